"""The training step's gradients and the AdamW update in 64 bits (plain torch), with
the error bounds that the GPU tests hold the kernels to.

A bound is a per-element limit on |kernel - reference| that follows from the kernels'
arithmetic: U(dtype) relative for each rounding to the layer's type, and A per addition
of an fp32 sum. A is 2^-23, twice the half step of a rounded addition, because the tensor
cores may truncate the addends that they align.
"""
from __future__ import annotations

import math

import torch

from sparse_mixture_experts_12_b200 import synth

A = 2.0 ** -23


def U(dt: torch.dtype) -> float:
    return torch.finfo(dt).eps / 2


def D(t):
    return None if t is None else t.double()


# ---------------------------------------------------------------- token movement
def combine_bwd(dy, y_perm, inv, gate, dy_perm):
    """(dy_perm, dgate, bound of dgate); rows of `dy_perm` that no slot owns are kept."""
    T, k = gate.shape
    out, dgate, lim = D(dy_perm).clone(), torch.zeros(T, k).to(D(gate)), torch.zeros(T, k).to(D(gate))
    iv = inv.reshape(T, k).long()
    for s in range(k):
        t = torch.nonzero(iv[:, s] >= 0)[:, 0]
        r = iv[t, s]
        out[r] = D(dy[t]) * D(gate[t, s])[:, None]
        dgate[t, s] = (D(dy[t]) * D(y_perm[r])).sum(1)
        lim[t, s] = (dy.shape[1] + 2) * A * (D(dy[t]) * D(y_perm[r])).abs().sum(1)
    return out, dgate, lim


def permute_bwd(dx_perm, inv, add, T, k):
    """(dx, sum of the magnitudes added)."""
    iv = inv.reshape(T, k).long()
    dx = D(add).clone() if add is not None else torch.zeros(T, dx_perm.shape[1]).to(D(dx_perm))
    mag = dx.abs()
    for s in range(k):
        t = torch.nonzero(iv[:, s] >= 0)[:, 0]
        dx[t] += D(dx_perm[iv[t, s]])
        mag[t] += D(dx_perm[iv[t, s]]).abs()
    return dx, mag


# ------------------------------------------------------------------------ router
def route_bwd(logits, idx, counts, dgate, d_losses, mode, alpha):
    """(dlogits, bound). `dgate` / `d_losses` may be None."""
    z, idx = D(logits), idx.long()
    T, E = z.shape
    k = idx.shape[1]
    top = z.max(1, keepdim=True).values
    ok = torch.isfinite(top)
    p = torch.where(ok, torch.softmax(z, 1), torch.zeros_like(z))
    lse = torch.where(ok, torch.logsumexp(z, 1, keepdim=True), torch.zeros_like(top))
    dz, mag = torch.zeros_like(z), torch.zeros_like(z)
    if dgate is not None:
        dg = D(dgate)
        if mode == synth.GATE_SOFTMAX_TOPK_RAW:
            ps = p.gather(1, idx)
            sd, sm = (ps * dg).sum(1, keepdim=True), (ps * dg).abs().sum(1, keepdim=True)
            dz -= p * sd
            mag += p * sm
            dz.scatter_add_(1, idx, ps * dg)
            mag.scatter_add_(1, idx, (ps * dg).abs())
        else:
            zs = z.gather(1, idx)
            fin = torch.isfinite(zs.max(1, keepdim=True).values)
            g = torch.where(fin, torch.softmax(zs, 1), torch.zeros_like(zs))
            dz.scatter_add_(1, idx, g * (dg - (g * dg).sum(1, keepdim=True)))
            mag.scatter_add_(1, idx, g * (dg.abs() + (g * dg).abs().sum(1, keepdim=True)))
    if d_losses is not None:
        f = D(counts) / (T * k)
        c0, c1 = D(d_losses)[0] * alpha * E / T, D(d_losses)[1] * 2 / T
        pf = (p * f).sum(1, keepdim=True)
        dz += p * (c0 * (f - pf) + c1 * lse)
        mag += p * (c0.abs() * (f + pf) + c1.abs() * lse.abs())
    # a probability is off by the exponent's rounding (|z - m| half steps), 2 ulp of expf, and
    # the sum of E terms; a handful of products, a second probability beside it, and the
    # k- and E-term sums follow: twice that, with 40 half steps for the products
    spread = torch.where(torch.isfinite(z), top - z, torch.zeros_like(z)).amax(1, keepdim=True)
    lim = mag * (40 + 4 * torch.where(ok, spread, torch.zeros_like(spread)) + E / 4 + k) * 2.0 ** -24
    return dz, lim


# ----------------------------------------------------------------------- experts
def _act(act, v):
    """act, act', and a bound of |act''|."""
    if act == synth.ACT_RELU:
        return v.clamp(min=0), (v > 0).double(), 0.0
    c = 0.5 * (1 + torch.erf(v / math.sqrt(2)))
    return v * c, c + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi), 1.13


def ffn_bwd(x, dy, off, p, act, dt, row_w=None):
    """Gradients of the grouped expert FFN in 64 bits, and their bounds, as two dicts (dx,
    w1, w3, w2, b1, b2, row_dot). `p`: w1, w3, w2, b1, b2; `off`: a list."""
    E, F, d = p["w1"].shape
    u = U(dt)
    new = lambda *s: torch.zeros(*s, dtype=torch.float64, device=x.device)  # noqa: E731
    R = x.shape[0]
    names = {"dx": (R, d), "w1": (E, F, d), "w2": (E, d, F), "w3": (E, F, d), "b1": (E, F),
             "b2": (E, d), "row_dot": (R,)}
    out, lim = {n: new(*s) for n, s in names.items()}, {n: new(*s) for n, s in names.items()}
    fp = 2.0 ** -20  # relative error of the activations' own evaluation: exp, erf, divisions (16 half steps)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if off[e + 1] <= off[e]:
            continue
        xe, ye = D(x[r]), D(dy[r])
        w = D(row_w[r])[:, None] if row_w is not None else torch.ones_like(xe[:, :1])
        w1, w2 = D(p["w1"][e]), D(p["w2"][e])
        a, q = xe @ w1.T, ye @ w2
        da_, dq = (d + 2) * A * (xe.abs() @ w1.abs().T), (d + 2) * A * (ye.abs() @ w2.abs())
        if act == synth.ACT_SWIGLU:
            w3 = D(p["w3"][e])
            up, dup = xe @ w3.T, (d + 2) * A * (xe.abs() @ w3.abs().T)
            s = torch.sigmoid(a)
            silu, sl = a * s, s * (1 + a * (1 - s))
            h, gu, ga = silu * up, q * silu, q * up * sl
            # |silu'| <= 1.1, |silu''| <= 0.5
            lh = 1.1 * da_ * up.abs() + silu.abs() * dup + fp * h.abs()
            lu = dq * silu.abs() + 1.1 * q.abs() * da_ + fp * gu.abs()
            la = dq * (up * sl).abs() + dup * (q * sl).abs() + 0.5 * da_ * (q * up).abs() \
                + fp * (q * up).abs() * (s * (1 + a.abs()))
        else:
            if p.get("b1") is not None:
                a = a + D(p["b1"][e])
                da_ = da_ + A * a.abs()
            h, sl, curv = _act(act, a)
            ga = q * sl
            lh = 1.13 * da_ + fp * (a.abs() + h.abs())
            la = dq * sl.abs() + q.abs() * (curv * da_ + fp)
            if act == synth.ACT_RELU:  # beside the kink either slope is right
                la = torch.where(a.abs() <= da_, la + q.abs(), la)
        dot, ldot = (q * h).sum(1), ((dq * h.abs() + q.abs() * lh).sum(1)
                                     + (F + 8) * A * (q * h).abs().sum(1))
        if p.get("b2") is not None:
            dot = dot + ye @ D(p["b2"][e])
            ldot = ldot + (d + 8) * A * (ye.abs() @ D(p["b2"][e]).abs())
        out["row_dot"][r], lim["row_dot"][r] = dot, ldot
        # weighted and rounded once to the layer's type
        h, ga, lh, la = w * h, w * ga, w.abs() * lh, w.abs() * la
        n = h.shape[0]
        out["b1"][e], lim["b1"][e] = ga.sum(0), la.sum(0) + (n + 4) * A * ga.abs().sum(0)
        out["b2"][e], lim["b2"][e] = (w * ye).sum(0), (n + 4) * A * (w * ye).abs().sum(0)
        lh, la = lh + u * (h.abs() + lh), la + u * (ga.abs() + la)
        dx, ldx = ga @ w1, la @ w1.abs() + 2 * (F + 2) * A * (ga.abs() @ w1.abs())
        out["w1"][e] = ga.T @ xe
        lim["w1"][e] = la.T @ xe.abs() + (n + 2) * A * (ga.abs().T @ xe.abs())
        if act == synth.ACT_SWIGLU:
            gu, lu = w * gu, w.abs() * lu
            lu = lu + u * (gu.abs() + lu)
            dx = dx + gu @ w3
            ldx = ldx + lu @ w3.abs() + 2 * (F + 2) * A * (gu.abs() @ w3.abs())
            out["w3"][e] = gu.T @ xe
            lim["w3"][e] = lu.T @ xe.abs() + (n + 2) * A * (gu.abs().T @ xe.abs())
        out["w2"][e] = ye.T @ h
        lim["w2"][e] = ye.abs().T @ lh + (n + 2) * A * (ye.abs().T @ h.abs())
        out["dx"][r], lim["dx"][r] = dx, ldx
    for n in ("dx", "w1", "w3", "w2"):  # the outputs' own rounding
        lim[n] = lim[n] + u * (out[n].abs() + lim[n])
    return out, lim


def layer_bwd(x, dy, taps, p, wl, d_losses=None):
    """The whole layer's gradients and bounds: the routed experts, the router, the shared
    experts. Returns two dicts with dx and the parameters' names."""
    T, d, E, k = wl.T, wl.d_model, wl.n_experts, wl.top_k
    dt = wl.torch_dtype
    iv = taps["inv"].reshape(T, k).long()
    R = T * k
    xp, yp = torch.zeros(R, d).to(x), torch.zeros(R, d).to(x)
    rw = torch.zeros(R).to(taps["topk_gate"])
    for s in range(k):
        t = torch.nonzero(iv[:, s] >= 0)[:, 0]
        xp[iv[t, s]], yp[iv[t, s]], rw[iv[t, s]] = x[t], dy[t], taps["topk_gate"][t, s]
    o, m = ffn_bwd(xp, yp, taps["offsets"].tolist(), p, wl.act, dt, rw)
    u = U(dt)
    dgate, ldg = torch.zeros(T, k).to(o["dx"]), torch.zeros(T, k).to(o["dx"])
    dx, ldx = torch.zeros(T, d).to(o["dx"]), torch.zeros(T, d).to(o["dx"])
    for s in range(k):
        t = torch.nonzero(iv[:, s] >= 0)[:, 0]
        dgate[t, s], ldg[t, s] = o["row_dot"][iv[t, s]], m["row_dot"][iv[t, s]]
        dx[t] += o["dx"][iv[t, s]]
        ldx[t] += m["dx"][iv[t, s]] + k * A * o["dx"][iv[t, s]].abs()
    dz, ldz = route_bwd(taps["logits"], taps["topk_idx"], taps["counts"], dgate, d_losses,
                        wl.gate_mode, wl.aux_alpha)
    # the gates' own gradients are off by ldg: |d dz| <= sum over the slots of p-weighted ldg
    ldz = ldz + (ldg.sum(1, keepdim=True)
                 * torch.ones(1, E).to(ldz)) * (1 if wl.gate_mode == synth.GATE_SOFTMAX_TOPK_RAW
                                                else _selected(taps["topk_idx"], E))
    wr = D(p["w_router"])
    out, lim = {n: o[n] for n in ("w1", "w3", "w2", "b1", "b2")}, \
        {n: m[n] for n in ("w1", "w3", "w2", "b1", "b2")}
    dx = dx + dz @ wr
    ldx = ldx + ldz @ wr.abs() + (E + 2) * A * (dz.abs() @ wr.abs())
    out["w_router"] = dz.T @ D(x)
    lim["w_router"] = ldz.T @ D(x).abs() + (T + 2) * A * (dz.abs().T @ D(x).abs())
    lim["w_router"] = lim["w_router"] + u * (out["w_router"].abs() + lim["w_router"])
    out["b_router"], lim["b_router"] = dz.sum(0), ldz.sum(0) + (T + 2) * A * dz.abs().sum(0)
    if wl.n_shared > 0:
        sp = {"w1": p["ws_gate"][None], "w3": p["ws_up"][None], "w2": p["ws_down"][None]}
        so, sm = ffn_bwd(x, dy, [0, T], sp, synth.ACT_SWIGLU, dt)
        dx, ldx = dx + so["dx"], ldx + sm["dx"] + A * so["dx"].abs()
        for a, b in (("ws_gate", "w1"), ("ws_up", "w3"), ("ws_down", "w2")):
            out[a], lim[a] = so[b][0], sm[b][0]
    out["dx"], lim["dx"] = dx, ldx + u * (dx.abs() + ldx)
    return out, lim


def _selected(idx, E):
    s = torch.zeros(idx.shape[0], E, dtype=torch.float64, device=idx.device)
    return s.scatter_(1, idx.long(), 1.0)


# ------------------------------------------------------------------------- AdamW
def adamw(p, g, m, v, step, lr, b1, b2, eps, wd, scale=1.0):
    """(p, m, v) after one step, 64 bits."""
    g = D(g) * scale
    m, v = b1 * D(m) + (1 - b1) * g, b2 * D(v) + (1 - b2) * g * g
    p = D(p) * (1 - lr * wd) - lr * (m / (1 - b1 ** step)) / ((v / (1 - b2 ** step)).sqrt() + eps)
    return p, m, v


def from_8(codes, scale, block=256):
    """The values that 8-bit codes stand for, 64 bits, flat."""
    n = codes.numel()
    at = torch.arange(n, device=codes.device) // block
    return codes.reshape(-1).double() * scale.double()[at]


def check(got, ref, lim, what):
    """Every element of `got` is within `lim` of `ref` (and finite where ref is)."""
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    over = err > lim + 1e-300
    if over.any():
        i = int(torch.argmax((err / (lim + 1e-300)).reshape(-1)))
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} elements off, worst "
                             f"{float(err.reshape(-1)[i]):.3e} against {float(lim.reshape(-1)[i]):.3e}"
                             f" at {i}")


def check_norm(got, ref, dt, what, roundings=2):
    """The error's 2-norm over the reference's: `roundings` independent roundings of at
    most U each, of random sign, are below U * sqrt(roundings) in the mean square; 1e-6 for
    fp32's sums."""
    n = float(ref.norm())
    if n > 0:
        rel = float((got.double() - ref).norm()) / n
        most = U(dt) * math.sqrt(roundings) + (1e-5 if dt == torch.float32 else 0.0)
        assert rel <= most, f"{what}: {rel:.3e} of the norm off, {most:.3e} allowed"
