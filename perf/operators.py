"""The operators of the layer's training step, as cases to be timed and compared.

Five operators: the gradient of the gate-weighted combine, the gradient of the
expert-contiguous permutation, the router's gradient (gates, load-balancing and
z-loss, projection), the expert FFNs' gradient, and an AdamW step over many tensors.
``run`` computes a case in elementary torch operations (``own`` false) or through
this framework's entry points (``own`` true).
"""
import math

import torch

own = False

RELU, GELU, SWIGLU = 0, 1, 2
TOPK_SOFTMAX, RENORM, RAW = 0, 1, 2
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.95, 1e-8, 0.1
ALPHA = 0.01       # weight of the load-balancing loss
BLOCK = 256        # elements that share one scale of an 8-bit state
E4M3_MAX = 448.0
E4M3_TINY = 2.0 ** -9
MIXTRAL_FFN = 8192 * 4096 * 14336   # rows x d x F of the largest listed expert case
MIXTRAL_W = 8 * 4096 * 14336


def listed():
    return [
        # fine-tuning on a batch of 32 tokens: launch latency counts
        dict(name="combine_bwd decode32", op="combine", T=32, d=4096, E=8, k=2, cf=0.0, skew=0.5, dtype="bf16"),
        # a training micro-batch of fine-grained experts: six slots a token
        dict(name="combine_bwd deepseek", op="combine", T=8192, d=2048, E=64, k=6, cf=0.0, skew=0.5, dtype="bf16"),
        # the smallest configured layer, fp32
        dict(name="permute_bwd tiny", op="permute", T=64, d=64, E=8, k=2, cf=0.0, skew=0.5, dtype="f32"),
        # top-1 with a capacity limit: overflowing tokens have no gradient of their own
        dict(name="permute_bwd switch", op="permute", T=16384, d=1024, E=128, k=1, cf=1.25, skew=1.0, dtype="bf16"),
        # few experts, no auxiliary losses: the gradient of the gates alone
        dict(name="route_bwd mixtral", op="route", T=4096, d=4096, E=8, k=2, mode=TOPK_SOFTMAX, losses=False, dtype="bf16"),
        # many experts, raw top-1 gates, load-balancing and z-loss gradients
        dict(name="route_bwd switch", op="route", T=16384, d=1024, E=128, k=1, mode=RAW, losses=True, dtype="bf16"),
        # the smallest configured layer's experts, fp32 with biases
        dict(name="ffn_bwd tiny", op="ffn", R=128, d=64, E=8, F=256, act=GELU, cap=0, skew=0.5, dtype="f32"),
        # many small capacity-limited experts: the weights' traffic counts
        dict(name="ffn_bwd switch", op="ffn", R=16384, d=1024, E=128, F=4096, act=GELU, cap=160, skew=1.0, dtype="bf16"),
        # few large experts: the matrix products count
        dict(name="ffn_bwd mixtral", op="ffn", R=8192, d=4096, E=8, F=14336, act=SWIGLU, cap=0, skew=0.3, dtype="bf16"),
        # sixteen small fp32 layers, 96 tensors from 8 to 131072 elements: launches count
        dict(name="adamw small tensors", op="adamw", layers=16, E=8, d=64, F=256, swiglu=False, dtype="f32", bits=32, master=False),
        # bf16 weights with an fp32 copy, fp32 states: the ordinary mixed-precision step
        dict(name="adamw bf16 master", op="adamw", layers=2, E=8, d=2048, F=4096, swiglu=True, dtype="bf16", bits=32, master=True),
        # the same weights twice over, 8-bit states, no copy: the step for little memory
        dict(name="adamw 8 bit", op="adamw", layers=4, E=8, d=2048, F=4096, swiglu=True, dtype="bf16", bits=8, master=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi, step):
        return max(step, log(lo, hi) // step * step)

    op = rng.choice(["combine", "permute", "route", "ffn", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    step = 64 if dtype == "bf16" else 4
    if op in ("combine", "permute"):
        E = log(1, 256)
        k = rng.randint(1, min(E, 8))
        d = width(64, 8192, step)
        T = log(1, 32768)
        while T * k * d > 8192 * 6 * 2048:
            T //= 2
        return dict(op=op, T=max(1, T), d=d, E=E, k=k, cf=rng.choice([0.0, 0.0, 0.5, 1.25]),
                    skew=rng.choice([0.0, 0.5, 1.5]), dtype=dtype)
    if op == "route":
        E = log(1, 256)
        T, d = log(1, 32768), width(64, 8192, step)
        while T * d * max(E, 8) > 16384 * 1024 * 128:
            T //= 2
        return dict(op=op, T=max(1, T), d=d, E=E, k=rng.randint(1, min(E, 8)),
                    mode=rng.choice([TOPK_SOFTMAX, RENORM, RAW]), losses=rng.random() < 0.6, dtype=dtype)
    if op == "ffn":
        E, R = log(1, 128), log(1, 16384)
        d, F = width(64, 4096, step), width(64, 14336, step)
        act = rng.choice([RELU, GELU, SWIGLU]) if dtype == "bf16" else rng.choice([GELU, SWIGLU])
        most = MIXTRAL_FFN if dtype == "bf16" else MIXTRAL_FFN // 64
        while R * d * F > most:
            R //= 2
        while E * d * F > MIXTRAL_W // (1 if dtype == "bf16" else 8):
            E //= 2
        return dict(op=op, R=max(1, R), d=d, E=max(1, E), F=F, act=act, cap=rng.choice([0, 0, 200]),
                    skew=rng.choice([0.0, 0.5, 1.5]), dtype=dtype)
    E, d, F, layers = log(1, 64), width(64, 4096, 4), width(64, 14336, 4), log(1, 32)
    while E * d * F * layers * 3 > 4 * 8 * 2048 * 4096 * 3:
        if layers > 1:
            layers //= 2
        elif E > 1:
            E //= 2
        else:
            F = F // 8 * 4
    return dict(op=op, layers=layers, E=E, d=d + rng.choice([0, 0, 1, 3]), F=F, swiglu=rng.random() < 0.5, dtype=dtype,
                bits=rng.choice([8, 32]), master=dtype == "bf16" and rng.random() < 0.5)


# ------------------------------------------------------------------- the inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _popularity(E, skew):
    """log probability of the experts: normal quantiles times `skew`."""
    q = (torch.arange(E, device="cuda", dtype=torch.float64) + 0.5) / E
    return torch.log_softmax(skew * math.sqrt(2.0) * torch.erfinv(2 * q - 1), 0).float()


def _experts_of(T, E, k, skew, g):
    """k experts for each of T tokens, in proportion to the popularity of each."""
    p = _popularity(E, skew)[torch.randperm(E, device="cuda", generator=g)]
    z = p - torch.log(-torch.log(torch.rand(T, E, device="cuda", generator=g).clamp_(1e-7, 1 - 1e-7)))
    return z.topk(k, 1).indices


def _capacity(case):
    return int(math.floor(case["cf"] * case["T"] * case["k"] / case["E"])) if case["cf"] > 0 else case["T"]


def _layout(idx, E, cap):
    """inv [T * k] of the expert-contiguous rows, in token order, and the kept rows' offsets."""
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    start = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device="cuda") - start[flat[order]]
    kept = counts.clamp(max=cap)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(kept, 0)
    inv = torch.where(rank < cap, offsets[flat] + rank, torch.full_like(flat, -1))
    return inv.int(), offsets.int(), counts.int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, op = _dt(case), case["op"]

    def normal(*shape, std=1.0, dtype=dt):
        return torch.randn(*shape, device="cuda", dtype=dtype, generator=g).mul_(std)

    s = dict(case=dict(case))
    if op in ("combine", "permute"):
        T, d, E, k = case["T"], case["d"], case["E"], case["k"]
        s["inv"], s["offsets"], _ = _layout(_experts_of(T, E, k, case["skew"], g), E, _capacity(case))
        if op == "combine":
            s["dy"], s["y_perm"] = normal(T, d), normal(T * k, d)
            s["gate"] = torch.softmax(normal(T, k, dtype=torch.float32), 1)
            s["dy_perm"] = torch.zeros(T * k, d, device="cuda", dtype=dt)  # rows behind the last kept one stay 0
            s["dgate"] = torch.empty(T, k, device="cuda")
        else:
            s["dx_perm"], s["dx_add"] = normal(T * k, d), normal(T, d, dtype=torch.float32)
            s["dx"] = torch.empty(T, d, device="cuda", dtype=dt)
    elif op == "route":
        T, d, E, k = case["T"], case["d"], case["E"], case["k"]
        s["x"], s["w_router"] = normal(T, d), normal(E, d, std=1 / math.sqrt(d))
        s["logits"] = s["x"].float() @ s["w_router"].float().T
        top = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, :k]
        s["topk_idx"] = top.int().contiguous()
        s["counts"] = torch.bincount(top.reshape(-1), minlength=E).int()
        s["dgate"] = normal(T, k, dtype=torch.float32)
        # upstream gradients of the mean losses, of the size that the gates' have in sum
        s["d_losses"] = torch.tensor([float(T), 0.001 * T], device="cuda") if case["losses"] else None
        s["dx"] = torch.empty(T, d, device="cuda")
        s["dlogits"] = torch.empty(T, E, device="cuda")
    elif op == "ffn":
        R, d, E, F = case["R"], case["d"], case["E"], case["F"]
        cap = case["cap"] or R
        _, s["offsets"], counts = _layout(_experts_of(R, E, 1, case["skew"], g), E, cap)
        s["most_rows"] = int(counts.clamp(max=cap).max())
        s["x_perm"], s["dy_perm"] = normal(R, d), normal(R, d)
        s["w1"], s["w2"] = normal(E, F, d, std=1 / math.sqrt(d)), normal(E, d, F, std=1 / math.sqrt(F))
        if case["act"] == SWIGLU:
            s["w3"] = normal(E, F, d, std=1 / math.sqrt(d))
        else:
            s["b1"], s["b2"] = normal(E, F, std=0.1, dtype=torch.float32), normal(E, d, std=0.1, dtype=torch.float32)
        s["dx_perm"] = torch.zeros(R, d, device="cuda", dtype=dt)
    else:
        E, d, F = case["E"], case["d"], case["F"]
        shapes = [((E, d), dt), ((E, F, d), dt), ((E, d, F), dt)]
        shapes += [((E, F, d), dt)] if case["swiglu"] else [((E, F), torch.float32), ((E, d), torch.float32)]
        shapes = (shapes + [((E,), torch.float32)]) * case["layers"]
        s["params"], s["grads"], s["master"], s["m"], s["v"], s["ms"], s["vs"] = [], [], [], [], [], [], []
        for shape, t in shapes:
            w = normal(*shape, std=0.02, dtype=torch.float32)
            s["params"].append(w.to(t))
            # mini-batch gradients: normal, of very different sizes from row to row
            s["grads"].append((normal(*shape, dtype=torch.float32) * 1e-3 * torch.exp(normal(*shape[:-1], 1, dtype=torch.float32))).to(t))
            s["master"].append(w if case["master"] and t != torch.float32 else None)
            m, r = normal(*shape, std=1e-3, dtype=torch.float32), normal(*shape, std=1e-3, dtype=torch.float32).abs_()
            if case["bits"] == 8:
                for x, codes, scales in ((m, "m", "ms"), (r, "v", "vs")):
                    q, sc = _to_8(x.reshape(-1), codes == "v")
                    s[codes].append(q.reshape(shape))
                    s[scales].append(sc)
            else:
                s["m"].append(m)
                s["v"].append(r.square_())
        s["step"] = 10
    return s


# ------------------------------------------------------------- the plain forms
def _blocks(x):
    n = x.numel()
    return torch.nn.functional.pad(x, (0, -n % BLOCK)).reshape(-1, BLOCK)


def _to_8(x, root):
    """e4m3 codes and a scale for each BLOCK elements: the largest stands at 448. A root of
    the second moment that is not zero keeps at least the smallest code."""
    b = _blocks(x)
    top = b.abs().amax(1).clamp_(min=2.0 ** -100)
    y = b * (E4M3_MAX / top)[:, None]
    if root:
        y = torch.where(b > 0, y.clamp(min=E4M3_TINY), y)
    return y.reshape(-1)[: x.numel()].to(torch.float8_e4m3fn), top / E4M3_MAX


def _from_8(q, scale):
    return (_blocks(q.reshape(-1).float()) * scale[:, None]).reshape(-1)[: q.numel()]


def _combine_bwd(s):
    case = s["case"]
    T, k, d = case["T"], case["k"], case["d"]
    inv = s["inv"].long()
    kept = inv >= 0
    dy = s["dy"].float().repeat_interleave(k, 0)
    y = s["y_perm"][inv.clamp(min=0)].float()
    dgate = torch.where(kept, (dy * y).sum(1), torch.zeros((), device="cuda")).reshape(T, k)
    rows = (dy * s["gate"].reshape(-1, 1)).to(s["dy"].dtype)
    s["dy_perm"][inv[kept]] = rows[kept]
    return dict(dy_perm=s["dy_perm"], dgate=dgate)


def _permute_bwd(s):
    case = s["case"]
    inv = s["inv"].long()
    rows = torch.where((inv >= 0)[:, None], s["dx_perm"][inv.clamp(min=0)].float(), torch.zeros((), device="cuda"))
    return (rows.reshape(case["T"], case["k"], -1).sum(1) + s["dx_add"]).to(s["dx_perm"].dtype)


def _route_bwd(s):
    case = s["case"]
    T, E, k = case["T"], case["E"], case["k"]
    z, idx, dg = s["logits"], s["topk_idx"].long(), s["dgate"]
    if case["mode"] == RAW or s["d_losses"] is not None:
        lse = torch.logsumexp(z, 1, keepdim=True)
        p = torch.exp(z - lse)
    if case["mode"] == RAW:
        sel = p.gather(1, idx)
        dz = -p * (sel * dg).sum(1, keepdim=True)
        dz.scatter_add_(1, idx, sel * dg)
    else:
        gt = torch.softmax(z.gather(1, idx), 1)
        dz = torch.zeros_like(z).scatter_(1, idx, gt * (dg - (gt * dg).sum(1, keepdim=True)))
    if s["d_losses"] is not None:
        f = s["counts"].float() / (T * k)
        dz += s["d_losses"][0] * (ALPHA * E / T) * p * (f - (p * f).sum(1, keepdim=True))
        dz += s["d_losses"][1] * (2.0 / T) * lse * p
    x, w = s["x"].float(), s["w_router"].float()
    return dict(dlogits=dz, dx=dz @ w, dw=(dz.T @ x).to(s["x"].dtype), db=dz.sum(0))


def _ffn_bwd(s):
    case = s["case"]
    E, R, dt = case["E"], case["R"], s["x_perm"].dtype
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["most_rows"], device="cuda")
    live = at < off[1:, None]
    at = at.clamp(max=R - 1)
    x = s["x_perm"][at].float() * live[..., None]
    dy = s["dy_perm"][at].float() * live[..., None]
    w1, w2 = s["w1"].float(), s["w2"].float()
    dh = dy @ w2
    out = {}
    a = x @ w1.transpose(1, 2)
    if case["act"] == SWIGLU:
        w3 = s["w3"].float()
        u = x @ w3.transpose(1, 2)
        sg = torch.sigmoid(a)
        h, du = a * sg * u, dh * a * sg
        da = dh * u * sg * (1 + a * (1 - sg))
        dx = da @ w1 + du @ w3
        out["dw3"] = (du.transpose(1, 2) @ x).to(dt)
    else:
        a = a + s["b1"][:, None, :]
        if case["act"] == RELU:
            h, da = a.clamp(min=0), dh * (a > 0)
        else:
            cdf = 0.5 * (1 + torch.erf(a * math.sqrt(0.5)))
            h, da = a * cdf, dh * (cdf + a * torch.exp(-0.5 * a * a) * (1 / math.sqrt(2 * math.pi)))
        da = da * live[..., None]
        dx = da @ w1
        out["db1"], out["db2"] = da.sum(1), dy.sum(1)
    out["dw1"] = (da.transpose(1, 2) @ x).to(dt)
    out["dw2"] = (dy.transpose(1, 2) @ h).to(dt)
    s["dx_perm"][at[live]] = dx[live].to(dt)
    out["dx_perm"] = s["dx_perm"]
    return out


def _adamw(s):
    s["step"] += 1
    c1, c2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
    for i, (p, gr) in enumerate(zip(s["params"], s["grads"])):  # a list of tensors is what the operator works on
        gr, m, v = gr.reshape(-1).float(), s["m"][i], s["v"][i]
        if s["ms"]:
            m, v = _from_8(m, s["ms"][i]), _from_8(v, s["vs"][i]).square_()
        w = s["master"][i] if s["master"][i] is not None else p
        m = BETA1 * m.reshape(-1) + (1 - BETA1) * gr
        v = BETA2 * v.reshape(-1) + (1 - BETA2) * gr * gr
        w32 = w.reshape(-1).float() * (1 - LR * DECAY)
        w32 -= (LR / c1) * (m / (v.sqrt() / math.sqrt(c2) + EPS))
        w.reshape(-1).copy_(w32)
        if w is not p:
            p.reshape(-1).copy_(w32)
        if s["ms"]:
            for x, codes, scales in ((m, "m", "ms"), (v.sqrt(), "v", "vs")):
                q, sc = _to_8(x, codes == "v")
                s[codes][i].reshape(-1).copy_(q)
                s[scales][i].copy_(sc)
        else:
            s["m"][i].reshape(-1).copy_(m)
            s["v"][i].reshape(-1).copy_(v)
    return _adamw_out(s)


#: Of many tensors the first layers' are returned: 64 outputs at most are looked at.
SHOWN = 10


def _adamw_out(s):
    out = dict(params=s["params"][:SHOWN], m=s["m"][:SHOWN], v=s["v"][:SHOWN])
    if s["ms"]:
        out |= dict(ms=s["ms"][:SHOWN], vs=s["vs"][:SHOWN])
    return out | dict(master=s["master"][:SHOWN])


# --------------------------------------------------- the framework's own calls
def _layer(s):
    """The layer handle that a program keeps next to its weights."""
    if "layer" not in s:
        from sparse_mixture_experts_12_b200 import binding, synth
        c = s["case"]
        wl = synth.Workload("case", T=c.get("T", c.get("R")), d_model=c["d"], n_experts=c["E"], top_k=c.get("k", 1),
                            d_ff=c.get("F", 64), act=c.get("act", SWIGLU), gate_mode=c.get("mode", TOPK_SOFTMAX),
                            dtype=synth.DT_BF16 if c["dtype"] == "bf16" else synth.DT_F32, aux_alpha=ALPHA,
                            capacity_factor=c.get("cf", 0.0))
        s["layer"] = binding.MoELayer(wl, {n: s.get(n) for n in ("w_router", "w1", "w3", "w2", "b1", "b2")})
        s["new"] = s["layer"].new_grads()
    return s["layer"]


def _own(s):
    op = s["case"]["op"]
    if op == "combine":
        _layer(s).combine_backward(s["dy"], s["y_perm"], s["inv"], s["gate"], s["dy_perm"], s["dgate"])
        return dict(dy_perm=s["dy_perm"], dgate=s["dgate"])
    if op == "permute":
        _layer(s).permute_backward(s["dx_perm"], s["inv"], s["dx_add"], s["dx"])
        return s["dx"]
    if op == "route":
        layer = _layer(s)
        layer.route_backward(s["x"], s["logits"], s["topk_idx"], s["counts"], s["dgate"], s["d_losses"], s["dlogits"],
                             s["dx"], s["new"])
        return dict(dlogits=s["dlogits"], dx=s["dx"], dw=s["new"]["w_router"], db=s["new"]["b_router"])
    if op == "ffn":
        layer = _layer(s)
        layer.expert_ffn_backward(s["x_perm"], s["offsets"], s["dy_perm"], s["dx_perm"], s["new"])
        return {("d" + n if n != "dx_perm" else n): t for n, t in {**s["new"], "dx_perm": s["dx_perm"]}.items()
                if n in ("w1", "w3", "w2", "b1", "b2", "dx_perm") and t is not None}
    if "opt" not in s:
        from sparse_mixture_experts_12_b200 import binding
        s["opt"] = binding.AdamW(s["params"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                                 state=dict(step=s["step"], exp_avg=s["m"], exp_avg_sq=s["v"],
                                            exp_avg_scale=s["ms"] or None, exp_avg_sq_scale=s["vs"] or None,
                                            master=s["master"]))
    s["opt"].step(s["grads"])
    return _adamw_out(s)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"combine": _combine_bwd, "permute": _permute_bwd, "route": _route_bwd, "ffn": _ffn_bwd, "adamw": _adamw}[op](state)


# -------------------------------------------------------------------- the work
def _kept(case):
    """Expected number of (token, slot) pairs that have a row."""
    R, cap = (case["R"], case["cap"] or case["R"]) if case["op"] == "ffn" else (case["T"] * case["k"], _capacity(case))
    q = [(i + 0.5) / case["E"] for i in range(case["E"])]
    # normal quantiles by bisection of erf
    def quantile(p):
        lo, hi = -6.0, 6.0
        for _ in range(50):
            mid = (lo + hi) / 2
            lo, hi = (mid, hi) if 0.5 * (1 + math.erf(mid / math.sqrt(2))) < p else (lo, mid)
        return lo
    w = [math.exp(case["skew"] * quantile(p)) for p in q]
    return sum(min(R * x / sum(w), cap) for x in w)


def work(case):
    eb, op = (2 if case["dtype"] == "bf16" else 4), case["op"]
    if op == "combine":
        T, d, k, K = case["T"], case["d"], case["k"], _kept(case)
        return dict(bytes=eb * d * (T + 2 * K) + 12 * T * k, flops=3 * K * d)
    if op == "permute":
        T, d, k, K = case["T"], case["d"], case["k"], _kept(case)
        return dict(bytes=eb * d * (T + K) + 4 * T * d + 4 * T * k, flops=(K + T) * d)
    if op == "route":
        T, d, E, k = case["T"], case["d"], case["E"], case["k"]
        return dict(bytes=eb * T * d + 4 * T * d + 8 * T * E + 8 * T * k + 2 * eb * E * d, flops=4 * T * E * d)
    if op == "ffn":
        R, d, E, F, K = case["R"], case["d"], case["E"], case["F"], _kept(case)
        mats, products = (3, 8) if case["act"] == SWIGLU else (2, 5)
        return dict(bytes=eb * (3 * K * d + 2 * mats * E * F * d), flops=2 * products * K * d * F)
    E, d, F, L = case["E"], case["d"], case["F"], case["layers"]
    n = L * (E * d + (3 if case["swiglu"] else 2) * E * d * F)
    n32 = L * (E + (0 if case["swiglu"] else E * F + E * d))
    state = 2 * (8 if case["bits"] == 32 else 2 + 8 / BLOCK)
    bytes_ = n * (3 * eb + state + (8 - eb if case["master"] else 0)) + n32 * (12 + state)
    return dict(bytes=bytes_, flops=16 * (n + n32))


# ------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    D = lambda t: t.double()  # noqa: E731
    op = case["op"]
    if op in ("combine", "permute"):
        T, k = case["T"], case["k"]
        inv = s["inv"].long().reshape(T, k)
        if op == "combine":
            dy_perm, dgate = D(s["dy_perm"]), torch.zeros(T, k, device="cuda", dtype=torch.float64)
            for j in range(k):
                t = torch.nonzero(inv[:, j] >= 0).reshape(-1)
                r = inv[t, j]
                dgate[t, j] = torch.einsum("td,td->t", D(s["dy"][t]), D(s["y_perm"][r]))
                dy_perm[r] = D(s["dy"][t]) * D(s["gate"][t, j])[:, None]
            return dict(dy_perm=dy_perm, dgate=dgate)
        dx = D(s["dx_add"])
        for j in range(k):
            t = torch.nonzero(inv[:, j] >= 0).reshape(-1)
            dx.index_add_(0, t, D(s["dx_perm"][inv[t, j]]))
        return dx
    if op == "route":
        # by differentiation of the gates and the losses themselves
        T, E, k = case["T"], case["E"], case["k"]
        z = D(s["logits"]).requires_grad_(True)
        p, idx = torch.softmax(z, 1), s["topk_idx"].long()
        gates = p.gather(1, idx)
        if case["mode"] != RAW:
            gates = torch.softmax(z.gather(1, idx), 1)
        total = (gates * D(s["dgate"])).sum()
        if s["d_losses"] is not None:
            f = D(s["counts"]) / (T * k)
            total = total + D(s["d_losses"])[0] * ALPHA * E * (f * p.mean(0)).sum()
            total = total + D(s["d_losses"])[1] * torch.logsumexp(z, 1).square().mean()
        (dz,) = torch.autograd.grad(total, z)
        return dict(dlogits=dz, dx=dz @ D(s["w_router"]), dw=dz.T @ D(s["x"]), db=dz.sum(0))
    if op == "ffn":
        E, off = case["E"], s["offsets"].tolist()
        if 16 * case["R"] * case["d"] * case["F"] > 1e13:
            return None
        out = dict(dx_perm=D(s["dx_perm"]), dw1=D(s["w1"]), dw2=D(s["w2"]))
        if case["act"] == SWIGLU:
            out["dw3"] = D(s["w3"])
        else:
            out["db1"], out["db2"] = D(s["b1"]), D(s["b2"])
        for e in range(E):
            x, dy = D(s["x_perm"][off[e]:off[e + 1]]), D(s["dy_perm"][off[e]:off[e + 1]])
            a, dh = x @ D(s["w1"][e]).T, dy @ D(s["w2"][e])
            if case["act"] == SWIGLU:
                u = x @ D(s["w3"][e]).T
                silu = a / (1 + torch.exp(-a))
                slope = (1 + silu * torch.exp(-a)) / (1 + torch.exp(-a))
                h, da, du = silu * u, dh * u * slope, dh * silu
                out["dw3"][e] = du.T @ x
                out["dx_perm"][off[e]:off[e + 1]] = da @ D(s["w1"][e]) + du @ D(s["w3"][e])
            else:
                a = a + D(s["b1"][e])
                if case["act"] == RELU:
                    h, da = torch.relu(a), dh * (a > 0).double()
                else:
                    cdf = torch.special.ndtr(a)
                    h, da = a * cdf, dh * (cdf + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi))
                out["db1"][e], out["db2"][e] = da.sum(0), dy.sum(0)
                out["dx_perm"][off[e]:off[e + 1]] = da @ D(s["w1"][e])
            out["dw1"][e], out["dw2"][e] = da.T @ x, dy.T @ h
        return out
    step = s["step"] + 1
    got = dict(params=[], m=[], v=[], ms=[], vs=[], master=[])
    for i, p in enumerate(s["params"][:SHOWN]):
        n, shape = p.numel(), p.shape
        gr = D(s["grads"][i]).reshape(-1)
        if case["bits"] == 8:
            each = torch.arange(n, device="cuda") // BLOCK
            m, v = D(s["m"][i]).reshape(-1) * D(s["ms"][i])[each], (D(s["v"][i]).reshape(-1) * D(s["vs"][i])[each]) ** 2
        else:
            m, v = D(s["m"][i]).reshape(-1), D(s["v"][i]).reshape(-1)
        m, v = m + (1 - BETA1) * (gr - m), v + (1 - BETA2) * (gr ** 2 - v)
        w = D(s["master"][i] if s["master"][i] is not None else p).reshape(-1)
        w = w - LR * DECAY * w - LR * (m / (1 - BETA1 ** step)) / ((v / (1 - BETA2 ** step)) ** 0.5 + EPS)
        got["params"].append(w.reshape(shape))
        got["master"].append(w.reshape(shape) if s["master"][i] is not None else None)
        if case["bits"] == 8:
            r = v ** 0.5
            for x, codes, scales in ((m, "m", "ms"), (r, "v", "vs")):
                top = torch.zeros(-(-n // BLOCK), device="cuda", dtype=torch.float64).scatter_reduce_(0, each, x.abs(), "amax")
                y = x * E4M3_MAX / top[each]
                got[codes].append((torch.where(x > 0, y.clamp(min=E4M3_TINY), y) if codes == "v" else y).reshape(shape))
                got[scales].append(top / E4M3_MAX)
        else:
            got["m"].append(m.reshape(shape))
            got["v"].append(v.reshape(shape))
    return got if case["bits"] == 8 else {n: t for n, t in got.items() if n not in ("ms", "vs")}
