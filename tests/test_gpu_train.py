"""The training step on the GPU against 64-bit references: the gradients of the token
movement, the router, the experts and the whole layer, and AdamW. The limits are those of
tests/train_ref.py: derived from the kernels' arithmetic, element by element."""
import ctypes
import itertools
import math

import pytest
import torch

from sparse_mixture_experts_12_b200 import binding as B
from sparse_mixture_experts_12_b200 import build as BUILD
from sparse_mixture_experts_12_b200 import synth
from tests import train_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = synth.DT_F32, synth.DT_BF16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    BUILD.build()
    yield B.load()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rand(g, *shape, dt=torch.float32, std=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * std).to(dt)


def _workload(T, d, E, k, dt, mode=0, F=64, act=synth.ACT_SWIGLU, cf=0.0, **kw):
    return synth.Workload("train_case", T=T, d_model=d, n_experts=E, top_k=k, d_ff=F, act=act,
                          gate_mode=mode, dtype=dt, capacity_factor=cf, **kw)


def _layout(idx, E, cap):
    """inv, offsets, counts (CPU lists would do; small sizes) of the stable layout."""
    flat = idx.reshape(-1).tolist()
    counts, ranks = [0] * E, []
    for e in flat:
        ranks.append(counts[e])
        counts[e] += 1
    off = [0]
    for c in counts:
        off.append(off[-1] + min(c, cap))
    inv = [off[e] + r if r < cap else -1 for e, r in zip(flat, ranks)]
    i32 = dict(dtype=torch.int32, device=DEV)
    return (torch.tensor(inv, **i32), torch.tensor(off, **i32), torch.tensor(counts, **i32))


def _picks(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(T, E, generator=g).topk(k, 1).indices.int()


# ---------------------------------------------------------------- token movement
TOKENS = [  # T, d, E, k, cap
    (1, 64, 1, 1, 9), (1, 4096, 8, 2, 9), (3, 64, 4, 2, 9), (33, 192, 64, 8, 99), (700, 256, 8, 2, 60),
    (517, 1024, 16, 6, 999), (2111, 128, 32, 1, 11), (5, 8192, 3, 3, 0), (2500, 64, 8, 3, 99999),
]


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,d,E,k,cap", TOKENS)
def test_combine_backward(T, d, E, k, cap, dt):
    wl = _workload(T, d, E, k, dt)
    layer, g, tdt = B.MoELayer(wl, {}, DEV), _gen(T), wl.torch_dtype
    inv, off, _ = _layout(_picks(T, E, k, T + d), E, cap)
    dy, yp = _rand(g, T, d, dt=tdt), _rand(g, T * k, d, dt=tdt)
    yp[int(off[-1]):] = float("nan")             # rows that no slot owns are not read
    gate = torch.softmax(_rand(g, T, k), 1)
    out, dgate = torch.full((T * k, d), 7.0, dtype=tdt, device=DEV), torch.full((T, k), 9.0, device=DEV)
    layer.combine_backward(dy, yp, inv, gate, out, dgate)
    ref, rdg, lim = R.combine_bwd(dy, yp, inv, gate, torch.full_like(out, 7.0))
    R.check(out, ref, (R.U(tdt) + 2.0 ** -23) * ref.abs(), "dy_perm")
    assert (out[int(off[-1]):] == 7.0).all()     # and not written
    R.check(dgate, rdg, lim, "dgate")
    assert (dgate.reshape(-1)[inv < 0] == 0).all()
    # one output at a time gives the same bits
    o2, d2 = torch.full_like(out, 7.0), torch.empty_like(dgate)
    layer.combine_backward(dy, None, inv, gate, o2, None)
    layer.combine_backward(dy, yp, inv, None, None, d2)
    assert torch.equal(o2, out) and torch.equal(d2, dgate)
    assert layer.last_backward_error() == (0, 0)


@pytest.mark.parametrize("add", [False, True], ids=["", "add"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,d,E,k,cap", TOKENS)
def test_permute_backward(T, d, E, k, cap, dt, add):
    wl = _workload(T, d, E, k, dt)
    layer, g, tdt = B.MoELayer(wl, {}, DEV), _gen(T + 1), wl.torch_dtype
    inv, off, _ = _layout(_picks(T, E, k, T + d), E, cap)
    dxp = _rand(g, T * k, d, dt=tdt)
    dxp[int(off[-1]):] = float("nan")
    da = _rand(g, T, d) if add else None
    dx = torch.full((T, d), 5.0, dtype=tdt, device=DEV)
    layer.permute_backward(dxp, inv, da, dx)
    ref, mag = R.permute_bwd(dxp, inv, da, T, k)
    R.check(dx, ref, (R.U(tdt) * (1 + 1e-6)) * ref.abs() + (k + 2) * 2.0 ** -24 * mag * 1.01, "dx")
    assert layer.last_backward_error() == (0, 0)


def test_rows_outside_the_buffer_are_reported_and_skipped():
    T, d, E, k = 40, 128, 4, 2
    wl = _workload(T, d, E, k, BF16)
    layer, g, b = B.MoELayer(wl, {}, DEV), _gen(5), torch.bfloat16
    inv, _, _ = _layout(_picks(T, E, k, 1), E, 99)
    inv[7], inv[50] = T * k, -2
    dy, yp, gate = _rand(g, T, d, dt=b), _rand(g, T * k, d, dt=b), torch.rand(T, k, device=DEV)
    out, dgate = torch.zeros(T * k, d, dtype=b, device=DEV), torch.ones(T, k, device=DEV)
    layer.combine_backward(dy, yp, inv, gate, out, dgate)
    code, info = layer.last_backward_error()
    assert code == 3 and info in (7, 50)
    assert dgate.reshape(-1)[7] == 0 and dgate.reshape(-1)[50] == 0
    dx = torch.zeros(T, d, dtype=b, device=DEV)
    layer.permute_backward(yp, inv, None, dx)
    assert layer.last_backward_error()[0] == 3
    assert layer.last_backward_error() == (0, 0)


# ------------------------------------------------------------------------ router
ROUTES = [  # T, d, E, k
    (1, 64, 1, 1), (1, 128, 8, 2), (37, 64, 20, 3), (300, 256, 8, 2), (131, 128, 33, 8),
    (1000, 192, 128, 1), (257, 64, 256, 8), (4100, 64, 4, 4), (700, 1088, 64, 4), (2049, 320, 200, 2),
    (50, 576, 16, 2), (611, 2112, 32, 3), (1, 64, 40, 2), (3, 128, 256, 8), (65, 64, 65, 1),
]


def _route_case(T, d, E, k, dt, mode, seed):
    wl = _workload(T, d, E, k, dt, mode=mode)
    g = _gen(seed)
    p = {"w_router": _rand(g, E, d, dt=wl.torch_dtype, std=1 / math.sqrt(d))}
    layer = B.MoELayer(wl, p, DEV)
    x = _rand(g, T, d, dt=wl.torch_dtype)
    z = x.float() @ layer.p["w_router"].float().T
    idx = z.topk(k, 1).indices.int()
    counts = torch.bincount(idx.reshape(-1), minlength=E).int()
    return wl, layer, x, z, idx, counts, _rand(g, T, k), torch.tensor([2.5 * T, 0.01 * T], device=DEV)


@pytest.mark.parametrize("what", ["gates", "losses", "both"])
@pytest.mark.parametrize("mode", [0, 1, 2], ids=["topk_softmax", "renorm", "raw"])
@pytest.mark.parametrize("T,d,E,k", ROUTES)
def test_route_backward(T, d, E, k, mode, what):
    for dt in (F32, BF16):
        wl, layer, x, z, idx, counts, dg, dl = _route_case(T, d, E, k, dt, mode, T + E)
        dg, dl = (None if what == "losses" else dg), (None if what == "gates" else dl)
        dz, dx, gr = torch.empty_like(z), torch.empty(T, d, device=DEV), layer.new_grads()
        layer.route_backward(x, z, idx, counts if dl is not None else None, dg, dl, dz, dx, gr)
        ref, lim = R.route_bwd(z, idx, counts, dg, dl, mode, wl.aux_alpha)
        R.check(dz, ref, lim, "dlogits")
        w, xd = layer.p["w_router"].double(), x.double()
        # the projection's own splitting of dz keeps 2^-22 of each value
        R.check(dx, ref @ w, lim @ w.abs() + ((E + 2) * R.A + 2.0 ** -22) * (ref.abs() @ w.abs()), "dx")
        rw = ref.T @ xd
        lw = lim.T @ xd.abs() + ((T + 2) * R.A + 2.0 ** -16) * (ref.abs().T @ xd.abs())
        R.check(gr["w_router"], rw, lw + R.U(wl.torch_dtype) * (rw.abs() + lw), "dw")
        R.check(gr["b_router"], ref.sum(0), lim.sum(0) + (T + 2) * R.A * ref.abs().sum(0), "db")
        if T > 30:
            R.check_norm(gr["w_router"], rw, wl.torch_dtype, "dw")
        # again, with fewer outputs: the same bits
        d2, g2 = torch.empty_like(dx), {"b_router": torch.empty(E, device=DEV)}
        layer.route_backward(None, z, idx, counts, dg, dl, None, d2, g2)
        assert torch.equal(d2, dx) and torch.equal(g2["b_router"], gr["b_router"])
        assert layer.last_backward_error() == (0, 0)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_route_backward_with_masked_experts(mode):
    """Logits of -inf (masked experts), rows with nothing left, and the type's lowest value."""
    T, d, E, k = 50, 64, 12, 3
    wl, layer, x, z, _, _, dg, dl = _route_case(T, d, E, k, F32, mode, 11)
    z[:, 3] = float("-inf")
    z[5, :-1] = float("-inf")            # fewer live experts than slots
    z[6] = float("-inf")                 # none
    z[7, :6] = torch.finfo(torch.float32).min
    z[8] = torch.finfo(torch.float32).min
    idx = z.topk(k, 1).indices.int()
    counts = torch.bincount(idx.reshape(-1), minlength=E).int()
    dz, dx, gr = torch.empty_like(z), torch.empty(T, d, device=DEV), layer.new_grads()
    dl = dl * torch.tensor([1.0, 0.0], device=DEV)   # lse^2 of the lowest value overflows
    layer.route_backward(x, z, idx, counts, dg, dl, dz, dx, gr)
    assert torch.isfinite(dz).all() and (dz[6] == 0).all()
    assert (dz[torch.isneginf(z)] == 0).all()   # row 8's equal lowest values share a probability
    keep = torch.tensor([t for t in range(T) if t not in (7, 8)], device=DEV)
    ref, lim = R.route_bwd(z, idx, counts, dg, dl, mode, wl.aux_alpha)
    R.check(dz[keep], ref[keep], lim[keep], "dlogits")
    assert layer.last_backward_error() == (0, 0)


def test_expert_indices_out_of_range_are_reported():
    wl, layer, x, z, idx, counts, dg, _ = _route_case(64, 64, 8, 2, F32, 0, 3)
    idx[9, 1] = 8
    dz = torch.empty_like(z)
    layer.route_backward(None, z, idx, None, dg, None, dz, None)
    assert layer.last_backward_error() == (1, 19)
    assert torch.isfinite(dz).all()


# ----------------------------------------------------------------------- experts
FFN = [  # d, F, rows per expert
    (64, 64, [1]), (64, 256, [5, 0, 64, 3]), (128, 320, [0, 1, 129, 300, 64, 0]), (256, 384, [65, 127, 128, 17]),
    (512, 192, [257]), (192, 640, [1, 2, 3, 4, 5, 6, 7, 8]), (64, 64, [0, 0]), (1024, 128, [31, 33]),
    (320, 576, [700, 255, 256, 511]), (64, 192, [i % 5 for i in range(100)]), (576, 64, [0, 0, 90, 0]),
    (64, 1088, [2, 0, 1]), (128, 832, [9, 30, 1]), (64, 2048, [70, 100]),
    (64, 7104, [1, 1]), (2112, 64, [1, 0, 2]),
]
ACTS = [synth.ACT_RELU, synth.ACT_GELU, synth.ACT_SWIGLU]


def _ffn_case(d, F, rows, act, dt, seed, spare=3):
    E, n = len(rows), sum(rows)
    wl = _workload(max(1, n + spare), d, E, 1, dt, F=F, act=act)
    g, tdt = _gen(seed), wl.torch_dtype
    p = {"w1": _rand(g, E, F, d, dt=tdt, std=1 / math.sqrt(d)),
         "w2": _rand(g, E, d, F, dt=tdt, std=1 / math.sqrt(F))}
    if act == synth.ACT_SWIGLU:
        p["w3"] = _rand(g, E, F, d, dt=tdt, std=1 / math.sqrt(d))
    else:
        p["b1"], p["b2"] = _rand(g, E, F, std=0.3), _rand(g, E, d, std=0.3)
    layer = B.MoELayer(wl, p, DEV)
    x, dy = _rand(g, wl.T, d, dt=tdt), _rand(g, wl.T, d, dt=tdt)
    x[n:] = float("nan")                       # rows past the last expert's are not read ...
    dy[n:] = float("inf")
    off = torch.tensor([0] + list(itertools.accumulate(rows)), dtype=torch.int32, device=DEV)
    return wl, layer, x, dy, off, n


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("act", ACTS, ids=["relu", "gelu", "swiglu"])
@pytest.mark.parametrize("d,F,rows", FFN)
def test_expert_ffn_backward(d, F, rows, act, dt):
    wl, layer, x, dy, off, n = _ffn_case(d, F, rows, act, dt, d + F + sum(rows))
    tdt = wl.torch_dtype
    gr = layer.new_grads()
    for t in gr.values():
        t.fill_(float("nan"))
    dx = torch.full((wl.T, d), 3.0, dtype=tdt, device=DEV)
    layer.expert_ffn_backward(x, off, dy, dx, gr)
    ref, lim = R.ffn_bwd(x, dy, off.tolist(), layer.p, act, tdt)
    for name, t in gr.items():
        if name not in ("w_router", "b_router"):
            R.check(t, ref[name], lim[name], name)
            if n > 100 and name in ("w1", "w2", "w3"):
                R.check_norm(t, ref[name], tdt, name)
    R.check(dx[:n], ref["dx"][:n], lim["dx"][:n], "dx")
    assert (dx[n:] == 3.0).all()               # ... nor written
    if n > 100:
        R.check_norm(dx[:n], ref["dx"][:n], tdt, "dx")
    for e, r in enumerate(rows):               # an expert without rows: zeros
        if r == 0:
            assert all((t[e] == 0).all() for nm, t in gr.items())
    # the same call again, and each output on its own, give the same bits
    g2, dx2 = layer.new_grads(), torch.full_like(dx, 3.0)
    for name in gr:
        layer.expert_ffn_backward(x, off, dy, None, {name: g2[name]})
    layer.expert_ffn_backward(x, off, dy, dx2, None)
    assert torch.equal(dx2, dx) and all(torch.equal(g2[nm], t) for nm, t in gr.items())
    assert layer.last_backward_error() == (0, 0)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_expert_ffn_backward_with_a_width_of_one_tile_and_a_bit(dt):
    """F and d that end inside every tile width (fp32: any F)."""
    d, F = (68, 161) if dt == F32 else (448, 832)
    wl, layer, x, dy, off, n = _ffn_case(d, F, [70, 1, 200], synth.ACT_GELU, dt, 5)
    gr, dx = layer.new_grads(), torch.empty_like(x)
    layer.expert_ffn_backward(x, off, dy, dx, gr)
    ref, lim = R.ffn_bwd(x, dy, off.tolist(), layer.p, synth.ACT_GELU, wl.torch_dtype)
    for name in ("w1", "w2", "b1", "b2"):
        R.check(gr[name], ref[name], lim[name], name)
    R.check(dx[:n], ref["dx"][:n], lim["dx"][:n], "dx")


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("bad", [[0, 5, 3, 9], [0, 5, 10, 9999], [2, 5, 6, 9], [0, -1, 3, 9]])
def test_invalid_offsets_are_reported_and_nothing_is_read(bad, dt):
    wl, layer, x, dy, _, n = _ffn_case(64, 64, [5, 5, 5], synth.ACT_SWIGLU, dt, 2)
    gr, dx = layer.new_grads(), torch.full_like(x, 3.0)
    layer.expert_ffn_backward(x, torch.tensor(bad, dtype=torch.int32, device=DEV), dy, dx, gr)
    assert layer.last_backward_error()[0] == 2
    assert (dx == 3.0).all() and all((gr[nm] == 0).all() for nm in ("w1", "w2", "w3"))


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("act", ACTS, ids=["relu", "gelu", "swiglu"])
def test_experts_do_not_touch_one_another(act, dt):
    """Infinities and NaN in one expert's rows and weights stay with it, and what the workspace
    held before is not read."""
    rows = [70, 3, 64, 129]
    wl, layer, x, dy, off, n = _ffn_case(192, 320, rows, act, dt, 77)
    dx, gr = torch.empty_like(x), layer.new_grads()
    layer.expert_ffn_backward(x, off, dy, dx, gr)
    x2, dy2 = x.clone(), dy.clone()
    x2[73 + 10], dy2[73 + 20, 5] = float("nan"), float("inf")      # rows of expert 2
    for nm in ("w1", "w2", "w3", "b1"):
        if layer.p.get(nm) is not None:
            layer.p[nm][2].reshape(-1)[7] = float("-inf")
    layer.bws[64:].fill_(255)                                      # NaN in every type
    dx2, g2 = torch.empty_like(x), layer.new_grads()
    layer.expert_ffn_backward(x2, off, dy2, dx2, g2)
    keep = [0, 1, 3]
    for nm in g2:
        if nm not in ("w_router", "b_router"):
            assert torch.equal(g2[nm][keep], gr[nm][keep]), nm
    assert torch.equal(dx2[:73], dx[:73]) and torch.equal(dx2[137:n], dx[137:n])
    assert not torch.isfinite(g2["w1"][2].float()).all()
    assert layer.last_backward_error() == (0, 0)


def test_expert_choice_rows_have_expert_gradients():
    """moe_expert_ffn_backward takes the expert-choice layout (E * C rows) as well."""
    wl = synth.SMALL["ec_small"]
    inp = synth.generate(wl, seed=4)
    layer = B.MoELayer(wl, inp, DEV)
    n = B.expert_rows(layer.cfg)
    C, g = n // wl.n_experts, _gen(6)
    x, dy = (_rand(g, n, wl.d_model, dt=torch.bfloat16) for _ in range(2))
    off = torch.arange(wl.n_experts + 1, device=DEV, dtype=torch.int32) * C
    gr, dx = layer.new_grads(), torch.empty_like(x)
    layer.expert_ffn_backward(x, off, dy, dx, gr)
    ref, lim = R.ffn_bwd(x, dy, off.tolist(), layer.p, wl.act, torch.bfloat16)
    R.check(dx, ref["dx"], lim["dx"], "dx")
    for nm in ("w1", "w2", "w3"):
        R.check(gr[nm], ref[nm], lim[nm], nm)
    with pytest.raises(B.MoeError):
        layer.permute_backward(torch.empty(wl.T, wl.d_model, dtype=torch.bfloat16, device=DEV),
                               torch.zeros(wl.T, dtype=torch.int32, device=DEV), None,
                               torch.empty(wl.T, wl.d_model, dtype=torch.bfloat16, device=DEV))


def test_offsets_past_32_bits():
    """Row buffers of more than 2^31 elements: the last rows are the right ones."""
    T, d, k, b = 33000, 8192, 8, torch.bfloat16
    wl = _workload(T, d, 8, k, BF16)
    layer, g = B.MoELayer(wl, {}, DEV), _gen(1)
    inv = torch.arange(T * k, device=DEV, dtype=torch.int32).flip(0).contiguous()
    dy, gate = _rand(g, T, d, dt=b), torch.rand(T, k, device=DEV, generator=g)
    yp = torch.empty(T * k, d, dtype=b, device=DEV).normal_(generator=g)
    out, dgate = torch.zeros_like(yp), torch.empty(T, k, device=DEV)
    layer.combine_backward(dy, yp, inv, gate, out, dgate)
    for t in (0, 1, T // 2, T - 1):
        rows = inv.reshape(T, k)[t].long()
        ref = dy[t].double() * gate[t].double()[:, None]
        R.check(out[rows], ref, (R.U(b) + 2.0 ** -23) * ref.abs(), "dy_perm")
        dot = yp[rows].double() * dy[t].double()
        R.check(dgate[t], dot.sum(1), (d + 2) * R.A * dot.abs().sum(1), "dgate")
    dx = torch.empty(T, d, dtype=b, device=DEV)
    layer.permute_backward(yp, inv, None, dx)
    for t in (0, T - 1):
        x = yp[inv.reshape(T, k)[t].long()].double()
        R.check(dx[t], x.sum(0), R.U(b) * 1.01 * x.sum(0).abs() + k * R.A * x.abs().sum(0), "dx")
    del yp, out, dx
    # and the experts' hidden rows
    rows, d, F = [1, 40000], 64, 57344
    wl, layer, x, dy, off, n = _ffn_case(d, F, rows, synth.ACT_RELU, BF16, 3)
    dx, gr = torch.empty_like(x), {m: layer.new_grads()[m] for m in ("w1", "w2")}
    layer.expert_ffn_backward(x, off, dy, dx, gr)
    p, e = {m: v[1:].double() for m, v in layer.p.items() if v is not None and m != "w_router"}, 1
    last = slice(n - 3, n)                       # three rows of expert 1 by themselves
    ref, lim = R.ffn_bwd(x[last], dy[last], [0, 3], {m: v for m, v in p.items()}, synth.ACT_RELU, b)
    R.check(dx[last], ref["dx"], lim["dx"], "dx")
    cols = slice(F - 64, F)                      # the last hidden columns, all rows
    few = {"w1": p["w1"][:, cols], "w2": p["w2"][:, :, cols].contiguous(), "b1": p["b1"][:, cols],
           "b2": p["b2"]}
    ref, lim = R.ffn_bwd(x[1:n], dy[1:n], [0, n - 1], few, synth.ACT_RELU, b)
    R.check(gr["w1"][1][cols], ref["w1"][0], lim["w1"][0], "w1")
    R.check(gr["w2"][1][:, cols], ref["w2"][0], lim["w2"][0], "w2")
    assert layer.last_backward_error() == (0, 0)


# --------------------------------------------------------------- the whole layer
LAYERS = ["tiny", "mixtral_small", "deepseek_small", "switch_small", "mixtral_cap", "decode_small",
          "deepseek_decode", "fp32_swiglu", "fp32_gelu_cap", "router_e20", "router_e256", "one_token"]


def _layer_workload(name):
    if name == "one_token":
        return synth.SMALL["deepseek_small"].replace(name="one_token", T=1)
    return synth.SMALL[name]


def _forward(wl, seed):
    inp = synth.generate(wl, seed=seed)
    layer = B.MoELayer(wl, inp, DEV)
    x, taps = inp["x"].to(DEV), layer.new_taps()
    layer.forward(x, taps=taps)
    return layer, x, taps, _rand(_gen(seed + 1), wl.T, wl.d_model, dt=wl.torch_dtype)


@pytest.mark.parametrize("losses", [False, True], ids=["", "losses"])
@pytest.mark.parametrize("name", LAYERS)
def test_layer_backward(name, losses):
    wl = _layer_workload(name)
    layer, x, taps, dy = _forward(wl, 8)
    dl = torch.tensor([3.0, 0.2], device=DEV) if losses else None
    dx, gr = layer.backward(x, dy, taps, d_losses=dl)
    assert layer.last_backward_error() == (0, 0) and layer.last_device_error() == (0, 0)
    ref, lim = R.layer_bwd(x, dy, taps, layer.p, wl, dl)
    R.check(dx, ref["dx"], lim["dx"], "dx")
    for nm, t in gr.items():
        R.check(t, ref[nm], lim[nm], nm)
        if wl.T > 100 and nm[0] == "w" and nm != "w_router":
            R.check_norm(t, ref[nm], wl.torch_dtype, nm)
    if wl.T > 100:
        R.check_norm(dx, ref["dx"], wl.torch_dtype, "dx")
    # the same bits again, and for each output on its own
    dx2, g2 = layer.backward(x, dy, taps, d_losses=dl)
    assert torch.equal(dx, dx2) and all(torch.equal(gr[nm], g2[nm]) for nm in gr)
    dx3, g3 = layer.backward(x, dy, taps, d_losses=dl, grads={})
    assert torch.equal(dx, dx3) and g3 == {}


@pytest.mark.parametrize("name", ["tiny", "deepseek_small", "switch_small"])
def test_layer_backward_is_the_steps_put_together(name):
    """The separate entry points, as a caller with experts of their own would run them,
    give the whole layer's gradients up to the roundings between them."""
    wl = _layer_workload(name).replace(n_shared=0, d_ff_shared=0)
    layer, x, taps, dy = _forward(wl, 21)
    T, d, k = wl.T, wl.d_model, wl.top_k
    dx, gr = layer.backward(x, dy, taps)
    xp, yp = (torch.zeros(T * k, d, dtype=x.dtype, device=DEV) for _ in range(2))
    c, o, pm, iv = (torch.empty_like(taps[n]) for n in ("counts", "offsets", "perm", "inv"))
    layer.permute(x, taps["topk_idx"], c, o, pm, iv, xp)
    assert torch.equal(iv, taps["inv"]) and torch.equal(o, taps["offsets"])
    layer.expert_ffn(xp, o, yp)
    dyp, dg = torch.zeros_like(xp), torch.empty_like(taps["topk_gate"])
    layer.combine_backward(dy, yp, iv, taps["topk_gate"], dyp, dg)
    dxp, g2 = torch.zeros_like(xp), layer.new_grads()
    layer.expert_ffn_backward(xp, o, dyp, dxp, g2)
    dxr, dx2 = torch.empty(T, d, device=DEV), torch.empty_like(dx)
    layer.route_backward(x, taps["logits"], taps["topk_idx"], None, dg, None, None, dxr, g2)
    layer.permute_backward(dxp, iv, dxr, dx2)
    ref, _ = R.layer_bwd(x, dy, taps, layer.p, wl)
    # up to five roundings on the way of a value (dy_perm, h and da, y_perm, dx_perm, dx)
    R.check_norm(dx2, ref["dx"], wl.torch_dtype, "dx", roundings=5)
    for nm in g2:
        R.check_norm(g2[nm], ref[nm], wl.torch_dtype, nm, roundings=5)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_no_tokens(dt):
    wl = _workload(0, 64, 4, 2, dt, n_shared=1, d_ff_shared=64)
    inp = synth.generate(wl, seed=0)
    layer = B.MoELayer(wl, inp, DEV)
    x, taps = inp["x"].to(DEV), layer.new_taps()
    gr = layer.new_grads()
    for t in gr.values():
        t.fill_(float("nan"))
    dx, _ = layer.backward(x, torch.empty_like(x), taps, grads=gr)
    assert dx.shape == (0, 64) and all((t == 0).all() for t in gr.values())


def test_binding_refuses_what_the_library_cannot_see():
    wl = synth.SMALL["mixtral_small"]
    layer, x, taps, dy = _forward(wl, 2)
    with pytest.raises(ValueError):
        layer.backward(x, dy.float(), taps)
    with pytest.raises(ValueError):
        layer.backward(x, dy[:-1], taps)
    with pytest.raises(ValueError):
        layer.backward(x, dy, {k: v for k, v in taps.items() if k != "inv"})
    with pytest.raises(ValueError):
        layer.backward(x, dy, taps, grads={"b1": torch.empty(8, 384, device=DEV)})
    with pytest.raises(ValueError):
        layer.backward(x, dy.cpu(), taps)
    with pytest.raises(ValueError):
        layer.permute_backward(x, taps["inv"], None, x)
    with pytest.raises(ValueError):
        layer.combine_backward(dy.t(), None, taps["inv"], taps["topk_gate"], None, None)


# ------------------------------------------------------------------------- AdamW
def _adam_case(sizes, pdt, gdt, bits, master, seed):
    g = _gen(seed)
    ps = [_rand(g, n, dt=pdt, std=0.5) for n in sizes]
    gs = [(_rand(g, n) * torch.exp(_rand(g, n))).to(gdt) for n in sizes]
    opt = B.AdamW(ps, lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1, state_bits=bits,
                  master=master)
    return ps, gs, opt


SIZES = [1, 7, 8, 255, 256, 257, 4095, 4096, 4097, 100003]


@pytest.mark.parametrize("master", [False, True], ids=["", "master"])
@pytest.mark.parametrize("pdt,gdt", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                     (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_adamw_32_bit_states(pdt, gdt, master):
    ps, gs, opt = _adam_case(SIZES, pdt, gdt, 32, master, 1)
    h = (0.01, 0.8, 0.95, 1e-6, 0.1)
    for t in range(1, 4):
        old = [(m.clone() if m is not None else p.clone(), a.clone(), b.clone())
               for p, m, a, b in zip(ps, opt.master, opt.exp_avg, opt.exp_avg_sq)]
        opt.step(gs)
        for i, (p, m, v) in enumerate(old):
            rp, rm, rv = R.adamw(p, gs[i], m, v, t, *h)
            e = 2.0 ** -24
            lm = 4 * e * (m.double().abs() + gs[i].double().abs())
            R.check(opt.exp_avg[i], rm, lm, "m")
            R.check(opt.exp_avg_sq[i], rv, 6 * e * rv + 1e-45, "v")
            # m, the quotient (v's and the root's roundings among it), two products and a sum
            upd = 0.01 / (1 - 0.8 ** t) / ((rv / (1 - 0.95 ** t)).sqrt() + 1e-6)
            lp = 4 * e * p.double().abs() + upd * (lm + 16 * e * rm.abs())
            w = opt.master[i] if opt.master[i] is not None else ps[i]
            R.check(w, rp, lp + (R.U(w.dtype) * (rp.abs() + lp)), "p")
            if opt.master[i] is not None:
                assert torch.equal(ps[i], opt.master[i].to(pdt))


@pytest.mark.parametrize("pdt", [torch.float32, torch.bfloat16])
def test_adamw_8_bit_states(pdt):
    ps, gs, opt = _adam_case(SIZES, pdt, pdt, 8, False, 2)
    gs[-1][1000:1300] = 0                       # a block whose second moment is 0 at first
    gs[-1][5000:5100] *= 1e-4                   # small beside large ones in one block
    for t in range(1, 4):
        old = [(p.clone(), a.clone(), b.clone(), c.clone(), d.clone()) for p, a, b, c, d in
               zip(ps, opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale)]
        opt.step(gs)
        for i, (p, a, b, sa, sb) in enumerate(old):
            m, r = R.from_8(a, sa), R.from_8(b, sb)
            rp, rm, rv = R.adamw(p, gs[i], m, r * r, t, 0.01, 0.8, 0.95, 1e-6, 0.1)
            e = 2.0 ** -24
            lm = 6 * e * (m.abs() + gs[i].double().abs())
            upd = 0.01 / (1 - 0.8 ** t) / ((rv / (1 - 0.95 ** t)).sqrt() + 1e-6)
            lp = 4 * e * p.double().abs() + upd * (lm + 20 * e * rm.abs())
            R.check(ps[i], rp, lp + R.U(pdt) * (rp.abs() + lp), "p")
            for val, codes, scale, root in ((rm, opt.exp_avg[i], opt.exp_avg_scale[i], False),
                                            (rv.sqrt(), opt.exp_avg_sq[i], opt.exp_avg_sq_scale[i], True)):
                n = val.numel()
                pad = torch.nn.functional.pad(val.abs(), (0, -n % 256)).reshape(-1, 256).amax(1)
                R.check(scale, (pad.clamp(min=2.0 ** -100)) / 448, 8 * e * pad.clamp(min=2.0 ** -100) / 448
                        + lm.max() / 448, "scale")
                each = scale.double()[torch.arange(n, device=DEV) // 256]
                # half a step of e4m3 (2^-4 of the value, 2^-10 of a scale below 2^-6), the
                # smallest code of a root, and the value's own error
                lim = 2.0 ** -4 * val.abs() * 1.001 + 2.0 ** -10 * each + lm
                if root:
                    lim = lim + 2.0 ** -9 * each
                R.check(R.from_8(codes, scale), val, lim, "codes")
                if root:
                    assert (R.from_8(codes, scale)[val > 0] > 0).all()


def test_adamw_many_tensors_one_step():
    """More tensors than one launch holds, empty ones among them."""
    sizes = [(i * 37) % 701 for i in range(700)]
    ps, gs, opt = _adam_case(sizes, torch.float32, torch.float32, 32, False, 3)
    old = [p.clone() for p in ps]
    opt.step(gs)
    for p, o, g in zip(ps, old, gs):
        rp, _, rv = R.adamw(o, g, torch.zeros_like(o), torch.zeros_like(o), 1, 0.01, 0.8, 0.95, 1e-6, 0.1)
        R.check(p, rp, 2.0 ** -20 * (rp.abs() + 0.01), "p")


def test_adamw_scalars_on_the_device():
    ps, gs, opt = _adam_case([1000, 31], torch.float32, torch.float32, 32, False, 4)
    q, _, ref = _adam_case([1000, 31], torch.float32, torch.float32, 32, False, 4)
    one = lambda v, dt=torch.float32: torch.tensor([v], dtype=dt, device=DEV)  # noqa: E731
    before = [p.clone() for p in ps]
    opt.step(gs, found_inf=one(1.0))
    assert all(torch.equal(p, b) for p, b in zip(ps, before)) and (opt.exp_avg[0] == 0).all()
    opt.t = 0
    opt.step(gs, grad_scale=one(0.5), found_inf=one(0.0))
    ref.step([g * 0.5 for g in gs])
    assert all(torch.equal(p, r) for p, r in zip(ps, q))
    opt.lr = 123.0
    opt.step(gs, step=one(2, torch.int64), lr=one(0.01))
    ref.step(gs)
    for p, r in zip(ps, q):  # the device's own powers: a rounding apart at most
        assert torch.allclose(p, r, rtol=1e-6, atol=1e-7)


def test_adamw_takes_gradients_by_name():
    ps, gs, opt = _adam_case([100, 100, 7], torch.float32, torch.float32, 32, False, 6)
    qs = {n: p.clone() for n, p in zip("abc", ps)}
    named = B.AdamW(qs, lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    opt.step(gs)
    named.step({"other": gs[0], "c": gs[2], "b": gs[1], "a": gs[0]})
    assert all(torch.equal(p, q) for p, q in zip(ps, qs.values()))
    with pytest.raises(ValueError):
        named.step({"a": gs[0], "b": gs[1]})
    with pytest.raises(ValueError):
        opt.step(dict(zip("abc", gs)))
    with pytest.raises(ValueError):
        B.AdamW([ps[0], ps[0]])


def test_adamw_refuses_what_does_not_fit():
    ps, gs, opt = _adam_case([100, 31], torch.float32, torch.float32, 32, False, 4)
    with pytest.raises(ValueError):
        opt.step(gs[:1])
    with pytest.raises(ValueError):
        opt.step([gs[0], gs[0]])
    with pytest.raises(ValueError):
        opt.step([g.cpu() for g in gs])
    with pytest.raises(ValueError):
        opt.step([g.half() for g in gs])
    with pytest.raises(ValueError):
        opt.step(gs, grad_scale=torch.ones(2, device=DEV))
    with pytest.raises(ValueError):
        B.AdamW(ps, state=dict(step=1, exp_avg=opt.exp_avg, exp_avg_sq=opt.exp_avg_sq[:1]))
    with pytest.raises(B.MoeError):   # a view that breaks the 16-byte rule
        base = torch.zeros(101, device=DEV)
        B.AdamW([base[1:]]).step([gs[0]])


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_state_continues_a_run(bits):
    ps, gs, opt = _adam_case([3000, 77], torch.bfloat16, torch.bfloat16, bits, bits == 32, 9)
    opt.step(gs)
    st = opt.state_dict()
    copy = lambda x: None if x is None else [None if t is None else t.clone() for t in x]  # noqa: E731
    ps2 = [p.clone() for p in ps]
    two = B.AdamW(ps2, lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1,
                  state={k: (v if k == "step" else copy(v)) for k, v in st.items()})
    opt.step(gs)
    two.step(gs)
    assert two.t == opt.t == 2 and all(torch.equal(a, b) for a, b in zip(ps, ps2))


# ------------------------------------------------------------- the step as a whole
def _train(wl, steps, seed, how):
    """`steps` training steps (forward, gradients, AdamW) on new inputs each: eagerly, on a
    side stream, or captured once and replayed. Returns outputs, gradients and weights."""
    inp = synth.generate(wl, seed=seed)
    layer = B.MoELayer(wl, inp, DEV)
    params = {n: layer.p[n] for n in layer.grad_shapes() if layer.p.get(n) is not None}
    opt = B.AdamW(params, lr=1e-2, betas=(0.9, 0.95), weight_decay=0.1, master=True)
    g = _gen(seed)
    xs = [_rand(g, wl.T, wl.d_model, dt=wl.torch_dtype) for _ in range(steps)]
    dys = [_rand(g, wl.T, wl.d_model, dt=wl.torch_dtype) for _ in range(steps)]
    dl = torch.tensor([3.0, 0.2], device=DEV)
    x, dy, y = torch.empty_like(xs[0]), torch.empty_like(dys[0]), torch.empty_like(xs[0])
    taps, aux, grads, dx = layer.new_taps(), layer.new_aux(), layer.new_grads(), torch.empty_like(x)
    count, lr = torch.zeros(1, dtype=torch.int64, device=DEV), torch.tensor([1e-2], device=DEV)
    layer.bws  # made before a capture

    def one():
        count.add_(1)
        layer.forward(x, y, aux=aux, taps=taps)
        layer.backward(x, dy, taps, dx=dx, grads=grads, d_losses=dl)
        opt.step(grads, step=count, lr=lr)

    seen = []
    side = torch.cuda.Stream()
    graph = None
    if how == "graph":
        saved = [t.clone() for t in list(params.values())]
        x.copy_(xs[0])
        dy.copy_(dys[0])
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            one()
        assert all(torch.equal(a, b) for a, b in zip(saved, params.values()))
        assert int(count) == 0
    for i in range(steps):
        if how == "side":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                x.copy_(xs[i])
                dy.copy_(dys[i])
                one()
            torch.cuda.current_stream().wait_stream(side)
        else:
            x.copy_(xs[i])
            dy.copy_(dys[i])
            graph.replay() if graph else one()
        seen.append([t.clone() for t in (y, aux, dx, *grads.values(), *params.values())])
    assert layer.last_backward_error() == (0, 0) and layer.last_device_error() == (0, 0)
    return seen


@pytest.mark.parametrize("how", ["side", "graph"])
@pytest.mark.parametrize("name", ["tiny", "deepseek_small", "switch_small", "decode_small"])
def test_training_steps_agree_however_they_are_launched(name, how):
    wl = synth.SMALL[name]
    a, b = _train(wl, 3, 5, "eager"), _train(wl, 3, 5, how)
    for s, t in zip(a, b):
        assert all(torch.equal(p, q) for p, q in zip(s, t))


@pytest.mark.parametrize("name", ["deepseek_small", "switch_small", "fp32_gelu_cap"])
def test_two_layers_at_once_and_a_stale_workspace(name):
    """Two layers on two streams give what each gives alone, from workspaces full of NaN."""
    wl = _layer_workload(name)
    made = [_forward(wl, seed) for seed in (31, 32)]
    alone = [layer.backward(x, dy, taps) for layer, x, taps, dy in made]
    for layer, *_ in made:
        layer.bws[64:].fill_(255)
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    out = []
    for _ in range(3):
        for s, (layer, x, taps, dy) in zip(streams, made):
            with torch.cuda.stream(s):
                out.append(layer.backward(x, dy, taps))
    torch.cuda.synchronize()
    for i, (dx, gr) in enumerate(out):
        rx, rg = alone[i % 2]
        assert torch.equal(dx, rx) and all(torch.equal(gr[n], rg[n]) for n in rg)
    assert all(layer.last_backward_error() == (0, 0) for layer, *_ in made)


def test_training_step_against_64_bits():
    """One step of an fp32 layer: the weights after it are the reference's, where the
    gradient is known well enough for AdamW's quotient (|g| far above its own error)."""
    wl = synth.SMALL["fp32_swiglu"]
    layer, x, taps, dy = _forward(wl, 13)
    old = {n: layer.p[n].clone() for n in layer.grad_shapes() if layer.p.get(n) is not None}
    dx, gr = layer.backward(x, dy, taps)
    ref, lim = R.layer_bwd(x, dy, taps, layer.p, wl)
    opt = B.AdamW({n: layer.p[n] for n in old}, lr=1e-2, betas=(0.9, 0.95), weight_decay=0.1)
    opt.step([gr[n] for n in old])
    for n, w in old.items():
        z = torch.zeros_like(w)
        rp, _, _ = R.adamw(w, ref[n], z, z, 1, 1e-2, 0.9, 0.95, 1e-8, 0.1)
        # the first step moves each weight by lr g / (|g| + eps): its slope in g is at most
        # lr eps / (|g| + eps)^2 beyond |g| - lim, and the sign holds there
        known = ref[n].abs() > 2 * lim[n] + 1e-4
        R.check(layer.p[n][known], rp[known], (1e-2 * 1e-8 / (ref[n].abs() / 2) ** 2 * lim[n]
                                               + 2.0 ** -20 * (rp.abs() + 1e-2))[known], n)
        assert known.double().mean() > 0.5
