"""The training step at the edges of what its documentation allows: storage that is
replaced between steps, steps with nothing between them, sizes past a launch's limits,
dispatch that needs wide fp32 layers. Limits as in tests/train_ref.py."""
import pytest
import torch

from sparse_mixture_experts_12_b200 import binding as B
from sparse_mixture_experts_12_b200 import build as BUILD
from sparse_mixture_experts_12_b200 import synth
from tests import test_gpu_train as G
from tests import train_ref as R
from tests.test_gpu_train import DEV, _adam_case, _forward, _gen, _rand, _workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    BUILD.build()
    yield B.load()


# ------------------------------------------------------------------------- AdamW
def test_adamw_refuses_a_parameter_whose_storage_was_replaced():
    for replace in ("data", "set_"):
        ps, gs, opt = _adam_case([100, 31], torch.float32, torch.float32, 32, False, 4)
        first, was = ps[1].detach(), ps[1].clone()   # an alias keeps the old storage
        if replace == "data":
            ps[1].data = torch.zeros_like(was)
        else:
            ps[1].set_(torch.zeros_like(was))
        with pytest.raises(ValueError, match="parameter 1"):
            opt.step(gs)
        assert opt.t == 0 and torch.equal(first, was) and (ps[1] == 0).all()
        assert all((m == 0).all() for m in opt.exp_avg)
        # a new optimizer goes on from the old one's state
        two = B.AdamW(ps, lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1,
                      state=opt.state_dict())
        two.step(gs)
        rp, _, _ = R.adamw(torch.zeros_like(was), gs[1], was * 0, was * 0, 1, 0.01, 0.8, 0.95,
                           1e-6, 0.1)
        # one step from zero is lr g / (|g| + eps), a handful of fp32 roundings
        R.check(ps[1], rp, 2.0 ** -20 * rp.abs() + 1e-12, "p")


def test_adamw_sees_a_replacement_of_the_freed_block():
    """A smaller tensor that takes the old storage's block is not taken for the parameter."""
    n = 8 << 20                                       # 32 MB: a block of its own
    p = torch.zeros(n, device=DEV)
    opt, g = B.AdamW([p]), torch.ones(n, device=DEV)
    torch.cuda.synchronize()
    p.data = torch.empty(0, device=DEV)
    small = torch.full((6 << 20,), 7.0, device=DEV)   # the allocator gives freed blocks first
    other = torch.full((2 << 20,), 7.0, device=DEV)
    p.data = small
    with pytest.raises(ValueError, match="parameter 0"):
        opt.step([g])
    assert (small == 7).all() and (other == 7).all()


def test_adamw_names_a_gradient_that_is_missing():
    ps, gs, opt = _adam_case([100, 31], torch.float32, torch.float32, 32, False, 4)
    was = [p.clone() for p in ps]
    named = B.AdamW({"a": ps[0], "b": ps[1]})
    for call in (lambda: opt.step([gs[0], None]), lambda: named.step({"a": gs[0], "b": None}),
                 lambda: opt.step([gs[0], gs[1].cpu().numpy()])):
        with pytest.raises(ValueError, match="gradient 1"):
            call()
    assert opt.t == named.t == 0 and all(torch.equal(p, w) for p, w in zip(ps, was))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_state_cannot_be_pulled_from_under_it(bits):
    """The state's tensors cannot be exchanged, and what happens to them leaves the memory that
    the step writes in place."""
    ps, gs, opt = _adam_case([1000], torch.float32, torch.float32, bits, False, 5)
    qs, _, ref = _adam_case([1000], torch.float32, torch.float32, bits, False, 5)
    for name in ("exp_avg", "exp_avg_sq", "master"):
        with pytest.raises(TypeError):
            getattr(opt, name)[0] = None
    opt.step(gs)
    ref.step(gs)
    size = opt.exp_avg[0].untyped_storage().nbytes()
    opt.exp_avg[0].set_(torch.empty(0, dtype=opt.exp_avg[0].dtype, device=DEV))
    torch.cuda.empty_cache()
    other = torch.full((size,), 7, dtype=torch.uint8, device=DEV)  # would take the freed block
    opt.step(gs)
    ref.step(gs)
    assert (other == 7).all() and all(torch.equal(p, q) for p, q in zip(ps, qs))


# ------------------------------------------------------------- the step as a whole
def _steps(wl, how, n=4):
    """n training steps on one input; the router's biases are trained too. "apart": the GPU is
    waited for after every call; "together": nothing lies between one call and the next;
    "graph": so, captured and replayed once. Returns what the last step left."""
    wl = wl.replace(router_bias=True, logit_bias_std=0.5, bias_std=0.1)
    layer, x, taps, dy = _forward(wl, 17)
    names = [m for m in layer.grad_shapes() if layer.p.get(m) is not None] + ["logit_bias"]
    opt = B.AdamW([layer.p[m] for m in names], lr=0.05, betas=(0.8, 0.9))
    gr, dx, y = layer.new_grads(), torch.empty_like(x), torch.empty_like(x)
    grads = [gr["b_router" if m == "logit_bias" else m] for m in names]
    layer.bws
    torch.cuda.synchronize()

    def run():
        for _ in range(n):
            for call in (lambda: layer.forward(x, y, taps=taps),
                         lambda: layer.backward(x, dy, taps, dx=dx, grads=gr),
                         lambda: opt.step(grads)):
                call()
                if how == "apart":
                    torch.cuda.synchronize()

    if how == "graph":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graph.replay()
    else:
        run()
    torch.cuda.synchronize()
    assert layer.last_backward_error() == (0, 0) and layer.last_device_error() == (0, 0)
    return [y, dx, taps["logits"], *grads, *(layer.p[m] for m in names)]


@pytest.mark.parametrize("how", ["together", "graph"])
@pytest.mark.parametrize("name", ["router_e20", "router_e256", "switch_small", "decode_e32", "tiny",
                                  "fp32_gelu_cap", "deepseek_small"])
def test_steps_with_nothing_between_them(name, how):
    """An optimizer step directly ahead of the next forward pass: its kernels see the weights
    and the biases that the step wrote."""
    wl = synth.SMALL[name]
    for a, b in zip(_steps(wl, "apart"), _steps(wl, how)):
        assert torch.equal(a, b)


def test_the_gradients_workspace_is_made_outside_a_capture():
    layer, x, taps, dy = _forward(synth.SMALL["mixtral_small"], 5)
    dx, gr = torch.empty_like(x), layer.new_grads()
    graph, one = torch.cuda.CUDAGraph(), torch.zeros(1, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        one.add_(1)
        with pytest.raises(RuntimeError, match="before a capture"):
            layer.backward(x, dy, taps, dx=dx, grads=gr)
    graph.replay()
    assert float(one) == 1
    layer.bws
    with torch.cuda.graph(graph2 := torch.cuda.CUDAGraph()):
        layer.backward(x, dy, taps, dx=dx, grads=gr)
    graph2.replay()
    dx2, g2 = layer.backward(x, dy, taps)
    assert torch.equal(dx, dx2) and all(torch.equal(gr[n], g2[n]) for n in gr)
    assert layer.last_backward_error() == (0, 0)


def test_the_gradients_workspace_is_ready_on_every_stream():
    """Made on a stream that is behind, it is initialised all the same when another uses it."""
    layer, x, taps, dy = _forward(synth.SMALL["mixtral_small"], 5)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)     # some 10 ms of clocks
        layer.bws
        assert side.query()
    assert layer.last_backward_error() == (0, 0)


def test_a_layers_weights_cannot_be_pulled_from_under_it():
    """The layer reads and differentiates the storage it was made with, whose memory stays."""
    layer, x, taps, dy = _forward(synth.SMALL["mixtral_small"], 6)
    y, (dx, gr) = layer.forward(x), layer.backward(x, dy, taps)
    sizes = {n: t.numel() for n, t in layer.p.items() if t is not None}
    layer.p["w1"].data = torch.empty(0, dtype=x.dtype, device=DEV)
    layer.p["w2"] = layer.p["w3"] = None
    torch.cuda.empty_cache()
    keep = [torch.full((n,), float("nan"), dtype=x.dtype, device=DEV) for n in sizes.values()]
    assert torch.equal(layer.forward(x), y)
    dx2, g2 = layer.backward(x, dy, taps, grads={"w_router": torch.empty_like(gr["w_router"])})
    assert torch.equal(dx2, dx) and torch.equal(g2["w_router"], gr["w_router"])
    assert all(torch.isnan(t).all() for t in keep)


@pytest.mark.parametrize("name,biases", [("switch_small", ("logit_bias",)), ("tiny", ("b_router",)),
                                         ("router_e20", ("b_router", "logit_bias")),
                                         ("mixtral_small", ())])
def test_every_parameter_is_trained(name, biases):
    """The optimizer over layer.parameters() moves all of them, the router's bias among them,
    under whichever name the layer has it."""
    layer, x, taps, dy = _forward(synth.SMALL[name], 3)
    params = layer.parameters()
    had = {n for n in layer.grad_shapes() if layer.p.get(n) is not None}
    assert set(params) == had | ({"b_router"} if biases else set())
    assert all(params[n] is layer.p[n] for n in had)
    assert tuple(n for n in ("b_router", "logit_bias") if layer.p.get(n) is not None) == biases
    old = {n: t.clone() for n, t in layer.p.items() if t is not None}
    _, gr = layer.backward(x, dy, taps)
    B.AdamW(params, lr=0.01, eps=1e-8, weight_decay=0.0).step(gr)
    for n, t in params.items():
        g = gr[n].double()
        if n == "b_router":
            # the first step: lr g / (|g| + eps)
            want = old[biases[0]].double() - 0.01 * g / (g.abs() + 1e-8)
            R.check(layer.p[biases[0]], want, 2.0 ** -20 * (want.abs() + 0.01), n)
            assert t is layer.p[biases[0]] and float(g.abs().max()) > 0
        else:
            assert not torch.equal(t, old[n]), n
    if biases == ("b_router", "logit_bias"):
        assert torch.equal(layer.p["logit_bias"], old["logit_bias"])


# ----------------------------------------------------------------------- experts
def test_output_biases_of_more_row_tiles_than_a_grid_dimension_holds():
    """bf16 MLP experts on 8.4 M rows: 65625 tiles of 128. dy holds small whole numbers, so
    that every partial sum of db2 is exact (below 2^24)."""
    rows, d, F, b = [3, 8_399_990, 7], 64, 64, torch.bfloat16
    n, E = sum(rows), len(rows)
    wl = _workload(n, d, E, 1, synth.DT_BF16, F=F, act=synth.ACT_RELU)
    g = _gen(3)
    p = {"w1": _rand(g, E, F, d, dt=b, std=1 / 8), "w2": _rand(g, E, d, F, dt=b, std=1 / 8),
         "b1": _rand(g, E, F, std=0.3), "b2": _rand(g, E, d, std=0.3)}
    layer = B.MoELayer(wl, p, DEV)
    x = torch.empty(n, d, dtype=b, device=DEV).normal_(generator=g)
    dy = torch.randint(-1, 2, (n, d), device=DEV, generator=g, dtype=torch.int8).to(b)
    off = torch.tensor([0, rows[0], rows[0] + rows[1], n], dtype=torch.int32, device=DEV)
    gr, dx = {m: layer.new_grads()[m] for m in ("b1", "b2")}, torch.empty_like(x)
    layer.expert_ffn_backward(x, off, dy, dx, gr)
    for e in range(E):
        want = dy[off[e]:off[e + 1]].sum(0, dtype=torch.int64)
        assert torch.equal(gr["b2"][e].double(), want.double())
    for e in (0, 2):  # the first and the last rows, by themselves
        r = slice(int(off[e]), int(off[e + 1]))
        ref, lim = R.ffn_bwd(x[r], dy[r], [0, rows[e]], {m: v[e:e + 1] for m, v in p.items()},
                             wl.act, b)
        R.check(dx[r], ref["dx"], lim["dx"], "dx")
        R.check(gr["b1"][e], ref["b1"][0], lim["b1"][0], "b1")
    assert layer.last_backward_error() == (0, 0)


def _fp32_tiles(d, F, rows):
    """(rows of a row tile, rows and columns of a tile of the weights' gradients) that the fp32
    experts' dispatch takes."""
    n, E = sum(rows), len(rows)
    tile = 8 if n <= 8 * E else (32 if n < 64 * E else 128)
    m = E * -(-F // 128)
    if tile == 128 and m * -(-d // 128) >= 296:
        return tile, (128, 128)
    return tile, ((128, 64) if m * -(-d // 64) >= 148 else (32, 64))


WIDE = [  # d, F, rows per expert, tiles: widths that end in either 64-column half of a tile
    (580, 1924, [70, 200, 130, 65], (128, (128, 128))), (580, 1923, [70, 200, 130, 65], (128, (128, 128))),
    (1220, 1137, [129, 1, 0, 300], (128, (128, 128))), (1028, 2500, [128, 190], (128, (128, 128))),
    (300, 1100, [70, 200, 130, 65], (128, (128, 64))), (300, 1101, [70, 200, 130, 65], (128, (128, 64))),
    (260, 520, [30] * 9 + [0, 64, 1, 33, 40, 32, 31], (32, (128, 64))),
    (260, 521, [30] * 9 + [0, 64, 1, 33, 40, 32, 31], (32, (128, 64))),
    (64, 193, [i % 5 for i in range(100)], (8, (128, 64))),
]


@pytest.mark.parametrize("act", G.ACTS, ids=["relu", "gelu", "swiglu"])
@pytest.mark.parametrize("d,F,rows,tiles", WIDE)
def test_fp32_experts_of_every_tile(d, F, rows, tiles, act):
    assert _fp32_tiles(d, F, rows) == tiles
    G.test_expert_ffn_backward(d, F, rows, act, synth.DT_F32)


@pytest.mark.parametrize("act", [synth.ACT_GELU, synth.ACT_SWIGLU], ids=["gelu", "swiglu"])
def test_fp32_layer_of_wide_experts(act):
    """The whole layer through the widest fp32 tiles, the shared experts' too."""
    T, d, E, k, F, Fs = 220, 1028, 4, 2, 1156, 2150
    assert _fp32_tiles(d, F, [T * k // E] * E)[1] == _fp32_tiles(d, 2 * Fs, [T])[1] == (128, 128)
    wl = _workload(T, d, E, k, synth.DT_F32, F=F, act=act, n_shared=2, d_ff_shared=Fs,
                   expert_bias=act == synth.ACT_GELU, bias_std=0.2, router_bias=True)
    layer, x, taps, dy = _forward(wl, 9)
    dl = torch.tensor([3.0, 0.2], device=DEV)
    dx, gr = layer.backward(x, dy, taps, d_losses=dl)
    ref, lim = R.layer_bwd(x, dy, taps, layer.p, wl, dl)
    for n, t in {"dx": dx, **gr}.items():
        R.check(t, ref[n], lim[n], n)
        R.check_norm(t, ref[n], torch.float32, n)
    assert layer.last_backward_error() == (0, 0)


@pytest.mark.parametrize("name", ["tiny", "mixtral_small", "deepseek_small", "switch_small", "fp32_gelu_cap"])
def test_layer_whose_capacity_drops_everything(name):
    """No expert has a row: their gradients are zero, x's is the losses' and the shared
    experts' (each token's gates have none)."""
    wl = synth.SMALL[name].replace(capacity_factor=1e-6)
    layer, x, taps, dy = _forward(wl, 4)
    assert (taps["inv"] == -1).all() and int(taps["offsets"][-1]) == 0
    for losses in (None, torch.tensor([3.0, 0.2], device=DEV)):
        layer.bws[64:].fill_(255)
        dx, gr = layer.backward(x, dy, taps, d_losses=losses)
        ref, lim = R.layer_bwd(x, dy, taps, layer.p, wl, losses)
        for n, t in {"dx": dx, **gr}.items():
            R.check(t, ref[n], lim[n], n)
        assert all((gr[n] == 0).all() for n in ("w1", "w3", "w2", "b1", "b2") if n in gr)
    assert layer.last_backward_error() == (0, 0)


@pytest.mark.parametrize("E,dt", [(8, synth.DT_BF16), (12, synth.DT_BF16), (100, synth.DT_BF16),
                                  (8, synth.DT_F32), (40, synth.DT_F32)])
def test_route_backward_keeps_infinities_to_their_column_and_token(E, dt):
    """An infinite weight or activation spoils its column of dx or dW (to infinity or NaN), a
    token without finite logits its row of dx; nothing else changes."""
    T, d, k = 300, 320, 2
    wl, layer, x, z, idx, counts, dg, _ = G._route_case(T, d, E, k, dt, 0, 5)
    full = lambda z: (torch.empty_like(z), torch.empty(T, d, device=DEV), layer.new_grads())  # noqa: E731
    dz, dx, gr = full(z)
    layer.route_backward(x, z, idx, None, dg, None, dz, dx, gr)
    x2 = x.clone()
    x2[7, 33] = float("inf")
    layer.p["w_router"][E - 1, 100] = float("-inf")
    dz2, dx2, g2 = full(z)
    layer.route_backward(x2, z, idx, None, dg, None, dz2, dx2, g2)
    cols = torch.arange(d, device=DEV)
    assert torch.equal(dz2, dz) and torch.equal(g2["b_router"], gr["b_router"])
    assert torch.equal(dx2[:, cols != 100], dx[:, cols != 100])
    assert torch.equal(g2["w_router"][:, cols != 33], gr["w_router"][:, cols != 33])
    hit = idx[7].long()                       # the experts that token chose
    assert not torch.isfinite(g2["w_router"][hit, 33].float()).any()
    assert not torch.isfinite(dx2[(idx == E - 1).any(1), 100]).any()
    layer.p["w_router"][E - 1, 100] = 0.25
    z2 = z.clone()
    z2[9, idx[9, 0].long()] = float("nan")
    dz, dx, gr = full(z)
    layer.route_backward(x, z, idx, None, dg, None, dz, dx, gr)
    dz2, dx2, g2 = full(z)
    layer.route_backward(x, z2, idx, None, dg, None, dz2, dx2, g2)
    rows = torch.arange(T, device=DEV) != 9
    assert torch.equal(dz2[rows], dz[rows]) and torch.equal(dx2[rows], dx[rows])
    assert torch.isnan(dx2[9]).all()
    assert layer.last_backward_error() == (0, 0)


# A running fp32 sum of n products of random sign is off by about U sqrt(n / 6) of its result
# (each rounding at most U of a partial sum whose size grows with the root of its length). The
# weights' gradients are sums of at most 1024, and of these parts.
def _sums(n, *others):
    return 2.0 ** -24 * (sum((m / 6) ** 0.5 for m in (min(n, 1024), n / 1024, *others)) + 8)


def test_fp32_weight_gradients_over_many_rows():
    n, d, F = 32768, 64, 64
    wl, layer, x, dy, off, n = G._ffn_case(d, F, [n, 5], synth.ACT_GELU, synth.DT_F32, 1)
    gr = layer.new_grads()
    layer.expert_ffn_backward(x, off, dy, None, gr)
    ref, _ = R.ffn_bwd(x, dy, off.tolist(), layer.p, wl.act, torch.float32)
    for m in ("w1", "w2"):  # the activations behind them are sums over d
        off_by = float((gr[m][0].double() - ref[m][0]).norm() / ref[m][0].norm())
        assert off_by <= _sums(n, d, d), f"{m}: {off_by:.2e}"


def test_fp32_router_gradient_over_many_tokens():
    T, d, E, k = 65536, 4096, 20, 2
    wl, layer, x, z, idx, counts, dg, _ = G._route_case(T, d, E, k, synth.DT_F32, 2, 3)
    dz, gr = torch.empty_like(z), layer.new_grads()
    layer.route_backward(x, z, idx, None, dg, None, dz, None, gr)
    ref = dz.double().T @ x.double()
    off_by = float((gr["w_router"].double() - ref).norm() / ref.norm())
    assert off_by <= _sums(T // 4, 4), f"{off_by:.2e}"
