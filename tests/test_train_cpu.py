"""The training step without a GPU: the 64-bit reference formulas against automatic
differentiation and against differences of the oracle's forward pass, the refusals of
the C entry points, struct layouts, and the binding's checks."""
import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_mixture_experts_12_b200 import binding as B
from sparse_mixture_experts_12_b200 import build as BUILD
from sparse_mixture_experts_12_b200 import synth
from tests import train_ref as R
from tests.gpu_harness import oracle_kwargs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

TINY = {
    "relu_top2": synth.TINY_FP32.replace(name="t", T=13, d_model=8, n_experts=4, d_ff=12,
                                         bias_std=0.3),
    "swiglu_raw_shared": synth.DEEPSEEK_FINE.replace(name="t", T=11, d_model=8, n_experts=5,
                                                     top_k=3, d_ff=6, n_shared=2, d_ff_shared=4,
                                                     dtype=synth.DT_F32, router_std=0.4,
                                                     gate_mode=synth.GATE_SOFTMAX_TOPK_RAW),
    "gelu_cap_renorm": synth.SWITCH_CAPACITY.replace(name="t", T=17, d_model=8, n_experts=4,
                                                     top_k=2, d_ff=12, dtype=synth.DT_F32,
                                                     router_std=0.4, bias_std=0.3,
                                                     capacity_factor=0.7, router_bias=True,
                                                     gate_mode=synth.GATE_SOFTMAX_TOPK_RENORM),
}


def _routed(wl, seed):
    inp = synth.generate(wl, seed=seed)
    p = {k: (None if v is None else v.double().numpy()) for k, v in inp.items()}
    r = O.route(p["x"], p, top_k=wl.top_k, gate_mode=oracle_kwargs(wl)["gate_mode"],
                capacity_factor=wl.capacity_factor)
    taps = {"logits": torch.tensor(r["logits"]), "topk_idx": torch.tensor(r["idx"]).int(),
            "topk_gate": torch.tensor(np.asarray(r["gates"], dtype=np.float64)),
            "counts": torch.tensor(r["counts"]).int(), "offsets": torch.tensor(r["offsets"]).int(),
            "inv": torch.tensor(r["inv"]).int().reshape(-1)}
    return inp, p, r, taps


@pytest.mark.parametrize("name", sorted(TINY))
def test_reference_against_differences_of_the_oracle(name):
    """d<dy, y> + c0 d aux + c1 d z_loss along random directions of x and of every
    parameter, by central differences of the oracle's forward pass with the routing of
    the base point (the selection has no gradient); step 1e-5 in 64 bits: the differences
    are good to about 1e-9 of the values' sizes. The oracle takes its logits in fp32, so
    the layer is put together from its parts here, in 64 bits."""
    wl = TINY[name]
    inp, p, r, taps = _routed(wl, seed=3)
    g = np.random.default_rng(7)
    dy = g.standard_normal(p["x"].shape)
    c = np.array([3.0, 0.2])
    act = oracle_kwargs(wl)["act"]
    T, E, k = wl.T, wl.n_experts, wl.top_k
    idx, inv = np.asarray(r["idx"]), np.asarray(r["inv"]).reshape(T, k)

    def value(q):
        z = q["x"] @ q["w_router"].T
        for b in ("b_router", "logit_bias"):
            if q.get(b) is not None:
                z = z + q[b]
        pr = O.softmax(z)
        gates = np.take_along_axis(pr, idx, 1)
        if wl.gate_mode != synth.GATE_SOFTMAX_TOPK_RAW:
            gates = gates / gates.sum(1, keepdims=True)
        y = np.zeros_like(q["x"])
        if wl.n_shared:
            y += O.shared_experts(q["x"], q["ws_gate"], q["ws_up"], q["ws_down"], wl.n_shared)
        for e in range(E):
            for s in range(k):
                m = (idx[:, s] == e) & (inv[:, s] >= 0)
                if m.any():
                    o = O.expert_ffn(q["x"][m], act, q["w1"][e], q["w2"][e],
                                     None if q["w3"] is None else q["w3"][e],
                                     None if q["b1"] is None else q["b1"][e],
                                     None if q["b2"] is None else q["b2"][e])
                    y[m] += gates[m, s][:, None] * o
        f = np.asarray(r["counts"]) / (T * k)
        aux = wl.aux_alpha * E * (f * pr.mean(0)).sum()
        mx = z.max(1)
        lse = mx + np.log(np.exp(z - mx[:, None]).sum(1))
        return (y * dy).sum() + c[0] * aux + c[1] * (lse ** 2).mean()

    # the reference at the same (64-bit) logits and gates
    z = p["x"] @ p["w_router"].T
    for b in ("b_router", "logit_bias"):
        if p.get(b) is not None:
            z = z + p[b]
    pr = O.softmax(z)
    gates = np.take_along_axis(pr, idx, 1)
    if wl.gate_mode != synth.GATE_SOFTMAX_TOPK_RAW:
        gates = gates / gates.sum(1, keepdims=True)
    taps["logits"], taps["topk_gate"] = torch.tensor(z), torch.tensor(gates)
    t64 = {n: (None if v is None else torch.tensor(v)) for n, v in p.items()}
    out, _ = R.layer_bwd(t64["x"], torch.tensor(dy), taps, t64, wl, torch.tensor(c))
    for n in ["x"] + [n for n in out if n != "dx"]:
        grad = out["dx" if n == "x" else n].numpy()
        key = "logit_bias" if n == "b_router" and p.get("b_router") is None else n
        if p.get(key) is None:
            continue
        for _ in range(2):
            v = g.standard_normal(p[key].shape)
            h = 1e-5
            up, dn = dict(p), dict(p)
            up[key], dn[key] = p[key] + h * v, p[key] - h * v
            num = (value(up) - value(dn)) / (2 * h)
            assert abs(num - (grad * v).sum()) <= 2e-6 * (1 + np.abs(grad * v).sum()), (n, num)


def test_adamw_reference_against_torch():
    g = torch.Generator().manual_seed(0)
    p = torch.randn(50, dtype=torch.float64, generator=g)
    q = p.clone().requires_grad_(True)
    opt = torch.optim.AdamW([q], lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    for t in range(1, 5):
        gr = torch.randn(50, dtype=torch.float64, generator=g)
        q.grad = gr.clone()
        opt.step()
        p, m, v = R.adamw(p, gr, m, v, t, 0.01, 0.8, 0.95, 1e-6, 0.1)
        assert torch.allclose(p, q.detach(), rtol=1e-12, atol=1e-14)


# ------------------------------------------------------------------ the C entry points
@pytest.fixture(scope="module")
def lib():
    BUILD.build()
    return B.load()


WS, GOOD, ODD = (ctypes.c_void_p(a) for a in (0x100000, 0x200000, 0x200008))


def _bytes(cfg):
    return B.backward_workspace_size(cfg)


def test_struct_layouts_match_the_header(tmp_path):
    prog = tmp_path / "layout.c"
    structs = (("moe_grads_t", B.MoeGrads), ("moe_adamw_tensor_t", B.MoeAdamWTensor),
               ("moe_adamw_t", B.MoeAdamW))
    prog.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "moe.h"\nint main(void) {\n'
                    + "".join(f'  printf("%zu ", offsetof({s}, {n}));\n'
                              for s, c in structs for n, _ in c._fields_)
                    + "".join(f'  printf("%zu ", sizeof({s}));\n' for s, _ in structs)
                    + '  printf("%d", MOE_ADAMW_BLOCK);\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", f"-I{os.path.join(ROOT, 'include')}", str(prog), "-o",
                    str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = [getattr(c, n).offset for _, c in structs for n, _ in c._fields_]
    want += [ctypes.sizeof(c) for _, c in structs] + [B.ADAMW_BLOCK]
    assert got == want


def test_backward_workspace_follows_the_layer(lib):
    small, big = synth.SMALL["mixtral_small"], synth.MIXTRAL_PREFILL
    assert 0 < _bytes(B.make_cfg(small)) < _bytes(B.make_cfg(big))
    ds = synth.SMALL["deepseek_small"]
    assert _bytes(B.make_cfg(ds)) > _bytes(B.make_cfg(ds, n_shared=0, d_ff_shared=0))
    assert _bytes(B.make_cfg(small, n_tokens=0)) > 0
    n = ctypes.c_size_t(0)
    assert lib.moe_backward_workspace_size(None, ctypes.byref(n)) == 1
    assert lib.moe_backward_workspace_size(ctypes.byref(B.make_cfg(small)), None) == 1
    # rows of h, da, du, x, dy and dx, and no more than 256 MB for the parts of dx
    wide = B.make_cfg(synth.SMALL["fp32_swiglu"], n_tokens=30000, d_model=1024, d_ff=8192)
    R = 30000 * wide.top_k
    assert _bytes(wide) < 4 * R * (3 * 8192 + 4 * 1024 + 8192 // 32 + 8) + (300 << 20)
    # the forward's own workspace did not grow for it
    R, F, d, T = small.T * 2, small.d_ff, small.d_model, small.T
    assert B.workspace_size(B.make_cfg(small)) < 2 * R * (F + 2 * d) + 40 * T * 64 + 65536


def test_token_gradients_refuse_before_launching(lib):
    cfg = B.make_cfg(synth.SMALL["mixtral_small"])
    n, c = _bytes(cfg), ctypes.byref(cfg)
    f = lib.moe_combine_backward
    assert f(c, None, GOOD, GOOD, GOOD, GOOD, GOOD, WS, n, None) == 1   # dy missing
    assert f(c, GOOD, None, GOOD, GOOD, GOOD, GOOD, WS, n, None) == 1   # dgate needs y_perm
    assert f(c, GOOD, GOOD, GOOD, None, GOOD, GOOD, WS, n, None) == 1   # dy_perm needs gates
    assert f(c, GOOD, GOOD, None, GOOD, GOOD, GOOD, WS, n, None) == 1
    assert f(c, ODD, GOOD, GOOD, GOOD, GOOD, GOOD, WS, n, None) == 3
    assert f(c, GOOD, GOOD, GOOD, GOOD, ODD, GOOD, WS, n, None) == 3
    assert f(c, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, WS, n - 1, None) == 4
    assert f(c, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, None, n, None) == 1
    assert f(c, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, ctypes.c_void_p(0x100010), n, None) == 3
    f = lib.moe_permute_backward
    assert f(c, None, GOOD, None, GOOD, WS, n, None) == 1
    assert f(c, GOOD, GOOD, ODD, GOOD, WS, n, None) == 3
    assert f(c, GOOD, GOOD, None, None, WS, n, None) == 1
    assert f(c, GOOD, GOOD, None, GOOD, WS, n - 1, None) == 4
    # no tokens: nothing to do, nothing launched
    z = B.make_cfg(synth.SMALL["mixtral_small"], n_tokens=0)
    assert lib.moe_combine_backward(ctypes.byref(z), None, None, None, None, None, None, WS,
                                    _bytes(z), None) == 0


def test_expert_choice_has_no_token_gradients(lib):
    cfg = B.make_cfg(synth.SMALL["ec_small"])
    n, c = _bytes(cfg), ctypes.byref(cfg)
    W, tp = B.MoeWeights(w_router=GOOD, w1=GOOD, w3=GOOD, w2=GOOD), B.MoeTaps()
    assert lib.moe_combine_backward(c, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, WS, n, None) == 1
    assert lib.moe_permute_backward(c, GOOD, GOOD, None, GOOD, WS, n, None) == 1
    assert lib.moe_route_backward(c, ctypes.byref(W), GOOD, GOOD, GOOD, None, GOOD, None, GOOD,
                                  GOOD, None, WS, n, None) == 1
    assert lib.moe_backward(c, ctypes.byref(W), GOOD, ctypes.byref(tp), GOOD, None, GOOD, None,
                            WS, n, None) == 1


def test_route_and_expert_gradients_refuse_before_launching(lib):
    cfg = B.make_cfg(synth.SMALL["mixtral_small"])
    n, c = _bytes(cfg), ctypes.byref(cfg)
    W = B.MoeWeights(w_router=GOOD, w1=GOOD, w3=GOOD, w2=GOOD)
    G = B.MoeGrads(w_router=GOOD)
    f = lib.moe_route_backward
    assert f(c, ctypes.byref(W), None, GOOD, GOOD, None, GOOD, None, GOOD, None, ctypes.byref(G),
             WS, n, None) == 1                       # w_router's gradient needs x
    assert f(c, ctypes.byref(W), GOOD, None, GOOD, None, GOOD, None, GOOD, None, None, WS, n,
             None) == 1                              # logits missing
    assert f(c, ctypes.byref(W), GOOD, GOOD, GOOD, None, GOOD, GOOD, GOOD, None, None, WS, n,
             None) == 1                              # the losses need counts
    assert f(c, None, GOOD, GOOD, GOOD, None, GOOD, None, GOOD, GOOD, None, WS, n, None) == 1
    assert f(c, ctypes.byref(B.MoeWeights()), GOOD, GOOD, GOOD, None, GOOD, None, GOOD, GOOD,
             None, WS, n, None) == 1                 # dx needs w_router
    assert f(c, ctypes.byref(W), GOOD, GOOD, ODD, None, GOOD, None, GOOD, GOOD, None, WS, n,
             None) == 3
    f = lib.moe_expert_ffn_backward
    args = lambda w=W, x=GOOD, o=GOOD, dy=GOOD, dx=GOOD, g=None, k=n: f(  # noqa: E731
        c, ctypes.byref(w), x, o, dy, dx, None if g is None else ctypes.byref(g), WS, k, None)
    assert args(x=None) == 1 and args(o=None) == 1 and args(dy=None) == 1
    assert args(dx=ODD) == 3 and args(k=n - 1) == 4
    assert args(w=B.MoeWeights(w1=GOOD, w2=GOOD)) == 1               # no w_up
    assert args(g=B.MoeGrads(b1=GOOD)) == 1                          # SwiGLU has no bias
    assert args(g=B.MoeGrads(w1=ODD)) == 3
    mlp = B.make_cfg(synth.SMALL["switch_small"])
    assert f(ctypes.byref(mlp), ctypes.byref(B.MoeWeights(w1=GOOD, w2=GOOD)), GOOD, GOOD, GOOD,
             GOOD, ctypes.byref(B.MoeGrads(w3=GOOD)), WS, _bytes(mlp), None) == 1
    assert f(ctypes.byref(mlp), ctypes.byref(B.MoeWeights(w1=GOOD, w2=GOOD)), GOOD, GOOD, GOOD,
             GOOD, ctypes.byref(B.MoeGrads(b2=GOOD)), WS, _bytes(mlp), None) == 1
    f = lib.moe_backward
    full = dict(logits=GOOD, topk_idx=GOOD, topk_gate=GOOD, offsets=GOOD, inv=GOOD)
    for missing in full:
        tp = B.MoeTaps(**{k: v for k, v in full.items() if k != missing})
        assert f(c, ctypes.byref(W), GOOD, ctypes.byref(tp), GOOD, None, GOOD, None, WS, n,
                 None) == 1, missing
    tp = B.MoeTaps(**full)
    assert f(c, ctypes.byref(W), GOOD, None, GOOD, None, GOOD, None, WS, n, None) == 1
    assert f(c, ctypes.byref(W), GOOD, ctypes.byref(tp), GOOD, GOOD, GOOD, None, WS, n, None) == 1
    assert f(c, ctypes.byref(W), GOOD, ctypes.byref(tp), GOOD, None, GOOD,
             ctypes.byref(B.MoeGrads(ws_gate=GOOD)), WS, n, None) == 1   # no shared experts
    assert f(c, ctypes.byref(W), GOOD, ctypes.byref(tp), None, None, GOOD, None, WS, n, None) == 1


def _adam(lib, t=None, o=None, n=1):
    tensor = dict(n=4, param=GOOD, grad=GOOD, exp_avg=GOOD, exp_avg_sq=GOOD, param_dtype=1,
                  grad_dtype=1, state_bits=32)
    opt = dict(beta1=0.9, beta2=0.99, lr=1e-3, eps=1e-8, weight_decay=0.1, step=1)
    tensor.update(t or {})
    opt.update(o or {})
    for k, v in tensor.items():
        tensor[k] = v.value if isinstance(v, ctypes.c_void_p) else v
    for k, v in opt.items():
        opt[k] = v.value if isinstance(v, ctypes.c_void_p) else v
    arr = (B.MoeAdamWTensor * 1)(B.MoeAdamWTensor(**tensor))
    return lib.moe_adamw_step(arr, n, ctypes.byref(B.MoeAdamW(**opt)), None)


@pytest.mark.parametrize("t,o,expect", [
    ({"n": -1}, {}, 1), ({"param": None}, {}, 1), ({"grad": None}, {}, 1),
    ({"exp_avg": None}, {}, 1), ({"exp_avg_sq": None}, {}, 1), ({"param": ODD}, {}, 3),
    ({"param_dtype": 2}, {}, 1), ({"grad_dtype": -1}, {}, 1), ({"state_bits": 16}, {}, 1),
    ({"state_bits": 8}, {}, 1), ({"state_bits": 8, "exp_avg_scale": GOOD}, {}, 1),
    ({"exp_avg_scale": GOOD}, {}, 1), ({"param_dtype": 0, "master": GOOD}, {}, 1),
    ({"master": ODD}, {}, 3),
    ({}, {"beta1": 1.0}, 1), ({}, {"beta2": -0.1}, 1), ({}, {"beta1": float("nan")}, 1),
    ({}, {"eps": -1e-8}, 1), ({}, {"lr": float("inf")}, 1), ({}, {"step": 0}, 1),
    ({}, {"weight_decay": float("nan")}, 1), ({}, {"step_dev": ctypes.c_void_p(0x200004)}, 3),
    ({}, {"grad_scale": ctypes.c_void_p(0x200002)}, 3), ({"n": 1 << 43}, {}, 2),
])
def test_adamw_refuses_before_launching(lib, t, o, expect):
    assert _adam(lib, t, o) == expect


@pytest.mark.parametrize("n", [1 << 42, (1 << 42) - 2047, (1 << 62) + 5])
def test_adamw_refuses_a_tensor_of_more_blocks_than_a_grid_holds(n):
    """2048 elements a block, 2^31 - 1 blocks: one element more is refused (in a process of its
    own, which an endless loop on the host would not hold up for good)."""
    prog = ("import ctypes; from sparse_mixture_experts_12_b200 import binding as B; "
            f"t = (B.MoeAdamWTensor * 1)(B.MoeAdamWTensor(n={n}, param=4096, grad=4096, "
            "exp_avg=4096, exp_avg_sq=4096, param_dtype=1, grad_dtype=1, state_bits=32)); "
            "o = B.MoeAdamW(beta1=0.9, beta2=0.9, step=1); "
            "print(B.load().moe_adamw_step(t, 1, ctypes.byref(o), None))")
    r = subprocess.run([sys.executable, "-c", prog], cwd=ROOT, capture_output=True, text=True,
                       timeout=120)
    assert r.stdout.strip() == "2", r.stderr


def test_adamw_with_nothing_to_do(lib):
    assert _adam(lib, {"n": 0, "param": None, "grad": None, "exp_avg": None,
                       "exp_avg_sq": None}) == 0
    assert lib.moe_adamw_step(None, 0, ctypes.byref(B.MoeAdamW(beta1=0.9, beta2=0.9, step=1)),
                              None) == 0
    assert lib.moe_adamw_step(None, 1, ctypes.byref(B.MoeAdamW(beta1=0.9, beta2=0.9, step=1)),
                              None) == 1
    assert lib.moe_adamw_step(None, 0, None, None) == 1


def test_binding_checks_tensors():
    cpu = torch.device("cpu")
    x = torch.zeros(4, 6)
    B.check_tensor(x, (4, 6), torch.float32, "x", cpu)
    B.check_tensor(None, (4, 6), torch.float32, "x", cpu, optional=True)
    for bad, shape, dt, dev in ((None, (4, 6), torch.float32, cpu), (x, (6, 4), torch.float32, cpu),
                                (x, (4, 6), torch.bfloat16, cpu),
                                (x.t(), (6, 4), torch.float32, cpu),
                                (x, (4, 6), torch.float32, torch.device("cuda", 0))):
        with pytest.raises(ValueError):
            B.check_tensor(bad, shape, dt, "x", dev)
    with pytest.raises(ValueError):
        B.AdamW([])
    with pytest.raises(ValueError):
        B.AdamW([x])


def test_errors_are_read_on_the_layers_own_device(monkeypatch):
    """The gradients run on the layer's device whichever is current; their errors are read
    there too, on that device's stream."""
    layer, seen = object.__new__(B.MoELayer), []

    class Lib:
        @staticmethod
        def moe_last_device_error(ws, code, info, stream):
            seen.append(stream)
            code._obj.value, info._obj.value = 2, 5
            return 6

    layer.lib, layer._index = Lib, 3
    layer.ws = layer._bws = torch.zeros(64, dtype=torch.uint8)
    monkeypatch.setattr(B, "_on_device", lambda index, call, *a: call(*a, ("stream of", index)))
    assert layer.last_backward_error() == layer.last_device_error() == (2, 5)
    assert seen == [("stream of", 3)] * 2


def _kernels_launched_ahead():
    """(name, body before the first wait) of every kernel that calls pdl_wait()."""
    csrc = os.path.join(ROOT, "sparse_mixture_experts_12_b200", "csrc")
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__.*?\bvoid\b.*?(k_\w+)\(", text, re.S):
            end = text.find("\n}\n", m.end())
            body = text[m.end():end]
            if "pdl_wait()" in body:
                yield f"{name}:{m.group(1)}", body[:body.index("pdl_wait()")]


def test_no_kernel_reads_a_bias_before_its_wait():
    """An optimizer step writes the biases and may stand directly ahead of a forward pass:
    their loads come after the wait for the kernel ahead. (The expert GEMMs read their
    weights before it, from behind a kernel of the same call that has waited.)"""
    seen = dict(_kernels_launched_ahead())
    assert len(seen) > 20 and "route_tc.cu:k_router_tc" in seen
    early = [k for k, body in seen.items()
             if re.search(r"\b(b_router|logit_bias|b1|b2|bias)\s*\[", body)]
    assert early == []
