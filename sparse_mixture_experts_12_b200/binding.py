"""Thin ctypes binding over ``libmoe.so`` (argument marshalling only).

Every step of the layer runs in the library's CUDA kernels; PyTorch only
provides device memory and the current stream. There is no fallback: if the
library is missing or no CUDA device is present, the calls raise.

Function names follow the C ABI in ``include/moe.h``.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import numpy as np
import torch

from . import synth

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")
_lib = None

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
                3: "MOE_ERR_MISALIGNED", 4: "MOE_ERR_WORKSPACE", 5: "MOE_ERR_CUDA",
                6: "MOE_ERR_DEVICE"}
DEVERR_NAMES = {0: "none", 1: "expert index out of range", 2: "invalid offsets",
                3: "row index out of range", 4: "pipeline wait timeout"}

EXPORTED = ("moe_workspace_size", "moe_workspace_init", "moe_route", "moe_route_noisy",
            "moe_route_expert_choice", "moe_permute", "moe_permute_noalloc", "moe_forward_noisy",
            "moe_expert_ffn", "moe_combine", "moe_aux_stats", "moe_forward",
            "moe_route_shard", "moe_permute_shard", "moe_forward_shard", "moe_aux_finalize",
            "moe_forward_staged", "moe_noise_draws", "moe_route_noisy_seeded",
            "moe_forward_noisy_seeded", "moe_backward_workspace_size", "moe_combine_backward",
            "moe_permute_backward", "moe_route_backward", "moe_expert_ffn_backward",
            "moe_backward", "moe_adamw_step", "moe_test_set_wait_limit", "moe_test_withhold_load",
            "moe_last_device_error", "moe_status_string")

ADAMW_BLOCK = 256  # MOE_ADAMW_BLOCK: elements that share a scale of an 8-bit state
_ADAMW_DTYPES = {torch.float32: synth.DT_F32, torch.bfloat16: synth.DT_BF16}

# stages of one layer call (MOE_STAGE_*), in launch order
STAGES = ("route", "scan", "permute", "shared_ffn", "expert_ffn", "combine")


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class MoeCfg(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("d_ff", ctypes.c_int32), ("act", ctypes.c_int32),
                ("gate_mode", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("capacity_factor", ctypes.c_float), ("aux_alpha", ctypes.c_float),
                ("n_shared", ctypes.c_int32), ("d_ff_shared", ctypes.c_int32),
                ("routing", ctypes.c_int32)]


class MoeWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("w_router", "b_router", "logit_bias", "w1", "w3", "w2", "b1", "b2",
                 "ws_gate", "ws_up", "ws_down", "w_noise")]


class MoeTaps(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("logits", "topk_idx", "topk_gate", "counts", "offsets", "perm", "inv")]


class MoeShard(ctypes.Structure):
    _fields_ = [("n_tokens_total", ctypes.c_longlong), ("n_shards", ctypes.c_int32),
                ("shard", ctypes.c_int32), ("counts_all", ctypes.c_void_p)]


class MoeStageEvents(ctypes.Structure):
    _fields_ = [("ev", ctypes.c_void_p * (len(STAGES) + 1))]


class MoeGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("w_router", "b_router", "w1", "w3", "w2", "b1", "b2", "ws_gate", "ws_up",
                 "ws_down")]


class MoeAdamWTensor(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64)] + [(n, ctypes.c_void_p) for n in
                ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale",
                 "master")] + [(n, ctypes.c_int32) for n in
                               ("param_dtype", "grad_dtype", "state_bits")]


class MoeAdamW(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("lr", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("step", ctypes.c_int64), ("step_dev", ctypes.c_void_p),
                ("lr_dev", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p),
                ("found_inf", ctypes.c_void_p)]


class MoeNoise(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_void_p), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64)]


def lib_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                           "`python -m sparse_mixture_experts_12_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, S = ctypes.c_void_p, ctypes.c_size_t
    cfgp, wp = ctypes.POINTER(MoeCfg), ctypes.POINTER(MoeWeights)
    sig = {
        "moe_workspace_size": [cfgp, ctypes.POINTER(ctypes.c_size_t)],
        "moe_workspace_init": [P, S, P],
        "moe_route": [cfgp, wp, P, P, P, P, P, S, P],
        "moe_permute": [cfgp, P, P, P, P, P, P, P, P, S, P],
        "moe_permute_noalloc": [cfgp, P, P, P, P, P, P, P, P],
        "moe_expert_ffn": [cfgp, wp, P, P, P, P, S, P],
        "moe_combine": [cfgp, P, P, P, P, P, P, S, P],
        "moe_aux_stats": [cfgp, P, P, P, P, S, P],
        "moe_forward": [cfgp, wp, P, P, P, ctypes.POINTER(MoeTaps), P, S, P],
        "moe_route_shard": [cfgp, wp, P, P, P, P, P, P, P, S, P],
        "moe_permute_shard": [cfgp, ctypes.POINTER(MoeShard), P, P, P, P, P, P, P, P, S, P],
        "moe_forward_shard": [cfgp, ctypes.POINTER(MoeShard), wp, P, ctypes.POINTER(MoeTaps), P,
                              P, S, P],
        "moe_aux_finalize": [cfgp, ctypes.c_longlong, P, P, P],
        "moe_forward_staged": [cfgp, wp, P, ctypes.POINTER(MoeNoise), P, P,
                               ctypes.POINTER(MoeTaps), ctypes.POINTER(MoeStageEvents), P, S,
                               P],
        "moe_noise_draws": [ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64, ctypes.c_uint64, P,
                            P, P],
        "moe_route_noisy_seeded": [cfgp, wp, P, ctypes.c_uint64, ctypes.c_uint64, P, P, P, P, S,
                                   P],
        "moe_forward_noisy_seeded": [cfgp, wp, P, ctypes.c_uint64, ctypes.c_uint64, P, P,
                                     ctypes.POINTER(MoeTaps), P, S, P],
        "moe_backward_workspace_size": [cfgp, ctypes.POINTER(ctypes.c_size_t)],
        "moe_combine_backward": [cfgp, P, P, P, P, P, P, P, S, P],
        "moe_permute_backward": [cfgp, P, P, P, P, P, S, P],
        "moe_route_backward": [cfgp, wp, P, P, P, P, P, P, P, P, ctypes.POINTER(MoeGrads), P, S,
                               P],
        "moe_expert_ffn_backward": [cfgp, wp, P, P, P, P, ctypes.POINTER(MoeGrads), P, S, P],
        "moe_backward": [cfgp, wp, P, ctypes.POINTER(MoeTaps), P, P, P,
                         ctypes.POINTER(MoeGrads), P, S, P],
        "moe_adamw_step": [ctypes.POINTER(MoeAdamWTensor), ctypes.c_int32,
                           ctypes.POINTER(MoeAdamW), P],
        "moe_test_set_wait_limit": [ctypes.c_uint64],
        "moe_test_withhold_load": [ctypes.c_int32],
        "moe_last_device_error": [P, ctypes.POINTER(ctypes.c_int32),
                                  ctypes.POINTER(ctypes.c_int32), P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def expert_rows(cfg: MoeCfg) -> int:
    """Rows of the expert-contiguous buffers (x_perm, y_perm) the library reads and
    writes for this configuration: T * k under token choice, E * C with
    C = floor(cf * T / E) under expert choice (evaluated in double, as the library
    does)."""
    if cfg.routing == synth.ROUTING_EXPERT_CHOICE:
        if not cfg.capacity_factor > 0:
            return 0
        return cfg.n_experts * math.floor(float(cfg.capacity_factor) * cfg.n_tokens /
                                          cfg.n_experts)
    return cfg.n_tokens * cfg.top_k


def check_rows(t: Optional[torch.Tensor], rows: int, cols: int, name: str):
    """The C ABI takes raw pointers and cannot see a buffer's size: a tensor with
    fewer than the `rows` rows of `cols` elements that the library will access is
    refused here, before anything is launched."""
    if t is None:
        return
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] != cols or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [>= {rows}, {cols}] tensor, "
                         f"not {tuple(t.shape)}")


def check_tensor(t: Optional[torch.Tensor], shape, dtype: torch.dtype, name: str, device,
                 optional: bool = False):
    """A tensor handed to the training entry points: contiguous, of this shape and dtype,
    on `device` (the C ABI sees none of these)."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is missing")
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor, not "
                         f"{tuple(t.shape)} {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _on_device(index: int, call, *args):
    """call(*args, stream) with device `index` current and its current stream."""
    if torch._C._cuda_getDevice() == index:
        return call(*args, torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(index):
        return call(*args, torch._C._cuda_getCurrentRawStream(index))


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _taps(taps: Optional[dict]):
    if taps is None:
        return None
    return MoeTaps(**{k: _ptr(taps.get(k)) for k, _ in MoeTaps._fields_})


def stage_events(events) -> MoeStageEvents:
    """MoeStageEvents from len(STAGES) + 1 torch.cuda.Event (None entries allowed)."""
    if len(events) != len(STAGES) + 1:
        raise ValueError(f"{len(STAGES) + 1} events expected, got {len(events)}")
    ev = MoeStageEvents()
    for i, e in enumerate(events):
        if e is not None and not e.cuda_event:
            raise ValueError("a torch.cuda.Event has no CUDA event until its first record()")
        ev.ev[i] = None if e is None else e.cuda_event
    return ev


def make_cfg(w: synth.Workload, **over) -> MoeCfg:
    c = MoeCfg(n_tokens=w.T, d_model=w.d_model, n_experts=w.n_experts, top_k=w.top_k,
               d_ff=w.d_ff, act=w.act, gate_mode=w.gate_mode, dtype=w.dtype,
               capacity_factor=w.capacity_factor, aux_alpha=w.aux_alpha,
               n_shared=w.n_shared, d_ff_shared=w.d_ff_shared, routing=w.routing)
    for k, v in over.items():
        setattr(c, k, v)
    return c


def workspace_size(cfg: MoeCfg) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def backward_workspace_size(cfg: MoeCfg) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_backward_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "moe_backward_workspace_size")
    return n.value


def new_workspace(cfg: MoeCfg, device="cuda", backward: bool = False) -> torch.Tensor:
    """A prepared workspace of the forward entry points, or (backward) of the gradients'."""
    nbytes = backward_workspace_size(cfg) if backward else workspace_size(cfg)
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + nbytes]
    _check(load().moe_workspace_init(_ptr(ws), nbytes, _stream()), "moe_workspace_init")
    return ws


class MoELayer:
    """One MoE FFN layer whose weights live on the GPU.

    ``params`` is the dict of ``synth.generate`` (CPU or CUDA tensors); they are
    moved to ``device`` once. ``forward`` runs the whole layer through
    ``moe_forward`` on the current stream. The layer works on the storage that the tensors
    of ``p`` have then: new values are written into them (``copy_``, an optimizer step).
    """

    def __init__(self, workload: synth.Workload, params: dict, device="cuda"):
        self.w = workload
        self.cfg = make_cfg(workload)
        self.device = torch.device(device)
        self.p = {k: (None if v is None else v.to(self.device).contiguous())
                  for k, v in params.items() if k != "x"}
        self.weights = MoeWeights(**{k: _ptr(self.p.get(k)) for k, _ in MoeWeights._fields_})
        # what these addresses point to, whatever becomes of the entries of p
        self._held = [v.detach() for v in self.p.values() if v is not None]
        self.ws = new_workspace(self.cfg, self.device)
        self.lib = load()
        self._bws = None
        self._index, self._dtype = self.ws.get_device(), workload.torch_dtype

    # -------------------------------------------------------------- whole layer
    def forward(self, x: torch.Tensor, y: Optional[torch.Tensor] = None,
                aux: Optional[torch.Tensor] = None, taps: Optional[dict] = None,
                events: Optional[list] = None) -> torch.Tensor:
        """The whole layer (moe_forward). ``events``: len(STAGES) + 1 torch.cuda.Event
        objects recorded at the stage boundaries (moe_forward_staged)."""
        if y is None:
            y = torch.empty_like(x)
        tp = _taps(taps)
        tpr = ctypes.byref(tp) if tp is not None else None
        if events is None:
            _check(self.lib.moe_forward(ctypes.byref(self.cfg), ctypes.byref(self.weights),
                                        _ptr(x), _ptr(y), _ptr(aux), tpr, _ptr(self.ws),
                                        self.ws.numel(), _stream()), "moe_forward")
        else:
            self._staged(x, None, y, aux, tpr, events)
        return y

    def _staged(self, x, noise, y, aux, tpr, events):
        ev = stage_events(events)
        _check(self.lib.moe_forward_staged(ctypes.byref(self.cfg), ctypes.byref(self.weights),
                                           _ptr(x), ctypes.byref(noise) if noise else None,
                                           _ptr(y), _ptr(aux), tpr, ctypes.byref(ev),
                                           _ptr(self.ws), self.ws.numel(), _stream()),
               "moe_forward_staged")

    def forward_noisy(self, x: torch.Tensor, eps: Optional[torch.Tensor] = None,
                      y: Optional[torch.Tensor] = None, aux: Optional[torch.Tensor] = None,
                      taps: Optional[dict] = None, events: Optional[list] = None,
                      seed: Optional[int] = None, offset: int = 0) -> torch.Tensor:
        """The layer with noisy top-k gating: eps [T, E] fp32 standard normal draws, or
        (eps None) the library's counter-based draws for (seed, offset)."""
        if (eps is None) == (seed is None):
            raise ValueError("give either eps or seed")
        if y is None:
            y = torch.empty_like(x)
        tp = _taps(taps)
        tpr = ctypes.byref(tp) if tp is not None else None
        if events is not None:
            self._staged(x, MoeNoise(eps=_ptr(eps), seed=seed or 0, offset=offset), y, aux, tpr,
                         events)
        elif eps is not None:
            _check(self.lib.moe_forward_noisy(ctypes.byref(self.cfg), ctypes.byref(self.weights),
                                              _ptr(x), _ptr(eps), _ptr(y), _ptr(aux), tpr,
                                              _ptr(self.ws), self.ws.numel(), _stream()),
                   "moe_forward_noisy")
        else:
            _check(self.lib.moe_forward_noisy_seeded(
                ctypes.byref(self.cfg), ctypes.byref(self.weights), _ptr(x), seed, offset,
                _ptr(y), _ptr(aux), tpr, _ptr(self.ws), self.ws.numel(), _stream()),
                "moe_forward_noisy_seeded")
        return y

    def new_taps(self) -> dict:
        T, E, k = self.w.T, self.w.n_experts, self.w.top_k
        dev = self.device
        i32 = dict(dtype=torch.int32, device=dev)
        return {"logits": torch.empty((T, E), dtype=torch.float32, device=dev),
                "topk_idx": torch.empty((T, k), **i32),
                "topk_gate": torch.empty((T, k), dtype=torch.float32, device=dev),
                "counts": torch.empty((E,), **i32), "offsets": torch.empty((E + 1,), **i32),
                "perm": torch.empty((T * k,), **i32), "inv": torch.empty((T * k,), **i32)}

    def new_aux(self) -> torch.Tensor:
        return torch.zeros(3 + 2 * self.w.n_experts, dtype=torch.float32, device=self.device)

    # ------------------------------------------------------------- single steps
    def route(self, x: Optional[torch.Tensor], logits: torch.Tensor, topk_idx: torch.Tensor,
              topk_gate: torch.Tensor):
        _check(self.lib.moe_route(ctypes.byref(self.cfg), ctypes.byref(self.weights), _ptr(x),
                                  _ptr(logits), _ptr(topk_idx), _ptr(topk_gate), _ptr(self.ws),
                                  self.ws.numel(), _stream()), "moe_route")

    def route_noisy(self, x: torch.Tensor, eps: torch.Tensor, logits: torch.Tensor,
                    topk_idx: torch.Tensor, topk_gate: torch.Tensor):
        _check(self.lib.moe_route_noisy(ctypes.byref(self.cfg), ctypes.byref(self.weights),
                                        _ptr(x), _ptr(eps), _ptr(logits), _ptr(topk_idx),
                                        _ptr(topk_gate), _ptr(self.ws), self.ws.numel(),
                                        _stream()), "moe_route_noisy")

    def route_noisy_seeded(self, x: torch.Tensor, seed: int, offset: int, logits: torch.Tensor,
                           topk_idx: torch.Tensor, topk_gate: torch.Tensor):
        _check(self.lib.moe_route_noisy_seeded(ctypes.byref(self.cfg), ctypes.byref(self.weights),
                                               _ptr(x), seed, offset, _ptr(logits),
                                               _ptr(topk_idx), _ptr(topk_gate), _ptr(self.ws),
                                               self.ws.numel(), _stream()),
               "moe_route_noisy_seeded")

    def route_expert_choice(self, x: Optional[torch.Tensor], logits: torch.Tensor,
                            ec_idx: torch.Tensor, ec_score: torch.Tensor):
        """Expert-Choice routing: logits [T, E] (input when x is None), ec_idx [E, C],
        ec_score [E, C]."""
        _check(self.lib.moe_route_expert_choice(
            ctypes.byref(self.cfg), ctypes.byref(self.weights), _ptr(x), _ptr(logits),
            _ptr(ec_idx), _ptr(ec_score), _ptr(self.ws), self.ws.numel(), _stream()),
            "moe_route_expert_choice")

    def permute(self, x, topk_idx, counts, offsets, perm, inv, x_perm):
        check_rows(x_perm, expert_rows(self.cfg), self.cfg.d_model, "x_perm")
        _check(self.lib.moe_permute(ctypes.byref(self.cfg), _ptr(x), _ptr(topk_idx), _ptr(counts),
                                    _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(x_perm),
                                    _ptr(self.ws), self.ws.numel(), _stream()), "moe_permute")

    def expert_ffn(self, x_perm, offsets, y_perm, cfg: Optional[MoeCfg] = None,
                   weights: Optional[MoeWeights] = None):
        c = cfg or self.cfg
        check_rows(x_perm, expert_rows(c), c.d_model, "x_perm")
        check_rows(y_perm, expert_rows(c), c.d_model, "y_perm")
        _check(self.lib.moe_expert_ffn(ctypes.byref(cfg or self.cfg),
                                       ctypes.byref(weights or self.weights), _ptr(x_perm),
                                       _ptr(offsets), _ptr(y_perm), _ptr(self.ws),
                                       self.ws.numel(), _stream()), "moe_expert_ffn")

    def combine(self, y_perm, inv, topk_gate, shared_y, y):
        check_rows(y_perm, expert_rows(self.cfg), self.cfg.d_model, "y_perm")
        _check(self.lib.moe_combine(ctypes.byref(self.cfg), _ptr(y_perm), _ptr(inv),
                                    _ptr(topk_gate), _ptr(shared_y), _ptr(y), _ptr(self.ws),
                                    self.ws.numel(), _stream()), "moe_combine")

    def aux_stats(self, logits, topk_idx, out):
        _check(self.lib.moe_aux_stats(ctypes.byref(self.cfg), _ptr(logits), _ptr(topk_idx),
                                      _ptr(out), _ptr(self.ws), self.ws.numel(), _stream()),
               "moe_aux_stats")

    # ------------------------------------------------- one shard of a larger batch
    def route_shard(self, x: Optional[torch.Tensor], logits: Optional[torch.Tensor],
                    topk_idx: torch.Tensor, topk_gate: torch.Tensor, counts: torch.Tensor,
                    aux_part: Optional[torch.Tensor] = None):
        """moe_route on this shard + its pre-drop counts [E] int32 and, optionally, its
        fp64 sums aux_part [1 + 2E] for the statistics."""
        _check(self.lib.moe_route_shard(ctypes.byref(self.cfg), ctypes.byref(self.weights),
                                        _ptr(x), _ptr(logits), _ptr(topk_idx), _ptr(topk_gate),
                                        _ptr(counts), _ptr(aux_part), _ptr(self.ws),
                                        self.ws.numel(), _stream()), "moe_route_shard")

    def permute_shard(self, shard: MoeShard, x, topk_idx, counts, offsets, perm, inv, x_perm):
        check_rows(x_perm, expert_rows(self.cfg), self.cfg.d_model, "x_perm")
        _check(self.lib.moe_permute_shard(ctypes.byref(self.cfg), ctypes.byref(shard), _ptr(x),
                                          _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                                          _ptr(perm), _ptr(inv), _ptr(x_perm), _ptr(self.ws),
                                          self.ws.numel(), _stream()), "moe_permute_shard")

    def forward_shard(self, shard: MoeShard, x: torch.Tensor, taps: dict,
                      y: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The layer on this shard, routed by route_shard: taps["topk_idx"] and
        taps["topk_gate"] are inputs."""
        if y is None:
            y = torch.empty_like(x)
        tp = MoeTaps(**{k: _ptr(taps.get(k)) for k, _ in MoeTaps._fields_})
        _check(self.lib.moe_forward_shard(ctypes.byref(self.cfg), ctypes.byref(shard),
                                          ctypes.byref(self.weights), _ptr(x), ctypes.byref(tp),
                                          _ptr(y), _ptr(self.ws), self.ws.numel(), _stream()),
               "moe_forward_shard")
        return y

    def aux_finalize(self, n_tokens_total: int, aux_part: torch.Tensor,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
        if out is None:
            out = self.new_aux()
        _check(self.lib.moe_aux_finalize(ctypes.byref(self.cfg), int(n_tokens_total),
                                         _ptr(aux_part), _ptr(out), _stream()),
               "moe_aux_finalize")
        return out

    # ------------------------------------------------------------ the training step
    @property
    def bws(self) -> torch.Tensor:
        """The workspace of the gradients, made at the first use, and ready on every stream from
        then on. Calls that share it must not overlap. In a capture it cannot be made (the
        captured initialisation would not have run): make that use before."""
        if self._bws is None:
            with torch.cuda.device(self.ws.device):
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("the gradients' workspace must be made before a capture: "
                                       "read layer.bws first")
                ws = new_workspace(self.cfg, self.ws.device, backward=True)
                torch.cuda.current_stream().synchronize()
                self._bws = ws
        return self._bws

    def _call(self, name: str, *args):
        """lib.name(cfg, *args, workspace, its size, stream) on this layer's device, on
        that device's current stream."""
        bws = self._bws if self._bws is not None else self.bws
        st = _on_device(self._index, getattr(self.lib, name), ctypes.byref(self.cfg), *args,
                        bws.data_ptr(), bws.numel())
        if st:
            _check(st, name)

    def _want(self, t, shape, name, dtype=None, optional=False):
        dtype = dtype or self._dtype
        if (t is None or t.shape != shape or t.dtype is not dtype or not t.is_contiguous()
                or t.get_device() != self._index):
            check_tensor(t, shape, dtype, name, self.ws.device, optional)

    def grad_shapes(self) -> dict:
        """name -> (shape, dtype) of every parameter's gradient: the parameters this layer
        has (b_router also stands for logit_bias)."""
        w, dt, f32 = self.w, self.w.torch_dtype, torch.float32
        E, d, F, Fs = w.n_experts, w.d_model, w.d_ff, w.n_shared * w.d_ff_shared
        shapes = {"w_router": ((E, d), dt), "b_router": ((E,), f32), "w1": ((E, F, d), dt),
                  "w3": ((E, F, d), dt), "w2": ((E, d, F), dt), "b1": ((E, F), f32),
                  "b2": ((E, d), f32), "ws_gate": ((Fs, d), dt), "ws_up": ((Fs, d), dt),
                  "ws_down": ((d, Fs), dt)}
        has = {n for n in shapes if self.p.get(n) is not None}
        if self.p.get("w_router") is not None:
            has.add("b_router")
        return {n: s for n, s in shapes.items() if n in has}

    def parameters(self) -> dict:
        """name of the gradient -> this layer's parameter of it, for AdamW. The router's bias
        (b_router) is logit_bias in a layer that has no other; next to a b_router, logit_bias is
        left out: the logits take their sum, and trained both it would move twice as far."""
        bias = self.p.get("b_router")
        own = dict(self.p, b_router=self.p.get("logit_bias") if bias is None else bias)
        return {n: own[n] for n in self.grad_shapes() if own.get(n) is not None}

    def new_grads(self) -> dict:
        """Buffers for the gradients of this layer's parameters."""
        return {n: torch.empty(s, dtype=dt, device=self.ws.device)
                for n, (s, dt) in self.grad_shapes().items()}

    def _grads(self, grads: Optional[dict], names) -> MoeGrads:
        shapes, out = self.grad_shapes(), MoeGrads()
        for n, t in (grads or {}).items():
            if t is None or n not in names:
                continue
            if n not in shapes:
                raise ValueError(f"this layer has no {n}")
            self._want(t, shapes[n][0], f"grads[{n!r}]", shapes[n][1])
            setattr(out, n, t.data_ptr())
        return out

    def combine_backward(self, dy: torch.Tensor, y_perm: Optional[torch.Tensor],
                         inv: torch.Tensor, topk_gate: Optional[torch.Tensor],
                         dy_perm: Optional[torch.Tensor], dgate: Optional[torch.Tensor]):
        """Gradient of combine: dy [T, d] -> dy_perm [R, d] and dgate [T, k] (each may be
        None; y_perm is read for dgate, topk_gate for dy_perm)."""
        T, d, k, i32, f32 = self.w.T, self.w.d_model, self.w.top_k, torch.int32, torch.float32
        self._want(dy, (T, d), "dy")
        self._want(y_perm, (T * k, d), "y_perm", optional=dgate is None)
        self._want(inv, (T * k,), "inv", i32)
        self._want(topk_gate, (T, k), "topk_gate", f32, optional=dy_perm is None)
        self._want(dy_perm, (T * k, d), "dy_perm", optional=True)
        self._want(dgate, (T, k), "dgate", f32, optional=True)
        self._call("moe_combine_backward", _addr(dy), _addr(y_perm), _addr(inv), _addr(topk_gate),
                   _addr(dy_perm), _addr(dgate))

    def permute_backward(self, dx_perm: torch.Tensor, inv: torch.Tensor,
                         dx_add: Optional[torch.Tensor], dx: torch.Tensor):
        """Gradient of permute: dx_perm [R, d] -> dx [T, d] (plus dx_add [T, d] fp32)."""
        T, d, k = self.w.T, self.w.d_model, self.w.top_k
        self._want(dx_perm, (T * k, d), "dx_perm")
        self._want(inv, (T * k,), "inv", torch.int32)
        self._want(dx_add, (T, d), "dx_add", torch.float32, optional=True)
        self._want(dx, (T, d), "dx")
        self._call("moe_permute_backward", _addr(dx_perm), _addr(inv), _addr(dx_add), _addr(dx))

    def route_backward(self, x: Optional[torch.Tensor], logits: torch.Tensor,
                       topk_idx: torch.Tensor, counts: Optional[torch.Tensor],
                       dgate: Optional[torch.Tensor], d_losses: Optional[torch.Tensor],
                       dlogits: Optional[torch.Tensor], dx: Optional[torch.Tensor],
                       grads: Optional[dict] = None):
        """Gradient of route and aux_stats: from dgate [T, k] and d_losses [2] (the upstream
        gradients of aux and z_loss, with counts) the gradients of the logits [T, E] fp32,
        of x ([T, d] fp32) and grads["w_router"], grads["b_router"]."""
        T, d, E, k = self.w.T, self.w.d_model, self.w.n_experts, self.w.top_k
        i32, f32 = torch.int32, torch.float32
        g = self._grads(grads, ("w_router", "b_router"))
        self._want(x, (T, d), "x", optional=not g.w_router)
        self._want(logits, (T, E), "logits", f32)
        self._want(topk_idx, (T, k), "topk_idx", i32)
        self._want(counts, (E,), "counts", i32, optional=d_losses is None)
        self._want(dgate, (T, k), "dgate", f32, optional=True)
        self._want(d_losses, (2,), "d_losses", f32, optional=True)
        self._want(dlogits, (T, E), "dlogits", f32, optional=True)
        self._want(dx, (T, d), "dx", f32, optional=True)
        self._call("moe_route_backward", ctypes.byref(self.weights), _addr(x), _addr(logits),
                   _addr(topk_idx), _addr(counts), _addr(dgate), _addr(d_losses), _addr(dlogits),
                   _addr(dx), ctypes.byref(g))

    def expert_ffn_backward(self, x_perm: torch.Tensor, offsets: torch.Tensor,
                            dy_perm: torch.Tensor, dx_perm: Optional[torch.Tensor],
                            grads: Optional[dict] = None):
        """Gradient of expert_ffn: dx_perm [R, d] and grads["w1"], ["w3"], ["w2"], ["b1"],
        ["b2"] (those that `grads` names)."""
        R, d = expert_rows(self.cfg), self.w.d_model
        self._want(x_perm, (R, d), "x_perm")
        self._want(offsets, (self.w.n_experts + 1,), "offsets", torch.int32)
        self._want(dy_perm, (R, d), "dy_perm")
        self._want(dx_perm, (R, d), "dx_perm", optional=True)
        g = self._grads(grads, ("w1", "w3", "w2", "b1", "b2"))
        self._call("moe_expert_ffn_backward", ctypes.byref(self.weights), _addr(x_perm),
                   _addr(offsets), _addr(dy_perm), _addr(dx_perm), ctypes.byref(g))

    def backward(self, x: torch.Tensor, dy: torch.Tensor, taps: dict,
                 dx: Optional[torch.Tensor] = None, grads: Optional[dict] = None,
                 d_losses: Optional[torch.Tensor] = None):
        """Gradient of forward: `taps` as the forward filled them (new_taps); returns (dx,
        grads), into the buffers given or new ones (a dict without some names: those
        gradients are not computed)."""
        T, d, E, k = self.w.T, self.w.d_model, self.w.n_experts, self.w.top_k
        i32, f32 = torch.int32, torch.float32
        self._want(x, (T, d), "x")
        self._want(dy, (T, d), "dy")
        for n, s, t in (("logits", (T, E), f32), ("topk_idx", (T, k), i32),
                        ("topk_gate", (T, k), f32), ("offsets", (E + 1,), i32),
                        ("inv", (T * k,), i32)):
            self._want(taps.get(n), s, f"taps[{n!r}]", t)
        self._want(taps.get("counts"), (E,), "taps['counts']", i32, optional=d_losses is None)
        self._want(d_losses, (2,), "d_losses", f32, optional=True)
        if dx is None:
            dx = torch.empty_like(x)
        self._want(dx, (T, d), "dx")
        if grads is None:
            grads = self.new_grads()
        g = self._grads(grads, tuple(self.grad_shapes()) + tuple(grads))
        tp = _taps(taps)
        self._call("moe_backward", ctypes.byref(self.weights), _addr(x), ctypes.byref(tp),
                   _addr(dy), _addr(d_losses), _addr(dx), ctypes.byref(g))
        return dx, grads

    def last_backward_error(self):
        """(code, info) of the gradients' workspace, cleared (see last_device_error)."""
        return self._device_error(self.bws)

    def last_device_error(self):
        return self._device_error(self.ws)

    def _device_error(self, ws):
        code, info = ctypes.c_int32(0), ctypes.c_int32(0)
        st = _on_device(self._index, self.lib.moe_last_device_error, _ptr(ws),
                        ctypes.byref(code), ctypes.byref(info))
        if st not in (MOE_OK, 6):
            raise MoeError(st, "moe_last_device_error")
        return code.value, info.value


def noise_draws(n_tokens: int, n_experts: int, seed: int, offset: int, eps: torch.Tensor,
                raw: Optional[torch.Tensor] = None):
    """moe_noise_draws: eps [T, E] fp32 and optionally raw [T, ceil(E/4), 4] int32 words
    (the uint32 bit patterns), both on the current device and stream."""
    _check(load().moe_noise_draws(n_tokens, n_experts, seed, offset, _ptr(eps), _ptr(raw),
                                  _stream()), "moe_noise_draws")


class AdamW:
    """AdamW over CUDA tensors on one device (moe_adamw_step), a list or a dict of them,
    updated in place.

    ``state_bits``: 32, or 8 (e4m3 with one fp32 scale for each ADAMW_BLOCK elements).
    ``master``: keep fp32 copies of the bf16 parameters, which the step works on.
    ``state`` continues a former run: a dict of ``step`` and lists ``exp_avg``,
    ``exp_avg_sq``, with 8 bits ``exp_avg_scale`` and ``exp_avg_sq_scale``, and optionally
    ``master`` (None where a parameter has none), used as they are; `state_dict` gives one.
    With 8 bits exp_avg_sq holds the root of the second moment.

    The step works on the storage that the parameters and the state had at first. A step
    after a parameter got another one (``p.data = ...``, ``p.set_()``) raises ValueError: make
    a new optimizer from `state_dict`. The state's tensors are for reading and for updates
    in place.
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 1e-2, state_bits: int = 32, master: bool = False,
                 state: Optional[dict] = None):
        self.names = list(params) if isinstance(params, dict) else None
        self.params = list(params.values() if isinstance(params, dict) else params)
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        if not self.params:
            raise ValueError("no parameters")
        self.device = self.params[0].device
        if self.device.type != "cuda":
            raise ValueError("the parameters must be CUDA tensors")
        if state is None:
            if state_bits not in (8, 32):
                raise ValueError("state_bits must be 32 or 8")
            self.bits, self.t = state_bits, 0
            dt = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
            new = lambda p: torch.zeros(p.shape, dtype=dt, device=p.device)  # noqa: E731
            self.exp_avg = tuple(new(p) for p in self.params)
            self.exp_avg_sq = tuple(new(p) for p in self.params)
            self.exp_avg_scale = self.exp_avg_sq_scale = None
            if state_bits == 8:
                scale = lambda p: torch.zeros(-(-p.numel() // ADAMW_BLOCK), device=p.device)  # noqa: E731
                self.exp_avg_scale = tuple(scale(p) for p in self.params)
                self.exp_avg_sq_scale = tuple(scale(p) for p in self.params)
            self.master = tuple(p.float() if master and p.dtype == torch.bfloat16 else None
                                for p in self.params)
        else:
            self.t = int(state["step"])
            self.exp_avg, self.exp_avg_sq = tuple(state["exp_avg"]), tuple(state["exp_avg_sq"])
            scales = [state.get(n) for n in ("exp_avg_scale", "exp_avg_sq_scale")]
            self.exp_avg_scale, self.exp_avg_sq_scale = (None if x is None else tuple(x)
                                                         for x in scales)
            self.bits = 32 if self.exp_avg_scale is None else 8
            self.master = tuple(state.get("master") or [None] * len(self.params))
        self._lib = load()
        n_params = len(self.params)
        if len({p.data_ptr() for p in self.params if p.numel()}) != sum(1 for p in self.params
                                                                        if p.numel()):
            raise ValueError("the same parameter twice")
        dt = torch.float32 if self.bits == 32 else torch.float8_e4m3fn
        lists = [self.exp_avg, self.exp_avg_sq, self.master]
        if self.bits == 8:
            lists += [self.exp_avg_scale, self.exp_avg_sq_scale]
        if any(x is None or len(x) != n_params for x in lists):
            raise ValueError("the state has not one entry for each parameter")
        self._batch = (MoeAdamWTensor * n_params)()
        for i, p in enumerate(self.params):
            if p.dtype not in _ADAMW_DTYPES:
                raise ValueError(f"parameter {i} is {p.dtype}: fp32 or bf16 are supported")
            check_tensor(p, p.shape, p.dtype, f"parameter {i}", self.device)
            check_tensor(self.exp_avg[i], p.shape, dt, f"exp_avg[{i}]", self.device)
            check_tensor(self.exp_avg_sq[i], p.shape, dt, f"exp_avg_sq[{i}]", self.device)
            check_tensor(self.master[i], p.shape, torch.float32, f"master[{i}]", self.device,
                         optional=True)
            if self.master[i] is not None and p.dtype == torch.float32:
                raise ValueError(f"master[{i}]: parameter {i} is fp32 already")
            e = self._batch[i]
            e.n, e.param, e.exp_avg, e.exp_avg_sq = (p.numel(), p.data_ptr(),
                                                     self.exp_avg[i].data_ptr(),
                                                     self.exp_avg_sq[i].data_ptr())
            e.master = _addr(self.master[i])
            if self.bits == 8:
                n = (-(-p.numel() // ADAMW_BLOCK),)
                for name, x in (("exp_avg_scale", self.exp_avg_scale[i]),
                                ("exp_avg_sq_scale", self.exp_avg_sq_scale[i])):
                    check_tensor(x, n, torch.float32, f"{name}[{i}]", self.device)
                    setattr(e, name, x.data_ptr())
            e.param_dtype, e.state_bits = _ADAMW_DTYPES[p.dtype], self.bits
        # views of the two members that every step sets, all tensors at once
        self._grad_ptrs = np.ndarray((n_params,), np.uint64, self._batch, MoeAdamWTensor.grad.offset,
                                     (ctypes.sizeof(MoeAdamWTensor),))
        self._grad_types = np.ndarray((n_params,), np.int32, self._batch,
                                      MoeAdamWTensor.grad_dtype.offset,
                                      (ctypes.sizeof(MoeAdamWTensor),))
        self._grad_dtypes = None  # the types that _grad_types holds
        # what the addresses above point to is kept by aliases of our own, whatever is done to the
        # tensors; the parameters' addresses are compared at every step (and no other tensor
        # can get one of them meanwhile)
        self._addresses = [p.data_ptr() for p in self.params]
        self._held = [x.detach() for xs in (self.params, *lists) for x in xs if x is not None]
        self._shapes = [p.shape for p in self.params]
        self._devices = [p.get_device() for p in self.params]
        self._index = self.params[0].get_device()

    def step(self, grads, grad_scale: Optional[torch.Tensor] = None,
             found_inf: Optional[torch.Tensor] = None, step: Optional[torch.Tensor] = None,
             lr: Optional[torch.Tensor] = None):
        """One step from ``grads``: a list in the parameters' order, or a dict with an entry for
        each name of a dict of parameters (others are left alone).
        Device scalars, read when the kernel runs: ``grad_scale`` multiplies the gradients,
        ``found_inf`` nonzero skips the update (the step still counts: a program that counts
        updates only passes its own ``step``), ``step`` (int64) and ``lr`` (fp32) take the place
        of the counter and of self.lr (a captured step needs them to move, and the program's
        count is then the one to save: self.t moves with calls, not with replays)."""
        if isinstance(grads, dict):
            if self.names is None or any(n not in grads for n in self.names):
                raise ValueError("a dict of gradients needs the names of a dict of parameters")
            grads = [grads[n] for n in self.names]
        else:
            grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} parameters")
        # list by list: a hundred tensors are checked in the time of a launch or two
        data_ptr = torch.Tensor.data_ptr
        if list(map(data_ptr, self.params)) != self._addresses:
            moved = [i for i, p in enumerate(self.params) if p.data_ptr() != self._addresses[i]]
            raise ValueError(f"parameter {moved[0]} has another storage than when the optimizer "
                             "was made")
        try:
            fit = ([g.shape for g in grads] == self._shapes
                   and list(map(torch.Tensor.get_device, grads)) == self._devices
                   and all(map(torch.Tensor.is_contiguous, grads)))
        except (AttributeError, TypeError):  # no tensor: None where nothing was computed
            fit = False
        if not fit:
            for i, (g, p) in enumerate(zip(grads, self.params)):  # which one
                if not isinstance(g, torch.Tensor):
                    raise ValueError(f"gradient {i} is missing" if g is None else
                                     f"gradient {i} is no tensor")
                check_tensor(g, p.shape, g.dtype, f"gradient {i}", self.device)
        dtypes = [g.dtype for g in grads]
        if dtypes != self._grad_dtypes:
            bad = [i for i, dt in enumerate(dtypes) if dt not in _ADAMW_DTYPES]
            if bad:
                raise ValueError(f"gradient {bad[0]} is {dtypes[bad[0]]}: fp32 or bf16 are "
                                 "supported")
            self._grad_types[:] = [_ADAMW_DTYPES[dt] for dt in dtypes]
            self._grad_dtypes = dtypes
        self._grad_ptrs[:] = list(map(data_ptr, grads))
        o = MoeAdamW(self.betas[0], self.betas[1], self.lr, self.eps, self.weight_decay, self.t + 1)
        for name, t, dt in (("grad_scale", grad_scale, torch.float32),
                            ("found_inf", found_inf, torch.float32),
                            ("step_dev", step, torch.int64), ("lr_dev", lr, torch.float32)):
            if t is not None:
                if t.numel() != 1:
                    raise ValueError(f"{name} must hold one value")
                check_tensor(t, t.shape, dt, name, self.device)
                setattr(o, name, t.data_ptr())
        st = _on_device(self._index, self._lib.moe_adamw_step, self._batch, len(self.params),
                        ctypes.byref(o))
        if st:
            _check(st, "moe_adamw_step")
        self.t += 1

    def state_dict(self) -> dict:
        lists = {n: getattr(self, n) for n in ("exp_avg", "exp_avg_sq", "exp_avg_scale",
                                               "exp_avg_sq_scale", "master")}
        return {"step": self.t, **{n: None if x is None else list(x) for n, x in lists.items()}}


def shared_as_experts(layer: MoELayer):
    """(cfg, weights) that run the layer's shared experts through moe_expert_ffn:
    one group, d_ff = n_shared * d_ff_shared, rows = all tokens."""
    w = layer.w
    cfg = make_cfg(w, n_experts=1, top_k=1, d_ff=w.n_shared * w.d_ff_shared,
                   act=synth.ACT_SWIGLU, n_shared=0, d_ff_shared=0, capacity_factor=0.0)
    p = layer.p
    wt = MoeWeights(w1=_ptr(p["ws_gate"]), w3=_ptr(p["ws_up"]), w2=_ptr(p["ws_down"]))
    return cfg, wt
