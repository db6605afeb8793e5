"""Python binding of libtq (block-quantized decode GEMV and top-k MoE expert FFN on gfx950).

Argument marshalling only: every call forwards device pointers, sizes and the current HIP stream
to the C ABI declared in ``include/tq.h``; all computation happens in the library's kernels.
PyTorch supplies device memory and streams. The library must be built
(``python -m moe_expert_ffn_q4_amd.build``); there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")

Q4_K, Q6_K, Q8_0, Q5_K, Q4_0 = 1, 2, 3, 4, 5
TYPES = {"q4_k": Q4_K, "q6_k": Q6_K, "q8_0": Q8_0, "q5_k": Q5_K, "q4_0": Q4_0}
F32, BF16, F16 = 0, 1, 2
PATH_AUTO, PATH_F32, PATH_BF16_MFMA = 0, 1, 2
MOE_ROUTE, MOE_EXPERTS, MOE_COMBINE, MOE_ALL = 1, 2, 4, 7
STATUS = {0: "TQ_OK", 1: "TQ_EINVAL", 2: "TQ_ESHAPE", 3: "TQ_EALIGN", 4: "TQ_ENOSPC",
          5: "TQ_EUNSUPPORTED", 6: "TQ_EDEVICE"}


class TQError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def lib() -> C.CDLL:
    """The loaded libtq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libtq.so not found at {LIB_PATH}; build it with "
                               "`python -m moe_expert_ffn_q4_amd.build`")
        _lib = C.CDLL(LIB_PATH)
        _declare(_lib)
    return _lib


_vp, _i64, _int = C.c_void_p, C.c_int64, C.c_int


class Expert(C.Structure):
    _fields_ = [("gate", _vp), ("up", _vp), ("down", _vp)]


class MoeDesc(C.Structure):
    _fields_ = [("type", _int), ("hidden", _i64), ("ffn", _i64), ("n_experts", _i64),
                ("top_k", _i64), ("router_w", _vp), ("experts", _vp), ("experts_host", _vp),
                ("shared", Expert), ("renormalize", _int), ("experts_on_host", _int),
                ("copy_stream", _vp), ("path", _int), ("expert_cache", _vp)]


class ExpertCacheStats(C.Structure):
    _fields_ = [("calls", _i64), ("hits", _i64), ("misses", _i64), ("fallbacks", _i64),
                ("prefetched", _i64), ("prefetch_hits", _i64), ("bytes_copied", _i64)]


class ChainOp(C.Structure):
    _fields_ = [("nparts", _int), ("swiglu", _int), ("w", _vp * 4), ("n", _i64 * 4),
                ("y", _vp * 4), ("k", _i64), ("x", _vp)]


class KvCacheDesc(C.Structure):
    _fields_ = [("kv_heads", _i64), ("head_dim", _i64), ("page_tokens", _i64), ("pages", _i64),
                ("data", _vp)]


class HeadRows(C.Structure):
    _fields_ = [("data", _vp), ("heads", _i64), ("row_stride", _i64), ("head_stride", _i64)]


class KvStepDesc(C.Structure):
    _fields_ = ([(f, _i64) for f in ("requests", "max_blocks", "rows")] +
                [(f, _vp) for f in ("kv_len", "new_len", "block_table", "free_pages", "free_count",
                                    "cu_new", "seq_len", "slots", "positions", "requests_of",
                                    "free_count_out", "status")])


class RopeDesc(C.Structure):
    _fields_ = [("inv_freq", _vp), ("positions", _vp), ("axis_stride", _i64), ("pairs", _i64),
                ("axes", _i64), ("sections", _i64 * 4), ("interleaved", _int)]


class KvAttnDesc(C.Structure):
    _fields_ = [("rows", _i64), ("requests", _i64), ("max_blocks", _i64), ("q", HeadRows),
                ("out", HeadRows), ("lse", _vp), ("block_table", _vp), ("seq_len", _vp),
                ("cu_new", _vp), ("scale", C.c_float), ("window", _i64)]


class MoeRouting(C.Structure):
    _fields_ = [("topk_ids", _vp), ("topk_w", _vp), ("logits", _vp), ("counts", _vp),
                ("offsets", _vp), ("pairs", _vp)]


def _declare(L: C.CDLL) -> None:
    L.tq_block_weights.argtypes = [_int]
    L.tq_block_weights.restype = _i64
    L.tq_block_bytes.argtypes = [_int]
    L.tq_block_bytes.restype = _i64
    L.tq_row_bytes.argtypes = [_int, _i64]
    L.tq_row_bytes.restype = _i64
    L.tq_last_error.argtypes = []
    L.tq_last_error.restype = C.c_char_p
    L.tq_dequant.argtypes = [_int, _vp, _i64, _i64, _int, _vp, _vp]
    L.tq_dequant.restype = _int
    L.tq_gemv_workspace_bytes.argtypes = [_int, _i64, _i64, _i64]
    L.tq_gemv_workspace_bytes.restype = C.c_size_t
    L.tq_gemv.argtypes = [_int, _vp, _i64, _i64, _vp, _i64, _vp, _vp, C.c_size_t, _vp]
    L.tq_gemv.restype = _int
    L.tq_gemv_noalloc.argtypes = [_int, _vp, _i64, _i64, _vp, _i64, _vp, _vp]
    L.tq_gemv_noalloc.restype = _int
    L.tq_swiglu.argtypes = [_vp, _vp, _i64, _vp, _vp]
    L.tq_swiglu.restype = _int
    L.tq_gemv_multi_workspace_bytes.argtypes = [_int, _int, C.POINTER(_i64), _i64, _i64]
    L.tq_gemv_multi_workspace_bytes.restype = C.c_size_t
    L.tq_gemv_multi.argtypes = [_int, _int, C.POINTER(_vp), C.POINTER(_i64), C.POINTER(_vp), _i64,
                                _vp, _i64, _vp, C.c_size_t, _vp]
    L.tq_gemv_multi.restype = _int
    L.tq_gemv_swiglu_workspace_bytes.argtypes = [_int, _i64, _i64, _i64]
    L.tq_gemv_swiglu_workspace_bytes.restype = C.c_size_t
    L.tq_gemv_swiglu.argtypes = [_int, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, C.c_size_t, _vp]
    L.tq_gemv_swiglu.restype = _int
    L.tq_chain_plan_bytes.argtypes = [_int]
    L.tq_chain_plan_bytes.restype = C.c_size_t
    L.tq_chain_prepare.argtypes = [_int, C.POINTER(ChainOp), _int, _vp, C.c_size_t]
    L.tq_chain_prepare.restype = _int
    L.tq_chain_run.argtypes = [_vp, _vp]
    L.tq_chain_run.restype = _int
    L.tq_chain_status.argtypes = [_vp, _vp]
    L.tq_chain_status.restype = _int
    L.tq_kv_page_bytes.argtypes = [_vp]
    L.tq_kv_page_bytes.restype = C.c_size_t
    L.tq_kv_plan.argtypes = [_vp, _vp, _vp]
    L.tq_kv_plan.restype = _int
    L.tq_kv_append.argtypes = [_vp, _int, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    L.tq_kv_append.restype = _int
    L.tq_kv_read.argtypes = [_vp, _int, _i64, _vp, _vp, _vp, _vp]
    L.tq_kv_read.restype = _int
    L.tq_kv_attention_workspace_bytes.argtypes = [_vp, _int, _vp]
    L.tq_kv_attention_workspace_bytes.restype = C.c_size_t
    L.tq_kv_attention.argtypes = [_vp, _int, _vp, _vp, C.c_size_t, _vp]
    L.tq_kv_attention.restype = _int
    if hasattr(L, "tq_moe_ffn"):
        L.tq_moe_workspace_bytes.argtypes = [C.POINTER(MoeDesc), _i64]
        L.tq_moe_workspace_bytes.restype = C.c_size_t
        L.tq_moe_ffn.argtypes = [C.POINTER(MoeDesc), _vp, _i64, _vp, _vp, C.c_size_t,
                                 C.POINTER(MoeRouting), _vp]
        L.tq_moe_ffn.restype = _int
        L.tq_moe_ffn_stages.argtypes = [C.POINTER(MoeDesc), _vp, _i64, _vp, _vp, C.c_size_t,
                                        C.POINTER(MoeRouting), _int, _vp]
        L.tq_moe_ffn_stages.restype = _int
        L.tq_tuning_set.argtypes = [_int, _int]
        L.tq_tuning_set.restype = _int
        L.tq_tuning_get.argtypes = [_int]
        L.tq_tuning_get.restype = _int
        L.tq_expert_cache_slot_bytes.argtypes = [C.POINTER(MoeDesc)]
        L.tq_expert_cache_slot_bytes.restype = C.c_size_t
        L.tq_expert_cache_state_bytes.argtypes = [C.POINTER(MoeDesc), _i64]
        L.tq_expert_cache_state_bytes.restype = C.c_size_t
        L.tq_expert_cache_init.argtypes = [_vp, C.c_size_t, C.POINTER(MoeDesc), _i64, _i64, _vp,
                                           C.c_size_t]
        L.tq_expert_cache_init.restype = _int
        L.tq_expert_cache_stats_get.argtypes = [_vp, C.POINTER(ExpertCacheStats)]
        L.tq_expert_cache_stats_get.restype = _int
        L.tq_expert_cache_destroy.argtypes = [_vp]
        L.tq_expert_cache_destroy.restype = _int


def _check(rc: int) -> None:
    if rc != 0:
        raise TQError(rc, lib().tq_last_error().decode())


def _type(t) -> int:
    return TYPES[t] if isinstance(t, str) else int(t)


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def row_bytes(t, k: int) -> int:
    return int(lib().tq_row_bytes(_type(t), k))


def dequant(t, w: torch.Tensor, n: int, k: int, out_dtype: str = "f32", out=None, stream=None):
    """Dense [n][k] weights: fp32 values, or bf16 bit patterns as int16 ('bf16')."""
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32 if out_dtype == "f32" else torch.int16,
                          device=w.device)
    _check(lib().tq_dequant(_type(t), _ptr(w), n, k, F32 if out_dtype == "f32" else BF16,
                            _ptr(out), _stream(stream)))
    return out


_workspaces: dict = {}


def workspace(nbytes: int, device=None, purpose: str = "gemv") -> torch.Tensor:
    """A device scratch buffer of at least nbytes, reused across calls on one stream. The
    library takes workspaces with any contents; one buffer per (device, purpose) keeps calls
    that the caller runs on different streams from sharing one."""
    dev = torch.device(device if device is not None else "cuda")
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    key = (dev.type, dev.index, purpose)
    buf = _workspaces.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
        _workspaces[key] = buf
    return buf


def gemv_workspace_bytes(t, n: int, k: int, batch: int) -> int:
    return int(lib().tq_gemv_workspace_bytes(_type(t), n, k, batch))


def gemv(t, w: torch.Tensor, n: int, k: int, x: torch.Tensor, out=None, ws=None, stream=None):
    """y[b][r] = sum_c W[r][c] x[b][c] for x of shape [batch, k] (or [k]); fp32.

    ws: workspace tensor (default: the shared per-device buffer); pass False for none.
    """
    x2 = x.reshape(-1, k)
    batch = x2.shape[0]
    if out is None:
        out = torch.empty((batch, n), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(gemv_workspace_bytes(t, n, k, batch), x.device)
    wsp, wsn = (None, 0) if ws is False else (ws.data_ptr(), ws.numel() * ws.element_size())
    _check(lib().tq_gemv(_type(t), _ptr(w), n, k, _ptr(x2), batch, _ptr(out), wsp, wsn,
                         _stream(stream)))
    return out


GEMV_NOALLOC_MAX_BYTES = 16 << 20  # TQ_GEMV_NOALLOC_MAX_BYTES


def gemv_noalloc(t, w: torch.Tensor, n: int, k: int, x: torch.Tensor, out: torch.Tensor,
                 stream=None):
    """tq_gemv_noalloc: y = W x into the preallocated out [batch, n], with the library's own
    per-device scratch instead of a workspace (nothing is allocated)."""
    x2 = x.reshape(-1, k)
    _check(lib().tq_gemv_noalloc(_type(t), _ptr(w), n, k, _ptr(x2), x2.shape[0], _ptr(out),
                                 _stream(stream)))
    return out


def gemv_multi(t, ws_: list, ns: list, k: int, x: torch.Tensor, outs=None, ws=None, stream=None):
    """[W_p x for each p] in one call (matrices ws_[p] of ns[p] rows sharing x [batch, k])."""
    x2 = x.reshape(-1, k)
    batch, P = x2.shape[0], len(ns)
    if outs is None:
        outs = [torch.empty((batch, n), dtype=torch.float32, device=x.device) for n in ns]
    narr = (_i64 * P)(*ns)
    if ws is None:
        ws = workspace(int(lib().tq_gemv_multi_workspace_bytes(_type(t), P, narr, k, batch)),
                       x.device)
    _check(lib().tq_gemv_multi(_type(t), P, (_vp * P)(*[w.data_ptr() for w in ws_]), narr,
                               (_vp * P)(*[o.data_ptr() for o in outs]), k, x2.data_ptr(), batch,
                               ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)))
    return outs


def gemv_swiglu(t, w_gate: torch.Tensor, w_up: torch.Tensor, n: int, k: int, x: torch.Tensor,
                out=None, ws=None, stream=None):
    """h = silu(W_gate x) * (W_up x), fp32 [batch, n]."""
    x2 = x.reshape(-1, k)
    batch = x2.shape[0]
    if out is None:
        out = torch.empty((batch, n), dtype=torch.float32, device=x.device)
    if ws is None:
        need = int(lib().tq_gemv_swiglu_workspace_bytes(_type(t), n, k, batch))
        ws = workspace(need, x.device, "swiglu")
    _check(lib().tq_gemv_swiglu(_type(t), w_gate.data_ptr(), w_up.data_ptr(), n, k, x2.data_ptr(),
                                batch, out.data_ptr(), ws.data_ptr(),
                                ws.numel() * ws.element_size(), _stream(stream)))
    return out


def swiglu(g: torch.Tensor, u: torch.Tensor, out=None, stream=None):
    if out is None:
        out = torch.empty_like(g)
    _check(lib().tq_swiglu(_ptr(g), _ptr(u), g.numel(), _ptr(out), _stream(stream)))
    return out


class Chain:
    """A prepared chain of batch-1 Q4_K products (tq_chain_prepare / tq_chain_run), run as one
    persistent launch. ops: list of dicts with keys w (list of uint8 blobs), n (list of rows),
    y (list of fp32 output tensors), k, x (fp32 input tensor), and optionally swiglu=True (w =
    [gate, up], y = [h]). Op i reads its x only after op i-1 has stored all of its outputs. The
    tensors are kept alive here."""

    def __init__(self, t, ops: list, device=None):
        self.keep = []
        arr = (ChainOp * len(ops))()
        for i, op in enumerate(ops):
            c = arr[i]
            sw = bool(op.get("swiglu", False))
            c.nparts = len(op["w"])
            c.swiglu = int(sw)
            for p, w in enumerate(op["w"]):
                c.w[p] = w.data_ptr()
                c.n[p] = int(op["n"][p])
            for p, y in enumerate(op["y"]):
                c.y[p] = y.data_ptr()
            c.k = int(op["k"])
            c.x = op["x"].data_ptr()
            self.keep += list(op["w"]) + list(op["y"]) + [op["x"]]
        self.ops = arr
        nbytes = int(lib().tq_chain_plan_bytes(len(ops)))
        if nbytes == 0:
            raise ValueError(f"chain of {len(ops)} ops is out of range")
        dev = device if device is not None else ops[0]["x"].device
        self.plan = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _check(lib().tq_chain_prepare(_type(t), arr, len(ops), self.plan.data_ptr(), nbytes))

    def run(self, stream=None):
        _check(lib().tq_chain_run(self.plan.data_ptr(), _stream(stream)))

    def status(self, stream=None) -> int:
        """0 (TQ_OK) or TQ_EDEVICE if a run gave up a wait since the last call (the reason is in
        last_error())."""
        rc = int(lib().tq_chain_status(self.plan.data_ptr(), _stream(stream)))
        self.last_error = lib().tq_last_error().decode() if rc else ""
        return rc


class MoeLayer:
    """MoE layer for tq_moe_ffn: router weights, the expert blobs and an optional shared expert.
    Blobs are torch uint8 tensors (kept alive here). Routed experts on the device (a device
    table of blob pointers), or, when they are CPU tensors, in pinned host memory (the
    host-resident variant: the selected experts are copied per call on `copy_stream`, a
    torch.cuda.Stream, or on the call's stream when None). The shared expert is always on the
    device."""

    def __init__(self, t, hidden: int, ffn: int, router_w: torch.Tensor, experts, shared=None,
                 top_k: int = 2, renormalize: bool = True, path: int = PATH_AUTO,
                 copy_stream=None):
        self.blobs = [b for e in experts for b in e] + (list(shared) if shared else [])
        self.router_w = router_w
        E = len(experts)
        on_host = experts[0][0].device.type == "cpu"
        if on_host and not all(b.is_pinned() for e in experts for b in e):
            raise ValueError("host-resident expert blobs must be pinned (pin_memory=True)")
        self.copy_stream = copy_stream
        if on_host:
            self.host_table = (Expert * E)(*[Expert(*[b.data_ptr() for b in e]) for e in experts])
            self.table = None
        else:
            table = torch.tensor([[b.data_ptr() for b in e] for e in experts], dtype=torch.int64)
            self.table = table.to(router_w.device)
        self.desc = MoeDesc()
        self.desc.type = _type(t)
        self.desc.hidden, self.desc.ffn = hidden, ffn
        self.desc.n_experts, self.desc.top_k = E, top_k
        self.desc.router_w = router_w.data_ptr()
        self.desc.experts = None if on_host else self.table.data_ptr()
        self.desc.experts_host = C.addressof(self.host_table) if on_host else None
        if shared:
            self.desc.shared = Expert(*[b.data_ptr() for b in shared])
        self.desc.renormalize = int(renormalize)
        self.desc.experts_on_host = int(on_host)
        self.desc.copy_stream = copy_stream.cuda_stream if copy_stream is not None else None
        self.desc.path = path

    def attach_cache(self, slots: int, prefetch: int = 0) -> "ExpertCache":
        """A residency cache of `slots` device slots (host-resident experts only), used by every
        later call of this layer; returns it (its stats() count hits, misses, prefetches)."""
        self.cache = ExpertCache(self, slots, prefetch)
        self.desc.expert_cache = self.cache.state_ptr
        return self.cache

    def detach_cache(self) -> None:
        self.desc.expert_cache = None
        if getattr(self, "cache", None) is not None:
            self.cache.close()
            self.cache = None

    def workspace_bytes(self, tokens: int) -> int:
        """Bytes of workspace tq_moe_ffn needs (0 when the descriptor is invalid)."""
        return int(lib().tq_moe_workspace_bytes(C.byref(self.desc), tokens))

    def __call__(self, x: torch.Tensor, out=None, ws=None, routing: dict | None = None,
                 stream=None, stages: int = MOE_ALL):
        """y = MoE(x) for x [T, hidden] fp32. routing: dict of preallocated device tensors
        (topk_ids, topk_w, logits, counts, offsets, pairs) to receive the routing. stages: a
        subset of MOE_ROUTE | MOE_EXPERTS | MOE_COMBINE (tq_moe_ffn_stages); the same ws must
        then be passed to the calls that run the later stages."""
        T = x.shape[0]
        if out is None and stages & MOE_COMBINE:
            out = torch.empty_like(x)
        if ws is None:
            need = self.workspace_bytes(T)
            ws = workspace(need, x.device, "moe") if need else None
        r = None
        if routing is not None:
            r = MoeRouting(*[(routing[f].data_ptr() if routing.get(f) is not None else None)
                             for f, _ in MoeRouting._fields_])
        nbytes = 0 if ws is None else ws.numel() * ws.element_size()
        rr = C.byref(r) if r is not None else None
        if stages == MOE_ALL:
            _check(lib().tq_moe_ffn(C.byref(self.desc), x.data_ptr(), T, out.data_ptr(),
                                    _ptr(ws), nbytes, rr, _stream(stream)))
        else:
            _check(lib().tq_moe_ffn_stages(C.byref(self.desc), x.data_ptr(), T, _ptr(out),
                                           _ptr(ws), nbytes, rr, stages, _stream(stream)))
        return out


class ExpertCache:
    """The device slots and host state of a residency cache (tq_expert_cache_init) for one
    host-resident MoE layer. Keeps its memory alive; close() releases the state's events."""

    def __init__(self, layer: MoeLayer, slots: int, prefetch: int = 0):
        L = lib()
        nstate = int(L.tq_expert_cache_state_bytes(C.byref(layer.desc), slots))
        nslot = int(L.tq_expert_cache_slot_bytes(C.byref(layer.desc)))
        if not nstate or not nslot:
            raise TQError(1, "invalid layer descriptor or slot count for an expert cache")
        self._state = (C.c_char * (nstate + 64))()  # host memory, 64-byte aligned below
        base = C.addressof(self._state)
        self.state_ptr = (base + 63) & ~63
        self.slots = torch.empty(slots * nslot, dtype=torch.uint8, device=layer.router_w.device)
        _check(L.tq_expert_cache_init(self.state_ptr, nstate, C.byref(layer.desc), slots, prefetch,
                                      self.slots.data_ptr(), self.slots.numel()))
        self.open = True

    def stats(self) -> dict:
        s = ExpertCacheStats()
        _check(lib().tq_expert_cache_stats_get(self.state_ptr, C.byref(s)))
        return {f: getattr(s, f) for f, _ in ExpertCacheStats._fields_}

    def close(self) -> None:
        if self.open:
            torch.cuda.synchronize()
            _check(lib().tq_expert_cache_destroy(self.state_ptr))
            self.open = False


# ---- a paged key/value cache held in 4 bits (tq_kv_*) --------------------------------------------

ACT_TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _kv_refuse(t, name: str, dtype, shape, device, strided: bool):
    """Says what is wrong with a tensor argument that _kv_tensor found wrong."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if len(shape) != t.dim() or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must have the shape {list(shape)}, not {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    raise ValueError(f"the last dimension of {name} must be dense" if strided
                     else f"{name} must be contiguous")


def _kv_tensor(t, name: str, dtype, shape, device, strided: bool = False):
    """Checks a tensor argument of a tq_kv_* call: dtype, shape (None in it: any size), device,
    density (strided: of the last dimension only). These calls take microseconds on the device, so
    the checks are one expression."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device
            and (t.shape == shape or (None in shape and len(shape) == t.dim()
                                      and all(w is None or w == n for w, n in zip(shape, t.shape))))
            and (t.is_contiguous() or (strided and (t.stride(-1) == 1 or t.shape[-1] <= 1 or not t.numel())))):
        return t
    _kv_refuse(t, name, dtype, shape, device, strided)


_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


class _On:
    """The cache's device and the call's stream as the current ones: outputs and workspaces that a
    call makes then belong to the stream that uses them."""

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {device}")
        self.ctx = torch.cuda.stream(stream) if stream is not None else torch.cuda.device(device)

    def __enter__(self):
        return self.ctx.__enter__()

    def __exit__(self, *exc):
        return self.ctx.__exit__(*exc)


def _elsewhere(device, stream) -> bool:
    """Whether a call has to change the current device or stream first (_On)."""
    if device.type != "cuda":
        raise ValueError(f"the cache is on {device}, not on a GPU")
    return stream is not None or _current_device() != device.index


class KvCache:
    """Pages of keys and values held as 4-bit blocks (tq_kv_cache). Makes its memory (`pages` on
    `device`; uint8 [pages, page bytes], contents irrelevant until written) or takes `data`.
    head_dim 64, 96, 128 or 256; page_tokens 16, 32, ... 1024."""

    def __init__(self, kv_heads: int, head_dim: int, page_tokens: int, pages: int | None = None,
                 data: torch.Tensor | None = None, device=None):
        d = KvCacheDesc(kv_heads, head_dim, page_tokens, 1, None)
        self.page_bytes = int(lib().tq_kv_page_bytes(C.byref(d)))
        if not self.page_bytes:
            raise ValueError(f"a cache of {kv_heads} heads of {head_dim} in pages of {page_tokens} "
                             "tokens is not supported")
        if (pages is None) == (data is None):
            raise ValueError("give either pages or data")
        if data is None:
            data = torch.empty((pages, self.page_bytes), dtype=torch.uint8,
                               device=device if device is not None else "cuda")
        else:
            _kv_tensor(data, "data", torch.uint8, (None, self.page_bytes), data.device)
        self.kv_heads, self.head_dim, self.page_tokens = kv_heads, head_dim, page_tokens
        self.data, self.pages, self.device = data, data.shape[0], data.device
        d.pages, d.data = self.pages, data.data_ptr()
        self.desc = d
        self.ref = C.byref(d)
        self.attn_bytes: dict = {}  # workspace sizes of kv_attention by what they depend on


class Rope:
    """Rotary positions: inv_freq fp32 [pairs]; sections: how many pairs take their position from
    each axis (default: all from one); interleaved: pairs (2p, 2p + 1), else (p, p + pairs)."""

    def __init__(self, inv_freq: torch.Tensor, sections=None, interleaved: bool = False):
        if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a dense fp32 vector")
        self.inv_freq, self.pairs = inv_freq, inv_freq.shape[0]
        self.sections = [self.pairs] if sections is None else [int(n) for n in sections]
        if not 1 <= len(self.sections) <= 4 or min(self.sections) < 0 or sum(self.sections) != self.pairs:
            raise ValueError(f"sections {self.sections} must be 1 to 4 counts that add up to {self.pairs}")
        self.interleaved = bool(interleaved)
        self.desc = RopeDesc(inv_freq.data_ptr(), None, 0, self.pairs, len(self.sections),
                             (_i64 * 4)(*self.sections), int(interleaved))


def _head_rows(t: torch.Tensor, heads: int) -> HeadRows:
    rows, head, _ = t.stride()
    return HeadRows(t.data_ptr(), heads, rows, head)


def _heads_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a tensor of rows, heads and head_dim")
    return t.shape[1]


def kv_plan(cache: KvCache, kv_len: torch.Tensor, new_len: torch.Tensor, block_table: torch.Tensor,
            rows: int, free_pages: torch.Tensor | None = None,
            free_count: torch.Tensor | None = None, stream=None) -> dict:
    """Tables, slots and positions of a step from its requests' lengths (tq_kv_plan): new_len[r]
    more tokens for request r, or -1 when it has ended. block_table [requests, max_blocks] and
    free_pages [pages] are updated in place (free_pages None: the table already holds the new
    tokens' pages). Returns a dict with block_table, cu_new, seq_len, slots, positions, requests
    (int32; -1 in the rows after the last token), free_pages, free_count (the new one) and status
    [1], on the device: 0, or the sum of reasons why nothing was done (1 pages, 2 rows, 4 table
    columns, 8 lengths)."""
    R, dev, i32 = kv_len.numel(), cache.device, torch.int32
    _kv_tensor(kv_len, "kv_len", i32, (R,), dev)
    _kv_tensor(new_len, "new_len", i32, (R,), dev)
    _kv_tensor(block_table, "block_table", i32, (R, block_table.shape[-1]), dev)
    if (free_pages is None) != (free_count is None):
        raise ValueError("free_pages and free_count go together")
    if free_pages is not None:
        _kv_tensor(free_pages, "free_pages", i32, (cache.pages,), dev)
        _kv_tensor(free_count, "free_count", i32, (1,), dev)
    if rows < 0:
        raise ValueError("rows must not be negative")
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return kv_plan(cache, kv_len, new_len, block_table, rows, free_pages, free_count)
    out = torch.empty(2 * R + 3 + 3 * rows, dtype=i32, device=dev)
    cu, seq, count, status, slots, pos, req = out.split((R + 1, R, 1, 1, rows, rows, rows))
    base = out.data_ptr()
    at = base + 4 * (2 * R + 3)
    managed = free_pages is not None
    d = KvStepDesc(R, block_table.shape[1], rows, kv_len.data_ptr(), new_len.data_ptr(),
                   block_table.data_ptr(), free_pages.data_ptr() if managed else None,
                   free_count.data_ptr() if managed else None, base, base + 4 * (R + 1),
                   at if rows else None, at + 4 * rows if rows else None,
                   at + 8 * rows if rows else None, base + 4 * (2 * R + 1) if managed else None,
                   base + 4 * (2 * R + 2))
    rc = lib().tq_kv_plan(cache.ref, C.byref(d), _raw_stream(dev.index))
    if rc:
        _check(rc)
    res = {"block_table": block_table, "cu_new": cu, "seq_len": seq, "slots": slots,
           "positions": pos, "requests": req, "status": status}
    if managed:
        res["free_pages"], res["free_count"] = free_pages, count
    return res


def kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
              q: torch.Tensor | None = None, rope: Rope | None = None,
              positions: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
              stream=None):
    """Rounds the rows k, v [rows, kv_heads, head_dim] (fp32, bf16 or fp16; rows and heads at any
    stride) into their slots, keys and the queries q [rows, heads, head_dim] turned by `rope` at
    `positions` (int32 [rows] or [axes, rows]) (tq_kv_append). Returns the turned queries (q_out,
    which may be q; rows with slot -1 are left as they were), or None without q."""
    dev, D = cache.device, cache.head_dim
    if not isinstance(k, torch.Tensor) or k.dtype not in ACT_TYPES:
        raise ValueError("k must be a tensor of fp32, bf16 or fp16")
    rows = k.shape[0]
    shape = (rows, cache.kv_heads, D)
    _kv_tensor(k, "k", k.dtype, shape, dev, True)
    _kv_tensor(v, "v", k.dtype, shape, dev, True)
    _kv_tensor(slots, "slots", torch.int32, (rows,), dev)
    if (rope is None) != (positions is None):
        raise ValueError("rope and positions go together")
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    if q is not None and rope is None:
        raise ValueError("q needs a rope")
    r = None
    if rope is not None:
        if rope.inv_freq.device != dev:
            raise ValueError(f"inv_freq is on {rope.inv_freq.device}, the cache on {dev}")
        axes = len(rope.sections)
        if isinstance(positions, torch.Tensor) and positions.dim() == 1 and axes == 1:
            positions = positions[None]
        _kv_tensor(positions, "positions", torch.int32, (axes, rows), dev, strided=True)
        r = RopeDesc.from_buffer_copy(rope.desc)
        r.positions, r.axis_stride = positions.data_ptr(), positions.stride(0) if axes > 1 else 0
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return kv_append(cache, k, v, slots, q, rope, positions, q_out)
    qr = orr = None
    if q is not None:
        heads = _heads_of(q, "q")
        shape = (rows, heads, D)
        _kv_tensor(q, "q", k.dtype, shape, dev, True)
        if q_out is None:
            q_out = torch.empty(shape, dtype=k.dtype, device=dev)
        else:
            _kv_tensor(q_out, "q_out", k.dtype, shape, dev, True)
        qr, orr = C.byref(_head_rows(q, heads)), C.byref(_head_rows(q_out, heads))
    if rows:
        rc = lib().tq_kv_append(cache.ref, ACT_TYPES[k.dtype], rows, slots.data_ptr(),
                                C.byref(_head_rows(k, cache.kv_heads)),
                                C.byref(_head_rows(v, cache.kv_heads)), qr, orr,
                                None if r is None else C.byref(r), _raw_stream(dev.index))
        if rc:
            _check(rc)
    return q_out


def kv_read(cache: KvCache, slots: torch.Tensor, dtype: torch.dtype = torch.float32, stream=None):
    """The keys and values at `slots` (int32 [rows]) as the values they stand for, two tensors
    [rows, kv_heads, head_dim] of `dtype` (tq_kv_read); zeros for slots outside the cache."""
    dev = cache.device
    _kv_tensor(slots, "slots", torch.int32, (slots.numel(),), dev)
    if dtype not in ACT_TYPES:
        raise ValueError("dtype must be fp32, bf16 or fp16")
    rows = slots.numel()
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return kv_read(cache, slots, dtype)
    k = torch.empty((rows, cache.kv_heads, cache.head_dim), dtype=dtype, device=dev)
    v = torch.empty_like(k)
    if rows:
        rc = lib().tq_kv_read(cache.ref, ACT_TYPES[dtype], rows, slots.data_ptr(), k.data_ptr(),
                              v.data_ptr(), _raw_stream(dev.index))
        if rc:
            _check(rc)
    return k, v


def kv_attention(cache: KvCache, q: torch.Tensor, block_table: torch.Tensor, seq_len: torch.Tensor,
                 cu_new: torch.Tensor, scale: float | None = None, window: int = 0,
                 out: torch.Tensor | None = None, return_lse: bool = False,
                 ws: torch.Tensor | None = None, stream=None):
    """Softmax attention of q [rows, heads, head_dim] over the cache (tq_kv_attention): rows
    cu_new[r] .. cu_new[r + 1] are the last tokens of request r, whose seq_len[r] tokens (their
    own included) lie in the pages block_table[r]. scale: default head_dim ** -0.5; window: tokens
    a row sees, itself included (0: all). Returns out (q's type), or (out, lse) with lse fp32
    [rows, heads]. Rows outside cu_new are left as they were in `out` (undefined in a new one)."""
    dev, D, i32 = cache.device, cache.head_dim, torch.int32
    if not isinstance(q, torch.Tensor) or q.dtype not in ACT_TYPES:
        raise ValueError("q must be a tensor of fp32, bf16 or fp16")
    heads = _heads_of(q, "q")
    rows = q.shape[0]
    shape = (rows, heads, D)
    _kv_tensor(q, "q", q.dtype, shape, dev, True)
    if heads == 0 or heads % cache.kv_heads:
        raise ValueError(f"{heads} heads of q are no multiple of the cache's {cache.kv_heads}")
    R = seq_len.numel()
    _kv_tensor(seq_len, "seq_len", i32, (R,), dev)
    mb = block_table.shape[-1]
    _kv_tensor(block_table, "block_table", i32, (R, mb), dev)
    _kv_tensor(cu_new, "cu_new", i32, (R + 1,), dev)
    t = ACT_TYPES[q.dtype]
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return kv_attention(cache, q, block_table, seq_len, cu_new, scale, window, out,
                                return_lse, ws)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=dev)
    else:
        _kv_tensor(out, "out", q.dtype, shape, dev, True)
    lse = torch.empty((rows, heads), dtype=torch.float32, device=dev) if return_lse else None
    d = KvAttnDesc(rows, R, mb, _head_rows(q, heads), _head_rows(out, heads), _ptr(lse), block_table.data_ptr(),
                   seq_len.data_ptr(), cu_new.data_ptr(), D ** -0.5 if scale is None else scale,
                   window)
    ref = C.byref(d)
    if ws is None:  # of the calling stream: calls on other streams, and graphs, have their own
        need = cache.attn_bytes.get((t, rows, R, heads, mb))
        if need is None:
            need = int(lib().tq_kv_attention_workspace_bytes(cache.ref, t, ref))
            if need:  # 0: an argument that the call below refuses
                cache.attn_bytes[t, rows, R, heads, mb] = need
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    rc = lib().tq_kv_attention(cache.ref, t, ref, ws.data_ptr() or None,
                               ws.numel() * ws.element_size(), _raw_stream(dev.index))
    if rc:
        _check(rc)
    return (out, lse) if return_lse else out


# Tuning knobs (TQ_KNOB_* of tq.h), for tests and tuning sweeps: the defaults are the production
# choices; an override changes which kernel or launch shape a call takes.
KNOBS = {
    "gemv_target_wg": 0,
    "gemv_max_waves": 1,
    "gemv_klane": 2,
    "kl_groups": 3,
    "kl_rows": 4,
    "kl_target_waves": 5,
    "gemm_f32m": 6,
    "f32m_upk": 7,
    "gemv_i8": 8,
    "i8_upk": 9,
    "moe_qmm": 10,
    "qmm_nt": 11,
    "moe_nt": 12,
    "router_kl": 13,
    "router_steps": 14,
    "router_mf": 15,
    "group1": 16,
    "combine4": 17,
    "fuse_combine": 18,
    "gemv_qmm": 19,
    "qmm_upk": 20,
    "qmm_inline": 21,
    "qmm_inline_upk": 22,
    "qmm_inline_nr": 23,
    "gemv_mf": 24,
    "mf_wgs": 25,
    "mf_kb": 26,
    "mf_deep": 27,
    "moe_mf": 28,
    "moe_route1": 29,
    "f32m_t4": 30,
    "mf_ksplit": 31,
}


def set_knob(name: str, value: int) -> None:
    """Override a tuning knob process-wide (value < 0: back to the default)."""
    _check(lib().tq_tuning_set(KNOBS[name], int(value)))


def get_knob(name: str) -> int:
    """The knob's override, or -1 while its default is in effect."""
    return int(lib().tq_tuning_get(KNOBS[name]))


class knobs:
    """Context manager: knobs(gemv_i8=2, kl_rows=2) sets overrides and restores the previous
    values on exit."""

    def __init__(self, **values):
        self.values = values

    def __enter__(self):
        self.old = {k: get_knob(k) for k in self.values}
        for k, v in self.values.items():
            set_knob(k, v)
        return self

    def __exit__(self, *exc):
        for k, v in self.old.items():
            set_knob(k, v)
        return False
