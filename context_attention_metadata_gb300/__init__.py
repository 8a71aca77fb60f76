"""Python binding of libmarble: exact mask-aware blockwise attention over packed
multimodal sequences with the online-softmax state carried in fp32 across KV shards.

This module only marshals arguments to the C ABI declared in ``include/marble.h``; every
step of the computation runs in the library's CUDA kernels.  PyTorch provides device
memory and streams.  There is no CPU fallback: importing works without a GPU, but every
call needs the built library (``__graft_entry__.build()``) and a CUDA device.

Sources (page title and section): "MARBLE: exact sequence parallelism for packed
multimodal masks" s01 (tracks and mask), s03 (block classification, PTRR, exact ring
accumulation), s04 (sparse all-to-all, layout transforms).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Dict, Optional

# The library queues work on up to five streams of its own (four side streams and a teardown
# stream) beside the caller's.  With CUDA's default of 8 hardware work queues, streams share
# queues, and work on one waits behind unrelated work on another: in a training loop the
# input and output copies then wait for the attention kernels.  More queues are asked for
# here, before the CUDA context exists, unless the caller chose a value; it has no effect if
# the process created its CUDA context before importing this module.
os.environ.setdefault("CUDA_DEVICE_MAX_CONNECTIONS", "32")

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libmarble.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_OOM, ERR_TIMEOUT = range(6)
BLOCK = 128
WINDOW_INF = 2147483647
TILE_FULL, TILE_PARTIAL = 1, 2
KV_NEEDED = -1
STEP_FIRST = 1
STEP_BF16_MERGE = 2  # standard ring merge in bf16 (the comparison baseline)
STEP_FP32_MERGE = 4  # merge of fp32 partials by their LSE
_MERGE = {None: 0, "carried": 0, "bf16": STEP_BF16_MERGE, "fp32": STEP_FP32_MERGE}
ORDERS = {"contiguous": 0, "ptrr_block": 1, "ptrr_chunk": 2, "chunk_search": 3}
FIELDS = {
    "perm": (0, "int32"), "block_perm": (1, "int32"), "tracks_perm": (2, "int32"),
    "tile_rowptr": (3, "int64"), "tile_col": (4, "int32"), "tile_tag": (5, "uint8"),
    "step_ptr": (6, "int64"), "step_col": (7, "int32"), "step_tag": (8, "uint8"),
    "colT_ptr": (9, "int64"), "colT_row": (10, "int32"), "colT_tag": (11, "uint8"),
    "needed_ptr": (12, "int64"), "needed": (13, "int32"),
    "key_intervals": (14, "int32"), "interval_blocks": (15, "uint8"),
}


class MarbleError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"marble error {status}: {msg}")
        self.status = status


class _PlanDesc(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("sample_id", ctypes.c_void_p),
                ("seg_id", ctypes.c_void_p), ("noise_id", ctypes.c_void_p),
                ("window", ctypes.c_int32), ("num_shards", ctypes.c_int32),
                ("order", ctypes.c_int32), ("chunk_tokens", ctypes.c_int32),
                ("range_cost", ctypes.c_int64), ("no_key_intervals", ctypes.c_int32),
                ("pos_id", ctypes.c_void_p)]


class _PlanStats(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int64) for name in (
        "n_tokens", "n_blocks", "num_shards", "nnz", "n_full", "n_partial", "legal_pairs",
        "shard_cost_max", "shard_cost_sum", "step_cost", "needed_total", "needed_remote",
        "chunks_per_rank", "layout_cost", "layout_step_cost", "step_cost_pairs")]


class _QKV(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("scale", ctypes.c_float)]


PAIRINGS = {"halves": 0, "adjacent": 1}
ROPE_WORKSPACE_BYTES = 1048576


class _Rope(ctypes.Structure):
    _fields_ = [("n_axes", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("pairing", ctypes.c_int32), ("inv_freq", ctypes.c_void_p),
                ("axis", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class _Heads(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32),
                ("d", ctypes.c_int32)]


class _State(ctypes.Structure):
    _fields_ = [("o_acc", ctypes.c_void_p), ("m", ctypes.c_void_p), ("l", ctypes.c_void_p)]


class _Score(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("slopes", ctypes.c_void_p)]


_lib = None

# every symbol the header declares, with its ctypes signature
_SIGS = {
    "marble_plan": ([ctypes.POINTER(_PlanDesc), ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]),
    "marble_plan_destroy": ([ctypes.c_void_p]),
    "marble_plan_stats": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(_PlanStats)]),
    "marble_layout_vision_groups": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                     ctypes.c_void_p]),
    "marble_chunk_layout_search": ([ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                    ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "marble_plan_field_bytes": ([ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "marble_plan_export": ([ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t,
                            ctypes.c_void_p]),
    "marble_permute": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                        ctypes.c_int32, ctypes.c_void_p]),
    "marble_permute_cast_bf16": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p]),
    "marble_release_memory": ([]),
    "marble_rope": ([ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_Rope),
                     ctypes.POINTER(_Heads), ctypes.POINTER(_Heads), ctypes.c_void_p]),
    "marble_rope_bwd": ([ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_Rope),
                         ctypes.POINTER(_Heads), ctypes.POINTER(_Heads), ctypes.POINTER(_Heads),
                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "marble_attn_step": ([ctypes.c_void_p, ctypes.POINTER(_QKV), ctypes.c_int32, ctypes.c_int32,
                          ctypes.POINTER(_State), ctypes.c_uint32, ctypes.c_void_p]),
    "marble_attn_finalize": ([ctypes.c_void_p, ctypes.POINTER(_State), ctypes.c_int32,
                              ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "marble_attn_bwd_prep": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                              ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]),
    "marble_attn_bwd": ([ctypes.c_void_p, ctypes.POINTER(_QKV), ctypes.c_void_p, ctypes.c_void_p,
                         ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]),
    "marble_attn_steps": ([ctypes.c_void_p, ctypes.POINTER(_QKV), ctypes.c_int32,
                           ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                           ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(_State),
                           ctypes.c_void_p]),
    "marble_attn_bwd_steps": ([ctypes.c_void_p, ctypes.POINTER(_QKV), ctypes.c_void_p,
                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                               ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                               ctypes.c_void_p]),
    "marble_attn_fwd_fused": ([ctypes.c_void_p, ctypes.POINTER(_QKV), ctypes.POINTER(_State),
                               ctypes.c_void_p]),
    "marble_attn_bwd_fused": ([ctypes.c_void_p, ctypes.POINTER(_QKV), ctypes.c_void_p,
                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "marble_attn_steps_scored": ([ctypes.c_void_p, ctypes.POINTER(_QKV), ctypes.POINTER(_Score),
                                  ctypes.c_int32, ctypes.POINTER(ctypes.c_int32),
                                  ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_uint32),
                                  ctypes.POINTER(_State), ctypes.c_void_p]),
    "marble_attn_fwd_fused_scored": ([ctypes.c_void_p, ctypes.POINTER(_QKV),
                                      ctypes.POINTER(_Score), ctypes.POINTER(_State),
                                      ctypes.c_void_p]),
    "marble_attn_bwd_steps_scored": ([ctypes.c_void_p, ctypes.POINTER(_QKV),
                                      ctypes.POINTER(_Score), ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_int32,
                                      ctypes.POINTER(ctypes.c_int32),
                                      ctypes.POINTER(ctypes.c_int32), ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "marble_attn_bwd_fused_scored": ([ctypes.c_void_p, ctypes.POINTER(_QKV),
                                      ctypes.POINTER(_Score), ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p]),
    "marble_cast_bf16": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "marble_check": ([ctypes.c_void_p, ctypes.c_void_p]),
    "marble_set_wait_limit_ns": ([ctypes.c_uint64]),
    "marble_set_side_streams": ([ctypes.c_int32]),
    "marble_debug_wait_timeout": ([ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]),
    "marble_timing_enable": ([ctypes.c_int]),
    "marble_timing_read": ([ctypes.c_void_p]),
    "marble_tile_map_static": ([ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                ctypes.c_void_p]),
    "marble_last_error": ([]),
    "marble_version": ([]),
}


def lib():
    """Load libmarble.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_char_p if name in ("marble_last_error", "marble_version") \
                else ctypes.c_int
        _lib = L
    return _lib


def _call(name, *args):
    st = getattr(_lib or lib(), name)(*args)
    if st != OK:
        raise MarbleError(st, lib().marble_last_error().decode())


def _raw_stream(torch, stream, index=None):
    """The stream's handle; None: the current stream of GPU ``index`` (None: the current GPU).
    That one is read directly where this torch has the (private) call for it: building the stream
    object costs a single-token call as much as its kernel takes."""
    if stream is not None:
        return stream.cuda_stream
    direct = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if direct is None:
        return torch.cuda.current_stream(index).cuda_stream
    return direct(torch.cuda.current_device() if index is None else index)


def _stream(stream):
    import torch
    return ctypes.c_void_p(_raw_stream(torch, stream))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _need(t, dtype, name, shape=None):
    if getattr(t, "dtype", None) is dtype and t.is_cuda and t.is_contiguous() and \
            (shape is None or t.shape == shape):
        return
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


class Plan:
    """A plan: tile map, token order, per-step lists and needed-KV index of one pack.

    sample/seg/noise: int32 CUDA tensors [N] in original token order (see marble.h)."""

    def __init__(self, sample, seg, noise, window: int, num_shards: int,
                 order: str = "contiguous", chunk_tokens: int = 0, stream=None,
                 range_cost: int = 0, key_intervals: bool = True, pos=None):
        import torch
        for t, nm in ((sample, "sample"), (seg, "seg"), (noise, "noise")):
            _need(t, torch.int32, nm, (sample.shape[0],))
        if pos is not None:
            _need(pos, torch.int32, "pos", (sample.shape[0],))
        self.n = int(sample.shape[0])
        self.num_shards = int(num_shards)
        self.window = int(window)
        self.order = order
        d = _PlanDesc(self.n, sample.data_ptr(), seg.data_ptr(), noise.data_ptr(),
                      int(window), int(num_shards), ORDERS[order], int(chunk_tokens),
                      int(range_cost), 0 if key_intervals else 1,
                      pos.data_ptr() if pos is not None else None)
        h = ctypes.c_void_p()
        _call("marble_plan", ctypes.byref(d), _stream(stream), ctypes.byref(h))
        self._h = h
        self.n_blocks = self.n // BLOCK
        self.blocks_per_shard = self.n_blocks // self.num_shards

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().marble_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def stats(self, stream=None) -> Dict[str, int]:
        s = _PlanStats()
        _call("marble_plan_stats", self._h, _stream(stream), ctypes.byref(s))
        return {name: int(getattr(s, name)) for name, _ in _PlanStats._fields_}

    def export(self, field: str, stream=None):
        """Copy a plan field into a new CUDA tensor."""
        import torch
        fid, dt = FIELDS[field]
        nbytes = ctypes.c_size_t()
        _call("marble_plan_field_bytes", self._h, fid, ctypes.byref(nbytes))
        dtype = getattr(torch, dt)
        elem = torch.tensor([], dtype=dtype).element_size()
        out = torch.empty(nbytes.value // elem, dtype=dtype, device="cuda")
        _call("marble_plan_export", self._h, fid, ctypes.c_void_p(out.data_ptr() if out.numel() else 0),
              nbytes.value, _stream(stream))
        return out

    def permute(self, src, inverse: bool = False, out=None, stream=None):
        """Gather rows into plan order (inverse=False) or scatter back (inverse=True)."""
        import torch
        if not src.is_cuda or not src.is_contiguous() or src.shape[0] != self.n:
            raise ValueError("src must be a contiguous CUDA tensor with N rows")
        out = torch.empty_like(src) if out is None else out
        row_bytes = src.numel() // self.n * src.element_size()
        _call("marble_permute", self._h, _ptr(src), _ptr(out), row_bytes, 1 if inverse else 0,
              _stream(stream))
        return out

    def permute_cast_bf16(self, src, inverse: bool = True, out=None, stream=None):
        """permute() of an fp32 tensor, written as bf16 (round to nearest even)."""
        import torch
        _need(src, torch.float32, "src")
        if src.shape[0] != self.n:
            raise ValueError("src must have N rows")
        out = torch.empty(src.shape, dtype=torch.bfloat16, device=src.device) if out is None else out
        _need(out, torch.bfloat16, "out", src.shape)
        _call("marble_permute_cast_bf16", self._h, _ptr(src), _ptr(out), src.numel() // self.n,
              1 if inverse else 0, _stream(stream))
        return out

    def check(self, stream=None):
        _call("marble_check", self._h, _stream(stream))


def rope_frequencies(sections, theta: float = 10000.0, layout: str = "sections"):
    """(inv_freq float64 [pairs], axis int32 [pairs]) of rotary positions with len(sections)
    axes, sections[a] of the pairs belonging to axis a.  With pairs = sum(sections):

    "sections"     one sequence theta^(-i / pairs) over all pairs, the first sections[0] of
                   them turned by axis 0, the next by axis 1, ...
    "interleaved"  the same sequence, the axes taking turns pair by pair while theirs last
    "axial"        a sequence of its own for every axis: theta^(-j / sections[a]), axis by axis

    One axis is the usual rotary position in each of them."""
    import numpy as np
    sec = [int(x) for x in sections]
    if not sec or min(sec) < 0 or sum(sec) == 0:
        raise ValueError("sections must hold the pairs of every axis")
    if layout not in ("sections", "interleaved", "axial"):
        raise ValueError("layout must be 'sections', 'interleaved' or 'axial'")
    axis = np.repeat(np.arange(len(sec)), sec)
    i = np.concatenate([np.arange(x) for x in sec])
    if layout == "axial":
        return float(theta) ** -(i / np.repeat(sec, sec)), axis.astype(np.int32)
    if layout == "interleaved":
        axis = axis[np.lexsort((axis, i))]
    return float(theta) ** -(np.arange(len(axis)) / len(axis)), axis.astype(np.int32)


class Rope:
    """The frequencies of rotary positions: radians per position and the axis of every rotated
    pair (see marble.h), host arrays of rot_dim / 2 entries; axis None: all on axis 0.
    ``pairing``: "halves" pairs channels (i, i + rot_dim / 2), "adjacent" (2 i, 2 i + 1)."""

    def __init__(self, inv_freq, axis=None, pairing: str = "halves"):
        if pairing not in PAIRINGS:
            raise ValueError(f"pairing must be one of {sorted(PAIRINGS)}")
        self.pairing = pairing
        self._set(inv_freq, axis)

    def _set(self, inv_freq, axis):
        import numpy as np
        # copies: the caller's arrays may change after this
        freq = np.array(inv_freq, dtype=np.float64)
        axis = np.zeros(freq.shape, np.int32) if axis is None else np.array(axis, dtype=np.int32)
        if freq.ndim != 1 or axis.shape != freq.shape:
            raise ValueError("inv_freq and axis must be 1-D arrays of one length")
        self._freq, self._axis = freq, axis
        self._tables = (freq.ctypes.data, axis.ctypes.data)  # of these two arrays, no others

    # a copy (copy, pickle) has arrays, and with them addresses, of its own
    def __getstate__(self):
        return {"inv_freq": self._freq, "axis": self._axis, "pairing": self.pairing}

    def __setstate__(self, state):
        self.pairing = state["pairing"]
        self._set(state["inv_freq"], state["axis"])

    @property
    def inv_freq(self):
        return self._freq

    @inv_freq.setter
    def inv_freq(self, value):
        self._set(value, self._axis)

    @property
    def axis(self):
        return self._axis

    @axis.setter
    def axis(self, value):
        self._set(self._freq, value)

    @property
    def rot_dim(self):
        return 2 * len(self._freq)

    def _c(self, pos, q_weight, k_weight, eps):
        return _Rope(pos.shape[0], self.rot_dim, PAIRINGS[self.pairing], *self._tables,
                     pos.data_ptr(),
                     None if q_weight is None else q_weight.data_ptr(),
                     None if k_weight is None else k_weight.data_ptr(), float(eps))


def _heads(parts, n, dtype, index, what):
    """marble_heads_t of the tensors q, k, v in ``parts``, [n, heads, d] on GPU ``index`` (None:
    absent), whose tokens may be strided."""
    ptr, step, count = [None, None, None], [0, 0, 0], [0, 0, 0]
    d = 0
    for i, t in enumerate(parts):
        if t is None:
            continue
        try:
            (rows, heads, dd), (s0, s1, s2) = t.shape, t.stride()
            ok = t.dtype is dtype and t.is_cuda
        except (AttributeError, ValueError, TypeError):
            ok = False
        if not ok or t.get_device() != index:
            raise ValueError(f"{what}{'qkv'[i]} must be a {dtype} tensor [n, heads, d] on cuda:{index}")
        if rows != n or (d and dd != d) or (i == 2 and count[1] and heads != count[1]):
            raise ValueError(f"{what}{'qkv'[i]} has shape {tuple(t.shape)}: n, d or the kv heads "
                             "differ")
        if n > 0 and ((heads > 1 and s1 != dd) or s2 != 1):
            raise ValueError(f"{what}{'qkv'[i]}: the heads of a token must be contiguous")
        d, count[i], ptr[i], step[i] = dd, heads, t.data_ptr(), s0 if n > 1 else heads * dd
    return _Heads(*ptr, *step, count[0], count[1] or count[2], d)


def _rope_args(torch, pos, plan, q_weight, k_weight, first):
    """(n, GPU) of a rotary call, its small tensors checked."""
    try:
        n, d = pos.shape[1], first.shape[2]
        ok = pos.dim() == 2 and pos.dtype is torch.int32 and pos.is_cuda and pos.is_contiguous()
    except (AttributeError, IndexError):
        ok = False
    if not ok:
        raise ValueError("pos must be a contiguous int32 CUDA tensor [axes, n], q a tensor "
                         "[n, heads, d]")
    if plan is not None:
        if plan.handle is None:  # NULL would be "no plan": the tokens left in their order
            raise ValueError("the plan is closed")
        if n != plan.n:
            raise ValueError("pos must have the plan's N columns")
    index = pos.get_device()
    for w, nm in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _need(w, torch.float32, nm, (d,))
            if w.get_device() != index:
                raise ValueError(f"{nm} must be on cuda:{index}")
    return n, index


def _rope_out(torch, like, heads, out, n, dtype, index, what, stream):
    """(tensors, their marble_heads_t): ``out`` checked against the tensors it is for (``heads``:
    theirs), or new tensors like them, which belong to the stream that writes them."""
    if out is None:
        if stream is not None:
            with torch.cuda.stream(stream):
                return _rope_out(torch, like, heads, None, n, dtype, index, what, None)
        dense = torch.contiguous_format
        out = tuple([None if t is None else torch.empty_like(t, dtype=dtype, memory_format=dense)
                     for t in like])
        d, hq, hkv = heads.d, heads.hq, heads.hkv
        return out, _Heads(*[None if t is None else t.data_ptr() for t in out],
                           hq * d, hkv * d, hkv * d, hq, hkv, d)
    if len(out) != 3 or any((a is None) != (b is None) or (a is not None and a.shape != b.shape)
                            for a, b in zip(out, like)):
        raise ValueError("out must hold one tensor of the same shape for each of "
                         f"{what}q, {what}k and {what}v")
    return tuple(out), _heads(out, n, dtype, index, "out " + what)


def rope(rope: Rope, pos, q, k=None, v=None, plan: Optional[Plan] = None, q_weight=None,
         k_weight=None, eps: float = 1e-6, out=None, stream=None):
    """Rotary positions of q and k, after their heads' RMS norm where a weight is given, and the
    move of q, k and v into plan order, in one pass (marble_rope).

    pos: int32 [axes, n], original order.  q [n, hq, d], k and v [n, hkv, d]: bf16, original
    order, each token's heads contiguous (slices of a fused projection are fine); k and v may
    be None.  plan None: the order stays, any n, and ``out`` may be (q, k, v) itself.
    Returns (q, k, v) in plan order, ``out`` or new tensors."""
    import torch
    n, index = _rope_args(torch, pos, plan, q_weight, k_weight, q)
    bf16 = torch.bfloat16
    parts = (q, k, v)
    src = _heads(parts, n, bf16, index, "")
    out, dst = _rope_out(torch, parts, src, out, n, bf16, index, "", stream)
    c = rope._c(pos, q_weight, None if k is None else k_weight, eps)
    _call("marble_rope", None if plan is None else plan.handle, n, ctypes.byref(c),
          ctypes.byref(src), ctypes.byref(dst), _raw_stream(torch, stream, index))
    return out


def rope_bwd(rope: Rope, pos, dq, dk=None, dv=None, plan: Optional[Plan] = None, q=None, k=None,
             q_weight=None, k_weight=None, eps: float = 1e-6, out=None, stream=None):
    """The gradient of rope() (marble_rope_bwd): fp32 gradients dq, dk, dv of its results in
    plan order (the accumulators of backward()) to bf16 gradients of its inputs in original
    order, in one pass.  Where the forward had a norm weight, q / k are its inputs.
    Returns (dq, dk, dv, dq_weight, dk_weight), the first three in ``out`` (a token's heads
    contiguous: slices of a fused gradient are fine) or new tensors, the weights' fp32 or None."""
    import torch
    n, index = _rope_args(torch, pos, plan, q_weight, k_weight, dq)
    bf16 = torch.bfloat16
    if dk is None:
        k_weight = None
    parts = (dq, dk, dv)
    grad = _heads(parts, n, torch.float32, index, "d")
    out, dx = _rope_out(torch, parts, grad, out, n, bf16, index, "d", stream)
    dwq = dwk = ws = x = None
    if q_weight is not None or k_weight is not None:
        for w, t, g, nm in ((q_weight, q, dq, "q"), (k_weight, k, dk, "k")):
            if w is not None and (t is None or t.shape != g.shape):
                raise ValueError(f"{nm}, the input of rope(), is needed for the norm's gradient")
        x = _heads((q if q_weight is not None else None, k if k_weight is not None else None, None),
                   n, bf16, index, "")
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            dwq = None if q_weight is None else torch.empty_like(q_weight)
            dwk = None if k_weight is None else torch.empty_like(k_weight)
            ws = pos.new_empty(ROPE_WORKSPACE_BYTES, dtype=torch.uint8)
    c = rope._c(pos, q_weight, k_weight, eps)
    _call("marble_rope_bwd", None if plan is None else plan.handle, n, ctypes.byref(c),
          None if x is None else ctypes.byref(x), ctypes.byref(grad), ctypes.byref(dx),
          None if dwq is None else _ptr(dwq), None if dwk is None else _ptr(dwk),
          None if ws is None else _ptr(ws), _raw_stream(torch, stream, index))
    return (*out, dwq, dwk)


class State:
    """fp32 online-softmax state (O_acc [N, hq, d], m [hq, N], l [hq, N]), plan order."""

    def __init__(self, n, hq, d, device="cuda"):
        import torch
        self.o_acc = torch.empty((n, hq, d), dtype=torch.float32, device=device)
        self.m = torch.empty((hq, n), dtype=torch.float32, device=device)
        self.l = torch.empty((hq, n), dtype=torch.float32, device=device)

    def _c(self):
        return _State(self.o_acc.data_ptr(), self.m.data_ptr(), self.l.data_ptr())


def _qkv(plan, q, k, v, scale):
    import torch
    n = plan.n
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k, v must be [N, heads, d]")
    hq, d = q.shape[1], q.shape[2]
    hkv = k.shape[1]
    _need(q, torch.bfloat16, "q", (n, hq, d))
    _need(k, torch.bfloat16, "k", (n, hkv, d))
    _need(v, torch.bfloat16, "v", (n, hkv, d))
    return _QKV(q.data_ptr(), k.data_ptr(), v.data_ptr(), hq, hkv, d, float(scale))


class Score:
    """What happens to a score before the softmax (marble_score_t): ``cap`` c > 0 makes it
    c tanh(score / c), ``slopes`` (fp32 CUDA tensor [hq], 16-byte aligned: a slice of a longer table
    may need a clone()) then takes slopes[h] * |pos_q - pos_k| off.  The same Score goes to every
    call of a pass, forward and backward."""

    def __init__(self, cap: float = 0.0, slopes=None):
        import torch
        if slopes is not None:
            _need(slopes, torch.float32, "slopes")
            if slopes.dim() != 1:
                raise ValueError("slopes must be [hq]")
        self.cap = float(cap)
        self.slopes = slopes

    def _c(self, hq):
        if self.slopes is not None and self.slopes.shape[0] != hq:
            raise ValueError(f"slopes must have {hq} entries, one for each q head")
        return _Score(self.cap, None if self.slopes is None else self.slopes.data_ptr())


def _call_scored(name, plan, c, score, *args):
    """The call, or its scored variant."""
    if score is None:
        _call(name, plan.handle, ctypes.byref(c), *args)
    else:
        _call(name + "_scored", plan.handle, ctypes.byref(c), ctypes.byref(score._c(c.hq)), *args)


def _flags(first: bool, merge) -> int:
    if merge not in _MERGE:
        raise ValueError(f"merge must be one of {sorted(k for k in _MERGE if k)}")
    return (STEP_FIRST if first else 0) | _MERGE[merge]


def attn_step(plan: Plan, q, k, v, q_shard: int, kv_shard: int, state: State,
              first: bool = False, scale: float = 0.0, stream=None, merge: str = "carried",
              score: Optional[Score] = None):
    """One forward ring step (marble_attn_step).  ``merge``: "carried" (the fp32 state
    carried across steps), "bf16" (the standard per-step merge of bf16 partials) or "fp32"
    (the same merge of fp32 partials).  ``score``: cap and distance bias of the scores."""
    if score is not None:
        attn_steps(plan, q, k, v, [(q_shard, kv_shard, first)], state, scale=scale, stream=stream,
                   merge=merge, score=score)
        return
    c = _qkv(plan, q, k, v, scale)
    st = state._c()
    _call("marble_attn_step", plan.handle, ctypes.byref(c), int(q_shard), int(kv_shard),
          ctypes.byref(st), _flags(first, merge), _stream(stream))


def attn_finalize(plan: Plan, state: State, o, lse, stream=None):
    import torch
    n, hq, d = state.o_acc.shape
    _need(o, torch.bfloat16, "o", (n, hq, d))
    _need(lse, torch.float32, "lse", (hq, n))
    st = state._c()
    _call("marble_attn_finalize", plan.handle, ctypes.byref(st), hq, d, _ptr(o), _ptr(lse),
          _stream(stream))


def attn_bwd_prep(plan: Plan, o, do, delta, stream=None):
    import torch
    n, hq, d = o.shape
    _need(o, torch.bfloat16, "o")
    _need(do, torch.bfloat16, "do", o.shape)
    _need(delta, torch.float32, "delta", (hq, n))
    _call("marble_attn_bwd_prep", plan.handle, _ptr(o), _ptr(do), hq, d, _ptr(delta),
          _stream(stream))


def attn_bwd(plan: Plan, q, k, v, do, lse, delta, q_shard: int, kv_shard: int, dq_acc, dk_acc,
             dv_acc, scale: float = 0.0, stream=None, score: Optional[Score] = None):
    """One backward ring step (marble_attn_bwd); accumulators are fp32 and caller-zeroed."""
    import torch
    if score is not None:
        attn_bwd_steps(plan, q, k, v, do, lse, delta, [(q_shard, kv_shard, False)], dq_acc, dk_acc,
                       dv_acc, scale=scale, stream=stream, score=score)
        return
    c = _qkv(plan, q, k, v, scale)
    _need(do, torch.bfloat16, "do", q.shape)
    _need(lse, torch.float32, "lse", (q.shape[1], plan.n))
    _need(delta, torch.float32, "delta", (q.shape[1], plan.n))
    _need(dq_acc, torch.float32, "dq_acc", q.shape)
    _need(dk_acc, torch.float32, "dk_acc", k.shape)
    _need(dv_acc, torch.float32, "dv_acc", k.shape)
    _call("marble_attn_bwd", plan.handle, ctypes.byref(c), _ptr(do), _ptr(lse), _ptr(delta),
          int(q_shard), int(kv_shard), _ptr(dq_acc), _ptr(dk_acc), _ptr(dv_acc), 0,
          _stream(stream))


def cast_bf16(src, dst, stream=None):
    import torch
    _need(src, torch.float32, "src")
    _need(dst, torch.bfloat16, "dst", src.shape)
    _call("marble_cast_bf16", _ptr(src), _ptr(dst), src.numel(), _stream(stream))


def set_wait_limit_ns(ns: int):
    _call("marble_set_wait_limit_ns", int(ns))


def release_memory():
    """Give the memory the library keeps for reuse (cached dS scratch of destroyed plans, the
    pool's unused blocks) back to the current device."""
    _call("marble_release_memory")


def set_side_streams(n: int):
    """Cap the side streams the step-list calls use (0: all launches on the caller's
    stream, in list order)."""
    _call("marble_set_side_streams", int(n))


def timing_enable(on: bool = True):
    """Per-kernel device timing of later attention calls (CUDA events on each kernel's stream)."""
    _call("marble_timing_enable", 1 if on else 0)


def timing_read() -> dict:
    """Summed device ms and launch counts per kernel since the previous read."""
    buf = (ctypes.c_double * 6)()
    _call("marble_timing_read", ctypes.cast(buf, ctypes.c_void_p))
    return {"fwd_ms": buf[0], "fwd_launches": int(buf[1]), "dq_ms": buf[2],
            "dq_launches": int(buf[3]), "dkdv_ms": buf[4], "dkdv_launches": int(buf[5])}


def debug_wait_timeout(plan: Plan, limit_ns: int, stream=None):
    _call("marble_debug_wait_timeout", plan.handle, int(limit_ns), _stream(stream))


TILE_MAP_STATIC_MAX_TOKENS = 2097152


def tile_map_static(sample, seg, noise, window: int, row_ptr, col, tag, stream=None):
    """Global tile map into caller-provided CUDA tensors without any allocation by the
    library (marble_tile_map_static): row_ptr int64[nb+1], col int32[cap], tag uint8[cap]."""
    import torch
    n = int(sample.shape[0])
    for t, nm in ((sample, "sample"), (seg, "seg"), (noise, "noise")):
        _need(t, torch.int32, nm, (n,))
    _need(row_ptr, torch.int64, "row_ptr", (n // BLOCK + 1,))
    _need(col, torch.int32, "col")
    _need(tag, torch.uint8, "tag", (col.numel(),))
    _call("marble_tile_map_static", n, _ptr(sample), _ptr(seg), _ptr(noise), int(window),
          _ptr(row_ptr), _ptr(col), _ptr(tag), col.numel(), _stream(stream))


def ring_schedule(num_shards: int, needed: bool = False):
    """The (q_shard, kv_shard, first) calls of one pass: r-major, kv shard (r - s) mod P at
    step s (MARBLE s03 ring pairing); with ``needed`` one call per q shard."""
    P = num_shards
    if needed:
        return [(r, KV_NEEDED, True) for r in range(P)]
    return [(r, (r - s) % P, s == 0) for r in range(P) for s in range(P)]


def attn_steps(plan: Plan, q, k, v, schedule, state: State, scale: float = 0.0, stream=None,
               merge: str = "carried", score: Optional[Score] = None):
    """A list of forward ring steps [(q_shard, kv_shard, first), ...] in one C call."""
    c = _qkv(plan, q, k, v, scale)
    st = state._c()
    n = len(schedule)
    qs = (ctypes.c_int32 * n)(*[int(r) for r, _, _ in schedule])
    ks = (ctypes.c_int32 * n)(*[int(j) for _, j, _ in schedule])
    fl = (ctypes.c_uint32 * n)(*[_flags(f, merge) for _, _, f in schedule])
    _call_scored("marble_attn_steps", plan, c, score, n, qs, ks, fl, ctypes.byref(st),
                 _stream(stream))


def attn_bwd_steps(plan: Plan, q, k, v, do, lse, delta, schedule, dq_acc, dk_acc, dv_acc,
                   scale: float = 0.0, stream=None, score: Optional[Score] = None):
    """A list of backward ring steps [(q_shard, kv_shard, _), ...] in one C call."""
    import torch
    c = _qkv(plan, q, k, v, scale)
    _need(do, torch.bfloat16, "do", q.shape)
    _need(lse, torch.float32, "lse", (q.shape[1], plan.n))
    _need(delta, torch.float32, "delta", (q.shape[1], plan.n))
    _need(dq_acc, torch.float32, "dq_acc", q.shape)
    _need(dk_acc, torch.float32, "dk_acc", k.shape)
    _need(dv_acc, torch.float32, "dv_acc", k.shape)
    n = len(schedule)
    qs = (ctypes.c_int32 * n)(*[int(r) for r, _, _ in schedule])
    ks = (ctypes.c_int32 * n)(*[int(j) for _, j, _ in schedule])
    _call_scored("marble_attn_bwd_steps", plan, c, score, _ptr(do), _ptr(lse), _ptr(delta), n, qs,
                 ks, _ptr(dq_acc), _ptr(dk_acc), _ptr(dv_acc), _stream(stream))


def attn_fwd_fused(plan: Plan, q, k, v, state: State, scale: float = 0.0, stream=None,
                   score: Optional[Score] = None):
    """Every forward ring step in one launch, the state on chip between steps
    (marble_attn_fwd_fused)."""
    c = _qkv(plan, q, k, v, scale)
    st = state._c()
    _call_scored("marble_attn_fwd_fused", plan, c, score, ctypes.byref(st), _stream(stream))


def attn_bwd_fused(plan: Plan, q, k, v, do, lse, delta, dq_acc, dk_acc, dv_acc,
                   scale: float = 0.0, stream=None, score: Optional[Score] = None):
    """Every backward ring step, dK/dV of a kv block kept on chip over its whole ring
    (marble_attn_bwd_fused); accumulators fp32 and caller-zeroed."""
    import torch
    c = _qkv(plan, q, k, v, scale)
    _need(do, torch.bfloat16, "do", q.shape)
    _need(lse, torch.float32, "lse", (q.shape[1], plan.n))
    _need(delta, torch.float32, "delta", (q.shape[1], plan.n))
    _need(dq_acc, torch.float32, "dq_acc", q.shape)
    _need(dk_acc, torch.float32, "dk_acc", k.shape)
    _need(dv_acc, torch.float32, "dv_acc", k.shape)
    _call_scored("marble_attn_bwd_fused", plan, c, score, _ptr(do), _ptr(lse), _ptr(delta),
                 _ptr(dq_acc), _ptr(dk_acc), _ptr(dv_acc), _stream(stream))


def forward(plan: Plan, q, k, v, state: State, o, lse, needed: bool = False, scale: float = 0.0,
            stream=None, merge: str = "carried", fused: bool = False,
            score: Optional[Score] = None):
    """All forward ring steps (r-major, keeping shard r's state hot in L2) + finalize;
    ``fused``: the whole ring in one launch (marble_attn_fwd_fused); ``score``: cap and
    distance bias of the scores."""
    if fused:
        if needed or merge not in (None, "carried"):
            raise ValueError("the fused ring carries the fp32 state over the ring steps only")
        attn_fwd_fused(plan, q, k, v, state, scale=scale, stream=stream, score=score)
    else:
        attn_steps(plan, q, k, v, ring_schedule(plan.num_shards, needed), state, scale=scale,
                   stream=stream, merge=merge, score=score)
    attn_finalize(plan, state, o, lse, stream=stream)


def backward(plan: Plan, q, k, v, o, do, lse, delta, dq_acc, dk_acc, dv_acc,
             needed: bool = False, scale: float = 0.0, stream=None, fused: bool = False,
             score: Optional[Score] = None):
    """bwd preprocessing + all backward ring steps (accumulators must be zeroed);
    ``fused``: dK/dV of a kv block kept on chip over its whole ring (marble_attn_bwd_fused);
    ``score``: the forward's."""
    attn_bwd_prep(plan, o, do, delta, stream=stream)
    if fused:
        if needed:
            raise ValueError("the fused ring runs the ring steps, not the needed-block mode")
        attn_bwd_fused(plan, q, k, v, do, lse, delta, dq_acc, dk_acc, dv_acc, scale=scale,
                       stream=stream, score=score)
    else:
        attn_bwd_steps(plan, q, k, v, do, lse, delta, ring_schedule(plan.num_shards, needed),
                       dq_acc, dk_acc, dv_acc, scale=scale, stream=stream, score=score)


def layout_vision_groups(sample, seg):
    """The vision-group layout (marble_layout_vision_groups) of host int32 tracks: returns
    perm (new index -> index), an int32 numpy array."""
    import numpy as np
    s_ = np.ascontiguousarray(sample, dtype=np.int32)
    g_ = np.ascontiguousarray(seg, dtype=np.int32)
    if s_.shape != g_.shape or s_.ndim != 1:
        raise ValueError("sample and seg must be 1-D arrays of one length")
    perm = np.empty(len(s_), np.int32)
    _call("marble_layout_vision_groups", s_.ctypes.data, g_.ctypes.data, len(s_),
          perm.ctypes.data)
    return perm


def chunk_layout_search(block_pairs, num_shards: int, range_cost: int = 0):
    """The chunk-layout search (marble_chunk_layout_search) on a host int64 [nb, nb] matrix
    of work between blocks.  Returns (k, layout cost C, step cost, rank of every chunk)."""
    import numpy as np
    w = np.ascontiguousarray(block_pairs, dtype=np.int64)
    nb = w.shape[0]
    if w.shape != (nb, nb):
        raise ValueError("block_pairs must be square")
    rank = np.zeros(min(nb, 1024), np.int32)
    out = np.zeros(3, np.int64)
    _call("marble_chunk_layout_search", w.ctypes.data, nb, int(num_shards), int(range_cost),
          rank.ctypes.data, out.ctypes.data)
    k = int(out[0])
    return k, int(out[1]), int(out[2]), rank[:k * int(num_shards)].astype(np.int64)


def version() -> str:
    return lib().marble_version().decode()
