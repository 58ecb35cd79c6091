"""Grouped routed-expert decode for the verify window, GB300-native (sm_103a).

A thin ctypes binding over the C ABI in ``include/moe_grouped.h``, ``moe_kv8.h`` and ``moe_decode.h`` (library
``_build/libmoe_grouped.so``, built by ``build.py``). The functions here only marshal
arguments: torch tensors supply device memory and the current CUDA stream; every step runs in
the library's kernels. There is no CPU fallback: a missing library raises.

q8_1 rows are uint8 tensors of shape [rows, cols/32, 36].
"""
from __future__ import annotations

import ctypes
import math
import operator
import os
import struct

import torch

__all__ = [
    "Q8_0", "Q4B", "NL4", "CB2", "CB3", "CB3X", "CB2X", "MoeError", "transcode_cb", "lib", "row_bytes", "strerror",
    "quantize_q8_1", "route_group", "grouped_gu", "swiglu_q8_1", "grouped_down",
    "expert_grouped", "ExpertCall", "STATIC_SCRATCH_BYTES", "test_block_isum", "ERR_BITS", "F_PDL",
    "LayerCall", "layer_sync_ints", "router_topk", "combine", "F_SYNC_PAIR", "F_SYNC_ODD", "F_TEST_EXPIRE",
    "qsa_block_scores", "grouped_fused_sync_ints", "stage_blobs",
    "kv8_block_bytes", "kv8_pool", "kv8_write", "kv8_read", "kv8_attention", "kv8_attention_workspace",
    "add_rms_norm_q8_1", "dequantize_q8_1", "Rope", "head_norm_rope", "kv8_append", "token_logprobs",
]

Q8_0, Q4B, NL4, CB2, CB3, CB3X, CB2X = 1, 2, 3, 4, 5, 6, 7
F_PDL = 1
F_SYNC_PAIR = 2  # moe_expert_layer: sync holds two halves used by alternate calls
F_SYNC_ODD = 4   # ... and this call uses the second half
F_TEST_EXPIRE = 8  # test hook: the down staging waits for a flag no call writes (timeout path)
STATIC_SCRATCH_BYTES = 4 << 20
ERR_BITS = {1: "NGROUPS", 2: "EXPERT", 4: "START", 8: "ENTRY", 16: "ALIGN", 32: "CODEBOOK",
            64: "TIMEOUT", 128: "ROUTE", 256: "PAGE", 512: "LEN"}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmoe_grouped.so")
_LIB = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64


class MoeError(RuntimeError):
    pass


class WFmt(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("codebook", ctypes.c_void_p)]


class ExpertCallC(ctypes.Structure):
    _fields_ = [
        ("gu_fmt", WFmt), ("down_fmt", WFmt),
        ("n_embd", ctypes.c_int32), ("n_ff", ctypes.c_int32), ("n_experts", ctypes.c_int32),
        ("w_gu", _P), ("w_down", _P), ("grp_expert", _P), ("grp_start", _P), ("n_groups", _P),
        ("cap_groups", ctypes.c_int32), ("grid_groups", ctypes.c_int32), ("cap_entries", ctypes.c_int32),
        ("xq", _P), ("n_xq_rows", ctypes.c_int32), ("ent_src", _P), ("ent_dst", _P),
        ("gu", _P), ("hq", _P), ("out", _P), ("out_rows", ctypes.c_int64), ("out_row_stride", ctypes.c_int64),
        ("err", _P), ("flags", ctypes.c_int32),
    ]


class LayerCallC(ctypes.Structure):
    _fields_ = [
        ("gu_fmt", WFmt), ("down_fmt", WFmt),
        ("n_embd", ctypes.c_int32), ("n_ff", ctypes.c_int32), ("n_experts", ctypes.c_int32),
        ("w_gu", _P), ("w_down", _P), ("topk_ids", _P), ("T", ctypes.c_int32), ("k", ctypes.c_int32),
        ("x", _P), ("out", _P), ("out_row_stride", ctypes.c_int64), ("gu", _P), ("hq", _P), ("sync", _P),
        ("grp_expert", _P), ("grp_start", _P), ("n_groups", _P), ("ent_src", _P), ("ent_dst", _P), ("xq", _P),
        ("err", _P), ("flags", ctypes.c_int32),
    ]


class KV8CacheC(ctypes.Structure):
    _fields_ = [
        ("pool", _P), ("n_pages", _I64), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32), ("page_table", _P), ("table_stride", _I64),
        ("max_pages", ctypes.c_int32), ("n_seqs", ctypes.c_int32),
    ]


class KV8RowsC(ctypes.Structure):
    _fields_ = [
        ("k", _P), ("v", _P), ("type", ctypes.c_int32), ("n_tokens", _I64),
        ("k_token_stride", _I64), ("k_head_stride", _I64), ("v_token_stride", _I64), ("v_head_stride", _I64),
    ]


class KV8AttentionC(ctypes.Structure):
    _fields_ = [
        ("cache", KV8CacheC), ("q", _P), ("type", ctypes.c_int32), ("T", ctypes.c_int32),
        ("n_heads", ctypes.c_int32), ("q_seq_stride", _I64), ("q_token_stride", _I64), ("q_head_stride", _I64),
        ("lens", _P), ("tree", _P), ("window", ctypes.c_int32), ("scale", ctypes.c_float), ("out", _P),
        ("lse", _P), ("workspace", _P), ("workspace_bytes", _I64), ("err", _P), ("depth", _P),
        ("flags", ctypes.c_int32),
    ]


class NormCallC(ctypes.Structure):
    _fields_ = [
        ("x", _P), ("residual", _P), ("weight", _P), ("sum", _P), ("y", _P), ("xq", _P),
        ("type", ctypes.c_int32), ("w_type", ctypes.c_int32), ("rows", _I64), ("x_stride", _I64),
        ("residual_stride", _I64), ("cols", ctypes.c_int32), ("eps", ctypes.c_float),
    ]


class RopeC(ctypes.Structure):
    _fields_ = [("turns", _P), ("rot", ctypes.c_int32), ("start", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("factor", ctypes.c_float)]


class HeadsC(ctypes.Structure):
    _fields_ = [
        ("x", _P), ("out", _P), ("weight", _P), ("x_token_stride", _I64), ("x_head_stride", _I64),
        ("out_token_stride", _I64), ("out_head_stride", _I64), ("n_heads", ctypes.c_int32),
    ]


class HeadNormCallC(ctypes.Structure):
    _fields_ = [
        ("q", HeadsC), ("k", HeadsC), ("rope", RopeC), ("positions", _P), ("n_tokens", _I64),
        ("type", ctypes.c_int32), ("w_type", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("eps", ctypes.c_float),
    ]


class KV8AppendC(ctypes.Structure):
    _fields_ = [
        ("cache", KV8CacheC), ("rows", KV8RowsC), ("q", HeadsC), ("rope", RopeC), ("k_weight", _P), ("cu_tokens", _P),
        ("start", _P), ("positions", _P), ("w_type", ctypes.c_int32), ("eps", ctypes.c_float), ("err", _P),
    ]


class LogprobsCallC(ctypes.Structure):
    _fields_ = [
        ("logits", _P), ("row_stride", _I64), ("type", ctypes.c_int32), ("rows", ctypes.c_int32), ("vocab", ctypes.c_int32),
        ("n_ids", ctypes.c_int32), ("top", ctypes.c_int32), ("scale", ctypes.c_float), ("ids", _P), ("logprobs", _P),
        ("top_logprobs", _P), ("top_ids", _P), ("entropy", _P), ("lse", _P),
    ]


_ELEM = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def lib():
    """Load the CUDA library (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise MoeError(f"CUDA library not built: {LIB_PATH} (run __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        L.moe_row_bytes.argtypes = [_I, _I]
        L.moe_row_bytes.restype = _I64
        L.moe_strerror.argtypes = [_I]
        L.moe_strerror.restype = ctypes.c_char_p
        L.moe_quantize_q8_1.argtypes = [_P, _I64, _I64, _P, _P]
        L.moe_route_group.argtypes = [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]
        L.moe_grouped_gu.argtypes = [WFmt, _I, _I, _P, _I, _P, _P, _P, _I, _I, _P, _I, _P, _I, _P, _P, _P]
        L.moe_swiglu_q8_1.argtypes = [_P, _I, _P, _P, _I, _I, _P, _P, _P]
        L.moe_grouped_down.argtypes = [WFmt, _I, _I, _P, _I, _P, _P, _P, _I, _I, _P, _I, _P, _P, _I64, _I64,
                                       _P, _P]
        L.moe_expert_grouped.argtypes = [ctypes.POINTER(ExpertCallC), _P]
        L.moe_expert_grouped_static.argtypes = [ctypes.POINTER(ExpertCallC), _P]
        L.moe_test_block_isum.argtypes = [WFmt, _I, _P, _I, _P, _P, _P]
        L.moe_transcode_cb.argtypes = [WFmt, _I, _I, _I, _I, _P, _P, _P, _P]
        L.moe_expert_layer.argtypes = [ctypes.POINTER(LayerCallC), _P]
        L.moe_layer_sync_ints.argtypes = [_I, _I, _I]
        L.moe_layer_sync_ints.restype = _I64
        L.moe_router_topk.argtypes = [_P, _I, _I, _I, _P, _P, _P]
        L.moe_combine.argtypes = [_P, _I64, _P, _P, _I, _I, _I, _I, _P, _I64, _P]
        L.moe_qsa_block_scores.argtypes = [_P, _I, _P, _P, _I64, _P, _P]
        L.moe_expert_grouped_fused.argtypes = [ctypes.POINTER(ExpertCallC), _P, _P]
        L.moe_grouped_fused_sync_ints.argtypes = [_I, _I, _I]
        L.moe_grouped_fused_sync_ints.restype = _I64
        L.moe_stage_blobs.argtypes = [_P, _P, _P, _I, _P]
        L.moe_kv8_block_bytes.argtypes = [_I]
        L.moe_kv8_block_bytes.restype = _I64
        L.moe_kv8_write.argtypes = [_P, _P, _P, _P, _P, _P]
        L.moe_kv8_read.argtypes = [_P, _P, _P, _P, _P, _P]
        L.moe_kv8_attention_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
        L.moe_kv8_attention_workspace_bytes.restype = _I64
        L.moe_kv8_attention.argtypes = [_P, _P]
        L.moe_add_rms_norm_q8_1.argtypes = [_P, _P]
        L.moe_dequantize_q8_1.argtypes = [_P, _I64, _I64, _P, _I, _P]
        L.moe_head_norm_rope.argtypes = [_P, _P]
        L.moe_kv8_append.argtypes = [_P, _P]
        L.moe_token_logprobs.argtypes = [_P, _P]
        for f in ("moe_quantize_q8_1", "moe_route_group", "moe_grouped_gu", "moe_swiglu_q8_1",
                  "moe_grouped_down", "moe_expert_grouped", "moe_expert_grouped_static", "moe_test_block_isum",
                  "moe_transcode_cb", "moe_expert_layer", "moe_router_topk", "moe_combine",
                  "moe_qsa_block_scores", "moe_expert_grouped_fused", "moe_stage_blobs", "moe_kv8_write",
                  "moe_kv8_read", "moe_kv8_attention", "moe_add_rms_norm_q8_1", "moe_dequantize_q8_1",
                  "moe_head_norm_rope", "moe_kv8_append", "moe_token_logprobs"):
            getattr(L, f).restype = _I
        _LIB = L
    return _LIB


def row_bytes(typ: int, K: int) -> int:
    return int(lib().moe_row_bytes(typ, K))


def strerror(status: int) -> str:
    return lib().moe_strerror(status).decode()


def _check(rc: int):
    if rc != 0:
        raise MoeError(f"{rc}: {strerror(rc)}")


def _dp(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise MoeError("device tensor expected")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _fmt(typ, codebook):
    return WFmt(typ, None if codebook is None else codebook.data_ptr())


def quantize_q8_1(x: torch.Tensor, xq: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x: fp32 [rows, cols] (contiguous, device) -> uint8 q8_1 [rows, cols/32, 36]."""
    rows, cols = x.shape
    if xq is None:
        xq = torch.empty((rows, cols // 32, 36), dtype=torch.uint8, device=x.device)
    _check(lib().moe_quantize_q8_1(_dp(x), rows, cols, _dp(xq), _stream(stream)))
    return xq


def route_group(topk_ids, n_experts, entry_base, grp_expert, grp_start, n_groups, ent_src, ent_dst,
                err=None, stream=None):
    T, k = topk_ids.shape
    _check(lib().moe_route_group(_dp(topk_ids), T, k, n_experts, entry_base, _dp(grp_expert), _dp(grp_start),
                                 _dp(n_groups), _dp(ent_src), _dp(ent_dst), _dp(err), _stream(stream)))


def grouped_gu(typ, codebook, n_embd, n_ff, w_table, n_experts, grp_expert, grp_start, n_groups, cap_groups,
               grid_groups, xq, ent_src, cap_entries, gu, err=None, stream=None):
    _check(lib().moe_grouped_gu(_fmt(typ, codebook), n_embd, n_ff, _dp(w_table), n_experts, _dp(grp_expert),
                                _dp(grp_start), _dp(n_groups), cap_groups, grid_groups, _dp(xq), xq.shape[0],
                                _dp(ent_src), cap_entries, _dp(gu), _dp(err), _stream(stream)))


def swiglu_q8_1(gu, n_ff, grp_start, n_groups, cap_groups, cap_entries, hq, err=None, stream=None):
    _check(lib().moe_swiglu_q8_1(_dp(gu), n_ff, _dp(grp_start), _dp(n_groups), cap_groups, cap_entries, _dp(hq),
                                 _dp(err), _stream(stream)))


def grouped_down(typ, codebook, n_embd, n_ff, w_table, n_experts, grp_expert, grp_start, n_groups, cap_groups,
                 grid_groups, hq, cap_entries, ent_dst, out, err=None, stream=None):
    _check(lib().moe_grouped_down(_fmt(typ, codebook), n_embd, n_ff, _dp(w_table), n_experts, _dp(grp_expert),
                                  _dp(grp_start), _dp(n_groups), cap_groups, grid_groups, _dp(hq), cap_entries,
                                  _dp(ent_dst), _dp(out), out.shape[0], out.stride(0), _dp(err),
                                  _stream(stream)))


class ExpertCall:
    """Arguments of one moe_expert_grouped call, kept alive with their tensors."""

    def __init__(self, gu_type, gu_codebook, down_type, down_codebook, n_embd, n_ff, w_gu_table, w_down_table,
                 n_experts, grp_expert, grp_start, n_groups, cap_groups, grid_groups, cap_entries, xq, ent_src,
                 ent_dst, gu, hq, out, err=None, flags=F_PDL):
        self._keep = (gu_codebook, down_codebook, w_gu_table, w_down_table, grp_expert, grp_start, n_groups, xq,
                      ent_src, ent_dst, gu, hq, out, err)
        self.c = ExpertCallC(
            _fmt(gu_type, gu_codebook), _fmt(down_type, down_codebook), n_embd, n_ff, n_experts,
            w_gu_table.data_ptr(), w_down_table.data_ptr(), grp_expert.data_ptr(), grp_start.data_ptr(),
            n_groups.data_ptr(), cap_groups, grid_groups, cap_entries, xq.data_ptr(), xq.shape[0],
            ent_src.data_ptr(), ent_dst.data_ptr(), gu.data_ptr(), hq.data_ptr(), out.data_ptr(), out.shape[0],
            out.stride(0), None if err is None else err.data_ptr(), flags)

    def __call__(self, stream=None):
        _check(lib().moe_expert_grouped(ctypes.byref(self.c), _stream(stream)))

    def call_fused(self, sync, stream=None):
        """The same call in one fused launch (moe_expert_grouped_fused); sync: int32 device tensor
        of grouped_fused_sync_ints(cap_groups, cap_entries, n_ff) words, zeroed before the first
        call (flags MOE_F_SYNC_PAIR / MOE_F_SYNC_ODD in self.c.flags select its halves)."""
        _check(lib().moe_expert_grouped_fused(ctypes.byref(self.c), _dp(sync), _stream(stream)))

    def call_static(self, stream=None):
        """The same call through moe_expert_grouped_static: gu/hq are ignored and the library's
        static device scratch buffer is used instead (nothing is allocated)."""
        _check(lib().moe_expert_grouped_static(ctypes.byref(self.c), _stream(stream)))


def stage_blobs(host_blobs, dev_slots, stream=None):
    """Copy host-resident blobs (uint8 CPU tensors, pinned for the copy kernel) into device staging
    slots (uint8 CUDA tensors, at least as large) with moe_stage_blobs."""
    n = len(host_blobs)
    assert len(dev_slots) == n and all(d.numel() >= h.numel() for h, d in zip(host_blobs, dev_slots))
    src = (ctypes.c_void_p * n)(*[h.data_ptr() for h in host_blobs])
    dst = (ctypes.c_void_p * n)(*[d.data_ptr() for d in dev_slots])
    by = (ctypes.c_int64 * n)(*[h.numel() * h.element_size() for h in host_blobs])
    _check(lib().moe_stage_blobs(src, dst, by, n, _stream(stream)))


def grouped_fused_sync_ints(cap_groups: int, cap_entries: int, n_ff: int) -> int:
    """int32 sync words a moe_expert_grouped_fused call needs (zero them before the first call)."""
    return int(lib().moe_grouped_fused_sync_ints(cap_groups, cap_entries, n_ff))


def layer_sync_ints(T: int, k: int, n_ff: int) -> int:
    """int32 sync words a moe_expert_layer call needs: counters, the call epoch and the flagged h
    copies (zero them once before the first call; torch allocations are 8-byte aligned)."""
    return int(lib().moe_layer_sync_ints(T, k, n_ff))


class LayerCall:
    """Arguments of one moe_expert_layer call (the whole layer in one launch), kept alive with their
    tensors. topk_ids int32 [T, k], x fp32 [T, n_embd], out fp32 [T*k, >= n_embd]; gu / hq scratch
    as for ExpertCall; sync int32 [layer_sync_ints(T, k, n_ff)] zeroed before the first call.
    grp_expert .. xq: optional tensors that receive the grouping and the activation q8_1."""

    def __init__(self, gu_type, gu_codebook, down_type, down_codebook, n_embd, n_ff, w_gu_table, w_down_table,
                 n_experts, topk_ids, x, out, gu, hq, sync, err=None, flags=F_PDL, grp_expert=None, grp_start=None,
                 n_groups=None, ent_src=None, ent_dst=None, xq=None):
        T, k = topk_ids.shape
        opt = (grp_expert, grp_start, n_groups, ent_src, ent_dst, xq)
        self._keep = (gu_codebook, down_codebook, w_gu_table, w_down_table, topk_ids, x, out, gu, hq, sync,
                      err) + opt
        ptr = lambda t: None if t is None else t.data_ptr()
        self.c = LayerCallC(
            _fmt(gu_type, gu_codebook), _fmt(down_type, down_codebook), n_embd, n_ff, n_experts,
            w_gu_table.data_ptr(), w_down_table.data_ptr(), topk_ids.data_ptr(), T, k, x.data_ptr(),
            out.data_ptr(), out.stride(0), gu.data_ptr(), hq.data_ptr(), sync.data_ptr(),
            *[ptr(t) for t in opt], ptr(err), flags)

    def __call__(self, stream=None):
        _check(lib().moe_expert_layer(ctypes.byref(self.c), _stream(stream)))


def router_topk(logits, k, topk_ids=None, weights=None, stream=None):
    """logits fp32 [T, n_experts] -> (topk_ids int32 [T, k], weights fp32 [T, k]) on the device."""
    T, E = logits.shape
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if weights is None:
        weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(lib().moe_router_topk(_dp(logits), T, E, k, _dp(topk_ids), _dp(weights), _stream(stream)))
    return topk_ids, weights


def combine(out, topk_ids, weights, n_experts, y=None, stream=None):
    """out fp32 [T*k, >= n_embd] (row t*k + j = entry (t, j)); -> y fp32 [T, n_embd]."""
    T, k = topk_ids.shape
    N = out.shape[1]
    if y is None:
        y = torch.empty((T, N), dtype=torch.float32, device=out.device)
    _check(lib().moe_combine(_dp(out), out.stride(0), _dp(topk_ids), _dp(weights), T, k, n_experts, N, _dp(y),
                             y.stride(0), _stream(stream)))
    return y


def qsa_block_scores(q, keys, key_scale, scores=None, stream=None):
    """QSA decode block scores: q fp32 [T, 4, 128] (T <= 4), keys int8 [n_blocks, 128], key_scale
    fp32 [n_blocks] -> scores fp32 [T, n_blocks] on the device (the tail block + 1e9)."""
    T = q.shape[0]
    nb = keys.shape[0]
    if scores is None:
        scores = torch.empty((T, nb), dtype=torch.float32, device=q.device)
    _check(lib().moe_qsa_block_scores(_dp(q), T, _dp(keys), _dp(key_scale), nb, _dp(scores), _stream(stream)))
    return scores


# ---------------------------------------------------------------- the attention side (moe_kv8.h)
# A small call's time is the binding's, so these pass packed structures and plain integers, and
# check only what the library cannot see (devices, types, shapes and strides of tensors); everything
# else is checked by the library.

_CACHE = "PqiiiPqii"                             # moe_kv8_cache
_pack_rows = struct.Struct("@" + _CACHE + "0q").pack, struct.Struct("@PPiqqqqq").pack
_pack_attn = struct.Struct("@" + _CACHE + "0qPiiiqqqPPifPPPqPPi0q").pack
_pack_norm = struct.Struct("@PPPPPPiiqqqif").pack
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _elem(t):
    try:
        return _ELEM[t.dtype]
    except KeyError:
        raise MoeError(f"float32, float16 or bfloat16 expected, got {t.dtype}") from None


def _device(t):
    dev = t.get_device()
    if dev < 0:
        raise MoeError("device tensor expected")
    return dev


def _ptr(t, dev):
    if t.get_device() != dev:
        raise MoeError(f"a tensor on device {dev} expected")
    return t.data_ptr()


def _ints(t, name, numel, dev):
    if t.dtype is not torch.int32 or t.numel() != numel or not t.is_contiguous():
        raise MoeError(f"{name}: a contiguous int32 tensor of {numel} elements expected")
    return _ptr(t, dev)


def _err(err, dev):
    return 0 if err is None else _ints(err, "err", 1, dev)


def _pack(pack, *values):
    """A structure's bytes; what its fields do not hold is an argument error."""
    try:
        return pack(*values)
    except (struct.error, OverflowError) as e:
        raise MoeError(f"an argument is out of its type's range: {e}") from None


def _empty(stream, shape, dtype, device):
    """A tensor of the caching allocator, of the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _launch(f, dev, stream, tensors, *args):
    """Call f(*args, stream) on device dev, which has to be the current one (the library launches there); tensors
    are marked as used on a stream that is not the current one."""
    if dev != _current_device() or (stream is not None and stream.device_index != dev):
        raise MoeError(f"tensors on device {dev}: the current device, and the stream's, expected")
    if stream is None:
        rc = f(*args, _raw_stream(dev))
    else:
        rc = f(*args, stream.cuda_stream)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    if rc:
        raise MoeError(f"{rc}: {strerror(rc)}")


def _kv8_cache(pool, page_table):
    """The fields of moe_kv8_cache, and the device."""
    dev = _device(pool)
    shape, rows = pool.shape, page_table.shape
    if pool.dtype is not torch.uint8 or len(shape) != 4 or not pool.is_contiguous():
        raise MoeError("pool: contiguous uint8 [pages, kv heads, page tokens / 32, block bytes] expected")
    if page_table.dtype is not torch.int32 or len(rows) != 2 or (page_table.stride(1) != 1 and rows[1] > 1):
        raise MoeError("page_table: int32 [sequences, pages] with contiguous rows expected")
    n_pages, hkv, nb, rec = shape
    if rec < 16 or (rec - 16) % 64:
        raise MoeError(f"pool: records of {rec} bytes are of no head size")
    n, pages = rows
    return (pool.data_ptr(), n_pages, hkv, (rec - 16) // 64, nb * 32, _ptr(page_table, dev),
            page_table.stride(0) if n > 1 else pages, pages, n), dev


def kv8_block_bytes(head_dim: int) -> int:
    """Bytes of one record of the cache: 32 tokens of one key/value head."""
    return int(lib().moe_kv8_block_bytes(head_dim))


def kv8_pool(n_pages: int, n_kv_heads: int, head_dim: int, page_tokens: int = 64, device="cuda") -> torch.Tensor:
    """A zeroed cache pool: uint8 [n_pages, n_kv_heads, page_tokens / 32, block bytes]."""
    rec = kv8_block_bytes(head_dim)
    if not rec or page_tokens <= 0 or page_tokens % 32:
        raise MoeError("head_dim: a multiple of 32 up to 256; page_tokens: a multiple of 32")
    return torch.zeros((n_pages, n_kv_heads, page_tokens // 32, rec), dtype=torch.uint8, device=device)


def _kv8_move(f, pool, page_table, cu_tokens, start, n_tokens, dtype, k, v, err, stream):
    c, dev = _kv8_cache(pool, page_table)
    hkv, D, n = c[2], c[3], c[8]
    if n_tokens is None:
        n_tokens = k.shape[0]
    if k is None:
        k = _empty(stream, (n_tokens, hkv, D), dtype, pool.device)
    if v is None:
        v = _empty(stream, (n_tokens, hkv, D), k.dtype, pool.device)
    ks, vs = k.stride(), v.stride()
    if k.shape != (n_tokens, hkv, D) or v.shape != k.shape or v.dtype is not k.dtype or ks[2] != 1 or vs[2] != 1:
        raise MoeError(f"k, v: [{n_tokens}, {hkv}, {D}] of one type, contiguous in the last dimension, expected")
    if n == 0 and n_tokens == 0:  # no sequences (the library takes one at least)
        return k, v
    rows = _pack(_pack_rows[1], _ptr(k, dev), _ptr(v, dev), _elem(k), n_tokens, ks[0], ks[1], vs[0], vs[1])
    _launch(f, dev, stream, (k, v, pool, page_table, cu_tokens, start, err), _pack(_pack_rows[0], *c), rows,
            _ints(cu_tokens, "cu_tokens", n + 1, dev), _ints(start, "start", n, dev), _err(err, dev))
    return k, v


def kv8_write(k, v, pool, page_table, cu_tokens, start, err=None, stream=None):
    """Quantise rows k, v [tokens, kv heads, head_dim] into the cache: rows cu_tokens[b] ..
    cu_tokens[b+1] become positions start[b] .. of sequence b, which ends with them. cu_tokens int32
    [sequences + 1], start int32 [sequences], page_table int32 [sequences, pages]; all on the device."""
    _kv8_move(lib().moe_kv8_write, pool, page_table, cu_tokens, start, None, None, k, v, err, stream)


def kv8_read(pool, page_table, cu_tokens, start, n_tokens, dtype=torch.bfloat16, k=None, v=None, err=None,
             stream=None):
    """Read positions start[b] .. of each sequence back as rows cu_tokens[b] .. cu_tokens[b+1] of
    k, v [n_tokens, kv heads, head_dim] (allocated as `dtype` when not given). n_tokens is
    cu_tokens' last value. Rows of a sequence or block that is refused (err) are left as they were."""
    return _kv8_move(lib().moe_kv8_read, pool, page_table, cu_tokens, start, n_tokens, dtype, k, v, err, stream)


def kv8_attention_workspace(n_seqs: int, T: int, n_heads: int, n_kv_heads: int, head_dim: int,
                            device="cuda") -> torch.Tensor:
    """A workspace for kv8_attention calls of these sizes, or of fewer sequences, dims, and rows of a key/value
    head (T * n_heads / n_kv_heads), to be kept between calls (one for each stream that calls run on at the
    same time)."""
    n = int(lib().moe_kv8_attention_workspace_bytes(n_seqs, T, n_heads, n_kv_heads, head_dim))
    if not n:
        raise MoeError(strerror(-3))
    return torch.empty(n, dtype=torch.uint8, device=device)


def kv8_attention(q, pool, page_table, lens, scale=None, window=0, tree=None, workspace=None, out=None, lse=None,
                  with_lse=False, err=None, stream=None, depth=None):
    """Attention of q [sequences, T, heads, head_dim] (the last T of lens[b] cached positions; T <= 32)
    over the cache. window: a query sees that many positions up to its own (0: all); tree: int32
    [sequences, T], bit j of tree[b, t] lets query t see window token j (else: causal); depth: int32
    [sequences, T], a token's number of ancestors in the tree, from which `window` is then counted (else: from
    its index in the window, which in a path with fewer ancestors hides the oldest tokens). Returns out
    [sequences, T, heads, head_dim] of q's type, and with_lse (or a given lse) also the log of the
    softmax sums, fp32 [sequences, T, heads]; a query that sees nothing gives zeros and -inf."""
    c, dev = _kv8_cache(pool, page_table)
    shape, qs = q.shape, q.stride()
    if len(shape) != 4 or shape[0] != c[8] or shape[3] != c[3] or qs[3] != 1:
        raise MoeError(f"q: [{c[8]}, T, heads, {c[3]}], contiguous in the last dimension, expected")
    B, T, hq, D = shape
    if workspace is None:
        workspace = _empty(stream, (max(16, lib().moe_kv8_attention_workspace_bytes(B, T, hq, c[2], D)),), torch.uint8, q.device)
    if out is None:
        out = _empty(stream, shape, q.dtype, q.device)
    elif out.dtype is not q.dtype or out.shape != shape or not out.is_contiguous():
        raise MoeError("out: contiguous, of q's shape and type, expected")
    if lse is None:
        if with_lse:
            lse = _empty(stream, (B, T, hq), torch.float32, q.device)
    elif lse.dtype is not torch.float32 or lse.shape != (B, T, hq) or not lse.is_contiguous():
        raise MoeError("lse: contiguous float32 [sequences, T, heads] expected")
    if not workspace.is_contiguous():
        raise MoeError("workspace: a contiguous tensor expected")
    if B == 0:  # no sequences (the library takes one at least)
        return out if lse is None else (out, lse)
    a = _pack(_pack_attn, *c, _ptr(q, dev), _elem(q), T, hq, qs[0], qs[1], qs[2], _ints(lens, "lens", B, dev),
                   0 if tree is None else _ints(tree, "tree", B * T, dev), window, D ** -0.5 if scale is None else scale,
                   _ptr(out, dev), 0 if lse is None else _ptr(lse, dev), _ptr(workspace, dev), workspace.nbytes,
                   _err(err, dev), 0 if depth is None else _ints(depth, "depth", B * T, dev), 0)
    _launch(lib().moe_kv8_attention, dev, stream, (q, pool, page_table, lens, tree, depth, out, lse, workspace, err), a)
    return out if lse is None else (out, lse)


def add_rms_norm_q8_1(x, weight, residual=None, eps=1e-6, sum_out=None, y=None, xq=None, with_y=False, stream=None):
    """h = x + residual, y = h * (1 / sqrt(mean(h^2) + eps)) * weight, and y's q8_1 rows, in one pass.
    x, residual [rows, cols] of one type, weight [cols]. Returns (sum, y, xq): h in x's type (None
    without a residual, unless sum_out is given; sum_out may be the residual itself), y in x's type
    (with_y or a given y, else None), xq uint8 [rows, cols/32, 36]."""
    dev, shape, dtype, device = _device(x), x.shape, x.dtype, x.device
    if len(shape) != 2 or x.stride(1) != 1 or weight.shape != shape[1:] or not weight.is_contiguous():
        raise MoeError("x: [rows, cols] with contiguous rows, weight: contiguous [cols], expected")
    rows, cols = shape
    if residual is not None:
        if residual.shape != shape or residual.dtype is not dtype or residual.stride(1) != 1:
            raise MoeError("residual: x's shape and type, with contiguous rows, expected")
        if sum_out is None:
            sum_out = _empty(stream, shape, dtype, device)
    if y is None and with_y:
        y = _empty(stream, shape, dtype, device)
    for t in (sum_out, y):
        if t is not None and (t.shape != shape or t.dtype is not dtype or not t.is_contiguous()):
            raise MoeError("sum_out, y: contiguous, of x's shape and type, expected")
    if xq is None:
        xq = _empty(stream, (rows, cols // 32, 36), torch.uint8, device)
    elif xq.dtype is not torch.uint8 or xq.shape != (rows, cols // 32, 36) or not xq.is_contiguous():
        raise MoeError("xq: contiguous uint8 [rows, cols/32, 36] expected")
    if rows:
        c = _pack(_pack_norm, x.data_ptr(), 0 if residual is None else _ptr(residual, dev), _ptr(weight, dev),
                       0 if sum_out is None else _ptr(sum_out, dev), 0 if y is None else _ptr(y, dev), _ptr(xq, dev),
                       _elem(x), _elem(weight), rows, x.stride(0) if rows > 1 else cols,
                       0 if residual is None else residual.stride(0) if rows > 1 else cols, cols, eps)
        _launch(lib().moe_add_rms_norm_q8_1, dev, stream, (x, residual, weight, sum_out, y, xq), c)
    return sum_out, y, xq


def dequantize_q8_1(xq, dtype=torch.float32, out=None, stream=None):
    """The values that q8_1 rows [rows, cols/32, 36] stand for, [rows, cols] of `dtype`."""
    dev, shape = _device(xq), xq.shape
    if xq.dtype is not torch.uint8 or len(shape) != 3 or shape[2] != 36 or not xq.is_contiguous():
        raise MoeError("xq: contiguous uint8 [rows, cols/32, 36] expected")
    rows, cols = shape[0], shape[1] * 32
    if out is None:
        out = _empty(stream, (rows, cols), dtype, xq.device)
    elif out.shape != (rows, cols) or not out.is_contiguous():
        raise MoeError("out: contiguous [rows, cols] expected")
    if rows:
        _launch(lib().moe_dequantize_q8_1, dev, stream, (xq, out), xq.data_ptr(), rows, cols, _ptr(out, dev), _elem(out))
    return out


# ---------------------------------------------------------------- around the attention side (moe_decode.h)

_ROWS, _HEADS, _ROPE = "PPiqqqqq", "PPPqqqqi0q", "Piiif"
_pack_heads = struct.Struct("@" + _HEADS * 2 + _ROPE + "Pqiiif").pack
_pack_append = struct.Struct("@" + _CACHE + "0q" + _ROWS + _HEADS + _ROPE + "PPPPifP").pack
_pack_logprobs = struct.Struct("@PqiiiiifPPPPPP").pack
_NO_HEADS, _NO_ROPE = (0,) * 8, (0, 0, 0, 0, 0.0)
_TWO_PI = 2 * 314159265358979323846264338327950288419716939937510, 10 ** 50  # as a fraction


class Rope:
    """A rotation of heads by position, kept between calls: dims start .. start + rot of a head are rot / 2 pairs, dims
    (start + i, start + i + rot / 2), or interleaved (start + 2 i, start + 2 i + 1), and pair i turns by position * f_i.
    rot is a multiple of 16, start of 8. f_i = theta^(-2 i / rot) (theta 10000 where not given), or inv_freq[i] where given (say,
    frequencies that were rounded to fp32). scaling: None, or for long contexts
      {"kind": "linear", "scale": s}: all divided by s;
      {"kind": "yarn", "scale": s, "original": o, "fast": 32, "slow": 1}: pairs that turn less than `slow` times over the
        original length o are divided by s, those that turn more than `fast` times are kept, with a line in i between (whose
        ends are moved outward to whole pairs); the rotated dims are multiplied by 0.1 log s + 1. The ends come from theta: with
        inv_freq, which have to be its powers (to 2^-7 of themselves), it has to be given. fast is above slow, s at least 1;
      {"kind": "bands", "scale": s, "original": o, "low": 1, "high": 4}: the same by low and high, with a line in the number
        of turns, and without a factor.
    factor (of the rotated dims) overrides the scaling's. Angles are exact to 1e-7 at any 32-bit position."""

    def __init__(self, rot, theta=None, start=0, interleaved=False, scaling=None, inv_freq=None, factor=None, device="cuda"):
        try:
            rot, start = operator.index(rot), operator.index(start)
            if rot <= 0 or rot % 16 or start < 0 or start % 8:
                raise MoeError("rot: a multiple of 16, start: a multiple of 8, expected")
            if inv_freq is None:
                theta = 10000.0 if theta is None else theta
                if not (theta > 0 and math.isfinite(theta)):
                    raise MoeError("theta: a positive number expected")
                f = [float(theta) ** (-2 * i / rot) for i in range(rot // 2)]
            else:
                f = [float(x) for x in inv_freq]
            if len(f) != rot // 2 or not all(math.isfinite(x) for x in f):
                raise MoeError(f"inv_freq: {rot // 2} finite numbers expected")
            f, scaled = self._scaled(f, rot, theta, dict(scaling or {"kind": "none"}))
            factor = scaled if factor is None else float(factor)
        except (TypeError, ValueError, OverflowError) as e:
            raise MoeError(f"rope: an argument is not of its kind, or out of its range: {e}") from None
        if not all(math.isfinite(x) for x in f) or not abs(factor) <= 3.4028234663852886e38:
            raise MoeError("rope: frequencies out of range, or a factor that fp32 does not hold")
        self.inv_freq, self.factor = f, factor
        self.rot, self.start, self.interleaved = rot, start, bool(interleaved)
        # fractions of a turn a position, rounded to 64 bits (as int64 tensors hold them)
        turns = []
        for x in f:
            n, d = x.as_integer_ratio()
            n, d = n * _TWO_PI[1] << 64, d * _TWO_PI[0]
            turns.append(((2 * n + d) // (2 * d) + 2 ** 63) % 2 ** 64 - 2 ** 63)
        self.turns = torch.tensor(turns, dtype=torch.int64, device=device)
        self._device = self.turns.get_device()
        self._fields = (rot, start, int(self.interleaved), self.factor)  # (without the address: a copy has its own)

    def __setstate__(self, state):  # (loading may move tensors to another device)
        self.__dict__.update(state)
        self._device = self.turns.get_device()

    @staticmethod
    def _scaled(f, rot, theta, p):
        kind, s = p.pop("kind", None), p.pop("scale", 1.0)
        known = {"none": {}, "linear": {}, "yarn": {"original": None, "fast": 32.0, "slow": 1.0}, "bands": {"original": None, "low": 1.0, "high": 4.0}}
        if kind not in known or not (s > 0 and math.isfinite(s)) or set(p) - set(known[kind]):
            raise MoeError(f"scaling: unknown kind or fields, or no positive scale: {kind!r}, {sorted(p)}")
        p = {**known[kind], **p}
        if kind in ("none", "linear"):
            return [x / s for x in f], 1.0
        if not all(x is not None and x > 0 for x in p.values()):
            raise MoeError(f"scaling: {kind} takes positive {', '.join(p)}")
        turns = [p["original"] * abs(x) / (2 * math.pi) for x in f]
        if kind == "bands":
            if p["high"] <= p["low"]:
                raise MoeError("scaling: high above low expected")
            keep = [min(max((t - p["low"]) / (p["high"] - p["low"]), 0.0), 1.0) for t in turns]
            factor = 1.0
        else:
            if p["fast"] <= p["slow"] or s < 1:
                raise MoeError("scaling: yarn takes fast above slow, and a scale of at least 1")
            if theta is None or not 1 < theta < math.inf:
                raise MoeError("scaling: yarn takes a theta above 1, with inv_freq the one whose powers they are")
            if any(not abs(x * float(theta) ** (2 * i / rot) - 1) <= 2.0 ** -7 for i, x in enumerate(f)):
                raise MoeError("scaling: yarn takes frequencies that are theta's powers")
            at = [rot * math.log(p["original"] / (2 * math.pi * p[r])) / (2 * math.log(theta)) for r in ("fast", "slow")]
            lo, hi = max(math.floor(at[0]), 0), math.ceil(at[1])
            # (hi <= lo: pair 0, where a line starts at the earliest, lies behind its end)
            keep = [1 - min(max((i - lo) / (hi - lo), 0.0), 1.0) if hi > lo else 0.0 for i in range(rot // 2)]
            factor = 0.1 * math.log(s) + 1
        return [x * k + x / s * (1 - k) for x, k in zip(f, keep)], factor


def _rope(rope, dev, D):
    if rope is None:
        return _NO_ROPE
    if rope._device != dev:
        raise MoeError(f"rope: on device {dev} expected")
    if rope.start + rope.rot > D:
        raise MoeError(f"rope: dims {rope.start} .. {rope.start + rope.rot} of heads of {D}")
    return (rope.turns.data_ptr(), *rope._fields)


def _heads(x, weight, out, N, D, dtype, dev, stream, name):
    """The fields of moe_heads, and the rows that they are written to."""
    shape = x.shape
    if len(shape) != 3 or x.dtype is not dtype or x.get_device() != dev:
        raise MoeError(f"{name}: [{N}, heads, {D}] of {dtype} on device {dev} expected")
    n, H, d = shape
    xt, xh, xd = x.stride()
    if n != N or d != D or (xd != 1 and N):
        raise MoeError(f"{name}: [{N}, heads, {D}], contiguous in the last dimension, expected")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device) if stream is None else _empty(stream, shape, dtype, x.device)
        ot, oh = H * D, D
    else:
        if out.shape != shape or out.dtype is not dtype or (out.stride(2) != 1 and N) or out.get_device() != dev:
            raise MoeError(f"{name}_out: {name}'s shape, type and device, contiguous in the last dimension, expected")
        ot, oh, _ = out.stride()
    w = 0
    if weight is not None:
        w = weight.data_ptr()
        if weight.numel() != D or weight.dim() != 1 or not weight.is_contiguous() or weight.get_device() != dev:
            raise MoeError(f"{name}_weight: contiguous [{D}] on device {dev} expected")
    return (x.data_ptr(), out.data_ptr(), w, xt, xh, ot, oh, H), out


def _w_type(a, b):
    if a is None or b is None:
        return 0 if a is b else _elem(b if a is None else a)
    if a.dtype is not b.dtype:
        raise MoeError("q_weight and k_weight: one type expected")
    return _elem(a)


def head_norm_rope(q, positions, rope=None, k=None, q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None, stream=None):
    """Norm of each head (where it has a weight [head_dim]) and rotation by position (where there is a Rope) of rows q, and
    k, [tokens, heads, head_dim], in one pass; positions int32 [tokens] (None without a rotation), negative ones turn back. Returns (q_out,
    k_out), k_out None without k; q_out may be q itself, k_out k. head_dim: a multiple of 16 up to 256."""
    dev = _device(q)
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3:
        raise MoeError("q: [tokens, heads, head_dim] expected")
    N, _, D = shape
    if rope is not None and positions is None:
        raise MoeError("positions: expected with a rotation")
    a, q_out = _heads(q, q_weight, q_out, N, D, dtype, dev, stream, "q")
    b, k_out = (_NO_HEADS, None) if k is None else _heads(k, k_weight, k_out, N, D, dtype, dev, stream, "k")
    c = _pack(_pack_heads, *a, *b, *_rope(rope, dev, D), 0 if positions is None else _ints(positions, "positions", N, dev), N, _elem(q),
              _w_type(q_weight, None if k is None else k_weight), D, eps)
    _launch(lib().moe_head_norm_rope, dev, stream, (q, k, q_weight, k_weight, positions, q_out, k_out, None if rope is None else rope.turns), c)
    return q_out, k_out


def kv8_append(k, v, pool, page_table, cu_tokens, start, rope=None, q=None, q_weight=None, k_weight=None, eps=1e-6, positions=None,
               q_out=None, err=None, stream=None):
    """kv8_write of keys that are normed (k_weight [head_dim]) and rotated on the way, and the queries of the same tokens, q
    [tokens, heads, head_dim], normed and rotated beside them: one launch from the projection's rows to what kv8_attention
    takes. positions int32 [tokens]: what each row turns by (a draft token by its depth in a tree), None: its
    position in the cache. Returns q_out (None without q); q_out may be q itself. Rows of q_out of a sequence that is refused (err), and
    rows behind the last sequence, are left as they were."""
    c, dev = _kv8_cache(pool, page_table)
    hkv, D, n = c[2], c[3], c[8]
    N, ks, vs = k.shape[0] if k.dim() else 0, k.stride(), v.stride()
    if k.shape != (N, hkv, D) or v.shape != k.shape or v.dtype is not k.dtype or (N and (ks[2] != 1 or vs[2] != 1)):
        raise MoeError(f"k, v: [tokens, {hkv}, {D}] of one type, contiguous in the last dimension, expected")
    if k_weight is not None and (k_weight.shape != (D,) or not k_weight.is_contiguous()):
        raise MoeError(f"k_weight: contiguous [{D}] expected")
    a, q_out = (_NO_HEADS, None) if q is None else _heads(q, q_weight, q_out, N, D, k.dtype, dev, stream, "q")
    if n == 0 and N == 0:  # no sequences (the library takes one at least)
        return q_out
    x = _pack(_pack_append, *c, _ptr(k, dev), _ptr(v, dev), _elem(k), N, ks[0], ks[1], vs[0], vs[1], *a, *_rope(rope, dev, D),
              0 if k_weight is None else _ptr(k_weight, dev), _ints(cu_tokens, "cu_tokens", n + 1, dev), _ints(start, "start", n, dev),
              0 if positions is None else _ints(positions, "positions", N, dev), _w_type(None if q is None else q_weight, k_weight), eps, _err(err, dev))
    _launch(lib().moe_kv8_append, dev, stream, (k, v, q, q_out, q_weight, k_weight, pool, page_table, cu_tokens, start, positions, err,
                                                None if rope is None else rope.turns), x)
    return q_out


def token_logprobs(logits, ids=None, top=0, scale=1.0, stream=None):
    """Of rows of logits [rows, vocab], with p = softmax(scale * logits): log p of the given tokens, ids int32 [rows, n] (-inf for
    an id outside the vocabulary, such as -1 for none); the `top` (up to 32) most likely tokens' log p and ids, equal logits in order of
    their ids; the entropy; and the log-sum-exp. Log p is at most 0, the entropy at least 0. Returns (logprobs fp32 [rows, n], top_logprobs fp32 [rows, top], top_ids
    int32 [rows, top], entropy fp32 [rows], lse fp32 [rows]), None for what was not asked for."""
    dev = _device(logits)
    shape = logits.shape
    if len(shape) != 2 or (logits.stride(1) != 1 and shape[1] > 1):
        raise MoeError("logits: [rows, vocab] with contiguous rows expected")
    if not 0 <= top <= 32:
        raise MoeError("top: 0 to 32 expected")
    R, V = shape
    n, given = 0, 0
    if ids is not None:
        if len(ids.shape) != 2 or ids.shape[0] != R:
            raise MoeError(f"ids: [{R}, n] expected")
        n = ids.shape[1]
        given = _ints(ids, "ids", R * n, dev)
    device = logits.device
    logprobs = None if ids is None else _empty(stream, (R, n), torch.float32, device)
    top_lp, top_ids = (_empty(stream, (R, top), torch.float32, device), _empty(stream, (R, top), torch.int32, device)) if top else (None, None)
    entropy, lse = _empty(stream, (R,), torch.float32, device), _empty(stream, (R,), torch.float32, device)
    if R:
        x = _pack(_pack_logprobs, logits.data_ptr(), logits.stride(0) if R > 1 else V, _elem(logits), R, V, n, top, scale, given,
                  logprobs.data_ptr() if n else 0, top_lp.data_ptr() if top else 0, top_ids.data_ptr() if top else 0, entropy.data_ptr(), lse.data_ptr())
        _launch(lib().moe_token_logprobs, dev, stream, (logits, ids, logprobs, top_lp, top_ids, entropy, lse), x)
    return logprobs, top_lp, top_ids, entropy, lse


def expert_grouped(*args, stream=None, **kw):
    ExpertCall(*args, **kw)(stream)


def transcode_cb(src_type, codebook, dst_type, K, rows, src_table, dst_table, err=None, stream=None):
    """Load-time transcoding of CB2/CB3 blobs (device pointer tables) into slot layouts."""
    _check(lib().moe_transcode_cb(_fmt(src_type, codebook), dst_type, K, rows, src_table.shape[0], _dp(src_table),
                                  _dp(dst_table), _dp(err), _stream(stream)))


def test_block_isum(typ, codebook, K, blob, rows, xq_row, isum, stream=None):
    """Test hook: per-block integer sums of `rows` rows of `blob` against one q8_1 row."""
    _check(lib().moe_test_block_isum(_fmt(typ, codebook), K, _dp(blob), rows, _dp(xq_row), _dp(isum),
                                     _stream(stream)))
