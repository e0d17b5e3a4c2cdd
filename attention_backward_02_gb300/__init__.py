"""GB300 (sm_103a) SDPA backward (FlashAttention-2 form) and NSA selected-attention
backward behind a C ABI (include/attnbwd.h).

The functions here marshal torch CUDA tensors into the C ABI: pointers,
strides, the caller's stream and a caller-sized workspace.  PyTorch only
provides device memory and streams; all arithmetic runs in the library's
CUDA kernels.
"""
from __future__ import annotations

import ctypes as C
import math
import struct

from . import _lib
from ._lib import (ATTN_BF16, ATTN_CAUSAL_BOTTOM_RIGHT, ATTN_CAUSAL_TOP_LEFT, ATTN_DQ_ATOMIC, ATTN_DQ_ORDERED,
                   ATTN_DQ_SPLIT, ATTN_E4M3, ATTN_F16, ATTN_F32, ATTN_MASK_NONE, AttnError, attn_nsa_desc_t,
                   attn_paged_cache_t, attn_qk_norm_desc_t, attn_relbias_t, attn_sdpa_desc_t,
                   attn_view_t, check)

__all__ = ["sdpa_desc", "nsa_desc", "view_bhsd", "view_tnd", "sdpa_workspace_size", "sdpa_fwd_stats",
           "sdpa_bwd", "nsa_workspace_size", "nsa_selected_attn_bwd", "nsa_block_lists",
           "nsa_fwd_workspace_size", "nsa_selected_attn_fwd",
           "relbias", "relbias_bucket", "sdpa_relbias_workspace_size", "sdpa_relbias_fwd_stats", "sdpa_relbias_bwd",
           "sdpa_relbias_decode_workspace_size", "sdpa_relbias_decode",
           "paged_cache", "paged_cache_workspace_size", "paged_cache_write", "paged_cache_read",
           "sdpa_paged_workspace_size", "sdpa_paged_fwd",
           "qk_norm_rope_desc", "qk_norm_rope_workspace_size", "qk_norm_rope_fwd", "qk_norm_rope_bwd",
           "attn_query_status", "AttnError", "ATTN_F16", "ATTN_BF16", "ATTN_F32", "ATTN_E4M3",
           "ATTN_MASK_NONE",
           "ATTN_CAUSAL_TOP_LEFT", "ATTN_CAUSAL_BOTTOM_RIGHT"]


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float16:
        return ATTN_F16
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    raise TypeError(f"fp16 or bf16 expected, got {t.dtype}")


def _stream_ptr(stream) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


class _Keep:
    """Holds ctypes arrays alive for the duration of a call."""

    def __init__(self):
        self.items = []


def _cu_array(keep, cu):
    if cu is None:
        return None
    arr = (C.c_int64 * len(cu))(*[int(x) for x in cu])
    keep.items.append(arr)
    return C.cast(arr, C.POINTER(C.c_int64))


def sdpa_desc(*, dtype, b, h, h_kv, s_q, s_kv, d, scale, mask=ATTN_MASK_NONE, cu_seqlens_q=None,
              cu_seqlens_kv=None, deterministic=False, dq_splits=0, _keep=None):
    """An attn_sdpa_desc_t.  Fixed-length mode: b sequences of s_q queries and s_kv keys.  Packed
    (varlen) mode: cu_seqlens_q / cu_seqlens_kv, b inclusive cumulative lengths each (s_q, s_kv then
    ignored).  scale multiplies q.k; mask is ATTN_MASK_NONE, ATTN_CAUSAL_TOP_LEFT or
    ATTN_CAUSAL_BOTTOM_RIGHT.  deterministic: False / ATTN_DQ_ATOMIC, True / ATTN_DQ_SPLIT (dq_splits
    partial buffers, 0: a default) or ATTN_DQ_ORDERED (one buffer, adds in a fixed order); the last two
    make dQ bitwise reproducible.  The host arrays live as long as the descriptor."""
    keep = _keep if _keep is not None else _Keep()
    mode = int(deterministic) if not isinstance(deterministic, bool) else int(deterministic)
    desc = attn_sdpa_desc_t(int(dtype), int(b), int(h), int(h_kv), int(s_q), int(s_kv), int(d), float(scale),
                            int(mask), _cu_array(keep, cu_seqlens_q), _cu_array(keep, cu_seqlens_kv),
                            mode, int(dq_splits))
    desc._keep = keep
    return desc


def nsa_desc(*, dtype, cu_seqlens_q, cu_seqlens_kv, n1, n2, d, scale, block_size, block_count, sparse_mode,
             deterministic=False, d_v=0, grad_fp32=False, atten_mask=None):
    """An attn_nsa_desc_t: TND layout, b = len(cu_seqlens_q) sequences with inclusive cumulative query /
    key lengths, n1 query and n2 kv heads, query / key head dim d and value head dim d_v (0: d),
    scaleValue, selectedBlockSize / Count, sparseMode 0 (selection only) or 2 (also causal,
    bottom-right per sequence); deterministic makes dq, dk, dv bitwise reproducible (tensor-core head
    groups only): False / 0 atomic adds, True / 1 per-slot dQ partials summed in slot order, 2 one dQ
    accumulator whose adds per token go in decreasing block order (ATTN_DQ_ORDERED); grad_fp32 makes dq, dk, dv fp32; atten_mask (attenMaskOptional) is a 2-D uint8 CUDA
    tensor [rows, cols] over local (query, key) positions, nonzero = key removed, covering every
    sequence (held by the descriptor)."""
    keep = _Keep()
    if atten_mask is not None:
        if atten_mask.dim() != 2 or not atten_mask.is_contiguous() or atten_mask.element_size() != 1:
            raise ValueError("atten_mask: a contiguous 2-D tensor of 1-byte elements")
        keep.items.append(atten_mask)
    desc = attn_nsa_desc_t(int(dtype), len(cu_seqlens_q), _cu_array(keep, cu_seqlens_q),
                           _cu_array(keep, cu_seqlens_kv), int(n1), int(n2), int(d), float(scale),
                           int(block_size), int(block_count), int(sparse_mode), int(deterministic),
                           int(d_v), int(bool(grad_fp32)),
                           atten_mask.data_ptr() if atten_mask is not None else None,
                           int(atten_mask.shape[0]) if atten_mask is not None else 0,
                           int(atten_mask.shape[1]) if atten_mask is not None else 0)
    desc._keep = keep
    return desc


def view_bhsd(t) -> attn_view_t:
    """A [B, H, S, D] tensor (any strides, innermost 1) as an attn_view_t."""
    if t.dim() != 4 or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError("expected a [B,H,S,D] tensor with unit innermost stride")
    sb, sh, ss, _ = t.stride()
    return attn_view_t(t.data_ptr(), sb, sh, ss)


def view_tnd(t) -> attn_view_t:
    """A packed [T, H, D] tensor as an attn_view_t (token stride = ss)."""
    if t.dim() != 3 or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError("expected a [T,H,D] tensor with unit innermost stride")
    st, sh, _ = t.stride()
    return attn_view_t(t.data_ptr(), 0, sh, st)


def sdpa_workspace_size(desc):
    """(forward bytes, backward bytes) of device workspace for this descriptor (host only)."""
    fwd, bwd = C.c_size_t(), C.c_size_t()
    check(_lib.load().sdpa_workspace_size(C.byref(desc), C.byref(fwd), C.byref(bwd)), "sdpa_workspace_size")
    return fwd.value, bwd.value


def _workspace(nbytes, device, workspace, stream):
    """The caller's workspace, or memory of the stream that the call runs on: that of the current stream might
    still be in use by earlier work there, and would go back to it before the call is done."""
    torch = _torch()
    if workspace is not None:
        return workspace
    if stream is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def sdpa_fwd_stats(desc, q, k, v, o, lse, *, workspace=None, stream=None):
    """q, k, v, o: views (attn_view_t) or tensors; lse: fp32 CUDA tensor."""
    fwd, _ = sdpa_workspace_size(desc)
    ws = _workspace(fwd, lse.device, workspace, stream)
    vq, vk, vv, vo = (x if isinstance(x, attn_view_t) else view_bhsd(x) for x in (q, k, v, o))
    st = _lib.load().sdpa_fwd_stats(C.byref(desc), vq, vk, vv, vo,
                                    C.cast(C.c_void_p(lse.data_ptr()), C.POINTER(C.c_float)),
                                    C.c_void_p(ws.data_ptr()), C.c_size_t(ws.numel()), C.c_void_p(_stream_ptr(stream)))
    check(st, "sdpa_fwd_stats")
    return ws


def sdpa_bwd(desc, q, k, v, o, dO, lse, dQ, dK, dV, *, workspace=None, stream=None):
    """dQ, dK, dV of scaled dot-product attention from O, dO and the fp32 stats lse (as sdpa_fwd_stats
    writes them).  Tensors are attn_view_t views or [B, H, S, D] CUDA tensors (view_bhsd); the call is
    asynchronous on `stream` (default: the current stream).  A workspace of the size
    sdpa_workspace_size gives is allocated when none is passed; it is returned, for attn_query_status."""
    _, bwd = sdpa_workspace_size(desc)
    ws = _workspace(bwd, lse.device, workspace, stream)
    views = [x if isinstance(x, attn_view_t) else view_bhsd(x) for x in (q, k, v, o, dO, dQ, dK, dV)]
    st = _lib.load().sdpa_bwd(C.byref(desc), *views[:5],
                              C.cast(C.c_void_p(lse.data_ptr()), C.POINTER(C.c_float)), *views[5:],
                              C.c_void_p(ws.data_ptr()), C.c_size_t(ws.numel()), C.c_void_p(_stream_ptr(stream)))
    check(st, "sdpa_bwd")
    return ws


def nsa_workspace_size(desc):
    """Bytes of device workspace nsa_selected_attn_bwd needs for this descriptor (host only)."""
    n = C.c_size_t()
    check(_lib.load().nsa_workspace_size(C.byref(desc), C.byref(n)), "nsa_workspace_size")
    return n.value


def nsa_selected_attn_bwd(desc, q, k, v, o, dO, softmax_max, softmax_sum, topk, dq, dk, dv, *, workspace=None,
                          stream=None):
    """NSA selected-attention backward on contiguous TND CUDA tensors: q, o, dO, dq [T1, n1, d]; k, v,
    dk, dv [T2, n2, d]; softmax_max / softmax_sum [T1, n1, 8] fp32; topk [T1, n2, block_count] int32.
    Asynchronous on `stream`; returns the workspace (allocated when none is passed) for
    attn_query_status, which reports indices that were out of range or repeated."""
    ws = _workspace(nsa_workspace_size(desc), q.device, workspace, stream)
    fp = lambda t: C.cast(C.c_void_p(t.data_ptr()), C.POINTER(C.c_float))
    st = _lib.load().nsa_selected_attn_bwd(
        C.byref(desc), *(C.c_void_p(t.data_ptr()) for t in (q, k, v, o, dO)), fp(softmax_max), fp(softmax_sum),
        C.cast(C.c_void_p(topk.data_ptr()), C.POINTER(C.c_int32)),
        *(C.c_void_p(t.data_ptr()) for t in (dq, dk, dv)), C.c_void_p(ws.data_ptr()), C.c_size_t(ws.numel()),
        C.c_void_p(_stream_ptr(stream)))
    check(st, "nsa_selected_attn_bwd")
    return ws


def nsa_fwd_workspace_size(desc):
    """Bytes of device workspace nsa_selected_attn_fwd needs (host only)."""
    n = C.c_size_t()
    check(_lib.load().nsa_fwd_workspace_size(C.byref(desc), C.byref(n)), "nsa_fwd_workspace_size")
    return n.value


def nsa_selected_attn_fwd(desc, q, k, v, topk, o, softmax_max, softmax_sum, *, workspace=None, stream=None):
    """NSA selected-attention forward on contiguous TND CUDA tensors: q [T1, n1, d], k [T2, n2, d],
    v [T2, n2, d_v], topk [T1, n2, block_count] int32 -> o [T1, n1, d_v] (input dtype), softmax_max /
    softmax_sum [T1, n1, 8] fp32.  Asynchronous on `stream`; returns the workspace (its first word is the
    device status)."""
    ws = _workspace(nsa_fwd_workspace_size(desc), q.device, workspace, stream)
    fp = lambda t: C.cast(C.c_void_p(t.data_ptr()), C.POINTER(C.c_float))
    st = _lib.load().nsa_selected_attn_fwd(
        C.byref(desc), *(C.c_void_p(t.data_ptr()) for t in (q, k, v)),
        C.cast(C.c_void_p(topk.data_ptr()), C.POINTER(C.c_int32)), C.c_void_p(o.data_ptr()), fp(softmax_max),
        fp(softmax_sum), C.c_void_p(ws.data_ptr()), C.c_size_t(ws.numel()), C.c_void_p(_stream_ptr(stream)))
    check(st, "nsa_selected_attn_fwd")
    return ws


def nsa_block_lists(desc, topk, offsets, tokens, *, workspace=None, stream=None):
    """Fills device int32 tensors offsets / tokens; returns nblk_max."""
    ws = _workspace(nsa_workspace_size(desc), topk.device, workspace, stream)
    ip = lambda t: C.cast(C.c_void_p(t.data_ptr()), C.POINTER(C.c_int32))
    nblk = C.c_int64()
    st = _lib.load().nsa_block_lists(C.byref(desc), ip(topk), ip(offsets), ip(tokens), C.byref(nblk),
                                     C.c_void_p(ws.data_ptr()), C.c_size_t(ws.numel()),
                                     C.c_void_p(_stream_ptr(stream)))
    check(st, "nsa_block_lists")
    return nblk.value, ws


class _Call:
    """One call on CUDA tensors that all live on one device: checks them, makes that device current for
    the call, and holds the stream and workspace it runs with.  These checks are most of a small call's
    time, so they read each property of a tensor once (the raw stream and device queries are the ones
    torch's own generated code uses: 0.1 us instead of 1.5)."""

    __slots__ = ("where", "dtype", "device", "stream", "given")

    def __init__(self, where, dtype, device, stream):
        torch = _torch()
        self.where, self.dtype, self.device = where, torch.float16 if dtype == ATTN_F16 else torch.bfloat16, device
        if device < 0:
            raise ValueError(f"{where}: CUDA tensors expected")
        self.given = stream
        if stream is None:
            self.stream = torch._C._cuda_getCurrentRawStream(device)
        else:
            self.stream = stream.cuda_stream
            if stream.device.index != device:
                raise ValueError(f"{where}: tensors on cuda:{device}, stream on {stream.device}")

    def refuse(self, name, t, dtype, shape):
        raise ValueError(f"{self.where}: {name} must be {dtype} {tuple(shape)} on cuda:{self.device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}, strides {t.stride()}")

    def ptr(self, name, t, dtype, shape):
        """Address of a contiguous tensor (None stays None: a NULL pointer)."""
        if t is None:
            return None
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self.device or not t.is_contiguous():
            self.refuse(name, t, dtype, shape)
        return t.data_ptr()

    def view(self, name, x, shape):
        """x: an attn_view_t, or a [B, H, S, D] tensor of this shape with a unit innermost stride."""
        if type(x) is attn_view_t:
            return x
        st = x.stride()
        if x.dtype is not self.dtype or x.shape != shape or x.get_device() != self.device or st[3] != 1:
            self.refuse(name, x, self.dtype, shape)
        return attn_view_t(x.data_ptr(), st[0], st[1], st[2])

    def workspace(self, nbytes, workspace):
        if workspace is None:
            return _workspace(nbytes, _torch().device("cuda", self.device), None, self.given)
        if workspace.get_device() != self.device or not workspace.is_contiguous():
            raise ValueError(f"{self.where}: workspace on {workspace.device}, tensors on cuda:{self.device}")
        return workspace

    def run(self, fn, *args):
        torch = _torch()
        if torch._C._cuda_getDevice() == self.device:
            st = fn(*args, self.stream)
        else:
            with torch.cuda.device(self.device):
                st = fn(*args, self.stream)
        if st:
            check(st, self.where)


def relbias(table, *, max_distance=128, bidirectional=True):
    """An attn_relbias_t: a learned relative position bias.  table [num_buckets, h] (fp32, fp16 or bf16; held by
    the result, and read anew by every call): table[bucket(key position - query position), head] is added to
    the score.  Half of a direction's buckets are exact distances, the rest grow to max_distance;
    bidirectional: keys after the query have buckets of their own."""
    bias = attn_relbias_t(None, 0, 0, int(max_distance), int(bool(bidirectional)))
    bias.tensor = table
    _read_table(bias)
    return bias


def _read_table(bias):
    """The table's address, type and number of buckets, as its tensor is now: its memory may have been replaced
    (tensor.data = ...) since the last call."""
    torch, t = _torch(), bias.tensor
    code = ATTN_F32 if t.dtype is torch.float32 else {torch.float16: ATTN_F16, torch.bfloat16: ATTN_BF16}.get(t.dtype)
    if code is None or t.dim() != 2 or not t.is_contiguous():
        raise ValueError("relbias: a contiguous [num_buckets, h] table of fp32, fp16 or bf16")
    bias.table, bias.table_type, bias.num_buckets = t.data_ptr(), code, t.shape[0]


def relbias_bucket(bias, delta):
    """Bucket of a key `delta` positions after its query (host only)."""
    n = C.c_int64()
    check(_lib.load().attn_relbias_bucket(C.byref(bias), int(delta), C.byref(n)), "attn_relbias_bucket")
    return n.value


def sdpa_relbias_workspace_size(desc, bias):
    """(forward bytes, backward bytes) of device workspace for this descriptor and bias (host only)."""
    fwd, bwd = C.c_size_t(), C.c_size_t()
    check(_lib.load().sdpa_relbias_workspace_size(C.byref(desc), C.byref(bias), C.byref(fwd), C.byref(bwd)),
          "sdpa_relbias_workspace_size")
    return fwd.value, bwd.value


def _dense_shapes(desc):
    """Shapes of the query-side and key-side tensors and of lse (None where packed views are expected)."""
    if desc.cu_seqlens_q:
        return None, None, None
    return ((desc.b, desc.h, desc.s_q, desc.d), (desc.b, desc.h_kv, desc.s_kv, desc.d), (desc.b, desc.h, desc.s_q))


def _packed_or(call, name, x, shape):
    if shape is None and not isinstance(x, attn_view_t):
        raise ValueError(f"{call.where}: {name}: packed tensors are passed as view_tnd views")
    return call.view(name, x, shape)


def _relbias_call(where, desc, bias, on, stream):
    """The call on the device of the tensor `on`."""
    call = _Call(where, desc.dtype, on.get_device(), stream)
    _read_table(bias)
    if bias.tensor.shape[1] != desc.h or bias.tensor.get_device() != call.device:
        raise ValueError(f"{where}: bias table {tuple(bias.tensor.shape)} on {bias.tensor.device}, {desc.h} heads on "
                         f"{on.device}")
    return call


def _same_order(got, want):
    """Whether a contiguous tensor of shape `got` is one of shape `want` with neighbouring dimensions merged or
    dimensions of 1 added; of other shapes the order of the elements is not known."""
    ends = [{math.prod(s[i:]) for i in range(len(s) + 1)} for s in (got, want)]
    return math.prod(got) == math.prod(want) and ends[0] <= ends[1]


def _lse_ptr(call, desc, lse, shape):
    torch = _torch()
    if shape is None:
        shape = (desc.h, int(desc.cu_seqlens_q[desc.b - 1]))
    if (lse.dtype is not torch.float32 or lse.get_device() != call.device or not lse.is_contiguous() or
            (lse.shape != shape and not _same_order(lse.shape, shape))):
        call.refuse("lse", lse, torch.float32, shape)
    return lse.data_ptr()


def sdpa_relbias_fwd_stats(desc, bias, q, k, v, o, lse, *, workspace=None, stream=None):
    """sdpa_fwd_stats with a learned relative position bias (see relbias) in the scores.  q, k, v, o: views or
    [B, H, S, D] tensors; lse: fp32 [B, h, S_q] (packed: [h, T_q]), or the same elements in a shape that merges
    neighbouring dimensions.  Returns the workspace."""
    call = _relbias_call("sdpa_relbias_fwd_stats", desc, bias, lse, stream)
    ws = call.workspace(sdpa_relbias_workspace_size(desc, bias)[0] if workspace is None else 0, workspace)
    sq, sk, sl = _dense_shapes(desc)
    views = [_packed_or(call, n, x, s) for n, x, s in (("q", q, sq), ("k", k, sk), ("v", v, sk), ("o", o, sq))]
    call.run(_lib.load().sdpa_relbias_fwd_stats, C.byref(desc), C.byref(bias), *views, _lse_ptr(call, desc, lse, sl),
             ws.data_ptr(), ws.numel())
    return ws


def sdpa_relbias_bwd(desc, bias, q, k, v, o, dO, lse, dQ, dK, dV, dtable, *, workspace=None, stream=None):
    """sdpa_bwd with a learned relative position bias in the scores; also the gradient of the bias table,
    dtable: fp32 [num_buckets, h], bitwise reproducible.  lse as in the forward.  Returns the workspace."""
    torch = _torch()
    call = _relbias_call("sdpa_relbias_bwd", desc, bias, lse, stream)
    ws = call.workspace(sdpa_relbias_workspace_size(desc, bias)[1] if workspace is None else 0, workspace)
    sq, sk, sl = _dense_shapes(desc)
    views = [_packed_or(call, n, x, s) for n, x, s in (
        ("q", q, sq), ("k", k, sk), ("v", v, sk), ("o", o, sq), ("dO", dO, sq), ("dQ", dQ, sq), ("dK", dK, sk),
        ("dV", dV, sk))]
    dt = call.ptr("dtable", dtable, torch.float32, tuple(bias.tensor.shape))
    call.run(_lib.load().sdpa_relbias_bwd, C.byref(desc), C.byref(bias), *views[:5], _lse_ptr(call, desc, lse, sl),
             *views[5:], dt, ws.data_ptr(), ws.numel())
    return ws


def sdpa_relbias_decode_workspace_size(desc, bias):
    """Bytes of device workspace sdpa_relbias_decode needs (host only)."""
    n = C.c_size_t()
    check(_lib.load().sdpa_relbias_decode_workspace_size(C.byref(desc), C.byref(bias), C.byref(n)),
          "sdpa_relbias_decode_workspace_size")
    return n.value


def sdpa_relbias_decode(desc, bias, q, k, v, lens, o, *, workspace=None, stream=None):
    """Attention with a learned relative position bias for one new token per sequence: q, o [B, h, 1, D], the
    cache k, v [B, h_kv, S_kv, D] (tensors or views), lens int32 CUDA [B] the keys cached, the new token's
    among them (None: S_kv).  desc: s_q = 1 and ATTN_CAUSAL_BOTTOM_RIGHT.  Returns the workspace, for
    attn_query_status (lengths out of range)."""
    torch = _torch()
    call = _relbias_call("sdpa_relbias_decode", desc, bias, bias.tensor, stream)
    ws = call.workspace(sdpa_relbias_decode_workspace_size(desc, bias) if workspace is None else 0, workspace)
    sq, sk = (desc.b, desc.h, 1, desc.d), (desc.b, desc.h_kv, desc.s_kv, desc.d)
    views = [call.view(n, x, s) for n, x, s in (("q", q, sq), ("k", k, sk), ("v", v, sk), ("o", o, sq))]
    call.run(_lib.load().sdpa_relbias_decode, C.byref(desc), C.byref(bias), *views[:3],
             call.ptr("lens", lens, torch.int32, (desc.b,)), views[3], ws.data_ptr(), ws.numel())
    return ws


def paged_cache(k, v, *, k_scale=None, v_scale=None):
    """An attn_paged_cache_t: a key / value cache in pages.  k, v: [n_pages, page_size, h_kv, d] of the calls' dtype
    or float8_e4m3fn, any strides with a unit innermost one, alike in both (a cache stored by heads is passed
    transposed); float8: k_scale, v_scale fp32 [n_pages, page_size, h_kv] of either sign, strides alike in both.  The tensors
    are held by the result, and read anew by every call."""
    cache = attn_paged_cache_t()
    cache.tensors, cache.as_read = (k, v, k_scale, v_scale), None
    _read_cache(cache)
    return cache


def _read_cache(cache):
    """The pages' addresses, type and strides, as their tensors are now: their memory may have been replaced
    (tensor.data = ...) since the last call.  The struct is written where something has changed (most of a call's
    time here goes into its fields)."""
    k, v, ks, vs = cache.tensors
    now = (k.data_ptr(), v.data_ptr(), k.dtype, v.dtype, k.shape, v.shape, k.stride(), v.stride(), k.get_device(),
           v.get_device())
    if ks is not None and vs is not None:
        now += (ks.data_ptr(), vs.data_ptr(), ks.dtype, vs.dtype, ks.shape, vs.shape, ks.stride(), vs.stride(),
                ks.get_device(), vs.get_device())
    if now == cache.as_read:
        return now[8]
    torch = _torch()
    code = {torch.float16: ATTN_F16, torch.bfloat16: ATTN_BF16, torch.float8_e4m3fn: ATTN_E4M3}.get(k.dtype)
    shape, st = k.shape, k.stride()
    if (code is None or k.dim() != 4 or v.dtype is not k.dtype or v.shape != shape or v.stride() != st or
            now[8] != now[9] or (st[3] != 1 and shape[3] > 1)):
        raise ValueError("paged_cache: k, v [n_pages, page_size, h_kv, d] of fp16, bf16 or float8_e4m3fn with the same "
                         f"strides on one device, got {k.dtype} {tuple(shape)} {st} and {v.dtype} {tuple(v.shape)} "
                         f"{v.stride()}")
    if code == ATTN_E4M3 and (len(now) == 10 or ks.dtype is not torch.float32 or vs.dtype is not torch.float32 or
                              ks.shape != shape[:3] or vs.shape != ks.shape or vs.stride() != ks.stride() or
                              now[18] != now[8] or now[19] != now[8]):
        raise ValueError("paged_cache: float8 pages need k_scale, v_scale fp32 [n_pages, page_size, h_kv] with the "
                         "same strides on the pages' device")
    cache.k, cache.v, cache.type = now[0], now[1], code
    cache.n_pages, cache.page_size = shape[0], shape[1]
    cache.sp, cache.ss, cache.sh = st[0], st[1], st[2]
    if code == ATTN_E4M3:
        cache.k_scale, cache.v_scale = now[10], now[11]
        cache.scale_sp, cache.scale_ss, cache.scale_sh = ks.stride()
    cache.as_read = now
    return now[8]


# an attn_paged_seqs_t's fields (six of 64 bits): packed in a third of the time that a ctypes structure takes
_pack_seqs = struct.Struct("=QqqQQq").pack


def _paged_call(where, desc, cache, page_table, lens, cu_new, tokens, stream):
    """The call on the device of the pages, and its attn_paged_seqs_t."""
    int32 = _torch().int32
    call = _Call(where, desc.dtype, _read_cache(cache), stream)
    shape, dev, b = cache.as_read[4], call.device, desc.b
    if shape[2] != desc.h_kv or shape[3] != desc.d:
        raise ValueError(f"{where}: pages {tuple(shape)}, {desc.h_kv} kv heads of {desc.d}")
    ts, st = page_table.shape, page_table.stride()
    if (page_table.dtype is not int32 or len(ts) != 2 or ts[0] != b or page_table.get_device() != dev or
            (ts[1] > 1 and st[1] != 1)):
        call.refuse("page_table", page_table, int32, (b, -1))
    cu = 0 if cu_new is None else call.ptr("cu_new", cu_new, int32, (b + 1,))
    return call, _pack_seqs(page_table.data_ptr(), st[0], ts[1], call.ptr("lens", lens, int32, (b,)) or 0, cu,
                            tokens)


def _packed_tokens(where, x):
    if type(x) is attn_view_t:
        raise ValueError(f"{where}: packed rows are passed as [T, heads, D] tensors")
    return x.shape[0]


def _paged_rows(call, desc, name, x, heads, packed, tokens):
    """View of the new tokens' rows: [B, heads, S_q, D], packed [tokens, heads, D]."""
    if not packed:
        return call.view(name, x, (desc.b, heads, desc.s_q, desc.d))
    st = x.stride()
    if x.dtype is not call.dtype or x.shape != (tokens, heads, desc.d) or x.get_device() != call.device or st[2] != 1:
        call.refuse(name, x, call.dtype, (tokens, heads, desc.d))
    return attn_view_t(x.data_ptr(), 0, st[1], st[0])


def paged_cache_workspace_size(desc, cache):
    """Bytes of device workspace paged_cache_write and paged_cache_read need (host only)."""
    n = C.c_size_t()
    check(_lib.load().paged_cache_workspace_size(C.byref(desc), C.byref(cache), C.byref(n)), "paged_cache_workspace_size")
    return n.value


def _paged_copy(where, fn, desc, cache, page_table, lens, k, v, cu_new, workspace, stream):
    packed = cu_new is not None
    tokens = _packed_tokens(where, k) if packed else 0
    call, seqs = _paged_call(where, desc, cache, page_table, lens, cu_new, tokens, stream)
    ws = call.workspace(256, workspace)
    views = [_paged_rows(call, desc, n, x, desc.h_kv, packed, tokens) for n, x in (("k", k), ("v", v))]
    call.run(fn, C.byref(desc), C.byref(cache), seqs, *views, ws.data_ptr(), ws.numel())
    return ws


def paged_cache_write(desc, cache, page_table, lens, k, v, *, cu_new=None, workspace=None, stream=None):
    """The new tokens' keys and values into their places of a paged_cache: the last tokens of each sequence, whose
    lens [B] (int32 CUDA) cached tokens they are counted in, page_table [B, pages] (int32 CUDA) naming its pages
    in order.  desc: an sdpa_desc with s_kv = the most tokens a sequence may have cached, s_q = the new tokens
    of each.  k, v: [B, h_kv, S_q, D] tensors or views; with cu_new (int32 CUDA [B + 1], first rows) packed
    [T, h_kv, D] tensors.  float8 pages: each row rounded to e4m3 with a scale of its own (expanded scales, of
    stride 0, can be read through but not written: AttnError).  Returns the
    workspace, for attn_query_status (lengths, counts or page ids out of range)."""
    return _paged_copy("paged_cache_write", _lib.load().paged_cache_write, desc, cache, page_table, lens, k, v, cu_new,
                       workspace, stream)


def paged_cache_read(desc, cache, page_table, lens, k, v, *, cu_new=None, workspace=None, stream=None):
    """The inverse of paged_cache_write: the last tokens of each sequence from the cache into k, v (float8 pages:
    number times scale, rounded).  Returns the workspace, for attn_query_status."""
    return _paged_copy("paged_cache_read", _lib.load().paged_cache_read, desc, cache, page_table, lens, k, v, cu_new,
                       workspace, stream)


def sdpa_paged_workspace_size(desc, cache):
    """Bytes of device workspace sdpa_paged_fwd needs (host only)."""
    n = C.c_size_t()
    check(_lib.load().sdpa_paged_workspace_size(C.byref(desc), C.byref(cache), C.byref(n)), "sdpa_paged_workspace_size")
    return n.value


def sdpa_paged_fwd(desc, cache, page_table, lens, q, o, *, lse=None, cu_new=None, workspace=None, stream=None):
    """Attention of each sequence's new tokens over everything it has in a paged_cache (their own keys and values
    included: paged_cache_write comes first).  desc, page_table, lens, cu_new as there, mask
    ATTN_CAUSAL_BOTTOM_RIGHT (up to a token's own position) or ATTN_MASK_NONE; q, o: [B, h, S_q, D] tensors or
    views, packed [T, h, D]; lse: fp32 [B, h, S_q], packed [h, T], or None.  Returns the workspace, for
    attn_query_status."""
    torch = _torch()
    packed = cu_new is not None
    tokens = _packed_tokens("sdpa_paged_fwd", q) if packed else 0
    call, seqs = _paged_call("sdpa_paged_fwd", desc, cache, page_table, lens, cu_new, tokens, stream)
    ws = call.workspace(sdpa_paged_workspace_size(desc, cache) if workspace is None else 0, workspace)
    views = [_paged_rows(call, desc, n, x, desc.h, packed, tokens) for n, x in (("q", q), ("o", o))]
    stats = call.ptr("lse", lse, torch.float32, (desc.h, tokens) if packed else (desc.b, desc.h, desc.s_q))
    call.run(_lib.load().sdpa_paged_fwd, C.byref(desc), C.byref(cache), seqs, *views, stats, ws.data_ptr(), ws.numel())
    return ws


def qk_norm_rope_desc(*, dtype, b, s, h, h_kv, d, rotary_dim=0, interleaved=False, eps=1e-6, weight_fp32=False,
                      max_pos=0):
    """An attn_qk_norm_desc_t: b sequences of s tokens (packed tensors: b = 1, s = all tokens), h query and
    h_kv key heads of dim d (64, 128 or 192).  The first rotary_dim elements of a head (a multiple of 16;
    0: none) are rotated in pairs (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved, by the rows
    of cos / sin tables of max_pos rows.  weight_fp32: the norm weights are fp32 (else dtype)."""
    return attn_qk_norm_desc_t(int(dtype), int(b), int(s), int(h), int(h_kv), int(d), int(rotary_dim),
                               int(bool(interleaved)), float(eps), int(bool(weight_fp32)), int(max_pos))


def qk_norm_rope_workspace_size(desc):
    """(forward bytes, backward bytes) of device workspace for this descriptor (host only)."""
    fwd, bwd = C.c_size_t(), C.c_size_t()
    check(_lib.load().qk_norm_rope_workspace_size(C.byref(desc), C.byref(fwd), C.byref(bwd)),
          "qk_norm_rope_workspace_size")
    return fwd.value, bwd.value


_NO_VIEW = attn_view_t(None, 0, 0, 0)


def _qk_views(call, desc, named):
    """Views of (name, query tensor, key tensor) triples; a side without heads has none."""
    out = []
    b, n, d = desc.b, desc.s, desc.d
    sq, sk = (b, desc.h, n, d), (b, desc.h_kv, n, d)
    for name, q, k in named:
        out.append(call.view(name + "q", q, sq) if sq[1] else _NO_VIEW)
        out.append(call.view(name + "k", k, sk) if sk[1] else _NO_VIEW)
    return out


def _qk_tables(call, desc, q_weight, k_weight, cos, sin, positions):
    f32 = _torch().float32
    wt, d = (f32 if desc.weight_fp32 else call.dtype), (desc.d,)
    wq, wk = call.ptr("q_weight", q_weight, wt, d), call.ptr("k_weight", k_weight, wt, d)
    rot = desc.rotary_dim
    if not rot:
        return wq, wk, None, None, None
    shape = (desc.max_pos, rot // 2)
    return (wq, wk, call.ptr("cos", cos, f32, shape), call.ptr("sin", sin, f32, shape),
            call.ptr("positions", positions, _torch().int32, (desc.b, desc.s)))


def _qk_device(*tensors):
    for t in tensors:
        if t is not None and type(t) is not attn_view_t:
            return t.get_device()
    return _torch().cuda.current_device()


def qk_norm_rope_fwd(desc, q, k, q_weight, k_weight, cos, sin, q_out, k_out, *, positions=None, workspace=None,
                     stream=None):
    """RMS norm of every query and key head with the rotary position embedding in the same pass: q, q_out
    [B, h, S, D], k, k_out [B, h_kv, S, D] (tensors of any strides with a unit innermost one, or
    attn_view_t views; an output may be its input), weights [D] or None, cos / sin fp32 [max_pos,
    rotary_dim / 2], positions int32 [B, S] (None: a token's index in its sequence).  Asynchronous on
    `stream`; returns the workspace, for attn_query_status (positions out of range)."""
    call = _Call("qk_norm_rope_fwd", desc.dtype, _qk_device(q, k, cos, q_weight, workspace), stream)
    ws = call.workspace(256, workspace)
    views = _qk_views(call, desc, (("", q, k), ("output of ", q_out, k_out)))
    tables = _qk_tables(call, desc, q_weight, k_weight, cos, sin, positions)
    call.run(_lib.load().qk_norm_rope_fwd, C.byref(desc), *views[:2], *tables, *views[2:], ws.data_ptr(), ws.numel())
    return ws


def qk_norm_rope_bwd(desc, q, k, dq_out, dk_out, q_weight, k_weight, cos, sin, dq, dk, dq_weight=None, dk_weight=None,
                     *, positions=None, workspace=None, stream=None):
    """Gradients of qk_norm_rope_fwd: dq, dk (which may be dq_out, dk_out) and the weights' fp32 [D]
    gradients (None: not wanted) from the call's inputs and the gradients dq_out, dk_out of its outputs,
    as sdpa_bwd returns them.  Bitwise reproducible.  Asynchronous on `stream`; returns the workspace."""
    torch = _torch()
    call = _Call("qk_norm_rope_bwd", desc.dtype, _qk_device(q, k, cos, q_weight, workspace), stream)
    ws = call.workspace(qk_norm_rope_workspace_size(desc)[1] if workspace is None else 0, workspace)
    views = _qk_views(call, desc, (("", q, k), ("gradient of the output of ", dq_out, dk_out), ("d", dq, dk)))
    tables = _qk_tables(call, desc, q_weight, k_weight, cos, sin, positions)
    dws = [call.ptr(n, t, torch.float32, (desc.d,)) for n, t in (("dq_weight", dq_weight), ("dk_weight", dk_weight))]
    call.run(_lib.load().qk_norm_rope_bwd, C.byref(desc), *views[:4], *tables, *views[4:], *dws, ws.data_ptr(),
             ws.numel())
    return ws


def attn_query_status(workspace, stream=None):
    """Synchronises the stream (default: the current stream of the workspace's device); returns the device status
    bits (0 = clean)."""
    torch = _torch()
    flags = C.c_uint32()
    with torch.cuda.device(workspace.get_device()):  # a default stream is that of the device that is current
        st = _lib.load().attn_query_status(C.c_void_p(workspace.data_ptr()), C.c_void_p(_stream_ptr(stream)),
                                           C.byref(flags))
    if st not in (_lib.ATTN_OK, _lib.ATTN_ERR_DEVICE):
        check(st, "attn_query_status")
    return flags.value
