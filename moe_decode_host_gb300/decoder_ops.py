"""The decoder-layer operators around the MoE layer: norm, cache append, attention, linear.

Binding of moe_add_rms_norm, moe_kv_* and moe_linear (include/moehost.h) for torch
tensors.  Shapes, strides and element types are read from the tensors and checked
here, since the C side sees only pointers; a call that does not fit raises MoeError
with MOE_ERR_INVALID_ARG and launches nothing.  Outputs are the caller's tensors.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import (MOE_ACT_GELU, MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_SILU, MOE_BF16, MOE_E4M3, MOE_ERR_INVALID_ARG,
                   MOE_F16, MOE_F32, MoeError, check, lib, moe_kv_params, stream_handle)

_TYPE = {torch.bfloat16: MOE_BF16, torch.float16: MOE_F16, torch.float32: MOE_F32, torch.float8_e4m3fn: MOE_E4M3}
_ACT = {None: MOE_ACT_NONE, "none": MOE_ACT_NONE, "relu": MOE_ACT_RELU, "silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU}


# cudaStream_t of a device's current torch stream, without building a Stream object (3 us)
_raw_stream = torch._C._cuda_getCurrentRawStream


def _refuse(where: str, why: str):
    raise MoeError(MOE_ERR_INVALID_ARG, f"{where}: {why}")


def _stream(stream, t) -> int:
    return _raw_stream(t.get_device()) if stream is None else stream_handle(stream)


def _type(t, where: str, name: str) -> int:
    """Type code of a tensor of one of the four types."""
    code = _TYPE.get(t.dtype, -1)
    if code < 0:
        _refuse(where, f"{name} has type {t.dtype}")
    return code


def _rows(t, shape, where: str, name: str) -> int:
    """Row stride of a CUDA tensor [rows, n] of that shape with contiguous rows."""
    if t.shape != shape or not t.is_cuda:
        _refuse(where, f"{name} is not a CUDA tensor {list(shape)}")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        _refuse(where, f"{name} is not contiguous in its last dimension")
    return s0


def _vector(t, n: int, where: str, name: str, dtype=None) -> int:
    """Pointer of a contiguous CUDA vector of n elements (of one type)."""
    if (dtype is not None and t.dtype != dtype) or not t.is_cuda or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        _refuse(where, f"{name} is not a contiguous CUDA vector of {n} {'elements' if dtype is None else dtype}")
    return t.data_ptr()


def moe_add_rms_norm(x, weight, y, residual=None, sum_out=None, scale=None, eps=1e-6, stream=None):
    """s = x + residual; sum_out = s; y = s * rsqrt(mean(s^2) + eps) * weight, row by row.

    x [T, H]; residual and sum_out [T, H] of one type (each may be None); weight [H] or
    None; y [T, H].  A float8_e4m3fn y holds y / scale[t], scale [T] fp32 being the
    row's largest |y| / 448.  sum_out may be residual or x; y may be x."""
    w = "moe_add_rms_norm"
    shape = x.shape
    if len(shape) != 2:
        _refuse(w, "x is not [T, H]")
    T, H = shape
    xt, xs = _type(x, w, "x"), _rows(x, shape, w, "x")
    yt, ys = _type(y, w, "y"), _rows(y, shape, w, "y")
    rp = rs = sp = ss = wp = wt = rt = cp = 0
    if residual is not None:
        rt, rs, rp = _type(residual, w, "residual"), _rows(residual, shape, w, "residual"), residual.data_ptr()
    if sum_out is not None:
        if residual is not None and sum_out.dtype != residual.dtype:
            _refuse(w, "sum_out has another type than residual")
        rt, ss, sp = _type(sum_out, w, "sum_out"), _rows(sum_out, shape, w, "sum_out"), sum_out.data_ptr()
    if weight is not None:
        wt, wp = _type(weight, w, "weight"), _vector(weight, H, w, "weight")
    if scale is not None:
        cp = _vector(scale, T, w, "scale", torch.float32)
    check(lib.moe_add_rms_norm(x.data_ptr(), xt, xs, rp, rt, rs, wp, wt, eps, T, H, sp, ss, y.data_ptr(), yt, ys, cp,
                               _stream(stream, x)), w)


class KvCache:
    """Handle of one layer's paged key-value cache (moe_kv_create).

    k, v: [n_pages, page_size, kv_heads, head_dim] (a transposed view of pages that
    hold their heads first fits too), bfloat16, float16, or float8_e4m3fn with k_scale
    and v_scale fp32 [kv_heads].  The tensors are borrowed and kept alive by the
    handle.  max_batch: most sequences of one moe_kv_attend call."""

    def __init__(self, k, v, *, q_heads: int, max_batch: int, k_scale=None, v_scale=None):
        w = "moe_kv_create"
        self.handle = None
        t = _type(k, w, "k")
        if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride() or v.dtype != k.dtype:
            _refuse(w, "k and v are not [n_pages, page_size, kv_heads, head_dim] of one type and one set of strides")
        if not k.is_cuda or not v.is_cuda or k.stride(3) != 1:
            _refuse(w, "k and v are not on a GPU or not contiguous in their last dimension")
        n_pages, page, kv_heads, dim = k.shape
        ks = vs = 0
        if k_scale is not None:
            ks = _vector(k_scale, kv_heads, w, "k_scale", torch.float32)
        if v_scale is not None:
            vs = _vector(v_scale, kv_heads, w, "v_scale", torch.float32)
        p = moe_kv_params(n_pages, page, kv_heads, q_heads, dim, t, max_batch, k.stride(0), k.stride(1), k.stride(2))
        h = ctypes.c_void_p()
        check(lib.moe_kv_create(ctypes.byref(p), k.data_ptr(), v.data_ptr(), ks, vs, ctypes.byref(h)), w)
        self.handle = h
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.type, self.q_heads, self.kv_heads, self.head_dim = t, q_heads, kv_heads, dim
        self.page_size, self.n_pages, self.max_batch = page, n_pages, max_batch

    def close(self):
        if self.handle:
            lib.moe_kv_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def status(self) -> int:
        s = ctypes.c_int()
        check(lib.moe_kv_get_status(self.handle, ctypes.byref(s)), "moe_kv_get_status")
        return int(s.value)

    def clear_status(self):
        check(lib.moe_kv_clear_status(self.handle), "moe_kv_clear_status")


def _heads(t, shape, dtype, where: str, name: str):
    """(pointer, outer stride, head stride) of a [rows, heads, head_dim] tensor."""
    if t.shape != shape or t.dtype != dtype or not t.is_cuda:
        _refuse(where, f"{name} is not a CUDA tensor {list(shape)} of the call's type")
    s0, s1, s2 = t.stride()
    if s2 != 1:
        _refuse(where, f"{name} is not contiguous in its last dimension")
    return t.data_ptr(), s0, s1


def moe_kv_append(kv: KvCache, q, k, v, positions, slots, cos_sin, q_out, interleaved=False, stream=None):
    """Rotates q and k by position, writes q to q_out and k, v to their cache slots.

    q, q_out [T, q_heads, head_dim]; k, v [T, kv_heads, head_dim], strided views of a
    fused projection's rows among them; positions int32 [T]; slots int64 [T] (page *
    page_size + entry, negative: not appended); cos_sin fp32 [positions, rot_dim]
    (cosines, then sines), or None for no rotation.  interleaved pairs (2i, 2i + 1)
    instead of (i, i + rot_dim / 2).  q_out may be q."""
    w = "moe_kv_append"
    code = _type(q, w, "q")
    T, dtype = len(q), q.dtype
    qs, ks = (T, kv.q_heads, kv.head_dim), (T, kv.kv_heads, kv.head_dim)
    qp, q0, q1 = _heads(q, qs, dtype, w, "q")
    kp, k0, k1 = _heads(k, ks, dtype, w, "k")
    vp, v0, v1 = _heads(v, ks, dtype, w, "v")
    op, o0, o1 = _heads(q_out, qs, dtype, w, "q_out")
    pp = tp = n_pos = rot = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32 or not cos_sin.is_cuda or not cos_sin.is_contiguous():
            _refuse(w, "cos_sin is not a contiguous CUDA fp32 [positions, rot_dim]")
        tp = cos_sin.data_ptr()
        n_pos, rot = cos_sin.shape
        pp = _vector(positions, T, w, "positions", torch.int32)
    sp = _vector(slots, T, w, "slots", torch.int64)
    check(lib.moe_kv_append(kv.handle, code, qp, q0, q1, kp, k0, k1, vp, v0, v1, pp, sp, tp, n_pos, rot,
                            1 if interleaved else 0, T, op, o0, o1, _stream(stream, q)), w)


def moe_kv_attend(kv: KvCache, q, page_table, lengths, out, scale=None, window=0, lse=None, stream=None):
    """Attention of one query token per sequence over the cache.

    q, out [B, q_heads, head_dim] bfloat16 or float16; page_table int32 [B, max_pages]
    (an expanded single row fits); lengths int32 [B]; scale defaults to
    head_dim ** -0.5; window: only the last `window` tokens count (0: all); lse fp32
    [B, q_heads] receives the log of the softmax sums."""
    w = "moe_kv_attend"
    code = _type(q, w, "q")
    B, dtype = len(q), q.dtype
    shape = (B, kv.q_heads, kv.head_dim)
    qp, q0, q1 = _heads(q, shape, dtype, w, "q")
    op, o0, o1 = _heads(out, shape, dtype, w, "out")
    if page_table.dtype != torch.int32 or not page_table.is_cuda or page_table.dim() != 2 or len(page_table) != B:
        _refuse(w, "page_table is not a CUDA int32 [B, max_pages]")
    per = page_table.shape[1]
    t0, t1 = page_table.stride()
    if per > 1 and t1 != 1:
        _refuse(w, "page_table is not contiguous in its last dimension")
    lp = _vector(lengths, B, w, "lengths", torch.int32)
    zp = 0
    if lse is not None:
        if lse.dtype != torch.float32 or not lse.is_cuda or lse.shape != (B, kv.q_heads) or not lse.is_contiguous():
            _refuse(w, "lse is not a contiguous CUDA fp32 [B, q_heads]")
        zp = lse.data_ptr()
    if scale is None:
        scale = kv.head_dim ** -0.5
    check(lib.moe_kv_attend(kv.handle, qp, code, q0, q1, page_table.data_ptr(), t0, per, lp, B, scale, window, op, o0,
                            o1, zp, _stream(stream, q)), w)


def moe_linear(x, w, y, bias=None, act="none", residual=None, x_scale=None, w_scale=None, status=None,
               stream=None):
    """y = act(x w^T [* x_scale[t] * w_scale[n]] + bias) + residual.

    x [T, K] and w [N, K] of one type: bfloat16, float16, or float8_e4m3fn with
    x_scale fp32 [T] and w_scale fp32 [N]; y [T, N] bfloat16, float16 or float32;
    bias [N]; residual [T, N] of y's type (may be y); act "none", "relu", "silu" or
    "gelu" (exact); status int32 [1], set to MOE_ERR_TIMEOUT if a device wait ran out."""
    f = "moe_linear"
    shape, wide = x.shape, w.shape
    if len(shape) != 2 or len(wide) != 2 or shape[1] != wide[1]:
        _refuse(f, "x is not [T, K] or w is not [N, K]")
    T, K = shape
    N = wide[0]
    code, yt = _type(x, f, "x"), _type(y, f, "y")
    if w.dtype != x.dtype:
        _refuse(f, "x and w have different types")
    xs, ws, ys = _rows(x, shape, f, "x"), _rows(w, wide, f, "w"), _rows(y, (T, N), f, "y")
    bp = bt = rp = rs = xp = wp = sp = 0
    if bias is not None:
        bt, bp = _type(bias, f, "bias"), _vector(bias, N, f, "bias")
    if residual is not None:
        if residual.dtype != y.dtype:
            _refuse(f, "residual has another type than y")
        rp, rs = residual.data_ptr(), _rows(residual, (T, N), f, "residual")
    if x_scale is not None:
        xp = _vector(x_scale, T, f, "x_scale", torch.float32)
    if w_scale is not None:
        wp = _vector(w_scale, N, f, "w_scale", torch.float32)
    if status is not None:
        sp = _vector(status, 1, f, "status", torch.int32)
    check(lib.moe_linear(x.data_ptr(), xs, w.data_ptr(), ws, code, T, N, K, xp, wp, bp, bt, _ACT.get(act, -1), rp, rs,
                         y.data_ptr(), yt, ys, sp, _stream(stream, x)), f)
