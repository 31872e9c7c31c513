"""The decoder-layer operators around the MoE layer: norm, cache append, attention, linear.

Binding of moe_add_rms_norm, moe_kv_* and moe_linear (include/moehost.h) for torch
tensors.  Types, shapes and strides are read from the tensors and checked before the C
call, which sees only pointers; a call that does not fit raises MoeError with
MOE_ERR_INVALID_ARG and launches nothing.  Outputs are the caller's tensors.  The checks
of the four calls are native code (csrc/binding.cc), since a call on small inputs takes
longer on the host than on the GPU.
"""
from __future__ import annotations

import ctypes

import torch

try:
    from . import _decoder_ops
except ImportError as e:  # as for the library itself: there is no other path
    raise ImportError("the extension moe_decode_host_gb300/_decoder_ops is missing or does not load: build the library first "
                      "(python moe_decode_host_gb300/build.py, or __graft_entry__.build())") from e
from ._lib import MOE_ERR_INVALID_ARG, MoeError, check, lib, moe_kv_params

_TYPES = (torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn)  # MOE_BF16 .. MOE_E4M3

# the C entry points that the binding calls
_CALLS = tuple(ctypes.cast(f, ctypes.c_void_p).value
               for f in (lib.moe_add_rms_norm, lib.moe_kv_append, lib.moe_kv_attend, lib.moe_linear))


def _bind(raw_stream=torch._C._cuda_getCurrentRawStream, current_device=torch._C._cuda_getDevice, calls=_CALLS):
    _decoder_ops.bind(MoeError, raw_stream, current_device, _TYPES + (torch.int32, torch.int64), calls)


_bind()

moe_add_rms_norm = _decoder_ops.moe_add_rms_norm
moe_kv_append = _decoder_ops.moe_kv_append
moe_kv_attend = _decoder_ops.moe_kv_attend
moe_linear = _decoder_ops.moe_linear


class KvCache:
    """Handle of one layer's paged key-value cache (moe_kv_create).

    k, v: [n_pages, page_size, kv_heads, head_dim] (a transposed view of pages that
    hold their heads first fits too), bfloat16, float16, or float8_e4m3fn with k_scale
    and v_scale fp32 [kv_heads].  The tensors are borrowed and kept alive by the
    handle.  max_batch: most sequences of one moe_kv_attend call."""

    def __init__(self, k, v, *, q_heads: int, max_batch: int, k_scale=None, v_scale=None):
        w = "moe_kv_create"
        self.handle = self._call = None

        def refuse(why):
            raise MoeError(MOE_ERR_INVALID_ARG, f"{w}: {why}")

        if k.dtype not in _TYPES or v.dtype != k.dtype:
            refuse("k and v are not of one known type")
        if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride():
            refuse("k and v are not [n_pages, page_size, kv_heads, head_dim] with one set of strides")
        if not k.is_cuda or not v.is_cuda or k.stride(3) != 1:
            refuse("k and v are not on a GPU or not contiguous in their last dimension")
        # the handle's workspace is on the current device, and its calls run there
        device = k.get_device()
        if device != torch._C._cuda_getDevice():
            refuse("k is not on the current GPU")
        if any(t is not None and t.get_device() != device for t in (v, k_scale, v_scale)):
            refuse("its tensors are not on one GPU")
        n_pages, page, kv_heads, dim = k.shape
        for s in (k_scale, v_scale):
            if s is not None and (s.dtype != torch.float32 or not s.is_cuda or s.shape != (kv_heads,)
                                  or (kv_heads > 1 and s.stride(0) != 1)):
                refuse("a scale is not a contiguous CUDA fp32 [kv_heads]")
        if any(not 0 <= n < 1 << 31 for n in (n_pages, page, kv_heads, q_heads, dim, max_batch)):
            refuse("a size is out of range")  # the structure below would take its low 32 bits
        p = moe_kv_params(n_pages, page, kv_heads, q_heads, dim, _TYPES.index(k.dtype), max_batch, k.stride(0),
                          k.stride(1), k.stride(2))
        h = ctypes.c_void_p()
        check(lib.moe_kv_create(ctypes.byref(p), k.data_ptr(), v.data_ptr(),
                                0 if k_scale is None else k_scale.data_ptr(),
                                0 if v_scale is None else v_scale.data_ptr(), ctypes.byref(h)), w)
        self.handle = h
        self._call = (h.value, q_heads, kv_heads, dim, device)  # what the calls read
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, dim
        self.page_size, self.n_pages, self.max_batch = page, n_pages, max_batch

    def close(self):
        if self.handle:
            self._call = None
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
