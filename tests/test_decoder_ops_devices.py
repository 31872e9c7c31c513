"""The GPU that a call of the decoder-layer operators runs on: tensors, cache and stream of
one GPU, the current one, or a refusal before the C call.

Tensors here are stand-ins with the attributes that the binding reads, and the C entry
points are replaced by functions that record the call, so no GPU is needed."""
import ctypes

import pytest
import torch

BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


class FakeTensor:
    is_cuda = True

    def __init__(self, shape, dtype=BF16, device=0):
        self.shape, self.dtype, self.device_index = tuple(shape), dtype, device

    def stride(self, i=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 1 << 20

    def get_device(self):
        return self.device_index


class FakeStream:
    def __init__(self, device, handle):
        self.device_index, self.cuda_stream = device, handle


class FakeCache:
    def __init__(self, device):
        self._call = (1 << 20, 4, 2, 64, device)


@pytest.fixture
def ops():
    """The binding over recording entry points: ops.calls lists (function, stream), ops.current
    is the current device, whose current stream is 100 + its index."""
    import __graft_entry__

    __graft_entry__.build()
    import moe_decode_host_gb300 as m
    from moe_decode_host_gb300 import decoder_ops

    class Ops:
        calls, current, mod = [], 0, m

    o = Ops()
    o.calls, keep = [], []

    def entry(name):
        sig = m._lib._SIGS[name][1]
        f = ctypes.CFUNCTYPE(ctypes.c_int, *sig)(lambda *a: o.calls.append((name, a[-1])) or 0)
        keep.append(f)
        return ctypes.cast(f, ctypes.c_void_p).value

    decoder_ops._bind(lambda d: 100 + d, lambda: o.current,
                      tuple(entry(n) for n in ("moe_add_rms_norm", "moe_kv_append", "moe_kv_attend", "moe_linear")))
    yield o
    decoder_ops._bind()


def _arguments(op, device):
    """A valid call: its positional and keyword arguments, everything on `device`."""
    t = lambda *shape, dtype=BF16: FakeTensor(shape, dtype, device)  # noqa: E731
    if op == "moe_add_rms_norm":
        return dict(x=t(3, 64), weight=t(64), y=t(3, 64), residual=t(3, 64), sum_out=t(3, 64))
    if op == "moe_kv_append":
        return dict(kv=FakeCache(device), q=t(3, 4, 64), k=t(3, 2, 64), v=t(3, 2, 64), positions=t(3, dtype=I32),
                    slots=t(3, dtype=I64), cos_sin=t(8, 64, dtype=F32), q_out=t(3, 4, 64))
    if op == "moe_kv_attend":
        return dict(kv=FakeCache(device), q=t(3, 4, 64), page_table=t(3, 5, dtype=I32), lengths=t(3, dtype=I32),
                    out=t(3, 4, 64), lse=t(3, 4, dtype=F32))
    return dict(x=t(3, 64), w=t(8, 64), y=t(3, 8), bias=t(8), residual=t(3, 8), status=t(1, dtype=I32))


OPS = ("moe_add_rms_norm", "moe_kv_append", "moe_kv_attend", "moe_linear")


@pytest.mark.parametrize("op", OPS)
def test_calls_on_the_current_gpu_use_its_current_stream(ops, op):
    for ops.current in (0, 1):
        getattr(ops.mod, op)(**_arguments(op, ops.current))
    getattr(ops.mod, op)(**_arguments(op, 1), stream=FakeStream(1, 7))
    getattr(ops.mod, op)(**_arguments(op, 1), stream=9)
    assert ops.calls == [(op, 100), (op, 101), (op, 7), (op, 9)]


@pytest.mark.parametrize("op", OPS)
def test_another_gpu_than_the_current_one_is_refused(ops, op):
    for ops.current, device in ((0, 1), (1, 0), (0, -1)):
        with pytest.raises(ops.mod.MoeError) as e:
            getattr(ops.mod, op)(**_arguments(op, device))
        assert e.value.code == ops.mod.MOE_ERR_INVALID_ARG
    assert ops.calls == []


@pytest.mark.parametrize("op", OPS)
def test_one_argument_of_another_gpu_is_refused(ops, op):
    for name in _arguments(op, 0):
        args = _arguments(op, 0)
        args[name] = _arguments(op, 1)[name]
        with pytest.raises(ops.mod.MoeError) as e:
            getattr(ops.mod, op)(**args)
        assert e.value.code == ops.mod.MOE_ERR_INVALID_ARG
    with pytest.raises(ops.mod.MoeError):
        getattr(ops.mod, op)(**_arguments(op, 0), stream=FakeStream(1, 7))
    assert ops.calls == []


def test_scales_of_another_gpu_are_refused(ops):
    e4m3 = torch.float8_e4m3fn
    t = FakeTensor
    for bad in ("x_scale", "w_scale"):
        a = dict(x=t((3, 64), e4m3), w=t((8, 64), e4m3), y=t((3, 8)), x_scale=t((3,), F32), w_scale=t((8,), F32))
        ops.mod.moe_linear(**a)
        a[bad].device_index = 1
        with pytest.raises(ops.mod.MoeError):
            ops.mod.moe_linear(**a)
    a = dict(x=t((3, 64)), weight=None, y=t((3, 64), e4m3), scale=t((3,), F32, 1))
    with pytest.raises(ops.mod.MoeError):
        ops.mod.moe_add_rms_norm(**a)
    assert len(ops.calls) == 2


def test_cache_of_another_gpu_is_refused(ops, monkeypatch):
    """The handle's workspace is made on the current device: k, v and the scales have to be there."""
    created = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    real = ops.mod.lib.moe_kv_create
    monkeypatch.setattr(ops.mod.lib, "moe_kv_create", lambda *a: created.append(1) or -1)
    assert real is not ops.mod.lib.moe_kv_create
    shape = (2, 4, 2, 64)
    for k, v, ks, vs in ((1, 1, 1, 1), (0, 1, 0, 0), (1, 0, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1)):
        with pytest.raises(ops.mod.MoeError, match="GPU"):
            ops.mod.KvCache(FakeTensor(shape, torch.float8_e4m3fn, k), FakeTensor(shape, torch.float8_e4m3fn, v), q_heads=4,
                            max_batch=1, k_scale=FakeTensor((2,), F32, ks), v_scale=FakeTensor((2,), F32, vs))
    assert created == []
    with pytest.raises(ops.mod.MoeError):  # the stand-in's own refusal: every check before it passed
        ops.mod.KvCache(FakeTensor(shape), FakeTensor(shape), q_heads=4, max_batch=1)
    assert created == [1]
