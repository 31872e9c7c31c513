"""Argument checks of the operators with fine scales and of positions with several axes, on the host: every
refusal comes before any CUDA call, so no GPU is needed."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # an aligned address that no refused call follows
F32, BF16, F16, E4M3 = 2, 0, 1, 3


@pytest.fixture(scope="module")
def m():
    import __graft_entry__

    __graft_entry__.build()
    import moe_decode_host_gb300 as mod

    return mod


def _quant(m, **kw):
    a = dict(x=FAKE, xt=BF16, xs=256, T=2, K=256, y=FAKE, ys=256, s=FAKE, ss=2)
    a.update(kw)
    return m.lib.moe_quant_e4m3(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(K=0), dict(K=-128), dict(xt=E4M3), dict(xt=7), dict(x=None), dict(y=None),
                                 dict(s=None)])
def test_quant_refusals(m, bad):
    assert _quant(m, **bad) == m.MOE_ERR_INVALID_ARG


def test_calls_of_nothing(m):
    assert _quant(m, T=0, x=None, y=None, s=None) == m.MOE_OK
    assert _product(m, T=0, x=None, y=None, xsc=None) == m.MOE_OK


def _product(m, **kw):
    a = dict(x=FAKE, xs=64, w=FAKE, ws=64, T=2, N=8, K=64, xsc=FAKE, xss=1, wsc=FAKE, wss=1, bias=None, bt=F32, act=0,
             res=None, rs=8, y=FAKE, yt=BF16, ys=8)
    a.update(kw)
    return m.lib.moe_linear_blocks(*a.values(), None, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(N=0), dict(K=0), dict(yt=E4M3), dict(yt=-2), dict(act=-1), dict(act=4), dict(bias=FAKE, bt=E4M3),
    dict(x=None), dict(w=None), dict(y=None), dict(xsc=None), dict(wsc=None), dict(xs=56), dict(ws=56), dict(K=60),
    dict(K=56), dict(xs=72), dict(ws=68), dict(x=FAKE + 8), dict(w=FAKE + 2), dict(N=(1 << 22) + 1), dict(T=(1 << 22) + 1)])
def test_product_refusals(m, bad):
    assert _product(m, **bad) == m.MOE_ERR_INVALID_ARG


def _create(m, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, tokens=8, **kw):
    a = dict(n_pages=4, page_size=16, kv_heads=2, q_heads=8, head_dim=64, type=E4M3, max_batch=4, page_stride=16 * 128,
             token_stride=128, head_stride=64)
    a.update(kw)
    out = ctypes.c_void_p()
    return m.lib.moe_kv_create_blocks(ctypes.byref(m._lib.moe_kv_params(*a.values())), k, v, ks, vs, tokens, ctypes.byref(out))


@pytest.mark.parametrize("bad", [
    dict(tokens=0), dict(tokens=-8), dict(tokens=3), dict(tokens=32), dict(tokens=2048, page_size=2048), dict(type=BF16), dict(type=F16),
    dict(page_size=0), dict(page_size=65537, tokens=1), dict(ks=None), dict(vs=None), dict(ks=None, vs=None), dict(head_dim=72),
    dict(q_heads=7), dict(k=None), dict(v=FAKE + 2), dict(max_batch=0)])
def test_cache_refusals(m, bad):
    assert _create(m, **bad) == m.MOE_ERR_INVALID_ARG


def test_cache_without_parameters(m):
    out = ctypes.c_void_p()
    assert m.lib.moe_kv_create_blocks(None, FAKE, FAKE, FAKE, FAKE, 8, ctypes.byref(out)) == m.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("axes,n", [(None, 3), (bytes(32), 0), (bytes(32), 5), (bytes(32), -1), (bytes(32), 3)])
def test_append_axes_refusals(m, axes, n):
    """The last of them has no cache."""
    assert m.lib.moe_kv_append_axes(None, BF16, FAKE, 64, 64, FAKE, 64, 64, FAKE, 64, 64, FAKE, 1, n, axes, FAKE, FAKE, 8, 64, 0,
                                    1, FAKE, 64, 64, None) == m.MOE_ERR_INVALID_ARG


def test_tensor_checks_refuse_what_is_not_on_a_gpu(m):
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    y, s = torch.empty(2, 256, dtype=torch.float8_e4m3fn), torch.empty(2, 2)
    with pytest.raises(m.MoeError) as e:
        m.moe_quant_e4m3(x, y, s)
    assert e.value.code == m.MOE_ERR_INVALID_ARG
    with pytest.raises(m.MoeError):
        m.moe_linear_blocks(y, y, torch.empty(2, 2), s, s[:1])
    c = torch.zeros(2, 4, 1, 64).to(torch.float8_e4m3fn)
    with pytest.raises(m.MoeError):
        m.KvCache(c, c, q_heads=1, max_batch=1, k_scale=torch.zeros(2, 1, 1), v_scale=torch.zeros(2, 1, 1))


class Fake:
    """A tensor's attributes, as the binding reads them."""

    def __init__(self, shape, dtype, strides=None, device=0):
        self.shape, self.dtype, self.device = tuple(shape), dtype, device
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        self.strides = tuple(strides or s)

    def stride(self):
        return self.strides

    def data_ptr(self):
        return FAKE

    def get_device(self):
        return self.device


class FakeCache:
    def __init__(self, device=0):
        self._call = (FAKE, 4, 2, 64, device)


@pytest.fixture
def ops(m):
    """The binding over recording entry points: ops.calls lists (function, arguments)."""
    from moe_decode_host_gb300 import decoder_ops

    class Ops:
        mod = m

    o, keep = Ops(), []
    o.calls = []

    def entry(name):
        f = ctypes.CFUNCTYPE(ctypes.c_int, *m._lib._SIGS[name][1])(lambda *a: o.calls.append((name, a)) or 0)
        keep.append(f)
        return ctypes.cast(f, ctypes.c_void_p).value

    names = ("moe_add_rms_norm", "moe_kv_append", "moe_kv_attend", "moe_linear", "moe_quant_e4m3", "moe_kv_append_axes", "moe_linear_blocks")
    decoder_ops._bind(lambda d: 100 + d, lambda: 0, tuple(entry(n) for n in names))
    yield o
    decoder_ops._bind()


E8, I32, I64, F, B = torch.float8_e4m3fn, torch.int32, torch.int64, torch.float32, torch.bfloat16


def test_arguments_reach_the_library(ops):
    m = ops.mod
    m.moe_quant_e4m3(Fake((3, 300), B, (400, 1)), Fake((3, 300), E8), Fake((3, 3), F, (8, 1)))
    m.moe_linear_blocks(Fake((3, 256), E8), Fake((200, 256), E8, (512, 1)), Fake((3, 200), B), Fake((3, 2), F, (5, 1)),
                        Fake((2, 2), F, (7, 1)), bias=Fake((200,), F), act="gelu")
    pos = Fake((3, 5), I32, (9, 1))
    args = dict(kv=FakeCache(), q=Fake((5, 4, 64), B), k=Fake((5, 2, 64), B), v=Fake((5, 2, 64), B), slots=Fake((5,), I64),
                cos_sin=Fake((10, 64), F), q_out=Fake((5, 4, 64), B))
    m.moe_kv_append(positions=pos, axes=[0, 1, 2, 0] * 8, **args)
    m.moe_kv_append(positions=Fake((5,), I32), **args)
    (n0, a0), (n1, a1), (n2, a2), (n3, _) = ops.calls
    assert (n0, n1, n2, n3) == ("moe_quant_e4m3", "moe_linear_blocks", "moe_kv_append_axes", "moe_kv_append")
    assert a0[1:5] == (BF16, 400, 3, 300) and a0[6] == 300 and a0[8:] == (8, 100)
    assert a1[1] == 256 and a1[3:7] == (512, 3, 200, 256) and a1[8] == 5 and a1[10] == 7 and a1[12:14] == (F32, 3) and a1[-1] == 100
    assert a2[11:14] == (FAKE, 9, 3) and a2[17:21] == (10, 64, 0, 5)


@pytest.mark.parametrize("axes", [[0, 1], b"\0" * 33, [0] * 31 + [256], [0] * 31 + [-1], [], [0] * 129])
def test_lists_of_axes_that_do_not_fit(ops, axes):
    with pytest.raises(ops.mod.MoeError):
        ops.mod.moe_kv_append(FakeCache(), Fake((5, 4, 64), B), Fake((5, 2, 64), B), Fake((5, 2, 64), B), Fake((3, 5), I32),
                              Fake((5,), I64), Fake((10, 64), F), Fake((5, 4, 64), B), axes=axes)
    assert not ops.calls


@pytest.mark.parametrize("op", ["moe_quant_e4m3", "moe_linear_blocks", "moe_kv_append"])
def test_everything_is_on_the_current_gpu(ops, op):
    make = {"moe_quant_e4m3": lambda d: [Fake((3, 256), B, device=d[0]), Fake((3, 256), E8, device=d[1]), Fake((3, 2), F, device=d[2])],
            "moe_linear_blocks": lambda d: [Fake((3, 256), E8, device=d[0]), Fake((8, 256), E8, device=d[0]), Fake((3, 8), B, device=d[0]),
                                            Fake((3, 2), F, device=d[1]), Fake((1, 2), F, device=d[2])],
            "moe_kv_append": lambda d: [FakeCache(d[0]), Fake((5, 4, 64), B, device=d[0]), Fake((5, 2, 64), B, device=d[0]),
                                        Fake((5, 2, 64), B, device=d[0]), Fake((2, 5), I32, device=d[1]), Fake((5,), I64, device=d[2]),
                                        Fake((10, 64), F, device=d[0]), Fake((5, 4, 64), B, device=d[0])]}[op]
    kw = dict(axes=[0, 1] * 16) if op == "moe_kv_append" else {}
    for devices in ((1, 1, 1), (0, 1, 0), (0, 0, 1), (-1, -1, -1), (0, -1, 0)):
        with pytest.raises(ops.mod.MoeError) as e:
            getattr(ops.mod, op)(*make(devices), **kw)
        assert e.value.code == ops.mod.MOE_ERR_INVALID_ARG
    assert not ops.calls
    getattr(ops.mod, op)(*make((0, 0, 0)), **kw)
    assert len(ops.calls) == 1
