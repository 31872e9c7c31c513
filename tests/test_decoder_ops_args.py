"""Argument checks of the decoder-layer operators on the host: every refusal comes
before any CUDA call, so no GPU is needed."""
import ctypes

import pytest

FAKE = 1 << 20  # an aligned address that no refused call follows
F32, BF16, F16, E4M3 = 2, 0, 1, 3


@pytest.fixture(scope="module")
def m():
    import __graft_entry__

    __graft_entry__.build()
    import moe_decode_host_gb300 as mod

    return mod


def _norm(m, **kw):
    a = dict(x=FAKE, xt=BF16, xs=64, res=None, rt=BF16, rs=64, w=None, wt=BF16, eps=1e-6, T=2, H=64, sum=None, ss=64,
             y=FAKE, yt=BF16, ys=64, scale=None)
    a.update(kw)
    return m.lib.moe_add_rms_norm(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(H=32769), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(xt=E4M3), dict(xt=7), dict(yt=4), dict(yt=-1), dict(res=FAKE, rt=E4M3), dict(sum=FAKE, rt=9),
    dict(w=FAKE, wt=E4M3), dict(x=None), dict(y=None), dict(yt=E4M3), dict(scale=FAKE)])
def test_norm_refusals(m, bad):
    assert _norm(m, **bad) == m.MOE_ERR_INVALID_ARG


def test_norm_of_nothing(m):
    assert _norm(m, T=0, x=None, y=None) == m.MOE_OK


def _create(m, k=FAKE, v=FAKE, ks=None, vs=None, **kw):
    a = dict(n_pages=4, page_size=16, kv_heads=2, q_heads=8, head_dim=64, type=BF16, max_batch=4,
             page_stride=16 * 128, token_stride=128, head_stride=64)
    a.update(kw)
    out = ctypes.c_void_p()
    return m.lib.moe_kv_create(ctypes.byref(m._lib.moe_kv_params(*a.values())), k, v, ks, vs, ctypes.byref(out))


@pytest.mark.parametrize("bad", [
    dict(n_pages=0), dict(page_size=0), dict(page_size=65537), dict(kv_heads=0), dict(q_heads=7), dict(q_heads=1),
    dict(q_heads=65536), dict(head_dim=0), dict(head_dim=72), dict(head_dim=272), dict(type=F32), dict(type=5),
    dict(max_batch=0), dict(max_batch=65536), dict(page_stride=-16), dict(token_stride=4), dict(head_stride=63),
    dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 2)])
def test_cache_refusals(m, bad):
    assert _create(m, **bad) == m.MOE_ERR_INVALID_ARG


def test_calls_without_a_cache(m):
    lib = m.lib
    assert lib.moe_kv_create(None, FAKE, FAKE, None, None, None) == m.MOE_ERR_INVALID_ARG
    assert lib.moe_kv_destroy(None) == m.MOE_ERR_INVALID_ARG
    assert lib.moe_kv_append(None, BF16, FAKE, 64, 64, FAKE, 64, 64, FAKE, 64, 64, FAKE, FAKE, FAKE, 8, 64, 0, 1, FAKE,
                             64, 64, None) == m.MOE_ERR_INVALID_ARG
    assert lib.moe_kv_attend(None, FAKE, BF16, 64, 64, FAKE, 4, 4, FAKE, 1, 1.0, 0, FAKE, 64, 64, None,
                             None) == m.MOE_ERR_INVALID_ARG
    s = ctypes.c_int()
    assert lib.moe_kv_get_status(None, ctypes.byref(s)) == m.MOE_ERR_INVALID_ARG
    assert lib.moe_kv_clear_status(None) == m.MOE_ERR_INVALID_ARG


def _linear(m, **kw):
    a = dict(x=FAKE, xs=64, w=FAKE, ws=64, it=BF16, T=2, N=8, K=64, xsc=None, wsc=None, bias=None, bt=F32, act=0,
             res=None, rs=8, y=FAKE, yt=BF16, ys=8)
    a.update(kw)
    return m.lib.moe_linear(*a.values(), None, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(N=0), dict(K=0), dict(it=F32), dict(it=8), dict(yt=E4M3), dict(yt=-2), dict(act=-1), dict(act=4),
    dict(bias=FAKE, bt=E4M3), dict(x=None), dict(w=None), dict(y=None), dict(it=E4M3), dict(it=E4M3, xsc=FAKE),
    dict(it=E4M3, wsc=FAKE), dict(xsc=FAKE, wsc=FAKE), dict(xs=56), dict(ws=56), dict(K=60), dict(xs=66), dict(ws=68),
    dict(x=FAKE + 8), dict(w=FAKE + 2), dict(it=E4M3, xsc=FAKE, wsc=FAKE, K=56)])
def test_linear_refusals(m, bad):
    assert _linear(m, **bad) == m.MOE_ERR_INVALID_ARG


def test_linear_of_nothing(m):
    assert _linear(m, T=0, x=None, y=None) == m.MOE_OK


def test_tensor_checks_refuse_what_is_not_on_a_gpu(m):
    """The binding reads shapes and types from the tensors and refuses before the C call."""
    import torch

    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(m.MoeError) as e:
        m.moe_add_rms_norm(x, None, torch.empty_like(x))
    assert e.value.code == m.MOE_ERR_INVALID_ARG
    with pytest.raises(m.MoeError):
        m.moe_linear(x, x, torch.empty(2, 2))
    with pytest.raises(m.MoeError):
        m.moe_linear(x, torch.zeros(2, 32, dtype=torch.bfloat16), torch.empty(2, 2))
    c = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(m.MoeError):
        m.KvCache(c, c, q_heads=1, max_batch=1)


def test_status_text(m):
    assert b"range" in m.lib.moe_strerror(m.MOE_ERR_BAD_INDEX)
