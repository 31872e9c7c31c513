"""Sizes of a key-value cache that the C structure's integers cannot hold."""
import pytest
import torch

from test_decoder_ops_devices import FakeTensor


@pytest.mark.parametrize("bad", [dict(n_pages=(1 << 32) + 5), dict(n_pages=1 << 31), dict(q_heads=(1 << 32) + 4),
                                 dict(max_batch=(1 << 32) + 1), dict(max_batch=-(1 << 32) + 1)])
def test_sizes_past_32_bits_are_refused(monkeypatch, bad):
    """They must not reach the library cut to their low bits."""
    import __graft_entry__

    __graft_entry__.build()
    import moe_decode_host_gb300 as m

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    created = []
    monkeypatch.setattr(m.lib, "moe_kv_create", lambda p, *a: created.append(p) or -1)
    size = dict(n_pages=7, q_heads=4, max_batch=1)
    for s in (size, {**size, **bad}):
        t = FakeTensor((s["n_pages"], 1, 2, 64))
        with pytest.raises(m.MoeError) as e:
            m.KvCache(t, t, q_heads=s["q_heads"], max_batch=s["max_batch"])
        assert e.value.code == m.MOE_ERR_INVALID_ARG
    assert len(created) == 1  # the sizes that fit: the stand-in's refusal
