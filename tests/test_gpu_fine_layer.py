"""The example's decoder layer with fine scales: every operator's output against the 64-bit form of its own inputs, step
by step, and the whole step captured in a graph.

The bounds are those of the operators' own tests."""
import os
import sys

import pytest
import torch

from test_gpu_fine_scales import E4M3, U, attend64, e4m3_tol, quant64, rows64, turn64, within
from test_gpu_linear_blocks import product64

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decoder_layer

    return decoder_layer


def check_quant(x, y, s):
    y64, s64 = quant64(x)
    within(s, s64, s64 * 2.0 ** -23, "scale")
    within(y.float(), y64, e4m3_tol(y64), "codes")


def check_product(x, w, xs, ws, y, add, what):
    y64, size = product64(x, w, xs, ws)
    want = y64 + add.double()
    tol = size * (12 * 2.0 ** -22 + (xs.shape[1] + 4) * 2.0 ** -24) + want.abs() * (2.0 ** -22 + U[BF16]) + 2.0 ** -134
    within(y, want, tol, what)


@pytest.mark.parametrize("T", [1, 5])
def test_steps_of_the_layer(example, T):
    steps = 20
    layer, pages, keep = example.random_layer(T, max_len=64, fine=True, seed=T)
    hq, hkv, D, c = layer.q_heads, layer.kv_heads, layer.head_dim, layer.cache
    g = torch.Generator(device="cuda").manual_seed(T)
    lengths = torch.zeros(T, dtype=torch.int32, device="cuda")
    h = torch.zeros(T, layer.moe.H, dtype=BF16, device="cuda")
    keys, vals = [], []
    for _ in range(steps):
        x = torch.randn(T, layer.moe.H, generator=g, device="cuda").to(BF16)
        _, slots = example.token_places(pages, lengths, c.page_size)
        positions = torch.randint(0, 64, (3, T), generator=g, device="cuda", dtype=torch.int32)
        lengths += 1
        h0 = (h.double() + x.double()).to(BF16)
        out = layer.step(x, h, positions, slots, pages, lengths)
        assert out.isfinite().all() and c.status() == 0 and layer.moe.status() == 0
        # self.n now holds the second norm's rows: the first ones are made again
        n = torch.empty_like(layer.n)
        example.m.moe_add_rms_norm(h0, layer.norm1, n, eps=layer.eps)
        a8, a8s = torch.empty_like(layer.a8), torch.empty_like(layer.a8_scale)
        example.m.moe_quant_e4m3(n, a8, a8s)
        check_quant(n, a8, a8s)
        qkv = layer.qkv.view(T, hq + 2 * hkv, D)
        # keys, values and turned queries from the layer's own rows
        y64, size = product64(layer.a8, layer.wqkv, layer.a8_scale, layer.wqkv_scale)
        y64 = (y64 + layer.bqkv.double()).view(T, hq + 2 * hkv, D)
        tol = size.view_as(y64) * (12 * 2.0 ** -22 + 8 * 2.0 ** -24) + y64.abs() * (2.0 ** -22 + U[BF16]) + 2.0 ** -134
        within(qkv[:, hq:], y64[:, hq:], tol[:, hq:], "k and v")
        cos, sin = rows64(layer.table, positions, list(layer.axes))
        q64, _ = turn64(y64[:, :hq], cos, sin, False)
        loss, _ = turn64(tol[:, :hq], cos.abs(), -sin.abs(), False)  # both parts of a pair's error in full
        other, _ = turn64(tol[:, :hq], cos.abs(), sin.abs(), False)
        within(qkv[:, :hq], q64, torch.maximum(loss.abs(), other.abs()) + q64.abs() * (U[BF16] + 2.0 ** -22) + size.max() * 2.0 ** -22, "q")
        keys.append(turn64(qkv[:, hq:hq + hkv], cos, sin, False)[0])
        vals.append(qkv[:, hq + hkv:].double())
        # what the cache holds is within E4M3 of what went in
        for t in range(len(keys)):
            p, e = pages[:, t // c.page_size].long(), t % c.page_size
            for codes, scales, want in ((c.k, c.k_scale, keys[t]), (c.v, c.v_scale, vals[t])):
                per = scales[p, e // c.scale_tokens].double()[..., None]
                within(codes[p, e].double() * per, want, want.abs() * (2.0 ** -4 + 1e-6) + per * 2.0 ** -10 * 2.01, "cache")
        o64, _, ot, _ = attend64(qkv[:, :hq], c.k, c.v, c.k_scale, c.v_scale, pages, lengths.tolist(), D ** -0.5, 0)
        within(layer.o, o64, ot, "attention")
        check_quant(layer.o.view(T, -1), layer.o8, layer.o8_scale)
        check_product(layer.o8, layer.wo, layer.o8_scale, layer.wo_scale, h, h0, "h")
    del keep


def test_a_captured_step_is_the_same(example):
    T = 4
    results = []
    for captured in (False, True):
        layer, pages, keep = example.random_layer(T, max_len=64, fine=True, seed=7)
        g = torch.Generator(device="cuda").manual_seed(3)
        lengths, slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.full((T,), -1, dtype=torch.int64, device="cuda")
        positions = torch.zeros(3, T, dtype=torch.int32, device="cuda")
        x, h = (torch.zeros(T, layer.moe.H, dtype=BF16, device="cuda") for _ in range(2))

        def attention():
            layer.attention(x, h, positions, slots, pages, lengths)

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            attention()  # nothing appended, nothing attended
            s.synchronize()
            if captured:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=s):
                    attention()
        torch.cuda.synchronize()
        h.zero_()
        seen = []
        for _ in range(12):
            p, at = example.token_places(pages, lengths, layer.cache.page_size)
            slots.copy_(at), positions.copy_(p.expand(3, -1)), lengths.add_(1)
            x.copy_(torch.randn(T, layer.moe.H, generator=g, device="cuda"))
            torch.cuda.synchronize()
            if captured:
                graph.replay()
            else:
                attention()
            torch.cuda.synchronize()
            seen.append((h.clone(), layer.n.clone(), layer.o.clone()))
        seen.append((layer.cache.k.view(torch.uint8).clone(), layer.cache.v.view(torch.uint8).clone(), layer.cache.k_scale.clone()))
        results.append(seen)
        del keep
    for a, b in zip(*results):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
