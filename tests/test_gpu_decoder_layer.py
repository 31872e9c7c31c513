"""The example's decoder layer, all operators together, against a plain 64-bit layer.

The plain form takes the quantised weights as given and rounds the first norm's rows to
E4M3 as the layer does; every other value stays unrounded.  The layer's bf16 roundings (the
projections, the rotated keys and queries, the weights of the softmax, the attention's
output and the residual stream) are each 2^-9 relative in the root mean square or less;
eight of them in a row stay under 8 * 2^-9 / sqrt(3) = 9e-3."""
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

REL = 9e-3


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decoder_layer

    return decoder_layer


def _norm(s, w, eps):
    return s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * w.double()


class PlainLayer:
    def __init__(self, layer):
        self.l, self.k, self.v = layer, [[] for _ in range(layer.T)], [[] for _ in range(layer.T)]

    def attention(self, x, h, positions):
        lay = self.l
        T, hq, hkv, D = lay.T, lay.q_heads, lay.kv_heads, lay.head_dim
        h = h + x.double()
        a = _norm(h, lay.norm1, lay.eps)
        scale = (a.abs().amax(1) / 448).clamp(min=2.0 ** -126)
        a = (a / scale[:, None]).float().to(torch.float8_e4m3fn).double() * scale[:, None]
        qkv = a @ (lay.wqkv.double() * lay.wqkv_scale.double()[:, None]).t() + lay.bqkv.double()
        qkv = qkv.view(T, hq + 2 * hkv, D)
        cs = lay.table[positions.long()].double()[:, None, :]
        c, s = cs[..., : D // 2], cs[..., D // 2:]
        r, v = qkv[:, : hq + hkv], qkv[:, hq + hkv:]
        u, w = r[..., : D // 2], r[..., D // 2:]
        r = torch.cat([u * c - w * s, u * s + w * c], -1)
        o = []
        for t in range(T):
            self.k[t].append(r[t, hq:])
            self.v[t].append(v[t])
            k, vv = torch.stack(self.k[t]), torch.stack(self.v[t])
            q = r[t, :hq].view(hkv, hq // hkv, D)
            p = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) * D ** -0.5, -1)
            o.append(torch.einsum("hgn,nhd->hgd", p, vv).reshape(hq * D))
        h = h + torch.stack(o) @ lay.wo.double().t()
        n = _norm(h, lay.norm2, lay.eps)
        return h, n, n @ lay.wr.double().t()


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("T,heads,page", [(4, (8, 2, 64), 16), (1, (4, 4, 128), 5), (9, (6, 1, 96), 7)])
def test_decoder_layer_steps(example, T, heads, page):
    import oracle
    from gpu_helpers import bf16_bits

    oracle.build()
    hq, hkv, D = heads
    layer, pages, keep = example.random_layer(T, q_heads=hq, kv_heads=hkv, head_dim=D, page_size=page, max_len=24,
                                              seed=T)
    plain = PlainLayer(layer)
    g = torch.Generator(device="cuda").manual_seed(100 + T)
    lengths = torch.zeros(T, dtype=torch.int32, device="cuda")
    for step in range(20):
        x = torch.randn(T, layer.moe.H, generator=g, device="cuda").to(torch.bfloat16)
        h = (2 * torch.randn(T, layer.moe.H, generator=g, device="cuda")).to(torch.bfloat16)
        h64, n64, logits64 = plain.attention(x, h.double(), lengths)
        positions, slots = example.token_places(pages, lengths, page)
        lengths += 1
        out = layer.step(x, h, positions, slots, pages, lengths)
        assert _rel(h, h64) <= REL and _rel(layer.n, n64) <= REL and _rel(layer.logits, logits64) <= REL
        if step % 10 == 9:  # the experts, on the layer's own logits and activations
            bits = bf16_bits(layer.n)
            blobs = [b.numpy() for b in keep[0]]
            rc, ids, _, want = oracle.layer(layer.logits.cpu().numpy(), bits, layer.moe.k, 0, layer.moe.H, layer.moe.I,
                                            blobs)
            assert rc == 0 and np.array_equal(layer.buf.topk_ids.cpu().numpy(), ids)
            got = out.cpu().double().numpy()
            assert np.linalg.norm(got - want) / np.linalg.norm(want) <= 5e-3
    assert layer.cache.status() == 0 and layer.moe.status() == 0


def test_decoder_layer_attention_half_in_a_graph(example):
    """The operators capture: one graph of the attention half gives what the calls give."""
    T = 4
    layer, pages, keep = example.random_layer(T, max_len=64, seed=3)
    lengths = torch.full((T,), 10, dtype=torch.int32, device="cuda")
    positions, slots = example.token_places(pages, lengths, 16)
    lengths += 1
    x = torch.randn(T, layer.moe.H, device="cuda").to(torch.bfloat16)
    h0 = torch.randn(T, layer.moe.H, device="cuda").to(torch.bfloat16)
    h = h0.clone()
    layer.attention(x, h, positions, slots, pages, lengths)
    want = h.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            layer.attention(x, h, positions, slots, pages, lengths)
    h.copy_(h0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want)
    del keep
