"""A whole decoder layer on the library's kernels: 8-bit attention projections, a paged
cache, and the mixture-of-experts layer with host-resident cold experts.

One decode step of T sequences, one new token each:

  h    += x                          x: the previous layer's output
  a8    = norm(h)                    E4M3 rows with one scale each     moe_add_rms_norm
  qkv   = a8 Wqkv^T + b              8-bit product                     moe_linear
  q, k  rotated; k, v appended                                         moe_kv_append
  o     = attention over the cache                                     moe_kv_attend
  h    += o Wo^T                     residual in the epilogue          moe_linear
  n     = norm(h)                                                      moe_add_rms_norm
  logits = n Wr^T                    fp32                              moe_linear
  out   = experts(n, logits)         router, gather, experts, combine  run_step

The next layer takes x = out and the same h.  Run as a program it builds a small random
layer and decodes a few steps:  python examples/decoder_layer.py

With --fine-scales the attention's half is in 8 bits throughout, with a scale for each 128
elements of a row, each 128 x 128 block of a weight and each block of tokens of the cache:

  n     = norm(h + x)                                                  moe_add_rms_norm
  a8    = E4M3 of n, a scale for each 128 elements                     moe_quant_e4m3
  qkv   = a8 Wqkv^T + b                                                moe_linear_blocks
  q, k  rotated by positions with three axes; k, v to the block cache  moe_kv_append
  o     = attention over it                                            moe_kv_attend
  h    += E4M3(o) Wo^T                          moe_quant_e4m3, moe_linear_blocks
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_decode_host_gb300 as m  # noqa: E402


def quantize_rows(w):
    """E4M3 rows of a weight matrix and their fp32 scales (largest magnitude / 448)."""
    scale = (w.float().abs().amax(1) / 448).clamp_(min=2.0 ** -126)
    return (w.float() / scale[:, None]).to(torch.float8_e4m3fn), scale


def rotation_table(positions: int, dim: int, base: float = 10000.0, device="cuda"):
    """cos | sin of every position, fp32 [positions, dim]."""
    inv = base ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float64) / dim)
    a = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


class DecoderLayer:
    """Weights, cache and buffers of one layer for T sequences.

    moe: the Layer of its experts (hidden size moe.H, moe.E experts).  Weights: wqkv
    [(q_heads + 2 kv_heads) head_dim, H] and its bias, wo [H, q_heads head_dim], wr
    [E, H], norm1 and norm2 [H]; k and v caches [n_pages, page_size, kv_heads, head_dim]."""

    def __init__(self, moe, T, *, q_heads, kv_heads, head_dim, wqkv, bqkv, wo, wr, norm1, norm2, k_cache, v_cache,
                 table, eps=1e-6):
        H, dev, bf16 = moe.H, wqkv.device, torch.bfloat16
        self.moe, self.T, self.eps, self.table = moe, T, eps, table
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.wqkv, self.wqkv_scale = quantize_rows(wqkv)
        self.bqkv, self.wo, self.wr, self.norm1, self.norm2 = bqkv, wo, wr, norm1, norm2
        self.cache = m.KvCache(k_cache, v_cache, q_heads=q_heads, max_batch=T)
        self.buf = m.StepBuffers(moe, T, dev)
        self.a8 = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=dev)
        self.a8_scale = torch.empty(T, dtype=torch.float32, device=dev)
        self.qkv = torch.empty(T, (q_heads + 2 * kv_heads) * head_dim, dtype=bf16, device=dev)
        self.o = torch.empty(T, q_heads, head_dim, dtype=bf16, device=dev)
        self.n = torch.empty(T, H, dtype=bf16, device=dev)
        self.logits = torch.empty(T, moe.E, dtype=torch.float32, device=dev)

    def attention(self, x, h, positions, slots, page_table, lengths):
        """Up to the second norm: h is updated in place, self.n holds norm(h)."""
        T, hq, hkv, D = self.T, self.q_heads, self.kv_heads, self.head_dim
        m.moe_add_rms_norm(x, self.norm1, self.a8, residual=h, sum_out=h, scale=self.a8_scale, eps=self.eps)
        m.moe_linear(self.a8, self.wqkv, self.qkv, bias=self.bqkv, x_scale=self.a8_scale, w_scale=self.wqkv_scale)
        qkv = self.qkv.view(T, hq + 2 * hkv, D)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        m.moe_kv_append(self.cache, q, k, v, positions, slots, self.table, q)
        m.moe_kv_attend(self.cache, q, page_table, lengths, self.o)
        m.moe_linear(self.o.view(T, hq * D), self.wo, h, residual=h)
        m.moe_add_rms_norm(h, self.norm2, self.n, eps=self.eps)

    def step(self, x, h, positions, slots, page_table, lengths):
        """One token of every sequence; lengths count it.  Returns the experts' output;
        h, the residual stream, is updated in place."""
        self.attention(x, h, positions, slots, page_table, lengths)
        m.moe_linear(self.n, self.wr, self.logits)
        m.run_step(self.moe, self.buf, self.logits, self.n)
        return self.buf.out


def quantize_blocks(w):
    """E4M3 codes of a weight matrix with one fp32 scale for each 128 x 128 block."""
    n, k = w.shape
    nb, kb = -(-n // 128), -(-k // 128)
    p = torch.zeros(nb * 128, kb * 128, dtype=torch.float32, device=w.device)
    p[:n, :k] = w
    p = p.view(nb, 128, kb, 128)
    scale = (p.abs().amax((1, 3)) / 448).clamp_(min=2.0 ** -126)
    codes = (p / scale[:, None, :, None]).view(nb * 128, kb * 128)[:n, :k]
    return codes.to(torch.float8_e4m3fn).contiguous(), scale


class FineDecoderLayer(DecoderLayer):
    """The layer with fine scales: E4M3 caches with scales [n_pages, blocks, kv_heads], and positions
    int32 [axes, T] of which `axes` gives each pair of the rotation its own."""

    def __init__(self, moe, T, *, q_heads, kv_heads, head_dim, wqkv, bqkv, wo, wr, norm1, norm2, k_cache, v_cache,
                 k_scale, v_scale, table, axes, eps=1e-6):
        H, dev = moe.H, wqkv.device
        self.moe, self.T, self.eps, self.table, self.axes = moe, T, eps, table, bytes(axes)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        (self.wqkv, self.wqkv_scale), (self.wo, self.wo_scale) = quantize_blocks(wqkv), quantize_blocks(wo)
        self.bqkv, self.wr, self.norm1, self.norm2 = bqkv, wr, norm1, norm2
        self.cache = m.KvCache(k_cache, v_cache, q_heads=q_heads, max_batch=T, k_scale=k_scale, v_scale=v_scale)
        self.buf = m.StepBuffers(moe, T, dev)
        bf16, f8, wide = torch.bfloat16, torch.float8_e4m3fn, q_heads * head_dim
        self.n = torch.empty(T, H, dtype=bf16, device=dev)
        self.a8, self.a8_scale = torch.empty(T, H, dtype=f8, device=dev), torch.empty(T, -(-H // 128), device=dev)
        self.qkv = torch.empty(T, (q_heads + 2 * kv_heads) * head_dim, dtype=bf16, device=dev)
        self.o = torch.empty(T, q_heads, head_dim, dtype=bf16, device=dev)
        self.o8, self.o8_scale = torch.empty(T, wide, dtype=f8, device=dev), torch.empty(T, -(-wide // 128), device=dev)
        self.logits = torch.empty(T, moe.E, dtype=torch.float32, device=dev)

    def attention(self, x, h, positions, slots, page_table, lengths):
        T, hq, hkv, D = self.T, self.q_heads, self.kv_heads, self.head_dim
        m.moe_add_rms_norm(x, self.norm1, self.n, residual=h, sum_out=h, eps=self.eps)
        m.moe_quant_e4m3(self.n, self.a8, self.a8_scale)
        m.moe_linear_blocks(self.a8, self.wqkv, self.qkv, self.a8_scale, self.wqkv_scale, bias=self.bqkv)
        qkv = self.qkv.view(T, hq + 2 * hkv, D)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        m.moe_kv_append(self.cache, q, k, v, positions, slots, self.table, q, axes=self.axes)
        m.moe_kv_attend(self.cache, q, page_table, lengths, self.o)
        m.moe_quant_e4m3(self.o.view(T, hq * D), self.o8, self.o8_scale)
        m.moe_linear_blocks(self.o8, self.wo, h, self.o8_scale, self.wo_scale, residual=h)
        m.moe_add_rms_norm(h, self.norm2, self.n, eps=self.eps)


def random_layer(T, *, H=256, I=512, E=16, n_hot=12, k=2, q_heads=8, kv_heads=2, head_dim=64, page_size=16,
                 max_len=256, seed=0, fine=False):
    """A layer with random weights, its page table [T, pages], and the pinned and device
    memory of its experts (to be kept alive beside it)."""
    import synth

    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    n_cold, eb = E - n_hot, m.expert_bytes(H, I)
    blobs = synth.gen_blobs(E, H, I, seed=seed)
    hot, cold = blobs[:n_hot].cuda(), blobs[n_hot:].clone().pin_memory()
    slots = torch.empty((max(1, n_cold), eb), dtype=torch.uint8, device="cuda")
    scratch = m.Scratch(n_cold, eb, slots)
    moe = m.Layer(E=E, k=k, H=H, I=I, n_hot=n_hot, n_cold=n_cold, scratch=scratch, hot_ptrs=list(hot),
                  cold_ptrs=list(cold), init_loc=synth.loc_identity(E, n_hot), swap_every=0)
    per = -(-max_len // page_size)
    order = torch.randperm(T * per, generator=g, device="cuda").to(torch.int32).view(T, per)
    bf16 = torch.bfloat16
    cache = torch.zeros(2, T * per, page_size, kv_heads, head_dim, device="cuda").to(torch.float8_e4m3fn if fine else bf16)
    kinds = {}
    if fine:  # blocks of half a page; pairs take their axes in turn
        kinds = dict(zip(("k_scale", "v_scale"), torch.zeros(2, T * per, 2, kv_heads, device="cuda")))
        kinds["axes"] = [i % 3 for i in range(head_dim // 2)]
    layer = (FineDecoderLayer if fine else DecoderLayer)(
        moe, T, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
        wqkv=randn((q_heads + 2 * kv_heads) * head_dim, H) / H ** 0.5, bqkv=0.1 * randn((q_heads + 2 * kv_heads) * head_dim),
        wo=(randn(H, q_heads * head_dim) / (q_heads * head_dim) ** 0.5).to(bf16), wr=(randn(E, H) / H ** 0.5).to(bf16),
        norm1=(1 + 0.1 * randn(H)).to(bf16), norm2=(1 + 0.1 * randn(H)).to(bf16), k_cache=cache[0], v_cache=cache[1],
        table=rotation_table(max_len, head_dim), **kinds)
    return layer, order, (blobs, hot, cold, slots, scratch, cache)


def token_places(page_table, lengths, page_size):
    """Positions and cache slots of the tokens that the sequences are about to append."""
    at = lengths.long()
    page = page_table.gather(1, (at // page_size)[:, None])[:, 0].long()
    return lengths.clone(), page * page_size + at % page_size


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--fine-scales", action="store_true")
    a = ap.parse_args()
    layer, pages, keep = random_layer(a.sequences, max_len=a.steps, fine=a.fine_scales)
    lengths = torch.zeros(a.sequences, dtype=torch.int32, device="cuda")
    h = torch.zeros(a.sequences, layer.moe.H, dtype=torch.bfloat16, device="cuda")
    x = torch.randn_like(h)
    for step in range(a.steps):
        positions, slots = token_places(pages, lengths, layer.cache.page_size)
        lengths += 1
        if a.fine_scales:  # text: the same position along every axis
            positions = positions.expand(3, -1)
        out = layer.step(x, h, positions, slots, pages, lengths)
        x.copy_(torch.randn_like(x))
        h.zero_()
    torch.cuda.synchronize()
    assert layer.cache.status() == 0 and layer.moe.status() == 0
    print(f"{a.steps} steps of {a.sequences} sequences; last output rms {out.float().square().mean().sqrt():.4f}")
    del keep


if __name__ == "__main__":
    main()
