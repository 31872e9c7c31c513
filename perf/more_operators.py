"""Performance cases of the decoder layer in 8 bits with fine scales, and of positions with several axes.

  quant   rows to E4M3 with one scale for each 128 elements
  linear  the product of such rows with a weight that has one scale for each 128 x 128 block, with its
          epilogue
  append  position rotation and append to a paged cache; here E4M3 with one scale for each block of
          tokens and key head, which grows with the tokens it takes in
  axes    the same call where a token's position has several axes (time, height, width)
  attend  attention of one new token per sequence over the block-scaled cache

Sizes follow the MoE layer's workloads (hidden size 4096; 1, 8 and 8192 tokens) with generic head
layouts.

`own` selects between the plain form (elementary torch operations in 32 bits) and the library's entry
points.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0
TINY = 2.0 ** -126
GROUP = 128  # elements of K under one scale

# No drawn case costs more than the largest listed one of its operator.
QUANT_ELEMS = 8192 * 4096
MM_FLOPS = 2 * 8192 * 6144 * 4096
APPEND_ELEMS = 8192 * 48 * 128
KV_BYTES = 64 * 12288 * 8 * 128 * 2


def listed():
    return [
        # the attention's output of a decode step of 8 sequences, on its way into the output projection
        dict(name="quant-decode-8", op="quant", T=8, K=4096, x="bf16"),
        # the rows of a prompt of 8192 tokens
        dict(name="quant-prompt-8192", op="quant", T=8192, K=4096, x="bf16"),
        # output projection of one decode token, onto the residual
        dict(name="linear-decode-1", op="linear", T=1, N=4096, K=4096, y="bf16", bias=False, act="none", res=True),
        # a ragged batch of prompts through a layer of odd width, where no tile is whole
        dict(name="linear-ragged-777", op="linear", T=777, N=5003, K=1424, y="f16", bias=True, act="gelu", res=False),
        # the q/k/v projection of a prompt with its bias
        dict(name="linear-prompt-8192", op="linear", T=8192, N=6144, K=4096, y="bf16", bias=True, act="none", res=False),
        # a decode step of 8 sequences, each in the middle of a block whose scale may grow
        dict(name="append-decode-8", op="append", T=8, seqs=8, mid=True, hq=32, hkv=8, D=128, page=64, block=32,
             x="bf16", kv="e4m3", rot=128, interleaved=False, axes=1, pattern="sections"),
        # a prompt of 8192 tokens into new blocks
        dict(name="append-prompt-8192", op="append", T=8192, seqs=1, mid=False, hq=32, hkv=8, D=128, page=64,
             block=64, x="bf16", kv="e4m3", rot=128, interleaved=False, axes=1, pattern="sections"),
        # a decode step behind images: three axes, taken in turn by the pairs
        dict(name="axes-decode-8", op="axes", T=8, seqs=8, mid=True, hq=32, hkv=8, D=128, page=16, block=0, x="bf16",
             kv="bf16", rot=128, interleaved=False, axes=3, pattern="turns"),
        # a prompt of 8192 tokens of text and images: three axes, a section of the pairs each
        dict(name="axes-prompt-8192", op="axes", T=8192, seqs=1, mid=False, hq=32, hkv=8, D=128, page=64, block=0,
             x="bf16", kv="bf16", rot=128, interleaved=False, axes=3, pattern="sections"),
        # one user's conversation: a single sequence, where the split over its length counts
        dict(name="attend-1x4097", op="attend", B=1, lo=4097, hi=4097, hq=32, hkv=8, D=128, page=64, block=64, q="bf16",
             window=0),
        # a small model's short ragged batch: one key head per query head, 96-wide heads, a sliding window, pages
        # and blocks that end inside a tile, and sequences with no token yet
        dict(name="attend-window-ragged", op="attend", B=19, lo=0, hi=2500, hq=12, hkv=12, D=96, page=14, block=7,
             q="f16", window=1000),
        # the largest batch: 64 long sequences, groups of 16 query heads
        dict(name="attend-64-long", op="attend", B=64, lo=8192, hi=16384, hq=128, hkv=8, D=128, page=64, block=32,
             q="bf16", window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _page_and_block(rng):
    page = rng.choice([1, 7, 16, 24, 32, 64, 128])
    return page, rng.choice([n for n in range(1, page + 1) if page % n == 0 and n * 8 >= page])


def draw(rng):
    op = rng.choice(["quant", "linear", "append", "axes", "attend"])
    if op == "quant":
        T, K = _log(rng, 1, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.6:
            K = max(64, K // 64 * 64)
        return dict(op=op, T=max(1, min(T, QUANT_ELEMS // K)), K=K, x=rng.choice(["bf16", "f16", "f32"]))
    if op == "linear":
        N, K = _log(rng, 64, 8192), max(64, _log(rng, 64, 8192) // 16 * 16)
        T = max(1, min(_log(rng, 1, 8192), MM_FLOPS // (2 * N * K)))
        return dict(op=op, T=T, N=N, K=K, y=rng.choice(["bf16", "f16", "f32"]), bias=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "gelu", "silu"]), res=rng.random() < 0.5)
    if op in ("append", "axes"):
        hkv, g, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 8]), rng.choice([64, 80, 96, 128, 256])
        T = min(_log(rng, 1, 8192), APPEND_ELEMS // ((g + 2) * hkv * D))
        x = rng.choice(["bf16", "f16"])
        page, block = _page_and_block(rng)
        kv = "e4m3" if op == "append" else rng.choice([x, "e4m3"])
        return dict(op=op, T=T, seqs=min(T, _log(rng, 1, 64)), mid=rng.random() < 0.7, hq=g * hkv, hkv=hkv, D=D,
                    page=page, block=block if kv == "e4m3" else 0, x=x, kv=kv, rot=rng.choice([D, D // 2]),
                    interleaved=rng.random() < 0.3, axes=1 if op == "append" else rng.choice([2, 3, 4]),
                    pattern=rng.choice(["sections", "turns"]))
    hkv, g, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 7, 8, 16]), rng.choice([64, 96, 128, 192, 256])
    page, block = _page_and_block(rng)
    B = _log(rng, 1, 64)
    hi = _log(rng, 16, max(17, min(16384, KV_BYTES // (2 * B * hkv * D))))
    return dict(op=op, B=B, lo=rng.choice([0, 1, hi // 4, hi]), hi=hi, hq=g * hkv, hkv=hkv, D=D, page=page, block=block,
                q=rng.choice(["bf16", "f16"]), window=rng.choice([0, 0, 0, 1 + hi // 3]))


def _lengths(case):
    """The batch's lengths: spread evenly from lo to hi, so that their sum is the case's own."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _runs(case):
    """(first entry, tokens) of each sequence of an append: where it stands in its first page, and what it adds."""
    T, n, page = case["T"], case["seqs"], case["page"]
    return [((7 * i + 3) % page if case["mid"] else 0, T // n + (i < T % n)) for i in range(n)]


def _axis_of_pair(case):
    """The axis that turns each pair: a section each (the first the shortest), or one after the other."""
    n, pairs = case["axes"], case["rot"] // 2
    if case["pattern"] == "turns":
        return [i % n for i in range(pairs)]
    first = pairs // (n + 1) // 2 * 2 if n > 1 else pairs
    rest = -(-(pairs - first) // max(1, n - 1))
    return [0 if i < first else 1 + (i - first) // rest for i in range(pairs)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed & 0x7FFFFFFF)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _page_order(g, n):
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32)


def _prepare_quant(c, g):
    T, K = c["T"], c["K"]
    s = dict(c)
    # activations with a few wide channels
    s["xt"] = (_randn(g, T, K) * torch.exp(0.8 * _randn(g, K))).to(DT[c["x"]])
    s["yt"] = torch.empty(T, K, dtype=DT["e4m3"], device="cuda")
    s["scale"] = torch.empty(T, -(-K // GROUP), dtype=torch.float32, device="cuda")
    return s


def _blocks_of_k(K):
    return -(-K // GROUP)


def _prepare_linear(c, g):
    T, N, K = c["T"], c["N"], c["K"]
    G, NB = _blocks_of_k(K), -(-N // GROUP)
    s = dict(c)
    x = _randn(g, T, G * GROUP) * torch.exp(0.5 * _randn(g, T, G)).repeat_interleave(GROUP, 1)
    w = _randn(g, NB * GROUP, G * GROUP) / math.sqrt(K)
    w = w * torch.exp(0.3 * _randn(g, NB, G)).repeat_interleave(GROUP, 0).repeat_interleave(GROUP, 1)
    x[:, K:], w[:, K:], w[N:] = 0, 0, 0
    xb, wb = x.view(T, G, GROUP), w.view(NB, GROUP, G, GROUP)
    s["xs"] = xb.abs().amax(2).clamp_(min=TINY) / E4M3_MAX
    s["ws"] = wb.abs().amax((1, 3)).clamp_(min=TINY) / E4M3_MAX
    s["xt"] = (xb / s["xs"][:, :, None]).reshape(T, -1)[:, :K].to(DT["e4m3"]).contiguous()
    s["wt"] = (wb / s["ws"][:, None, :, None]).reshape(NB * GROUP, -1)[:N, :K].to(DT["e4m3"]).contiguous()
    s["b"] = 0.1 * _randn(g, N) if c["bias"] else None
    s["rt"] = _randn(g, T, N).to(DT[c["y"]]) if c["res"] else None
    s["yt"] = torch.empty(T, N, dtype=DT[c["y"]], device="cuda")
    return s


def _rotation_table(positions, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([torch.cos(a), torch.sin(a)], 1).to(torch.float32)


def _exponent(top):
    """The smallest e with top <= 448 * 2^e, held to the range of a scale (2^-126 to 2^119)."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(top > 0, e, torch.full_like(e, -126)).clamp(-126, 119)


def _power(e):
    return torch.ldexp(torch.ones((), device="cuda"), e)


def _fill_blocks(n_pages, page, block, hkv, D, size, g):
    """A cache of E4M3 codes with the scales of its blocks [pages, blocks, heads]."""
    v = _randn(g, n_pages * (page // block), block, hkv, D)
    v.mul_(size * torch.exp(0.4 * _randn(g, v.shape[0], 1, hkv, 1)))
    scale = _power(_exponent(v.abs().amax((1, 3))))
    codes = v.div_(scale[:, None, :, None]).to(DT["e4m3"])
    return codes.view(n_pages, page, hkv, D), scale.view(n_pages, page // block, hkv).contiguous()


def _prepare_append(c, g):
    T, hq, hkv, D, page = c["T"], c["hq"], c["hkv"], c["D"], c["page"]
    s = dict(c)
    # the three parts of a fused projection's rows
    qkv = _randn(g, T, hq + 2 * hkv, D).to(DT[c["x"]])
    s["qt"], s["kt"], s["vt"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    runs = _runs(c)
    n_pages = sum(-(-(at + n) // page) for at, n in runs) + 2
    order = _page_order(g, n_pages)
    slots, pos, first = [], [], 0
    for i, (at, n) in enumerate(runs):
        t = at + torch.arange(n, device="cuda")
        slots.append(order[first + t // page].to(torch.int64) * page + t % page)
        pos.append(t + 97 * i)  # positions need not be places in the cache
        first += -(-(at + n) // page)
    s["slots"] = torch.cat(slots).contiguous()
    t = torch.cat(pos) + 40
    n_positions = T + page + 97 * len(runs) + 512
    if c["axes"] == 1:
        s["pos"], s["axis"] = t.to(torch.int32), None
    else:
        # text (all axes alike), then images of 16 x 24 patches behind it
        at, per = (t - 300).clamp(min=0), 16 * 24
        image, grid = t >= 300, [(at // per) * 24, (at // per) * 24 + at % per // 24, (at // per) * 24 + at % 24, at // per]
        s["pos"] = torch.stack([torch.where(image, 300 + grid[a], t) for a in range(c["axes"])]).to(torch.int32).contiguous()
        s["axis"] = bytes(_axis_of_pair(c))
    s["table"] = _rotation_table(n_positions, c["rot"])
    s["ks"] = s["vs"] = None
    if c["block"]:
        s["kc"], s["ks"] = _fill_blocks(n_pages, page, c["block"], hkv, D, 0.5, g)
        s["vc"], s["vs"] = _fill_blocks(n_pages, page, c["block"], hkv, D, 0.5, g)
    else:
        s["kc"], s["vc"] = (_randn(g, n_pages, page, hkv, D).to(DT[c["kv"]]) for _ in range(2))
    s["qo"] = torch.empty(T, hq, D, dtype=DT[c["x"]], device="cuda")
    s["cache"] = _cache(s, hq, 1)
    return s


def _prepare_attend(c, g):
    B, hq, hkv, D, page = c["B"], c["hq"], c["hkv"], c["D"], c["page"]
    s = dict(c)
    lens = torch.tensor(_lengths(c), device="cuda")
    s["lens"] = lens[torch.randperm(B, generator=g, device="cuda")].to(torch.int32)
    per = max(1, -(-c["hi"] // page))
    need = (s["lens"].long() + page - 1) // page
    first = torch.cumsum(need, 0) - need
    n_pages = sum(-(-n // page) for n in _lengths(c)) + 2
    order = _page_order(g, n_pages)
    at = torch.arange(per, device="cuda")[None, :]
    # rows of pages past a sequence's end hold page 0, as an engine's table does
    s["pages"] = torch.where(at < need[:, None], order[(first[:, None] + at).clamp(max=n_pages - 1)],
                             torch.zeros((), dtype=torch.int32, device="cuda")).contiguous()
    s["qt"] = _randn(g, B, hq, D).to(DT[c["q"]])
    s["kc"], s["ks"] = _fill_blocks(n_pages, page, c["block"], hkv, D, 1.0, g)
    s["vc"], s["vs"] = _fill_blocks(n_pages, page, c["block"], hkv, D, 1.0, g)
    s["scale"] = 1.0 / math.sqrt(D)
    s["ot"] = torch.empty(B, hq, D, dtype=DT[c["q"]], device="cuda")
    s["lse"] = torch.empty(B, hq, dtype=torch.float32, device="cuda")
    s["cache"] = _cache(s, hq, B)
    return s


def _cache(s, hq, batch):
    """The cache handle that a user's program keeps."""
    if not own:
        return None
    import moe_decode_host_gb300 as m

    return m.KvCache(s["kc"], s["vc"], q_heads=hq, max_batch=batch, k_scale=s["ks"], v_scale=s["vs"])


def prepare(case, seed):
    return {"quant": _prepare_quant, "linear": _prepare_linear, "append": _prepare_append, "axes": _prepare_append,
            "attend": _prepare_attend}[case["op"]](case, _gen(seed))


# ---- plain forms: 32 bits throughout, one rounding at the end -----------------


def _plain_quant(s):
    T, K = s["T"], s["K"]
    G = _blocks_of_k(K)
    x = torch.zeros(T, G * GROUP, dtype=torch.float32, device="cuda")
    x[:, :K] = s["xt"].float()
    x = x.view(T, G, GROUP)
    scale = (x.abs().amax(2) / E4M3_MAX).clamp(min=TINY)
    y = (x / scale[:, :, None]).view(T, G * GROUP)[:, :K]
    return [y.to(DT["e4m3"]), scale]


def _activated(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y / math.sqrt(2.0)))
    return y


def _plain_linear(s):
    N, K = s["N"], s["K"]
    x = s["xt"].float() * s["xs"].repeat_interleave(GROUP, 1)[:, :K]
    w = s["wt"].float() * s["ws"].repeat_interleave(GROUP, 0)[:N].repeat_interleave(GROUP, 1)[:, :K]
    y = torch.matmul(x, w.t())
    if s["b"] is not None:
        y = y + s["b"]
    y = _activated(y, s["act"])
    if s["rt"] is not None:
        y = y + s["rt"].float()
    return y.to(s["yt"].dtype)


def _rotated(x, table, rot, interleaved):
    cos, sin = table[:, None, : rot // 2], table[:, None, rot // 2:]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _table_rows(s):
    """Cosines and sines [T, rot] of every token, each pair's from its own axis' position."""
    if s["axis"] is None:
        return s["table"][s["pos"].long()]
    axis = torch.tensor(list(s["axis"]), device="cuda")
    rows = s["pos"].long()[axis].t()  # [T, pairs]
    pair = torch.arange(s["rot"] // 2, device="cuda")
    return torch.cat([s["table"][rows, pair], s["table"][rows, pair + s["rot"] // 2]], 1)


def _plain_put(codes, scales, slots, v, block):
    """Tokens v [T, heads, D] into the blocks that hold their slots."""
    _, hkv, D = v.shape
    all_codes, all_scales = codes.view(-1, block, hkv, D), scales.view(-1, hkv)
    at = slots // block
    touched, which = torch.unique(at, return_inverse=True)
    top = torch.zeros(len(touched), hkv, device="cuda")
    top.scatter_reduce_(0, which[:, None].expand(-1, hkv), v.abs().amax(2), "amax")
    fresh = torch.zeros(len(touched), dtype=torch.bool, device="cuda")
    fresh[which[slots % block == 0]] = True  # a block that gets its first entry starts anew
    need, before = _power(_exponent(top)), all_scales[touched]
    now = torch.where(fresh[:, None], need, torch.maximum(need, before))
    kept = all_codes[touched].float()
    # what the block held keeps its values; a block that starts anew keeps its codes
    factor = torch.where(fresh[:, None], torch.ones_like(now), before / now)
    kept = kept * factor[:, None, :, None]
    kept[which, slots % block] = (v / now[which][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    all_codes[touched] = kept.to(DT["e4m3"])
    all_scales[touched] = now


def _plain_append(s):
    table = _table_rows(s)
    q = _rotated(s["qt"].float(), table, s["rot"], s["interleaved"])
    k = _rotated(s["kt"].float(), table, s["rot"], s["interleaved"])
    v = s["vt"].float()
    if s["block"]:
        _plain_put(s["kc"], s["ks"], s["slots"], k, s["block"])
        _plain_put(s["vc"], s["vs"], s["slots"], v, s["block"])
        return [q.to(s["qo"].dtype), s["kc"], s["vc"], s["ks"], s["vs"]]
    page = s["page"]
    s["kc"][s["slots"] // page, s["slots"] % page] = k.to(s["kc"].dtype)
    s["vc"][s["slots"] // page, s["slots"] % page] = v.to(s["vc"].dtype)
    return [q.to(s["qo"].dtype), s["kc"], s["vc"]]


def _plain_attend(s):
    B, hq, hkv, D, block = s["B"], s["hq"], s["hkv"], s["D"], s["block"]
    pages = s["pages"].long()
    k, v = s["kc"][pages].float(), s["vc"][pages].float()
    k.mul_(s["ks"][pages].repeat_interleave(block, 2)[..., None])
    v.mul_(s["vs"][pages].repeat_interleave(block, 2)[..., None])
    L = k.shape[1] * k.shape[2]
    k, v = k.view(B, L, hkv, D), v.view(B, L, hkv, D)
    q = s["qt"].float().view(B, hkv, hq // hkv, D)
    a = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    at, n = torch.arange(L, device="cuda")[None, :], s["lens"].long()[:, None]
    seen = at < n
    if s["window"]:
        seen = seen & (at >= n - s["window"])
    a = a.masked_fill(~seen[:, None, None, :], -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - top.clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / total.clamp(min=1e-30)
    return [o.reshape(B, hq, D).to(s["ot"].dtype), (top + torch.log(total)).reshape(B, hq)]


# ---- the library's entry points ----------------------------------------------


def _own(s):
    import moe_decode_host_gb300 as m

    op = s["op"]
    if op == "quant":
        m.moe_quant_e4m3(s["xt"], s["yt"], s["scale"])
        return [s["yt"], s["scale"]]
    if op == "linear":
        m.moe_linear_blocks(s["xt"], s["wt"], s["yt"], s["xs"], s["ws"], bias=s["b"], act=s["act"], residual=s["rt"])
        return s["yt"]
    if op == "attend":
        m.moe_kv_attend(s["cache"], s["qt"], s["pages"], s["lens"], s["ot"], scale=s["scale"], window=s["window"],
                        lse=s["lse"])
        return [s["ot"], s["lse"]]
    m.moe_kv_append(s["cache"], s["qt"], s["kt"], s["vt"], s["pos"], s["slots"], s["table"], s["qo"],
                    interleaved=s["interleaved"], axes=s["axis"])
    return [s["qo"], s["kc"], s["vc"]] + ([s["ks"], s["vs"]] if s["block"] else [])


def run(state):
    if own:
        return _own(state)
    return {"quant": _plain_quant, "linear": _plain_linear, "append": _plain_append, "axes": _plain_append,
            "attend": _plain_attend}[state["op"]](state)


def work(case):
    op = case["op"]
    if op == "quant":
        T, K = case["T"], case["K"]
        return {"bytes": T * K * (SIZE[case["x"]] + 1) + 4 * T * _blocks_of_k(K), "flops": 3 * T * K}
    if op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        G = _blocks_of_k(K)
        b = (T + N) * K + T * N * SIZE[case["y"]] * (2 if case["res"] else 1) + 4 * G * (T + -(-N // GROUP))
        return {"bytes": b + (4 * N if case["bias"] else 0), "flops": 2 * T * N * K}
    if op == "attend":
        n = sum(min(v, case["window"]) if case["window"] else v for v in _lengths(case))
        B, hq, hkv, D = case["B"], case["hq"], case["hkv"], case["D"]
        b = 2 * n * hkv * D + 8 * n * hkv // case["block"] + B * hq * (2 * D * SIZE[case["q"]] + 4)
        return {"bytes": b + 4 * n // case["page"] + 4 * B, "flops": 4 * n * hq * D}
    T, hq, hkv, D = case["T"], case["hq"], case["hkv"], case["D"]
    b = T * D * (2 * hq * SIZE[case["x"]] + 2 * hkv * (SIZE[case["x"]] + SIZE[case["kv"]]))
    if case["block"]:
        blocks = sum(-(-(at + n) // case["block"]) - at // case["block"] for at, n in _runs(case))
        b += 2 * 2 * 4 * blocks * hkv
    return {"bytes": b + T * (8 + 4 * case["axes"] + 4 * case["rot"]), "flops": 3 * T * (hq + hkv) * case["rot"]}


# ---- definitions in 64 bits ----------------------------------------------------


def _exact_quant(s):
    y, scales = [], []
    for k0 in range(0, s["K"], GROUP):
        x = s["xt"][:, k0:k0 + GROUP].double()
        scale = torch.clamp(torch.linalg.vector_norm(x, math.inf, dim=1) / 448, min=TINY)
        y.append(x / scale[:, None])
        scales.append(scale)
    return [torch.cat(y, 1), torch.stack(scales, 1)]


def _exact_linear(s):
    """A block of K at a time, its partial products under their two scales."""
    T, N, K = s["T"], s["N"], s["K"]
    y = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    block = torch.arange(N, device="cuda") // GROUP
    for i, k0 in enumerate(range(0, K, GROUP)):
        part = torch.einsum("tk,nk->tn", s["xt"][:, k0:k0 + GROUP].double(), s["wt"][:, k0:k0 + GROUP].double())
        y.addcmul_(part.mul_(s["xs"][:, i].double()[:, None]), s["ws"][:, i].double()[block][None, :])
    if s["b"] is not None:
        y += s["b"].double()
    if s["act"] == "relu":
        y = torch.relu(y)
    elif s["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif s["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    return y if s["rt"] is None else y + s["rt"].double()


def _exact_turn(x, cs, rot, interleaved):
    """Each pair as a complex number, turned by its angle."""
    turn = torch.complex(cs[:, : rot // 2], cs[:, rot // 2:])[:, None, :]
    head, tail = x[..., :rot], x[..., rot:]
    if interleaved:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
        head = torch.view_as_real(z).reshape(head.shape)
    else:
        z = torch.complex(head[..., : rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, tail], -1)


def _exact_put(codes, scales, slots, v, block):
    """Block after block of the tokens in the order in which they come."""
    _, hkv, D = v.shape
    out, outs = codes.double().view(-1, block, hkv, D), scales.double().view(-1, hkv)
    home = (slots // block).tolist()
    t0 = 0
    while t0 < len(home):
        t1 = t0
        while t1 < len(home) and home[t1] == home[t0]:
            t1 += 1
        entry = (slots[t0:t1] % block).tolist()
        top = v[t0:t1].abs().amax((0, 2)).tolist()
        for h in range(hkv):
            e = -126
            if top[h] > 0:
                e = max(-126, math.ceil(math.log2(top[h] / 448)) - 1)
                while top[h] > 448 * 2.0 ** e:
                    e += 1
            top[h] = 2.0 ** e
        now, old = torch.tensor(top, dtype=torch.float64, device="cuda"), outs[home[t0]].clone()
        if 0 not in entry:
            now = torch.maximum(now, old)
            out[home[t0]] *= (old / now)[None, :, None]
        out[home[t0], entry[0]:entry[0] + t1 - t0] = v[t0:t1] / now[None, :, None]
        outs[home[t0]] = now
        t0 = t1
    return out.view(codes.shape), outs.view(scales.shape)


def _exact_append(s):
    pair = list(s["axis"]) if s["axis"] is not None else [0] * (s["rot"] // 2)
    pos = s["pos"].view(s["axes"], -1).long()
    cos = torch.stack([s["table"][pos[a], i] for i, a in enumerate(pair)], 1).double()
    sin = torch.stack([s["table"][pos[a], len(pair) + i] for i, a in enumerate(pair)], 1).double()
    cs = torch.cat([cos, sin], 1)
    q = _exact_turn(s["qt"].double(), cs, s["rot"], s["interleaved"])
    k = _exact_turn(s["kt"].double(), cs, s["rot"], s["interleaved"])
    v = s["vt"].double()
    if s["block"]:
        kc, ks = _exact_put(s["kc"], s["ks"], s["slots"], k, s["block"])
        vc, vs = _exact_put(s["vc"], s["vs"], s["slots"], v, s["block"])
        return [q, kc, vc, ks, vs]
    shape, width = s["kc"].shape, s["hkv"] * s["D"]
    kc, vc = s["kc"].double().reshape(-1, width), s["vc"].double().reshape(-1, width)
    kc.index_copy_(0, s["slots"], k.reshape(-1, width))
    vc.index_copy_(0, s["slots"], v.reshape(-1, width))
    return [q, kc.view(shape), vc.view(shape)]


def _exact_sequence(s, b, n):
    """One sequence over its own tokens alone."""
    hq, hkv, D, page, block = s["hq"], s["hkv"], s["D"], s["page"], s["block"]
    first = max(0, n - s["window"]) if s["window"] else 0
    if n <= first:
        return (torch.zeros(hq, D, dtype=torch.float64, device="cuda"),
                torch.full((hq,), -math.inf, dtype=torch.float64, device="cuda"))
    t = torch.arange(first, n, device="cuda")
    where = s["pages"][b].long()[t // page] * page + t % page
    k, v = s["kc"].reshape(-1, hkv, D)[where].double(), s["vc"].reshape(-1, hkv, D)[where].double()
    k = k * s["ks"].reshape(-1, hkv)[where // block].double()[:, :, None]
    v = v * s["vs"].reshape(-1, hkv)[where // block].double()[:, :, None]
    q = s["qt"][b].double().reshape(hkv, hq // hkv, D)
    a = torch.einsum("hgd,thd->hgt", q, k) * s["scale"]
    z = torch.logsumexp(a, -1)
    return torch.einsum("hgt,thd->hgd", torch.exp(a - z[..., None]), v).reshape(hq, D), z.reshape(hq)


def _exact_attend(s):
    each = [_exact_sequence(s, b, n) for b, n in enumerate(s["lens"].tolist())]
    return [torch.stack([o for o, _ in each]), torch.stack([z for _, z in each])]


def exact(case, seed):
    s = prepare(case, seed)
    return {"quant": _exact_quant, "linear": _exact_linear, "append": _exact_append, "axes": _exact_append,
            "attend": _exact_attend}[case["op"]](s)
