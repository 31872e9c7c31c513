"""Rows and caches in E4M3 with fine scales, and positions with several axes, against plain 64-bit forms.

Bounds come from the arithmetic, not from runs: U is half a step of an output type relative to the
value (2^-8, 2^-11, 2^-24; E4M3 2^-4), sums and factors are fp32 (2^-24 a step), and each test
states the rest."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
SUB = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}  # below the smallest normal the spacing is absolute
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import moe_decode_host_gb300 as mod

    return mod


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def within(got, want, tol, what=""):
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= tol) & ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist())


def e4m3_tol(v):
    """Half the spacing of E4M3 at v (2^-4 relative, 2^-10 below the smallest normal), widened by what
    fp32 adds before the rounding."""
    return v.abs() * (2.0 ** -4 + 1e-6) + 2.0 ** -10 * (1 + 1e-6)


# ---- quant --------------------------------------------------------------------


def quant64(x):
    T, K = x.shape
    G = -(-K // 128)
    p = torch.zeros(T, G * 128, dtype=torch.float64, device="cuda")
    p[:, :K] = x.double()
    s = (p.view(T, G, 128).abs().amax(2) / 448).clamp(min=TINY)
    return (p.view(T, G, 128) / s[:, :, None]).view(T, -1)[:, :K], s


def check_quant(m, x, y, s):
    m.moe_quant_e4m3(x, y, s)
    y64, s64 = quant64(x)
    # a product with the rounded 1 / 448: two roundings
    within(s, s64, s64 * 2.0 ** -23, "scale")
    within(y.float(), y64, e4m3_tol(y64), "codes")


@pytest.mark.parametrize("T,K", [(1, 1), (1, 127), (1, 128), (2, 129), (3, 136), (8, 4096), (5, 1000), (64, 2048), (33, 5003),
                                 (2, 16384), (700, 392), (1, 100000)])
@pytest.mark.parametrize("xt", [BF16, F16, F32])
def test_quant(m, T, K, xt):
    g = gen(T * 31 + K)
    x = (randn(g, T, K) * torch.exp(randn(g, K))).to(xt)
    check_quant(m, x, torch.empty(T, K, dtype=E4M3, device="cuda"), torch.empty(T, -(-K // 128), device="cuda"))


@pytest.mark.parametrize("offset", [0, 1, 4, 8])
def test_quant_of_views(m, offset):
    """Rows of wider tensors at any alignment; what lies beside the outputs stays."""
    g = gen(offset)
    x = randn(g, 50, 900).to(BF16)[:, offset:offset + 640]
    y = torch.full((50, 700), 3.0, device="cuda").to(E4M3)
    s = torch.full((50, 9), -1.0, device="cuda")
    check_quant(m, x, y[:, offset:offset + 640], s[:, 1:6])
    assert (y[:, :offset].float() == 3).all() and (y[:, offset + 640:].float() == 3).all()
    assert (s[:, 0] == -1).all() and (s[:, 6:] == -1).all()


@pytest.mark.parametrize("K", [384, 381])
def test_quant_special_groups(m, K):
    """Zeros, tiny and huge values, NaN and infinities: each stays in its group."""
    x = torch.ones(8, K, device="cuda")
    x[0, :128] = 0
    x[1, :128] = 2.0 ** -149
    x[2, :128] = 3.4e38
    x[3, 5], x[4, 130], x[5, K - 1] = float("nan"), float("inf"), -float("inf")
    x[6, :128] = 1e-38
    y, s = torch.empty(8, K, dtype=E4M3, device="cuda"), torch.empty(8, 3, device="cuda")
    m.moe_quant_e4m3(x, y, s)
    spoilt = torch.zeros(8, 3, dtype=torch.bool, device="cuda")
    spoilt[3, 0] = spoilt[4, 1] = spoilt[5, 2] = True
    assert (s.isnan() == spoilt).all()
    assert (y.float().isnan() == spoilt.repeat_interleave(128, 1)[:, :K]).all()
    y64, s64 = quant64(x.masked_fill(spoilt.repeat_interleave(128, 1)[:, :K], 0))
    keep = ~spoilt
    within(s[keep], s64[keep], s64[keep] * 2.0 ** -23)
    cols = keep.repeat_interleave(128, 1)[:, :K]
    within(y.float()[cols], y64[cols], e4m3_tol(y64[cols]))
    assert s[0, 0] == TINY and s[1, 0] == TINY and (y[0, :128].float() == 0).all()


def test_quant_same_scale_as_the_norm_and_no_rows(m):
    """A row of one group is what the norm's E4M3 form gives for it, codes apart by a rounding at most."""
    g = gen(3)
    x = randn(g, 40, 128).to(BF16)
    y, s = torch.empty(40, 128, dtype=E4M3, device="cuda"), torch.empty(40, 1, device="cuda")
    m.moe_quant_e4m3(x, y, s)
    assert ((y.float() * s).sub(x.float()).abs() <= x.float().abs() * (2.0 ** -4 + 1e-6) + s * 2.0 ** -9).all()
    m.moe_quant_e4m3(x[:0], y[:0], s[:0])


def test_quant_refusals(m):
    x = torch.zeros(4, 256, dtype=BF16, device="cuda")
    y, s = torch.empty(4, 256, dtype=E4M3, device="cuda"), torch.empty(4, 2, device="cuda")
    for kw in (dict(x=y), dict(y=x), dict(y=y[:, :128]), dict(scale=s[:, :1]), dict(scale=s.double()), dict(scale=s.half()),
               dict(x=x.t()), dict(scale=s.t().contiguous().t()), dict(x=x.cpu()), dict(scale=s[0]), dict(x=x[0])):
        with pytest.raises(m.MoeError) as err:
            m.moe_quant_e4m3(**{**dict(x=x, y=y, scale=s), **kw})
        assert err.value.code == m.MOE_ERR_INVALID_ARG
    with pytest.raises(m.MoeError):
        m.moe_quant_e4m3(x[:, :0], y[:, :0], s[:, :0])


# ---- positions with several axes ------------------------------------------------


def table(n, rot):
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(1, rot))
    return torch.cat([a.cos(), a.sin()], 1).float()


def turn64(x, cos, sin, interleaved):
    """x [T, heads, D] with pairs turned by cos, sin [T, pairs]; and the size of what is added up."""
    x = x.double().clone()
    rot = 2 * cos.shape[1]
    c, s = cos.double()[:, None, :], sin.double()[:, None, :]
    ia = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    ib = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = x[..., ia].clone(), x[..., ib].clone()
    x[..., ia], x[..., ib] = a * c - b * s, a * s + b * c
    size = torch.zeros_like(x)
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return x, size


def rows64(cs, pos, axes):
    pairs = cs.shape[1] // 2
    pick = [pos[a] for a in axes]
    cos = torch.stack([cs[p.long(), i] for i, p in enumerate(pick)], 1)
    return cos, torch.stack([cs[p.long(), pairs + i] for i, p in enumerate(pick)], 1)


AXES = {"sections": lambda n, a: [min(a - 1, i * a // n) for i in range(n)], "turns": lambda n, a: [i % a for i in range(n)],
        "fours": lambda n, a: [i // 4 % a for i in range(n)], "last": lambda n, a: [a - 1] * n}


@pytest.mark.parametrize("T,hq,hkv,D,rot,il", [
    (1, 32, 8, 128, 128, False), (5, 4, 4, 64, 64, True), (19, 6, 2, 80, 40, False), (3, 1, 1, 16, 2, False),
    (130, 8, 1, 256, 64, False), (17, 5, 1, 48, 18, True), (40, 12, 4, 256, 256, True), (700, 3, 1, 96, 96, False)])
@pytest.mark.parametrize("n_axes,pattern", [(1, "last"), (2, "sections"), (3, "turns"), (3, "fours"), (4, "sections"), (4, "turns")])
@pytest.mark.parametrize("xt,ct", [(BF16, BF16), (F16, E4M3), (F32, BF16)])
def test_axes(m, T, hq, hkv, D, rot, il, n_axes, pattern, xt, ct):
    g = gen(T * 31 + D + n_axes)
    qkv = randn(g, T, hq + 2 * hkv, D).to(xt)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    axes = AXES[pattern](rot // 2, n_axes)
    pos = torch.randint(0, 50, (n_axes, T + 3), generator=g, device="cuda", dtype=torch.int32)[:, :T]
    cs = table(50, rot)
    n_pages = -(-T // 16) + 1
    kc, vc = torch.zeros(2, n_pages, 16, hkv, D, device="cuda").to(ct)
    ks, vs = (torch.full((hkv,), 0.02, device="cuda"), torch.full((hkv,), 0.02, device="cuda")) if ct == E4M3 else (None, None)
    slots = torch.randperm(n_pages * 16, generator=g, device="cuda")[:T].contiguous()
    kv = m.KvCache(kc, vc, q_heads=hq, max_batch=1, k_scale=ks, v_scale=vs)
    qo = torch.empty(T, hq, D, dtype=xt, device="cuda")
    m.moe_kv_append(kv, q, k, v, pos, slots, cs, qo, interleaved=il, axes=bytes(axes) if T % 2 else axes)
    assert kv.status() == 0
    cos, sin = rows64(cs, pos, axes)
    q64, qsz = turn64(q, cos, sin, il)
    k64, ksz = turn64(k, cos, sin, il)
    within(qo, q64, q64.abs() * U[xt] + qsz * 2.0 ** -23 + SUB[xt], "q")  # two products and a sum in fp32
    gk, gv = kc.view(-1, hkv, D)[slots], vc.view(-1, hkv, D)[slots]
    if ct == E4M3:
        k64, v64, ksz = (k64 / ks.double()[:, None]).clamp(-448, 448), (v.double() / vs.double()[:, None]).clamp(-448, 448), ksz / 0.02
        within(gk.float(), k64, e4m3_tol(k64) + ksz * 2.0 ** -22, "k")
        within(gv.float(), v64, e4m3_tol(v64) + v64.abs() * 2.0 ** -22, "v")
    else:
        within(gk, k64, k64.abs() * U[ct] + ksz * 2.0 ** -23 + SUB[ct], "k")
        within(gv, v.double(), v.double().abs() * U[ct] + SUB[ct], "v")


@pytest.mark.parametrize("ct", [BF16, E4M3])
def test_axes_alike_are_one_position(m, ct):
    """Text has the same position along every axis: the bits are those of the call without axes."""
    g = gen(8)
    T, hq, hkv, D = 50, 8, 2, 64
    x = randn(g, T, hq + 2 * hkv, D).to(BF16)
    pos = torch.randint(0, 300, (T,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.arange(T, device="cuda")
    cs = table(300, D)
    res = []
    for axes in (None, [0] * 32, AXES["fours"](32, 3), AXES["turns"](32, 3)):
        c = torch.zeros(2, 4, 16, hkv, D, device="cuda").to(ct)
        sc = torch.zeros(2, 4, 2, hkv, device="cuda")
        kv = m.KvCache(c[0], c[1], q_heads=hq, max_batch=1, k_scale=sc[0] if ct == E4M3 else None, v_scale=sc[1] if ct == E4M3 else None)
        qo = torch.empty(T, hq, D, dtype=BF16, device="cuda")
        m.moe_kv_append(kv, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos if axes is None else pos.expand(3, T), slots, cs,
                        qo, axes=axes)
        res.append((qo, c.view(torch.uint8), sc))
    for r in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, res[0]))


@pytest.mark.parametrize("block", [0, 8])
def test_axes_out_of_the_table_and_refusals(m, block):
    g = gen(9)
    T, D = 6, 32
    x = randn(g, T, 4, D).to(BF16)
    ct = E4M3 if block else BF16
    c = torch.zeros(2, 2, 8, 1, D, device="cuda").to(ct)
    sc = torch.zeros(2, 2, 8 // block if block else 1, 1, device="cuda") if block else (None, None)
    kv = m.KvCache(c[0], c[1], q_heads=2, max_batch=1, k_scale=sc[0], v_scale=sc[1])
    pos = torch.tensor([[0, 1, 2, 3, 4, 5], [0, 9, 2, 10, 4, 5], [0, 1, -1, 3, 4, 5]], dtype=torch.int32, device="cuda")
    qo = torch.full((T, 2, D), 7.0, device="cuda").to(BF16)
    cs, axes = table(10, D), [0, 1, 2, 0] * 4
    args = lambda **kw: {**dict(kv=kv, q=x[:, :2], k=x[:, 2:3], v=x[:, 3:], positions=pos, slots=torch.arange(T, device="cuda"),  # noqa: E731
                                cos_sin=cs, q_out=qo, axes=axes), **kw}
    m.moe_kv_append(**args())
    assert kv.status() == m.MOE_ERR_BAD_INDEX
    kv.clear_status()
    keep = torch.tensor([True, True, False, False, True, True], device="cuda")
    cos, sin = rows64(cs, pos.clamp(0, 9), axes)
    q64, qsz = turn64(x[:, :2], cos, sin, False)
    within(qo[keep], q64[keep], q64[keep].abs() * U[BF16] + qsz[keep] * 2.0 ** -23)
    assert (qo[~keep].float() == 7).all()
    written = (c[0].view(-1, D)[:T].float() != 0).any(1)
    assert (written == keep).all()
    for bad in (dict(axes=axes[:-1]), dict(axes=[0, 1, 2, 3] * 4), dict(axes=[0, -1] * 8), dict(axes=b"\x00" * 17),
                dict(positions=pos[0]), dict(positions=pos[:, :5]), dict(positions=pos.long()), dict(axes=None),
                dict(positions=pos[:0]), dict(positions=pos.repeat(2, 1)[:5]), dict(cos_sin=None),
                dict(positions=pos.t().contiguous().t())):
        with pytest.raises(m.MoeError) as err:
            m.moe_kv_append(**args(**bad))
        assert err.value.code == m.MOE_ERR_INVALID_ARG, bad
    with pytest.raises(TypeError):
        m.moe_kv_append(**args(axes=5))
    assert kv.status() == 0


# ---- append to a cache with scales of blocks -----------------------------------


def power_for(top):
    """The smallest power of two s with top <= 448 s, from 2^-126 to 2^119 (exact, in 64 bits)."""
    f, e = torch.frexp(top.double())
    e = torch.where(f <= 0.875, e - 9, e - 8)
    e = torch.where(top > 0, e, torch.full_like(e, -126)).clamp(-126, 119)
    # by a table: torch.ldexp in 64 bits is off by an ulp for some e
    return torch.tensor([2.0 ** i for i in range(-126, 120)], dtype=torch.float64, device="cuda")[(e + 126).long()]


def put64(codes, scales, slots, x, block, ok):
    """What the cache holds after x [T, heads, D] (64 bits) went to its slots: codes unrounded, scales, and
    which entries were written."""
    hkv, D = x.shape[1:]
    out, sc = codes.double().reshape(-1, hkv, D).clone(), scales.double().view(-1, hkv).clone()
    wrote = torch.zeros(out.shape[0], dtype=torch.bool, device="cuda")
    slots = slots.tolist()
    t = 0
    while t < len(slots):
        u = t
        while u < len(slots) and slots[t] >= 0 and slots[u] >= 0 and slots[u] // block == slots[t] // block:
            u += 1
        if slots[t] < 0 or slots[t] >= out.shape[0]:
            t = t + 1
            continue
        who = [i for i in range(t, u) if ok[i]]
        home, at = slots[t] // block, [slots[i] for i in who]
        if who:
            now = power_for(x[who].abs().nan_to_num(nan=0.0, posinf=math.inf).amax((0, 2)).clamp(max=3e38))
            if home * block not in at:
                old = sc[home].clone()
                now = torch.maximum(now, old)
                out[home * block:(home + 1) * block] *= (old / now)[None, :, None]
            out[at] = (x[who] / now[None, :, None]).clamp(-448, 448)
            sc[home] = now
            wrote[at] = True
        t = u
    return out.view(codes.shape), sc.view(scales.shape), wrote


def block_cache(g, n_pages, page, block, hkv, D, size=1.0, hnd=False):
    v = size * randn(g, n_pages * page // block, block, hkv, D) * torch.exp(0.5 * randn(g, n_pages * page // block, 1, hkv, 1))
    s = power_for(v.abs().amax((1, 3))).float()
    c = (v / s[:, None, :, None]).to(E4M3).view(n_pages, page, hkv, D)
    if hnd:
        c = c.transpose(1, 2).contiguous().transpose(1, 2)
    return c, s.view(n_pages, page // block, hkv).contiguous()


def check_blocks(m, g, slots, hq, hkv, D, page, block, rot, xt, il=False, gain=1.0, size=0.3, hnd=False, x=None, n_pages=None):
    T = len(slots)
    n_pages = n_pages or max(slots) // page + 2
    slots = torch.tensor(slots, device="cuda")
    x = (gain * randn(g, T, hq + 2 * hkv, D)).to(xt) if x is None else x
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    kc, ks = block_cache(g, n_pages, page, block, hkv, D, size, hnd)
    vc, vs = block_cache(g, n_pages, page, block, hkv, D, size, hnd)
    k0, v0, ks0, vs0 = kc.clone(), vc.clone(), ks.clone(), vs.clone()
    kv = m.KvCache(kc, vc, q_heads=hq, max_batch=1, k_scale=ks, v_scale=vs)
    pos = torch.randint(0, 60, (T,), generator=g, device="cuda", dtype=torch.int32)
    cs = table(60, rot) if rot else None
    qo = torch.empty(T, hq, D, dtype=xt, device="cuda")
    m.moe_kv_append(kv, q, k, v, pos, slots, cs, qo, interleaved=il)
    assert kv.status() == 0
    cos, sin = rows64(cs, [pos], [0] * (rot // 2)) if rot else (torch.zeros(T, 0, device="cuda"),) * 2
    q64, qsz = turn64(q, cos, sin, il)
    within(qo, q64, q64.abs() * U[xt] + qsz * 2.0 ** -23 + SUB[xt], "q")
    k64, ksz = turn64(k, cos, sin, il)
    for codes, scales, c0, s0, x64, sz in ((kc, ks, k0, ks0, k64, ksz), (vc, vs, v0, vs0, v.double(), torch.zeros_like(ksz))):
        want, sc, wrote = put64(c0, s0, slots, x64, block, [True] * T)
        assert torch.equal(scales.double(), sc)
        per = sc.view(-1, hkv).repeat_interleave(block, 0).view(codes.shape[0], page, hkv, 1)
        slack = torch.zeros(n_pages * page, hkv, D, dtype=torch.float64, device="cuda")
        slack[slots[slots >= 0]] = sz[slots >= 0] * 2.0 ** -22
        within(codes.float(), want, e4m3_tol(want) + slack.view(want.shape) / per, "codes")
        # nothing else changed: blocks that the call did not touch, and others under a scale that stayed
        same = (sc == s0.double()).view(-1, 1, hkv, 1).expand(-1, block, -1, D).reshape(-1, hkv, D) & ~wrote[:, None, None]
        flat, flat0 = codes.view(torch.uint8).reshape(-1, hkv, D), c0.view(torch.uint8).reshape(-1, hkv, D)
        assert torch.equal(flat[same], flat0[same])
    return kv


def order(g, n):
    return torch.randperm(n, generator=g, device="cuda").tolist()


def run_slots(g, page, runs):
    """Slots of sequences, (first entry in its first page, tokens) each, on pages in any order."""
    need = [-(-(a + n) // page) for a, n in runs]
    pages = order(g, sum(need) + 1)
    out, p = [], 0
    for (a, n), k in zip(runs, need):
        out += [pages[p + (a + i) // page] * page + (a + i) % page for i in range(n)]
        p += k
    return out


@pytest.mark.parametrize("page,block", [(16, 16), (64, 32), (64, 64), (7, 7), (14, 7), (24, 6), (32, 1), (1, 1), (128, 128),
                                        (512, 256), (2048, 1024), (30, 10), (16, 4)])
@pytest.mark.parametrize("runs", [[(0, 1)], [(3, 1), (0, 1), (9, 1)], [(0, 70)], [(5, 200), (0, 3), (11, 40)]])
def test_blocks_pages(m, page, block, runs):
    g = gen(page + len(runs))
    check_blocks(m, g, run_slots(g, page, [(a % page, n) for a, n in runs]), 4, 2, 64, page, block, 64, BF16)


@pytest.mark.parametrize("hq,hkv,D,rot,il", [(32, 8, 128, 128, False), (3, 3, 80, 40, False), (1, 1, 16, 2, True), (8, 1, 256, 64, False),
                                             (5, 1, 48, 18, True), (6, 2, 96, 96, False), (12, 4, 256, 256, True), (2, 2, 112, 0, False)])
@pytest.mark.parametrize("xt", [BF16, F16, F32])
@pytest.mark.parametrize("block", [4, 16])
def test_blocks_heads(m, hq, hkv, D, rot, il, xt, block):
    g = gen(D + rot)
    check_blocks(m, g, run_slots(g, 32, [(3, 60), (0, 32), (17, 1)]), hq, hkv, D, 32, block, rot, xt, il)
    check_blocks(m, g, run_slots(g, 32, [(30, 5)]), hq, hkv, D, 32, block, rot, xt, il, hnd=True)


def test_blocks_many_tokens(m):
    g = gen(4)
    check_blocks(m, g, run_slots(g, 64, [(0, 3000), (13, 1500)]), 4, 2, 128, 64, 64, 128, BF16)
    check_blocks(m, g, run_slots(g, 16, [(0, 700), (1, 2100), (15, 2)]), 2, 1, 64, 16, 2, 64, F16)
    check_blocks(m, g, run_slots(g, 64, [(i % 64, 1) for i in range(600)]), 8, 8, 128, 64, 32, 128, BF16)


@pytest.mark.parametrize("size", [1e-6, 50.0])
@pytest.mark.parametrize("xt,block", [(BF16, 64), (F16, 16), (F32, 64), (BF16, 4)])
def test_blocks_long_and_short_runs(m, xt, block, size):
    """Runs of one token to many blocks, which begin at every place among four tokens and in blocks that hold
    some, under scales that are too small for the new tokens and such that are large enough."""
    g = gen(block)
    lens = [1, 1, 2, 70, 3, 1, 1, 1, 5, 4, 66, 1, 8, 40, 1, 1, 1, 1, 2, 33]
    check_blocks(m, g, run_slots(g, 64, [((7 * i + 1) % 64, n) for i, n in enumerate(lens)]), 4, 2, 128, 64, block, 128, xt, size=size)
    check_blocks(m, g, run_slots(g, 64, [(0, 200)]), 32, 8, 128, 64, block, 64, xt, size=size)


def test_blocks_tokens_left_out(m):
    """Negative slots, in the middle of a block's tokens too; every scale large enough, and every one too small."""
    g = gen(5)
    s = run_slots(g, 32, [(0, 40), (5, 20)])
    s[3] = s[50] = -1
    # a run ends at a token that is left out: the block's tokens then do not follow one another, so the hole
    # lies where one block ends
    s = [x for x in s if x >= 0]
    cut = next(i for i in range(1, len(s)) if s[i] // 16 != s[i - 1] // 16)
    s = s[:cut] + [-1, -5] + s[cut:]
    check_blocks(m, g, s, 4, 2, 64, 32, 16, 64, BF16)
    mid = run_slots(g, 32, [(5, 8), (20, 4), (1, 1)])
    check_blocks(m, g, mid, 4, 2, 64, 32, 16, 64, BF16, size=50.0)
    check_blocks(m, g, mid, 4, 2, 64, 32, 16, 64, BF16, size=1e-6)
    check_blocks(m, g, mid, 4, 2, 64, 32, 16, 64, F32, gain=1e30, size=1e-30)
    check_blocks(m, g, mid, 4, 2, 64, 32, 16, 64, F32, gain=1e-35, size=1e-38)


def test_blocks_special_values(m):
    """Zeros, NaN, infinities and values at the ends of the range and at a scale's edge."""
    g = gen(6)
    D, n = 32, 12
    x = torch.zeros(n, 3, D, device="cuda")
    x[1, :, 3] = 448.0
    x[2, :, 3] = 448.0 * (1 + 2.0 ** -23)
    x[3, :, 0] = float("nan")
    x[4, :, 1] = float("inf")
    x[5, :, 2] = -3.4e38
    x[6, :, 2] = 2.0 ** -149
    x[7] = 1e-3
    x[8, :, 0] = float("nan")
    x[8, :, 1] = 1.0
    slots = torch.arange(n, device="cuda") * 4  # a block each
    kc, ks = torch.full((2, 4 * n // 2, 1, D), 1.0, device="cuda").to(E4M3), torch.ones(2, n // 2, 1, device="cuda")
    vc, vs = kc.clone(), ks.clone()
    kv = m.KvCache(kc, vc, q_heads=1, max_batch=1, k_scale=ks, v_scale=vs)
    m.moe_kv_append(kv, x[:, :1], x[:, 1:2], x[:, 2:], None, slots, None, torch.empty(n, 1, D, device="cuda"))
    assert kv.status() == 0
    top, low = 2.0 ** 119, TINY
    want = [low, 1.0, 2.0, low, top, top, low, 2.0 ** -18, 2.0 ** -8, low, low, low]
    assert 448 * 2.0 ** -19 < 1e-3 <= 448 * 2.0 ** -18 and 448 * 2.0 ** -9 < 1.0 <= 448 * 2.0 ** -8
    for codes, scales in ((kc, ks), (vc, vs)):
        assert scales.view(-1).tolist() == want
        c = codes.view(n, 4, D).float()[:, 0]
        assert c[3, 0].isnan() and not c[3, 1:].isnan().any() and c[8, 0].isnan() and c[8, 1] == 256
        assert c[4, 1] == 448 and c[5, 2] == -448 and (c[0] == 0).all() and c[1, 3] == 448 and c[2, 3] == 224 and c[6, 2] == 0
        assert (codes.view(n, 4, D).float()[:, 1:] == 1).all()  # the blocks start anew: their other bytes stay


def test_blocks_grow_and_keep(m):
    """Token by token, as a decode step does: what a block holds keeps its values as its scale grows."""
    g = gen(7)
    D, hkv, block = 64, 2, 16
    kc = torch.zeros(1, 32, hkv, D, device="cuda").to(E4M3)
    vc, ks, vs = kc.clone(), torch.zeros(1, 2, hkv, device="cuda"), torch.zeros(1, 2, hkv, device="cuda")
    kv = m.KvCache(kc, vc, q_heads=2, max_batch=1, k_scale=ks, v_scale=vs)
    all_k = []
    for t in range(32):
        x = (randn(g, 1, 6, D) * 1.5 ** (t % block)).to(BF16)
        m.moe_kv_append(kv, x[:, :2], x[:, 2:4], x[:, 4:], None, torch.tensor([t], device="cuda"), None, torch.empty_like(x[:, :2]))
        all_k.append(x[:, 2:4].double())
        want = torch.cat(all_k)
        per = ks.double().repeat_interleave(block, 1).view(-1, hkv, 1)[:t + 1]
        got = kc.view(-1, hkv, D)[:t + 1].double() * per
        # half a step of E4M3 at first and at most half a step of each subnormal rewriting after it; a scale
        # doubles at most 20 times here, and each step is half as large as the next
        within(got, want, want.abs() * 2.0 ** -4 + per * 2.0 ** -10 * 2)
        first = t // block * block
        top = want[first:].abs().amax((0, 2))
        assert torch.equal(ks.view(2, hkv)[t // block].double(), power_for(top))


def test_blocks_in_place_graph_stream_and_bad_slots(m):
    g = gen(10)
    T, hq, hkv, D, page, block = 5, 4, 2, 64, 32, 16
    x = randn(g, T, hq + 2 * hkv, D).to(BF16)
    slots = torch.tensor([3, 40, 100, 70, 1 << 40], device="cuda")  # 100 and the last are past the last page
    kc, ks = block_cache(g, 3, page, block, hkv, D, 0.01)
    vc, vs = block_cache(g, 3, page, block, hkv, D, 0.01)
    k0, ks0 = kc.clone(), ks.clone()
    kv = m.KvCache(kc, vc, q_heads=hq, max_batch=1, k_scale=ks, v_scale=vs)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    cs = table(T, D)
    cos, sin = rows64(cs, [pos], [0] * (D // 2))
    q64, qsz = turn64(x[:, :hq], cos, sin, False)
    k64, _ = turn64(x[:, hq:hq + hkv], cos, sin, False)
    y = x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m.moe_kv_append(kv, y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:], pos, slots, cs, y[:, :hq], stream=s)  # q in place
    s.synchronize()
    assert kv.status() == m.MOE_ERR_BAD_INDEX
    within(y[:, :hq], q64, q64.abs() * U[BF16] + qsz * 2.0 ** -23)
    want, sc, _ = put64(k0, ks0, slots, k64, block, [True] * T)
    assert torch.equal(ks.double(), sc)
    within(kc.float(), want, e4m3_tol(want) + 1e-3)
    kv.clear_status()
    # captured: the slots are read at each replay
    slots.copy_(torch.tensor([8, 9, 10, 64, 65], device="cuda"))
    qo = torch.empty(T, hq, D, dtype=BF16, device="cuda")
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            m.moe_kv_append(kv, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, slots, cs, qo)
    for first in (8, 16, 27):
        slots[:3] = torch.arange(first, first + 3, device="cuda")
        k1, ks1 = kc.clone(), ks.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, sc, _ = put64(k1, ks1, slots, k64, block, [True] * T)
        assert torch.equal(ks.double(), sc)
        within(kc.float(), want, e4m3_tol(want) + 1e-3)
    assert kv.status() == 0
    m.moe_kv_append(kv, x[:0, :hq], x[:0, hq:hq + hkv], x[:0, hq + hkv:], pos[:0], slots[:0], cs, qo[:0])


def test_block_cache_refusals(m):
    k = torch.zeros(4, 24, 2, 64, device="cuda").to(E4M3)
    s = torch.zeros(4, 3, 2, device="cuda")
    for a, b, kc in ((s[:, :, :1], s, k), (s, s[:3], k), (s.double(), s, k), (s.transpose(0, 1), s, k), (s, None, k), (None, s, k),
                     (torch.zeros(4, 5, 2, device="cuda"),) * 2 + (k,), (s, s, k.to(BF16)), (s.cpu(), s, k), (s, s[0, 0], k),
                     (torch.zeros(4, 0, 2, device="cuda"),) * 2 + (k,)):
        with pytest.raises(m.MoeError) as err:
            m.KvCache(kc, kc, q_heads=2, max_batch=1, k_scale=a, v_scale=b)
        assert err.value.code == m.MOE_ERR_INVALID_ARG
    big = torch.zeros(1, 2048, 1, 16, device="cuda").to(E4M3)
    with pytest.raises(m.MoeError):  # a block of 2048 tokens
        m.KvCache(big, big, q_heads=1, max_batch=1, k_scale=torch.zeros(1, 1, 1, device="cuda"), v_scale=torch.zeros(1, 1, 1, device="cuda"))


# ---- attention over a cache with scales of blocks -------------------------------


def attend64(q, k, v, ks, vs, pages, lens, scale, window):
    """Per sequence: output, log-sum, and the bounds of both.

    A score is a sum of D products in fp32 and a product with its key's scale (D + 3 steps of 2^-24 of
    sum |q||k|).  A weight has an exponential good to 2^-21 and the score's error on top, is multiplied by
    its value's scale (2^-23 with the reference) and goes into the products as two f16 terms, which lose
    2^-22 of it and, below f16's range, 2^-31 of the largest weight times the largest scale; the weighted
    sum adds one fp32 step for every 16 tokens."""
    page, hkv, D = k.shape[1], k.shape[2], k.shape[3]
    block = page // ks.shape[1]
    g = q.shape[1] // hkv
    outs, lses, otol, ltol = [], [], [], []
    for b, n in enumerate(lens):
        t = torch.arange(max(0, n - window) if window else 0, n, device="cuda")
        if t.numel() == 0:
            z = torch.zeros(q.shape[1], D, dtype=torch.float64, device="cuda")
            outs.append(z), otol.append(z), ltol.append(z[:, 0]), lses.append(z[:, 0] - math.inf)
            continue
        p, e = pages[b].long()[t // page], t % page
        kk = k[p, e].double() * ks[p, e // block].double()[..., None]
        vsc = vs[p, e // block].double()[..., None]
        vv = v[p, e].double() * vsc
        qq = q[b].double().view(hkv, g, D)
        s = torch.einsum("hgd,thd->hgt", qq, kk) * scale
        es = torch.einsum("hgd,thd->hgt", qq.abs(), kk.abs()).amax(-1) * abs(scale) * (D + 3) * 2.0 ** -24
        lse = torch.logsumexp(s, -1)
        w = torch.exp(s - lse[..., None])
        o = torch.einsum("hgt,thd->hgd", w, vv)
        size = torch.einsum("hgt,thd->hgd", w, vv.abs())
        rel = 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -23 + 2 * es + (len(t) / 16 + 8) * 2.0 ** -24
        floor = w.amax(-1)[..., None] * 2.0 ** -31 * (v[p, e].double().abs().sum(0) * vsc.abs().amax(0))[:, None, :]
        outs.append(o.reshape(-1, D)), lses.append(lse.reshape(-1))
        otol.append((size * rel[..., None] * 1.01 + floor + o.abs() * U[q.dtype] * 1.01 + SUB[q.dtype]).reshape(-1, D))
        ltol.append((es + 2.0 ** -21 + (len(t) / 16 + 8) * 2.0 ** -24 + lse.abs() * 2.0 ** -22).reshape(-1))
    return torch.stack(outs), torch.stack(lses), torch.stack(otol), torch.stack(ltol)


def check_attend(m, g, lens, hq, hkv, D, page, block, qt, window=0, scale=None, hnd=False, gain=1.0, odd=False):
    per = max(1, -(-max(lens + [0]) // page))
    n_pages = sum(-(-n // page) for n in lens) + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    pages = torch.full((len(lens), per), 2 ** 30, dtype=torch.int32, device="cuda")  # past a sequence's end: never read
    at = 0
    for b, n in enumerate(lens):
        need = -(-n // page)
        pages[b, :need] = perm[at:at + need]
        at += need
    k, ks = block_cache(g, n_pages, page, block, hkv, D, 1.0, hnd)
    v, vs = block_cache(g, n_pages, page, block, hkv, D, 1.0, hnd)
    if odd:  # scales of the caller's own: any numbers
        ks = ks * (randn(g, *ks.shape) + 1.5)
        vs = vs * (randn(g, *vs.shape) - 0.5)
    q = (gain * randn(g, len(lens), hq, D)).to(qt)
    kv = m.KvCache(k, v, q_heads=hq, max_batch=len(lens), k_scale=ks, v_scale=vs)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    outs = []
    for _ in range(3):  # the same call gives the same bits
        o = torch.full_like(q, float("nan"))
        lse = torch.full((len(lens), hq), float("nan"), device="cuda")
        m.moe_kv_attend(kv, q, pages, n, o, scale=scale, window=window, lse=lse)
        outs.append((o, lse))
    assert kv.status() == 0
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
    o64, l64, ot, lt = attend64(q, k, v, ks, vs, pages, lens, D ** -0.5 if scale is None else scale, window)
    within(outs[0][0], o64, ot, "out")
    within(outs[0][1], l64, lt, "lse")


@pytest.mark.parametrize("hq,hkv,D", [(1, 1, 16), (4, 4, 64), (32, 8, 128), (7, 1, 96), (16, 1, 128), (24, 2, 80), (6, 2, 256),
                                      (40, 1, 64), (3, 1, 192), (64, 1, 112), (128, 2, 128), (17, 1, 208)])
@pytest.mark.parametrize("qt", [BF16, F16])
@pytest.mark.parametrize("block", [16, 4])
def test_attend_heads(m, hq, hkv, D, qt, block):
    check_attend(m, gen(hq * 100 + D), [0, 1, 2, 15, 16, 17, 63, 64, 65, 300], hq, hkv, D, 16, block, qt)


@pytest.mark.parametrize("page,block", [(1, 1), (3, 3), (7, 1), (14, 7), (33, 11), (64, 64), (64, 32), (128, 8), (1000, 500), (1024, 1024)])
@pytest.mark.parametrize("window", [0, 1, 5, 16, 100])
def test_attend_pages_and_windows(m, page, block, window):
    check_attend(m, gen(page), [0, 1, 99, 100, 101, 250, 17], 8, 2, 64, page, block, BF16, window=window)
    check_attend(m, gen(page + 1), [33, 0, 40], 4, 4, 96, page, block, F16, window=window, hnd=True, odd=True)


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [5000], [1, 40000], [20000, 0, 3], list(range(0, 700, 3)), [700] * 40,
                                  [1] * 500, [320] * 76])
@pytest.mark.parametrize("hq,D", [(8, 128), (32, 64), (4, 256)])
def test_attend_batches(m, lens, hq, D):
    check_attend(m, gen(len(lens)), lens, hq, 2, D, 32, 16, BF16)


def test_attend_scores_and_scales_far_apart(m):
    check_attend(m, gen(1), [300, 50], 8, 2, 64, 16, 8, BF16, scale=8.0, gain=4.0)
    check_attend(m, gen(2), [300, 50], 8, 2, 64, 16, 8, F16, scale=-1.0, odd=True)
    check_attend(m, gen(3), [300, 50], 8, 2, 64, 16, 8, BF16, scale=0.0)
    check_attend(m, gen(4), [300, 50], 8, 2, 64, 16, 8, BF16, gain=1e4)
    # value blocks 2^20 apart, in both orders along the sequence, the small ones with nearly all of the weight
    g = gen(5)
    n, D = 200, 64
    k, ks = block_cache(g, 13, 16, 16, 1, D)
    v, vs = block_cache(g, 13, 16, 16, 1, D)
    pages = torch.arange(13, dtype=torch.int32, device="cuda")[None]
    for large in (slice(0, 6), slice(6, 13), slice(3, 13, 4)):
        big = torch.zeros(13, dtype=torch.bool, device="cuda")
        big[large] = True
        sc = vs * torch.where(big, 2.0 ** 10, 2.0 ** -10)[:, None, None]
        kk = (k.float().abs() * torch.where(big, -1.0, 1.0)[:, None, None, None]).to(E4M3)
        q = torch.full((1, 4, D), 0.25, device="cuda").to(BF16)
        kv = m.KvCache(kk, v, q_heads=4, max_batch=1, k_scale=ks, v_scale=sc)
        o, lse = torch.empty_like(q), torch.empty(1, 4, device="cuda")
        m.moe_kv_attend(kv, q, pages, torch.tensor([n], dtype=torch.int32, device="cuda"), o, lse=lse)
        o64, l64, ot, lt = attend64(q, kk, v, ks, sc, pages, [n], D ** -0.5, 0)
        within(o, o64, ot)
        within(lse, l64, lt)


@pytest.mark.parametrize("e", [-126, -60, 60, 96])
def test_attend_scales_at_the_ends(m, e):
    """Values' scales from 2^-126 to 2^96, and keys' with scores of ordinary size under them."""
    g = gen(6)
    k, ks = block_cache(g, 6, 16, 8, 2, 64)
    v, vs = block_cache(g, 6, 16, 8, 2, 64)
    p = 2.0 ** e
    ks, vs = torch.full_like(ks, p), torch.full_like(vs, p)
    pages = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    q = randn(g, 1, 4, 64).to(BF16)
    scale = 2.0 ** max(-120, -10 - e)
    kv = m.KvCache(k, v, q_heads=4, max_batch=1, k_scale=ks, v_scale=vs)
    o, lse = torch.empty_like(q), torch.empty(1, 4, device="cuda")
    n = torch.tensor([90], dtype=torch.int32, device="cuda")
    m.moe_kv_attend(kv, q, pages, n, o, scale=scale, lse=lse)
    o64, l64, ot, lt = attend64(q, k, v, ks, vs, pages, [90], scale, 0)
    within(o, o64, ot + p * 2.0 ** -133)
    within(lse, l64, lt)


def test_attend_ignores_what_is_not_attended(m):
    """NaN and infinities in codes and scales behind a sequence's end, before its window and in pages of no
    sequence leave every result as it was."""
    g = gen(9)
    lens, page, block = [37, 5, 100], 16, 4
    k, ks = block_cache(g, 16, page, block, 2, 64)
    v, vs = block_cache(g, 16, page, block, 2, 64)
    perm = torch.randperm(16, generator=g, device="cuda").to(torch.int32)
    pages = torch.stack([perm[:7], perm[7:14], perm[[14, 15, 3, 4, 5, 6, 2]]])
    pages[0, 3:], pages[1, 1:] = 99, -5
    q = randn(g, 3, 8, 64).to(BF16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kv = m.KvCache(k, v, q_heads=8, max_batch=3, k_scale=ks, v_scale=vs)
    clean = torch.empty_like(q)
    m.moe_kv_attend(kv, q, pages, n, clean, window=30)
    seen = torch.zeros(16, page, dtype=torch.bool, device="cuda")
    for b, x in enumerate(lens):
        t = torch.arange(max(0, x - 30), x, device="cuda")
        seen[pages[b].long()[t // page], t % page] = True
    used = seen.view(16, page // block, block).any(2)
    k.view(torch.uint8)[~seen] = v.view(torch.uint8)[~seen] = 0x7f  # NaN
    for bad in (float("nan"), float("inf"), -float("inf"), 3e38):
        ks[~used], vs[~used] = bad, bad
        got = torch.empty_like(q)
        m.moe_kv_attend(kv, q, pages, n, got, window=30)
        assert torch.equal(got, clean)
    assert kv.status() == 0


def test_attend_nan_where_it_is_attended(m):
    """A NaN among a head's keys' or values' scales or codes shows in that head's outputs alone."""
    g = gen(12)
    k, ks = block_cache(g, 4, 16, 8, 2, 64)
    v, vs = block_cache(g, 4, 16, 8, 2, 64)
    pages = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    q = randn(g, 1, 4, 64).to(BF16)
    n = torch.tensor([60], dtype=torch.int32, device="cuda")
    for what in range(3):
        a, b, c = ks.clone(), vs.clone(), v.clone()
        if what == 0:
            a[2, 1, 1] = float("nan")
        elif what == 1:
            b[2, 1, 1] = float("nan")
        else:
            c.view(torch.uint8)[2, 3, 1] = 0x7f  # NaN
        kv = m.KvCache(k, c, q_heads=4, max_batch=1, k_scale=a, v_scale=b)
        o, lse = torch.empty_like(q), torch.empty(1, 4, device="cuda")
        m.moe_kv_attend(kv, q, pages, n, o, lse=lse)
        assert o[0, 2:].isnan().all() and o[0, :2].isfinite().all() and lse[0, :2].isfinite().all()
        assert lse[0, 2:].isnan().all() if what == 0 else lse[0, 2:].isfinite().all()


def test_attend_reports_and_clamps(m):
    g = gen(13)
    k, ks = block_cache(g, 12, 8, 4, 1, 32)
    v, vs = block_cache(g, 12, 8, 4, 1, 32)
    pages = torch.randperm(12, generator=g, device="cuda").to(torch.int32)[:10].view(2, 5).contiguous()
    q = randn(g, 2, 2, 32).to(BF16)
    kv = m.KvCache(k, v, q_heads=2, max_batch=2, k_scale=ks, v_scale=vs)
    out = torch.empty_like(q)
    n = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    m.moe_kv_attend(kv, q, pages, n(1000, -3), out)  # longer than its row of the table, and negative
    assert kv.status() == m.MOE_ERR_BAD_INDEX and (out[1] == 0).all()
    o64, _, ot, _ = attend64(q, k, v, ks, vs, pages, [40, 0], 32 ** -0.5, 0)
    within(out, o64, ot)
    kv.clear_status()
    for wrong in (12, -1, 2 ** 31 - 1):
        bad = pages.clone()
        bad[0, 2] = wrong  # tokens 16..23 are left out
        m.moe_kv_attend(kv, q, bad, n(40, 30), out)
        assert kv.status() == m.MOE_ERR_BAD_INDEX
        kv.clear_status()
        short = pages.clone()
        short[0, 2:4] = pages[0, 3:5]
        o64, _, ot, _ = attend64(q, k, v, ks, vs, short, [32, 30], 32 ** -0.5, 0)
        within(out, o64, ot)


def test_attend_far_offsets(m):
    """Scales past 2^31 bytes and a cache whose later pages lie past 2^32."""
    n_pages, page, hkv, D = 3000, 1024, 1, 16
    stride = (5 << 30) // n_pages // 16 * 16
    room = torch.empty(2, n_pages * stride, dtype=torch.uint8, device="cuda").view(E4M3)
    g = gen(14)
    k, v = (r.as_strided((n_pages, page, hkv, D), (stride, D, D, 1)) for r in room)
    c, s = block_cache(g, 4, page, 1, hkv, D)
    pages = torch.tensor([[0, n_pages - 1, 1500, n_pages - 2]], dtype=torch.int32, device="cuda")
    ks = torch.full((n_pages, page, hkv), float("nan"), device="cuda")
    vs = ks.clone()
    for i, p in enumerate(pages[0].tolist()):
        k[p], v[p], ks[p], vs[p] = c[i], c[3 - i], s[i], s[3 - i]
    q = randn(g, 1, 4, D).to(BF16)
    kv = m.KvCache(k, v, q_heads=4, max_batch=1, k_scale=ks, v_scale=vs)
    o = torch.empty_like(q)
    m.moe_kv_attend(kv, q, pages, torch.tensor([4 * page - 9], dtype=torch.int32, device="cuda"), o)
    o64, _, ot, _ = attend64(q, k, v, ks, vs, pages, [4 * page - 9], D ** -0.5, 0)
    within(o, o64, ot)
    # and the append writes there
    x = randn(g, 2, 6, D).to(BF16)
    slots = torch.tensor([(n_pages - 1) * page + 7, (n_pages - 1) * page + 8], device="cuda")
    m.moe_kv_append(kv, x[:, :4], x[:, 4:5], x[:, 5:], None, slots, None, torch.empty(2, 4, D, dtype=BF16, device="cuda"))
    got = k[n_pages - 1, 7:9].double() * ks[n_pages - 1, 7:9].double()[..., None]
    within(got, x[:, 4:5].double(), x[:, 4:5].double().abs() * 2.0 ** -4)


# ---- together ------------------------------------------------------------------


def test_append_then_attend_as_decoding_goes(m):
    """A prompt, then steps of one token each, captured once: the attention sees what the appends left."""
    g = gen(15)
    hq, hkv, D, page, block = 8, 2, 64, 16, 8
    start, steps = [21, 0, 40], 20
    per = -(-(max(start) + steps) // page)
    pages = torch.randperm(3 * per + 2, generator=g, device="cuda").to(torch.int32)[:3 * per].view(3, per).contiguous()
    kc = torch.zeros(3 * per + 2, page, hkv, D, device="cuda").to(E4M3)
    vc, ks = kc.clone(), torch.zeros(3 * per + 2, page // block, hkv, device="cuda")
    vs = ks.clone()
    kv = m.KvCache(kc, vc, q_heads=hq, max_batch=3, k_scale=ks, v_scale=vs)
    cs, axes = table(200, D), AXES["fours"](D // 2, 3)
    keys, vals = [[] for _ in start], [[] for _ in start]

    def place(b, t):
        return int(pages[b, t // page]) * page + t % page

    def note(x, pos, who):
        cos, sin = rows64(cs, pos, axes)
        k64, _ = turn64(x[:, hq:hq + hkv], cos, sin, False)
        for i, b in enumerate(who):
            keys[b].append(k64[i]), vals[b].append(x[i, hq + hkv:].double())

    who = [b for b, n in enumerate(start) for _ in range(n)]
    slots = torch.tensor([place(b, t) for b, n in enumerate(start) for t in range(n)], device="cuda")
    x = randn(g, len(who), hq + 2 * hkv, D).to(BF16)
    pos = torch.randint(0, 200, (3, len(who)), generator=g, device="cuda", dtype=torch.int32)
    m.moe_kv_append(kv, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, slots, cs, torch.empty(len(who), hq, D, dtype=BF16, device="cuda"), axes=axes)
    note(x, pos, who)
    x = torch.empty(3, hq + 2 * hkv, D, dtype=BF16, device="cuda")
    pos, slots = torch.zeros(3, 3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    q, o = torch.empty(3, hq, D, dtype=BF16, device="cuda"), torch.empty(3, hq, D, dtype=BF16, device="cuda")
    slots.fill_(-1)

    def step():
        m.moe_kv_append(kv, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, slots, cs, q, axes=bytes(axes))
        m.moe_kv_attend(kv, q, pages, lens, o)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    for i in range(steps):
        x.copy_(randn(g, 3, hq + 2 * hkv, D) * 1.3 ** i)
        pos.copy_(torch.randint(0, 200, (3, 3), generator=g, device="cuda"))
        slots.copy_(torch.tensor([place(b, n + i) for b, n in enumerate(start)]))
        lens.copy_(torch.tensor([n + i + 1 for n in start]))
        graph.replay()
        torch.cuda.synchronize()
        note(x, pos, range(3))
        # what the cache holds is within E4M3 of what went in; the attention is that of what it holds
        o64, _, ot, _ = attend64(q, kc, vc, ks, vs, pages, lens.tolist(), D ** -0.5, 0)
        within(o, o64, ot)
        for b, n in enumerate(lens.tolist()):
            t = torch.arange(n, device="cuda")
            p, e = pages[b].long()[t // page], t % page
            for c, sc, want in ((kc, ks, torch.stack(keys[b])), (vc, vs, torch.stack(vals[b]))):
                per_t = sc[p, e // block].double()[..., None]
                within(c[p, e].double() * per_t, want, want.abs() * (2.0 ** -4 + 1e-6) + per_t * 2.0 ** -10 * 2.01)
    assert kv.status() == 0
