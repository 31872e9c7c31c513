"""Rows and caches in E4M3 with fine scales, where their definitions are easiest to miss: codes at a tie, scales of the
caller's own making, sums at the end of fp32, tokens that do not follow one another, and the kernels for many tokens on
every kind of input.

Bounds come from the arithmetic; helpers and their bounds are those of the operators' own tests."""
import pytest
import torch

from test_gpu_fine_scales import (AXES, BF16, E4M3, F16, F32, SUB, U, attend64, block_cache, e4m3_tol, gen, m, put64,  # noqa: F401
                                  randn, rows64, run_slots, table, turn64, within)
from test_gpu_linear_blocks import operands

pytestmark = pytest.mark.gpu


# ---- quant --------------------------------------------------------------------


def check_quotients(m, x):  # noqa: F811
    """Codes are those of x / scale under the scale that the call returns: one division in fp32, one rounding."""
    T, K = x.shape
    y, s = torch.empty(T, K, dtype=E4M3, device="cuda"), torch.empty(T, -(-K // 128), device="cuda")
    m.moe_quant_e4m3(x, y, s)
    per = s.repeat_interleave(128, 1)[:, :K]
    want = (x.float() / per).to(E4M3)  # |x / scale| is at most 448 and a few roundings: no saturation
    bad = y.view(torch.uint8) != want.view(torch.uint8)
    assert not bad.any(), (int(bad.sum()), x[bad][:4].tolist(), per[bad][:4].tolist(), y.float()[bad][:4].tolist())


@pytest.mark.parametrize("xt", [BF16, F16, F32])
@pytest.mark.parametrize("K", [4096, 1003])
def test_quant_codes_are_quotients(m, xt, K):  # noqa: F811
    g = gen(K)
    check_quotients(m, randn(g, 300, K).to(xt))
    # whole numbers and halves: many quotients lie on or beside a tie between two codes
    check_quotients(m, torch.randint(-250, 251, (300, K), generator=g, device="cuda").to(xt))
    check_quotients(m, (torch.randint(-15, 16, (300, K), generator=g, device="cuda") / 16).to(xt))


@pytest.mark.parametrize("K", [512, 509])
@pytest.mark.parametrize("e", [-149, -140, -130, -126, -120, -117, -105, -100, -60, 60, 100, 118, 119])
def test_quant_codes_are_quotients_at_the_ends(m, K, e):  # noqa: F811
    """Scales from where they are held at 2^-126 to the largest; ties lie at whole numbers under those."""
    g = gen(e + 200)
    x = torch.randint(-448, 449, (200, K), generator=g, device="cuda").double() * torch.randint(1, 8, (200, 1), generator=g, device="cuda")
    check_quotients(m, (x * 2.0 ** e / 8).clamp(-3.4e38, 3.4e38).float())


# ---- append onto scales of the caller's own making ---------------------------------


@pytest.mark.parametrize("hkv,D,block", [(2, 64, 16), (1, 128, 64), (3, 80, 5)])
@pytest.mark.parametrize("T", [1, 9, 3000])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_append_onto_scales_of_either_sign(m, hkv, D, block, T, xt):  # noqa: F811
    """Tokens in the middle of blocks under scales of both signs, powers of two and others, large enough and too small: a
    scale that is large enough stays, and whatever a block held keeps its value."""
    g = gen(T + D)
    page, n_pages = 4 * block, T // 4 + 2
    nb = n_pages * 4
    x = (3 * randn(g, T, 1 * hkv + 2 * hkv, D)).to(xt)
    # one to three tokens a block, behind its first entry
    home = torch.randperm(nb, generator=g, device="cuda").tolist()
    slots, i = [], 0
    while len(slots) < T:
        n = min(1 + i % 3, T - len(slots), block - 1)
        slots += [home[i] * block + 1 + i % (block - n) + j for j in range(n)]
        i += 1
    slots = torch.tensor(slots, device="cuda")
    wrote = torch.zeros(nb * block, dtype=torch.bool, device="cuda")
    wrote[slots] = True
    touched = torch.zeros(nb, dtype=torch.bool, device="cuda")
    touched[slots // block] = True
    top = torch.zeros(2, nb, hkv, device="cuda")
    for side in range(2):
        v = x[:, hkv * (1 + side):hkv * (2 + side)].float().abs().amax(2)
        top[side].scatter_reduce_(0, (slots // block)[:, None].expand(-1, hkv), v, "amax")
    for power in (True, False):
        codes = [(100 * randn(g, n_pages, page, hkv, D)).clamp(-448, 448).to(E4M3) for _ in range(2)]
        e = torch.randint(-9, 3, (2, n_pages, 4, hkv), generator=g, device="cuda").float()
        scales = torch.exp2(e) * (1 if power else 0.3) * (torch.randint(0, 2, e.shape, generator=g, device="cuda") * 2 - 1)
        old_codes, old = [c.clone() for c in codes], scales.clone()
        kv = m.KvCache(codes[0], codes[1], q_heads=hkv, max_batch=1, k_scale=scales[0], v_scale=scales[1])
        m.moe_kv_append(kv, x[:, :hkv], x[:, hkv:2 * hkv], x[:, 2 * hkv:], None, slots, None, torch.empty(T, hkv, D, dtype=xt, device="cuda"))
        assert kv.status() == 0
        for side in range(2):
            s0, s1 = old[side].view(nb, hkv), scales[side].view(nb, hkv)
            keeps = (448 * s0.double().abs() >= top[side].double()) | ~touched[:, None]
            assert torch.equal(s1[keeps], s0[keeps])
            new = s1[~keeps].double()
            assert (new > 0).all() and (448 * new >= top[side][~keeps]).all() and (224 * new < top[side][~keeps]).all()
            assert (torch.frexp(new)[0] == 0.5).all()
            per = s1.double().repeat_interleave(block, 0)[..., None]
            got = codes[side].double().view(-1, hkv, D) * per
            was = old_codes[side].double().view(-1, hkv, D) * s0.double().repeat_interleave(block, 0)[..., None]
            # half a step of a subnormal code; under scales that are no powers of two half a step of every code
            slack = per.abs() * 2.0 ** -10 + (0 if power else was.abs() * 2.0 ** -4 * 1.000001)
            grown = ~keeps.repeat_interleave(block, 0)[..., None]
            err = (got - was).abs()
            assert (err <= torch.where(grown, slack, torch.zeros_like(slack)))[~wrote].all()
            want = x[:, hkv * (1 + side):hkv * (2 + side)].double()
            assert ((got[slots] - want).abs() <= want.abs() * 2.0 ** -4 * 1.000001 + per[slots].abs() * 2.0 ** -10 * 1.000001).all()


# ---- attention under large scales ------------------------------------------------


@pytest.mark.parametrize("hq,D", [(4, 64), (32, 128), (2, 256)])
@pytest.mark.parametrize("lens", [[20000] * 32, [4000], [1, 17, 5000, 900]])
@pytest.mark.parametrize("e", [-126, 96])
def test_attend_long_under_scales_at_the_ends(m, hq, D, lens, e):  # noqa: F811
    """Values' scales at both ends of their range, and values of one sign at the end of theirs, under long sequences in
    which runs of tokens, the first among them, score a few units less than the rest, so that weights are counted from
    a reference below their maximum."""
    g = gen(D + e)
    page, block = 16, 8
    per = -(-max(lens) // page)
    n_pages = len(lens) * per
    pages = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).view(len(lens), per)
    k, ks = block_cache(g, n_pages, page, block, 2, D, 0.02)
    v = torch.randint(320, 449, (n_pages, page, 2, D), generator=g, device="cuda").float().to(E4M3)
    vs = torch.full_like(ks, 2.0 ** e)
    q = torch.ones(len(lens), hq, D, device="cuda").to(BF16)
    scale = 0.5
    far = pages[:, torch.arange(per, device="cuda") // 8 % 8 == 0].reshape(-1).long()  # 128 tokens of 1024
    k[far] = torch.full_like(k[far].float(), -1.0).to(E4M3)
    ks[far] = 5.0 / (D * scale)  # scores of -5
    kv = m.KvCache(k, v, q_heads=hq, max_batch=len(lens), k_scale=ks, v_scale=vs)
    o, lse = torch.empty_like(q), torch.empty(len(lens), hq, device="cuda")
    m.moe_kv_attend(kv, q, pages, torch.tensor(lens, dtype=torch.int32, device="cuda"), o, scale=scale, lse=lse)
    o64, l64, ot, lt = attend64(q, k, v, ks, vs, pages, lens, scale, 0)
    assert o64.abs().max() < 2.0 ** (e + 9)
    within(o, o64, ot + 2.0 ** (e - 133))
    within(lse, l64, lt)


# ---- tokens of a block that do not follow one another --------------------------------


def calls_that_come_apart(page, block, filler):
    """Slots of calls in which one block's tokens, in the first page, are not in one run, and the same without those."""
    def runs(at, *counts):  # consecutive tokens, each lot from a block's beginning on
        for k in counts:
            yield list(range(at, at + k))
            at += -(-k // block) * block

    n = block // 2
    for between in (0, 1, filler):
        for first, second in ((range(n), range(n, block)),  # begun, left and gone on with
                              (range(n, block), range(n)),  # the other way about
                              ([1], range(2, block))):      # both behind the first entry
            head, middle, tail = runs(page, 3, between, filler)
            middle = middle or [-1]
            yield head + [*first] + middle + [*second] + tail, head + [-1] * len(first) + middle + [-1] * len(second) + tail


@pytest.mark.parametrize("xt,hq,hkv,D,rot", [(BF16, 4, 2, 64, 64), (F16, 2, 1, 128, 64), (F32, 4, 2, 64, 64), (BF16, 5, 1, 48, 18),
                                             (BF16, 16, 8, 128, 128)])
@pytest.mark.parametrize("page,block", [(16, 4), (64, 32), (12, 6), (256, 128)])
@pytest.mark.parametrize("filler", [2, 31, 5000])
def test_append_tells_of_tokens_that_come_apart(m, xt, hq, hkv, D, rot, page, block, filler):  # noqa: F811
    """The status is set, and blocks whose tokens follow one another are as in the call without the others."""
    g = gen(D + block + filler)
    n_pages = 5 + 2 * filler // page
    k, ks = block_cache(g, n_pages, page, block, hkv, D, 0.01)
    v, vs = block_cache(g, n_pages, page, block, hkv, D, 0.01)
    cs = table(60, rot)
    for slots, kept in calls_that_come_apart(page, block, filler):
        T = len(slots)
        x = (2 * randn(g, T, hq + 2 * hkv, D)).to(xt)
        pos = torch.randint(0, 60, (T,), generator=g, device="cuda", dtype=torch.int32)
        seen = []
        for s, status in ((slots, m.MOE_ERR_BAD_INDEX), (kept, 0)):
            c = [t.clone() for t in (k, v, ks, vs)]
            kv = m.KvCache(c[0], c[1], q_heads=hq, max_batch=1, k_scale=c[2], v_scale=c[3])
            qo = torch.full((T, hq, D), 7.0, device="cuda").to(xt)
            m.moe_kv_append(kv, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, torch.tensor(s, device="cuda"), cs, qo)
            assert kv.status() == status, (slots[:8], T)
            seen.append([t.view(torch.uint8)[1:] for t in c] + [qo.view(torch.uint8)])
        assert all(torch.equal(p, q) for p, q in zip(*seen))
        assert not torch.equal(seen[0][0], k.view(torch.uint8)[1:])


# ---- kernels for many tokens, and blocks that a team cannot hold at once -----------------


def check_many(m, g, xt, hkv, D, page, block, rot, il, axes, runs, n_axes=3):  # noqa: F811
    hq = hkv
    slots = run_slots(g, page, runs)
    T = len(slots)
    assert T * 2 * hkv > 16384  # else they are few
    n_pages = max(slots) // page + 2
    x = randn(g, T, hq + 2 * hkv, D).to(xt)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    slots = torch.tensor(slots, device="cuda")
    cs = table(90, rot)
    pos = torch.randint(0, 90, (n_axes, T), generator=g, device="cuda", dtype=torch.int32)
    pair = AXES[axes](rot // 2, n_axes) if axes else [0] * (rot // 2)
    cos, sin = rows64(cs, pos, pair)
    q64, qsz = turn64(q, cos, sin, il)
    k64, ksz = turn64(k, cos, sin, il)
    for size in (1e-4, 30.0):  # scales that are too small for the tokens, and such that are large enough
        kc, ks = block_cache(g, n_pages, page, block, hkv, D, size)
        vc, vs = block_cache(g, n_pages, page, block, hkv, D, size)
        k0, v0, ks0, vs0 = kc.clone(), vc.clone(), ks.clone(), vs.clone()
        kv = m.KvCache(kc, vc, q_heads=hq, max_batch=1, k_scale=ks, v_scale=vs)
        qo = torch.empty(T, hq, D, dtype=xt, device="cuda")
        m.moe_kv_append(kv, q, k, v, pos if axes else pos[0], slots, cs, qo, interleaved=il, axes=pair if axes else None)
        assert kv.status() == 0
        within(qo, q64, q64.abs() * U[xt] + qsz * 2.0 ** -23 + SUB[xt], "q")
        for codes, scales, c0, s0, x64, sz in ((kc, ks, k0, ks0, k64, ksz), (vc, vs, v0, vs0, v.double(), torch.zeros_like(ksz))):
            want, sc, wrote = put64(c0, s0, slots, x64, block, [True] * T)
            assert torch.equal(scales.double(), sc)
            per = sc.view(-1, hkv).repeat_interleave(block, 0)
            slack = torch.zeros(n_pages * page, hkv, D, dtype=torch.float64, device="cuda")
            slack[slots] = sz * 2.0 ** -22
            within(codes.float().view(-1, hkv, D), want.view(-1, hkv, D), e4m3_tol(want.view(-1, hkv, D)) + slack / per[..., None], "codes")
            same = (sc == s0.double()).view(-1, 1, hkv, 1).expand(-1, block, -1, D).reshape(-1, hkv, D) & ~wrote[:, None, None]
            assert torch.equal(codes.view(torch.uint8).view(-1, hkv, D)[same], c0.view(torch.uint8).view(-1, hkv, D)[same])


@pytest.mark.parametrize("xt", [BF16, F16, F32])
@pytest.mark.parametrize("axes,il", [(None, True), ("turns", False), ("turns", True), ("fours", True), ("sections", False)])
@pytest.mark.parametrize("block", [1, 8, 64])
def test_many_tokens_of_every_kind(m, xt, il, block, axes):  # noqa: F811
    check_many(m, gen(block), xt, 8, 32, 64, block, 32, il, axes, [(0, 700), (13, 400), (63, 2), (5, 100)])


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("D,rot,page,block", [(128, 128, 128, 128), (256, 128, 64, 64), (256, 256, 32, 32), (64, 64, 1024, 1024), (128, 64, 512, 256),
                                              (48, 18, 64, 64), (80, 40, 200, 100)])
def test_blocks_longer_than_a_team_holds(m, xt, D, rot, page, block):  # noqa: F811
    """Read twice, with other runs before and behind them."""
    check_many(m, gen(D + block), xt, 8, D, page, block, rot, False, None, [(0, 600), (7, 500), (page // 2, 3)])
    check_many(m, gen(D + block), xt, 8, D, page, block, rot, True, "turns", [(page - 1, 1100), (0, 5)])


# ---- what the quantiser and the product share with others ------------------------------


def test_quant_of_the_norms_rows(m):  # noqa: F811
    """The norm's own E4M3 rows and the quantiser's of the norm's fp32 rows: one group a row, so the scales are those of
    the same numbers, a few roundings of fp32 apart, and either's codes are within half a step of them."""
    g = gen(3)
    x, w = (3 * randn(g, 500, 128)).to(BF16), randn(g, 128).to(BF16)
    y32, y8, s8 = torch.empty(500, 128, device="cuda"), torch.empty(500, 128, dtype=E4M3, device="cuda"), torch.empty(500, device="cuda")
    m.moe_add_rms_norm(x, w, y32)
    m.moe_add_rms_norm(x, w, y8, scale=s8)
    q, s = torch.empty(500, 128, dtype=E4M3, device="cuda"), torch.empty(500, 1, device="cuda")
    m.moe_quant_e4m3(y32, q, s)
    within(s[:, 0], s8.double(), s8.double() * 2.0 ** -22, "scale")  # a rounding each on the way to the maximum and to the scale
    for codes, scale in ((y8, s8[:, None]), (q, s)):
        want = y32.double() / scale.double()
        within(codes.float(), want, e4m3_tol(want) + want.abs() * 2.0 ** -22, "codes")


@pytest.mark.parametrize("T,N,K", [(1, 256, 512), (30, 300, 1024), (100, 256, 2048), (300, 512, 512), (1000, 1024, 512)])
def test_a_products_row_does_not_depend_on_its_neighbours(m, T, N, K):  # noqa: F811
    g = gen(T)
    x, w, xs, ws = operands(g, T, N, K)
    keep = torch.arange(0, T, 7, device="cuda")
    y, z = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
    m.moe_linear_blocks(x, w, y, xs, ws)
    x2, _, xs2, _ = operands(g, T, N, K)
    x2.view(torch.uint8)[keep] = x.view(torch.uint8)[keep]
    xs2[keep] = xs[keep]
    m.moe_linear_blocks(x2, w, z, xs2, ws)
    assert torch.equal(y[keep], z[keep]) and (T == 1 or not torch.equal(y, z))
