"""The decoder-layer operators against plain 64-bit forms of the same formulas.

Bounds come from the arithmetic, not from runs: U is the unit roundoff of an output
type (2^-p for a significand of p bits, the hidden one among them: 8, 11 and 24), sums and
factors are fp32 (2^-24 a step), and each test states the rest."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
# below the smallest normal the spacing is absolute
SUB = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}


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
    """Half the spacing of E4M3 at v (2^-4 relative, 2^-10 below the smallest normal),
    widened by the fp32 arithmetic before the rounding."""
    return v.abs() * (2.0 ** -4 + 1e-5) + 2.0 ** -10 * (1 + 1e-5)


# ---- norm ---------------------------------------------------------------------


def norm64(x, r, w, eps):
    s = x.double() + (0 if r is None else r.double())
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return s, y if w is None else y * w.double()


# fp32 sum of squares: at most 32 + 5 + 32 steps of 2^-24 in a row, halved by the square
# root, and a handful of roundings after it
NORM_REL = 4e-6


@pytest.mark.parametrize("T,H", [(1, 1), (1, 64), (3, 7), (2, 255), (5, 256), (1, 4096), (33, 1000), (7, 5003), (130, 96),
                                 (3, 8192), (2, 8200), (2, 8193), (1, 32768), (1, 32767), (2, 16384)])
@pytest.mark.parametrize("xt,rt,yt", [(BF16, BF16, BF16), (F16, F32, F16), (F32, F32, F32), (BF16, F32, E4M3),
                                      (F32, BF16, BF16), (F16, F16, E4M3)])
def test_norm(m, T, H, xt, rt, yt):
    g = gen(T * 7919 + H)
    x, r = randn(g, T, H).to(xt), (3 * randn(g, T, H)).to(rt)
    w = (1 + 0.2 * randn(g, H)).to(xt)
    y, so = torch.empty(T, H, dtype=yt, device="cuda"), torch.empty(T, H, dtype=rt, device="cuda")
    sc = torch.empty(T, device="cuda") if yt == E4M3 else None
    m.moe_add_rms_norm(x, w, y, residual=r, sum_out=so, scale=sc, eps=1e-5)
    s64, y64 = norm64(x, r, w, 1e-5)
    within(so, s64, s64.abs() * (U[rt] + U[F32]) + SUB[rt], "sum")
    if yt == E4M3:
        s = (y64.abs().amax(1) / 448).clamp(min=2.0 ** -126)
        within(sc, s, s * 2 * NORM_REL, "scale")
        within(y.float(), y64 / s[:, None], e4m3_tol(y64 / s[:, None]), "y8")
    else:
        within(y, y64, y64.abs() * (U[yt] + NORM_REL) + SUB[yt], "y")


def test_norm_without_parts_in_place_and_strided(m):
    g = gen(5)
    wide = randn(g, 9, 700).to(BF16)
    x = wide[:, 100:612]  # rows 700 apart, 8-byte aligned
    y = torch.empty(9, 512, dtype=BF16, device="cuda")
    m.moe_add_rms_norm(x, None, y)
    within(y, norm64(x, None, None, 1e-6)[1], norm64(x, None, None, 1e-6)[1].abs() * (U[BF16] + NORM_REL))
    # residual stream updated in place, y over x
    x, r = randn(g, 6, 1024).to(BF16), randn(g, 6, 1024).to(BF16)
    s64, y64 = norm64(x, r, None, 0.0)
    m.moe_add_rms_norm(x, None, x, residual=r, sum_out=r, eps=0.0)
    within(r, s64, s64.abs() * (U[BF16] + U[F32]))
    within(x, y64, y64.abs() * (U[BF16] + NORM_REL))
    # one row broadcast to every output row
    one = randn(g, 1, 512).to(F16)
    y = torch.empty(4, 512, dtype=F16, device="cuda")
    m.moe_add_rms_norm(one.expand(4, 512), None, y)
    assert all(torch.equal(y[0], y[i]) for i in range(4))


def test_norm_special_rows(m):
    """Zero rows, tiny rows, a NaN, an infinity: each stays in its row."""
    x = torch.ones(6, 256, device="cuda")
    x[1] = 0
    x[2] = 1e-30
    x[3, 5] = float("nan")
    x[4, 5] = float("inf")
    y = torch.empty(6, 256, device="cuda")
    m.moe_add_rms_norm(x, None, y, eps=1e-6)
    want = norm64(x, None, None, 1e-6)[1]
    for i in (0, 1, 2, 5):
        within(y[i], want[i], want[i].abs() * 1e-5)
    assert y[3].isnan().all() and y[4, 5].isnan() and (y[4].nan_to_num() == 0).all()
    y8, sc = torch.empty(6, 256, dtype=E4M3, device="cuda"), torch.empty(6, device="cuda")
    m.moe_add_rms_norm(x, None, y8, scale=sc, eps=1e-6)
    assert sc[1] == 2.0 ** -126 and (y8[1].float() == 0).all()
    assert sc[3].isnan() and sc[4].isnan() and sc[[0, 2, 5]].isfinite().all()
    within(y8[2].float(), torch.full((256,), 448.0, device="cuda"), 0.0)


def test_norm_of_no_rows_and_refusals(m):
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    m.moe_add_rms_norm(e, None, e.clone())
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    for kw in (dict(y=torch.empty(4, 32, dtype=BF16, device="cuda")), dict(weight=x[0, :32]),
               dict(residual=x[:2]), dict(scale=torch.empty(4, device="cuda")),
               dict(y=torch.empty(4, 64, dtype=E4M3, device="cuda")), dict(y=x.t().contiguous().t()),
               dict(residual=x.float(), sum_out=x.clone()), dict(weight=x[0].cpu())):
        a = dict(x=x, weight=None, y=torch.empty_like(x))
        a.update(kw)
        with pytest.raises(m.MoeError) as err:
            m.moe_add_rms_norm(**a)
        assert err.value.code == m.MOE_ERR_INVALID_ARG


# ---- append -------------------------------------------------------------------


def table(n, rot):
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(1, rot))
    return torch.cat([a.cos(), a.sin()], 1).float()


def turn64(x, cs, rot, interleaved):
    x = x.double().clone()
    cs = cs.double()[:, None, :]
    c, s = cs[..., : rot // 2], cs[..., rot // 2:]
    ia = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    ib = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = x[..., ia].clone(), x[..., ib].clone()
    x[..., ia], x[..., ib] = a * c - b * s, a * s + b * c
    size = torch.zeros_like(x)
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return x, size


@pytest.mark.parametrize("T,hq,hkv,D,page,rot,il", [
    (1, 32, 8, 128, 16, 128, False), (5, 4, 4, 64, 7, 64, True), (19, 6, 2, 80, 1, 40, False),
    (3, 1, 1, 16, 5, 2, False), (3, 1, 1, 16, 5, 2, True), (130, 8, 1, 256, 64, 128, False), (9, 3, 3, 96, 32, 0, False),
    (17, 5, 1, 48, 16, 18, True), (40, 12, 4, 256, 128, 256, True), (2, 64, 64, 128, 16, 128, False)])
@pytest.mark.parametrize("xt,ct", [(BF16, BF16), (F16, F16), (BF16, E4M3), (F32, E4M3), (F32, BF16)])
def test_append(m, T, hq, hkv, D, page, rot, il, xt, ct):
    g = gen(T * 31 + D)
    qkv = randn(g, T, hq + 2 * hkv, D).to(xt)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    n_pages = -(-T // page) + 2
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:T].contiguous()
    if T > 2:
        slots[1] = -1
    pos = torch.randint(0, 50, (T,), generator=g, device="cuda", dtype=torch.int32)
    cs = table(50, rot) if rot else None
    kc, vc = randn(g, n_pages, page, hkv, D).to(ct), randn(g, n_pages, page, hkv, D).to(ct)
    ks = vs = None
    if ct == E4M3:
        ks, vs = 0.004 + 0.01 * torch.rand(hkv, generator=g, device="cuda"), 0.01 + torch.rand(hkv, generator=g, device="cuda")
    k0, v0 = kc.clone(), vc.clone()
    qo = torch.empty(T, hq, D, dtype=xt, device="cuda")
    kv = m.KvCache(kc, vc, q_heads=hq, max_batch=1, k_scale=ks, v_scale=vs)
    m.moe_kv_append(kv, q, k, v, pos, slots, cs, qo, interleaved=il)
    assert kv.status() == 0
    rows = cs[pos.long()] if rot else torch.zeros(T, 0, device="cuda")
    q64, qsz = turn64(q, rows, rot, il)
    k64, ksz = turn64(k, rows, rot, il)
    # two products and a sum in fp32, then one rounding
    within(qo, q64, q64.abs() * U[xt] + qsz * 2.0 ** -23 + SUB[xt], "q")
    keep = slots >= 0
    flat = lambda c: c.view(n_pages * page, hkv, D)  # noqa: E731
    gk, gv = flat(kc)[slots[keep]], flat(vc)[slots[keep]]
    k64, ksz, v64 = k64[keep], ksz[keep], v[keep].double()
    if ct == E4M3:
        k64 = (k64 / ks.double()[:, None]).clamp(-448, 448)
        v64 = (v64 / vs.double()[:, None]).clamp(-448, 448)
        within(gk.float(), k64, e4m3_tol(k64) + ksz / ks[:, None] * 2.0 ** -22, "k")
        within(gv.float(), v64, e4m3_tol(v64), "v")
    else:
        within(gk, k64, k64.abs() * U[ct] + ksz * 2.0 ** -23 + SUB[ct], "k")
        assert torch.equal(gv, v[keep].to(ct))
    # nothing but the slots of the call was written
    rest = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    rest[slots[keep]] = False
    bits = torch.uint8 if ct == E4M3 else torch.int16
    assert torch.equal(flat(kc)[rest].view(bits), flat(k0)[rest].view(bits))
    assert torch.equal(flat(vc)[rest].view(bits), flat(v0)[rest].view(bits))


def test_append_layouts_in_place_and_unaligned(m):
    """Heads before tokens in a page, q rotated in place, and rows at odd addresses."""
    g = gen(3)
    T, hq, hkv, D, page = 11, 4, 2, 64, 8
    k_hnd = torch.zeros(4, hkv, page, D, dtype=F16, device="cuda")
    v_hnd = torch.zeros_like(k_hnd)
    kv = m.KvCache(k_hnd.transpose(1, 2), v_hnd.transpose(1, 2), q_heads=hq, max_batch=1)
    raw = randn(g, T * (hq + 2 * hkv) * D + 1).to(F16)[1:].view(T, hq + 2 * hkv, D)  # 2-byte aligned
    q, k, v = raw[:, :hq], raw[:, hq:hq + hkv], raw[:, hq + hkv:]
    cs, pos = table(64, D), torch.arange(T, device="cuda", dtype=torch.int32) + 7
    slots = torch.arange(T, device="cuda") + 5
    q64, qsz = turn64(q, cs[pos.long()], D, False)
    k64, ksz = turn64(k, cs[pos.long()], D, False)
    m.moe_kv_append(kv, q, k, v, pos, slots, cs, q)
    within(q, q64, q64.abs() * U[F16] + qsz * 2.0 ** -23 + SUB[F16])
    got = k_hnd.transpose(1, 2)[slots // page, slots % page]
    within(got, k64, k64.abs() * U[F16] + ksz * 2.0 ** -23 + SUB[F16])
    assert torch.equal(v_hnd.transpose(1, 2)[slots // page, slots % page], v)


def test_append_reports_what_is_out_of_range(m):
    g = gen(4)
    kc, vc = torch.zeros(2, 4, 1, 16, dtype=BF16, device="cuda"), torch.zeros(2, 4, 1, 16, dtype=BF16, device="cuda")
    kv = m.KvCache(kc, vc, q_heads=1, max_batch=1)
    q = randn(g, 3, 1, 16).to(BF16)
    cs = table(8, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    for pos, slots in ((torch.tensor([1, 2, 3], **i32), torch.tensor([0, 8, 2], device="cuda")),
                       (torch.tensor([1, 8, 3], **i32), torch.tensor([0, 1, 2], device="cuda")),
                       (torch.tensor([1, -1, 3], **i32), torch.tensor([0, 1, 2], device="cuda"))):
        kc.zero_(), vc.zero_()
        m.moe_kv_append(kv, q, q, q, pos, slots, cs, torch.empty_like(q))
        assert kv.status() == m.MOE_ERR_BAD_INDEX
        kv.clear_status()
        assert kv.status() == 0
        written = vc.view(8, 16).abs().sum(1) > 0
        assert written.tolist() == [True, False, True] + [False] * 5
    with pytest.raises(m.MoeError):  # odd rotation
        m.moe_kv_append(kv, q, q, q, torch.zeros(3, **i32), torch.zeros(3, dtype=torch.int64, device="cuda"),
                        torch.zeros(8, 15, device="cuda"), torch.empty_like(q))
    with pytest.raises(m.MoeError):  # slots of the wrong width
        m.moe_kv_append(kv, q, q, q, torch.zeros(3, **i32), torch.zeros(3, **i32), cs, torch.empty_like(q))
    with pytest.raises(m.MoeError):  # another type
        m.moe_kv_append(kv, q, q.float(), q, torch.zeros(3, **i32), torch.zeros(3, dtype=torch.int64, device="cuda"),
                        cs, torch.empty_like(q))


# ---- attend -------------------------------------------------------------------


def make_cache(g, lens, page, hkv, D, ct, per=None, spare=2, hnd=False):
    need = [-(-n // page) for n in lens]
    per = max(need + [1]) if per is None else per
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    pages = torch.full((len(lens), per), -7, dtype=torch.int32, device="cuda")  # never to be read
    at = 0
    for b, n in enumerate(need):
        pages[b, :n] = order[at:at + n]
        at += n
    ks = vs = None
    k, v = randn(g, n_pages, page, hkv, D), randn(g, n_pages, page, hkv, D)
    if ct == E4M3:
        ks, vs = 0.005 + 0.01 * torch.rand(hkv, generator=g, device="cuda"), 0.005 + 0.01 * torch.rand(hkv, generator=g, device="cuda")
        k, v = (k / ks[:, None]).clamp(-448, 448), (v / vs[:, None]).clamp(-448, 448)
    k, v = k.to(ct), v.to(ct)
    if hnd:
        k = k.transpose(1, 2).contiguous().transpose(1, 2)
        v = v.transpose(1, 2).contiguous().transpose(1, 2)
    return k, v, ks, vs, pages


def attend64(q, k, v, ks, vs, pages, lens, scale, window):
    """Per sequence: output, log-sum, and the bounds of both.

    A score is a sum of D products in fp32 (D + 2 steps of 2^-24 of sum |q||k|); a weight
    is rounded once to 16 bits (U of bf16 for a bf16 cache, of f16 else) with an
    exponential good to 2^-21 and the score's error on top; the weighted sum adds at most
    one fp32 step for every 16 tokens."""
    page, hkv, D = k.shape[1], k.shape[2], k.shape[3]
    g = q.shape[1] // hkv
    outs, lses, otol, ltol = [], [], [], []
    uw = U[BF16] if k.dtype == BF16 else U[F16]
    for b, n in enumerate(lens):
        t = torch.arange(max(0, n - window) if window else 0, n, device="cuda")
        if t.numel() == 0:
            z = torch.zeros(q.shape[1], D, dtype=torch.float64, device="cuda")
            outs.append(z), otol.append(z), ltol.append(z[:, 0]), lses.append(z[:, 0] - math.inf)
            continue
        p, e = pages[b].long()[t // page], t % page
        kk, vv = k[p, e].double(), v[p, e].double()
        if ks is not None:
            kk, vv = kk * ks.double()[:, None], vv * vs.double()[:, None]
        qq = q[b].double().view(hkv, g, D)
        s = torch.einsum("hgd,thd->hgt", qq, kk) * scale
        es = torch.einsum("hgd,thd->hgt", qq.abs(), kk.abs()).amax(-1) * abs(scale) * (D + 2) * 2.0 ** -24
        lse = torch.logsumexp(s, -1)
        w = torch.exp(s - lse[..., None])
        o = torch.einsum("hgt,thd->hgd", w, vv)
        size = torch.einsum("hgt,thd->hgd", w, vv.abs())
        rel = uw + 2.0 ** -21 + 2 * es + (len(t) / 16 + 8) * 2.0 ** -24
        outs.append(o.reshape(-1, D)), lses.append(lse.reshape(-1))
        otol.append((size * rel[..., None] * 1.01 + o.abs() * U[q.dtype] * 1.01 + SUB[q.dtype]).reshape(-1, D))
        ltol.append((es + 2.0 ** -21 + (len(t) / 16 + 8) * 2.0 ** -24 + lse.abs() * 2.0 ** -22).reshape(-1))
    return torch.stack(outs), torch.stack(lses), torch.stack(otol), torch.stack(ltol)


def check_attend(m, g, lens, hq, hkv, D, page, qt, ct, window=0, scale=None, hnd=False, gain=1.0):
    k, v, ks, vs, pages = make_cache(g, lens, page, hkv, D, ct, hnd=hnd)
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


@pytest.mark.parametrize("hq,hkv,D", [(1, 1, 16), (4, 4, 64), (32, 8, 128), (7, 1, 96), (16, 1, 128), (24, 2, 80),
                                      (6, 2, 256), (40, 1, 64), (3, 1, 192), (64, 1, 112), (128, 2, 128)])
@pytest.mark.parametrize("qt,ct", [(BF16, BF16), (F16, F16), (BF16, E4M3), (F16, E4M3)])
def test_attend_heads(m, hq, hkv, D, qt, ct):
    check_attend(m, gen(hq * 100 + D), [0, 1, 2, 15, 16, 17, 63, 64, 65, 300], hq, hkv, D, 16, qt, ct)


@pytest.mark.parametrize("page", [1, 3, 7, 16, 33, 64, 128, 1000])
@pytest.mark.parametrize("window", [0, 1, 5, 16, 100])
def test_attend_pages_and_windows(m, page, window):
    check_attend(m, gen(page), [0, 1, 99, 100, 101, 250, 17], 8, 2, 64, page, BF16, BF16, window=window)
    check_attend(m, gen(page + 1), [33, 0, 40], 4, 4, 96, page, F16, E4M3, window=window, hnd=True)


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [5000], [1, 40000], [20000, 0, 3], list(range(0, 700, 3)),
                                  [700] * 40, [1] * 500])
@pytest.mark.parametrize("ct", [BF16, E4M3])
def test_attend_batches(m, lens, ct):
    check_attend(m, gen(len(lens)), lens, 8, 2, 128, 16, BF16, ct)


@pytest.mark.parametrize("lens", [[320], [321], [319, 0, 1, 320], [640, 641, 639], [0, 17, 0, 0, 300], [320] * 76, [16] * 128,
                                  [16] * 129])
@pytest.mark.parametrize("hq,hkv,D,ct", [(8, 2, 128, BF16), (32, 2, 64, E4M3), (3, 1, 256, F16)])
def test_attend_short_sequences(m, lens, hq, hkv, D, ct):
    """Lengths about the most that one block takes whole, and batches about the most it does so for."""
    check_attend(m, gen(len(lens) + D), lens, hq, hkv, D, 16, F16 if ct == F16 else BF16, ct)


def test_attend_sharp_and_flat_scores(m):
    """Scores far apart (one key takes all), negative scale, and scale zero (a mean)."""
    check_attend(m, gen(1), [300, 50], 8, 2, 64, 16, BF16, BF16, scale=8.0, gain=4.0)
    check_attend(m, gen(2), [300, 50], 8, 2, 64, 16, F16, F16, scale=-1.0)
    check_attend(m, gen(3), [300, 50], 8, 2, 64, 16, BF16, E4M3, scale=0.0)
    check_attend(m, gen(4), [300, 50], 8, 2, 64, 16, BF16, E4M3, gain=1e4)


def test_attend_ignores_what_is_not_attended(m):
    """Infinities and NaN behind a sequence's end, before its window and in pages of no
    sequence leave every result as it was."""
    g = gen(9)
    lens, page = [37, 5, 100], 16
    k, v, _, _, pages = make_cache(g, lens, page, 2, 64, BF16)
    q = randn(g, 3, 8, 64).to(BF16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kv = m.KvCache(k, v, q_heads=8, max_batch=3)
    clean = torch.empty_like(q)
    m.moe_kv_attend(kv, q, pages, n, clean, window=30)
    seen = torch.zeros(k.shape[0], page, dtype=torch.bool, device="cuda")
    for b, x in enumerate(lens):
        t = torch.arange(max(0, x - 30), x, device="cuda")
        seen[pages[b].long()[t // page], t % page] = True
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(BF16).min):
        k[~seen], v[~seen] = bad, bad
        got = torch.empty_like(q)
        m.moe_kv_attend(kv, q, pages, n, got, window=30)
        assert torch.equal(got, clean)


def test_attend_strided_rows_shared_table_and_other_stream(m):
    g = gen(11)
    k, v, _, _, pages = make_cache(g, [200], 16, 2, 64, F16)
    big = randn(g, 5, 12, 64).to(F16)
    q = big[:, 2:10]  # rows of a wider tensor
    lens = [200, 1, 0, 77, 150]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.zeros(5, 10, 64, dtype=F16, device="cuda")
    kv = m.KvCache(k, v, q_heads=8, max_batch=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    # the verification of several tokens of one sequence: one table row, lengths of their own
    m.moe_kv_attend(kv, q, pages.expand(5, -1), n, out[:, 1:9], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    o64, _, ot, _ = attend64(q, k, v, None, None, pages.expand(5, -1), lens, 64 ** -0.5, 0)
    within(out[:, 1:9], o64, ot)
    assert (out[:, 0] == 0).all() and (out[:, 9] == 0).all()


def test_attend_far_offsets(m):
    """A cache whose later pages lie past 2^32 bytes and 2^31 elements."""
    n_pages, page, hkv, D = 40, 64, 8, 128
    stride = (5 << 30) // 2 // n_pages // 8 * 8 * 2  # elements between pages: about 10 GB in all
    room = torch.empty(n_pages * stride, dtype=BF16, device="cuda")
    k = room.as_strided((n_pages, page, hkv, D), (stride, hkv * D, D, 1))
    g = gen(12)
    k.copy_(randn(g, n_pages, page, hkv, D))
    lens = [n_pages * page - 5]
    pages = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)[None]
    q = randn(g, 1, 32, D).to(BF16)
    out, lse = torch.empty_like(q), torch.empty(1, 32, device="cuda")
    kv = m.KvCache(k, k, q_heads=32, max_batch=1)
    m.moe_kv_attend(kv, q, pages, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, lse=lse)
    o64, l64, ot, lt = attend64(q, k, k, None, None, pages, lens, D ** -0.5, 0)
    within(out, o64, ot)
    within(lse, l64, lt)
    # and the append writes there
    slots = torch.tensor([(n_pages - 1) * page + 3], device="cuda")
    x = randn(g, 1, 48, D).to(BF16)
    # k and v are the same memory here: both get the same values
    m.moe_kv_append(kv, x[:, :32], x[:, 40:], x[:, 40:], None, slots, None, torch.empty_like(q))
    assert torch.equal(k[n_pages - 1, 3], x[0, 40:])


def test_attend_reports_and_clamps(m):
    g = gen(13)
    k, v, _, _, pages = make_cache(g, [40, 30], 8, 1, 32, BF16)
    q = randn(g, 2, 2, 32).to(BF16)
    kv = m.KvCache(k, v, q_heads=2, max_batch=2)
    out = torch.empty_like(q)
    n = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    m.moe_kv_attend(kv, q, pages, n(40, -3), out)
    assert kv.status() == m.MOE_ERR_BAD_INDEX and (out[1] == 0).all()
    kv.clear_status()
    m.moe_kv_attend(kv, q, pages, n(1000, 1), out)  # longer than its row of the table: clamped
    assert kv.status() == m.MOE_ERR_BAD_INDEX
    o64, _, ot, _ = attend64(q, k, v, None, None, pages, [40, 1], 32 ** -0.5, 0)
    within(out, o64, ot)
    kv.clear_status()
    bad = pages.clone()
    bad[0, 2] = k.shape[0]  # tokens 16..23 are left out
    m.moe_kv_attend(kv, q, bad, n(40, 30), out)
    assert kv.status() == m.MOE_ERR_BAD_INDEX
    short = pages.clone()
    short[0, 2:4] = pages[0, 3:5]
    o64, _, ot, _ = attend64(q, k, v, None, None, short, [32, 30], 32 ** -0.5, 0)
    within(out, o64, ot)
    kv.clear_status()
    m.moe_kv_attend(kv, q, pages, n(40, 30), out)
    assert kv.status() == 0
    with pytest.raises(m.MoeError):
        m.moe_kv_attend(kv, q[:1].expand(3, 2, 32), pages[:1].expand(3, -1), n(1, 1, 1), torch.empty(3, 2, 32, dtype=BF16, device="cuda"))
    with pytest.raises(m.MoeError):
        m.moe_kv_attend(kv, q.half(), pages, n(1, 1), out.half())
    with pytest.raises(m.MoeError):
        m.moe_kv_attend(kv, q, pages, n(1, 1), out, scale=float("nan"))
    with pytest.raises(m.MoeError):
        m.moe_kv_attend(kv, q, pages.long(), n(1, 1), out)
    m.moe_kv_attend(kv, q[:0], pages[:0], n(), out[:0])


def test_attend_in_a_graph_with_growing_lengths(m):
    """One captured call serves later steps: lengths, table and cache are read on the GPU."""
    g = gen(14)
    lens = [90, 200, 3]
    k, v, _, _, pages = make_cache(g, [300, 300, 300], 16, 2, 128, BF16)
    q = randn(g, 3, 8, 128).to(BF16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kv = m.KvCache(k, v, q_heads=8, max_batch=3)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.moe_kv_attend(kv, q, pages, n, out)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            m.moe_kv_attend(kv, q, pages, n, out)
    torch.cuda.synchronize()
    for step in range(4):
        graph.replay()
        o64, _, ot, _ = attend64(q, k, v, None, None, pages, [x + 25 * step for x in lens], 128 ** -0.5, 0)
        within(out, o64, ot)
        n += 25


# ---- linear -------------------------------------------------------------------


def act64(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "silu":
        return y * torch.sigmoid(y)
    if act == "gelu":
        return y * torch.special.ndtr(y)
    return y


def check_linear(m, g, T, N, K, xt, yt, act="none", bias=None, res=False, ragged=False):
    x, w = randn(g, T, K), randn(g, N, K) / math.sqrt(K)
    xs = ws = None
    if xt == E4M3:
        xs, ws = x.abs().amax(1) / 448 + 1e-30, w.abs().amax(1) / 448 + 1e-30
        x, w = x / xs[:, None], w / ws[:, None]
    x, w = x.to(xt), w.to(xt)
    if ragged:  # rows further apart than they are long
        x = torch.cat([x.float(), randn(g, T, 32)], 1).to(xt)[:, :K]
        w = torch.cat([w.float(), randn(g, N, 16)], 1).to(xt)[:, :K]
    b = None if bias is None else (0.3 * randn(g, N)).to(bias)
    wide = torch.full((T, N + 3), float("nan"), dtype=yt, device="cuda")
    y = wide[:, :N] if ragged else torch.full((T, N), float("nan"), dtype=yt, device="cuda")
    r = randn(g, T, N).to(yt) if res else None
    m.moe_linear(x, w, y, bias=b, act=act, residual=r, x_scale=xs, w_scale=ws)
    x64, w64 = x.double(), w.double()
    if xs is not None:
        x64, w64 = x64 * xs.double()[:, None], w64 * ws.double()[:, None]
    y64, size = x64 @ w64.t(), x64.abs() @ w64.abs().t()
    # tensor cores add 16 products or more a step; each step may lose 2^-22 of the sum of
    # sizes; no activation is steeper than 1.13
    tol = size * (K / 16 + 4) * 2.0 ** -22
    if b is not None:
        y64 = y64 + b.double()
    tol = 1.13 * tol + y64.abs() * 2.0 ** -20 + 1e-6
    y64 = act64(y64, act)
    if res:
        y64 = y64 + r.double()
        tol = tol + y64.abs() * 2.0 ** -23
    within(y, y64, tol + y64.abs() * U[yt] + SUB[yt])
    if ragged:
        assert wide[:, N:].isnan().all()


@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 8, 64), (1, 4096, 4096), (2, 100, 208), (7, 384, 512), (16, 129, 256),
                                   (17, 1000, 1040), (32, 6144, 4096), (33, 65, 80), (64, 256, 4096), (65, 127, 144),
                                   (100, 4096, 64), (127, 640, 1024), (128, 128, 128), (129, 257, 272), (200, 72, 8192),
                                   (256, 512, 4096), (511, 1021, 528), (1000, 1536, 768), (2049, 640, 320),
                                   (3000, 2056, 192), (5001, 1023, 80), (2500, 4100, 1040), (8192, 640, 4096)])
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (F16, F32), (E4M3, BF16)])
def test_linear(m, T, N, K, xt, yt):
    check_linear(m, gen(T + N + K), T, N, K, xt, yt)


@pytest.mark.parametrize("T", [1, 5, 40, 130, 300, 10001])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("xt,yt,bias,res", [(BF16, BF16, BF16, True), (BF16, F32, F32, False), (F16, F16, F16, True),
                                            (E4M3, BF16, F32, True), (E4M3, F32, None, True), (F16, BF16, None, False)])
def test_linear_epilogue(m, T, act, xt, yt, bias, res):
    check_linear(m, gen(T), T, 333, 256, xt, yt, act, bias, res, ragged=True)


@pytest.mark.parametrize("K", [16, 64, 80, 128, 192, 1040])  # blocks of K in odd and even numbers, the last one short
@pytest.mark.parametrize("T,N", [(257, 1023), (300, 72), (513, 2050), (1000, 8100)])
@pytest.mark.parametrize("yt", [BF16, F16, F32])
def test_linear_tiles_end_inside_a_run(m, T, N, K, yt):
    """Aligned rows whose last run of outputs is cut short, with residual, in tiles of several widths."""
    g = gen(T + N + K)
    x, w = randn(g, T, K).to(BF16), (randn(g, N, K) / math.sqrt(K)).to(BF16)
    wide = torch.full((T, (N + 15) // 8 * 8), float("nan"), dtype=yt, device="cuda")
    y = wide[:, :N]
    r = randn(g, T, wide.shape[1]).to(yt)[:, :N]
    m.moe_linear(x, w, y, residual=r)
    sums, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    want = sums + r.double()
    tol = size * (K / 16 + 4) * 2.0 ** -22 + sums.abs() * 2.0 ** -20 + want.abs() * 2.0 ** -23 + 1e-6
    within(y, want, tol + want.abs() * U[yt] + SUB[yt])
    assert wide[:, N:].isnan().all()


def test_linear_residual_in_place_and_special_values(m):
    g = gen(21)
    x, w = randn(g, 70, 128).to(BF16), (randn(g, 200, 128) / 11).to(BF16)
    y = randn(g, 70, 200).to(BF16)
    y0 = y.clone()
    m.moe_linear(x, w, y, residual=y)
    want = x.double() @ w.double().t() + y0.double()
    within(y, want, want.abs() * U[BF16] + 2.0 ** -14)
    # a row with an infinity or a NaN spoils its own outputs alone
    clean = torch.empty(70, 200, dtype=F32, device="cuda")
    m.moe_linear(x, w, clean)
    x[3, 5], x[69, 0] = float("inf"), float("nan")
    got = torch.empty_like(clean)
    m.moe_linear(x, w, got)
    keep = torch.ones(70, dtype=torch.bool, device="cuda")
    keep[[3, 69]] = False
    assert torch.equal(got[keep], clean[keep]) and not got[3].isfinite().any() and got[69].isnan().all()
    # activations far out: no overflow of their exponentials
    far = torch.tensor([[1e4], [-1e4]], device="cuda").expand(2, 16).to(BF16).contiguous()
    one = torch.ones(8, 16, device="cuda").to(BF16)
    for act in ("silu", "gelu", "relu"):
        o = torch.empty(2, 8, device="cuda")
        m.moe_linear(far, one, o, act=act)
        within(o[0], torch.full((8,), float(far[0, 0]) * 16, device="cuda"), 1.0)
        assert (o[1] == 0).all()


def test_linear_same_bits_and_no_rows(m):
    g = gen(22)
    for T, K in ((1, 4096), (32, 4096), (300, 512)):
        x, w = randn(g, T, K).to(BF16), randn(g, 512, K).to(BF16)
        a = [torch.empty(T, 512, device="cuda") for _ in range(3)]
        for y in a:
            m.moe_linear(x, w, y)
        assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[2])
    m.moe_linear(x[:0], w, torch.empty(0, 512, device="cuda"))
    with pytest.raises(m.MoeError):
        m.moe_linear(x, w.half(), a[0])
    with pytest.raises(m.MoeError):
        m.moe_linear(x, w, a[0], act="tanh")
    with pytest.raises(m.MoeError):
        m.moe_linear(x, w, a[0], residual=a[0].half())
    with pytest.raises(m.MoeError):
        m.moe_linear(x, w, a[0], x_scale=torch.ones(300, device="cuda"))
    with pytest.raises(m.MoeError):
        m.moe_linear(x.to(E4M3), w.to(E4M3), a[0])
