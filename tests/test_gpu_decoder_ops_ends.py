"""The decoder-layer operators at the ends of their ranges, against plain 64-bit forms.

Bounds are derived as in test_gpu_decoder_ops.py, whose helpers are used here."""
import math

import pytest
import torch

from test_gpu_decoder_ops import (BF16, E4M3, F16, F32, SUB, U, attend64, e4m3_tol, gen, m, make_cache,  # noqa: F401
                                  norm64, randn, within)

pytestmark = pytest.mark.gpu


# ---- norm ---------------------------------------------------------------------


def norm8(m, x, w, eps=1e-6):
    y, sc = torch.empty(x.shape, dtype=E4M3, device="cuda"), torch.empty(x.shape[0], device="cuda")
    m.moe_add_rms_norm(x, w, y, scale=sc, eps=eps)
    return y.float(), sc


@pytest.mark.parametrize("H", [64, 200, 4096, 4097])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_norm_square_past_fp32(m, H, xt):
    """A finite row whose squares overflow: a NaN scale in E4M3, zeros in the other types, and no
    other row touched."""
    x = randn(gen(H), 5, H).to(xt)
    clean8, cleans = norm8(m, x, None)
    clean = torch.empty_like(x)
    m.moe_add_rms_norm(x, None, clean)
    x[1] = 1e20  # every square overflows
    x[3, H // 2] = 3e19  # one does
    y8, sc = norm8(m, x, None)
    assert sc[1].isnan() and sc[3].isnan() and y8[1].isnan().all() and y8[3].isnan().all()
    assert torch.equal(sc[[0, 2, 4]], cleans[[0, 2, 4]]) and torch.equal(y8[[0, 2, 4]], clean8[[0, 2, 4]])
    y = torch.empty_like(x)
    m.moe_add_rms_norm(x, None, y)
    assert (y[[1, 3]] == 0).all() and torch.equal(y[[0, 2, 4]], clean[[0, 2, 4]])


@pytest.mark.parametrize("H", [64, 200, 4096, 4097])
def test_norm_nan_of_a_weight(m, H):
    """A NaN that the weights bring, or an infinity times a zero weight, reaches the scale of every
    row that it is in."""
    x, w = randn(gen(H), 3, H), torch.ones(H, device="cuda")
    w[H - 1] = float("nan")
    y8, sc = norm8(m, x, w)
    assert sc.isnan().all() and y8.isnan().all()
    w[H - 1] = 0.0
    x[1, H - 1] = float("inf")
    y8, sc = norm8(m, x, w)
    assert sc[1].isnan() and y8[1].isnan().all() and sc[[0, 2]].isfinite().all() and (y8[[0, 2], H - 1] == 0).all()


@pytest.mark.parametrize("H", [64, 200, 4096, 4097])
@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("size,weight,eps", [(1e8, 1e-37, 1e-6), (1.0, 1e-22, 1e30), (1.0, 1e-34, 1e-6), (1e-31, 1.0, 1e12)])
def test_norm_scale_held_at_its_least(m, H, xt, size, weight, eps):
    """Rows whose largest |y| / 448 is below 2^-126: the scale stays there and the codes are y over
    that scale (y stays normal or loses less than E4M3 does: 2^-149 against half of 2^-9 2^-126)."""
    x = (size * (0.5 + torch.rand(4, H, generator=gen(H), device="cuda"))).to(xt)
    w = (weight * (0.1 + torch.rand(H, generator=gen(H + 1), device="cuda"))).to(xt)
    y64 = norm64(x, None, w, eps)[1]
    s = (y64.abs().amax(1) / 448).clamp(min=2.0 ** -126)
    y8, sc = norm8(m, x, w, eps)
    within(sc, s, s * 8e-6, "scale")
    within(y8, y64 / s[:, None], e4m3_tol(y64 / s[:, None]) + 2.0 ** -22, "codes")


# ---- append -------------------------------------------------------------------


@pytest.mark.parametrize("D", [64, 80])  # runs of 8 through the ring, and the kernel for any rows
def test_append_over_subnormal_scales(m, D):
    """Scales whose inverse is past fp32: zeros stay zeros, and values are divided all the same."""
    ks = torch.tensor([2.0 ** -130, 2.0 ** -126, 0.5], device="cuda")
    vs = torch.tensor([2.0 ** -149, -(2.0 ** -129), 1.0], device="cuda")
    kc, vc = (torch.ones(2, 4, 3, D, device="cuda").to(E4M3) for _ in range(2))
    kv = m.KvCache(kc, vc, q_heads=3, max_batch=1, k_scale=ks, v_scale=vs)
    x = torch.zeros(5, 3, D, device="cuda").to(BF16)
    x[:, :, 1], x[:, :, 2], x[:, :, 3] = 2.0 ** -126, 3 * 2.0 ** -129, -7 * 2.0 ** -131
    x[:, :, 4], x[:, :, 5] = 1.0, -3.0
    raw = x if D == 64 else torch.cat([x.flatten()[:1], x.flatten()])[1:].view_as(x)  # at an odd address
    slots = torch.arange(5, device="cuda")
    m.moe_kv_append(kv, raw, raw, raw, None, slots, None, torch.empty_like(x))
    for cache, scale in ((kc, ks), (vc, vs)):
        want = (x.double() / scale.double()[:, None]).clamp(-448, 448)
        assert torch.equal(cache.view(8, 3, D)[:5].float(), want.float().to(E4M3).float())


# ---- attend -------------------------------------------------------------------


def attend(m, q, k, v, ks, vs, pages, lens, **kw):
    kv = m.KvCache(k, v, q_heads=q.shape[1], max_batch=len(lens), k_scale=ks, v_scale=vs)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    m.moe_kv_attend(kv, q, pages, torch.tensor(lens, dtype=torch.int32, device="cuda"), o, lse=lse, **kw)
    assert kv.status() == 0
    return o, lse


@pytest.mark.parametrize("qt", [BF16, F16])
@pytest.mark.parametrize("scale", [0.125, -0.25])
def test_attend_signed_scales(m, qt, scale):
    """A cache's value is scale * code whatever the scale's sign, and a NaN scale spoils its heads."""
    g = gen(31)
    lens = [1, 40, 0, 700, 3000]
    k, v, ks, vs, pages = make_cache(g, lens, 16, 4, 64, E4M3)
    ks[1], vs[2] = -ks[1], -vs[2]
    ks[3], vs[3] = -ks[3], -vs[3]
    q = randn(g, len(lens), 12, 64).to(qt)
    o, lse = attend(m, q, k, v, ks, vs, pages, lens, scale=scale)
    o64, l64, ot, lt = attend64(q, k, v, ks, vs, pages, lens, scale, 0)
    within(o, o64, ot, "out")
    within(lse, l64, lt, "lse")
    ks[1] = float("nan")
    o2, lse2 = attend(m, q, k, v, ks, vs, pages, lens, scale=scale)
    some = torch.tensor([n > 0 for n in lens], device="cuda")
    assert o2[some, 3:6].isnan().all() and lse2[some, 3:6].isnan().all()
    keep = [0, 1, 2, 6, 7, 8, 9, 10, 11]
    assert torch.equal(o2[:, keep], o[:, keep]) and torch.equal(lse2[:, keep], lse[:, keep])


@pytest.mark.parametrize("ct", [BF16, F16, E4M3])
@pytest.mark.parametrize("lens,where", [([1, 5], 0), ([40, 7], 20), ([300, 300], 299), ([300, 20], 70), ([6000, 100], 4321)])
def test_attend_nan_keys_reach_the_log_sum(m, ct, lens, where):
    """One NaN among the keys of a head: that head's outputs and log-sums are NaN, wherever the token
    lies in the split; a NaN query likewise.  The others stay as they were."""
    g = gen(32)
    qt = F16 if ct == F16 else BF16
    k, v, ks, vs, pages = make_cache(g, lens, 16, 2, 64, ct)
    q = randn(g, 2, 6, 64).to(qt)
    o, lse = attend(m, q, k, v, ks, vs, pages, lens)
    page, e = int(pages[0, where // 16]), where % 16
    kb = k.float()
    kb[page, e, 1, 7] = float("nan")
    o2, lse2 = attend(m, q, kb.to(ct), v, ks, vs, pages, lens)
    assert o2[0, 3:].isnan().all() and lse2[0, 3:].isnan().all()
    assert torch.equal(o2[0, :3], o[0, :3]) and torch.equal(lse2[0, :3], lse[0, :3])
    assert torch.equal(o2[1], o[1]) and torch.equal(lse2[1], lse[1])
    q[0, 2, 63] = float("nan")
    o3, lse3 = attend(m, q, k, v, ks, vs, pages, lens)
    assert o3[0, 2].isnan().all() and lse3[0, 2].isnan()
    rest = [0, 1, 3, 4, 5]
    assert torch.equal(o3[0, rest], o[0, rest]) and torch.equal(lse3[0, rest], lse[0, rest])


@pytest.mark.parametrize("ct,qt", [(F16, F16), (E4M3, F16), (BF16, BF16)])
def test_attend_many_small_weights(m, ct, qt):
    """One key outweighs each of the others by e^17.5 = 2^25.3, and there are 2^18 others, whose
    values alone are not zero: together they are 0.6% of the weight and all of the output."""
    n, B = (1 << 18) + 1, 512  # more sequences than blocks: a block walks a whole sequence
    page = 4096
    n_pages = -(-n // page)
    k = torch.zeros(n_pages, page, 1, 64, device="cuda")
    v = torch.ones_like(k)
    k[0, 0, 0, 0], v[0, 0] = 17.5, 0.0
    ks = vs = torch.ones(1, device="cuda") if ct == E4M3 else None
    if ct == E4M3:
        k[0, 0, 0, 0] = 16.0
        k[0, 0, 0, 1] = 1.5
    q = torch.zeros(1, 1, 64, device="cuda")
    q[..., :2] = 1.0
    pages = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    k, v, q = k.to(ct), v.to(ct), q.to(qt)
    o, lse = attend(m, q.expand(B, 1, 64).contiguous(), k, v, ks, vs, pages.expand(B, -1), [n] * B, scale=1.0)
    o64, l64, ot, lt = attend64(q, k, v, ks, vs, pages, [n], 1.0, 0)
    within(o, o64.expand(B, 1, 64), ot.expand(B, 1, 64), "out")
    within(lse, l64.expand(B, 1), lt.expand(B, 1), "lse")


@pytest.mark.parametrize("ct,qt", [(BF16, BF16), (F16, F16), (E4M3, BF16), (E4M3, F16)])
def test_attend_dominant_key_after_the_first(m, ct, qt):
    """Two keys in one warp's hands, the later one e^c times the earlier one's weight, the rest below
    e^-24; values of one.  The outputs are one: what is left of the weights' two terms (2^-16) and
    of fp32 sums is below half of the type's spacing under one (2^-9 for bf16; 2^-12 for f16, whose
    weights lose 2^-22)."""
    c = torch.linspace(3.0, 5.4, 48, device="cuda")  # below 2^8, where the softmax's reference stays
    k, v = torch.zeros(1, 256, 1, 128, device="cuda"), torch.ones(1, 256, 1, 128, device="cuda")
    k[0, :, 0, 0] = -8.0
    k[0, 0], k[0, 128, 0, 0] = 0.0, 1.0
    q = torch.zeros(48, 1, 128, device="cuda")
    q[:, 0, 0] = c
    one = torch.ones(1, device="cuda") if ct == E4M3 else None
    pages = torch.zeros(48, 1, dtype=torch.int32, device="cuda")
    o, _ = attend(m, q.to(qt), k.to(ct), v.to(ct), one, one, pages, [129] * 48, scale=1.0)
    assert (o == 1).all(), float((o.double() - 1).abs().max())


@pytest.mark.parametrize("ct,qt", [(BF16, BF16), (F16, F16), (E4M3, BF16), (E4M3, F16)])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (16, 1, 64), (32, 1, 96), (2, 2, 256)])
def test_attend_adds_little_to_the_outputs_rounding(m, ct, qt, hq, hkv, D):
    """The bound of attend64 with the weights' two 16-bit terms in the place of one: 2^-16 of a weight
    for bf16 caches and 2^-22 for the others."""
    g = gen(34)
    lens = [5000, 33, 2000, 320]
    k, v, ks, vs, pages = make_cache(g, lens, 16, hkv, D, ct)
    q = randn(g, len(lens), hq, D).to(qt)
    o, _ = attend(m, q, k, v, ks, vs, pages, lens)
    o64, _, tol, _ = attend64(q, k, v, ks, vs, pages, lens, D ** -0.5, 0)
    own = o64.abs() * U[qt] * 1.01 + SUB[qt]
    size = attend64(q, k, v.float().abs().to(ct), ks, vs, pages, lens, D ** -0.5, 0)[0]
    one = U[BF16] if ct == BF16 else U[F16]
    tol = tol - size * (one - one * one)
    assert (tol >= own).all()
    within(o, o64, tol)


def test_attend_refuses_the_query_as_output(m):
    """Parts of a sequence read its query while another's join may have written the output."""
    g = gen(35)
    k, v, _, _, pages = make_cache(g, [40], 16, 1, 64, BF16)
    kv = m.KvCache(k, v, q_heads=4, max_batch=1)
    q = randn(g, 1, 4, 64).to(BF16)
    keep, n = q.clone(), torch.tensor([40], dtype=torch.int32, device="cuda")
    with pytest.raises(m.MoeError) as e:
        m.moe_kv_attend(kv, q, pages, n, q)
    assert e.value.code == m.MOE_ERR_INVALID_ARG and torch.equal(q, keep) and kv.status() == 0
    both = torch.cat([q, torch.zeros_like(q)], 1)  # one tensor's heads, apart from one another
    o = torch.empty_like(q)
    m.moe_kv_attend(kv, q, pages, n, o)
    m.moe_kv_attend(kv, both[:, :4], pages, n, both[:, 4:])
    assert torch.equal(both[:, 4:], o) and torch.equal(both[:, :4], keep)


# ---- linear -------------------------------------------------------------------


@pytest.mark.parametrize("T,N,K", [(1, 64, 4096), (3, 1000, 8192), (32, 512, 4096), (128, 256, 4096), (300, 520, 2048),
                                   (600, 1023, 1040), (1024, 2048, 512)])
@pytest.mark.parametrize("xt", [BF16, F16, E4M3])
def test_linear_of_whole_numbers_is_exact(m, T, N, K, xt):
    """Whole numbers up to 8 (their sums below 2^24): fp32 holds every partial sum, so that nothing may
    be rounded on the way, in whatever parts the product is made and joined."""
    g = gen(T + K)
    x = torch.randint(-8, 9, (T, K), generator=g, device="cuda").to(xt)
    w = torch.randint(-8, 9, (N, K), generator=g, device="cuda").to(xt)
    one = (lambda n: torch.ones(n, device="cuda")) if xt == E4M3 else (lambda n: None)
    r = torch.randint(-1000, 1000, (T, N), generator=g, device="cuda").float()
    b = torch.randint(-1000, 1000, (N,), generator=g, device="cuda").float()
    y = torch.empty(T, N, device="cuda")
    m.moe_linear(x, w, y, bias=b, residual=r, x_scale=one(T), w_scale=one(N))
    assert torch.equal(y.double(), x.double() @ w.double().t() + b.double() + r.double())


def activation_points():
    v = torch.cat([torch.linspace(-14, 14, 40001), torch.linspace(-0.01, 0.01, 4001), torch.linspace(-90, 90, 18001),
                   torch.tensor([0.0, 1e-30, -1e-30, 1e30, -1e30, 3e38, -3e38])]).cuda()
    return v[: v.numel() // 8 * 8]


def as_stored(want, yt):
    """Infinite where the output type's nearest value is."""
    top = torch.finfo(yt).max * (1 + U[yt] / 2)
    return torch.where(want.abs() >= top, want.sign() * math.inf, want)


@pytest.mark.parametrize("T", [1, 300])  # the split kernel and the tiled one
@pytest.mark.parametrize("yt", [F32, F16, BF16])
def test_linear_gelu_everywhere(m, T, yt):
    """v Phi(v) of the bias alone, to 2^-18 of its value in fp32 and below 2^-126 absolutely (header)."""
    v = activation_points()
    x, w = torch.zeros(T, 16, device="cuda").to(BF16), torch.zeros(v.numel(), 16, device="cuda").to(BF16)
    y = torch.empty(T, v.numel(), dtype=yt, device="cuda")
    m.moe_linear(x, w, y, bias=v, act="gelu")
    want = (0.5 * v.double() * torch.special.erfc(-v.double() / math.sqrt(2.0))).expand(T, -1)
    within(y, as_stored(want, yt), want.abs() * (2.0 ** -18 + U[yt]) + 2.0 ** -126 + SUB[yt])


@pytest.mark.parametrize("T", [1, 300])
@pytest.mark.parametrize("yt", [F32, F16, BF16])
def test_linear_silu_everywhere(m, T, yt):
    """v / (1 + exp(-v)) of the bias alone, to 2^-20 of its value in fp32 and below 2^-126 absolutely:
    an exponential good to 2^-22 and its factor, a sum, a reciprocal of 1 unit and two products (2^-24,
    2^-24, 2^-23, 2^-23): 2.5 2^-22 in all."""
    v = activation_points()
    x, w = torch.zeros(T, 16, device="cuda").to(BF16), torch.zeros(v.numel(), 16, device="cuda").to(BF16)
    y = torch.empty(T, v.numel(), dtype=yt, device="cuda")
    m.moe_linear(x, w, y, bias=v, act="silu")
    want = (v.double() * torch.sigmoid(v.double())).expand(T, -1)
    within(y, as_stored(want, yt), want.abs() * (2.0 ** -20 + U[yt]) + 2.0 ** -126 + SUB[yt])
