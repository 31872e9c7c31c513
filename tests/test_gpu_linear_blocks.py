"""The product of E4M3 operands with a scale for each block of 128, against its 64-bit form.

Bounds come from the arithmetic: a block of K is at most eight steps of the tensor cores, each of which may lose
2^-22 of the sum of sizes; a block's two scales are multiplied (2^-24), meet its sum in a fused product and
addition (2^-24 of the running sum a block), and the epilogue adds a few steps of fp32."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
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
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


def act64(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "silu":
        return y * torch.sigmoid(y)
    if act == "gelu":
        return y * torch.special.ndtr(y)
    return y


def operands(g, T, N, K, pad=0):
    """E4M3 rows, `pad` apart from the next beyond their length, and scales that differ widely from block to block."""
    G, NB = -(-K // 128), -(-N // 128)
    x = (100 * randn(g, T, K + pad)).clamp(-448, 448).to(E4M3)[:, :K]
    w = (100 * randn(g, N, K + pad)).clamp(-448, 448).to(E4M3)[:, :K]
    xs = 0.01 * torch.exp(1.5 * randn(g, T, G + (3 if pad else 0)))[:, :G]
    ws = 0.01 / math.sqrt(K) * torch.exp(1.5 * randn(g, NB, G + (1 if pad else 0)))[:, :G]
    return x, w, xs, ws


def product64(x, w, xs, ws):
    """The product and the sum of its sizes."""
    K, N = x.shape[1], w.shape[0]
    x64 = x.double() * xs.double().repeat_interleave(128, 1)[:, :K]
    w64 = w.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return x64 @ w64.t(), x64.abs() @ w64.abs().t()


def check(m, g, T, N, K, yt, act="none", bias=None, res=False, ragged=False):
    x, w, xs, ws = operands(g, T, N, K, 16 if ragged else 0)
    G = xs.shape[1]
    b = None if bias is None else (0.3 * randn(g, N)).to(bias)
    wide = torch.full((T, N + 3), float("nan"), dtype=yt, device="cuda")
    y = wide[:, :N] if ragged else torch.full((T, N), float("nan"), dtype=yt, device="cuda")
    r = randn(g, T, N).to(yt) if res else None
    m.moe_linear_blocks(x, w, y, xs, ws, bias=b, act=act, residual=r)
    y64, size = product64(x, w, xs, ws)
    tol = size * (12 * 2.0 ** -22 + (G + 4) * 2.0 ** -24)
    if b is not None:
        y64 = y64 + b.double()
    tol = 1.13 * tol + y64.abs() * 2.0 ** -18  # no activation is steeper than 1.13; GELU is good to 2^-18
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
                                   (256, 512, 4096), (511, 1021, 528), (1000, 1536, 768), (2049, 640, 320), (240, 2000, 176),
                                   (3000, 2056, 192), (5001, 1023, 80), (2500, 4100, 1040), (8192, 640, 4096), (300, 130, 16384)])
@pytest.mark.parametrize("yt", [BF16, F32])
def test_sizes(m, T, N, K, yt):
    check(m, gen(T + N + K), T, N, K, yt)


@pytest.mark.parametrize("T", [1, 5, 40, 90, 130, 300, 3001])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("yt,bias,res", [(BF16, BF16, True), (F32, F32, False), (F16, F16, True), (F32, None, True), (BF16, None, False)])
def test_epilogue(m, T, act, yt, bias, res):
    check(m, gen(T), T, 333, 272, yt, act, bias, res, ragged=True)


@pytest.mark.parametrize("K", [16, 112, 128, 144, 640])
@pytest.mark.parametrize("T,N", [(257, 1023), (300, 72), (513, 2050), (1000, 8100), (700, 192), (5000, 320)])
def test_tiles_end_inside_a_run(m, T, N, K):
    """Aligned rows whose last run of outputs is cut short, with residual, in tiles of several widths."""
    g = gen(T + N + K)
    for yt in (BF16, F16, F32):
        x, w, xs, ws = operands(g, T, N, K)
        wide = torch.full((T, (N + 15) // 8 * 8), float("nan"), dtype=yt, device="cuda")
        y, r = wide[:, :N], randn(g, T, wide.shape[1]).to(yt)[:, :N]
        m.moe_linear_blocks(x, w, y, xs, ws, residual=r)
        y64, size = product64(x, w, xs, ws)
        want = y64 + r.double()
        tol = size * (12 * 2.0 ** -22 + (xs.shape[1] + 4) * 2.0 ** -24) + want.abs() * 2.0 ** -23
        within(y, want, tol + want.abs() * U[yt] + SUB[yt])
        assert wide[:, N:].isnan().all()


@pytest.mark.parametrize("T,N,K", [(3, 200, 512), (100, 300, 1024), (400, 520, 640)])
def test_each_block_meets_its_own_scales(m, T, N, K):
    """Whole numbers under powers of two: the products are exact, whatever parts they are made and joined in."""
    g = gen(T)
    x = torch.randint(-8, 9, (T, K), generator=g, device="cuda").float().to(E4M3)
    w = torch.randint(-8, 9, (N, K), generator=g, device="cuda").float().to(E4M3)
    xs = 2.0 ** torch.randint(-2, 3, (T, K // 128), generator=g, device="cuda").float()
    ws = 2.0 ** torch.randint(-2, 3, (-(-N // 128), K // 128), generator=g, device="cuda").float()
    y = torch.empty(T, N, device="cuda")
    m.moe_linear_blocks(x, w, y, xs, ws)
    assert torch.equal(y.double(), product64(x, w, xs, ws)[0])


def test_signs_zeros_and_nan_of_scales(m):
    g = gen(5)
    for T in (20, 400):
        x, w, xs, ws = operands(g, T, 300, 512)
        xs, ws = -xs, ws.clone()
        xs[3] = 0
        ws[1, 2] = 0
        y = torch.empty(T, 300, device="cuda")
        m.moe_linear_blocks(x, w, y, xs, ws)
        y64, size = product64(x, w, xs, ws)
        within(y, y64, size * 16 * 2.0 ** -22)
        assert (y[3] == 0).all()
        # a NaN or an infinity in a row's scales spoils that row, in a block of w those 128 outputs; no others
        bad, badw = xs.clone(), ws.clone()
        bad[7, 1], badw[2, 0] = float("nan"), float("inf")
        z = torch.empty_like(y)
        m.moe_linear_blocks(x, w, z, bad, badw)
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[7] = False
        assert torch.equal(z[keep, :256], y[keep, :256]) and z[7].isnan().all()
        assert not z[:, 256:][(x[:, :128].float() @ w[256:, :128].float().t() != 0) & (xs[:, :1] != 0)].isfinite().any()


def test_far_scales(m):
    """Scales whose products with a block's sum are far apart, and large sums that cancel between blocks."""
    g = gen(6)
    T, N, K = 130, 140, 384
    x, w, _, _ = operands(g, T, N, K)
    xs = torch.tensor([2.0 ** 60, 2.0 ** -60, 1.0], device="cuda").expand(T, 3)
    ws = torch.tensor([2.0 ** -50, 2.0 ** 55, 2.0 ** -20], device="cuda").expand(2, 3)
    y = torch.empty(T, N, device="cuda")
    m.moe_linear_blocks(x, w, y, xs, ws)
    y64, size = product64(x, w, xs, ws)
    within(y, y64, size * 16 * 2.0 ** -22)


def test_same_bits_in_place_graph_stream_and_no_rows(m):
    g = gen(7)
    for T, N, K in ((1, 512, 4096), (32, 300, 1024), (300, 512, 512), (1000, 1024, 512)):
        x, w, xs, ws = operands(g, T, N, K)
        r = randn(g, T, N)
        outs = []
        for _ in range(3):
            y = r.clone()
            m.moe_linear_blocks(x, w, y, xs, ws, residual=y)
            outs.append(y)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        y = torch.empty(T, N, device="cuda")
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                m.moe_linear_blocks(x, w, y, xs, ws, residual=r)
        for _ in range(2):
            y.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, outs[0])
        # a row's result does not depend on the rows beside it where the kernel and its split are the same
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        z = torch.empty(T, N, device="cuda")
        m.moe_linear_blocks(x, w, z, xs, ws, residual=r, status=status, stream=s)
        s.synchronize()
        assert torch.equal(z, y) and status.item() == 0
    m.moe_linear_blocks(x[:0], w, z[:0], xs[:0], ws)


def test_from_the_quantiser(m):
    """Rows as moe_quant_e4m3 leaves them, a weight quantised by blocks: within what E4M3 loses of the exact product."""
    g = gen(8)
    T, N, K = 70, 400, 1000 // 16 * 16
    a, w = randn(g, T, K).to(BF16), randn(g, N, K)
    x, xs = torch.empty(T, K, dtype=E4M3, device="cuda"), torch.empty(T, -(-K // 128), device="cuda")
    m.moe_quant_e4m3(a, x, xs)
    G, NB = -(-K // 128), -(-N // 128)
    p = torch.zeros(NB * 128, G * 128, device="cuda")
    p[:N, :K] = w
    ws = p.view(NB, 128, G, 128).abs().amax((1, 3)) / 448
    w8 = (p.view(NB, 128, G, 128) / ws[:, None, :, None]).view(NB * 128, -1)[:N, :K].to(E4M3).contiguous()
    y = torch.empty(T, N, device="cuda")
    m.moe_linear_blocks(x, w8, y, xs, ws)
    exact, size = a.double() @ w.double().t(), a.double().abs() @ w.double().abs().t()
    # each factor is off by 2^-4 of itself, or 2^-10 of its scale
    slack = (xs.double().repeat_interleave(128, 1)[:, :K] * 2.0 ** -10) @ w.double().abs().t() * 1.1
    slack += a.double().abs() @ (ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K] * 2.0 ** -10).t() * 1.1
    within(y, exact, size * (2 * 2.0 ** -4 + 2.0 ** -7) + slack)


def test_refusals(m):
    x, w, xs, ws = operands(gen(9), 4, 200, 256)
    y = torch.empty(4, 200, device="cuda")
    ok = dict(x=x, w=w, y=y, x_scale=xs, w_scale=ws)
    m.moe_linear_blocks(**ok)
    for kw in (dict(x=x.to(BF16), w=w.to(BF16)), dict(w=w[:, :128]), dict(x_scale=xs[:, :1]), dict(x_scale=xs[:3]), dict(w_scale=ws[:1]),
               dict(x_scale=xs[:, 0]), dict(w_scale=ws.half()), dict(w_scale=ws.t().contiguous().t()), dict(y=y.to(E4M3)), dict(act="tanh"),
               dict(residual=y.half()), dict(bias=y[0, :100]), dict(x_scale=xs.cpu()), dict(x=x[:, 4:], w=w[:, 4:]),
               dict(x=x[:, :248], w=w[:, :248]), dict(status=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(m.MoeError) as err:
            m.moe_linear_blocks(**{**ok, **kw})
        assert err.value.code == m.MOE_ERR_INVALID_ARG, kw
    with pytest.raises(TypeError):
        m.moe_linear_blocks(x, w, y, xs)
