"""Rows and caches in E4M3 with fine scales, where their definitions are easiest to miss: codes at a tie, scales of the
caller's own making, sums at the end of fp32, tokens that do not follow one another, and the kernels for many tokens on
every kind of input.

Bounds come from the arithmetic; helpers and their bounds are those of the operators' own tests."""
import pytest
import torch

from test_gpu_fine_scales import BF16, E4M3, F16, F32, gen, m, randn  # noqa: F401

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
