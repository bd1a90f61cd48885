"""Scales of 2^15 and more, whose outputs the many-row products compute term by term: with many tiles for each pair of
blocks, so that later tiles' results depend on how long that takes, and with a residual that is the output itself."""
import numpy as np
import pytest

from oracle import layer_oracle as L
from tests.layer_cases import check, f64, half, weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gemm_tern_gemv_b200 as T  # noqa: E402


def _dev(a):
    return torch.from_numpy(a).cuda()


@pytest.mark.parametrize("layout", [T.Q2_0_G128, T.T3_5PB_G128])
def test_dx_of_a_long_sum_in_three_rounds_of_tiles(layout):
    # 2048 x 4096 of dx are 176 tiles for 74 pairs of blocks; one scale concerns 128 columns, 2048 sums of 151936 terms
    m, n, k = 2048, 151936, 4096
    g = torch.Generator(device="cuda").manual_seed(5)
    W = T.empty_matrix(layout, n, k)
    if layout == T.Q2_0_G128:
        W.codes.copy_(torch.tensor([0x00, 0x01, 0x43, 0x5C, 0x37, 0xD0, 0x1F, 0x74], dtype=torch.uint8, device="cuda")[
            torch.randint(0, 8, W.codes.shape, generator=g, device="cuda", dtype=torch.int32)])
    else:
        W.codes.copy_(torch.randint(0, 243, W.codes.shape, generator=g, device="cuda", dtype=torch.int32))
    W.scales[:, :k // 128] = 2.0 ** -9
    W.scales[77, 3] = 40000.0
    W.scales[n - 1, 3] = -33000.0
    dz = (torch.randn(m, n, generator=g, device="cuda") * 2.0 ** -7).half()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, _, _ = T.linear_backward(W, dz, need_dbias=False, status=status)
    assert int(status.item()) == 0
    w = T.unpack(W, want_t=False)[0]
    worst = 0.0
    for c0 in range(0, k, 512):  # every column, some at a time
        wd = w[:, c0:c0 + 512].double()
        want, a = torch.zeros(m, 512, dtype=torch.float64, device="cuda"), torch.zeros(m, 512, dtype=torch.float64, device="cuda")
        for r in range(0, n, 1 << 14):
            d = dz[:, r:r + (1 << 14)].double()
            want += d @ wd[r:r + (1 << 14)]
            a += d.abs() @ wd[r:r + (1 << 14)].abs()
        # n / 16 + 64 steps of the tensor cores, or n fp32 additions one after the other (2^-24 each): n 2^-24 holds both
        bound = n * 2.0 ** -24 * a * (1 + L.HALF_F16) + L.HALF_F16 * want.abs() + L.TINY_F16
        worst = max(worst, float(((dx[:, c0:c0 + 512].double() - want).abs() / bound).max()))
    assert worst <= 1.0, worst


@pytest.mark.parametrize("layout", [T.Q2_0_G128, T.T3_5PB_G128])
@pytest.mark.parametrize("gated", [False, True])
def test_in_place_residual_beside_large_scales(layout, gated):
    m, n, k = 200, 40000 + 46 * gated, 384  # four tiles and more for a pair
    codes, s, w = weights(layout, n, k, 90)
    s[:] = np.float16(2.0 ** -16)
    for r in (0, 3, 77, n // 2 - 1, n // 2, n // 2 + 3, n - 60, n - 1):
        s[r, r % 3] = np.float16(40000.0 if r % 2 else -32768.0)
    w = np.sign(w) * np.repeat(s.astype(np.float64), 128, axis=1)
    W = T.from_packed(_dev(codes), _dev(s), layout, k)
    nout = n // 2 if gated else n
    x, res, b = half(91, m, k, scale=2.0 ** -12), half(92, m, nout), half(93, n)
    y, z = _dev(res), torch.empty(m, n, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    T.linear(W, _dev(x), _dev(b), act="silu", gated=gated, residual=y, y=y, preact=z, status=status)
    assert int(status.item()) == 0
    args = (w, f64(x), f64(b), "silu", gated, f64(res))
    # the rows of large scales are summed one term after the other: k 2^-24 is less than the (k / 16 + 64) 2^-23 allowed for
    check(y.cpu().numpy(), L.linear(*args), L.linear_bound(*args), "y")
    check(z.cpu().numpy(), L.preact(w, f64(x), f64(b)), L.preact_bound(w, f64(x), f64(b)), "preact")
