"""Nine to sixteen rows of x at the lengths where their operands stop fitting on chip at once, with several tiles for each block."""
import numpy as np
import pytest

from oracle import layer_oracle as L
from tests.layer_cases import check, f64, half, weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gemm_tern_gemv_b200 as T  # noqa: E402


@pytest.mark.parametrize("layout,k", [(T.T3_5PB_G128, k) for k in (1920, 2048, 4096, 5120, 5248)] +
                         [(T.Q1_0_G128, k) for k in (4096, 4224, 5120, 5248)] + [(T.Q2_0_G128, k) for k in (5120, 6400, 17408)])
@pytest.mark.parametrize("m", [9, 13, 16])
@pytest.mark.parametrize("gated", [False, True])
def test_operands_in_one_or_several_passes(layout, k, m, gated):
    # 320 rows of weights repeated to three tiles for a block and more; the last tile is cut short
    n0, times = 320, 24
    codes, s, w = weights(layout, n0, k, k)
    x = half(1, m, k)
    x[:, :2] *= 8
    b = half(2, n0, scale=0.5)
    rep = lambda a: torch.from_numpy(np.tile(a, (times,) + (1,) * (a.ndim - 1))).cuda()  # noqa: E731
    if gated:  # the same gate and up rows under the repetition: both halves of it hold whole periods
        W = T.from_packed(rep(codes), rep(s), layout, k)
        y = T.linear(W, torch.from_numpy(x).cuda(), rep(b), act="silu", gated=True).cpu().numpy()
        args = (np.concatenate([w, w]), f64(x), f64(np.concatenate([b, b])), "silu", True)
        want = L.linear(*args)
        check(y[:, :n0], want, L.linear_bound(*args, common=False), "gated")
        assert np.array_equal(y, np.tile(y[:, :n0], (1, times // 2)))
    else:
        W = T.from_packed(rep(codes)[:-5], rep(s)[:-5], layout, k)
        y = T.linear(W, torch.from_numpy(x).cuda(), rep(b)[:-5], act="silu").cpu().numpy()
        args = (w, f64(x), f64(b), "silu")
        check(y[:, :n0], L.linear(*args), L.linear_bound(*args, common=False), "plain")
        assert np.array_equal(y, np.tile(y[:, :n0], (1, times))[:, :-5])
