"""The derivatives of T.linear_backward at infinite and NaN z, where fp16 pre-activations overflowed: the formulas' own values."""
import numpy as np
import pytest

from oracle import layer_oracle as L
from tests.layer_cases import f64, weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gemm_tern_gemv_b200 as T  # noqa: E402


def _want(act, z):
    """act(z) and act'(z) of the formulas in fp64, as they are written (a limit is not taken)."""
    s = lambda u: 1 / (1 + np.exp(-u))  # noqa: E731
    with np.errstate(all="ignore"):
        if act == "silu":
            return z * s(z), s(z) + z * s(z) * (1 - s(z))
        if act == "gelu":
            c = (1 + L._erf(z / np.sqrt(2))) / 2
            return z * c, c + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        if act == "gelu_tanh":
            a = np.sqrt(2 / np.pi)
            t = np.tanh(a * (z + 0.044715 * z ** 3))
            return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t * t) / 2 * a * (1 + 3 * 0.044715 * z * z)
        if act == "relu":  # NaN stays NaN
            return np.where(z < 0, 0, z), np.where(np.isnan(z), z, z > 0)
        if act == "relu2":
            return np.where(z < 0, 0, z * z), np.where(z < 0, 0, 2 * z)
        return z, np.ones_like(z)


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("n", [8, 6])  # 16-byte and 2-byte accesses
def test_derivatives_at_infinities(act, n):
    z = np.zeros((3, n), np.float16)
    z[0], z[1], z[2] = -np.inf, np.inf, np.nan
    codes, s, _ = weights(T.Q2_0_G128, 2 * n, 128, 3)
    W = T.from_packed(torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda(), T.Q2_0_G128, 128)
    f, df = _want(act, f64(z))
    zz = torch.from_numpy(np.concatenate([z, np.ones_like(z)], 1)).cuda()  # gated: up = 1
    dy = torch.ones(3, n, dtype=torch.float16, device="cuda")
    _, dz, _ = T.linear_backward(W, dy, zz, act=act, gated=True, need_dx=False)
    got = f64(dz.cpu().numpy())
    assert np.array_equal(got[:, :n], df, equal_nan=True) and np.array_equal(got[:, n:], f, equal_nan=True)
    if act != "none":
        _, dz, _ = T.linear_backward(W, torch.ones(3, 2 * n, dtype=torch.float16, device="cuda"),
                                     torch.from_numpy(np.concatenate([z, z], 1)).cuda(), act=act, need_dx=False)
        assert np.array_equal(f64(dz.cpu().numpy()), np.concatenate([df, df], 1), equal_nan=True)
