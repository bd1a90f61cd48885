"""T.moe where the two products of an expert take different forms: the forms go by layout and pairs per expert."""
import numpy as np
import pytest

from oracle import layer_oracle as L
from tests.layer_cases import check, f64, half, weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gemm_tern_gemv_b200 as T  # noqa: E402

LAYOUTS = [T.Q2_0_G128, T.T3_5PB_G128, T.Q1_0_G128]
PAIRS = [(a, b) for a in LAYOUTS for b in LAYOUTS]


def _dev(a):
    return torch.from_numpy(a).cuda()


def _layer(up, down, d, f, experts, up_scale, down_scale, seed=0):
    gc, gs, gw = weights(up, experts * 2 * f, d, seed, scale=up_scale)
    dc, ds, dw = weights(down, experts * d, f, seed + 1, scale=down_scale)
    G, D = T.from_packed(_dev(gc), _dev(gs), up, d), T.from_packed(_dev(dc), _dev(ds), down, f)
    return G, D, gw.reshape(experts, 2 * f, d), dw.reshape(experts, d, f), half(seed + 2, experts, d, scale=1.5 / np.sqrt(d))


@pytest.mark.parametrize("up,down", PAIRS)
@pytest.mark.parametrize("tokens", [1, 3, 4, 6, 8, 16])
@pytest.mark.parametrize("size", ["large", "small"])
def test_expert_activations_outside_fp16s_range(up, down, tokens, size):
    # 8 experts, 2 chosen: 1/4, 3/4, 1, 3/2, 2 and 4 pairs for each. |h| beyond 65504 with down scales that bring y back,
    # or far below fp16's smallest normal with scales that keep y in range
    experts, top_k, d, f = 8, 2, 256, 256
    up_scale, x_scale, down_scale = (0.5, 300.0, 2.0 ** -13) if size == "large" else (2.0 ** -12, 2.0 ** -4, 2.0 ** 12)
    G, D, gw, dw, r = _layer(up, down, d, f, experts, up_scale, down_scale)
    x = half(3, tokens, d, scale=x_scale)
    y, w, ids = T.moe(G, D, _dev(r), _dev(x), top_k, act="relu", return_routing=True)
    args = (gw, dw, f64(r), f64(x), top_k, "relu", True)
    want, _, wi = L.moe(*args)
    h = np.concatenate([L.linear(gw[e], f64(x[t:t + 1]), None, "relu", True).ravel() for t in range(tokens) for e in wi[t]])
    assert np.abs(h).max() > 1e5 if size == "large" else np.median(np.abs(h)[h != 0]) < 2.0 ** -24
    assert np.abs(want).max() < 6e4 and np.array_equal(ids.cpu().numpy(), wi)
    check(y.cpu().numpy(), want, L.moe_bound(*args, held="fp16"), f"up {up} down {down}, {tokens} tokens")


@pytest.mark.parametrize("up", LAYOUTS)
@pytest.mark.parametrize("tokens", [1, 3, 8, 40])
def test_activations_beside_an_overflow_keep_their_size(up, tokens):
    # one h of each token is beyond fp32's range, the others are far beyond fp16's: what the down rows make of them is the
    # infinity with their weight's sign (binary: no weight is zero), not the difference of two
    experts, d, f, j = 2, 2048, 128, 5
    G, D, gw, dw, r = _layer(up, T.Q1_0_G128, d, f, experts, 1.0, 2.0 ** -13)
    plus = weights(up, 1, d, 0)[0].copy()
    plus[:] = {T.Q2_0_G128: 0x55, T.T3_5PB_G128: 242, T.Q1_0_G128: 0xFF}[up]  # every t = +1
    for row in (j, f + j, 2 * f + j, 3 * f + j):
        G.codes[row] = _dev(plus)[0]
        G.scales[row] = 65504.0
    x = np.minimum(np.abs(half(4, tokens, d)).astype(np.float64) * 1e4 + 55e3, 65504).astype(np.float16)
    # (65504 55e3 2048)^3 = 4.0e38, fp32 ends at 3.4e38; elsewhere at most (6.6e4 2048)^3 = 2.4e24
    y, _, ids = T.moe(G, D, _dev(r), _dev(x), 1, act="relu2", return_routing=True)
    want = np.sign(dw[ids.cpu().numpy()[:, 0], :, j]) * np.inf
    assert np.array_equal(y.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("tokens,experts,top_k,held", [(1, 4, 2, "integers"), (4, 64, 8, "integers"), (3, 24, 4, "integers"),
                                                      (4, 6, 3, "fp16"), (16, 4, 2, "fp16"), (30, 2, 1, "fp16")])
def test_activations_are_held_as_documented(layout, tokens, experts, top_k, held):
    # one token and up to half a pair per expert: integers; from two pairs (binary: more) on: fp16
    d, f = 256, 640
    if layout == T.Q1_0_G128 and held == "fp16":
        tokens *= 2
    G, D, gw, dw, r = _layer(layout, layout, d, f, experts, 0.02, 0.02, seed=20)
    x = half(21, tokens, d)
    args = (gw, dw, f64(r), f64(x), top_k, "silu", True)
    y = T.moe(G, D, _dev(r), _dev(x), top_k)
    check(y.cpu().numpy(), L.moe(*args)[0], L.moe_bound(*args, held=held), f"{held} {layout}")
