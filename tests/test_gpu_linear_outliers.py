"""Few rows of x with huge activations beside tiny ones: an output whose weights at the huge ones are zero has to be as
exact as any sum in fp32, so the bounds here hold nothing for a common exponent of neighbouring activations."""
import numpy as np
import pytest

from oracle import layer_oracle as L
from tests.layer_cases import check, f64, half, weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gemm_tern_gemv_b200 as T  # noqa: E402

LAYOUTS = [T.Q2_0_G128, T.T3_5PB_G128, T.Q1_0_G128]


def _dev(a):
    return torch.from_numpy(a).cuda()


def _outliers(seed, m, k, tiny, every):
    x = half(seed, m, k, scale=tiny)
    rng = np.random.default_rng(seed)
    for i in range(m):
        for u in range(0, k, every):
            x[i, u + rng.integers(0, min(every, k - u))] = rng.choice([60000.0, -2000.0, 511.0])
    return x


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n", [64, 2500, 9700])
@pytest.mark.parametrize("m", [1, 2, 3])
@pytest.mark.parametrize("tiny", [1e-2, 1e-3, 2.0 ** -22])
def test_huge_beside_tiny(layout, n, m, tiny):
    k = 896
    codes, s, w = weights(layout, n, k, n)
    W = T.from_packed(_dev(codes), _dev(s), layout, k)
    x = _outliers(1, m, k, tiny, 160)
    args = (w, f64(x))
    check(T.linear(W, _dev(x)).cpu().numpy(), L.linear(*args), L.linear_bound(*args, common=False), "plain")
    args = (w, f64(x), None, "relu", True)
    y, want = T.linear(W, _dev(x), act="relu", gated=True).cpu().numpy(), L.linear(*args)
    fits = np.abs(want) < 65000  # products of two sums of huge ones do not
    check(np.where(fits, y, 0), np.where(fits, want, 0), L.linear_bound(*args, common=False), "gated")
    assert np.isinf(y[np.abs(want) > 66000]).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("k", [128 * 300, 128 * 1400])
def test_outliers_in_long_rows(layout, k):
    # rows in several passes, and more units of a row than a word for each 32 of 1024 tells apart; 64 rows repeated
    n, m = 9536, 1
    codes, s, w = weights(layout, 64, k, 3)
    W = T.from_packed(_dev(np.tile(codes, (n // 64, 1))), _dev(np.tile(s, (n // 64, 1))), layout, k)
    for every in (k // 2, 1280):
        x = _outliers(4, m, k, 1e-3, every)
        y = T.linear(W, _dev(x)).cpu().numpy()
        check(y[:, :64], L.linear(w, f64(x)), L.linear_bound(w, f64(x), common=False), "long rows")
        assert np.array_equal(y, np.tile(y[:, :64], (1, n // 64)))
        assert torch.equal(_dev(y), T.linear(W, _dev(x)))


@pytest.mark.parametrize("layout", [T.Q2_0_G128, T.T3_5PB_G128])
def test_one_weight_in_a_row(layout):
    # row i picks activation i % k: the result is that activation, whatever stands beside it
    n, k = 9600, 640
    from tests.gpu_cases import pack_rows
    t = np.zeros((n, k), np.int8)
    t[np.arange(n), np.arange(n) % k] = 1
    W = T.from_packed(_dev(pack_rows(t, layout)), _dev(np.ones((n, k // 128), np.float16)), layout, k)
    x = half(5, 1, k, scale=1.0)
    x[0] *= np.float16(2.0) ** np.random.default_rng(6).integers(-16, 15, k).astype(np.float16)
    y = T.linear(W, _dev(x)).cpu().numpy()
    assert np.array_equal(y[0], x[0][np.arange(n) % k])


@pytest.mark.parametrize("layout", LAYOUTS)
def test_experts_of_one_token(layout):
    experts, d, f = 4, 640, 2432
    gc, gs, gw = weights(layout, experts * 2 * f, d, 7)
    dc, ds, dw = weights(layout, experts * d, f, 8, scale=64.0 if layout != T.Q1_0_G128 else 2.0 ** -8)
    G, D = T.from_packed(_dev(gc), _dev(gs), layout, d), T.from_packed(_dev(dc), _dev(ds), layout, f)
    r = half(9, experts, d, scale=1e-3)
    x = _outliers(10, 1, d, 1e-3, 320)
    # gates that skip the huge activations: only those rows' h are small enough to compare
    big = np.abs(x[0]) > 1
    if layout != T.Q1_0_G128:
        from tests.gpu_cases import pack_rows
        t = np.sign(gw).astype(np.int8)
        t[:, big] = 0
        gw = np.where(big, 0.0, gw)
        G = T.from_packed(_dev(pack_rows(t, layout)), _dev(gs), layout, d)
    else:
        x[0, big] = 100.0
    args = (gw.reshape(experts, 2 * f, d), dw.reshape(experts, d, f), f64(r), f64(x), 2, "relu", True)
    y, _, ids = T.moe(G, D, _dev(r), _dev(x), 2, act="relu", return_routing=True)
    assert np.array_equal(ids.cpu().numpy(), L.moe(*args)[2])
    check(y.cpu().numpy(), L.moe(*args)[0], L.moe_bound(*args, held="integers"), "one token")


@pytest.mark.parametrize("layout", [T.Q2_0_G128, T.T3_5PB_G128])
def test_experts_that_two_tokens_share(layout):
    # few pairs per expert, some of them with two: huge activations whose weights are zero beside tiny ones in each
    experts, d, f, tokens, top_k = 24, 640, 384, 3, 4
    from tests.gpu_cases import pack_rows
    _, gs, gw = weights(layout, experts * 2 * f, d, 11)
    dc, ds, dw = weights(layout, experts * d, f, 12, scale=64.0)
    x = _outliers(13, tokens, d, 1e-3, 320)
    big = (np.abs(x) > 1).any(0)
    t = np.sign(gw).astype(np.int8)
    t[:, big] = 0
    gw = np.where(big, 0.0, gw)
    G = T.from_packed(_dev(pack_rows(t, layout)), _dev(gs), layout, d)
    D = T.from_packed(_dev(dc), _dev(ds), layout, f)
    r = half(14, experts, d, scale=1e-3)
    args = (gw.reshape(experts, 2 * f, d), dw.reshape(experts, d, f), f64(r), f64(x), top_k, "relu", True)
    y, _, ids = T.moe(G, D, _dev(r), _dev(x), top_k, act="relu", return_routing=True)
    assert np.array_equal(ids.cpu().numpy(), L.moe(*args)[2])
    assert np.bincount(ids.cpu().numpy().ravel()).max() > 1
    check(y.cpu().numpy(), L.moe(*args)[0], L.moe_bound(*args, held="integers"), "shared experts")


def _few_tiny(seed, m, k, count):
    """x with huge, ordinary and `count` tiny activations, the tiny ones alone below what stands beside the huge ones; their places."""
    rng = np.random.default_rng(seed)
    x = (np.round(rng.standard_normal((m, k)) * 64) / 64).astype(np.float16)
    x[:, rng.choice(k, 5, replace=False)] = 30000.0
    tiny = rng.choice(np.flatnonzero(x[0] < 100), count, replace=False)
    x[:, tiny] = (rng.standard_normal((m, count)) * 1e-3).astype(np.float16)
    return x, tiny


@pytest.mark.parametrize("layout", [T.Q2_0_G128, T.T3_5PB_G128])
@pytest.mark.parametrize("k,count", [(640, 1), (640, 30), (4224, 200), (4224, 1200), (38400, 250)])
@pytest.mark.parametrize("gated", [False, True])
def test_outputs_of_the_tiny_activations_alone(layout, k, count, gated):
    # weights at every other activation are zero; few and many of the tiny ones stand beside a huge one
    from tests.gpu_cases import pack_rows
    n0, times = 64, 150
    x, tiny = _few_tiny(15, 1, k, count)
    t = np.zeros((n0, k), np.int8)
    t[:, tiny] = np.random.default_rng(16).integers(-1, 2, (n0, count))
    s = half(17, n0, k // 128, scale=0.05)
    w = t * np.repeat(f64(s), 128, axis=1)
    W = T.from_packed(_dev(np.tile(pack_rows(t, layout), (times, 1))), _dev(np.tile(s, (times, 1))), layout, k)
    act = "relu" if gated else "none"
    args = (np.concatenate([w, w]) if gated else w, f64(x), None, act, gated)
    scale = 2.0 ** 10 if gated else 1.0  # a gate times an up sum of 1e-3 would fall below fp16's steps
    if gated:
        W.scales *= scale
        args = (args[0] * scale,) + args[1:]
    y = T.linear(W, _dev(x), act=act, gated=gated)
    check(y[:, :n0].cpu().numpy(), L.linear(*args), L.linear_bound(*args, common=False), "tiny alone")
    assert torch.equal(y, y[:, :n0].repeat(1, y.shape[1] // n0))
    for _ in range(5):
        assert torch.equal(y, T.linear(W, _dev(x), act=act, gated=gated))


@pytest.mark.parametrize("layout", [T.Q2_0_G128, T.T3_5PB_G128])
def test_tiny_activations_of_tokens_that_share_experts(layout):
    from tests.gpu_cases import pack_rows
    experts, d, f, tokens, top_k = 24, 640, 384, 3, 4
    x, tiny = _few_tiny(18, tokens, d, 30)
    t = np.zeros((experts * 2 * f, d), np.int8)
    t[:, tiny] = np.random.default_rng(19).integers(-1, 2, (t.shape[0], 30))
    gs = half(20, experts * 2 * f, d // 128, scale=16.0)
    gw = t * np.repeat(f64(gs), 128, axis=1)
    dc, ds, dw = weights(layout, experts * d, f, 21, scale=1.0)
    G, D = T.from_packed(_dev(pack_rows(t, layout)), _dev(gs), layout, d), T.from_packed(_dev(dc), _dev(ds), layout, f)
    r = half(22, experts, d, scale=1e-3)
    args = (gw.reshape(experts, 2 * f, d), dw.reshape(experts, d, f), f64(r), f64(x), top_k, "relu", True)
    y, _, ids = T.moe(G, D, _dev(r), _dev(x), top_k, act="relu", return_routing=True)
    assert np.array_equal(ids.cpu().numpy(), L.moe(*args)[2])
    check(y.cpu().numpy(), L.moe(*args)[0], L.moe_bound(*args, held="integers"), "shared experts")
