"""GPU parity of the linear layer's backward (T.linear_backward) against the fp64 oracle and differences."""
import numpy as np
import pytest

from oracle import layer_oracle as L
from tests.layer_cases import check, f64, half, weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gemm_tern_gemv_b200 as T  # noqa: E402

LAYOUTS = [T.Q2_0_G128, T.T3_5PB_G128, T.Q1_0_G128]


def _dev(a):
    return None if a is None else torch.from_numpy(a).cuda()


def _matrix(codes, s, layout, k):
    return T.from_packed(_dev(codes), _dev(s), layout, k)


def _check(layout, m, n, k, act="silu", gated=False, zscale=1.0, seed=0):
    codes, s, w = weights(layout, n, k, seed + n + k + layout)
    z = half(seed + 1, m, n, scale=zscale)
    dy = half(seed + 2, m, n // 2 if gated else n)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dz, db = T.linear_backward(_matrix(codes, s, layout, k), _dev(dy), _dev(z), act=act, gated=gated, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want = L.linear_backward(w, f64(dy), f64(z), act, gated)
    bound = L.backward_bounds(w, f64(dy), f64(z), act, gated)
    for name, got, a, b in zip(("dx", "dz", "dbias"), (dx, dz, db), want, bound):
        check(got.cpu().numpy(), a, b, f"{name} layout {layout} {m}x{n}x{k} {act} gated={gated}")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [1, 2, 5, 16, 17, 64, 77, 130, 300])
def test_rows(layout, m):
    _check(layout, m, 200, 640)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,k", [(1, 128), (3, 256), (7, 384), (63, 128), (65, 640), (129, 896), (1001, 1280), (2000, 256),
                                 (4100, 128)])
@pytest.mark.parametrize("m", [1, 19, 70])
def test_odd_sizes(layout, n, k, m):
    _check(layout, m, n, k, act="gelu")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("f,k", [(1, 128), (33, 384), (500, 1152)])
@pytest.mark.parametrize("m", [1, 40, 257])
def test_gated(layout, f, k, m):
    _check(layout, m, 2 * f, k, gated=True)


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_activations(act, gated):
    _check(T.Q2_0_G128, 33, 128, 256, act=act, gated=gated, zscale=4.0)


def test_tails_of_the_activations():
    # far negative and positive z, zeros: derivatives vanish or saturate without NaN
    z = np.array([[-60000, -200, -90, -20, -6, -1e-3, 0, 1e-3, 6, 20, 90, 60000]], dtype=np.float16)
    codes, s, w = weights(T.Q2_0_G128, 12, 128, 3)
    dy = np.ones((1, 12), np.float16)
    for act in L.ACTS:
        dx, dz, db = T.linear_backward(_matrix(codes, s, T.Q2_0_G128, 128), _dev(dy), _dev(z), act=act)
        with np.errstate(over="ignore"):
            want = L.act_grad(act, f64(z))
            bound = L.backward_bounds(w, f64(dy), f64(z), act)[1]
        got, keep = dz.cpu().numpy().astype(np.float64), np.abs(want) < 65504
        assert np.isfinite(db.cpu().numpy()).all()
        assert (np.abs(got - want) <= bound)[keep].all() and np.isinf(got[~keep]).all(), act


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu2"])
def test_against_differences(act, gated):
    # <dy, y(x + e v) - y(x - e v)> / 2e = <dx, v>, the forward in fp64; likewise for the bias
    m, n, k = 6, 64, 256
    codes, s, w = weights(T.T3_5PB_G128, n, k, 9)
    W = _matrix(codes, s, T.T3_5PB_G128, k)
    x, b = half(1, m, k), half(2, n, scale=0.3)
    z = torch.empty(m, n, dtype=torch.float16, device="cuda")
    T.linear(W, _dev(x), _dev(b), act=act, gated=gated, preact=z)
    dy = half(3, m, n // 2 if gated else n)
    dx, dz, db = T.linear_backward(W, _dev(dy), z, act=act, gated=gated)
    rng, e = np.random.default_rng(4), 1e-5
    f = lambda xx, bb: (f64(dy) * L.linear(w, xx, bb, act, gated)).sum()  # noqa: E731
    bx, bz, bb = L.backward_bounds(w, f64(dy), f64(z.cpu().numpy()), act, gated)
    # the stored z is rounded (2^-11 |z|): dz moves by at most its slope times that; |act''| <= 2 for all four
    zz = np.abs(f64(z.cpu().numpy())) * 2.0 ** -11
    h = n // 2
    g = np.abs(f64(dy))
    if gated:
        zc = np.abs(f64(z.cpu().numpy()))
        slack = np.concatenate([g * (2 * zz[:, :h] * zc[:, h:] + 4 * (1 + zc[:, :h]) * zz[:, h:]),
                                g * 4 * (1 + zc[:, :h]) * zz[:, :h]], axis=1)
    else:
        slack = g * 2 * zz
    for _ in range(4):
        v, u = rng.standard_normal((m, k)), rng.standard_normal(n)
        want = (f(f64(x) + e * v, f64(b)) - f(f64(x) - e * v, f64(b))) / (2 * e)
        got = (f64(dx.cpu().numpy()) * v).sum()
        assert abs(got - want) <= ((bx + slack @ np.abs(w)) * np.abs(v)).sum() + 1e-6 * abs(want) + 1e-6
        want = (f(f64(x), f64(b) + e * u) - f(f64(x), f64(b) - e * u)) / (2 * e)
        got = (f64(db.cpu().numpy()) * u).sum()
        assert abs(got - want) <= ((bb + slack.sum(0)) * np.abs(u)).sum() + 1e-6 * abs(want) + 1e-6


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [1, 30])
def test_dx_is_exact_on_integers(layout, m):
    n, k = 200, 640
    codes, s, w = weights(layout, n, k, 5, scale=1.0)
    dy = np.random.default_rng(5).integers(-2, 3, size=(m, n)).astype(np.float16)
    dx, dz, db = T.linear_backward(_matrix(codes, s, layout, k), _dev(dy))
    assert np.array_equal(f64(dx.cpu().numpy()), f64(dy) @ w)
    assert np.array_equal(f64(db.cpu().numpy()), f64(dy).sum(0)) and torch.equal(dz, _dev(dy))


def test_parts_asked_for():
    codes, s, w = weights(T.Q2_0_G128, 96, 256, 6)
    W = _matrix(codes, s, T.Q2_0_G128, 256)
    dy, z = _dev(half(1, 20, 96)), _dev(half(2, 20, 96))
    dx, dz, db = T.linear_backward(W, dy, z, act="silu")
    a = T.linear_backward(W, dy, z, act="silu", need_dx=False)
    b = T.linear_backward(W, dy, z, act="silu", need_dbias=False)
    assert a[0] is None and torch.equal(a[1], dz) and torch.equal(a[2], db)
    assert b[2] is None and torch.equal(b[0], dx) and torch.equal(b[1], dz)
    none = T.linear_backward(W, dy, need_dx=False, need_dbias=False)
    assert none[0] is None and none[2] is None and torch.equal(none[1], dy)


def test_infinite_gradient_stays_in_its_row():
    codes, s, w = weights(T.Q2_0_G128, 64, 256, 7)
    dy, z = half(1, 40, 64), half(2, 40, 64)
    dy[3, 5] = np.inf
    dx, dz, db = T.linear_backward(_matrix(codes, s, T.Q2_0_G128, 256), _dev(dy), _dev(z), act="silu")
    bad = ~torch.isfinite(dx).all(1).cpu().numpy()
    assert bad.tolist() == [i == 3 for i in range(40)]
    assert (~torch.isfinite(db)).cpu().numpy().tolist() == [j == 5 for j in range(64)]


@pytest.mark.parametrize("m", [1, 20, 200])
def test_graph_replay_and_repeats_agree(m):
    codes, s, w = weights(T.Q1_0_G128, 2 * 160, 512, 8)
    W = _matrix(codes, s, T.Q1_0_G128, 512)
    dy, z = _dev(half(1, m, 160)), _dev(half(2, m, 320))
    want = T.linear_backward(W, dy, z, act="silu", gated=True)
    live = T.linear_backward(W, dy, z, act="silu", gated=True)  # an eager result alive during capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = T.linear_backward(W, dy, z, act="silu", gated=True)
    for _ in range(2):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, live):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_refused_operands():
    codes, s, _ = weights(T.Q2_0_G128, 32, 256, 60)
    W = _matrix(codes, s, T.Q2_0_G128, 256)
    dy = torch.zeros(2, 32, dtype=torch.float16, device="cuda")
    for bad in (dict(dy=dy.float(), preact=dy), dict(act="silu"), dict(preact=dy[:, :16], act="silu"), dict(gated=True),
                dict(preact=dy.cpu(), act="silu"), dict(act="sine"), dict(dy=dy[0])):
        with pytest.raises(ValueError):
            T.linear_backward(W, **{"dy": dy, **bad})
    with pytest.raises(T.TernError):
        T.linear_backward(W, dy[:0])


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [1, 40])
def test_extreme_scales(layout, m):
    # scales whose double does not fit fp16, beside subnormal ones
    n, k = 200, 384
    codes, s, w = weights(layout, n, k, 70)
    s[:] = np.float16(2.0 ** -16)
    s[5, 1], s[150, 1], s[7, 2] = 65504.0, -40000.0, np.float16(2.0 ** -24)
    w = np.sign(w) * np.repeat(s.astype(np.float64), 128, axis=1)
    dy = half(71, m, n, scale=2.0 ** -10)
    dx, _, _ = T.linear_backward(_matrix(codes, s, layout, k), _dev(dy))
    check(dx.cpu().numpy(), f64(dy) @ w, L.backward_bounds(w, f64(dy), None)[0], "extreme scales")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,k", [(2600, 1024), (1500, 4096), (700, 7680), (9001, 128)])
@pytest.mark.parametrize("m", [1, 33, 77, 190])
def test_sums_shared_by_several_pairs(layout, n, k, m):
    # few tiles of dx with many weight rows: two or four pairs of blocks take a part of the sum each
    _check(layout, m, n, k, act="gelu_tanh")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [3, 100])
def test_extreme_scale_in_one_part_of_the_sum(layout, m):
    n, k = 2000, 384
    codes, s, w = weights(layout, n, k, 74)
    s[:] = np.float16(2.0 ** -16)
    s[1999, 1] = -40000.0
    w = np.sign(w) * np.repeat(s.astype(np.float64), 128, axis=1)
    dy = half(75, m, n, scale=2.0 ** -10)
    dx, _, _ = T.linear_backward(_matrix(codes, s, layout, k), _dev(dy))
    check(dx.cpu().numpy(), f64(dy) @ w, L.backward_bounds(w, f64(dy), None)[0], "one extreme scale")
