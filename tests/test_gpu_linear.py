"""GPU parity of the fused linear layer (T.linear) against the fp64 oracle, within derived bounds."""
import numpy as np
import pytest

import oracle as O
from oracle import layer_oracle as L
from tests.layer_cases import check, f64, guarded, guards_kept, half, weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gemm_tern_gemv_b200 as T  # noqa: E402

LAYOUTS = [T.Q2_0_G128, T.T3_5PB_G128, T.Q1_0_G128]


def _matrix(codes, s, layout, k):
    return T.from_packed(torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda(), layout, k)


def _dev(a):
    return None if a is None else torch.from_numpy(a).cuda()


def _case(layout, m, n, k, act, gated, bias, residual, seed=0, xscale=1.0):
    codes, s, w = weights(layout, n, k, seed + n + k + layout)
    x = half(seed + 1, m, k, scale=xscale)
    x[:, np.random.default_rng(seed).integers(0, k, 2)] *= 8  # a few large channels
    b = half(seed + 2, n, scale=0.5) if bias else None
    r = half(seed + 3, m, n // 2 if gated else n) if residual else None
    return _matrix(codes, s, layout, k), w, x, b, r


def _check(layout, m, n, k, act="none", gated=False, bias=False, residual=False, preact=False, **kw):
    W, w, x, b, r = _case(layout, m, n, k, act, gated, bias, residual, **kw)
    n_out = n // 2 if gated else n
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ybuf, y = guarded(torch, (m, n_out), torch.float16, 777.0)
    zbuf, z = guarded(torch, (m, n), torch.float16, 333.0) if preact else (None, None)
    out = T.linear(W, _dev(x), _dev(b), act=act, gated=gated, residual=_dev(r), y=y, preact=z, status=status)
    torch.cuda.synchronize()
    assert out is y and int(status.item()) == 0
    args = (w, f64(x), f64(b), act, gated, f64(r))
    what = f"linear layout {layout} {m}x{n}x{k} {act} gated={gated}"
    check(y.cpu().numpy(), L.linear(*args), L.linear_bound(*args), what)
    assert guards_kept(ybuf, 777.0), what
    if preact:
        check(z.cpu().numpy(), L.preact(w, f64(x), f64(b)), L.preact_bound(w, f64(x), f64(b)), what + " preact")
        assert guards_kept(zbuf, 333.0), what


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 64, 65, 130])
def test_rows_of_x(layout, m):
    _check(layout, m, 200, 640, act="silu", bias=True, residual=True)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [1, 2, 7, 16, 40, 300])
def test_gated_rows_of_x(layout, m):
    _check(layout, m, 2 * 136, 1152, act="silu", gated=True, bias=True, residual=True, preact=True)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,k", [(1, 128), (2, 256), (7, 384), (15, 128), (17, 640), (33, 1280), (129, 896), (1000, 2176),
                                 (2050, 128), (64, 17408), (4100, 512)])
@pytest.mark.parametrize("m", [1, 6, 21])
def test_odd_widths_and_lengths(layout, n, k, m):
    _check(layout, m, n, k, residual=True)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("f,k", [(1, 128), (3, 384), (9, 256), (65, 640), (500, 1280), (2048, 256)])
@pytest.mark.parametrize("m", [1, 3, 12, 35])
def test_odd_gated_widths(layout, f, k, m):
    _check(layout, m, 2 * f, k, act="gelu", gated=True, preact=True)


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m", [1, 5, 50])
def test_activations(act, gated, m):
    _check(T.Q2_0_G128, m, 96, 512, act=act, gated=gated, bias=True, preact=True, xscale=4.0)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [1, 2, 11, 16])
def test_long_rows_in_several_passes(layout, m):
    # rows too long to keep every row of x on chip at once
    _check(layout, m, 48, 128 * 300, bias=True)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [1, 2, 4, 24])
def test_integers_are_exact(layout, m):
    n, k = 264, 1920
    codes, s, w = weights(layout, n, k, 5, scale=1.0)
    x = np.random.default_rng(5).integers(-1, 2, size=(m, k)).astype(np.float16)
    y = T.linear(_matrix(codes, s, layout, k), _dev(x)).cpu().numpy()
    assert np.array_equal(y.astype(np.float64), f64(x) @ w.T)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [1, 2, 5, 20])
def test_wide_dynamic_range(layout, m):
    # one huge activation per row next to tiny ones: rows whose weight there is zero depend on the tiny ones
    n, k = 96, 512
    codes, s, w = weights(layout, n, k, 6)
    x = half(7, m, k, scale=1e-2)
    x[np.arange(m), np.arange(m) * 37 % k] = 60000.0
    y = T.linear(_matrix(codes, s, layout, k), _dev(x)).cpu().numpy().astype(np.float64)
    check(y, L.linear(w, f64(x)), L.linear_bound(w, f64(x)), "wide range")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [1, 2, 4, 16, 20])
def test_infinities_and_nan_reach_the_rows_they_belong_to(layout, m):
    n, k = 70, 640
    codes, s, w = weights(layout, n, k, 8)
    x = half(9, m, k)
    x[0, 5] = np.inf
    if m > 1:
        x[1, k - 1] = np.nan
    if m > 3:
        x[3, 128], x[3, 129] = -np.inf, np.inf
    y = T.linear(_matrix(codes, s, layout, k), _dev(x)).cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        want = (f64(x)[:, None, :] * w[None]).sum(2)
    assert np.array_equal(np.isnan(y), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(y[inf], want[inf])
    fin = [i for i in range(m) if np.isfinite(f64(x)[i]).all()]
    check(y[fin], want[fin], L.linear_bound(w, f64(x)[fin]), "finite rows beside them")


@pytest.mark.parametrize("m", [1, 3, 40])
def test_zero_rows_and_zero_scales(m):
    n, k = 40, 384
    codes, s, w = weights(T.Q2_0_G128, n, k, 10)
    s[3] = 0
    s[5, 1] = 0
    w = w * np.repeat(s != 0, 128, axis=1)
    x = half(11, m, k)
    x[0] = 0
    W = _matrix(codes, s, T.Q2_0_G128, k)
    y = T.linear(W, _dev(x), act="silu").cpu().numpy()
    assert (y[0] == 0).all() and (y[:, 3] == 0).all()
    check(y, L.linear(w, f64(x), None, "silu"), L.linear_bound(w, f64(x), None, "silu"), "zeros")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [1, 4, 30])
def test_padded_rows_of_codes_and_scales(layout, m):
    # rows of a wider allocation: nothing between them may count
    n, k, f = 50, 896, 25
    codes, s, w = weights(layout, n, k, 12)
    wide = torch.full((n, codes.shape[1] + 48), 0x55, dtype=torch.uint8, device="cuda")
    wide[:, :codes.shape[1]] = _dev(codes)
    ws = torch.full((n, 24), float("nan"), dtype=torch.float16, device="cuda")
    ws[:, :k // 128] = _dev(s)
    W = T.TernMatrix(layout, n, k, wide, ws)
    x = half(13, m, k)
    y = T.linear(W, _dev(x), act="silu", gated=True).cpu().numpy()
    check(y, L.linear(w, f64(x), None, "silu", True), L.linear_bound(w, f64(x), None, "silu", True), "padded rows")


@pytest.mark.parametrize("m", [1, 9, 80])
def test_in_place_residual_and_strided_inputs(m):
    n, k = 256, 256
    codes, s, w = weights(T.Q2_0_G128, n, k, 14)
    W = _matrix(codes, s, T.Q2_0_G128, k)
    x, r = half(15, m, 2 * k), half(16, m, n)
    xs = _dev(x)[:, ::2]
    y = _dev(r).clone()
    T.linear(W, xs, residual=y, y=y)
    args = (w, f64(x[:, ::2]), None, "none", False, f64(r))
    check(y.cpu().numpy(), L.linear(*args), L.linear_bound(*args), "in place")
    one = T.linear(W, xs[0])
    assert one.shape == (n,) and torch.equal(one, T.linear(W, xs[:1])[0])
    odd = torch.empty(m * k + 1, dtype=torch.float16, device="cuda")[1:].view(m, k)  # 2-byte aligned x
    odd.copy_(xs)
    assert torch.equal(T.linear(W, odd), T.linear(W, xs))


@pytest.mark.parametrize("m", [1, 2, 6, 16, 90])
def test_graph_replay_streams_and_repeats_agree(m):
    n, k = 2 * 320, 1024
    codes, s, w = weights(T.T3_5PB_G128, n, k, 17)
    W = _matrix(codes, s, T.T3_5PB_G128, k)
    x, r = _dev(half(18, m, k)), _dev(half(19, m, n // 2))
    y0 = T.linear(W, x, act="silu", gated=True, residual=r)
    assert torch.equal(y0, T.linear(W, x, act="silu", gated=True, residual=r, static_weights=True))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1 = T.linear(W, x, act="silu", gated=True, residual=r)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y0, y1)
    g = torch.cuda.CUDAGraph()
    yg = torch.empty_like(y0)
    with torch.cuda.graph(g):
        T.linear(W, x, act="silu", gated=True, residual=r, y=yg)
    for _ in range(3):
        yg.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y0, yg)
    x.copy_(_dev(half(20, m, k)))  # new inputs in the captured buffers
    g.replay()
    assert torch.equal(yg, T.linear(W, x, act="silu", gated=True, residual=r))


@pytest.mark.parametrize("static", [False, True])
def test_dependent_chain_of_layers(static):
    # each layer reads what the one before writes; launched back to back
    d, f = 512, 768
    mats = []
    for i in range(4):
        gc, gs, gw = weights(T.Q2_0_G128, 2 * f, d, 30 + i)
        dc, ds, dw = weights(T.T3_5PB_G128, d, f, 40 + i)
        mats.append((_matrix(gc, gs, T.Q2_0_G128, d), gw, _matrix(dc, ds, T.T3_5PB_G128, f), dw))
    x = half(50, 2, d)
    h = _dev(x)
    for G, _, D, _ in mats:
        u = T.linear(G, h, act="silu", gated=True, static_weights=static)
        T.linear(D, u, residual=h, y=h, static_weights=static)
    got = h.cpu().numpy()
    ref = _dev(x)
    for G, _, D, _ in mats:
        torch.cuda.synchronize()
        u = T.linear(G, ref, act="silu", gated=True)
        torch.cuda.synchronize()
        ref = T.linear(D, u, residual=ref)
    assert np.array_equal(got, ref.cpu().numpy())


def test_far_offsets():
    # codes and outputs past 2^31 bytes / elements: the last rows are read from and written to the right place
    n, k, m = 2_200_000, 4096, 1
    W = T.empty_matrix(T.Q2_0_G128, n, k)
    W.codes.zero_()
    W.codes[-1].fill_(0x55)  # every t = +1
    W.codes[n // 2 + 3].fill_(0xFF)  # every t = -1
    W.scales[:, :k // 128] = 0.25
    x = torch.ones(m, k, dtype=torch.float16, device="cuda")
    y = T.linear(W, x)
    assert y[0, -1].item() == k * 0.25 and y[0, n // 2 + 3].item() == -k * 0.25
    assert int((y != 0).sum()) == 2
    y = T.linear(W, x.expand(20, k).contiguous())
    assert (y[:, -1] == k * 0.25).all() and (y[:, n // 2 + 3] == -k * 0.25).all() and int((y != 0).sum()) == 40


def test_refused_operands():
    codes, s, _ = weights(T.Q2_0_G128, 32, 256, 60)
    W = _matrix(codes, s, T.Q2_0_G128, 256)
    x = torch.zeros(2, 256, dtype=torch.float16, device="cuda")
    for bad in (dict(x=x.float()), dict(x=x[:, :128]), dict(x=x.cpu()), dict(bias=x[0, :31]), dict(act="tanh"),
                dict(residual=x), dict(y=torch.empty(2, 32, device="cuda")), dict(preact=x),
                dict(y=torch.empty(2, 64, dtype=torch.float16, device="cuda")[:, ::2]), dict(x=x[None])):
        with pytest.raises(ValueError):
            T.linear(W, **{"x": x, **bad})
    with pytest.raises(T.TernError):
        T.linear(W, x[:0])
    codes, s, _ = weights(T.Q2_0_G128, 33, 256, 60)
    with pytest.raises(T.TernError):
        T.linear(_matrix(codes, s, T.Q2_0_G128, 256), x, gated=True)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [1, 7, 40, 200])
@pytest.mark.parametrize("gated", [False, True])
def test_extreme_scales(layout, m, gated):
    # scales near fp16's largest value (twice them does not fit) and in its subnormal range, side by side
    n, k = 300, 384
    codes, s, w = weights(layout, n, k, 70)
    t = np.sign(w)
    s[:] = np.float16(2.0 ** -16)
    s[5, 1], s[17, 0], s[n // 2 + 5, 2], s[n - 1, 2] = 65504.0, 40000.0, -33000.0, 32768.0
    s[20, 0], s[21, 1] = np.float16(2.0 ** -24), np.float16(3 * 2.0 ** -24)
    w = t * np.repeat(s.astype(np.float64), 128, axis=1)
    x = half(71, m, k, scale=2.0 ** -10)
    for rows in (slice(0, m),):
        y = T.linear(_matrix(codes, s, layout, k), _dev(x[rows]), act="relu" if gated else "none", gated=gated).cpu().numpy()
        args = (w, f64(x[rows]), None, "relu" if gated else "none", gated)
        want, bound = L.linear(*args), L.linear_bound(*args)
        fits = np.abs(want) < 65000
        check(np.where(fits, y, 0), np.where(fits, want, 0), bound, "extreme scales")
        assert np.isinf(y[~fits]).all() or fits.all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,k", [(1000, 2176), (2500, 1664), (8100, 1152), (72, 17408)])
@pytest.mark.parametrize("m", [17, 48, 100, 191])
def test_sums_shared_by_several_pairs(layout, n, k, m):
    # few tiles with long rows: two or four pairs of blocks take a part of the sum each
    _check(layout, m, n, k, act="gelu", bias=True, residual=True)
    _check(layout, m, n, k, act="silu", gated=True, preact=True)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [20, 90])
def test_extreme_scale_in_one_part_of_the_sum(layout, m):
    # only the blocks that meet the scale know of it; whoever finishes the output has to learn it
    n, k = 300, 2304
    codes, s, w = weights(layout, n, k, 74)
    s[:] = np.float16(2.0 ** -16)
    s[3, 0], s[140, 9], s[n - 1, 17] = 65504.0, -40000.0, 32768.0
    w = np.sign(w) * np.repeat(s.astype(np.float64), 128, axis=1)
    x = half(75, m, k, scale=2.0 ** -10)
    y = T.linear(_matrix(codes, s, layout, k), _dev(x)).cpu().numpy()
    want, bound = L.linear(w, f64(x), None, "none", False), L.linear_bound(w, f64(x), None, "none", False)
    fits = np.abs(want) < 65000
    check(np.where(fits, y, 0), np.where(fits, want, 0), bound, "one extreme scale")
    assert np.isinf(y[~fits]).all() or fits.all()


@pytest.mark.parametrize("m", [30, 150])
def test_shared_sums_repeat_in_graphs(m):
    W, _, x, _, r = _case(T.T3_5PB_G128, m, 1500, 2560, "none", False, False, True)
    x, r = _dev(x), _dev(r)
    want = T.linear(W, x, residual=r)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=other):
        ys = [T.linear(W, x, residual=r) for _ in range(3)]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,m", [(2500, 1), (9700, 1), (9700, 2)])
def test_one_and_two_rows_on_many_outputs(layout, n, m):
    # large matrices take other forms of the product than small ones
    _check(layout, m, n, 640, act="silu", bias=True, residual=True, preact=True)
    _check(layout, m, 2 * n, 1152, act="gelu", gated=True)
    k = 384
    codes, s, w = weights(layout, n, k, 80)
    W = _matrix(codes, s, layout, k)
    x = half(81, m, k, scale=1e-2)
    x[np.arange(m), np.arange(m) * 37 + 5] = 60000.0  # one huge activation beside tiny ones
    check(T.linear(W, _dev(x)).cpu().numpy(), L.linear(w, f64(x)), L.linear_bound(w, f64(x)), "wide range")
    x = half(82, m, k)
    x[0, 5] = np.inf
    if m > 1:
        x[1, k - 1] = np.nan
    y = T.linear(W, _dev(x)).cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        want = np.stack([(f64(x)[i] * w).sum(1) for i in range(m)])
    assert np.array_equal(np.isnan(y), np.isnan(want)) and np.array_equal(y[np.isinf(want)], want[np.isinf(want)])
    codes, s, w = weights(layout, n, k, 83, scale=1.0)
    x = np.random.default_rng(84).integers(-1, 2, size=(m, k)).astype(np.float16)
    y = T.linear(_matrix(codes, s, layout, k), _dev(x)).cpu().numpy()
    assert np.array_equal(y.astype(np.float64), f64(x) @ w.T)
    # scales whose double does not fit fp16 and subnormal ones
    s[:] = np.float16(2.0 ** -16)
    s[7, 0], s[n - 1, 2], s[n // 2, 1], s[20, 1] = 65504.0, -33000.0, 40000.0, np.float16(2.0 ** -24)
    w = np.sign(w) * np.repeat(s.astype(np.float64), 128, axis=1)
    x = half(85, m, k, scale=2.0 ** -10)
    y, want = T.linear(_matrix(codes, s, layout, k), _dev(x)).cpu().numpy(), L.linear(w, f64(x))
    fits = np.abs(want) < 65000
    check(np.where(fits, y, 0), np.where(fits, want, 0), L.linear_bound(w, f64(x)), "extreme scales")
