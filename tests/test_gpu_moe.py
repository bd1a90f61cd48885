"""GPU parity of the mixture-of-experts layer (T.moe) against the fp64 oracle, within derived bounds."""
import numpy as np
import pytest

from oracle import layer_oracle as L
from tests.layer_cases import check, f64, guarded, guards_kept, half, weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gemm_tern_gemv_b200 as T  # noqa: E402

LAYOUTS = [T.Q2_0_G128, T.T3_5PB_G128, T.Q1_0_G128]


def _dev(a):
    return None if a is None else torch.from_numpy(a).cuda()


class Layer:
    def __init__(self, layout, d, f, experts, seed=0, down_layout=None):
        self.d, self.f, self.experts = d, f, experts
        gc, gs, gw = weights(layout, experts * 2 * f, d, seed + d)
        dc, ds, dw = weights(down_layout or layout, experts * d, f, seed + f + 1)
        self.G = T.from_packed(_dev(gc), _dev(gs), layout, d)
        self.D = T.from_packed(_dev(dc), _dev(ds), down_layout or layout, f)
        self.gw, self.dw = gw.reshape(experts, 2 * f, d), dw.reshape(experts, d, f)
        self.r = half(seed + 2, experts, d, scale=1.5 / np.sqrt(d))

    def check(self, x, top_k, act="silu", renorm=True, residual=None, what=""):
        t = x.shape[0]
        ybuf, y = guarded(torch, (t, self.d), torch.float16, 777.0)
        out, w, ids = T.moe(self.G, self.D, _dev(self.r), _dev(x), top_k, act=act, renormalize=renorm, residual=_dev(residual),
                            y=y, return_routing=True)
        torch.cuda.synchronize()
        assert out is y
        args = (self.gw, self.dw, f64(self.r), f64(x), top_k, act, renorm, f64(residual))
        want, ww, wi = L.moe(*args)
        assert np.array_equal(ids.cpu().numpy(), wi), what
        check(w.cpu().numpy(), ww, (16 + self.experts) * L.HALF_F32 * np.maximum(ww, 1e-30), what + " weights")
        check(y.cpu().numpy(), want, L.moe_bound(*args), what)
        assert guards_kept(ybuf, 777.0), what


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 8, 16, 17, 33, 64])
def test_tokens(layout, tokens):
    Layer(layout, 256, 384, 8).check(half(tokens, tokens, 256), 2, residual=half(9, tokens, 256))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("d,f,experts,top_k", [(128, 128, 1, 1), (128, 256, 3, 3), (384, 128, 5, 2), (640, 896, 4, 1),
                                               (256, 640, 40, 8), (128, 128, 256, 16), (1152, 128, 6, 6), (128, 2176, 2, 1)])
@pytest.mark.parametrize("tokens", [1, 7, 20])
def test_shapes(layout, d, f, experts, top_k, tokens):
    Layer(layout, d, f, experts, seed=3).check(half(tokens, tokens, d), top_k, renorm=tokens != 7)


@pytest.mark.parametrize("act", L.ACTS)
def test_activations(act):
    Layer(T.Q2_0_G128, 256, 256, 4, seed=5).check(half(1, 6, 256, scale=2.0), 2, act=act)


@pytest.mark.parametrize("up,down", [(T.Q2_0_G128, T.T3_5PB_G128), (T.T3_5PB_G128, T.Q1_0_G128), (T.Q1_0_G128, T.Q2_0_G128)])
def test_mixed_layouts(up, down):
    Layer(up, 384, 256, 6, seed=7, down_layout=down).check(half(2, 9, 384), 3)


@pytest.mark.parametrize("tokens", [1, 4, 64])
def test_every_token_to_the_same_experts(tokens):
    lay = Layer(T.Q2_0_G128, 256, 256, 16, seed=8)
    x = half(3, tokens, 256)
    x[:, 0] = 20.0
    lay.r[:, 0] = 0
    lay.r[5, 0], lay.r[11, 0] = 2.0, 3.0
    lay.check(x, 2, what="one pair of experts")


def test_ties_go_to_the_lower_index():
    lay = Layer(T.Q2_0_G128, 128, 128, 12, seed=9)
    lay.r[:] = lay.r[0]  # every logit equal
    lay.check(half(4, 5, 128), 4, what="all equal")
    lay.r[3] = lay.r[7] = lay.r[0] * np.float16(2)  # exact doubles of it
    lay.check(half(5, 5, 128), 3, what="pairs")


def test_wide_activations_do_not_overflow_between_the_products():
    # act(gate) * up beyond fp16's range, brought back by small down scales
    lay = Layer(T.Q2_0_G128, 256, 256, 4, seed=10)
    lay.D.scales[:, :2] = 2.0 ** -13
    lay.dw = np.sign(lay.dw) * 2.0 ** -13
    x = half(6, 3, 256, scale=300.0)
    for t in (1, 3):
        _, w, ids = T.moe(lay.G, lay.D, _dev(lay.r), _dev(x[:t]), 2, return_routing=True)
        lay.check(x[:t], 2, what=f"{t} wide tokens")


@pytest.mark.parametrize("tokens", [1, 6])
def test_nan_token_stays_alone(tokens):
    lay = Layer(T.T3_5PB_G128, 256, 128, 6, seed=11)
    x = half(7, tokens, 256)
    x[0, 3] = np.nan
    y, w, ids = T.moe(lay.G, lay.D, _dev(lay.r), _dev(x), 2, return_routing=True)
    assert torch.isnan(y[0]).all() and torch.isnan(w[0]).all()
    i = ids[0].cpu().numpy()
    assert ((i >= 0) & (i < 6)).all() and len(set(i.tolist())) == 2
    assert torch.isfinite(y[1:]).all() and torch.isfinite(w[1:]).all()
    if tokens > 1:
        z, _, _ = T.moe(lay.G, lay.D, _dev(lay.r), _dev(x[1:]), 2, return_routing=True)
        want = L.moe(lay.gw, lay.dw, f64(lay.r), f64(x[1:]), 2)[0]
        check(y[1:].cpu().numpy(), want, L.moe_bound(lay.gw, lay.dw, f64(lay.r), f64(x[1:]), 2), "beside a NaN token")


@pytest.mark.parametrize("tokens", [1, 12])
def test_in_place_residual_workspace_and_graph(tokens):
    lay = Layer(T.Q2_0_G128, 256, 256, 8, seed=12)
    x, r = _dev(half(8, tokens, 256)), _dev(lay.r)
    want = T.moe(lay.G, lay.D, r, x, 2, residual=x)
    ws = torch.full((T.moe_workspace_bytes(lay.G, lay.D, r, tokens, 2),), 0xFF, dtype=torch.uint8, device="cuda")
    h = x.clone()
    T.moe(lay.G, lay.D, r, h, 2, residual=h, y=h, workspace=ws)
    assert torch.equal(h, want)
    # two graphs over one workspace, replayed in turn on one stream
    graphs, outs, ins = [], [], [x.clone(), _dev(half(9, tokens, 256))]
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        y = torch.empty_like(x)
        with torch.cuda.graph(g):
            T.moe(lay.G, lay.D, r, ins[i], 2, y=y, workspace=ws)
        graphs.append(g)
        outs.append(y)
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], T.moe(lay.G, lay.D, r, ins[i], 2))


def test_unused_experts_are_not_read():
    lay = Layer(T.Q2_0_G128, 128, 128, 8, seed=13)
    x = half(10, 2, 128)
    _, _, ids = T.moe(lay.G, lay.D, _dev(lay.r), _dev(x), 2, return_routing=True)
    want = T.moe(lay.G, lay.D, _dev(lay.r), _dev(x), 2)
    for e in set(range(8)) - set(ids.flatten().tolist()):
        lay.G.scales[e * 256:(e + 1) * 256] = float("nan")
        lay.D.scales[e * 128:(e + 1) * 128] = float("nan")
    assert torch.equal(want, T.moe(lay.G, lay.D, _dev(lay.r), _dev(x), 2))


def test_refused_operands():
    lay = Layer(T.Q2_0_G128, 128, 128, 4, seed=14)
    x, r = torch.zeros(2, 128, dtype=torch.float16, device="cuda"), _dev(lay.r)
    for kw in (dict(x=x.float()), dict(x=x[0]), dict(router=r[:, :64]), dict(router=r.cpu()), dict(act="x"),
               dict(residual=x[:1]), dict(y=x.float()), dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            T.moe(**{"gate_up": lay.G, "down": lay.D, "router": r, "x": x, "top_k": 2, **kw})
    for kw in (dict(top_k=0), dict(top_k=5), dict(router=r[:3]), dict(x=torch.zeros(65, 128, dtype=torch.float16, device="cuda")),
               dict(x=x[:0]), dict(down=lay.G), dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(T.TernError):
            T.moe(**{"gate_up": lay.G, "down": lay.D, "router": r, "x": x, "top_k": 2, **kw})


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("tokens,f", [(2, 16384), (20, 6400), (40, 12416)])
def test_long_down_rows(layout, tokens, f):
    # down products whose K is cut into slices
    Layer(layout, 128, f, 2, seed=15).check(half(11, tokens, 128), 1, residual=half(12, tokens, 128))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("tokens,experts,top_k", [(2, 3, 3), (5, 40, 8), (16, 16, 2), (40, 64, 2), (64, 200, 4), (9, 8, 4), (30, 6, 3)])
def test_pairs_per_expert(layout, tokens, experts, top_k):
    # from less than one pair for each expert to fifteen: every form of the product, and experts of many pairs in each
    lay = Layer(layout, 256, 384, experts, seed=60)
    x = half(tokens, tokens, 256)
    lay.check(x, top_k, residual=half(9, tokens, 256))
    lay.r[:] *= np.float16(0)
    lay.r[0] = 1  # one expert is taken by every token with a positive sum, the others by index
    lay.check(x, top_k)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_infinite_activations_of_some_tokens(layout):
    # pairs of tokens with and without infinities in the same experts
    lay = Layer(layout, 256, 384, 24, seed=61)
    x = half(62, 12, 256)
    want = T.moe(lay.G, lay.D, _dev(lay.r), _dev(x), 2)
    x[3, 7], x[8, 0] = np.inf, np.nan
    got = T.moe(lay.G, lay.D, _dev(lay.r), _dev(x), 2)
    rest = [i for i in range(12) if i not in (3, 8)]
    assert torch.equal(got[rest], want[rest]) and not torch.isfinite(got[[3, 8]]).all(1).any()
