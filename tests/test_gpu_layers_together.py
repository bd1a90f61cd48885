"""The layer operators in a run, as a model uses them: each one's output is the next one's input, in one stream and
in a captured graph. Every stage is checked with the fp64 oracle on the input that it really got."""
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


def _np(t):
    return t.cpu().numpy().astype(np.float64)


class Block:
    """Output projection + residual, gated feed-forward + residual, mixture of experts + residual."""

    def __init__(self, layout, d=256, f=640, experts=6, seed=0):
        self.dense = {}
        for i, (name, n, k) in enumerate((("o", d, d), ("gu", 2 * f, d), ("dn", d, f), ("eg", experts * 256, d), ("ed", experts * d, 128))):
            codes, s, w = weights(layout, n, k, seed + i)
            setattr(self, name, T.from_packed(_dev(codes), _dev(s), layout, k))
            self.dense[name] = w
        self.router = half(seed + 9, experts, d, scale=1.5 / np.sqrt(d))
        self.router_dev = _dev(self.router)
        self.dense["eg"] = self.dense["eg"].reshape(experts, 256, d)
        self.dense["ed"] = self.dense["ed"].reshape(experts, d, 128)

    def run(self, attn, x):
        h = T.linear(self.o, attn, residual=x)
        g = T.linear(self.gu, h, act="silu", gated=True)
        y = T.linear(self.dn, g, residual=h)
        z, w, ids = T.moe(self.eg, self.ed, self.router_dev, y, 2, residual=y, return_routing=True)
        return h, g, y, z, w, ids

    def check(self, attn, x, outs, what):
        h, g, y, z, w, ids = outs
        for got, args in ((h, (self.dense["o"], _np(attn), None, "none", False, _np(x))),
                          (g, (self.dense["gu"], _np(h), None, "silu", True, None)),
                          (y, (self.dense["dn"], _np(g), None, "none", False, _np(h)))):
            check(got.cpu().numpy(), L.linear(*args), L.linear_bound(*args), what)
        args = (self.dense["eg"], self.dense["ed"], f64(self.router), _np(y), 2, "silu", True, _np(y))
        want, ww, wi = L.moe(*args)
        assert np.array_equal(ids.cpu().numpy(), wi), what
        check(z.cpu().numpy(), want, L.moe_bound(*args), what + " moe")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("tokens", [1, 2, 6, 40])
def test_block(layout, tokens):
    b = Block(layout)
    attn, x = _dev(half(1, tokens, 256)), _dev(half(2, tokens, 256))
    b.check(attn, x, b.run(attn, x), f"block layout {layout}, {tokens} tokens")


@pytest.mark.parametrize("tokens", [1, 6, 40])
def test_blocks_in_a_graph(tokens):
    # three blocks in a row, replayed on inputs that change; two such graphs take turns
    b = Block(T.T3_5PB_G128, seed=20)
    attn, x = _dev(half(3, tokens, 256)), _dev(half(4, tokens, 256))
    b.run(attn, x)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, v = [], x
            for _ in range(3):
                o.append(b.run(attn, v))
                v = o[-1][3]
        graphs.append(g)
        outs.append(o)
    for seed in (5, 6):
        attn.copy_(_dev(half(seed, tokens, 256)))
        x.copy_(_dev(half(seed + 10, tokens, 256)))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, c in zip(outs[0], outs[1]):
            assert all(torch.equal(p, q) for p, q in zip(a, c))
        v = x
        for i, o in enumerate(outs[0]):
            b.check(attn, v, o, f"graph, block {i}")
            v = o[3]


def test_two_streams_at_once():
    b, c = Block(T.Q2_0_G128, seed=30), Block(T.Q1_0_G128, seed=40)
    attn, x = _dev(half(7, 5, 256)), _dev(half(8, 5, 256))
    want = [b.run(attn, x)[3], c.run(attn, x)[3]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i, blk in enumerate((b, c)):
            with torch.cuda.stream(streams[i]):
                got[i].append(blk.run(attn, x)[3])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m", [3, 70])
def test_training_pass(layout, m):
    # a gated feed-forward's forward and backward with the stored preactivations
    d, f = 384, 520
    (cu, su, wu), (cd, sd, wd) = weights(layout, 2 * f, d, 50), weights(layout, d, 640, 51)
    up, down = T.from_packed(_dev(cu), _dev(su), layout, d), T.from_packed(_dev(cd), _dev(sd), layout, 640)
    x, bias, dy = _dev(half(52, m, d)), _dev(half(53, 2 * f, scale=0.3)), _dev(half(54, m, d))
    z1 = torch.empty((m, 2 * f), dtype=torch.float16, device="cuda")
    h = torch.zeros((m, 640), dtype=torch.float16, device="cuda")
    h[:, :f] = T.linear(up, x, bias=bias, act="silu", gated=True, preact=z1)
    y = T.linear(down, h, residual=x)
    dh, dz2, db2 = T.linear_backward(down, dy)
    dx, dz1, db1 = T.linear_backward(up, dh[:, :f], z1, act="silu", gated=True)
    torch.cuda.synchronize()
    args = (wd, _np(h), None, "none", False, _np(x))
    check(y.cpu().numpy(), L.linear(*args), L.linear_bound(*args), "y")
    for got, a in (((dh, dz2, db2), (wd, _np(dy), None, "none", False)), ((dx, dz1, db1), (wu, _np(dh)[:, :f], _np(z1), "silu", True))):
        for name, g, want, bound in zip(("dx", "dz", "dbias"), got, L.linear_backward(*a), L.backward_bounds(*a)):
            check(g.cpu().numpy(), want, bound, name)
    # the whole gradient of x against the formula's from x on: every rounding to fp16 on the way is off by at
    # most 2^-11, the sums of the three products at most 2^-20 of what they add up
    z = f64(x.cpu().numpy()) @ wu.T + f64(bias.cpu().numpy())
    whole, _, _ = L.linear_backward(wu, (f64(dy.cpu().numpy()) @ wd)[:, :f], z, "silu", True)
    size = (np.abs(f64(dy.cpu().numpy())) @ np.abs(wd))[:, :f]  # dh's terms
    zs = np.abs(f64(x.cpu().numpy())) @ np.abs(wu).T + np.abs(f64(bias.cpu().numpy()))  # and z's
    # |silu| <= |z|, |silu'| <= 1.1, |silu''| <= 0.5: d(dz) <= step (dh's (1.1 |u| + |g|) + |dh| z's (1 + 0.5 |u| + 1.1 + 1))
    step = 2.0 ** -11 + 2.0 ** -20
    part = size * (1.1 * zs[:, f:] + zs[:, :f]) + size * (zs[:, :f] * 0.5 * zs[:, f:] + 1.1 * zs[:, f:] + 1.1 * zs[:, :f])
    both = 2 * part + size * (1.1 * zs[:, f:] + zs[:, :f])  # and dz's own rounding
    bound = step * np.concatenate([both, both], 1) @ np.abs(wu) + 2.0 ** -11 * np.abs(whole) + 1e-6
    check(dx.cpu().numpy(), whole, bound, "gradient of the whole")
