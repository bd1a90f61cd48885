"""Layer operators: host-side checks of the C ABI and the oracle's own pins. No GPU needed: the rejected
calls return before any launch and their pointers are never dereferenced."""
import ctypes

import numpy as np
import pytest

import gemm_tern_gemv_b200 as T
from oracle import layer_oracle as L
from tests.layer_cases import f64, half, weights

FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    from gemm_tern_gemv_b200 import build
    build.build()
    return T.lib()


def _mat(**kw):
    d = dict(layout=1, n=64, k=1024, codes=FAKE, code_row_stride=256, scales=FAKE + 4096, scale_row_stride=8)
    d.update(kw)
    return T.TernMatrixC(d["layout"], d["n"], d["k"], d["codes"], d["code_row_stride"], d["scales"], d["scale_row_stride"])


def _p(v):
    return ctypes.c_void_p(v)


@pytest.mark.parametrize("kw,status", [(dict(layout=7), 2), (dict(n=0), 1), (dict(k=1000), 1), (dict(codes=0), 1),
                                       (dict(code_row_stride=128), 1), (dict(codes=FAKE + 8), 3), (dict(scale_row_stride=12), 3)])
def test_bad_matrix(lib, kw, status):
    m, ok = _mat(**kw), _mat()
    assert lib.tern_linear(m, _p(FAKE), 1, _p(FAKE), None, 0, None, None) == status
    assert lib.tern_linear_backward(m, _p(FAKE), None, 1, 0, 0, _p(FAKE), None, 0, None, None, None) == status
    for g, d in ((m, ok), (ok, m)):
        layer = T.TernMoeLayerC(ctypes.pointer(g), ctypes.pointer(d), FAKE, 4, 2, 3, 1)
        assert lib.tern_moe(layer, _p(FAKE), 1, None, _p(FAKE), None, None, _p(FAKE), 1 << 30, None) == status
        assert lib.tern_moe_workspace_bytes(layer, 1) == 0


def test_linear_rejects(lib):
    m = _mat()
    f = lambda x=FAKE, rows=1, y=FAKE, e=None, flags=0, status=None: lib.tern_linear(  # noqa: E731
        m, _p(x), rows, _p(y), e, flags, _p(status), None)
    assert f(x=0) == 1 and f(y=0) == 1 and f(rows=0) == 1 and f(rows=-3) == 1 and f(rows=1 << 31) == 1
    assert f(flags=2) == 1 and f(x=FAKE + 2) == 3 and f(y=FAKE + 1) == 3 and f(status=FAKE + 2) == 3
    E = T.TernEpilogueC
    assert f(e=E(6, 0, None, None, None)) == 2 and f(e=E(-1, 0, None, None, None)) == 2
    assert f(e=E(0, 2, None, None, None)) == 1
    for i in range(2, 5):
        args = [0, 0, None, None, None]
        args[i] = FAKE + 1
        assert f(e=E(*args)) == 3
    odd = _mat(n=63)
    assert lib.tern_linear(odd, _p(FAKE), 1, _p(FAKE), E(3, 1, None, None, None), 0, None, None) == 1
    assert lib.tern_linear(None, _p(FAKE), 1, _p(FAKE), None, 0, None, None) == 1


def test_linear_backward_rejects(lib):
    m = _mat()
    f = lambda dy=FAKE, z=FAKE, rows=1, act=3, gated=0, dx=FAKE, dz=FAKE, stride=64, db=FAKE, status=None: lib.tern_linear_backward(  # noqa: E731
        m, _p(dy), _p(z), rows, act, gated, _p(dx), _p(dz), stride, _p(db), _p(status), None)
    assert f(dy=0) == 1 and f(z=0) == 1 and f(rows=0) == 1 and f(gated=3) == 1 and f(act=9) == 2
    assert f(dx=0, dz=0, db=0) == 1 and f(dz=0) == 1  # dx needs dz once there is an activation
    assert f(act=0, dz=0, dy=FAKE + 2) == 3  # dz is dy: 16-byte aligned
    assert f(stride=56) == 1 and f(stride=68) == 3
    odd = _mat(n=63)
    assert lib.tern_linear_backward(odd, _p(FAKE), None, 1, 0, 0, _p(FAKE), None, 0, None, None, None) == 1  # rows of dy unaligned
    assert f(dz=FAKE + 8) == 3 and f(dx=FAKE + 1) == 3 and f(db=FAKE + 2) == 3 and f(z=FAKE + 1) == 3 and f(status=FAKE + 1) == 3


def test_moe_rejects_and_workspace(lib):
    d, f, e = 256, 384, 4
    g = _mat(n=e * 2 * f, k=d)
    dn = _mat(n=e * d, k=f)
    def layer(g=g, dn=dn, router=FAKE, experts=e, top_k=2, act=3, renorm=1):
        return T.TernMoeLayerC(ctypes.pointer(g), ctypes.pointer(dn), router, experts, top_k, act, renorm)
    def call(lay, x=FAKE, tokens=3, res=None, y=FAKE, w=None, ids=None, ws=FAKE, wsb=1 << 30):
        return lib.tern_moe(lay, _p(x), tokens, _p(res), _p(y), _p(w), _p(ids), _p(ws), wsb, None)
    for kw, st in ((dict(experts=0), 1), (dict(experts=5), 1), (dict(top_k=0), 1), (dict(top_k=5), 1), (dict(act=6), 2),
                   (dict(renorm=2), 1), (dict(g=_mat(n=e * 2 * f + 2, k=d)), 1), (dict(dn=_mat(n=e * d, k=d)), 1),
                   (dict(router=0), 1), (dict(router=FAKE + 2), 3)):
        assert call(layer(**kw)) == st, kw
    lay = layer()
    assert call(lay, x=0) == 1 and call(lay, y=0) == 1 and call(lay, tokens=0) == 1 and call(lay, tokens=65) == 2
    assert call(lay, x=FAKE + 8) == 3 and call(lay, y=FAKE + 1) == 3 and call(lay, w=FAKE + 2) == 3 and call(lay, ids=FAKE + 1) == 3
    assert call(lay, res=FAKE + 1) == 3
    need = lib.tern_moe_workspace_bytes(lay, 3)
    assert need > 0 and call(lay, ws=0) == 4 and call(lay, wsb=need - 1) == 4 and call(lay, ws=FAKE + 8) == 3
    assert lib.tern_moe_workspace_bytes(lay, 65) == 0 and lib.tern_moe_workspace_bytes(None, 1) == 0
    many = layer(g=_mat(n=300 * 2 * f, k=d), dn=_mat(n=300 * d, k=f), experts=300)
    assert call(many) == 2
    wide = layer(g=_mat(n=2 * 32896, k=d), dn=_mat(n=d, k=32896, code_row_stride=8224, scale_row_stride=264), experts=1, top_k=1)
    assert call(wide) == 2


def test_python_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    W = T.TernMatrix(1, 8, 128, torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 8, dtype=torch.float16))
    x = torch.zeros(1, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        T.linear(W, x)
    with pytest.raises(ValueError):
        T.linear_backward(W, torch.zeros(1, 8, dtype=torch.float16))
    with pytest.raises(ValueError):
        T.moe(W, W, x, x, 1)


# ---- the oracle's pins --------------------------------------------------------------------------
def test_activation_values():
    one = np.array([1.0])
    assert L.act("silu", one)[0] == pytest.approx(0.7310585786300049, rel=1e-15)  # 1 / (1 + e^-1)
    assert L.act("gelu", one)[0] == pytest.approx(0.8413447460685429, rel=1e-14)  # Phi(1)
    assert L.act("gelu_tanh", one)[0] == pytest.approx(0.8411919906082768, rel=1e-14)
    z = np.array([-3.0, 0.0, 2.0])
    assert L.act("relu", z).tolist() == [0, 0, 2] and L.act("relu2", z).tolist() == [0, 0, 4]
    assert L.act_grad("relu", z).tolist() == [0, 0, 1] and L.act_grad("relu2", z).tolist() == [0, 0, 4]


@pytest.mark.parametrize("name", L.ACTS)
def test_derivatives_by_differences(name):
    z = np.random.default_rng(1).standard_normal(200) * 3
    z = z[np.abs(z) > 1e-3]
    d = (L.act(name, z + 1e-5) - L.act(name, z - 1e-5)) / 2e-5
    assert np.allclose(d, L.act_grad(name, z), atol=1e-7)
    slope = L._slope(name, np.linspace(-12, 12, 20001), 0.0)
    assert (np.abs(L.act_grad(name, np.linspace(-12, 12, 20001))) <= slope + 1e-12).all()  # the bounds' slopes hold


def test_backward_by_differences():
    _, _, w = weights(1, 24, 128, 3)
    x, b = f64(half(1, 3, 128)), f64(half(2, 24))
    for gated in (False, True):
        dy = f64(half(3, 3, 12 if gated else 24))
        dx, dz, db = L.linear_backward(w, dy, L.preact(w, x, b), "silu", gated)
        f = lambda xx, bb: (dy * L.linear(w, xx, bb, "silu", gated)).sum()  # noqa: E731
        for i, j in ((0, 0), (2, 100)):
            e = np.zeros_like(x)
            e[i, j] = 1e-6
            assert (f(x + e, b) - f(x - e, b)) / 2e-6 == pytest.approx(dx[i, j], rel=1e-5, abs=1e-8)
        e = np.zeros_like(b)
        e[5] = 1e-6
        assert (f(x, b + e) - f(x, b - e)) / 2e-6 == pytest.approx(db[5], rel=1e-5, abs=1e-8)
        assert np.allclose(dz.sum(0), db)


def test_routing_ties_and_moe_by_hand():
    w, ids = L.route(np.array([[1.0, 2.0, 2.0, 0.0], [0.0, 0.0, 0.0, 0.0]]), 2, True)
    assert ids.tolist() == [[1, 2], [0, 1]] and np.allclose(w, 0.5)
    w, _ = L.route(np.zeros((1, 4)), 2, False)
    assert np.allclose(w, 0.25)
    # one expert of ones: h = relu(sum x) * sum x, y = f * h
    y, _, _ = L.moe(np.ones((1, 4, 3)), np.ones((1, 3, 2)), np.zeros((1, 3)), np.array([[1.0, 2.0, 3.0]]), 1, "relu", True)
    assert y.tolist() == [[72.0, 72.0, 72.0]]
