"""fp64 oracle of the layer operators: fused linear layer, its backward, mixture of experts.

Plain numpy on dense weights w = s * t from `dequantize`; besides each result it returns the magnitudes
its error bounds are made of (see the bound functions)."""
from __future__ import annotations

import math

import numpy as np

GROUP = 128
_erf = np.vectorize(math.erf, otypes=[np.float64])
# half a unit in the last place relative to the value: rounding to fp16 / fp32 is off by at most this
HALF_F16, HALF_F32 = 2.0 ** -11, 2.0 ** -24
TINY_F16 = 2.0 ** -25  # half the smallest fp16 step, for results in the subnormal range

ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")
_A = math.sqrt(2 / math.pi)


def _sigmoid(z):
    return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))


def act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return np.maximum(z, 0)
    if name == "relu2":
        return np.maximum(z, 0) ** 2
    if name == "silu":
        return z * _sigmoid(z)
    if name == "gelu":
        return z * (1 + _erf(z / math.sqrt(2))) / 2
    assert name == "gelu_tanh"
    return z * (1 + np.tanh(_A * (z + 0.044715 * z ** 3))) / 2


def act_grad(name, z):
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "relu2":
        return 2 * np.maximum(z, 0)
    if name == "silu":
        s = _sigmoid(z)
        return s + z * s * (1 - s)
    if name == "gelu":
        return (1 + _erf(z / math.sqrt(2))) / 2 + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    assert name == "gelu_tanh"
    t = np.tanh(_A * (z + 0.044715 * z ** 3))
    return (1 + t) / 2 + z * (1 - t * t) / 2 * _A * (1 + 3 * 0.044715 * z * z)


def preact(w, x, bias=None):
    """z = x w^T + bias with x [m][k], w [n][k]."""
    z = x @ w.T
    return z if bias is None else z + bias


def linear(w, x, bias=None, name="none", gated=False, residual=None):
    z = preact(w, x, bias)
    f = z.shape[1] // 2
    y = act(name, z[:, :f]) * z[:, f:] if gated else act(name, z)
    return y if residual is None else y + residual


def linear_backward(w, dy, z, name="none", gated=False):
    """(dx, dz, dbias) from the stored z."""
    if gated:
        f = z.shape[1] // 2
        dz = np.concatenate([dy * z[:, f:] * act_grad(name, z[:, :f]), dy * act(name, z[:, :f])], axis=1)
    else:
        dz = dy * act_grad(name, z) if z is not None else dy
    return dz @ w, dz, dz.sum(0)


def route(logits, top_k, renormalize):
    """(weights, ids): the top_k largest logits of each row, ties to the lower index, softmax weights."""
    p = np.exp(logits - logits.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    w = np.take_along_axis(p, ids, 1)
    return (w / w.sum(1, keepdims=True) if renormalize else w), ids


def moe(gate_up, down, router, x, top_k, name="silu", renormalize=True, residual=None):
    """gate_up [e][2f][d], down [e][d][f], router [e][d], x [t][d] -> (y, weights, ids)."""
    weights, ids = route(x @ router.T, top_k, renormalize)
    y = np.zeros_like(x) if residual is None else residual.copy()
    for t in range(x.shape[0]):
        for j in range(top_k):
            e = ids[t, j]
            z = gate_up[e] @ x[t]
            f = z.shape[0] // 2
            y[t] += weights[t, j] * (down[e] @ (act(name, z[:f]) * z[f:]))
    return y, weights, ids


# ------------------------------------------------------------------------------------- error bounds
def product_bound(w, x, common=True):
    """Bound on a kernel's error of x w^T before rounding. Sums run in fp32: at most k / 16 + 64 dependent
    additions (tensor-core steps of 16, then the joining of partial sums), each off by at most one unit
    (2^-23, tensor cores may truncate) of a partial sum no larger than A = sum |w x|. `common`: where x is
    held as integers with a common exponent for 128 of them, each x is off by at most 2^-25 of the largest."""
    k = x.shape[1]
    a = np.abs(x) @ np.abs(w).T
    sums = 2.0 ** -23 * (k / 16 + 64) * a
    if not common:
        return sums
    top = np.repeat(np.abs(x).reshape(x.shape[0], k // GROUP, GROUP).max(2), GROUP, axis=1)
    return sums + 2.0 ** -25 * (top @ np.abs(w).T)


def _slope(name, z, dz):
    """Largest |act'| within dz of z: 1.13 bounds silu's, gelu's and its tanh form's derivative."""
    return 2 * (np.maximum(z, 0) + dz) if name == "relu2" else np.full_like(z, 1.0 if name in ("none", "relu") else 1.13)


def _linear_error(w, x, bias=None, name="none", gated=False, residual=None, common=True):
    """(y, bound on the error of y before its rounding): see linear_bound."""
    z = preact(w, x, bias)
    dz = product_bound(w, x, common) + 2 * HALF_F32 * np.abs(z)
    f = z.shape[1] // 2
    if gated:
        a, u = act(name, z[:, :f]), z[:, f:]
        da = _slope(name, z[:, :f], dz[:, :f]) * dz[:, :f] + 16 * HALF_F32 * np.abs(z[:, :f]) * np.maximum(1, np.abs(z[:, :f])
                                                                                             if name == "relu2" else 1)
        err = da * np.abs(u) + np.abs(a) * dz[:, f:] + da * dz[:, f:]
        y = a * u
    else:
        y = act(name, z)
        err = _slope(name, z, dz) * dz + 16 * HALF_F32 * np.maximum(np.abs(y), np.abs(z) if name != "relu2" else 0)
    if residual is not None:
        y = y + residual
        err = err + 2 * HALF_F32 * (np.abs(y) + np.abs(residual))
    return y, err


def linear_bound(w, x, bias=None, name="none", gated=False, residual=None, common=True):
    """Bound on |y - linear()| for an fp16 y: the product's error through the activation, 16 units of fp32
    for evaluating activation, bias, gate and residual, and one rounding to fp16."""
    y, err = _linear_error(w, x, bias, name, gated, residual, common)
    return err * (1 + HALF_F16) + HALF_F16 * np.abs(y) + TINY_F16


def preact_bound(w, x, bias=None):
    z = preact(w, x, bias)
    err = product_bound(w, x) + 2 * HALF_F32 * np.abs(z)
    return err * (1 + HALF_F16) + HALF_F16 * np.abs(z) + TINY_F16


def backward_bounds(w, dy, z, name="none", gated=False):
    """(dx, dz, dbias) bounds. dz: 32 units of fp32 for the derivative's terms (they are at most
    1.2 (1 + |z|) each, and may cancel), one rounding. dbias: the unrounded error summed, and m fp32
    additions. dx: the rounded dz through |w|, and the product's sums."""
    def term(a, g):  # error of g * act'(a), of g * act(a)
        if name == "none":
            return 4 * HALF_F32 * np.abs(g), 4 * HALF_F32 * np.abs(g * a)
        if name in ("relu", "relu2"):
            return 4 * HALF_F32 * np.abs(g * act_grad(name, a)), 4 * HALF_F32 * np.abs(g * act(name, a))
        return 32 * HALF_F32 * np.abs(g) * 1.2 * (1 + np.abs(a)), 32 * HALF_F32 * np.abs(g * a)
    dx, dzv, _ = linear_backward(w, dy, z, name, gated)
    if gated:
        f = z.shape[1] // 2
        e = np.concatenate([term(z[:, :f], dy * z[:, f:])[0], term(z[:, :f], dy)[1]], axis=1)
    else:
        e = term(z, dy)[0] if z is not None else np.zeros_like(dy)
    m, n = dzv.shape
    round_dz = HALF_F16 * np.abs(dzv) + TINY_F16 if (z is not None and (gated or name != "none")) else 0.0
    b_dz = e * (1 + HALF_F16) + round_dz
    b_db = e.sum(0) + HALF_F32 * (m + 4) * np.abs(dzv).sum(0)
    s = np.abs(dzv) @ np.abs(w)
    b_dx = (b_dz @ np.abs(w) if np.ndim(b_dz) else 0.0) + 2.0 ** -23 * (n / 16 + 64) * s
    return b_dx * (1 + HALF_F16) + HALF_F16 * np.abs(dx) + TINY_F16, b_dz + TINY_F16, b_db


def moe_bound(gate_up, down, router, x, top_k, name="silu", renormalize=True, residual=None, held=None):
    """Bound on |y - moe()|: each expert's h = act(gate) * up with its bound as in linear_bound, rounded to
    at most 11 bits for the second product (2^-11 |h|, with 2^-24 of the largest h of the row where a
    common exponent holds it), the product's sums, weights off by 16 units of fp32, one rounding.
    `held` says how h comes to the second product and leaves out what that does not do: "fp16" (times a power of two
    that brings the pair's largest to [2^14, 2^15): 2^-11 |h|, and 2^-25 of a scaled value, so 2^-39 of the largest)
    or "integers" (2^-27 of the largest)."""
    weights, ids = route(x @ router.T, top_k, renormalize)
    y, _, _ = moe(gate_up, down, router, x, top_k, name, renormalize, residual)
    err = np.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(top_k):
            g, dn = gate_up[ids[t, j]], down[ids[t, j]]
            f = dn.shape[1]
            h = linear(g, x[t:t + 1], None, name, True)
            if held is None:
                eh = linear_bound(g, x[t:t + 1], None, name, True) + 2.0 ** -24 * np.abs(h).max()  # holds the 2^-11 |h|
            else:
                eh = _linear_error(g, x[t:t + 1], None, name, True, None, False)[1]
                eh = eh * (1 + HALF_F16) + (HALF_F16 * np.abs(h) + 2.0 ** -39 * np.abs(h).max() if held == "fp16" else 2.0 ** -27 * np.abs(h).max())
            s = np.abs(h) @ np.abs(dn).T
            e = eh @ np.abs(dn).T + 2.0 ** -23 * (f / 16 + 64) * s
            err[t] += weights[t, j] * (e[0] + 18 * HALF_F32 * s[0])
    if residual is not None:
        err += 2 * HALF_F32 * (np.abs(residual) + np.abs(y))
    return err * (1 + HALF_F16) + HALF_F16 * np.abs(y) + TINY_F16
