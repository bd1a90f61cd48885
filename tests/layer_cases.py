"""Shared helpers of the layer-operator tests: seeded operands, and the elementwise bound check."""
from __future__ import annotations

import numpy as np

import oracle as O
from gemm_tern_gemv_b200 import synth
from tests.gpu_cases import pack_rows

GUARD = 64  # elements kept on both sides of a guarded output


def weights(layout, n, k, seed, scale=None):
    """(codes uint8, scales fp16, dense fp64 w [n][k])."""
    t = synth.codes_for(layout, n, k, seed)
    s = synth.group_scales(n, k // 128, seed) if scale is None else np.full((n, k // 128), scale, np.float16)
    return pack_rows(t, layout), s, O.dequantize(t, s).astype(np.float64)


def half(seed, *shape, scale=1.0):
    return (np.random.default_rng(seed).standard_normal(shape) * scale).astype(np.float16)


def f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def check(got, want, bound, what):
    """Asserts |got - want| <= bound elementwise; returns the worst ratio."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    ratio = np.abs(got - want) / bound
    worst = float(ratio.max()) if ratio.size else 0.0
    if worst > 1.0:
        i = np.unravel_index(int(ratio.argmax()), ratio.shape)
        raise AssertionError(f"{what}: {worst:.3g} times the bound at {i}: {got[i]!r}, exact {want[i]!r}, bound {bound[i]!r}")
    return worst


def guarded(torch, shape, dtype, fill):
    """(whole buffer, view of `shape` inside it): GUARD elements of `fill` before and after the view."""
    size = int(np.prod(shape))
    whole = torch.full((size + 2 * GUARD,), fill, dtype=dtype, device="cuda")
    return whole, whole[GUARD:GUARD + size].view(*shape)


def guards_kept(whole, fill):
    return bool((whole[:GUARD] == fill).all()) and bool((whole[-GUARD:] == fill).all())
