"""The router of T.moe under small sizes, where its blocks reach one another's shared memory soonest."""
import numpy as np
import pytest

from oracle import layer_oracle as L
from tests.layer_cases import f64, half, weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gemm_tern_gemv_b200 as T  # noqa: E402


@pytest.mark.parametrize("experts,top_k", [(1, 1), (2, 1), (3, 3), (9, 2), (33, 4), (64, 8), (65, 8)])
@pytest.mark.parametrize("tokens", [1, 5, 20, 64])
def test_repeated_small_routings(experts, top_k, tokens):
    d, f = 128, 128
    packed = []
    for n, k in ((experts * 2 * f, d), (experts * d, f)):
        codes, s, _ = weights(T.Q2_0_G128, n, k, experts + n)
        packed.append(T.from_packed(torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda(), T.Q2_0_G128, k))
    router, x = half(1, experts, d, scale=0.2), half(tokens, tokens, d)
    want_w, want_ids = L.route(f64(x) @ f64(router).T, top_k, True)
    r, xd = torch.from_numpy(router).cuda(), torch.from_numpy(x).cuda()
    runs = [T.moe(*packed, r, xd, top_k, return_routing=True) for _ in range(60)]
    for y, w, ids in runs:
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert torch.equal(w, runs[0][1]) and torch.equal(y, runs[0][0])
    # fp32 exponentials, sums over the experts and a quotient: 16 + experts units of 2^-24
    assert (np.abs(f64(runs[0][1].cpu().numpy()) - want_w) <= (16 + experts) * L.HALF_F32 * np.maximum(want_w, 1e-30)).all()
