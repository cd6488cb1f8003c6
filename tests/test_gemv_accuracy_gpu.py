"""The few-token products' error against 64-bit sums, as a whole, where tokens
are two FP16 values (fp32 or rotated ones, fp32 results)."""
import numpy as np
import pytest
import torch

from tests import serving_refs as R
from tests.test_gemv_gpu import BF, FP, SEED, U, _f64, _grouped, _values, _x  # noqa: F401

pytestmark = pytest.mark.gpu


# The second values' products do not pass through the sums of the first: 8
# additions to a chunk's sum, each losing half a unit of its last place (0.72 of
# 2^-23, on average over a binade) where it truncates, on sums that grow with the
# square root of the steps: 5.35 * 0.5 * 0.72 * 2^-23 = 2.3e-7 of the result.
BOUND = 2.3e-7


@pytest.mark.parametrize("tokens", [1, 4, 8, 13, 32])
@pytest.mark.parametrize("dtype,rht", [(FP, False), (FP, True), (BF, True)])
def test_two_values_a_token(U, tokens, dtype, rht):  # noqa: F811
    g = np.random.default_rng([tokens, int(rht)])
    w = torch.from_numpy(g.standard_normal((1024, 2048)).astype(np.float32)).cuda()
    for grid in (U.UFP4_E2M1, U.UFP4_E1M2):
        q = U.ufp4_quantize(w, grid, rht=rht, rht_seed=SEED)
        x = _x(g, (tokens, 2048), dtype)
        got = _f64(U.ufp4_gemv(x, q, rht=rht, rht_seed=SEED, dtype=FP))
        want, _ = R.gemv(_f64(x), _values(q, grid)[0], rht, SEED, 0.0)
        assert np.linalg.norm(got - want) <= BOUND * np.linalg.norm(want)


def test_two_values_a_token_by_expert(U):  # noqa: F811
    g = np.random.default_rng(5)
    q, v = _grouped(U, g, 4, 512, 1408, U.UFP4_E1M2, True)
    plan = U.ufp4_moe_sort(torch.from_numpy(g.integers(0, 4, size=(16, 2))).cuda(), 4)
    x = _x(g, (32, 1408), BF)
    got, off = _f64(U.ufp4_gemv_grouped(x, q, plan, 512, rht=True, rht_seed=SEED, dtype=FP)), plan.offsets.tolist()
    for e in range(4):
        want, _ = R.gemv(_f64(x[off[e]:off[e + 1]]), v[e], True, SEED, 0.0)
        assert np.linalg.norm(got[off[e]:off[e + 1]] - want) <= BOUND * np.linalg.norm(want)
