"""The error of the attention's scores against 64-bit sums, as a whole, where
queries are two FP16 values (fp32 or rotated ones)."""
import numpy as np
import pytest
import torch

from tests import serving_refs as R
from tests.test_attn_gpu import BF, FP, SEED, Case, U, _f64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [8, 16, 64])
@pytest.mark.parametrize("dtype,rht", [(FP, False), (FP, True), (BF, True)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scores(U, group, dtype, rht, dim):  # noqa: F811
    """Sequences of one key, whose lse is the score.  The second values'
    products do not pass through the sums of the first: dim / 16 additions, each
    losing half a unit of the sum's last place (0.72 of 2^-23, on average over a
    binade) where it truncates, on sums that grow with the square root of the
    steps; and four roundings by factors, of 2^-25 each."""
    g = np.random.default_rng([group, dim, int(rht)])
    c = Case(U, g, [1] * 40, 1, 2 * group, 2, dim, 16, 1, rht, dtype, sizes=0)
    _, lse = U.ufp4_cache_attn(**c.args(), lse=True)
    want = np.zeros(lse.shape)
    for b in range(40):
        k, _ = c.rows((c.cache.k_codes, c.cache.k_scales, c.cache.k_row_scale), b)
        q = _f64(c.q[b]).reshape(2, group, dim)
        q = R.rotate(q, SEED) if rht else q
        want[b] = (np.einsum("hgd,hd->hg", q, k[:, 0]) * dim ** -0.5).reshape(-1)
    n = dim // 16
    bound = np.sqrt(np.arange(1, n + 1) / n).sum() * 0.5 * 0.72 * 2.0 ** -23 + 4 * 2.0 ** -25
    assert np.linalg.norm(_f64(lse) - want) <= bound * np.linalg.norm(want)
