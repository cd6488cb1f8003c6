"""GPU parity of the attention over the 4-bit cache at the ends of its range:
queries and scales whose product leaves fp32, and rows of values far above
those that count for a query (bounds: tests/serving_refs.py)."""
import numpy as np
import pytest
import torch

from tests import serving_refs as R
from tests.test_attn_gpu import BF, FP, SEED, Case, U, _f64, _tree  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------ queries times small scales
# A query of zeros (padding, say) or a tiny one, times the scale: nothing that
# a query does not see may turn it into NaN.  heads: 4 and 24 queries a head of
# the cache, 12 and 72 with the three tokens.
@pytest.mark.parametrize("scale", [1e-9, -1e-9, 1e-12, 1e-30, 1e-38])
@pytest.mark.parametrize("heads", [4, 24])
@pytest.mark.parametrize("grid", [0, 1])
def test_queries_of_zeros_and_small_scales(U, scale, heads, grid):  # noqa: F811
    g = np.random.default_rng(31)
    c = Case(U, g, [77, 128, 5], 3, heads, 1, 64, 16, grid, False, FP)
    c.q[1] = 0
    c.q[3, 1::2] = 0
    c.q[4] *= 2.0 ** -100
    c.q[8, 0] *= 2.0 ** -120
    scale = float(np.float32(scale))
    c.check(*U.ufp4_cache_attn(**c.args(), lse=True, scale=scale), scale=scale, dtype=FP)
