"""GPU parity of the few-token products near the lower end of fp32 (bounds:
tests/serving_refs.py, tests/test_gemv_gpu.py)."""
import numpy as np
import pytest
import torch

from tests.test_gemv_gpu import BF, FP, SEED, U, _check, _values, _x  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [1e-25, 1e-28, 1e-30, 1e-32, 1e-34])
@pytest.mark.parametrize("dtype,rht", [(FP, False), (FP, True), (BF, False), (BF, True)])
@pytest.mark.parametrize("tokens", [1, 11, 20])
def test_small_tokens(U, size, dtype, rht, tokens):  # noqa: F811
    """Tokens far below 1 with a model's weights: results that fp32 holds are
    as exact as others'."""
    g = np.random.default_rng(6)
    w = torch.from_numpy((g.standard_normal((64, 1040)) * 0.02).astype(np.float32)).cuda()
    x = (_x(g, (tokens, 1040), FP) * size).to(dtype)
    for grid in (U.UFP4_E2M1, U.UFP4_E1M2):
        q = U.ufp4_quantize(w, grid, rht=rht, rht_seed=SEED)
        _check(U.ufp4_gemv(x, q, rht=rht, rht_seed=SEED, dtype=FP), x, _values(q, grid)[0], rht, FP)
