"""The bounded waits of the attention for many queries, through the test-only
probe build of the library (tests/probe)."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_attn_gpu import BF, FP, Case
from tests.test_probe_gpu import _through, probe  # noqa: F401

pytestmark = pytest.mark.gpu


# One tile of keys, two, many, and sequences split over CTAs (joined by a
# second kernel, which then reads whatever the scratch holds).
@pytest.mark.parametrize("lens,m,heads,kv,extra", [([40], 32, 2, 2, 0), ([100, 0, 7], 9, 8, 2, 0),
                                                   ([700, 64], 6, 24, 2, 0), ([5000], 20, 2, 1, 900)])
@pytest.mark.parametrize("dim,out", [(64, BF), (128, FP)])
def test_a_wait_that_runs_out(probe, lens, m, heads, kv, extra, dim, out):  # noqa: F811
    """With a short budget (about a millisecond) and the MMA thread held on a
    barrier that nothing arrives on, the kernel gives up and returns;
    ufp4_check reports UFP4_ERR_TIMEOUT once and clears it; the next call is
    right.  Nothing faults: every role leaves its loop and the tensor memory
    is freed, or the next call's CTAs would not get theirs."""
    U, P = probe
    P.ufp4probe_attn_waits.argtypes = [ctypes.c_longlong, ctypes.c_int]
    P.ufp4probe_attn_waits.restype = None
    c = Case(U, np.random.default_rng(41), lens, m, heads, kv, dim, 16, 1, True, BF, extra=extra)
    want = U.ufp4_cache_attn(**c.args(), dtype=out, lse=True)
    with _through(U, P):
        assert U.ufp4_check() == U.UFP4_OK
        for _ in range(2):
            P.ufp4probe_attn_waits(2_000_000, 1)
            try:
                U.ufp4_cache_attn(**c.args(), dtype=out, lse=True)
                torch.cuda.synchronize()
            finally:
                P.ufp4probe_attn_waits(0, 0)
            assert U.ufp4_check() == U.UFP4_ERR_TIMEOUT
            assert U.ufp4_check() == U.UFP4_OK          # the flag was cleared
            got = U.ufp4_cache_attn(**c.args(), dtype=out, lse=True)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert U.ufp4_check() == U.UFP4_OK
