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


# ----------------------------------------- values far above those that count
def _check(c, out, scale, dtype):
    """Case.check of `out`, with what falls below FP16's normal numbers counted
    from the largest probability times row scale that the query itself sees,
    and not from the largest row scale of the sequence.  (Where it lies within
    2^10 of that, that one counts.)"""
    cache, group, m, out = c.cache, c.heads // c.kv, c.m, _f64(out)
    for b in range(len(c.lens)):
        at = slice(b * m, (b + 1) * m)
        sees = c.sees(b)
        some = sees.any(0)
        k, _ = c.rows((cache.k_codes, cache.k_scales, cache.k_row_scale), b)
        v, vs = c.rows((cache.v_codes, cache.v_scales, cache.v_row_scale), b)
        for h in range(c.heads):
            kk, vv, vss = k[h // group][some], v[h // group][some], np.abs(vs[h // group][some])
            q = _f64(c.q[at, h])
            if c.rht:
                q = R.rotate(q, SEED)
            s = np.where(sees[:, some], (q @ kk.T) * scale, -np.inf)
            top = (np.exp(s - s.max(-1, keepdims=True)) * vss).max(-1, keepdims=True) * 448 * R.QMAX[c.grid]
            o, _, tol, _ = R.attn(q, kk, vv, None, sees[:, some], scale, c.q.dtype is BF and not c.rht, dtype is FP,
                                  top * 2 ** 10, c.dim)
            if c.rht:
                spread = lambda t: np.repeat(t.reshape(m, -1, 16).sum(-1) / 4, 16, -1)  # noqa: E731
                tol = spread(tol + 8 * R.U24 * np.abs(o))
                o = R.rotate(o, SEED, back=True)
            tol = tol + R.half_step(dtype) * (np.abs(o) + tol) + 1e-40
            bad = ~(np.abs(out[at, h] - o) <= tol)
            assert not bad.any(), (b, h, np.argwhere(bad)[:4], out[at, h][bad][:4], o[bad][:4], tol[bad][:4])


def _put(c, b, j, k=None, v=None):
    """Writes the key or value of position j of sequence b again (the other as it was drawn)."""
    g = np.random.default_rng([b, j])
    kv = [g.standard_normal((1, c.kv, c.dim)).astype(np.float32) if x is None else
          np.broadcast_to(np.asarray(x, np.float32), (1, c.kv, c.dim)).copy() for x in (k, v)]
    at = int(c.table[b, j // c.page]) * c.page + j % c.page
    c.U.ufp4_cache_append(torch.from_numpy(kv[0]).cuda(), torch.from_numpy(kv[1]).cuda(),
                          torch.tensor([at], device="cuda"), c.cache)


@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 40, 2.0 ** 100, 3e38])
@pytest.mark.parametrize("heads", [4, 16])         # (12 and 48 queries a head of the cache)
@pytest.mark.parametrize("rht,out", [(False, FP), (False, BF), (True, BF)])
def test_large_values_that_a_query_does_not_see(U, size, heads, rht, out):  # noqa: F811
    """A drafted token's values, far above all others, count for the queries
    that see it and for no other."""
    if rht and size > 1e37:
        size = 1e37                                # (16 of them are added in the rotation)
    g = np.random.default_rng(32)
    mask = _tree(g, 2, 6)
    c = Case(U, g, [300, 40], 6, heads, 2, 64, 16, 1, rht, FP, mask=mask)
    _put(c, 0, 300 - 6 + 1, v=g.choice([-1.0, 1.0], (c.kv, c.dim)) * size)
    _put(c, 1, 40 - 6 + 2, v=g.choice([-1.0, 1.0], (c.kv, c.dim)) * size)
    scale = 0.125
    _check(c, U.ufp4_cache_attn(**c.args(), dtype=out, scale=scale), scale, out)


@pytest.mark.parametrize("size", [2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("where", [0, 150, 399])
@pytest.mark.parametrize("heads", [2, 24])
@pytest.mark.parametrize("out", [FP, BF])
@pytest.mark.parametrize("dim", [64, 128])
def test_large_values_of_no_probability(U, size, where, heads, out, dim):  # noqa: F811
    """One row of values far above all others, at a score that leaves it nothing."""
    g = np.random.default_rng(33)
    c = Case(U, g, [400, 1000], 1, heads, 1, dim, 16, 0, False, FP)
    c.q[..., 0] = 16.0
    for b in range(2):
        _put(c, b, where, k=np.eye(dim)[0] * -100.0, v=g.choice([-1.0, 1.0], (1, dim)) * size)
    scale = 0.125                                  # (a score of -200)
    _check(c, U.ufp4_cache_attn(**c.args(), dtype=out, scale=scale), scale, out)


@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -60])
@pytest.mark.parametrize("where", [0, 150, 399])
@pytest.mark.parametrize("heads", [2, 24])
@pytest.mark.parametrize("out", [FP, BF])
def test_small_values_of_all_probability(U, size, where, heads, out):  # noqa: F811
    """The key with nearly all of the probability has values far below the others'."""
    g = np.random.default_rng(34)
    c = Case(U, g, [400, 1000], 1, heads, 1, 64, 16, 1, False, FP)
    c.q[..., 0] = 16.0
    for b in range(2):
        _put(c, b, where, k=np.eye(64)[0] * 8.0, v=g.standard_normal((1, 64)) * size)
    scale = 1.0                                    # (a score of 128, the others' below some 80)
    _check(c, U.ufp4_cache_attn(**c.args(), dtype=out, scale=scale), scale, out)


@pytest.mark.parametrize("size", [1e-30, 1e-36, 1e30, 1e37])
@pytest.mark.parametrize("heads", [2, 24])
@pytest.mark.parametrize("lens", [[300, 64], [40000, 3]])
def test_values_at_the_ends_of_fp32(U, size, heads, lens):  # noqa: F811
    g = np.random.default_rng(35)
    c = Case(U, g, lens, 1, heads, 1, 64, 64, 1, False, FP)
    k = torch.from_numpy(c.k).cuda()
    v = torch.from_numpy(c.v * np.float32(size / 8)).cuda()
    slots = torch.cat([torch.from_numpy(c.table[b, np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64)
                       for b, n in enumerate(lens)]).cuda()
    U.ufp4_cache_append(k, v, slots, c.cache)
    c.check(*U.ufp4_cache_attn(**c.args(), lse=True), dtype=FP)


@pytest.mark.parametrize("size", [1e-36, 1e-28, 1e-20, 1e20, 1e32, 1e35, 1e37])
@pytest.mark.parametrize("heads", [2, 24])
@pytest.mark.parametrize("grid", [0, 1])
@pytest.mark.parametrize("by", ["queries", "scale"])
def test_keys_at_the_ends_of_fp32(U, size, heads, grid, by):  # noqa: F811
    """Keys far from 1, the queries or the scale as far on the other side: ordinary scores."""
    g = np.random.default_rng(36)
    c = Case(U, g, [300, 64], 1, heads, 1, 64, 64, grid, False, FP)
    k = torch.from_numpy(c.k * np.float32(size / 8)).cuda()
    slots = torch.cat([torch.from_numpy(c.table[b, np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64)
                       for b, n in enumerate(c.lens)]).cuda()
    U.ufp4_cache_append(k, torch.from_numpy(c.v).cuda(), slots, c.cache)
    scale = 0.125
    if by == "queries":
        c.q *= np.float32(1 / size)
    else:
        scale = float(np.float32(0.125 / size))
    c.check(*U.ufp4_cache_attn(**c.args(), lse=True, scale=scale), scale=scale, dtype=FP)


@pytest.mark.parametrize("scale", [1e4, 1e8, 1e12])
@pytest.mark.parametrize("size", [2.0 ** -40, 2.0 ** 30])
@pytest.mark.parametrize("heads", [2, 24])
@pytest.mark.parametrize("out", [FP, BF])
@pytest.mark.parametrize("spread", [0, 20])
def test_scores_so_large_that_one_key_has_all(U, scale, size, heads, out, spread):  # noqa: F811
    """Scores beside which the scales' exponents vanish in fp32: the result is
    the values of the key with the largest score (of orthogonal keys here, so
    that it is the same key in any precision).  Its probability is 1, its weight
    within half a step of FP16 (2^-12; two values: 2^-22) of its row's scale."""
    g = np.random.default_rng(37)
    c = Case(U, g, [200, 70], 1, heads, 1, 64, 16, 1, False, FP)
    c.q.zero_()
    for h in range(heads):
        c.q[:, h, h % 4] = 4.0
    for b, n in enumerate(c.lens):
        for j in range(n):
            _put(c, b, j, k=np.eye(64)[j % 4] * (j + 1),
                 v=g.standard_normal((1, 64)) * size * 2.0 ** g.integers(-spread, spread + 1))
    o = _f64(U.ufp4_cache_attn(**c.args(), dtype=out, scale=scale))
    for b, n in enumerate(c.lens):
        v, _ = c.rows((c.cache.v_codes, c.cache.v_scales, c.cache.v_row_scale), b)
        for h in range(heads):
            want = v[0, max(j for j in range(n) if j % 4 == h % 4)]
            assert np.all(np.abs(o[b, h] - want) <= (2.0 ** -20 if out is FP else 2.0 ** -8 + 2.0 ** -11) * np.abs(want)), (b, h)
