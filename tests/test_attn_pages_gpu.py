"""GPU parity of the attention over the 4-bit cache where a sequence's table
names pages outside the cache: their positions are rows of zeros, which count
in the softmax (score 0) and add nothing (bounds: tests/serving_refs.py)."""
import numpy as np
import pytest
import torch

from tests.test_attn_gpu import BF, FP, Case, U, _tree  # noqa: F401

pytestmark = pytest.mark.gpu


class Outside(Case):
    """Case with the pages `lost`, (sequence, place in its table), outside the cache."""

    def lose(self, lost, number):
        self.kept, self.lost = self.table.copy(), lost
        for b, p in lost:
            self.table[b, p] = number

    def rows(self, half, b):
        table, self.table = self.table, self.kept
        v, rs = super().rows(half, b)
        self.table = table
        v, rs = v.copy(), rs.copy()
        for c, p in self.lost:
            if c == b:
                v[:, p * self.page:(p + 1) * self.page] = 0
                rs[:, p * self.page:(p + 1) * self.page] = 0
        return v, rs


# A page of one 16-row half of a tile, first, middle and last (partly filled)
# ones, all of a sequence, the new tokens' own; split sequences.
CASES = [([70, 40], 1, 16, [(0, 1), (0, 4), (1, 2)]), ([70, 33], 3, 32, [(0, 0), (1, 1)]),
         ([100], 1, 64, [(0, 0), (0, 1)]), ([6000, 20], 2, 16, [(0, 0), (0, 77), (0, 374), (1, 0)]),
         ([129, 65], 6, 64, [(0, 1), (0, 2), (1, 1)])]


@pytest.mark.parametrize("lens,m,page,lost", CASES)
@pytest.mark.parametrize("heads", [2, 8, 48])
@pytest.mark.parametrize("dim,grid,rht,out", [(64, 1, False, FP), (128, 0, True, BF), (256, 1, True, FP)])
def test_pages_outside_the_cache_are_zeros(U, lens, m, page, lost, heads, dim, grid, rht, out):  # noqa: F811
    g = np.random.default_rng([sum(lens), m, heads, dim])
    c = Outside(U, g, lens, m, heads, 2, dim, page, grid, rht, FP, mask=_tree(g, len(lens), m) if m > 3 else None)
    for number in (-1, c.cache.pages, 2 ** 31 - 1, -2 ** 31):
        c.lose(lost, number)
        c.check(*U.ufp4_cache_attn(**c.args(), dtype=out, lse=True), dtype=out)
        c.table = c.kept
