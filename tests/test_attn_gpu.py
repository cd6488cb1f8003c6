"""GPU parity of the attention over the 4-bit cache against plain 64-bit sums
over what the cache's rows stand for (tests/serving_refs.py, which derives the
bounds)."""
import numpy as np
import pytest
import torch

from tests import serving_refs as R

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
SEED = 7


@pytest.fixture(scope="module")
def U():
    from fp4_quantized_numerics_gb300 import build, ufp4
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return ufp4


def _np(t):
    return t.detach().cpu().numpy()


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Case:
    """Sequences of lengths `lens` in scattered pages of a cache whose every
    other byte is 0xFF (scales that are NaN), m new tokens each."""

    def __init__(self, U, g, lens, m, heads, kv, dim, page, grid, rht, dtype, mask=None, extra=0, sizes=1):
        self.U, self.lens, self.m, self.heads, self.kv, self.dim, self.page = U, list(lens), m, heads, kv, dim, page
        self.grid, self.rht, batch = grid, rht, len(lens)
        width = max(-(-max(lens) // page), 1) + extra
        used = [-(-n // page) for n in lens]
        pages = sum(used) + 2
        order = g.permutation(pages)
        self.table = np.full((batch, width), -1, np.int32)             # (entries past a length are not used)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = c = U.Cache.empty(pages, kv, page, dim, grid, rht=rht, rht_seed=SEED)
        for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
            t.fill_(0xFF)
        c.k_row_scale.fill_(float("nan"))
        c.v_row_scale.fill_(float("nan"))
        self.mask = mask
        slots = []
        for b, n in enumerate(lens):
            sees = self.sees(b)
            for j in range(n):
                if sees[:, j].any():
                    slots.append(int(self.table[b, j // page]) * page + j % page)
        total = len(slots)
        if total:
            scale = 2.0 ** g.integers(-sizes, sizes + 1, size=(total, 1, 1))
            self.k = (g.standard_normal((total, kv, dim)) * scale).astype(np.float32)
            self.v = (g.standard_normal((total, kv, dim)) * scale).astype(np.float32)
            U.ufp4_cache_append(torch.from_numpy(self.k).cuda(), torch.from_numpy(self.v).cuda(),
                                torch.tensor(slots, device="cuda"), c)
        self.q = torch.from_numpy(g.standard_normal((batch * m, heads, dim)).astype(np.float32)).cuda().to(dtype)

    def sees(self, b):
        """[m, len] of sequence b."""
        n, m = self.lens[b], self.m
        s = np.ones((m, n), bool)
        for i in range(m):
            bits = (2 << i) - 1 if self.mask is None else int(self.mask[b, i]) & (2 ** 64 - 1)
            for r in range(m):
                j = n - m + r
                if 0 <= j < n:
                    s[i, j] = bits >> r & 1
        return s

    def args(self):
        mask = None if self.mask is None else torch.from_numpy(self.mask.view(np.int64)).cuda()
        return dict(q=self.q, cache=self.cache, table=torch.from_numpy(self.table).cuda(),
                    lens=torch.tensor(self.lens, dtype=torch.int32, device="cuda"), mask=mask)

    def rows(self, half, b):
        """The values of sequence b's rows as kept, [kv, len, dim], and their scales."""
        codes, scales, rs = half
        n = self.lens[b]
        pages = torch.from_numpy(self.table[b, :-(-n // self.page)].astype(np.int64)).cuda()
        take = lambda t: _np(t[pages].transpose(0, 1).reshape(self.kv, len(pages) * self.page, -1)[:, :n])  # noqa: E731
        rs = take(rs.unsqueeze(-1)).astype(np.float64)
        return R.values(R.unpack(take(codes)), take(scales), self.grid)[..., :self.dim] * rs, rs[..., 0]

    def check(self, out, lse, scale=None, dtype=BF):
        scale = self.dim ** -0.5 if scale is None else scale
        c, group, m = self.cache, self.heads // self.kv, self.m
        out, lse = _f64(out), _f64(lse)
        for b in range(len(self.lens)):
            at = slice(b * m, (b + 1) * m)
            sees = self.sees(b)
            if not sees.any():
                assert (out[at] == 0).all() and (lse[at] == -np.inf).all()
                continue
            k, _ = self.rows((c.k_codes, c.k_scales, c.k_row_scale), b)
            v, vs = self.rows((c.v_codes, c.v_scales, c.v_row_scale), b)
            some = sees.any(0)
            sees_ = sees[:, some]
            for h in range(self.heads):
                kv = h // group
                kk, vv = k[kv][some], v[kv][some]
                q = _f64(self.q[at, h])
                if self.rht:
                    q = R.rotate(q, SEED)
                top_v = np.abs(vs[kv][some]).max() * 448 * R.QMAX[self.grid]
                o, z, tol, ztol = R.attn(q, kk, vv, None, sees_, scale, self.q.dtype is BF and not self.rht,
                                         dtype is FP, top_v, self.dim)
                if self.rht:
                    # the inverse rotation: 16 elements' errors over 4, and its own additions
                    spread = lambda t: np.repeat(t.reshape(m, -1, 16).sum(-1) / 4, 16, -1)  # noqa: E731
                    tol = spread(tol + 8 * R.U24 * np.abs(o))
                    o = R.rotate(o, SEED, back=True)
                tol = tol + R.half_step(dtype) * (np.abs(o) + tol) + 1e-40
                bad = ~(np.abs(out[at, h] - o) <= tol)
                assert not bad.any(), (b, h, np.argwhere(bad)[:4], out[at, h][bad][:4], o[bad][:4], tol[bad][:4])
                bad = ~((np.abs(lse[at, h] - z) <= ztol) | (lse[at, h] == z))
                assert not bad.any(), ("lse", b, h, lse[at, h][bad][:4], z[bad][:4], ztol[bad][:4])


def _tree(g, batch, m):
    mask = np.zeros((batch, m), np.uint64)
    for b in range(batch):
        for i in range(m):
            p = int(g.integers(-1, i)) if i else -1
            mask[b, i] = (mask[b, p] if p >= 0 else np.uint64(0)) | np.uint64(1 << i)
    return mask


# lens, m, heads, kv, dim, page
CASES = [([1], 1, 1, 1, 16, 16), ([1, 0, 2], 1, 2, 1, 64, 16), ([15, 16, 17], 1, 4, 2, 48, 16),
         ([31, 32, 33, 64], 1, 8, 1, 64, 32), ([127, 128, 129, 300], 1, 8, 2, 128, 64), ([1000], 1, 32, 8, 128, 64),
         ([5000], 1, 3, 1, 80, 128), ([700, 3, 0, 257], 2, 6, 3, 128, 16), ([40, 90], 5, 10, 2, 128, 32),
         ([64, 65, 200], 64, 2, 2, 64, 16), ([500, 129], 17, 8, 2, 128, 64), ([300, 77], 3, 4, 2, 256, 32),
         ([900], 1, 7, 1, 144, 64), ([150], 64, 8, 1, 128, 16), ([3, 10], 8, 4, 4, 64, 16),
         # (more than 16 queries a head: one token of a wide group, groups past 128 queries, splits, short and empty ones)
         ([333, 0, 64], 1, 20, 1, 128, 32), ([63, 64, 65, 129], 5, 8, 2, 64, 16), ([3000, 17], 9, 30, 2, 80, 64),
         ([12000], 3, 32, 2, 128, 64)]


@pytest.mark.parametrize("lens,m,heads,kv,dim,page", CASES)
@pytest.mark.parametrize("grid,rht,dtype,out", [(1, True, BF, BF), (0, False, FP, FP), (2, False, BF, FP),
                                                (1, False, BF, BF), (0, True, FP, BF)])
def test_sizes(U, lens, m, heads, kv, dim, page, grid, rht, dtype, out):
    g = np.random.default_rng([sum(lens), m, heads, dim])
    c = Case(U, g, lens, m, heads, kv, dim, page, grid, rht, dtype)
    o, lse = U.ufp4_cache_attn(**c.args(), dtype=out, lse=True)
    assert o.dtype is out and o.shape == c.q.shape
    c.check(o, lse, dtype=out)
    o2, lse2 = U.ufp4_cache_attn(**c.args(), dtype=out, lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(o, U.ufp4_cache_attn(**c.args(), dtype=out))


@pytest.mark.parametrize("lens,m,heads,kv,dim,page", [c for c in CASES if c[1] > 1])
@pytest.mark.parametrize("kind", ["tree", "self", "gaps"])
def test_masks(U, lens, m, heads, kv, dim, page, kind):
    """Trees; tokens that see only themselves; words with empty rows and new
    tokens that nobody sees (their rows were never written)."""
    g = np.random.default_rng([sum(lens), m, heads])
    if kind == "tree":
        mask = _tree(g, len(lens), m)
    elif kind == "self":
        mask = np.broadcast_to(np.uint64(1) << np.arange(m, dtype=np.uint64), (len(lens), m)).copy()
    else:
        some = g.integers(0, 2 ** 63, size=(len(lens), m), dtype=np.uint64) << np.uint64(1)
        seen = g.integers(0, 2 ** 63, size=(len(lens), 1), dtype=np.uint64)
        mask = np.where(g.random((len(lens), m)) < 0.3, np.uint64(0), some & seen)
    c = Case(U, g, lens, m, heads, kv, dim, page, 1, True, BF, mask=mask)
    c.check(*U.ufp4_cache_attn(**c.args(), lse=True))


def test_one_token_that_does_not_see_itself(U):
    g = np.random.default_rng(2)
    c = Case(U, g, [50, 1], 1, 4, 2, 64, 16, 0, False, BF, mask=np.zeros((2, 1), np.uint64))
    c.check(*U.ufp4_cache_attn(**c.args(), lse=True))


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
def test_a_long_sequence_beside_short_ones(U, dim, page):
    """Split over CTAs, with splits that some sequences do not reach; a table
    wider than any of them."""
    g = np.random.default_rng(dim)
    c = Case(U, g, [20011, 5, 0, 4096], 2, 4, 2, dim, page, 1, True, FP, extra=37)
    c.check(*U.ufp4_cache_attn(**c.args(), lse=True), dtype=FP)


@pytest.mark.parametrize("heads", [8, 40])
def test_keys_and_values_of_differing_size(U, heads):
    """Rows whose scales differ by 2^24, scores far apart."""
    g = np.random.default_rng(9)
    c = Case(U, g, [777], 1, heads, 2, 128, 32, 0, False, FP, sizes=12)
    c.check(*U.ufp4_cache_attn(**c.args(), lse=True, scale=2.0 ** -12), scale=2.0 ** -12, dtype=FP)


@pytest.mark.parametrize("scale", [0.0, -0.25, 1e-4, 3.0])
@pytest.mark.parametrize("heads", [8, 16])
def test_scales(U, scale, heads):
    g = np.random.default_rng(10)
    c = Case(U, g, [300], 3, heads, 2, 64, 32, 1, False, FP)
    c.check(*U.ufp4_cache_attn(**c.args(), lse=True, scale=scale), scale=scale, dtype=FP)


def test_lengths_past_the_table(U):
    """A length longer than the table is held to it; a negative one is none."""
    g = np.random.default_rng(11)
    c = Case(U, g, [64, 10], 1, 4, 2, 64, 16, 1, False, BF)
    a = c.args()
    want = U.ufp4_cache_attn(**dict(a, lens=torch.tensor([64, 0], dtype=torch.int32, device="cuda")))
    got = U.ufp4_cache_attn(**dict(a, lens=torch.tensor([70000, -5], dtype=torch.int32, device="cuda")))
    assert torch.equal(got, want) and bool((got[1] == 0).all())


@pytest.mark.parametrize("heads", [2, 20])
def test_pages_outside_the_cache(U, heads):
    """They read as rows of zeros, whatever their number."""
    g = np.random.default_rng(12)
    c = Case(U, g, [64], 1, heads, 1, 64, 16, 1, False, FP)
    for bad in (-1, c.cache.pages, 2 ** 31 - 1, -2 ** 31):
        c.table[0, 1] = bad
        out, lse = U.ufp4_cache_attn(**c.args(), lse=True)
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("heads", [4, 16])         # (12 and 48 queries a head of the cache)
def test_non_finite_rows(U, where, heads):
    """A NaN row reaches the queries that see it, and no other."""
    g = np.random.default_rng(13)
    mask = _tree(g, 2, 6)
    c = Case(U, g, [70, 40], 6, heads, 2, 64, 16, 1, False, FP, mask=mask)
    clean, _ = U.ufp4_cache_attn(**c.args(), lse=True)
    j, head = 40 - 6 + 2, 1                     # new token 2 of the second sequence, the cache's second head
    page, at = int(c.table[1, j // 16]), j % 16
    getattr(c.cache, where + "_row_scale")[page, head, at] = float("nan")
    out, _ = U.ufp4_cache_attn(**c.args(), lse=True)
    hit = torch.zeros(12, heads, dtype=torch.bool, device="cuda")
    for i in range(6):
        if int(mask[1, i]) >> 2 & 1:
            hit[6 + i, heads // 2:] = True
    assert bool(hit.any()) and bool(torch.isnan(out[hit]).all()) and torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads", [4, 24])
def test_non_finite_queries(U, bad, heads):
    g = np.random.default_rng(14)
    c = Case(U, g, [70, 40], 3, heads, 2, 64, 16, 1, True, FP)
    clean = U.ufp4_cache_attn(**c.args())
    c.q[4, 1, 5] = bad
    out = U.ufp4_cache_attn(**c.args())
    hit = torch.zeros(6, heads, dtype=torch.bool, device="cuda")
    hit[4, 1] = True
    assert bool(torch.isnan(out[hit]).all()) and torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("m", [2, 9])              # (6 and 27 queries a head of the cache)
def test_strides(U, dtype, m):
    """q and out inside wider tensors, off their alignment; the rest stays."""
    g = np.random.default_rng(15)
    c = Case(U, g, [100, 33], m, 6, 2, 48, 16, 0, True, dtype)
    want = U.ufp4_cache_attn(**c.args())
    wide = torch.full((2 * m, 9, 51), 3.0, device="cuda", dtype=dtype)
    wide[:, 2:8, 1:49] = c.q
    res = torch.full((2 * m, 7, 53), 4.0, device="cuda", dtype=dtype)
    args = dict(c.args(), q=wide[:, 2:8, 1:49], out=res[:, 1:, 3:51])
    table = torch.full((2, c.table.shape[1] + 5), 99, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = args["table"]
    U.ufp4_cache_attn(**dict(args, table=table[:, :c.table.shape[1]]))
    assert torch.equal(res[:, 1:, 3:51], want)
    res[:, 1:, 3:51] = 4.0
    assert bool((res == 4.0).all())


def test_two_graphs_and_streams(U):
    """Captured calls keep their scratch apart; replayed with other lengths and queries."""
    g = np.random.default_rng(16)
    cases = [Case(U, g, [3000, 700], 1, 8, 2, 128, 32, 1, True, BF) for _ in range(2)]
    args = [c.args() for c in cases]
    graphs, outs = [], []
    for a in args:
        U.ufp4_cache_attn(**a)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(U.ufp4_cache_attn(**a))
        graphs.append(graph)
    for lens in ([3000, 700], [11, 650], [0, 1]):
        for a in args:
            a["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
            a["q"].normal_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for a, o in zip(args, outs):
            assert torch.equal(o, U.ufp4_cache_attn(**a))
    side = torch.cuda.Stream()
    got = U.ufp4_cache_attn(**args[0], stream=side)
    side.synchronize()
    assert torch.equal(got, outs[0])


def test_offsets_past_32_bits(U):
    """Pages more than 2^32 bytes into the codes."""
    g = np.random.default_rng(17)
    c = Case(U, g, [200], 1, 8, 8, 128, 128, 1, False, BF)
    want = U.ufp4_cache_attn(**c.args())
    far, small = U.Cache.empty(66000, 8, 128, 128, 1), c.cache
    to = torch.tensor([65999, 65000], device="cuda")
    at = torch.from_numpy(c.table[0, :2].astype(np.int64)).cuda()
    for n in ("k_codes", "k_scales", "k_row_scale", "v_codes", "v_scales", "v_row_scale"):
        getattr(far, n)[to] = getattr(small, n)[at]
    c.table[0, :2] = [65999, 65000]
    assert torch.equal(U.ufp4_cache_attn(**dict(c.args(), cache=far)), want)


def test_a_run_of_decoding(U):
    """Prompt, then tokens one by one: appended, attended over, and equal to
    the attention of a prompt's last tokens at once."""
    g = np.random.default_rng(18)
    heads, kv, dim, page, n, new = 4, 2, 64, 16, 45, 6
    c = U.Cache.empty(8, kv, page, dim, U.UFP4_E1M2, rht=True, rht_seed=SEED)
    table = torch.from_numpy(g.permutation(8)[:4].astype(np.int32)).cuda()[None]
    kvs = torch.randn(2, n + new, kv, dim, device="cuda", dtype=BF)
    q = torch.randn(new, heads, dim, device="cuda", dtype=BF)
    place = torch.arange(n + new, device="cuda")
    slots = table[0].long()[place // page] * page + place % page
    U.ufp4_cache_append(kvs[0, :n], kvs[1, :n], slots[:n], c)
    outs = []
    for i in range(new):
        U.ufp4_cache_append(kvs[0, n + i:n + i + 1], kvs[1, n + i:n + i + 1], slots[n + i:n + i + 1], c)
        lens = torch.tensor([n + i + 1], dtype=torch.int32, device="cuda")
        outs.append(U.ufp4_cache_attn(q[i:i + 1], c, table, lens, dtype=FP))
    at_once = U.ufp4_cache_attn(q, c, table, torch.tensor([n + new], dtype=torch.int32, device="cuda"), dtype=FP)
    # the same products, joined in another order: some 50 terms of 2^-21, through weights that sum to one
    assert (torch.cat(outs) - at_once).abs().max() <= 64 * 2.0 ** -21 * kvs[1].abs().max().float()


def test_empty(U):
    c = U.Cache.empty(1, 2, 16, 64, U.UFP4_E1M2)
    none = U.ufp4_cache_attn(torch.empty(0, 4, 64, device="cuda"), c, torch.empty(0, 3, dtype=torch.int32, device="cuda"),
                             torch.empty(0, dtype=torch.int32, device="cuda"))
    assert none.shape == (0, 4, 64)
    out, lse = U.ufp4_cache_attn(torch.randn(2, 4, 64, device="cuda"), c,
                                 torch.empty(2, 0, dtype=torch.int32, device="cuda"),
                                 torch.tensor([5, 0], dtype=torch.int32, device="cuda"), lse=True)
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())


def test_refusals(U):
    g = np.random.default_rng(19)
    c = Case(U, g, [40, 20], 2, 4, 2, 64, 16, 1, False, BF)
    a = c.args()
    call = lambda **kw: U.ufp4_cache_attn(**dict(a, **kw))  # noqa: E731
    mask = torch.zeros(2, 2, dtype=torch.int64, device="cuda")
    for kw in (dict(q=c.q[:3]), dict(q=c.q[..., :48]), dict(q=c.q[0]), dict(lens=a["lens"][:1]),
               dict(table=a["table"][:1]), dict(table=a["table"].t()), dict(mask=mask[:1]), dict(mask=mask.int()),
               dict(lse=torch.empty(4, 3, device="cuda")), dict(out=torch.empty(3, 4, 64, device="cuda", dtype=BF))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=c.q.half()), dict(lens=a["lens"].long()), dict(table=a["table"].long()), dict(dtype=torch.float16),
               dict(q=c.q.cpu())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=torch.randn(4, 3, 64, device="cuda")), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(q=torch.randn(130, 4, 64, device="cuda"))):
        with pytest.raises(U.UFP4Error):
            call(**kw)
    long = Case(U, g, [4000], 1, 2, 1, 64, 16, 1, False, BF, extra=4000)
    need = U.lib().ufp4_cache_attn_workspace_bytes(1, 1, 2, long.table.shape[1], long.cache.c())
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(U.ufp4_cache_attn(**long.args(), ws=ws), U.ufp4_cache_attn(**long.args()))
    with pytest.raises(U.UFP4Error):
        U.ufp4_cache_attn(**long.args(), ws=ws[:need - 1])


@pytest.mark.parametrize("m", [1, 32])
def test_workspace_on_16_bytes(U, m):
    """Scratch that starts 16 bytes past a larger boundary, and what lies before and behind it stays."""
    c = Case(U, np.random.default_rng(23), [4000], m, 2, 1, 128, 16, 1, True, BF, extra=4000)
    need = U.lib().ufp4_cache_attn_workspace_bytes(1, m, 2, c.table.shape[1], c.cache.c())
    assert need > 0
    room = torch.full((need + 48,), 0x5A, dtype=torch.uint8, device="cuda")
    assert room.data_ptr() % 32 == 0
    got = U.ufp4_cache_attn(**c.args(), ws=room[16:16 + need])
    assert torch.equal(got, U.ufp4_cache_attn(**c.args()))
    assert bool((room[:16] == 0x5A).all()) and bool((room[16 + need:] == 0x5A).all())
