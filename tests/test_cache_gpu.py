"""GPU parity of the 4-bit cache: rows written (codes, block scales and row
scales bit for bit the plain quantization of each row; with the rotation, a
neighbouring grid value where a rotated value lies within its fp32 error of a
border), read back, and what a call leaves alone."""
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


def _filled(U, pages, heads, page, dim, grid, rht=False, byte=0xA5):
    c = U.Cache.empty(pages, heads, page, dim, grid, rht=rht, rht_seed=SEED)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.fill_(byte)
    c.k_row_scale.fill_(-3.0)
    c.v_row_scale.fill_(-3.0)
    return c


def _halves(c):
    return ((c.k_codes, c.k_scales, c.k_row_scale), (c.v_codes, c.v_scales, c.v_row_scale))


def _kv(g, tokens, heads, dim, dtype, shift=0, pad=0):
    buf = torch.full((tokens * (heads * dim + pad) + shift + 1,), float("nan"), device="cuda", dtype=dtype)
    t = buf[shift:shift + tokens * (heads * dim + pad)].view(tokens, -1)[:, :heads * dim].view(tokens, heads, dim)
    v = g.standard_normal((tokens, heads, dim)) * 2.0 ** g.integers(-6, 7, size=(tokens, heads, 1))
    t.copy_(torch.from_numpy(v.astype(np.float32)))
    return t


def _stands_for(half, slot, dim, grid):
    """The values at a place, [heads, dim] (as kept, rotated or not)."""
    codes, scales, rs = half
    page = codes.shape[2]
    at = (slot // page, slice(None), slot % page)
    v = R.values(R.unpack(_np(codes[at])), _np(scales[at]), grid) * _np(rs[at]).astype(np.float64)[:, None]
    return v[:, :dim]


CASES = [(1, 1, 16, 16, 0), (5, 2, 16, 48, 1), (7, 3, 32, 64, 2), (9, 1, 64, 80, 0), (13, 2, 128, 128, 1),
         (6, 5, 16, 144, 0), (4, 2, 16, 256, 1), (3, 2, 32, 192, 2)]


@pytest.mark.parametrize("tokens,heads,page,dim,grid", CASES)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rht", [False, True])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 3)])
def test_rows(U, tokens, heads, page, dim, grid, dtype, rht, shift, pad):
    g = np.random.default_rng([tokens, heads, dim])
    pages = 3
    c = _filled(U, pages, heads, page, dim, grid, rht)
    k, v = _kv(g, tokens, heads, dim, dtype, shift, pad), _kv(g, tokens, heads, dim, dtype, shift, pad)
    k[0, 0] = 0.0                                                     # a row of zeros
    v[-1, -1, :16] *= 2.0 ** -30                                      # a block that vanishes beside its row
    slots = torch.from_numpy(g.permutation(pages * page)[:tokens]).cuda()
    U.ufp4_cache_append(k, v, slots, c)
    written = np.zeros((pages, page), bool)
    total = off = 0
    for i, s in enumerate(slots.tolist()):
        written[s // page, s % page] = True
        for half, x in zip(_halves(c), (k, v)):
            for h in range(heads):
                want = R.quantize_row(_np(x[i, h].float()), grid, rht, SEED)
                got = [_np(t[s // page, h, s % page]) for t in half]
                codes = R.unpack(got[0])
                assert (codes[dim:] == 0).all() and (got[1][dim // 16:] == 0).all()
                if not rht:
                    assert np.array_equal(codes[:dim], want[0]) and np.array_equal(got[1][:dim // 16], want[1])
                    assert got[2] == want[2]
                else:
                    # the row's scale within the butterflies' 4 roundings (of a sum of 16 magnitudes: 16 half steps)
                    assert abs(got[2] - want[2]) <= 16 * R.U24 * want[2]
                    a = R.values(codes[:dim], got[1][:dim // 16], grid) * got[2]
                    b = R.values(want[0], want[1], grid) * want[2]
                    step = np.repeat(R.e4m3(np.maximum(got[1][:dim // 16], want[1])), 16) * got[2] * \
                        (2.0 if grid == 0 else 0.5)
                    differ = np.abs(a - b) > 1e-5 * np.abs(b) + 1e-30
                    assert (np.abs(a - b)[differ] <= 1.13 * step[differ]).all()     # (a scale's step is an eighth)
                    off, total = off + differ.sum(), total + dim
    # codes one step away: 1e-4 of them is the bar of the quantizer; some 2000 are looked at here
    assert off <= max(2, 1e-4 * total)
    for half in _halves(c):
        rest = ~torch.from_numpy(written).cuda()
        assert bool((half[0].transpose(1, 2)[rest] == 0xA5).all()) and bool((half[1].transpose(1, 2)[rest] == 0xA5).all())
        assert bool((half[2].transpose(1, 2)[rest] == -3.0).all())

    for out in (BF, FP):
        lk, lv = U.ufp4_cache_load(c, slots, dtype=out)
        for half, t in zip(_halves(c), (lk, lv)):
            for i, s in enumerate(slots.tolist()):
                want = _stands_for(half, s, dim, grid)
                if rht:
                    want = R.rotate(want, SEED, back=True)
                    tol = 8 * R.U24 * np.abs(want).max(-1, keepdims=True) * 16
                else:
                    tol = R.U24 * np.abs(want)                        # the product with the row's scale
                tol = tol + R.half_step(out) * 1.001 * np.abs(want) + 1e-44
                assert (np.abs(_np(t[i].float()).astype(np.float64) - want) <= tol).all()


def test_skipped_and_foreign_places(U):
    """Places outside the cache: nothing is written, zeros are read."""
    c, g = _filled(U, 2, 2, 16, 64, U.UFP4_E1M2), np.random.default_rng(0)
    x = _kv(g, 6, 2, 64, BF)
    slots = torch.tensor([-1, 3, 32, 31, 1 << 40, -(1 << 40)], device="cuda")
    U.ufp4_cache_append(x, x, slots, c)
    hit = torch.zeros(2, 16, dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[1, 15] = True
    assert bool((c.k_codes.transpose(1, 2)[~hit] == 0xA5).all()) and bool((c.v_row_scale.transpose(1, 2)[~hit] == -3).all())
    k, v = U.ufp4_cache_load(c, slots)
    dead = torch.tensor([0, 2, 4, 5], device="cuda")
    assert bool((k[dead] == 0).all()) and bool((v[dead] == 0).all()) and bool((k[[1, 3]] != 0).any())
    again, _ = U.ufp4_cache_load(c, slots[[1, 1, 3, 1]])              # a place more than once
    assert torch.equal(again[0], again[1]) and torch.equal(again[0], again[3]) and torch.equal(again[2], k[3])


@pytest.mark.parametrize("rht", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_rows(U, rht, bad):
    c, g = _filled(U, 1, 3, 16, 128, U.UFP4_E2M1, rht), np.random.default_rng(0)
    k, v = _kv(g, 4, 3, 128, FP), _kv(g, 4, 3, 128, FP)
    k[1, 2, 77] = bad
    slots = torch.arange(4, device="cuda")
    U.ufp4_cache_append(k, v, slots, c)
    lk, lv = U.ufp4_cache_load(c, slots)
    hit = torch.zeros(4, 3, dtype=torch.bool, device="cuda")
    hit[1, 2] = True
    assert bool(torch.isnan(lk[hit]).all()) and bool(torch.isfinite(lk[~hit]).all()) and bool(torch.isfinite(lv).all())
    assert bool((c.k_codes[0, 2, 1] == 0).all()) and bool((c.k_scales[0, 2, 1] == 0).all())


@pytest.mark.parametrize("scale", [2.0 ** -140, 2.0 ** -100, 2.0 ** 100, 2.0 ** 126])
def test_range(U, scale):
    """Rows far from 1 are rounded relative to themselves."""
    c, g = _filled(U, 1, 1, 16, 64, U.UFP4_E1M2), np.random.default_rng(4)
    x = torch.from_numpy((g.uniform(-1, 1, size=(1, 1, 64)) * scale).astype(np.float32)).cuda()
    U.ufp4_cache_append(x, x, torch.zeros(1, dtype=torch.int64, device="cuda"), c)
    codes, scales, dec = R.quantize_row(_np(x[0, 0]), U.UFP4_E1M2)
    assert np.array_equal(R.unpack(_np(c.k_codes[0, 0, 0])), codes) and np.array_equal(_np(c.k_scales[0, 0, 0]), scales)
    assert float(c.k_row_scale[0, 0, 0]) == dec


def test_strided_results(U):
    """Reading into the heads of a wider tensor leaves the rest."""
    c, g = _filled(U, 2, 2, 16, 48, U.UFP4_E1M2), np.random.default_rng(2)
    x = _kv(g, 10, 2, 48, BF)
    slots = torch.arange(10, device="cuda") * 3
    U.ufp4_cache_append(x, x, slots, c)
    want, _ = U.ufp4_cache_load(c, slots)
    wide = torch.full((10, 5, 57), 9.0, device="cuda", dtype=BF)
    k, v = wide[:, 1:3, 4:52], torch.empty_like(want)
    U.ufp4_cache_load(c, slots, k=k, v=v)
    assert torch.equal(k, want) and torch.equal(v, want)
    wide[:, 1:3, 4:52] = 9.0
    assert bool((wide == 9.0).all())


def test_empty(U):
    c = _filled(U, 1, 1, 16, 16, U.UFP4_E1M2)
    none = torch.empty(0, 1, 16, device="cuda")
    U.ufp4_cache_append(none, none, torch.empty(0, dtype=torch.int64, device="cuda"), c)
    assert U.ufp4_cache_load(c, torch.empty(0, dtype=torch.int64, device="cuda"))[0].shape == (0, 1, 16)
    assert bool((c.k_codes == 0xA5).all())


def test_offsets_past_32_bits(U):
    """A place more than 2^32 bytes into the codes."""
    pages, heads, page, dim = 66000, 8, 128, 128
    c = U.Cache.empty(pages, heads, page, dim, U.UFP4_E2M1)
    x = _kv(np.random.default_rng(3), 3, heads, dim, BF)
    slots = torch.tensor([pages * page - 1, pages * page // 2 + 5, 0], device="cuda")
    U.ufp4_cache_append(x, x, slots, c)
    k, v = U.ufp4_cache_load(c, slots, dtype=FP)
    for i, s in enumerate(slots.tolist()):
        for h in range(heads):
            codes, scales, dec = R.quantize_row(_np(x[i, h].float()), 0)
            want = R.values(codes, scales, 0) * float(dec)
            assert (np.abs(_np(k[i, h]) - want) <= 2 * R.U24 * np.abs(want)).all() and torch.equal(k[i, h], v[i, h])


def test_streams_and_graphs(U):
    c, g = _filled(U, 4, 2, 32, 128, U.UFP4_E1M2, True), np.random.default_rng(8)
    x, slots = _kv(g, 40, 2, 128, BF), torch.from_numpy(g.permutation(128)[:40]).cuda()
    U.ufp4_cache_append(x, x, slots, c)
    want = U.ufp4_cache_load(c, slots)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = U.ufp4_cache_load(c, slots, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        U.ufp4_cache_append(x, x, slots, c)
        got = U.ufp4_cache_load(c, slots)
    slots.copy_(torch.from_numpy(g.permutation(128)[:40]).cuda())
    x.copy_(_kv(g, 40, 2, 128, BF))
    graph.replay()
    other = _filled(U, 4, 2, 32, 128, U.UFP4_E1M2, True)
    U.ufp4_cache_append(x, x, slots, other)
    want = U.ufp4_cache_load(other, slots)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals(U):
    c = _filled(U, 2, 2, 16, 64, U.UFP4_E1M2)
    x, slots = torch.randn(3, 2, 64, device="cuda"), torch.arange(3, device="cuda")
    with pytest.raises(TypeError):
        U.ufp4_cache_append(x, x.bfloat16(), slots, c)
    with pytest.raises(TypeError):
        U.ufp4_cache_append(x.half(), x.half(), slots, c)
    for bad in (x[:, :1], x[..., :48], x[0], x.transpose(1, 2)):
        with pytest.raises(ValueError):
            U.ufp4_cache_append(bad, x, slots, c)
    for bad in (slots[:2], slots.int(), slots[None], torch.arange(6, device="cuda")[::2]):
        with pytest.raises(ValueError):
            U.ufp4_cache_append(x, x, bad, c)
    with pytest.raises(ValueError):
        U.ufp4_cache_load(c, slots, k=x)
    with pytest.raises(TypeError):
        U.ufp4_cache_load(c, slots, dtype=torch.float16)
    with pytest.raises(ValueError):
        U.Cache(c.k_codes, c.k_scales, c.k_row_scale, c.v_codes, c.v_scales[:1], c.v_row_scale, 64, U.UFP4_E1M2)
    for page, dim, grid in ((8, 64, 1), (16, 512, 1), (16, 64, U.UFP4_MXFP4)):
        with pytest.raises((U.UFP4Error, ValueError)):
            bad = U.Cache.empty(2, 2, page, dim, grid)
            U.ufp4_cache_append(torch.randn(3, 2, dim, device="cuda"), torch.randn(3, 2, dim, device="cuda"), slots, bad)
