"""GPU parity of the 8-bit checkpoints and the gated activation against plain
64-bit forms (tests/rowop_refs.py, which also derives the error bounds).
Scale bytes and restored values are compared exactly."""
import numpy as np
import pytest
import torch

from tests import rowop_refs as R

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
FORMATS = [0, 1]


@pytest.fixture(scope="module")
def U():
    from fp4_quantized_numerics_gb300 import build, ufp4
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return ufp4


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _tensor(v, dtype, pad=0, shift=0):
    rows, cols = v.shape
    buf = torch.full((rows * (cols + pad) + shift + 1,), float("nan"), device="cuda", dtype=dtype)
    t = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)))
    return t


def _values(g, rows, cols):
    """Rows of very different size, some zeros, a heavy column."""
    v = g.standard_normal((rows, cols)) * 2.0 ** g.integers(-6, 7, size=(rows, 1))
    v[g.random((rows, cols)) < 0.05] = 0
    v[:, cols // 2] *= 30
    return v


# (rows, cols, pad, shift): blocks that end inside a row, rows off 16 bytes, one element, one block
SHAPES = [(1, 1, 0, 0), (1, 32, 0, 0), (3, 8, 0, 0), (5, 40, 0, 0), (5, 40, 8, 0), (5, 40, 3, 0), (7, 64, 0, 1),
          (9, 33, 0, 0), (2, 1001, 0, 0), (4, 1408, 0, 0), (65, 72, 0, 0),
          (6, 34, 0, 0), (3, 1002, 0, 0), (5, 96, 2, 2), (5, 48, 0, 0)]


@pytest.mark.parametrize("rows,cols,pad,shift", SHAPES)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("fmt", FORMATS)
def test_ckpt(U, rows, cols, pad, shift, dtype, fmt):
    x = _tensor(_values(np.random.default_rng(cols), rows, cols), dtype, pad, shift)
    c = U.ufp4_ckpt_save(x, fmt)
    scales, back = R.ckpt(_f64(x), fmt)
    np.testing.assert_array_equal(c.scales.cpu().numpy(), scales)
    for dt in (BF, FP):
        np.testing.assert_array_equal(_f64(U.ufp4_ckpt_load(c, dtype=dt)), back)
    out = _tensor(np.zeros((rows, cols)), dtype, pad, shift)
    assert U.ufp4_ckpt_load(c, out=out) is out
    np.testing.assert_array_equal(_f64(out), back)


@pytest.mark.parametrize("cols", [32, 31, 30])   # the layouts of the work
@pytest.mark.parametrize("fmt", FORMATS)
def test_ckpt_edges(U, fmt, cols):
    """Powers of two and their neighbours at the top of a block (the scale's
    steps, E4M3's 1.75), ties of the rounding, the smallest and largest fp32
    magnitudes, all-zero blocks, signs of zero."""
    tops = []
    for e in (-149, -140, -127, -126, -125, -122, -120, -119, -118, -117, -20, 0, 3, 126, 127):
        for m in (1.0, 1.0 + 2.0 ** -23, 1.5, 1.75, 1.75 + 2.0 ** -23, 1.875, 2.0 - 2.0 ** -23):
            tops.append(np.float32(m * 2.0 ** e))
    v = np.zeros((len(tops) + 2, cols), np.float32)
    for r, top in enumerate(tops):
        frac = np.linspace(-1, 1, cols)
        frac[1:8] = [0.5, 0.25 + 1 / 512, -3 / 256, 63.5 / 64, 2.5 / 64, -3.5 / 64, 1 / 1024]
        v[r] = (frac * np.float64(top)).astype(np.float32)
        v[r, 0] = top
    v[-1, ::2] = -0.0
    x = torch.from_numpy(v).cuda()
    c = U.ufp4_ckpt_save(x, fmt)
    scales, back = R.ckpt(v.astype(np.float64), fmt)
    np.testing.assert_array_equal(c.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(_f64(U.ufp4_ckpt_load(c, dtype=FP)), back)


@pytest.mark.parametrize("cols", [96, 95, 94])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_ckpt_keeps_non_finite_blocks_visible(U, fmt, bad, cols):
    v = np.ones((3, cols))
    v[1, 40] = bad
    c = U.ufp4_ckpt_save(_tensor(v, BF), fmt)
    back = _f64(U.ufp4_ckpt_load(c))
    assert c.scales[1, 1].item() == 255 and torch.all(c.codes[1, 32:64] == 0)
    assert np.all(np.isnan(back[1, 32:64]))
    back[1, 32:64] = 1
    assert np.all(back == 1)


@pytest.mark.parametrize("rows,cols,pad,shift", SHAPES)
@pytest.mark.parametrize("dtypes", [(BF, BF, FP, FP), (FP, BF, FP, BF), (BF, FP, BF, BF), (FP, FP, BF, FP)],
                         ids=lambda d: "-".join(str(t)[6:] for t in d))
@pytest.mark.parametrize("fmt", FORMATS)
def test_swiglu(U, rows, cols, pad, shift, dtypes, fmt):
    ti, th, td, to = dtypes
    g = np.random.default_rng(cols + 1)
    both = _tensor(np.concatenate([_values(g, rows, cols), _values(g, rows, cols)], axis=1), ti, pad, shift)
    gate, up = both[:, :cols], both[:, cols:]          # two halves of one product
    h = _tensor(np.zeros((rows, cols)), th, pad, shift)
    _, kg, ku = U.ufp4_swiglu(gate, up, ckpt=fmt, out=h)
    g64, u64 = _f64(gate), _f64(up)
    want = R.swiglu(g64, u64)
    assert np.all(np.abs(_f64(h) - want) <= R.swiglu_tol(g64, u64, want, th))
    for c, v in ((kg, g64), (ku, u64)):
        scales, back = R.ckpt(v, fmt)
        np.testing.assert_array_equal(c.scales.cpu().numpy(), scales)
        np.testing.assert_array_equal(_f64(U.ufp4_ckpt_load(c, dtype=FP)), back)
    # without checkpoints: the same h
    alone, none_g, none_u = U.ufp4_swiglu(gate, up, dtype=th)
    assert none_g is None and none_u is None and torch.equal(alone, h)

    dh = _tensor(g.standard_normal((rows, cols)) * 1e-3, td, pad, shift)
    dgate, dup = _tensor(np.zeros((rows, cols)), to, pad, shift), _tensor(np.zeros((rows, cols)), to, pad, shift)
    U.ufp4_swiglu_bwd(dh, kg, ku, dgate=dgate, dup=dup)
    g64, u64, d64 = R.ckpt(g64, fmt)[1], R.ckpt(u64, fmt)[1], _f64(dh)
    wg, wu = R.swiglu_bwd(d64, g64, u64)
    tg, tu = R.swiglu_bwd_tol(d64, g64, u64, wg, wu, to)
    assert np.all(np.abs(_f64(dgate) - wg) <= tg)
    assert np.all(np.abs(_f64(dup) - wu) <= tu)
    assert U.ufp4_swiglu_bwd(dh, kg, ku)[0].dtype == td


@pytest.mark.parametrize("th", [BF, FP])
def test_swiglu_far_gates(U, th):
    """Gates far on both sides: silu goes to 0 and to the gate itself, its
    derivative to 0 and 1, and nothing overflows into a NaN."""
    gate = torch.tensor([[0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 88.0, -88.0, 89.0, -89.0, 104.0, -104.0, 1e4, -1e4,
                          1e30, -1e30]], device="cuda")
    up = torch.full_like(gate, 3.0)
    h, kg, ku = U.ufp4_swiglu(gate, up, ckpt=1, dtype=th)
    want = R.swiglu(_f64(gate), 3.0)
    assert np.all(np.abs(_f64(h) - want) <= R.swiglu_tol(_f64(gate), 3.0, want, th))
    dh = torch.ones_like(gate)
    for lo in (0, 4, 12, 14):   # gates of one size at a time: a block has one scale
        part = gate[:, lo:lo + 2].contiguous()
        _, kg, ku = U.ufp4_swiglu(part, up[:, :2].contiguous(), ckpt=1, dtype=th)
        dg, du = U.ufp4_swiglu_bwd(dh[:, :2].contiguous(), kg, ku, dtype=th)
        g64, u64 = _f64(U.ufp4_ckpt_load(kg, dtype=FP)), _f64(U.ufp4_ckpt_load(ku, dtype=FP))
        wg, wu = R.swiglu_bwd(1.0, g64, u64)
        tg, tu = R.swiglu_bwd_tol(1.0, g64, u64, wg, wu, th)
        assert np.all(np.abs(_f64(dg) - wg) <= tg) and np.all(np.abs(_f64(du) - wu) <= tu)


def test_swiglu_gradients_by_differences(U):
    """The gradients against central differences of silu(g) u in 64 bits, at
    the restored values.  The differences' own error: step^2 / 6 times the
    third derivative (silu''' < 1), plus 64-bit cancellation."""
    g = np.random.default_rng(12)
    gate, up, dh = (_tensor(g.standard_normal((6, 64)), FP) for _ in range(3))
    _, kg, ku = U.ufp4_swiglu(gate, up, ckpt=0)
    dg, du = U.ufp4_swiglu_bwd(dh, kg, ku)
    g64, u64, d64 = _f64(U.ufp4_ckpt_load(kg, dtype=FP)), _f64(U.ufp4_ckpt_load(ku, dtype=FP)), _f64(dh)
    e = 1e-4
    ng = d64 * (R.swiglu(g64 + e, u64) - R.swiglu(g64 - e, u64)) / (2 * e)
    nu = d64 * (R.swiglu(g64, u64 + e) - R.swiglu(g64, u64 - e)) / (2 * e)
    tg, tu = R.swiglu_bwd_tol(d64, g64, u64, ng, nu, FP)
    assert np.all(np.abs(_f64(dg) - ng) <= tg + np.abs(d64 * u64) * e * e / 6 + 1e-11)
    assert np.all(np.abs(_f64(du) - nu) <= tu + 1e-11)


@pytest.mark.parametrize("fmt", FORMATS)
def test_non_finite_gradient_flow(U, fmt):
    """A NaN in gate reaches h there, and the block's gradients."""
    v = np.full((2, 64), 0.5)
    v[0, 3] = np.nan
    gate, up = _tensor(v, BF), _tensor(np.ones((2, 64)), BF)
    h, kg, ku = U.ufp4_swiglu(gate, up, ckpt=fmt)
    assert np.isnan(_f64(h)[0, 3]) and np.isnan(_f64(h)).sum() == 1
    dg, du = U.ufp4_swiglu_bwd(_tensor(np.ones((2, 64)), BF), kg, ku)
    for t in (dg, du):
        nan = np.isnan(_f64(t))
        assert nan[0, :32].all() and nan.sum() == 32


@pytest.mark.parametrize("fmt", FORMATS)
def test_kept_buffers_of_the_caller(U, fmt):
    """Checkpoints written into the caller's, on a side stream and in a graph;
    a pair of another shape or of two formats is refused."""
    g = np.random.default_rng(13)
    gate, up = _tensor(_values(g, 40, 96), BF), _tensor(_values(g, 40, 96), BF)
    h, kg, ku = U.ufp4_swiglu(gate, up, ckpt=fmt)
    keep = U.Ckpt.empty(40, 96, fmt), U.Ckpt.empty(40, 96, fmt)
    out = torch.empty_like(gate)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert U.ufp4_swiglu(gate, up, out=out, keep=keep, stream=side)[1] is keep[0]
    side.synchronize()
    for a, b in ((keep[0], kg), (keep[1], ku)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
        a.codes.zero_()
        a.scales.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        U.ufp4_swiglu(gate, up, out=out, keep=keep)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, h)
    for a, b in ((keep[0], kg), (keep[1], ku)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    for bad in ((keep[0], U.Ckpt.empty(40, 96, 1 - fmt)), (keep[0], U.Ckpt.empty(40, 64, fmt))):
        with pytest.raises(U.UFP4Error):
            U.ufp4_swiglu(gate, up, keep=bad)


def test_no_rows(U):
    e = torch.empty(0, 64, device="cuda")
    h, kg, ku = U.ufp4_swiglu(e, e, ckpt=0)
    dg, du = U.ufp4_swiglu_bwd(e, kg, ku)
    assert h.shape == dg.shape == du.shape == U.ufp4_ckpt_load(U.ufp4_ckpt_save(e)).shape == (0, 64)


def test_codes_of_a_wide_row_stride(U):
    """Row offsets past 2^31 elements of the input."""
    rows, cols, ld = 3, 64, (1 << 30) + 8
    free, _ = torch.cuda.mem_get_info()
    need = ((rows - 1) * ld + cols) * 2
    if free < need + (4 << 30):
        pytest.skip("needs %d GB of device memory" % (need >> 30))
    x = torch.empty(need // 2, device="cuda", dtype=BF).as_strided((rows, cols), (ld, 1))
    x.copy_(torch.from_numpy(_values(np.random.default_rng(2), rows, cols)))
    np.testing.assert_array_equal(_f64(U.ufp4_ckpt_load(U.ufp4_ckpt_save(x, 0))), R.ckpt(_f64(x), 0)[1])
