"""GPU parity of the sort by expert, dispatch, combine and combine's
gradients against plain 64-bit forms (tests/rowop_refs.py).

Integers and copies are compared exactly.  Sums: combine adds topk terms in
fp32, each addition within 2^-24 of the sum of magnitudes so far; dw adds
`hidden` products likewise; a bf16 result adds its own 2^-8.
"""
import numpy as np
import pytest
import torch

from tests import rowop_refs as R

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def U():
    from fp4_quantized_numerics_gb300 import build, ufp4
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return ufp4


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _ids(g, tokens, topk, experts, dropped):
    """dropped: 'none', 'some' (tokens and single slots, both sides of the
    range), 'all'."""
    ids = g.integers(0, experts, size=(tokens, topk))
    if dropped == "some":
        ids[g.random(tokens) < 0.3] = -1
        ids[g.random(ids.shape) < 0.1] = experts
    elif dropped == "all":
        ids[:] = -1
    return ids


def _tensor(g, rows, cols, dtype, pad=0, shift=0, std=1.0):
    """rows x cols N(0, std) on the GPU, row stride cols + pad, first element
    `shift` elements into its allocation."""
    buf = torch.full((rows * (cols + pad) + shift + 1,), float("nan"), device="cuda", dtype=dtype)
    t = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    if rows and cols:
        t.copy_(torch.from_numpy(g.standard_normal((rows, cols)).astype(np.float32) * np.float32(std)))
    return t


def _close(got, want, tol):
    got = _f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


SIZES = [(0, 2, 4), (1, 1, 1), (1, 6, 64), (2, 8, 256), (33, 2, 3), (257, 6, 64), (1000, 3, 7), (1024, 1, 2),
         (2049, 8, 256), (70001, 2, 16)]


@pytest.mark.parametrize("tokens,topk,experts", SIZES)
@pytest.mark.parametrize("dropped", ["none", "some", "all"])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(U, tokens, topk, experts, dropped, dtype):
    ids = _ids(np.random.default_rng(tokens + topk), tokens, topk, experts, dropped)
    p = U.ufp4_moe_sort(torch.from_numpy(ids).to(dtype).cuda(), experts)
    pos, src, counts, offsets = R.sort(ids, experts)
    np.testing.assert_array_equal(p.pos.cpu().numpy(), pos)
    np.testing.assert_array_equal(p.src.cpu().numpy(), src)
    np.testing.assert_array_equal(p.counts.cpu().numpy(), counts)
    np.testing.assert_array_equal(p.offsets.cpu().numpy(), offsets)
    assert (p.tokens, p.topk, p.n_experts) == (tokens, topk, experts)


def test_sort_of_one_expert_and_of_far_ids(U):
    """Every slot to one expert stays in slot order; int64 ids whose low 32
    bits look valid are dropped all the same."""
    n = 5000
    p = U.ufp4_moe_sort(torch.full((n, 2), 5, device="cuda", dtype=torch.int64), 8)
    assert torch.equal(p.src.cpu(), torch.arange(2 * n, dtype=torch.int32))
    assert p.counts.tolist() == [0] * 5 + [2 * n, 0, 0]
    far = torch.tensor([[1, (1 << 32) + 1, -(1 << 40), (1 << 62), 0]], device="cuda")
    p = U.ufp4_moe_sort(far, 4)
    assert p.pos.tolist() == [[1, 2, 3, 4, 0]] and p.offsets.tolist() == [0, 1, 2, 2, 2]


def _plan(U, g, tokens, topk, experts, dropped):
    ids = _ids(g, tokens, topk, experts, dropped)
    plan = U.ufp4_moe_sort(torch.from_numpy(ids).cuda(), experts)
    pos, _, _, offsets = R.sort(ids, experts)
    return plan, pos, int(offsets[-1])


# (tokens, topk, experts, hidden, pad, shift): rows on and off 16 bytes, rows shorter than a vector, long rows
SHAPES = [(1, 6, 64, 2048, 0, 0), (5, 1, 3, 8, 0, 0), (37, 2, 5, 96, 0, 0), (37, 2, 5, 96, 8, 0), (37, 2, 5, 96, 3, 0),
          (37, 2, 5, 96, 0, 1), (29, 8, 64, 27, 0, 0), (29, 9, 64, 40, 0, 0), (13, 13, 200, 1001, 0, 0),
          (3, 2, 4, 8200, 0, 0), (130, 6, 64, 1, 0, 0), (2, 17, 32, 264, 0, 0), (11, 3, 7, 10, 0, 0),
          (7, 4, 9, 1002, 0, 0), (7, 4, 9, 600, 2, 2)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dropped", ["none", "some", "all"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_dispatch(U, shape, dropped, dtype):
    tokens, topk, experts, hidden, pad, shift = shape
    g = np.random.default_rng(3)
    plan, pos, routed = _plan(U, g, tokens, topk, experts, dropped)
    x = _tensor(g, tokens, hidden, dtype, pad, shift)
    out = _tensor(g, tokens * topk, hidden, dtype, pad, shift)
    want = R.dispatch(_f64(x), pos, routed)
    np.testing.assert_array_equal(_f64(U.ufp4_moe_dispatch(x, plan)), want)
    assert U.ufp4_moe_dispatch(x, plan, out=out) is out
    np.testing.assert_array_equal(_f64(out), want)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dropped", ["none", "some", "all"])
@pytest.mark.parametrize("y_dtype", [BF, FP])
@pytest.mark.parametrize("out_dtype", [BF, FP])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(U, shape, dropped, y_dtype, out_dtype, weighted):
    tokens, topk, experts, hidden, pad, shift = shape
    g = np.random.default_rng(4)
    plan, pos, routed = _plan(U, g, tokens, topk, experts, dropped)
    y = _tensor(g, tokens * topk, hidden, y_dtype, pad, shift)
    y[routed:] = float("nan")          # dropped rows are not read into the sum
    w = torch.from_numpy(g.random((tokens, topk)).astype(np.float32)).cuda() if weighted else None
    if weighted:
        w[torch.from_numpy(pos >= routed).cuda()] = float("inf")
    out = _tensor(g, tokens, hidden, out_dtype, pad, shift)
    U.ufp4_moe_combine(y, plan, w, out=out)
    want, mag = R.combine(_f64(y), pos, routed, None if w is None else _f64(w))
    _close(out, want, topk * R.U32 * mag + R.unit(out_dtype) * 1.001 * np.abs(want))
    assert U.ufp4_moe_combine(y, plan, w).dtype == y_dtype


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dropped", ["none", "some", "all"])
@pytest.mark.parametrize("dtypes", [(BF, FP, BF), (FP, BF, FP), (BF, BF, FP), (FP, FP, BF), (FP, FP, FP)],
                         ids=lambda d: "-".join(str(t)[6:] for t in d))
def test_combine_bwd(U, shape, dropped, dtypes):
    tokens, topk, experts, hidden, pad, shift = shape
    g = np.random.default_rng(5)
    plan, pos, routed = _plan(U, g, tokens, topk, experts, dropped)
    dout = _tensor(g, tokens, hidden, dtypes[0], pad, shift, 1e-3)
    y = _tensor(g, tokens * topk, hidden, dtypes[1], pad, shift)
    y[routed:] = float("nan")
    w = torch.from_numpy(g.random((tokens, topk)).astype(np.float32)).cuda()
    w[torch.from_numpy(pos >= routed).cuda()] = float("nan")
    dy = _tensor(g, tokens * topk, hidden, dtypes[2], pad, shift)
    dw = torch.full((tokens, topk), float("nan"), device="cuda")
    U.ufp4_moe_combine_bwd(dout, y, plan, w, dy=dy, dw=dw)
    want, want_w, mag = R.combine_bwd(_f64(dout), _f64(y), pos, routed, _f64(w))
    _close(dy, want, (R.U32 + R.unit(dtypes[2]) * 1.001) * np.abs(want))
    _close(dw, want_w, (hidden + 1) * R.U32 * mag)
    again = U.ufp4_moe_combine_bwd(dout, y, plan, w, dtype=dtypes[2])
    assert torch.equal(again[0], dy) and torch.equal(again[1], dw)


def test_combine_gradients_by_differences(U):
    """combine is linear in y and in w: its differences along any direction
    are the gradients' inner products.  The kernel's fp32 sums round within
    topk 2^-24 of their magnitudes, each side once."""
    g = np.random.default_rng(6)
    tokens, topk, experts, hidden = 50, 4, 9, 72
    plan, pos, routed = _plan(U, g, tokens, topk, experts, "some")
    y, step = _tensor(g, tokens * topk, hidden, FP), _tensor(g, tokens * topk, hidden, FP)
    dout = _tensor(g, tokens, hidden, FP)
    w = torch.from_numpy(g.random((tokens, topk)).astype(np.float32)).cuda()
    wstep = torch.from_numpy(g.random((tokens, topk)).astype(np.float32)).cuda()
    dy, dw = U.ufp4_moe_combine_bwd(dout, y, plan, w)
    up, down = U.ufp4_moe_combine(y + step, plan, w), U.ufp4_moe_combine(y - step, plan, w)
    diff = np.sum(_f64(dout) * (_f64(up) - _f64(down))) / 2
    _, mag = R.combine(np.abs(_f64(y)) + np.abs(_f64(step)), pos, routed, _f64(w))
    tol = np.sum(np.abs(_f64(dout)) * mag) * (topk + 3) * R.U32
    assert abs(diff - np.sum(_f64(dy) * _f64(step))) <= tol
    up, down = U.ufp4_moe_combine(y, plan, w + wstep), U.ufp4_moe_combine(y, plan, w - wstep)
    diff = np.sum(_f64(dout) * (_f64(up) - _f64(down))) / 2
    _, mag = R.combine(np.abs(_f64(y)), pos, routed, _f64(w) + _f64(wstep))
    tol = np.sum(np.abs(_f64(dout)) * mag) * (hidden + topk + 3) * R.U32
    assert abs(diff - np.sum(_f64(dw) * _f64(wstep))) <= tol


def test_dispatch_gradient_is_combine_without_weights(U):
    """<dispatch(x), d> = <x, combine(d)>: the dispatch copies, so the left
    side is exact in 64 bits; combine adds topk terms in fp32."""
    g = np.random.default_rng(7)
    tokens, topk, experts, hidden = 41, 5, 6, 104
    plan, pos, routed = _plan(U, g, tokens, topk, experts, "some")
    x, d = _tensor(g, tokens, hidden, FP), _tensor(g, tokens * topk, hidden, FP)
    left = np.sum(_f64(U.ufp4_moe_dispatch(x, plan)) * _f64(d))
    right = np.sum(_f64(x) * _f64(U.ufp4_moe_combine(d, plan)))
    _, mag = R.combine(np.abs(_f64(d)), pos, routed)
    assert abs(left - right) <= np.sum(np.abs(_f64(x)) * mag) * (topk + 1) * R.U32


def test_rows_far_apart(U):
    """Row offsets past 2^31 elements and 2^32 bytes."""
    free, _ = torch.cuda.mem_get_info()
    tokens, topk, hidden, ld = 3, 2, 40, (1 << 29) + 8
    need = ((tokens * topk - 1) * ld + hidden) * 4
    if free < need + (4 << 30):
        pytest.skip("needs %d GB of device memory" % (need >> 30))
    g = np.random.default_rng(8)
    buf = torch.empty(need // 4, device="cuda")
    wide = buf.as_strided((tokens * topk, hidden), (ld, 1))
    plan, pos, routed = _plan(U, g, tokens, topk, 2, "none")
    x = _tensor(g, tokens, hidden, FP)
    U.ufp4_moe_dispatch(x, plan, out=wide)
    np.testing.assert_array_equal(_f64(wide), R.dispatch(_f64(x), pos, routed))
    want, mag = R.combine(_f64(wide), pos, routed)
    _close(U.ufp4_moe_combine(wide, plan), want, topk * R.U32 * mag)
    w = torch.ones(tokens, topk, device="cuda")
    dy, dw = U.ufp4_moe_combine_bwd(x, wide, plan, w)
    _, want_w, mag = R.combine_bwd(_f64(x), _f64(wide), pos, routed, _f64(w))
    _close(dw, want_w, (hidden + 1) * R.U32 * mag)


def test_side_stream_and_graph(U):
    """The calls run on the stream they are given and can be captured; the
    graph's replay follows new inputs."""
    g = np.random.default_rng(9)
    tokens, topk, experts, hidden = 64, 4, 8, 256
    ids = torch.from_numpy(_ids(g, tokens, topk, experts, "some")).cuda()
    x = _tensor(g, tokens, hidden, BF)
    w = torch.from_numpy(g.random((tokens, topk)).astype(np.float32)).cuda()
    plan = U.MoePlan.empty(tokens, topk, experts)
    xs = torch.empty(tokens * topk, hidden, device="cuda", dtype=BF)
    out = torch.empty(tokens, hidden, device="cuda", dtype=FP)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(stream=None):
        U.ufp4_moe_sort(ids, experts, out=plan, stream=stream)
        U.ufp4_moe_dispatch(x, plan, out=xs, stream=stream)
        U.ufp4_moe_combine(xs, plan, w, out=out, stream=stream)

    step(side)
    side.synchronize()
    want = out.clone()
    assert torch.any(want != 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -want)
