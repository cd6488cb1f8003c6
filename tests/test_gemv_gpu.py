"""GPU parity of the few-token products, dense and by expert, against plain
64-bit sums over what the quantized weights stand for (tests/serving_refs.py,
which derives the bounds)."""
import numpy as np
import pytest
import torch

from tests import serving_refs as R
from tests.layouts import kpad, rpad, unpack_codes, unpack_scales

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
SEED = 7


@pytest.fixture(scope="module")
def U():
    from fp4_quantized_numerics_gb300 import build, ufp4
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return ufp4


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _values(q, grid, rows=None, segments=1):
    """What a QTensor stands for, [segments, rows, k] (no rotation undone)."""
    codes = unpack_codes(q.codes.cpu().numpy(), q.rows, q.k)
    scales, _ = unpack_scales(q.scales.cpu().numpy(), q.rows, q.k)
    v = R.values(codes, scales, grid).reshape(segments, -1, q.k)
    v = v * _f64(q.tensor_scale)[:segments, None, None]
    return v if rows is None else v[:, :rows]


def _x(g, shape, dtype, pad=0, shift=0, spread=0):
    """N(0, 1) tokens, each times 2^(-spread .. spread), with a row stride of
    k + pad, `shift` elements into their allocation (NaN around them)."""
    t, k = shape
    buf = torch.full((t * (k + pad) + shift + 1,), float("nan"), device="cuda", dtype=dtype)
    x = buf[shift:shift + t * (k + pad)].view(t, k + pad)[:, :k]
    v = g.standard_normal(shape) * 2.0 ** g.integers(-spread, spread + 1, size=(t, 1))
    if t and k:
        x.copy_(torch.from_numpy(v.astype(np.float32)))
    return x


def _check(y, x, w, rht, out, tag=""):
    # exact, one FP16 value (11 bits), or two
    unit = 0.0 if x.dtype is BF and not rht else 2.0 ** -11 if out is BF else 2.0 ** -22
    want, tol = R.gemv(_f64(x), w, rht, SEED, unit)
    got = _f64(y)
    tol = tol + R.half_step(out) * (np.abs(want) + tol) + 1e-44
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (tag, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


# tokens, rows, k: single ones, sizes that fill nothing, column groups of 8, 16 and 32 and past them, phases of k
SIZES = [(1, 1, 16), (1, 16, 64), (1, 128, 128), (1, 129, 80), (2, 130, 208), (3, 256, 2048), (4, 97, 1040), (5, 640, 512),
         (8, 300, 1408), (9, 128, 64), (13, 1001, 1040), (16, 64, 4096), (17, 200, 720), (32, 131, 2064), (33, 96, 320),
         (70, 257, 272), (8, 96, 8208), (32, 64, 8192), (1, 4096, 16384), (16, 4100, 5136)]


@pytest.mark.parametrize("tokens,rows,k", SIZES)
@pytest.mark.parametrize("rht", [False, True])
def test_sizes(U, tokens, rows, k, rht):
    g = np.random.default_rng([tokens, rows, k, int(rht)])
    for grid, dx, dy in ((U.UFP4_E2M1, BF, FP), (U.UFP4_E1M2, FP, BF), (U.UFP4_E2M1C, FP, FP)):
        w = torch.from_numpy(g.standard_normal((rows, k)).astype(np.float32)).cuda()
        q = U.ufp4_quantize(w, grid, rht=rht, rht_seed=SEED)
        x = _x(g, (tokens, k), dx, spread=2)
        y = U.ufp4_gemv(x, q, rht=rht, rht_seed=SEED, dtype=dy)
        assert y.shape == (tokens, rows) and y.dtype is dy
        _check(y, x, _values(q, grid)[0], rht, dy, (grid, dx))
        assert torch.equal(y, U.ufp4_gemv(x, q, rht=rht, rht_seed=SEED, dtype=dy))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 5), (8, 0)])
def test_strides(U, dtype, pad, shift):
    """Any row stride and alignment; what lies between a result's rows stays."""
    g = np.random.default_rng([pad, shift])
    w = U.ufp4_quantize(torch.randn(200, 400, device="cuda"), U.UFP4_E1M2)
    x = _x(g, (6, 400), dtype, pad, shift)
    buf = torch.full((6 * (200 + pad) + shift,), 77.0, device="cuda", dtype=dtype)
    out = buf[shift:].view(6, 200 + pad)[:, :200]
    assert U.ufp4_gemv(x, w, out=out) is out
    _check(out, x, _values(w, U.UFP4_E1M2)[0], False, dtype)
    rest = buf.clone()
    rest[shift:].view(6, 200 + pad)[:, :200] = 77.0
    assert bool((rest == 77.0).all())


@pytest.mark.parametrize("scale", [2.0 ** -120, 1e-30, 1e30, 2.0 ** 120])
@pytest.mark.parametrize("rht", [False, True])
def test_range(U, scale, rht):
    """Tokens far from 1, weights too: neither passes through FP16's range."""
    g = np.random.default_rng(5)
    w = torch.from_numpy(g.standard_normal((64, 256)).astype(np.float32) / np.float32(scale)).cuda()
    q = U.ufp4_quantize(w, U.UFP4_E2M1, rht=rht, rht_seed=SEED)
    x = _x(g, (3, 256), FP) * scale
    y = U.ufp4_gemv(x, q, rht=rht, rht_seed=SEED)
    _check(y, x, _values(q, U.UFP4_E2M1)[0], rht, FP)


def test_uneven_token(U):
    """Chunks of a token that differ by 2^60, and one element far above its chunk's others."""
    x = torch.randn(2, 1024, device="cuda")
    x[0, 128:256] *= 2.0 ** 60
    x[0, 512:640] *= 2.0 ** -60
    x[1, 77] = 2.0 ** 20
    q = U.ufp4_quantize(torch.randn(40, 1024, device="cuda"), U.UFP4_E1M2)
    _check(U.ufp4_gemv(x, q), x, _values(q, U.UFP4_E1M2)[0], False, FP)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rht", [False, True])
def test_non_finite_tokens(U, dtype, rht):
    """A NaN makes its token's results NaN, an infinity non-finite, and no other token's."""
    g = np.random.default_rng(1)
    q = U.ufp4_quantize(torch.randn(50, 320, device="cuda"), U.UFP4_E1M2, rht=rht, rht_seed=SEED)
    clean = _x(g, (5, 320), dtype)
    x = clean.clone()
    x[1, 130], x[3, 7] = float("nan"), float("inf")
    a, b = (U.ufp4_gemv(t, q, rht=rht, rht_seed=SEED, dtype=FP) for t in (clean, x))
    assert torch.isnan(b[1]).all() and not torch.isfinite(b[3]).any()
    assert torch.equal(a[[0, 2, 4]], b[[0, 2, 4]])
    if not rht:      # an infinity times a weight is that infinity, or NaN where the weight is zero
        w = torch.from_numpy(_values(q, U.UFP4_E1M2)[0][:, 7]).cuda()
        assert torch.equal(torch.isnan(b[3]), w == 0)
        assert bool(((b[3] > 0) == (w > 0))[w != 0].all())


def test_empty(U):
    q = U.ufp4_quantize(torch.randn(32, 64, device="cuda"), U.UFP4_E2M1)
    assert U.ufp4_gemv(torch.empty(0, 64, device="cuda"), q).shape == (0, 32)
    none = U.QTensor.empty(32, 0, U.UFP4_E2M1)
    assert bool((U.ufp4_gemv(torch.empty(3, 0, device="cuda"), none) == 0).all())


def test_offsets_past_32_bits(U):
    """A matrix of 5 GB of codes: its first and last rows."""
    rows, k = 1200128 + 3, 8192
    q = U.QTensor.empty(rows, k, U.UFP4_E2M1)
    step = 1 << 28
    for a in range(0, q.codes.numel(), step):
        q.codes[a:a + step].random_(0, 256)
    q.scales.random_(0x30, 0x40)
    q.tensor_scale.fill_(0.125)
    x = torch.randn(1, k, device="cuda")
    y = U.ufp4_gemv(x, q)
    nkt = kpad(k) // 64
    for r in (0, 130, rows // 2, rows - 129, rows - 2, rows - 1):
        codes = R.unpack(q.codes_2d()[r].cpu().numpy())
        b = np.arange(k // 16)
        at = ((r // 128) * nkt + b // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + b % 4
        w = R.values(codes, q.scales[torch.from_numpy(at).cuda()].cpu().numpy(), 0) * 0.125
        _check(y[:, r:r + 1], x, w[None], False, FP)


# ------------------------------------------------------------------ by expert
def _grouped(U, g, experts, rows, k, grid, rht):
    w = torch.from_numpy(g.standard_normal((experts * rows, k)).astype(np.float32)).cuda()
    q = U.ufp4_quantize_grouped(w.to(BF), grid, [rows] * experts, rht=rht, rht_seed=SEED)
    v = _values(q, grid, rows, experts)
    assert q.rows == experts * rpad(rows)
    return q, v


def _ids(g, tokens, topk, experts, kind):
    ids = g.integers(0, experts, size=(tokens, topk))
    if kind == "some":
        ids[g.random(tokens) < 0.3] = -1
        ids[g.random(ids.shape) < 0.1] = experts
    elif kind == "one":
        ids[:] = experts - 1
    elif kind == "none":
        ids[:] = -1
    return ids


@pytest.mark.parametrize("tokens,topk,experts,rows,k", [(1, 1, 1, 16, 16), (1, 6, 64, 200, 208), (1, 4, 3, 130, 64),
                                                         (5, 2, 7, 128, 512), (8, 8, 256, 33, 144),
                                                         (33, 3, 5, 257, 1040), (64, 6, 16, 96, 704),
                                                         (200, 2, 4, 64, 320), (9, 2, 3, 40, 8208)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("kind", ["all", "some", "one", "none"])
def test_by_expert(U, tokens, topk, experts, rows, k, gather, kind):
    """Experts without tokens, dropped slots, every token at one expert (an
    expert that a token names more than once among them)."""
    g = np.random.default_rng([tokens, topk, experts, rows, k])
    rht, grid = bool(tokens % 2), (U.UFP4_E1M2, U.UFP4_E2M1)[topk % 2]
    dx, dy = ((BF, FP), (FP, BF))[gather]
    q, v = _grouped(U, g, experts, rows, k, grid, rht)
    ids = _ids(g, tokens, topk, experts, kind)
    plan = U.ufp4_moe_sort(torch.from_numpy(ids).cuda(), experts)
    x = _x(g, (tokens if gather else tokens * topk, k), dx)
    buf = torch.full((tokens * topk, rows + 3), 5.0, device="cuda", dtype=dy)
    y = U.ufp4_gemv_grouped(x, q, plan, rows, gather=gather, rht=rht, rht_seed=SEED, out=buf[:, :rows])
    assert bool((buf[:, rows:] == 5.0).all())
    src, off = plan.src.cpu().numpy(), plan.offsets.cpu().numpy()
    for e in range(experts):
        a, b = off[e], off[e + 1]
        if a < b:
            at = src[a:b] // topk if gather else np.arange(a, b)
            _check(y[a:b], x[torch.from_numpy(np.asarray(at)).cuda()], v[e], rht, dy, e)
    assert bool((y[int(off[-1]):] == 0).all())


def test_a_decoding_step_in_a_graph(U):
    """The whole routed layer for a few tokens, captured once and replayed
    with other tokens and other experts: sort, both products, gated activation
    and the way back, without a count on the host."""
    tokens, topk, experts, hidden, ffn = 4, 2, 8, 256, 192
    g = np.random.default_rng(3)
    w13, v13 = _grouped(U, g, experts, 2 * ffn, hidden, U.UFP4_E1M2, True)
    w2, v2 = _grouped(U, g, experts, hidden, ffn, U.UFP4_E1M2, True)
    rot = dict(rht=True, rht_seed=SEED)

    def layer(x, ids, weights):
        plan = U.ufp4_moe_sort(ids, experts)
        gu = U.ufp4_gemv_grouped(x, w13, plan, 2 * ffn, gather=True, dtype=FP, **rot)
        h, _, _ = U.ufp4_swiglu(gu[:, :ffn], gu[:, ffn:], dtype=FP)
        y = U.ufp4_gemv_grouped(h, w2, plan, hidden, **rot)
        return U.ufp4_moe_combine(y, plan, weights)

    new = lambda: (torch.randn(tokens, hidden, device="cuda"),  # noqa: E731
                   torch.from_numpy(_ids(g, tokens, topk, experts, "some")).cuda(),
                   torch.rand(tokens, topk, device="cuda"))
    held = new()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(*held)
    r = R.rotation(SEED)
    turn = lambda w: (w.reshape(w.shape[:-1] + (-1, 16)) @ r).reshape(w.shape)  # noqa: E731
    u13, u2 = turn(v13), turn(v2)
    for _ in range(3):
        args = new()
        for a, b in zip(held, args):
            a.copy_(b)
        graph.replay()
        assert torch.equal(out, layer(*args))
        x, ids, w = _f64(args[0]), args[1].cpu().numpy(), _f64(args[2])
        want = np.zeros((tokens, hidden))
        for t in range(tokens):
            for j in range(topk):
                if 0 <= ids[t, j] < experts:
                    gu = u13[ids[t, j]] @ x[t]
                    want[t] += w[t, j] * (u2[ids[t, j]] @ (gu[:ffn] / (1 + np.exp(-gu[:ffn])) * gu[ffn:]))
        # each product's sums (some 300 additions of 2^-23), through a product of norms: 1e-4 is 3 times their sum
        assert np.linalg.norm(_f64(out) - want) <= 1e-4 * np.linalg.norm(want)


def test_results_on_a_side_stream(U):
    q = U.ufp4_quantize(torch.randn(512, 512, device="cuda"), U.UFP4_E1M2)
    x = torch.randn(4, 512, device="cuda")
    want, side = U.ufp4_gemv(x, q), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = U.ufp4_gemv(x, q, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_refusals(U):
    q = U.ufp4_quantize(torch.randn(32, 64, device="cuda"), U.UFP4_E2M1)
    x = torch.randn(2, 64, device="cuda")
    with pytest.raises(U.UFP4Error):
        U.ufp4_gemv(x, U.ufp4_quantize(torch.randn(32, 64, device="cuda"), U.UFP4_MXFP4))
    for bad in (x[:, :48], x[0], x.t()):
        with pytest.raises(ValueError):
            U.ufp4_gemv(bad, q)
    with pytest.raises(TypeError):
        U.ufp4_gemv(x.half(), q)
    with pytest.raises(TypeError):
        U.ufp4_gemv(x, q, dtype=torch.float16)
    with pytest.raises(TypeError):
        U.ufp4_gemv(x.cpu(), q)
    w = U.ufp4_quantize_grouped(torch.randn(64, 64, device="cuda"), U.UFP4_E2M1, [32, 32])
    plan = U.ufp4_moe_sort(torch.zeros(2, 2, dtype=torch.int64, device="cuda"), 2)
    four = torch.randn(4, 64, device="cuda")
    assert U.ufp4_gemv_grouped(four, w, plan, 32).shape == (4, 32)
    with pytest.raises(ValueError):
        U.ufp4_gemv_grouped(x, w, plan, 32)
    with pytest.raises(ValueError):
        U.ufp4_gemv_grouped(four, w, plan, 32, gather=True)
    with pytest.raises(U.UFP4Error):
        U.ufp4_gemv_grouped(four, w, plan, 200)
    other = U.ufp4_moe_sort(torch.zeros(2, 2, dtype=torch.int64, device="cuda"), 3)
    with pytest.raises(ValueError):
        U.ufp4_gemv_grouped(four, w, other, 32)
