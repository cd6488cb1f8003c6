"""What the calls around the grouped GEMMs write: every element of their
results and nothing else.  Each result is a view into a larger buffer filled
with a known byte; the call is made twice, with different bytes, and has to
give the same view and leave the rest as it was (rows' gaps, what comes before
and after, the padding of rows of 8-bit codes)."""
import numpy as np
import pytest
import torch

from tests import rowop_refs as R

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
FILLS = (0xA5, 0x5A)
LEAD = 256                                   # bytes before a result, and after it


@pytest.fixture(scope="module")
def U():
    from fp4_quantized_numerics_gb300 import build, ufp4
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return ufp4


class Guarded:
    """A rows x cols view, row stride cols + pad, `shift` elements and LEAD
    bytes into a buffer."""

    def __init__(self, rows, cols, dtype, pad=0, shift=0):
        size = torch.empty(0, dtype=dtype).element_size()
        ld = cols + pad
        self.bytes = torch.empty(2 * LEAD + (rows * ld + shift) * size, device="cuda", dtype=torch.uint8)
        at = LEAD // size + shift
        self.view = self.bytes.view(dtype)[at:at + rows * ld].view(rows, ld)[:, :cols]
        mine = torch.zeros_like(self.bytes, dtype=torch.bool)
        mine[at * size:(at + rows * ld) * size].view(rows, ld * size)[:, :cols * size] = True
        self.others = ~mine

    def fill(self, byte):
        self.byte = byte
        self.bytes.fill_(byte)

    def check(self):
        assert bool((self.bytes[self.others] == self.byte).all()), "written outside the result"


def _twice(results, call):
    seen = []
    for byte in FILLS:
        for r in results:
            r.fill(byte)
        call()
        for r in results:
            r.check()
        seen.append([r.view.contiguous().view(torch.uint8) for r in results])
    for a, b in zip(*seen):
        assert torch.equal(a, b), "an element was not written"


def _values(g, rows, cols, dtype, pad=0, shift=0):
    buf = torch.zeros(rows * (cols + pad) + shift, device="cuda", dtype=dtype)
    t = buf[shift:].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.from_numpy(g.standard_normal((rows, cols)).astype(np.float32)))
    return t


# (rows, cols, pad, shift): sixteens, eights, pairs and singles a thread; blocks and rows that end early
SHAPES = [(5, 48, 16, 0), (3, 272, 0, 0), (5, 40, 8, 0), (9, 8, 0, 0), (6, 34, 2, 2), (4, 1002, 0, 0), (5, 40, 2, 0),
          (7, 72, 3, 1), (9, 33, 0, 0), (3, 1001, 1, 0), (3, 1, 0, 0), (5, 1, 6, 1), (2, 31, 1, 1), (257, 16, 0, 0)]
DTYPES = [(BF, FP), (FP, BF), (BF, BF), (FP, FP)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtypes", DTYPES, ids=lambda d: "-".join(str(t)[6:] for t in d))
def test_rows_in_and_out_of_expert_order(U, shape, dtypes):
    tokens, hidden, pad, shift = shape
    ti, to = dtypes
    g = np.random.default_rng(20)
    topk, experts = 3, 5
    ids = g.integers(-1, experts + 1, size=(tokens, topk))
    plan = U.ufp4_moe_sort(torch.from_numpy(ids).cuda(), experts)
    w = torch.from_numpy(g.random((tokens, topk)).astype(np.float32)).cuda()
    x, y = _values(g, tokens, hidden, ti, pad, shift), _values(g, tokens * topk, hidden, ti, pad, shift)
    xs, out = Guarded(tokens * topk, hidden, ti, pad, shift), Guarded(tokens, hidden, to, pad, shift)
    dy, dw = Guarded(tokens * topk, hidden, to, pad, shift), Guarded(tokens, topk, FP)
    _twice([xs], lambda: U.ufp4_moe_dispatch(x, plan, out=xs.view))
    _twice([out], lambda: U.ufp4_moe_combine(y, plan, w, out=out.view))
    _twice([out], lambda: U.ufp4_moe_combine(y, plan, out=out.view))
    _twice([dy, dw], lambda: U.ufp4_moe_combine_bwd(x, y, plan, w, dy=dy.view, dw=dw.view))


def _ckpt(U, rows, cols, fmt):
    """A checkpoint in guarded buffers: codes (padding beside them) and scales."""
    width = (cols + 15) // 16 * 16
    codes, scales = Guarded(rows, cols, torch.uint8, width - cols), Guarded(rows, (cols + 31) // 32, torch.uint8)
    whole = codes.bytes[LEAD:LEAD + rows * width].view(rows, width)
    return U.Ckpt(whole, scales.view, rows, cols, fmt), codes, scales


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtypes", DTYPES, ids=lambda d: "-".join(str(t)[6:] for t in d))
@pytest.mark.parametrize("fmt", [0, 1])
def test_checkpoints_and_activation(U, shape, dtypes, fmt):
    rows, cols, pad, shift = shape
    ti, to = dtypes
    g = np.random.default_rng(21)
    gate, up = _values(g, rows, cols, ti, pad, shift), _values(g, rows, cols, ti, pad, shift)
    (kg, *cg), (ku, *cu) = _ckpt(U, rows, cols, fmt), _ckpt(U, rows, cols, fmt)
    h, back = Guarded(rows, cols, to, pad, shift), Guarded(rows, cols, to, pad, shift)
    _twice(cg, lambda: U.ufp4_ckpt_save(gate, fmt, out=kg))
    _twice([back], lambda: U.ufp4_ckpt_load(kg, out=back.view))
    _twice([h], lambda: U.ufp4_swiglu(gate, up, out=h.view))
    _twice([h, *cg, *cu], lambda: U.ufp4_swiglu(gate, up, out=h.view, keep=(kg, ku)))
    dgate, dup = Guarded(rows, cols, to, pad, shift), Guarded(rows, cols, to, pad, shift)
    _twice([dgate, dup], lambda: U.ufp4_swiglu_bwd(gate, kg, ku, dgate=dgate.view, dup=dup.view))


# one, eight and sixteen CTAs, on both sides of each change; slots that end inside a warp's share; many slots
@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 6, 64), (512, 2, 64), (205, 5, 64), (1025, 1, 256),
                                                 (2048, 4, 64), (8193, 1, 7), (16384, 6, 64), (65537, 8, 256),
                                                 (131072, 4, 1)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(U, tokens, topk, experts, dtype):
    n = tokens * topk
    g = np.random.default_rng(n)
    ids = g.integers(-1 if experts > 1 else 0, experts + (experts > 7), size=(tokens, topk))
    pos, src = Guarded(tokens, topk, torch.int32), Guarded(1, n, torch.int32)
    counts, offsets = Guarded(1, experts, torch.int64), Guarded(1, experts + 1, torch.int64)
    plan = U.MoePlan(pos.view, src.view.view(-1), counts.view.view(-1), offsets.view.view(-1))
    given = torch.from_numpy(ids).to(dtype).cuda()
    _twice([pos, src, counts, offsets], lambda: U.ufp4_moe_sort(given, experts, out=plan))
    want = R.sort(ids, experts)
    for got, exact in zip((plan.pos, plan.src, plan.counts, plan.offsets), want):
        np.testing.assert_array_equal(got.cpu().numpy(), exact)
