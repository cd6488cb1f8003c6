"""CPU-only checks of the calls around the grouped GEMMs: arguments they
refuse (before any launch), sizes they give, and the plain forms that the GPU
tests compare with."""
import ctypes

import numpy as np
import pytest

from tests import rowop_refs as R


@pytest.fixture(scope="module")
def U():
    from fp4_quantized_numerics_gb300 import build, ufp4
    build.build()
    ufp4.lib()
    return ufp4


P = 0x10000     # never dereferenced: every call here is refused


def _plan(U, tokens=8, topk=2, experts=4, **kw):
    f = dict(pos=P, src=P, counts=P, offsets=P, tokens=tokens, topk=topk, n_experts=experts, reserved=0)
    f.update(kw)
    return ctypes.byref(U.MoePlanC(*[f[n] for n, _ in U.MoePlanC._fields_]))


def _ckpt(U, rows=8, cols=64, fmt=0, codes=P, scales=P, reserved=0):
    return ctypes.byref(U.CkptC(codes, scales, rows, cols, fmt, reserved))


BAD_PLANS = [dict(reserved=1), dict(tokens=-1), dict(topk=0), dict(experts=0), dict(experts=257), dict(pos=None),
             dict(src=None), dict(counts=None), dict(offsets=None), dict(pos=P + 2), dict(src=P + 1),
             dict(counts=P + 4), dict(offsets=P + 4)]


def _calls(U):
    """Each call with a plan as a function of that plan."""
    L = U.lib()
    return [lambda p: L.ufp4_moe_sort(P, 8, p, None),
            lambda p: L.ufp4_moe_dispatch(P, 0, 64, 64, p, P, 64, None),
            lambda p: L.ufp4_moe_combine(P, 1, 64, 64, p, P, P, 0, 64, None),
            lambda p: L.ufp4_moe_combine_bwd(P, 0, 64, P, 1, 64, 64, p, P, P, 0, 64, P, None)]


@pytest.mark.parametrize("bad", BAD_PLANS, ids=str)
def test_bad_plans_are_refused(U, bad):
    for call in _calls(U):
        assert call(_plan(U, **bad)) == U.UFP4_ERR_INVALID
        assert call(None) == U.UFP4_ERR_INVALID


def test_plans_past_the_limits(U):
    for call in _calls(U):
        assert call(_plan(U, tokens=1 << 30, topk=2)) == U.UFP4_ERR_UNSUPPORTED


def test_sort_refusals(U):
    L = U.lib()
    assert L.ufp4_moe_sort(P, 2, _plan(U), None) == U.UFP4_ERR_INVALID        # id size
    assert L.ufp4_moe_sort(None, 8, _plan(U), None) == U.UFP4_ERR_INVALID
    assert L.ufp4_moe_sort(P + 4, 8, _plan(U), None) == U.UFP4_ERR_INVALID    # alignment


def test_moe_row_refusals(U):
    L, p, INV, UNS = U.lib(), _plan(U), U.UFP4_ERR_INVALID, U.UFP4_ERR_UNSUPPORTED

    def disp(x=P, dt=0, h=64, lx=64, xs=P, ls=64):
        return L.ufp4_moe_dispatch(x, dt, h, lx, p, xs, ls, None)

    def comb(y=P, ty=1, h=64, ly=64, w=P, o=P, to=0, lo=64):
        return L.ufp4_moe_combine(y, ty, h, ly, p, w, o, to, lo, None)

    def bwd(d=P, td=0, ld=64, y=P, ty=1, ly=64, h=64, w=P, dy=P, ty2=0, ldy=64, dw=P):
        return L.ufp4_moe_combine_bwd(d, td, ld, y, ty, ly, h, p, w, dy, ty2, ldy, dw, None)

    for kw in (dict(x=None), dict(xs=None), dict(dt=2), dict(h=-1), dict(lx=63), dict(ls=63), dict(x=P + 1),
               dict(xs=P + 1), dict(dt=1, x=P + 2)):
        assert disp(**kw) == INV, kw
    for kw in (dict(y=None), dict(o=None), dict(ty=2), dict(to=-1), dict(h=-1), dict(ly=63), dict(lo=63),
               dict(y=P + 2), dict(o=P + 1), dict(w=P + 2)):
        assert comb(**kw) == INV, kw
    for kw in (dict(d=None), dict(y=None), dict(w=None), dict(dy=None), dict(dw=None), dict(td=3), dict(ty=3),
               dict(ty2=3), dict(ld=63), dict(ly=63), dict(ldy=63), dict(h=-1), dict(w=P + 1), dict(dw=P + 2)):
        assert bwd(**kw) == INV, kw
    big = 1 << 25
    assert disp(h=big, lx=big, ls=big) == UNS
    assert comb(h=big, ly=big, lo=big) == UNS
    assert bwd(h=big, ld=big, ly=big, ldy=big) == UNS
    assert disp(lx=1 << 31) == UNS and comb(ly=1 << 31) == UNS and bwd(ldy=1 << 31) == UNS
    p = _plan(U, tokens=1 << 20, topk=2)
    wide = 1 << 18
    assert disp(h=wide, lx=wide, ls=wide) == UNS          # 2^21 rows of 2^18
    p = _plan(U, tokens=0, pos=None, src=None)
    assert disp(x=None, xs=None) == comb(y=None, o=None, w=None) == bwd(d=None, y=None, w=None, dy=None, dw=None) == 0
    p = _plan(U)
    assert disp(h=0) == comb(h=0) == U.UFP4_OK


def test_ckpt_refusals(U):
    L, INV, UNS = U.lib(), U.UFP4_ERR_INVALID, U.UFP4_ERR_UNSUPPORTED
    bad = [_ckpt(U, reserved=1), _ckpt(U, rows=-1), _ckpt(U, cols=-1), _ckpt(U, fmt=2), _ckpt(U, codes=None),
           _ckpt(U, scales=None), _ckpt(U, codes=P + 8), None]
    for c in bad:
        assert L.ufp4_ckpt_save(P, 0, 64, c, None) == INV
        assert L.ufp4_ckpt_load(c, P, 0, 64, None) == INV
        assert L.ufp4_swiglu_bwd(P, 0, 64, c, _ckpt(U), P, 64, P, 64, 0, None) == INV
        assert L.ufp4_swiglu_bwd(P, 0, 64, _ckpt(U), c, P, 64, P, 64, 0, None) == INV
        if c is not None:
            assert L.ufp4_swiglu(P, 64, P, 64, 0, 8, 64, P, 0, 64, c, _ckpt(U), None) == INV
            assert L.ufp4_swiglu(P, 64, P, 64, 0, 8, 64, P, 0, 64, _ckpt(U), c, None) == INV
    for kw in ((None, 0, 64), (P, 2, 64), (P, 0, 63), (P + 1, 0, 64), (P + 2, 1, 64)):
        assert L.ufp4_ckpt_save(*kw, _ckpt(U), None) == INV
        assert L.ufp4_ckpt_load(_ckpt(U), *kw, None) == INV
    assert L.ufp4_ckpt_save(P, 0, 1 << 25, _ckpt(U, cols=1 << 25), None) == UNS
    assert L.ufp4_ckpt_load(_ckpt(U, rows=1 << 20, cols=1 << 18), P, 0, 1 << 18, None) == UNS
    assert L.ufp4_ckpt_save(None, 0, 64, _ckpt(U, rows=0, codes=None, scales=None), None) == U.UFP4_OK


def test_swiglu_refusals(U):
    L, INV, UNS = U.lib(), U.UFP4_ERR_INVALID, U.UFP4_ERR_UNSUPPORTED

    def fwd(g=P, lg=64, u=P, lu=64, ti=0, rows=8, cols=64, h=P, th=0, lh=64, kg=None, ku=None):
        return L.ufp4_swiglu(g, lg, u, lu, ti, rows, cols, h, th, lh, kg, ku, None)

    for kw in (dict(g=None), dict(u=None), dict(h=None), dict(ti=2), dict(th=2), dict(lg=63), dict(lu=63),
               dict(lh=63), dict(rows=-1), dict(cols=-1), dict(g=P + 1), dict(kg=_ckpt(U)), dict(ku=_ckpt(U)),
               dict(kg=_ckpt(U), ku=_ckpt(U, fmt=1)), dict(kg=_ckpt(U, rows=7), ku=_ckpt(U, rows=7)),
               dict(kg=_ckpt(U), ku=_ckpt(U, cols=32))):
        assert fwd(**kw) == INV, kw
    big = 1 << 25
    assert fwd(cols=big, lg=big, lu=big, lh=big) == UNS
    assert fwd(rows=0, g=None, u=None, h=None) == U.UFP4_OK

    def bwd(d=P, td=0, ld=64, kg=None, ku=None, dg=P, lg=64, du=P, lu=64, to=0):
        return L.ufp4_swiglu_bwd(d, td, ld, kg or _ckpt(U), ku or _ckpt(U), dg, lg, du, lu, to, None)

    for kw in (dict(d=None), dict(dg=None), dict(du=None), dict(td=2), dict(to=2), dict(ld=63), dict(lg=63),
               dict(lu=63), dict(ku=_ckpt(U, fmt=1)), dict(ku=_ckpt(U, rows=7)), dict(ku=_ckpt(U, cols=32))):
        assert bwd(**kw) == INV, kw
    assert bwd(kg=_ckpt(U, cols=big), ku=_ckpt(U, cols=big), ld=big, lg=big, lu=big) == UNS


def test_ckpt_sizes(U):
    L = U.lib()
    for cols, ld, nb in ((0, 0, 0), (1, 16, 1), (16, 16, 1), (33, 48, 2), (1408, 1408, 44)):
        assert L.ufp4_ckpt_ld(cols) == ld
        assert L.ufp4_ckpt_codes_bytes(3, cols) == 3 * ld
        assert L.ufp4_ckpt_scales_bytes(3, cols) == 3 * nb
    assert L.ufp4_ckpt_codes_bytes(0, 64) == L.ufp4_ckpt_scales_bytes(-1, 64) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes(U):
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        U.ufp4_moe_sort(torch.zeros(4, 2, dtype=torch.int64), 4)
    with pytest.raises(TypeError):
        U.ufp4_ckpt_save(x)
    with pytest.raises(TypeError):
        U.ufp4_swiglu(x, x)
    with pytest.raises(TypeError):
        U.MoePlan(torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                  torch.zeros(4, dtype=torch.int64), torch.zeros(5, dtype=torch.int64))


# ------------------------------------------------- the plain forms themselves
def test_plain_e4m3_is_the_format(U):
    """Every value of the plain E4M3 grid is an E4M3 number, and every E4M3
    number comes back unchanged."""
    import torch
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    every = every[np.isfinite(every)]
    for lo in range(0, every.size, 31):
        part = every[lo:lo + 31]
        block = np.concatenate([[256.0], part])[None]     # at the top of the block: scale 1 unless 448 is passed
        scales, back = R.ckpt(block, 1)
        assert scales[0, 0] == 127
        np.testing.assert_array_equal(back[0, 1:], part)
    g = np.random.default_rng(1)
    v = g.standard_normal((20, 32))
    scales, back = R.ckpt(v, 1)
    u = back / 2.0 ** (scales.astype(np.float64) - 127)
    t = torch.from_numpy(u).float()
    np.testing.assert_array_equal(t.to(torch.float8_e4m3fn).float().numpy(), u)


def test_plain_int8_error_and_range():
    g = np.random.default_rng(2)
    v = g.standard_normal((50, 100)) * 2.0 ** g.integers(-30, 30, size=(50, 1))
    scales, back = R.ckpt(v, 0)
    step = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, axis=1)[:, :100]
    assert np.all(np.abs(back / step) <= 127) and np.all(np.abs(v - back) <= step)
    within = np.abs(v / step) <= 127.5
    assert np.all(np.abs(v - back)[within] <= 0.5 * step[within]) and within.mean() > 0.99


def test_plain_combine_and_its_gradients_agree():
    g = np.random.default_rng(3)
    ids = g.integers(-1, 5, size=(20, 3))
    pos, src, counts, offsets = R.sort(ids, 5)
    routed = offsets[-1]
    assert sorted(pos.reshape(-1)) == list(range(60)) and np.array_equal(pos.reshape(-1)[src], np.arange(60))
    x, y, d = g.standard_normal((20, 7)), g.standard_normal((60, 7)), g.standard_normal((20, 7))
    w = g.random((20, 3))
    dy, dw, _ = R.combine_bwd(d, y, pos, routed, w)
    out = R.combine(y, pos, routed, w)[0]
    assert np.sum(d * out) == pytest.approx(np.sum(dy * y)) == pytest.approx(np.sum(dw * w))
    assert np.sum(R.dispatch(x, pos, routed) * y) == pytest.approx(np.sum(x * R.combine(y, pos, routed)[0]))


def test_plain_swiglu_gradient_by_differences():
    g = np.random.default_rng(4)
    a, b, d = g.standard_normal((3, 200)) * 3
    da, db = R.swiglu_bwd(d, a, b)
    e = 1e-6
    np.testing.assert_allclose(d * (R.swiglu(a + e, b) - R.swiglu(a - e, b)) / (2 * e), da, rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(d * (R.swiglu(a, b + e) - R.swiglu(a, b - e)) / (2 * e), db, rtol=1e-6, atol=1e-7)
