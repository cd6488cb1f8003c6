"""CPU-only checks of the calls that answer with a quantized model: arguments
they refuse (before any launch), sizes they give, and the plain forms that the
GPU tests compare with."""
import ctypes

import numpy as np
import pytest

from tests import serving_refs as R


@pytest.fixture(scope="module")
def U():
    from fp4_quantized_numerics_gb300 import build, ufp4
    build.build()
    ufp4.lib()
    return ufp4


P = 0x10000     # never dereferenced: every call here is refused, or has nothing to do


def _w(U, rows=128, k=64, grid=1, codes=P, scales=P, ts=P, reserved=0):
    return ctypes.byref(U.QTensorC(codes, scales, ts, rows, k, grid, reserved, None))


def _plan(U, tokens=8, topk=2, experts=4, **kw):
    f = dict(pos=P, src=P, counts=P, offsets=P, tokens=tokens, topk=topk, n_experts=experts, reserved=0)
    f.update(kw)
    return ctypes.byref(U.MoePlanC(*[f[n] for n, _ in U.MoePlanC._fields_]))


def _cache(U, **kw):
    f = dict(k_codes=P, k_scales=P, k_row_scale=P, v_codes=P, v_scales=P, v_row_scale=P, pages=4, heads=2, page=16,
             head_dim=64, grid=1, rht=0, reserved=0, rht_seed=0)
    f.update(kw)
    return ctypes.byref(U.CacheC(*[f[n] for n, _ in U.CacheC._fields_]))


def test_gemv_refusals(U):
    L, INV, UNS = U.lib(), U.UFP4_ERR_INVALID, U.UFP4_ERR_UNSUPPORTED

    def call(x=P, dt=0, t=3, ld=64, w=None, rht=0, y=P, ty=1, ly=128):
        return L.ufp4_gemv(x, dt, t, ld, _w(U) if w is None else w, rht, 7, y, ty, ly, None)

    for kw in (dict(x=None), dict(y=None), dict(dt=2), dict(ty=-1), dict(t=-1), dict(ld=63), dict(ly=127), dict(x=P + 1),
               dict(dt=1, x=P + 2), dict(y=P + 2), dict(rht=2)):
        assert call(**kw) == INV, kw
    for w in (_w(U, codes=None), _w(U, scales=None), _w(U, ts=None), _w(U, codes=P + 8), _w(U, k=72), _w(U, rows=-1),
              _w(U, grid=9), _w(U, reserved=1)):
        assert call(w=w) == INV
    assert L.ufp4_gemv(P, 0, 3, 64, None, 0, 7, P, 1, 128, None) == INV
    assert call(w=_w(U, grid=U.UFP4_MXFP4)) == UNS
    assert call(w=_w(U, k=1 << 25), ld=1 << 25) == UNS
    assert call(ld=1 << 31) == UNS and call(ly=1 << 31) == UNS and call(t=(1 << 30) + 1) == UNS
    assert call(t=0, x=None, y=None) == U.UFP4_OK
    assert call(w=_w(U, rows=0, codes=None, scales=None, ts=None), y=None, ly=0) == U.UFP4_OK


def test_gemv_grouped_refusals(U):
    L, INV, UNS = U.lib(), U.UFP4_ERR_INVALID, U.UFP4_ERR_UNSUPPORTED

    def call(x=P, dt=0, ld=64, gather=0, w=None, rows=100, plan=None, rht=0, y=P, ty=1, ly=100):
        return L.ufp4_gemv_grouped(x, dt, ld, gather, _w(U, rows=512) if w is None else w, rows,
                                   _plan(U) if plan is None else plan, rht, 7, y, ty, ly, None)

    for kw in (dict(x=None), dict(y=None), dict(dt=2), dict(ty=2), dict(ld=63), dict(ly=99), dict(gather=2), dict(rht=-1),
               dict(rows=-1), dict(rows=129), dict(x=P + 1), dict(y=P + 1), dict(w=_w(U, rows=500)),
               dict(w=_w(U, rows=512, codes=None)), dict(plan=_plan(U, reserved=1)), dict(plan=_plan(U, experts=257)),
               dict(plan=_plan(U, src=None)), dict(plan=_plan(U, offsets=None))):
        assert call(**kw) == INV, kw
    assert call(w=_w(U, rows=512, grid=U.UFP4_MXFP4)) == UNS
    assert call(ld=1 << 31) == UNS
    assert call(plan=_plan(U, tokens=1 << 30)) == UNS
    assert call(plan=_plan(U, tokens=0, pos=None, src=None), x=None, y=None) == U.UFP4_OK


BAD_CACHES = [dict(reserved=1), dict(pages=-1), dict(heads=0), dict(page=0), dict(page=24), dict(head_dim=0),
              dict(head_dim=40), dict(rht=2), dict(grid=7), dict(k_codes=None), dict(v_codes=None), dict(k_scales=None),
              dict(v_row_scale=None), dict(k_codes=P + 8), dict(v_scales=P + 4), dict(k_row_scale=P + 4)]
OTHER_CACHES = [dict(page=8), dict(page=1 << 16), dict(head_dim=272), dict(grid=3), dict(heads=1 << 17)]


def _cache_calls(U):
    L = U.lib()
    return [lambda c: L.ufp4_cache_append(P, P, 0, 3, 1024, 512, 1024, 512, P, c, None),
            lambda c: L.ufp4_cache_load(c, P, 3, P, P, 0, 1024, 512, 1024, 512, None),
            lambda c: L.ufp4_cache_attn(P, 0, 1024, 512, 1, 1, 2, c, P, 4, 4, P, None, 1.0, P, 0, 1024, 512, None, None, 0,
                                        None)]


@pytest.mark.parametrize("bad", BAD_CACHES + [None], ids=str)
def test_bad_caches_are_refused(U, bad):
    for call in _cache_calls(U):
        assert call(None if bad is None else _cache(U, **bad)) == U.UFP4_ERR_INVALID


@pytest.mark.parametrize("other", OTHER_CACHES, ids=str)
def test_caches_that_are_not_supported(U, other):
    for call in _cache_calls(U):
        assert call(_cache(U, **other)) == U.UFP4_ERR_UNSUPPORTED


def test_append_and_load_refusals(U):
    L, INV, UNS = U.lib(), U.UFP4_ERR_INVALID, U.UFP4_ERR_UNSUPPORTED

    def both(k=P, v=P, dt=0, t=3, lk=128, hk=64, lv=128, hv=64, slots=P):
        a = L.ufp4_cache_append(k, v, dt, t, lk, hk, lv, hv, slots, _cache(U), None)
        b = L.ufp4_cache_load(_cache(U), slots, t, k, v, dt, lk, hk, lv, hv, None)
        assert a == b
        return a

    for kw in (dict(k=None), dict(v=None), dict(dt=2), dict(t=-1), dict(lk=63), dict(hk=63), dict(lv=63), dict(hv=63),
               dict(slots=None), dict(slots=P + 4), dict(k=P + 1), dict(dt=1, v=P + 2)):
        assert both(**kw) == INV, kw
    assert both(lk=1 << 31) == UNS and both(hv=1 << 31) == UNS and both(t=1 << 31) == UNS
    assert both(t=0, k=None, v=None, slots=None) == U.UFP4_OK


def test_attn_refusals(U):
    L, INV, UNS = U.lib(), U.UFP4_ERR_INVALID, U.UFP4_ERR_UNSUPPORTED

    def call(q=P, dt=0, lq=256, hq=64, batch=2, m=1, heads=4, c=None, table=P, lt=8, width=8, lens=P, mask=None,
             scale=1.0, out=P, to=0, lo=256, ho=64, lse=None, ws=None, size=0):
        return L.ufp4_cache_attn(q, dt, lq, hq, batch, m, heads, c or _cache(U), table, lt, width, lens, mask, scale, out,
                                 to, lo, ho, lse, ws, size, None)

    for kw in (dict(q=None), dict(out=None), dict(dt=2), dict(to=2), dict(lq=63), dict(hq=63), dict(lo=63), dict(ho=63),
               dict(batch=-1), dict(m=0), dict(heads=0), dict(heads=3), dict(table=None), dict(lt=7), dict(width=-1),
               dict(lens=None), dict(lens=P + 2), dict(table=P + 2), dict(mask=P + 4), dict(lse=P + 2),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(q=P + 1), dict(to=1, out=P + 2)):
        assert call(**kw) == INV, kw
    assert call(width=(1 << 26) + 1, lt=(1 << 26) + 1) == UNS       # pages of 16: one more than 2^30 positions
    assert call(m=65) == UNS and call(width=1 << 27, lt=1 << 27) == UNS and call(lq=1 << 31) == UNS
    assert call(ho=1 << 31) == UNS and call(batch=1 << 30) == UNS
    assert call(batch=0, q=None, out=None, lens=None, table=None) == U.UFP4_OK


def test_workspace_bytes(U):
    f = U.lib().ufp4_cache_attn_workspace_bytes
    assert f(1, 1, 4, 1, _cache(U)) == 0                              # one CTA a head takes a page
    for bad in ((0, 1, 4, 8, _cache(U)), (1, 0, 4, 8, _cache(U)), (1, 65, 4, 8, _cache(U)), (1, 1, 3, 8, _cache(U)),
                (1, 1, 4, -1, _cache(U)), (1, 1, 4, 1 << 27, _cache(U)), (1, 1, 4, 8, _cache(U, page=24)),
                (1 << 30, 1, 4, 8, _cache(U)), (1, 1, 4, 8, None)):
        assert f(*bad) == 0


def test_cache_dim(U):
    for dim, want in ((-16, 0), (0, 0), (16, 64), (64, 64), (80, 128), (128, 128), (144, 256), (256, 256), (272, 0)):
        assert U.lib().ufp4_cache_dim(dim) == want


# ------------------------------------------------------------ the plain forms
@pytest.mark.parametrize("grid", [0, 1, 2])
def test_plain_row_is_the_oracles(oracle, grid):
    """quantize_row is the oracle's quantization of a one-row tensor."""
    g = np.random.default_rng(grid)
    for n in (16, 64, 208):
        x = (g.standard_normal(n) * 2.0 ** g.integers(-8, 9, size=n)).astype(np.float32)
        want = oracle.quantize(x[None], grid)
        codes, scales, dec = R.quantize_row(x, grid)
        assert np.array_equal(codes, want["codes"][0]) and np.array_equal(scales, want["scales"][0])
        assert dec == np.float32(want["tensor_scale"])


def test_plain_rotation_keeps_products():
    g = np.random.default_rng(1)
    a, b = g.standard_normal((2, 3, 64))
    assert np.allclose(R.rotate(a, 5) @ R.rotate(b, 5).T, a @ b.T)
    assert np.allclose(R.rotate(R.rotate(a, 5), 5, back=True), a)


def test_plain_attention_of_one_key_is_its_value():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((3, 4, 16))
    sees = np.eye(4, dtype=bool)
    out, lse, tol, ltol = R.attn(q, k, v, None, sees, 0.25, True, False, 1.0, 16)
    assert np.allclose(out, v) and np.allclose(lse, 0.25 * (q * k).sum(-1)) and (tol > 0).all() and (ltol > 0).all()
    sees[2] = False
    out, lse, _, _ = R.attn(q, k, v, None, sees, 0.25, True, False, 1.0, 16)
    assert (out[2] == 0).all() and lse[2] == -np.inf
