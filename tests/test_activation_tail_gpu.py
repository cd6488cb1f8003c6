"""The gated activation and its gradients far on the negative side, where
exp(-g) nears the end of fp32's range while the results, times a large factor,
are ordinary numbers.

The bounds, relative to each result.  expf is within 2 ulp (4 * 2^-24), __expf
within 2 + 1.173 |x| ulp, __fdividef within 2; 2^x and the reciprocal as the
hardware gives them, with x rounded before, are within the same.  A result
takes at most two exponentials of g / 2 (or one of g) and five more roundings
of 2^-24: fp32 13 * 2^-24, bf16 2 * (8 + 1.173 |g|) * 2^-24 and its own 2^-8.
Nothing else is allowed but half a step of the type's subnormal numbers."""
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


def _cuda(v):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).cuda()


def _close(got, want, g, dtype):
    rel = 13 * R.U32 if dtype is FP else 2 * (8 + 1.173 * np.abs(g)) * R.U32 + 1.001 * R.UBF
    bad = ~(np.abs(_f64(got) - want) <= rel * np.abs(want) + 1.001 * R.half_step(dtype))
    assert not bad.any(), (np.argwhere(bad)[:3], _f64(got)[bad][:3], want[bad][:3])


@pytest.mark.parametrize("cols", [64, 62, 61])      # the three layouts
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("up", [1.0, -2.0 ** 40, 2.0 ** 100, 3e38])
def test_activation_far_below_zero(U, cols, dtype, up):
    """Gates from -60 to -170 around every step of the exponentials' range."""
    gate = _cuda(-np.linspace(60, 170, 40 * cols).reshape(40, cols))
    h = U.ufp4_swiglu(gate, _cuda(np.full((40, cols), up)), dtype=dtype)[0]
    g, u = _f64(gate), float(np.float32(up))
    _close(h, R.swiglu(g, u), g, dtype)


def test_activation_near_the_end_of_exp(U):
    """silu(-88.73) is a normal fp32 number, and exp(88.73) is not."""
    gate = torch.tensor([[-88.73, -100.0]], device="cuda")
    h = _f64(U.ufp4_swiglu(gate, torch.ones_like(gate))[0])
    assert abs(h[0, 0]) > 2.0 ** -126 and h[0, 1] < 0
    far = torch.tensor([[-1e4, -1e30, -3e38]], device="cuda")
    for dtype in (BF, FP):
        assert not U.ufp4_swiglu(far, torch.full_like(far, 3e38), dtype=dtype)[0].any()


@pytest.mark.parametrize("cols", [64, 62, 61])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("size", [1e-3, 1e15, 1e30])
def test_gradients_far_below_zero(U, cols, dtype, size):
    """Gates -64 .. -127, which INT8's step of 1 keeps as they are, and up a
    power of two."""
    gate = np.repeat(-np.arange(64.0, 128.0), cols).reshape(64, cols)
    up = np.full((64, cols), 2.0 ** 10)
    _, kg, ku = U.ufp4_swiglu(_cuda(gate), _cuda(up), ckpt=U.UFP4_CKPT_INT8, dtype=FP)
    np.testing.assert_array_equal(_f64(U.ufp4_ckpt_load(kg, dtype=FP)), gate)
    np.testing.assert_array_equal(_f64(U.ufp4_ckpt_load(ku, dtype=FP)), up)
    dh = _cuda(np.random.default_rng(cols).standard_normal((64, cols)) * size)
    dgate, dup = U.ufp4_swiglu_bwd(dh, kg, ku, dtype=dtype)
    wg, wu = R.swiglu_bwd(_f64(dh), gate, up)
    _close(dgate, wg, gate, dtype)
    _close(dup, wu, gate, dtype)
