"""Calls that answer with a quantized model, on tensors that held something else before."""
import pytest
import torch

from tests.test_gemv_gpu import U  # noqa: F401

pytestmark = pytest.mark.gpu


def test_dense_and_grouped_weights_in_one_tensor(U):  # noqa: F811
    """A dense product refuses grouped weights, and takes them again when the
    tensor has been quantized as a whole since."""
    w, x = torch.randn(256, 64, device="cuda"), torch.randn(3, 64, device="cuda")
    q = U.ufp4_quantize_grouped(w, U.UFP4_E1M2, [128, 128])
    with pytest.raises(ValueError):
        U.ufp4_gemv(x, q)
    want = U.ufp4_gemv(x, U.ufp4_quantize(w, U.UFP4_E1M2))
    assert torch.equal(U.ufp4_gemv(x, U.ufp4_quantize(w, U.UFP4_E1M2, out=q)), want)
    U.ufp4_quantize_grouped(w, U.UFP4_E1M2, [128, 128], out=q)
    with pytest.raises(ValueError):
        U.ufp4_gemv(x, q)
    other = U.QTensor.empty(64, 256, U.UFP4_E1M2)
    U.ufp4_quantize_dual(w, U.UFP4_E1M2, out_row=q, out_col=other)
    assert torch.equal(U.ufp4_gemv(x, q), want)
    U.ufp4_quantize_grouped(w, U.UFP4_E1M2, [128, 128], out=q)
    q, _ = U.ufp4_quantize_stats(w, U.UFP4_E1M2, out=q)
    assert torch.equal(U.ufp4_gemv(x, q), want)
