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


def test_attention_after_a_refused_cache_of_the_same_sizes(U):  # noqa: F811
    """A table that needs scratch, with a cache that is refused first."""
    good = U.Cache.empty(256, 1, 16, 64, U.UFP4_E1M2)
    bad = U.Cache(good.k_codes, good.k_scales, good.k_row_scale, good.v_codes, good.v_scales, good.v_row_scale, 64,
                  U.UFP4_MXFP4)
    kv = torch.randn(256 * 16, 1, 64, device="cuda")
    U.ufp4_cache_append(kv, kv, torch.arange(256 * 16, device="cuda"), good)
    q = torch.randn(1, 2, 64, device="cuda")
    table = torch.arange(4000, dtype=torch.int32, device="cuda").remainder(256)[None]
    lens = torch.tensor([50000], dtype=torch.int32, device="cuda")
    assert U.lib().ufp4_cache_attn_workspace_bytes(1, 1, 2, 4000, good.c()) > 0
    U._attn_needs.clear()
    with pytest.raises(U.UFP4Error):
        U.ufp4_cache_attn(q, bad, table, lens)
    out = U.ufp4_cache_attn(q, good, table, lens)
    U._attn_needs.clear()
    assert torch.equal(U.ufp4_cache_attn(q, good, table, lens), out)
