"""Results that a call makes on another stream than the current one: never in
memory that work queued on the current stream still uses, and never given to
the current stream while the call's own work may write it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ROWS, COLS = 1000, 1000            # a million elements: results of a few MB, no other test's sizes


@pytest.fixture(scope="module")
def U():
    from fp4_quantized_numerics_gb300 import build, ufp4
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return ufp4


def _calls(U):
    """name -> call(stream), the tensors it makes first."""
    x = torch.randn(ROWS, COLS, device="cuda")
    ids = torch.randint(0, 8, (ROWS, 1), device="cuda")
    plan, w = U.ufp4_moe_sort(ids, 8), torch.ones(ROWS, 1, device="cuda")
    h, kg, ku = U.ufp4_swiglu(x, x, ckpt=U.UFP4_CKPT_INT8)
    a = torch.randn(1024, 1024, device="cuda", dtype=torch.bfloat16)
    q = U.ufp4_quantize(a, U.UFP4_E1M2)
    many = torch.randint(0, 8, (ROWS * COLS, 1), device="cuda")
    return {
        "moe_sort": lambda s: U.ufp4_moe_sort(many, 8, stream=s).pos,
        "moe_dispatch": lambda s: U.ufp4_moe_dispatch(x, plan, stream=s),
        "moe_combine": lambda s: U.ufp4_moe_combine(x, plan, w, stream=s),
        "moe_combine_bwd": lambda s: U.ufp4_moe_combine_bwd(x, x, plan, w, stream=s)[0],
        "ckpt_save": lambda s: U.ufp4_ckpt_save(x, stream=s).codes[:, :COLS],   # (rows' padding is not written)
        "ckpt_load": lambda s: U.ufp4_ckpt_load(kg, stream=s),
        "swiglu": lambda s: U.ufp4_swiglu(x, x, stream=s)[0],
        "quantize": lambda s: U.ufp4_quantize(a, U.UFP4_E1M2, stream=s).codes,
        "quantize_dual": lambda s: U.ufp4_quantize_dual(a, U.UFP4_E1M2, stream=s)[1].codes,
        "quantize_grouped": lambda s: U.ufp4_quantize_grouped(a, U.UFP4_E1M2, [512, 512], stream=s).codes,
        "dequantize": lambda s: U.ufp4_dequantize(q, stream=s),
        "gemm": lambda s: U.ufp4_gemm(q, q, stream=s),
        "swiglu_bwd": lambda s: U.ufp4_swiglu_bwd(x, kg, ku, stream=s)[0],
    }


NAMES = ["moe_sort", "moe_dispatch", "moe_combine", "moe_combine_bwd", "ckpt_save", "ckpt_load", "swiglu",
         "swiglu_bwd", "quantize", "quantize_dual", "quantize_grouped", "dequantize", "gemm"]


@pytest.mark.parametrize("name", NAMES)
def test_results_on_a_side_stream(U, name):
    call = _calls(U)[name]
    want = call(None)
    size, want = want.untyped_storage().nbytes(), want.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    # a block of the result's size, dropped while queued work still reads it
    held, seen = torch.full((size,), 7, dtype=torch.uint8, device="cuda"), torch.zeros(size, dtype=torch.uint8,
                                                                                      device="cuda")
    at = held.data_ptr()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    seen.copy_(held)
    del held
    got = call(side)
    assert not at <= got.data_ptr() < at + size
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool((seen == 7).all())

    # a result dropped while its call is still queued: its memory stays the side stream's
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = call(side)
    at = got.data_ptr()
    del got
    other = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
    assert not other.data_ptr() <= at < other.data_ptr() + size
    side.synchronize()
    assert bool((other == 7).all())
