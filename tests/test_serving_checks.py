"""CPU-only checks of what the binding of the calls that answer with a
quantized model refuses, and what it remembers between calls."""
import pytest
import torch

from fp4_quantized_numerics_gb300 import ufp4 as U
from tests.test_binding import On0, _rows, _t
from tests.test_serving_binding import machine  # noqa: F401


def _weights(segments):
    w = U.QTensor(_t(On0, 256 * 32, dtype=torch.uint8), _t(On0, 256 * 4, dtype=torch.uint8), _t(On0, len(segments)), 256,
                  64, U.UFP4_E1M2)
    w.seg_rows = segments
    return w


@pytest.mark.parametrize("segments", [[128, 128], [256, 0], [100, 0, 7]])
def test_a_dense_product_refuses_grouped_weights(machine, segments):  # noqa: F811
    """Every segment has a tensor scale of its own; a dense product knows one."""
    with pytest.raises(ValueError):
        U.ufp4_gemv(_rows(4, 64)(On0), _weights(segments))
    assert not machine.calls
    U.ufp4_gemv(_rows(4, 64)(On0), _weights([256]))       # (one segment is a matrix)
    assert [n for n, _ in machine.calls] == ["ufp4_gemv"]


def test_a_tensor_that_was_grouped_before(machine):  # noqa: F811
    w = _weights([128, 128])
    w.ungrouped()
    U.ufp4_gemv(_rows(4, 64)(On0), w)
    assert [n for n, _ in machine.calls] == ["ufp4_gemv"]
