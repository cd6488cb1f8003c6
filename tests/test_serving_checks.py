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


class _Attention:
    """The library's attention with `need` bytes of scratch, which answers the
    size of a refused cache with 0; `given`: scratch of each call that ran."""

    def __init__(self, need):
        self.need, self.given, self.asked = need, [], 0

    def ufp4_cache_attn_workspace_bytes(self, batch, m, heads, width, cache):
        self.asked += 1
        return self.need if cache._obj.grid == U.UFP4_E1M2 else 0

    def ufp4_cache_attn(self, *args):
        if args[7]._obj.grid != U.UFP4_E1M2:
            return U.UFP4_ERR_UNSUPPORTED
        if args[-2] < self.need:
            return U.UFP4_ERR_INVALID
        self.given.append(args[-2])
        return U.UFP4_OK

    def ufp4_status_string(self, status):
        return b"refused"


def test_a_refused_cache_leaves_no_scratch_size_behind(machine, monkeypatch):  # noqa: F811
    """A call that was refused says nothing of the scratch that the next one of its sizes needs."""
    monkeypatch.setattr(U, "_attn_needs", {})
    fake = _Attention(512)
    monkeypatch.setattr(U, "lib", lambda: fake)
    new = lambda *tail, dtype=torch.uint8: _t(On0, 4, 2, 16, *tail, dtype=dtype)  # noqa: E731
    parts = [new(32), new(4), new(dtype=torch.float32), new(32), new(4), new(dtype=torch.float32)]
    call = lambda grid: U.ufp4_cache_attn(_t(On0, 4, 4, 64), U.Cache(*parts, 64, grid),  # noqa: E731
                                          _t(On0, 2, 3, dtype=torch.int32), _t(On0, 2, dtype=torch.int32))
    with pytest.raises(U.UFP4Error):
        call(U.UFP4_MXFP4)
    call(U.UFP4_E1M2)
    call(U.UFP4_E1M2)
    assert fake.given == [512, 512] and fake.asked == 2
    with pytest.raises(U.UFP4Error):
        call(U.UFP4_MXFP4)


def test_scratch_with_gaps_is_refused(machine):  # noqa: F811
    """What lies between the elements of a strided view is not scratch."""
    new = lambda *tail, dtype=torch.uint8: _t(On0, 4, 2, 16, *tail, dtype=dtype)  # noqa: E731
    cache = U.Cache(new(32), new(4), new(dtype=torch.float32), new(32), new(4), new(dtype=torch.float32), 64, U.UFP4_E1M2)
    call = lambda ws: U.ufp4_cache_attn(_t(On0, 4, 4, 64), cache, _t(On0, 2, 3, dtype=torch.int32),  # noqa: E731
                                        _t(On0, 2, dtype=torch.int32), ws=ws)
    room = _t(On0, 1024, dtype=torch.uint8)
    with pytest.raises(ValueError):
        call(room[::2])
    with pytest.raises(ValueError):
        call(room.view(32, 32)[:, :16])
    assert not machine.calls
    call(room[:512])
    assert [n for n, _ in machine.calls] == ["ufp4_cache_attn"]
