"""CPU-only checks of the Python binding of the calls that answer with a
quantized model: operands and streams of another device are refused, and
results belong to the stream of the call."""
import pytest
import torch

from fp4_quantized_numerics_gb300 import ufp4 as U
from tests.test_binding import FP, Machine, On0, On1, Stream, _plan, _rows, _t

HEADS, DIM = 2, 64


@pytest.fixture
def machine(monkeypatch):
    return Machine(monkeypatch)


def _weights(rows):
    def make(kind):
        return U.QTensor(_t(kind, rows * 32, dtype=torch.uint8), _t(kind, rows * 4, dtype=torch.uint8), _t(kind, 3), rows,
                         64, U.UFP4_E1M2)
    return make


def _cache(kind):
    new = lambda *tail, dtype=torch.uint8: _t(kind, 4, HEADS, 16, *tail, dtype=dtype)  # noqa: E731
    return U.Cache(new(32), new(4), new(dtype=FP), new(32), new(4), new(dtype=FP), DIM, U.UFP4_E1M2)


def _heads(tokens, heads=HEADS):
    return lambda kind: _t(kind, tokens, heads, DIM)


def _ints(*shape, dtype=torch.int32):
    return lambda kind: _t(kind, *shape, dtype=dtype)


# tensors on a device; results among them, which a call also makes by itself
CALLS = {
    "ufp4_gemv": dict(x=_rows(4, 64), w=_weights(128), out=_rows(4, 128)),
    "ufp4_gemv_grouped": dict(x=_rows(8, 64), w=_weights(384), plan=_plan, out=_rows(8, 100)),
    "ufp4_cache_append": dict(k=_heads(3), v=_heads(3), slots=_ints(3, dtype=torch.int64), cache=_cache),
    "ufp4_cache_load": dict(cache=_cache, slots=_ints(3, dtype=torch.int64), k=_heads(3), v=_heads(3)),
    "ufp4_cache_attn": dict(q=_heads(4, 4), cache=_cache, table=_ints(2, 3), lens=_ints(2),
                            mask=_ints(2, 2, dtype=torch.int64), out=_heads(4, 4), lse=lambda kind: _t(kind, 4, 4),
                            ws=_ints(64, dtype=torch.uint8)),
}
PLAIN = {"ufp4_gemv_grouped": dict(rows=100)}
MADE = {"ufp4_gemv": ("out",), "ufp4_gemv_grouped": ("out",), "ufp4_cache_append": (), "ufp4_cache_load": ("k", "v"),
        "ufp4_cache_attn": ("out", "lse", "ws")}


@pytest.fixture(autouse=True)
def sizes(monkeypatch):
    monkeypatch.setattr(U, "_attn_needs", {(0, 2, 2, 4, 3, HEADS, 16, DIM): 512})


def _call(name, made, **kw):
    make = CALLS[name]
    given = {k: (kw[k] if k in kw else m(On0)) for k, m in make.items()
             if made or k in kw or k not in MADE[name]}
    return getattr(U, name)(**given, **PLAIN.get(name, {}), **{k: v for k, v in kw.items() if k not in make})


@pytest.mark.parametrize("name", CALLS)
def test_operands_of_one_device_reach_the_library(machine, name):
    _call(name, True)
    assert machine.calls == [(name, 100)] and not machine.made


@pytest.mark.parametrize("name,which", [(n, k) for n, make in CALLS.items() for k in make])
def test_operands_of_another_device_are_refused(machine, name, which):
    with pytest.raises(ValueError):
        _call(name, True, **{which: CALLS[name][which](On1)})
    assert not machine.calls


@pytest.mark.parametrize("name", CALLS)
def test_everything_on_another_device_than_the_current_one_is_refused(machine, name):
    with pytest.raises(ValueError):
        _call(name, False, **{k: m(On1) for k, m in CALLS[name].items() if k not in MADE[name]})
    assert not machine.calls and not machine.made


@pytest.mark.parametrize("name", CALLS)
def test_streams_of_another_device_are_refused(machine, name):
    with pytest.raises(ValueError):
        _call(name, True, stream=Stream(1, 300))
    assert not machine.calls


@pytest.mark.parametrize("name", CALLS)
def test_results_belong_to_the_calls_stream(machine, name):
    more = dict(lse=True) if name == "ufp4_cache_attn" else {}
    _call(name, False, stream=Stream(0, 300), **more)
    assert machine.calls == [(name, 300)] and {s for _, s in machine.made} <= {300}
    assert len(machine.made) == len(MADE[name])


@pytest.mark.parametrize("name,which", [(n, k) for n, make in CALLS.items() for k in make
                                        if k not in ("w", "plan", "cache")])
def test_cpu_tensors_are_refused(machine, name, which):
    with pytest.raises(TypeError):
        _call(name, True, **{which: CALLS[name][which](torch.Tensor)})
    assert not machine.calls


def test_caches_of_mixed_parts_are_refused(machine):
    new = lambda *tail, dtype=torch.uint8, kind=On0: _t(kind, 4, HEADS, 16, *tail, dtype=dtype)  # noqa: E731
    good = [new(32), new(4), new(dtype=FP), new(32), new(4), new(dtype=FP)]
    U.Cache(*good, DIM, U.UFP4_E1M2)
    for i, bad in ((1, new(8)), (2, new(dtype=torch.float64)), (3, new(64)), (4, new(4, kind=On1)), (0, new(32)[0]),
                   (5, new(dtype=FP).transpose(0, 1))):
        with pytest.raises(ValueError):
            U.Cache(*(good[:i] + [bad] + good[i + 1:]), DIM, U.UFP4_E1M2)
    with pytest.raises(ValueError):
        U.Cache(*good, 2 * DIM, U.UFP4_E1M2)
