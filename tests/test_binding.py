"""CPU-only checks of the Python binding: what it refuses before a call
reaches the library, and where its results come from.

No GPU is needed: tensors are CPU tensors that report a CUDA device, the
current device and streams are stand-ins, and the library's entry points are
replaced by ones that record the call."""
import contextlib

import pytest
import torch

from fp4_quantized_numerics_gb300 import ufp4 as U

BF, FP = torch.bfloat16, torch.float32


class On0(torch.Tensor):
    """A tensor that reports to be on a CUDA device."""
    is_cuda, index = True, 0

    def get_device(self):
        return self.index

    @property
    def device(self):
        return torch.device("cuda", self.index)


class On1(On0):
    index = 1


class Stream:
    def __init__(self, index, handle):
        self.device_index, self.cuda_stream = index, handle


class Machine:
    """Two devices, 0 current; `calls`: (entry point, stream handle) of each
    call; `made`: (shape, stream handle) of each allocation."""

    def __init__(self, patch):
        self.calls, self.made, self.stream, self.current = [], [], 100, 0
        plain = torch.empty

        def empty(*shape, dtype=None, device=None):
            t = plain(*shape, dtype=dtype).as_subclass(On0)
            self.made.append((tuple(t.shape), self.stream))
            return t

        @contextlib.contextmanager
        def on(stream):
            before, self.stream = self.stream, self.stream if stream is None else stream.cuda_stream
            yield
            self.stream = before

        patch.setattr(U, "_empty_strided_cuda", lambda shape, strides, dtype: empty(shape, dtype=dtype))
        patch.setattr(U, "_current_device", lambda: self.current)
        patch.setattr(U, "_current_raw_stream", lambda dev: 100)
        patch.setattr(U, "lib", lambda: self)
        patch.setattr(torch, "empty", empty)
        patch.setattr(torch.cuda, "stream", on)
        patch.setattr(torch.cuda, "current_stream", lambda *a: Stream(self.current, 100))

    def __getattr__(self, name):
        if name in ("ufp4_codes_bytes", "ufp4_scales_bytes", "ufp4_grouped_rows", "ufp4_grouped_kpad",
                    "ufp4_workspace_bytes"):
            return lambda *args: 64
        if not name.startswith("ufp4_"):
            raise AttributeError(name)

        def call(*args):
            last = args[-1]
            self.calls.append((name, getattr(last, "value", last)))
            return U.UFP4_OK
        return call


@pytest.fixture
def machine(monkeypatch):
    return Machine(monkeypatch)


def _t(kind, *shape, dtype=FP):
    return torch.zeros(shape, dtype=dtype).as_subclass(kind)


def _plan(kind):
    return U.MoePlan(_t(kind, 4, 2, dtype=torch.int32), _t(kind, 8, dtype=torch.int32),
                     _t(kind, 3, dtype=torch.int64), _t(kind, 4, dtype=torch.int64))


def _ckpt(kind, fmt=0):
    return U.Ckpt(_t(kind, 4, 32, dtype=torch.uint8), _t(kind, 4, 1, dtype=torch.uint8), 4, 32, fmt)


# every call of 4 tokens x 2 choices, 32 wide: its operands by name, a maker of each
def _rows(n, width=32, dtype=FP):
    return lambda kind: _t(kind, n, width, dtype=dtype)


CALLS = {
    "ufp4_moe_sort": dict(ids=_rows(4, 2, torch.int64), n_experts=lambda kind: 3, out=_plan),
    "ufp4_moe_dispatch": dict(x=_rows(4), plan=_plan, out=_rows(8)),
    "ufp4_moe_combine": dict(y=_rows(8), plan=_plan, weights=_rows(4, 2), out=_rows(4)),
    "ufp4_moe_combine_bwd": dict(dout=_rows(4), y=_rows(8), plan=_plan, weights=_rows(4, 2), dy=_rows(8),
                                 dw=_rows(4, 2)),
    "ufp4_ckpt_save": dict(x=_rows(4), out=_ckpt),
    "ufp4_ckpt_load": dict(c=_ckpt, out=_rows(4)),
    "ufp4_swiglu": dict(gate=_rows(4), up=_rows(4), out=_rows(4), keep=lambda kind: (_ckpt(On0), _ckpt(kind))),
    "ufp4_swiglu_bwd": dict(dh=_rows(4), keep_gate=_ckpt, keep_up=_ckpt, dgate=_rows(4), dup=_rows(4)),
}
OUTPUTS = ("out", "dy", "dw", "dgate", "dup", "keep")


@pytest.mark.parametrize("name", CALLS)
def test_operands_of_one_device_reach_the_library(machine, name):
    f, make = getattr(U, name), CALLS[name]
    f(**{k: m(On0) for k, m in make.items()})
    assert machine.calls == [(name, 100)] and not machine.made


@pytest.mark.parametrize("name,elsewhere", [(n, k) for n, make in CALLS.items() for k in make if k != "n_experts"])
def test_operands_of_another_device_are_refused(machine, name, elsewhere):
    """One operand on device 1, the others and the current device 0; then all
    of them, with any result allocated by the call."""
    make = CALLS[name]
    with pytest.raises(ValueError):
        getattr(U, name)(**{k: m(On1 if k == elsewhere else On0) for k, m in make.items()})
    with pytest.raises(ValueError):
        getattr(U, name)(**{k: m(On1) for k, m in make.items() if k not in OUTPUTS})
    assert not machine.calls and not machine.made


@pytest.mark.parametrize("name", CALLS)
def test_streams_of_another_device_are_refused(machine, name):
    given = {k: m(On0) for k, m in CALLS[name].items()}
    with pytest.raises(ValueError):
        getattr(U, name)(**given, stream=Stream(1, 300))
    assert not machine.calls
    getattr(U, name)(**given, stream=Stream(0, 300))
    assert machine.calls == [(name, 300)]


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream,where", [(None, 100), (Stream(0, 100), 100), (Stream(0, 300), 300)])
def test_results_are_made_on_the_stream_of_the_call(machine, name, stream, where):
    given = {k: m(On0) for k, m in CALLS[name].items() if k not in OUTPUTS}
    if name == "ufp4_swiglu":
        given["ckpt"] = 0
    getattr(U, name)(**given, stream=stream)
    assert machine.calls == [(name, where)] and machine.made
    assert {s for _, s in machine.made} == {where}


def test_a_plan_or_checkpoint_is_on_one_device(machine):
    with pytest.raises(ValueError):
        U.MoePlan(_t(On0, 4, 2, dtype=torch.int32), _t(On0, 8, dtype=torch.int32), _t(On1, 3, dtype=torch.int64),
                  _t(On0, 4, dtype=torch.int64))
    with pytest.raises(ValueError):
        U.Ckpt(_t(On0, 4, 32, dtype=torch.uint8), _t(On1, 4, 1, dtype=torch.uint8), 4, 32, 0)


def _q(kind):
    return U.QTensor(_t(kind, 64, dtype=torch.uint8), _t(kind, 64, dtype=torch.uint8), _t(kind, 1), 4, 32,
                     U.UFP4_E2M1)


OLDER = {
    "ufp4_quantize": (lambda k, s: U.ufp4_quantize(_t(k, 4, 32), U.UFP4_E2M1, ws=_t(k, 8), stream=s)),
    "ufp4_quantize_dual": (lambda k, s: U.ufp4_quantize_dual(_t(k, 4, 32), U.UFP4_E2M1, ws=_t(k, 8), stream=s)),
    "ufp4_dequantize": (lambda k, s: U.ufp4_dequantize(_q(k), stream=s)),
    "ufp4_gemm": (lambda k, s: U.ufp4_gemm(_q(k), _q(k), stream=s)),
    "ufp4_gemm_amax": (lambda k, s: U.ufp4_gemm_amax(_q(k), _q(k), stream=s)),
    "ufp4_quantize_stats": (lambda k, s: U.ufp4_quantize_stats(_t(k, 4, 32), U.UFP4_E2M1, ws=_t(k, 8), stream=s)),
    "ufp4_stats": (lambda k, s: U.ufp4_stats(_t(k, 4, 32), _q(k), ws=_t(k, 8), stream=s)),
    "ufp4_gemm_grouped": (lambda k, s: U.ufp4_gemm_grouped(_q(k), _q(k), [], stream=s)),
    "ufp4_quantize_grouped": (lambda k, s: U.ufp4_quantize_grouped(_t(k, 4, 32), U.UFP4_E1M2, [4], ws=_t(k, 8),
                                                                   stream=s)),
    "ufp4_quantize_grouped_dual": (lambda k, s: U.ufp4_quantize_grouped_dual(_t(k, 4, 32), U.UFP4_E1M2, [4],
                                                                             ws=_t(k, 8), stream=s)),
}


@pytest.mark.parametrize("name", OLDER)
def test_quantizer_and_gemm_calls_of_another_device_are_refused(machine, name):
    with pytest.raises(ValueError):
        OLDER[name](On1, None)
    with pytest.raises(ValueError):
        OLDER[name](On0, Stream(1, 300))
    assert not machine.calls
    OLDER[name](On0, Stream(0, 300))
    assert machine.calls == [(name, 300)]


@pytest.mark.parametrize("name", OLDER)
@pytest.mark.parametrize("stream,where", [(None, 100), (Stream(0, 300), 300)])
def test_quantizer_and_gemm_results_are_made_on_the_stream_of_the_call(machine, name, stream, where):
    OLDER[name](On0, stream)
    assert machine.calls[-1] == (name, where)
    assert machine.made or name in ("ufp4_stats", "ufp4_gemm_grouped")
    assert {s for _, s in machine.made} <= {where}


def test_the_workspace_is_made_on_the_stream_of_the_first_call(machine, monkeypatch):
    monkeypatch.setattr(U, "_workspaces", {})
    U.ufp4_quantize(_t(On0, 4, 32), U.UFP4_E2M1, stream=Stream(0, 300))
    assert ((64,), 300) in machine.made and {s for _, s in machine.made} == {300}


# ----------------------------------------------------- arguments that disagree
DTYPED = {"ufp4_moe_combine": ["out"], "ufp4_moe_combine_bwd": ["dy"], "ufp4_ckpt_load": ["out"],
          "ufp4_swiglu": ["out"], "ufp4_swiglu_bwd": ["dgate", "dup"]}


@pytest.mark.parametrize("name,result", [(n, r) for n, results in DTYPED.items() for r in results])
def test_a_dtype_that_a_given_result_does_not_have_is_refused(machine, name, result):
    given = {k: m(On0) for k, m in CALLS[name].items() if k not in OUTPUTS or k == result}
    with pytest.raises(TypeError):
        getattr(U, name)(**given, dtype=BF)
    assert not machine.calls
    getattr(U, name)(**given, dtype=FP)
    getattr(U, name)(**given)
    assert len(machine.calls) == 2


def test_results_of_another_dtype_than_each_other_are_refused(machine):
    with pytest.raises(TypeError):
        U.ufp4_moe_dispatch(_t(On0, 4, 32), _plan(On0), out=_t(On0, 8, 32, dtype=BF))
    with pytest.raises(TypeError):
        U.ufp4_swiglu_bwd(_t(On0, 4, 32), _ckpt(On0), _ckpt(On0), dgate=_t(On0, 4, 32),
                          dup=_t(On0, 4, 32, dtype=BF))
    assert not machine.calls


def test_a_format_that_the_kept_checkpoints_do_not_have_is_refused(machine):
    x = _t(On0, 4, 32)
    for keep in ((_ckpt(On0, 0), _ckpt(On0, 0)), (_ckpt(On0, 1), _ckpt(On0, 0)), (None, None)):
        with pytest.raises(ValueError):
            U.ufp4_swiglu(x, x, ckpt=U.UFP4_CKPT_E4M3, keep=keep)
    assert not machine.calls and not machine.made
    pair = _ckpt(On0, 1), _ckpt(On0, 1)
    assert U.ufp4_swiglu(x, x, ckpt=U.UFP4_CKPT_E4M3, keep=pair)[1] is pair[0]
    assert U.ufp4_swiglu(x, x, keep=pair)[2] is pair[1]
    assert U.ufp4_ckpt_load(pair[0]).dtype is BF


def test_results_are_made_by_the_public_call_where_the_short_one_is_another(machine, monkeypatch):
    def takes_other_arguments(*args):
        raise TypeError("3 arguments given")
    monkeypatch.setattr(U, "_empty_strided_cuda", takes_other_arguments)
    for _ in range(2):
        assert U.ufp4_moe_dispatch(_t(On0, 4, 32), _plan(On0)).shape == (8, 32)
    assert U._empty_strided_cuda is None and len(machine.made) == 2


def test_a_wrong_size_leaves_the_short_call_in_use(machine):
    with pytest.raises(TypeError):
        U.ufp4_moe_sort(_t(On0, 4, 2, dtype=torch.int64), "three")
    assert U._empty_strided_cuda is not None
