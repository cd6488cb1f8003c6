"""examples/moe_step.py where no token reaches an expert: all of them padding,
and no tokens at all.  The layer's output and every gradient are zeros."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [40, 0])
def test_step_without_routed_tokens(tokens):
    from fp4_quantized_numerics_gb300 import build, ufp4
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location("moe_step", os.path.join(ROOT, "examples", "moe_step.py"))
    step = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(step)
    experts, hidden, ffn = 4, 128, 64
    d = step.make(tokens, 2, experts, hidden, ffn)
    d["ids"][:] = -1
    w13, w2 = step.quantize_weights(d["w13"], experts), step.quantize_weights(d["w2"], experts)
    out, kept = step.forward(d["x"], d["ids"], d["weights"], w13, w2, experts, ffn)
    assert kept.counts == [0] * experts
    grads = step.backward(d["dout"], kept, w13, w2)
    for got, like in zip((out, *grads), (d["x"], d["x"], d["weights"], d["w13"], d["w2"])):
        assert got.shape == like.shape and not got.any()
    assert ufp4.ufp4_check() == ufp4.UFP4_OK
