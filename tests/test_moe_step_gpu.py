"""examples/moe_step.py: the operators around the grouped GEMMs together with
them, as one training step of a mixture-of-experts layer, against the same
layer in fp32.

The bounds: with the transform, E1M2 with 16-element scales keeps Gaussian
operands at about 22 dB, 8 % of their norm, and stochastic rounding of the
gradients costs about 3 dB more (11 %).  A product of two such operands is off
by sqrt(2) of that; errors of independent steps add in squares.  forward: two
operands, the activation (which about doubles a relative error of its inputs
in the worst case), two operands: 0.08 sqrt(2) = 0.11, 0.23, with two more
0.25.  Gradients: dw2 0.23 and 0.11 together 0.26; dx and dw13 pass the second
product, the activation's derivative at inputs that are off by 0.11, and the
first product: sqrt(0.14^2 + 0.25^2 + 0.14^2) = 0.32.  0.35 and 0.45 leave
room for the spread of small tensors; a wrong row, expert or weight gives 1 or
more."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def step():
    from fp4_quantized_numerics_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location("moe_step", os.path.join(ROOT, "examples", "moe_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,topk,experts,hidden,ffn,dropped", [
    (300, 2, 8, 256, 192, 0.0),
    (129, 4, 6, 128, 320, 0.3),      # padding tokens
    (7, 1, 16, 128, 64, 0.0),        # most experts without a token
])
def test_step_against_fp32(step, tokens, topk, experts, hidden, ffn, dropped):
    d = step.make(tokens, topk, experts, hidden, ffn, seed=tokens)
    if dropped:
        d["ids"][: int(tokens * dropped)] = -1
    w13, w2 = step.quantize_weights(d["w13"], experts), step.quantize_weights(d["w2"], experts)
    out, kept = step.forward(d["x"], d["ids"], d["weights"], w13, w2, experts, ffn)
    got = (out, *step.backward(d["dout"], kept, w13, w2))
    want = step.plain(**d, experts=experts, ffn=ffn)
    for name, u, v, bound in zip(("out", "dx", "dweights", "dw13", "dw2"), got, want, (0.35, 0.45, 0.35, 0.45, 0.35)):
        assert u.shape == v.shape, name
        assert torch.isfinite(u.float()).all(), name
        off = ((u.float() - v).norm() / v.norm()).item()
        assert off <= bound, (name, off)
    if dropped:
        n = int(tokens * dropped)
        assert not out[:n].any() and not got[1][:n].any() and not got[2][:n].any()
    from fp4_quantized_numerics_gb300 import ufp4
    assert ufp4.ufp4_check() == ufp4.UFP4_OK
