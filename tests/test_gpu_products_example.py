"""The example of experts in three precisions: its parts agree with fp32 and its
tuning steps lower the loss.

Bound of the FP8 parts: every operand rounds to E4M3 with a relative error of at
most 2^-4, about 2^-4 / sqrt(3) = 0.036 rms over a code's interval and 0.026 over
all values of a binade; the two products round three operands (tokens, activation,
and the weights of each product: four roundings that add in quadrature), so the
output's relative error is about 2 * 0.026 = 0.05; twice that is the bound."""
import importlib.util
import os

import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    need_gpu()
    spec = importlib.util.spec_from_file_location("mixed_precision_experts",
                                                  os.path.join(ROOT, "examples", "mixed_precision_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens", [1, 5, 64, 300])
def test_shared_expert(example, tokens):
    out, mlp, want = example.serve(tokens=tokens)
    assert out.shape == want.shape
    assert example.relative(mlp, want) < 0.1


@pytest.mark.parametrize("tokens", [1, 96, 700])
def test_routed_fp8_experts(example, tokens):
    out, want = example.experts_fp8(tokens=tokens)
    assert example.relative(out, want) < 0.1


def test_tuning_lowers_the_loss(example):
    losses = example.tune()
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert losses[-1] < 0.8 * losses[0], losses
