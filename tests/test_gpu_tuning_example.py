"""The example's adapters and router (examples/mixed_precision_experts.py): they run, and
their gradients are those of the same step in fp32."""
import os
import sys

import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    need_gpu()
    import mixed_precision_experts
    return mixed_precision_experts


def test_gradients_of_a_step(example):
    leaves, grads, want = example.tune_adapters()
    for leaf, got, ref in zip(leaves, grads, want):
        assert got.shape == leaf.shape and got.dtype is leaf.dtype
        # rows, their products and gradients are rounded to bf16 (2^-8) on the way: some roundings' worth of the norm
        assert example.relative(got, ref) < 4 * 2.0 ** -8


def test_adapters_of_many_requests(example):
    # the projection in FP8: two operands, each off by about 0.026 of its size (rms over E4M3's intervals), in quadrature
    # 0.037; the adapters' part, which is not rounded so, only lowers that
    assert example.relative(*example.serve_adapters()) < 2.0 ** -4
