"""Fp8Mlp in the orders and shapes that a program uses it in: serving between a
forward and its backward, tensors changed under a pending backward, any token
count, weights frozen again under a captured decode, first steps of a fresh
block.

Bounds as in test_mlp_gpu.py: 0.08 of a value's 2-norm for outputs, 0.16 for
gradients; equal call sequences have to give equal bits."""
import pytest
import torch

from tests import block_ref as R
from tests.gpu_util import DEV
from tests.test_mlp_gpu import BF, G_BOUND, Y_BOUND, make, off, reference

pytestmark = pytest.mark.gpu
fp8mi = pytest.importorskip("fp8_tensor_scaled_quantize_amd")
from fp8_tensor_scaled_quantize_amd.mlp import Fp8Mlp  # noqa: E402


def batch(rows, d, seed, sigma=1.0):
    return R.rand((rows, d), sigma, BF, seed).to(DEV)


def same(got, want):
    torch.cuda.synchronize()
    for name, g in got.items():
        assert (g is None) == (want[name] is None), name
        assert g is None or torch.equal(g, want[name]), name


@pytest.mark.parametrize("act,gated", [("gelu", False), ("silu", True)])
def test_decode_between_forward_and_backward(act, gated):
    """Serving steps leave a pending backward as it was."""
    d, f = 256, 512
    _, _, a = make(d, f, act, gated, True)
    _, _, b = make(d, f, act, gated, True)
    x, dy, tok = batch(48, d, 1), batch(48, d, 2, 1e-2), batch(3, d, 3)
    a.freeze()
    for step in range(2):  # a fresh block's scales are far from each other, later ones nearly equal
        a.forward(x), b.forward(x)
        a.decode(tok, tok.clone())
        same(a.backward(dy), b.backward(dy))
