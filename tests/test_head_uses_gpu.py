"""Fp8Head in uses that its own kernels' tests do not make."""
import pytest
import torch

from fp8_tensor_scaled_quantize_amd.head import Fp8Head

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rand(*shape, sigma=1.0, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * sigma).to(dtype)


def test_what_the_loss_cannot_take_is_refused_before_a_ring_moves():
    """More rows than fp8_cross_entropy takes, and weights that the quantize refuses."""
    many = torch.zeros((1 << 20) + 1, 16, dtype=torch.bfloat16, device=DEV)
    few = rand(4, 16, seed=1)
    for weight, x, text in [
        (rand(32, 16), many, "more than"), (rand(32, 16).double(), few, "weight must be"),
        (rand(16, 32).t(), few, "unit column stride"), (rand(32, 16).cpu(), few, "weight is on"),
    ]:
        head = Fp8Head(torch.ones(16, device=DEV), weight)
        rings = {k: r.clone() for k, r in head.rings.items()}
        with pytest.raises(ValueError, match=text):
            head.forward(x, torch.zeros(x.shape[0], dtype=torch.int64, device=DEV))
        assert all(torch.equal(r, head.rings[k]) for k, r in rings.items())
    head = Fp8Head(torch.ones(16, device=DEV), rand(32, 16))
    loss = head.forward(many[:-1], torch.zeros(1 << 20, dtype=torch.int64, device=DEV))  # as many as it takes
    assert abs(float(loss) - torch.log(torch.tensor(32.0)).item()) < 1e-5
