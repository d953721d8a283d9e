"""Uses of the operators that end a training step which need no GPU: names, and
refusals of the binding and of the objects before anything is launched."""
import pytest
import torch

import fp8_tensor_scaled_quantize_amd as fp8mi
from fp8_tensor_scaled_quantize_amd.head import Fp8Head


def test_the_optimizers_names():
    """The step and the norm are reached with and without the prefix."""
    for name in ("adamw_step", "grad_norm"):
        assert name in fp8mi.__all__ and "fp8_" + name in fp8mi.__all__
        assert getattr(fp8mi, name) is getattr(fp8mi, "fp8_" + name)


OTHERS = [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.bool]


def test_cross_entropy_refuses_other_formats():
    """Operands are E4M3 codes: tensors of another fp8 type have other values."""
    a, b, t = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(9, 32, dtype=torch.uint8), torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)

    def calls(x, y):
        return (lambda: fp8mi.fp8_cross_entropy(x, y, t), lambda: fp8mi.fp8_cross_entropy_grad(x, y, t, f, f))

    for dtype in OTHERS:
        for x, y in ((a.view(dtype), b), (a, b.view(dtype))):
            for call in calls(x, y):
                with pytest.raises(ValueError, match="E4M3 codes"):
                    call()
    for dtype in (torch.int8, torch.float8_e4m3fn):  # only the device is wrong here
        for call in calls(a.view(dtype), b.view(dtype)):
            with pytest.raises(ValueError, match="host tensor"):
                call()


def test_eight_bit_states_refuse_other_formats():
    w, one = torch.zeros(4), torch.zeros(1)

    def step(m, v):
        fp8mi.fp8_adamw_step([w], [w], [m], [v], 1, exp_avg_scales=[one], exp_avg_sq_scales=[one])

    codes = torch.zeros(4, dtype=torch.uint8)
    for dtype in OTHERS:
        for m, v in ((codes.view(dtype), codes), (codes, codes.view(dtype))):
            with pytest.raises(ValueError, match="E4M3 codes"):
                step(m, v)
    for dtype in (torch.int8, torch.float8_e4m3fn):  # only the device is wrong here
        with pytest.raises(ValueError, match="host tensor"):
            step(codes.view(dtype), codes.view(dtype))


def test_a_freeze_that_fails_leaves_nothing_to_score_with():
    head = Fp8Head(torch.ones(32), torch.zeros(9, 32))
    for _ in range(2):
        with pytest.raises(ValueError, match="host tensor"):
            head.freeze()
        with pytest.raises(RuntimeError, match="freeze"):
            head.score(torch.zeros(2, 32), torch.zeros(2, dtype=torch.int64))
