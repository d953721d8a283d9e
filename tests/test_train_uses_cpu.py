"""Uses of the operators that end a training step which need no GPU: names, and
refusals of the binding and of the objects before anything is launched."""
import fp8_tensor_scaled_quantize_amd as fp8mi


def test_the_optimizers_names():
    """The step and the norm are reached with and without the prefix."""
    for name in ("adamw_step", "grad_norm"):
        assert name in fp8mi.__all__ and "fp8_" + name in fp8mi.__all__
        assert getattr(fp8mi, name) is getattr(fp8mi, "fp8_" + name)
