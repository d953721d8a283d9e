"""fp8_rmsnorm and its gradient in the kernel forms that test_rmsnorm_gpu.py's
shapes do not reach: one wave a row with four vectors a lane (1537 .. 2048
columns), the gradient's with two, and the wide forms in every type, with fp32
weights and 16-bit ones.  Bounds are that file's."""
import pytest
import torch

from tests import block_ref as R
from tests.test_rmsnorm_gpu import BF, F16, F32, check_forward, check_grad

pytestmark = pytest.mark.gpu
fp8mi = pytest.importorskip("fp8_tensor_scaled_quantize_amd")


@pytest.mark.parametrize("dt", [BF, F16, F32])
@pytest.mark.parametrize("wt", [F16, F32])
@pytest.mark.parametrize("rows,cols", [(1030, 2001), (3, 9003), (2, 16384), (2, 20001), (1, 32768)])
def test_forward_forms(dt, wt, rows, cols):
    x, res, w = R.rand((rows, cols), 2.0, dt, 70), R.rand((rows, cols), 1.0, dt, 71), R.rand((cols,), 1.0, wt, 72)
    for mode in ("row", "ring"):
        print(f"rmsnorm {rows}x{cols} {dt} weight {wt} {mode}", flush=True)
        check_forward(x, res, w, 0, mode, f"{rows}x{cols} {dt} {mode}", ld=cols % 2, shift=cols % 2)


@pytest.mark.parametrize("dt", [BF, F16, F32])
@pytest.mark.parametrize("wt", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(2050, 1001), (2050, 2001), (3, 9003), (2, 16384), (1, 32768), (600, 20001)])
def test_grad_forms(dt, wt, rows, cols):
    print(f"rmsnorm grad {rows}x{cols} {dt} weight {wt}", flush=True)
    check_grad(rows, cols, dt, R.rand((cols,), 1.0, wt, 73), True, f"{rows}x{cols} {dt}", cols % 2, cols % 2)
