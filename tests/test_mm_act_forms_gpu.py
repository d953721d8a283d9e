"""fp8_mm_act in the kernel forms that test_mm_act_gpu.py's shapes do not reach,
or reach without activation, gating, residual or fp8 output.  The form that a
shape takes on 256 CUs stands beside it.  Bounds are that file's."""
import pytest
import torch

from tests import block_ref as R
from tests.gpu_util import DEV
from tests.test_mm_act_gpu import BF, F16, F32, codes, run

pytestmark = pytest.mark.gpu
fp8mi = pytest.importorskip("fp8_tensor_scaled_quantize_amd")

# ragged in M and N
FORMS = [
    (31, 3590, 272),     # rows, two blocks of 16, 4 waves
    (31, 3590, 1040),    # rows, two blocks of 16, 8 waves
    (20, 4090, 2080),    # rows, two blocks of 16, 16 waves
    (9, 3000, 2064),     # rows, one block of 16, 16 waves: one step a wave, one has two
    (60, 1538, 6912),    # 64 x 32 tiles, eight stages
    (2040, 1530, 1040),  # 64 x 128 tiles
    (1990, 1530, 256),   # 64 x 128 tiles, short K
    (4090, 3586, 128),   # 128 x 128 tiles, short K
    (4350, 4090, 2064),  # 128 x 192 tiles, K above 2048
]


def some_rows(M):
    """All rows of a small product; of a large one a few and the last."""
    return None if M <= 64 else torch.cat([torch.arange(0, M, 331), torch.arange(M - 3, M)])


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out_fmt", [None, 0])
def test_forms(M, N, K, gated, out_fmt):
    act = ["silu", "gelu", "relu"][(M + N // 2) % 3]
    run(M, N, K, act, gated, out_fmt, res_dt=[BF, F32, F16][M % 3], bias_dt=[F32, BF, F16][N // 2 % 3], keep_z=True,
        row_scales=True, ring=M % 2 == 0, rows=some_rows(M), tag="forms")


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("res_dt", [None, BF, F16, F32])
def test_activations_and_residuals_in_tiles(act, gated, res_dt):
    """64 x 64 tiles: every activation with every residual type."""
    for out_fmt in (None, 0):
        run(330, 1030, 272, act, gated, out_fmt, res_dt, F32, keep_z=out_fmt is None, rows=some_rows(330), tag=f"{res_dt}")


# shapes whose product runs in tiles: they sum K in the plain product's order
TILED = [(300, 2050, 272), (129, 4098, 800), (60, 1538, 6912), (2040, 1530, 1040), (1990, 1530, 256), (300, 520, 48),
         (4090, 3586, 128), (4090, 3586, 288), (4350, 4090, 2064), (8190, 6910, 272)]


@pytest.mark.parametrize("M,N,K", TILED)
def test_bits_of_the_plain_product(M, N, K):
    """No activation, no residual: fp8_mm's bits, in y and in z alike."""
    a, b = codes(M, K, 11).to(DEV), codes(N, K, 12).to(DEV)
    s, bias = torch.tensor([0.02], device=DEV), R.rand((N,), 1.0, BF, 13).to(DEV)
    z = torch.empty(M, N, dtype=BF, device=DEV)
    print(f"mm_act bits {M}x{N}x{K}", flush=True)
    want = fp8mi.fp8_mm(a, b, 0, 0, s, s, bias)
    got = fp8mi.fp8_mm_act(a, b, s, s, bias, z_out=z)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(z, want)


@pytest.mark.parametrize("M,N,K", [(31, 3590, 1040), (60, 1538, 6912), (2040, 1530, 1040), (4350, 4090, 2064)])
def test_residual_in_place_in_every_form(M, N, K):
    run(M, N, K, "gelu", res_dt=BF, bias_dt=BF, inplace=True, rows=some_rows(M), tag="in place")
