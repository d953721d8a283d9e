"""The cross entropy where single values, not norms, are what a caller sees."""
import numpy as np
import pytest
import torch

import fp8_tensor_scaled_quantize_amd as fp8mi
import train_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32 = 2.0 ** -24


def code(x):
    """E4M3 codes of values that it holds."""
    c = torch.as_tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn)
    assert torch.equal(c.float(), torch.as_tensor(x, dtype=torch.float32))
    return c.view(torch.uint8)


def f64(t):
    return t.detach().cpu().double().numpy()


# rows straight from the codes, tiles of 64, 128 and 256 with a band
@pytest.mark.parametrize("M,N", [(4, 300), (300, 3000), (500, 9000), (300, 50000)])
@pytest.mark.parametrize("top", [40.0, 100.0, 1000.0])
def test_loss_of_a_confident_token(M, N, top):
    """One logit, the target's, stands some 14 above all others: the loss, their sum,
    is 10^-4 to 10^-2 and has to come out as such whatever the logits' size is."""
    K = 16
    step = {40.0: (160.0, 224.0), 100.0: (64.0, 224.0), 1000.0: (8.0, 176.0)}[top]
    a, b = torch.zeros(M, K), torch.zeros(N, K)
    a[:, 0] = torch.tensor([448.0, 416.0, 384.0, 352.0])[torch.arange(M) % 4]  # sums of products below 2^18: exact
    a[:, 1] = step[0]
    b[:, 0], b[:, 1] = 448.0, -step[1]
    b[N // 3, 1] = step[1]
    sa, sb = np.float32(2.0 ** -9), np.float32(top / 448 ** 2 * 2.0 ** 9)
    t = torch.full((M,), N // 3, device=DEV)
    mean = torch.empty(2, device=DEV)
    loss, lse = fp8mi.fp8_cross_entropy(code(a).to(DEV), code(b).to(DEV), t, torch.tensor([sa], device=DEV),
                                        torch.tensor([sb], device=DEV), mean_out=mean)
    l = (a.double() @ b.double().t()).numpy() * (float(sa) * float(sb))
    own = l[:, N // 3]
    # (log1p: the 64-bit form must not lose it either)
    want = np.log1p((N - 1) * np.exp(l[:, 0] - own))
    # Relative: each logit is rounded at most three times (two products of scales, the product), so a difference of
    # two is off by 6 half steps of the logits, and exp2's and the sum's terms by a few of 1.  Absolute: additions to
    # a sum of 1 or more, half a step of [1, 2) each: at most 64 in a tile's lane, 16 lanes and waves, 8 a round of the
    # join (at most 2 here) and 8 halves of its segments; log2's two steps of the result beside them.
    err = want * (6 * U32 * (np.abs(l).max() + 4) + 16 * U32) + (64 + 16 + 16 + 8) * U32
    assert (want > 8 * err).all()  # the bound says something
    assert (np.abs(f64(loss) - want) <= err).all(), (np.abs(f64(loss) - want) / err).max()
    assert abs(float(mean[0]) - want.mean()) <= err.max() + U32
    assert (np.abs(f64(lse) - (own + want)) <= 8 * U32 * (own + 1) + err).all()
