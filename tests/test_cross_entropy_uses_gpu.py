"""The cross entropy where single values, not norms, are what a caller sees."""
import numpy as np
import pytest
import torch

import fp8_tensor_scaled_quantize_amd as fp8mi
import train_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF, U32 = 2.0 ** -8, 2.0 ** -24


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


@pytest.mark.parametrize("M,N", [(8, 300), (300, 3000), (500, 9000), (300, 50000)])
def test_infinite_logits(M, N):
    """-inf is a probability of zero (a loss of +inf at the target), +inf and NaN make
    the row's loss NaN, as does a row of nothing but -inf."""
    K = 16
    a, b = torch.zeros(M, K), torch.zeros(N, K)
    a[:, 0] = 1.0
    a[:, 1] = 448.0
    b[:, 0] = (torch.arange(N) % 3).float() - 1
    sb = torch.ones(N)
    sb[7] = 1e38  # 448 * 448 * 1e38 is beyond fp32
    b[7, 1] = -448.0
    t = torch.arange(M) % 5
    t[3] = 7
    sb, t = sb.to(DEV), t.to(DEV)
    loss, lse = fp8mi.fp8_cross_entropy(code(a).to(DEV), code(b).to(DEV), t, None, sb)
    l = b[:, 0].double().numpy()
    l[7] = -np.inf
    all_ = np.log(np.exp(l).sum())
    err = 200 * U32 * (1 + all_)
    for i in range(M):
        want = np.inf if int(t[i]) == 7 else all_ - l[int(t[i])]
        assert (float(loss[i]) == want) if np.isinf(want) else abs(float(loss[i]) - want) <= err
    assert (np.abs(f64(lse) - all_) <= err).all()
    b[7, 1] = 448.0  # +inf
    loss, lse = fp8mi.fp8_cross_entropy(code(a).to(DEV), code(b).to(DEV), t, None, sb)
    assert torch.isnan(loss).all()
    a[:, 1] = 0.0
    a[2, 1] = 448.0  # row 2's logits are all -inf: its own scale as well as the columns'
    b[:, 1] = -448.0
    sb.fill_(1e38)
    sa = torch.zeros(M, device=DEV)
    sa[2] = 1.0
    loss, lse = fp8mi.fp8_cross_entropy(code(a).to(DEV), code(b).to(DEV), t, sa, sb)
    assert torch.isnan(loss[2]) and int(torch.isnan(loss).sum()) == 1


# rows straight from the codes, the same in K splits of G^T A, tiles, tiles in K splits
@pytest.mark.parametrize("M,N", [(40, 300), (1030, 700), (300, 3000), (1500, 600)])
@pytest.mark.parametrize("size", [1.0, 1e-25, 1e25])
def test_rows_of_little_weight(M, N, size):
    """Vocabulary rows whose gradient comes from a single row of small dloss: each is
    the formula's by itself, whatever the batch's largest dloss."""
    ratios = [1e-5, 1e-7, 1e-8, 1e-9]
    Q, S, K = len(ratios), 16, 128
    rng = np.random.default_rng(M)
    a, b = (torch.from_numpy(rng.integers(0x28, 0x70, (n, K)) | (rng.integers(0, 2, (n, K)) << 7)).to(torch.uint8)
            for n in (M, N))  # magnitudes of 2^-2 to 2^7
    low, high = int(code(-448.0)), int(code(448.0))
    # S columns of K for each small row q: only it has no -448 there, and only the vocabulary's row q has 448
    a[:, :Q * S] = low
    b[:, :Q * S] = 0
    for q in range(Q):
        a[5 + q, q * S:(q + 1) * S] = 0
        b[9 + q] = 0
        b[9 + q, q * S:(q + 1) * S] = high
    t = torch.randint(9 + Q, N, (M,))
    t[5:5 + Q] = 9 + torch.arange(Q)
    sa, sb = np.float32(2.0 ** -7), np.float32(2.0 ** -7)  # those columns: -196 elsewhere
    d = torch.rand(M) * 0.5 + 0.5
    d[5:5 + Q] = torch.tensor(ratios)
    d *= size
    args = [x.to(DEV) for x in (a, b, t)]
    scales = [torch.tensor([s], device=DEV) for s in (sa, sb)]
    _, lse = fp8mi.fp8_cross_entropy(*args, *scales)
    da, db = fp8mi.fp8_cross_entropy_grad(*args, lse, d.to(DEV), *scales)
    A, B = R.decode_e4m3(a.numpy()), R.decode_e4m3(b.numpy())
    l = (A @ B.T) * (float(sa) * float(sb))
    el = (np.abs(A) @ np.abs(B).T) * float(sa) * float(sb) * K * 2 * U32 + 4 * U32 * np.abs(l)
    p = np.exp(l - f64(lse)[:, None])
    G = p.copy()
    G[np.arange(M), t.numpy()] -= 1
    w, most = d.double().numpy(), float(d.max())
    # G before its rounding (the argument's errors), then fp16's half step or the smallest one, which a row of little
    # weight has up to 2^8 times larger
    eg = p * (el + 4 * U32 * (np.abs(l) + np.abs(f64(lse))[:, None]) + 4 * U32) + 2 * U32 * np.abs(G)
    eg = eg + 2.0 ** -11 * (np.abs(G) + eg) + np.where(w < most * 2.0 ** -20, 2.0 ** -31, 2.0 ** -39)[:, None]
    for q in range(Q):
        i, j = 5 + q, 9 + q
        rest = np.delete(p[:, j], i).max()
        assert rest < 1e-30  # the row is alone
        x = w[i] * float(sa) * A[i]
        want = G[i, j] * x
        # dloss A in fp16: half a step, or 2^-39 of the largest dloss per unit of a code
        ex = 2.0 ** -11 * np.abs(x) + 2.0 ** -39 * most * float(sa)
        err = np.abs(G[i, j]) * ex + eg[i, j] * (np.abs(x) + ex) + (M + 8) * 2 * U32 * np.abs(want)
        got = f64(db[j])
        assert (np.abs(got - want) <= err + HALF * (np.abs(want) + err)).all(), (q, np.abs(got - want).max() / np.abs(want).max())
        assert np.linalg.norm(got - want) <= 0.02 * np.linalg.norm(want)
    dwant = w[:, None] * float(sb) * (G @ B)
    derr = w[:, None] * float(sb) * (eg @ np.abs(B) + (N + 8) * 2 * U32 * (np.abs(G) @ np.abs(B)))
    assert (np.abs(f64(da) - dwant) <= derr + HALF * (np.abs(dwant) + derr)).all()
    # alone, each is the same
    assert torch.equal(da, fp8mi.fp8_cross_entropy_grad(*args, lse, d.to(DEV), *scales, need_db=False)[0])
    assert torch.equal(db, fp8mi.fp8_cross_entropy_grad(*args, lse, d.to(DEV), *scales, need_da=False)[1])
