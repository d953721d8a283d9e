"""The cross entropy at sizes that reach its larger tiles, K splits, pieces and
row counts, against a 64-bit computation on the GPU."""
import pytest
import torch

import fp8_tensor_scaled_quantize_amd as fp8mi

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
HALF, U32 = 2.0 ** -8, 2.0 ** -24


def operands(M, N, K, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    out = []
    for rows, sigma in ((M, 1.0), (N, 2.0 / K ** 0.5)):
        v = torch.randn(rows, K, generator=g, device=DEV) * sigma
        s = 448 / v.abs().amax()
        out.append(((v * s).to(E4M3).view(torch.uint8), (1 / s).reshape(1)))
    t = torch.randint(0, N, (M,), generator=g, device=DEV)
    t[::5] = -100
    return out[0][0], out[1][0], t, out[0][1], out[1][1], g


def exact(a, b, t, sa, sb, d):
    a, b = a.view(E4M3).double() * sa.double(), b.view(E4M3).double() * sb.double()
    bt = b.t().contiguous()
    lse, loss, da, db = [], [], [], torch.zeros_like(b)
    for i in range(0, a.shape[0], 2048):
        l = a[i:i + 2048] @ bt
        p = torch.softmax(l, 1)
        lse.append(torch.logsumexp(l, 1))
        ti = t[i:i + 2048]
        rows = torch.arange(l.shape[0], device=DEV)
        loss.append(torch.where(ti >= 0, lse[-1] - l[rows, ti.clamp(min=0)], 0.0))
        p[rows, ti.clamp(min=0)] -= 1
        p *= torch.where(ti >= 0, d.double().expand(a.shape[0])[i:i + 2048], 0.0)[:, None]
        da.append(p @ b)
        db += p.t().contiguous() @ a[i:i + 2048]
    return torch.cat(loss), torch.cat(lse), torch.cat(da), db


# 64-wide, 128-wide, 256-wide tiles with and without edges, one and more pieces, K from a step to long
SHAPES = [(2048, 20000, 512), (1111, 33001, 640), (4100, 9000, 1040), (600, 70001, 256), (96, 50001, 512), (64, 40000, 768),
          (33, 8200, 2048), (17, 8191, 4096), (200, 3000, 4112), (300, 300, 8192), (5000, 700, 96), (129, 131072, 64),
          (8000, 33000, 32), (1500, 2000, 16), (150, 9000, 16)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forms(M, N, K):
    a, b, t, sa, sb, g = operands(M, N, K, seed=M + N)
    d = torch.rand(M, generator=g, device=DEV) + 0.1
    mean = torch.empty(2, device=DEV)
    loss, lse = fp8mi.fp8_cross_entropy(a, b, t, sa, sb, mean_out=mean)
    wloss, wlse, wda, wdb = exact(a, b, t, sa, sb, d)
    # a logit's terms add up to at most |a| |b| (Cauchy-Schwarz), its sums are off by K 2^-23 of that at most and in
    # truth by the root of it: the bound below is the worst case
    na = (a.view(E4M3).double() * sa.double()).norm(dim=1)
    nb = (b.view(E4M3).double() * sb.double()).norm(dim=1).max()
    el = na * nb * K * 2 * U32
    assert ((lse - wlse).abs() <= el + 200 * U32 * (1 + wlse.abs())).all()
    assert ((loss - wloss).abs() <= 2 * el + 200 * U32 * (1 + wlse.abs() + na * nb)).all()
    # and as a whole: errors of single sums are independent, of the order of 2^-22 of a logit
    assert (lse - wlse).norm() / wlse.norm() < 1e-6
    n = int((t >= 0).sum())
    assert abs(float(mean[0]) - float(wloss.sum()) / n) <= 1e-5 and abs(float(mean[1]) * n - 1) < 1e-6
    da, db = fp8mi.fp8_cross_entropy_grad(a, b, t, lse, d, sa, sb)
    # the outputs round to bf16, G and the rows of d A to fp16 (an eighth of it), independently
    for got, want in ((da, wda), (db, wdb)):
        assert (got - want).norm() / want.norm() <= 1.25 * HALF
        big = want.abs().amax(1)
        # no row is off as a whole
        assert ((got - want).norm(dim=1) <= 4 * HALF * want.norm(dim=1) + 1e-6 * big.max()).all()
    assert not da[::5].any()


@pytest.mark.parametrize("M,N,K", [(40, 600, 48), (300, 5000, 208), (2100, 3000, 336), (300, 33000, 80)])
def test_nothing_beside_the_operands_is_used(M, N, K):
    """Rows of a wider buffer that ends with the last row's last code: what lies
    between the rows (NaN codes) and behind them stays out."""
    a, b, t, sa, sb, g = operands(M, N, K, seed=7)
    d = torch.rand(M, generator=g, device=DEV)
    loss, lse = fp8mi.fp8_cross_entropy(a, b, t, sa, sb)
    da, db = fp8mi.fp8_cross_entropy_grad(a, b, t, lse, d, sa, sb)

    def wide(x):
        ld = x.shape[1] + 48
        buf = torch.full((x.shape[0] * ld - 48,), 0x7F, dtype=torch.uint8, device=DEV)
        view = torch.as_strided(buf, x.shape, (ld, 1))
        view.copy_(x)
        return view

    a2, b2 = wide(a), wide(b)
    loss2, lse2 = fp8mi.fp8_cross_entropy(a2, b2, t, sa, sb)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    assert all(torch.equal(x, y) for x, y in zip((da, db), fp8mi.fp8_cross_entropy_grad(a2, b2, t, lse, d, sa, sb)))


def test_rows_as_far_apart_as_allowed():
    """ldb = 2^22: a buffer's offsets hold 256 such rows, so the vocabulary is taken in pieces."""
    M, N, K, ld = 3000, 300, 64, 1 << 22
    a, b, t, sa, sb, g = operands(M, N, K, seed=9)
    far = torch.as_strided(torch.empty((N - 1) * ld + K, dtype=torch.uint8, device=DEV), (N, K), (ld, 1))
    far.copy_(b)
    d = torch.rand(M, generator=g, device=DEV)
    loss, lse = fp8mi.fp8_cross_entropy(a, b, t, sa, sb)
    loss2, lse2 = fp8mi.fp8_cross_entropy(a, far, t, sa, sb)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    da, db = fp8mi.fp8_cross_entropy_grad(a, b, t, lse, d, sa, sb)
    da2, db2 = fp8mi.fp8_cross_entropy_grad(a, far, t, lse, d, sa, sb)
    assert torch.equal(db, db2)
    # da's sums are split elsewhere: each side is off by its own bf16 rounding
    assert (da.double() - da2.double()).norm() <= 2 * HALF * da.double().norm()
    few, flse = fp8mi.fp8_cross_entropy(a[:9], far, t[:9], sa, sb)
    assert (few - loss[:9]).abs().max() < 1e-5


def test_the_same_whatever_the_workspace_holds():
    a, b, t, sa, sb, g = operands(1500, 20011, 528, 3)
    d = torch.ones(1, device=DEV)
    size = fp8mi.fp8_cross_entropy_workspace_bytes(1500, 20011, 528), fp8mi.fp8_cross_entropy_grad_workspace_bytes(1500, 20011, 528)
    out = []
    for fill in (0, 0xFF, 0x7F):
        ws = [torch.full((n + 16,), fill, dtype=torch.uint8, device=DEV)[16:] for n in size]
        loss, lse = fp8mi.fp8_cross_entropy(a, b, t, sa, sb, workspace=ws[0])
        out.append((loss, lse, *fp8mi.fp8_cross_entropy_grad(a, b, t, lse, d, sa, sb, workspace=ws[1])))
    for o in out[1:]:
        assert all(torch.equal(x, y) for x, y in zip(o, out[0]))


def test_more_logits_than_a_grid_holds():
    """2^39 logits: two launches.  Rows of A are 0 or (1, 0, ...), B's are (1, 0, ...) or (2, 0, ...)."""
    M, N, K = 1 << 20, 1 << 19, 16
    one, two = (int(torch.tensor(x).to(E4M3).view(torch.uint8)) for x in (1.0, 2.0))
    a, b = torch.zeros(M, K, dtype=torch.uint8, device=DEV), torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    a[::3, 0] = one
    b[:, 0] = one
    b[1::2, 0] = two
    t = torch.arange(M, device=DEV) % N
    loss, lse = fp8mi.fp8_cross_entropy(a, b, t)
    on = a[:, 0] == one
    e = torch.tensor(1.0, dtype=torch.float64, device=DEV).exp()
    want = torch.where(on, (N / 2 * (e + e * e)).log(), torch.tensor(float(N), device=DEV).double().log())
    logit = torch.where(on, 1.0 + (t % 2).double(), 0.0)
    # a sum's terms pass fewer than 256 roundings (64 in a tile, 128 tiles to a segment of the join, 16 segments), each
    # of 2^-23 with its exponential's; lse and loss, below 16, round by 2^-21 at most
    for got, w in ((lse, want), (loss, want - logit)):
        assert (got.double() - w).abs().max() <= 256 * 2.0 ** -23 + 2 * 2.0 ** -21


# many rows of few codes: G^T A in K splits, over one and over several pieces; sums that are complete at once
SPLIT_SHAPES = [(300000, 1000, 32), (6000, 60, 1024), (3000, 300, 512), (1500, 1500, 768), (100000, 2, 16), (70000, 65, 48),
                (1024, 1000, 16), (4097, 129, 272), (1023, 1, 16), (1025, 1500, 1040)]


@pytest.mark.parametrize("M,N,K", SPLIT_SHAPES)
def test_splits_over_the_rows(M, N, K):
    if N > 1:
        return test_forms(M, N, K)
    # A vocabulary of one: G = exp(l - lse) - 1 is 0 in truth, as are the gradients.  lse is l times ln 2 and is taken
    # times log2 e again: with the two constants' roundings and the exponential's, fewer than 16 half steps of 1 + |l|, and
    # |l| <= |a| |b|.  G's rounding to fp16 adds 2^-11 of it, the outputs' 2^-8 (together below a hundredth), dA is d G b and
    # dB at most the sum of d |G| |a|.
    a, b, t, sa, sb, g = operands(M, N, K, seed=M + N)
    d = torch.rand(M, generator=g, device=DEV) + 0.1
    loss, lse = fp8mi.fp8_cross_entropy(a, b, t, sa, sb)
    da, db = fp8mi.fp8_cross_entropy_grad(a, b, t, lse, d, sa, sb)
    na = (a.view(E4M3).double() * sa.double()).norm(dim=1)
    nb = (b.view(E4M3).double() * sb.double()).norm()
    most = d.double() * 1.01 * 16 * U32 * (1 + na * nb)
    assert (da.double().norm(dim=1) <= most * nb).all() and db.double().norm() <= (most * na).sum()


@pytest.mark.parametrize("M,N,K", [(6000, 60, 1024), (1500, 1500, 768), (512, 2000, 1024), (100, 20000, 512)])
def test_each_gradient_alone(M, N, K):
    """Alone, a product may run in other tiles than beside the other: the sums' order is the same."""
    a, b, t, sa, sb, g = operands(M, N, K, seed=5)
    d = torch.rand(M, generator=g, device=DEV)
    _, lse = fp8mi.fp8_cross_entropy(a, b, t, sa, sb)
    for dloss in (d, d[:1].clone()):
        da, db = fp8mi.fp8_cross_entropy_grad(a, b, t, lse, dloss, sa, sb)
        assert torch.equal(da, fp8mi.fp8_cross_entropy_grad(a, b, t, lse, dloss, sa, sb, need_db=False)[0])
        assert torch.equal(db, fp8mi.fp8_cross_entropy_grad(a, b, t, lse, dloss, sa, sb, need_da=False)[1])
        wide = [torch.full((x.shape[0], K + 3), 7.0, dtype=torch.bfloat16, device=DEV) for x in (da, db)]
        fp8mi.fp8_cross_entropy_grad(a, b, t, lse, dloss, sa, sb, da=wide[0][:, :K], db=wide[1][:, :K])
        assert torch.equal(wide[0][:, :K], da) and torch.equal(wide[1][:, :K], db)
        assert all((w[:, K:] == 7).all() for w in wide)


def test_ignored_rows_of_complete_sums():
    """A dloss that is NaN where the row is ignored, with sums finished by the product itself."""
    a, b, t, sa, sb, g = operands(700, 200, 64, seed=6)
    _, lse = fp8mi.fp8_cross_entropy(a, b, t, sa, sb)
    d = torch.rand(700, generator=g, device=DEV)
    want = fp8mi.fp8_cross_entropy_grad(a, b, t, lse, d, sa, sb)
    d[t < 0] = float("nan")
    a[t < 0] = 0x7F
    got = fp8mi.fp8_cross_entropy_grad(a, b, t, lse, d, sa, sb)
    assert all(torch.equal(x, y) for x, y in zip(want, got)) and not got[0][t < 0].any()
