"""fp8_cross_entropy and its gradient against 64-bit forms (train_ref.py)."""
import numpy as np
import pytest
import torch

import fp8_tensor_scaled_quantize_amd as fp8mi
import train_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = 2.0 ** -8  # half a bf16 step


def f64(t):
    return t.detach().cpu().double().numpy()


class Case:
    def __init__(self, M, N, K, seed=0, ignored=0.25, row_scales=False, spread=3.0, pad=0, targets=torch.int64):
        rng = np.random.default_rng(seed)
        # codes below 2^6: logits of a few units at these scales
        a, b = (rng.integers(0, 0x58, (n, K)) | (rng.integers(0, 2, (n, K)) << 7) for n in (M, N))
        rms = [np.sqrt((R.decode_e4m3(x) ** 2).mean()) if x.size else 1.0 for x in (a, b)]
        self.sa = np.float32(1 / rms[0]) * np.ones(1, np.float32)
        self.sb = np.float32(spread / (rms[1] * np.sqrt(K))) * np.ones(1, np.float32)
        if row_scales:
            self.sa = (self.sa * np.exp(rng.normal(0, 0.3, M))).astype(np.float32)
            self.sb = (self.sb * np.exp(rng.normal(0, 0.3, N))).astype(np.float32)
        t = rng.integers(0, N, M)
        self.t = np.where(rng.random(M) < ignored, rng.choice([-1, -100], M), t)
        self.a, self.b = (self._place(x.astype(np.uint8), pad) for x in (a, b))
        self.targets = torch.from_numpy(self.t).to(targets).to(DEV)
        self.scales = [torch.from_numpy(s).to(DEV) for s in (self.sa, self.sb)]
        self.codes = a, b
        self.l = R.logits(a, b, self.sa.astype(np.float64), self.sb.astype(np.float64))
        # A logit's terms: exact products; K - 1 sums, each rounded by half a step of at most the terms' magnitudes (the
        # MFMA may cut instead of round: a whole step), and four roundings of its scales
        mag = R.logits(np.asarray(a) & 127, np.asarray(b) & 127, self.sa.astype(np.float64), self.sb.astype(np.float64))
        self.el = mag * (K * 2 * R.U32) + 4 * R.U32 * np.abs(self.l)

    @staticmethod
    def _place(x, pad):
        buf = torch.full((x.shape[0], x.shape[1] + pad), 0x7F, dtype=torch.uint8, device=DEV)  # NaN beside the rows
        buf[:, :x.shape[1]] = torch.from_numpy(x)
        return buf[:, :x.shape[1]]

    def forward(self, **kw):
        return fp8mi.fp8_cross_entropy(self.a, self.b, self.targets, *self.scales, **kw)

    def check_forward(self, loss, lse, mean=None):
        want, wlse, wmean = R.cross_entropy(self.l, self.t)
        # lse: the logits' own error (a weighted mean of them), the exponentials' (arguments in powers of two of at most
        # 2^8 units: 2^-16 ulp-wise relative each would be the argument's rounding 2^8 U32; 2 U32 of exp2), the sum's
        # and the logarithm's roundings: N-term sums in tiles of at most 64 terms per lane, then pairs
        top = np.abs(self.l).max(1)
        el = self.el.max(1)
        e_lse = el + (8 + 64 + 4 * top) * R.U32 + 4 * R.U32 * np.abs(wlse)
        assert (np.abs(f64(lse) - wlse) <= e_lse).all()
        e_loss = e_lse + el + 4 * R.U32 * top
        assert (np.abs(f64(loss) - want) <= np.where(self.t >= 0, e_loss, 0.0)).all()
        if mean is not None:
            assert (np.abs(f64(mean) - wmean) <= np.array([e_loss.max(), 0.0]) + 2 * R.U32 * np.abs(wmean)).all()

    def check_grad(self, da, db, dloss, lse):
        l, M = self.l, len(self.t)
        g = np.exp(l - f64(lse)[:, None])
        # G's error before its rounding: the argument's (logit, lse, product with log2 e) and exp2's
        eg = g * (self.el + 4 * R.U32 * (np.abs(l) + np.abs(f64(lse))[:, None]) + 4 * R.U32)
        g[np.arange(M), np.maximum(self.t, 0)] -= 1
        eg = eg + 2 * R.U32 * np.abs(g)
        before = eg
        eg = eg + (np.abs(g) + eg) * 2.0 ** -11 + 2.0 ** -39  # rounded to fp16, in units of 2^-14
        d = np.where(self.t >= 0, np.broadcast_to(dloss, M), 0.0)[:, None]
        a, b = R.decode_e4m3(self.codes[0]) * float(self.sa[0]), R.decode_e4m3(self.codes[1]) * float(self.sb[0])
        # with a dloss per row db takes fp16 rows of d A: a half step (or 2^-25 of the largest d's unit) of each more
        ea = np.abs(d * a) * 2.0 ** -11 + 2.0 ** -24 * np.abs(d).max() * float(self.sa[0]) if np.size(dloss) > 1 else 0 * a
        for got, x, y, ex, e0, ey, n in ((da, d * g, b, np.abs(d) * eg, np.abs(d) * before, 0 * b, len(b)),
                                         (db, g.T, d * a, eg.T, before.T, ea, len(a))):
            if got is None:
                continue
            want = x @ y
            # sums of n terms in fp32, their factors' roundings, and one rounding to bf16
            err = ex @ np.abs(y) + (np.abs(x) + ex) @ ey + (n + 8) * 2 * R.U32 * (np.abs(x) @ np.abs(y))
            assert (np.abs(f64(got) - want) <= err + HALF * (np.abs(want) + err)).all()
            # and as a whole: the output's half steps, G's and d A's (an eighth of those each; all independent), apart from
            # what G is off by before it is rounded (with one column G is that alone)
            off = np.linalg.norm(f64(got) - want)
            tiny = 2.0 ** -39 * np.sqrt(x.size) * np.linalg.norm(y)
            assert off <= 1.25 * HALF * np.linalg.norm(want) + np.linalg.norm(e0 @ np.abs(y)) + tiny, off


SHAPES = [(1, 2, 16), (1, 1, 16), (3, 17, 32), (16, 255, 64), (17, 256, 128), (64, 257, 144), (65, 1000, 512), (127, 513, 48),
          (128, 2048, 256), (200, 4001, 96), (255, 300, 1040), (257, 777, 80), (700, 5003, 64), (1030, 1500, 32)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("row_scales", [False, True])
def test_forward(M, N, K, row_scales):
    c = Case(M, N, K, seed=M, row_scales=row_scales, pad=16 if row_scales else 0,
             targets=torch.int32 if row_scales else torch.int64)
    mean = torch.empty(2, device=DEV)
    loss, lse = c.forward(mean_out=mean)
    c.check_forward(loss, lse, mean)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("per_row", [False, True])
def test_gradient(M, N, K, per_row):
    c = Case(M, N, K, seed=M + 1, pad=16 if per_row else 0)
    _, lse = c.forward()
    dloss = torch.rand(M if per_row else 1, device=DEV) + 0.1
    da, db = fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, dloss, *c.scales)
    c.check_grad(da, db, f64(dloss), lse)


def test_big_tiles_and_several_pieces():
    """Sizes at which the largest tiles, K splits and more than one piece are taken
    (pieces of 8192 columns with 8192 rows), checked on some rows and columns."""
    M, N, K = 8192, 17000, 64
    c = Case(64, N, K, seed=5)
    a = c.a.repeat(M // 64, 1)
    t = c.targets.repeat(M // 64)
    mean = torch.empty(2, device=DEV)
    loss, lse = fp8mi.fp8_cross_entropy(a, c.b, t, *c.scales, mean_out=mean)
    for k in (0, 31, 127):
        c.check_forward(loss[64 * k:64 * k + 64], lse[64 * k:64 * k + 64])
    # every row block is the same: da too, and db is 128 times one block's
    dl = torch.full((1,), 0.5, device=DEV)
    da, db = fp8mi.fp8_cross_entropy_grad(a, c.b, t, lse, dl, *c.scales)
    for k in (0, 31, 127):
        assert torch.equal(da[64 * k:64 * k + 64], da[:64])
    c.check_grad(da[:64], None, 0.5, lse[:64])
    c.check_grad(None, db / 128, 0.5, lse[:64])


def test_scales_and_values_at_the_edges():
    """Logits far apart (exp underflows), all alike, and a vocabulary of one."""
    for spread in (100.0, 1e-6):
        c = Case(70, 300, 64, seed=2, spread=spread)
        loss, lse = c.forward()
        c.check_forward(loss, lse)
        da, db = fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, torch.ones(1, device=DEV), *c.scales)
        assert torch.isfinite(da).all() and torch.isfinite(db).all()
        if spread < 1:
            c.check_grad(da, db, 1.0, lse)
    c = Case(5, 1, 16, seed=3, ignored=0.0)
    loss, lse = c.forward()
    assert (loss.abs() <= 1e-5).all()


def test_everything_ignored_and_no_rows():
    c = Case(40, 100, 32, ignored=1.0)
    mean = torch.full((2,), 7.0, device=DEV)
    loss, lse = c.forward(mean_out=mean)
    assert not loss.any() and not mean.any() and torch.isfinite(lse).all()
    da, db = fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, torch.ones(1, device=DEV), *c.scales)
    assert not da.any() and not db.any()
    mean.fill_(7)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    loss, lse = fp8mi.fp8_cross_entropy(c.a[:0], c.b, none, *c.scales, mean_out=mean)
    assert loss.numel() == 0 and not mean.any()
    da, db = fp8mi.fp8_cross_entropy_grad(c.a[:0], c.b, none, lse, torch.ones(1, device=DEV), *c.scales)
    assert da.shape == (0, 32) and db.shape == (100, 32) and not db.any()


@pytest.mark.parametrize("M", [20, 300])
def test_nan_rows_and_targets_past_the_vocabulary(M):
    """A NaN code makes its own row's loss NaN; an ignored row with one, or with a
    NaN dloss, stays out of both gradients; a target past the vocabulary gives NaN."""
    c = Case(M, 400, 64, seed=8, ignored=0.0)
    c.a[3, 5] = 0x7F
    c.targets[3] = -1
    loss, lse = c.forward()
    assert loss[3] == 0 and torch.isnan(lse[3]) and torch.isfinite(loss).all()
    da, db = fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, torch.ones(1, device=DEV), *c.scales)
    assert not da[3].any() and torch.isfinite(da).all() and torch.isfinite(db).all()
    dl = torch.full((M,), 0.25, device=DEV)
    same = fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, dl, *c.scales)
    dl[3] = float("nan")
    odd = fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, dl, *c.scales)
    assert torch.equal(odd[0], same[0]) and torch.equal(odd[1], same[1])
    assert torch.equal(same[0], (0.25 * da.float()).to(torch.bfloat16))  # powers of two leave the roundings alone
    assert torch.equal(same[1], (0.25 * db.float()).to(torch.bfloat16))
    c.targets[3] = 7
    loss, lse = c.forward()
    assert torch.isnan(loss[3]) and int(torch.isnan(loss).sum()) == 1
    c.a[3, 5] = 0
    for bad in (400, 1 << 40):
        c.targets[3] = bad
        loss, lse = c.forward()
        assert torch.isnan(loss[3]) and int(torch.isnan(loss).sum()) == 1 and torch.isfinite(lse).all()
        da, _ = fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, torch.ones(1, device=DEV), *c.scales)
        assert torch.isnan(da[3]).all() and int(torch.isnan(da).any(1).sum()) == 1


def test_one_gradient_alone_and_padded_outputs():
    c = Case(130, 500, 96, seed=4)
    _, lse = c.forward()
    dl = torch.ones(1, device=DEV)
    both = fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, dl, *c.scales)
    assert fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, dl, *c.scales, need_db=False)[1] is None
    assert torch.equal(fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, dl, *c.scales, need_db=False)[0], both[0])
    assert torch.equal(fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, dl, *c.scales, need_da=False)[1], both[1])
    for rows, k in ((130, 0), (500, 1)):
        buf = torch.full((rows + 2, 96 + 5), 9.0, dtype=torch.bfloat16, device=DEV)
        view = buf[1:-1, 3:99]
        fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, dl, *c.scales, **{("da", "db")[k]: view})
        assert torch.equal(view, both[k])
        view.fill_(9)
        assert (buf == 9).all()


def test_captured_on_a_stream_and_the_same_every_time():
    c = Case(300, 5000, 128, seed=6)
    mean, dl = torch.empty(2, device=DEV), torch.ones(1, device=DEV)
    loss, lse = c.forward(mean_out=mean)
    want = [t.clone() for t in (loss, lse, mean, *fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, dl, *c.scales))]
    da, db = torch.empty_like(want[3]), torch.empty_like(want[4])
    ws = [torch.empty(f(300, 5000, 128), dtype=torch.uint8, device=DEV)
          for f in (fp8mi.fp8_cross_entropy_workspace_bytes, fp8mi.fp8_cross_entropy_grad_workspace_bytes)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward(loss=loss, lse=lse, mean_out=mean, workspace=ws[0])
        fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, dl, *c.scales, da=da, db=db, workspace=ws[1])
    for _ in range(3):
        for t in (loss, lse, mean, da, db):
            t.fill_(float("nan"))
        for w in ws:
            w.fill_(0xFF)  # NaN in every type that the workspace holds
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((loss, lse, mean, da, db), want):
            assert torch.equal(got, w)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e6, 1e30])
def test_dloss_of_any_size(size):
    """One dloss, and rows a factor of 10^4 apart: each of da's rows has its own
    precision, db that of its largest terms."""
    c = Case(100, 300, 64, seed=14, ignored=0.1)
    _, lse = c.forward()
    for d in (torch.full((1,), size, device=DEV), torch.logspace(-4, 0, 100, device=DEV) * size):
        da, db = fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, d, *c.scales)
        c.check_grad(da, db, f64(d), lse)


def test_gradient_against_differences():
    """Along a direction of B's scale: dloss/dsb = sum(db * B) / ... by the chain
    rule, against the loss at two scales."""
    c = Case(64, 300, 128, seed=11, ignored=0.2, spread=1.0)
    _, lse = c.forward()
    dl = torch.ones(1, device=DEV)
    da, db = fp8mi.fp8_cross_entropy_grad(c.a, c.b, c.targets, lse, dl, *c.scales)
    b = R.decode_e4m3(c.codes[1])
    by_grad = (f64(db) * b).sum()
    h = 2.0 ** -6
    losses = []
    for s in (1 - h, 1 + h):
        l = R.logits(*c.codes, c.sa.astype(np.float64), c.sb.astype(np.float64) * s)
        losses.append(R.cross_entropy(l, c.t)[0].sum())
    by_difference = (losses[1] - losses[0]) / (2 * h * float(c.sb[0]))
    # central difference: h^2 / 6 of the third derivative (order of the value itself); bf16: its half step of the terms
    terms = np.abs(f64(db) * b).sum()
    assert abs(by_grad - by_difference) <= 4 * h * h * abs(by_difference) + 2 * HALF * terms
