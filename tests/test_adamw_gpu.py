"""fp8_adamw_step and fp8_grad_norm against 64-bit forms (train_ref.py)."""
import numpy as np
import pytest
import torch

import fp8_tensor_scaled_quantize_amd as fp8mi
import train_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 0.0}  # fp32's own rounding is among the bounds
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}        # half an fp16 subnormal step
HP = dict(lr=3e-3, b1=0.9, b2=0.95, eps=1e-8)
DEV = "cuda:0"


def f64(t):
    return t.detach().cpu().double().numpy()


def view(n, dtype, rng, sigma, offset=0, positive=False):
    """A flat device tensor of n values that starts `offset` elements into its storage."""
    x = torch.from_numpy(rng.standard_normal(n + offset) * sigma)
    return (x.abs() if positive else x).to(dtype).to(DEV)[offset:]


class Case:
    """Tensors of one step, with copies of everything before it."""

    def __init__(self, sizes, pdt="bf16", gdt="bf16", bits=32, master=True, offset=0, seed=0):
        rng = np.random.default_rng(seed)
        torch.manual_seed(seed)  # two cases of one seed are alike
        self.sizes, self.bits = sizes, bits
        self.w = [view(n, torch.float32, rng, 0.05, offset) for n in sizes]
        self.p = [w.to(DT[pdt]) if master or pdt != "f32" else w for w in self.w]
        self.masters = self.w if master else None
        self.g = [view(n, DT[gdt], rng, 10.0 ** rng.uniform(-4, 0), offset) for n in sizes]
        m = [view(n, torch.float32, rng, 1e-2, offset) for n in sizes]
        v = [view(n, torch.float32, rng, 1e-3, offset, positive=True) for n in sizes]
        if bits == 32:
            self.m, self.v, self.ms, self.vs = m, v, None, None
        else:
            self.m, self.v = ([torch.randint(0, 127, (n + offset,), dtype=torch.uint8, device=DEV)[offset:] for n in sizes]
                              for _ in range(2))
            for t in self.m:
                t[::2] |= 128  # negative ones
            self.ms, self.vs = ([torch.rand(-(-n // 256), device=DEV) * 1e-4 + 1e-6 for n in sizes] for _ in range(2))
        self.pdt = pdt

    def old(self):
        """(w, g, m, v) of every tensor in 64 bits."""
        out = []
        for i, n in enumerate(self.sizes):
            w = f64(self.w[i] if self.masters is not None else self.p[i])
            m, v = self.m[i].cpu().numpy(), self.v[i].cpu().numpy()
            if self.bits == 8:
                m = R.decode_e4m3(m) * np.repeat(f64(self.ms[i]), 256)[:n]
                v = (R.decode_e4m3(v) * np.repeat(f64(self.vs[i]), 256)[:n]) ** 2
            out.append((w, f64(self.g[i]), m.astype(np.float64), v.astype(np.float64)))
        return out

    def run(self, t, wd, c=None, seed=0, **kw):
        fp8mi.fp8_adamw_step(self.p, self.g, self.m, self.v, t, lr=kw.pop("lr", HP["lr"]), betas=(HP["b1"], HP["b2"]),
                             eps=HP["eps"], weight_decay=wd, masters=self.masters, exp_avg_scales=self.ms,
                             exp_avg_sq_scales=self.vs, grad_scale=c, seed=seed, **kw)
        torch.cuda.synchronize()

    def check(self, old, t, wd, c=1.0, seed=0):
        for i, (w0, g0, m0, v0) in enumerate(old):
            if not self.sizes[i]:
                continue
            d = wd[i] if isinstance(wd, list) else wd
            w, m, v = R.adamw(w0, g0, m0, v0, t, HP["lr"], HP["b1"], HP["b2"], HP["eps"], d, c)
            ew, em, ev = R.adamw_bounds(w0, g0, m0, v0, t, HP["lr"], HP["b1"], HP["b2"], HP["eps"], d, c)
            if self.bits == 8:
                # decoded states carry two more roundings (code times scale, its square), and the update's root and
                # reciprocal are within an ulp instead of half of one
                ew, em, ev = 1.5 * ew, 1.5 * em, 1.5 * ev
            if self.masters is not None:
                assert (np.abs(f64(self.w[i]) - w) <= ew).all(), i
            p = f64(self.p[i])
            assert (np.abs(p - w) <= ew + HALF[self.pdt] * (np.abs(w) + ew) + TINY[self.pdt]).all(), i
            if self.bits == 32:
                assert (np.abs(f64(self.m[i]) - m) <= em).all() and (np.abs(f64(self.v[i]) - v) <= ev).all(), i
            else:
                self.check_codes(i, m, v, em, ev, t, seed)

    def check_codes(self, i, m, v, em, ev, t, seed):
        n = self.sizes[i]
        um, uv = R.uniforms(n, seed, t, i)
        r = np.sqrt(v)
        # m may be off by em (its terms can cancel), r by half of v's relative error and its root's ulp: the largest of a
        # block is off by at most the largest of those, and two roundings (1 / 448 and the product) more
        er = r * (ev / np.maximum(v, 1e-300) / 2 + 2 * R.U32)
        for x, ex, codes, scales, u, root in ((m, em, self.m[i], self.ms[i], um, False), (r, er, self.v[i], self.vs[i], uv, True)):
            s, per = R.block_scales(x)
            es, eper = R.block_scales(ex)
            assert (np.abs(f64(scales) - s) <= es + 3 * R.U32 * s).all()
            # and y = |x| / s by both, and two roundings of the division
            off = (ex + np.abs(x) * eper / per) / per + 4 * R.U32 * 448
            got = R.decode_e4m3(codes.cpu().numpy())
            y = np.minimum(np.abs(x) / per, 448.0)
            k, f, step = R.grid(y)
            # always the grid point below or above (the next finer step lies below a power of two)
            assert (np.abs(np.abs(got) - y) <= step + off).all(), i
            up = (u * (2 * k + 1) < f * (2 * k + f)) | ((k == 0) & (f > 0)) if root else u < f
            same = np.abs(got) == (k + up) * step
            # a code falls the other way where u is nearer to f than f is off: the expected number of them is the sum of
            # off / step, and u's own step 2^-16 makes a few more possible
            assert (~same).sum() <= 3 + 4 * np.minimum(off / step, 1).sum(), (i, (~same).sum())
            if root:
                assert (got[x > 0] > 0).all()
            else:
                assert (np.sign(got) * np.sign(x) >= 0).all()


SIZES = [1536, 1, 0, 255, 256, 257, 4096, 4097, 12345, 100003, 3]


@pytest.mark.parametrize("master", [True, False])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("offset", [0, 1])
def test_step(pdt, gdt, bits, master, offset):
    if master and pdt == "f32":
        master = False
    c = Case(SIZES, pdt, gdt, bits, master, offset, seed=offset)
    old = c.old()
    wd = [0.1 * (i % 2) for i in range(len(SIZES))]
    c.run(7, wd, seed=5)
    c.check(old, 7, wd, seed=5)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_steps_and_scale(bits):
    """Zero states, a scaled gradient, and a second step on what the first left."""
    c = Case([1000, 70000], "bf16", "bf16", bits, True, 0, seed=3)
    for t in c.m + c.v + (c.ms + c.vs if bits == 8 else []):
        t.zero_()
    scale = torch.full((1,), 0.37, device=DEV)
    for t in (1, 2):
        old = c.old()
        c.run(t, 0.01, scale)
        c.check(old, t, 0.01, float(scale))


@pytest.mark.parametrize("gdt", ["bf16", "f32"])
def test_codes_are_those_of_ieee_arithmetic(gdt):
    """Each code and scale is the formula's in fp32, bit for bit (a code that fell
    the other way now and then would make runs of other builds drift apart).
    Values below 2^-6 of a code step's grid (2^-15 of a block's largest) are left
    out: there the sum of the rounding's number and the value is rounded once more."""
    c = Case([300000, 777], "bf16", gdt, 8, True, 0, seed=21)
    before = [[t.cpu().numpy().copy() for t in ts] for ts in (c.m, c.ms, c.v, c.vs, [x.float() for x in c.g])]
    scale = torch.full((1,), 0.61, device=DEV)
    c.run(12, 0.1, scale, seed=31)
    for i in range(2):
        m, ms, v, vs, g = (b[i] for b in before)
        wm, wms, wr, wvs = R.adamw8_fp32(m, ms, v, vs, g, 31, 12, i, HP["b1"], HP["b2"], float(scale))
        assert (c.ms[i].cpu().numpy() == wms).all() and (c.vs[i].cpu().numpy() == wvs).all()
        assert (R.decode_e4m3(c.v[i].cpu().numpy()) == wr).all()
        normal = np.abs(wm) > 2.0 ** -6
        got = R.decode_e4m3(c.m[i].cpu().numpy())
        assert (got == wm)[normal].all() and (got != wm).sum() <= 1


def test_more_tensors_than_a_launch_holds():
    for bits in (32, 8):
        c = Case([100 + i for i in range(130)], "bf16", "f32", bits, True, 0, seed=9)
        old = c.old()
        c.run(2, 0.0, seed=77)
        c.check(old, 2, 0.0, seed=77)


def test_mixed_states_and_types():
    """32- and 8-bit states, masters and none, in one call."""
    a, b = Case([5000, 300], "bf16", "bf16", 32, True, 0, 1), Case([3000, 70], "f16", "f32", 8, False, 1, 2)
    oa, ob = a.old(), b.old()
    fp8mi.fp8_adamw_step(a.p + b.p, a.g + b.g, a.m + b.m, a.v + b.v, 3, lr=HP["lr"], betas=(HP["b1"], HP["b2"]),
                         eps=HP["eps"], weight_decay=0.0, masters=a.masters + [None, None],
                         exp_avg_scales=[None, None] + b.ms, exp_avg_sq_scales=[None, None] + b.vs, seed=4)
    a.check(oa, 3, 0.0)
    got = [R.decode_e4m3(t.cpu().numpy()) for t in b.m]  # (the rounding's numbers go by the place in the list: 2, 3)
    for i, (w0, g0, m0, v0) in enumerate(ob):
        w, m, v = R.adamw(w0, g0, m0, v0, 3, HP["lr"], HP["b1"], HP["b2"], HP["eps"], 0.0)
        s, per = R.block_scales(m)
        um, _ = R.uniforms(len(m), 4, 3, 2 + i)
        k, f, step = R.grid(np.minimum(np.abs(m) / per, 448.0))
        assert (np.abs(got[i]) != (k + (um < f)) * step).sum() <= 3


def test_zero_blocks_and_masked_gradients():
    """Blocks of zeros stay zero; without a gradient v never becomes zero before m
    does, so the update stays small."""
    n = 1024
    c = Case([n], "f32", "f32", 8, False, 0, 0)
    for t in c.m + c.v + c.ms + c.vs:
        t.zero_()
    c.g[0][512:].zero_()
    c.g[0][:512] *= torch.logspace(-9, 0, 512, device=DEV)
    c.run(1, 0.0)
    assert not c.m[0][512:].any() and not c.v[0][512:].any() and not c.ms[0][2:].any() and not c.vs[0][2:].any()
    c.g[0].zero_()
    for t in range(2, 40):
        w = c.p[0].clone()
        c.run(t, 0.0)
        # |m| <= (1 - b1) |g| b1^t' and sqrt(v) >= its rounding down to half: a few lr at most
        assert (c.p[0] - w).abs().max() <= 8 * HP["lr"]
        assert torch.isfinite(c.p[0]).all()


def test_eight_bit_average_does_not_stand_still():
    """A constant squared gradient: v's mean over many elements follows 1 - b2^t,
    though each step changes v by less than half a code step.  Per element the
    rounding leaves a spread of at most half of v, so the mean over 2^16 elements
    is within 0.5 / 2^8 = 0.2 per cent of it at one sigma: 1 per cent is allowed."""
    n, b2 = 1 << 16, 0.999
    p, g = torch.zeros(n, device=DEV), torch.ones(n, device=DEV)
    g[::2] = -1
    g[::256] = 3.0  # the blocks' largest: the others' codes lie inside the range
    m, v = torch.zeros(n, dtype=torch.uint8, device=DEV), torch.zeros(n, dtype=torch.uint8, device=DEV)
    ms, vs = torch.zeros(n // 256, device=DEV), torch.zeros(n // 256, device=DEV)
    for t in range(1, 301):
        fp8mi.fp8_adamw_step([p], [g], [m], [v], t, lr=0.0, betas=(0.9, b2), exp_avg_scales=[ms], exp_avg_sq_scales=[vs])
    got = (R.decode_e4m3(v.cpu().numpy()) * np.repeat(f64(vs), 256)) ** 2
    inner = np.arange(n) % 256 != 0
    assert abs(got[inner].mean() / (1 - b2 ** 300) - 1) <= 0.01
    gm = R.decode_e4m3(m.cpu().numpy()) * np.repeat(f64(ms), 256) * np.sign(f64(g))
    assert abs(gm[inner].mean() - 1) <= 0.01


def test_non_finite_scale_skips_the_step():
    for bits in (32, 8):
        for bad in (float("nan"), float("inf"), -float("inf")):
            c = Case([3000], "bf16", "bf16", bits, True, 0, 1)
            kept = [t.clone() for t in c.p + c.w + c.m + c.v + (c.ms + c.vs if bits == 8 else [])]
            words = torch.tensor([4, 0, 0, 0], dtype=torch.int32, device=DEV)
            c.run(words, 0.1, torch.full((1,), bad, device=DEV))
            c.run(5, 0.1, torch.full((1,), bad, device=DEV))
            now = c.p + c.w + c.m + c.v + (c.ms + c.vs if bits == 8 else [])
            assert all(torch.equal(a, b) for a, b in zip(kept, now)) and int(words[0]) == 4


@pytest.mark.parametrize("bits", [32, 8])
def test_non_finite_gradients_stay_in_their_block(bits):
    c, d = (Case([1024], "f32", "f32", bits, False, 0, 1) for _ in range(2))
    c.g[0][300], c.g[0][301] = float("nan"), float("inf")
    d.g[0].copy_(c.g[0])
    d.g[0][300:302] = 0
    c.run(3, 0.0)
    d.run(3, 0.0)
    other = torch.arange(1024, device=DEV) // 256 != 1
    for a, b in zip((c.p[0], c.m[0], c.v[0]), (d.p[0], d.m[0], d.v[0])):
        assert torch.equal(a[other], b[other])
    assert torch.isnan(c.p[0][300]) and torch.isfinite(c.p[0][:300]).all() and torch.isfinite(c.p[0][302:]).all()
    if bits == 8:
        assert not torch.isfinite(c.ms[0][1]) and not torch.isfinite(c.vs[0][1])


@pytest.mark.parametrize("bits", [32, 8])
def test_device_step_in_a_graph(bits):
    """Captured once, replayed: the step counts itself, lr and the clip are read
    anew, and every replay gives what eager calls with host numbers give."""
    a, b = (Case([5000, 77], "bf16", "bf16", bits, True, 0, 4) for _ in range(2))
    words = torch.zeros(fp8mi.ADAMW_STEP_WORDS, dtype=torch.int32, device=DEV)
    lr, clip = torch.full((1,), HP["lr"], device=DEV), torch.ones(1, device=DEV)
    kept = [t.clone() for t in a.p + a.w + a.m + a.v + (a.ms + a.vs if bits == 8 else [])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.run(words, 0.1, clip, lr=lr)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8mi.fp8_adamw_step(a.p, a.g, a.m, a.v, words, lr=lr, betas=(HP["b1"], HP["b2"]), eps=HP["eps"], weight_decay=0.1,
                             masters=a.masters, exp_avg_scales=a.ms, exp_avg_sq_scales=a.vs, grad_scale=clip)
    for t, k in zip(a.p + a.w + a.m + a.v + (a.ms + a.vs if bits == 8 else []), kept):
        t.copy_(k)
    words.zero_()
    for t in range(1, 5):
        lr.fill_(HP["lr"] * t)
        clip.fill_(0.5 if t % 2 else 2.0)
        graph.replay()
        torch.cuda.synchronize()
        assert int(words[0]) == t
        # the device takes lr as the fp32 word holds it
        b.run(t, 0.1, clip, lr=float(lr))
        for x, y in zip(a.p + a.w + a.m + a.v, b.p + b.w + b.m + b.v):
            if bits == 32:
                torch.testing.assert_close(x, y, rtol=1e-6 if x.dtype == torch.float32 else 2.0 ** -7, atol=1e-9)
            else:
                assert (x.float() - y.float()).abs().mean() < 1e-2
        if bits == 32:
            assert torch.equal(a.m[0], b.m[0]) and torch.equal(a.v[0], b.v[0])


def test_same_every_time_and_on_another_stream():
    cases = [Case([70001, 300], "bf16", "bf16", 8, True, 0, 6) for _ in range(2)]
    cases[0].run(3, 0.1, seed=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cases[1].run(3, 0.1, seed=9)
    s.synchronize()
    a, b = cases
    assert all(torch.equal(x, y) for x, y in zip(a.p + a.w + a.m + a.v + a.ms + a.vs, b.p + b.w + b.m + b.v + b.ms + b.vs))


def test_autograd_sees_the_change():
    p = torch.nn.Parameter(torch.ones(10, device=DEV))
    before = p._version
    fp8mi.fp8_adamw_step([p], [torch.ones(10, device=DEV)], [torch.zeros(10, device=DEV)], [torch.zeros(10, device=DEV)], 1)
    assert p._version > before


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [4096], [4097, 1, 255], [100003] * 3, [1000 + i for i in range(300)], [5000011]])
def test_norm(dt, sizes):
    rng = np.random.default_rng(1)
    g = [view(n, DT[dt], rng, 0.1, offset=1) for n in sizes]
    clip = torch.empty(1, device=DEV)
    exact = np.sqrt(sum((f64(t) ** 2).sum() for t in g))
    norm = fp8mi.fp8_grad_norm(g, 0.5, clip_out=clip)
    # fp64 sums: one fp32 rounding of the norm; the clip's sum and quotient two more
    assert abs(float(norm) - exact) <= 1.01 * U(exact)
    assert abs(float(clip) - min(1.0, 0.5 / (exact + 1e-6))) <= 4 * U(min(1.0, 0.5 / (exact + 1e-6)))


def U(x):
    return R.U32 * abs(x)


def test_norm_beyond_fp32_squares_and_not_finite():
    clip = torch.empty(1, device=DEV)
    big = torch.full((1000,), 1e30, device=DEV)
    assert abs(float(fp8mi.fp8_grad_norm([big], 1.0, clip_out=clip)) / (1e30 * np.sqrt(1000)) - 1) < 1e-6 and float(clip) > 0
    tiny = torch.full((1000,), 1e-30, device=DEV)
    assert abs(float(fp8mi.fp8_grad_norm([tiny], 1.0, clip_out=clip)) / (1e-30 * np.sqrt(1000)) - 1) < 1e-6 and float(clip) == 1
    for bad in (float("nan"), float("inf")):
        big[7] = bad
        fp8mi.fp8_grad_norm([tiny, big], 1.0, clip_out=clip)
        assert torch.isnan(clip).all()
    assert float(fp8mi.fp8_grad_norm([], 1.0, out=torch.empty(1, device=DEV), clip_out=clip)) == 0 and float(clip) == 1


def test_norm_without_a_limit_and_in_a_graph():
    rng = np.random.default_rng(2)
    g = [view(n, torch.bfloat16, rng, 1.0) for n in (5000, 70000, 3)]
    out, clip = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    ws = torch.empty(4096, dtype=torch.uint8, device=DEV)
    fp8mi.fp8_grad_norm(g, out=out, clip_out=clip, workspace=ws)
    assert float(clip) == 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8mi.fp8_grad_norm(g, 2.0, out=out, clip_out=clip, workspace=ws)
    for k in range(3):
        g[1].mul_(1.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), clip.clone()
        assert torch.equal(got[0], fp8mi.fp8_grad_norm(g, 2.0, clip_out=clip)) and torch.equal(got[1], clip)


def test_more_elements_than_a_grid_holds():
    """Five tensors of 2^31 elements: four to a launch.  All weights go from 0 to -lr, a power of two, which bf16 holds
    (fp32's few roundings are far below its half step), and every code of m and sqrt(v) is its block's largest."""
    n, lr = 1 << 31, 2.0 ** -9
    params = [torch.zeros(n, dtype=torch.bfloat16, device=DEV) for _ in range(5)]
    m, v = ([torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(5)] for _ in range(2))
    ms, vs = ([torch.zeros(n // 256, device=DEV) for _ in range(5)] for _ in range(2))
    grad = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    fp8mi.fp8_adamw_step(params, [grad] * 5, m, v, 1, lr, (0.9, 0.95), 1e-8, 0.0, None, ms, vs)
    for t, want in (*((p, -lr) for p in params), *((c, 0x7E) for c in (*m, *v))):
        lo, hi = torch.aminmax(t)
        assert lo == want and hi == want
    norm = fp8mi.fp8_grad_norm([grad] * 5)
    assert abs(float(norm) - (5 * n) ** 0.5) <= 2.0 ** -23 * (5 * n) ** 0.5
