"""fp8_mm_act against its formula in 64 bits: every tile of the dispatch, plain
and gated activations, residual and bias types, per-row scales, both outputs,
pre-activations, ragged and strided operands."""
import numpy as np
import pytest
import torch

import oracle as O
from tests import block_ref as R
from tests.gpu_util import DEV, ring_from_oracle, ring_state_words

pytestmark = pytest.mark.gpu
fp8mi = pytest.importorskip("fp8_tensor_scaled_quantize_amd")

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = R.F32_ULP
TAB = torch.from_numpy(O.decode_table(O.E4M3))


def codes(rows, cols, seed):
    """Random finite E4M3 codes, mid-range exponents."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, cols, generator=g) * 8
    return torch.from_numpy(O.encode(v.numpy(), O.E4M3))


def p_of(t, act):
    """p and the slope factor q' of silu / gelu, and |q|."""
    q = t if act == "silu" else 2 * R.GELU_C * (t + R.GELU_A * t ** 3)
    return torch.sigmoid(q), q.abs()


def act_slack(t, e, act):
    """Bound on the fp32 activation's error for an argument within e of t."""
    v, slope = R.act(t, act)
    if act in ("none", "relu"):
        return e
    p, q = p_of(t, act)
    own = v.abs() * ((1 - p) * (q + 2) * U + 4 * U)
    return 1.13 * e + own + 1e-37  # both slopes are at most 1.13


def reference(a, b, sa, sb, bias, act, gated, res, rows):
    """t, y and bounds on their fp32 errors, for the given rows."""
    A, B = TAB[a[rows].long()], TAB[b.long()]
    s = sa.double().reshape(-1, 1) if sa.numel() == 1 else sa.double()[rows].reshape(-1, 1)
    w = s * sb.double().reshape(1, -1)
    t = (A @ B.t()) * w
    e = 1e-5 * (A.abs() @ B.abs().t()) * w.abs()
    if bias is not None:
        t = t + bias.double()
    e = e + 3 * U * t.abs() + 1e-40
    if gated:
        g, u, eg, eu = t[:, 0::2], t[:, 1::2], e[:, 0::2], e[:, 1::2]
        v, ev = R.act(g, act)[0], act_slack(g, eg, act)
        y, ey = v * u, ev * u.abs() + (v.abs() + ev) * eu + 2 * U * (v * u).abs()
    else:
        y, ey = R.act(t, act)[0], act_slack(t, e, act)
    if res is not None:
        y = y + res[rows].double()
        ey = ey + U * y.abs()
    return t, y, e, ey


def run(M, N, K, act="none", gated=False, out_fmt=None, res_dt=None, bias_dt=None, keep_z=False, row_scales=False, pad=0,
        shift=0, ring=False, rows=None, tag="", a=None, b=None, inplace=False):
    No = N // 2 if gated else N
    a = codes(M, K, 1) if a is None else a
    b = codes(N, K, 2) if b is None else b
    sa, sb = torch.tensor([0.03]), torch.tensor([0.9 / max(1, K) ** 0.5 / 8])
    if row_scales:
        sa, sb = sa * (0.5 + torch.rand(M, generator=torch.Generator().manual_seed(3))), sb * (
            0.5 + torch.rand(N, generator=torch.Generator().manual_seed(4)))
    bias = None if bias_dt is None else R.rand((N,), 0.5, bias_dt, 5)
    res = None if res_dt is None else R.rand((M, No), 1.0, res_dt, 6)
    ad, bd = R.place(a, K + 16 * pad, 16 * shift), R.place(b, K + 32 * pad, 16 * shift)
    odt = torch.uint8 if out_fmt is not None else BF
    fill = 0xA5 if out_fmt is not None else 5.0
    out = R.place(torch.zeros(M, No, dtype=odt), No + pad, shift, fill)
    resd = None if res is None else R.place(res, No + 3 * pad, shift)
    if inplace:
        out = resd
    z = R.place(torch.zeros(M, N, dtype=BF), N + pad, shift, 5.0) if keep_z else None
    ring0 = O.Ring.new(4, 30.0)
    ring0.hist[0], ring0.idx = 2.0, 1
    rg = ring_from_oracle(ring0) if ring else None
    sinv, amax = torch.full((1,), -1.0, device=DEV), torch.full((1,), -1.0, device=DEV)
    kw = {}
    if out_fmt is not None:
        kw = dict(out_fmt=out_fmt, out_scale=None if ring else torch.tensor([30.0], device=DEV), out_ring=rg,
                  out_scale_inv=sinv, out_amax=amax)
    print(f"mm_act {M}x{N}x{K} {act} gated={gated} out={out_fmt} {tag}", flush=True)
    got = fp8mi.fp8_mm_act(ad, bd, sa.to(DEV), sb.to(DEV), None if bias is None else bias.to(DEV), act, gated, resd, z,
                           out, **kw)
    torch.cuda.synchronize()
    rows = torch.arange(M) if rows is None else rows
    t, y, e, ey = reference(a, b, sa, sb, bias, act, gated, res, rows)
    if keep_z:
        R.assert_close(z[rows.to(DEV)], t, e + R.half_ulp(t.abs() + e, BF), f"{tag} z")
        assert R.around_untouched(z, 5.0), "wrote outside z"
    if not inplace:
        assert R.around_untouched(out, fill), "wrote outside the output"
    if out_fmt is None:
        R.assert_close(got[rows.to(DEV)], y, ey + R.half_ulp(y.abs() + ey, BF), f"{tag} y")
    else:
        R.assert_codes(got[rows.to(DEV)], y * 30.0, 0, 30.0 * (ey + U * y.abs()) + 1e-40, f"{tag} codes")
        assert float(sinv) == float(np.float32(1) / np.float32(30))
        if len(rows) == M:
            m = y.abs().max().reshape(1)
            R.assert_close(amax.cpu(), m, ey.max().reshape(1), f"{tag} amax")
        if ring:
            assert np.array_equal(ring_state_words(rg), O.fold(ring0, np.float32(float(amax)), O.E4M3).words())


SMALL = [(1, 2, 16), (1, 16, 16), (3, 18, 48), (64, 64, 256), (65, 130, 272), (1, 1536, 6912), (17, 500, 4096),
         (64, 512, 1024), (200, 2050, 512), (520, 1030, 272), (129, 4098, 800)]


@pytest.mark.parametrize("M,N,K", SMALL)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out_fmt", [None, 0])
def test_shapes(M, N, K, gated, out_fmt):
    act = ["silu", "gelu", "relu", "none"][(M + N // 2 + K // 16) % 4]
    run(M, N, K, act, gated, out_fmt, res_dt=[None, BF, F32, F16][(M + K // 16) % 4], bias_dt=[BF, F32, F16][M % 3],
        keep_z=True, row_scales=True, ring=M % 2 == 0, tag="shapes")


@pytest.mark.parametrize("M,N,K", [(17, 512, 2048), (40, 516, 1040), (64, 1008, 528), (33, 30, 6912), (130, 250, 528),
                                   (250, 256, 1024), (4001, 10, 272)])
@pytest.mark.parametrize("gated,out_fmt", [(False, None), (True, 0), (False, 0)])
def test_row_blocks(M, N, K, gated, out_fmt):
    """16 x 16 blocks, a workgroup each: few rows and columns, ragged edges."""
    run(M, N, K, "silu", gated, out_fmt, res_dt=BF, bias_dt=F32, keep_z=True, row_scales=True, ring=M % 2 == 0, tag="blocks")


# the big tiles of the dispatch: 256 x 192, 256 x 256, the mixed grid; ragged edges
BIG = [(4096, 2560, 272), (4090, 3586, 288), (8190, 6910, 272)]


@pytest.mark.parametrize("M,N,K", BIG)
@pytest.mark.parametrize("gated,out_fmt", [(False, None), (True, None), (False, 0), (True, 0)])
def test_big_tiles(M, N, K, gated, out_fmt):
    rows = torch.cat([torch.arange(0, M, 331), torch.arange(M - 3, M)])
    run(M, N, K, "gelu", gated, out_fmt, res_dt=BF, bias_dt=BF, keep_z=True, rows=rows, tag="big")


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("res_dt", [None, BF, F16, F32])
def test_activations_and_residuals(act, gated, res_dt):
    run(70, 200, 320, act, gated, None, res_dt, F32, tag=f"{res_dt}")
    run(70, 200, 320, act, gated, 0, res_dt, F32, tag=f"{res_dt}")


@pytest.mark.parametrize("M,N,K", [(5, 35, 64), (64, 96, 1040), (300, 1537, 272), (2, 1537, 1024)])
@pytest.mark.parametrize("out_fmt", [None, 0])
def test_strides_and_shifts(M, N, K, out_fmt):
    """Odd widths, padded rows, bases that no vector access is aligned to."""
    for pad, shift in ((0, 0), (1, 1), (3, 5)):
        run(M, N, K, "silu", False, out_fmt, BF, F16, keep_z=True, row_scales=True, pad=pad, shift=shift, tag=f"{pad} {shift}")


@pytest.mark.parametrize("M,N,K", [(33, 257, 512), (1, 256, 2048), (700, 520, 272)])
def test_residual_in_place(M, N, K):
    run(M, N, K, "none", res_dt=BF, bias_dt=BF, inplace=True, tag="in place")


def test_scales_of_one_and_absent():
    """No multipliers, no bias: plain products."""
    a, b = codes(9, 64, 7), codes(20, 64, 8)
    got = fp8mi.fp8_mm_act(a.to(DEV), b.to(DEV))
    torch.cuda.synchronize()
    t, y, e, ey = reference(a, b, torch.ones(1), torch.ones(1), None, "none", False, None, torch.arange(9))
    R.assert_close(got, y, ey + R.half_ulp(y.abs() + ey, BF), "plain")


@pytest.mark.parametrize("M", [2, 300])
def test_nan_infinite_and_saturated(M):
    """NaN codes spoil their rows, an infinite residual saturates the code, and
    the amax leaves NaN out."""
    N, K = 96, 320
    a, b = codes(M, K, 9), codes(N, K, 10)
    a[1, 5] = 0x7F
    res = torch.zeros(M, N, dtype=BF)
    res[0, 3], res[0, 4] = float("inf"), -1e30
    amax, one = torch.empty(1, device=DEV), torch.tensor([1.0], device=DEV)
    sa, sb = torch.tensor([0.01]), torch.tensor([0.01])
    q = fp8mi.fp8_mm_act(a.to(DEV), b.to(DEV), sa.to(DEV), sb.to(DEV), act="relu", residual=res.to(DEV), out_fmt=0,
                         out_scale=one, out_amax=amax)
    y = fp8mi.fp8_mm_act(a.to(DEV), b.to(DEV), sa.to(DEV), sb.to(DEV), act="relu", residual=res.to(DEV))
    torch.cuda.synchronize()
    q, y = q.cpu(), y.cpu()
    assert (q[1] & 0x7F == 0x7F).all() and torch.isnan(y[1].float()).all()
    assert q[0, 3] == 0x7E and q[0, 4] == 0xFE and float(amax) == float("inf")
    assert y[0, 3] == float("inf") and torch.isfinite(y[0, 5:].float()).all()


def test_large_arguments():
    """Pre-activations whose cube and exponential overflow: act(t) = t or 0."""
    a = torch.full((2, 64), 0x7E, dtype=torch.uint8)   # 448
    b = torch.full((32, 64), 0x7E, dtype=torch.uint8)
    a[1] = 0xFE                                       # -448
    for act in ("gelu", "silu"):
        y = fp8mi.fp8_mm_act(a.to(DEV), b.to(DEV), torch.tensor([1e15], device=DEV), torch.tensor([1e10], device=DEV),
                             act=act).cpu().float()
        torch.cuda.synchronize()
        assert (y[0] > 1e31).all() and (y[1] == 0).all(), act


def test_empty():
    ring0 = O.Ring.new(4, 3.0)
    ring = ring_from_oracle(ring0)
    a, b = torch.empty(0, 64, dtype=torch.uint8, device=DEV), torch.zeros(8, 64, dtype=torch.uint8, device=DEV)
    assert fp8mi.fp8_mm_act(a, b, act="gelu").shape == (0, 8)
    amax = torch.full((1,), -1.0, device=DEV)
    fp8mi.fp8_mm_act(b, a, act="gelu", out_fmt=0, out_ring=ring, out_amax=amax)
    # K = 0: t is the bias
    bias = R.rand((6,), 1.0, F32, 1).to(DEV)
    e = torch.empty(4, 0, dtype=torch.uint8, device=DEV)
    y = fp8mi.fp8_mm_act(e, torch.empty(6, 0, dtype=torch.uint8, device=DEV), bias=bias, act="relu")
    torch.cuda.synchronize()
    assert np.array_equal(ring_state_words(ring), O.fold(ring0, np.float32(0), O.E4M3).words()) and float(amax) == 0
    assert torch.equal(y.cpu(), bias.clamp(min=0).to(BF).cpu().expand(4, 6))


def test_equals_fp8_mm_without_activation():
    """No activation, no residual: the plain GEMM's bits."""
    for M, N, K in ((300, 520, 272), (64, 1536, 6912), (2048, 1536, 1536)):
        a, b = codes(M, K, 11).to(DEV), codes(N, K, 12).to(DEV)
        s, bias = torch.tensor([0.02], device=DEV), R.rand((N,), 1.0, BF, 13).to(DEV)
        y = fp8mi.fp8_mm(a, b, 0, 0, s, s, bias)
        z = fp8mi.fp8_mm_act(a, b, s, s, bias)
        torch.cuda.synchronize()
        # few rows may sum K in another order: then within one rounding
        d = (y.float() - z.float()).abs()
        assert (d <= 2.0 ** -7 * y.float().abs() + 1e-5 * K).all()


def test_graph_replays_on_a_side_stream():
    M, N, K = 260, 1536, 512
    a = torch.empty(M, K, dtype=torch.uint8, device=DEV)
    b, s = codes(N, K, 21).to(DEV), torch.tensor([0.02], device=DEV)
    res = R.rand((M, N // 2), 1.0, BF, 22).to(DEV)
    ring, eager = fp8mi.new_ring(8, 10.0, DEV), fp8mi.new_ring(8, 10.0, DEV)
    out = torch.empty(M, N // 2, dtype=torch.uint8, device=DEV)
    z = torch.empty(M, N, dtype=BF, device=DEV)
    amax = torch.empty(1, device=DEV)

    def step(rg):
        fp8mi.fp8_mm_act(a, b, s, s, act="silu", gated=True, residual=res, z_out=z, out=out, out_fmt=0, out_ring=rg,
                         out_amax=amax)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    a.copy_(codes(M, K, 23))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(ring)
    for k in range(4):
        a.copy_(codes(M, K, 24 + k))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, z, amax, ring)]
        with torch.cuda.stream(side):
            step(eager)
        torch.cuda.synchronize()
        for x, y in zip(got, (out, z, amax, eager)):
            assert torch.equal(x, y), f"replay {k}"
