"""fp8_act_grad against its formula in 64 bits and against differences of the
activation."""
import numpy as np
import pytest
import torch

import oracle as O
from tests import block_ref as R
from tests.gpu_util import DEV, ring_from_oracle, ring_state_words

pytestmark = pytest.mark.gpu
fp8mi = pytest.importorskip("fp8_tensor_scaled_quantize_amd")

BF, F16 = torch.bfloat16, torch.float16
U = R.F32_ULP


def slope_slack(t, act):
    """Bound on the fp32 slope's error: p is within (1 - p)(|q| + 2) u + 2 u of
    exact (relative), 1 - p inherits that, 6 roundings join the terms."""
    if act in ("relu", "none"):
        return torch.zeros_like(t)
    q = t if act == "silu" else 2 * R.GELU_C * (t + R.GELU_A * t ** 3)
    dq = torch.ones_like(t) if act == "silu" else 2 * R.GELU_C * (1 + 3 * R.GELU_A * t * t)
    p = torch.sigmoid(q)
    ep = (1 - p) * (q.abs() + 2) * U + 2 * U
    tq = t.abs() * dq
    return p * ep + tq * p * (ep + 2 * U) + 6 * U * (p + tq * p * (1 - p)) + 1e-37


def value_slack(t, act):
    if act in ("relu", "none"):
        return torch.zeros_like(t)
    q = t if act == "silu" else 2 * R.GELU_C * (t + R.GELU_A * t ** 3)
    p = torch.sigmoid(q)
    return (t * p).abs() * ((1 - p) * (q.abs() + 2) * U + 4 * U) + 1e-37


def reference(dy, z, act, gated):
    dy, z = dy.double(), z.double()
    if not gated:
        sl = R.act(z, act)[1]
        return dy * sl, dy.abs() * (slope_slack(z, act) + U * sl.abs())
    g, u = z[:, 0::2], z[:, 1::2]
    v, sl = R.act(g, act)
    dz = torch.stack([dy * u * sl, dy * v], dim=2).flatten(1)
    e = torch.stack([(dy * u).abs() * (slope_slack(g, act) + 2 * U * sl.abs()),
                     dy.abs() * (value_slack(g, act) + U * v.abs())], dim=2).flatten(1)
    return dz, e


def check(rows, cols, act, gated, fmt, dt=BF, ring=True, bias=True, pad=0, shift=0, dy=None, z=None, tag=""):
    """cols counts dz columns."""
    dy = R.rand((rows, cols // 2 if gated else cols), 1e-3, dt, 1) if dy is None else dy
    z = R.rand((rows, cols), 2.0, BF, 2) if z is None else z
    s0 = O.FMT_MAX[R.FMT_NAME[fmt]] / 5e-3
    ring0 = O.Ring.new(4, s0)
    ring0.hist[:2], ring0.idx = [5e-3, 1e-3], 2
    rg = ring_from_oracle(ring0) if ring else None
    out = R.place(torch.zeros(rows, cols, dtype=torch.uint8), cols + pad, shift, 0xA5)
    out_t = R.place(torch.zeros(cols, rows, dtype=torch.uint8), rows + pad, shift, 0xA5)
    sinv, amax = torch.full((1,), -1.0, device=DEV), torch.full((1,), -1.0, device=DEV)
    print(f"act_grad {rows}x{cols} {act} gated={gated} fmt={fmt} {dt} ring={ring} {tag}", flush=True)
    scale = None if ring else torch.tensor([s0], dtype=torch.float32, device=DEV)
    c, ct, db = fp8mi.fp8_act_grad(R.place(dy, dy.shape[1] + pad, shift), R.place(z, cols + 2 * pad, shift), act, gated,
                                   fmt, out, out_t, scale=scale, ring=rg, scale_inv_out=sinv, amax_out=amax,
                                   need_bias_grad=bias)
    torch.cuda.synchronize()
    dz, e = reference(dy, z, act, gated)
    s = float(np.float32(s0))
    R.assert_codes(c, dz * s, fmt, s * (e + 2 * U * dz.abs()) + 1e-40, f"{tag} codes")
    assert torch.equal(ct.cpu(), c.cpu().t()), f"{tag}: the transposed codes differ"
    assert R.around_untouched(out, 0xA5) and R.around_untouched(out_t, 0xA5), "wrote outside its output"
    fin = dz.abs().nan_to_num(nan=0.0)
    R.assert_close(amax.cpu(), fin.max().reshape(1), e.nan_to_num(nan=0.0, posinf=0.0).max().reshape(1) + 1e-30, f"{tag} amax")
    assert float(sinv) == float(np.float32(1) / np.float32(s))
    if ring:
        assert np.array_equal(ring_state_words(rg), O.fold(ring0, np.float32(float(amax)), R.FMT_NAME[fmt]).words())
    if bias:
        t, mag = dz.sum(0), (e + 2 * U * dz.abs()).sum(0)
        R.assert_close(db, t, mag + R.half_ulp(t.abs() + mag, BF), f"{tag} bias gradient")
    else:
        assert db is None


SHAPES = [(1, 2), (1, 64), (2, 6), (127, 62), (128, 64), (129, 66), (250, 1538), (1000, 1536), (33, 6912), (2050, 130)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_shapes(rows, cols, gated, act):
    check(rows, cols, act, gated, 1, ring=cols % 4 == 0, bias=rows % 2 == 0, tag="shapes")


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,cols,pad,shift", [(70, 200, 0, 0), (131, 130, 3, 1), (128, 128, 8, 8), (40, 66, 1, 3)])
def test_types_and_strides(dt, fmt, gated, rows, cols, pad, shift):
    for ring in (False, True):
        check(rows, cols, "gelu", gated, fmt, dt, ring, True, pad, shift, tag=f"{pad} {shift}")


def test_gated_without_activation():
    check(65, 70, "none", True, 1)


@pytest.mark.parametrize("rows,cols", [(5, 3), (130, 1537), (1, 1)])
def test_odd_widths(rows, cols):
    for act in ("relu", "silu"):
        check(rows, cols, act, False, 1, ring=False, tag="odd")


def test_nan_and_infinite():
    """A NaN or infinite gradient or pre-activation spoils its own element."""
    rows, cols = 140, 72
    dy, z = R.rand((rows, cols), 1e-3, BF, 5), R.rand((rows, cols), 1.0, BF, 6)
    dy[0, 0], z[1, 1], dy[2, 2], z[3, 3], z[3, 4] = float("nan"), float("nan"), float("inf"), float("inf"), float("-inf")
    dy[139, 71] = float("-inf")
    amax = torch.empty(1, device=DEV)
    c, ct, _ = fp8mi.fp8_act_grad(dy.to(DEV), z.to(DEV), "relu", scale=torch.tensor([1e5], device=DEV), amax_out=amax)
    torch.cuda.synchronize()
    c = c.cpu()
    dz = dy.double() * (z.double() > 0)
    got = O.decode_table(O.E5M2)[c.numpy()]
    assert np.array_equal(np.isnan(got), torch.isnan(dz).numpy()) and torch.equal(ct.cpu(), c.t())
    want = float(dz.abs().nan_to_num(nan=0.0, posinf=float("inf")).max())
    assert float(amax) == want
    if z[2, 2] > 0:
        assert got[2, 2] == 57344.0


def test_large_arguments():
    """z whose cube overflows: slope 1 or 0, never NaN."""
    z = torch.tensor([[1e30, -1e30, 3e38, -3e38, 30.0, -30.0, 0.0, 200.0]], dtype=BF)
    dy = torch.full((1, 8), 0.5, dtype=BF)
    for act in ("gelu", "silu"):
        _, _, db = fp8mi.fp8_act_grad(dy.to(DEV), z.to(DEV), act, scale=torch.tensor([1.0], device=DEV),
                                      need_bias_grad=True)
        torch.cuda.synchronize()
        d = db.cpu().float()
        assert torch.equal(d[:4], torch.tensor([0.5, 0.0, 0.5, 0.0])) and d[4] == 0.5 and abs(d[5]) < 1e-10
        assert d[6] == 0.25 and d[7] == 0.5, act


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("gated", [False, True])
def test_against_differences(act, gated):
    """One row: the bias gradient is dz itself, rounded to bf16; compared with
    central differences of L = sum dy y (error ~ step^2, far below 2^-8)."""
    n = 64
    z, dy = R.rand((1, n), 1.5, BF, 8), R.rand((1, n // 2 if gated else n), 1.0, BF, 9)
    _, _, db = fp8mi.fp8_act_grad(dy.to(DEV), z.to(DEV), act, gated, scale=torch.tensor([1.0], device=DEV),
                                  need_bias_grad=True)
    torch.cuda.synchronize()

    def loss(t):
        y = R.act(t[:, 0::2], act)[0] * t[:, 1::2] if gated else R.act(t, act)[0]
        return float((dy.double() * y).sum())

    step = 1e-4
    for j in range(n):
        e = torch.zeros(1, n, dtype=torch.float64)
        e[0, j] = step
        num = (loss(z.double() + e) - loss(z.double() - e)) / (2 * step)
        assert abs(float(db[j]) - num) <= 2.0 ** -8 * abs(num) + 1e-6, j


@pytest.mark.parametrize("rows,cols", [(0, 64), (4, 0)])
def test_empty(rows, cols):
    ring0 = O.Ring.new(4, 3.0)
    ring = ring_from_oracle(ring0)
    e = torch.empty(rows, cols, dtype=BF, device=DEV)
    amax = torch.full((1,), -1.0, device=DEV)
    _, _, db = fp8mi.fp8_act_grad(e, e, "gelu", ring=ring, amax_out=amax, need_bias_grad=True)
    torch.cuda.synchronize()
    assert np.array_equal(ring_state_words(ring), O.fold(ring0, np.float32(0), O.E5M2).words())
    assert float(amax) == 0 and db.shape == (cols,) and (db.cpu() == 0).all()


def test_repeatable():
    rows, cols = 3000, 1536
    dy, z = R.rand((rows, cols), 1e-3, BF, 12).to(DEV), R.rand((rows, cols), 1.0, BF, 13).to(DEV)
    one = torch.tensor([1e6], device=DEV)
    a = fp8mi.fp8_act_grad(dy, z, "silu", scale=one, need_bias_grad=True)
    b = fp8mi.fp8_act_grad(dy, z, "silu", scale=one, need_bias_grad=True)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
