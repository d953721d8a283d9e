"""fp8_rmsnorm and fp8_rmsnorm_grad against their formulas in 64 bits (and the
gradient against differences of the formula)."""
import numpy as np
import pytest
import torch

import oracle as O
from tests import block_ref as R
from tests.gpu_util import DEV, ring_from_oracle, ring_state_words

pytestmark = pytest.mark.gpu
fp8mi = pytest.importorskip("fp8_tensor_scaled_quantize_amd")

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5
# every kernel form: one wave a row (1..6 vectors a lane), four waves, sixteen
SHAPES = [(1, 1), (1, 7), (3, 8), (2, 64), (5, 511), (4, 512), (1, 1535), (1, 4096), (37, 513), (1030, 520),
          (1100, 1535), (1025, 2050), (1024, 2561), (3, 2048), (2, 2049), (3, 6000), (2, 8191), (2, 8193), (3, 16385),
          (1, 32768)]


def forward(x, res, w, fmt, mode, ld=0, shift=0, s_given=None, ring=None, **kw):
    """One call with padded, shifted operands; returns codes, scale_inv, amax, h, rstd."""
    rows, cols = x.shape
    L = cols + ld
    xd = R.place(x, L, shift)
    rd = None if res is None else R.place(res, L + ld, shift)
    wd = None if w is None else R.place(w.reshape(1, -1), None, shift)[0]
    out = R.place(torch.zeros(rows, cols, dtype=torch.uint8), L + ld, shift, 0xA5)
    hs = R.place(torch.zeros_like(x), L, shift, 3.0)
    n = rows if mode == "row" else 1
    sinv, amax = torch.full((n,), -1.0, device=DEV), torch.full((n,), -1.0, device=DEV)
    rstd = torch.full((rows,), -1.0, device=DEV)
    got = fp8mi.fp8_rmsnorm(xd, wd, fmt, EPS, residual=rd, out=out, row_scaled=mode == "row",
                            scale=s_given if mode == "tensor" else None, ring=ring if mode == "ring" else None,
                            scale_inv_out=sinv, amax_out=amax, sum_out=hs, rstd_out=rstd, **kw)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    if rows and cols:
        assert R.around_untouched(out, 0xA5) and R.around_untouched(hs, 3.0), "wrote outside its output"
    return out.cpu(), sinv.cpu(), amax.cpu(), hs.cpu(), rstd.cpu()


def check_forward(x, res, w, fmt, mode, tag, **kw):
    rows, cols = x.shape
    rel = R.rms_rel(cols)
    h, rstd, y = R.rmsnorm(x, res, w, EPS)
    ring0 = O.Ring.new(4, O.FMT_MAX[R.FMT_NAME[fmt]] / 9.0)
    ring0.hist[:2], ring0.idx = [9.0, 2.0], 2
    ring = ring_from_oracle(ring0)
    given = torch.tensor([12.5], device=DEV)
    codes, sinv, amax, hs, rs = forward(x, res, w, fmt, mode, s_given=given, ring=ring, **kw)
    exact_h = x.float() if res is None else x.float() + res.float()
    assert torch.equal(hs.float(), exact_h.to(x.dtype).float()), f"{tag}: h is not x + residual rounded once"
    R.assert_close(rs, rstd.reshape(-1), rel * rstd.reshape(-1), f"{tag} rstd")
    if mode == "row":
        a = y.abs().amax(1)
        R.assert_close(amax, a, rel * a, f"{tag} amax")
        s = R.scale_of(a, fmt)
        R.assert_close(sinv, 1 / s, (rel + 4 * R.F32_ULP) / s, f"{tag} scale_inv")
        R.assert_codes(codes, y * s[:, None], fmt, 2 * rel + 6 * R.F32_ULP, tag)
    else:
        a = y.abs().max().reshape(1)
        s = 12.5 if mode == "tensor" else float(ring0.scale)
        R.assert_close(amax, a, rel * a, f"{tag} amax")
        assert float(sinv) == float(np.float32(1.0) / np.float32(s)), f"{tag}: scale_inv"
        R.assert_codes(codes, y * s, fmt, rel + 2 * R.F32_ULP, tag)
        if mode == "ring":
            want = O.fold(ring0, np.float32(float(amax)), R.FMT_NAME[fmt])
            assert np.array_equal(ring_state_words(ring), want.words()), f"{tag}: ring"


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_shapes(rows, cols):
    """Every kernel form, bf16 with a residual, per-row and per-tensor scales."""
    x, res = R.rand((rows, cols), 2.0, BF, 1), R.rand((rows, cols), 1.0, BF, 2)
    w = R.rand((cols,), 1.0, BF, 3)
    for mode in ("row", "ring"):
        print(f"rmsnorm {rows}x{cols} {mode}", flush=True)
        check_forward(x, res, w, 0, mode, f"{rows}x{cols} {mode}")


@pytest.mark.parametrize("dt", [BF, F16, F32])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("mode", ["row", "tensor", "ring"])
@pytest.mark.parametrize("rows,cols,ld,shift", [(9, 333, 0, 0), (70, 1536, 8, 8), (5, 1537, 3, 1), (3, 3000, 5, 7)])
def test_forward_types_and_strides(dt, fmt, mode, rows, cols, ld, shift):
    print(f"rmsnorm {rows}x{cols} {dt} fmt {fmt} {mode} ld +{ld} shift {shift}", flush=True)
    x = R.rand((rows, cols), 1.0, dt, 10)
    res = R.rand((rows, cols), 0.5, dt, 11) if ld else None
    w = [None, R.rand((cols,), 1.0, F16, 12), R.rand((cols,), 1.0, F32, 13)][(ld + fmt) % 3]
    check_forward(x, res, w, fmt, mode, f"{dt} {fmt} {mode}", ld=ld, shift=shift)


@pytest.mark.parametrize("mode", ["row", "tensor", "ring"])
@pytest.mark.parametrize("cols", [40, 1536, 5000])
def test_zero_nan_and_infinite_rows(mode, cols):
    """A row of zeros gives zeros; a NaN or an infinity spoils its own row only
    (as the formula says) and the amax leaves NaN out."""
    x = R.rand((6, cols), 1.0, BF, 20)
    x[1] = 0.0
    x[2, 3] = float("nan")
    x[3, cols - 1] = float("inf")
    x[4, 0] = float("-inf")
    w = R.rand((cols,), 1.0, BF, 21)
    h, rstd, y = R.rmsnorm(x, None, w, EPS)
    ring = ring_from_oracle(O.Ring.new(4, 20.0))
    codes, sinv, amax, _, rs = forward(x, None, w, 0, mode, s_given=torch.tensor([20.0], device=DEV), ring=ring)
    print(f"rmsnorm specials {mode} {cols}", flush=True)
    rel = R.rms_rel(cols)
    R.assert_close(rs, rstd.reshape(-1), rel * rstd.reshape(-1), "rstd")
    a = torch.nan_to_num(y, nan=0.0).abs().amax(1)
    if mode == "row":
        R.assert_close(amax, a, rel * a, "amax")
        s = R.scale_of(a, 0)
        R.assert_codes(codes, y * s[:, None], 0, 2 * rel + 6 * R.F32_ULP, "codes")
        assert float(sinv[1]) == 1.0
    else:
        R.assert_close(amax, a.max().reshape(1), rel * a.max().reshape(1), "amax")
        R.assert_codes(codes, y * 20.0, 0, rel + 2 * R.F32_ULP, "codes")
    assert (codes[1] & 0x7F == 0).all()


def test_zero_row_without_eps_is_nan():
    """0 / 0: the formula's NaN, not a hidden zero."""
    x = torch.zeros(2, 24, dtype=BF, device=DEV)
    sinv = torch.empty(2, device=DEV)
    codes = fp8mi.fp8_rmsnorm(x, None, fp8mi.E4M3, 0.0, row_scaled=True, scale_inv_out=sinv)
    torch.cuda.synchronize()
    assert (codes.cpu() & 0x7F == 0x7F).all() and (sinv.cpu() == 1.0).all()


@pytest.mark.parametrize("s", [0.0, float("inf"), float("nan")])
def test_irregular_scale(s):
    """An explicit scale of 0, infinity or NaN encodes the products themselves."""
    x = R.rand((3, 72), 1.0, F32, 22)
    x[0, 5] = 0.0
    _, _, y = R.rmsnorm(x, None, None, EPS)
    got = fp8mi.fp8_rmsnorm(x.to(DEV), None, fp8mi.E5M2, EPS, scale=torch.tensor([s], device=DEV))
    torch.cuda.synchronize()
    t = y * s
    fin = t.nan_to_num(nan=float("nan"), posinf=1e9, neginf=-1e9)  # saturates
    R.assert_codes(got, fin, 1, 1e-5, f"scale {s}")


@pytest.mark.parametrize("rows,cols", [(0, 64), (4, 0), (0, 0)])
def test_empty(rows, cols):
    x = torch.empty(rows, cols, dtype=BF, device=DEV)
    ring0 = O.Ring.new(4, 3.0)
    ring0.hist[0], ring0.idx = 2.0, 1
    ring = ring_from_oracle(ring0)
    sinv, amax = torch.full((1,), -1.0, device=DEV), torch.full((1,), -1.0, device=DEV)
    fp8mi.fp8_rmsnorm(x, None, fp8mi.E4M3, EPS, ring=ring, scale_inv_out=sinv, amax_out=amax)
    rowinv = torch.full((rows,), -1.0, device=DEV)
    fp8mi.fp8_rmsnorm(x, None, fp8mi.E4M3, EPS, row_scaled=True, scale_inv_out=rowinv)
    dx, dw = fp8mi.fp8_rmsnorm_grad(x, x, None, torch.ones(rows, device=DEV))
    torch.cuda.synchronize()
    assert np.array_equal(ring_state_words(ring), O.fold(ring0, np.float32(0), O.E4M3).words())
    assert float(amax) == 0.0 and float(sinv) == float(np.float32(1) / np.float32(3))
    assert (rowinv.cpu() == 1.0).all() and dx.shape == (rows, cols) and (dw.cpu() == 0).all()


@pytest.mark.parametrize("rows,cols", [(4, 1536), (1200, 600), (2, 9000)])
def test_residual_stream_in_place(rows, cols):
    """sum_out may be the residual or x itself."""
    x, res = R.rand((rows, cols), 1.0, BF, 30).to(DEV), R.rand((rows, cols), 1.0, BF, 31).to(DEV)
    sinv = torch.empty(rows, device=DEV)
    h = torch.empty_like(x)
    a = fp8mi.fp8_rmsnorm(x, None, fp8mi.E4M3, EPS, residual=res, row_scaled=True, scale_inv_out=sinv, sum_out=h)
    r2, x2 = res.clone(), x.clone()
    b = fp8mi.fp8_rmsnorm(x, None, fp8mi.E4M3, EPS, residual=r2, row_scaled=True, scale_inv_out=sinv, sum_out=r2)
    c = fp8mi.fp8_rmsnorm(x2, None, fp8mi.E4M3, EPS, residual=res, row_scaled=True, scale_inv_out=sinv, sum_out=x2)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(h, r2) and torch.equal(h, x2)


def test_offsets_past_32_bits():
    """Rows whose element offsets (and the codes' byte offsets) pass 2^32."""
    rows, cols, ld = 3, 200, (1 << 31) + 24
    x = R.rand((rows, cols), 1.0, BF, 33)
    buf = torch.empty(2 * ld + cols, dtype=BF, device=DEV)
    xd = torch.as_strided(buf, (rows, cols), (ld, 1))
    xd.copy_(x.to(DEV))
    ob = torch.empty(2 * ld + cols, dtype=torch.uint8, device=DEV)
    out = torch.as_strided(ob, (rows, cols), (ld, 1))
    sinv = torch.empty(rows, device=DEV)
    fp8mi.fp8_rmsnorm(xd, None, fp8mi.E4M3, EPS, out=out, row_scaled=True, scale_inv_out=sinv, sum_out=xd)
    dense = fp8mi.fp8_rmsnorm(x.to(DEV), None, fp8mi.E4M3, EPS, row_scaled=True, scale_inv_out=sinv)
    dx, dw = fp8mi.fp8_rmsnorm_grad(xd, xd, None, sinv, dx=xd)
    dx2, dw2 = fp8mi.fp8_rmsnorm_grad(x.to(DEV), x.to(DEV), None, sinv)
    torch.cuda.synchronize()
    assert torch.equal(out, dense) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def check_grad(rows, cols, dt, w, with_dsum, tag, ld=0, shift=0):
    dy, h = R.rand((rows, cols), 1e-2, dt, 40), R.rand((rows, cols), 2.0, dt, 41)
    h[rows // 2] = 0.0
    dsum = R.rand((rows, cols), 1e-2, dt, 42) if with_dsum else None
    rstd = (1 / torch.sqrt(h.float().square().mean(1) + EPS))
    L = cols + ld
    dxd = R.place(torch.zeros(rows, cols, dtype=dt), L, shift, 7.0)
    dw = torch.full((cols,), -1.0, device=DEV)
    args = (R.place(dy, L, shift), R.place(h, L + ld, shift), None if w is None else w.to(DEV), rstd.to(DEV))
    kw = dict(dsum=None if dsum is None else R.place(dsum, L, shift))
    fp8mi.fp8_rmsnorm_grad(*args, dx=dxd, dweight=dw, **kw)
    dx2, none = fp8mi.fp8_rmsnorm_grad(*args, need_dweight=False, **kw)
    torch.cuda.synchronize()
    assert none is None and torch.equal(dx2, dxd), f"{tag}: dx depends on whether dweight is wanted"
    assert R.around_untouched(dxd, 7.0), f"{tag}: wrote outside dx"
    dx64, dw64, mag, wmag = R.rmsnorm_grad(dy, h, w, rstd, dsum)
    # the row's dot product: 32 + 22 additions; 8 more roundings
    rel = (min(cols, 32) + 30) * R.F32_ULP
    R.assert_close(dxd.cpu(), dx64, R.half_ulp(dx64, dt) + rel * mag, f"{tag} dx")
    # per lane ceil(rows / (512 workgroups)) rows one by one, 8 waves, then fp64; 3 roundings a term
    R.assert_close(dw.cpu(), dw64, (rows / 512 + 14) * R.F32_ULP * wmag, f"{tag} dweight")


@pytest.mark.parametrize("rows,cols", SHAPES + [(2500, 1536), (3000, 130)])
def test_grad_shapes(rows, cols):
    print(f"rmsnorm grad {rows}x{cols}", flush=True)
    check_grad(rows, cols, BF, R.rand((cols,), 1.0, BF, 43), rows % 2 == 0, f"{rows}x{cols}")


@pytest.mark.parametrize("dt", [BF, F16, F32])
@pytest.mark.parametrize("rows,cols,ld,shift", [(9, 333, 0, 0), (70, 1536, 8, 8), (5, 1537, 3, 1), (3, 3000, 5, 7),
                                                (2, 20001, 1, 1)])
def test_grad_types_and_strides(dt, rows, cols, ld, shift):
    print(f"rmsnorm grad {rows}x{cols} {dt} ld +{ld} shift {shift}", flush=True)
    w = [None, R.rand((cols,), 1.0, F16, 44), R.rand((cols,), 1.0, F32, 45)][rows % 3]
    check_grad(rows, cols, dt, w, ld % 2 == 1, f"{dt}", ld, shift)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("size", [1e14, 1e-14])
@pytest.mark.parametrize("cols", [300, 3001, 9000])
def test_grad_of_extreme_rows(dt, size, cols):
    """rstd^3 alone is outside fp32's range; the gradient is not."""
    print(f"rmsnorm grad extreme {dt} {size} {cols}", flush=True)
    dy, h, w = R.rand((3, cols), 1e-2, dt, 53), R.rand((3, cols), size, dt, 54), R.rand((cols,), 1.0, BF, 55)
    rstd = (1 / torch.sqrt(h.double().square().mean(1))).float()
    dx, dw = fp8mi.fp8_rmsnorm_grad(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV))
    torch.cuda.synchronize()
    dx64, dw64, mag, wmag = R.rmsnorm_grad(dy, h, w, rstd, None)
    rel = (min(cols, 32) + 30) * R.F32_ULP  # as check_grad
    R.assert_close(dx.cpu(), dx64, R.half_ulp(dx64, dt) + rel * mag, "dx")
    R.assert_close(dw.cpu(), dw64, 14 * R.F32_ULP * wmag, "dweight")


def test_grad_in_place_and_repeatable():
    rows, cols = 2300, 1535
    dy, h = R.rand((rows, cols), 1.0, BF, 46).to(DEV), R.rand((rows, cols), 1.0, BF, 47).to(DEV)
    ds, rstd = R.rand((rows, cols), 1.0, BF, 48).to(DEV), torch.rand(rows, device=DEV) + 0.5
    a, wa = fp8mi.fp8_rmsnorm_grad(dy, h, None, rstd, dsum=ds)
    d2, s2 = dy.clone(), ds.clone()
    b, wb = fp8mi.fp8_rmsnorm_grad(dy, h, None, rstd, dsum=s2, dx=s2)
    c, wc = fp8mi.fp8_rmsnorm_grad(d2, h, None, rstd, dsum=ds, dx=d2)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(wa, wb) and torch.equal(wa, wc)


@pytest.mark.parametrize("rows,cols", [(3, 5), (4, 130), (2, 1030)])
def test_grad_against_differences(rows, cols):
    """dx and dweight against central differences of L = sum dy * y in 64 bits."""
    x, w = R.rand((rows, cols), 1.0, F32, 50), R.rand((cols,), 1.0, F32, 51)
    dy = R.rand((rows, cols), 1.0, F32, 52)
    _, rstd, _ = R.rmsnorm(x, None, w, EPS)
    dx, dw = fp8mi.fp8_rmsnorm_grad(dy.to(DEV), x.to(DEV), w.to(DEV), rstd.reshape(-1).float().to(DEV))
    torch.cuda.synchronize()

    def loss(xx, ww):
        return float((dy.double() * R.rmsnorm(xx, None, ww, EPS)[2]).sum())

    step = 1e-5  # difference error ~ step^2 |f'''| and 1e-16 L / step: both below 1e-8 here
    for i, j in ((0, 0), (rows - 1, cols - 1), (rows // 2, cols // 2)):
        e = torch.zeros(rows, cols, dtype=torch.float64)
        e[i, j] = step
        num = (loss(x.double() + e, w.double()) - loss(x.double() - e, w.double())) / (2 * step)
        assert abs(float(dx[i, j]) - num) <= 1e-5 * (1 + abs(num)), (i, j)
        ew = torch.zeros(cols, dtype=torch.float64)
        ew[j] = step
        num = (loss(x.double(), w.double() + ew) - loss(x.double(), w.double() - ew)) / (2 * step)
        assert abs(float(dw[j]) - num) <= 1e-5 * (1 + abs(num)), j


def test_other_stream_and_graph_replays():
    """Work on a side stream, captured with its ring; every replay (with eager
    work between) equals an eager step from the same ring."""
    rows, cols = 300, 1536
    x = torch.empty(rows, cols, dtype=BF, device=DEV)
    res = R.rand((rows, cols), 1.0, BF, 61).to(DEV)
    w = R.rand((cols,), 1.0, BF, 62).to(DEV)
    ring, eager = (fp8mi.new_ring(8, 10.0, DEV) for _ in range(2))
    out, h = torch.empty(rows, cols, dtype=torch.uint8, device=DEV), torch.empty_like(x)
    rstd, dx, dw = torch.empty(rows, device=DEV), torch.empty_like(x), torch.empty(cols, device=DEV)
    ws = torch.empty(fp8mi.fp8_rmsnorm_grad_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)

    def step(rg):
        fp8mi.fp8_rmsnorm(x, w, fp8mi.E4M3, EPS, residual=res, out=out, ring=rg, sum_out=h, rstd_out=rstd)
        fp8mi.fp8_rmsnorm_grad(h, h, w, rstd, dx=dx, dweight=dw, workspace=ws)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    x.copy_(R.rand((rows, cols), 1.0, BF, 63))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(ring)
    for k in range(4):
        x.copy_(R.rand((rows, cols), 1.0 + k, BF, 64 + k))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, h, rstd, dx, dw, ring)]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(eager)
        torch.cuda.synchronize()
        for a, b in zip(got, (out, h, rstd, dx, dw, eager)):
            assert torch.equal(a, b), f"replay {k}"
