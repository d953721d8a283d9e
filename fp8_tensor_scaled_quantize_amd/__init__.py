"""fp8mi: FP8 per-tensor scaled quantize, delayed-scaling amax history fold
and per-tensor-scaled fp8 GEMM on MI355X (gfx950).

Thin Python binding over the C ABI in include/fp8mi.h (libfp8mi.so).  The
functions carry the ABI's names and only marshal arguments: shapes, strides
and device pointers of torch tensors, and torch's current HIP stream.  Every
step of the computation runs in the library's HIP kernels; when the library
is missing, every call raises.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import lib

__all__ = ["E4M3", "E5M2", "F32", "F16", "BF16", "Fp8Error", "fp8_quantize", "fp8_quantize_dual", "fp8_quantize_dual_bias_grad",
           "fp8_quantize_dual_bias_grad_noalloc", "NOALLOC_SCRATCH_BYTES", "stream_reference",
           "fp8_quantize_dynamic", "DYNAMIC_WORKSPACE_BYTES", "fp8_amax_fold", "fp8_mm", "fp8_mm_ex", "FP8_E4M3", "FP8_E5M2", "fp8_bias_grad", "fp8_bias_grad_workspace_bytes", "fp8_ring_seed", "new_ring", "ring_words", "version",
           "fp8_rmsnorm", "fp8_rmsnorm_grad", "fp8_rmsnorm_grad_workspace_bytes", "fp8_mm_act", "fp8_act_grad",
           "ACT_NONE", "ACT_RELU", "ACT_GELU", "ACT_SILU", "interleave_gated"]

E4M3, E5M2 = 0, 1
F32, F16, BF16 = 0, 1, 2
FP8_E4M3, FP8_E5M2 = 3, 4  # fp8 storage types (fp8 bias / fp8 GEMM output of fp8_mm_ex)

ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU = 0, 1, 2, 3  # activations of fp8_mm_act (gelu: the tanh form)
_ACT_GATED = 16

_ACT = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "silu": ACT_SILU, None: ACT_NONE,
        ACT_NONE: ACT_NONE, ACT_RELU: ACT_RELU, ACT_GELU: ACT_GELU, ACT_SILU: ACT_SILU}
_FMT = {"e4m3": E4M3, "e5m2": E5M2, E4M3: E4M3, E5M2: E5M2}
_DT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
RING_SCRATCH_WORDS = 1024  # FP8MI_RING_SCRATCH_WORDS
DYNAMIC_WORKSPACE_BYTES = 4096  # FP8MI_DYNAMIC_WORKSPACE_BYTES
NOALLOC_SCRATCH_BYTES = 8 * 1024 * 1024  # FP8MI_NOALLOC_SCRATCH_BYTES
LAYOUT_ROW, LAYOUT_T, LAYOUT_DUAL = 0, 1, 2


def ring_words_for(hist_len: int) -> int:
    """FP8MI_RING_WORDS(hist_len)."""
    return hist_len + 4 + RING_SCRATCH_WORDS


class Fp8Error(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"fp8mi status {status}: {detail}")
        self.status = status


def _check(status: int) -> None:
    if status != 0:
        L = lib()
        raise Fp8Error(status, f"{L.fp8mi_status_string(status).decode()} -- {L.fp8mi_last_error().decode()}")


def _fmt(f) -> int:
    try:
        return _FMT[f]
    except KeyError:
        raise ValueError(f"unknown fp8 format {f!r}") from None


def _ptr(t):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _current_device() -> int:
    """torch's current HIP device (the raw getter skips the lazy-init check,
    done already by the time a device tensor exists)."""
    return _raw_device() if _raw_device is not None else torch.cuda.current_device()


def _stream(t: torch.Tensor):
    """Handle of torch's current HIP stream on t's device (the raw getter
    skips building a Stream object: a few microseconds per call)."""
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _as_codes(t: torch.Tensor, name: str = "codes") -> torch.Tensor:
    if t.element_size() != 1:
        raise ValueError(f"{name} must hold 1-byte fp8 codes, got {t.dtype}")
    return t.view(torch.uint8) if t.dtype != torch.uint8 else t


# Argument checks.  The library takes raw device pointers and sizes, so the
# binding checks what only the tensors know -- device, dtype, shape -- before
# the call; the library itself checks sizes, strides and alignment.

def _on_device(*ts) -> None:
    """Every tensor argument lives on the current HIP device (the library
    launches there): a host tensor or another device's memory would be read
    as this device's."""
    dev = None
    for t in ts:
        if t is None:
            continue
        d = t.get_device()
        if d < 0:
            raise ValueError("tensor arguments must be HIP device tensors, got a host tensor")
        if dev is None:
            dev = d
        elif d != dev:
            raise ValueError(f"tensor arguments on devices cuda:{dev} and cuda:{d}")
    if dev is not None and dev != _current_device():
        raise ValueError(f"tensors on cuda:{dev} but the current device is cuda:{_current_device()}")


def _dt(t: torch.Tensor, name: str) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}") from None


def _scalar(t, name: str) -> None:
    """A device fp32 scalar argument (its first element is read or written)."""
    if t is not None and (t.dtype != torch.float32 or t.numel() < 1):
        raise ValueError(f"{name} must be a float32 tensor of at least one element")


def _matrix_out(t: torch.Tensor, shape, name: str) -> None:
    """A 2-D output of exactly `shape` with unit stride along its rows."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} needs unit stride along its rows")


def _vector(t: torch.Tensor, n: int, name: str) -> None:
    """A contiguous 1-D tensor of n elements."""
    if t.dim() != 1 or t.numel() != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous 1-D tensor of {n} elements, got {tuple(t.shape)}")


def _quant_checks(x, name, out_row, out_t, scale, scale_inv_out, amax_out):
    rows, cols = x.shape
    if out_row is not None:
        _matrix_out(out_row, (rows, cols), "out" if out_t is None else "out_row")
    if out_t is not None:
        _matrix_out(out_t, (cols, rows), "out" if out_row is None else "out_t")
    _scalar(scale, "scale")
    _scalar(scale_inv_out, "scale_inv_out")
    _scalar(amax_out, "amax_out")
    return _dt(x, name)


def _ring_args(ring):
    if ring is None:
        return None, 0
    if ring.dim() != 1 or ring.dtype not in (torch.int32, torch.uint32) or not ring.is_contiguous():
        raise ValueError("ring must be a contiguous 1-D int32 tensor of hist_len + 4 + 1024 words")
    h = ring.numel() - 4 - RING_SCRATCH_WORDS
    if h < 1:
        raise ValueError(f"ring of {ring.numel()} words is too short")
    return ring.data_ptr(), h


def version() -> str:
    return lib().fp8mi_version().decode()


def new_ring(hist_len: int, scale0: float = 1.0, device=None) -> torch.Tensor:
    """A zeroed ring (history 0, slot 0, ticket and scratch 0) holding scale0
    as its current scale: FP8MI_RING_WORDS(hist_len) int32 words on `device`."""
    w = torch.zeros(ring_words_for(hist_len), dtype=torch.int32)
    w[hist_len] = torch.tensor([scale0], dtype=torch.float32).view(torch.int32)[0]
    return w.to(device if device is not None else "cuda")


def ring_words(ring: torch.Tensor):
    """Host copy of a ring: dict of hist (fp32), scale, idx, ticket and
    whether the scratch region is all zero (as it is between calls)."""
    w = ring.detach().to("cpu")
    h = w.numel() - 4 - RING_SCRATCH_WORDS
    f = w.view(torch.float32)
    return {"hist": f[:h].clone(), "scale": float(f[h]), "idx": int(w[h + 1]),
            "ticket": int(w[h + 2]), "scratch_clear": bool((w[h + 3:] == 0).all())}


def fp8_quantize(x: torch.Tensor, fmt, transposed: bool = False, out: torch.Tensor | None = None,
                 scale: torch.Tensor | None = None, ring: torch.Tensor | None = None,
                 scale_inv_out: torch.Tensor | None = None, amax_out: torch.Tensor | None = None) -> torch.Tensor:
    """Quantize a 2-D bf16/fp16/fp32 tensor (unit column stride; any row
    stride and base offset) to fp8 codes (uint8) in row or transposed layout.
    Exactly one of `scale` (device fp32 scalar) or `ring` is given."""
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be 2-D with unit column stride")
    rows, cols = x.shape
    f = _fmt(fmt)
    if out is None:
        out = torch.empty((cols, rows) if transposed else (rows, cols), dtype=torch.uint8, device=x.device)
    out = _as_codes(out, "out")
    dt = _quant_checks(x, "x", None if transposed else out, out if transposed else None, scale, scale_inv_out,
                       amax_out)
    ld_x = x.stride(0) if rows > 1 else cols
    ld_out = out.stride(0) if out.shape[0] > 1 else out.shape[1]
    rp, h = _ring_args(ring)
    _on_device(x, out, scale, ring, scale_inv_out, amax_out)
    _check(lib().fp8_quantize(_ptr(x), dt, rows, cols, ld_x, f, int(bool(transposed)), _ptr(out),
                              ld_out, _ptr(scale), rp, h, _ptr(scale_inv_out), _ptr(amax_out), _stream(x)))
    return out


def fp8_quantize_dual(x: torch.Tensor, fmt, out_row: torch.Tensor | None = None, out_t: torch.Tensor | None = None,
                      scale: torch.Tensor | None = None, ring: torch.Tensor | None = None,
                      scale_inv_out: torch.Tensor | None = None, amax_out: torch.Tensor | None = None):
    """Both layouts from one read; returns (codes [rows, cols], codes_t [cols, rows])."""
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be 2-D with unit column stride")
    rows, cols = x.shape
    f = _fmt(fmt)
    if out_row is None:
        out_row = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if out_t is None:
        out_t = torch.empty((cols, rows), dtype=torch.uint8, device=x.device)
    out_row, out_t = _as_codes(out_row, "out_row"), _as_codes(out_t, "out_t")
    dt = _quant_checks(x, "x", out_row, out_t, scale, scale_inv_out, amax_out)
    ld_x = x.stride(0) if rows > 1 else cols
    ld_r = out_row.stride(0) if out_row.shape[0] > 1 else out_row.shape[1]
    ld_t = out_t.stride(0) if out_t.shape[0] > 1 else out_t.shape[1]
    rp, h = _ring_args(ring)
    _on_device(x, out_row, out_t, scale, ring, scale_inv_out, amax_out)
    _check(lib().fp8_quantize_dual(_ptr(x), dt, rows, cols, ld_x, f, _ptr(out_row), ld_r, _ptr(out_t),
                                   ld_t, _ptr(scale), rp, h, _ptr(scale_inv_out), _ptr(amax_out), _stream(x)))
    return out_row, out_t


def fp8_quantize_dual_bias_grad(dy: torch.Tensor, fmt, out_row: torch.Tensor | None = None,
                                out_t: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                                ring: torch.Tensor | None = None, scale_inv_out: torch.Tensor | None = None,
                                amax_out: torch.Tensor | None = None, bias_grad_out: torch.Tensor | None = None,
                                workspace: torch.Tensor | None = None):
    """fp8_quantize_dual of a 2-D bf16/fp16 gradient plus its bias gradient
    from the same read; returns (codes, codes_t, bias_grad bf16 [cols])."""
    if dy.dim() != 2 or (dy.shape[1] > 1 and dy.stride(1) != 1):
        raise ValueError("dy must be 2-D with unit column stride")
    rows, cols = dy.shape
    f = _fmt(fmt)
    if out_row is None:
        out_row = torch.empty((rows, cols), dtype=torch.uint8, device=dy.device)
    if out_t is None:
        out_t = torch.empty((cols, rows), dtype=torch.uint8, device=dy.device)
    if bias_grad_out is None:
        bias_grad_out = torch.empty(cols, dtype=torch.bfloat16, device=dy.device)
    need = fp8_bias_grad_workspace_bytes(rows, cols)
    if workspace is None:
        workspace = torch.empty(max(need, 8), dtype=torch.uint8, device=dy.device)
    out_row, out_t = _as_codes(out_row, "out_row"), _as_codes(out_t, "out_t")
    dt = _quant_checks(dy, "dy", out_row, out_t, scale, scale_inv_out, amax_out)
    _vector(bias_grad_out, cols, "bias_grad_out")
    if bias_grad_out.dtype != torch.bfloat16:
        raise ValueError("bias_grad_out must be bfloat16")
    ld_x = dy.stride(0) if rows > 1 else cols
    ld_r = out_row.stride(0) if out_row.shape[0] > 1 else out_row.shape[1]
    ld_t = out_t.stride(0) if out_t.shape[0] > 1 else out_t.shape[1]
    rp, h = _ring_args(ring)
    _on_device(dy, out_row, out_t, scale, ring, scale_inv_out, amax_out, bias_grad_out, workspace)
    _check(lib().fp8_quantize_dual_bias_grad(_ptr(dy), dt, rows, cols, ld_x, f, _ptr(out_row), ld_r,
                                             _ptr(out_t), ld_t, _ptr(scale), rp, h, _ptr(scale_inv_out),
                                             _ptr(amax_out), _ptr(bias_grad_out), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), _stream(dy)))
    return out_row, out_t, bias_grad_out


def fp8_quantize_dual_bias_grad_noalloc(dy: torch.Tensor, fmt, out_row: torch.Tensor, out_t: torch.Tensor,
                                        bias_grad_out: torch.Tensor, scale: torch.Tensor | None = None,
                                        ring: torch.Tensor | None = None, scale_inv_out: torch.Tensor | None = None,
                                        amax_out: torch.Tensor | None = None):
    """fp8_quantize_dual_bias_grad with the library's own scratch instead of a
    workspace: every output is the caller's (nothing is allocated here or in
    the library).  Returns (codes, codes_t, bias_grad)."""
    if dy.dim() != 2 or (dy.shape[1] > 1 and dy.stride(1) != 1):
        raise ValueError("dy must be 2-D with unit column stride")
    rows, cols = dy.shape
    f = _fmt(fmt)
    out_row, out_t = _as_codes(out_row, "out_row"), _as_codes(out_t, "out_t")
    dt = _quant_checks(dy, "dy", out_row, out_t, scale, scale_inv_out, amax_out)
    _vector(bias_grad_out, cols, "bias_grad_out")
    if bias_grad_out.dtype != torch.bfloat16:
        raise ValueError("bias_grad_out must be bfloat16")
    ld_x = dy.stride(0) if rows > 1 else cols
    ld_r = out_row.stride(0) if out_row.shape[0] > 1 else out_row.shape[1]
    ld_t = out_t.stride(0) if out_t.shape[0] > 1 else out_t.shape[1]
    rp, h = _ring_args(ring)
    _on_device(dy, out_row, out_t, scale, ring, scale_inv_out, amax_out, bias_grad_out)
    _check(lib().fp8_quantize_dual_bias_grad_noalloc(_ptr(dy), dt, rows, cols, ld_x, f, _ptr(out_row), ld_r,
                                                     _ptr(out_t), ld_t, _ptr(scale), rp, h, _ptr(scale_inv_out),
                                                     _ptr(amax_out), _ptr(bias_grad_out), _stream(dy)))
    return out_row, out_t, bias_grad_out


def stream_reference(src: torch.Tensor, dst: torch.Tensor) -> torch.Tensor:
    """Measurement aid: fp8mi_stream_reference over two contiguous device
    tensors (dst of src's byte size or its half) -- the HBM traffic of a
    quantize moving the same bytes, with no arithmetic."""
    for t, name in ((src, "src"), (dst, "dst")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    _on_device(src, dst)
    _check(lib().fp8mi_stream_reference(src.data_ptr(), src.numel() * src.element_size(), dst.data_ptr(),
                                        dst.numel() * dst.element_size(), _stream(src)))
    return dst


def fp8_quantize_dynamic(x: torch.Tensor, fmt, layout: int = LAYOUT_ROW, out_row: torch.Tensor | None = None,
                         out_t: torch.Tensor | None = None, scale_inv_out: torch.Tensor | None = None,
                         amax_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Current scaling: quantize a 2-D bf16/fp16/fp32 tensor with
    s = fmt_max / amax(x) measured in the same call (no ring).  layout 0 row,
    1 transposed, 2 both; returns (codes or None, codes_t or None)."""
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be 2-D with unit column stride")
    if layout not in (LAYOUT_ROW, LAYOUT_T, LAYOUT_DUAL):
        raise ValueError(f"layout must be 0, 1 or 2, got {layout!r}")
    rows, cols = x.shape
    f = _fmt(fmt)
    if layout != LAYOUT_T and out_row is None:
        out_row = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if layout != LAYOUT_ROW and out_t is None:
        out_t = torch.empty((cols, rows), dtype=torch.uint8, device=x.device)
    if workspace is None:
        workspace = torch.empty(DYNAMIC_WORKSPACE_BYTES, dtype=torch.uint8, device=x.device)
    out_row = None if out_row is None else _as_codes(out_row, "out_row")
    out_t = None if out_t is None else _as_codes(out_t, "out_t")
    dt = _quant_checks(x, "x", out_row if layout != LAYOUT_T else None, out_t if layout != LAYOUT_ROW else None,
                       None, scale_inv_out, amax_out)
    _on_device(x, out_row, out_t, scale_inv_out, amax_out, workspace)
    ld_x = x.stride(0) if rows > 1 else cols
    ld_r = 0 if out_row is None else (out_row.stride(0) if out_row.shape[0] > 1 else out_row.shape[1])
    ld_t = 0 if out_t is None else (out_t.stride(0) if out_t.shape[0] > 1 else out_t.shape[1])
    _check(lib().fp8_quantize_dynamic(_ptr(x), dt, rows, cols, ld_x, f, layout, _ptr(out_row), ld_r,
                                      _ptr(out_t), ld_t, _ptr(scale_inv_out), _ptr(amax_out), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(x)))
    return out_row, out_t


def fp8_amax_fold(ring: torch.Tensor, amax: torch.Tensor, fmt) -> None:
    """Fold a device fp32 amax into the ring (the fold a ring-mode quantize
    performs in its last workgroup)."""
    rp, h = _ring_args(ring)
    _scalar(amax, "amax")
    _on_device(ring, amax)
    _check(lib().fp8_amax_fold(rp, h, _ptr(amax), _fmt(fmt), _stream(ring)))


def fp8_mm(a: torch.Tensor, b: torch.Tensor, fmt_a=E4M3, fmt_b=E4M3, a_scale_inv: torch.Tensor | None = None,
           b_scale_inv: torch.Tensor | None = None, bias: torch.Tensor | None = None,
           out: torch.Tensor | None = None) -> torch.Tensor:
    """C = bf16(A B^T * sa * sb + bias) for fp8 codes A [(batch,) M, K] and
    B [(batch,) N, K]; a size-1 (or stride-0) batch dimension broadcasts.
    An operand that is a transposed view (unit stride along its rows, e.g.
    codes_t.t()) is read K-major through fp8_mm_ex's layout tags."""
    return _mm_call(a, b, fmt_a, fmt_b, a_scale_inv, b_scale_inv, bias, None, None, out, None, ex=False)


def fp8_mm_ex(a: torch.Tensor, b: torch.Tensor, fmt_a=E4M3, fmt_b=E4M3, a_scale_inv: torch.Tensor | None = None,
              b_scale_inv: torch.Tensor | None = None, bias: torch.Tensor | None = None,
              bias_fmt=None, bias_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
              out_fmt=None, out_scale: torch.Tensor | None = None, out_ring: torch.Tensor | None = None,
              out_scale_inv: torch.Tensor | None = None, out_amax: torch.Tensor | None = None) -> torch.Tensor:
    """fp8_mm with an fp8-stored bias (codes `bias` of format `bias_fmt`,
    dequantized by `bias_scale`) and/or a quantizing epilogue: with `out_fmt`
    (E4M3 / E5M2) the output is fp8 codes quantized with `out_scale` or the
    ring `out_ring` (which then folds the output's amax); `out_scale_inv` and
    `out_amax` receive 1/s and amax."""
    return _mm_call(a, b, fmt_a, fmt_b, a_scale_inv, b_scale_inv, bias, bias_fmt, bias_scale, out, out_fmt,
                    out_scale, out_ring, out_scale_inv, out_amax)


def _operand(t: torch.Tensor, name: str):
    """(batch, rows, K, batch stride, leading dimension, K-major) of a
    [rows, K] or [batch, rows, K] operand.  An operand that is a transposed
    view of [K, rows] storage (unit stride along its rows) is K-major: the
    library reads it through the FP8MI_A_KM / FP8MI_B_KM layout tags."""
    if t.dim() == 3:
        batch, rows, K = t.shape
        sb, sr, sk = t.stride()
    elif t.dim() == 2:
        batch, (rows, K), sb = 1, t.shape, 0
        sr, sk = t.stride()
    else:
        raise ValueError(f"operand {name} must be [rows, K] or [batch, rows, K], got {tuple(t.shape)}")
    if batch == 1:
        sb = 0
    if K <= 1 or sk == 1:
        return batch, rows, K, sb, (sr if rows > 1 else K), False
    if rows <= 1 or sr == 1:
        ld = sk
        # the library reads K full rows of ld bytes (the last row's padding included)
        last = t.storage_offset() + (batch - 1) * sb + K * ld
        if last > t.untyped_storage().nbytes():
            raise ValueError(f"K-major operand {name} must span {K} full rows of {ld} bytes in its storage")
        return batch, rows, K, sb, ld, True
    raise ValueError(f"operand {name} needs unit stride along K or along its rows")


def _operand_ld(t: torch.Tensor, name: str):
    """Leading dimension of an operand and whether it is K-major."""
    return _operand(t, name)[4:]


def _mm_call(a, b, fmt_a, fmt_b, a_scale_inv, b_scale_inv, bias, bias_fmt, bias_scale, out, out_fmt,
             out_scale=None, out_ring=None, out_scale_inv=None, out_amax=None, ex=True):
    a, b = _as_codes(a, "a"), _as_codes(b, "b")
    ba, M, K, sa, lda, a_km = _operand(a, "a")
    bb, N, Kb, sb, ldb, b_km = _operand(b, "b")
    if K != Kb:
        raise ValueError(f"K mismatch: {tuple(a.shape)} vs {tuple(b.shape)}")
    batch = ba if ba > 1 else bb
    if ba not in (1, batch) or bb not in (1, batch):
        raise ValueError("batch sizes must match or be 1")
    layout = (1 if a_km else 0) | (2 if b_km else 0)
    c_dt = BF16 if out_fmt is None else FP8_E4M3 + _fmt(out_fmt)
    batched = a.dim() == 3 or b.dim() == 3
    if out is None:
        out = torch.empty((batch, M, N) if batched else (M, N), dtype=torch.bfloat16 if c_dt == BF16 else torch.uint8,
                          device=a.device)
    if c_dt != BF16:
        out = _as_codes(out, "out")
    elif out.dtype != torch.bfloat16:
        raise ValueError(f"out must be bfloat16, got {out.dtype}")
    if out.dim() == 3:
        cshape, (sc, ldc, scn) = tuple(out.shape), out.stride()
    else:
        cshape, (ldc, scn) = (1,) + tuple(out.shape), out.stride()
        sc = M * ldc
    if cshape != (batch, M, N):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(batch, M, N) if batch > 1 else (M, N)}")
    if N > 1 and scn != 1:
        raise ValueError("out needs unit stride along N")
    if M <= 1:
        ldc = N
    if batch <= 1:
        sc = M * ldc
    if bias is None:
        bias_dt = 0
    elif bias_fmt is not None:
        bias, bias_dt = _as_codes(bias, "bias"), FP8_E4M3 + _fmt(bias_fmt)
    else:
        bias_dt = _dt(bias, "bias")
    if bias is not None:
        _vector(bias, N, "bias")
    _scalar(a_scale_inv, "a_scale_inv")
    _scalar(b_scale_inv, "b_scale_inv")
    if ex:
        for t, name in ((bias_scale, "bias_scale"), (out_scale, "out_scale"), (out_scale_inv, "out_scale_inv"),
                        (out_amax, "out_amax")):
            _scalar(t, name)
        _on_device(a, b, a_scale_inv, b_scale_inv, bias, bias_scale, out, out_scale, out_ring, out_scale_inv,
                   out_amax)
    else:
        _on_device(a, b, a_scale_inv, b_scale_inv, bias, out)
    L = lib()
    if not ex and layout == 0:
        _check(L.fp8_mm(a.data_ptr(), _fmt(fmt_a), lda, sa, b.data_ptr(), _fmt(fmt_b), ldb, sb, M, N, K, batch,
                        _ptr(a_scale_inv), _ptr(b_scale_inv), _ptr(bias), bias_dt, out.data_ptr(), ldc, sc,
                        _stream(a)))
        return out
    rp, h = _ring_args(out_ring)
    _check(L.fp8_mm_ex(a.data_ptr(), _fmt(fmt_a), lda, sa, b.data_ptr(), _fmt(fmt_b), ldb, sb, M, N, K, batch,
                       layout, _ptr(a_scale_inv), _ptr(b_scale_inv), _ptr(bias), bias_dt, _ptr(bias_scale),
                       out.data_ptr(), c_dt, ldc, sc, _ptr(out_scale), rp, h, _ptr(out_scale_inv), _ptr(out_amax),
                       _stream(a)))
    return out


def fp8_bias_grad_workspace_bytes(rows: int, cols: int) -> int:
    """Device workspace fp8_bias_grad needs for a [rows, cols] gradient."""
    return int(lib().fp8_bias_grad_workspace_bytes(rows, cols))


def fp8_bias_grad(dy: torch.Tensor, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Bias gradient: sum of a bf16/fp16 gradient over every leading
    dimension (fp64 accumulation in a fixed order, one bf16 rounding) ->
    bf16 [cols].  `workspace` (any dtype, device) is scratch of at least
    fp8_bias_grad_workspace_bytes(rows, cols) bytes; one is allocated from
    torch's caching allocator when it is not given."""
    if dy.dim() < 1 or (dy.shape[-1] > 1 and dy.stride(-1) != 1):
        raise ValueError("dy needs unit stride along its last dimension")
    cols = dy.shape[-1]
    d2 = dy.reshape(-1, cols)
    rows = d2.shape[0]
    ld = d2.stride(0) if rows > 1 else cols
    if out is None:
        out = torch.empty(cols, dtype=torch.bfloat16, device=dy.device)
    need = fp8_bias_grad_workspace_bytes(rows, cols)
    if workspace is None:
        workspace = torch.empty(max(need, 8), dtype=torch.uint8, device=dy.device)
    dt = _dt(dy, "dy")
    _vector(out, cols, "out")
    if out.dtype != torch.bfloat16:
        raise ValueError("out must be bfloat16")
    _on_device(d2, out, workspace)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().fp8_bias_grad(_ptr(d2), dt, rows, cols, ld, _ptr(out), _ptr(workspace), nbytes,
                               _stream(dy)))
    return out


def fp8_ring_seed(ring: torch.Tensor, amax: torch.Tensor, fmt) -> None:
    """Reset a ring and publish the scale a fold of `amax` into an empty
    window gives (fmt_max / amax, or 1.0)."""
    rp, h = _ring_args(ring)
    _scalar(amax, "amax")
    _on_device(ring, amax)
    _check(lib().fp8_ring_seed(rp, h, _ptr(amax), _fmt(fmt), _stream(ring)))


# A serving step calls the operators below once per token, when the host's
# share of a call is longer than the kernel: their checks read each tensor's
# shape and strides once and call as little as they can.

def _rows2d(t: torch.Tensor, name: str):
    """(shape, rows, cols, leading dimension) of a 2-D tensor with unit column
    stride."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    rows, cols = shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return shape, rows, cols, ld if rows > 1 else cols


def _ld(t: torch.Tensor, shape, dtype, name: str) -> int:
    """Leading dimension of a matrix of exactly this shape and dtype."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {str(dtype)[6:]}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name} needs unit stride along its rows")
    return ld if shape[0] > 1 else shape[1]


def _typed_vector(t: torch.Tensor, n: int, name: str, dtypes=_DT) -> int:
    """Type code of a contiguous 1-D tensor of n elements."""
    dt = dtypes.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be " + " or ".join(str(d)[6:] for d in dtypes) + f", got {t.dtype}")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous 1-D tensor of {n} elements, got {tuple(t.shape)}")
    return dt


# autograd's record that a tensor was changed in place: the operators below bump
# it where an output is one of their inputs, as torch's in-place operations do
_changed_in_place = torch.autograd.graph.increment_version

_F32_ONLY, _BF16_ONLY = {torch.float32: F32}, {torch.bfloat16: BF16}


def fp8_rmsnorm(x: torch.Tensor, weight: torch.Tensor | None, fmt=E4M3, eps: float = 1e-6,
                residual: torch.Tensor | None = None, out: torch.Tensor | None = None, row_scaled: bool = False,
                scale: torch.Tensor | None = None, ring: torch.Tensor | None = None,
                scale_inv_out: torch.Tensor | None = None, amax_out: torch.Tensor | None = None,
                sum_out: torch.Tensor | None = None, rstd_out: torch.Tensor | None = None) -> torch.Tensor:
    """Root-mean-square norm of each row of x (+ residual), times weight, as
    fp8 codes.  Exactly one of `scale`, `ring` and `row_scaled` picks the scale:
    given, the ring's (which folds this call's amax), or measured per row --
    then scale_inv_out [rows] receives the rows' dequantisation multipliers.
    sum_out receives x + residual (it may be residual or x itself: in place),
    rstd_out [rows] the 1 / rms values that fp8_rmsnorm_grad reads."""
    shape, rows, cols, ld_x = _rows2d(x, "x")
    dtype = x.dtype
    dt = _dt(x, "x")
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=x.device)
    elif out.dtype is not torch.uint8:
        out = _as_codes(out, "out")
    ld_out = _ld(out, shape, torch.uint8, "out")
    wdt = 0 if weight is None else _typed_vector(weight, cols, "weight")
    ld_res = 0 if residual is None else _ld(residual, shape, dtype, "residual")
    ld_sum = 0 if sum_out is None else _ld(sum_out, shape, dtype, "sum_out")
    if row_scaled:
        if scale is not None or ring is not None:
            raise ValueError("row_scaled measures its scales: give neither scale nor ring")
        if scale_inv_out is None:
            raise ValueError("row_scaled needs scale_inv_out [rows]")
        _typed_vector(scale_inv_out, rows, "scale_inv_out", _F32_ONLY)
        if amax_out is not None:
            _typed_vector(amax_out, rows, "amax_out", _F32_ONLY)
    else:
        _scalar(scale, "scale")
        _scalar(scale_inv_out, "scale_inv_out")
        _scalar(amax_out, "amax_out")
    if rstd_out is not None:
        _typed_vector(rstd_out, rows, "rstd_out", _F32_ONLY)
    rp, h = (None, 0) if ring is None else _ring_args(ring)
    _on_device(x, weight, residual, out, scale, ring, scale_inv_out, amax_out, sum_out, rstd_out)
    px, pr = x.data_ptr(), None if residual is None else residual.data_ptr()
    ps = None if sum_out is None else sum_out.data_ptr()
    status = lib().fp8_rmsnorm(
        px, dt, rows, cols, ld_x, pr, ld_res,
        None if weight is None else weight.data_ptr(), wdt, ctypes.byref(ctypes.c_float(eps)), _fmt(fmt),
        out.data_ptr(), ld_out, 1 if row_scaled else 0, None if scale is None else scale.data_ptr(), rp, h,
        None if scale_inv_out is None else scale_inv_out.data_ptr(), None if amax_out is None else amax_out.data_ptr(),
        ps, ld_sum, None if rstd_out is None else rstd_out.data_ptr(), _stream(x))
    if status:
        _check(status)
    if ps and (ps == pr or ps == px):
        _changed_in_place(sum_out)
    return out


def fp8_rmsnorm_grad_workspace_bytes(rows: int, cols: int) -> int:
    """Device workspace fp8_rmsnorm_grad needs for its weight gradient."""
    return int(lib().fp8_rmsnorm_grad_workspace_bytes(rows, cols))


def fp8_rmsnorm_grad(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor | None, rstd: torch.Tensor,
                     dsum: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                     dweight: torch.Tensor | None = None, need_dweight: bool = True,
                     workspace: torch.Tensor | None = None):
    """Gradient of fp8_rmsnorm's normalised rows: returns (dx, dweight fp32 or
    None).  h and rstd are the forward call's sum_out (or x) and rstd_out, dsum
    the gradient that reaches h by the residual path (added into dx; dx may be
    dsum or dy itself)."""
    shape, rows, cols, ld_dy = _rows2d(dy, "dy")
    dtype = dy.dtype
    dt = _dt(dy, "dy")
    ld_h = _ld(h, shape, dtype, "h")
    wdt = 0 if weight is None else _typed_vector(weight, cols, "weight")
    _typed_vector(rstd, rows, "rstd", _F32_ONLY)
    ld_ds = 0 if dsum is None else _ld(dsum, shape, dtype, "dsum")
    if dx is None:
        dx = torch.empty(shape, dtype=dtype, device=dy.device)
    ld_dx = _ld(dx, shape, dtype, "dx")
    nbytes = 0
    if need_dweight or dweight is not None:
        if dweight is None:
            dweight = torch.empty(cols, dtype=torch.float32, device=dy.device)
        _typed_vector(dweight, cols, "dweight", _F32_ONLY)
        if workspace is None:
            workspace = torch.empty(max(fp8_rmsnorm_grad_workspace_bytes(rows, cols), 4), dtype=torch.uint8,
                                    device=dy.device)
        nbytes = workspace.numel() * workspace.element_size()
    _on_device(dy, h, weight, rstd, dsum, dx, dweight, workspace)
    py, ph, pd, pg = dy.data_ptr(), h.data_ptr(), None if dsum is None else dsum.data_ptr(), dx.data_ptr()
    status = lib().fp8_rmsnorm_grad(
        py, dt, rows, cols, ld_dy, ph, ld_h, None if weight is None else weight.data_ptr(), wdt, rstd.data_ptr(), pd,
        ld_ds, pg, ld_dx,
        None if dweight is None else dweight.data_ptr(), None if workspace is None else workspace.data_ptr(), nbytes,
        _stream(dy))
    if status:
        _check(status)
    if pg and (pg == pd or pg == py or pg == ph):
        _changed_in_place(dx)
    return dx, dweight


def _act(act, gated: bool) -> int:
    try:
        return _ACT[act] | (_ACT_GATED if gated else 0)
    except (KeyError, TypeError):
        raise ValueError(f"unknown activation {act!r}") from None


def interleave_gated(gate: torch.Tensor, value: torch.Tensor) -> torch.Tensor:
    """The weight (or bias, or its codes) of a gated product from its two
    halves: rows 2j and 2j + 1 are row j of gate and of value."""
    if gate.shape != value.shape or gate.dtype != value.dtype:
        raise ValueError(f"gate {tuple(gate.shape)} {gate.dtype} and value {tuple(value.shape)} {value.dtype} differ")
    return torch.stack((gate, value), dim=1).flatten(0, 1)


def _row_scales(t, n: int, name: str) -> int:
    """1 where t holds one multiplier per row, 0 for one per tensor (or none)."""
    if t is None:
        return 0
    k = t.numel()
    if t.dtype is not torch.float32 or (k != 1 and k != n):
        raise ValueError(f"{name} must be a float32 tensor of 1 or {n} elements")
    if k > 1:
        _typed_vector(t, n, name, _F32_ONLY)
        return 1
    return 0


def fp8_mm_act(a: torch.Tensor, b: torch.Tensor, a_scale_inv: torch.Tensor | None = None,
               b_scale_inv: torch.Tensor | None = None, bias: torch.Tensor | None = None, act=ACT_NONE,
               gated: bool = False, residual: torch.Tensor | None = None, z_out: torch.Tensor | None = None,
               out: torch.Tensor | None = None, out_fmt=None, out_scale: torch.Tensor | None = None,
               out_ring: torch.Tensor | None = None, out_scale_inv: torch.Tensor | None = None,
               out_amax: torch.Tensor | None = None) -> torch.Tensor:
    """E4M3 codes A [M, K] and B [N, K]: f(A B^T sa sb + bias) + residual as
    bf16, or with out_fmt=E4M3 as codes quantized with out_scale or out_ring.
    The scale multipliers hold one word, or one per row of their operand.
    gated: B's rows alternate gate and value (interleave_gated) and the output
    is f(gate) * value + residual, [M, N / 2].  z_out (bf16 [M, N]) receives
    the values before the activation, for fp8_act_grad.  A bf16 residual may be
    `out` itself."""
    if a.dtype is not torch.uint8:
        a = _as_codes(a, "a")
    if b.dtype is not torch.uint8:
        b = _as_codes(b, "b")
    _, M, K, lda = _rows2d(a, "a")
    _, N, Kb, ldb = _rows2d(b, "b")
    if K != Kb:
        raise ValueError(f"K mismatch: {tuple(a.shape)} vs {tuple(b.shape)}")
    code = _act(act, gated)
    if gated and N % 2:
        raise ValueError(f"a gated product needs an even number of rows in b, got {N}")
    shape = (M, N // 2 if gated else N)
    fp8_out = out_fmt is not None
    if fp8_out:
        if _fmt(out_fmt) != E4M3:
            raise ValueError("fp8_mm_act's fp8 output is E4M3")
        for t, name in ((out_scale, "out_scale"), (out_scale_inv, "out_scale_inv"), (out_amax, "out_amax")):
            if t is not None:
                _scalar(t, name)
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8 if fp8_out else torch.bfloat16, device=a.device)
    elif fp8_out and out.dtype is not torch.uint8:
        out = _as_codes(out, "out")
    ldc = _ld(out, shape, torch.uint8 if fp8_out else torch.bfloat16, "out")
    rows = _row_scales(a_scale_inv, M, "a_scale_inv") | (_row_scales(b_scale_inv, N, "b_scale_inv") << 1)
    bias_dt = 0 if bias is None else _typed_vector(bias, N, "bias")
    res_dt = ld_res = ld_z = 0
    if residual is not None:
        res_dt = _dt(residual, "residual")
        ld_res = _ld(residual, shape, residual.dtype, "residual")
    if z_out is not None:
        ld_z = _ld(z_out, (M, N), torch.bfloat16, "z_out")
    rp, h = (None, 0) if out_ring is None else _ring_args(out_ring)
    _on_device(a, b, a_scale_inv, b_scale_inv, bias, residual, z_out, out, out_scale, out_ring, out_scale_inv, out_amax)
    pr, pc = None if residual is None else residual.data_ptr(), out.data_ptr()
    status = lib().fp8_mm_act(
        a.data_ptr(), lda, b.data_ptr(), ldb, M, N, K, None if a_scale_inv is None else a_scale_inv.data_ptr(),
        None if b_scale_inv is None else b_scale_inv.data_ptr(), rows, None if bias is None else bias.data_ptr(),
        bias_dt, code, pr, res_dt, ld_res, None if z_out is None else z_out.data_ptr(), ld_z, pc,
        FP8_E4M3 if fp8_out else BF16, ldc,
        None if out_scale is None else out_scale.data_ptr(), rp, h,
        None if out_scale_inv is None else out_scale_inv.data_ptr(), None if out_amax is None else out_amax.data_ptr(),
        _stream(a))
    if status:
        _check(status)
    if pc and pc == pr:
        _changed_in_place(out)
    return out


def fp8_act_grad(dy: torch.Tensor, z: torch.Tensor, act, gated: bool = False, fmt=E5M2,
                 out_row: torch.Tensor | None = None, out_t: torch.Tensor | None = None,
                 scale: torch.Tensor | None = None, ring: torch.Tensor | None = None,
                 scale_inv_out: torch.Tensor | None = None, amax_out: torch.Tensor | None = None,
                 need_bias_grad: bool = False, bias_grad_out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None):
    """Gradient dz of fp8_mm_act's pre-activations (z, its z_out) from the
    gradient dy of its output, quantized with `scale` or `ring`: returns
    (codes [rows, cols], codes_t [cols, rows], bias gradient bf16 or None)."""
    _, drows, dcols, ld_dy = _rows2d(dy, "dy")
    shape, rows, cols, ld_z = _rows2d(z, "z")
    if z.dtype is not torch.bfloat16:
        raise ValueError(f"z must be bfloat16, got {z.dtype}")
    if drows != rows or dcols * (2 if gated else 1) != cols:
        raise ValueError(f"dy {tuple(dy.shape)} does not fit z {tuple(z.shape)}" + (" (gated)" if gated else ""))
    dt, code, f = _dt(dy, "dy"), _act(act, gated), _fmt(fmt)
    if out_row is None:
        out_row = torch.empty(shape, dtype=torch.uint8, device=dy.device)
    elif out_row.dtype is not torch.uint8:
        out_row = _as_codes(out_row, "out_row")
    if out_t is None:
        out_t = torch.empty((cols, rows), dtype=torch.uint8, device=dy.device)
    elif out_t.dtype is not torch.uint8:
        out_t = _as_codes(out_t, "out_t")
    ld_row = _ld(out_row, shape, torch.uint8, "out_row")
    ld_t = _ld(out_t, (cols, rows), torch.uint8, "out_t")
    for t, name in ((scale, "scale"), (scale_inv_out, "scale_inv_out"), (amax_out, "amax_out")):
        if t is not None:
            _scalar(t, name)
    nbytes = 0
    if need_bias_grad or bias_grad_out is not None:
        if bias_grad_out is None:
            bias_grad_out = torch.empty(cols, dtype=torch.bfloat16, device=dy.device)
        _typed_vector(bias_grad_out, cols, "bias_grad_out", _BF16_ONLY)
        if workspace is None:
            workspace = torch.empty(max(fp8_bias_grad_workspace_bytes(rows, cols), 8), dtype=torch.uint8,
                                    device=dy.device)
        nbytes = workspace.numel() * workspace.element_size()
    rp, h = (None, 0) if ring is None else _ring_args(ring)
    _on_device(dy, z, out_row, out_t, scale, ring, scale_inv_out, amax_out, bias_grad_out, workspace)
    status = lib().fp8_act_grad(
        dy.data_ptr(), dt, rows, cols, ld_dy, z.data_ptr(), ld_z, code, f, out_row.data_ptr(), ld_row,
        out_t.data_ptr(), ld_t, None if scale is None else scale.data_ptr(), rp, h,
        None if scale_inv_out is None else scale_inv_out.data_ptr(), None if amax_out is None else amax_out.data_ptr(),
        None if bias_grad_out is None else bias_grad_out.data_ptr(),
        None if workspace is None else workspace.data_ptr(), nbytes, _stream(dy))
    if status:
        _check(status)
    return out_row, out_t, bias_grad_out
