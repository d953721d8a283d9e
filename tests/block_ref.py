"""Plain 64-bit forms of the operators around an fp8 linear layer, and the
bounds their fp32 kernels are held to.  Torch on the CPU, one formula per
line; no code of the library.

Bounds.  A kernel's fp32 value v of an exact value t has |v - t| <= rel |t| (or
rel times the sum of the terms' magnitudes where terms cancel).  Codes are then
checked without a tolerance of their own: the code must lie between the codes
of t s moved down and up by that much (encoding is monotonic)."""
import math

import numpy as np
import torch

import oracle as O

FMT_NAME = {0: O.E4M3, 1: O.E5M2}
GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715
F32_ULP = 2.0 ** -24  # relative error of one fp32 rounding


def rms_rel(cols: int) -> float:
    """Relative error of fp32 rstd and of the scaled products that follow: a
    lane adds up to 48 squares one by one, 6 + 16 more additions join lanes and
    waves; half of that (square root), plus 8 roundings of the square root,
    the divisions and the products."""
    return (0.5 * (min(cols, 48) + 22) + 8) * F32_ULP


def codes64(t: torch.Tensor, fmt: int) -> np.ndarray:
    """fp8 codes of 64-bit values (through fp32, which the encoder reads)."""
    return O.encode(t.numpy().astype(np.float32), FMT_NAME[fmt])


def assert_codes(codes: torch.Tensor, t: torch.Tensor, fmt: int, rel, tag="") -> None:
    """codes of values within rel |t| (or an absolute tensor rel) of t."""
    tab = O.decode_table(FMT_NAME[fmt])
    slack = rel if isinstance(rel, torch.Tensor) else rel * t.abs() + 1e-45
    got = tab[codes.cpu().numpy()]
    nan = torch.isnan(t).numpy()
    assert np.array_equal(np.isnan(got), nan), f"{tag}: NaN codes differ"
    lo, hi = tab[codes64(t - slack, fmt)], tab[codes64(t + slack, fmt)]
    bad = ~nan & ~((got >= lo) & (got <= hi))
    assert not bad.any(), f"{tag}: {bad.sum()} of {bad.size} codes outside their bounds"


def assert_close(got: torch.Tensor, t: torch.Tensor, slack, tag="") -> None:
    """|got - t| <= slack (same NaN and infinity places)."""
    g = got.detach().cpu().double()
    fin = torch.isfinite(t)
    assert torch.equal(torch.isnan(g), torch.isnan(t)), f"{tag}: NaN places differ"
    assert torch.equal(g[~fin & ~torch.isnan(t)], t[~fin & ~torch.isnan(t)]), f"{tag}: infinities differ"
    s = slack if isinstance(slack, torch.Tensor) else torch.full_like(t, slack)
    bad = (g[fin] - t[fin]).abs() > s[fin]
    assert not bad.any(), (f"{tag}: {int(bad.sum())} of {bad.numel()} outside the bound, worst "
                           f"{float(((g[fin] - t[fin]).abs() / s[fin].clamp_min(1e-300)).max()):.2f} x")


def half_ulp(t: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """Largest error of one rounding of values near t to dtype."""
    bits, tiny = {torch.bfloat16: (8, 2.0 ** -134), torch.float16: (11, 2.0 ** -25),
                  torch.float32: (24, 2.0 ** -150)}[dtype]
    return t.abs() * 2.0 ** -bits * (1 + 2.0 ** -7) + tiny


def scale_of(amax: torch.Tensor, fmt: int) -> torch.Tensor:
    """fmt_max / amax, 1 where amax is 0 or not finite."""
    q = O.FMT_MAX[FMT_NAME[fmt]] / amax
    return torch.where((amax > 0) & torch.isfinite(amax) & torch.isfinite(q), q, torch.ones_like(q))


def rmsnorm(x, res, w, eps):
    """h, rstd [rows, 1] and y in 64 bits."""
    h = x.double() if res is None else x.double() + res.double()
    rstd = 1.0 / torch.sqrt((h * h).sum(1, keepdim=True) / max(1, h.shape[1]) + eps)
    y = h * rstd
    return h, rstd, y if w is None else y * w.double()


def rmsnorm_grad(dy, h, w, rstd, dsum):
    """dx, dw and the magnitudes of the sums they hold."""
    dy, h, r = dy.double(), h.double(), rstd.double().reshape(-1, 1)
    g = dy if w is None else dy * w.double()
    n = max(1, h.shape[1])
    dx = r * g - r ** 3 * ((g * h).sum(1, keepdim=True) / n) * h
    mag = (r * g).abs() + r ** 3 * ((g * h).abs().sum(1, keepdim=True) / n) * h.abs()
    if dsum is not None:
        dx, mag = dx + dsum.double(), mag + dsum.double().abs()
    t = dy * h * r
    return dx, t.sum(0), mag, t.abs().sum(0)


def act(t, name):
    """The activation and its slope."""
    if name == "relu":
        return torch.where(t > 0, t, torch.zeros_like(t)), (t > 0).to(t.dtype)
    if name == "none":
        return t, torch.ones_like(t)
    if name == "silu":
        p, dp = torch.sigmoid(t), 1.0
    else:
        p, dp = torch.sigmoid(2 * GELU_C * (t + GELU_A * t ** 3)), 2 * GELU_C * (1 + 3 * GELU_A * t * t)
    return t * p, p + t * p * (1 - p) * dp


def rand(shape, sigma, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(dtype)


def place(t: torch.Tensor, ld=None, shift=0, fill=0.0, device="cuda:0") -> torch.Tensor:
    """A copy of the matrix t on the device with row stride ld, its first
    element `shift` elements past an allocation's start; everything around it
    holds `fill`."""
    rows, cols = t.shape
    ld = cols if ld is None else ld
    buf = torch.full((shift + max(rows, 1) * ld + 16,), fill, dtype=t.dtype, device=device)
    view = torch.as_strided(buf, (rows, cols), (ld, 1), shift)
    if t.numel():
        view.copy_(t.to(device))
    return view


def around_untouched(view: torch.Tensor, fill) -> bool:
    """Every element of the view's buffer outside the view still holds fill."""
    full = torch.empty(0, dtype=view.dtype, device=view.device).set_(view.untyped_storage()).clone()
    torch.as_strided(full, view.shape, view.stride(), view.storage_offset()).fill_(fill)
    return bool((full == torch.tensor(fill, dtype=view.dtype, device=view.device)).all())
