"""A pre-norm feed-forward block in fp8, driven through the C ABI: the norm
with the residual's addition, the up-projection with its activation and the
down-projection with the residual stream, each one call.

    h = x + residual                       (residual optional)
    n = rmsnorm(h) * norm_weight           fp8_rmsnorm     -> E4M3 codes, h, 1 / rms
    u = act(n W_up^T + b_up)               fp8_mm_act      -> E4M3 codes, pre-activations
        (gated: act(gate) * value, W_up's rows alternating gate and value)
    y = u W_down^T + b_down + h            fp8_mm_act      -> bf16

forward / backward (training, delayed scaling): every quantized tensor has its
amax-history ring, as Fp8Linear's have; a step has no host synchronisation.
seed() gives a fresh block's rings the scales of a first batch.

    dY  -> E5M2 codes in both layouts, db_down       fp8_quantize_dual_bias_grad
    dU  = dY W_down                                  fp8_mm
    dZ  -> E5M2 codes in both layouts, db_up         fp8_act_grad (from dU, pre-activations;
        without activation and gating dZ is dU, quantized as dY is)
    dN  = dZ W_up                                    fp8_mm
    dW_down = dY^T U, dW_up = dZ^T N                 fp8_mm (U, N read K-major; any
        token count: zero codes up to a multiple of 16)
    dX  = gradient of the norm + dY, dnorm_weight    fp8_rmsnorm_grad

decode (serving): weights quantized once by freeze(), the norm's codes with one
scale per row, the activation's with the trained (or calibrated) scale; the
residual stream is updated in place.
"""
from __future__ import annotations

import torch

from . import (ACT_NONE, E4M3, E5M2, LAYOUT_ROW, fp8_act_grad, fp8_mm, fp8_mm_act, fp8_quantize,
               fp8_quantize_dual, fp8_quantize_dual_bias_grad, fp8_quantize_dynamic, fp8_ring_seed, fp8_rmsnorm,
               fp8_rmsnorm_grad, new_ring)


def _version(t: torch.Tensor):
    """t's count of in-place changes (inference tensors keep none)."""
    return None if t.is_inference() else t._version


# The weight gradients sum over tokens, and a product's K is a multiple of 16:
# codes that they read have that many tokens, the last ones zero.
def _token_rows(rows: int, cols: int, dev):
    """Storage for codes [rows, cols] with zero rows up to a multiple of 16, and
    the codes' part of it."""
    pad = -rows % 16
    buf = torch.empty(rows + pad, cols, dtype=torch.uint8, device=dev)
    if pad == 0:
        return buf, buf
    buf[rows:].zero_()
    return buf, buf[:rows]


def _token_cols(cols: int, rows: int, dev):
    """The same for transposed codes [cols, rows]: zero columns."""
    pad = -rows % 16
    buf = torch.empty(cols, rows + pad, dtype=torch.uint8, device=dev)
    if pad == 0:
        return buf, buf
    buf[:, rows:].zero_()
    return buf, buf[:, :rows]


class Fp8Mlp:
    """norm_weight [d]; w_up [F, d], or [2F, d] with interleaved rows when
    gated (interleave_gated); w_down [d, F]; biases optional."""

    def __init__(self, norm_weight: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                 b_up: torch.Tensor | None = None, b_down: torch.Tensor | None = None, act="silu",
                 gated: bool = False, eps: float = 1e-6, hist_len: int = 16):
        d, n_up = norm_weight.shape[0], w_up.shape[0]
        f = n_up // 2 if gated else n_up
        if tuple(w_up.shape) != (n_up, d) or tuple(w_down.shape) != (d, f) or (gated and n_up % 2):
            raise ValueError(f"weights {tuple(w_up.shape)} and {tuple(w_down.shape)} do not fit a width of {d}"
                             + (" (gated)" if gated else ""))
        self.norm_weight, self.w_up, self.w_down = norm_weight, w_up, w_down
        self.b_up, self.b_down = b_up, b_down
        self.act, self.gated, self.eps, self.hist_len = act, gated, eps, hist_len
        dev = norm_weight.device
        # n, W_up, u, W_down, dY, dZ
        self.rings = {k: new_ring(hist_len, 1.0, dev) for k in ("n", "w_up", "u", "w_down", "g", "z")}
        self.scale_inv = {k: torch.empty(1, dtype=torch.float32, device=dev) for k in self.rings}
        self._one = torch.ones(1, dtype=torch.float32, device=dev)
        self._amax = torch.empty(1, dtype=torch.float32, device=dev)
        self._seed_gradients = False  # set by seed() for the next backward
        self._frozen = None
        # decode's multiplier of u: scale_inv holds a pending backward's
        self._u_inv = torch.empty(1, dtype=torch.float32, device=dev)
        self._saved = None
        self._forwards = 0

    def _rows(self, t: torch.Tensor, name: str) -> torch.Tensor:
        """t as rows of d: its last dimension, or its last ones together, hold d
        (another width would be read as other rows)."""
        d, n = self.norm_weight.shape[0], 1
        for size in reversed(t.shape):
            n *= size
            if n >= d:
                break
        if n != d:
            raise ValueError(f"{name} must be [..., {d}], got {tuple(t.shape)}")
        return t.reshape(-1, d)

    def seed(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> None:
        """Seed the rings from the weights and a first batch, and those of the
        gradients in the next backward from what it quantizes, so that the
        first step has the tensors' own scales.  A fresh block's rings hold
        scale 1: its first steps lose what E5M2 cannot hold there, gradients
        below 2^-17.  (Call it before a step is captured in a graph.)"""
        x2, r2 = self._rows(x, "x"), None if residual is None else self._rows(residual, "residual")
        self._seed("w_up", E4M3, lambda s, amax: fp8_quantize(self.w_up, E4M3, scale=s, amax_out=amax))
        self._seed("w_down", E4M3, lambda s, amax: fp8_quantize(self.w_down, E4M3, scale=s, amax_out=amax))
        self._seed("n", E4M3, lambda s, amax: fp8_rmsnorm(x2, self.norm_weight, E4M3, self.eps, residual=r2, scale=s,
                                                          amax_out=amax))
        self._seed("u", E4M3, lambda s, amax: self._up(x2, r2, None, out_scale=s, out_amax=amax))
        self._seed_gradients = True

    def _seed(self, name: str, fmt, measure) -> None:
        """Seed a ring with the amax that `measure` finds at scale 1, its codes unused."""
        measure(self._one, self._amax)
        fp8_ring_seed(self.rings[name], self._amax, fmt)

    def _weight(self, name: str, w: torch.Tensor, both: bool):
        """w's codes, and the transposed ones that only a backward reads."""
        if both:
            return fp8_quantize_dual(w, E4M3, ring=self.rings[name], scale_inv_out=self.scale_inv[name])
        return fp8_quantize(w, E4M3, ring=self.rings[name], scale_inv_out=self.scale_inv[name]), None

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None, save_for_backward: bool = True):
        """x (and residual) bf16, fp16 or fp32 [..., d] -> the residual stream
        after the block, bf16 [..., d]."""
        x2, r2 = self._rows(x, "x"), None if residual is None else self._rows(residual, "residual")
        d = x2.shape[1]
        rows, dev, s = x2.shape[0], x.device, self.scale_inv
        h = x2 if r2 is None else torch.empty_like(x2)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        n_buf, n_out = _token_rows(rows, d, dev) if save_for_backward else (None, None)
        nq = fp8_rmsnorm(x2, self.norm_weight, E4M3, self.eps, residual=r2, out=n_out, ring=self.rings["n"],
                         scale_inv_out=s["n"], sum_out=None if r2 is None else h, rstd_out=rstd)
        self._saved = None  # its multipliers are being replaced, whatever comes of this forward
        wu, wu_t = self._weight("w_up", self.w_up, save_for_backward)
        wd, wd_t = self._weight("w_down", self.w_down, save_for_backward)
        z = None
        if save_for_backward and (self.gated or self.act not in ("none", None, ACT_NONE)):
            z = torch.empty(rows, self.w_up.shape[0], dtype=torch.bfloat16, device=dev)
        u_buf, u_out = _token_rows(rows, self.w_down.shape[1], dev) if save_for_backward else (None, None)
        uq = fp8_mm_act(nq, wu, s["n"], s["w_up"], self.b_up, self.act, self.gated, z_out=z, out=u_out, out_fmt=E4M3,
                        out_ring=self.rings["u"], out_scale_inv=s["u"])
        y = fp8_mm_act(uq, wd, s["u"], s["w_down"], self.b_down, residual=h)
        # the norm's weight is not a copy, and h is x itself without a residual:
        # backward, which reads both again, checks their versions
        nw = self.norm_weight
        self._saved = ((n_buf, h, rstd, z, u_buf, wu_t, wd_t, x.shape, nw, _version(h), _version(nw))
                       if save_for_backward else None)
        self._forwards += 1 if save_for_backward else 0
        return y.reshape(x.shape)

    def _gradient(self, name: str, dy: torch.Tensor, out_t: torch.Tensor, bias: bool):
        """dy's codes in both layouts; returns the row codes and the bias gradient."""
        ring, inv = self.rings[name], self.scale_inv[name]
        if self._seed_gradients:
            self._seed(name, E5M2, lambda s, amax: fp8_quantize(dy, E5M2, scale=s, amax_out=amax))
        if bias:
            codes, _, db = fp8_quantize_dual_bias_grad(dy, E5M2, out_t=out_t, ring=ring, scale_inv_out=inv)
            return codes, db
        return fp8_quantize_dual(dy, E5M2, out_t=out_t, ring=ring, scale_inv_out=inv)[0], None

    def backward(self, dy: torch.Tensor) -> dict:
        """Gradients of the latest saved forward: dx (x's and the residual's),
        norm_weight, w_up, w_down, b_up, b_down.  The norm's weight, and x of a
        forward without a residual, must not have been changed in place since."""
        if self._saved is None:
            raise RuntimeError("backward needs a forward with save_for_backward=True")
        n_buf, h, rstd, z, u_buf, wu_t, wd_t, x_shape, nw, h_version, nw_version = self._saved
        dy2 = self._rows(dy, "dy")
        if dy.dtype is not torch.bfloat16 or dy2.shape != h.shape:
            raise ValueError(f"dy must be bfloat16 {tuple(x_shape)} like the output, got {dy.dtype} {tuple(dy.shape)}")
        if _version(h) != h_version:
            raise RuntimeError("backward reads x again, which was changed in place since the forward pass")
        if _version(nw) != nw_version:
            raise RuntimeError("backward reads norm_weight again, which was changed in place since the forward pass")
        s, r = self.scale_inv, self.rings
        rows, d = h.shape
        g_t, g_out = _token_cols(d, rows, h.device)
        z_t, z_out = _token_cols(self.w_up.shape[0], rows, h.device)
        gq, db_down = self._gradient("g", dy2, g_out, self.b_down is not None)
        du = fp8_mm(gq, wd_t, E5M2, E4M3, s["g"], s["w_down"])
        if z is None:  # no activation
            zq, db_up = self._gradient("z", du, z_out, self.b_up is not None)
        else:
            if self._seed_gradients:
                self._seed("z", E5M2, lambda q, amax: fp8_act_grad(du, z, self.act, self.gated, E5M2, scale=q,
                                                                   amax_out=amax))
            zq, _, db_up = fp8_act_grad(du, z, self.act, self.gated, E5M2, out_t=z_out, ring=r["z"],
                                        scale_inv_out=s["z"], need_bias_grad=self.b_up is not None)
        self._seed_gradients = False
        dn = fp8_mm(zq, wu_t, E5M2, E4M3, s["z"], s["w_up"])
        dw_down = fp8_mm(g_t, u_buf.t(), E5M2, E4M3, s["g"], s["u"])
        dw_up = fp8_mm(z_t, n_buf.t(), E5M2, E4M3, s["z"], s["n"])
        if h.dtype is torch.bfloat16:
            dx, dnw = fp8_rmsnorm_grad(dn, h, nw, rstd, dsum=dy2)
        else:  # the products' gradients are bf16: fp32 holds both types, fp16 would not
            dx, dnw = fp8_rmsnorm_grad(dn.float(), h.float(), nw, rstd, dsum=dy2.float())
            dx = dx.to(h.dtype)
        return {"x": dx.reshape(x_shape), "norm_weight": dnw, "w_up": dw_up, "w_down": dw_down, "b_up": db_up,
                "b_down": db_down}

    # ------------------------------------------------------------------ serving
    def freeze(self) -> None:
        """Quantize the weights for decode (current scaling).  Called again, it
        fills the same storage, so that a captured decode has the new weights."""
        weights = (self.w_up, self.w_down)
        kept = self._frozen
        if kept is None:
            kept = [(torch.empty(w.shape, dtype=torch.uint8, device=w.device),
                     torch.empty(1, dtype=torch.float32, device=w.device)) for w in weights]
        for w, (codes, inv) in zip(weights, kept):
            fp8_quantize_dynamic(w, E4M3, LAYOUT_ROW, out_row=codes, scale_inv_out=inv)
        self._frozen = kept

    def calibrate(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> None:
        """Fold one batch's amax into the activation's ring, for decode of a
        block that was not trained here: the up-projection as decode runs it
        (the frozen weights where there are some), nothing else touched."""
        x2, r2 = self._rows(x, "x"), None if residual is None else self._rows(residual, "residual")
        self._up(x2, r2, None if self._frozen is None else self._frozen[0], out_ring=self.rings["u"])

    def _up(self, x2, r2, weight, **out) -> None:
        """The up-projection under current scaling, for its output's amax;
        weight: W_up's codes and multiplier, where they are at hand."""
        nq, row_inv = self._decode_norm(x2, r2, None)
        if weight is None:
            inv = torch.empty(1, dtype=torch.float32, device=x2.device)
            weight = fp8_quantize_dynamic(self.w_up, E4M3, LAYOUT_ROW, scale_inv_out=inv)[0], inv
        fp8_mm_act(nq, weight[0], row_inv, weight[1], self.b_up, self.act, self.gated, out_fmt=E4M3, **out)

    def _decode_norm(self, x, residual, sum_out):
        """The norm's codes with one scale per row, and the rows' multipliers."""
        row_inv = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        return fp8_rmsnorm(x, self.norm_weight, E4M3, self.eps, residual=residual, row_scaled=True,
                           scale_inv_out=row_inv, sum_out=sum_out), row_inv

    def decode(self, x: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
        """One serving step on bf16 [tokens, d]: adds x to residual and the block's
        output to that, in place; returns residual."""
        if self._frozen is None:
            raise RuntimeError("decode needs freeze()")
        if residual.dtype is not torch.bfloat16:  # before the norm has written to it
            raise ValueError(f"residual must be bfloat16, got {residual.dtype}")
        (wu, s_wu), (wd, s_wd) = self._frozen
        nq, row_inv = self._decode_norm(x, residual, residual)
        scale = self.rings["u"].view(torch.float32)[self.hist_len:self.hist_len + 1]  # the ring's current scale
        uq = fp8_mm_act(nq, wu, row_inv, s_wu, self.b_up, self.act, self.gated, out_fmt=E4M3, out_scale=scale,
                        out_scale_inv=self._u_inv)
        return fp8_mm_act(uq, wd, self._u_inv, s_wd, self.b_down, residual=residual, out=residual)


class _Fp8MlpFn(torch.autograd.Function):
    """One Fp8Mlp step on torch's autograd tape; a backward must belong to the
    block's latest saved forward."""

    @staticmethod
    def forward(ctx, x, residual, norm_weight, w_up, w_down, b_up, b_down, block):
        y = block.forward(x, residual)
        ctx.block, ctx.step = block, block._forwards
        ctx.residual_shape = None if residual is None else residual.shape
        ctx.dtypes = [None if t is None else t.dtype for t in (x, residual, norm_weight, w_up, w_down, b_up, b_down)]
        return y

    @staticmethod
    def backward(ctx, dy):
        block = ctx.block
        if block._forwards != ctx.step:
            raise RuntimeError("fp8_mlp: the block ran another forward since the one being differentiated")
        g = block.backward(dy.contiguous())
        g_res = None if ctx.residual_shape is None else g["x"].reshape(ctx.residual_shape)
        grads = [g["x"], g_res, g["norm_weight"], g["w_up"], g["w_down"], g["b_up"], g["b_down"]]
        out = [None if t is None or dt is None or not need else t.to(dt)
               for t, dt, need in zip(grads, ctx.dtypes, ctx.needs_input_grad)]
        return (*out, None)


def fp8_mlp(x: torch.Tensor, block: Fp8Mlp, residual: torch.Tensor | None = None) -> torch.Tensor:
    """y = block.forward(x, residual) recorded for autograd: the backward pass
    fills the gradients of x, residual and the block's weights and biases."""
    return _Fp8MlpFn.apply(x, residual, block.norm_weight, block.w_up, block.w_down, block.b_up, block.b_down, block)
