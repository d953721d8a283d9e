"""The end of a model in fp8, driven through the C ABI: the last norm, the
vocabulary's product and the softmax cross entropy, the logits never written.

    h = x + residual                       (residual optional)
    n = rmsnorm(h) * norm_weight           fp8_rmsnorm             -> E4M3 codes, h, 1 / rms
    W -> E4M3 codes                        fp8_quantize
    loss = mean over the targets           fp8_cross_entropy       -> loss and lse per row, mean

forward / backward (training, delayed scaling: rings for n and W, as Fp8Mlp's):

    dN, dW                                 fp8_cross_entropy_grad
    dX = gradient of the norm, dnorm_weight    fp8_rmsnorm_grad

score (serving): each target's loss (its negative log-probability), the weights
quantized once by freeze(), the norm's codes with one scale per row.
"""
from __future__ import annotations

import torch

from . import (E4M3, LAYOUT_ROW, fp8_cross_entropy, fp8_cross_entropy_grad, fp8_cross_entropy_workspace_bytes,
               fp8_quantize, fp8_quantize_dynamic, fp8_ring_seed, fp8_rmsnorm, fp8_rmsnorm_grad, new_ring)
from .mlp import _version


class Fp8Head:
    """norm_weight [d]; weight [vocabulary, d], d a multiple of 16."""

    def __init__(self, norm_weight: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, hist_len: int = 16):
        d = norm_weight.shape[0]
        if weight.dim() != 2 or weight.shape[1] != d or weight.shape[0] < 1:
            raise ValueError(f"weight {tuple(weight.shape)} does not fit a width of {d}")
        if d % 16:
            raise ValueError(f"the width must be a multiple of 16, got {d}")
        self.norm_weight, self.weight, self.eps, self.hist_len = norm_weight, weight, eps, hist_len
        dev = norm_weight.device
        self.rings = {k: new_ring(hist_len, 1.0, dev) for k in ("n", "w")}
        self.scale_inv = {k: torch.empty(1, dtype=torch.float32, device=dev) for k in self.rings}
        self._frozen = None
        self._saved = None
        self._forwards = 0

    def _rows(self, x, residual, targets):
        d = self.norm_weight.shape[0]
        if x.shape[-1] != d or (residual is not None and residual.shape[-1] != d):
            raise ValueError(f"x and residual must be [..., {d}], got {tuple(x.shape)}"
                             + ("" if residual is None else f" and {tuple(residual.shape)}"))
        x2, r2 = x.reshape(-1, d), None if residual is None else residual.reshape(-1, d)
        if targets is None:
            return x2, r2, None
        # before a ring moves
        if targets.dtype not in (torch.int64, torch.int32):
            raise ValueError(f"targets must be int64 or int32, got {targets.dtype}")
        if targets.numel() != x2.shape[0]:
            raise ValueError(f"{targets.numel()} targets for {x2.shape[0]} rows")
        if targets.device != x.device:
            raise ValueError(f"targets are on {targets.device}, x on {x.device}")
        return x2, r2, targets.reshape(-1).contiguous()

    def _check_weight(self, x2) -> None:
        """What the weight's quantize and the loss would refuse, before the norm's ring moves."""
        w, (rows, d) = self.weight, x2.shape
        if w.dtype not in (torch.bfloat16, torch.float16, torch.float32):
            raise ValueError(f"weight must be bfloat16, float16 or float32, got {w.dtype}")
        if w.dim() != 2 or w.shape[1] != d or w.stride(1) != 1:
            raise ValueError(f"weight must be [vocabulary, {d}] with unit column stride, got {tuple(w.shape)}")
        if w.device != x2.device:
            raise ValueError(f"weight is on {w.device}, x on {x2.device}")
        if rows and not fp8_cross_entropy_workspace_bytes(rows, w.shape[0], d):
            raise ValueError(f"{rows} rows of {d} over a vocabulary of {w.shape[0]}: more than fp8_cross_entropy takes")

    def seed(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> None:
        """Seed the rings from the weight and a first batch, so that the first
        step has the tensors' own scales (a fresh ring holds scale 1)."""
        x2, r2, _ = self._rows(x, residual, None)
        one = torch.ones(1, dtype=torch.float32, device=x.device)
        amax = torch.empty_like(one)
        fp8_quantize(self.weight, E4M3, scale=one, amax_out=amax)
        fp8_ring_seed(self.rings["w"], amax, E4M3)
        fp8_rmsnorm(x2, self.norm_weight, E4M3, self.eps, residual=r2, scale=one, amax_out=amax)
        fp8_ring_seed(self.rings["n"], amax, E4M3)

    def forward(self, x: torch.Tensor, targets: torch.Tensor, residual: torch.Tensor | None = None,
                save_for_backward: bool = True) -> torch.Tensor:
        """x (and residual) bf16, fp16 or fp32 [..., d], targets [...] -> the mean
        loss over the targets that are not negative, an fp32 scalar (0 without
        any)."""
        x2, r2, t = self._rows(x, residual, targets)
        self._check_weight(x2)
        s, dev = self.scale_inv, x.device
        h = x2 if r2 is None else torch.empty_like(x2)
        rstd = torch.empty(x2.shape[0], dtype=torch.float32, device=dev)
        self._saved = None  # its multipliers are being replaced, whatever comes of this forward
        nq = fp8_rmsnorm(x2, self.norm_weight, E4M3, self.eps, residual=r2, ring=self.rings["n"], scale_inv_out=s["n"],
                         sum_out=None if r2 is None else h, rstd_out=rstd)
        wq = fp8_quantize(self.weight, E4M3, ring=self.rings["w"], scale_inv_out=s["w"])
        mean = torch.empty(2, dtype=torch.float32, device=dev)
        _, lse = fp8_cross_entropy(nq, wq, t, s["n"], s["w"], mean_out=mean)
        if save_for_backward:
            # h is x itself without a residual, the norm's weight and the targets are no copies either
            kept = (h, self.norm_weight, t)
            self._saved = (nq, wq, lse, mean, rstd, kept, [_version(k) for k in kept], x.shape)
            self._forwards += 1
        return mean[0].clone()

    def backward(self, dloss: torch.Tensor) -> dict:
        """Gradients of dloss times the latest saved forward's mean loss: x (x's
        and the residual's), norm_weight, weight.  x of a forward without a
        residual, the norm's weight and the targets must not have been changed in
        place since."""
        if self._saved is None:
            raise RuntimeError("backward needs a forward with save_for_backward=True")
        nq, wq, lse, mean, rstd, kept, versions, x_shape = self._saved
        for k, v, name in zip(kept, versions, ("x", "norm_weight", "targets")):
            if _version(k) != v:
                raise RuntimeError(f"backward reads {name} again, which was changed in place since the forward pass")
        h, nw, t = kept
        s = self.scale_inv
        dn, dw = fp8_cross_entropy_grad(nq, wq, t, lse, mean[1:] * dloss.float(), s["n"], s["w"])
        if h.dtype is torch.bfloat16:
            dx, dnw = fp8_rmsnorm_grad(dn, h, nw, rstd)
        else:  # dn is bf16: fp32 holds both types, fp16 would not
            dx, dnw = fp8_rmsnorm_grad(dn.float(), h.float(), nw, rstd)
            dx = dx.to(h.dtype)
        return {"x": dx.reshape(x_shape), "norm_weight": dnw, "weight": dw}

    # ------------------------------------------------------------------ serving
    def freeze(self) -> None:
        """Quantize the weight for score (current scaling).  Called again, it fills
        the same storage, so that a captured score has the new weight."""
        kept = self._frozen
        if kept is None:
            w = self.weight
            kept = (torch.empty(w.shape, dtype=torch.uint8, device=w.device),
                    torch.empty(1, dtype=torch.float32, device=w.device))
        fp8_quantize_dynamic(self.weight, E4M3, LAYOUT_ROW, out_row=kept[0], scale_inv_out=kept[1])
        self._frozen = kept

    def score(self, x: torch.Tensor, targets: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        """Loss of each target (0 where it is negative), fp32 of targets' shape;
        exp(-loss) is the target's probability."""
        if self._frozen is None:
            raise RuntimeError("score needs freeze()")
        x2, r2, t = self._rows(x, residual, targets)
        row_inv = torch.empty(x2.shape[0], dtype=torch.float32, device=x.device)
        nq = fp8_rmsnorm(x2, self.norm_weight, E4M3, self.eps, residual=r2, row_scaled=True, scale_inv_out=row_inv)
        loss, _ = fp8_cross_entropy(nq, self._frozen[0], t, row_inv, self._frozen[1])
        return loss.reshape(targets.shape)


class _Fp8HeadFn(torch.autograd.Function):
    """One Fp8Head loss on torch's autograd tape; a backward must belong to the
    head's latest saved forward."""

    @staticmethod
    def forward(ctx, x, residual, norm_weight, weight, targets, head):
        loss = head.forward(x, targets, residual)
        ctx.head, ctx.step = head, head._forwards
        ctx.residual_shape = None if residual is None else residual.shape
        ctx.dtypes = [None if t is None else t.dtype for t in (x, residual, norm_weight, weight)]
        return loss

    @staticmethod
    def backward(ctx, dloss):
        head = ctx.head
        if head._forwards != ctx.step:
            raise RuntimeError("fp8_head_loss: the head ran another forward since the one being differentiated")
        g = head.backward(dloss)
        g_res = None if ctx.residual_shape is None else g["x"].reshape(ctx.residual_shape)
        out = [None if dt is None or not need else t.to(dt)
               for t, dt, need in zip((g["x"], g_res, g["norm_weight"], g["weight"]), ctx.dtypes, ctx.needs_input_grad)]
        return (*out, None, None)


def fp8_head_loss(x: torch.Tensor, targets: torch.Tensor, head: Fp8Head,
                  residual: torch.Tensor | None = None) -> torch.Tensor:
    """loss = head.forward(x, targets, residual) recorded for autograd: the
    backward pass fills the gradients of x, residual and the head's weights.  (Its
    backward is captured into a graph only while no eager graph of the same leaves is
    alive; head.forward and head.backward capture at any time.)"""
    return _Fp8HeadFn.apply(x, residual, head.norm_weight, head.weight, targets, head)
