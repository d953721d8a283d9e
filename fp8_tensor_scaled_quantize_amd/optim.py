"""AdamW over the weights of fp8 layers, driven through the C ABI: one or few
launches for all of them (fp8_adamw_step), with their gradients' norm and the
clipping factor (fp8_grad_norm) before it and no host synchronisation.

    opt = AdamW([block.w_up, block.w_down, ...], lr=3e-4, max_norm=1.0, state_bits=8)
    fp8_head_loss(fp8_mlp(x, block), targets, head).backward()
    opt.step()
    opt.zero_grad()
"""
from __future__ import annotations

import torch

from . import ADAMW_BLOCK, ADAMW_STEP_WORDS, fp8_adamw_step, fp8_grad_norm


class AdamW:
    """params: contiguous fp32, fp16 or bf16 device tensors.  masters: 16-bit ones
    get fp32 weights that the step updates and rounds to them.  state_bits 8: the
    states are E4M3 codes with a scale per 256 elements.  weight_decay: a number,
    or one per param.  max_norm: the gradients are scaled to at most that norm,
    and a step whose gradients are not finite is skipped (without a look from the
    host: `steps` counts it all the same, the device's count does not).
    capturable: the step's number and lr are device words (lr_word), so that a
    captured step goes on."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01,
                 state_bits: int = 32, masters: bool = True, max_norm: float | None = None, capturable: bool = False,
                 seed: int = 0):
        self.params = list(params)
        if not self.params:
            raise ValueError("no params")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        self.lr, self.betas, self.eps, self.max_norm, self.seed = lr, betas, eps, max_norm, seed
        n = len(self.params)
        self.weight_decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        if len(self.weight_decay) != n:
            raise ValueError(f"{len(self.weight_decay)} weight decays for {n} params")
        dev = self.params[0].device
        self.masters = [p.detach().float() if masters and p.dtype is not torch.float32 else None for p in self.params]
        kind = torch.float32 if state_bits == 32 else torch.uint8
        self.exp_avg, self.exp_avg_sq = ([torch.zeros(p.numel(), dtype=kind, device=dev) for p in self.params]
                                         for _ in range(2))
        self.exp_avg_scale, self.exp_avg_sq_scale = (
            [torch.zeros(-(-p.numel() // ADAMW_BLOCK), device=dev) if state_bits == 8 else None for p in self.params]
            for _ in range(2))
        self.steps = 0
        self.step_words = torch.zeros(ADAMW_STEP_WORDS, dtype=torch.int32, device=dev) if capturable else None
        self.lr_word = torch.full((1,), lr, dtype=torch.float32, device=dev) if capturable else None
        self.norm = torch.zeros(1, dtype=torch.float32, device=dev)  # of the latest step's gradients, with max_norm
        self._clip = torch.empty_like(self.norm)

    def zero_grad(self) -> None:
        for p in self.params:
            p.grad = None

    def step(self, grads=None) -> None:
        """One step with the given gradients, or the params' own; a param whose
        gradient is None is left as it is."""
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} params")
        at = [i for i, g in enumerate(grads) if g is not None]
        if not at:
            return
        grads = [grads[i].contiguous() for i in at]

        def pick(ts):
            return [ts[i] for i in at]

        scale = None
        if self.max_norm is not None:
            fp8_grad_norm(grads, self.max_norm, out=self.norm, clip_out=self._clip)
            scale = self._clip
        device = self.step_words is not None
        fp8_adamw_step(pick(self.params), grads, pick(self.exp_avg), pick(self.exp_avg_sq),
                       self.step_words if device else self.steps + 1, self.lr_word if device else self.lr, self.betas,
                       self.eps, pick(self.weight_decay), pick(self.masters), pick(self.exp_avg_scale),
                       pick(self.exp_avg_sq_scale), scale, self.seed)
        if not device:
            self.steps += 1

    def sync_masters(self) -> None:
        """Take the masters from the params anew (after a param was loaded or set)."""
        for p, m in zip(self.params, self.masters):
            if m is not None:
                m.copy_(p.detach())

    def state_dict(self) -> dict:
        steps = self.steps if self.step_words is None else int(self.step_words[0])
        return {"steps": steps, "masters": self.masters, "exp_avg": self.exp_avg, "exp_avg_sq": self.exp_avg_sq,
                "exp_avg_scale": self.exp_avg_scale, "exp_avg_sq_scale": self.exp_avg_sq_scale}

    def load_state_dict(self, state: dict) -> None:
        """Fill the states from another optimizer's over the same params (same
        state_bits and masters), in place."""
        for name in ("masters", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
            mine, theirs = getattr(self, name), state[name]
            if [None if t is None else (t.numel(), t.dtype) for t in mine] != \
                    [None if t is None else (t.numel(), t.dtype) for t in theirs]:
                raise ValueError(f"the state's {name} do not fit these params")
        for name in ("masters", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
            for a, b in zip(getattr(self, name), state[name]):
                if a is not None:
                    a.copy_(b.reshape(a.shape))
        self.steps = int(state["steps"])
        if self.step_words is not None:
            self.step_words[0] = self.steps
