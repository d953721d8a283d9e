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

from . import (ADAMW_BLOCK, ADAMW_STEP_WORDS, _all_on_device, _dtypes, _flat, _numel, fp8_adamw_step, fp8_grad_norm)


class AdamW:
    """params: contiguous fp32, fp16 or bf16 device tensors.  masters: 16-bit ones
    get fp32 weights that the step updates and rounds to them.  state_bits 8: the
    states are E4M3 codes with a scale per 256 elements.  weight_decay: a number,
    or one per param.  max_norm: the gradients are scaled to at most that norm,
    and a step whose gradients are not finite is skipped (without a look from the
    host: `steps` counts it all the same, the device's count does not).
    capturable: the step's number and lr are device words (lr_word), so that a
    captured step goes on.

    Each param counts its own steps, those that had a gradient for it, and its bias
    corrections go by them.  Params that had theirs in the same steps are updated in
    one call, and any others in a call for each such group."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01,
                 state_bits: int = 32, masters: bool = True, max_norm: float | None = None, capturable: bool = False,
                 seed: int = 0):
        self.params = list(params)
        if not self.params:
            raise ValueError("no params")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        self.lr, self.betas, self.eps, self.max_norm, self.seed = lr, betas, eps, max_norm, seed
        self.state_bits = state_bits
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
        # groups of params with one count, ascending: it is at the first param's place
        self._groups = [list(range(n))]
        self._counts = [0] * n  # steps issued from the host
        self._words = torch.zeros(n, ADAMW_STEP_WORDS, dtype=torch.int32, device=dev) if capturable else None
        self.step_words = None if self._words is None else self._words[0]  # the first param's
        self._captured = set()  # the groups of captured steps, by their first params: they stay together
        self._none = torch.empty(0, dtype=torch.float32, device=dev)  # stands for a param without a gradient
        self.lr_word = torch.full((1,), lr, dtype=torch.float32, device=dev) if capturable else None
        self.norm = torch.zeros(1, dtype=torch.float32, device=dev)  # of the latest step's gradients, with max_norm
        self._clip = torch.empty_like(self.norm)

    def zero_grad(self) -> None:
        for p in self.params:
            p.grad = None

    @property
    def steps(self) -> int:
        """The most steps that a param has had."""
        return max(self._counts)

    @steps.setter
    def steps(self, count: int) -> None:
        self._set_counts([int(count)] * len(self.params))

    def _regroup(self, counts) -> list:
        """The groups for new counts."""
        kept = [g for g in self._groups if g[0] in self._captured]
        rest = sorted(i for g in self._groups if g[0] not in self._captured for i in g)
        if any(len({counts[i] for i in g}) > 1 for g in kept):
            raise ValueError("these step counts differ among params that a captured step counts together")
        return kept + [[i for i in rest if counts[i] == c] for c in dict.fromkeys(counts[i] for i in rest)]

    def _set_counts(self, counts) -> None:
        self._groups, self._counts = self._regroup(counts), list(counts)
        if self._words is not None:
            self._words.copy_(torch.tensor([[c] + [0] * (ADAMW_STEP_WORDS - 1) for c in counts], dtype=torch.int32))

    def _parted(self, have):
        """The groups, those parted of which some params have a gradient and some have
        none, and where such parts' counts come from and go to."""
        parts, moved = [], []
        for g in self._groups:
            yes, no = [i for i in g if i in have], [i for i in g if i not in have]
            parts += [p for p in (yes, no) if p]
            if yes and no:
                moved.append((g[0], no[0] if yes[0] == g[0] else yes[0]))
                # (a count of 0 needs no copy, so a first step may be captured with some gradients missing)
                if self._words is not None and self._counts[g[0]] and (g[0] in self._captured or
                                                                       torch.cuda.is_current_stream_capturing()):
                    raise RuntimeError("a captured step keeps the params that were updated together: these gradients "
                                       "are there for a part of them (run one such step before the capture)")
        return parts, moved

    def step(self, grads=None) -> None:
        """One step with the given gradients, or the params' own; a param whose
        gradient is None is left as it is, and does not count the step."""
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} params")
        at = [i for i, g in enumerate(grads) if g is not None]
        if not at:
            return
        for i in at:
            grads[i] = grads[i].contiguous()
        given, have = [grads[i] for i in at], set(at)
        groups, moved = (self._groups, ()) if len(at) == len(grads) else self._parted(have)
        active = [g for g in groups if g[0] in have]
        if len(active) > 1:  # several calls: what one of them would refuse, before the first has run
            params = [self.params[i] for i in at]
            _flat(params, "params")
            _flat(given, "grads", list(map(_numel, params)))
            _dtypes(params, "params"), _dtypes(given, "grads")
            _all_on_device(params, given)
            filled = [p.data_ptr() for p in params if p.numel()]
            if len(set(filled)) != len(filled):
                raise ValueError("the same param is there twice")
        scale = None
        if self.max_norm is not None:
            fp8_grad_norm(given, self.max_norm, out=self.norm, clip_out=self._clip)
            scale = self._clip
        for a, b in moved:
            if self._counts[a] and self._words is not None:
                self._words[b].copy_(self._words[a])
            self._counts[b] = self._counts[a]
        self._groups = groups
        device = self._words is not None
        for g in active:
            inside = set(g)

            def pick(ts, other=self._none):
                if len(g) == len(ts):
                    return ts
                if self.state_bits == 32:
                    return [ts[i] for i in g]
                # 8-bit states are rounded by a tensor's place: those of other groups keep theirs
                return [t if i in inside else other for i, t in enumerate(ts)]

            fp8_adamw_step(pick(self.params), pick(grads), pick(self.exp_avg), pick(self.exp_avg_sq),
                           self._words[g[0]] if device else self._counts[g[0]] + 1, self.lr_word if device else self.lr,
                           self.betas, self.eps, pick(self.weight_decay, 0.0), pick(self.masters, None),
                           pick(self.exp_avg_scale, None), pick(self.exp_avg_sq_scale, None), scale, self.seed)
            if device and torch.cuda.is_current_stream_capturing():
                self._captured.add(g[0])
            for i in g:
                self._counts[i] += 1

    def sync_masters(self) -> None:
        """Take the masters from the params anew (after a param was loaded or set)."""
        for p, m in zip(self.params, self.masters):
            if m is not None:
                m.copy_(p.detach())

    def state_dict(self) -> dict:
        counts = list(self._counts)
        if self._words is not None:
            words = self._words[:, 0].tolist()
            for g in self._groups:
                for i in g:
                    counts[i] = words[g[0]]
        return {"steps": max(counts), "param_steps": counts, "masters": self.masters, "exp_avg": self.exp_avg,
                "exp_avg_sq": self.exp_avg_sq, "exp_avg_scale": self.exp_avg_scale,
                "exp_avg_sq_scale": self.exp_avg_sq_scale}

    def load_state_dict(self, state: dict) -> None:
        """Fill the states from another optimizer's over the same params (same
        state_bits and masters), in place.  A state without "param_steps" has one
        count, "steps", for all."""
        for name in ("masters", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
            mine, theirs = getattr(self, name), state[name]
            if [None if t is None else (t.numel(), t.dtype) for t in mine] != \
                    [None if t is None else (t.numel(), t.dtype) for t in theirs]:
                raise ValueError(f"the state's {name} do not fit these params")
        counts = [int(c) for c in state.get("param_steps", [state["steps"]] * len(self.params))]
        if len(counts) != len(self.params):
            raise ValueError("the state's param_steps do not fit these params")
        self._regroup(counts)  # refuses what it refuses before anything is written
        for name in ("masters", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
            for a, b in zip(getattr(self, name), state[name]):
                if a is not None:
                    a.copy_(b.reshape(a.shape))
        self._set_counts(counts)
