"""AdamW over all tensors of a model in one call, in the library's kernels
(sp24_grad_norm, sp24_adamw_step).

Per tensor: the fp32 values P, their states M and V, in 32 bits or in 8, and
optionally an fp16 copy W that the products take.  A step does, in place,

    g = G / loss_scale, clipped so that all gradients' norm is at most max_norm
    M <- b1 M + (1 - b1) g,   V <- b2 V + (1 - b2) g^2
    P <- (1 - lr weight_decay) P - lr (M / (1 - b1^t)) / (sqrt(V / (1 - b2^t)) + eps)
    W  = fp16(P)

All of G carries the loss scale, what was added to the loss's own gradient (a
layer's decay term) too.

With a loss scale or a largest norm, t and the gradients' factor stay in device
memory: a step whose gradients are not all finite is left out (and t with it)
without the host's waiting for it, and a captured step counts on as it is
replayed.  Without either, t is counted here and a step is not captured.

Everything else of a captured step is a constant of its graph: the learning rate
and the decay, betas, eps, the scale and the largest norm.  A replay after
``set_lr`` still takes the rate that it was captured with; capture it again.
"""
from __future__ import annotations

import warnings

import torch

from . import sp24


class AdamW:
    """``params``: fp32 tensors of any shapes, updated in place; ``copies``: their
    fp16 copies or None, each; ``weight_decay`` one number or one each; ``bits`` of
    the states, 32 or 8."""

    def __init__(self, params, copies=None, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01,
                 bits: int = 32, max_norm: float | None = None, loss_scale: float = 1.0, seed: int = 0):
        if bits not in (8, 32):
            raise ValueError("states are of 32 bits or of 8")
        # here and not in the call, which comes after the norm has counted the step
        if not all(0.0 <= b < 1.0 for b in betas) or not eps >= 0.0:
            raise ValueError("betas must be from 0 up to below 1, eps 0 or more")
        self.params = list(params)
        n = len(self.params)
        self.copies = [None] * n if copies is None else list(copies)
        self.betas, self.eps, self.seed = tuple(float(b) for b in betas), float(eps), int(seed)
        self.weight_decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else list(weight_decay)
        if bits == 32:
            self.states = [(torch.zeros_like(p), torch.zeros_like(p)) for p in self.params]
            exps = {}
        else:
            self.states = [(*sp24.state8(p), *sp24.state8(p)) for p in self.params]
            exps = {"M_exps": [s[1] for s in self.states], "V_exps": [s[3] for s in self.states]}
        self.plan = sp24.sp24_adamw_plan(self.params, [s[0] for s in self.states], [s[1 if bits == 32 else 2] for s in self.states],
                                         self.copies, lrs=lr, decays=[lr * w for w in self.weight_decay], **exps)
        self.max_norm, self.loss_scale = max_norm, float(loss_scale)
        self.guarded = max_norm is not None or self.loss_scale != 1.0
        self.steps = 0
        self._captured = False
        device = self.params[0].device if n else torch.device("cuda", torch.cuda.current_device())
        self.control = sp24.step_control(device) if self.guarded else None
        # the norm's parts: the same for every step
        sizes, at = sp24._int64s(self.plan.sizes)
        self._work = torch.empty(sp24.lib().sp24_grad_norm_workspace(at, n), dtype=torch.uint8, device=device) if self.guarded else None

    def set_lr(self, lr: float) -> None:
        """The learning rate of the steps from here on; those that were captured
        before keep theirs, which is warned of."""
        if self._captured:
            warnings.warn("a captured step keeps its learning rate when it is replayed: capture it again", RuntimeWarning, stacklevel=2)
            self._captured = False
        for job, w in zip(self.plan.jobs, self.weight_decay):
            job.lr, job.decay = lr, lr * w

    def step(self, grads) -> None:
        """One step with the gradients of all tensors, in their order and shapes
        (all fp32 or all fp16)."""
        # before any count goes on
        self.plan.check(grads, [g.numel() for g in grads])
        capturing = torch.cuda.is_current_stream_capturing()
        if not self.guarded:
            if capturing:
                raise RuntimeError("a captured step would replay its t: with a max_norm (infinity clips nothing) it counts on")
            sp24.sp24_adamw_step(self.plan, grads, self.betas, self.eps, step=self.steps + 1, seed=self.seed)
            self.steps += 1
            return
        sp24.sp24_grad_norm(grads, 1.0 / self.loss_scale, float("inf") if self.max_norm is None else self.max_norm,
                            control=self.control, workspace=self._work)
        sp24.sp24_adamw_step(self.plan, grads, self.betas, self.eps, control=self.control, seed=self.seed)
        self._captured |= capturing
