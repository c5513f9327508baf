"""The optimiser step of the 2:4 layers' dense weights: momentum and updates
orthogonalised by Newton-Schulz products, all in the library's kernels
(sp24_muon_step).

Per weight: the fp32 master P, its momentum M, and the fp16 copy W that the
layer searches, compresses and multiplies.  A step takes the weights' fp32
gradients (sp24_weight_grad's) and does, in place,

    M <- momentum M + G,   U = G + momentum M (or M)
    P <- (1 - lr weight_decay) P - lr 0.2 sqrt(max(R, C)) orthogonalise(U)
    W  = fp16(P)

The factor makes an update's entries 0.2 lr in the mean square whatever the
weight's shape, so that a learning rate and a weight decay suit weights of all
shapes.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import sp24


class Muon:
    """``weights``: the fp16 weights of the layers, updated in place; the
    masters start as their values unless given.  ``precise=False`` orthogonalises
    with products of fp16 operands, a third of the matrix work."""

    def __init__(self, weights, masters=None, lr: float = 3e-4, momentum: float = 0.95, weight_decay: float = 0.0,
                 nesterov: bool = True, steps: int = 5, coeffs=None, precise: bool = True):
        self.weights = list(weights)
        self.masters = [w.float() for w in self.weights] if masters is None else list(masters)
        self.momenta = [torch.zeros_like(p) for p in self.masters]
        self.lr, self.momentum, self.weight_decay = lr, momentum, weight_decay
        self.nesterov, self.steps, self.coeffs, self.precise = nesterov, steps, coeffs, precise
        self._workspace = None

    def _groups(self):
        """Up to 8 weights a call, in order."""
        n = len(self.weights)
        return [range(k, min(n, k + sp24.MAX_BATCH)) for k in range(0, n, sp24.MAX_BATCH)]

    def _work(self, device):
        """One workspace for all groups: they run one after the other."""
        if self._workspace is None:
            need = 0
            for group in self._groups():
                jobs = (sp24.MuonJob * len(group))(*[sp24.MuonJob(R=self.masters[k].shape[0], C=self.masters[k].shape[1])
                                                     for k in group])
                need = max(need, sp24.lib().sp24_muon_workspace(ctypes.cast(jobs, ctypes.c_void_p), len(group)))
            self._workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return self._workspace

    def _check(self, grads):
        """What a call refuses, for all of them before the first: otherwise the
        weights of earlier calls would have taken the step."""
        for g, m, p, w in zip(grads, self.momenta, self.masters, self.weights):
            for t, dtype, name in ((g, torch.float32, "the gradient"), (m, torch.float32, "the momentum"),
                                   (p, torch.float32, "the weight"), (w, torch.float16, "the float16 weight")):
                sp24._need(t, p.shape, dtype, name)
                sp24._ptr(t)
                if t.data_ptr() % 16:
                    raise ValueError(f"{name} must be 16-byte aligned")

    def step(self, grads) -> None:
        """One step with the gradients of all weights, in their order."""
        if len(grads) != len(self.weights):
            raise ValueError("one gradient per weight")
        groups = self._groups()
        if len(groups) > 1:
            self._check(grads)
        for group in groups:
            sp24.sp24_muon_step(
                [grads[k] for k in group], [self.momenta[k] for k in group], [self.masters[k] for k in group],
                [self.weights[k] for k in group],
                [self.lr * 0.2 * math.sqrt(max(self.masters[k].shape)) for k in group],
                decays=[self.lr * self.weight_decay] * len(group), momentum=self.momentum, nesterov=self.nesterov,
                steps=self.steps, coeffs=self.coeffs, precise=self.precise, workspace=self._work(grads[0].device))
