"""A training step from token ids to new weights: the token embedding, a gated
2:4-sparse FFN layer (ffn.py) and its optimiser (muon.py), in the library's
kernels; the table itself takes plain gradient descent, in torch.

    X = scale table[ids]                         sp24_embed_fwd
    Y = FFN(X)                                   SparseGegluFFN.forward
    dX, dW1, dW2 from dY                         SparseGegluFFN.backward
    dtable += scale sum over tokens of dX        sp24_embed_bwd
    new W1, W2                                   Muon, then refresh()
    table -= table_lr dtable, dtable = 0         torch, two passes over the dense table

``python -m structured_sparse_transformer_amd.token_step`` trains one such
layer to map tokens to the outputs of a fixed random one and prints its loss.

TokenMLP is the same step around the plain layer (SparseFFN), all of whose
parameters, the table's too, one call of AdamW (adamw.py) updates; ``python -m
structured_sparse_transformer_amd.token_step plain`` trains that one.
"""
from __future__ import annotations

import sys

import torch

from . import sp24
from .adamw import AdamW
from .ffn import SparseFFN, SparseGegluFFN
from .muon import Muon


class TokenFFN:
    """``table`` fp32 [V, d]; W1, W2 as SparseGegluFFN takes them.  The table's
    gradient is kept in ``dtable`` (a tied output layer would add its own to
    it) until ``update`` takes it."""

    def __init__(self, table: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, scale: float = 1.0, decay: float = 0.0,
                 **muon):
        if table.dim() != 2 or table.dtype != torch.float32 or table.shape[1] != W1.shape[1]:
            raise ValueError("the table must be float32 [V, d], d the layer's width")
        self.table, self.scale = table, float(scale)
        self.layer = SparseGegluFFN(W1, W2, decay)
        self.optimizer = Muon([W1, W2], **muon)
        self.dtable = torch.zeros_like(table)
        self.layer.refresh()

    def forward(self, ids: torch.Tensor):
        X = sp24.sp24_embed_fwd(ids, self.table, self.scale)
        return self.layer.forward(X)

    def backward(self, ids: torch.Tensor, dY: torch.Tensor, saved):
        dX, dW1, dW2 = self.layer.backward(dY, saved)
        sp24.sp24_embed_bwd(ids, dX, self.table.shape[0], self.scale, dtable=self.dtable, accumulate=True)
        return dW1, dW2

    def update(self, grads, table_lr: float) -> None:
        self.optimizer.step(grads)
        self.layer.refresh()
        self.table.add_(self.dtable, alpha=-table_lr)
        self.dtable.zero_()


class TokenMLP:
    """``table`` fp32 [V, d]; W1, b1, W2, b2 as SparseFFN takes them.  The fp32
    masters of W1 and W2 start as their values.  ``decay`` is of the unscaled
    gradients, whatever the loss scale.  ``adamw``: AdamW's arguments."""

    def __init__(self, table: torch.Tensor, W1: torch.Tensor, b1: torch.Tensor, W2: torch.Tensor, b2: torch.Tensor,
                 act: str = "gelu", scale: float = 1.0, decay: float = 0.0, **adamw):
        if table.dim() != 2 or table.dtype != torch.float32 or table.shape[1] != W1.shape[1]:
            raise ValueError("the table must be float32 [V, d], d the layer's width")
        self.table, self.scale = table, float(scale)
        self.layer = SparseFFN(W1, b1, W2, b2, act=act, decay=decay)
        # biases and the table take no weight decay
        weight_decay = adamw.pop("weight_decay", 0.01)
        self.optimizer = AdamW([table, W1.float(), b1, W2.float(), b2], [None, W1, None, W2, None],
                               weight_decay=[0.0, weight_decay, 0.0, weight_decay, 0.0], **adamw)
        self.layer.refresh()

    def forward(self, ids: torch.Tensor):
        X = sp24.sp24_embed_fwd(ids, self.table, self.scale)
        return self.layer.forward(X)

    def backward(self, ids: torch.Tensor, dY: torch.Tensor, saved):
        """The gradients of table, W1, b1, W2 and b2, of the loss as dY is: multiplied
        with the optimiser's loss_scale."""
        dX, *grads = self.layer.backward(dY, saved, self.optimizer.loss_scale)
        return [sp24.sp24_embed_bwd(ids, dX, self.table.shape[0], self.scale), *grads]

    def update(self, grads) -> None:
        self.optimizer.step(grads)
        self.layer.refresh()


def train(steps: int = 60, tokens: int = 4096, vocabulary: int = 1000, d: int = 128, hidden: int = 256, seed: int = 0):
    """Mean square errors, one a step, of learning a random layer's outputs."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    make = lambda: (rand(2 * hidden, d).mul_(d ** -0.5).half(), rand(d, hidden).mul_(hidden ** -0.5).half())  # noqa: E731
    table = rand(vocabulary, d)
    teacher, student = TokenFFN(table.clone(), *make()), TokenFFN(table, *make(), lr=0.03)
    losses = []
    for _ in range(steps):
        ids = torch.randint(0, vocabulary, (tokens,), generator=gen, device="cuda")
        want, _ = teacher.forward(ids)
        Y, saved = student.forward(ids)
        error = Y.float() - want.float()
        losses.append(error.square().mean())
        # the mean over tokens, times 2^10 so that fp16 keeps it
        dW1, dW2 = student.backward(ids, (error * (2.0 ** 10 / tokens)).half(), saved)
        student.update([dW1, dW2], table_lr=2.0 ** -10)
    return [float(v) for v in losses]


def train_plain(steps: int = 60, tokens: int = 4096, vocabulary: int = 1000, d: int = 128, hidden: int = 512,
                seed: int = 0, bits: int = 8):
    """As train(), for the plain layer: fp16 gradients of a loss scaled by 2^10."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    make = lambda: (rand(hidden, d).mul_(d ** -0.5).half(), rand(hidden).mul_(0.1),  # noqa: E731
                    rand(d, hidden).mul_(hidden ** -0.5).half(), rand(d).mul_(0.1))
    table = rand(vocabulary, d)
    teacher = TokenMLP(table.clone(), *make())
    student = TokenMLP(table, *make(), lr=1e-2, bits=bits, max_norm=1.0, loss_scale=2.0 ** 10)
    losses = []
    for _ in range(steps):
        ids = torch.randint(0, vocabulary, (tokens,), generator=gen, device="cuda")
        want, _ = teacher.forward(ids)
        Y, saved = student.forward(ids)
        error = Y.float() - want.float()
        losses.append(error.square().mean())
        student.update(student.backward(ids, (error * (2.0 ** 10 / tokens)).half(), saved))
    return [float(v) for v in losses]


if __name__ == "__main__":
    run = train_plain if sys.argv[1:] == ["plain"] else train
    for k, loss in enumerate(run()):
        if k % 10 == 0 or k == 59:
            print(f"step {k:3d}  mean square error {loss:.4f}")
