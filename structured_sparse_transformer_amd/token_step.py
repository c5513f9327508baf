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
"""
from __future__ import annotations

import torch

from . import sp24
from .ffn import SparseGegluFFN
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


if __name__ == "__main__":
    for k, loss in enumerate(train()):
        if k % 10 == 0 or k == 59:
            print(f"step {k:3d}  mean square error {loss:.4f}")
