"""Timed cases of the operators around the 2:4 FFN step: the token embedding
that makes the layer's input, its gradient, the orthogonalisation of a weight
update by Newton-Schulz products, and the optimiser step built on it.

A case is a dict of plain values.  `run` computes it in its plain form
(elementary torch operations in 32 bits, rounded once at the end) while `own`
is false, and through the library's entry points while it is true.

  embed_fwd   out[t] = scale * table[ids[t]], fp16 [T, d]; ids outside [0, V)
              (padding) give zero rows
  embed_bwd   dtable[v] (+)= scale * sum over t with ids[t] == v of dout[t],
              fp32 [V, d]
  ortho       X_0 = G / (|G|_F + eps);  A = X X^T, X <- a X + (b A + c A^2) X,
              `steps` times.  fp16 results, or fp32 ones that are held to
              fp32 accuracy
  muon        M <- mu M + G, X = orthogonalised G + mu M, P <- (1 - lr wd) P - lr X,
              W = fp16(P), for all the weights of one layer in one call
"""
import math

import numpy as np
import torch

own = False

A, B, C = 3.4445, -4.7750, 2.0315   # the usual quintic: pulls singular values into about [0.7, 1.2]
EPS = 1e-7
MU, DECAY = 0.95, 0.1
DEV = "cuda"


def listed():
    return [
        # one token of a decoder's step: launch latency alone
        {"name": "embed_fwd one token", "op": "embed_fwd", "T": 1, "V": 50257, "d": 1600, "table": "f16", "ids": "i64", "scale": 1.0},
        # a training batch's tokens from the fp32 master table, scaled
        {"name": "embed_fwd batch fp32 table", "op": "embed_fwd", "T": 16384, "V": 50257, "d": 1600, "table": "f32", "ids": "i64", "scale": 40.0},
        # a small vocabulary and an odd width: rows that no vector load is aligned to
        {"name": "embed_bwd small odd", "op": "embed_bwd", "T": 517, "V": 1003, "d": 67, "ids": "i32", "scale": 1.0, "accumulate": False},
        # the training batch's dense gradient: most rows of the table are zeros
        {"name": "embed_bwd batch", "op": "embed_bwd", "T": 16384, "V": 50257, "d": 1600, "ids": "i64", "scale": 1.0, "accumulate": False},
        # a long batch added to the gradient that a tied output layer has left there
        {"name": "embed_bwd long accumulate", "op": "embed_bwd", "T": 131072, "V": 50257, "d": 1024, "ids": "i64", "scale": 1.0, "accumulate": True},
        # the smallest weight of the tests: latency of the chain of products
        {"name": "ortho 64x64", "op": "ortho", "shapes": "64x64", "g": "f16", "out": "f16", "steps": 5},
        # an odd, tall update in fp32 throughout
        {"name": "ortho 1001x357 fp32", "op": "ortho", "shapes": "1001x357", "g": "f32", "out": "f32", "steps": 5},
        # one FFN weight of the widest layer
        {"name": "ortho 1600x6400", "op": "ortho", "shapes": "1600x6400", "g": "f32", "out": "f16", "steps": 5},
        # both weights of the 1024-wide layer, held to fp32 accuracy
        {"name": "ortho 4096x1024+1024x4096 fp32", "op": "ortho", "shapes": "4096x1024,1024x4096", "g": "f32", "out": "f32", "steps": 5},
        # both weights of a small layer
        {"name": "muon 256x64+64x256", "op": "muon", "shapes": "256x64,64x256", "lr": 3e-4, "steps": 5},
        # the gated layer of the 1600-wide model: W1 holds values and gates
        {"name": "muon 3200x1600+1600x1600", "op": "muon", "shapes": "3200x1600,1600x1600", "lr": 3e-4, "steps": 5},
        # the widest layer's both weights: the largest case
        {"name": "muon 6400x1600+1600x6400", "op": "muon", "shapes": "6400x1600,1600x6400", "lr": 2e-4, "steps": 5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "ortho", "muon"])
    if op.startswith("embed"):
        case = {"op": op, "T": _log_int(rng, 1 if op == "embed_fwd" else 64, 65536), "V": _log_int(rng, 300, 60000),
                "d": _log_int(rng, 32, 2048), "ids": rng.choice(["i32", "i64"]), "scale": rng.choice([1.0, 0.5, 32.0])}
        if rng.random() < 0.7:
            case["d"] = -(-case["d"] // 16) * 16
        if op == "embed_fwd":
            case["table"] = rng.choice(["f16", "f32"])
        else:
            case["accumulate"] = rng.choice([False, True])
        return case
    mult = rng.choice([1, 16, 64])   # weights of the 2:4 path are multiples of 16; others (heads, odd test sizes) are not

    def shape():
        r, c = (-(-_log_int(rng, 48, 2560) // mult) * mult for _ in range(2))
        return "%dx%d" % (r, c)

    steps = rng.choice([4, 5, 5, 6])
    if op == "ortho":
        return {"op": op, "shapes": ",".join(shape() for _ in range(rng.choice([1, 1, 2, 3]))), "g": rng.choice(["f16", "f32"]),
                "out": rng.choice(["f16", "f16", "f32"]), "steps": steps}
    r, c = shape().split("x")
    return {"op": op, "shapes": "%sx%s,%sx%s" % (r, c, c, r), "lr": rng.choice([1e-4, 2e-4, 3e-4]), "steps": steps}


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def work(case):
    if case["op"] == "embed_fwd":
        T, d = case["T"], case["d"]
        rows = _distinct(T, case["V"])
        return {"bytes": T * (4 if case["ids"] == "i32" else 8) + rows * d * (2 if case["table"] == "f16" else 4) + T * d * 2,
                "flops": T * d}
    if case["op"] == "embed_bwd":
        T, V, d = case["T"], case["V"], case["d"]
        rows = 2 * _distinct(T, V) if case["accumulate"] else V   # read and written, or all written
        return {"bytes": T * (4 if case["ids"] == "i32" else 8) + T * d * 2 + rows * d * 4, "flops": T * d}
    bytes_, flops = 0, 0
    for r, c in _shapes(case):
        m, n = min(r, c), max(r, c)
        # A and A^2 are symmetric: half of each product
        flops += case["steps"] * (m * m * n + m * m * m + 2 * m * m * n)
        if case["op"] == "ortho":
            bytes_ += r * c * ((2 if case["g"] == "f16" else 4) + (2 if case["out"] == "f16" else 4))
        else:
            bytes_ += r * c * (4 + 8 + 8 + 2)   # G read; M and P read and written; W written
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------ inputs

def _distinct(T, V):
    """Expected number of table rows that T of _ids()'s draws touch."""
    edges = np.log(np.arange(1, V + 2)) / math.log(V + 1)
    p = np.diff(edges)
    return int(np.sum(-np.expm1(T * np.log1p(-p))) + 0.5)


def _ids(gen, T, V, dtype):
    """Token ids whose frequencies fall as 1 / rank, as words' do; a thirtieth
    of a longer batch is padding (-1)."""
    u = torch.rand(T, generator=gen, device=DEV, dtype=torch.float64)
    ids = ((u * math.log(V + 1)).exp().floor().long() - 1).clamp_(0, V - 1)
    if T >= 30:
        ids[torch.randperm(T, generator=gen, device=DEV)[: T // 30]] = -1
    return ids.to(torch.int32 if dtype == "i32" else torch.int64)


def _update(gen, r, c):
    """A weight gradient: an eighth of the directions carry most of it, over a
    floor of noise."""
    k = max(1, min(r, c) // 8)
    low = torch.randn(r, k, generator=gen, device=DEV) @ torch.randn(k, c, generator=gen, device=DEV)
    return (low / math.sqrt(k) + 0.3 * torch.randn(r, c, generator=gen, device=DEV)) * 1e-3


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": case, "dtype": torch.float16 if case.get("out") == "f16" else torch.float32}
    if case["op"].startswith("embed"):
        T, V, d = case["T"], case["V"], case["d"]
        st["ids"] = _ids(gen, T, V, case["ids"])
        if case["op"] == "embed_fwd":
            st["table"] = (torch.randn(V, d, generator=gen, device=DEV) * 0.02).to(
                torch.float16 if case["table"] == "f16" else torch.float32)
        else:
            st["dout"] = torch.randn(T, d, generator=gen, device=DEV).half()
            if case["accumulate"]:
                st["dtable"] = torch.randn(V, d, generator=gen, device=DEV)
        return st
    st["G"] = [_update(gen, r, c) for r, c in _shapes(case)]
    if case["op"] == "ortho":
        st["G"] = [g.to(torch.float16 if case["g"] == "f16" else torch.float32) for g in st["G"]]
    else:
        st["M"] = [5 * _update(gen, r, c) for r, c in _shapes(case)]
        st["P"] = [0.02 * torch.randn(r, c, generator=gen, device=DEV) for r, c in _shapes(case)]
        st["W"] = [p.half() for p in st["P"]]
    return st


# ------------------------------------------------------------------ plain forms

def _lookup(ids, table, scale):
    real = (ids >= 0) & (ids < table.shape[0])
    rows = table[torch.where(real, ids, 0).long()].float() * scale
    return torch.where(real[:, None], rows, 0.0).half()


def _scatter(ids, dout, V, scale, dtable):
    real = (ids >= 0) & (ids < V)
    at = torch.where(real, ids, 0).long()
    rows = torch.where(real[:, None], dout.float() * scale, 0.0)
    if dtable is None:
        dtable = torch.zeros(V, dout.shape[1], dtype=torch.float32, device=dout.device)
    return dtable.index_add_(0, at, rows)


def _orthogonalise(G, steps):
    X = G.float()
    X = X / (X.square().sum().sqrt() + EPS)
    if G.shape[0] > G.shape[1]:
        X = X.t()
    for _ in range(steps):
        S = X @ X.t()
        X = A * X + (B * S + C * (S @ S)) @ X
    return X.t() if G.shape[0] > G.shape[1] else X


def _muon(G, M, P, W, lr, steps):
    M.mul_(MU).add_(G)
    X = _orthogonalise(G + MU * M, steps)
    P.mul_(1 - lr * DECAY).sub_(_rate(lr, P) * X)
    W.copy_(P)


def _rate(lr, P):
    """The step's size for a weight of this shape: updates of 0.2 lr in every entry's mean square."""
    return lr * 0.2 * math.sqrt(max(P.shape))


def run(state):
    case = state["case"]
    if own:
        return _run_own(state)
    if case["op"] == "embed_fwd":
        return _lookup(state["ids"], state["table"], case["scale"])
    if case["op"] == "embed_bwd":
        return _scatter(state["ids"], state["dout"], case["V"], case["scale"], state.get("dtable"))
    if case["op"] == "ortho":
        return [_orthogonalise(g, case["steps"]).to(state["dtype"]).contiguous() for g in state["G"]]
    for g, m, p, w in zip(state["G"], state["M"], state["P"], state["W"]):
        _muon(g, m, p, w, case["lr"], case["steps"])
    return {"M": state["M"], "P": state["P"], "W": state["W"]}


def _run_own(state):
    from structured_sparse_transformer_amd import sp24
    case = state["case"]
    if case["op"] == "embed_fwd":
        return sp24.sp24_embed_fwd(state["ids"], state["table"], case["scale"])
    if case["op"] == "embed_bwd":
        return sp24.sp24_embed_bwd(state["ids"], state["dout"], case["V"], case["scale"], dtable=state.get("dtable"),
                                   accumulate=case["accumulate"])
    if case["op"] == "ortho":
        return sp24.sp24_orthogonalize_batch(state["G"], steps=case["steps"], coeffs=(A, B, C), eps=EPS, dtype=state["dtype"])
    # lr scales the orthogonalised update, decay the weights: both as the step applies them
    sp24.sp24_muon_step(state["G"], state["M"], state["P"], state["W"], [_rate(case["lr"], p) for p in state["P"]],
                        decays=[case["lr"] * DECAY] * len(state["P"]), momentum=MU, nesterov=True, steps=case["steps"],
                        coeffs=(A, B, C), eps=EPS)
    return {"M": state["M"], "P": state["P"], "W": state["W"]}


# ------------------------------------------------------------------ 64 bits, from the definitions

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("embed"):
        V, d = case["V"], case["d"]
        ids = st["ids"].long()
        keep = torch.nonzero((ids >= 0) & (ids < V)).squeeze(1)
        if case["op"] == "embed_fwd":
            out = torch.zeros(len(ids), d, dtype=torch.float64, device=DEV)
            out[keep] = st["table"].double()[ids[keep]] * case["scale"]
            return out
        out = st["dtable"].double() if case["accumulate"] else torch.zeros(V, d, dtype=torch.float64, device=DEV)
        out.index_put_((ids[keep],), st["dout"][keep].double() * case["scale"], accumulate=True)
        return out

    def polar(U):
        # the step's odd polynomial on the short side's Gram matrix
        U = U.double()
        U = U / (torch.linalg.vector_norm(U) + EPS)
        wide = U.shape[0] <= U.shape[1]
        for _ in range(case["steps"]):
            S = torch.matmul(U, U.mT) if wide else torch.matmul(U.mT, U)
            Q = A * torch.eye(len(S), dtype=torch.float64, device=DEV) + torch.matmul(B * torch.eye(len(S), dtype=torch.float64, device=DEV) + C * S, S)
            U = torch.matmul(Q, U) if wide else torch.matmul(U, Q)
        return U

    if case["op"] == "ortho":
        return [polar(g) for g in st["G"]]
    out = {"M": [], "P": [], "W": []}
    for g, m, p in zip(st["G"], st["M"], st["P"]):
        m = MU * m.double() + g.double()
        p = (1 - case["lr"] * DECAY) * p.double() - case["lr"] * 0.2 * math.sqrt(max(p.shape)) * polar(g.double() + MU * m)
        out["M"].append(m)
        out["P"].append(p)
        out["W"].append(p)
    return out
