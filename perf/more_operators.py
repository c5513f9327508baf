"""Timed cases of the operators of a plain feed-forward layer's training step
and its serving: the 2:4 products with bias, activation and residual in their
epilogues, the bias gradient, and AdamW over many tensors at once with the
gradients' norm that it clips by.

A case is a dict of plain values.  `run` computes it in its plain form
(elementary torch operations in 32 bits, rounded once at the end) while `own`
is false, and through the library's entry points while it is true.  The plain
forms multiply by the pruned weight Ws as a dense matrix; the library takes
its 2:4 forms.

  fwd        U = X Ws^T + bias,  Y = act(U) + residual; U is kept for the
             backward where `keep` says so
  bwd        dU = (dY Ws) * act'(U), dbias = the sum of dU over tokens
  bias_grad  dbias = the sum of dY over tokens
  norm       the norm of all gradients together, what it leaves of them
             (factor), and the step's count unless some entry is not finite
  adamw      M <- b1 M + (1 - b1) g, V <- b2 V + (1 - b2) g^2,
             P <- (1 - lr wd) P - lr M / (1 - b1^t) / (sqrt(V / (1 - b2^t)) + eps),
             W = fp16(P), g = factor * G.  M and V in 32 bits, or in 8: groups
             of 64 entries share an exponent, M is held with 3 fraction bits
             and a sign, sqrt V with 4, both rounded at random by a hash of
             the seed, the step, the tensor's place and the entry's
"""
import itertools
import math

import numpy as np
import torch

own = False

B1, B2, EPS, DECAY = 0.9, 0.999, 1e-8, 0.1
DEV = "cuda"


def listed():
    return [
        # one token of a decoder's step through the widest layer's first linear: the weight's bytes and launch latency
        {"name": "fwd one token", "op": "fwd", "T": 1, "R": 6400, "C": 1600, "act": "gelu", "bias": True, "residual": False, "keep": False},
        # a batch of requests through the second linear, added to the residual stream
        {"name": "fwd 24 tokens residual", "op": "fwd", "T": 24, "R": 1600, "C": 6400, "act": "none", "bias": True, "residual": True, "keep": False},
        # the training batch's first linear, its pre-activation kept for the backward
        {"name": "fwd training batch", "op": "fwd", "T": 16384, "R": 6400, "C": 1600, "act": "gelu", "bias": True, "residual": False, "keep": True},
        # a short batch of odd length, backward through the 1024-wide layer's activation
        {"name": "bwd odd batch", "op": "bwd", "T": 1021, "R": 1024, "C": 4096, "act": "gelu_tanh"},
        # the training batch's backward through the activation: the largest product
        {"name": "bwd training batch", "op": "bwd", "T": 16384, "R": 1600, "C": 6400, "act": "gelu"},
        # an odd, short batch's bias gradient
        {"name": "bias_grad odd batch", "op": "bias_grad", "T": 517, "R": 1600},
        # the training batch's, at the hidden width
        {"name": "bias_grad training batch", "op": "bias_grad", "T": 16384, "R": 6400},
        # the biases of a 24-layer model, fp16 gradients: launch latency
        {"name": "norm 48 biases", "op": "norm", "shapes": "4096*24,1024*24", "g": "f16", "scale": 2.0 ** -10, "max": 1.0},
        # a layer's weights and biases
        {"name": "norm 1600-wide layer", "op": "norm", "shapes": "10240000*2,6400*1,1600*1", "g": "f32", "scale": 1.0, "max": 1.0},
        # the biases of the 24-layer model
        {"name": "adamw 48 biases", "op": "adamw", "shapes": "4096*24,1024*24", "g": "f32", "bits": 32, "copy": False, "t": 3, "control": False},
        # a layer's weights and biases, with fp16 copies for the products
        {"name": "adamw 1600-wide layer", "op": "adamw", "shapes": "10240000*2,6400*1,1600*1", "g": "f32", "bits": 32, "copy": True, "t": 1000, "control": True},
        # the token table, its states in 8 bits: the most bytes
        {"name": "adamw table 8 bits", "op": "adamw", "shapes": "80411200*1", "g": "f32", "bits": 8, "copy": False, "t": 100, "control": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bias_grad", "norm", "adamw", "adamw"])
    if op in ("fwd", "bwd"):
        # widths of the 2:4 path are multiples of 16; most of 64
        R, C = (-(-_log_int(rng, 64, 6400) // m) * m for m in (rng.choice([16, 64, 64]) for _ in range(2)))
        case = {"op": op, "T": _log_int(rng, 1 if op == "fwd" else 16, 16384), "R": R, "C": C}
        while case["T"] * R * C > 16384 * 6400 * 1600:
            case["T"] = case["T"] // 2 + 1
        if op == "bwd":
            return {**case, "act": rng.choice(["gelu", "gelu_tanh", "relu", "relu2", "silu"])}
        return {**case, "act": rng.choice(["none", "gelu", "gelu_tanh", "relu", "relu2", "silu"]), "bias": rng.random() < 0.8,
                "residual": rng.random() < 0.4, "keep": rng.random() < 0.4}
    if op == "bias_grad":
        return {"op": op, "T": _log_int(rng, 1, 16384), "R": 16 * _log_int(rng, 4, 400)}
    sizes, left = [], 40_000_000
    for _ in range(rng.choice([1, 2, 5, 60])):
        n = min(_log_int(rng, 1, 12_000_000 if len(sizes) < 8 else 20_000), left)
        if n:
            sizes.append("%d*1" % n)
            left -= n
    case = {"op": op, "shapes": ",".join(sizes), "g": rng.choice(["f32", "f32", "f16"])}
    if op == "norm":
        return {**case, "scale": rng.choice([1.0, 2.0 ** -10, 2.0 ** -13]), "max": rng.choice([0.1, 1.0, 1e6])}
    return {**case, "bits": rng.choice([32, 8]), "copy": rng.random() < 0.5, "t": _log_int(rng, 1, 100_000), "control": rng.random() < 0.5}


def _sizes(case):
    pairs = (s.split("*") for s in case["shapes"].split(","))
    return [int(n) for n, k in pairs for _ in range(int(k))]


def work(case):
    if case["op"] in ("fwd", "bwd"):
        T, R, C = case["T"], case["R"], case["C"]
        weight = R * C + R * C // 8                      # two fp16 values of four, 16 index bits of sixteen
        if case["op"] == "fwd":
            rows = 1 + case["residual"] + case["keep"]
            bytes_ = 2 * T * C + weight + 2 * T * R * rows + 4 * R * case["bias"]
        else:
            bytes_ = 2 * T * R + weight + 2 * T * C * 2 + 4 * C
        return {"bytes": bytes_, "flops": T * R * C}     # of the kept products
    if case["op"] == "bias_grad":
        return {"bytes": 2 * case["T"] * case["R"] + 4 * case["R"], "flops": case["T"] * case["R"]}
    n, g = sum(_sizes(case)), 2 if case["g"] == "f16" else 4
    if case["op"] == "norm":
        return {"bytes": n * g, "flops": 2 * n}
    # P, M and V read and written; what an 8-bit state stands for is written out as values
    state = 16 if case["bits"] == 32 else 4 + 4 / 64 + 4
    return {"bytes": int(n * (g + 8 + state + 2 * case["copy"])), "flops": 15 * n}


# ------------------------------------------------------------------ inputs

def _patterns():
    """The 90 masks of a 4 x 4 block with two entries kept in every row and
    column, in the order of their rows' pairs, as [90, 16]."""
    pairs = list(itertools.combinations(range(4), 2))
    rows = [[float(c in p) for c in range(4)] for p in pairs]
    kept = [sum((rows[k] for k in ks), []) for ks in itertools.product(range(6), repeat=4)
            if all(sum(rows[k][c] for k in ks) == 2 for c in range(4))]
    return torch.tensor(kept, device=DEV)


def _mask(W):
    """The best of the 90 masks for every block of |W|, as [R, C]."""
    R, C = W.shape
    blocks = W.float().abs().reshape(R // 4, 4, C // 4, 4).transpose(1, 2).reshape(-1, 16)
    P = _patterns()
    keep = P[(blocks @ P.t()).argmax(1)]
    return keep.reshape(R // 4, C // 4, 4, 4).transpose(1, 2).reshape(R, C) > 0


def _blocked(x, width):
    """The library's order of a 2:4 form: bands of 64 rows, each band's blocks
    of `width` columns one after the other."""
    n, m = x.shape
    whole, parts = m // width * width, []
    for band in (x[: n // 64 * 64].reshape(-1, 64, m), x[n // 64 * 64:][None]):
        if band.numel():
            k, h, _ = band.shape
            full = band[:, :, :whole].reshape(k, h, whole // width, width).transpose(1, 2).reshape(k, -1)
            parts.append(torch.cat([full, band[:, :, whole:].reshape(k, -1)], 1).reshape(-1))
    return torch.cat(parts).reshape(n, m).contiguous()


def _form(W, keep):
    """The 2:4 row form of W's kept entries: their values, and 16-bit words of
    four groups' index pairs."""
    n, m = W.shape
    at = keep.reshape(n, m // 4, 4).to(torch.int8)
    i0 = at.argmax(2)
    i1 = 3 - at.flip(2).argmax(2)
    vals = torch.stack([W.reshape(n, m // 4, 4).gather(2, i[..., None])[..., 0] for i in (i0, i1)], 2).reshape(n, m // 2)
    nibbles = (i0 | i1 << 2).reshape(n, m // 16, 4)
    words = sum(nibbles[:, :, j] << (4 * j) for j in range(4))
    words = torch.where(words >= 1 << 15, words - (1 << 16), words).to(torch.int16)
    return _blocked(vals, 32), _blocked(words, 4)


def _spans(case):
    """Where the tensors lie in buffers that hold them all, each from a multiple
    of 64 entries on, and the buffers' length."""
    starts = np.cumsum([0] + [-(-n // 64) * 64 for n in _sizes(case)]).tolist()
    return starts[:-1], starts[-1]


def _views(flat, case):
    return [flat[a: a + n] for a, n in zip(_spans(case)[0], _sizes(case))]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    st = {"case": case}
    if case["op"] == "bias_grad":
        st["dY"] = (rand(case["T"], case["R"]) + 0.1 * rand(case["R"])).half()
        return st
    if case["op"] in ("fwd", "bwd"):
        T, R, C = case["T"], case["R"], case["C"]
        W = (rand(R, C) / math.sqrt(C / 2)).half()       # pre-activations of about unit size
        keep = _mask(W)
        st["Ws"] = torch.where(keep, W, 0)
        if case["op"] == "fwd":
            st["forms"] = _form(W, keep)
            st["X"] = rand(T, C).half()
            st["bias"] = 0.1 * rand(R) if case["bias"] else None
            st["residual"] = rand(T, R).half() if case["residual"] else None
        else:
            st["forms"] = _form(W.t().contiguous(), keep.t().contiguous())
            st["dY"] = (rand(T, R) + 0.1 * rand(R)).half()
            st["U"] = rand(T, C).half()
        return st
    sizes, (_, total) = _sizes(case), _spans(case)
    # gradients that fp16 holds, their size from tensor to tensor apart; zeros between the tensors
    own_size = (rand(len(sizes)).clamp_(-2, 2) * 0.5).exp()
    size = torch.zeros(total, device=DEV)
    for view, s in zip(_views(size, case), own_size):
        view.fill_(0.01 * s)
    st["G"] = (rand(total) * size).to(torch.float16 if case["g"] == "f16" else torch.float32)
    st["Gs"] = _views(st["G"], case)
    st["control"] = torch.zeros(8, dtype=torch.int32, device=DEV)
    if case["op"] == "norm":
        return st
    if case["control"]:
        # as a call of the norm leaves it: the step's count and the gradients' factor
        st["control"].view(torch.int64)[0] = case["t"]
        st["control"].view(torch.float32)[3] = 0.5
    st["P"] = rand(total) * 0.02 * (size > 0)
    st["W"] = st["P"].half() if case["copy"] else None
    M = rand(total) * 0.3 * size
    root = size * (0.2 + 0.05 * rand(total).abs())
    if case["bits"] == 8:
        st["M"], st["ME"] = _held(M, 3)
        st["V"], st["VE"] = _held(root, 4)
    else:
        st["M"], st["V"] = M, root.square()
    for k in ("P", "W", "M", "V"):
        st[k + "s"] = _views(st[k], case) if st[k] is not None else [None] * len(sizes)
    if case["bits"] == 8:
        for k in ("ME", "VE"):
            st[k + "s"] = [st[k][a // 64: -(-(a + n) // 64)] for a, n in zip(_spans(case)[0], sizes)]
    st["lr"], st["seed"] = 1e-3, seed & 0x7FFFFFFF
    if own:   # the plan of the tensors, which an optimiser keeps
        from structured_sparse_transformer_amd import sp24
        eight = {"M_exps": st["MEs"], "V_exps": st["VEs"]} if case["bits"] == 8 else {}
        st["plan"] = sp24.sp24_adamw_plan(st["Ps"], st["Ms"], st["Vs"], st["Ws"], lrs=st["lr"], decays=st["lr"] * DECAY, **eight)
    return st


# ------------------------------------------------------------------ plain forms

def _logistic(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _act(name, u):
    if name == "none":
        return u
    if name == "relu":
        return torch.where(u < 0, 0.0, u)
    if name == "relu2":
        return torch.where(u < 0, 0.0, u * u)
    if name == "gelu":
        return 0.5 * u * torch.erfc(u * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return u * _logistic(2.0 * math.sqrt(2.0 / math.pi) * (u + 0.044715 * u * u * u))
    return u * _logistic(u)


def _slope(name, u):
    if name == "relu":
        return torch.where(u > 0, 1.0, 0.0)
    if name == "relu2":
        return torch.where(u > 0, 2.0 * u, 0.0)
    if name == "gelu":
        return 0.5 * torch.erfc(u * -math.sqrt(0.5)) + u * torch.exp(-0.5 * u * u) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        k = 2.0 * math.sqrt(2.0 / math.pi)
        s = _logistic(k * (u + 0.044715 * u * u * u))
        return s + u * s * (1.0 - s) * k * (1.0 + 3.0 * 0.044715 * u * u)
    s = _logistic(u)
    return s + u * s * (1.0 - s)


def _fwd(st):
    U = st["X"].float() @ st["Ws"].float().t()
    if st["bias"] is not None:
        U = U + st["bias"]
    Y = _act(st["case"]["act"], U)
    if st["residual"] is not None:
        Y = Y + st["residual"].float()
    return {"Y": Y.half(), "U": U.half() if st["case"]["keep"] else None}


def _bwd(st):
    dU = (st["dY"].float() @ st["Ws"].float()) * _slope(st["case"]["act"], st["U"].float())
    return {"dU": dU.half(), "dbias": dU.sum(0)}


def _norm(st):
    case, control = st["case"], st["control"]
    norm = st["G"].double().square().sum().sqrt() * case["scale"]
    fine = torch.isfinite(norm)
    factor = torch.where(fine, case["scale"] * torch.clamp(case["max"] / norm, max=1.0), 0.0)
    control.view(torch.int64)[0] += fine
    control.view(torch.float32)[2] = norm.float()
    control.view(torch.float32)[3] = factor.float()
    control[4] = ~fine
    return _control(control)


def _control(control):
    return {"t": control.view(torch.int64)[0], "norm": control.view(torch.float32)[2], "factor": control.view(torch.float32)[3],
            "skip": control[4]}


def _mix(x):
    """A 32-bit hash of 32-bit values, held in 64 bits (the multipliers are the
    roots of 2 and 3, their fractions' first bits)."""
    x = (x ^ x >> 16) * 0x6A09E667 & 0xFFFFFFFF
    x = (x ^ x >> 15) * 0xBB67AE85 & 0xFFFFFFFF
    return x ^ x >> 16


def _random(case, seed, t):
    """32 random bits for each entry, by its place in its tensor and the
    tensor's among all."""
    starts, total = _spans(case)
    starts = torch.tensor(starts, device=DEV) // 64
    group = torch.arange(total // 64, device=DEV)
    place = torch.bucketize(group, starts, right=True) - 1
    keys = _mix(_mix(_mix(t & 0xFFFFFFFF) ^ seed) ^ place)
    entry = (group - starts[place])[:, None] * 64 + torch.arange(64, device=DEV)
    return _mix(entry ^ keys[:, None]).view(-1)


def _scaled(x, E):
    """x 2^E for groups of 64 entries; the power itself may be out of 32 bits' range."""
    return (x.view(-1, 64).double() * torch.exp2(E.double())[:, None]).float().view(-1)


def _values(code, E, fraction):
    """The entries that an 8-bit state stands for: M's, or the roots of V's."""
    code = code.int()
    y = ((code & 127 if fraction == 3 else code) << (23 - fraction)).view(torch.float32)
    x = _scaled(y, E.int() - 15)
    return torch.where(code > 127, -x, x) if fraction == 3 else x


def _held(x, fraction, bits=None):
    """Entries in 8 bits with their groups' exponents, rounded to nearest, or up
    or down at random as `bits` has it.  A root above zero stays above it."""
    shift = 23 - fraction
    E = (x.view(-1, 64).abs().amax(1).view(torch.int32) + (1 << shift) - 1) >> 23
    y = _scaled(x.abs(), 15 - E).view(torch.int32)
    more = (1 << (shift - 1)) - 1 + (y >> shift & 1) if bits is None else ((bits << (shift - 16)) + (1 << (shift - 17))).int()
    code = (y + more) >> shift
    code = code | (x < 0).int() << 7 if fraction == 3 else torch.where(x > 0, code.clamp(min=1), code)
    return code.to(torch.uint8), E.to(torch.uint8)


def _adamw(st):
    case, control = st["case"], st["control"]
    t = control.view(torch.int64)[0] if case["control"] else torch.tensor(case["t"], device=DEV)
    g = st["G"].float() * control.view(torch.float32)[3] if case["control"] else st["G"].float()
    c1, c2 = -torch.expm1(t * math.log(B1)), -torch.expm1(t * math.log(B2))
    eight = case["bits"] == 8
    m = (_values(st["M"], st["ME"], 3) if eight else st["M"]) * B1 + g * (1.0 - B1)
    v = (_values(st["V"], st["VE"], 4).square() if eight else st["V"]) * B2 + g * g * (1.0 - B2)
    r = v.sqrt()
    st["P"].mul_(1.0 - st["lr"] * DECAY).sub_(st["lr"] / c1 * m / (r * torch.rsqrt(c2) + EPS))
    if case["copy"]:
        st["W"].copy_(st["P"])
    out = {"P": st["P"], "W": st["W"]}
    if not eight:
        st["M"].copy_(m)
        st["V"].copy_(v)
        return {**out, "M": st["M"], "V": st["V"]}
    bits = _random(case, st["seed"], t)
    for k, x, low, fraction in (("M", m, bits & 0xFFFF, 3), ("V", r, bits >> 16, 4)):
        code, E = _held(x, fraction, low)
        st[k].copy_(code)
        st[k + "E"].copy_(E)
        # bfloat16 holds such values whole
        out["M" if k == "M" else "root V"] = _values(code, E, fraction).bfloat16()
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"fwd": _fwd, "bwd": _bwd, "bias_grad": lambda s: s["dY"].float().sum(0), "norm": _norm, "adamw": _adamw}[state["case"]["op"]](state)


def _run_own(st):
    from structured_sparse_transformer_amd import sp24
    case = st["case"]
    if case["op"] == "fwd":
        Y, U = sp24.sp24_spmm_fwd_act(st["X"], *st["forms"], case["R"], case["C"], act=case["act"], bias=st["bias"],
                                      residual=st["residual"], U=case["keep"])
        return {"Y": Y, "U": U}
    if case["op"] == "bwd":
        dU, dbias = sp24.sp24_spmm_bwd_input_act(st["dY"], *st["forms"], case["R"], case["C"], st["U"], act=case["act"])
        return {"dU": dU, "dbias": dbias}
    if case["op"] == "bias_grad":
        return sp24.sp24_bias_grad(st["dY"])
    if case["op"] == "norm":
        return _control(sp24.sp24_grad_norm(st["Gs"], scale=case["scale"], max_norm=case["max"], control=st["control"]))
    at = {"control": st["control"]} if case["control"] else {"step": case["t"]}
    sp24.sp24_adamw_step(st["plan"], st["Gs"], betas=(B1, B2), eps=EPS, seed=st["seed"], **at)
    out = {"P": st["P"], "W": st["W"]}
    if case["bits"] == 32:
        return {**out, "M": st["M"], "V": st["V"]}
    return {**out, "M": sp24.sp24_state8_values(st["M"], st["ME"], dtype=torch.bfloat16),
            "root V": sp24.sp24_state8_values(st["V"], st["VE"], root=True, dtype=torch.bfloat16)}


# ------------------------------------------------------------------ 64 bits, from the definitions

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "bias_grad":
        return torch.ones(case["T"], dtype=torch.float64, device=DEV) @ st["dY"].double()
    if op in ("fwd", "bwd"):
        def phi(u):   # the normal distribution's function
            return 0.5 * (1 + torch.erf(u / math.sqrt(2)))

        def f(u):
            if case["act"] == "gelu_tanh":
                return 0.5 * u * (1 + torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
            return {"none": lambda: u, "relu": lambda: torch.relu(u), "relu2": lambda: torch.relu(u) ** 2,
                    "gelu": lambda: torch.where(u > -5, u * phi(u), u * torch.erfc(-u / math.sqrt(2)) / 2),
                    "silu": lambda: u * torch.sigmoid(u)}[case["act"]]()
        if op == "fwd":
            U = torch.matmul(st["X"].double(), st["Ws"].double().mT) + (0 if st["bias"] is None else st["bias"].double())
            return {"Y": f(U) + (0 if st["residual"] is None else st["residual"].double()), "U": U if case["keep"] else None}
        with torch.enable_grad():
            U = st["U"].double().requires_grad_()
            slope, = torch.autograd.grad(f(U).sum(), U)
        dU = torch.matmul(st["dY"].double(), st["Ws"].double()) * slope
        return {"dU": dU, "dbias": torch.ones(len(dU), dtype=torch.float64, device=DEV) @ dU}
    if op == "norm":
        norm = case["scale"] * math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in st["Gs"]))
        as64 = lambda v: torch.tensor(v, dtype=torch.float64, device=DEV)  # noqa: E731
        return {"t": None, "norm": as64(norm), "factor": as64(case["scale"] * min(1.0, case["max"] / norm)), "skip": None}
    eight, g = case["bits"] == 8, st["G"].double() * (0.5 if case["control"] else 1.0)

    def read(code, E, fraction):
        # a sign, four bits of the power of two and the fraction's
        code, E = code.long(), E.long().repeat_interleave(64)
        size = code % 128 if fraction == 3 else code
        power, part = size >> fraction, (size % (1 << fraction)).double() / (1 << fraction)
        x = torch.where(power > 0, 1 + part, part) * torch.exp2((E - 127 - 15 + power.clamp(min=1)).double())
        return torch.where((code > 127) & (fraction == 3), -x, x)

    def rounded(x, u, fraction):
        # whole numbers of steps: 2^-fraction of the entry's power of two, or of the least that its group holds
        a = x.abs()
        top = a.view(-1, 64).amax(1)
        q = torch.exp2(torch.floor(torch.log2(top)) - fraction)
        top = torch.floor(torch.log2(torch.ceil(top / q) * q)).repeat_interleave(64)
        step = torch.exp2(torch.maximum(torch.floor(torch.log2(a)), top - 14) - fraction)
        y = torch.floor(a / step + (u + 0.5) / 65536) * step
        y = torch.where((y > 0) | (fraction == 3), y, torch.exp2(top - 14 - fraction))
        return torch.where(a > 0, torch.copysign(y, x), 0.0)

    m = B1 * (read(st["M"], st["ME"], 3) if eight else st["M"].double()) + (1 - B1) * g
    v = B2 * (read(st["V"], st["VE"], 4) ** 2 if eight else st["V"].double()) + (1 - B2) * g ** 2
    p = st["P"].double() * (1 - st["lr"] * DECAY) - st["lr"] * (m / (1 - B1 ** case["t"])) / ((v / (1 - B2 ** case["t"])) ** 0.5 + EPS)
    out = {"P": p, "W": p if case["copy"] else None}
    if not eight:
        return {**out, "M": m, "V": v}
    bits = _random(case, st["seed"], torch.tensor(case["t"], device=DEV))
    return {**out, "M": rounded(m, bits & 0xFFFF, 3), "root V": rounded(v ** 0.5, bits >> 16, 4)}
