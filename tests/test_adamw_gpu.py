"""GPU checks of the gradients' norm and of AdamW over many tensors, in 32 and
in 8 bits.

32 bits: against the formulas in float64.  M is a sum of two products: 3
roundings of the larger's magnitude, 2^-24 each; V has one more; P's update
divides M by the root, whose errors are at most 16 roundings' together.
8 bits: the state after a step, decoded here, has to be one of the two held
values around the exact state (or a rounding error off, at a border), the mean
over many entries has to come out unbiased, and with the library's hash written
out here the codes have to be the very ones.
"""
import math

import pytest

from gpu_checks import Guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
U32 = 2.0 ** -24
SIZES = [1, 3, 64, 65, 1600, 4095, 4096, 4097, 70001]


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def decode(codes, exps, fraction):
    code, E = codes.long(), exps.long().repeat_interleave(64)[: codes.numel()]
    size = code % 128 if fraction == 3 else code
    power, part = size >> fraction, (size % (1 << fraction)).double() / (1 << fraction)
    x = torch.where(power > 0, 1 + part, part) * torch.exp2((E - 142 + power.clamp(min=1)).double())
    return torch.where((code > 127) & (fraction == 3), -x, x)


def mix(x):
    x = (x ^ x >> 16) * 0x6A09E667 & 0xFFFFFFFF
    x = (x ^ x >> 15) * 0xBB67AE85 & 0xFFFFFFFF
    return x ^ x >> 16


def hash_bits(seed, t, place, n):
    return mix(torch.arange(n, device="cuda") ^ mix(mix(mix(t) ^ seed) ^ place))


# ------------------------------------------------------------------ the norm

@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 16384], [16385, 3], SIZES, [7] * 300, [3_000_001]])
def test_norm(sp, dtype, sizes):
    gen = gen_of(sum(sizes))
    grads = [torch.randn(n, generator=gen, device="cuda").to(dtype) for n in sizes]
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    control = Guarded((8,), torch.int32)
    control.t.zero_()
    for k, (scale, most) in enumerate([(1.0, math.inf), (0.25, norm / 8), (2.0 ** -10, 1e9)]):
        got = sp.control_values(sp.sp24_grad_norm(grads, scale=scale, max_norm=most, control=control.t))
        assert int(got["step"]) == k + 1 and int(got["skip"]) == 0
        assert abs(float(got["norm"]) - scale * norm) <= 2 * U32 * scale * norm
        want = scale * min(1.0, most / (scale * norm))
        assert abs(float(got["factor"]) - want) <= 2 * U32 * want
    control.check()


def test_norm_of_nothing_and_of_zeros(sp):
    for grads in ([], [torch.empty(0, device="cuda")], [torch.zeros(5, device="cuda")]):
        got = sp.control_values(sp.sp24_grad_norm(grads, scale=0.5, max_norm=1.0))
        assert [float(got[k]) for k in ("norm", "factor", "skip", "step")] == [0.0, 0.5, 0, 1]


def test_norm_does_not_overflow(sp):
    g = torch.full((1000,), 3e38, device="cuda")
    got = sp.control_values(sp.sp24_grad_norm([g], scale=1e-3, max_norm=1.0))
    assert int(got["skip"]) == 0 and abs(float(got["norm"]) / (3e35 * math.sqrt(1000)) - 1) < 1e-6
    tiny = torch.full((1000,), 1e-30, device="cuda")
    assert abs(float(sp.control_values(sp.sp24_grad_norm([tiny]))["norm"]) / (1e-30 * math.sqrt(1000)) - 1) < 1e-6


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_what_is_not_finite_skips_the_step(sp, bad, dtype):
    grads = [torch.ones(n, device="cuda", dtype=dtype) for n in (5, 40000)]
    grads[1][39999] = bad
    control = sp.sp24_grad_norm([torch.ones(4, device="cuda", dtype=dtype)])
    sp.sp24_grad_norm(grads, control=control)
    got = sp.control_values(control)
    assert int(got["skip"]) == 1 and int(got["step"]) == 1 and float(got["factor"]) == 0.0
    for state8 in (False, True):
        P = [torch.randn(g.numel(), device="cuda") for g in grads]
        W = [p.half() for p in P]
        if state8:
            S = [[sp.state8(p) for p in P] for _ in range(2)]
            plan = sp.sp24_adamw_plan(P, [s[0] for s in S[0]], [s[0] for s in S[1]], W,
                                      M_exps=[s[1] for s in S[0]], V_exps=[s[1] for s in S[1]])
        else:
            plan = sp.sp24_adamw_plan(P, [torch.zeros_like(p) for p in P], [torch.zeros_like(p) for p in P], W)
        before = [t.clone() for part in plan.tensors for t in part]
        sp.sp24_adamw_step(plan, grads, control=control)
        assert all(torch.equal(a, b) for a, b in zip(before, [t for part in plan.tensors for t in part]))
    # and the next finite step counts on
    sp.sp24_grad_norm(grads[:1], control=control)
    assert int(got["skip"]) == 0 and int(got["step"]) == 2


# ------------------------------------------------------------------ 32 bits

def reference(P, M, V, g, lr, decay, b1, b2, eps, t):
    m = b1 * M + (1 - b1) * g
    v = b2 * V + (1 - b2) * g * g
    step = lr / (1 - b1 ** t) * m / ((v / (1 - b2 ** t)).sqrt() + eps)
    return (1 - decay) * P - step, m, v, step


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("sizes,t,b1,b2,copy", [(SIZES, 1, 0.9, 0.999, True), ([33] * 130, 7, 0.9, 0.95, False),
                                                ([1_000_003, 5], 100_000, 0.95, 0.999, True), ([200], 3, 0.0, 0.0, True)])
def test_32_bits(sp, dtype, sizes, t, b1, b2, copy):
    gen = gen_of(t)
    rand = lambda n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    P, M, V, W = ([Guarded((n,), d) for n in sizes] for d in (torch.float32,) * 3 + (torch.float16,))
    G = [(rand(n) * 0.01).to(dtype) for n in sizes]
    start = []
    for k, n in enumerate(sizes):
        P[k].t.copy_(rand(n))
        M[k].t.copy_(rand(n) * 0.01)
        V[k].t.copy_((rand(n) * 0.01).square())
        start.append([x[k].t.double() for x in (P, M, V)])
    lrs, decays = [1e-3 * (k + 1) for k in range(len(sizes))], [1e-4 * (k % 3) for k in range(len(sizes))]
    plan = sp.sp24_adamw_plan([x.t for x in P], [x.t for x in M], [x.t for x in V], [x.t if copy else None for x in W],
                              lrs=lrs, decays=decays)
    sp.sp24_adamw_step(plan, G, betas=(b1, b2), eps=1e-8, step=t)
    for k in range(len(sizes)):
        p, m, v, step = reference(*start[k], G[k].double(), lrs[k], decays[k], b1, b2, 1e-8, t)
        g, m0 = G[k].double(), start[k][1]
        for x in (P, M, V):
            x[k].check()
        assert ((M[k].t.double() - m).abs() <= 4 * U32 * ((b1 * m0).abs() + ((1 - b1) * g).abs()) + 1e-40).all()
        assert ((V[k].t.double() - v).abs() <= 5 * U32 * v + 1e-40).all()
        # M's error beside the root's, which with V's half is at most 6 roundings, and the bias corrections'
        m_err = 4 * U32 * ((b1 * m0).abs() + ((1 - b1) * g).abs())
        scale = lrs[k] / (1 - b1 ** t) / ((v / (1 - b2 ** t)).sqrt() + 1e-8)
        tol = scale * m_err + 24 * U32 * step.abs() + 3 * U32 * (start[k][0].abs() + step.abs())
        assert ((P[k].t.double() - p).abs() <= tol).all()
        if copy:
            W[k].check()
            assert torch.equal(W[k].t, P[k].t.half())


def test_no_epsilon_needed_for_zero_gradients(sp):
    P = torch.ones(100, device="cuda")
    plan = sp.sp24_adamw_plan([P], [torch.zeros(100, device="cuda")], [torch.zeros(100, device="cuda")], lrs=0.1, decays=0.5)
    sp.sp24_adamw_step(plan, [torch.zeros(100, device="cuda")], step=1)
    assert (P == 0.5).all()


def test_factor_and_step_from_the_control(sp):
    """A step with a control equals one with scaled gradients and the step given."""
    gen = gen_of(8)
    sizes = [1000, 77]
    G = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
    state = lambda: [[torch.full((n,), v, device="cuda") for n in sizes] for v in (0.5, 0.01, 0.02)]  # noqa: E731
    control = sp.sp24_grad_norm(G)
    control = sp.sp24_grad_norm(G, scale=0.5, max_norm=1e9, control=control)   # a power of two: exact
    a, b = state(), state()
    sp.sp24_adamw_step(sp.sp24_adamw_plan(*a), G, control=control)
    sp.sp24_adamw_step(sp.sp24_adamw_plan(*b), [g * 0.5 for g in G], step=2)
    assert all(torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


def test_a_control_before_the_first_step(sp):
    """No step counted yet: nothing is written (and no division by 1 - b^0)."""
    P = torch.ones(100, device="cuda")
    plan = sp.sp24_adamw_plan([P], [torch.ones(100, device="cuda")], [torch.ones(100, device="cuda")])
    sp.sp24_adamw_step(plan, [torch.ones(100, device="cuda")], control=sp.step_control())
    assert all((t == 1).all() for part in plan.tensors[:3] for t in part)


def test_refusals_on_the_gpu(sp):
    """What needs tensors on the GPU to be refused."""
    P = torch.ones(100, device="cuda")
    plan = sp.sp24_adamw_plan([P], [torch.zeros_like(P)], [torch.zeros_like(P)])
    for bad in ([P.cpu()], [torch.ones(100, 2, device="cuda")[:, 0]], [P.double()], [P, P]):
        with pytest.raises(ValueError):
            sp.sp24_adamw_step(plan, bad, step=1)
        with pytest.raises(ValueError):
            sp.sp24_grad_norm([P.cpu()] if bad[0] is P else bad)
    with pytest.raises(sp.Sp24Error):   # 4 bytes past a multiple of 16
        sp.sp24_adamw_step(plan, [torch.ones(101, device="cuda")[1:]], step=1)
    with pytest.raises(sp.Sp24Error):
        sp.sp24_grad_norm([P], max_norm=0.0)
    assert (P == 1).all()


# ------------------------------------------------------------------ 8 bits

def eight(sp, sizes, gen, steps=0):
    rand = lambda n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    P = [rand(n) for n in sizes]
    M, V = [sp.state8(p) for p in P], [sp.state8(p) for p in P]
    plan = sp.sp24_adamw_plan(P, [c for c, _ in M], [c for c, _ in V], M_exps=[e for _, e in M],
                              V_exps=[e for _, e in V], lrs=1e-3, decays=1e-4)
    return P, M, V, plan


def neighbours(x, top, fraction):
    """The held values below and above x >= 0, in a group whose largest is top."""
    q = torch.exp2(torch.floor(torch.log2(top)) - fraction)
    E = torch.floor(torch.log2(torch.ceil(top / q) * q))
    step = torch.exp2(torch.maximum(torch.floor(torch.log2(x)), E - 14) - fraction)
    low = torch.floor(x / step) * step
    return low, low + step


def group_top(x):
    n = x.numel()
    return torch.nn.functional.pad(x.abs(), (0, -n % 64)).reshape(-1, 64).amax(1).repeat_interleave(64)[:n]


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("sizes", [SIZES, [50] * 90])
def test_8_bits_step_by_step(sp, dtype, sizes):
    """Every step from the state as it is held: P as in 32 bits, M and the root
    of V one of the two held values next to the exact ones, and the one that
    the hash's bits say wherever rounding errors cannot decide."""
    gen = gen_of(len(sizes))
    P, M, V, plan = eight(sp, sizes, gen)
    seed = 0x12345678
    for t in range(1, 5):
        # sizes over many powers of two, zeros among them
        G = [(torch.randn(n, generator=gen, device="cuda") * torch.exp2(torch.randint(-12, 1, (n,), generator=gen, device="cuda").float())
              * (torch.rand(n, generator=gen, device="cuda") > 0.1)).to(dtype) for n in sizes]
        start = [(p.double(), decode(*m, 3), decode(*v, 4).square()) for p, m, v in zip(P, M, V)]
        sp.sp24_adamw_step(plan, G, step=t, seed=seed)
        for k, n in enumerate(sizes):
            p, m, v, step = reference(*start[k], G[k].double(), 1e-3, 1e-4, 0.9, 0.999, 1e-8, t)
            g = G[k].double()
            m_err = 4 * U32 * ((0.9 * start[k][1]).abs() + (0.1 * g).abs())
            scale = 1e-3 / (1 - 0.9 ** t) / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8)
            assert ((P[k].double() - p).abs() <= scale * m_err + 24 * U32 * step.abs() + 3 * U32 * (start[k][0].abs() + step.abs())).all()
            bits = hash_bits(seed, t, k, n)
            for (codes, exps), x, err, fraction, u in ((M[k], m, m_err, 3, bits & 0xFFFF), (V[k], v.sqrt(), 6 * U32 * v.sqrt(), 4, bits >> 16)):
                got = decode(codes, exps, fraction)
                assert ((got == 0) == (x == 0)).all() if fraction == 4 else (got[x == 0] == 0).all()
                some = x != 0
                a, got, err, u = x.abs()[some], got[some] * torch.sign(x[some]), err[some], u[some]
                low, high = neighbours(a, group_top(x)[some], fraction)
                near = torch.minimum(a - low, high - a) <= err + 2.0 ** -40 * a
                least = high if fraction == 4 else torch.zeros_like(high)
                assert ((got == low) | (got == high) | near | ((low == 0) & (got == least))).all()
                z = (a - low) / (high - low) + (u + 0.5) / 65536
                clear = ((z - 1).abs() > err / (high - low) + 1e-9) & ~near & (low > 0)
                assert torch.equal((got == high)[clear], (z >= 1)[clear]) and int(clear.sum()) >= 0.3 * int(some.sum()) - 2


def test_8_bits_are_unbiased_over_steps(sp):
    """One state value, held with many different random bits: the mean is the
    value, within 5 standard deviations of a mean of n coins."""
    n = 1 << 18
    P, M, V, plan = eight(sp, [n], gen_of(1))
    G = torch.full((n,), 0.3, device="cuda")
    G[63::64] = 1.0     # sets the groups' exponents, and keeps 0.03 between held values
    sp.sp24_adamw_step(plan, [G], step=1, seed=99)
    rest = torch.arange(n, device="cuda") % 64 != 63
    for (codes, exps), fraction, x in ((M[0], 3, 0.03), (V[0], 4, math.sqrt(0.001) * 0.3)):
        got = decode(codes, exps, fraction)[rest]
        held = got.unique()
        assert len(held) == 2 and held[0] < x < held[1]
        width = float(held[1] - held[0])
        assert abs(float(got.mean()) - x) <= 5 * 0.5 * width / math.sqrt(len(got)) + 2.0 ** -16 * width


def test_8_bits_follow_a_falling_gradient(sp):
    """Where gradients vanish V falls as in 32 bits: rounding to nearest would
    hold it where it is."""
    n = 4096
    gen = gen_of(5)
    P, M, V, plan = eight(sp, [n], gen)
    exact = torch.zeros(n, dtype=torch.float64, device="cuda")
    for t in range(1, 601):
        g = torch.randn(n, generator=gen, device="cuda") * (1.0 if t <= 100 else 0.05)
        exact = 0.999 * exact + 0.001 * g.double().square()
        sp.sp24_adamw_step(plan, [g], step=t, seed=7)
    got = sp.sp24_state8_values(V[0][0], V[0][1], root=True).double()
    # A root moves by a 2000th of itself a step, so of a held step (a 16th to a 32nd of it) at most a 62nd: rounding
    # adds a variance of at most 1/62 (1/16)^2 a step, 0.031 relative in 500 steps, a standard deviation of 18%,
    # 0.3% over 4096 entries; the term g^2 / 2r bends the mean by no more than that variance.  3.1% + 5 * 0.3%
    assert abs(float(got.mean() / exact.sqrt().mean()) - 1) <= 0.05


def test_8_bits_not_finite(sp):
    P, M, V, plan = eight(sp, [200], gen_of(2))
    G = torch.ones(200, device="cuda")
    G[70] = math.nan
    G[130] = 1e30       # its square overflows: V is infinite
    sp.sp24_adamw_step(plan, [G], step=1)
    m, v = sp.sp24_state8_values(*M[0]), sp.sp24_state8_values(*V[0], root=True)
    groups = torch.arange(200, device="cuda") // 64
    assert torch.equal(torch.isnan(m), groups == 1) and torch.equal(torch.isnan(v), (groups == 1) | (groups == 2))
    # magnitudes at the range's end are held, not lost
    P, M, V, plan = eight(sp, [64], gen_of(3))
    big = torch.full((64,), 3.4e38, device="cuda")
    sp.sp24_adamw_step(plan, [big], step=1, betas=(0.0, 0.5))
    assert torch.isfinite(sp.sp24_state8_values(*M[0])).all()


def test_values_of_all_codes(sp):
    codes = torch.arange(256, device="cuda").to(torch.uint8)
    for E in (0, 1, 100, 127, 200, 254):
        exps = torch.full((4,), E, dtype=torch.uint8, device="cuda")
        for root in (False, True):
            want = decode(codes, exps, 4 if root else 3)
            got = sp.sp24_state8_values(codes, exps, root=root)
            assert torch.equal(got.double(), want)
            if E > 17:
                assert torch.equal(sp.sp24_state8_values(codes, exps, root=root, dtype=torch.bfloat16).double(), want)
    out = Guarded((131,), torch.bfloat16)
    sp.sp24_state8_values(torch.full((131,), 120, dtype=torch.uint8, device="cuda"),
                          torch.full((3,), 127, dtype=torch.uint8, device="cuda"), dtype=torch.bfloat16, out=out.t)
    out.check()
    assert (out.t == 1.0).all()


def test_states_between_guards(sp):
    for n in (1, 63, 64, 130, 5000):
        P, M, V = Guarded((n,), torch.float32), Guarded((n,), torch.uint8, fill=0), Guarded((n,), torch.uint8, fill=0)
        ME, VE = (Guarded((-(-n // 64),), torch.uint8, fill=0) for _ in range(2))
        P.t.zero_()
        plan = sp.sp24_adamw_plan([P.t], [M.t], [V.t], M_exps=[ME.t], V_exps=[VE.t])
        sp.sp24_adamw_step(plan, [torch.ones(n, device="cuda")], step=1)
        for g in (P, M, V, ME, VE):
            g.check()


def test_norm_and_step_in_a_graph(sp):
    """A captured norm and step, replayed with eager work between, go the way
    of eager calls: the step's count and the random bits move on."""
    for state8 in (False, True):
        sizes = [1000, 77, 20000]
        runs = []
        for captured in (False, True):
            gen = gen_of(11)
            P = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
            if state8:
                M, V = [sp.state8(p) for p in P], [sp.state8(p) for p in P]
                plan = sp.sp24_adamw_plan(P, [c for c, _ in M], [c for c, _ in V], M_exps=[e for _, e in M],
                                          V_exps=[e for _, e in V])
            else:
                plan = sp.sp24_adamw_plan(P, [torch.zeros_like(p) for p in P], [torch.zeros_like(p) for p in P])
            G = [torch.zeros(n, device="cuda") for n in sizes]
            control = sp.step_control()
            ws = torch.empty(sum(-(-n // 16384) for n in sizes) * 8, dtype=torch.uint8, device="cuda")

            def step():
                sp.sp24_grad_norm(G, max_norm=1.0, control=control, workspace=ws)
                sp.sp24_adamw_step(plan, G, control=control, seed=3)

            if captured:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            for k in range(5):
                for g in G:
                    g.copy_(torch.randn(g.numel(), generator=gen, device="cuda"))
                if k == 3:
                    G[1][5] = math.nan
                graph.replay() if captured else step()
                torch.cuda.synchronize()
            assert int(sp.control_values(control)["step"]) == 4
            runs.append([t for part in plan.tensors for t in part if t is not None])
        assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_entries_past_32_bits(sp):
    """A tensor of more than 2^31 entries: offsets past 32 bits of bytes and
    of entries."""
    n = (1 << 31) + 1000
    P = torch.zeros(n, device="cuda")
    G = torch.zeros(n, dtype=torch.float16, device="cuda")
    at = torch.tensor([0, 5, (1 << 30) + 3, (1 << 31) - 1, 1 << 31, n - 1], device="cuda")
    G[at] = 1.0
    M, V = sp.state8(P), sp.state8(P)
    got = sp.control_values(sp.sp24_grad_norm([G]))
    assert abs(float(got["norm"]) - math.sqrt(6)) < 1e-6
    sp.sp24_adamw_step(sp.sp24_adamw_plan([P], [M[0]], [V[0]], M_exps=[M[1]], V_exps=[V[1]], lrs=0.5), [G], step=1)
    # m / sqrt v = 1 after the first step
    assert ((P[at] + 0.5).abs() <= 1e-5).all() and int(torch.count_nonzero(P)) == 6
    assert int(torch.count_nonzero(M[0])) == 6
