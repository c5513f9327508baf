"""Host model of the address arithmetic of the products with an epilogue, the
bias gradient, the norm and AdamW (CPU only, no kernel runs): every tile, part
and pass is dealt once, every direct load lies inside its operand or beyond all
of it (where it reads as zero), what goes straight to registers is in bounds,
and partial sums stay in the workspace that the library asks for.  The formulas
are transcribed from csrc/sp24_linear.hip, csrc/sp24_spmm_loop.inc and
csrc/sp24_adamw.hip; a change to a kernel's indexing has to be mirrored here."""
import os

import numpy as np
import pytest

CUS = 256
SIZES = [(1, 6400, 1600), (17, 1600, 6400), (24, 1600, 6400), (33, 16, 16), (64, 112, 6400), (65, 1024, 320), (127, 64, 1616),
         (150, 528, 6416), (192, 6400, 1600), (257, 272, 128), (512, 1600, 6400), (1021, 4096, 1024), (1000, 128, 48),
         (2500, 528, 656), (8192, 2064, 336), (1500, 6400, 1600), (2048, 4096, 1024), (3000, 1600, 6400), (16384, 6400, 1600), (16384, 1600, 6400), (70000, 64, 6400), (350000, 6400, 64)]


def cdiv(a, b):
    return -(-a // b)


def plan(T, N, K):
    tiles = lambda f, t: cdiv(T, t) * cdiv(N, f)  # noqa: E731
    fits = K >= 64 and K * 512 < 2 ** 31 and N * K < 2 ** 31 and tiles(64, 64) < 2 ** 22
    if not fits or T <= 16 or (T <= 32 and K <= 1024):
        return "thin", 1, 16 if T <= 16 else 32 if T <= 32 else 64
    if tiles(64, 64) <= CUS:
        rounds = (K // 64 + 3) // 4
        parts = min(CUS // tiles(64, 64), rounds // 2)
        if parts > 1 and rounds - cdiv(rounds, parts) >= 7:
            return "mid", parts, 16
        return "mid", 1, 64
    if tiles(128, 128) <= CUS and K >= 128:
        return "pairs", 1, 128
    return "small" if tiles(256, 128) < CUS else "large", 1, 128


def tile_at(lin, tiles_m, tiles_n):
    group = lin // (8 * tiles_n)
    gm0 = group * 8
    gsize = min(8, tiles_m - gm0)
    in_group = lin - group * 8 * tiles_n
    return gm0 + in_group % gsize, in_group // gsize


def runs(count):
    """Positions of a launch's workgroups in runs by XCD."""
    per = cdiv(count, 8)
    return [b % 8 * per + b // 8 for b in range(cdiv(count, 8) * 8) if b % 8 * per + b // 8 < count]


@pytest.fixture(scope="module")
def lib():
    from structured_sparse_transformer_amd import build, sp24
    if not os.path.exists(sp24.LIB_PATH):
        build.build()
    return sp24.lib()


@pytest.mark.parametrize("T,N,K", SIZES)
def test_every_output_has_one_tile(T, N, K):
    how, parts, _ = plan(T, N, K)
    seen = {}
    if how == "large":
        tiles_n, slots = cdiv(T, 128), 2 * CUS
        rounds = tiles_n * cdiv(N, 256) // slots
        big = min(N // 256, rounds * slots // tiles_n)
        if cdiv(N - big * 256, 128) * tiles_n > slots:
            big = N // 256
        small = cdiv(N - big * 256, 128)
        nbig, nsmall = big * tiles_n, small * tiles_n
        pb, ps = cdiv(nbig, 8), cdiv(nsmall, 8)
        for b in range((pb + ps) * 8):
            x, at = b % 8, b // 8
            if at < pb:
                lin = x * pb + at
                if lin >= nbig:
                    continue
                tm, tn = tile_at(lin, big, tiles_n)
                cells = [(2 * tm, tn), (2 * tm + 1, tn)]
            else:
                lin = x * ps + at - pb
                if at - pb >= ps or lin >= nsmall:
                    continue
                tm, tn = tile_at(lin, small, tiles_n)
                cells = [(2 * big + tm, tn)]
            for c in cells:
                seen[c] = seen.get(c, 0) + 1
        want = {(m, n) for m in range(2 * big + small) for n in range(tiles_n)}
        assert (2 * big + small) * 128 >= N and (2 * big + small - 1) * 128 < N and big * 256 <= N
    elif how in ("small", "pairs"):
        tiles_m, tiles_n = cdiv(N, 128), cdiv(T, 128)
        for lin in runs(tiles_m * tiles_n):
            c = tile_at(lin, tiles_m, tiles_n)
            seen[c] = seen.get(c, 0) + 1
        want = {(m, n) for m in range(tiles_m) for n in range(tiles_n)}
    elif how == "mid":
        tiles_m, tiles_n = cdiv(N, 64), cdiv(T, 64)
        for lin in runs(tiles_m * tiles_n * parts):
            tn, strip = lin % tiles_n, lin // tiles_n
            c = (strip // parts, tn, strip % parts)
            seen[c] = seen.get(c, 0) + 1
        want = {(m, n, p) for m in range(tiles_m) for n in range(tiles_n) for p in range(parts)}
    else:
        return
    assert set(seen) == want and set(seen.values()) == {1}


@pytest.mark.parametrize("n", list(range(1, 40)) + [100, 101])
@pytest.mark.parametrize("parts", [1, 2, 3, 8])
def test_stages_are_dealt_once(n, parts):
    """The mid kernel's parts and groups, and the pairs' halves with their barriers."""
    if parts <= n:
        got = []
        for p in range(parts):
            first = p * n // parts
            count = (p + 1) * n // parts - first
            rounds = (count + 3) // 4
            for kg in range(4):
                mine = max(0, (count - kg + 3) // 4)
                assert mine <= rounds
                got += [first + kg + 4 * j for j in range(mine)]
        assert sorted(got) == list(range(n))
    if n >= 2:
        half = (n + 1) // 2
        assert n - half >= 1
        meet = [1 + half, 1 + (n - half) + (1 if n % 2 else 0)]
        assert meet[0] == meet[1]


@pytest.mark.parametrize("slots", [2, 3])
@pytest.mark.parametrize("nk", [1, 2, 3, 4, 5, 7, 25])
def test_ring(slots, nk):
    """The loop's ring: a stage is loaded before it is read, and no slot is loaded
    while a stage that it holds is still to be read."""
    held = {s: s for s in range(min(slots, nk))}
    for kt in range(nk):
        assert held[kt % slots] == kt
        # past the barrier in stage kt nobody reads its slot again
        if kt + slots < nk:
            held[kt % slots] = kt + slots


@pytest.mark.parametrize("rounds", [1, 2, 3, 4, 7, 25])
def test_mid_ring(rounds):
    """Stage j + 2 is issued past the barrier of round j, into the slot that round
    j - 1 read; the wait before it allows one stage's loads under way."""
    issued, read = [0, 1][:rounds], []
    for j in range(rounds):
        flying = [s for s in issued if s > j]
        assert j in issued and len(flying) <= 1
        if j + 2 < rounds:
            assert all(s % 3 != (j + 2) % 3 or s in read for s in issued)
            issued.append(j + 2)
        read.append(j)
    assert read == list(range(rounds))


def direct(offset, size, limit, whole):
    """A direct load of `size` bytes: inside the operand, or past all of it."""
    assert offset >= 0
    assert (offset + size <= whole) or offset >= limit, (offset, size, limit, whole)
    return offset + size <= whole


@pytest.mark.parametrize("T,N,K", [s for s in SIZES if plan(*s)[0] != "thin"])
def test_direct_loads(T, N, K):
    how, parts, _ = plan(T, N, K)
    bm, bn = {"large": (256, 128), "small": (128, 128), "pairs": (128, 128), "mid": (64, 64)}[how]
    lane = np.arange(64)
    swz_s = lambda r: ((r >> 1) ^ (r >> 2)) & 3  # noqa: E731
    swz_b = lambda r: (r & 7) ^ ((r >> 3) & 1)  # noqa: E731
    n = K // 64
    rows_m, rows_n = cdiv(N, bm), cdiv(T, bn)
    for tm in {0, rows_m // 2, rows_m - 1}:
        m0 = tm * bm
        whole = (N - m0) * K                       # bytes of vals from the tile's first row on
        for q in range(bm // 16):
            r = 16 * q + lane // 4
            h = max(0, min(64, N - m0 - 64 * (16 * q // 64)))
            off = (r // 64) * 64 * K + (r % 64) * 64 + ((lane % 4) ^ swz_s(r)) * 16
            for kt in {0, n - 1}:
                o = off + kt * h * 64
                assert (o >= 0).all() and o.max() + 16 < 2 ** 31
                # rows that are stored read their own block: inside
                real = m0 + r < N
                assert (o[real] + 16 <= whole).all()
                assert sorted((o[real] - off[real]) // 64 // max(h, 1)) == [kt] * int(real.sum())
        for q in range(max(1, bm // 32)):
            r = 32 * q + lane // 2
            h = max(0, min(64, N - m0 - 64 * (32 * q // 64)))
            o = (r // 64) * 8 * K + (r % 64) * 8 + (lane % 2) * 4 + (n - 1) * h * 8
            real = m0 + r < N
            assert (o[real] + 4 <= (N - m0) * (K // 8)).all()
    for tn in {0, rows_n // 2, rows_n - 1}:
        tokens = min(bn, T - tn * bn)
        whole = tokens * K * 2
        assert whole < 2 ** 31
        for q in range(bn // 8):
            r = 8 * q + lane // 8
            o = r * K * 2 + ((lane % 8) ^ swz_b(r)) * 16 + (n - 1) * 128
            assert o.max() + 16 < 2 ** 31
            for rr, oo in zip(r, o):
                inside = direct(int(oo), 16, whole, whole)
                assert inside == (rr < tokens)     # rows past the last read zeros


@pytest.mark.parametrize("T,N,K", SIZES)
def test_straight_loads(T, N, K):
    """The thin kernel's operands and the tails of all: inside the operands, and
    each kept value where the forms' blocked order has it."""
    left, k0 = K % 64, K // 64 * 64

    def form(r, c, n, m, b):
        r0, c0 = r // 64 * 64, c // b * b
        return r0 * m + c0 * min(64, n - r0) + (r - r0) * min(b, m - c0) + (c - c0)

    for row in {0, 15, N // 2, N - 16, N - 1}:
        r0 = row // 64 * 64
        h = min(64, N - r0)
        for b in {0, k0 // 64 - 1}:
            if b < 0 or b >= K // 64:
                continue
            for g in range(4):
                v = r0 * (K // 2) + b * 32 * h + (row - r0) * 32 + g * 8
                assert v == form(row, b * 32 + g * 8, N, K // 2, 32) and v + 8 <= N * K // 2
                assert r0 * (K // 16) + b * 4 * h + (row - r0) * 4 + g == form(row, b * 4 + g, N, K // 16, 4)
        for c in range(left // 16):
            v = r0 * (K // 2) + k0 // 2 * h + (row - r0) * (left // 2) + 8 * c
            assert v == form(row, k0 // 2 + 8 * c, N, K // 2, 32) and v + 8 <= N * K // 2
            assert r0 * (K // 16) + k0 // 16 * h + (row - r0) * (left // 16) + c == form(row, k0 // 16 + c, N, K // 16, 4)
    for g in range(4):      # the thin kernel's tokens: 16-byte pieces of a row, or none
        for at in (8 * g, 32 + 8 * g):
            assert not at < left or k0 + at + 8 <= K


@pytest.mark.parametrize("T,N,K", SIZES)
def test_partial_sums_fit_the_workspace(lib, T, N, K):
    how, parts, block = plan(T, N, K)
    rows = cdiv(T, block)
    floats = parts * T * N if parts > 1 else 0
    assert lib.sp24_spmm_fwd_act_workspace(T, N, K) == 4 * floats
    assert lib.sp24_spmm_bwd_input_act_workspace(T, K, N) == 4 * (floats + (rows * N if rows > 1 else 0))
    last = {"thin": lambda: (T - 1) // block, "mid": lambda: (T - 1) // (16 if parts > 1 else 64),
            "pairs": lambda: (T - 1) // 128, "small": lambda: (T - 1) // 128, "large": lambda: (T - 1) // 128}[how]()
    assert last == rows - 1


@pytest.mark.parametrize("T", [1, 64, 517, 1024, 1025, 4096, 16384, 100000, 2 ** 31 - 1])
@pytest.mark.parametrize("R", [16, 80, 512, 528, 6400])
def test_bias_grad_chunks(lib, T, R):
    if R >= 2 ** 40 // T:
        return
    P = 1 if T <= 1024 else max(1, min(cdiv(T, 64), max(1, 2048 // cdiv(R, 512))))
    assert lib.sp24_bias_grad_workspace(T, R) == (4 * P * R if P > 1 else 0)
    rows = cdiv(T, P)
    assert P * rows >= T and P <= 65535


@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [4096] * 200, [1, 4095, 4096, 4097, 70001], [2 ** 34 - 1, 3]])
@pytest.mark.parametrize("most,chunk", [(44, 4096), (64, 4096), (128, 16384)])
def test_chunks_find_their_tensor(lib, sizes, most, chunk):
    launches, table, chunks = [], [], 0
    for k, n in enumerate(sizes):
        c = cdiv(n, chunk)
        if c == 0:
            continue
        if len(table) == most or chunks + c > 2 ** 24 - 1:
            launches.append((table, chunks))
            table, chunks = [], 0
        table = table + [(k, chunks)]
        chunks += c
    launches.append((table, chunks))
    covered = {}
    for table, chunks in launches:
        assert chunks <= 2 ** 24 - 1
        firsts = [f for _, f in table]
        probe = sorted({c for f in firsts for c in (f, f + 1, f - 1)} | {chunks - 1})
        for c in probe:
            if not 0 <= c < chunks:
                continue
            lo, hi = 0, len(table) - 1
            while lo < hi:
                mid = (lo + hi + 1) // 2
                if firsts[mid] <= c:
                    lo = mid
                else:
                    hi = mid - 1
            k = table[lo][0]
            assert firsts[lo] <= c and (c - firsts[lo]) * chunk < sizes[k]
            covered[k] = True
    assert set(covered) == {k for k, n in enumerate(sizes) if n}
