"""Host model of the Newton-Schulz products' and the embedding gradient's
address arithmetic (CPU only, no kernel runs): every tile and item is dealt
once, every entry of the symmetric matrices is stored, every direct load lies
inside the operand or beyond all of it (where it reads as zero), and the
embedding's chunks, parts and cleared runs cover what they should.  The formulas
are transcribed from csrc/sp24_ns.hip and csrc/sp24_embed.hip; a change to a
kernel's indexing has to be mirrored here."""
import numpy as np
import pytest

TILES = [(128, 128), (64, 128), (320, 256), (128, 256)]
SIZES = [(1, 1), (33, 1000), (129, 130), (357, 1001), (500, 500), (1024, 4096), (1600, 1600), (1600, 6400), (2049, 5000)]


def cdiv(a, b):
    return -(-a // b)


def upper_tiles(m, bm, bn):
    q = bn // bm
    rows, cols = cdiv(m, bm), cdiv(m, bn)
    full, rest = divmod(rows, q)
    return rows * cols - q * (full * (full - 1) // 2) - rest * full


def upper_tile(m, k, bm, bn):
    q, cols, tm = bn // bm, cdiv(m, bn), 0
    while k >= cols - tm // q:
        k -= cols - tm // q
        tm += 1
    return tm, tm // q + k


@pytest.mark.parametrize("bm,bn", [t for t in TILES if t[1] % t[0] == 0])
@pytest.mark.parametrize("m", sorted({s[0] for s in SIZES}))
def test_symmetric_tiles_cover_the_matrix(bm, bn, m):
    blocks = cdiv(m, 32)
    seen = np.zeros((blocks + bm // 32 + bn // 32, blocks + bm // 32 + bn // 32), int)
    tiles = [upper_tile(m, k, bm, bn) for k in range(upper_tiles(m, bm, bn))]
    assert len(set(tiles)) == len(tiles)
    for tm, tn in tiles:
        assert tm * bm < m and tn * bn < m
        rows, cols = slice(tm * bm // 32, (tm + 1) * bm // 32), slice(tn * bn // 32, (tn + 1) * bn // 32)
        seen[rows, cols] += 1
        if tn != tm // (bn // bm):
            assert (tm + 1) * bm <= m          # whole rows above: what is mirrored exists
            seen[cols, rows] += 1
    assert (seen[:blocks, :blocks] == 1).all()


@pytest.mark.parametrize("items", [1, 7, 8, 9, 91, 250, 455, 650, 1300])
def test_runs_by_xcd_deal_every_item_once(items):
    run = cdiv(items, 8)
    got = [b % 8 * run + b // 8 for b in range(cdiv(items, 8) * 8) if b // 8 < run and b % 8 * run + b // 8 < items]
    assert sorted(got) == list(range(items))


@pytest.mark.parametrize("bm,bn", TILES)
@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("parts", [1, 2])
def test_direct_loads_stay_inside_or_read_zero(bm, bn, m, n, parts):
    na, nx, waves = cdiv(m, 32), cdiv(n, 32), {(128, 128): 4, (64, 128): 4, (320, 256): 8, (128, 256): 8}[bm, bn]
    lane = np.arange(64)
    for kind in ("gram", "poly", "apply"):
        if bn % bm and kind != "apply":
            continue
        lnb, rnb = (nx if kind == "gram" else na), (na if kind == "poly" else nx)
        lplane, rplane = na * lnb * 1024, na * rnb * 1024     # elements of a part
        nk = lnb
        tiles_n = cdiv(m if kind != "apply" else n, bn)
        for m0, n0 in {(0, 0), ((cdiv(m, bm) - 1) * bm, (tiles_n - 1) * bn)}:
            for side in ("left", "right"):
                rows, plane = (bm, lplane) if side == "left" else (bn, rplane)
                per_part, records = rows * 64 // 1024, parts * plane * 2
                assert records <= 2 ** 31
                slots = set()
                for ld in range(parts * per_part):
                    s = ld % per_part * 64 + lane
                    row, blk, q = s // 4 % 32, (m0 if side == "left" else n0) // 32 + s // 128, (s & 3) ^ (s // 4 % 32 >> 2 & 3)
                    across = kind == "apply" and side == "right"
                    first = blk if across else blk * (lnb if side == "left" else rnb)
                    at = ld // per_part * plane * 2 + first * 2048 + row * 64 + q * 16
                    step = rnb * 2048 if across else 2048
                    real = blk < (rnb if across else na)
                    end = at + (nk - 1) * step + 16
                    assert (end[real] <= records).all() and (at[real] >= 0).all()
                    # all of a part's chunks of a block, each once
                    slots |= {(ld // per_part, int(b), int(r), int(c)) for b, r, c in zip(s // 128, row, q)}
                assert len(slots) == parts * rows // 32 * 128
        assert max(cdiv(parts * bm * 64 // 1024, waves), 1) * waves >= parts * bm * 64 // 1024


@pytest.mark.parametrize("T", [1, 15, 16, 517, 8191, 8192, 65535, 65536, 131072, 200001])
def test_embedding_segments_and_chunks(T):
    unit = 512
    seg = max(cdiv(T, 16 * unit) * unit, 2048)
    segs = cdiv(T, seg)
    assert segs <= 16 and seg % 512 == 0
    chunk = 64 if T >= 65536 else 32 if T >= 8192 else 16
    chunks = cdiv(T, chunk)
    assert chunks * chunk >= T > (chunks - 1) * chunk
    # a run over chunks a .. b leaves its parts in 2 a + 1 and 2 k, k = a + 1 .. b: inside 2 chunks rows
    assert 2 * (chunks - 1) + 1 < 2 * chunks


@pytest.mark.parametrize("d", [1, 3, 7, 8, 9, 67, 1600, 1999, 2056, 4097])
def test_embedding_columns(d):
    vec = 8 if d >= 8 else 1
    team = 8
    while team < 256 and team * vec < d:
        team *= 2
    added = np.zeros(d, int)
    for y in range(cdiv(d, team * vec)):
        for t in range(team):
            mine = (y * team + t) * vec
            if mine >= d:
                continue
            col = min(mine, d - vec)
            assert 0 <= col and col + vec <= d
            added[mine:col + vec] += 1
    assert (added == 1).all()
    # cleared runs: 16 rows of d entries in pieces of 4, dealt to the slices
    for rows in (1, 5, 16):
        pieces, slices = cdiv(rows * d, 4), cdiv(d, team * vec)
        cuts = [pieces * y // slices for y in range(slices + 1)]
        assert cuts[0] == 0 and cuts[-1] == pieces
        i = np.arange(pieces)
        r, r3 = 4 * i // d, (4 * i + 3) // d
        whole = (r == r3) & (r < rows)
        assert (4 * i[whole] + 4 <= rows * d).all() and (r3 <= 16 + 3).all()
