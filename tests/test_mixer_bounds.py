"""CPU replay of the index arithmetic of the delta rule and query and key norm kernels
(the same names as in their sources): every element is written by one lane, operands
agree on the summed places, and every address formed lies inside its buffer."""
import numpy as np
import pytest

LANE = np.arange(64)
C, G = LANE & 15, LANE >> 4


def rho(tile, x):
    return 32 * (tile >> 1) + 8 * (x >> 2) + 4 * (tile & 1) + (x & 3)


def rho_tile(n):
    return 2 * (n >> 5) + ((n >> 2) & 1)


def rho_row(n):
    return 4 * ((n >> 3) & 3) + (n & 3)


def row_place(lane=LANE):
    return lane ^ (lane >> 4 << 2)


def lower_frag(i, kt):
    return (i >> 1) * ((i >> 1) + 1) + (i & 1) * ((i >> 1) + 1) + kt


def upper_frag(KC, j, kt):
    return 2 * ((j >> 1) * KC - (j >> 1) * ((j >> 1) - 1) // 2) + (j & 1) * (KC - (j >> 1)) + kt - (j >> 1)


def test_rho_is_a_numbering_whose_results_chain():
    n = np.arange(128)
    tile, row = np.meshgrid(np.arange(8), np.arange(16), indexing="ij")
    assert sorted(rho(tile, row).ravel()) == list(n)
    assert np.array_equal(rho(rho_tile(n), rho_row(n)), n)
    # a lane's results (rows 4 g + r of tiles 2 m, 2 m + 1) are its eight places of the next product
    for m in range(4):
        for e in range(8):
            assert np.array_equal(rho(2 * m + (e >> 2), 4 * G + (e & 3)), 32 * m + 8 * G + e)


@pytest.mark.parametrize("KC", [1, 2])
def test_triangles(KC):
    RT = 2 * KC
    assert sorted(lower_frag(i, kt) for i in range(RT) for kt in range(i // 2 + 1)) == list(range(KC * (KC + 1)))
    assert sorted(upper_frag(KC, j, kt) for j in range(RT) for kt in range(j // 2, KC)) == list(range(KC * (KC + 1)))


def row_image(X, KD, NP, frag=None):
    """fetch_rows: the image of rows X [C][32 KD] (words apart by NP), as elements of two bytes."""
    RT = len(X) // 16
    frag = frag or (lambda i, ks: i * KD + ks)
    img = np.full(RT * KD * NP * 512, -1, np.int64)
    seen = np.zeros(len(img), int)
    for i in range(RT):
        for ks in range(KD):
            if frag(i, ks) is None:
                continue
            for w in range(NP):
                c = row_place() & 15   # lane l of the fetch brings the row of its place
                for e in range(8):
                    at = (frag(i, ks) * NP + w) * 512 + LANE * 8 + e
                    img[at] = X[rho(i, c), 32 * ks + 8 * G + e] * NP + w
                    seen[at] += 1
    return img, seen


def turned4(img, at):
    """The transposing read: lane p of 16 names four elements (4 (p % 4) .. of row p / 4); lane c gets column c of the rows."""
    out = np.zeros((64, 4), np.int64)
    for g in range(4):
        rows = np.array([[img[at[16 * g + 4 * k + q] + e] for q in range(4) for e in range(4)] for k in range(4)])
        out[16 * g:16 * g + 16] = rows.T
    return out


def turned_frag(img, NP, j, frag0, frag1, w):
    p, x, g = C, 4 * G + (C >> 2), C & 3
    at = (16 * g + (x ^ (4 * g))) * 8 + 4 * (j & 1)
    assert at.min() >= 0 and at.max() + 4 <= 512
    return np.concatenate([turned4(img, at + (f * NP + w) * 512) for f in (frag0, frag1)], axis=1)


@pytest.mark.parametrize("RT,KD,NP", [(4, 4, 1), (4, 2, 1), (2, 4, 3), (2, 2, 3), (4, 2, 2)])
def test_rows_and_turned_rows(RT, KD, NP):
    X = np.arange(16 * RT * 32 * KD).reshape(16 * RT, 32 * KD)
    img, seen = row_image(X, KD, NP)
    assert (seen == 1).all()
    for w in range(NP):
        for i in range(RT):
            for ks in range(KD):   # row_frag: row rho(i, c), places 8 g ..
                for e in range(8):
                    got = img[((i * KD + ks) * NP + w) * 512 + row_place() * 8 + e]
                    assert np.array_equal(got, X[rho(i, C), 32 * ks + 8 * G + e] * NP + w)
        for j in range(2 * KD):
            for kt in range(RT // 2):   # row rho(j, c) of the transpose, places 32 kt + 8 g ..
                got = turned_frag(img, NP, j, 2 * kt * KD + (j >> 1), (2 * kt + 1) * KD + (j >> 1), w)
                for e in range(8):
                    assert np.array_equal(got[:, e], X[32 * kt + 8 * G + e, rho(j, C)] * NP + w)


@pytest.mark.parametrize("KC", [1, 2])
def test_pair_matrices(KC):
    """The pair tiles' stores fill the lower image; it is read as it stands and turned."""
    RT, NP = 2 * KC, 2
    pairs = [(p >> 1, p & 1) if p < 4 else (2 + ((p - 4) >> 2), (p - 4) & 3) for p in range(2 * KC * (KC + 1))]
    assert sorted(pairs) == [(i, j) for i in range(RT) for j in range(2 * (i // 2) + 2)]
    X = np.arange(16 * RT * 16 * RT).reshape(16 * RT, 16 * RT)
    img = np.full(KC * (KC + 1) * NP * 512, -1, np.int64)
    for i, j in pairs:
        at = lower_frag(i, j >> 1) * NP * 512 + row_place() * 8 + (j & 1) * 4
        for r in range(4):
            assert (img[at + r] == -1).all()
            img[at + r] = X[rho(i, C), rho(j, 4 * G + r)]
    for i in range(RT):
        for kt in range(i // 2 + 1):
            for e in range(8):
                assert np.array_equal(img[lower_frag(i, kt) * NP * 512 + row_place() * 8 + e], X[rho(i, C), 32 * kt + 8 * G + e])
    for kt in range(KC):
        for j in range(2 * kt + 2):
            got = turned_frag(img, NP, j, lower_frag(2 * kt, j >> 1), lower_frag(2 * kt + 1, j >> 1), 0)
            for e in range(8):
                assert np.array_equal(got[:, e], X[32 * kt + 8 * G + e, rho(j, C)])


@pytest.mark.parametrize("es,RT", [(2, 4), (4, 2)])
def test_columns(es, RT):
    """16 columns of a chunk in 2048 bytes: fetch_columns, take_columns."""
    rows, lanes = 16 * RT, es
    img = np.full(2048 // es, -1, np.int64)
    for j in range(2):
        t, part = j * (64 // lanes) + LANE // lanes, LANE % lanes
        assert t.max() < rows
        for e in range(16 // es):
            img[(1024 * j + 16 * LANE) // es + e] = t * 16 + part * (16 // es) + e
    assert np.array_equal(img, np.arange(rows * 16))
    for i in range(RT):
        if es == 4:
            for r in range(4):
                assert np.array_equal(img[(rho(i, r) * 64 + G * 8 * 64 + C * 4) // 4], rho(i, 4 * G + r) * 16 + C)
        else:
            got = turned4(img, ((rho(i, 0) + 8 * G + (C >> 2)) * 32 + (C & 3) * 8) // 2)
            for r in range(4):
                assert np.array_equal(got[:, r], rho(i, 4 * G + r) * 16 + C)


def test_turned_tile():
    """lds_tile, lds_turned: a result tile back with rows and columns changed."""
    tile = np.zeros(256, np.int64)
    for r in range(4):
        tile[(LANE ^ (LANE >> 4)) * 4 + r] = (4 * G + r) * 16 + C
    for r in range(4):
        at = (16 * (C >> 2) + 4 * G) * 16 + (C & 3) * 4 + 16 * (r ^ (C >> 2))
        assert np.array_equal(tile[at // 4], C * 16 + 4 * G + r)
        assert sorted(at // 4 % 64) == list(range(64))   # every bank once


@pytest.mark.parametrize("RT,kv,NP", [(4, 4, 2), (4, 2, 2), (2, 4, 3), (2, 2, 3)])
def test_image_of_columns(RT, kv, NP):
    """put_image from all column tiles is read by lds_frag: row rho(i, c), places 8 g .."""
    img = np.full(RT * kv * NP * 512, -1, np.int64)
    for v0 in range(0, 128, 16):
        if v0 >= 32 * kv:
            continue
        v = v0 + 4 * G
        to = (v >> 5) * NP * 512 + (16 * ((v >> 3) & 3) + C) * 8 + (v & 7)
        for i in range(RT):
            for p in range(NP):
                for r in range(4):
                    at = to + (i * kv * NP + p) * 512 + r
                    assert (img[at] == -1).all()
                    img[at] = (rho(i, C) * 128 + v + r) * NP + p
    for i in range(RT):
        for k in range(kv):
            for p in range(NP):
                for e in range(8):
                    assert np.array_equal(img[((i * kv + k) * NP + p) * 512 + LANE * 8 + e], (rho(i, C) * 128 + 32 * k + 8 * G + e) * NP + p)


def test_state_blocks():
    """store_block, and the gradients' loads of its rows, at every size."""
    for dk in (1, 15, 48, 64, 96, 127, 128):
        for dv in (1, 16, 17, 80, 100, 128):
            blocks = -(-dv // 16)
            mem = np.full(dk * 16 * blocks, -1, np.int64)
            for j in range(blocks):
                for i in range(8 if dk > 64 else 4):
                    d = rho(i, C)
                    for r in range(4):
                        at = (16 * j * dk + d * 16 + 4 * G + r)[d < dk]
                        assert (mem[at] == -1).all()
                        mem[at] = (d * 128 + 16 * j + 4 * G + r)[d < dk]
            assert (mem >= 0).all()
            for i in range(8 if dk > 64 else 4):
                d = rho(i, C)
                for kv in range(4 if dv > 64 else 2):
                    block = 2 * kv + (G >> 1)
                    off = (np.where(16 * block < dv, block, 0) * dk + np.where(d < dk, d, 0)) * 16 + 8 * (G & 1)
                    for e in range(8):
                        assert off.min() >= 0 and (off + e).max() < len(mem)
                        v = 32 * kv + 8 * G + e
                        ok = (d < dk) & (v < dv)
                        assert np.array_equal(mem[off + e][ok], (d * 128 + v)[ok])


def groups(N, NW, first, RT=1):
    n = (N + 3) // 4
    return [[(g // n) * N + 4 * (g % n) + j for g in range(RT * n) if (g + first) % NW == w for j in range(min(4, N - 4 * (g % n)))]
            for w in range(NW)]


@pytest.mark.parametrize("N,RT", [(4, 4), (2, 4), (12, 2), (6, 2), (20, 1), (12, 1), (18, 1), (7, 1), (6, 1), (2, 1), (1, 1), (32, 1), (24, 1)])
@pytest.mark.parametrize("NW", [1, 8])
def test_fetches_bring_every_fragment_once(N, RT, NW):
    for first in (0, 4, 5, 7):
        assert sorted(f for w in groups(N, NW, first, RT) for f in w) == list(range(N * RT))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("DK", [64, 128])
def test_lds_sizes(bf16, DK):
    """What the chains and the gradients hold in LDS fits 160 KiB, and a fetch is at most 63 loads of a wave behind."""
    kIn, kOut, C_ = (1, 2, 64) if bf16 else (3, 3, 32)
    RT, KC, KD, DT = C_ // 16, C_ // 32, DK // 32, DK // 16
    tri, gates = KC * (KC + 1), -(-8 * C_ * 4 // 1024)
    rows, head, p_fwd, p_bwd = RT * KD * kIn, tri * 3 + gates, tri * kOut, tri * 3
    fwd = 2 * (2 * rows + head + p_fwd)
    bwd = 2 * (2 * rows + head + p_bwd)
    assert max(fwd + 4 + KD * kOut + RT, fwd + 16, bwd + 4 + 2 * RT + DT, bwd + 16) <= 160
    assert rows + p_fwd <= 63 and 2 * rows + head <= 63 and p_bwd + 2 <= 63
    for DV in (64, 128):
        KV, NW = DV // 32, max(DK, DV) // 16
        lds = (2 * rows + RT * KV * (kIn + 2 * kOut) + 2 * tri * kOut + 2 * gates) * 1024
        assert lds + (NW * C_ + 2 * NW + C_ + 2 * RT * RT * 16) * 4 <= 163840


@pytest.mark.parametrize("VB", [32, 64, 128])
def test_step_rows_and_columns(VB):
    cols = VB // 4
    groups = 256 // cols
    rows = 128 // groups
    tid = np.arange(256)
    cg, rg = tid % cols, tid // cols
    seen = np.zeros((128, VB), int)
    for i in range(rows):
        for j in range(4):
            np.add.at(seen, (i * groups + rg, 4 * cg + j), 1)
    assert (seen == 1).all()


def clamp(offs, T):
    return np.maximum.accumulate(np.clip(np.asarray(offs, np.int64), 0, T))


@pytest.mark.parametrize("log_c", [5, 6])
@pytest.mark.parametrize("T,offs", [(1000, [0, 7, 7, 400, 1000]), (64, [0, 64]), (130, list(range(131))), (500, [5, 3, 499, 9000]),
                                    (0, [0, 0]), (77, [80, 90])])
def test_chunks_fit_the_states(T, offs, log_c):
    """Sequences' chunks, numbered one after the other, never pass T >> log_c plus the sequences."""
    b = clamp(offs, T)
    n = (b[1:] - b[:-1] + (1 << log_c) - 1) >> log_c
    assert n.sum() <= (T >> log_c) + len(n)


def qk_pairs(D, half, halves):
    """Channels of both sides of every pair of a row, by lane: channel() and Spot."""
    lanes = 1
    while 16 * lanes < D:
        lanes *= 2
    out = []
    for lane in range(lanes):
        p0 = 8 * lane
        split = halves and p0 < half
        off = (p0, p0 + half) if split else (2 * p0, 2 * p0 + 8)
        fast = p0 + 8 <= half if split else 2 * p0 + 16 <= D
        chans = []
        for p in range(p0, p0 + 8):
            for s in range(2):
                d = p + s * half if halves and p < half else 2 * p + s
                chans.append(d if 2 * p < D + 1 and d < D else D)
        out.append((off, fast, split, chans))
    return lanes, out


@pytest.mark.parametrize("halves", [False, True])
def test_qk_channels(halves):
    for D in list(range(1, 70)) + [80, 96, 100, 127, 128, 192, 250, 256, 511, 512, 513, 1000, 1023, 1024]:
        for R in sorted({0, 2, D // 2 // 2 * 2, D // 2 * 2, D // 4 // 2 * 2, min(D // 2 * 2, 64)}):
            if R > D:
                continue
            lanes, rows = qk_pairs(D, R // 2, halves)
            assert lanes <= 64
            cells = [d for _, _, _, chans in rows for d in chans if d < D]
            assert sorted(cells) == list(range(D)), (D, R)
            for off, fast, split, chans in rows:
                if fast:   # the two runs are those channels
                    assert off[0] >= 0 and off[1] + 8 <= D
                    run = [off[0] + i for i in range(8)], [off[1] + i for i in range(8)]
                    if split:
                        assert chans[0::2] == run[0] and chans[1::2] == run[1]
                    else:
                        assert chans == run[0] + run[1]
            # the launch's choices of whole runs for all lanes that have any, and of one kind for all
            if D % 16 == 0 and (not halves or R == 0 or R // 2 % 8 == 0 or R == D):
                live = [row for lane, row in enumerate(rows) if 16 * lane < D]
                assert all(fast for _, fast, _, _ in live)
                assert all(d >= D for lane, row in enumerate(rows) if 16 * lane >= D for d in row[3])
                if not halves or R == 0 or R == D:
                    assert all(split == (halves and R > 0) for _, _, split, _ in live)


def qk_tokens(T, D, heads, most):
    lanes = 1
    while 16 * lanes < D:
        lanes *= 2
    rows, room = 256 // lanes, 2048 // (8 * lanes)
    n = max(1, min(room, max(min(-(-4 * rows // heads), -(-T // 1024)), min(rows // heads, T // 256))))
    turns = -(-(-(-T // n)) // most)
    return (min(n, -(-T // (most * turns))) if turns > 1 else n), lanes


def test_qk_turns_fit():
    for most in (1024, 4096):
        for T in (1, 2, 255, 1000, 1024, 1501, 5000, 8191, 40000, 1 << 20, 1 << 40):
            for D in (1, 16, 17, 64, 80, 128, 300, 1024):
                for heads in (1, 3, 10, 40, 1000):
                    n, lanes = qk_tokens(T, D, heads, most)
                    assert n >= 1 and n * 8 * lanes <= 2048 and 2 * 8 * lanes <= 1024
                    groups = min(-(-T // n), most)
                    assert -(-(-(-T // n)) // groups) * groups * n >= T
