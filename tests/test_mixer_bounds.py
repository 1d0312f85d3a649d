"""CPU replay of the index arithmetic of the delta rule and query and key norm kernels
(the same names as in their sources): every element is written by one lane, operands
agree on the summed places, and every address formed lies inside its buffer."""
import numpy as np
import pytest


def image(RT, KS):
    group, frag = 272, 4 * 272
    tile = (KS * frag + 239) // 256 * 256 + 16
    return group, frag, tile, RT * tile


def at(RT, KS, row, place):
    group, frag, tile, _ = image(RT, KS)
    return (row >> 4) * tile + (place >> 5) * frag + ((place >> 2) & 3) * group + (row & 15) * 16 + ((place >> 4) & 1) * 8


@pytest.mark.parametrize("RT,KS", [(4, 4), (4, 2), (8, 2), (2, 4), (2, 2), (8, 1), (4, 1), (2, 1)])
def test_image(RT, KS):
    """Four places of every row have eight bytes of their own; a lane's fragment holds the places 32 ks + 4 g + r and
    32 ks + 16 + 4 g + r of its row, in this order."""
    group, frag, tile, word = image(RT, KS)
    row, place = np.meshgrid(np.arange(16 * RT), np.arange(0, 32 * KS, 4), indexing="ij")
    a = at(RT, KS, row, place).ravel()
    assert a.min() >= 0 and a.max() + 8 <= word and tile % 16 == 0 and tile >= KS * frag
    cells = (a[:, None] + np.arange(8)[None]).ravel()
    assert len(np.unique(cells)) == len(cells)
    lane = np.arange(64)
    for rt in range(RT):
        for ks in range(KS):
            base = rt * tile + ks * frag + (lane >> 4) * group + (lane & 15) * 16
            assert (base % 16 == 0).all() and base.max() + 16 <= word
            for e in range(8):
                want = 32 * ks + 16 * (e >> 2) + 4 * (lane >> 4) + (e & 3)
                got = at(RT, KS, 16 * rt + (lane & 15), want & ~3) + (want & 3) * 2
                assert np.array_equal(got, base + 2 * e)


@pytest.mark.parametrize("C", [64, 32])
@pytest.mark.parametrize("DK", [64, 128])
@pytest.mark.parametrize("NW", [1, 2, 4, 8])
def test_chunk_staging(C, DK, NW):
    """Blocks of four tokens by four channels, and of four by four of the inverse, over the threads."""
    threads = 64 * NW
    blocks = C * DK // 16
    seen = np.zeros((C, DK), int)
    for b in range(-(-blocks // threads)):
        i = b * threads + np.arange(threads)
        i = i[i < blocks]
        t, d = i // (DK // 4) * 4, i % (DK // 4) * 4
        for j in range(4):
            for e in range(4):
                np.add.at(seen, (t + j, d + e), 1)
    assert (seen == 1).all()
    blocks, seen = C * C // 16, np.zeros((C, C), int)
    for b in range(-(-blocks // threads)):
        i = b * threads + np.arange(threads)
        i = i[i < blocks]
        r, c = i // (C // 4) * 4, i % (C // 4) * 4
        for j in range(4):
            for e in range(4):
                np.add.at(seen, (r + j, c + e), 1)
    assert (seen == 1).all()


@pytest.mark.parametrize("RT,NW", [(4, 1), (4, 2), (4, 4), (4, 8), (2, 1), (2, 4), (2, 8)])
def test_pair_tiles(RT, NW):
    n = RT * (RT + 1) // 2
    tiles = []
    for wave in range(NW):
        for p in range(wave, n, NW):
            i, j = 0, p
            while j > i:
                i += 1
                j -= i
            assert p == i * (i + 1) // 2 + j and j <= i < RT
            tiles.append((i, j))
    assert sorted(tiles) == [(i, j) for i in range(RT) for j in range(i + 1)]


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
            # the launch's choice of one kind for all lanes
            if D == 16 * lanes and (not halves or R == 0 or R == D):
                assert all(fast for _, fast, _, _ in rows)
                assert all(split == (halves and R > 0) for _, _, split, _ in rows)


def qk_tokens(T, D, heads):
    lanes = 1
    while 16 * lanes < D:
        lanes *= 2
    rows = 256 // lanes
    n = min(-(-4 * rows // heads), 1 if T < 1024 else T // 1024, 2048 // (8 * lanes))
    return max(n, 1), lanes


def test_qk_turns_fit():
    for T in (1, 1000, 1024, 5000, 40000, 1 << 20):
        for D in (1, 16, 17, 64, 128, 300, 1024):
            for heads in (1, 3, 40, 1000):
                n, lanes = qk_tokens(T, D, heads)
                assert n * 8 * lanes <= 2048 and 2 * 8 * lanes <= 1024
