"""CPU replay of the index arithmetic of the router, distillation and norm kernels
(the same names as in their sources): every element is read and written by
exactly one lane, and every address formed lies inside its buffer."""
import numpy as np
import pytest


def cdiv(a, b):
    return -(-a // b)


def cols(N, lanes, tiny):
    """Cols::set for every lane: (base, lo, hi)."""
    col = np.arange(lanes) * 8
    hi = N if tiny and N < 8 else 8
    base = np.where(col + 8 <= N, col, np.where((col < N) & (hi == 8), N - 8, 0))
    lo = np.where(col < N, col - base, 8)
    return base, lo, hi


def check_cols(N, lanes, tiny):
    base, lo, hi = cols(N, lanes, tiny)
    width = hi if tiny and N < 8 else 8          # elements a lane loads
    assert base.min() >= 0 and (base + width).max() <= N, (N, lanes)
    j = np.arange(8)
    own = (j[None] >= lo[:, None]) & (j[None] < hi if tiny else np.ones((1, 8), bool))
    cells = (base[:, None] + j[None])[own]
    assert np.array_equal(np.sort(cells), np.arange(N)), (N, lanes)


def router_lanes(E):
    lpr, ni = 1, 2 if E > 16 else 1
    while lpr * ni * 8 < E:
        lpr *= 2
    return lpr, ni


def test_router_columns():
    for E in range(1, 1025):
        lpr, ni = router_lanes(E)
        check_cols(E, lpr * ni, tiny=lpr == 1)


def norm_threads(D):
    t = 64
    while t < 1024 and t * 8 < D:
        t *= 2
    return t


def test_norm_columns():
    for D in list(range(1, 2100)) + [4095, 4096, 4097, 8191, 8192, 8193, 10000, 16383, 16384]:
        t = norm_threads(D)
        check_cols(D, t * (2 if D > 8192 else 1), tiny=t == 64)


def tile_log(T, E, threads, ahead, target):
    lpr, ni = router_lanes(E)
    step = threads // 64 * (64 // lpr) * (ahead // ni)
    lg = 0
    while (1 << lg) < step or (T >> lg) > target:
        lg += 1
    return lg


def clamp_bounds(offs, T):
    return np.maximum.accumulate(np.clip(np.asarray(offs, np.int64), 0, T))


@pytest.mark.parametrize("T,E,offs", [(65536, 256, [0, 7, 7, 40000, 65536]), (9001, 160, [5, 100, 9000]),
                                      (5000, 1, [0, 5000]), (3000, 1024, [0, 1, 2, 3, 2999]),
                                      (777, 600, [9, 3, 2000, 100]), (0, 4, [0, 0])])
def test_router_tiles_cover_every_token_once(T, E, offs):
    """segment_tile over the launch's worst-case grid, and every lane group's rows of a tile."""
    b = clamp_bounds(offs, T)
    S = len(b) - 1
    for threads, ahead, target in ((512, 2, 512), (256, 2, 1024)):
        lg = tile_log(T, E, threads, ahead, target)
        grid = cdiv(T, 1 << lg) + S
        tiles = [(s, r) for s in range(S) for r in range(b[s], b[s + 1], 1 << lg)]
        assert len(tiles) <= grid
        seen = np.zeros(T, int)
        lpr, ni = router_lanes(E)
        rpw, W, a = 64 // lpr, threads // 64, ahead // ni
        for s, r0 in tiles:
            r1 = min(r0 + (1 << lg), b[s + 1])
            for wave in range(W):
                for r in range(r0 + wave * rpw, r1, a * W * rpw):
                    rows = (r + np.arange(a)[:, None] * W * rpw + np.arange(rpw)[None]).ravel()
                    seen[rows[rows < r1]] += 1
        inside = np.zeros(T, int)
        inside[b[0]:b[-1]] = 1
        assert np.array_equal(seen, inside)


def fwd_split(T, V):
    threads = 1024 if T < 512 or V >= 131072 else 512 if V >= 65536 else 256
    want = 1 if T >= 256 or T == 0 else cdiv(512, T)
    n = max(1, min(want, cdiv(V, 1 << 18)))
    piece = cdiv(cdiv(V, n), 8192) * 8192
    return threads, cdiv(V, piece), piece


@pytest.mark.parametrize("T,V", [(1, 1), (3, 131072), (3, 600001), (1021, 50001), (2000, 2049), (7, 8193), (1, 262145),
                                 (300, 16384), (600, 7), (5000, 70001), (5000, 140001)])
def test_distill_forward_pieces_cover_every_word_once(T, V):
    threads, n, piece = fwd_split(T, V)
    assert n >= 1 and (n - 1) * piece < V <= n * piece
    step = threads * 8
    seen = np.zeros(V, int)
    for k in range(n):
        i, c1 = k * piece, min(V, (k + 1) * piece)
        for u in (8, 2):
            while i + u * step <= c1:
                seen[i:i + u * step] += 1
                i += u * step
        while i < c1:
            seen[i:min(i + step, c1)] += 1
            i += step
    assert (seen == 1).all()


@pytest.mark.parametrize("V", [1, 5, 63, 64, 65, 8191, 8192, 8193, 8255, 8256, 8257, 50001, 131072, 131100])
@pytest.mark.parametrize("phase", [0, 2, 14, 126])
@pytest.mark.parametrize("K", [0, 64, 128, 129, 1024])
def test_distill_backward_pieces_cover_every_word_once(V, phase, K):
    """Pieces from the first 128-byte line of dz (bf16, the row starting at byte `phase` of a line), the lead with the
    first; the loops of four, two and one accesses."""
    piece = cdiv(max(64 * K, 8192), 8192) * 8192
    step = 2048
    lead = min((-phase % 128) // 2, V)
    assert lead <= 256
    seen = np.zeros(V, int)
    for k in range(cdiv(V, piece)):
        at = k * piece
        c0, c1 = (lead + at if at else 0), min(lead + at + piece, V)
        if c0 >= c1:
            continue
        i = lead + at
        if at == 0:
            seen[:lead] += 1
        for u in (4, 2):
            while i + u * step <= c1:
                assert (phase // 2 + i) % 64 == 0
                seen[i:i + u * step] += 1
                i += u * step
        while i < c1:
            seen[i:min(i + step, c1)] += 1
            i += step
    assert (seen == 1).all()


def groups_for(T, D, bwd):
    full = 256 * (1024 // norm_threads(D)) if bwd else 512 * (2048 // norm_threads(D))
    g = max(cdiv(T, 6 if bwd else 3), 512 if bwd else 1024)
    return min(T, min(g, full))


def test_norm_rows_and_slots():
    for T in (1, 5, 511, 512, 3001, 8192, 20011, 100000):
        for D in (1, 64, 512, 513, 1407, 2048, 4096, 8192, 16384):
            for bwd in (False, True):
                G = groups_for(T, D, bwd)
                assert 1 <= G <= T
            # the fold's waves read every slot once, and only slots
            seen = np.zeros(G, int)
            for wave in range(16):
                for b in range(wave, G, 256):
                    k = b + 16 * np.arange(16)
                    seen[k[k < G]] += 1
                    assert (np.where(k < G, k, wave) < G).all()
            assert (seen == 1).all()
