"""CPU replay of how det_delta_rule_bwd's kernel forms dg's sums over the pairs i >= t > j of a chunk, with its names:
from runs of four columns j of the pair tiles, no pair that does not cross t being added and taken off again."""
import numpy as np
import pytest

from tests.test_mixer_bounds import C as COL, G, rho, rho_tile


@pytest.mark.parametrize("C", [32, 64])
@pytest.mark.parametrize("NW", [4, 8])
def test_crossing_sums(C, NW):
    RT, KC, runs = C // 16, C // 32, C // 4
    pairs = [(p >> 1, p & 1) if p < 4 else (2 + ((p - 4) >> 2), (p - 4) & 3) for p in range(2 * KC * (KC + 1))]
    E = np.tril(np.random.default_rng(C).integers(1, 1000, (C, C)).astype(float), -1)   # whole: sums are exact
    run_e, near_e, far_e = np.full((C, runs), np.nan), np.full((RT, C), np.nan), np.full(C, np.nan)
    for i, j in pairs:
        row, at0 = rho(i, COL), rho(j, 4 * G)
        ev = np.stack([E[row, at0 + r] for r in range(4)])
        assert np.isnan(run_e[row, at0 >> 2]).all()
        run_e[row, at0 >> 2] = ev.sum(0)
        before = ev[0].copy()
        for r in (1, 2, 3):
            masked = np.where(row >= at0 + r, before, 0.0)
            for g in range(4):
                assert np.isnan(near_e[i, at0[16 * g] + r])
                near_e[i, at0[16 * g] + r] = masked[16 * g:16 * g + 16].sum()
            before += ev[r]
    lane = np.arange(64)
    for m in [m for w in range(NW) for m in range(w, runs, NW)]:
        p = np.where(np.arange(runs) < m, run_e[lane & (C - 1)], 0.0).sum(1)
        t = [0.0] * 4
        t[3] = np.where((lane >= 4 * m + 4) & (lane < C), p, 0.0).sum()
        for r in (3, 2, 1, 0):
            t[r] = (t[r + 1] if r < 3 else t[3]) + p[4 * m + r]
        far_e[4 * m:4 * m + 4] = t
    for t in range(C):
        got = far_e[t] + sum(near_e[i, t] for i in range(RT) if i // 2 >= rho_tile(t) // 2 and t & 3)
        assert got == E[t:, :t].sum(), t
