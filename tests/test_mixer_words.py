"""CPU replay of where the delta rule's kernels hold their operands in LDS, with three words for all but bf16 inputs
(the same names as in their sources)."""
import pytest


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("DK", [64, 128])
def test_chains_fit(bf16, DK):
    kIn, C = (1, 64) if bf16 else (3, 32)
    RT, KC, KD, DT = C // 16, C // 32, DK // 32, DK // 16
    tri, gates = 3 * KC * (KC + 1), -(-8 * C * 4 // 1024)
    rows, head = RT * KD * kIn, tri + gates
    buf = 2 * rows + head + tri
    assert 2 * buf + max(4 + 3 * KD + RT, 4 + 2 * RT + DT, 16) <= 160
    # the counted waits: at most 63 loads of a wave
    assert rows + tri <= 63 and 2 * rows + head <= 63 and tri + 2 <= 63


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("DK", [64, 128])
@pytest.mark.parametrize("DV", [64, 128])
def test_gradients_fit_and_share(bf16, DK, DV):
    kIn, C = (1, 64) if bf16 else (3, 32)
    RT, KC, KD, KV, NW = C // 16, C // 32, DK // 32, DV // 32, max(DK, DV) // 16
    nK, nO, nV, nTri, nGate = RT * KD * kIn, RT * KV * kIn, RT * KV * 3, KC * (KC + 1) * 3, -(-8 * C * 4 // 1024)
    share = 2 * nK + nO + 2 * nV + 2 * nTri + 2 * nGate > 148
    assert share == (bf16 and DV == 128)
    oN = 2 * nK
    oO = oN + nV
    oY = oO + nO
    oA = oY if share else oY + nV
    oZ = oA + nTri
    oGate = oY + nV if share else oZ + nTri
    floats = 2 * NW * C + NW + C + C * (C // 4 + 4) + RT * C + C
    assert (oGate + 2 * nGate) * 1024 + 4 * floats + 64 <= 163840
    # what comes for the next head while the pair matrices are read: none of theirs
    n, y, o = range(oN, oN + nV), range(oY, oY + nV), range(oO, oO + nO)
    pairs = set(range(oA, oA + 2 * nTri))
    assert not pairs & (set(n) | set(o) | set(range(2 * nK)) | set(range(oGate, oGate + 2 * nGate)))
    assert pairs <= set(y) if share else not pairs & set(y)
