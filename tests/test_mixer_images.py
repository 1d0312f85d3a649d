"""CPU replay of the float32 images of N and dY that the delta rule's chains leave and its gradients read (the same
names as in their sources): every element is written once, and a wave's lanes get the places of a fragment."""
import numpy as np
import pytest

from tests.test_mixer_bounds import C as COL, G, LANE, rho


@pytest.mark.parametrize("C,DV", [(64, 64), (64, 128), (32, 64), (32, 128)])
def test_float_images(C, DV):
    RT, kv = C // 16, DV // 32
    img = np.full(C * DV, -1)
    for v0 in range(0, 128, 16):
        if v0 >= 32 * kv:
            continue
        v = v0 + 4 * G
        to = (v >> 5) * 512 + ((v >> 2) & 1) * 256 + (16 * ((v >> 3) & 3) + COL) * 4
        for i in range(RT):
            for r in range(4):
                at = to + i * kv * 512 + r
                assert (img[at] == -1).all() and (to % 4 == 0).all()
                img[at] = rho(i, COL) * 128 + v + r
    assert (img >= 0).all()
    for NW in {DV // 16, 8}:
        each, seen = -(-RT * kv // NW), set()
        for wave in range(NW):
            for u in range(each):
                f = wave + u * NW
                if RT * kv % NW and f >= RT * kv:
                    continue
                assert f < RT * kv and f not in seen
                seen.add(f)
                for e in range(8):   # the fragment's row rho(i, c), places 32 k + 8 g .. of it
                    at = f * 512 + (e >> 2) * 256 + LANE * 4 + (e & 3)
                    assert np.array_equal(img[at], rho(f // kv, COL) * 128 + 32 * (f % kv) + 8 * G + e)
        assert len(seen) == RT * kv
