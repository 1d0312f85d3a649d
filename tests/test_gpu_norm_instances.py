"""det_block_norm and its backward where outputs are larger than the last-level cache,
with one gate per token, none, and more than 8192 channels: every row has the bits of a
small call, and the parameter gradients agree with float64 column sums."""
import pytest
import torch

from tests import ref64
from tests.test_gpu_block_norm import BF, F32, bwd, fwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,T,D,gate", [(BF, 4200, 16384, "row"), (BF, 3000, 16000, "full"), (F32, 2200, 16384, "none"),
                                            (F32, 2100, 16001, "full"), (BF, 16500, 4100, "row"), (F32, 9000, 4096, "full"),
                                            (F32, 70000, 500, "none")])
def test_outputs_past_the_caches(dtype, T, D, gate):
    assert 2 * T * D * torch.finfo(dtype).bits // 8 >= 256 << 20 or gate == "full"
    g = torch.Generator(device="cuda").manual_seed(3)

    def rows(n):
        return torch.randn(T, n, device="cuda", dtype=dtype, generator=g)
    d = dict(x=rows(D), f=rows(D), gate={"none": None, "row": rows(1), "full": rows(D)}[gate], dy=rows(D), dh=rows(D),
             **{k: 1 + 0.1 * torch.randn(D, device="cuda", generator=g) for k in ("w_post", "alpha", "w_pre")})
    o = fwd(d)
    r = bwd(d, o)
    for a in range(0, T, T // 6):
        e = {k: v[a:a + 5] if v is not None and v.dim() == 2 else v for k, v in d.items()}
        p = fwd(e)
        assert all(torch.equal(p[k], o[k][a:a + 5]) for k in o), a
        q = bwd(e, p)
        assert all(q[k] is None or torch.equal(q[k], r[k][a:a + 5]) for k in ("dx", "df", "dgate")), a
    # dw_pre = sum dh yh from the stored y (off by half a step each) and the call's factors; a workgroup's chain of at
    # most T / 256 rows in float32
    want, mag = torch.zeros(D, device="cuda", dtype=torch.float64), torch.zeros(D, device="cuda", dtype=torch.float64)
    for a in range(0, T, 1000):
        s = slice(a, a + 1000)
        t = d["dh"][s].double() * o["y"][s].double() * o["rstd_pre"][s].double()[:, None]
        want += t.sum(0)
        mag += t.abs().sum(0)
    tol = (ref64.HALF_STEP[dtype] + (100 + T / 256) * ref64.U) * mag
    assert bool(((r["dw_pre"].double() - want).abs() <= tol).all())
