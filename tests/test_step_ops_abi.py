"""Refusals of the router balance, distillation and block norm entry points: every
one is made on the host before any HIP call (CPU only, no kernel launches)."""
import ctypes
import os

import pytest
import torch

import deterministic_gradient_reductions_amd as dg

pytestmark = pytest.mark.skipif(not os.path.exists(dg.library_path), reason="libdetgrad.so not built")

P = ctypes.c_void_p
INVALID, UNSUPPORTED, WORKSPACE, OVERLAP = (dg.DET_ERR_INVALID_ARG, dg.DET_ERR_UNSUPPORTED, dg.DET_ERR_WORKSPACE,
                                            dg.DET_ERR_OVERLAP)
MB = 1 << 20
A = [P(0x10000000 + i * 64 * MB) for i in range(24)]   # never dereferenced: every call fails validation first
BIG = 32 * MB


def run(fn, defaults, **kw):
    assert set(kw) <= set(defaults), set(kw) - set(defaults)
    return getattr(dg.lib(), fn)(*{**defaults, **kw}.values())


ROUTER = dict(logits=A[0], ld=64, dtype=0, ids=A[1], ids_ld=4, T=100000, E=64, K=4, offs=A[2], S=2, score=0, coeff=0.01,
              counts=A[3], prob_sum=A[4], loss=A[5], ws=A[6], ws_bytes=BIG, stream=None)
ROUTER_BWD = dict(dlogits=A[0], ld_d=64, logits=A[1], ld=64, dtype=0, T=100, E=64, K=4, offs=A[2], S=2, counts=A[3],
                  dloss=A[4], score=0, coeff=0.01, stream=None)
DISTILL = dict(logits=A[0], ld=300000, dtype=0, ids=A[1], ids_ld=8, teacher=A[2], teacher_ld=8, teacher_dtype=1, T=10,
               V=300000, K=8, tau=1.0, loss=A[3], lse=A[4], ws=A[5], ws_bytes=BIG, stream=None)
DISTILL_BWD = dict(dlogits=A[0], ld_d=30000, logits=A[1], ld=30000, dtype=0, ids=A[2], ids_ld=8, teacher=A[3],
                   teacher_ld=8, teacher_dtype=1, T=10, V=30000, K=8, tau=1.0, lse=A[4], dloss=A[5], stream=None)
NORM = dict(x=A[0], x_ld=64, f=A[1], f_ld=64, gate=A[2], gate_ld=64, gate_cols=64, w_post=A[3], alpha=A[4], w_pre=A[5],
            dtype=0, T=100, D=64, eps=1e-6, y=A[6], y_ld=64, h=A[7], h_ld=64, rstd_post=A[8], rstd_pre=A[9],
            stream=None)
NORM_BWD = dict(dy=A[0], dy_ld=64, dh=A[1], dh_ld=64, x=A[2], x_ld=64, f=A[3], f_ld=64, gate=A[4], gate_ld=64,
                gate_cols=64, w_post=A[5], alpha=A[6], w_pre=A[7], rstd_post=A[8], rstd_pre=A[9], dtype=0, T=100, D=64,
                dx=A[10], dx_ld=64, df=A[11], df_ld=64, dgate=A[12], dgate_ld=64, dw_post=A[13], dalpha=A[14],
                dw_pre=A[15], ws=A[16], ws_bytes=BIG, stream=None)
FAR = P(A[0].value + 16)    # inside the first buffer

CASES = [
    ("det_router_balance", ROUTER, INVALID, [dict(T=-1), dict(S=-1), dict(E=0), dict(K=0), dict(dtype=2), dict(score=2),
                                             dict(ld=63), dict(ids_ld=3), dict(coeff=float("nan")),
                                             dict(coeff=float("inf")), dict(logits=None), dict(ids=None),
                                             dict(offs=None), dict(counts=None), dict(prob_sum=None), dict(loss=None)]),
    ("det_router_balance", ROUTER, UNSUPPORTED, [dict(E=1025, ld=1025), dict(S=65536), dict(K=65537, ids_ld=65537),
                                                 dict(T=1 << 29, K=4), dict(ld=1 << 60), dict(ids_ld=1 << 60)]),
    ("det_router_balance", ROUTER, INVALID, [dict(logits=P(A[0].value + 1)), dict(ids=P(A[1].value + 2)),
                                             dict(counts=P(A[3].value + 1)), dict(loss=P(A[5].value + 2))]),
    ("det_topk_distill_bwd", DISTILL_BWD, INVALID, [dict(dlogits=P(A[0].value + 1)), dict(teacher=P(A[3].value + 2))]),
    ("det_topk_distill", DISTILL, UNSUPPORTED, [dict(T=1 << 24, V=8, ld=8)]),
    ("det_topk_distill_bwd", DISTILL_BWD, UNSUPPORTED, [dict(T=1 << 24, V=8, ld=8, ld_d=8)]),
    ("det_block_norm", NORM, INVALID, [dict(x=P(A[0].value + 1)), dict(w_pre=P(A[5].value + 2))]),
    ("det_block_norm_bwd", NORM_BWD, INVALID, [dict(dgate=P(A[12].value + 1)), dict(dw_pre=P(A[15].value + 2))]),
    ("det_router_balance", ROUTER, WORKSPACE, [dict(ws=None), dict(ws=P(A[6].value + 16)), dict(ws_bytes=300)]),
    ("det_router_balance", ROUTER, OVERLAP, [dict(counts=FAR), dict(loss=FAR), dict(prob_sum=A[3]), dict(loss=A[1]),
                                             dict(ws=A[0]), dict(counts=A[2]), dict(loss=A[6])]),
    ("det_router_balance_bwd", ROUTER_BWD, INVALID, [dict(T=-1), dict(E=0), dict(K=0), dict(dtype=3), dict(score=-1),
                                                     dict(ld=63), dict(ld_d=63), dict(dlogits=None), dict(logits=None),
                                                     dict(offs=None), dict(counts=None), dict(dloss=None)]),
    ("det_router_balance_bwd", ROUTER_BWD, UNSUPPORTED, [dict(E=2000, ld=2000, ld_d=2000), dict(ld_d=1 << 60)]),
    ("det_router_balance_bwd", ROUTER_BWD, OVERLAP, [dict(dlogits=A[1]), dict(counts=FAR), dict(dloss=FAR)]),
    ("det_topk_distill", DISTILL, INVALID, [dict(T=-1), dict(V=0), dict(K=-1), dict(dtype=2), dict(teacher_dtype=2),
                                            dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")),
                                            dict(tau=float("inf")), dict(tau=1e-9), dict(ld=299999), dict(ids_ld=7),
                                            dict(teacher_ld=7), dict(logits=None), dict(ids=None), dict(teacher=None),
                                            dict(loss=None), dict(lse=None)]),
    ("det_topk_distill", DISTILL, UNSUPPORTED, [dict(K=1025, ids_ld=1025, teacher_ld=1025), dict(V=1 << 31, ld=1 << 31),
                                                dict(T=1 << 32), dict(ld=1 << 60)]),
    ("det_topk_distill", DISTILL, WORKSPACE, [dict(ws=None), dict(ws=P(A[5].value + 8)), dict(ws_bytes=256)]),
    ("det_topk_distill", DISTILL, OVERLAP, [dict(loss=FAR), dict(lse=A[3]), dict(ws=A[0]), dict(lse=A[2])]),
    ("det_topk_distill_bwd", DISTILL_BWD, INVALID, [dict(T=-1), dict(V=0), dict(tau=0.0), dict(ld=29999),
                                                    dict(ld_d=29999), dict(dlogits=None), dict(lse=None),
                                                    dict(dloss=None), dict(ids=None)]),
    ("det_topk_distill_bwd", DISTILL_BWD, UNSUPPORTED, [dict(K=1025, ids_ld=1025, teacher_ld=1025),
                                                        dict(ld_d=1 << 60)]),
    ("det_topk_distill_bwd", DISTILL_BWD, OVERLAP, [dict(dlogits=A[1]), dict(ids=FAR), dict(lse=FAR), dict(dloss=FAR)]),
    ("det_block_norm", NORM, INVALID, [dict(T=-1), dict(D=-1), dict(dtype=2), dict(eps=-1e-6), dict(eps=float("nan")),
                                       dict(x_ld=63), dict(f_ld=63), dict(gate_ld=63), dict(y_ld=63), dict(h_ld=63),
                                       dict(gate_cols=2), dict(x=None), dict(f=None), dict(y=None), dict(h=None),
                                       dict(rstd_pre=None), dict(rstd_post=None), dict(w_pre=None),
                                       dict(w_post=None)]),
    ("det_block_norm", NORM, UNSUPPORTED, [dict(D=16385, x_ld=16385), dict(x_ld=1 << 60)]),
    ("det_block_norm", NORM, OVERLAP, [dict(y=A[0]), dict(h=A[6]), dict(rstd_post=FAR), dict(y=A[2]), dict(h=A[5])]),
    ("det_block_norm_bwd", NORM_BWD, INVALID, [dict(T=-1), dict(dtype=2), dict(dy_ld=63), dict(dh_ld=63), dict(x_ld=63),
                                               dict(f_ld=63), dict(dx_ld=63), dict(df_ld=63), dict(dgate_ld=63),
                                               dict(gate_cols=63), dict(dy=None), dict(f=None), dict(x=None),
                                               dict(dx=None), dict(df=None), dict(dgate=None), dict(dh=None),
                                               dict(w_pre=None), dict(dw_pre=None), dict(rstd_pre=None),
                                               dict(dw_post=None), dict(rstd_post=None), dict(dalpha=None),
                                               dict(alpha=None), dict(gate=None)]),
    ("det_block_norm_bwd", NORM_BWD, UNSUPPORTED, [dict(D=16385), dict(dy_ld=1 << 60)]),
    ("det_block_norm_bwd", NORM_BWD, WORKSPACE, [dict(ws=None), dict(ws=P(A[16].value + 4)), dict(ws_bytes=512)]),
    ("det_block_norm_bwd", NORM_BWD, OVERLAP, [dict(dx=A[0]), dict(df=A[10]), dict(dgate=A[4]), dict(dw_pre=A[13]),
                                               dict(dalpha=FAR), dict(ws=A[3])]),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_refusals(i):
    fn, defaults, status, cases = CASES[i]
    for kw in cases:
        assert run(fn, defaults, **kw) == status, (fn, kw, dg.lib().det_last_error())
        assert dg.lib().det_last_error()


def test_empty_problems_touch_nothing():
    none = {k: None for k, v in ROUTER.items() if isinstance(v, P)}
    assert run("det_router_balance", ROUTER, **{**none, "S": 0}) == dg.DET_OK
    none = {k: None for k, v in ROUTER_BWD.items() if isinstance(v, P)}
    assert run("det_router_balance_bwd", ROUTER_BWD, **{**none, "T": 0}) == dg.DET_OK
    assert run("det_router_balance_bwd", ROUTER_BWD, **{**none, "S": 0}) == dg.DET_OK
    for fn, d in (("det_topk_distill", DISTILL), ("det_topk_distill_bwd", DISTILL_BWD), ("det_block_norm", NORM),
                  ("det_block_norm_bwd", NORM_BWD)):
        assert run(fn, d, **{**{k: None for k, v in d.items() if isinstance(v, P)}, "T": 0}) == dg.DET_OK
    assert run("det_block_norm", NORM, **{**{k: None for k, v in NORM.items() if isinstance(v, P)}, "D": 0}) == dg.DET_OK


def test_workspace_sizes():
    assert dg.det_router_balance_workspace_size(100, 64, 4, 0) == 0
    assert dg.det_router_balance_workspace_size(100, 64, 4, 2) == 0     # a workgroup per sequence
    assert dg.det_router_balance_workspace_size(100000, 64, 4, 2) > 256 + 2 * 64 * 8
    assert dg.det_topk_distill_workspace_size(0, 1000, 4) == 0
    assert dg.det_topk_distill_workspace_size(2000, 131072, 4) == 0     # a workgroup per row
    assert dg.det_topk_distill_workspace_size(3, 131072, 4) == 0
    assert dg.det_topk_distill_workspace_size(3, 300000, 4) >= 256 + 3 * 8 * 2
    assert dg.det_block_norm_bwd_workspace_size(0, 64) == 0
    assert dg.det_block_norm_bwd_workspace_size(1, 64) >= 256 + 2 * 64 * 4
    n = ctypes.c_size_t()
    L = dg.lib()
    assert L.det_router_balance_workspace_size(100, 64, 4, 2, None) == INVALID
    assert L.det_router_balance_workspace_size(100, 1025, 4, 2, ctypes.byref(n)) == UNSUPPORTED
    assert L.det_topk_distill_workspace_size(10, 100, 2000, ctypes.byref(n)) == UNSUPPORTED
    assert L.det_block_norm_bwd_workspace_size(10, 20000, ctypes.byref(n)) == UNSUPPORTED


def test_binding_refusals():
    """Shapes, dtypes, strides and devices are checked before any library call (CPU tensors suffice)."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    z, ids, offs = torch.zeros(6, 8, dtype=bf), torch.zeros(6, 2, dtype=i32), torch.tensor([0, 6], dtype=i32)
    cnt, ps, ls = torch.zeros(1, 8, dtype=i32), torch.zeros(1, 8), torch.zeros(1)

    def refuse(exc, fn, *a, **k):
        with pytest.raises(exc):
            fn(*a, **k)
    f = dg.det_router_balance
    refuse(TypeError, f, z.half(), ids, offs, cnt, ps, ls)
    refuse(TypeError, f, z, ids.long(), offs, cnt, ps, ls)
    refuse(TypeError, f, z, ids, offs.long(), cnt, ps, ls)
    refuse(TypeError, f, z, ids, offs, cnt.float(), ps, ls)
    refuse(TypeError, f, z, ids, offs, cnt, ps.double(), ls)
    refuse(ValueError, f, z, ids[:5], offs, cnt, ps, ls)
    refuse(ValueError, f, z, ids, offs, cnt, ps, torch.zeros(2))
    refuse(ValueError, f, z, ids, offs, torch.zeros(2, 8, dtype=i32), ps, ls)
    refuse(ValueError, f, torch.zeros(8, 6, dtype=bf).t(), ids, offs, cnt, ps, ls)
    refuse(ValueError, f, z, ids, offs, cnt, ps, ls, score="tanh")
    refuse(ValueError, f, z, ids, offs, cnt, ps, ls)                        # not on a GPU
    f = dg.det_router_balance_bwd
    refuse(TypeError, f, z.float(), z, offs, cnt, ls, 2)
    refuse(ValueError, f, z[:5].clone(), z, offs, cnt, ls, 2)
    refuse(ValueError, f, z.clone(), z, offs, cnt, ls, 2)
    t, lse = torch.zeros(6, 2), torch.zeros(6)
    f = dg.det_topk_distill
    refuse(TypeError, f, z.double(), ids, t, lse, lse.clone())
    refuse(TypeError, f, z, ids, t.half(), lse, lse.clone())
    refuse(TypeError, f, z, ids.long(), t, lse, lse.clone())
    refuse(ValueError, f, z, ids, torch.zeros(6, 3), lse, lse.clone())
    refuse(ValueError, f, z, ids, t, torch.zeros(5), lse.clone())
    refuse(ValueError, f, z, ids, t, torch.zeros(12)[::2], lse.clone())
    refuse(ValueError, f, z, ids, t, lse, lse.clone())
    f = dg.det_topk_distill_bwd
    refuse(TypeError, f, z.float(), z, ids, t, lse, lse)
    refuse(TypeError, f, z.clone(), z, ids, t, lse.double(), lse)
    refuse(ValueError, f, z.clone(), z, ids, t, lse, lse)
    x, w = torch.zeros(6, 8), torch.zeros(8)
    f = dg.det_block_norm
    refuse(TypeError, f, x.half(), x.half(), x.half())
    refuse(TypeError, f, x, x.bfloat16(), x.clone())
    refuse(TypeError, f, x, x, x.clone(), w_post=w.bfloat16())
    refuse(ValueError, f, x, x, x.clone(), gate=torch.zeros(6, 2))
    refuse(ValueError, f, x, x, x.clone(), w_post=torch.zeros(7))
    refuse(ValueError, f, x, x[:5], x.clone())
    refuse(ValueError, f, x, torch.zeros(6, 16)[:, ::2], x.clone())
    refuse(ValueError, f, x, x, x.clone())
    f = dg.det_block_norm_bwd
    refuse(TypeError, f, x, x.bfloat16(), x, x.clone(), x.clone())
    refuse(ValueError, f, x, x, x, x.clone(), x.clone(), gate=torch.zeros(5, 1))
    refuse(ValueError, f, x, x, x, x.clone(), x.clone(), alpha=w, dalpha=torch.zeros(9))
    refuse(ValueError, f, x, x, x, x.clone(), x.clone())
