"""Refusals of the delta rule and query and key norm entry points: every one is made on
the host before any HIP call (CPU only, no kernel launches)."""
import ctypes
import os

import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests.test_step_ops_abi import INVALID, MB, OVERLAP, P, UNSUPPORTED, WORKSPACE, run

pytestmark = pytest.mark.skipif(not os.path.exists(dg.library_path), reason="libdetgrad.so not built")

A = [P(0x100000000 + i * 64 * MB) for i in range(32)]   # never dereferenced: every call fails validation first
BIG = 48 * MB
X = dict(q=A[0], q_st=128, q_sh=64, k=A[1], k_st=128, k_sh=64, v=A[2], v_st=192, v_sh=48, g=A[3], g_ld=4, beta=A[4], beta_ld=4)
N = dict(dtype=0, T=1000, Hk=2, H=4, dk=64, dv=48)
RULE = dict(X, **N, offs=A[5], S=3, scale=0.1, s0=A[6], o=A[7], o_st=192, o_sh=48, s1=A[8], states=A[9], ws=A[10], ws_bytes=BIG,
            stream=None)
RULE_BWD = dict(dict(d_o=A[11], do_st=192, do_sh=48), **X, **N, offs=A[5], S=3, scale=0.1, states=A[9], ds1=A[12], dq=A[13],
                dq_st=128, dq_sh=64, dk_out=A[14], dk_st=128, dk_sh=64, dv_out=A[15], dv_st=192, dv_sh=48, dg=A[16], dg_ld=4,
                dbeta=A[17], dbeta_ld=4, ds0=A[18], ws=A[10], ws_bytes=BIG, stream=None)
STEP = dict(X, dtype=0, B=100, Hk=2, H=4, dk=64, dv=48, scale=0.1, state=A[6], N=200, slots=A[5], o=A[7], o_st=192, o_sh=48,
            stream=None)
ROT = dict(dtype=0, T=1000, D=64, w_q=A[2], w_k=A[3], norm=1, eps=1e-6, pos=A[4], pos_ld=1000, axes=2, inv_freq=A[5], axis=A[6],
           R=64, pairs=0)
QK = dict(q=A[0], q_st=256, q_sh=64, Hq=4, k=A[1], k_st=128, k_sh=64, Hk=2, **ROT, q_out=A[7], qo_st=256, qo_sh=64, k_out=A[8],
          ko_st=128, ko_sh=64, stream=None)
QK_BWD = dict(dqo=A[9], dqo_st=256, dqo_sh=64, dko=A[10], dko_st=128, dko_sh=64, q=A[0], q_st=256, q_sh=64, Hq=4, k=A[1],
              k_st=128, k_sh=64, Hk=2, **ROT, dq=A[11], dq_st=256, dq_sh=64, dk=A[12], dk_st=128, dk_sh=64, dw_q=A[13],
              dw_k=A[14], ws=A[15], ws_bytes=BIG, stream=None)


def inside(p, n=16):
    return P(p.value + n)


NUL = dict.fromkeys
SIZES = [dict(T=-1), dict(Hk=0), dict(H=0), dict(H=3), dict(dk=0), dict(dv=0), dict(dtype=2), dict(scale=float("nan")),
         dict(scale=float("inf")), dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(beta=None), dict(q_sh=63),
         dict(q_st=127), dict(v_sh=0), dict(v_st=0), dict(g_ld=3), dict(beta_ld=3), dict(q=inside(A[0], 1)), dict(g=inside(A[3], 2))]
LARGE = [dict(dk=129, q_sh=129, q_st=258, k_sh=129, k_st=258), dict(dv=129), dict(T=1 << 31), dict(q_st=1 << 50), dict(g_ld=1 << 50)]
CASES = [
    ("det_delta_rule", RULE, INVALID, SIZES + [dict(S=-1), dict(offs=None), dict(o=None), dict(o_sh=47), dict(o_st=191),
                                               dict(s0=inside(A[6], 2)), dict(states=inside(A[9], 1))]),
    ("det_delta_rule", RULE, UNSUPPORTED, LARGE + [dict(S=65536), dict(H=1 << 20), dict(T=1 << 28, H=64)]),
    ("det_delta_rule", RULE, WORKSPACE, [dict(ws=None), dict(ws=inside(A[10])), dict(ws_bytes=300)]),
    ("det_delta_rule", RULE, OVERLAP, [dict(o=A[0]), dict(o=A[2]), dict(s1=A[6]), dict(states=inside(A[6])), dict(ws=A[7]),
                                       dict(o=inside(A[5], 8)), dict(s1=inside(A[9])), dict(ws=A[3]), dict(o=A[4]), dict(o=A[1])]),
    ("det_delta_rule_bwd", RULE_BWD, INVALID, SIZES + [dict(S=-1)] + [{n: None} for n in (
        "offs", "d_o", "states", "dq", "dk_out", "dv_out", "dg", "dbeta")] + [dict(dg_ld=3), dict(dbeta_ld=0), dict(dq_sh=10),
                                                                             dict(do_st=100), dict(dv_st=100)]),
    ("det_delta_rule_bwd", RULE_BWD, UNSUPPORTED, LARGE + [dict(S=65536), dict(dv_st=1 << 50), dict(dg_ld=1 << 50)]),
    ("det_delta_rule_bwd", RULE_BWD, WORKSPACE, [dict(ws=None), dict(ws=inside(A[10])), dict(ws_bytes=300)]),
    ("det_delta_rule_bwd", RULE_BWD, OVERLAP, [dict(dq=A[0]), dict(dk_out=A[13]), dict(dv_out=A[11]), dict(dg=A[3]),
                                               dict(dbeta=A[16]), dict(ds0=A[12]), dict(ws=A[9]), dict(dq=A[5]), dict(ds0=A[18], dg=A[18])]),
    ("det_delta_rule_step", STEP, INVALID, [dict(B=-1), dict(Hk=0), dict(H=3), dict(dk=0), dict(dtype=2), dict(N=-1),
                                            dict(N=1 << 31), dict(slots=None, N=99), dict(q=None), dict(state=None), dict(o=None),
                                            dict(q_sh=63), dict(o_st=191), dict(g_ld=3), dict(scale=float("nan")),
                                            dict(slots=inside(A[5], 2))]),
    ("det_delta_rule_step", STEP, UNSUPPORTED, [dict(dk=129, q_sh=129, q_st=258, k_sh=129, k_st=258), dict(B=65536),
                                                dict(q_st=1 << 50), dict(H=65536)]),
    ("det_delta_rule_step", STEP, OVERLAP, [dict(o=A[6]), dict(o=A[2]), dict(state=A[0]), dict(state=A[5]), dict(o=A[5])]),
    ("det_qk_norm", QK, INVALID, [dict(T=-1), dict(D=-1), dict(Hq=-1), dict(R=65), dict(R=66), dict(R=-2), dict(dtype=3),
                                  dict(norm=3), dict(norm=-1), dict(pairs=2), dict(eps=-1.0), dict(eps=float("nan")),
                                  dict(pos=None), dict(inv_freq=None), dict(axes=0), dict(axis=None), dict(pos_ld=999),
                                  dict(q=None), dict(k_out=None), dict(q_sh=60), dict(qo_st=255), dict(k=inside(A[1], 1)),
                                  dict(pos=inside(A[4], 2))]),
    ("det_qk_norm", QK, UNSUPPORTED, [dict(D=1025, R=64, q_sh=1025, q_st=1 << 14), dict(Hq=65536), dict(q_st=1 << 50),
                                      dict(pos_ld=1 << 50), dict(T=1 << 41)]),
    ("det_qk_norm", QK, OVERLAP, [dict(q_out=A[0]), dict(k_out=A[7]), dict(q_out=A[2]), dict(k_out=A[4]), dict(q_out=A[5]),
                                  dict(k_out=A[6]), dict(q_out=inside(A[1]))]),
    ("det_qk_norm_bwd", QK_BWD, INVALID, [dict(T=-1), dict(R=65), dict(norm=3), dict(pairs=-1), dict(dw_q=None), dict(w_k=None),
                                          dict(dqo=None), dict(dk=None), dict(pos=None), dict(dq_sh=1), dict(dko_st=100)]),
    ("det_qk_norm_bwd", QK_BWD, WORKSPACE, [dict(ws=None), dict(ws=inside(A[15])), dict(ws_bytes=300)]),
    ("det_qk_norm_bwd", QK_BWD, OVERLAP, [dict(dq=A[9]), dict(dk=A[0]), dict(dw_q=A[2]), dict(dw_k=A[13]), dict(ws=A[9]),
                                          dict(dq=inside(A[4])), dict(ws=A[13])]),
]


@pytest.mark.parametrize("fn,args,status,kw", [(f, a, s, k) for f, a, s, ks in CASES for k in ks])
def test_refused(fn, args, status, kw):
    assert run(fn, args, **kw) == status, (fn, kw, dg.lib().det_last_error())
    if status != WORKSPACE:     # (the message about a workspace is one for all calls)
        assert dg.lib().det_last_error().startswith(fn[4:].encode())


def test_nothing_to_do():
    none = lambda d: {k: None for k, v in d.items() if isinstance(v, P)}  # noqa: E731
    assert run("det_delta_rule", RULE, **{**none(RULE), "S": 0}) == dg.DET_OK
    assert run("det_delta_rule_bwd", RULE_BWD, **{**none(RULE_BWD), "S": 0}) == dg.DET_OK
    assert run("det_delta_rule_step", STEP, **{**none(STEP), "B": 0}) == dg.DET_OK
    for fn, d in (("det_qk_norm", QK), ("det_qk_norm_bwd", QK_BWD)):
        for kw in (dict(T=0), dict(D=0, R=0), dict(Hq=0, Hk=0)):
            assert run(fn, d, **{**none(d), **kw}) == dg.DET_OK, (fn, kw, dg.lib().det_last_error())


def test_column_ranges_of_one_buffer_are_no_overlap():
    """dq, dk and dv as ranges of one [T, 2 Hk dk + H dv] buffer pass the overlap check, one column less does not (the
    calls end at the workspace)."""
    st = 128 + 128 + 192
    ok = dict(dq_st=st, dk_st=st, dv_st=st, dk_out=P(A[13].value + 256), dv_out=P(A[13].value + 512))
    late = dict(ds0=A[12])   # an overlap that is looked for after those
    assert run("det_delta_rule_bwd", RULE_BWD, **ok, **late) == OVERLAP
    assert b"dinitial_state" in dg.lib().det_last_error()
    assert run("det_delta_rule_bwd", RULE_BWD, **dict(ok, dv_out=P(A[13].value + 510)), **late) == OVERLAP
    assert b"dk overlaps dv" in dg.lib().det_last_error()


def test_sizes():
    n, b = ctypes.c_int64(), ctypes.c_size_t()
    L = dg.lib()
    f = ctypes.c_int64()
    size = lambda *a: L.det_delta_rule_states_size(*a, ctypes.byref(n), ctypes.byref(f))  # noqa: E731
    assert size(1000, 3, 64, 48, 0) == 0 and n.value == 1000 // 64 + 3 and f.value >= 64 * 48 + 64 * 48
    assert size(1000, 3, 63, 47, 1) == 0 and n.value == 1000 // 32 + 3 and f.value % 4 == 0 and f.value >= 63 * 47 + 32 * 47
    assert L.det_delta_rule_states_size(1000, 3, 64, 48, 0, None, ctypes.byref(f)) == INVALID
    assert L.det_delta_rule_states_size(1000, 3, 64, 48, 0, ctypes.byref(n), None) == INVALID
    assert size(1000, 3, 64, 48, 5) == INVALID and size(1000, 3, 64, 129, 0) == UNSUPPORTED
    assert dg.det_delta_rule_workspace_size(0, 3, 2, 4, 64, 48, 0) == 0
    assert dg.det_delta_rule_workspace_size(1000, 3, 2, 4, 64, 48, 0) >= 256 + 18 * 4 * (64 * 64 * 3 // 4 * 6 + 6 * 64 * 4)
    assert dg.det_delta_rule_bwd_workspace_size(1000, 3, 2, 4, 64, 48, 0) >= 256 + 18 * 4 * (64 * 64 * 3 // 4 * 12 + 6 * 64 * 4 + 64 * 48 * 8)
    assert L.det_delta_rule_workspace_size(10, 1, 1, 1, 8, 8, 0, None) == INVALID
    assert L.det_delta_rule_bwd_workspace_size(10, 1, 1, 1, 200, 8, 0, ctypes.byref(b)) == UNSUPPORTED
    assert dg.det_qk_norm_bwd_workspace_size(0, 4, 2, 64) == 0
    assert dg.det_qk_norm_bwd_workspace_size(1, 4, 2, 64) >= 256 + 2 * 64 * 4
    assert L.det_qk_norm_bwd_workspace_size(10, 4, 2, 2000, ctypes.byref(b)) == UNSUPPORTED


def test_binding_refusals():
    """Shapes, dtypes, strides and devices are checked before any library call (CPU tensors suffice)."""
    bf, i32 = torch.bfloat16, torch.int32

    def refuse(exc, fn, *a, **k):
        with pytest.raises(exc):
            fn(*a, **k)
    q, v, g, b = torch.zeros(6, 2, 8, dtype=bf), torch.zeros(6, 4, 5, dtype=bf), torch.zeros(6, 4), torch.zeros(6, 4, dtype=bf)
    offs, s = torch.tensor([0, 6], dtype=i32), torch.zeros(1, 4, 8, 5)
    f = dg.det_delta_rule
    refuse(TypeError, f, q.half(), q.half(), v, g, b, v, offs)
    refuse(TypeError, f, q, q.float(), v, g, b, v, offs)
    refuse(TypeError, f, q, q, v, g.to(bf), b, v, offs)
    refuse(TypeError, f, q, q, v, g, b.float(), v, offs)
    refuse(TypeError, f, q, q, v, g, b, v.float(), offs)
    refuse(TypeError, f, q, q, v, g, b, v, offs.long())
    refuse(TypeError, f, q, q, v, g, b, v, offs, final_state=s.to(bf))
    refuse(ValueError, f, q[0], q, v, g, b, v, offs)
    refuse(ValueError, f, q, q[:5], v, g, b, v, offs)
    refuse(ValueError, f, q, q, v, g[:, :3], b, v, offs)
    refuse(ValueError, f, q, q, v, g, b, v[..., :4], offs)
    refuse(ValueError, f, q, q, v, g, b, v, offs[None])
    refuse(ValueError, f, q, q, v, g, b, v, offs, initial_state=s[:, :2])
    refuse(ValueError, f, q, q, v, g, b, v, offs, states=torch.zeros(2, 4, 64 * 64 + 128))
    refuse(ValueError, f, q.transpose(1, 2).contiguous().transpose(1, 2), q, v, g, b, v, offs)
    refuse(ValueError, f, q, q, v, g, b, v.clone(), offs)                        # not on a GPU
    assert dg.det_delta_rule_states_shape(q, v, offs) == (1, 4, 64 * 64 + 128)
    f, st = dg.det_delta_rule_bwd, torch.zeros(dg.det_delta_rule_states_shape(q, v, offs))
    refuse(TypeError, f, v.float(), q, q, v, g, b, offs, st, q, q, v, b, b)
    refuse(TypeError, f, v, q, q, v, g, b, offs, st, q, q, v, g, b)
    refuse(ValueError, f, v, q, q, v, g, b, offs, st[:0], q, q, v, b, b)
    refuse(ValueError, f, v, q, q, v, g, b, offs, st, q, q[:, :1], v, b, b)
    refuse(ValueError, f, v, q, q, v, g, b, offs, st, q, q, v, b, b)
    f, c = dg.det_delta_rule_step, torch.zeros(9, 4, 8, 5)
    refuse(TypeError, f, q, q, v, g, b, c.to(bf), v)
    refuse(TypeError, f, q, q, v, g, b, c, v, slots=torch.zeros(6))
    refuse(ValueError, f, q, q, v, g, b, c[0], v)
    refuse(ValueError, f, q, q, v, g, b, c[:, :2], v)
    refuse(ValueError, f, q, q, v, g, b, c, v, slots=torch.zeros(5, dtype=i32))
    refuse(ValueError, f, q, q, v, g, b, c, v)
    f, x, k, w = dg.det_qk_norm, torch.zeros(6, 4, 8), torch.zeros(6, 2, 8), torch.zeros(8)
    pos, fr = torch.zeros(6, dtype=i32), torch.zeros(4)
    refuse(ValueError, f, None, None, None, None)
    refuse(ValueError, f, x, None, x, k)
    refuse(ValueError, f, x, k, x, None)
    refuse(TypeError, f, x.half(), k.half(), x, k)
    refuse(TypeError, f, x, k.to(bf), x, k)
    refuse(TypeError, f, x, k, x, k, w_q=w.to(bf))
    refuse(TypeError, f, x, k, x, k, pos=pos.long(), inv_freq=fr)
    refuse(TypeError, f, x, k, x, k, pos=pos, inv_freq=fr.double())
    refuse(ValueError, f, x, k, x, k, w_q=torch.zeros(7))
    refuse(ValueError, f, x, k, x, k, norm="layer")
    refuse(ValueError, f, x, k, x, k, pairs="both")
    refuse(ValueError, f, x, k, x, k, pos=pos)
    refuse(ValueError, f, x, k, x, k, inv_freq=fr)
    refuse(ValueError, f, x, k, x, k, axis=pos)
    refuse(ValueError, f, x, k, x, k, pos=pos[:5], inv_freq=fr)
    refuse(ValueError, f, x, k, x, k, pos=torch.zeros(2, 6, dtype=i32), inv_freq=fr)
    refuse(ValueError, f, x, k, x, k, pos=pos, inv_freq=fr, axis=torch.zeros(3, dtype=i32))
    refuse(ValueError, f, x[..., ::2], k, x, k)
    refuse(ValueError, f, x, k, x.clone(), k.clone())
    f = dg.det_qk_norm_bwd
    refuse(ValueError, f, x, None, x, k, x, k)
    refuse(ValueError, f, x, k, x, k, x, k[:5])
    refuse(TypeError, f, x, k, x, k, x, k, w_q=w, dw_q=w.double())
    refuse(ValueError, f, x, k, x, k, x.clone(), k.clone())
