"""Refusals of the gated form, the q/k norm with rotation and the slot calls, before
anything reaches the device (no GPU needed)."""

import ctypes

import pytest
import torch

from linear_attention_la2_b200 import build as la2_build

la2_build.build()
from linear_attention_la2_b200 import la2  # noqa: E402

NULL = ctypes.c_void_p(0)
BAD = ctypes.c_size_t(-1).value
INVALID, UNSUPPORTED, OK = la2.LA2_ERR_INVALID_ARG, la2.LA2_ERR_UNSUPPORTED, la2.LA2_OK


def at(i, off=0):
    return ctypes.c_void_p(0x10000000 * (i + 1) + off)


def fwd(q=at(0), k=at(1), v=at(2), g=at(3), o=at(4), B=1, H=1, N=16, d=64, dv=64, dt=la2.LA2_F32, ws=NULL, n=0):
    return la2.la2_forward_gated(q, k, v, g, o, B, H, N, d, dv, dt, ws, n, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(d=0), INVALID), (dict(dv=0), INVALID), (dict(dt=5), INVALID),
    (dict(d=129), UNSUPPORTED), (dict(dv=200), UNSUPPORTED), (dict(dt=la2.LA2_BF16, d=96), UNSUPPORTED),
    (dict(dt=la2.LA2_BF16, dv=32), UNSUPPORTED), (dict(B=1 << 20, H=1 << 12), UNSUPPORTED),
    (dict(B=0), OK), (dict(H=0), OK), (dict(N=0, q=NULL, k=NULL, v=NULL, g=NULL, o=NULL), OK),
    (dict(g=NULL), INVALID), (dict(g=at(3, 2)), INVALID), (dict(o=at(4, 8)), INVALID), (dict(o=at(3)), INVALID),
    (dict(o=at(1, 64)), INVALID),
])
def test_forward_gated(kw, code):
    assert fwd(**kw) == code
    if code != OK and all(x in ("B", "N", "d", "dv", "dt", "H") for x in kw):
        a = dict(B=1, H=1, N=16, d=64, dv=64, dt=la2.LA2_F32)
        a.update(kw)
        for bwd in (0, 1):
            assert la2.la2_workspace_size_gated(a["B"], a["H"], a["N"], a["d"], a["dv"], a["dt"], bwd) == BAD
        assert la2.la2_kv_state_gated_workspace_size(a["B"], a["H"], a["N"], a["d"], a["dv"], a["dt"]) == BAD


def test_backward_gated():
    def bwd(*p, N=16):
        return la2.la2_backward_gated(*p, 1, 1, N, 64, 64, la2.LA2_F32, NULL, 0, NULL)

    good = [at(i) for i in range(9)]
    for i in range(9):
        assert bwd(*good[:i], NULL, *good[i + 1:]) == INVALID
        assert bwd(*good[:i], at(i, 4), *good[i + 1:]) == INVALID
    for out in range(5, 9):  # over an input, over another output
        assert bwd(*good[:out], at(2, 128), *good[out + 1:]) == INVALID
    assert bwd(*good[:6], good[5], *good[7:]) == INVALID
    assert bwd(*[NULL] * 9, N=0) == OK


def test_kv_state_and_decode_gated():
    def state(k=at(0), v=at(1), g=at(2), s=at(3), slots=at(4), S=4, B=2, dt=la2.LA2_F32):
        return la2.la2_kv_state_gated(k, v, g, s, slots, S, B, 1, 8, 64, 64, dt, NULL, 0, NULL)

    assert state(S=-1) == INVALID and state(S=1 << 31) == INVALID
    assert state(slots=NULL, S=1) == INVALID           # fewer slots than rows
    assert state(slots=at(4, 2)) == INVALID and state(s=at(3, 4)) == INVALID
    assert state(slots=at(3, 64)) == INVALID            # the list inside the pool
    assert state(k=at(3, 16384)) == INVALID
    assert state(B=0) == OK

    def dec(q=at(0), k=at(1), v=at(2), g=at(3), o=at(4), s=at(5), slots=at(6), S=4, B=2, d=64, dt=la2.LA2_BF16):
        return la2.la2_decode_step_gated(q, k, v, g, o, s, slots, S, B, 2, d, 32, dt, NULL)

    for kw in (dict(q=NULL), dict(g=NULL), dict(s=NULL), dict(g=at(3, 1)), dict(s=at(5, 2)), dict(slots=at(6, 1)),
               dict(o=at(0)), dict(o=at(5, 64)), dict(g=at(5, 64)), dict(slots=at(5, 64)), dict(slots=at(4)),
               dict(S=-1), dict(slots=NULL, S=1), dict(d=0), dict(dt=3), dict(B=-1)):
        assert dec(**kw) == INVALID, kw
    assert dec(B=0) == OK


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def rope(q=at(0), k=at(1), qs=strides(512, 128, 64), ks=strides(512, 128, 64), wq=at(2), wk=at(3), pos=at(4), qo=at(5),
         ko=at(6), B=2, N=4, H=2, Hkv=2, d=64, rot=64, axes=1, sec=None, base=10.0, eps=1e-6, s=1.0, dt=la2.LA2_F32):
    sec = None if sec is None else (ctypes.c_int64 * len(sec))(*sec)
    return la2.la2_qk_norm_rope(q, k, qs, ks, wq, wk, pos, qo, ko, B, N, H, Hkv, d, rot, axes, sec, base, eps, s, 1.0,
                                dt, NULL)


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(H=-1), INVALID), (dict(d=0), INVALID), (dict(rot=63), INVALID), (dict(rot=66), INVALID),
    (dict(rot=-2), INVALID), (dict(axes=0), INVALID), (dict(axes=2), INVALID), (dict(axes=2, sec=(16, 15)), INVALID),
    (dict(axes=2, sec=(33, -1)), INVALID), (dict(base=0.0), INVALID), (dict(base=NAN), INVALID), (dict(base=INF), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(s=INF), INVALID), (dict(dt=9), INVALID),
    (dict(d=258), UNSUPPORTED), (dict(axes=5, sec=(32, 0, 0, 0, 0)), UNSUPPORTED), (dict(B=1 << 16, N=1 << 16), UNSUPPORTED),
    (dict(qs=None), INVALID), (dict(qs=strides(-1, 128, 64)), INVALID), (dict(q=NULL), INVALID), (dict(ko=NULL), INVALID),
    (dict(q=at(0, 2)), INVALID), (dict(wq=at(2, 1)), INVALID), (dict(pos=at(4, 2)), INVALID),
    (dict(qo=at(0, 1024)), INVALID), (dict(ko=at(5, 64)), INVALID), (dict(qo=at(2)), INVALID), (dict(ko=at(4)), INVALID),
    (dict(N=0), OK), (dict(H=0, Hkv=0), OK),
])
def test_qk_norm_rope(kw, code):
    assert rope(**kw) == code


def test_qk_norm_rope_backward():
    s = strides(512, 128, 64)

    def bwd(p, ws=NULL, n=0, N=4):
        return la2.la2_qk_norm_rope_backward(p[0], p[1], p[2], p[3], s, s, p[4], p[5], p[6], p[7], p[8], p[9], p[10], 2, N,
                                             2, 2, 64, 64, 1, None, 10.0, 1e-6, 1.0, 1.0, la2.LA2_F32, ws, n, NULL)

    good = [at(i) for i in range(11)]  # dyq dyk q k wq wk pos dq dk dwq dwk
    for i in (0, 1, 2, 3, 4, 5, 7, 8, 9, 10):  # a weight without its gradient, and the other way round
        assert bwd(good[:i] + [NULL] + good[i + 1:]) == INVALID
    assert la2.la2_qk_norm_rope_backward_workspace_size(2, 4, 2, 2, 300) == BAD
    assert la2.la2_qk_norm_rope_backward_workspace_size(-1, 4, 2, 2, 64) == BAD
    assert la2.la2_qk_norm_rope_backward_workspace_size(2, 0, 2, 2, 64) == 0


def test_slot_calls():
    def copy(s=at(0), a=at(1), b=at(2), n=3, S=4, H=2, d=16):
        return la2.la2_state_copy(s, a, b, n, S, H, d, 16, NULL)

    for kw in (dict(s=NULL), dict(a=NULL), dict(b=NULL), dict(s=at(0, 2)), dict(a=at(1, 1)), dict(a=at(0, 64)),
               dict(n=-1), dict(S=-1), dict(H=-1), dict(d=0), dict(S=1 << 31)):
        assert copy(**kw) == INVALID, kw
    assert copy(n=0) == OK and copy(S=0) == OK and copy(H=0) == OK
    assert copy(n=1 << 31) == UNSUPPORTED

    def compact(s=at(0), live=at(1), moved=at(2), S=4, H=2):
        return la2.la2_state_compact(s, live, moved, S, H, 16, 16, NULL)

    for kw in (dict(s=NULL), dict(live=NULL), dict(moved=NULL), dict(moved=at(1, 4)), dict(moved=at(0, 64)), dict(S=-1)):
        assert compact(**kw) == INVALID, kw
    assert compact(S=32769) == UNSUPPORTED and compact(S=0) == OK


def test_binding_refuses_host_and_mismatched_tensors():
    x, g, s = torch.zeros(1, 2, 8, 64), torch.zeros(1, 2, 8), torch.zeros(1, 2, 64, 64)
    i = torch.zeros(1, dtype=torch.int32)
    for fn, args in ((la2.forward_gated, (x, x, x, g)), (la2.backward_gated, (x, x, x, g, x)),
                     (la2.kv_state_gated, (x, x, g)), (la2.decode_step_gated, (x[:, :, 0], x[:, :, 0], x[:, :, 0], g[..., 0], s)),
                     (la2.qk_norm_rope, (x, x)), (la2.qk_norm_rope_backward, (x, x, x, x)),
                     (la2.state_copy, (s, i, i)), (la2.state_compact, (s, i))):
        with pytest.raises(la2.La2Error) as e:
            fn(*args)
        assert e.value.code == INVALID
