"""The CPU model of qk_norm_rope against closed forms and differences, and the refusals of the C calls and the binding
(no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import rope as OR


@pytest.fixture(scope="module")
def L():
    from bit_mixed_precision_gb300 import build, kvq
    build.build()
    return kvq.lib()


def test_turn_by_hand():
    x = np.arange(1.0, 9.0)[None, None, None]                       # one row of 8 channels, 4 of them rotated
    quarter = np.full((1, 1, 2), math.pi / 2)
    got = OR.forward(x, None, 0.0, quarter, False)[0, 0, 0]
    np.testing.assert_allclose(got, [-3, -4, 1, 2, 5, 6, 7, 8], atol=1e-15)
    got = OR.forward(x, None, 0.0, quarter, True)[0, 0, 0]
    np.testing.assert_allclose(got, [-2, 1, -4, 3, 5, 6, 7, 8], atol=1e-15)


def test_norm_by_hand():
    x = np.array([3.0, 4.0, 0.0, 0.0])[None, None, None]
    got = OR.forward(x, np.array([1.0, 2.0, 1.0, 1.0]), 0.0, np.zeros((1, 1, 0)), False)[0, 0, 0]
    np.testing.assert_allclose(got, [1.2, 3.2, 0, 0])
    assert (OR.forward(0 * x, np.ones(4), 1e-6, np.zeros((1, 1, 0)), False) == 0).all()


def test_angles_of_several_axes():
    pos = np.array([[[1, 2]], [[10, 20]]])
    got = OR.angles(pos, [0.5, 0.25, 0.125], [0, 1, 0])
    np.testing.assert_array_equal(got[0], [[0.5, 2.5, 0.125], [1.0, 5.0, 0.25]])


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(interleaved):
    rng = np.random.default_rng(0)
    x, w, d = rng.normal(size=(2, 3, 2, 8)), rng.normal(size=8), rng.normal(size=(2, 2, 3, 8))
    angle = rng.normal(size=(2, 3, 2))
    f = lambda x, w: (OR.forward(x, w, 1e-3, angle, interleaved) * d).sum()
    dx, dw = OR.backward(d, x, w, 1e-3, angle, interleaved)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(8):
        e = np.zeros(8)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_fractions_of_a_turn():
    """turn[i] / 2^64 is f / 2 pi modulo 1, to the last bit of the float64 quotient."""
    from bit_mixed_precision_gb300 import kvq
    f = [1.0, 1e-4, 7.5, -0.3, 0.0, 2 * math.pi, 1e-12, 3.0]
    d = kvq.make_rope(64, rot=16, inv_freq=f, axis=[0, 1, 2, 3, 0, 1, 2, 3]).desc
    assert (d.rot, d.interleaved, d.n_axes) == (16, 0, 4) and list(d.axis[:8]) == [0, 1, 2, 3, 0, 1, 2, 3]
    for x, t in zip(f, d.turn[:8]):
        off = (t / 2.0 ** 64 - x / (2 * math.pi)) % 1.0
        assert min(off, 1.0 - off) <= 2.0 ** -52 * max(1.0, abs(x)), (x, t)
    d = kvq.make_rope(128, base=500000.0).desc
    assert d.rot == 128 and d.turn[0] == round(2.0 ** 64 / (2 * math.pi))
    assert d.turn[32] / 2.0 ** 64 == pytest.approx(500000.0 ** -0.5 / (2 * math.pi), rel=1e-12)


def test_struct_layout_matches_header(tmp_path):
    import os
    import shutil
    import subprocess
    from bit_mixed_precision_gb300 import kvq
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "kvq.h"', "int main(void) {",
             'printf("%zu\\n", sizeof(kvq_rope));']
    lines += [f'printf("%zu\\n", offsetof(kvq_rope, {n}));' for n, _ in kvq.KvqRope._fields_]
    (tmp_path / "l.c").write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call([cc, "-I", inc, str(tmp_path / "l.c"), "-o", str(tmp_path / "l")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "l")], text=True).split()]
    assert got == [ctypes.sizeof(kvq.KvqRope)] + [getattr(kvq.KvqRope, n).offset for n, _ in kvq.KvqRope._fields_]


def test_bad_arguments_are_refused(L):
    from bit_mixed_precision_gb300 import kvq
    p, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p(8 + (1 << 20))
    E, X, W, OK = kvq.KVQ_EINVAL, kvq.KVQ_EUNSUPPORTED, kvq.KVQ_EWORKSPACE, kvq.KVQ_OK
    big, f = 1 << 40, ctypes.c_float
    good = kvq.make_rope(128).desc

    def change(**kw):
        d = kvq.KvqRope.from_buffer_copy(good)
        for k, v in kw.items():
            if k == "axis0":
                d.axis[0] = v
            else:
                setattr(d, k, v)
        return ctypes.byref(d)

    def fwd(r=ctypes.byref(good), dt=0, B=1, T=2, Hq=4, Hkv=2, D=128, q=p, k=p, v=p, st=None, pos=p, qw=p, kw=p, eps=1e-6,
            qo=p, ko=p, vo=p):
        return L.qk_norm_rope(r, dt, B, T, Hq, Hkv, D, q, k, v, st, pos, qw, kw, 0, f(eps), qo, ko, vo, None)

    def bwd(r=ctypes.byref(good), dt=0, B=1, T=2, Hq=4, Hkv=2, D=128, dq=p, dk=p, dv=p, q=p, k=p, st=None, pos=p, qw=p,
            kw=p, eps=1e-6, gq=p, gk=p, gv=p, gst=None, gqw=p, gkw=p, ws=p, wsb=big):
        return L.qk_norm_rope_bwd(r, dt, B, T, Hq, Hkv, D, dq, dk, dv, q, k, st, pos, qw, kw, 0, f(eps), gq, gk, gv, gst,
                                  gqw, gkw, ws, wsb, None)

    st9 = lambda i, x: (ctypes.c_int64 * 9)(*[x if j == i else 128 for j in range(9)])
    for call in (fwd, bwd):
        assert call(r=None) == E and call(dt=2) == E and call(D=96) == X and call(Hq=3) == E and call(Hkv=0) == E
        assert call(B=-1) == E and call(T=-1) == E and call(B=1 << 20, T=1 << 20) == X
        for kw in (dict(rot=24), dict(rot=144), dict(rot=-16), dict(interleaved=2), dict(n_axes=0), dict(n_axes=5),
                   dict(axis0=1)):
            assert call(r=change(**kw)) == E, kw
        assert call(eps=-1.0) == E and call(eps=float("nan")) == E and call(eps=float("inf")) == E
        assert call(q=None) == E and call(k=None) == E and call(q=odd) == E and call(k=odd) == E and call(pos=None) == E
        assert call(qw=odd) == E and call(kw=odd) == E
        for i in range(6):
            assert call(B=2, st=st9(i, 4)) == E and call(B=2, st=st9(i, -8)) == E
    assert fwd(B=0, q=None) == OK and fwd(T=0) == OK
    assert fwd(v=odd) == E and fwd(qo=None) == E and fwd(ko=None) == E and fwd(vo=None) == E
    assert fwd(qo=odd) == E and fwd(ko=odd) == E and fwd(vo=odd) == E and fwd(B=2, st=st9(7, 4)) == E
    for name in ("dq", "dk", "gq", "gk", "gv", "gqw", "gkw"):
        assert bwd(**{name: None}) == E, name
    for name in ("dq", "dk", "dv", "gq", "gk", "gv"):
        assert bwd(**{name: odd}) == E, name
    for i in range(9):
        assert bwd(B=2, gst=st9(i, 4)) == E and bwd(B=2, gst=st9(i, 0)) == E
    need = L.qk_norm_rope_bwd_workspace_bytes(1, 2, 128, 1)
    assert need > 0 and bwd(ws=None) == W and bwd(wsb=need - 1) == W and bwd(ws=odd) == E
    assert L.qk_norm_rope_bwd_workspace_bytes(1, 2, 128, 0) == 0
    assert L.qk_norm_rope_bwd_workspace_bytes(1, 2, 96, 1) == ctypes.c_size_t(-1).value
    assert b"qk_norm_rope" in L.kvq_last_error()


def test_make_rope_refusals():
    from bit_mixed_precision_gb300 import kvq
    for bad in (dict(D=96), dict(D=128, rot=24), dict(D=64, rot=128), dict(D=64, inv_freq=[1.0] * 5),
                dict(D=64, rot=16, inv_freq=[1.0] * 9), dict(D=64, rot=16, axis=[0] * 7), dict(D=64, rot=16, axis=[4] * 8),
                dict(D=64, rot=16, axis=[-1] * 8), dict(D=64, rot=16, inv_freq=[math.inf] * 8)):
        with pytest.raises(ValueError):
            kvq.make_rope(**bad)


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    from bit_mixed_precision_gb300 import kvq
    q, k, pos = torch.zeros(1, 2, 4, 64).half(), torch.zeros(1, 2, 2, 64).half(), torch.zeros(1, 2, dtype=torch.int32)
    r = kvq.make_rope(64)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.qk_norm_rope(q, k, k, pos, r)
    with pytest.raises(ValueError, match="pos must be"):
        kvq.qk_norm_rope(q, k, k, pos[:, :1], r)
    with pytest.raises(ValueError, match="128 channels"):
        kvq.qk_norm_rope(q, k, k, pos, kvq.make_rope(128))
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        kvq.qk_norm_rope(q.float(), k.float(), None, pos, r)
    with pytest.raises(ValueError, match="multiple"):
        kvq.qk_norm_rope(q[:, :, :3], k, None, pos, r)
    with pytest.raises(ValueError, match="for a step"):
        kvq.qk_norm_rope(q, k[0], None, pos, r)


def test_overlapping_outputs_are_refused(L):
    """Rows that share memory: of one gradient, of two, of an output and an input; addresses are made up, nothing is read."""
    from bit_mixed_precision_gb300 import kvq
    B, T, Hq, Hkv, D = 2, 5, 4, 2, 64
    desc, n = ctypes.byref(kvq.make_rope(D).desc), Hq + 2 * Hkv
    need = L.qk_norm_rope_bwd_workspace_bytes(B, T, D, 1)
    room = 1 << 16
    names = ["q", "k", "v", "pos", "qw", "kw", "qo", "ko", "vo", "gq", "gk", "gv", "gqw", "gkw", "ws"]
    where = {x: (1 << 20) + i * room for i, x in enumerate(names)}
    dense = lambda h: [T * h * D, h * D, D]
    wide = [T * n * D, n * D, D]

    def refused(st):
        return st == kvq.KVQ_EINVAL and b"overlap" in L.kvq_last_error()

    def fwd(strides=None, **kw):
        p = {x: ctypes.c_void_p(y) for x, y in {**where, **kw}.items()}
        st = strides or dense(Hq) + dense(Hkv) + dense(Hkv)
        return refused(L.qk_norm_rope(desc, 0, B, T, Hq, Hkv, D, p["q"], p["k"], p["v"], (ctypes.c_int64 * 9)(*st), p["pos"],
                                      p["qw"], p["kw"], 0, ctypes.c_float(1e-6), p["qo"], p["ko"], p["vo"], None))

    def bwd(g=None, **kw):
        p = {x: ctypes.c_void_p(y) for x, y in {**where, **kw}.items()}
        g = g or dense(Hq) + dense(Hkv) + dense(Hkv)
        st = dense(Hq) + dense(Hkv) + dense(Hkv)
        return refused(L.qk_norm_rope_bwd(desc, 0, B, T, Hq, Hkv, D, p["qo"], p["ko"], p["vo"], p["q"], p["k"],
                                          (ctypes.c_int64 * 9)(*st), p["pos"], p["qw"], p["kw"], 0, ctypes.c_float(1e-6),
                                          p["gq"], p["gk"], p["gv"], (ctypes.c_int64 * 9)(*g), p["gqw"], p["gkw"], p["ws"],
                                          need, None))

    size = dict(q=B * T * Hq * D * 2, k=B * T * Hkv * D * 2, v=B * T * Hkv * D * 2, pos=B * T * 4, qw=D * 2, kw=D * 2)
    size.update(qo=size["q"], ko=size["k"], vo=size["k"], gq=size["q"], gk=size["k"], gv=size["k"], gqw=D * 4, gkw=D * 4, ws=need)
    for call, outs, ins in ((fwd, ["qo", "ko", "vo"], ["q", "k", "v", "pos", "qw", "kw"]),
                            (bwd, ["gq", "gk", "gv", "gqw", "gkw", "ws"], ["qo", "ko", "vo", "q", "k", "pos", "qw", "kw"])):
        for out in outs:
            for other in ins + outs:
                if out == other:
                    continue
                step = 256 if out == "ws" else 16
                assert call(**{out: where[other] + (size[other] - 1) // step * step}), (out, other)
                assert call(**{out: where[other] - (size[out] - 1) // step * step}), (out, other)
    # rows of one gradient: a head, a token or a sequence that does not step over what lies inside it
    for i, x in ((2, 8), (2, D - 8), (1, D), (1, Hq * D - 8), (0, Hq * D), (0, T * Hq * D - 8), (5, 8), (8, 8)):
        g = dense(Hq) + dense(Hkv) + dense(Hkv)
        g[i] = x
        assert bwd(g=g), (i, x)
    # parts of one array that share a head
    for gk, gv in ((Hq - 1, Hq + Hkv), (Hq, Hq + Hkv - 1), (Hq, Hq), (0, Hq + Hkv)):
        assert bwd(g=wide * 3, gk=where["gq"] + 2 * D * gk, gv=where["gq"] + 2 * D * gv)
    # in place only where every row keeps its place
    assert fwd(qo=where["q"]) and fwd(ko=where["k"]) and fwd(vo=where["v"])
    assert fwd(strides=[0, Hq * D, D] + dense(Hkv) * 2, qo=where["q"])
    assert bwd(gq=where["qo"]) and bwd(gk=where["ko"]) and bwd(gv=where["vo"]) and bwd(g=wide * 3, gq=where["q"])
    assert bwd(gv=where["k"]) and bwd(gk=where["q"])
