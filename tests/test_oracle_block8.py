"""The CPU model of the 8-bit block cache against hand-worked values, and the host-side refusals of block8_*."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import block8 as O8


def test_e4m3_rounding_matches_torch_and_the_grid():
    x = np.concatenate([np.linspace(-470, 470, 4001), np.geomspace(1e-4, 448, 2000), O8.E4M3, -O8.E4M3,
                        (O8.E4M3[1:] + O8.E4M3[:-1]) / 2]).astype(np.float32)
    ref = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O8.round_e4m3(x), ref)
    # every code value is its own rounding; a midpoint goes to the even code
    assert np.array_equal(O8.round_e4m3(O8.E4M3.astype(np.float32)), np.arange(127))
    mid = ((O8.E4M3[1:] + O8.E4M3[:-1]) / 2).astype(np.float32)
    assert (O8.round_e4m3(mid) % 2 == 0).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_codes_are_within_half_a_step(kind):
    x = np.random.default_rng(0).standard_normal((37, 64)).astype(np.float16).astype(np.float32)
    codes, s = O8.quantise(x, kind)
    err = np.abs(O8.decode(codes, kind) * np.float64(s) - x)
    # e4m3: half a step is 2^-4 of the value, or 2^-10 of the scale below the normal range; int8: half the scale.
    # The float32 product with the reciprocal moves the midpoint by 2 * 2^-24 of the value.
    step = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) if kind == "e4m3" else np.full_like(x, 0.5 * s)
    assert (err <= step + 2.0 ** -22 * np.abs(x)).all()
    assert O8.quantise(np.zeros((2, 64)), kind)[1] == np.float32(2.0 ** -64)
    x[3, 5] = np.inf
    codes, s = O8.quantise(x, kind)
    assert np.isnan(s) and not codes.any()


def test_bounds_hold_the_keys_and_scores_are_upper_bounds():
    rng = np.random.default_rng(1)
    b = O8.Block(0, 64)
    b.k = rng.standard_normal((16, 64)).astype(np.float16).astype(np.float32)
    bd, s = O8.bounds(b.k)
    slack = 2.0 ** -22 * np.abs(b.k).max()
    assert (bd[0] * np.float64(s) <= b.k.min(axis=0) + slack).all()
    assert (bd[1] * np.float64(s) >= b.k.max(axis=0) - slack).all()
    q = rng.integers(-127, 128, (3, 64)).astype(np.float32)
    q[:, 0] = 127                                        # q8 == q exactly, sq == 1
    score = O8.block_scores(q, [b])[0]
    assert score >= (q @ b.k.T).max() * (1 - 1e-6)


def test_choose_by_hand():
    assert O8.choose([5, 1, 9, 9, 2, 0], 4, 1, 1) == [0, 2, 3, 5]
    assert O8.choose([5, 7, 7, 7, 7, 0], 4, 1, 1) == [0, 1, 2, 5]          # ties: the lower blocks
    assert O8.choose([0, 1, np.nan, 3, 4], 2, 0, 1) == [2, 4]              # NaN is the largest
    assert O8.choose([0, -0.0, 0.0, -0.0, 0], 3, 0, 1) == [0, 1, 4]        # zeros of both signs are equal
    assert O8.choose([1, 2], 5, 1, 1) == [0, 1]


def test_attend_closed_forms():
    v = np.arange(12.0).reshape(4, 3)
    mask = np.array([[1, 1, 1, 0], [0, 0, 0, 0], [0, 1, 0, 0]], bool)
    o, lse, p = O8.attend(np.zeros((3, 3)), np.ones((4, 3)), v, mask, 0.5)
    assert np.allclose(o, [v[:3].mean(0), [0, 0, 0], v[1]])
    assert np.allclose(lse, [np.log(3), -np.inf, 0.0]) and np.allclose(p.sum(1), [1, 0, 1])


def test_unit_life_cycle_by_hand():
    u = O8.Unit(2, 2, "int8")
    rows = np.arange(10, dtype=np.float32).reshape(5, 2)
    u.append(rows[:1], rows[:1], [0.5])
    u.append(rows[1:], rows[1:], [1, 2, 4, 8])
    assert [len(b.k) for b in u.blocks] == [2, 2, 1] and [b.acc for b in u.blocks] == [1.5, 6, 8]
    assert [b.pos for b in u.blocks] == [0, 2, 4] and u.seq_len == 5
    assert list(u.seen(4, [1, 2])) == [False, False, True, True, False]
    assert u.evict(2, 0, 1) == 1 and [b.pos for b in u.blocks] == [2, 4] and u.count == 3 and u.seq_len == 5


# ------------------------------------------------------------------ refusals (no GPU)

@pytest.fixture(scope="module")
def L():
    from bit_mixed_precision_gb300 import build, kvq
    build.build()
    return kvq.lib()


def _desc(**kw):
    from bit_mixed_precision_gb300 import kvq
    c = kvq.KvqBlock8()
    for k, v in dict(B=2, Hq=8, Hkv=2, D=128, dtype=kvq.F16, code=kvq.CODE_E4M3, block=64, max_blocks=8, n_blocks=32).items():
        setattr(c, k, v)
    for name, _ in kvq.KvqBlock8._fields_[9:]:
        setattr(c, name, 1 << 20)                       # aligned, never read
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [(dict(B=0), "EINVAL"), (dict(Hkv=3), "EINVAL"), (dict(Hq=2 * 65), "EUNSUPPORTED"),
              (dict(D=96), "EUNSUPPORTED"), (dict(dtype=2), "EINVAL"), (dict(code=2), "EINVAL"),
              (dict(block=48), "EINVAL"), (dict(max_blocks=0), "EINVAL"), (dict(n_blocks=0), "EINVAL"),
              (dict(max_blocks=(1 << 24) + 1), "EUNSUPPORTED"), (dict(B=1 << 20, max_blocks=1 << 20), "EUNSUPPORTED"),
              (dict(n_blocks=(1 << 31) - 1, block=128), "EUNSUPPORTED"), (dict(acc=0), "EINVAL"), (dict(k_codes=8 + (1 << 20)), "EINVAL"), (dict(table=2 + (1 << 20)), "EINVAL")]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(L, kw, status):
    from bit_mixed_precision_gb300 import kvq
    c, p, f = ctypes.byref(_desc(**kw)), ctypes.c_void_p(1 << 20), ctypes.c_float(0.1)
    want = getattr(kvq, "KVQ_" + status)
    assert L.block8_reset(c, None, None) == want
    assert L.block8_append(c, p, None, p, None, 1, None, None, None) == want
    assert L.block8_attn(p, None, 1, None, c, f, None, None, 0, 0, p, p, p, 1 << 40, None) == want
    assert L.block8_select(p, None, 1, None, c, 4, 1, 1, p, p, p, 1 << 40, None) == want
    assert L.block8_evict(c, p, 1, 1, p, None) == want
    assert L.block8_attn_workspace_bytes(c, 1, 0, 0) == ctypes.c_size_t(-1).value
    assert L.block8_select_workspace_bytes(c, 1) == ctypes.c_size_t(-1).value
    assert b"block8_select_workspace_bytes" in L.kvq_last_error()


def test_bad_arguments_are_refused(L):
    from bit_mixed_precision_gb300 import kvq
    d = _desc()
    c, p, f = ctypes.byref(d), ctypes.c_void_p(1 << 20), ctypes.c_float(0.1)
    odd = ctypes.c_void_p(8 + (1 << 20))
    st = lambda *x: (ctypes.c_int64 * 3)(*x)
    big = 1 << 40
    E, X, W = kvq.KVQ_EINVAL, kvq.KVQ_EUNSUPPORTED, kvq.KVQ_EWORKSPACE
    assert L.block8_reset(None, None, None) == E
    assert L.block8_append(c, p, None, p, None, 0, None, None, None) == kvq.KVQ_OK
    assert L.block8_append(c, p, None, p, None, -1, None, None, None) == E
    assert L.block8_append(c, p, None, p, None, 8 * 64 + 1, None, None, None) == E
    assert L.block8_append(c, None, None, p, None, 1, None, None, None) == E
    assert L.block8_append(c, p, None, odd, None, 1, None, None, None) == E
    assert L.block8_append(c, p, st(128, 4, 128), p, None, 1, None, None, None) == E
    assert L.block8_append(c, p, st(128, -128, 128), p, None, 1, None, None, None) == E
    attn = lambda q=p, s=None, n_q=1, scale=f, bl=None, ln=None, n_sel=0, o=p, ws=p, wsb=big: \
        L.block8_attn(q, s, n_q, None, c, scale, bl, ln, n_sel, 1, o, p, ws, wsb, None)
    assert attn(q=None) == E and attn(q=odd) == E and attn(o=None) == E and attn(o=odd) == E
    assert attn(s=st(1024, 128, 100)) == E
    assert attn(n_q=0) == E and attn(n_q=17) == X
    assert attn(scale=ctypes.c_float(0.0)) == E and attn(scale=ctypes.c_float(float("nan"))) == E
    assert attn(bl=p) == E and attn(bl=p, ln=p, n_sel=0) == E and attn(ln=p) == E and attn(n_sel=3) == E
    assert attn(bl=p, ln=p, n_sel=(1 << 20) + 1) == X
    sel = lambda q=p, n_q=1, n_sel=4, a=1, b=1, i=p, n=p, ws=p, wsb=big: \
        L.block8_select(q, None, n_q, None, c, n_sel, a, b, i, n, ws, wsb, None)
    assert sel(q=None) == E and sel(n_q=0) == E and sel(n_q=17) == X and sel(i=None) == E and sel(n=None) == E
    assert sel(n_sel=0) == E and sel(a=-1) == E and sel(b=-1) == E and sel(n_sel=4, a=3, b=2) == E
    need = L.block8_select_workspace_bytes(c, 1)
    assert need > 0 and sel(ws=None) == W and sel(wsb=need - 1) == W and sel(ws=odd) == E
    for n_sel, kw in ((0, {}), (4, dict(bl=p, ln=p, n_sel=4))):
        need = L.block8_attn_workspace_bytes(c, 1, n_sel, 1)
        if need:
            assert attn(ws=None, **kw) == W and attn(wsb=need - 1, **kw) == W and attn(ws=odd, **kw) == E
    assert L.block8_attn_workspace_bytes(c, 1, -1, 0) == ctypes.c_size_t(-1).value
    assert L.block8_evict(c, None, 1, 1, p, None) == E
    assert L.block8_evict(c, p, -1, 1, p, None) == E and L.block8_evict(c, p, 1, 0, p, None) == E
    assert L.block8_evict(c, p, 9, 1, p, None) == E
    # 1024 units of 2^21 tokens for 1024 rows each are more than one call counts
    wide = ctypes.byref(_desc(B=1024, Hkv=1, Hq=64, max_blocks=1 << 14, block=128))
    assert L.block8_attn(p, None, 16, None, wide, f, None, None, 0, 0, p, p, p, big, None) == X
    assert L.block8_attn_workspace_bytes(wide, 16, 0, 0) == ctypes.c_size_t(-1).value
    assert L.block8_attn_workspace_bytes(wide, 1, 0, 0) != ctypes.c_size_t(-1).value
    d.max_blocks = 51201
    assert L.block8_evict(c, p, 1, 1, p, None) == X


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
             'printf("%zu\\n", sizeof(kvq_block8));']
    lines += [f'printf("%zu\\n", offsetof(kvq_block8, {n}));' for n, _ in kvq.KvqBlock8._fields_]
    (tmp_path / "l.c").write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call([cc, "-I", inc, str(tmp_path / "l.c"), "-o", str(tmp_path / "l")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "l")], text=True).split()]
    assert got == [ctypes.sizeof(kvq.KvqBlock8)] + [getattr(kvq.KvqBlock8, n).offset for n, _ in kvq.KvqBlock8._fields_]


def test_binding_refuses_cpu_tensors_and_wrong_types():
    from bit_mixed_precision_gb300 import kvq
    with pytest.raises(ValueError, match="CUDA"):
        kvq.make_block8_cache(1, 2, 1, 64, torch.float16, 64, device="cpu")
    with pytest.raises(ValueError, match="block must be"):
        kvq.make_block8_cache(1, 2, 1, 64, torch.float16, 64, block=20, device="cpu")
    with pytest.raises(TypeError, match="codes"):
        kvq.make_block8_cache(1, 2, 1, 64, torch.float16, 64, codes=torch.uint8, device="cpu")


def test_workspace_of_lists_longer_than_the_table(L):
    """A unit has no more than max_blocks blocks to list, so longer lists need no more room (room for lists of the table's
    length is what a cache allocates)."""
    c = ctypes.byref(_desc())
    for acc in (0, 1):
        need = L.block8_attn_workspace_bytes(c, 2, 8, acc)
        assert need > L.block8_attn_workspace_bytes(c, 2, 7, acc) or not acc
        assert L.block8_attn_workspace_bytes(c, 2, 9, acc) == L.block8_attn_workspace_bytes(c, 2, 1 << 20, acc) == need


def test_calls_keep_the_cache_for_the_streams_they_run_on(monkeypatch):
    """The first call on a stream, given or torch's current one, tells the allocator that the stream uses the cache's
    tensors and its workspace; otherwise a cache that is dropped behind a call would be overwritten under it."""
    from types import SimpleNamespace as N
    from bit_mixed_precision_gb300 import kvq
    uses = []
    cache = N(_index=0, _streams=set(), _tensors=[N(record_stream=lambda s, i=i: uses.append((i, s.cuda_stream))) for i in range(14)])
    current = N(cuda_stream=5, device=N(index=0))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: current.cuda_stream, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i: current)
    for stream, raw in ((None, 5), (None, 5), (N(cuda_stream=9, device=N(index=0)), 9), (None, 5)):
        assert kvq._stream8(cache, stream) == raw
    assert uses == [(i, 5) for i in range(14)] + [(i, 9) for i in range(14)]
    with pytest.raises(ValueError, match="another device"):
        kvq._stream8(cache, N(cuda_stream=9, device=N(index=1)))
