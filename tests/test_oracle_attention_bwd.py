"""The float64 gradient of causal attention against differences of the forward pass, and the refusals of
prefill_attn_bwd (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import attention as OA


def forward(q, k, v, scale):
    """o [g, T, D] and lse [g, T] of one KV head's group, from the definition."""
    T = k.shape[0]
    z = np.where(np.tril(np.ones((T, T), bool)), np.einsum("gid,jd->gij", q, k) * scale, -np.inf)
    lse = np.log(np.exp(z).sum(-1))
    return np.exp(z - lse[..., None]) @ v, lse


@pytest.mark.parametrize("with_lse", [False, True])
def test_gradient_against_differences(with_lse):
    rng = np.random.default_rng(1)
    g, T, D, scale = 2, 5, 4, 0.7
    x = {"q": rng.normal(size=(g, T, D)), "k": rng.normal(size=(T, D)), "v": rng.normal(size=(T, D))}
    do, dlse = rng.normal(size=(g, T, D)), rng.normal(size=(g, T)) if with_lse else None

    def loss():
        o, lse = forward(**x, scale=scale)
        return (o * do).sum() + ((lse * dlse).sum() if with_lse else 0.0)

    o, lse = forward(**x, scale=scale)
    got = OA.prefill_backward(x["q"], x["k"], x["v"], o, do, lse, scale, dlse)[:3]
    h = 1e-6
    for name, grad in zip("qkv", got):
        for i in np.ndindex(x[name].shape):
            at = x[name][i]
            x[name][i] = at + h
            up = loss()
            x[name][i] = at - h
            down = loss()
            x[name][i] = at
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7, (name, i)


def test_forward_agrees_with_the_oracle():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(1, 7, 8)), rng.normal(size=(7, 8)), rng.normal(size=(7, 8))
    o, lse = forward(q, k, v, 0.3)
    oo, ol, _ = OA.prefill_head(q[0], k, v, 0.3)
    np.testing.assert_allclose(o[0], oo, atol=1e-12)
    np.testing.assert_allclose(lse[0], ol, atol=1e-12)


def test_one_token():
    """P = 1: dv is the sum of the heads' do, dq and dk are 0 but for dlse."""
    q, k, v, do = (np.ones((3, 1, 4)), np.ones((1, 4)), np.full((1, 4), 2.0), np.arange(12.0).reshape(3, 1, 4))
    o, lse = forward(q, k, v, 0.5)
    dq, dk, dv, _ = OA.prefill_backward(q, k, v, o, do, lse, 0.5, np.array([[1.0], [0.0], [0.0]]))
    np.testing.assert_allclose(dv, do.sum(0))
    np.testing.assert_allclose(dq[:, 0], [[0.5] * 4, [0] * 4, [0] * 4], atol=1e-12)
    np.testing.assert_allclose(dk[0], [0.5] * 4, atol=1e-12)


@pytest.fixture(scope="module")
def L():
    from bit_mixed_precision_gb300 import build, kvq
    build.build()
    return kvq.lib()


def test_bad_arguments_are_refused(L):
    from bit_mixed_precision_gb300 import kvq
    p, odd, f = ctypes.c_void_p(1 << 20), ctypes.c_void_p(8 + (1 << 20)), ctypes.c_float
    E, X, W = kvq.KVQ_EINVAL, kvq.KVQ_EUNSUPPORTED, kvq.KVQ_EWORKSPACE
    names = ["q", "k", "v", "o", "go", "dt", "B", "Hq", "Hkv", "T", "D", "scale", "causal", "lse", "glse", "dq", "dk", "dv",
             "ws", "wsb"]
    good = dict(zip(names, [p, p, p, p, p, 0, 1, 4, 2, 100, 64, 0.1, 1, p, None, p, p, p, p, 1 << 40]))

    def call(**kw):
        a = {**good, **kw}
        a["scale"] = f(a["scale"])
        return L.prefill_attn_bwd(*[a[n] for n in names], None)

    for n in ("q", "k", "v", "o", "go", "lse", "dq", "dk", "dv"):
        assert call(**{n: None}) == E, n
    for n in ("q", "k", "v", "o", "go", "dq", "dk", "dv"):
        assert call(**{n: odd}) == E, n
    assert call(glse=ctypes.c_void_p(2)) == E and call(lse=ctypes.c_void_p(2)) == E
    assert call(dt=2) == E and call(Hq=3) == E and call(T=0) == E and call(B=0) == E and call(B=-1) == E
    assert call(D=96) == X and call(causal=0) == X and call(B=1 << 20, Hq=2048) == X and call(T=(1 << 24) + 1) == X
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == E
    need = L.prefill_attn_bwd_workspace_bytes(1, 4, 2, 100)
    assert need >= 4 * 128 * 8 and call(ws=None) == W and call(wsb=need - 1) == W and call(ws=odd) == E
    assert L.prefill_attn_bwd_workspace_bytes(1, 3, 2, 100) == ctypes.c_size_t(-1).value
    # linear in the length: no buffer of pairs
    assert L.prefill_attn_bwd_workspace_bytes(1, 4, 2, 1 << 20) < 4 * (1 << 20) * 9
    assert b"prefill_attn_bwd" in L.kvq_last_error()


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    from bit_mixed_precision_gb300 import kvq
    q, k, lse = torch.zeros(1, 2, 5, 64).half(), torch.zeros(1, 1, 5, 64).half(), torch.zeros(1, 2, 5)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.prefill_attn_bwd(q, q, k, k, q, lse)
    with pytest.raises(ValueError, match="does not match"):
        kvq.prefill_attn_bwd(q, q, k[:, :, :4], k[:, :, :4], q, lse)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        kvq.prefill_attn_bwd(q.float(), q.float(), k.float(), k.float(), q.float(), lse)


def test_overlapping_outputs_are_refused(L):
    """An output on an input, on another output or on the workspace, in whole or by its last bytes; addresses are made up,
    nothing is read."""
    from bit_mixed_precision_gb300 import kvq
    B, Hq, Hkv, T, D = 2, 4, 2, 100, 64
    need = L.prefill_attn_bwd_workspace_bytes(B, Hq, Hkv, T)
    sizes = dict(q=B * Hq * T * D * 2, k=B * Hkv * T * D * 2, lse=B * Hq * T * 4)
    bytes_of = dict(q=sizes["q"], k=sizes["k"], v=sizes["k"], o=sizes["q"], go=sizes["q"], lse=sizes["lse"],
                    glse=sizes["lse"], dq=sizes["q"], dk=sizes["k"], dv=sizes["k"], ws=need)
    where, at = {}, 1 << 20
    for n, b in bytes_of.items():
        where[n] = at
        at += (b + 255) // 256 * 256 + 4096

    def call(**kw):
        p = {n: ctypes.c_void_p(x) for n, x in {**where, **kw}.items()}
        st = L.prefill_attn_bwd(p["q"], p["k"], p["v"], p["o"], p["go"], 0, B, Hq, Hkv, T, D, ctypes.c_float(0.1), 1, p["lse"],
                                p["glse"], p["dq"], p["dk"], p["dv"], p["ws"], need, None)
        return st == kvq.KVQ_EINVAL and b"overlap" in L.kvq_last_error()

    for out in ("dq", "dk", "dv", "ws"):
        for other in bytes_of:
            if out == other:
                continue
            step = 256 if out == "ws" else 16
            last = where[other] + (bytes_of[other] - 1) // step * step
            behind = where[other] - (bytes_of[out] - 1) // step * step
            for x in (where[other], last, behind):
                assert call(**{out: x}), (out, other)


def test_rows_that_share_memory(tmp_path):
    """rows.h against sets of addresses: views of one array by slicing and transposing, with room between rows, and any
    strides; exact where the header says so, never blind to a shared byte."""
    import os
    import shutil
    import subprocess
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no host C++ compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    (tmp_path / "r.cpp").write_text("""
#include <stdio.h>
#include "rows.h"
int main() {
    long long x[8], y[8];
    for (;;) {
        for (auto& e : x) if (scanf("%lld", &e) != 1) return 0;
        for (auto& e : y) if (scanf("%lld", &e) != 1) return 0;
        auto make = [](long long* e) {
            const int64_t size[3] = {e[2], e[3], e[4]}, stride[3] = {e[5], e[6], e[7]};
            return kvq::Rows(reinterpret_cast<const void*>((uintptr_t)e[0]), e[1], size, stride);
        };
        const kvq::Rows a = make(x), b = make(y);
        printf("%d %d %d %d\\n", kvq::rows_meet(a, b), kvq::rows_meet(b, a), a.nested(), b.nested());
    }
}
""")
    subprocess.check_call([cc, "-std=c++17", "-I", os.path.join(root, "bit_mixed_precision_gb300", "csrc"),
                           str(tmp_path / "r.cpp"), "-o", str(tmp_path / "r")])
    rng = np.random.default_rng(0)

    def view():
        """A view of an array [3, 4, 5, 8] of bytes at 0 as (start, row, sizes, strides), its axes in any order."""
        shape, strides = [3, 4, 5], [160, 40, 8]
        start = int(rng.integers(8)) * 0
        sizes = []
        for a in range(3):
            lo, step = int(rng.integers(shape[a])), int(rng.integers(1, 3))
            hi = int(rng.integers(lo + 1, shape[a] + 1))
            start += lo * strides[a]
            strides[a] *= step
            sizes.append((hi - lo + step - 1) // step)
        row, order = int(rng.choice([4, 8])), rng.permutation(3)
        return [start + (8 - row) * int(rng.integers(2)), row] + [sizes[i] for i in order] + [strides[i] for i in order]

    def anything():
        return [int(rng.integers(200)), int(rng.choice([1, 4, 8]))] + [int(x) for x in rng.integers(1, 5, 3)] + \
            [int(x) * 4 for x in rng.integers(0, 20, 3)]

    pairs = [(view(), view()) for _ in range(4000)] + [(anything(), anything()) for _ in range(4000)]
    pairs += [(view(), [int(rng.integers(480)), int(rng.integers(1, 200)), 1, 1, 1, 0, 0, 0]) for _ in range(1000)]
    text = "\n".join(" ".join(map(str, x + y)) for x, y in pairs)
    got = subprocess.run([str(tmp_path / "r")], input=text, capture_output=True, text=True, check=True).stdout.split()
    got = np.array(got, dtype=int).reshape(-1, 4)

    def addresses(x):
        at, row, *rest = x
        rows = [at + sum(i * s for i, s in zip(idx, rest[3:])) for idx in np.ndindex(*rest[:3])]
        return [r + j for r in rows for j in range(row)]

    shared = 0
    for i, ((x, y), g) in enumerate(zip(pairs, got)):
        ax, ay = addresses(x), addresses(y)
        want = bool(set(ax) & set(ay))
        shared += want
        assert g[0] >= want and g[1] >= want, (x, y)
        if not 4000 <= i < 8000:                            # views: exact
            assert g[0] == want and g[1] == want, (x, y)
            assert g[2] == 1
        for r, s, n in ((x, ax, g[2]), (y, ay, g[3])):
            live = [a for a in range(3) if r[2 + a] > 1 and r[5 + a] > 0]
            if n and len(live) == sum(r[2 + a] > 1 for a in range(3)):
                assert len(set(s)) == len(s), r
    assert 2000 < shared < 7000
