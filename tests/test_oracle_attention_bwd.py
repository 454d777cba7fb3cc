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
