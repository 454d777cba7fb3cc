"""prefill_attn_bwd on the GPU against the float64 gradient in oracle/attention.py, which takes the same o and lse.

Tolerances, u = 2^-24, h = half a step of the type (eps / 2), from the arithmetic of the kernels:
  logits    exact products, D added in float32 (a tensor core may cut: 2u each): 2 D u sigma sum_c |q_c k_c| <= e;
            exponent in base 2: three roundings of at most |z| + |lse| + 16, and exp2's 2^-22:
            P is off by eP = e + 4 u (max |z| + max |lse| + 16) + 2^-22, relatively
  P         rounded: h P; fp16 (kept times 2^15): 2^-40 at least
  dV        sum_i P_ij |do_i| (eP + h + 2 n u) + 2^-40 sum_i |do_i|, n products
  dS        P ((eP + 4 u) |dP - delta| + 2 D u A + D u C + 2 u (|dP| + |delta|)), A = sum_c |do_c v_c|, C = sum_c |do_c o_c|;
            rounded: h |dS|; fp16 (kept times 2^15 c, 1 / c <= 2 M): 2^-39 M, M = max |do| max |v| + max |delta| (2-norms)
  dQ, dK    sigma sum (error of dS + 2 n u |dS|) |k| or |q|
  output    h of it, fp16 below its normal range 2^-25
  underflow exp2 gives 0 below 2^-126 (its ftz form), and so may any float32 or bf16 number behind it: a P is off by 2^-126 at
            least, so dV by sum_i (1 + |do_i|) 2^-126, dS by (1 + |dP - delta|) 2^-126 and an output by 2^-126.  (Sharp rows
            in bf16 have probabilities of 1e-47, where every relative bound above is below what float32 can hold.)
"""
import math

import numpy as np
import pytest
import torch

from bit_mixed_precision_gb300 import kvq
from oracle import attention as OA
from tests.helpers import np_

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def status_is_clean():
    yield
    assert kvq.device_status() == 0


def make(B=1, Hq=2, Hkv=2, T=128, D=128, dtype=F16, seed=0, size=1.0, key=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda h: torch.randn((B, h, T, D), generator=g)
    q, k, v, do = r(Hq), r(Hkv) * key, r(Hkv), r(Hq) * size
    q, k, v, do = (x.to(dtype).cuda() for x in (q, k, v, do))
    o, lse, _ = kvq.prefill_attn_scores(q, k, v, colscore=False)
    return do, q, k, v, o, lse


def check(got, do, q, k, v, o, lse, scale=None, dlse=None, heads=None):
    """Every KV head's gradients, or those in `heads` (numbers b * Hkv + h), within the bounds above."""
    B, Hq, T, D = q.shape
    Hkv, dtype = k.shape[1], q.dtype
    g, scale = Hq // Hkv, D ** -0.5 if scale is None else scale
    h, f16 = torch.finfo(dtype).eps / 2, dtype == F16
    for u in (range(B * Hkv) if heads is None else heads):
        b, kv = divmod(u, Hkv)
        at = slice(kv * g, (kv + 1) * g)
        Q, DO, O, L = (np_(x[b, at]).astype(np.float64) for x in (q, do, o, lse))
        K, V = (np_(x[b, kv]).astype(np.float64) for x in (k, v))
        dl = None if dlse is None else np_(dlse[b, at]).astype(np.float64)
        dq, dk, dv, terms = OA.prefill_backward(Q, K, V, O, DO, L, scale, dl)
        tq, tk, tv = np.zeros_like(dq), np.zeros_like(dk), np.zeros_like(dv)
        nk = 2 * g * T * U
        norm = lambda x: np.sqrt((x * x).sum(-1)).max()
        most = norm(DO) * norm(V) + max(np.abs(t[2]).max() for t in terms)
        for i, (P, dP, delta, dS) in enumerate(terms):
            ok = ~np.isinf(L[i])
            z = np.abs(Q[i] @ K.T).max() * scale
            e = 2 * D * U * scale * (np.abs(Q[i]) @ np.abs(K).T).max()
            eP = e + 4 * U * (z + np.abs(L[i][ok]).max() + 16) + 2.0 ** -22
            low = 2.0 ** -126 * np.tril(np.ones((T, T)))
            tv += (P * (eP + h + nk)).T @ np.abs(DO[i]) + low.T @ (1 + np.abs(DO[i])) + (2.0 ** -40 * np.abs(DO[i]).sum(0) if f16 else 0)
            E = P * ((eP + 4 * U) * np.abs(dP - delta) + 2 * D * U * (np.abs(DO[i]) @ np.abs(V).T)
                     + D * U * (np.abs(DO[i]) * np.abs(O[i])).sum(-1, keepdims=True) + 2 * U * (np.abs(dP) + np.abs(delta)))
            E += (h + nk) * np.abs(dS) + (2.0 ** -39 * most * np.tril(np.ones((T, T))) if f16 else 0) + low * (1 + np.abs(dP - delta))
            tq[i] += scale * E @ np.abs(K)
            tk += scale * E.T @ np.abs(Q[i])
        for name, a, ref, tol in (("dq", got[0][b, at], dq, tq), ("dk", got[1][b, kv], dk, tk), ("dv", got[2][b, kv], dv, tv)):
            tol = tol + h * np.abs(ref) + (2.0 ** -25 if f16 else 2.0 ** -126)
            off = np.abs(np_(a).astype(np.float64) - ref)
            assert (off <= tol).all(), f"{name} unit {u}: {(off / tol).max()} of the bound, {np.isnan(off).sum()} NaN"


@pytest.mark.parametrize("B,Hq,Hkv,T,D,dtype", [
    (1, 1, 1, 128, 128, F16),
    (1, 1, 1, 128, 64, BF16),
    (1, 2, 2, 256, 128, BF16),
    (1, 2, 1, 256, 64, F16),
    (1, 1, 1, 1, 128, F16),
    (3, 4, 2, 1, 64, BF16),
    (1, 2, 1, 2, 128, BF16),
    (1, 1, 1, 63, 64, F16),
    (1, 1, 1, 64, 128, F16),
    (2, 1, 1, 65, 128, BF16),
    (1, 3, 1, 127, 64, F16),
    (1, 1, 1, 129, 128, F16),
    (2, 4, 2, 300, 128, F16),
    (1, 5, 1, 257, 128, BF16),
    (1, 8, 1, 385, 64, BF16),
    (2, 2, 2, 641, 128, F16),
    (1, 2, 1, 1023, 128, BF16),
    (1, 2, 2, 1400, 64, F16),
])
def test_gradients(B, Hq, Hkv, T, D, dtype):
    x = make(B, Hq, Hkv, T, D, dtype)
    check(kvq.prefill_attn_bwd(*x), *x)


@pytest.mark.parametrize("Hq,Hkv,T,D,dtype", [(8, 1, 900, 128, BF16), (5, 1, 640, 64, F16), (3, 1, 200, 128, F16), (2, 1, 1300, 64, BF16),
                                              (16, 2, 130, 128, F16), (1, 1, 1500, 128, BF16)])
def test_few_key_tiles(Hq, Hkv, T, D, dtype):
    """Fewer key tiles than SMs: clusters share a tile's query tiles, also where some of a cluster's CTAs get none."""
    x = make(1, Hq, Hkv, T, D, dtype)
    got = kvq.prefill_attn_bwd(*x)
    check(got, *x)
    assert all(torch.equal(a, b) for a, b in zip(got, kvq.prefill_attn_bwd(*x)))


@pytest.mark.parametrize("D,dtype", [(128, F16), (64, BF16)])
def test_long(D, dtype):
    x = make(1, 4, 2, 4100, D, dtype)
    check(kvq.prefill_attn_bwd(*x), *x, heads=[1])


def test_many_heads():
    """More tiles than the GPU holds CTAs, several groups of heads; some heads checked."""
    x = make(4, 64, 32, 700, 64, BF16)
    check(kvq.prefill_attn_bwd(*x), *x, heads=[0, 63, 127])
    x = make(2, 40, 8, 1537, 128, F16)
    check(kvq.prefill_attn_bwd(*x), *x, heads=[0, 15])
    # many sequences of one and of several tiles; a sequence's dQ is the same in a call of its own, whose launch order differs
    for B, Hq, Hkv, T, D, dtype in ((37, 64, 64, 100, 128, BF16), (31, 64, 16, 130, 64, F16), (9, 32, 8, 1290, 64, BF16),
                                    (7, 40, 40, 1290, 128, F16)):
        x = make(B, Hq, Hkv, T, D, dtype, seed=T)
        got = kvq.prefill_attn_bwd(*x)
        check(got, *x, heads=[0, B * Hkv - 1])
        assert all(torch.equal(a, b) for a, b in zip(got, kvq.prefill_attn_bwd(*x)))
        for b in (0, B // 2, B - 1):
            alone = kvq.prefill_attn_bwd(*[y[b:b + 1].contiguous() for y in x])
            assert torch.equal(alone[0][0], got[0][b])


def test_many_short_sequences():
    """More heads than a grid's second axis could count."""
    x = make(2200, 32, 8, 20, 64, BF16)
    check(kvq.prefill_attn_bwd(*x), *x, heads=[0, 9999, 2200 * 8 - 1])


@pytest.mark.parametrize("dtype,size", [(F16, 2.0 ** -14), (F16, 3000.0), (BF16, 2.0 ** -60), (BF16, 2.0 ** 40)])
def test_gradients_of_any_size(dtype, size):
    """fp16: dS below its normal range, or do.v beyond its largest number; results that overflow the type are avoided by
    values of size 2^-6."""
    do, q, k, v, o, lse = make(1, 2, 1, 300, 128, dtype, size=size)
    if size == 3000.0:
        v = (v * 2.0 ** -6).contiguous()
        o, lse, _ = kvq.prefill_attn_scores(q, k, v, colscore=False)
    x = (do, q, k, v, o, lse)
    check(kvq.prefill_attn_bwd(*x), *x)


def test_one_head_far_larger_than_another():
    """The scale of fp16's dS is one per KV head: heads of other groups, and batches, do not touch it."""
    do, q, k, v, o, lse = make(2, 4, 2, 200, 64, F16)
    do[0, :2] *= 2.0 ** 12
    do[1, 2:] *= 2.0 ** -12
    x = (do.contiguous(), q, k, v, o, lse)
    check(kvq.prefill_attn_bwd(*x), *x)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_sharp_rows(dtype):
    """Logits of up to a few hundred: most probabilities are 0, rows have one key."""
    x = make(1, 2, 2, 400, 128, dtype, key=25.0)
    check(kvq.prefill_attn_bwd(*x), *x)


def test_scale_and_gradient_of_lse():
    do, q, k, v, _, _ = make(2, 4, 2, 200, 128, F16)
    o, lse, _ = kvq.prefill_attn_scores(q, k, v, 0.21, colscore=False)
    dlse = torch.randn(lse.shape, generator=torch.Generator().manual_seed(4)).cuda()
    for dl in (None, dlse):
        check(kvq.prefill_attn_bwd(do, q, k, v, o, lse, 0.21, dlse=dl), do, q, k, v, o, lse, 0.21, dl)


def test_rows_without_gradient():
    """do = 0 behind the last token of a padded batch, and rows whose lse is -inf: zero dq there, dk and dv as without
    those rows."""
    do, q, k, v, o, lse = make(2, 2, 1, 260, 64, BF16)
    do[1, :, 150:] = 0
    got = kvq.prefill_attn_bwd(do, q, k, v, o, lse)
    check(got, do, q, k, v, o, lse)
    assert (got[0][1, :, 150:] == 0).all() and (got[1][1, :, 150:] == 0).all() and (got[2][1, :, 150:] == 0).all()
    s = [x[1:, :, :150].contiguous() for x in (do, q, k, v, o, lse)]
    small = kvq.prefill_attn_bwd(*s)
    assert torch.equal(small[0], got[0][1:, :, :150])
    lse2 = lse.clone()
    lse2[1, :, 150:] = -math.inf
    again = kvq.prefill_attn_bwd(do, q, k, v, o, lse2)
    assert all(torch.equal(a, b) for a, b in zip(again, got))
    do[1, :, 150:] = 1.0
    again = kvq.prefill_attn_bwd(do, q, k, v, o, lse2)
    assert all(torch.equal(a, b) for a, b in zip(again, got))
    zero = kvq.prefill_attn_bwd(torch.zeros_like(do), q, k, v, o, lse)
    assert all((x == 0).all() for x in zero)


def test_outputs_given_and_nothing_else_written():
    x = make(1, 2, 1, 130, 64, F16)
    base = kvq.prefill_attn_bwd(*x)
    n = [y.numel() for y in base]
    room = torch.full((sum(n) + 4 * 64,), 7.0, dtype=F16, device="cuda")
    out, at = [], 64
    for y in base:
        out.append(room[at:at + y.numel()].view(y.shape))
        at += y.numel() + 64
    got = kvq.prefill_attn_bwd(*x, out=out)
    assert all(a is b and torch.equal(a, w) for a, b, w in zip(got, out, base))
    gaps = [room[:64], room[64 + n[0]:128 + n[0]], room[128 + n[0] + n[1]:192 + n[0] + n[1]], room[-64:]]
    assert all((x == 7.0).all() for x in gaps)


def test_repeats_itself_on_any_workspace():
    x = make(2, 8, 2, 900, 128, F16)
    a = kvq.prefill_attn_bwd(*x)
    need = kvq.prefill_attn_bwd_ws_bytes(x[1], x[2])
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")      # NaN wherever it is read before it is written
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, kvq.prefill_attn_bwd(*x, ws=ws)))
    with pytest.raises(kvq.KvqError, match="workspace"):
        kvq.prefill_attn_bwd(*x, ws=ws[:need // 2])
    with pytest.raises(ValueError, match="ws must be"):
        kvq.prefill_attn_bwd(*x, ws=ws.cpu())


def test_graph_replay_and_streams():
    """Two graphs on one workspace and one with its own; calls on a given stream with temporaries dropped."""
    x = make(1, 4, 2, 333, 128, BF16)
    want = kvq.prefill_attn_bwd(*x)
    double = kvq.prefill_attn_bwd(x[0] * 2, *x[1:])
    ws = torch.empty(kvq.prefill_attn_bwd_ws_bytes(x[1], x[2]) + 256, dtype=torch.uint8, device="cuda")
    do, graphs = x[0].clone(), []
    for kw in (dict(ws=ws), dict(ws=ws), {}):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, kvq.prefill_attn_bwd(do, *x[1:], **kw)))
    for src, ref in ((x[0], want), (x[0] * 2, double)):
        do.copy_(src)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [kvq.prefill_attn_bwd(*x, stream=s) for _ in range(3)]
    junk = [torch.full_like(x[1], 9.0) for _ in range(6)]
    s.synchronize()
    assert all(torch.equal(a, b) for out in outs for a, b in zip(out, want))
    del junk


def test_first_calls_inside_a_capture():
    """A process whose first calls of all three operators are captured, with a second capture on another stream's graph."""
    import os
    import subprocess
    import sys
    code = """
import torch
from bit_mixed_precision_gb300 import kvq
g = torch.Generator().manual_seed(0)
x = torch.randn((2, 70, 8, 64), generator=g).half().cuda()
w, pos, rope = torch.ones(64).half().cuda(), torch.arange(70).int().repeat(2, 1).cuda(), kvq.make_rope(64, interleaved=True)
def step():
    q, k, v = kvq.qk_norm_rope(x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], pos, rope, w, w)
    o, lse, _ = kvq.prefill_attn_scores(q, k, v, colscore=False)
    d = kvq.prefill_attn_bwd(o, q, k, v, o, lse)
    return kvq.qk_norm_rope_bwd(*d, x[:, :, :4], x[:, :, 4:6], pos, rope, w, w)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step())) and kvq.device_status() == 0
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_two_calls_at_once():
    """Calls on two streams whose CTAs share the SMs, with a forward pass on a third."""
    x, y = make(1, 8, 2, 1500, 128, F16), make(2, 8, 8, 1100, 64, BF16, seed=1)
    wx, wy = kvq.prefill_attn_bwd(*x), kvq.prefill_attn_bwd(*y)
    wf = kvq.prefill_attn_scores(*x[1:4])
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):
        got.append((kvq.prefill_attn_bwd(*x, stream=s[0]), kvq.prefill_attn_bwd(*y, stream=s[1])))
        with torch.cuda.stream(s[2]):
            f = kvq.prefill_attn_scores(*x[1:4])
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(p, q) for p, q in zip(a, wx)) and all(torch.equal(p, q) for p, q in zip(b, wy))
    assert all(torch.equal(p, q) for p, q in zip(f, wf))


def test_beyond_32_bits():
    """Tensors of more than 2^32 bytes: the last head within the bounds (not bit for bit as in a call of its own: how many
    CTAs share a key tile goes by the number of heads), the one before it untouched by it."""
    B, H, T, D = 8191, 8, 257, 128
    last = make(1, 1, 1, T, D, F16)
    big = [torch.zeros((B, H, T, D), dtype=F16, device="cuda") for _ in range(5)] + [torch.zeros((B, H, T), device="cuda")]
    assert big[0].numel() > 1 << 31
    for a, b in zip(big, last):
        a[-1, -1] = b[0, 0]
    got = kvq.prefill_attn_bwd(*big)
    check(got, *big, heads=[B * H - 1])
    assert all((a[-1, -2] == 0).all() for a in got)


def test_gradient_against_differences():
    """The kernels' own forward pass in float64 differences of a smooth direction: sum of o * do along a step of v (linear),
    and along a small step of q."""
    do, q, k, v, o, lse = make(1, 2, 1, 200, 64, F16, seed=5)
    dq, dk, dv = kvq.prefill_attn_bwd(do, q, k, v, o, lse)
    loss = lambda qq, vv: float((kvq.prefill_attn_scores(qq, k, vv, colscore=False)[0].double() * do.double()).sum())
    # v: o is linear in v; each side's outputs are off by half a step and the rounding of P, 2^-10 of |o| |do| in all
    step = torch.where(dv >= 0, 0.25, -0.25).half()
    up, down = (v + step), (v - step)
    moved = float((dv.double() * (up.double() - down.double())).sum())
    noise = 2.0 ** -10 * float(sum((kvq.prefill_attn_scores(q, k, x.abs(), colscore=False)[0].double().abs()
                                    * do.double().abs()).sum() for x in (up, down)))
    assert abs(loss(q, up) - loss(q, down) - moved) <= noise + 2.0 ** -10 * abs(moved) * 2
    # q: central differences along the gradient's own direction; the third derivative's term (|dz| <= h |k| sigma each way)
    h = 2.0 ** -4
    step = torch.where(dq >= 0, h, -h).half()
    up, down = (q + step), (q - step)
    moved = float((dq.double() * (up.double() - down.double())).sum())
    dz = float((h * k.double().abs().sum(-1)).max()) * 64 ** -0.5
    third = dz ** 3 * float((do.double().abs() * v.double().abs().max()).sum()) * 4
    assert abs(loss(up, v) - loss(down, v) - moved) <= third + 2 * noise


def test_binding_refusals():
    do, q, k, v, o, lse = make(1, 2, 1, 100, 64, F16)
    for bad in ((do.float(), q, k, v, o, lse), (do[:, :, :50], q, k, v, o, lse), (do, q, k, v, o, lse.double()),
                (do, q, k, v, o, lse[:, :1]), (do, q, k, v, o.transpose(2, 3).contiguous().transpose(2, 3), lse)):
        with pytest.raises(ValueError):
            kvq.prefill_attn_bwd(*bad)
    with pytest.raises(ValueError, match="dlse must be"):
        kvq.prefill_attn_bwd(do, q, k, v, o, lse, dlse=lse[:, :, :50])
    with pytest.raises(ValueError, match=r"out\[1\]"):
        kvq.prefill_attn_bwd(do, q, k, v, o, lse, out=(q, q, v))
    with pytest.raises(kvq.KvqError, match="sm_scale"):
        kvq.prefill_attn_bwd(do, q, k, v, o, lse, 0.0)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 1), (128, 2, 2)])
def test_each_gradient_against_differences(D, Hq, Hkv):
    """The kernels' forward pass, sum of o * do + lse * dlse, along a step s of +-1 in every channel of q, k or v, as
    8 (f(s / 2) - f(-s / 2)) - (f(s) - f(-s)): what is cubic in the step drops out, 6 s f' is left.  Noise: an output is off
    by h for its own rounding and h for those of its weights, relatively to the attention over |v| and independently of the
    others, so f by `noise`; the four evaluations have 8, 8, 1 and 1 of it, together 11.4, taken six times.  The gradient
    is off by 8 h in the 2-norm (its own rounding, those of o, P and dS, each h / sqrt(3) of terms about as large as their
    sum).  A check that could miss a factor is none: the bound stays below 5 % of what is compared."""
    do, q, k, v, o, lse = make(1, Hq, Hkv, 200, D, F16, seed=5)
    dlse = torch.randn(lse.shape, generator=torch.Generator().manual_seed(6)).cuda()
    h = 2.0 ** -11
    size = kvq.prefill_attn_scores(q, k, v.abs(), colscore=False)[0].double()
    noise = 2 * h * float((size * do.double()).norm())

    def f(x):
        o, lse, _ = kvq.prefill_attn_scores(*x, colscore=False)
        return float((o.double() * do.double()).sum() + (lse.double() * dlse.double()).sum())

    for i, g in enumerate(kvq.prefill_attn_bwd(do, q, k, v, o, lse, dlse=dlse)):
        found = moved = far = 0.0
        for s, weight in ((2.0 ** -5, 8.0), (2.0 ** -4, -1.0)):
            step, x = torch.where(g >= 0, s, -s).half(), [q, k, v]
            ends = []
            for sign in (1, -1):
                x[i] = (q, k, v)[i] + sign * step
                ends.append((f(x), x[i].double()))
            found += weight * (ends[0][0] - ends[1][0])
            moved += weight * float((g.double() * (ends[0][1] - ends[1][1])).sum())
            far += abs(weight) * float((ends[0][1] - ends[1][1]).norm())
        tol = 6 * 11.4 * noise + 8 * h * float(g.double().norm()) * far
        assert tol < 0.05 * moved, ("qkv"[i], tol, moved)
        assert abs(found - moved) <= tol, ("qkv"[i], found, moved, tol)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("falling", [False, True])
def test_fp16_rows_of_differing_size(D, falling):
    """do of one head from 2^7 down to 2^-14, at random from row to row or falling with the position: fp16's scale of dS is
    a row's own for dQ (up to 2^15 within a tile, |do_i| taken up to 2), and that of the rows from a key's tile on for dK.
    Bounds as above, 2^-39 M with M_i = 2 max(|do_i|, 2^-15 its tile's largest) max |v| + |delta_i| for dQ, and for dK the
    largest |do| max |v| + |delta| of the rows from the key's tile on."""
    T, h = 700, 2.0 ** -11
    do, q, k, v, _, _ = make(1, 1, 1, T, D, F16, seed=9)
    e = torch.linspace(7, -14, T) if falling else 7 - 21 * torch.rand(T, generator=torch.Generator().manual_seed(1))
    do = (do.float() * torch.exp2(e).cuda()[:, None]).half()
    size = 64.0 if falling else 2.0 ** -6               # dQ goes with k, dK with q: above fp16's subnormal numbers
    q, k = (q * size).contiguous(), (k / size).contiguous()
    o, lse, _ = kvq.prefill_attn_scores(q, k, v, colscore=False)
    dq, dk, dv = kvq.prefill_attn_bwd(do, q, k, v, o, lse)
    Q, K, V, O, DO, L = (np_(x[0, 0]).astype(np.float64) for x in (q, k, v, o, do, lse))
    scale = D ** -0.5
    rq, rk, rv, ((P, dP, delta, dS),) = OA.prefill_backward(Q[None], K, V, O[None], DO[None], L[None], scale)
    z, n = np.abs(Q @ K.T).max() * scale, 2 * T * U
    eP = 2 * D * U * scale * (np.abs(Q) @ np.abs(K).T).max() + 4 * U * (z + np.abs(L).max() + 16) + 2.0 ** -22
    E = P * ((eP + 4 * U) * np.abs(dP - delta) + 2 * D * U * (np.abs(DO) @ np.abs(V).T)
             + D * U * (np.abs(DO) * np.abs(O)).sum(-1, keepdims=True) + 2 * U * (np.abs(dP) + np.abs(delta)))
    E += (h + n) * np.abs(dS)
    length = lambda x: np.sqrt((x * x).sum(-1))
    tile = np.arange(T) // 128
    x, most_v, keep = length(DO), length(V).max(), np.tril(np.ones((T, T)))
    largest = np.array([x[tile == t].max() for t in tile])
    M = 2 * np.maximum(x, 2.0 ** -15 * largest) * most_v + np.abs(delta[:, 0])
    tol = scale * (E + 2.0 ** -39 * M[:, None] * keep) @ np.abs(K) + h * np.abs(rq[0]) + 2.0 ** -25
    off = np.abs(np_(dq[0, 0]) - rq[0])
    assert (off <= tol).all(), ("dq", (off / tol).max())
    M = np.array([x[tile >= t].max() * most_v + np.abs(delta[tile >= t]).max() for t in tile])
    tol = scale * (E + 2.0 ** -39 * M[None] * keep).T @ np.abs(Q) + h * np.abs(rk) + 2.0 ** -25
    off = np.abs(np_(dk[0, 0]) - rk)
    assert (off <= tol).all(), ("dk", (off / tol).max())
    tol = (P * (eP + h + n)).T @ np.abs(DO) + 2.0 ** -40 * np.abs(DO).sum(0) + h * np.abs(rv) + 2.0 ** -25
    assert (np.abs(np_(dv[0, 0]) - rv) <= tol).all(), "dv"


def test_rows_without_gradient_leave_fp16s_scale():
    """Rows whose lse is -inf count for nothing, whatever their do: the others come out bit for bit as beside zeros."""
    do, q, k, v, o, lse = make(1, 2, 1, 300, 64, F16, size=2.0 ** -10)
    lse[0, :, 100:140] = -math.inf
    do[0, :, 100:140] = 0
    want = kvq.prefill_attn_bwd(do, q, k, v, o, lse)
    do[0, :, 100:140] = 3e4
    assert all(torch.equal(a, b) for a, b in zip(kvq.prefill_attn_bwd(do, q, k, v, o, lse), want))
