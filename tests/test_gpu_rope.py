"""qk_norm_rope and qk_norm_rope_bwd on the GPU against oracle/rope.py (float64).

Tolerances, u = 2^-24, from the arithmetic of the kernels:
  r       D squares added: D u, halved by the root, rsqrt 2^-22: r is off by at most (D / 2 + 4) u relatively
  y       two products more: (D / 2 + 8) u
  angle   a float32 in [-1, 1): 2^-25 half turns, so pi 2^-25; the fraction of a turn 2^-32; the float64 quotient behind it
          and the model's own product pos * f: |pos| 2^-51 each.  sincospi 2 u.  Together c = 2^-22 + |pos| 2^-50
  pair    (|a| + |b|) (c + (D / 2 + 12) u), a and b the exact sides of the pair before the turn
  output  half a step of its type (eps / 2 relatively, 2^-25 for fp16 below its normal range)
Backward: dy as `pair`; g = dy w, x r, their mean over D: each term of dx = r (g - x r mean(g x r)) is off by at most
  E = c + (2 D + 32) u relatively to r (G + |x r| mean(G |x r|)), G = (|a| + |b|) |w|.
  dw: E sum (|a| + |b|) |x r|, and n u of it for the additions, n rows.
"""
import math

import numpy as np
import pytest
import torch

from oracle import rope as OR
from tests.helpers import np_

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvq():
    from bit_mixed_precision_gb300 import kvq
    yield kvq


class Case:
    def __init__(self, kvq, B=2, T=5, Hq=4, Hkv=2, D=128, dtype=F16, rot=None, axes=1, interleaved=False, norm=(1, 1),
                 w_dtype=None, start=0, eps=1e-6, seed=0, step=False):
        g = torch.Generator().manual_seed(seed)
        self.kvq, self.B, self.T, self.Hq, self.Hkv, self.D, self.dtype, self.eps = kvq, B, T, Hq, Hkv, D, dtype, eps
        self.step, self.interleaved = step, interleaved
        rot = D if rot is None else rot
        n = rot // 2
        self.f = [10000.0 ** (-i / max(n, 1)) for i in range(n)]
        self.axis = [i % axes for i in range(n)]
        self.rope = kvq.make_rope(D, rot=rot, inv_freq=self.f, axis=self.axis, interleaved=interleaved)
        x = torch.randn((B, T, Hq + 2 * Hkv, D), generator=g) * torch.exp(torch.randn((Hq + 2 * Hkv, 1), generator=g))
        self.x = x.to(dtype).cuda()                         # one projection
        self.q, self.k, self.v = self.x[:, :, :Hq], self.x[:, :, Hq:Hq + Hkv], self.x[:, :, Hq + Hkv:]
        w = lambda on: (1 + 0.3 * torch.randn(D, generator=g)).to(w_dtype or dtype).cuda() if on else None
        self.qw, self.kw = w(norm[0]), w(norm[1])
        self.axes = max(self.axis, default=0) + 1
        pos = torch.randint(-50, 50, (self.axes, B, T), generator=g) + start
        self.pos = pos.to(torch.int32).cuda()
        self.angle = OR.angles(self.pos.cpu().numpy(), self.f, self.axis)
        self.c = 2.0 ** -22 + float(pos.abs().max()) * 2.0 ** -50
        self.d = [torch.randn((B, h, T, D), generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv)]

    def args(self):
        """q, k, v, pos as the call takes them."""
        if self.step:
            return self.q[:, 0], self.k[:, 0], self.v[:, 0], self.pos[:, :, 0] if self.axes > 1 else self.pos[0, :, 0]
        return self.q, self.k, self.v, self.pos if self.axes > 1 else self.pos[0]

    def forward(self, **kw):
        q, k, v, pos = self.args()
        return self.kvq.qk_norm_rope(q, k, v, pos, self.rope, self.qw, self.kw, self.eps, **kw)

    def backward(self, **kw):
        q, k, _, pos = self.args()
        d = [x[:, :, 0] for x in self.d] if self.step else self.d
        return self.kvq.qk_norm_rope_bwd(*[x.contiguous() for x in d], q, k, pos, self.rope, self.qw, self.kw, self.eps, **kw)

    def half(self, ref):
        return torch.finfo(self.dtype).eps / 2 * np.abs(ref) + (2.0 ** -25 if self.dtype == F16 else 0.0)

    def both_sides(self, y):
        """|a| + |b| at each channel of rows y [..., D] (|y| where it does not turn)."""
        out, p = np.abs(y), OR.pairs(len(self.f) * 2, self.interleaved)
        if len(p):
            out[..., p[:, 0]] = out[..., p[:, 1]] = np.abs(y[..., p[:, 0]]) + np.abs(y[..., p[:, 1]])
        return out

    def check_forward(self, got):
        for x, w, o in ((self.q, self.qw, got[0]), (self.k, self.kw, got[1])):
            x, w, o = np_(x).astype(np.float64), None if w is None else np_(w), np_(o)
            o = o[:, :, None] if self.step else o
            ref = OR.forward(x, w, self.eps, self.angle, self.interleaved)
            y = OR.forward(x, w, self.eps, 0 * self.angle, self.interleaved)
            tol = self.both_sides(y) * (self.c + (self.D / 2 + 12) * U) + self.half(ref)
            off = np.abs(o - ref)
            assert (off <= tol).all(), (off / tol).max()
        if got[2] is not None:
            o = got[2][:, :, None] if self.step else got[2]
            assert torch.equal(o, self.v.transpose(1, 2))

    def check_backward(self, got):
        E = self.c + (2 * self.D + 32) * U
        for x, w, d, o, ow in ((self.q, self.qw, self.d[0], got[0], got[3]), (self.k, self.kw, self.d[1], got[1], got[4])):
            x, w, d, o = np_(x).astype(np.float64), None if w is None else np_(w).astype(np.float64), np_(d), np_(o)
            o = o[:, None] if self.step else o
            ref, dw = OR.backward(d, x, w, self.eps, self.angle, self.interleaved)
            G = self.both_sides(d.astype(np.float64).transpose(0, 2, 1, 3))
            if w is None:
                tol = G * E
            else:
                r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + self.eps)
                xr, Gw = np.abs(x * r), G * np.abs(w)
                tol = E * r * (Gw + xr * (Gw * xr).mean(-1, keepdims=True))
                rows = x.size // self.D
                off, wtol = np.abs(np_(ow) - dw), (E + rows * U) * (G * xr).sum((0, 1, 2))
                assert (off <= wtol).all(), (off / wtol).max()
            off, tol = np.abs(o - ref), tol + self.half(ref)
            assert (off <= tol).all(), (off / tol).max()
        assert (got[3] is None) == (self.qw is None) and (got[4] is None) == (self.kw is None)
        if got[2] is not None:
            o = got[2][:, None] if self.step else got[2]
            assert torch.equal(o, self.d[2].transpose(1, 2))


KINDS = [
    dict(),
    dict(dtype=BF16, Hq=5, Hkv=1, T=1),
    dict(D=64, rot=16, interleaved=True, T=33),
    dict(D=64, Hq=9, Hkv=3, rot=48, axes=3, dtype=BF16),
    dict(rot=0, norm=(1, 1)),
    dict(rot=16, norm=(0, 0), interleaved=True),
    dict(norm=(1, 0), axes=4, B=1, T=37),
    dict(norm=(0, 1), axes=2, rot=112, interleaved=True, dtype=BF16),
    dict(w_dtype=F32, dtype=BF16, Hq=40, Hkv=8, T=3),
    dict(start=1 << 20, T=64, B=1),
    dict(start=2147483000, dtype=BF16),
    dict(start=-2147483000, D=64),
    dict(B=1, T=700, Hq=2, Hkv=2, D=64),
    dict(B=3, T=1, Hq=12, Hkv=4, step=True),
    dict(B=70, T=1, Hq=32, Hkv=8, step=True, axes=3, dtype=BF16, start=100000),
    dict(B=1, T=1, Hq=1, Hkv=1, step=True, D=64, rot=32),
    dict(eps=0.5),
]


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_forward(kvq, kind):
    c = Case(kvq, **kind)
    c.check_forward(c.forward())


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_backward(kvq, kind):
    c = Case(kvq, **kind)
    c.check_backward(c.backward())


def test_strides_and_missing_values(kvq):
    """Heads first, broadcast batches, every second token, rows of one axis; no values."""
    c = Case(kvq, B=2, T=6, Hq=4, Hkv=2, D=64)
    base = c.forward()
    heads_first = c.q.transpose(1, 2).contiguous().transpose(1, 2)
    far = torch.zeros((2, 12, 5, 64), dtype=F16, device="cuda")
    far[:, ::2, :2] = c.k
    o = kvq.qk_norm_rope(heads_first, far[:, ::2, :2], None, c.pos, c.rope, c.qw, c.kw, c.eps)
    assert torch.equal(o[0], base[0]) and torch.equal(o[1], base[1]) and o[2] is None
    same = c.q[:1].expand(2, 6, 4, 64)                      # stride 0 over the batch
    o = kvq.qk_norm_rope(same, c.k, None, c.pos, c.rope, c.qw, c.kw, c.eps)
    assert torch.equal(o[0][0], base[0][0]) and torch.equal(o[1], base[1])
    one = kvq.qk_norm_rope(c.q[:, 3:4], c.k[:, 3:4], c.v[:, 3:4], c.pos[0][:, 3:4].contiguous(), c.rope, c.qw, c.kw, c.eps)
    assert all(torch.equal(a[:, :, 0], b[:, :, 3]) for a, b in zip(one, base))
    step = kvq.qk_norm_rope(c.q[:, 3], c.k[:, 3], c.v[:, 3], c.pos[0][:, 3].contiguous(), c.rope, c.qw, c.kw, c.eps)
    assert all(torch.equal(a, b[:, :, 3]) for a, b in zip(step, base))


def test_outputs_given_and_nothing_else_written(kvq):
    c = Case(kvq, B=2, T=3, Hq=3, Hkv=1, D=64, dtype=BF16)
    base, grads = c.forward(), c.backward()
    out = tuple(torch.full_like(x, 7.0) for x in base)
    got = c.forward(out=out)
    assert all(a is b and torch.equal(a, w) for a, b, w in zip(got, out, base))
    wide = torch.full((2, 3, 9, 64), 7.0, dtype=BF16, device="cuda")        # the gradients inside a larger array
    gw = [torch.full((66,), 7.0, device="cuda") for _ in range(2)]
    got = c.backward(out=(wide[:, :, 1:4], wide[:, :, 5:6], wide[:, :, 7:8], gw[0][1:65], gw[1][1:65]))
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    assert (wide[:, :, [0, 4, 6, 8]] == 7.0).all() and all((g[[0, 65]] == 7.0).all() for g in gw)
    assert grads[0].stride() == (3 * 5 * 64, 5 * 64, 64, 1)                # views of one gradient of the projection


def test_rows_do_not_touch_one_another(kvq):
    """A row with NaN or infinity spoils itself only; rows of zeros stay zero."""
    c = Case(kvq, B=1, T=4, Hq=4, Hkv=4, D=128)
    base = c.forward()
    c.q[0, 1, 2, 5], c.k[0, 2, 0, 9] = float("nan"), float("inf")
    c.q[0, 3, 1] = 0.0
    q, k, _ = c.forward()
    ok = torch.ones((1, 4, 4), dtype=torch.bool, device="cuda")
    okq, okk = ok.clone(), ok.clone()
    okq[0, 2, 1] = okq[0, 1, 3] = okk[0, 0, 2] = False
    assert torch.equal(q[okq], base[0][okq]) and torch.equal(k[okk], base[1][okk])
    assert q[0, 2, 1].isnan().all() and (q[0, 1, 3] == 0).all()
    g = c.backward()
    assert g[0][0, 1, 2].isnan().all() and g[0][0, 0].isfinite().all() and g[0][0, 3, 1].isfinite().all()


def test_gradient_against_differences(kvq):
    """The kernels' own forward pass, differenced in float16: sum of out * d along a direction."""
    c = Case(kvq, B=1, T=3, Hq=2, Hkv=1, D=64, dtype=F16, w_dtype=F32, seed=3)
    gq, gk, gv, gqw, gkw = c.backward()
    f = lambda: sum((o.double() * d.double()).sum() for o, d in zip(c.forward(), c.d))
    h = 2.0 ** -3
    for w, g in ((c.qw, gqw), (c.kw, gkw)):                 # linear in the weights: no curvature
        step = torch.sign(g)
        w += h * step
        up = f()
        w -= 2 * h * step
        down = f()
        w += h * step
        # each side sums outputs off by half a step each, independent of one another
        size = float(torch.stack([(o.double().abs() * d.double().abs()).sum() for o, d in zip(c.forward(), c.d)]).sum())
        assert abs(float(up - down) / (2 * h) - float((g * step).sum())) <= 2.0 ** -11 * 1.5 * size / h


def test_backward_repeats_itself(kvq):
    c = Case(kvq, B=2, T=901, Hq=8, Hkv=8, D=128, dtype=BF16)
    a, b = c.backward(), c.backward()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    ws = torch.full((kvq.qk_norm_rope_bwd_ws_bytes(c.q) + 256,), 255, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(x, y) for x, y in zip(a, c.backward(ws=ws)))
    with pytest.raises(kvq.KvqError, match="workspace"):
        c.backward(ws=ws[:256])
    with pytest.raises(ValueError, match="ws must be"):
        c.backward(ws=ws.view(torch.int32))


@pytest.mark.parametrize("T", [4096, 1])
def test_many_tokens(kvq, T):
    """More tokens than the backward pass has warps, sampled; weight gradients in full."""
    c = Case(kvq, B=1 if T > 1 else 5000, T=T, Hq=8, Hkv=2, D=64, dtype=BF16, step=T == 1)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


def test_beyond_32_bits(kvq):
    """A projection of more than 2^32 bytes: its last tokens."""
    B, T, H, D = 1, 70001, 80, 128
    x = torch.zeros((B, T, 3 * H, D), dtype=F16, device="cuda")
    assert x.numel() > 1 << 31
    last = torch.randn((4, 3 * H, D), generator=torch.Generator().manual_seed(1)).half().cuda()
    x[0, -4:] = last
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    rope, w = kvq.make_rope(D), torch.ones(D, dtype=F16, device="cuda")
    small = kvq.qk_norm_rope(last[None, :, :H], last[None, :, H:2 * H], last[None, :, 2 * H:], pos[:, -4:].contiguous(), rope, w, w)
    got = kvq.qk_norm_rope(x[:, :, :H], x[:, :, H:2 * H], x[:, :, 2 * H:], pos, rope, w, w)
    assert all(torch.equal(a[:, :, -4:], b) for a, b in zip(got, small))
    g = kvq.qk_norm_rope_bwd(*got, x[:, :, :H], x[:, :, H:2 * H], pos, rope, w, w)
    s = kvq.qk_norm_rope_bwd(*small, last[None, :, :H], last[None, :, H:2 * H], pos[:, -4:].contiguous(), rope, w, w)
    assert all(torch.equal(a[:, -4:], b) for a, b in zip(g[:3], s[:3]))


def test_no_tokens(kvq):
    c = Case(kvq, B=2, T=3, D=64)
    e = lambda *s: torch.empty(s, dtype=F16, device="cuda")
    pos = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    q, k, v = kvq.qk_norm_rope(e(2, 0, 4, 64), e(2, 0, 2, 64), e(2, 0, 2, 64), pos, c.rope, c.qw, c.kw)
    assert q.shape == (2, 4, 0, 64) and v.shape == (2, 2, 0, 64)
    g = kvq.qk_norm_rope_bwd(q, k, v, e(2, 0, 4, 64), e(2, 0, 2, 64), pos, c.rope, c.qw, c.kw)
    assert g[0].shape == (2, 0, 4, 64) and (g[3] == 0).all() and (g[4] == 0).all()


def test_graph_replay_and_streams(kvq):
    """Two graphs that share a workspace, replayed with new inputs in place; a call on a stream given, whose temporaries go
    back to the allocator at once."""
    c = Case(kvq, B=2, T=200, Hq=8, Hkv=2, D=128, dtype=BF16)
    want, grads = c.forward(), c.backward()
    c.x.mul_(2.0)
    want2, grads2 = c.forward(), c.backward()
    ws = torch.empty(kvq.qk_norm_rope_bwd_ws_bytes(c.q) + 256, dtype=torch.uint8, device="cuda")
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, c.forward(), c.backward(ws=ws)))
    for scale, w, gr in ((0.5, want, grads), (2.0, want2, grads2)):
        c.x.mul_(scale)
        for g, fo, ba in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, fo, ba in graphs:
            assert all(torch.equal(x, y) for x, y in zip(fo, w)) and all(torch.equal(x, y) for x, y in zip(ba, gr))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [(c.forward(stream=s), c.backward(stream=s)) for _ in range(3)]
    junk = [torch.full_like(c.x, 9.0) for _ in range(3)]
    s.synchronize()
    for fo, ba in outs:
        assert all(torch.equal(x, y) for x, y in zip(fo, want2)) and all(torch.equal(x, y) for x, y in zip(ba, grads2))
    del junk


def test_binding_refusals(kvq):
    c = Case(kvq, B=2, T=3, Hq=4, Hkv=2, D=64)
    f = lambda **kw: kvq.qk_norm_rope(*[kw.get(n, d) for n, d in zip("q k v pos".split(), c.args())], c.rope,
                                      kw.get("qw", c.qw), kw.get("kw", c.kw), out=kw.get("out"))
    f()
    with pytest.raises(ValueError, match="last axis"):
        f(q=c.q.transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(ValueError, match="k must be"):
        f(k=c.k.bfloat16())
    with pytest.raises(ValueError, match="v must be"):
        f(v=c.v[:, :2])
    with pytest.raises(ValueError, match="pos must be"):
        f(pos=c.pos[0].long())
    with pytest.raises(ValueError, match="q_weight must be"):
        f(qw=c.qw[:32])
    with pytest.raises(TypeError, match="share one dtype"):
        f(qw=c.qw.float())
    with pytest.raises(kvq.KvqError, match="multiples of 8"):
        f(q=torch.empty((2, 3, 4, 68), dtype=F16, device="cuda")[..., :64])
    with pytest.raises(kvq.KvqError, match="aligned"):
        f(q=torch.empty(2 * 3 * 4 * 64 + 8, dtype=F16, device="cuda")[4:-4].view(2, 3, 4, 64))
    base = c.forward()
    with pytest.raises(ValueError, match=r"out\[0\]"):
        f(out=(base[0][:, :2], base[1], base[2]))
    with pytest.raises(ValueError, match="out must have a v"):
        f(out=(base[0], base[1], None))
    with pytest.raises(ValueError, match="dq must be"):
        kvq.qk_norm_rope_bwd(c.d[0][:, :2], c.d[1], c.d[2], c.q, c.k, c.pos[0], c.rope)
    with pytest.raises(ValueError, match="out must have a gradient"):
        kvq.qk_norm_rope_bwd(*c.d, c.q, c.k, c.pos[0], c.rope, c.qw, c.kw, out=(c.q, c.k, c.v, None, None))


def test_prompt_and_steps_through_the_block_cache(kvq):
    """Projection -> norm and rotation -> prefill attention, 8-bit cache, a step of attention over it, against float64."""
    B, T, Hq, Hkv, D = 2, 130, 4, 2, 64
    c = Case(kvq, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, dtype=F16, rot=32)
    c.pos.copy_(torch.arange(T, dtype=torch.int32, device="cuda").expand(1, B, T))
    c.angle = OR.angles(c.pos.cpu().numpy(), c.f, c.axis)
    n = T - 1
    cache = kvq.make_block8_cache(B, Hq, Hkv, D, F16, T, block=16)
    q, k, v = kvq.qk_norm_rope(c.q[:, :n], c.k[:, :n], c.v[:, :n], c.pos[0, :, :n].contiguous(), c.rope, c.qw, c.kw, c.eps)
    o, lse, cs = kvq.prefill_attn_scores(q, k, v)
    kvq.block8_append(cache, k, v, colscore=cs)
    q1, k1, v1 = kvq.qk_norm_rope(c.q[:, n], c.k[:, n], c.v[:, n], c.pos[0, :, n].contiguous(), c.rope, c.qw, c.kw, c.eps)
    kvq.block8_append(cache, k1, v1)
    o1, _ = kvq.block8_attn(q1, cache)
    rq = OR.forward(np_(c.q), np_(c.qw), c.eps, c.angle, False)
    rk = OR.forward(np_(c.k), np_(c.kw), c.eps, c.angle, False)
    rv = np_(c.v).astype(np.float64).transpose(0, 2, 1, 3)
    size = lambda x: np.sqrt((x * x).sum(-1)).max()
    for b in range(B):
        for h in range(Hq):
            u = b * Hkv + h // 2
            s = rq[b, h] @ rk[b, h // 2].T / math.sqrt(D)
            p = np.tril(np.exp(s - s.max(-1, keepdims=True)))
            ref = p / p.sum(-1, keepdims=True) @ rv[b, h // 2]
            # q and k rounded to fp16 move a logit by at most 2 2^-11 |q| |k| / sqrt(D) (and a little for float32), so the
            # weights by twice that relatively; the weights themselves are rounded to 2^-11, the output too
            most, logit = np.abs(rv[b, h // 2]).max(), 2.0 ** -9.9 * size(rq[b, h]) * size(rk[b, h // 2]) / math.sqrt(D)
            assert np.abs(np_(o[b, h]) - ref[:n]).max() <= (np.expm1(2 * logit) + 2.0 ** -9) * most
            # the cache's keys and values: a code is off by half a step of 3 bits, 2^-4 (below its normal range 2^-10 / 448
            # of the block's largest); the attention over what it holds: q rounded
            dk, dv = (np_(x).astype(np.float64) for x in cache.dequantised(u))
            for got, want in ((dk, rk[b, h // 2]), (dv, rv[b, h // 2])):
                assert (np.abs(got - want) <= (2.0 ** -4 + 2.0 ** -10) * np.abs(want) + 2.0 ** -18 * np.abs(want).max()).all()
            s = rq[b, h, n] @ dk.T / math.sqrt(D)
            p = np.exp(s - s.max())
            logit = 2.0 ** -10.9 * size(rq[b, h]) * size(dk) / math.sqrt(D)
            assert np.abs(np_(o1[b, h]) - p / p.sum() @ dv).max() <= (np.expm1(2 * logit) + 2.0 ** -10) * np.abs(dv).max()


@pytest.mark.parametrize("dtype,D,rot", [(F16, 64, 32), (BF16, 128, 128)])
def test_training_step(kvq, dtype, D, rot):
    """Forward and backward pass of a layer between its projection and its output: every call on what the calls before it
    gave, each within its own bounds, and the gradient of the projection's output against float64 autograd."""
    from tests.test_gpu_prefill_bwd import check
    B, T, Hq, Hkv = 2, 200, 4, 2
    c = Case(kvq, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, rot=rot, seed=5)
    got = c.forward()
    c.check_forward(got)
    q, k, v = got
    o, lse, _ = kvq.prefill_attn_scores(q, k, v)
    do = torch.randn(o.shape, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()
    d = kvq.prefill_attn_bwd(do, q, k, v, o, lse)
    check(d, do, q, k, v, o, lse)
    c.d = list(d)
    grads = c.backward()
    c.check_backward(grads)
    # the whole in float64
    x = c.x.double().cpu().requires_grad_()
    w = [y.double().cpu().requires_grad_() for y in (c.qw, c.kw)]
    phi, n = torch.from_numpy(c.angle)[:, :, None], rot // 2
    def normed(y, w):
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + c.eps) * w
        a, b = y[..., :n], y[..., n:rot]
        return torch.cat([a * phi.cos() - b * phi.sin(), b * phi.cos() + a * phi.sin(), y[..., rot:]], -1).transpose(1, 2)
    rq, rk = normed(x[:, :, :Hq], w[0]), normed(x[:, :, Hq:Hq + Hkv], w[1])
    rk, rv = (y.repeat_interleave(Hq // Hkv, 1) for y in (rk, x[:, :, Hq + Hkv:].transpose(1, 2)))
    s = (rq @ rk.transpose(-1, -2) * D ** -0.5).masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), -math.inf)
    ((s.softmax(-1) @ rv) * do.double().cpu()).sum().backward()
    # q, k rounded: a logit is off by at most `logit`, weights by expm1(2 logit) relatively; v, o, do, P, dS, dq, dk and dv
    # are off by half a step h each, relatively to terms that add up to sums sqrt(T) times smaller at worst (random signs):
    # in the 2-norm (8 h + expm1(2 logit)) times that, taken for the largest row norms
    h = torch.finfo(dtype).eps / 2
    logit = 2 * h * float((rq.norm(dim=-1).max() * rk.norm(dim=-1).max()).detach()) * D ** -0.5
    bound = (8 * h + math.expm1(2 * logit)) * math.sqrt(T)
    for a, ref in ((grads[0], x.grad[:, :, :Hq]), (grads[1], x.grad[:, :, Hq:Hq + Hkv]), (grads[2], x.grad[:, :, Hq + Hkv:]),
                   (grads[3], w[0].grad), (grads[4], w[1].grad)):
        off = float((a.double().cpu() - ref).norm() / ref.norm())
        assert off <= min(bound, 0.1), (off, bound)


@pytest.mark.parametrize("D,Hq,Hkv,interleaved,norm", [
    (64, 4, 4, False, (1, 1)),
    (64, 9, 3, True, (1, 1)),
    (128, 6, 2, False, (1, 1)),
    (128, 5, 1, True, (1, 0)),
    (64, 20, 4, False, (0, 1)),
    (128, 8, 4, False, (1, 1)),
])
def test_backward_without_eps(kvq, D, Hq, Hkv, interleaved, norm):
    """eps = 0 on rows that are not zero, also where the heads do not fill a warp's rows: 1 / sqrt(0) of a row that is not
    there must not reach the weights' gradients."""
    c = Case(kvq, B=2, T=9, Hq=Hq, Hkv=Hkv, D=D, interleaved=interleaved, norm=norm, eps=0.0, seed=7)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


BEHIND = [(64, 16, False), (64, 32, True), (128, 48, False), (128, 112, True), (64, 0, False), (128, 0, True)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,rot,interleaved", BEHIND)
def test_infinities_behind_the_rotated_channels(kvq, D, rot, interleaved, dtype):
    """Channels that do not turn leave without a norm as they came, and touch no other channel, both ways."""
    c = Case(kvq, B=1, T=6, Hq=6, Hkv=3, D=D, rot=rot, interleaved=interleaved, dtype=dtype, norm=(0, 0))
    base, grads = c.forward(), c.backward()
    put = [(rot, math.inf), (rot + 3, -math.inf), (D - 1, math.nan), ((rot + D) // 2, math.inf), (rot + 1, -0.0)]
    for i, (ch, x) in enumerate(put):
        c.q[0, i, i, ch] = c.k[0, i, i % 3, ch] = x
        c.d[0][0, i, i, ch] = c.d[1][0, i % 3, i, ch] = x
    got, back = c.forward(), c.backward()
    for raw, want, o in ((c.q, base[0], got[0]), (c.k, base[1], got[1])):
        want = want.clone()
        want[..., rot:] = raw.transpose(1, 2)[..., rot:]
        torch.testing.assert_close(o, want, rtol=0, atol=0, equal_nan=True)
        assert torch.equal(o.signbit()[..., rot:] | o[..., rot:].isnan(), want.signbit()[..., rot:] | want[..., rot:].isnan())
    for d, want, o in ((c.d[0], grads[0], back[0]), (c.d[1], grads[1], back[1])):
        want = want.clone()
        want[..., rot:] = d.transpose(1, 2)[..., rot:]
        torch.testing.assert_close(o, want, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("D,rot,interleaved", BEHIND)
def test_infinities_behind_the_rotated_channels_of_a_normed_row(kvq, D, rot, interleaved):
    """An infinite sum of squares leaves x * 0: zeros, and NaN in the infinite channel alone."""
    c = Case(kvq, B=1, T=2, Hq=3, Hkv=1, D=D, rot=rot, interleaved=interleaved)
    c.q[0, 1, 2, rot + 2], c.k[0, 0, 0, D - 2] = math.inf, -math.inf
    q, k, _ = c.forward()
    for row, ch in ((q[0, 2, 1], rot + 2), (k[0, 0, 0], D - 2)):
        assert row[ch].isnan() and (torch.cat([row[:ch], row[ch + 1:]]) == 0).all()


@pytest.mark.parametrize("kind", [dict(B=3, T=1, Hq=12, Hkv=4, step=True), dict(B=2, T=301, D=64, dtype=BF16),
                                  dict(B=1, T=40, Hq=5, Hkv=5, rot=32, interleaved=True)], ids=str)
def test_in_place(kvq, kind):
    """Outputs in place of their own inputs, and gradients beside one another in one array."""
    c = Case(kvq, **kind)
    base, grads = c.forward(), c.backward()
    at = (lambda x: x[:, 0]) if c.step else (lambda x: x)
    q, k, v = (x.clone() for x in base)                     # [B, heads, T, D] storage: raw rows as views of it
    turned = (lambda x: x) if c.step else (lambda x: x.transpose(1, 2))
    for dst, src in ((q, c.q), (k, c.k), (v, c.v)):
        turned(dst).copy_(at(src))
    pos = c.args()[3]
    got = kvq.qk_norm_rope(turned(q), turned(k), turned(v), pos, c.rope, c.qw, c.kw, c.eps, out=(q, k, v))
    assert all(a is b and torch.equal(a, w) for a, b, w in zip(got, (q, k, v), base))
    # the gradient over the projection itself (the values are not read)
    x = c.x.clone()
    parts = [at(y) for y in (x[:, :, :c.Hq], x[:, :, c.Hq:c.Hq + c.Hkv], x[:, :, c.Hq + c.Hkv:])]
    d = [(y[:, :, 0] if c.step else y).contiguous() for y in c.d]
    weights = [torch.empty(c.D, device="cuda") for _ in range(2)]
    got = kvq.qk_norm_rope_bwd(*d, parts[0], parts[1], pos, c.rope, c.qw, c.kw, c.eps, out=(*parts, *weights))
    assert all(torch.equal(a, w) for a, w in zip(got, grads))
    # over the gradients that come in
    d = [y.clone() for y in d]
    got = kvq.qk_norm_rope_bwd(*d, at(c.q), at(c.k), pos, c.rope, c.qw, c.kw, c.eps, out=(*[turned(y) for y in d], *weights))
    assert all(torch.equal(a, w) for a, w in zip(got, grads))


def test_gradients_as_views_of_one_array(kvq):
    """Layouts whose rows lie between one another but share nothing are taken."""
    c = Case(kvq, B=2, T=7, Hq=2, Hkv=2, D=64)
    grads, w = c.backward(), [torch.empty(64, device="cuda") for _ in range(2)]
    new = lambda *s: torch.full(s, 7.0, dtype=F16, device="cuda")
    a, b, e = new(2, 7, 2, 3, 64), new(3, 2, 2, 7, 64), new(2, 6, 14, 72)
    for out in ([a[:, :, :, i] for i in range(3)],                              # a head's query, key and value side by side
                [b[i].transpose(1, 2) for i in range(3)],                       # heads first
                [e[:, i::3, ::2, 8:].transpose(1, 2) for i in range(3)],        # every second token, room before each row
                [e[:, 2 * i:2 * i + 2, i % 2::2, :64].transpose(1, 2) for i in range(3)]):
        got = c.backward(out=(*out, *w))
        assert all(torch.equal(x, y) for x, y in zip(got, grads))


@pytest.mark.parametrize("dtype,D,rot", [(F16, 64, 32), (BF16, 128, 128)])
def test_training_step_row_by_row(kvq, dtype, D, rot):
    """The projection's gradient row by row against a float64 chain over the forward pass' stored q, k, v, o and lse.
    P and dS round to h each, every one by itself: a row of dq is off by h / sqrt(3) S in the 2-norm, S the root of the sum of
    its squared terms scale dS_ij |k_j| (dk: |q_i|, dv: P_ij |do_i|), and by h of itself for its own rounding.  The norm's
    gradient passes that on times r |w| at most, a channel of the weights' gradient times |x r|, rows adding up in
    squares; the result rounds to h (the weights' to float32).  6 times that, and float32's sums: dP and
    delta add D products each, so that dS is off by D 2^-23 P |do| |v| also where it is 0 (a sequence's first row)."""
    B, T, Hq, Hkv = 2, 200, 4, 2
    g = Hq // Hkv
    c = Case(kvq, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, rot=rot, seed=5)
    q, k, v = c.forward()
    o, lse, _ = kvq.prefill_attn_scores(q, k, v)
    do = torch.randn(o.shape, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()
    d = kvq.prefill_attn_bwd(do, q, k, v, o, lse)
    got = kvq.qk_norm_rope_bwd(*d, c.q, c.k, c.pos if c.axes > 1 else c.pos[0], c.rope, c.qw, c.kw, c.eps)
    from oracle import attention as OA
    f64 = lambda x: np_(x).astype(np.float64)
    ref = [np.zeros(x.shape) for x in d]
    S = [np.zeros(x.shape[:3]) for x in d]
    F = [np.zeros(x.shape[:3]) for x in d]
    length = lambda x: np.sqrt((x * x).sum(-1))
    for b in range(B):
        for u in range(Hkv):
            at = slice(u * g, (u + 1) * g)
            Q, K, V, O, DO, L = f64(q[b, at]), f64(k[b, u]), f64(v[b, u]), f64(o[b, at]), f64(do[b, at]), f64(lse[b, at])
            ref[0][b, at], ref[1][b, u], ref[2][b, u], terms = OA.prefill_backward(Q, K, V, O, DO, L, D ** -0.5)
            for i, (P, _, _, dS) in enumerate(terms):
                S[0][b, u * g + i] = np.sqrt((dS * dS) @ (length(K) ** 2)) * D ** -0.5
                S[1][b, u] += (dS * dS).T @ (length(Q[i]) ** 2) / D
                S[2][b, u] += (P * P).T @ (length(DO[i]) ** 2)
                low = D * 2.0 ** -23 * P * length(DO[i])[:, None] * length(V) * D ** -0.5
                F[0][b, u * g + i] = low @ length(K)
                F[1][b, u] += low.T @ length(Q[i])
    S[1], S[2] = np.sqrt(S[1]), np.sqrt(S[2])
    h = torch.finfo(dtype).eps / 2
    for i, (raw, w) in enumerate(((c.q, c.qw), (c.k, c.kw))):
        x, w = f64(raw), f64(w)
        dx, dw = OR.backward(ref[i], x, w, c.eps, c.angle, False)
        r = 1 / np.sqrt((x * x).mean(-1) + c.eps)
        err = (h * (S[i] + length(ref[i])) + F[i]).transpose(0, 2, 1)
        tol = 6 * (err * r * np.abs(w).max() + h * length(dx))
        off = length(f64(got[i]) - dx)
        assert (off <= tol).all(), (off / tol).max()
        tol = 6 * np.sqrt(((err[..., None] * x * r[..., None]) ** 2).sum((0, 1, 2)))
        assert (np.abs(f64(got[3 + i]) - dw) <= tol).all()
        # the bounds are worth something
        tol = 6 * (err * r * np.abs(w).max() + h * length(dx))
        assert np.median(tol) / np.median(length(dx)) < (0.02 if dtype == F16 else 0.15)
    dv = ref[2].transpose(0, 2, 1, 3)
    off, tol = length(f64(got[2]) - dv), 6 * h * (S[2].transpose(0, 2, 1) + length(dv))
    assert (off <= tol).all(), (off / tol).max()
