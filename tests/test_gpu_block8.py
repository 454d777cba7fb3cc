"""GPU parity of the 8-bit block cache (block8_*) against the CPU model in oracle/block8.py.

Codes, scales, bounds, positions, tables and chosen blocks are compared exactly.  Tolerances of the attention, derived
from its arithmetic (u = 2^-24, D channels, n tokens seen):
  logit      products of 16-bit queries and 8-bit codes are exact, D of them are added in float32 (a tensor core may cut
             instead of round: 2u each), then four float32 factors:  e = (2 D + 8) u sigma max_j sum_c |q_c k_jc|
  weight     exp2 of a logit: e, plus 2^-22 of the hardware's exp2 and the rounding of its argument, |s - max| 2u <= 2^-15
             where weights still count (|s - max| < 128);  the sum of n weights: n u;  the fp16 pair of a weight 2^-22
  output     n products added: 2 n u;  so |o - ref| <= (2 e + 2^-13 + 4 n u) sum_j p_j |v_j| + half a step of the
             16-bit output (eps/2 |ref|, 2^-25 below fp16's normal range);  2^-13 holds 2 * 2^-15 and the small terms
  lse        e + 2^-14 + n u + 2^-22 |lse|;   acc: (2 e + 2^-13 + 2 n u) relative, plus u of the sum it is added to
"""
import math

import numpy as np
import pytest
import torch

from oracle import block8 as O8

pytestmark = pytest.mark.gpu
U24 = 2.0 ** -24
F8, I8 = torch.float8_e4m3fn, torch.int8
KIND = {F8: "e4m3", I8: "int8"}


@pytest.fixture(scope="module")
def kvq():
    from bit_mixed_precision_gb300 import kvq
    yield kvq


@pytest.fixture(autouse=True)
def status_is_clean(kvq):
    yield
    assert kvq.device_status() == 0


class Pair:
    """A cache and its CPU model, fed the same tokens."""

    def __init__(self, kvq, B=2, Hq=4, Hkv=2, D=128, block=16, codes=F8, dtype=torch.float16, max_tokens=256, seed=0,
                 **kw):
        self.kvq, self.B, self.Hq, self.Hkv, self.D, self.g = kvq, B, Hq, Hkv, D, Hq // Hkv
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator().manual_seed(seed)
        self.c = kvq.make_block8_cache(B, Hq, Hkv, D, dtype, max_tokens, block=block, codes=codes, **kw)
        n = self.c.table.numel()
        perm = torch.randperm(n, generator=self.gen).to(torch.int32)
        self.c.table.copy_(perm.view_as(self.c.table))
        for x in (self.c.k_codes, self.c.v_codes):              # NaN codes (e4m3 0x7f) where nothing was written
            x.view(torch.uint8).fill_(0x7F)
        for x in (self.c.k_scale, self.c.v_scale, self.c.bound_scale, self.c.acc):
            x.fill_(float("nan"))
        self.units = [O8.Unit(D, block, KIND[codes]) for _ in range(B * Hkv)]

    def rand(self, *shape, outlier=True):
        x = torch.randn(shape, generator=self.gen)
        if outlier:
            x[..., 3] *= 9
        return x.to(self.c.dtype)

    def append(self, n, n_new=None, colscore=False, k=None, v=None, strided=False):
        B, Hkv = self.B, self.Hkv
        k = self.rand(B, Hkv, n, self.D) if k is None else k
        v = self.rand(B, Hkv, n, self.D, outlier=False) if v is None else v
        cs = torch.rand((B, self.Hq, n), generator=self.gen) if colscore else None
        kd, vd = k.cuda(), v.cuda()
        if strided:                                             # views of one [B, n, heads, D] projection
            both = torch.empty((B, n, 2 * Hkv + 1, self.D), dtype=k.dtype, device="cuda")
            both[:, :, 1:1 + Hkv] = kd.transpose(1, 2)
            both[:, :, 1 + Hkv:] = vd.transpose(1, 2)
            kd, vd = both[:, :, 1:1 + Hkv].transpose(1, 2), both[:, :, 1 + Hkv:].transpose(1, 2)
        nn = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device="cuda")
        self.kvq.block8_append(self.c, kd, vd, n_new=nn, colscore=None if cs is None else cs.cuda())
        for u, unit in enumerate(self.units):
            b, h = divmod(u, Hkv)
            m = n if n_new is None else n_new[b]
            w = None if cs is None else cs[b, h * self.g:(h + 1) * self.g, :m].double().sum(0).numpy()
            unit.append(k[b, h, :m].float().numpy(), v[b, h, :m].float().numpy(), w)

    def check(self, acc_rtol=None):
        c = self.c
        cpu = {k: getattr(c, k).cpu() for k in ("table", "count", "seq_len", "k_scale", "v_scale", "bound_scale",
                                                "k_bound", "block_pos", "acc", "tail_k", "tail_v")}
        codes = {"k": c.k_codes.view(torch.uint8).cpu().numpy(), "v": c.v_codes.view(torch.uint8).cpu().numpy()}
        rows_written = np.zeros(codes["k"].shape[:2], bool)
        for u, unit in enumerate(self.units):
            assert int(cpu["count"][u]) == unit.count and int(cpu["seq_len"][u]) == unit.seq_len
            for i, b in enumerate(unit.blocks):
                at, n = int(cpu["table"][u, i]), len(b.k)
                rows_written[at, :n] = True
                for name in ("k", "v"):
                    want, s = O8.quantise(getattr(b, name), unit.kind)
                    np.testing.assert_array_equal(codes[name][at, :n], want, err_msg=f"unit {u} block {i} {name}")
                    np.testing.assert_array_equal(cpu[name + "_scale"][at].numpy(), s)
                    if n < c.block:
                        np.testing.assert_array_equal(cpu["tail_" + name][u, :n].float().numpy(), getattr(b, name))
                bd, s = O8.bounds(b.k)
                np.testing.assert_array_equal(cpu["k_bound"][at].numpy(), bd)
                np.testing.assert_array_equal(cpu["bound_scale"][at].numpy(), s)
                assert int(cpu["block_pos"][at]) == b.pos
                if acc_rtol is not None:
                    assert abs(float(cpu["acc"][at]) - b.acc) <= acc_rtol * abs(b.acc) + 1e-30, (u, i)
        for name in ("k", "v"):                                 # nothing else was written
            rest = codes[name][~rows_written]
            assert self.evicted or (rest == 0x7F).all()

    evicted = False

    def attn(self, q, n_new=None, blocks=None, accumulate=False, scale=None, qd=None, **kw):
        """Runs block8_attn and compares it; returns (o, lse)."""
        c, B, Hq, n_q = self.c, self.B, self.Hq, q.shape[2]
        scale = scale or self.D ** -0.5
        nn = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device="cuda")
        acc0 = c.acc.double().cpu().numpy().copy()
        o, lse = self.kvq.block8_attn(q.cuda() if qd is None else qd, c, scale, blocks=blocks, accumulate=accumulate,
                                      n_new=nn, **kw)
        got, glse, acc1 = o.double().cpu().numpy(), lse.double().cpu().numpy(), c.acc.double().cpu().numpy()
        if blocks is not None:
            idx, ln = blocks[0].cpu().numpy(), blocks[1].cpu().numpy()
        table = c.table.cpu().numpy()
        for u, unit in enumerate(self.units):
            b, h = divmod(u, self.Hkv)
            m = n_q if n_new is None else n_new[b]
            k, v = unit.dequantised()
            share, share_tol = np.zeros(len(unit.blocks)), np.zeros(len(unit.blocks))
            for t in range(n_q):
                limit = unit.count - m + t + 1 if t < m else 0
                chosen = None if blocks is None else idx[b, h, t, :ln[b, h, t]]
                mask = np.broadcast_to(unit.seen(limit, chosen), (self.g, unit.count))
                qq = q[b, h * self.g:(h + 1) * self.g, t].float().numpy()
                ro, rl, p = O8.attend(qq, k, v, mask, scale)
                n = int(mask[0].sum())
                e = np.where(mask, scale * np.abs(qq.astype(np.float64)) @ np.abs(k).T, 0).max(axis=1, initial=0)
                e = e * (2 * self.D + 8) * U24
                eps = torch.finfo(c.dtype).eps / 2
                tol = (2 * e + 2.0 ** -13 + 4 * n * U24)[:, None] * (p @ np.abs(v)) + eps * np.abs(ro) + 2.0 ** -25
                go, gl = got[b, h * self.g:(h + 1) * self.g, t], glse[b, h * self.g:(h + 1) * self.g, t]
                if n == 0:
                    assert (go == 0).all() and (gl == -np.inf).all(), (u, t)
                    continue
                err = np.abs(go - ro) - tol
                assert np.isfinite(go).all() and (err <= 0).all(), (u, t, float(err.max()))
                assert (np.abs(gl - rl) <= e + 2.0 ** -14 + n * U24 + 2.0 ** -22 * np.abs(rl)).all(), (u, t)
                pb = np.zeros(len(unit.blocks))
                np.add.at(pb, np.arange(unit.count) // unit.P, p.sum(0))
                share += pb
                share_tol += pb * (2 * e.max() + 2.0 ** -13 + 2 * n * U24)
            for i, blk in enumerate(unit.blocks):
                at = table[u, i]
                if not accumulate:
                    assert acc1[at] == acc0[at] or np.isnan(acc0[at])
                    continue
                want = acc0[at] + share[i]
                # one addition of a float32 share to a float32 sum (a few, one per query, for lists)
                assert abs(acc1[at] - want) <= share_tol[i] + (1 + n_q) * U24 * abs(want) + 1e-37, (u, i)
                blk.acc = acc1[at]
        return o, lse


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", [F8, I8])
@pytest.mark.parametrize("D,block", [(128, 16), (64, 16), (128, 32), (64, 64), (128, 64), (64, 128), (128, 128)])
def test_append_any_split(kvq, D, block, codes, dtype):
    p = Pair(kvq, D=D, block=block, codes=codes, dtype=dtype, max_tokens=6 * block, seed=block + D)
    p.append(1)
    p.check()
    p.append(3, n_new=[3, 0], strided=True)             # a padded row: sequence 1 has no new token
    p.append(block - 2, n_new=[block - 4, block - 2])   # sequence 0 fills its block to the last row, 1 stays open
    p.check()
    p.append(2 * block + 3, strided=True, colscore=False)   # across three blocks, open at both ends
    p.check()
    for _ in range(3):
        p.append(1)
    p.append(block, n_new=[block, 1])                   # open block to open block, one CTA
    p.check()


@pytest.mark.parametrize("D,block", [(64, 16), (128, 32), (128, 128)])
def test_append_whole_blocks(kvq, D, block):
    """Calls that end on a block's last row, alone and among others, and a block filled row by row."""
    p = Pair(kvq, D=D, block=block, max_tokens=8 * block)
    p.append(block)
    p.check()
    p.append(block, n_new=[block, 0], colscore=True)
    p.append(2 * block, n_new=[2 * block, block])
    p.check()
    for _ in range(block if block == 16 else 3):
        p.append(1)
    p.check()
    p.append(block, n_new=[block - 3, block - 1] if block > 16 else [block, block])
    p.check()


@pytest.mark.parametrize("block", [16, 128])
def test_append_prompt_with_scores(kvq, block):
    p = Pair(kvq, B=3, Hq=6, Hkv=2, block=block, codes=I8, max_tokens=1000)
    p.append(777, n_new=[777, 5, 640], colscore=True)
    # g * block float32 additions of non-negative numbers
    p.check(acc_rtol=(3 * block + 2) * U24)
    for u in (0, 2, 5):                                 # code x scale, rounded to float32 once
        for got, want in zip(p.c.dequantised(u), p.units[u].dequantised()):
            np.testing.assert_allclose(got.cpu().numpy(), want, rtol=U24, atol=0)
    p.append(100, n_new=[100, 0, 33], colscore=True)
    p.check(acc_rtol=(6 * block + 4) * U24)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", [F8, I8])
def test_append_values_at_the_edges(kvq, codes, dtype):
    p = Pair(kvq, B=1, Hq=1, Hkv=1, D=64, codes=codes, dtype=dtype, max_tokens=128)
    k = torch.zeros((1, 1, 96, 64), dtype=dtype)
    k[0, 0, 16:32] = torch.finfo(dtype).max * torch.linspace(-1, 1, 64).to(dtype)
    k[0, 0, 32:48, ::2] = -0.0
    k[0, 0, 33, 7] = torch.finfo(dtype).smallest_normal / 4             # subnormal in the 16-bit type
    k[0, 0, 48:64] = torch.tensor(2.0 ** -14, dtype=dtype) * torch.arange(64).to(dtype)
    k[0, 0, 64 + 3, 5], k[0, 0, 80 + 9, 6] = float("nan"), float("-inf")
    v = k.flip(2).contiguous()
    p.append(96, k=k, v=v)
    p.check()
    # one token at a time, with scales that grow, stand, and become NaN, gives the same codes
    q = Pair(kvq, B=1, Hq=1, Hkv=1, D=64, codes=codes, dtype=dtype, max_tokens=128)
    for i in range(96):
        q.append(1, k=k[:, :, i:i + 1], v=v[:, :, i:i + 1])
    q.check()


def test_append_leaves_a_unit_alone_that_has_no_room(kvq):
    p = Pair(kvq, B=2, Hq=2, Hkv=2, max_tokens=48)
    p.append(40)
    p.c.table[1, 2] = -1                                # the open block of unit 1: in use, and now lost
    p.c.table[2, 2] = p.c.k_codes.shape[0]              # out of the pool
    p.append(0)
    before = [x.clone() for x in (p.c.count, p.c.seq_len, p.c.k_codes.view(torch.uint8), p.c.tail_k)]
    z = torch.ones((2, 2, 9, 128), dtype=torch.float16, device="cuda")
    kvq.block8_append(p.c, z, z)                        # 49 tokens fit nowhere
    kvq.block8_append(p.c, z, z, n_new=torch.tensor([0, -1], dtype=torch.int32, device="cuda"))
    assert kvq.device_status() == kvq.KVQ_EDEVICE
    for x, y in zip(before, (p.c.count, p.c.seq_len, p.c.k_codes.view(torch.uint8), p.c.tail_k)):
        assert torch.equal(x, y)
    kvq.block8_append(p.c, z[:, :, :3].contiguous(), z[:, :, :3].contiguous())
    assert kvq.device_status() == kvq.KVQ_EDEVICE
    assert p.c.count.tolist() == [43, 40, 40, 43]


def test_reset(kvq):
    p = Pair(kvq)
    p.append(33)
    kvq.block8_reset(p.c, torch.tensor([0, 1, 0, 2], dtype=torch.int32, device="cuda"))
    assert p.c.count.tolist() == [33, 0, 33, 0] and p.c.seq_len.tolist() == [33, 0, 33, 0]
    kvq.block8_reset(p.c)
    assert p.c.count.tolist() == [0] * 4
    p.units = [O8.Unit(128, 16, "e4m3") for _ in range(4)]
    p.evicted = True                                    # old codes lie around
    p.append(21)
    p.check()


# ------------------------------------------------------------------ attention

def _lengths(p, lens):
    """Appends so that sequence b holds lens[b] tokens."""
    if max(lens):
        p.append(max(lens), n_new=list(lens))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", [F8, I8])
@pytest.mark.parametrize("D,block,Hq,Hkv", [(128, 16, 4, 4), (128, 64, 10, 2), (64, 32, 16, 2), (128, 128, 24, 2),
                                            (64, 16, 3, 1), (128, 32, 40, 2), (64, 128, 64, 1)])
def test_attn_lengths(kvq, D, block, Hq, Hkv, codes, dtype):
    lens = [0, 1, 15, 16, 17, 33, 129, 512, 801]
    p = Pair(kvq, B=len(lens), Hq=Hq, Hkv=Hkv, D=D, block=block, codes=codes, dtype=dtype, max_tokens=896, seed=D + Hq)
    _lengths(p, lens)
    p.c.acc.zero_()
    q = p.rand(len(lens), Hq, 1, D)
    a = p.attn(q, accumulate=True)
    b = p.attn(q)                                       # the same call twice gives the same bits
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # a step's shape, without the axis of queries
    o, lse = kvq.block8_attn(q[:, :, 0].cuda(), p.c)
    assert torch.equal(o, a[0][:, :, 0]) and torch.equal(lse, a[1][:, :, 0])


@pytest.mark.parametrize("n_q,Hq,Hkv,D,block,codes", [(2, 4, 4, 128, 16, F8), (3, 10, 2, 128, 64, I8),
                                                      (8, 8, 1, 64, 32, F8), (16, 4, 2, 128, 128, I8),
                                                      (5, 24, 2, 64, 16, F8), (16, 64, 1, 128, 16, I8),
                                                      (9, 3, 1, 128, 32, F8)])
def test_attn_several_queries(kvq, n_q, Hq, Hkv, D, block, codes):
    """Causal among the last tokens; ragged numbers of queries, more queries than tokens, padding rows."""
    lens = [0, 1, 4, 31, 32, 65, 300]
    p = Pair(kvq, B=len(lens), Hq=Hq, Hkv=Hkv, D=D, block=block, codes=codes, dtype=torch.bfloat16, max_tokens=384,
             max_q=16, seed=n_q)
    _lengths(p, lens)
    p.c.acc.zero_()
    q = p.rand(len(lens), Hq, n_q, D)
    p.attn(q, accumulate=True)
    p.attn(q, n_new=[1, 0, n_q, n_q - 1, 2, n_q, 1], accumulate=True)
    # a strided query: a view of [B, n_q, heads, D]
    qd = q.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    assert not qd.is_contiguous() or n_q == 1
    p.attn(q, qd=qd)


@pytest.mark.parametrize("D,block,Hq,Hkv,n_q,codes,dtype", [
    (128, 16, 4, 4, 1, F8, torch.float16), (64, 64, 10, 2, 1, I8, torch.bfloat16), (128, 128, 12, 1, 1, F8, torch.bfloat16),
    (64, 16, 3, 1, 3, F8, torch.float16), (128, 32, 8, 1, 4, I8, torch.float16), (128, 16, 40, 1, 2, F8, torch.bfloat16)])
def test_attn_small_caches(kvq, D, block, Hq, Hkv, n_q, codes, dtype):
    """Room for 256 tokens a unit: one CTA per work unit writes the output itself."""
    lens = [0, 1, 15, 16, 17, 100, 255, 256]
    p = Pair(kvq, B=len(lens), Hq=Hq, Hkv=Hkv, D=D, block=block, codes=codes, dtype=dtype, max_tokens=256, max_q=4, seed=Hq)
    _lengths(p, lens)
    q = p.rand(len(lens), Hq, n_q, D)
    p.attn(q)
    n_new = [n_q, 1, 0, n_q, 1, n_q - 1, 1, n_q]
    qn = q.clone()
    for b, m in enumerate(n_new):
        qn[b, :, m:] = float("nan")
    p.attn(q, n_new=n_new, qd=qn.cuda())
    idx, n = kvq.block8_select(q.cuda(), p.c, max(2, 128 // block))
    p.attn(q, blocks=(idx, n))
    p.attn(q, blocks=(idx, torch.zeros_like(n)))


@pytest.mark.parametrize("room", [512, 544])
def test_attn_many_small_units(kvq, room):
    """320 units with room just at, and just above, what one CTA each takes; most hold little."""
    lens = [int(x) for x in np.random.default_rng(room).integers(0, 40, 160)]
    lens[7], lens[100] = room, 300
    p = Pair(kvq, B=160, Hq=2, Hkv=2, D=64, block=32, codes=I8, max_tokens=room)
    _lengths(p, lens)
    p.attn(p.rand(160, 2, 1, 64))
    p.c.acc.zero_()
    p.attn(p.rand(160, 2, 1, 64), accumulate=True)


@pytest.mark.parametrize("Hq,n_q", [(2, 4), (4, 3), (12, 3)])
def test_padding_rows_may_hold_anything(kvq, Hq, n_q):
    """Rows t >= n_new[b] of q, k and v are not looked at: NaN and infinities there change nothing."""
    p = Pair(kvq, B=4, Hq=Hq, Hkv=1, D=64, block=32, max_tokens=128, max_q=n_q)
    n_new = [1, n_q, 0, n_q - 1]
    _lengths(p, [70, 33, 64, 100])
    k, v, q = (p.rand(4, h, n_q, 64) for h in (1, 1, Hq))
    for b, m in enumerate(n_new):
        k[b, :, m:], v[b, :, m:], q[b, :, m:] = float("nan"), float("inf"), float("nan")
    p.append(n_q, n_new=n_new, k=k, v=v)
    p.check()
    p.c.acc.zero_()
    clean = torch.nan_to_num(q, 0.0)
    for blocks in (None, kvq.block8_select(q.cuda(), p.c, 3, n_new=torch.tensor(n_new, dtype=torch.int32, device="cuda"))):
        p.attn(clean, n_new=n_new, blocks=blocks, accumulate=True, qd=q.cuda())
        assert torch.isfinite(p.c.acc).all()
    if blocks is not None:
        _check_select(p, clean, 3, 1, 1, n_new=n_new)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attn_extreme_logits_and_scales(kvq, dtype):
    """Logits far above and below the usual, blocks whose value scales differ by many powers of two."""
    p = Pair(kvq, B=4, Hq=4, Hkv=1, D=64, block=16, dtype=dtype, max_tokens=512)
    k, v = p.rand(4, 1, 500, 64), p.rand(4, 1, 500, 64)
    k[0] *= 40                                          # one token wins, others underflow
    k[1] = 0                                            # all equal
    v[2, :, :256] *= 2.0 ** -12                         # later blocks dwarf the first ones
    v[2, :, 256:] *= 2.0 ** 8
    k[3, 0, 100] *= 30                                  # the largest logits in the middle
    v[3, 0, 100] *= 2.0 ** -10
    p.append(500, k=k, v=v)
    p.c.acc.zero_()
    p.attn(p.rand(4, 4, 1, 64), accumulate=True)
    q = p.rand(4, 4, 1, 64) * 200
    p.attn(q, accumulate=True)
    p.attn(torch.zeros_like(q))


@pytest.mark.parametrize("D,block,Hq,n_q,codes,room", [(64, 16, 1, 1, F8, 256), (128, 32, 4, 1, I8, 256), (64, 16, 12, 1, I8, 256),
                                                       (128, 16, 4, 1, F8, 2048), (64, 32, 6, 2, I8, 2048), (128, 64, 8, 4, F8, 2048)])
def test_attn_value_scales_over_all_of_bf16(kvq, D, block, Hq, n_q, codes, room):
    """Value scales from 2^-64 (a block of zeros) to 2^120: blocks of small values keep their part of the softmax, in
    the outputs, lse and acc; one kernel for a unit (room 256, no acc) and the joined partials of many."""
    n = min(room, 1400) - 7
    p = Pair(kvq, B=6, Hq=Hq, Hkv=1, D=D, block=block, codes=codes, dtype=torch.bfloat16, max_tokens=room, max_q=4, seed=D + Hq)
    k, v = p.rand(6, 1, n, D), torch.rand((6, 1, n, D), generator=p.gen) + 0.5
    v = v * torch.where(torch.rand(v.shape, generator=p.gen) < 0.5, -1.0, 1.0)
    power = torch.full((6, n), -math.inf)               # log2 of the values' size; -inf: zeros
    at = torch.arange(n) // block
    power[0, at == 3] = 80.0                            # equal logits, one block far above many of zeros
    power[1, at < 2] = 126.0                            # the large ones first
    power[2, at == int(at[-1]) - 1] = 126.0             # and last
    power[2, at == 0] = 0.0
    power[3] = torch.tensor([-100.0, -20.0, 0.0, 45.0, 126.0, -math.inf])[torch.randint(0, 6, (int(at[-1]) + 1,), generator=p.gen)[at]]
    power[4] = 0.0                                      # large values only where the softmax has next to nothing
    power[4, at == 1] = 100.0
    power[5] = 126.0                                    # and everywhere
    k[:3], k[4, 0, at == 1] = 0, k[4, 0, at == 1] * 0 + 8
    p.append(n, k=k, v=(v * torch.exp2(power)[:, None, :, None]).to(torch.bfloat16))
    q = p.rand(6, Hq, n_q, D)
    q[4] = -q[4].abs()
    p.c.acc.zero_()
    p.attn(q)
    p.attn(q, accumulate=True)
    held = int(at[-1]) + 1
    idx = torch.arange(held - 1, -1, -1, dtype=torch.int32, device="cuda").expand(6, 1, n_q, held).contiguous()
    p.attn(q, blocks=(idx, torch.full((6, 1, n_q), held, dtype=torch.int32, device="cuda")), accumulate=True)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Hq,D,codes,n,room", [(1, 64, I8, 250, 256), (8, 128, F8, 250, 256), (12, 128, I8, 250, 256), (32, 64, F8, 250, 256),
                                               (4, 128, I8, 2000, 2048), (16, 64, F8, 2000, 2048), (32, 128, I8, 2000, 2048)])
def test_attn_weights_have_22_bits(kvq, Hq, D, codes, n, room, dtype):
    """Two kinds of tokens, logit L with value 1 and logit 0 with value -1, in numbers that nearly cancel: the output is
    small, so that its own rounding hides nothing, and an error of the weights shows beside sum p |v| = 1.

    Only one channel of q and k is not 0, so a logit's products and their sum are exact.  It takes three float32 factors
    (each within u of |s| < 2) and two additions of numbers below 16 (each within 2^-21): 2^-19.9 in the exponent, ln 2 of
    that in the weight, 2^-22 of exp2, 2^-22 of the fp16 pair: the ratio of the two weights is within 2^-19, the output
    moves by half of it.  The sums: at most 32 additions of a warp (2000 tokens in 125 cells, 2 products each, spread
    over 8 warps at least, 250 in 16 cells over 4), cut instead of rounded: 2^-23 each of at most 1, 2^-18.  So 2^-17.
    With weights of fp16 alone the ratio would be off by 2^-12.6 at least, as the test asserts of its numbers."""
    n_a = n * 3 // 10
    sigma = D ** -0.5
    best = None
    for x in torch.arange(2.0, 16.0, 1 / 32).to(dtype).unique().tolist():       # q's only channel
        r = math.exp(-sigma * x)                        # weight of the second kind to the first's
        off = abs(float(np.float16(128 * r)) / (128 * r) - 1)
        o = (n_a - (n - n_a) * r) / (n_a + (n - n_a) * r)
        if off > 2.0 ** -12.6 and (best is None or abs(o) < abs(best[1])):
            best = x, o, off
    x, o, off = best
    assert abs(o) < 2.0 ** -5 and off / 2 > 4 * 2.0 ** -17
    p = Pair(kvq, B=1, Hq=Hq, Hkv=1, D=D, block=16, codes=codes, dtype=dtype, max_tokens=room)
    first = torch.zeros(n, dtype=torch.bool)
    first[torch.randperm(n, generator=p.gen)[:n_a]] = True
    k, v = torch.zeros((1, 1, n, D), dtype=dtype), torch.ones((1, 1, n, D), dtype=dtype)
    k[0, 0, first, 5] = 1.0
    v[0, 0, ~first] = -1.0
    p.append(n, k=k, v=v)
    q = torch.zeros((1, Hq, 1, D), dtype=dtype)
    q[..., 5] = x
    p.c.acc.zero_()
    kd, vd = p.units[0].dequantised()
    ro, rl, w = O8.attend(q[0, :, 0].float().numpy(), kd, vd, np.ones((Hq, n), bool), sigma)
    for accumulate in (False, True):
        got, lse = kvq.block8_attn(q.cuda(), p.c, accumulate=accumulate)
        err = np.abs(got[0, :, 0].double().cpu().numpy() - ro)
        assert (err <= 2.0 ** -17 + torch.finfo(dtype).eps / 2 * np.abs(ro)).all(), float(err.max())
        # the exponent's error, 32 additions (u each), log2 of a sum below 2^18 and its addition to the reference (2^-20 each)
        assert np.abs(lse[0, :, 0].double().cpu().numpy() - rl).max() <= 2.0 ** -17
    # acc: log2 of a cell's weights and of the sum, each added to a reference (numbers below 32: 2^-20 a rounding, ln 2 of
    # which counts), the sum's 32 additions and those of up to 32 heads (u each): 2^-17.3
    acc = p.c.acc[p.c.table[0].long()].double().cpu().numpy()
    want = np.zeros(-(-n // 16))
    np.add.at(want, np.arange(n) // 16, w.sum(0))
    assert (np.abs(acc[:len(want)] - want) <= 2.0 ** -17 * want).all()


def test_attn_lists(kvq):
    B, Hq, Hkv, n_q, n_sel = 3, 6, 2, 2, 7
    for codes, block in ((F8, 16), (I8, 32), (F8, 128)):
        p = Pair(kvq, B=B, Hq=Hq, Hkv=Hkv, block=block, codes=codes, max_tokens=20 * block, max_q=2)
        lens = [20 * block, 7 * block + 5, 3]
        _lengths(p, lens)
        p.c.acc.zero_()
        idx = torch.full((B, Hkv, n_q, n_sel), -1, dtype=torch.int32)
        n = torch.zeros((B, Hkv, n_q), dtype=torch.int32)
        for b in range(B):
            held = -(-lens[b] // block)
            for h in range(Hkv):
                for t in range(n_q):
                    m = int(p.rng.integers(0, min(n_sel, held) + 1)) if (b, h, t) != (0, 0, 0) else 0   # an empty list
                    pick = p.rng.permutation(held)[:m]              # any order
                    if m > 1 and held - 1 not in pick:
                        pick[0] = held - 1                          # the partly filled block among them
                    idx[b, h, t, :m], n[b, h, t] = torch.from_numpy(pick.astype(np.int32)), m
        blocks = (idx.cuda(), n.cuda())
        q = p.rand(B, Hq, n_q, 128)
        p.attn(q, blocks=blocks, accumulate=True)
        p.attn(q, blocks=blocks, n_new=[2, 1, 0])


def test_attn_list_numbers_that_are_not_there(kvq):
    p = Pair(kvq, B=1, Hq=2, Hkv=1, D=64, max_tokens=160, max_q=1)
    p.append(100)
    q = p.rand(1, 2, 1, 64)
    good = torch.tensor([[[[1, 3]]]], dtype=torch.int32, device="cuda"), torch.tensor([[[2]]], dtype=torch.int32, device="cuda")
    want = p.attn(q, blocks=good)
    bad = torch.tensor([[[[1, 7, -5, 3, 1 << 30]]]], dtype=torch.int32, device="cuda")
    got = kvq.block8_attn(q.cuda(), p.c, blocks=(bad, torch.tensor([[[9]]], dtype=torch.int32, device="cuda")))
    assert kvq.device_status() == kvq.KVQ_EDEVICE
    assert torch.equal(got[0], want[0])
    p.c.table[0, 2] = -1                                # a lost block is skipped, and told of
    kvq.block8_attn(q.cuda(), p.c, accumulate=True)
    assert kvq.device_status() == kvq.KVQ_EDEVICE


def test_attn_not_a_number(kvq):
    """A block that holds a NaN makes NaN of the queries that see it, and of no others."""
    p = Pair(kvq, B=3, Hq=2, Hkv=1, D=64, max_tokens=64, max_q=2)
    k, v = p.rand(3, 1, 33, 64), p.rand(3, 1, 33, 64)
    k[0, 0, 20, 1] = float("nan")                       # block 1
    v[1, 0, 32, 1] = float("inf")                       # block 2: only the last query sees it
    p.append(33, k=k, v=v)
    q = p.rand(3, 2, 2, 64).cuda()
    o, lse = kvq.block8_attn(q, p.c)
    assert o[0].isnan().all() and lse[0].isnan().all()
    assert o[1, :, 1].isnan().all() and not o[1, :, 0].isnan().any() and not o[2].isnan().any()
    blocks = (torch.tensor([0, 2], dtype=torch.int32, device="cuda").expand(3, 1, 2, 2).contiguous(),
              torch.full((3, 1, 2), 2, dtype=torch.int32, device="cuda"))
    o, _ = kvq.block8_attn(q, p.c, blocks=blocks)
    assert not o[0].isnan().any()                       # block 1 is not listed
    qn = q.clone()
    qn[2, 1, 0, 3] = float("nan")
    o, _ = kvq.block8_attn(qn, p.c)
    assert o[2, 1, 0].isnan().all() and not o[2, 0].isnan().any() and not o[2, 1, 1].isnan().any()


@pytest.mark.parametrize("Hq,n_q,dtype", [(8, 1, torch.float16), (16, 1, torch.bfloat16), (5, 8, torch.bfloat16)])
def test_attn_one_long_unit(kvq, Hq, n_q, dtype):
    """One unit's tokens spread over every CTA: many partials a row."""
    p = Pair(kvq, B=1, Hq=Hq, Hkv=1, block=64, codes=F8, dtype=dtype, max_tokens=30000, max_q=8)
    p.append(29991)
    p.c.acc.zero_()
    p.attn(p.rand(1, Hq, n_q, 128), accumulate=True)
    idx, n = kvq.block8_select(p.rand(1, Hq, n_q, 128).cuda(), p.c, 300)
    p.attn(p.rand(1, Hq, n_q, 128), blocks=(idx, n), accumulate=True)


def test_empty_cache(kvq):
    p = Pair(kvq, B=3, Hq=4, Hkv=2, max_q=2)
    p.c.acc.zero_()
    q = p.rand(3, 4, 2, 128)
    p.attn(q, accumulate=True)
    idx, n = kvq.block8_select(q.cuda(), p.c, 3)
    assert (idx == -1).all() and (n == 0).all()
    p.attn(q, blocks=(idx, n), accumulate=True)
    assert kvq.block8_evict(p.c, torch.zeros(6, dtype=torch.int32, device="cuda")).tolist() == [0] * 6
    p.append(1, n_new=[0, 0, 0])
    p.check()


def test_counters_out_of_range_are_refused_or_read_as_empty(kvq):
    """Counters that no call writes: nothing outside the cache is touched."""
    p = Pair(kvq, B=2, Hq=2, Hkv=1, max_tokens=64)
    p.append(40)
    p.c.acc.zero_()
    p.c.count.copy_(torch.tensor([-5, 1 << 30], dtype=torch.int32))
    z = torch.ones((2, 1, 1, 128), dtype=torch.float16, device="cuda")
    kvq.block8_append(p.c, z, z)
    assert kvq.device_status() == kvq.KVQ_EDEVICE and p.c.count.tolist() == [-5, 1 << 30]
    q = p.rand(2, 2, 1, 128).cuda()
    p.c.v_codes.view(torch.uint8).zero_()               # the 24 rows behind the 40 tokens are read as well here
    p.c.k_codes.view(torch.uint8).zero_()
    p.c.k_scale.fill_(1.0)
    p.c.v_scale.fill_(1.0)
    p.c.bound_scale.fill_(1.0)
    o, lse = kvq.block8_attn(q, p.c, accumulate=True)
    assert (lse[0] == -np.inf).all() and (o[0] == 0).all()
    assert torch.allclose(lse[1], torch.full_like(lse[1], float(np.log(64))), atol=1e-4)
    idx, n = kvq.block8_select(q, p.c, 2)
    assert n.flatten().tolist() == [0, 2]
    kvq.block8_evict(p.c, torch.full((2,), 2, dtype=torch.int32, device="cuda"))
    assert kvq.device_status() == 0


def test_attn_pool_beyond_32_bits(kvq):
    """Blocks whose byte offsets pass 2^32 in pools of keys and values."""
    n = (1 << 32) // (128 * 128) + 64
    p = Pair(kvq, B=1, Hq=2, Hkv=1, block=128, max_tokens=n * 128)
    p.c.table.copy_(torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda").view(1, n))
    p.append(333)
    q = p.rand(1, 2, 1, 128)
    p.c.acc.zero_()
    p.attn(q, accumulate=True)
    idx, m = kvq.block8_select(q.cuda(), p.c, 2)
    p.attn(q, blocks=(idx, m))


class StoredUnit(O8.Unit):
    """A unit known by its codes and scales."""

    def __init__(self, D, block, kind, n, k, v):
        super().__init__(D, block, kind)
        self.n, self.rows, self.seq_len, self.blocks = n, [k, v], n, [O8.Block(0, D) for _ in range(-(-n // block))]

    count = property(lambda self: self.n)

    def dequantised(self):
        return self.rows


class Stored(Pair):
    """A cache of lens[u] tokens whose codes, scales and bounds are random: many units without appending to each."""

    def __init__(self, kvq, lens, Hq, Hkv, D, block, codes, dtype, max_tokens, seed=0, values=True, v_power=None, **kw):
        B, dev = len(lens) // Hkv, "cuda"
        self.kvq, self.B, self.Hq, self.Hkv, self.D, self.g = kvq, B, Hq, Hkv, D, Hq // Hkv
        self.rng, self.gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.c = c = kvq.make_block8_cache(B, Hq, Hkv, D, dtype, max_tokens, block=block, codes=codes, **kw)
        gen, n = torch.Generator(dev).manual_seed(seed), c.table.numel()
        c.table.copy_(torch.randperm(n, generator=gen, device=dev).to(torch.int32).view_as(c.table))
        c.count.copy_(torch.tensor(lens, dtype=torch.int32))
        c.seq_len.copy_(c.count)
        for x in (c.k_codes, c.v_codes):
            if values:
                y = torch.randn(x.shape, generator=gen, device=dev) * 40
                x.view(torch.uint8).copy_((y.to(F8) if codes == F8 else y.round().clamp(-127, 127).to(I8)).view(torch.uint8))
        for x in (c.k_scale, c.v_scale, c.bound_scale):
            x.copy_(0.02 * torch.exp(0.3 * torch.randn(n, generator=gen, device=dev)))
        if v_power is not None:                         # log2 of the value scales [unit, logical block]
            c.v_scale[c.table.long()] = torch.exp2(v_power).cuda()
        c.k_bound.copy_(torch.randint(-127, 128, c.k_bound.shape, generator=gen, device=dev).sort(dim=1).values.to(I8))
        table, cpu = c.table.cpu(), {}
        for name in ("k", "v"):
            cpu[name] = getattr(c, name + "_codes").view(torch.uint8).cpu().numpy(), getattr(c, name + "_scale").double().cpu().numpy()
        self.units = []
        for u, m in enumerate(lens):
            ids = table[u, :-(-m // block)].numpy()
            rows = [(O8.decode(x[ids], KIND[codes]) * s[ids, None, None]).reshape(-1, D)[:m] if values else None
                    for x, s in cpu.values()]
            self.units.append(StoredUnit(D, block, KIND[codes], m, *rows))


def _stale(p, n_q, n_sel=0):
    """NaN where the workspace holds partial outputs, and cells' weights with accumulate."""
    c, g = p.c, p.g
    rows, sets = (g, p.B * p.Hkv * n_q) if n_sel else (g * n_q, p.B * p.Hkv)
    r = 8 if rows <= 8 else 16 if rows <= 16 else 32
    works = sets * -(-rows // r)
    at = -c.ws.data_ptr() % 256
    mass = works * (min(n_sel, c.table.shape[1]) or c.table.shape[1]) * (c.block // 16) * r * 4
    total = p.kvq.lib().block8_attn_workspace_bytes(c._ref, n_q, n_sel, 1)
    c.ws[at:at + (1024 + works) * r * p.D * 4] = 0xFF
    c.ws[at + total - (mass + 255) // 256 * 256:at + total] = 0xFF


# (sequences, most tokens, heads, KV heads, queries, D, block, codes, dtype): more runs of tiles than CTAs fit the GPU, so that
# CTAs come to several units, and units' first tiles stand behind 1 to 8 places without work
MANY = [(150, 700, 16, 4, 1, 128, 32, F8, torch.bfloat16), (300, 3500, 2, 1, 1, 64, 64, I8, torch.float16),
        (150, 700, 5, 5, 1, 128, 16, I8, torch.bfloat16), (200, 900, 24, 2, 1, 64, 128, F8, torch.float16),
        (160, 600, 16, 2, 4, 128, 16, I8, torch.bfloat16), (170, 700, 40, 1, 1, 64, 32, F8, torch.bfloat16)]


@pytest.mark.parametrize("B,most,Hq,Hkv,n_q,D,block,codes,dtype", MANY)
def test_attn_runs_over_many_units(kvq, B, most, Hq, Hkv, n_q, D, block, codes, dtype):
    lens = np.random.default_rng(most).integers(0, most + 1, B * Hkv)
    lens[::7], lens[3::50], lens[-4:] = 0, 1, (0, 0, most, 0)
    p = Stored(kvq, [int(x) for x in lens], Hq, Hkv, D, block, codes, dtype, most, seed=B, max_q=n_q)
    q = p.rand(B, Hq, n_q, D, outlier=False)
    p.c.acc.zero_()
    _stale(p, n_q)
    a = p.attn(q, accumulate=True)
    _stale(p, n_q)
    b = p.attn(q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    n_new = [int(x) for x in np.random.default_rng(B).integers(0, n_q + 1, B)]
    p.attn(q, n_new=n_new, accumulate=True)


@pytest.mark.parametrize("Hq,Hkv,n_q,D,block,codes,dtype", [(8, 2, 2, 64, 32, F8, torch.bfloat16), (12, 1, 1, 128, 64, I8, torch.float16),
                                                            (20, 1, 3, 64, 16, F8, torch.float16)])
def test_attn_lists_over_many_units(kvq, Hq, Hkv, n_q, D, block, codes, dtype):
    B, n_sel = 320 // Hkv, {16: 40, 32: 24, 64: 12}[block]
    lens = [int(x) for x in np.random.default_rng(D).integers(0, 40 * block, B * Hkv)]
    lens[5] = lens[-1] = 0
    p = Stored(kvq, lens, Hq, Hkv, D, block, codes, dtype, 40 * block, seed=Hq, max_q=n_q, max_sel=n_sel)
    idx, n = np.full((B * Hkv, n_q, n_sel), -1, np.int32), np.zeros((B * Hkv, n_q), np.int32)
    for u, m in enumerate(lens):
        for t in range(n_q):
            held = -(-m // block)
            n[u, t] = int(p.rng.integers(0, min(n_sel, held) + 1)) if u % 9 else 0      # every ninth unit's lists are empty
            idx[u, t, :n[u, t]] = p.rng.permutation(held)[:n[u, t]]
    blocks = (torch.from_numpy(idx.reshape(B, Hkv, n_q, n_sel)).cuda(), torch.from_numpy(n.reshape(B, Hkv, n_q)).cuda())
    q = p.rand(B, Hq, n_q, D, outlier=False)
    p.c.acc.zero_()
    _stale(p, n_q, n_sel)
    a = p.attn(q, blocks=blocks, accumulate=True)
    _stale(p, n_q, n_sel)
    b = p.attn(q, blocks=blocks)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("Hq,Hkv,D,codes", [(8, 2, 128, F8), (12, 1, 64, I8), (32, 1, 128, I8)])
def test_attn_runs_over_many_units_of_far_apart_value_scales(kvq, Hq, Hkv, D, codes):
    """CTAs come from units whose value scales span 2^170 to units whose scales do not, and back."""
    B = 480 // Hkv
    lens = [int(x) for x in np.random.default_rng(D).integers(0, 1001, B * Hkv)]
    gen = torch.Generator().manual_seed(D)
    power = torch.tensor([-64.0, -30.0, 0.0, 40.0, 100.0, 105.0])[torch.randint(0, 6, (B * Hkv, 32), generator=gen)]
    power[::3] = 0.0                                    # every third unit as usual
    p = Stored(kvq, lens, Hq, Hkv, D, 32, codes, torch.bfloat16, 1000, seed=Hq, v_power=power)
    p.c.acc.zero_()
    _stale(p, 1)
    x = p.rand(B, Hq, 1, D, outlier=False)
    a = p.attn(x, accumulate=True)
    b = p.attn(x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ selection

def _check_select(p, q, n_sel, n_first, n_last, n_new=None):
    nn = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device="cuda")
    idx, n = p.kvq.block8_select(q.cuda(), p.c, n_sel, n_first, n_last, n_new=nn)
    gi, gn = idx.cpu().numpy(), n.cpu().numpy()
    for u, unit in enumerate(p.units):
        b, h = divmod(u, p.Hkv)
        for t in range(q.shape[2]):
            m = q.shape[2] if n_new is None else n_new[b]
            limit = max(0, unit.count - m + t + 1) if t < m else 0
            seen = unit.blocks[:-(-limit // unit.P)]
            want = O8.choose(O8.block_scores(q[b, h * p.g:(h + 1) * p.g, t].float().numpy(), seen), n_sel, n_first, n_last)
            assert gn[b, h, t] == len(want)
            assert gi[b, h, t].tolist() == want + [-1] * (n_sel - len(want)), (u, t)
    return idx, n


@pytest.mark.parametrize("Hq,Hkv,D,block,codes,dtype", [(4, 2, 128, 16, F8, torch.float16), (12, 1, 64, 16, I8, torch.bfloat16),
                                                        (2, 2, 64, 32, I8, torch.float16), (40, 2, 128, 16, F8, torch.bfloat16)])
def test_select(kvq, Hq, Hkv, D, block, codes, dtype):
    lens = [0, 1, block, 5 * block + 3, 60 * block - 1]
    p = Pair(kvq, B=5, Hq=Hq, Hkv=Hkv, D=D, block=block, codes=codes, dtype=dtype, max_tokens=60 * block, max_q=3, seed=Hq)
    _lengths(p, lens)
    for n_sel, a, b in ((1, 0, 0), (1, 1, 0), (4, 1, 1), (6, 0, 6), (17, 3, 2), (64, 1, 1)):
        _check_select(p, p.rand(5, Hq, 3, D), n_sel, a, b)
    _check_select(p, p.rand(5, Hq, 3, D), 5, 1, 1, n_new=[3, 1, 0, 2, 3])
    _check_select(p, torch.zeros((5, Hq, 1, D), dtype=dtype), 7, 1, 2)          # every score ties


def test_select_many_blocks_ties_and_not_a_number(kvq):
    p = Pair(kvq, B=1, Hq=2, Hkv=2, D=64, block=16, max_tokens=16 * 2500)
    k = p.rand(1, 2, 16 * 2500, 64)
    k[:, :, 16 * 100:] = k[:, :, :16 * 2400]            # the scores repeat
    k[0, 1, 16 * 1234 + 5, 9] = float("inf")
    p.append(16 * 2500, k=k, v=k)
    q = p.rand(1, 2, 1, 64)
    for n_sel in (2, 33, 1100, 2499):
        idx, _ = _check_select(p, q, n_sel, 0, 1)
        assert 1234 in idx[0, 1, 0].tolist()
    q[0, 0, 0, 0] = float("nan")
    _check_select(p, q, 33, 1, 1)


def test_lists_longer_than_the_table(kvq):
    """n_sel above the units' number of blocks: what select returns is taken back by attn, with accumulate too."""
    p = Pair(kvq, B=2, Hq=8, Hkv=2, max_tokens=16 * 32)
    p.append(16 * 32 - 3)
    p.c.acc.zero_()
    q = p.rand(2, 8, 1, 128)
    blocks = _check_select(p, q, 64, 1, 1)
    a = p.attn(q, blocks=blocks, accumulate=True)
    b = p.attn(q, blocks=blocks)
    assert torch.equal(a[0], b[0])
    # more entries than blocks exist: the first ones count, and the call is told of
    p.attn(q, blocks=(blocks[0], torch.full_like(blocks[1], 32)))
    got = kvq.block8_attn(q.cuda(), p.c, blocks=(blocks[0], torch.full_like(blocks[1], 33)))
    assert kvq.device_status() == kvq.KVQ_EDEVICE
    assert torch.equal(got[0], b[0])


def _scores(p, q, u, t, nb):
    """float32 scores of unit u's first nb blocks for query t, from the bounds that the cache holds."""
    if not hasattr(p, "bounds"):
        p.bounds = p.c.k_bound.cpu().numpy().astype(np.int64), p.c.bound_scale.cpu().numpy(), p.c.table.cpu().numpy()
    kb, sb, table = p.bounds
    b, h = divmod(u, p.Hkv)
    x = q[b, h * p.g:(h + 1) * p.g, t].float().numpy()
    ids, best = table[u, :nb], None
    for row in x:
        s = O8.scale_of(row, 127.0)
        q8 = np.clip(np.rint(row * (np.float32(1.0) / s)), -127, 127).astype(np.int64)
        y = (kb[ids, 0] @ np.minimum(q8, 0) + kb[ids, 1] @ np.maximum(q8, 0)).astype(np.float32) * s
        best = y if best is None else np.maximum(best, y)
    return best * sb[ids]


def _choose(score, n_sel, n_first, n_last):
    """O8.choose for many blocks without NaN."""
    n = len(score)
    if n <= n_sel:
        return np.arange(n)
    order = np.argsort(-score[n_first:n - n_last], kind="stable")[:n_sel - n_first - n_last] + n_first
    return np.sort(np.concatenate([np.arange(n_first), order, np.arange(n - n_last, n)]))


def _check_stored_select(p, q, n_sel, n_first, n_last):
    n_q = q.shape[2]
    p.c.ws.fill_(0xFF)                                  # NaN scores would be chosen first
    idx, n = p.kvq.block8_select(q.cuda(), p.c, n_sel, n_first, n_last)
    gi, gn = idx.cpu().numpy(), n.cpu().numpy()
    for u, unit in enumerate(p.units):
        b, h = divmod(u, p.Hkv)
        for t in range(n_q):
            nb = -(-max(0, unit.count - n_q + t + 1) // unit.P)
            want = _choose(_scores(p, q, u, t, nb), n_sel, n_first, n_last) if nb else np.zeros(0, int)
            assert gn[b, h, t] == len(want), (u, t)
            assert np.array_equal(gi[b, h, t, :len(want)], want) and (gi[b, h, t, len(want):] == -1).all(), (u, t)


@pytest.mark.parametrize("B,Hq,Hkv,n_q,D,dtype", [(250, 24, 2, 2, 64, torch.float16), (600, 2, 2, 1, 128, torch.bfloat16)])
def test_select_runs_over_many_units(kvq, B, Hq, Hkv, n_q, D, dtype):
    """More runs of 64 blocks than CTAs fit the GPU: CTAs come to several queries, runs end inside one.  Units that are
    empty or hold no more than n_sel blocks between the others."""
    lens = np.random.default_rng(B).integers(0, 16 * 200 + 1, B * Hkv)
    lens[::6], lens[4::31], lens[-3:] = 0, 16 * 8, (0, 3200, 0)
    p = Stored(kvq, [int(x) for x in lens], Hq, Hkv, D, 16, I8, dtype, 3200, seed=D, values=False, max_q=n_q)
    q = p.rand(B, Hq, n_q, D, outlier=False)
    _check_stored_select(p, q, 8, 1, 1)
    _check_stored_select(p, q, 100, 0, 3)


def test_select_more_blocks_than_the_registers_hold(kvq):
    """Above 8192 blocks the top-k reads the scores again in every pass."""
    p = Stored(kvq, [16 * 9000 - 5, 16 * 8500, 0, 16 * 300], 4, 2, 64, 16, I8, torch.float16, 16 * 9000, values=False)
    p.c.k_bound.copy_(p.c.k_bound // 64)                # many scores are equal
    p.c.bound_scale.fill_(0.25)
    q = p.rand(2, 4, 1, 64)
    for n_sel, a, b in ((500, 1, 1), (1, 0, 0), (8999, 2, 3), (4000, 0, 4000), (8400, 0, 1)):
        _check_stored_select(p, q, n_sel, a, b)


# ------------------------------------------------------------------ eviction

def test_evict(kvq):
    p = Pair(kvq, B=4, Hq=2, Hkv=2, D=64, max_tokens=16 * 40 + 4 * 21)
    p.evicted = True
    _lengths(p, [16 * 40, 16 * 9 + 1, 16 * 8, 0])
    for rnd in range(4):
        acc = torch.randn(p.c.acc.shape, generator=p.gen).abs()
        acc[::3] = 0.5                                  # ties
        if rnd == 2:
            acc[::7] = float("nan")
        p.c.acc.copy_(acc)
        table = p.c.table.cpu().numpy()
        for u, unit in enumerate(p.units):
            for i, b in enumerate(unit.blocks):
                b.acc = float(acc[table[u, i]])
        keep, a, b = [([30, 40, 9, 3, 8, 8, 0, 5], 1, 1), ([20, 1, 0, 0, 2, 7, 1, 1], 2, 3),
                      ([11, 12, -4, 3, 1, 5, 0, 0], 0, 1), ([5] * 8, 1, 1)][rnd]
        want = [unit.evict(x, a, b) for unit, x in zip(p.units, keep)]
        gone = kvq.block8_evict(p.c, torch.tensor(keep, dtype=torch.int32, device="cuda"), a, b)
        assert gone.tolist() == want
        now = p.c.table.cpu().numpy()
        for u, unit in enumerate(p.units):              # those that left follow the kept ones, in order; then the free
            old = table[u].tolist()
            held = len(unit.blocks)
            left = [x for x in old[:held + want[u]] if x not in now[u, :held].tolist()]
            assert now[u, held:].tolist() == left + old[held + want[u]:], (rnd, u)
        p.check()
        if rnd != 2:
            p.c.acc.nan_to_num_(0.5)
            p.attn(p.rand(4, 2, 1, 64))
        p.append(21, n_new=[21, 3, 16, 0])
        p.check()


def test_evict_many_blocks(kvq):
    p = Pair(kvq, B=2, Hq=1, Hkv=1, D=64, max_tokens=16 * 5000)
    p.evicted = True
    p.c.count.copy_(torch.tensor([16 * 5000 - 3, 16 * 1025], dtype=torch.int32))
    acc = torch.rand(p.c.acc.shape, generator=p.gen).round(decimals=3)
    p.c.acc.copy_(acc)
    table = p.c.table.cpu()
    want = [O8.choose(acc[table[u, :n].long()].tolist(), 1024, 4, 1024 - 200) for u, n in ((0, 5000), (1, 1025))]
    gone = kvq.block8_evict(p.c, torch.full((2,), 1024, dtype=torch.int32, device="cuda"), 4, 824)
    assert gone.tolist() == [5000 - 1024, 1] and p.c.count.tolist() == [16 * 1024 - 3, 16 * 1024]
    for u in range(2):
        assert p.c.table[u, :1024].tolist() == table[u][torch.tensor(want[u])].tolist()
        assert sorted(p.c.table[u].tolist()) == sorted(table[u].tolist())


@pytest.mark.parametrize("max_blocks", [12000, 51200])
def test_evict_more_blocks_than_the_registers_hold(kvq, max_blocks):
    """More than 8192 blocks, and table rows of more than 40 KB in shared memory, up to the most that is allowed."""
    p = Pair(kvq, B=3, Hq=1, Hkv=1, D=64, max_tokens=16 * max_blocks)
    for rnd, (keep, a, b) in enumerate((([max_blocks // 3, 9000, 5], 1, 1), ([8200, max_blocks - 1, 700], 300, 400), ([0, 1, 2], 40, 60))):
        held = [max_blocks, max_blocks - 1, 8193]
        p.c.count.copy_(torch.tensor([16 * max_blocks - 3, 16 * held[1], 16 * held[2] - 9], dtype=torch.int32))
        before = p.c.count.tolist()
        acc = torch.rand(p.c.acc.shape, generator=p.gen).round(decimals=3)          # ties
        if rnd == 1:
            acc[::1111] = float("nan")
        p.c.acc.copy_(acc)
        table, acc = p.c.table.cpu().numpy(), acc.numpy()
        gone = p.kvq.block8_evict(p.c, torch.tensor(keep, dtype=torch.int32, device="cuda"), a, b).tolist()
        now, count = p.c.table.cpu().numpy(), p.c.count.tolist()
        for u in range(3):
            n, want = held[u], max(keep[u], a + b)
            if n <= want:
                assert gone[u] == 0 and count[u] == before[u] and np.array_equal(now[u], table[u])
                continue
            score = acc[table[u, :n]]
            kept = _choose(np.where(np.isnan(score), np.inf, score), want, a, b)
            rest = np.setdiff1d(np.arange(n), kept)
            assert gone[u] == n - want and count[u] == before[u] - 16 * (n - want)
            assert np.array_equal(now[u], np.concatenate([table[u, kept], table[u, rest], table[u, n:]])), (rnd, u)


# ------------------------------------------------------------------ as they are used

def test_decode_with_eviction_and_selection(kvq):
    """A prompt through prefill_attn_scores, its scores seeding the blocks' weights, then decode steps that append,
    attend (dense, accumulating) and every few steps evict; a second attention reads selected blocks only."""
    B, Hq, Hkv, D, T = 2, 8, 2, 128, 300
    p = Pair(kvq, B=B, Hq=Hq, Hkv=Hkv, D=D, block=16, codes=F8, dtype=torch.bfloat16, max_tokens=512)
    p.evicted = True
    q, k, v = p.rand(B, Hq, T, D, outlier=False), p.rand(B, Hkv, T, D), p.rand(B, Hkv, T, D, outlier=False)
    _, _, cs = kvq.prefill_attn_scores(q.cuda(), k.cuda(), v.cuda())
    kvq.block8_append(p.c, k.cuda(), v.cuda(), colscore=cs)
    for u, unit in enumerate(p.units):
        b, h = divmod(u, Hkv)
        unit.append(k[b, h].float().numpy(), v[b, h].float().numpy(),
                    cs[b, h * 4:h * 4 + 4].double().sum(0).cpu().numpy())
    p.check(acc_rtol=(4 * 16 + 2) * U24)
    for step in range(24):
        p.append(1)
        qs = p.rand(B, Hq, 1, D)
        p.attn(qs, accumulate=True)                     # takes the kernel's acc over into the model
        blocks = _check_select(p, qs, 6, 1, 2)
        p.attn(qs, blocks=blocks)
        if step % 8 == 7:
            keep = torch.tensor([12, 10, 30, 5], dtype=torch.int32)
            want = [unit.evict(int(x), 1, 2) for unit, x in zip(p.units, keep)]
            assert kvq.block8_evict(p.c, keep.cuda(), 1, 2).tolist() == want
            p.check()
    assert p.c.seq_len.tolist() == [T + 24] * 4


def _filled(kvq, **kw):
    p = Pair(kvq, B=2, Hq=8, Hkv=2, max_tokens=640, **kw)
    p.append(500, n_new=[500, 77])
    p.c.acc.zero_()
    return p


def test_graph_replay_and_shared_workspace(kvq):
    """Captured steps of two caches that share one workspace, replayed in turn, against eager steps of their twins."""
    a, b = _filled(kvq, seed=1), _filled(kvq, seed=2)
    shared = a.c.ws
    caches = []
    for x in (a, b):
        f = {k: getattr(x.c, k).clone() for k in ("k_codes", "v_codes", "k_scale", "v_scale", "k_bound", "bound_scale",
                                                  "tail_k", "tail_v", "table", "count", "seq_len", "block_pos", "acc")}
        caches.append(kvq.Block8Cache(2, 8, 2, 128, 16, torch.float16, ws=shared, **f))
    k, v = a.rand(2, 2, 1, 128).cuda(), a.rand(2, 2, 1, 128).cuda()
    q = a.rand(2, 8, 1, 128).cuda()
    keep = torch.full((4,), 20, dtype=torch.int32, device="cuda")

    def step(c):
        kvq.block8_append(c, k, v)
        o1, l1 = kvq.block8_attn(q, c, accumulate=True)
        idx, n = kvq.block8_select(q, c, 5)
        o2, l2 = kvq.block8_attn(q, c, blocks=(idx, n))
        gone = kvq.block8_evict(c, keep)
        return o1, l1, idx, n, o2, l2, gone

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for c in caches:
        arrays = [t.view(torch.uint8) for t in (c.k_codes, c.v_codes)] + [
            c.k_scale, c.v_scale, c.k_bound, c.bound_scale, c.tail_k, c.tail_v, c.table, c.count, c.seq_len, c.block_pos, c.acc]
        snap = [t.clone() for t in arrays]
        with torch.cuda.stream(s):
            step(c)                                     # before the capture, on the stream it uses
        s.synchronize()
        for t, o in zip(arrays, snap):
            t.copy_(o)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(step(c))
        graphs.append(g)
        for t, o in zip(arrays, snap):
            t.copy_(o)
    for rep in range(3):
        for t in (q, k, v):
            t.copy_(a.rand(*t.shape).cuda())
        for i, x in enumerate((a, b)):
            graphs[i].replay()
            want = step(x.c)
            torch.cuda.synchronize()
            for y, z in zip(outs[i], want):
                assert torch.equal(y, z), (rep, i)
            for name in ("count", "table", "acc", "k_scale"):
                y, z = getattr(caches[i], name), getattr(x.c, name)
                assert torch.equal(y.nan_to_num(), z.nan_to_num()), name


def test_first_calls_inside_a_capture(kvq):
    """Nothing of a cache has run before, on the capture's stream or any other."""
    p, twin = Pair(kvq, B=2, Hq=8, Hkv=2, max_tokens=640, seed=3), Pair(kvq, B=2, Hq=8, Hkv=2, max_tokens=640, seed=3)
    k, v, q = (p.rand(2, h, n, 128).cuda() for h, n in ((2, 300), (2, 300), (8, 1)))
    keep = torch.full((4,), 9, dtype=torch.int32, device="cuda")

    def calls(c):
        kvq.block8_reset(c)
        kvq.block8_append(c, k, v)
        o = kvq.block8_attn(q, c, accumulate=True)
        blocks = kvq.block8_select(q, c, 5)
        return *o, *blocks, *kvq.block8_attn(q, c, blocks=blocks), kvq.block8_evict(c, keep)

    table = p.c.table.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = calls(p.c)
    want = calls(twin.c)
    for _ in range(2):
        p.c.table.copy_(table)
        g.replay()
        torch.cuda.synchronize()
        for y, z in zip(got, want):
            assert torch.equal(y, z)
    del g, got, p                                       # the graph first, then the cache that it wrote to


def test_other_streams(kvq):
    """Calls on a stream that is not torch's current one, with inputs freed right after."""
    p, twin = _filled(kvq, seed=5), _filled(kvq, seed=5)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(5):
        k, v, q = twin.rand(2, 2, 1, 128), twin.rand(2, 2, 1, 128), twin.rand(2, 8, 1, 128)
        kvq.block8_append(twin.c, k.cuda(), v.cuda())
        want = kvq.block8_attn(q.cuda(), twin.c)
        kd, vd, qd = k.cuda(), v.cuda(), q.cuda()
        s.wait_stream(torch.cuda.current_stream())
        kvq.block8_append(p.c, kd, vd, stream=s)
        got = kvq.block8_attn(qd, p.c, stream=s)
        del kd, vd, qd
        torch.full((2, 2, 1, 128), float("nan"), device="cuda", dtype=torch.float16)
        s.synchronize()
        assert torch.equal(got[0], want[0])


def test_cache_dropped_behind_a_call_on_another_stream(kvq):
    """Its memory is not given out again while the call runs."""
    p = _filled(kvq, seed=9)
    names = ("k_codes", "v_codes", "k_scale", "v_scale", "k_bound", "bound_scale", "tail_k", "tail_v", "table", "count",
             "seq_len", "block_pos", "acc", "ws")
    sizes = [(getattr(p.c, x).data_ptr(), getattr(p.c, x).numel() * getattr(p.c, x).element_size()) for x in names]
    q = p.rand(2, 8, 1, 128).cuda()
    want = kvq.block8_attn(q, p.c)
    count, p.c.count = p.c.count, torch.zeros_like(p.c.count)       # a tensor put in another's place changes nothing
    assert count.data_ptr() == sizes[9][0]
    s = torch.cuda.Stream()
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in sizes]      # memory that the allocator has ready below
    del new
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(1 << 27)                      # a bounded wait of some 60 ms
    got = kvq.block8_attn(q, p.c, stream=s)
    del p, count
    new = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _, n in sizes]
    assert not s.query()
    for x in new:
        for at, n in sizes:
            assert x.data_ptr() + x.numel() <= at or at + n <= x.data_ptr()
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_binding_refusals(kvq):
    p = Pair(kvq, B=2, Hq=4, Hkv=2, max_tokens=64)
    z = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="k must be"):
        kvq.block8_append(p.c, z(2, 3, 1, 128), z(2, 3, 1, 128))
    with pytest.raises(ValueError, match="one shape"):
        kvq.block8_append(p.c, z(2, 2, 1, 128), z(2, 2, 2, 128))
    with pytest.raises(TypeError):
        kvq.block8_append(p.c, z(2, 2, 1, 128, dt=torch.bfloat16), z(2, 2, 1, 128))
    with pytest.raises(ValueError, match="contiguous"):
        kvq.block8_append(p.c, z(2, 2, 128, 2).transpose(2, 3), z(2, 2, 2, 128))
    with pytest.raises(kvq.KvqError, match="16-byte"):
        kvq.block8_append(p.c, z(2 * 2 * 128 + 8)[4:-4].view(2, 2, 1, 128), z(2, 2, 1, 128))
    with pytest.raises(kvq.KvqError, match="multiples of 8"):
        kvq.block8_append(p.c, z(2, 2, 2, 132)[..., :128], z(2, 2, 2, 128))
    with pytest.raises(kvq.KvqError, match="exceed"):
        kvq.block8_append(p.c, z(2, 2, 65, 128), z(2, 2, 65, 128))
    with pytest.raises(ValueError, match="n_new"):
        kvq.block8_append(p.c, z(2, 2, 1, 128), z(2, 2, 1, 128), n_new=i(3))
    with pytest.raises(ValueError, match="colscore"):
        kvq.block8_append(p.c, z(2, 2, 1, 128), z(2, 2, 1, 128), colscore=z(2, 2, 1, dt=torch.float32))
    with pytest.raises(ValueError, match="q must be"):
        kvq.block8_attn(z(2, 2, 1, 128), p.c)
    with pytest.raises(kvq.KvqError):
        kvq.block8_attn(z(2, 4, 17, 128), p.c)
    with pytest.raises(ValueError, match="blocks"):
        kvq.block8_attn(z(2, 4, 1, 128), p.c, blocks=(i(2, 2, 3), i(2, 2)))
    with pytest.raises(ValueError, match="o must be"):
        kvq.block8_attn(z(2, 4, 1, 128), p.c, o=z(2, 4, 128))
    with pytest.raises(kvq.KvqError, match="n_first"):
        kvq.block8_select(z(2, 4, 1, 128), p.c, 2, 2, 1)
    with pytest.raises(ValueError, match="keep"):
        kvq.block8_evict(p.c, i(3))
    with pytest.raises(kvq.KvqError, match="n_last"):
        kvq.block8_evict(p.c, i(4), 1, 0)
    with pytest.raises(ValueError, match="ws"):
        kvq.Block8Cache(**{f: getattr(p.c, f) for f in ("B", "Hq", "Hkv", "D", "block", "dtype", "k_codes", "v_codes",
                                                         "k_scale", "v_scale", "k_bound", "bound_scale", "tail_k", "tail_v",
                                                         "table", "count", "seq_len", "block_pos", "acc")},
                        ws=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="table"):
        kvq.Block8Cache(**{f: getattr(p.c, f) for f in ("B", "Hq", "Hkv", "D", "block", "dtype", "k_codes", "v_codes",
                                                         "k_scale", "v_scale", "k_bound", "bound_scale", "tail_k", "tail_v",
                                                         "count", "seq_len", "block_pos", "acc")}, table=i(3, 4))
