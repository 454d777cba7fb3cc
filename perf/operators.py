"""The operators of the 8-bit block cache as cases to measure: their inputs, their plain forms, their work.

A cache holds the keys and values of U = B * Hkv units (one sequence and KV head each) in 8-bit codes (e4m3 or int8).
The tokens of a unit lie in blocks of `block` tokens, one float32 scale for the keys and one for the values of each;
logical block i of unit u is block table[u][i] of a pool that all units share.  Four operators work on it:

  append  new tokens (one of a step, or a prompt) are quantised into the blocks, with bounds of the keys per channel
  attn    attention of n_q queries over all tokens, or over a list of blocks; optionally each block's share of the
          softmax weights is added to acc
  select  the blocks of the largest upper bound of q.k, for each query and KV head
  evict   blocks of the smallest acc leave the table until `keep` are left

`run` computes them with elementary torch operations, or by the framework's calls where `own` is set.
"""
import math

import torch

own = False

SMALLEST = 2.0 ** -64       # scales are never smaller, so that a block of zeros has one too


# ------------------------------------------------------------------ cases

def _case(name, op, B, Hq, Hkv, D, T, block, codes, dtype, low=0, n=1, n_q=1, n_sel=0, keep=0, acc=False, cap=0):
    """T: the most tokens that a unit holds; low: the fewest.  cap: tokens that a unit has room for (T and n if 0)."""
    room = max(cap, T + (n if op == "append" else 0), 1)
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T, "low": low or T, "block": block,
            "codes": codes, "dtype": dtype, "n": n, "n_q": n_q, "n_sel": n_sel, "keep": keep, "acc": acc,
            "max_blocks": -(-room // block)}


def listed():
    return [
        # one decode step's new token of 64 sequences, at ragged lengths: what every layer does at every step
        _case("append-step", "append", 64, 32, 8, 128, 4000, 64, "e4m3", "bf16", low=17),
        # 16 prompts of 16384 tokens of a layer with 32 KV heads put into an empty cache, with the prompt's scores
        _case("append-prompt", "append", 16, 32, 32, 128, 0, 32, "int8", "f16", n=16384, acc=True),
        # the smallest decode: one sequence, two heads of 64 channels, 256 tokens; latency is all
        _case("attn-tiny", "attn", 1, 2, 2, 64, 256, 16, "e4m3", "f16"),
        # one sequence of 4096 tokens, 32 heads without sharing
        _case("attn-4k", "attn", 1, 32, 32, 128, 4096, 64, "e4m3", "f16"),
        # 32 sequences of ragged lengths up to 8192, five query heads per KV head
        _case("attn-gqa5", "attn", 32, 40, 8, 128, 8192, 32, "int8", "f16", low=700),
        # the largest decode: 64 sequences of 32768 tokens, four heads per KV head, weights accumulated for eviction
        _case("attn-32k-acc", "attn", 64, 32, 8, 128, 32768, 64, "e4m3", "bf16", acc=True),
        # a step that feeds four known tokens of each sequence (a prompt's last piece), eight heads per KV head, causal
        _case("attn-4q", "attn", 8, 64, 8, 128, 20011, 128, "int8", "bf16", low=9000, n_q=4),
        # one long sequence: choose 64 of up to 2048 blocks
        _case("select-1", "select", 1, 32, 8, 128, 131072, 64, "e4m3", "bf16", n_sel=64),
        # 16 long sequences of ragged lengths
        _case("select-16", "select", 16, 32, 8, 128, 131072, 64, "e4m3", "bf16", low=60001, n_sel=64),
        # attention over the 64 chosen blocks of each of those
        _case("attn-blocks", "attn", 16, 32, 8, 128, 131072, 64, "e4m3", "bf16", low=60001, n_sel=64),
        # one sequence's blocks brought back to a budget
        _case("evict-1", "evict", 1, 32, 8, 128, 8192, 64, "e4m3", "f16", keep=64),
        # 64 sequences with up to 2048 blocks a head, down to 1024
        _case("evict-64", "evict", 64, 32, 8, 128, 32768, 16, "e4m3", "bf16", low=12000, keep=1024),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over the logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["append", "append", "attn", "attn", "attn", "select", "attn-blocks", "evict"])
    D = rng.choice([64, 128, 128])
    block = rng.choice([16, 32, 64, 128])
    codes, dtype = rng.choice(["e4m3", "int8"]), rng.choice(["f16", "bf16"])
    Hkv = rng.choice([1, 2, 4, 8, 8, 32])
    g = rng.choice([1, 2, 4, 5, 8, 12, 16]) if Hkv < 32 else rng.choice([1, 1, 2])
    n_q = rng.choice([1, 1, 1, 2, 4, 8])
    T = _spread(rng, 1, 131072)
    most = 64 * 8 * 32768 if op in ("attn", "append") else 16 * 8 * 131072
    B = _spread(rng, 1, max(1, min(64, most // (T * Hkv))))
    low = _spread(rng, max(1, T // 8), T)
    if op == "append" and rng.random() < 0.5:          # prompts into an empty cache
        n = _spread(rng, 2, 16384)
        B = _spread(rng, 1, max(1, min(64, 16 * 32 * 16384 // (2 * n * Hkv))))
        return _drawn(_case("", op, B, Hkv * g, Hkv, D, 0, block, codes, dtype, n=n, acc=rng.random() < 0.5))
    if op == "append":                                   # a step: no more tokens than fit the open block
        return _drawn(_case("", op, min(B, 64), Hkv * g, Hkv, D, min(T, 4096), block, codes, dtype,
                            low=min(low, T, 4096)))
    if op == "evict":
        return _drawn(_case("", op, B, Hkv * g, Hkv, D, T, block, codes, dtype, low=low,
                            keep=max(2, -(-T // block) * rng.randrange(20, 100) // 100)))
    if op == "attn":
        return _drawn(_case("", op, B, Hkv * g, Hkv, D, T, block, codes, dtype, low=low, n_q=n_q,
                            acc=rng.random() < 0.4))
    return _drawn(_case("", op.split("-")[0], B, Hkv * g, Hkv, D, T, block, codes, dtype, low=low,
                        n_q=min(n_q, 2), n_sel=min(_spread(rng, 2, 128), max(2, -(-T // block)))))


def _drawn(case):
    del case["name"]
    return case


def _lengths(case):
    """Tokens that each unit holds: between low and T, the longest first; known from the case alone."""
    U, T, low = case["B"] * case["Hkv"], case["T"], case["low"]
    return [T - int((T - low) * ((u * 0.6180339887498949) % 1.0)) for u in range(U)]


# ------------------------------------------------------------------ inputs

def _qmax(case):
    return 448.0 if case["codes"] == "e4m3" else 127.0


def _dtype(case):
    return torch.float16 if case["dtype"] == "f16" else torch.bfloat16


def _to_codes(case, x):
    if case["codes"] == "e4m3":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return x.round().clamp(-127.0, 127.0).to(torch.int8)


def _code_values(codes):
    return codes.float()


def _scale(amax, qmax):
    """The scale of a block whose largest absolute value is amax (float32 throughout)."""
    return (amax * torch.tensor(1.0 / qmax, dtype=torch.float32, device=amax.device)).clamp_min(SMALLEST)


def _keys(shape, D, gen, dev):
    """Keys: Gaussian with a spread of their own per channel, and two channels of outliers."""
    x = torch.randn(shape, generator=gen, device=dev)
    spread = torch.exp(0.5 * torch.randn(D, generator=gen, device=dev))
    spread[D // 5] *= 8.0
    spread[D - 3] *= 8.0
    return x * spread


def _quantise(case, x):
    """Codes, scale and key bounds of blocks x [..., block, D] (all tokens valid)."""
    s = _scale(x.abs().amax(dim=(-2, -1)), _qmax(case))
    codes = _to_codes(case, x * s.reciprocal()[..., None, None])
    sb = _scale(x.abs().amax(dim=(-2, -1)), 127.0)
    ib = sb.reciprocal()[..., None]
    low = torch.floor(x.amin(dim=-2) * ib).clamp(-127.0, 127.0)
    high = torch.ceil(x.amax(dim=-2) * ib).clamp(-127.0, 127.0)
    return codes, s, torch.stack([low, high], dim=-2).to(torch.int8), sb


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, Hq, Hkv, D, P, nb = case["B"], case["Hq"], case["Hkv"], case["D"], case["block"], case["max_blocks"]
    U, N, dt = B * Hkv, B * Hkv * nb, _dtype(case)
    st = {"case": case}
    full = case["op"] == "attn"                         # only attention reads the codes of all blocks
    if full or case["op"] == "select":
        k = _keys((N, P, D), D, gen, dev)
        st["k_codes"], st["k_scale"], st["k_bound"], st["bound_scale"] = _quantise(case, k)
        del k
    else:
        st["k_codes"] = torch.zeros((N, P, D), device=dev, dtype=torch.uint8).view(_to_codes(case, torch.zeros(1)).dtype)
        st["k_scale"] = torch.ones(N, device=dev)
        st["k_bound"] = torch.zeros((N, 2, D), dtype=torch.int8, device=dev)
        st["bound_scale"] = torch.ones(N, device=dev)
    if full:
        st["v_codes"], st["v_scale"] = _quantise(case, torch.randn((N, P, D), generator=gen, device=dev))[:2]
    else:
        st["v_codes"], st["v_scale"] = torch.zeros_like(st["k_codes"]), torch.ones(N, device=dev)
    # counters and table share one array, so that one copy brings them back to where they were; for append the scales
    # too: an open block's must be the old ones, or no new token would be larger than what the block holds already
    held = U * (nb + 2)
    meta = torch.empty(held + (3 * N if case["op"] == "append" else 0), dtype=torch.int32, device=dev)
    if case["op"] == "append":
        for name, x in zip(("k_scale", "v_scale", "bound_scale"), meta[held:].view(torch.float32).view(3, N)):
            st[name] = x.copy_(st[name])
    count = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
    meta[:U] = count
    meta[U:2 * U] = count + 11 * 16                     # some tokens were dropped before
    meta[2 * U:held] = torch.randperm(N, generator=gen, device=dev).to(torch.int32)
    if case["op"] == "append" and case["T"] == 0:
        meta[U:2 * U] = 0
    st["meta"], st["meta0"] = meta, meta.clone()
    st["count"], st["seq_len"], st["table"] = meta[:U], meta[U:2 * U], meta[2 * U:held].view(U, nb)
    # what attention left in the blocks: mostly little, much in a few
    st["acc0"] = torch.exp(2.0 * torch.randn(N, generator=gen, device=dev))
    st["acc"] = st["acc0"].clone()
    st["block_pos"] = torch.zeros(N, dtype=torch.int32, device=dev)
    st["tail_k"] = torch.zeros((U, P, D), dtype=dt, device=dev)
    st["tail_v"] = torch.zeros((U, P, D), dtype=dt, device=dev)
    if case["op"] == "append":
        n = case["n"]
        st["k"] = _keys((B, Hkv, n, D), D, gen, dev).to(dt)
        st["v"] = torch.randn((B, Hkv, n, D), generator=gen, device=dev).to(dt)
        st["colscore"] = torch.rand((B, Hq, n), generator=gen, device=dev) ** 4 if case["acc"] else None
        if case["T"]:
            _open_blocks(case, st, gen)
            st["meta0"].copy_(meta)
    else:
        st["q"] = torch.randn((B, Hq, case["n_q"], D), generator=gen, device=dev).to(dt)
        st["sm_scale"] = 1.0 / math.sqrt(D)
    if case["op"] == "attn" and case["n_sel"]:
        st["idx"], st["n"] = _lists(case, st, gen)
    if case["op"] == "evict":
        st["keep"] = torch.full((U,), case["keep"], dtype=torch.int32, device=dev)
    return st


def _open_blocks(case, st, gen):
    """The last, partly filled block of each unit: 16-bit rows, codes, scales and bounds that agree."""
    P, D, U = case["block"], case["D"], case["B"] * case["Hkv"]
    fill = st["count"] % P
    held = (torch.arange(P, device="cuda")[None] < fill[:, None])[..., None]
    at = st["table"].gather(1, (st["count"] // P).clamp_max(case["max_blocks"] - 1).long()[:, None])[:, 0].long()
    for name, x in (("k", _keys((U, P, D), D, gen, "cuda")), ("v", torch.randn((U, P, D), generator=gen, device="cuda"))):
        x = torch.where(held, x.to(_dtype(case)), torch.zeros((), dtype=_dtype(case), device="cuda"))
        st["tail_" + name].copy_(x)
        got = _blocks_of(case, x.float()[:, None], held[:, None, :, 0])
        new = torch.nonzero(fill)[:, 0]
        st[name + "_codes"].view(torch.uint8)[at[new]] = got[0][new, 0].view(torch.uint8)
        st[name + "_scale"][at[new]] = got[1][new, 0]
        if name == "k":
            st["k_bound"][at[new]] = got[2][new, 0]
            st["bound_scale"][at[new]] = got[3][new, 0]


def _lists(case, st, gen):
    """Block lists as select gives them: ascending, the first and the last block among them."""
    B, Hkv, n_q, n_sel, nb = case["B"], case["Hkv"], case["n_q"], case["n_sel"], case["max_blocks"]
    seen = _seen_blocks(case, st)[..., None]
    score = torch.rand((B, Hkv, n_q, nb), generator=gen, device="cuda")
    i = torch.arange(nb, device="cuda")
    score = torch.where((i == 0) | (i == seen - 1), 2.0, score)
    score = torch.where(i < seen, score, -1.0)
    if nb < n_sel:
        score = torch.nn.functional.pad(score, (0, n_sel - nb), value=-1.0)
    idx = score.topk(n_sel, dim=-1).indices.sort(dim=-1).values
    n = seen.clamp_max(n_sel)
    valid = torch.arange(n_sel, device="cuda") < n
    # where a unit has fewer blocks than n_sel, its blocks come first
    idx = torch.where(seen <= n_sel, torch.arange(n_sel, device="cuda"), idx)
    return torch.where(valid, idx, -1).to(torch.int32).contiguous(), n[..., 0].to(torch.int32).contiguous()


# ------------------------------------------------------------------ plain forms

def _limits(case, st):
    """[B, Hkv, n_q] tokens that each query sees: the queries are the unit's last n_q tokens."""
    t = torch.arange(case["n_q"], device="cuda")
    c = st["count"].view(case["B"], case["Hkv"], 1).long()
    return (c - case["n_q"] + t + 1).clamp_min(0)


def _seen_blocks(case, st):
    return (_limits(case, st) + case["block"] - 1) // case["block"]


def _blocks_of(case, x, valid):
    """_quantise for blocks [U, n, block, D] of which only `valid` [U, n, block] tokens count."""
    v = valid[..., None]
    amax = torch.where(v, x.abs(), 0.0).amax(dim=(-2, -1))
    s, sb = _scale(amax, _qmax(case)), _scale(amax, 127.0)
    codes = _to_codes(case, x * s.reciprocal()[..., None, None])
    ib = sb.reciprocal()[..., None]
    low = torch.floor(torch.where(v, x, math.inf).amin(dim=-2) * ib).clamp(-127.0, 127.0)
    high = torch.ceil(torch.where(v, x, -math.inf).amax(dim=-2) * ib).clamp(-127.0, 127.0)
    return codes, s, torch.stack([low, high], dim=-2).to(torch.int8), sb


def _placed(case, st):
    """Where the new tokens go: the touched blocks [U, m] (in the unit's order, in the pool), the first new and the
    first free token of the unit counted from the first touched block, and which tokens are held after the call."""
    P, n = case["block"], case["n"]
    U, m = case["B"] * case["Hkv"], (n + P - 2) // P + 1
    f0 = (st["count"].long() // P)
    blocks = f0[:, None] + torch.arange(m, device="cuda")
    a = (st["count"].long() - f0 * P)[:, None]
    pool = st["table"].gather(1, blocks.clamp_max(case["max_blocks"] - 1)).long()
    row = torch.arange(m * P, device="cuda")[None]
    return U, m, blocks, pool, a, row, row < a + n, blocks * P < st["count"].long()[:, None] + n


def _plain_append(case, st):
    st["meta"].copy_(st["meta0"])
    U, m, blocks, pool, a, row, held, touched = _placed(case, st)
    P, D, n, U2 = case["block"], case["D"], case["n"], torch.arange(case["B"] * case["Hkv"], device="cuda")[:, None]
    at = pool[touched]
    for name in ("k", "v"):
        new = st[name].view(U, n, D)[U2, (row - a).clamp(0, n - 1)]
        old = st["tail_" + name][U2, row.clamp_max(P - 1)]
        x = torch.where((row < a)[..., None], old, new).view(U, m, P, D)
        codes, s, bound, sb = _blocks_of(case, x.float(), held.view(U, m, P))
        c8 = st[name + "_codes"].view(torch.uint8)
        c8[at] = torch.where(held.view(U, m, P)[touched][..., None], codes.view(torch.uint8)[touched], c8[at])
        st[name + "_scale"][at] = s[touched]
        if name == "k":
            st["k_bound"][at] = bound[touched]
            st["bound_scale"][at] = sb[touched]
        # the open block, if there is one, stays in 16 bits too
        end = a[:, 0] + n
        last = x.gather(1, (end // P).clamp_max(m - 1)[:, None, None, None].expand(U, 1, P, D))[:, 0]
        kept = (torch.arange(P, device="cuda")[None] < (end % P)[:, None])[..., None]
        st["tail_" + name].copy_(torch.where(kept, last, st["tail_" + name]))
    opened = touched & (blocks * P >= st["count"].long()[:, None])
    first = st["seq_len"].long()[:, None] + blocks * P - st["count"].long()[:, None]
    st["block_pos"][pool[opened]] = first[opened].to(torch.int32)
    st["acc"][pool[opened]] = 0.0
    if st["colscore"] is not None:
        w = st["colscore"].view(case["B"], case["Hkv"], -1, n).sum(dim=2).view(U, n)
        w = torch.where(held & (row >= a), w[U2, (row - a).clamp(0, n - 1)], 0.0).view(U, m, P).sum(dim=-1)
        st["acc"][at] += w[touched]
    st["count"] += n
    st["seq_len"] += n
    return _append_outputs(st)


def _append_outputs(st):
    return {k: st[k] for k in ("k_codes", "v_codes", "k_scale", "v_scale", "k_bound", "bound_scale", "tail_k",
                               "tail_v", "count", "seq_len", "block_pos", "acc")}


def _plain_attn(case, st):
    B, Hq, Hkv, D, P, n_q = case["B"], case["Hq"], case["Hkv"], case["D"], case["block"], case["n_q"]
    U, g = B * Hkv, Hq // Hkv
    # dense: the unit's blocks once for all queries; with lists: each query's own blocks
    if case["n_sel"]:
        place = st["idx"].view(U, n_q, -1).long()
        listed_ = place >= 0
        place = place.clamp_min(0)
    else:
        place = torch.arange(case["max_blocks"], device="cuda").expand(U, 1, -1)
        listed_ = torch.ones_like(place, dtype=torch.bool)
    s, m = place.shape[1], place.shape[2]
    pool = st["table"].long().gather(1, place.reshape(U, s * m)).view(U, s, m)
    q = st["q"].view(B, Hkv, g, n_q, D).permute(0, 1, 3, 2, 4).reshape(U, s, n_q // s * g, D).float()
    k = _code_values(st["k_codes"].view(torch.uint8)[pool].view(st["k_codes"].dtype)).view(U, s, m * P, D)
    x = torch.matmul(q, k.transpose(-1, -2)).view(U, s, n_q // s, g, m, P)
    del k
    x = x * (st["k_scale"][pool] * st["sm_scale"])[:, :, None, None, :, None]
    token = place[..., None] * P + torch.arange(P, device="cuda")
    seen = token[:, :, None] < _limits(case, st).view(U, s, n_q // s, 1, 1)
    seen = (seen & listed_[:, :, None, :, None])[:, :, :, None]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(dim=(-2, -1), keepdim=True).clamp_min(-3.0e38)
    p = torch.exp(x - top)
    total = p.sum(dim=(-2, -1), keepdim=True)
    p = torch.where(seen, p / total, 0.0)
    lse = (torch.log(total) + top)[..., 0, 0]
    v = _code_values(st["v_codes"].view(torch.uint8)[pool].view(st["v_codes"].dtype)).view(U, s, m * P, D)
    w = (p * st["v_scale"][pool][:, :, None, None, :, None]).view(U, s, n_q // s * g, m * P)
    o = torch.matmul(w, v)
    del v
    o = o.view(B, Hkv, n_q, g, D).permute(0, 1, 3, 2, 4).reshape(B, Hq, n_q, D).to(st["q"].dtype)
    out = {"o": o, "lse": lse.reshape(B, Hkv, n_q, g).permute(0, 1, 3, 2).reshape(B, Hq, n_q)}
    if case["acc"]:
        out["acc"] = st["acc0"].index_add(0, pool.reshape(-1), p.sum(dim=(2, 3, 5)).reshape(-1))
    return out


def _chosen(score, seen, n_sel):
    """Of blocks [..., m] with scores, of which the first `seen` exist: the first, the last and those of the largest
    scores, n_sel in all, ascending; ties to the lower block."""
    m = score.shape[-1]
    i = torch.arange(m, device=score.device)
    score = torch.where((i == 0) | (i == seen - 1), math.inf, score)
    score = torch.where(i < seen, score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, i.expand_as(order))
    return (rank < n_sel) & (i < seen)


def _ascending(mask, n_sel):
    """The places of the ones of mask [..., m] in ascending order, -1 behind them: [..., n_sel]."""
    m = mask.shape[-1]
    i = torch.where(mask, torch.arange(m, device=mask.device), m).sort(dim=-1).values
    i = i[..., :n_sel] if m >= n_sel else torch.nn.functional.pad(i, (0, n_sel - m), value=m)
    return torch.where(i < m, i, -1).to(torch.int32), mask.sum(dim=-1).to(torch.int32)


def _plain_select(case, st):
    B, Hq, Hkv, D, n_q = case["B"], case["Hq"], case["Hkv"], case["D"], case["n_q"]
    U, g = B * Hkv, Hq // Hkv
    q = st["q"].view(B, Hkv, g, n_q, D).permute(0, 1, 3, 2, 4).reshape(U, n_q, g, D).float()
    sq = _scale(q.abs().amax(dim=-1), 127.0)
    q8 = (q * sq.reciprocal()[..., None]).round().clamp(-127.0, 127.0).reshape(U, n_q * g, D)
    bound = st["k_bound"][st["table"].long()].float()
    # sums of products of whole numbers below 2^24: float32 holds them exactly, in any order
    x = torch.matmul(q8.clamp_min(0.0), bound[:, :, 1].transpose(-1, -2))
    x = x + torch.matmul(q8.clamp_max(0.0), bound[:, :, 0].transpose(-1, -2))
    x = (x.view(U, n_q, g, -1) * sq[..., None]).amax(dim=2) * st["bound_scale"][st["table"].long()][:, None]
    mask = _chosen(x, _seen_blocks(case, st).view(U, n_q, 1), case["n_sel"])
    idx, n = _ascending(mask, case["n_sel"])
    return {"idx": idx.view(B, Hkv, n_q, -1), "n": n.view(B, Hkv, n_q)}


def _plain_evict(case, st):
    P, nb = case["block"], case["max_blocks"]
    st["meta"].copy_(st["meta0"])
    n = ((st["count"].long() + P - 1) // P)[:, None]
    mask = _chosen(st["acc0"][st["table"].long()], n, case["keep"])
    i = torch.arange(nb, device="cuda").expand_as(mask)
    # kept blocks first, then those that left, then those that were free: each in its order
    order = torch.where(mask, i, torch.where(i < n, i + nb, i + 2 * nb)).sort(dim=-1).values % nb
    gone = n[:, 0] - mask.sum(dim=-1)
    st["table"].copy_(st["table"].gather(1, order))
    st["count"] -= (gone * P).to(torch.int32)
    return {"table": st["table"], "count": st["count"], "seq_len": st["seq_len"], "gone": gone.to(torch.int32)}


# ------------------------------------------------------------------ one pass

def _cache(st):
    from bit_mixed_precision_gb300 import kvq
    if "cache" not in st:
        c = st["case"]
        st["cache"] = kvq.Block8Cache(
            B=c["B"], Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"], block=c["block"], dtype=_dtype(c), max_q=c["n_q"],
            **{k: st[k] for k in ("k_codes", "v_codes", "k_scale", "v_scale", "k_bound", "bound_scale", "tail_k",
                                  "tail_v", "table", "count", "seq_len", "block_pos", "acc")})
    return kvq, st["cache"]


def run(state):
    case, op = state["case"], state["case"]["op"]
    if not own:
        return {"append": _plain_append, "attn": _plain_attn, "select": _plain_select, "evict": _plain_evict}[op](case, state)
    kvq, cache = _cache(state)
    if op == "append":
        state["meta"].copy_(state["meta0"])
        kvq.block8_append(cache, state["k"], state["v"], colscore=state["colscore"])
        return _append_outputs(state)
    if op == "attn":
        if case["acc"]:
            state["acc"].copy_(state["acc0"])
        blocks = (state["idx"], state["n"]) if case["n_sel"] else None
        o, lse = kvq.block8_attn(state["q"], cache, state["sm_scale"], blocks=blocks, accumulate=case["acc"])
        return {"o": o, "lse": lse, "acc": state["acc"]} if case["acc"] else {"o": o, "lse": lse}
    if op == "select":
        idx, n = kvq.block8_select(state["q"], cache, case["n_sel"])
        return {"idx": idx, "n": n}
    state["meta"].copy_(state["meta0"])
    gone = kvq.block8_evict(cache, state["keep"])
    return {"table": state["table"], "count": state["count"], "seq_len": state["seq_len"], "gone": gone}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    B, Hq, Hkv, D, P, n_q = case["B"], case["Hq"], case["Hkv"], case["D"], case["block"], case["n_q"]
    U, n, lengths = B * Hkv, case["n"], _lengths(case)
    if case["op"] == "append":
        # 16-bit rows in, 8-bit codes out; a scale for keys, values and bounds, the bounds, acc and position of each
        # touched block; the rows of an open block in 16 bits
        blocks = sum(-(-(c + n) // P) - c // P for c in lengths)
        tail = sum(min(n, (c + n) % P) for c in lengths)
        rows = U * n * (2 * 2 * D + 2 * D) + tail * 2 * 2 * D
        return {"bytes": rows + blocks * (3 * 4 + 2 * D + 3 * 4) + 16 * U + (4 * B * Hq * n if case["acc"] else 0),
                "flops": 6 * U * n * D}
    if case["op"] == "evict":
        blocks = sum(-(-c // P) for c in lengths)
        return {"bytes": 12 * blocks + 16 * U, "flops": blocks}
    if case["op"] == "select":
        blocks = sum(-(-c // P) for c in lengths)
        return {"bytes": blocks * (2 * D + 8) + 2 * B * Hq * n_q * D + 4 * U * n_q * (case["n_sel"] + 1),
                "flops": 4 * blocks * D * n_q * (Hq // Hkv)}
    read = rows = blocks = 0
    for c in lengths:
        whole = -(-c // P)
        if case["n_sel"]:
            tokens = min(c, (min(case["n_sel"], whole) - 1) * P + (c - 1) % P + 1)
            read, rows, blocks = read + n_q * tokens, rows + n_q * tokens, blocks + n_q * min(case["n_sel"], whole)
        else:
            read, rows, blocks = read + c, rows + n_q * c, blocks + whole
    return {"bytes": read * 2 * D + blocks * (12 + (8 if case["acc"] else 0)) + B * Hq * n_q * (4 * D + 4) + 4 * U,
            "flops": 4 * D * rows * (Hq // Hkv)}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """Append: scales, code values before their rounding (e4m3) and accumulated scores, block by block.  Attention: one
    sequence, KV head and query at a time, from the definition of softmax.  The others give whole numbers only."""
    B, Hq, Hkv, D, P, n, n_q = (case[k] for k in ("B", "Hq", "Hkv", "D", "block", "n", "n_q"))
    if case["op"] in ("select", "evict"):
        return None
    if B * Hkv * n_q > 8192:
        return None
    st, g = prepare(case, seed), Hq // Hkv
    if case["op"] == "append" and case["T"] == 0:       # a prompt into an empty cache: its blocks are rows of one array
        nb = -(-n // P)
        table, out = st["table"][:, :nb].long(), {k: st[k].double() for k in ("k_scale", "v_scale", "bound_scale", "acc")}
        in_blocks = lambda x: torch.nn.functional.pad(x.double(), (0, nb * P - n)).unflatten(-1, (nb, P))  # noqa: E731
        for name, scale, most in (("k", "k_scale", _qmax(case)), ("v", "v_scale", _qmax(case)), ("k", "bound_scale", 127.0)):
            amax = in_blocks(st[name].abs().amax(dim=-1).view(B * Hkv, n)).amax(dim=-1)
            out[scale][table] = (amax / most).clamp_min(SMALLEST)
        out["acc"][table] = 0.0
        if case["acc"]:
            out["acc"][table] = in_blocks(st["colscore"].double().view(B * Hkv, g, n).sum(dim=1)).sum(dim=-1)
        return out
    if case["op"] == "append":
        eight = case["codes"] == "e4m3"
        names = ("k_scale", "v_scale", "bound_scale", "acc") + (("k_codes", "v_codes") if eight else ())
        out = {k: st[k].float().double().cpu() for k in names}
        tails = {"k": st["tail_k"].double().cpu(), "v": st["tail_v"].double().cpu()}
        news = {"k": st["k"].double().cpu(), "v": st["v"].double().cpu()}
        col = st["colscore"].double().cpu() if case["acc"] else None
        table = st["table"].tolist()
        for u, c in enumerate(st["count"].tolist()):
            b, h = divmod(u, Hkv)
            for block in range(c // P, -(-(c + n) // P)):
                lo, hi = block * P, min((block + 1) * P, c + n)
                at, old, a = table[u][block], max(0, min(c, hi) - lo), max(0, lo - c)
                for name in ("k", "v"):
                    x = torch.cat([tails[name][u, :old], news[name][b, h, a:hi - c]])
                    most = float(x.abs().max())
                    out[name + "_scale"][at] = max(most / (448.0 if eight else 127.0), SMALLEST)
                    if eight:
                        out[name + "_codes"][at, :hi - lo] = x / out[name + "_scale"][at]
                    if name == "k":
                        out["bound_scale"][at] = max(most / 127.0, SMALLEST)
                if lo >= c:
                    out["acc"][at] = 0.0
                if col is not None:
                    out["acc"][at] += float(col[b, h * g:(h + 1) * g, a:hi - c].sum())
        return out
    o = torch.zeros((B, Hq, n_q, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, n_q), -math.inf, dtype=torch.float64, device="cuda")
    acc = st["acc0"].double()
    codes = {k: st[k + "_codes"] for k in ("k", "v")}
    for u, c in enumerate(st["count"].tolist()):
        b, h = divmod(u, Hkv)
        for t in range(n_q):
            see = c - n_q + t + 1
            if see <= 0:
                continue
            which = st["idx"][b, h, t, :int(st["n"][b, h, t])].long() if case["n_sel"] else torch.arange(-(-see // P)).cuda()
            at = st["table"][u][which].long()
            token = (which[:, None] * P + torch.arange(P, device="cuda")).reshape(-1)
            there = token < see
            k, v = (((codes[x].view(torch.uint8)[at].view(codes[x].dtype).to(torch.float64)
                      * st[x + "_scale"][at].double()[:, None, None]).reshape(-1, D)[there]) for x in ("k", "v"))
            z = st["q"][b, h * g:(h + 1) * g, t].double() @ k.T * st["sm_scale"]
            p = torch.softmax(z, dim=-1)
            o[b, h * g:(h + 1) * g, t] = p @ v
            lse[b, h * g:(h + 1) * g, t] = torch.logsumexp(z, dim=-1)
            block = torch.arange(len(which), device="cuda").repeat_interleave(P)[there]
            acc.index_add_(0, at, torch.zeros(len(which), dtype=torch.float64, device="cuda").index_add_(0, block, p.sum(0)))
    return {"o": o, "lse": lse, "acc": acc} if case["acc"] else {"o": o, "lse": lse}
