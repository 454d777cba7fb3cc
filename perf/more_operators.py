"""From a layer's projection to its attention and back, as cases to measure: inputs, plain forms, work.

Three operators around the framework's prefill attention and caches:

  rope      queries, keys and values leave the projection's [B, T, heads, D] for [B, heads, T, D]; on the way the queries
            and keys of each head are RMS-normed (with a weight per channel, or not at all) and rotated by their
            positions, which may have several axes
  rope_bwd  its gradient: of the projection's output and of the norms' weights
  attn_bwd  the gradients of q, k and v through causal attention, from its output and row log-sum-exp

`run` computes them with elementary torch operations, or by the framework's calls where `own` is set.
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 500000.0
MOST_SCORES = 1 << 31       # query-key pairs of one attention case


# ------------------------------------------------------------------ cases

def _rope(name, op, B, T, Hq, Hkv, D, dtype, rot=0, axes=1, interleaved=False, norm=True, far=0):
    """rot: rotated channels (all if 0).  far: positions start at up to this."""
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype, "rot": rot or D,
            "axes": axes, "interleaved": interleaved, "norm": norm, "far": far}


def _attn(name, B, Hq, Hkv, T, D, dtype):
    return {"name": name, "op": "attn_bwd", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype}


def listed():
    return [
        # the smallest call: one new token of one sequence, what a layer does before it appends and attends
        _rope("rope-token", "rope", 1, 1, 32, 8, 128, "bf16", far=100000),
        # one decode step of 64 sequences far into their contexts
        _rope("rope-step", "rope", 64, 1, 40, 8, 128, "f16", far=1000000),
        # a prompt of one image or clip: time, height and width; heads without sharing, an odd length
        _rope("rope-3axes", "rope", 1, 9001, 32, 32, 128, "bf16", axes=3),
        # four prompts of 16384 tokens
        _rope("rope-prompt", "rope", 4, 16384, 32, 8, 128, "bf16"),
        # a small training batch, neighbouring channels paired, a quarter of the head rotated
        _rope("rope-bwd-small", "rope_bwd", 2, 1023, 16, 16, 64, "f16", rot=16, interleaved=True),
        # a large training batch
        _rope("rope-bwd", "rope_bwd", 16, 4096, 32, 8, 128, "bf16"),
        # the smallest training step of an attention layer; latency is all
        _attn("attn-bwd-tiny", 1, 2, 2, 256, 64, "f16"),
        # one sequence of 1024 tokens, eight query heads per KV head: few tiles
        _attn("attn-bwd-1k", 1, 32, 4, 1024, 128, "bf16"),
        # an odd length, five heads per KV head
        _attn("attn-bwd-odd", 2, 40, 8, 1999, 128, "f16"),
        # small heads without sharing
        _attn("attn-bwd-d64", 8, 16, 16, 2048, 64, "bf16"),
        # an ordinary training batch: four sequences of 4096 tokens, 32 heads
        _attn("attn-bwd-4k", 4, 32, 8, 4096, 128, "bf16"),
        # a long sequence
        _attn("attn-bwd-16k", 1, 8, 2, 16384, 128, "f16"),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over the logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    D, dtype = rng.choice([64, 128, 128]), rng.choice(["f16", "bf16"])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16, 32])
    Hq = Hkv * (rng.choice([1, 2, 4, 5, 8]) if Hkv < 16 else rng.choice([1, 2]))
    if rng.random() < 0.5:
        T = _spread(rng, 16, min(16384, math.isqrt(MOST_SCORES // Hq)))
        B = _spread(rng, 1, max(1, min(16, MOST_SCORES // (Hq * T * T))))
        case = _attn("", B, Hq, Hkv, T, D, dtype)
    else:
        op = rng.choice(["rope", "rope", "rope_bwd"])
        step = op == "rope" and rng.random() < 0.4
        tokens = 4 * 16384 * 48 * 128 // ((Hq + 2 * Hkv) * D)       # of the listed prompts' bytes
        T = 1 if step else _spread(rng, 2, min(32768, tokens * 2 // 3))
        B = _spread(rng, 1, max(1, min(256, tokens * 2 // 3 // T)))
        case = _rope("", op, B, T, Hq, Hkv, D, dtype, rot=rng.choice([0, 0, D // 2, 16, 48]),
                     axes=rng.choice([1, 1, 2, 3, 4]), interleaved=rng.random() < 0.3, norm=rng.random() < 0.8,
                     far=rng.choice([0, 5000, 1000000]))
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.float16 if case["dtype"] == "f16" else torch.bfloat16


def _axis(case):
    """The axis of each pair of rotated channels: consecutive shares of the pairs, the first axis the remainder."""
    n, a = case["rot"] // 2, case["axes"]
    share = n // a
    return [0] * (n - (a - 1) * share) + [x for x in range(1, a) for _ in range(share)]


def _inv_freq(case):
    n = case["rot"] // 2
    return [BASE ** (-i / n) for i in range(n)]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, T, Hq, Hkv, D, dt = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"], _dtype(case)
    rand = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    st = {"case": case}
    if case["op"] == "attn_bwd":
        # keys: a spread of their own per channel; output gradients: small, and of differing size from token to token
        st["q"] = rand(B, Hq, T, D).to(dt)
        st["k"] = (rand(B, Hkv, T, D) * torch.exp(0.3 * rand(D))).to(dt)
        st["v"] = rand(B, Hkv, T, D).to(dt)
        size = 2.0 ** -4 if case["dtype"] == "f16" else 2.0 ** -10      # f16 trains with a scaled loss
        st["do"] = (rand(B, Hq, T, D) * torch.exp(0.5 * rand(T, 1)) * size).to(dt)
        st["sm_scale"] = 1.0 / math.sqrt(D)
        # what the forward pass left: the output and the rows' log-sum-exp
        x = _scores(case, st)
        top = x.amax(dim=-1, keepdim=True)
        x = x.sub_(top).exp_()
        total = x.sum(dim=-1, keepdim=True)
        st["lse"] = (top + total.log()).view(B, Hq, T)
        st["o"] = (torch.matmul(x, st["v"].float()[:, :, None]) / total).view(B, Hq, T, D).to(dt)
        return st
    # the projection's output, all heads of a token beside one another: head by head of a size of its own
    x = (rand(B, T, Hq + 2 * Hkv, D) * torch.exp(0.5 * rand(Hq + 2 * Hkv, 1))).to(dt)
    st["q_in"], st["k_in"], st["v_in"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    st["q_weight"] = (1.0 + 0.2 * rand(D)).to(dt) if case["norm"] else None
    st["k_weight"] = (1.0 + 0.2 * rand(D)).to(dt) if case["norm"] else None
    start = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device=dev)
    t = torch.arange(T, device=dev)
    if case["axes"] == 1:
        pos = start + t
    else:                                       # rows of a grid: the last axis runs fastest
        side = max(1, int(round(T ** (1.0 / case["axes"]))))
        pos = torch.stack([t // side ** a % (side if a + 1 < case["axes"] else T) + start for a in reversed(range(case["axes"]))])
    st["pos"] = pos.to(torch.int32).contiguous()
    if case["op"] == "rope_bwd":
        st["dq"], st["dk"] = (rand(B, h, T, D).to(dt) for h in (Hq, Hkv))
        st["dv"] = rand(B, Hkv, T, D).to(dt)
    return st


# ------------------------------------------------------------------ plain forms

def _scores(case, st):
    """[B, Hkv, g, T, T] scaled scores in float32, -inf above the diagonal."""
    B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
    q = st["q"].float().view(B, Hkv, -1, T, D) * st["sm_scale"]
    x = torch.matmul(q, st["k"].float()[:, :, None].transpose(-1, -2))
    t = torch.arange(T, device=x.device)
    return x.masked_fill_(t[None] > t[:, None], -math.inf)


def _plain_attn_bwd(case, st):
    B, T, Hq, Hkv, D, dt = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"], _dtype(case)
    per = (B, Hkv, Hq // Hkv, T)
    p = _scores(case, st).sub_(st["lse"].view(per + (1,))).exp_()
    do, k, v = st["do"].float().view(per + (D,)), st["k"].float()[:, :, None], st["v"].float()[:, :, None]
    delta = (do * st["o"].float().view(per + (D,))).sum(dim=-1, keepdim=True)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(dim=2)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_(delta).mul_(p).mul_(st["sm_scale"])
    del p
    dq = torch.matmul(ds, k).view(B, Hq, T, D)
    dk = torch.matmul(ds.transpose(-1, -2), st["q"].float().view(per + (D,))).sum(dim=2)
    return {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt)}


def _angles(case, st):
    """Cosine and sine [B, T, 1, rot / 2] of each pair's angle, the angles in 64 bits."""
    f = torch.tensor(_inv_freq(case), dtype=torch.float64, device="cuda")
    pos = st["pos"].view(case["axes"], case["B"], case["T"])
    phi = pos[_axis(case)].permute(1, 2, 0).double() * f
    return torch.cos(phi).float()[:, :, None], torch.sin(phi).float()[:, :, None]


def _rotated(case, x, cos, sin):
    """x [B, T, H, D] with the pairs of its first rot channels turned."""
    rot, n = case["rot"], case["rot"] // 2
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2), x[..., rot:]], dim=-1)
    a, b = x[..., :n], x[..., n:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], dim=-1)


def _plain_rope(case, st):
    cos, sin = _angles(case, st)
    out = {"v": st["v_in"].transpose(1, 2).contiguous()}
    for name in ("q", "k"):
        x, w = st[name + "_in"].float(), st[name + "_weight"]
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w.float()
        out[name] = _rotated(case, x, cos, sin).to(_dtype(case)).transpose(1, 2).contiguous()
    return out


def _plain_rope_bwd(case, st):
    cos, sin = _angles(case, st)
    out = {"gv": st["dv"].transpose(1, 2).contiguous()}
    for name in ("q", "k"):
        g = _rotated(case, st["d" + name].float().transpose(1, 2), cos, -sin)
        w = st[name + "_weight"]
        if w is not None:
            x = st[name + "_in"].float()
            r = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)
            x = x * r
            out["g" + name + "_weight"] = (g * x).sum(dim=(0, 1, 2))
            g = g * w.float()
            g = r * (g - x * (g * x).mean(dim=-1, keepdim=True))
        out["g" + name] = g.to(_dtype(case))
    return out


# ------------------------------------------------------------------ one pass

def run(state):
    case, op = state["case"], state["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "attn_bwd": _plain_attn_bwd}[op](case, state)
    from bit_mixed_precision_gb300 import kvq
    if op == "attn_bwd":
        dq, dk, dv = kvq.prefill_attn_bwd(state["do"], state["q"], state["k"], state["v"], state["o"], state["lse"],
                                          state["sm_scale"])
        return {"dq": dq, "dk": dk, "dv": dv}
    if "rope" not in state:
        state["rope"] = kvq.make_rope(case["D"], inv_freq=_inv_freq(case), axis=_axis(case), interleaved=case["interleaved"])
    raw = (state["q_in"], state["k_in"])
    weights = (state["q_weight"], state["k_weight"], EPS)
    if op == "rope":
        q, k, v = kvq.qk_norm_rope(*raw, state["v_in"], state["pos"], state["rope"], *weights)
        return {"v": v, "q": q, "k": k}
    gq, gk, gv, gqw, gkw = kvq.qk_norm_rope_bwd(state["dq"], state["dk"], state["dv"], *raw, state["pos"], state["rope"],
                                                *weights)
    out = {"gv": gv, "gq": gq, "gk": gk}
    return {**out, "gq_weight": gqw, "gk_weight": gkw} if case["norm"] else out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    B, T, Hq, Hkv, D = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "attn_bwd":
        # q, o, do in and dq out, k, v in and dk, dv out; five products over the pairs at and below the diagonal
        return {"bytes": B * T * (2 * D * (4 * Hq + 4 * Hkv) + 4 * Hq), "flops": 5 * 2 * D * B * Hq * (T * (T + 1) // 2)}
    rows = B * T * (Hq + Hkv)
    extra = 4 * case["axes"] * B * T + (4 * D if case["norm"] else 0)
    if case["op"] == "rope":
        return {"bytes": 2 * D * (2 * rows + 2 * B * T * Hkv) + extra, "flops": rows * (4 * D + 3 * case["rot"])}
    reads = 2 if case["norm"] else 1            # without a norm the gradient does not need the projection's output
    return {"bytes": 2 * D * ((reads + 1) * rows + 2 * B * T * Hkv) + extra + (8 * D if case["norm"] else 0),
            "flops": rows * (10 * D + 3 * case["rot"])}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """Attention one query head at a time; rotations as products of complex numbers, one axis at a time."""
    st = prepare(case, seed)
    B, T, Hq, Hkv, D = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if case["op"] == "attn_bwd":
        g, c = Hq // Hkv, st["sm_scale"]
        dq, dk, dv = torch.zeros((B, Hq, T, D), **f64), torch.zeros((B, Hkv, T, D), **f64), torch.zeros((B, Hkv, T, D), **f64)
        for b in range(B):
            for h in range(Hq):
                q, k, v, do = (st[n][b, i].double() for n, i in (("q", h), ("k", h // g), ("v", h // g), ("do", h)))
                z = (q @ k.T).mul_(c)
                w = torch.tril(z.sub_(st["lse"][b, h].double()[:, None]).exp_())
                del z
                dv[b, h // g].addmm_(w.T, do)
                w.mul_((do @ v.T).sub_((do * st["o"][b, h].double()).sum(dim=1, keepdim=True)))
                dq[b, h] = w @ k * c
                dk[b, h // g].addmm_(w.T, q, alpha=c)
        return {"dq": dq, "dk": dk, "dv": dv}

    n, rot = case["rot"] // 2, case["rot"]
    phi = torch.empty((B, T, n), **f64)
    for i, (axis, f) in enumerate(zip(_axis(case), _inv_freq(case))):
        phi[..., i] = st["pos"].view(case["axes"], B, T)[axis].double() * f
    turn = torch.polar(torch.ones_like(phi), phi)[:, :, None]

    def turned(x, by):
        head = x[..., :rot].unflatten(-1, (n, 2) if case["interleaved"] else (2, n))
        z = torch.complex(*(y.contiguous() for y in head.unbind(-1 if case["interleaved"] else -2))) * by
        head = torch.stack([z.real, z.imag], dim=-1 if case["interleaved"] else -2).flatten(-2)
        return torch.cat([head, x[..., rot:]], dim=-1)

    out = {}
    for name in ("q", "k"):
        x, w = st[name + "_in"].double(), st[name + "_weight"]
        size = torch.sqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
        if case["op"] == "rope":
            out[name] = turned(x if w is None else x / size * w.double(), turn).transpose(1, 2)
            continue
        d = turned(st["d" + name].double().transpose(1, 2), turn.conj())
        if w is not None:
            out["g" + name + "_weight"] = (d * x / size).sum(dim=(0, 1, 2))
            d = d * w.double()
            # the derivative of x / sqrt(mean(x^2) + eps)
            d = d / size - x * (d * x).mean(dim=-1, keepdim=True) / size ** 3
        out["g" + name] = d
    out["v" if case["op"] == "rope" else "gv"] = None
    return out
