"""Serving and scoring operators: their plain forms, and the cases they are measured at.

What a served or scored token passes through, and what training by its log probability needs:

  append   keys and values into a paged cache of 16-bit rows, the position rotation applied to queries and keys on
           the way
  turn     the rotation alone and its inverse, as a training step applies them around the attention
  park     the same into a cache held in 4 bits, and back: a conversation put aside and taken up again
  decode   attention of one new token per sequence over a cache held in 4 bits
  score    log probabilities of given tokens, with entropy and the most probable alternatives
  learn    the same with the gradient, as a policy update calls the pair

`run` computes them in elementary torch operations in 32 bits (angles in 64), or, where `own` is true, calls the
framework.

Rotation: pair i of a head's first `rot` values turns by position times frequency i; the pair is (i, i + rot / 2), or
(2 i, 2 i + 1) where `interleaved`. A cache row in 4 bits holds, for its D values, the lowest one and a scale (bf16 both)
and a code 0..15 per value, two to a byte, the even value low: value = lowest + scale * code.
"""
import math

import torch

own = False

LOG2E = 1.0 / math.log(2.0)


# ------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoding step of a serving batch, GPT-2 small's heads: latency
        {"name": "append token", "op": "append", "B": 16, "T": 1, "H": 12, "Hkv": 12, "D": 64, "page": 16, "rot": 64,
         "interleaved": False, "weights": True},
        # the repository's own benchmark batch as prompts
        {"name": "append prompts", "op": "append", "B": 16, "T": 1024, "H": 12, "Hkv": 12, "D": 64, "page": 16,
         "rot": 64, "interleaved": False, "weights": True},
        # a training step's rotation and its inverse, ragged against every tile, half of each head turned
        {"name": "turn train", "op": "turn", "B": 8, "T": 1000, "H": 12, "Hkv": 12, "D": 64, "rot": 32,
         "interleaved": True},
        # three short conversations with shared key heads
        {"name": "park short", "op": "park", "B": 3, "T": 77, "H": 16, "Hkv": 4, "D": 64, "page": 32, "rot": 64,
         "interleaved": False},
        # a batch of whole conversations
        {"name": "park batch", "op": "park", "B": 16, "T": 1024, "H": 12, "Hkv": 12, "D": 64, "page": 16, "rot": 64,
         "interleaved": False},
        # one conversation of GPT-2 small's heads: latency
        {"name": "decode one", "op": "decode", "B": 1, "H": 12, "Hkv": 12, "D": 64, "page": 16, "min_len": 600,
         "max_len": 600, "window": 0, "sinks": 0},
        # a serving batch of ragged lengths with shared key heads
        {"name": "decode batch", "op": "decode", "B": 16, "H": 16, "Hkv": 4, "D": 64, "page": 16, "min_len": 1,
         "max_len": 1023, "window": 0, "sinks": 0},
        # long caches, every row read, a key head for each query head
        {"name": "decode long", "op": "decode", "B": 16, "H": 12, "Hkv": 12, "D": 64, "page": 64, "min_len": 9000,
         "max_len": 32000, "window": 0, "sinks": 0},
        # the answers' log probabilities while a batch of 16 is decoded, with five alternatives
        {"name": "score token", "op": "score", "M": 16, "V": 50257, "K": 5, "bf16": False},
        # whole prompts scored
        {"name": "score prompts", "op": "score", "M": 4096, "V": 50257, "K": 8, "bf16": False},
        # the small vocabulary of the repository's MiniGPT configuration
        {"name": "learn small", "op": "learn", "M": 256, "V": 5000, "bf16": False},
        # a policy update's batch, logits in 16 bits
        {"name": "learn batch", "op": "learn", "M": 4096, "V": 50257, "bf16": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "turn", "park", "decode", "decode", "decode", "score", "score", "learn"])
    if op in ("score", "learn"):
        V = _log(rng, 200, 60000)
        M = max(1, min(_log(rng, 1, 4096), 150_000_000 // V))
        case = {"op": op, "M": M, "V": V, "bf16": rng.random() < 0.5}
        return case | ({"K": rng.choice([0, 1, 2, 5, 10, 20, 32])} if op == "score" else {})
    D = rng.choice([64, 64, 64, 32])
    Hkv = rng.choice([1, 2, 3, 4, 6, 8, 12])
    H = Hkv * rng.choice([1, 1, 2, 3, 4, 12])
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "decode":
        top = _log(rng, 16, 32000)
        B = max(1, min(_log(rng, 1, 128), 400000 // top))
        window = rng.choice([0, 0, _log(rng, 8, 4000)])
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "D": D, "page": page, "min_len": rng.randrange(0, top),
                "max_len": top, "window": window, "sinks": rng.choice([0, 4]) if window else 0}
    T = _log(rng, 1, 4000)
    B = max(1, min(_log(rng, 1, 64), 30_000_000 // (T * (H + 2 * Hkv) * D)))
    case = {"op": op, "B": B, "T": T, "H": H, "Hkv": Hkv, "D": D, "rot": rng.choice([D, D, D // 2]),
            "interleaved": rng.random() < 0.5}
    if op != "turn":
        case["page"] = page
    if op == "append":
        case["weights"] = rng.random() < 0.5
    return case


def _lens(case):
    """The sequences' lengths: spread evenly over [min_len, max_len] (which sequence has which goes by the seed)."""
    B, lo, hi = case["B"], case["min_len"], case["max_len"]
    return [hi if B == 1 else lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _counts(case):
    """New tokens of each sequence: between half of T and T."""
    B, T = case["B"], case["T"]
    return [T - (b * T) // (2 * B) for b in range(B)]


# ------------------------------------------------------------------------------------------ inputs

def _normal(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(torch.bfloat16)


def _pages(gen, B, max_pages, spare=3):
    """A page table whose sequences hold their pages in shuffled order, and the pool's page count."""
    n = B * max_pages + spare
    return torch.randperm(n, generator=gen, device="cuda")[: B * max_pages].to(torch.int32).view(B, max_pages), n


def _frequencies(rot):
    """Radians per position of each pair, and the same in 2^-64 turns as the framework takes it."""
    freq = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    turns = [round(f / (2.0 * math.pi) * 2.0 ** 64) % 2 ** 64 for f in freq]
    turns = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns]
    return torch.tensor(freq, dtype=torch.float64).cuda(), torch.tensor(turns, dtype=torch.int64).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, s = case["op"], dict(case)
    if op in ("score", "learn"):
        return _prepare_logits(s, gen)
    B, D, H, Hkv = case["B"], case["D"], case["H"], case["Hkv"]
    row = (H + 2 * Hkv) * D
    if op == "decode":
        page = case["page"]
        lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        s["lens"] = lens[torch.randperm(B, generator=gen, device="cuda")].contiguous()
        s["table"], n = _pages(gen, B, max(1, (case["max_len"] + page - 1) // page))
        s["qkv"] = _normal(gen, B, row, scale=1.5)
        s["codes"] = torch.empty(n, 2, Hkv, page, D // 2, dtype=torch.uint8, device="cuda")
        s["ranges"] = torch.empty(n, 2, Hkv, page, 2, dtype=torch.bfloat16, device="cuda")
        step = max(1, (1 << 27) // (2 * Hkv * page * D))
        for p in range(0, n, step):
            x = _normal(gen, min(step, n - p), 2, Hkv, page, D)
            s["codes"][p: p + step], s["ranges"][p: p + step] = _quantised(x)
        s["y"] = torch.zeros(B, H * D, dtype=torch.bfloat16, device="cuda")
        s["lse2"] = torch.zeros(B, H, dtype=torch.float32, device="cuda")
        return s
    T = case["T"]
    s["freq"], s["turns"] = _frequencies(case["rot"])
    s["qkv"] = _normal(gen, B, T, row)
    s["out"] = torch.zeros_like(s["qkv"])
    # where the text stands: further than the cache's rows, once rows have been evicted
    s["pos"] = torch.randint(0, 100000, (B,), generator=gen, device="cuda", dtype=torch.int32)
    if op == "turn":
        s["dout"] = _normal(gen, B, T, row, scale=0.25)
        s["dqkv"] = torch.zeros_like(s["qkv"])
        return s
    page = case["page"]
    # sequences continue behind what their pages hold already, and are shorter than the batch's T
    s["start"] = torch.randint(0, 2 * page, (B,), generator=gen, device="cuda", dtype=torch.int32)
    s["count"] = torch.tensor(_counts(case), dtype=torch.int32, device="cuda")
    s["table"], n = _pages(gen, B, (T + 2 * page + page - 1) // page)
    if op == "append":
        s["pool"] = _normal(gen, n, 2, Hkv, page, D)
        s["weight"] = torch.rand(n, Hkv, page, generator=gen, device="cuda") if case["weights"] else None
        return s
    s["codes"], s["ranges"] = _quantised(_normal(gen, n, 2, Hkv, page, D))
    s["rows"] = torch.zeros(B, T, 2 * Hkv * D, dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_logits(s, gen):
    M, V = s["M"], s["V"]
    # logits of a trained model: a wide spread, a few tokens far above, a constraint that rules some tokens out
    z = torch.randn(M, V, generator=gen, device="cuda").mul_(2.5).sub_(4.0)
    hot = torch.randint(0, V, (M, 8), generator=gen, device="cuda")
    z.scatter_add_(1, hot, torch.rand(M, 8, generator=gen, device="cuda") * 12.0)
    ruled_out = torch.rand(V, generator=gen, device="cuda") < 0.1
    z[::4] = z[::4].masked_fill(ruled_out, -math.inf)
    z = z.to(torch.bfloat16 if s["bf16"] else torch.float32)
    s["logits"] = z
    # the given tokens: drawn ones that were not ruled out
    cold = torch.argmax(torch.rand(V, generator=gen, device="cuda").masked_fill(ruled_out, -1.0))
    pick = torch.where(torch.rand(M, generator=gen, device="cuda") < 0.7, hot[:, 0], cold)
    s["targets"] = torch.where(ruled_out[pick], cold, pick).to(torch.int32)
    f32 = dict(dtype=torch.float32, device="cuda")
    s["logp"], s["entropy"] = torch.zeros(M, **f32), torch.zeros(M, **f32)
    if s["op"] == "score":
        s["top_ids"] = torch.zeros(M, s["K"], dtype=torch.int32, device="cuda") if s["K"] else None
        s["top_logp"] = torch.zeros(M, s["K"], **f32) if s["K"] else None
        return s
    s["stats"] = torch.zeros(M, 2, **f32)
    # advantages, and a bonus for entropy
    s["dlogp"] = torch.randn(M, generator=gen, device="cuda") / M
    s["dentropy"] = torch.full((M,), 0.01 / M, **f32)
    s["dlogits"] = torch.zeros_like(z)
    return s


# ------------------------------------------------------------------------------------------ one pass

def run(state):
    return {"append": _append, "turn": _turn, "park": _park, "decode": _decode, "score": _score,
            "learn": _learn}[state["op"]](state)


def _rotated(x, s, sign=1.0):
    """Queries and keys of x [B, T, (H + 2 Hkv) D] turned by their positions, in 32 bits; values as they are."""
    B, T, _ = x.shape
    H, Hkv, D, R = s["H"], s["Hkv"], s["D"], s["rot"]
    at = s["pos"].double()[:, None] + torch.arange(T, device="cuda")
    angle = at[:, :, None, None] * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float() * sign
    x = x.float().view(B, T, H + 2 * Hkv, D)
    y = x.clone()
    turned = x[:, :, : H + Hkv]
    a, b = (slice(0, R, 2), slice(1, R, 2)) if s["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
    y[:, :, : H + Hkv, a] = turned[..., a] * cos - turned[..., b] * sin
    y[:, :, : H + Hkv, b] = turned[..., b] * cos + turned[..., a] * sin
    return y


def _new_rows(s):
    """Sequence, token, page and slot of every new token, in one list each."""
    t = torch.arange(s["T"], device="cuda")[None, :]
    b, t = (t < s["count"][:, None]).nonzero(as_tuple=True)
    r = t + s["start"].long()[b]
    return b, t, s["table"].long()[b, r // s["page"]], r % s["page"]


def _append(s):
    pool, weight = s["pool"], s["weight"]
    if own:
        from decoder_only_transformer_gpt_gb300 import binding
        binding.paged_append(s["qkv"], pool, s["table"], s["H"], turns=s["turns"], start=s["start"], count=s["count"],
                             pos=s["pos"], weight=weight, out=s["out"], interleaved=s["interleaved"])
        return {"out": s["out"], "pool": pool} | ({"weight": weight} if s["weights"] else {})
    H, Hkv = s["H"], s["Hkv"]
    x = _rotated(s["qkv"], s).to(torch.bfloat16)
    b, t, pages, slots = _new_rows(s)
    s["out"][b, t] = x[b, t].flatten(1)
    pool[pages, 0, :, slots] = x[b, t, H: H + Hkv]
    pool[pages, 1, :, slots] = x[b, t, H + Hkv:]
    if weight is not None:
        weight[pages, :, slots] = 0.0
    return {"out": s["out"], "pool": pool} | ({"weight": weight} if s["weights"] else {})


def _turn(s):
    if own:
        from decoder_only_transformer_gpt_gb300 import binding
        binding.rotary(s["qkv"], s["out"], s["H"], s["Hkv"], s["turns"], pos=s["pos"], interleaved=s["interleaved"])
        binding.rotary(s["dout"], s["dqkv"], s["H"], s["Hkv"], s["turns"], pos=s["pos"], interleaved=s["interleaved"],
                       inverse=True)
        return {"out": s["out"], "dqkv": s["dqkv"]}
    shape = s["qkv"].shape
    return {"out": _rotated(s["qkv"], s).to(torch.bfloat16).view(shape),
            "dqkv": _rotated(s["dout"], s, sign=-1.0).to(torch.bfloat16).view(shape)}


def _quantised(x):
    """Codes (two to a byte) and (scale, lowest) of rows of D values."""
    x = x.float()
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((high - low) * (1.0 / 15.0)).to(torch.bfloat16).float()
    n = ((x - low) * torch.where(scale > 0, scale, torch.ones_like(scale)).reciprocal()).round().clamp_(max=15.0)
    n = torch.where(scale > 0, n, torch.zeros_like(n)).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4), torch.cat([scale, low], dim=-1).to(torch.bfloat16)


def _values(codes, ranges):
    """What codes and ranges stand for, in 32 bits."""
    n = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float()
    r = ranges.float()
    return r[..., 1:] + r[..., :1] * n


def _park(s):
    codes, ranges = s["codes"], s["ranges"]
    if own:
        from decoder_only_transformer_gpt_gb300 import binding
        binding.paged_append4(s["qkv"], codes, ranges, s["table"], s["H"], turns=s["turns"], start=s["start"],
                              count=s["count"], pos=s["pos"], out=s["out"], interleaved=s["interleaved"])
        binding.paged_load4(codes, ranges, s["table"], s["rows"], start=s["start"], count=s["count"])
        return {"out": s["out"], "rows": s["rows"]}
    H, Hkv = s["H"], s["Hkv"]
    x = _rotated(s["qkv"], s).to(torch.bfloat16)
    b, t, pages, slots = _new_rows(s)
    s["out"][b, t] = x[b, t].flatten(1)
    c, r = _quantised(x[b, t, H:])
    codes[pages, 0, :, slots], codes[pages, 1, :, slots] = c[:, :Hkv], c[:, Hkv:]
    ranges[pages, 0, :, slots], ranges[pages, 1, :, slots] = r[:, :Hkv], r[:, Hkv:]
    back = _values(codes[pages, :, :, slots], ranges[pages, :, :, slots])
    s["rows"][b, t] = back.flatten(1).to(torch.bfloat16)
    return {"out": s["out"], "rows": s["rows"]}


def _decode(s):
    if own:
        from decoder_only_transformer_gpt_gb300 import binding
        binding.paged_attention4(s["qkv"], s["codes"], s["ranges"], s["table"], s["lens"], s["y"], s["H"],
                                 lse2=s["lse2"], window=s["window"], sinks=s["sinks"])
        return {"y": s["y"], "lse2": s["lse2"]}
    B, H, Hkv, D, page = s["B"], s["H"], s["Hkv"], s["D"], s["page"]
    rows = torch.arange(s["max_len"], device="cuda")[None, :].expand(B, -1)
    pages, slots = torch.gather(s["table"].long(), 1, rows // page), rows % page
    n = s["lens"].long()[:, None]
    seen = rows < n
    if s["window"]:
        seen = seen & ((n - 1 - rows < s["window"]) | (rows < s["sinks"]))
    q = s["qkv"].float()[:, : H * D].view(B, Hkv, H // Hkv, D)
    # rows that are not seen hold what others left there: they are no numbers of this sequence
    keys = _values(s["codes"][pages, 0, :, slots], s["ranges"][pages, 0, :, slots]).permute(0, 2, 3, 1)
    values = _values(s["codes"][pages, 1, :, slots], s["ranges"][pages, 1, :, slots]).permute(0, 2, 1, 3)
    z = (q @ keys / math.sqrt(D)).masked_fill(~seen[:, None, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = (z - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp()
    total = p.sum(-1, keepdim=True)
    # a sequence of no rows: zeros, and a log-sum-exp of -inf
    y = (p @ values) / torch.where(total > 0, total, torch.ones_like(total))
    lse2 = (top + total.log()).squeeze(-1) * LOG2E
    return {"y": y.reshape(B, H * D).to(torch.bfloat16), "lse2": lse2.reshape(B, H)}


def _log_probabilities(z):
    """Largest logit, sum of exponentials against it, log probabilities and entropy, in 32 bits."""
    z = z.float()
    top = z.amax(-1, keepdim=True)
    d = z - top
    total = d.exp().sum(-1, keepdim=True)
    lp = d - total.log()
    p = lp.exp()
    entropy = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(-1)
    return top, total, lp, p, entropy


def _score(s):
    if own:
        from decoder_only_transformer_gpt_gb300 import binding
        binding.logprobs(s["logits"], s["targets"], s["logp"], entropy=s["entropy"], top_ids=s["top_ids"],
                         top_logp=s["top_logp"])
        return {"logp": s["logp"], "entropy": s["entropy"]} | (
            {"top_ids": s["top_ids"], "top_logp": s["top_logp"]} if s["K"] else {})
    _, _, lp, _, entropy = _log_probabilities(s["logits"])
    out = {"logp": lp.gather(1, s["targets"].long()[:, None]).squeeze(1), "entropy": entropy}
    if s["K"]:
        # equal logits: the lowest index first
        ids = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True).indices[:, : s["K"]]
        out |= {"top_ids": ids.to(torch.int32), "top_logp": lp.gather(1, ids)}
    return out


def _learn(s):
    if own:
        from decoder_only_transformer_gpt_gb300 import binding
        binding.logprobs(s["logits"], s["targets"], s["logp"], entropy=s["entropy"], stats=s["stats"])
        binding.logprobs_bwd(s["logits"], s["targets"], s["stats"], s["dlogp"], s["dlogits"], entropy=s["entropy"],
                             dentropy=s["dentropy"])
        return {"logp": s["logp"], "entropy": s["entropy"], "dlogits": s["dlogits"]}
    _, _, lp, p, entropy = _log_probabilities(s["logits"])
    at = s["targets"].long()[:, None]
    g, e = s["dlogp"][:, None], s["dentropy"][:, None]
    dz = -g * p - e * torch.where(p > 0, p * (lp + entropy[:, None]), torch.zeros_like(p))
    dz.scatter_add_(1, at, g)
    return {"logp": lp.gather(1, at).squeeze(1), "entropy": entropy, "dlogits": dz.to(s["logits"].dtype)}


# ------------------------------------------------------------------------------------------ what a pass needs

def work(case):
    op = case["op"]
    if op in ("score", "learn"):
        M, V, size = case["M"], case["V"], 2 if case["bf16"] else 4
        if op == "score":
            return {"bytes": M * (V * size + 12 + 8 * case["K"]), "flops": 6 * M * V}
        return {"bytes": M * (2 * V * size + 28), "flops": 12 * M * V}
    B, D, H, Hkv = case["B"], case["D"], case["H"], case["Hkv"]
    row = (H + 2 * Hkv) * D
    if op == "decode":
        W, S = case["window"], case["sinks"]
        rows = sum(n if W == 0 or W + S >= n else W + S for n in _lens(case))
        return {"bytes": rows * Hkv * (D + 8) + B * (4 * H * D + 4 * H), "flops": 4 * D * H * rows}
    if op == "turn":
        tokens = B * case["T"]
        return {"bytes": tokens * 8 * row, "flops": tokens * 6 * case["rot"] * (H + Hkv)}
    tokens = sum(_counts(case))
    turned = tokens * 3 * case["rot"] * (H + Hkv)
    if op == "append":
        return {"bytes": tokens * (4 * row + 4 * Hkv * D + (4 * Hkv if case["weights"] else 0)), "flops": turned}
    return {"bytes": tokens * (4 * row + 2 * Hkv * (D // 2 + 4) + 4 * Hkv * D), "flops": turned}


# ------------------------------------------------------------------------------------------ from the definitions

def exact(case, seed):
    """What run returns, in 64 bits from the definitions; None in the place of copies and of whole numbers."""
    s = prepare(case, seed)
    return {"append": _exact_rows, "turn": _exact_turn, "park": _exact_rows, "decode": _exact_decode,
            "score": _exact_logits, "learn": _exact_logits}[case["op"]](s)


def _exact_turned(x, s, sign):
    """Every pair as a complex number times e^(i angle), in 64 bits: [B, T, heads, D]."""
    B, T, _ = x.shape
    H, Hkv, D, R = s["H"], s["Hkv"], s["D"], s["rot"]
    y = x.double().reshape(B, T, H + 2 * Hkv, D).clone()
    heads = y[:, :, : H + Hkv, :R]
    pairs = heads.unflatten(-1, (R // 2, 2)) if s["interleaved"] else heads.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    at = torch.arange(T, device="cuda", dtype=torch.float64) + s["pos"][:, None]
    angle = torch.einsum("bt,i->bti", at, s["freq"])
    turn = torch.polar(torch.ones_like(angle), sign * angle)[:, :, None]
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y[:, :, : H + Hkv, :R] = z.flatten(-2) if s["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return y


def _exact_turn(s):
    return {"out": _exact_turned(s["qkv"], s, 1.0).flatten(2), "dqkv": _exact_turned(s["dout"], s, -1.0).flatten(2)}


def _exact_rows(s):
    x = _exact_turned(s["qkv"], s, 1.0)
    out = s["out"].double()
    H, Hkv = s["H"], s["Hkv"]
    parked = s["op"] == "park"
    rows = s["rows"].double() if parked else None
    for b, n in enumerate(s["count"].tolist()):
        out[b, :n] = x[b, :n].flatten(1)
        if parked:
            # the cache holds 16-bit keys and values in 4 bits: the nearest of 16 steps from the lowest value up
            v = x[b, :n, H:].to(torch.bfloat16).double()
            low = v.min(-1, keepdim=True).values
            step = ((v.max(-1, keepdim=True).values - low) / 15.0).to(torch.bfloat16).double()
            n_steps = torch.clamp(torch.round((v - low) / step), max=15.0)
            rows[b, :n] = (low + step * n_steps).flatten(1)
    if parked:
        return {"out": out, "rows": rows}
    return {"out": out, "pool": None} | ({"weight": None} if s["weights"] else {})


def _exact_decode(s):
    H, Hkv, D, page = s["H"], s["Hkv"], s["D"], s["page"]
    G, W, S = H // Hkv, s["window"], s["sinks"]
    table = s["table"].long()
    y = torch.zeros(s["B"], H * D, dtype=torch.float64, device="cuda")
    lse2 = torch.full((s["B"], H), -math.inf, dtype=torch.float64, device="cuda")

    def held(pages, slots, which, j):
        c = s["codes"][pages, which, j, slots].to(torch.int64)
        v = torch.empty(len(pages), D, dtype=torch.float64, device="cuda")
        v[:, 0::2], v[:, 1::2] = (c % 16).double(), (c // 16).double()
        r = s["ranges"][pages, which, j, slots].double()
        return v * r[:, :1] + r[:, 1:]

    for b, n in enumerate(s["lens"].tolist()):
        r = torch.arange(n, device="cuda")
        if W:
            r = r[(r >= n - W) | (r < S)]
        if not len(r):
            continue
        pages, slots = table[b, r // page], r % page
        for j in range(Hkv):
            q = s["qkv"][b, j * G * D: (j + 1) * G * D].double().view(G, D)
            z = torch.einsum("gd,sd->gs", q, held(pages, slots, 0, j)) * D ** -0.5
            lz = torch.logsumexp(z, 1)
            a = torch.exp(z - lz[:, None])
            y[b, j * G * D: (j + 1) * G * D] = torch.einsum("gs,sd->gd", a, held(pages, slots, 1, j)).reshape(-1)
            lse2[b, j * G: (j + 1) * G] = lz / math.log(2.0)
    return {"y": y, "lse2": lse2}


def _exact_logits(s):
    M, V, learn = s["M"], s["V"], s["op"] == "learn"
    f64 = dict(dtype=torch.float64, device="cuda")
    out = {"logp": torch.empty(M, **f64), "entropy": torch.empty(M, **f64)}
    if learn:
        out["dlogits"] = torch.empty(M, V, **f64)
    elif s["K"]:
        out["top_logp"] = torch.empty(M, s["K"], **f64)
    step = max(1, (1 << 26) // V)
    for m in range(0, M, step):
        z = s["logits"][m: m + step].double()
        lse = torch.logsumexp(z, -1)
        p = torch.softmax(z, -1)
        own_logp = z.gather(1, s["targets"][m: m + step].long()[:, None])[:, 0] - lse
        # entropy = log-sum-exp less the mean logit
        mean = torch.where(p > 0, p * z, torch.zeros_like(p)).sum(-1)
        out["logp"][m: m + step], out["entropy"][m: m + step] = own_logp, lse - mean
        if learn:
            one = torch.nn.functional.one_hot(s["targets"][m: m + step].long(), V)
            g, e = s["dlogp"][m: m + step].double()[:, None], s["dentropy"][m: m + step].double()[:, None]
            # d entropy / d z = p (mean logit - z)
            away = torch.where(p > 0, p * (mean[:, None] - z), torch.zeros_like(p))
            out["dlogits"][m: m + step] = g * (one - p) + e * away
        elif s["K"]:
            out["top_logp"][m: m + step] = torch.topk(z, s["K"]).values - lse[:, None]
    if not learn and s["K"]:
        out["top_ids"] = None
    return out
