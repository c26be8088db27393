"""Long-context serving and training operators: their plain forms, and the cases they are measured at.

Five operators that belong together:

  prompt   causal attention in which a query sees a sliding window of recent keys and the first few keys
           ("sinks"), over a whole prompt
  train    the same with its derivative, as a training step calls the pair
  store    a prompt's keys and values into a paged key/value cache
  decode   attention of one new token per sequence over the paged cache: stores the token's own key and
           value, then attends over the cached rows (all of them, or window and sinks), and can add every
           cached row's attention weight to a running sum
  evict    keep the rows of a cache with the largest summed weight (and the first and last ones), in order,
           in fewer pages

`run` computes them in elementary torch operations in 32 bits, or, where `own` is true, calls the framework.
"""
import math

import torch

own = False

LOG2E = 1.0 / math.log(2.0)


# ------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # a short prompt of the small character of the repository's MiniGPT configuration: latency
        {"name": "prompt short", "op": "prompt", "B": 1, "T": 200, "H": 4, "Hkv": 4, "D": 32, "window": 64, "sinks": 4},
        # GPT-2 small's batch of the repository's own benchmark, each query over 256 recent tokens
        {"name": "prompt batch", "op": "prompt", "B": 16, "T": 1024, "H": 12, "Hkv": 12, "D": 64, "window": 256,
         "sinks": 4},
        # one long document of an odd length, 25 heads of 64 sharing 5 key heads
        {"name": "prompt long", "op": "prompt", "B": 1, "T": 12001, "H": 25, "Hkv": 5, "D": 64, "window": 1500,
         "sinks": 4},
        # a training step's attention at GPT-2 small's shape, ragged against every tile
        {"name": "train batch", "op": "train", "B": 8, "T": 1000, "H": 12, "Hkv": 12, "D": 64, "window": 250,
         "sinks": 5},
        # long-context training with shared key heads
        {"name": "train long", "op": "train", "B": 1, "T": 8192, "H": 16, "Hkv": 4, "D": 64, "window": 1024,
         "sinks": 4},
        # one conversation, every cached row visible: latency
        {"name": "decode one", "op": "decode", "B": 1, "H": 12, "Hkv": 12, "D": 64, "page": 16, "min_len": 600,
         "max_len": 600, "window": 0, "sinks": 0, "weights": False},
        # a serving batch of ragged lengths that also sums the attention weights
        {"name": "decode batch", "op": "decode", "B": 16, "H": 12, "Hkv": 12, "D": 64, "page": 16, "min_len": 0,
         "max_len": 1023, "window": 0, "sinks": 0, "weights": True},
        # long caches, the whole length read
        {"name": "decode long", "op": "decode", "B": 16, "H": 12, "Hkv": 12, "D": 64, "page": 64, "min_len": 9000,
         "max_len": 32000, "window": 0, "sinks": 0, "weights": False},
        # a prompt batch into its pages
        {"name": "store batch", "op": "store", "B": 16, "T": 1024, "H": 12, "Hkv": 12, "D": 64, "page": 16},
        # a few short chunks appended behind what the pages hold
        {"name": "store chunk", "op": "store", "B": 3, "T": 77, "H": 16, "Hkv": 4, "D": 64, "page": 32},
        # halving a serving batch's caches
        {"name": "evict batch", "op": "evict", "B": 16, "Hkv": 12, "D": 64, "page": 16, "min_len": 500,
         "max_len": 1024, "budget": 512, "sinks": 4, "recent": 128},
        # long caches down to an eighth
        {"name": "evict long", "op": "evict", "B": 4, "Hkv": 12, "D": 64, "page": 64, "min_len": 10000,
         "max_len": 20000, "budget": 2500, "sinks": 4, "recent": 500},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "decode", "decode", "decode", "store", "evict"])
    D = rng.choice([64, 64, 64, 32])
    Hkv = rng.choice([1, 2, 3, 4, 6, 8, 12])
    H = Hkv * rng.choice([1, 1, 2, 3, 4])
    page = rng.choice([8, 16, 32, 64, 128])
    if op in ("prompt", "train"):
        T = _log(rng, 16, 8000 if op == "prompt" else 4000)
        B = max(1, min(_log(rng, 1, 32), 16000 // T, int(1.4e9 / (float(T) * T * H))))
        return {"op": op, "B": B, "T": T, "H": H, "Hkv": Hkv, "D": D, "window": _log(rng, 8, max(16, T)),
                "sinks": rng.choice([0, 1, 4, 4, 16])}
    if op == "decode":
        top = _log(rng, 16, 32000)
        B = max(1, min(_log(rng, 1, 128), 300000 // top))
        window = rng.choice([0, 0, _log(rng, 8, 4000)])
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "D": D, "page": page, "min_len": rng.randrange(0, top),
                "max_len": top, "window": window, "sinks": rng.choice([0, 4]) if window else 0,
                "weights": rng.random() < 0.4}
    if op == "store":
        T = _log(rng, 1, 4000)
        return {"op": op, "B": max(1, min(_log(rng, 1, 64), 16000 // T)), "T": T, "H": H, "Hkv": Hkv, "D": D,
                "page": page}
    top = _log(rng, 200, 20000)
    budget = rng.randrange(64, top)
    recent = rng.randrange(0, budget // 2)
    return {"op": op, "B": max(1, min(_log(rng, 1, 64), 80000 // top)), "Hkv": Hkv, "D": D, "page": page,
            "min_len": rng.randrange(top // 4, top), "max_len": top, "budget": budget, "sinks": rng.choice([0, 4, 16]),
            "recent": recent}


def _lens(case):
    """The sequences' lengths: spread evenly over [min_len, max_len] (which sequence has which goes by the seed)."""
    B, lo, hi = case["B"], case["min_len"], case["max_len"]
    return [hi if B == 1 else lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _visible(n, window, sinks):
    """How many of n cached rows the newest query sees."""
    return n if window == 0 or window + sinks >= n else window + sinks


# ------------------------------------------------------------------------------------------ inputs

def _normal(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(torch.bfloat16)


def _pages(gen, B, max_pages, spare=3):
    """A page table whose sequences hold their pages in shuffled order, and the pool's page count."""
    n = B * max_pages + spare
    return torch.randperm(n, generator=gen, device="cuda")[: B * max_pages].to(torch.int32).view(B, max_pages), n


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, B, D, Hkv = case["op"], case["B"], case["D"], case["Hkv"]
    s = dict(case)
    if op in ("prompt", "train"):
        T, H = case["T"], case["H"]
        s["qkv"] = _normal(gen, B, T, (H + 2 * Hkv) * D)
        s["y"] = torch.empty(B, T, H * D, dtype=torch.bfloat16, device="cuda")
        s["lse2"] = torch.empty(B, H, T, dtype=torch.float32, device="cuda")
        if op == "train":
            s["dy"] = _normal(gen, B, T, H * D, scale=0.25)
            s["dqkv"] = torch.empty_like(s["qkv"])
        return s
    page = case["page"]
    if op == "store":
        T = case["T"]
        # sequences continue behind what their pages hold already, and are shorter than the batch's T
        start = torch.randint(0, 2 * page, (B,), generator=gen, device="cuda", dtype=torch.int32)
        count = torch.tensor([T - (b * T) // (2 * B) for b in range(B)], dtype=torch.int32, device="cuda")
        s["start"], s["count"] = start, count
        s["qkv"] = _normal(gen, B, T, (case["H"] + 2 * Hkv) * D)
        s["table"], n = _pages(gen, B, (T + 2 * page + page - 1) // page)
        s["pool"] = _normal(gen, n, 2, Hkv, page, D)
        s["weight"] = torch.rand(n, Hkv, page, generator=gen, device="cuda")
        return s
    lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    s["lens"] = lens[torch.randperm(B, generator=gen, device="cuda")].contiguous()
    s["table"], n = _pages(gen, B, (case["max_len"] + 1 + page - 1) // page)
    if op == "decode":
        H = case["H"]
        s["qkv"] = _normal(gen, B, (H + 2 * Hkv) * D, scale=1.5)
        s["pool"] = _normal(gen, n, 2, Hkv, page, D)
        s["weight"] = torch.rand(n, Hkv, page, generator=gen, device="cuda") if case["weights"] else None
        s["y"] = torch.empty(B, H * D, dtype=torch.bfloat16, device="cuda")
        s["lse2"] = torch.empty(B, H, dtype=torch.float32, device="cuda")
        return s
    # evict: into pages of the same pool, as when another sequence still uses the old ones
    budget = case["budget"]
    more = (budget + page - 1) // page
    s["dst_table"] = torch.arange(n, n + B * more, dtype=torch.int32, device="cuda").view(B, more)
    n += B * more
    s["pool"] = _normal(gen, n, 2, Hkv, page, D)
    # summed weights are heavy-tailed, and some rows were never looked at
    w = torch.randn(n, Hkv, page, generator=gen, device="cuda").mul_(2.0).exp_()
    s["weight"] = torch.where(torch.rand(n, Hkv, page, generator=gen, device="cuda") < 0.1, torch.zeros_like(w), w)
    s["new_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
    s["kept"] = torch.empty(B, Hkv, budget, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------ one pass

def run(state):
    return {"prompt": _prompt, "train": _train, "decode": _decode, "store": _store, "evict": _evict}[state["op"]](state)


def _split(qkv, H, Hkv, D):
    """Queries [.., Hkv, G, T, D], keys and values [.., Hkv, 1, T, D] of [B, T, (H + 2 Hkv) D], in 32 bits."""
    B, T, _ = qkv.shape
    x = qkv.float()
    q = x[..., : H * D].view(B, T, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)
    k = x[..., H * D: (H + Hkv) * D].view(B, T, Hkv, 1, D).permute(0, 2, 3, 1, 4)
    u = x[..., (H + Hkv) * D:].view(B, T, Hkv, 1, D).permute(0, 2, 3, 1, 4)
    return q, k, u


def _seen(T, window, sinks):
    t = torch.arange(T, device="cuda")[:, None]
    s = torch.arange(T, device="cuda")[None, :]
    return (s <= t) & ((t - s < window) | (s < sinks))


def _softmax(scores, seen):
    """Probabilities over the seen keys and the log of their exponentials' sum."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - top).exp()
    total = p.sum(-1, keepdim=True)
    return p / total, (top + total.log()).squeeze(-1)


def _merged(x):
    """[B, Hkv, G, T, D] -> [B, T, Hkv G D]"""
    B, K, G, T, D = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(B, T, K * G * D)


def _prompt(s):
    if own:
        from decoder_only_transformer_gpt_gb300 import binding
        binding.attention_window(s["qkv"], s["y"], s["H"], s["Hkv"], s["window"], s["sinks"], lse2=s["lse2"])
        return {"y": s["y"], "lse2": s["lse2"]}
    B, T, H, Hkv, D = s["B"], s["T"], s["H"], s["Hkv"], s["D"]
    q, k, u = _split(s["qkv"], H, Hkv, D)
    p, lse = _softmax(q @ k.transpose(-1, -2) / math.sqrt(D), _seen(T, s["window"], s["sinks"]))
    return {"y": _merged(p @ u).to(torch.bfloat16), "lse2": (lse * LOG2E).reshape(B, H, T)}


def _train(s):
    if own:
        from decoder_only_transformer_gpt_gb300 import binding
        binding.attention_window(s["qkv"], s["y"], s["H"], s["Hkv"], s["window"], s["sinks"], lse2=s["lse2"])
        binding.attention_window_bwd(s["qkv"], s["y"], s["dy"], s["lse2"], s["dqkv"], s["H"], s["Hkv"], s["window"],
                                     s["sinks"])
        return {"y": s["y"], "lse2": s["lse2"], "dqkv": s["dqkv"]}
    B, T, H, Hkv, D = s["B"], s["T"], s["H"], s["Hkv"], s["D"]
    q, k, u = _split(s["qkv"], H, Hkv, D)
    p, lse = _softmax(q @ k.transpose(-1, -2) / math.sqrt(D), _seen(T, s["window"], s["sinks"]))
    y = p @ u
    dy = s["dy"].float().view(B, T, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)
    dp = dy @ u.transpose(-1, -2)
    ds = p * (dp - (dy * y).sum(-1, keepdim=True)) / math.sqrt(D)
    dq = ds @ k
    dk = (ds.transpose(-1, -2) @ q).sum(2, keepdim=True)
    du = (p.transpose(-1, -2) @ dy).sum(2, keepdim=True)
    dqkv = torch.cat([_merged(dq), _merged(dk), _merged(du)], dim=-1)
    return {"y": _merged(y).to(torch.bfloat16), "lse2": (lse * LOG2E).reshape(B, H, T), "dqkv": dqkv.to(torch.bfloat16)}


def _places(table, page, rows):
    """Page and slot of cache rows `rows` [B, n] of each sequence."""
    return torch.gather(table.long(), 1, rows // page), rows % page


def _store(s):
    pool, weight, page = s["pool"], s["weight"], s["page"]
    if own:
        from decoder_only_transformer_gpt_gb300 import binding
        binding.paged_store(s["qkv"], pool, s["table"], s["H"], start=s["start"], count=s["count"], weight=weight)
        return {"pool": pool, "weight": weight}
    B, T, H, Hkv, D = s["B"], s["T"], s["H"], s["Hkv"], s["D"]
    t = torch.arange(T, device="cuda")[None, :]
    b, t = (t < s["count"][:, None]).nonzero(as_tuple=True)
    row = t + s["start"].long()[b]
    pages, slots = s["table"].long()[b, row // page], row % page
    pool[pages, 0, :, slots] = s["qkv"][b, t, H * D: (H + Hkv) * D].view(-1, Hkv, D)
    pool[pages, 1, :, slots] = s["qkv"][b, t, (H + Hkv) * D:].view(-1, Hkv, D)
    weight[pages, :, slots] = 0.0
    return {"pool": pool, "weight": weight}


def _decode(s):
    pool, weight, page, lens = s["pool"], s["weight"], s["page"], s["lens"]
    if own:
        from decoder_only_transformer_gpt_gb300 import binding
        binding.paged_attention(s["qkv"], pool, s["table"], lens, s["y"], s["H"], lse2=s["lse2"], weight=weight,
                                window=s["window"], sinks=s["sinks"])
        return {"y": s["y"], "lse2": s["lse2"], "pool": pool} | ({"weight": weight} if s["weights"] else {})
    B, H, Hkv, D = s["B"], s["H"], s["Hkv"], s["D"]
    q, k, u = _split(s["qkv"][:, None], H, Hkv, D)                       # [B, Hkv, G, 1, D]
    pages, slots = _places(s["table"], page, lens.long()[:, None])
    pool[pages[:, 0], 0, :, slots[:, 0]] = k[:, :, 0, 0].to(pool.dtype)
    pool[pages[:, 0], 1, :, slots[:, 0]] = u[:, :, 0, 0].to(pool.dtype)
    rows = torch.arange(s["max_len"] + 1, device="cuda")[None, :].expand(B, -1)
    pages, slots = _places(s["table"], page, rows)
    keys = pool[pages, 0, :, slots].float().permute(0, 2, 3, 1)          # [B, Hkv, D, n]
    values = pool[pages, 1, :, slots].float().permute(0, 2, 1, 3)        # [B, Hkv, n, D]
    last = lens.long()[:, None]
    seen = rows <= last
    if s["window"]:
        seen = seen & ((last - rows < s["window"]) | (rows < s["sinks"]))
    p, lse = _softmax(q[:, :, :, 0] @ keys / math.sqrt(D), seen[:, None, None, :])
    y = (p @ values).reshape(B, H * D).to(torch.bfloat16)
    out = {"y": y, "lse2": (lse * LOG2E).reshape(B, H), "pool": pool}
    if s["weights"]:
        w = weight[pages, :, slots]                                      # [B, n, Hkv]
        w = torch.where((rows == last)[..., None], torch.zeros_like(w), w) + p.sum(2).permute(0, 2, 1)
        b, n = (rows <= last).nonzero(as_tuple=True)
        weight[pages[b, n], :, slots[b, n]] = w[b, n]
        out["weight"] = weight
    return out


def _evict(s):
    pool, weight, page, lens = s["pool"], s["weight"], s["page"], s["lens"]
    budget, sinks, recent = s["budget"], s["sinks"], s["recent"]
    if own:
        from decoder_only_transformer_gpt_gb300 import binding
        binding.paged_evict(pool, weight, s["table"], lens, s["dst_table"], s["new_lens"], s["kept"], budget,
                            sinks=sinks, recent=recent)
        return {"pool": pool, "weight": weight, "new_lens": s["new_lens"], "kept": s["kept"]}
    B, Hkv = s["B"], s["Hkv"]
    rows = torch.arange(s["max_len"], device="cuda")[None, :].expand(B, -1)
    pages, slots = _places(s["table"], page, rows)
    n = lens.long()[:, None]
    w = weight[pages, :, slots].permute(0, 2, 1)                         # [B, Hkv, n]
    sure = ((rows < sinks) | (rows >= n - recent)) & (rows < n)
    w = w.masked_fill(sure[:, None], math.inf).masked_fill((rows >= n)[:, None], -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices  # equal weights: the lowest row first
    kept = order[..., : min(budget, s["max_len"])]
    new = torch.minimum(lens, torch.full_like(lens, budget))
    kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[-1]), value=1 << 30)
    at = torch.arange(budget, device="cuda")
    alive = at < new.long()[:, None, None]
    kept = kept.masked_fill(~alive, 1 << 30).sort(-1).values             # in the order of the rows
    b, h, i = (kept < (1 << 30)).nonzero(as_tuple=True)
    r = kept[b, h, i]
    src, src_slot = s["table"].long()[b, r // page], r % page
    dst, dst_slot = s["dst_table"].long()[b, i // page], i % page
    pool[dst, :, h, dst_slot] = pool[src, :, h, src_slot]
    weight[dst, h, dst_slot] = weight[src, h, src_slot]
    kept = kept.masked_fill(~alive, -1).to(torch.int32)
    return {"pool": pool, "weight": weight, "new_lens": new, "kept": kept}


# ------------------------------------------------------------------------------------------ what a pass needs

def work(case):
    op, B, D, Hkv = case["op"], case["B"], case["D"], case["Hkv"]
    if op in ("prompt", "train"):
        T, H, W, S = case["T"], case["H"], case["window"], case["sinks"]
        pairs = sum(_visible(t + 1, W, S) for t in range(T)) * B * H
        row = (H + 2 * Hkv) * D
        moved = B * T * (2 * row + 2 * H * D + 4 * H)
        if op == "prompt":
            return {"bytes": moved, "flops": 4.0 * D * pairs}
        # forward 2 products, derivative 5 (the scores once more, dP, dQ, dK, dU); reads dy, writes dqkv
        return {"bytes": moved + B * T * (2 * H * D + 2 * row), "flops": 14.0 * D * pairs}
    if op == "store":
        T = case["T"]
        rows = sum(T - (b * T) // (2 * B) for b in range(B))
        return {"bytes": rows * Hkv * (8 * D + 4), "flops": 0}
    lens = _lens(case)
    if op == "decode":
        H = case["H"]
        rows = sum(_visible(n + 1, case["window"], case["sinks"]) for n in lens)
        moved = 4 * D * Hkv * (rows + B) + B * (2 * (H + 2 * Hkv) * D + 2 * H * D + 4 * H)
        return {"bytes": moved + (8 * Hkv * rows if case["weights"] else 0), "flops": 4.0 * D * H * rows}
    kept = sum(min(n, case["budget"]) for n in lens)
    return {"bytes": Hkv * (4 * sum(lens) + kept * (8 * D + 4) + 4 * B * case["budget"]), "flops": 0}


# ------------------------------------------------------------------------------------------ from the definitions

def exact(case, seed):
    """What run returns, in 64 bits, query by query and head by head from the definitions. The cache itself holds
    copies, no computed numbers: None in its place, and for the operators that only move rows."""
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    if op in ("store", "evict"):
        return None
    s = prepare(case, seed)
    H, W, S = case["H"], case["window"], case["sinks"]
    G = H // Hkv
    if op == "decode":
        return _exact_decode(s, H, Hkv, G, D, W, S)
    B, T = case["B"], case["T"]
    x = s["qkv"].double()
    y = torch.empty(B, T, H * D, dtype=torch.float64, device="cuda")
    lse2 = torch.empty(B, H, T, dtype=torch.float64, device="cuda")
    grad = torch.zeros_like(x) if op == "train" else None
    step = 512
    for b in range(B):
        for h in range(H):
            qc, kc, uc = h * D, (H + h // G) * D, (H + Hkv + h // G) * D
            for t0 in range(0, T, step):
                t1 = min(T, t0 + step)
                first = max(0, t0 - W + 1)
                idx = torch.cat([torch.arange(0, min(S, first), device="cuda"), torch.arange(first, t1, device="cuda")])
                t = torch.arange(t0, t1, device="cuda")[:, None]
                ok = (idx[None] <= t) & ((idx[None] > t - W) | (idx[None] < S))
                q, k, u = x[b, t0:t1, qc: qc + D], x[b, idx, kc: kc + D], x[b, idx, uc: uc + D]
                z = torch.where(ok, torch.einsum("td,sd->ts", q, k) * D ** -0.5, torch.full((), -math.inf, device="cuda",
                                                                                           dtype=torch.float64))
                lz = torch.logsumexp(z, 1)
                a = torch.exp(z - lz[:, None])
                o = torch.einsum("ts,sd->td", a, u)
                y[b, t0:t1, qc: qc + D] = o
                lse2[b, h, t0:t1] = lz / math.log(2.0)
                if grad is not None:
                    g = s["dy"][b, t0:t1, qc: qc + D].double()
                    da = torch.einsum("td,sd->ts", g, u)
                    dz = a * (da - torch.einsum("ts,ts->t", a, da)[:, None]) * D ** -0.5
                    grad[b, t0:t1, qc: qc + D] = torch.einsum("ts,sd->td", dz, k)
                    grad[b, :, kc: kc + D].index_add_(0, idx, torch.einsum("ts,td->sd", dz, q))
                    grad[b, :, uc: uc + D].index_add_(0, idx, torch.einsum("ts,td->sd", a, g))
    out = {"y": y, "lse2": lse2}
    return out | ({"dqkv": grad} if grad is not None else {})


def _exact_decode(s, H, Hkv, G, D, W, S):
    pool, table, page = s["pool"], s["table"].long(), s["page"]
    lens = s["lens"].tolist()
    y = torch.empty(s["B"], H * D, dtype=torch.float64, device="cuda")
    lse2 = torch.empty(s["B"], H, dtype=torch.float64, device="cuda")
    weight = s["weight"].double() if s["weights"] else None
    for b, n in enumerate(lens):
        r = torch.arange(n + 1, device="cuda")
        if W:
            r = r[(r > n - W) | (r < S)]
        pg, sl = table[b, r // page], r % page
        new = s["qkv"][b].double()
        if weight is not None:
            weight[table[b, n // page], :, n % page] = 0.0
        for j in range(Hkv):
            k, u = pool[pg, 0, j, sl].double(), pool[pg, 1, j, sl].double()
            k[-1], u[-1] = new[(H + j) * D: (H + j + 1) * D], new[(H + Hkv + j) * D: (H + Hkv + j + 1) * D]
            q = new[j * G * D: (j + 1) * G * D].view(G, D)
            z = torch.einsum("gd,sd->gs", q, k) * D ** -0.5
            lz = torch.logsumexp(z, 1)
            a = torch.exp(z - lz[:, None])
            y[b, j * G * D: (j + 1) * G * D] = torch.einsum("gs,sd->gd", a, u).reshape(-1)
            lse2[b, j * G: (j + 1) * G] = lz / math.log(2.0)
            if weight is not None:
                weight[pg, j, sl] += a.sum(0)
    out = {"y": y, "lse2": lse2, "pool": None}
    return out | ({"weight": weight} if weight is not None else {})
