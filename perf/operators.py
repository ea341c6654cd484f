"""The operators of a decode step around the quantized linears, as they are measured.

Each case is one call (one launch or a few) of one operator, at sizes from a
single new token to long prompts, long caches and whole evaluation batches:

  norm      residual sum, gate and RMS norms before / after a block
  rope      rotary positions of q and k, k and v appended to the paged cache
  pages     block tables, slot maps and the free pages from the lengths
  attend    attention of one new token per sequence over the paged cache
  logprobs  log probabilities, rank, entropy and top alternatives of logits

With `own` false, run() computes them in elementary torch operations in 32 bits;
with it true, through this package.  exact() is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5


# ---- the cases -------------------------------------------------------------------

def listed():
    return [
        # one new token at the smallest hidden size here, fp32 as the linears have it
        {"name": "norm_token", "op": "norm", "tokens": 1, "width": 960, "act": "f32", "res": "f32",
         "post": False, "gate": "none", "alpha": 1.0},
        # a long prompt: norm after the block, gate for each element, scaled residual in fp32
        {"name": "norm_prompt", "op": "norm", "tokens": 8192, "width": 2048, "act": "bf16", "res": "f32",
         "post": True, "gate": "all", "alpha": 0.22},
        # four sequences' new tokens, fp32 from the linears, bf16 cache
        {"name": "rope_token", "op": "rope", "tokens": 4, "q_heads": 15, "kv_heads": 5, "dim": 64, "rot": 64,
         "inter": False, "act": "f32", "cache": "bf16", "page": 16, "start": 2000, "scale": 1.0},
        # a prompt late in a long context: interleaved pairs, half of the head rotated
        {"name": "rope_prompt", "op": "rope", "tokens": 16384, "q_heads": 16, "kv_heads": 2, "dim": 128, "rot": 64,
         "inter": True, "act": "bf16", "cache": "bf16", "page": 64, "start": 98304, "scale": 1.07},
        # every sequence of a decode batch grows by one token, a few end
        {"name": "pages_decode", "op": "pages", "seqs": 64, "page": 16, "longest": 4096, "grow": 1, "ending": 0.1,
         "tokens": 64},
        # prompts of many lengths admitted at once, chunks of long ones continued
        {"name": "pages_prompts", "op": "pages", "seqs": 509, "page": 16, "longest": 8192, "grow": 1000, "ending": 0.05,
         "tokens": 524288},
        # one sequence, a few pages: latency
        {"name": "attend_short", "op": "attend", "seqs": 1, "q_heads": 15, "kv_heads": 5, "dim": 64, "page": 16,
         "longest": 613, "ragged": False, "window": 0, "act": "f32", "cache": "bf16"},
        # one sequence with a long cache: the length has to be split over the GPU
        {"name": "attend_long", "op": "attend", "seqs": 1, "q_heads": 16, "kv_heads": 2, "dim": 128, "page": 64,
         "longest": 131072, "ragged": False, "window": 0, "act": "f32", "cache": "bf16"},
        # a serving batch of very different lengths
        {"name": "attend_batch", "op": "attend", "seqs": 384, "q_heads": 32, "kv_heads": 4, "dim": 64, "page": 16,
         "longest": 8192, "ragged": True, "window": 0, "act": "bf16", "cache": "bf16"},
        # the next token of one sequence, fp32 logits from the lm_head
        {"name": "logprobs_token", "op": "logprobs", "tokens": 1, "vocab": 151936, "act": "f32", "top": 20, "masked": 0.0},
        # a small batch over a vocabulary of odd size, part of it masked
        {"name": "logprobs_batch", "op": "logprobs", "tokens": 37, "vocab": 32003, "act": "f32", "top": 5, "masked": 0.2},
        # scoring of whole texts
        {"name": "logprobs_score", "op": "logprobs", "tokens": 2048, "vocab": 151936, "act": "bf16", "top": 8,
         "masked": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "pages", "attend", "logprobs"])
    act = rng.choice(["f32", "bf16", "f16"])
    if op == "norm":
        width = _log(rng, 576, 8192) if rng.random() < 0.3 else 64 * _log(rng, 9, 128)
        return {"op": op, "tokens": _log(rng, 1, 8192 * 2048 // width), "width": width, "act": act,
                "res": rng.choice(["f32", act]), "post": rng.random() < 0.5,
                "gate": rng.choice(["none", "row", "all"]), "alpha": round(rng.uniform(0.1, 1.0), 3)}
    kv = rng.choice([1, 2, 3, 4, 5, 8])
    q = kv * rng.choice([1, 2, 3, 4, 6, 8, 12])
    dim = rng.choice([64, 80, 96, 128, 128, 256])
    page = rng.choice([16, 16, 24, 32, 64, 128])
    cache = act if act != "f32" else rng.choice(["bf16", "f16"])
    if op == "rope":
        return {"op": op, "tokens": _log(rng, 1, 16384 * 20 * 128 // ((q + 2 * kv) * dim)), "q_heads": q, "kv_heads": kv,
                "dim": dim, "rot": rng.choice([dim, dim // 2]), "inter": rng.random() < 0.5, "act": act, "cache": cache,
                "page": page, "start": _log(rng, 1, 1000000), "scale": 1.0}
    if op == "pages":
        seqs, grow = _log(rng, 1, 512), rng.choice([1, 1, _log(rng, 2, 1000)])
        return {"op": op, "seqs": seqs, "page": page, "longest": _log(rng, 16, 8192), "grow": grow,
                "ending": rng.choice([0.0, 0.1]), "tokens": max(1, seqs * grow)}
    if op == "attend":
        seqs = _log(rng, 1, 256)
        longest = _log(rng, 1, max(1, min(131072, 384 * 1024 * 4 * 64 // (seqs * kv * dim))))
        return {"op": op, "seqs": seqs, "q_heads": q, "kv_heads": kv, "dim": dim, "page": page, "longest": longest,
                "ragged": rng.random() < 0.6, "window": rng.choice([0, 0, 0, 1024]), "act": act, "cache": cache}
    vocab = _log(rng, 1000, 151936)
    return {"op": op, "tokens": _log(rng, 1, max(1, 2048 * 151936 // (vocab * (2 if act == "f32" else 1)))), "vocab": vocab,
            "act": act, "top": rng.choice([0, 1, 5, 20]), "masked": rng.choice([0.0, 0.1])}


def _lengths(case):
    """Cache lengths of an attend case: the same for every seed, so that the work is the case's."""
    n, top = case["seqs"], case["longest"]
    if not case["ragged"]:
        return [top] * n
    # log-uniform from 1 to the longest, in an order that mixes them
    return [int(round(top ** (((i * 0.6180339887) % 1.0)))) if i else top for i in range(n)]


def _attended(case):
    w = case["window"]
    return [min(x, w) if w else x for x in _lengths(case)]


def work(case):
    op = case["op"]
    if op == "norm":
        t, c, a, r = case["tokens"], case["width"], SIZE[case["act"]], SIZE[case["res"]]
        gate = {"none": 0, "row": c * a, "all": t * c * a}[case["gate"]]
        return {"bytes": t * c * (2 * a + 2 * r) + gate + 4 * c * (2 if case["post"] else 1), "flops": 10 * t * c}
    if op == "rope":
        t, d, a, s = case["tokens"], case["dim"], SIZE[case["act"]], SIZE[case["cache"]]
        q, kv = case["q_heads"], case["kv_heads"]
        return {"bytes": t * d * (2 * q * a + 2 * kv * (a + s)) + 8 * t + 4 * case["rot"],
                "flops": 6 * t * (q + kv) * case["rot"] // 2}
    if op == "pages":
        return {"bytes": 12 * case["tokens"] + 20 * case["seqs"] + 8 * (case["tokens"] // case["page"]), "flops": 0}
    if op == "attend":
        keys, b, d = sum(_attended(case)), case["seqs"], case["dim"]
        return {"bytes": 2 * keys * case["kv_heads"] * d * SIZE[case["cache"]] + 2 * b * case["q_heads"] * d * SIZE[case["act"]]
                + 4 * sum(-(-x // case["page"]) for x in _attended(case)) + 4 * b,
                "flops": 4 * keys * case["q_heads"] * d}
    t, v, k = case["tokens"], case["vocab"], case["top"]
    return {"bytes": t * v * SIZE[case["act"]] + t * (16 + 8 * k), "flops": 6 * t * v}


# ---- inputs ----------------------------------------------------------------------

def _turns(rot, base=1000000.0):
    """Turns per position of each rotated pair, in units of 2^-64."""
    at = torch.arange(0, rot, 2, dtype=torch.float64) / rot
    return (torch.pow(torch.tensor(base, dtype=torch.float64), -at) / (2 * math.pi) * 2.0 ** 64).to(torch.int64)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    def ints(lo, hi, n):
        return torch.randint(lo, hi, (n,), generator=g, device=dev, dtype=torch.int32)

    op, s = case["op"], {"case": case}
    if op == "norm":
        t, c, act, res = case["tokens"], case["width"], DTYPES[case["act"]], DTYPES[case["res"]]
        s["x"], s["h"] = normal(t, c, dtype=act), normal(t, c, dtype=res, std=3.0)
        s["w"] = 1 + normal(c, std=0.1)
        s["post_w"] = 1 + normal(c, std=0.1) if case["post"] else None
        s["gate"] = None if case["gate"] == "none" else normal(1 if case["gate"] == "row" else t, c, dtype=act)
        s["h_out"], s["y"] = torch.empty_like(s["h"]), torch.empty_like(s["x"])
    elif op == "rope":
        t, d, q, kv, page = case["tokens"], case["dim"], case["q_heads"], case["kv_heads"], case["page"]
        act, cache = DTYPES[case["act"]], DTYPES[case["cache"]]
        s["q"], s["k"], s["v"] = normal(t, q, d, dtype=act), normal(t, kv, d, dtype=act), normal(t, kv, d, dtype=act)
        s["positions"] = torch.arange(t, device=dev, dtype=torch.int32) + case["start"]
        pages = -(-t // page) + 3
        order = torch.randperm(pages, generator=g, device=dev)
        at = torch.arange(t, device=dev)
        s["slots"] = (order[at // page] * page + at % page).to(torch.int32)
        s["turns"] = _turns(case["rot"]).to(dev)
        s["q_out"] = torch.empty_like(s["q"])
        s["k_cache"] = torch.zeros((pages, page, kv, d), device=dev, dtype=cache)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
    elif op == "pages":
        n, page, grow = case["seqs"], case["page"], case["grow"]
        lens = ints(0, case["longest"] + 1, n)
        more = torch.full((n,), 1, device=dev, dtype=torch.int32) if grow == 1 else ints(0, grow + 1, n)
        ends = torch.rand((n,), generator=g, device=dev) < case["ending"]
        s["lens"], s["targets"] = lens, torch.where(ends, torch.zeros_like(lens), lens + more)
        width = -(-(case["longest"] + grow) // page)
        pool = n * width + 64
        order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        s["table"] = order[: n * width].reshape(n, width).contiguous()
        used = (torch.arange(width, device=dev)[None] < ((lens + page - 1) // page)[:, None]).reshape(-1)
        # pages of no sequence, in a ring that begins somewhere in its buffer
        free = torch.cat([order[: n * width][~used], order[n * width:]])
        head = int(torch.randint(0, pool, (1,), generator=g, device=dev))
        s["ring"] = torch.zeros((pool,), device=dev, dtype=torch.int32)
        s["ring"][(torch.arange(free.numel(), device=dev) + head) % pool] = free
        s["ring_state"] = torch.tensor([head, free.numel()], device=dev, dtype=torch.int32)
        s["ring_state_out"] = torch.zeros_like(s["ring_state"])
        s["lens_out"] = torch.zeros_like(lens)
        s["status"] = torch.zeros_like(lens)
        s["starts"] = torch.zeros((n + 1,), device=dev, dtype=torch.int32)
        s["slots"], s["positions"], s["token_seqs"] = (torch.zeros((case["tokens"],), device=dev, dtype=torch.int32)
                                                       for _ in range(3))
    elif op == "attend":
        n, d, q, kv, page = case["seqs"], case["dim"], case["q_heads"], case["kv_heads"], case["page"]
        act, cache = DTYPES[case["act"]], DTYPES[case["cache"]]
        lens = _lengths(case)
        need = [-(-x // page) for x in lens]
        pool = sum(need) + 5
        s["q"] = normal(n, q, d, dtype=act, std=2.0)
        s["k_cache"], s["v_cache"] = normal(pool, page, kv, d, dtype=cache), normal(pool, page, kv, d, dtype=cache)
        order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        width = max(need)
        first = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
        at = torch.arange(width, device=dev)
        have = at[None] < torch.tensor(need, device=dev)[:, None]
        s["table"] = torch.where(have, order[torch.where(have, first[:, None] + at[None], 0)], -1).to(torch.int32)
        s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((n, q), device=dev)
    else:
        t, v, k = case["tokens"], case["vocab"], case["top"]
        x = normal(t, v, dtype=DTYPES[case["act"]], std=2.5)
        s["ids"] = ints(0, v, t)
        if case["masked"]:
            hide = torch.rand((v,), generator=g, device=dev) < case["masked"]
            x.masked_fill_(hide[None], -math.inf)
        s["logits"] = x
        s["logprobs"], s["entropy"] = torch.empty((t,), device=dev), torch.empty((t,), device=dev)
        s["ranks"] = torch.empty((t,), device=dev, dtype=torch.int32)
        s["top_ids"] = torch.empty((t, k), device=dev, dtype=torch.int32) if k else None
        s["top_logprobs"] = torch.empty((t, k), device=dev) if k else None
    return s


# ---- one pass --------------------------------------------------------------------

def _norm_plain(s):
    x, h = s["x"].float(), s["h"].float()
    if s["post_w"] is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["post_w"]
    if s["gate"] is not None:
        x = x * s["gate"].float()
    h = h + s["case"]["alpha"] * x
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"]
    return {"h": h.to(s["h"].dtype), "y": y.to(s["x"].dtype)}


def _rope_plain(s):
    case = s["case"]
    rot, kv, d = case["rot"], case["kv_heads"], case["dim"]
    # whole turns drop out of the 64-bit product; the upper half is the angle
    turn = (s["positions"].long()[:, None] * s["turns"][None]) >> 32
    angle = turn.float() * (2 * math.pi / 2 ** 32)
    cos, sin = torch.cos(angle)[:, None] * case["scale"], torch.sin(angle)[:, None] * case["scale"]

    def rotated(x):
        x = x.float()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        u, v = a * cos - b * sin, a * sin + b * cos
        both = torch.stack([u, v], -1).flatten(-2) if case["inter"] else torch.cat([u, v], -1)
        return torch.cat([both, x[..., rot:]], -1)

    at = s["slots"].long()
    s["k_cache"].view(-1, kv, d)[at] = rotated(s["k"]).to(s["k_cache"].dtype)
    s["v_cache"].view(-1, kv, d)[at] = s["v"].to(s["v_cache"].dtype)
    return {"q": rotated(s["q"]).to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _pages_plain(s):
    # the inputs here always fit; every sequence grows, shrinks or stays
    page, pool = s["case"]["page"], s["ring"].numel()
    lens, targets, table = s["lens"].long(), s["targets"].long(), s["table"]
    n, width = table.shape
    had, have = (lens + page - 1) // page, (targets + page - 1) // page
    taken, given = (have - had).clamp(min=0), (had - have).clamp(min=0)
    take_from, give_to = taken.cumsum(0) - taken, given.cumsum(0) - given
    head, count = s["ring_state"].long()[0], s["ring_state"].long()[1]
    col = torch.arange(width, device=table.device)[None]
    ring = s["ring"]
    fresh = ring[((head + take_from[:, None] + col - had[:, None]) % pool)]
    table.copy_(torch.where((col >= had[:, None]) & (col < have[:, None]), fresh, table))
    back = torch.where((col >= have[:, None]) & (col < had[:, None]), (head + count + give_to[:, None] + col - have[:, None]) % pool, pool)
    wide = torch.cat([ring, ring[:1]])
    wide.index_put_((back.reshape(-1),), table.reshape(-1))
    ring.copy_(wide[:pool])
    new = (targets - lens).clamp(min=0)
    ends = new.cumsum(0)
    starts = torch.cat([ends.new_zeros(1), ends])
    tok = torch.arange(s["case"]["tokens"], device=table.device)
    seq = torch.searchsorted(ends, tok, right=True)
    real = seq < n
    seq = seq.clamp(max=n - 1)
    pos = lens[seq] + tok - starts[seq]
    slot = table[seq, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    state = torch.stack([(head + taken.sum()) % pool, count - taken.sum() + given.sum()])
    i32 = torch.int32
    return {"table": table, "ring": ring, "ring_state": state.to(i32), "lens": targets.to(i32), "status": torch.zeros_like(s["lens"]),
            "starts": starts.to(i32), "slots": torch.where(real, slot, -1).to(i32),
            "positions": torch.where(real, pos, 0).to(i32), "token_seqs": torch.where(real, seq, -1).to(i32)}


def _attend_plain(s):
    case = s["case"]
    n, q, d = s["q"].shape
    page, kv = case["page"], case["kv_heads"]
    at = torch.arange(s["table"].shape[1] * page, device=s["q"].device)
    where = s["table"].long()[:, at // page] * page + (at % page)[None]
    keys, values = s["k_cache"].view(-1, kv, d)[where].float(), s["v_cache"].view(-1, kv, d)[where].float()
    x = s["q"].float().view(n, kv, q // kv, d) / math.sqrt(d)
    score = torch.einsum("ngrd,nlgd->ngrl", x, keys)
    lens = s["lens"].long()[:, None]
    seen = at[None] < lens
    if case["window"]:
        seen = seen & (at[None] >= lens - case["window"])
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    out = torch.einsum("ngrl,nlgd->ngrd", e, values) / total
    return {"out": out.reshape(n, q, d).to(s["q"].dtype), "lse": (top + torch.log(total)).reshape(n, q)}


def _logprobs_plain(s):
    raw, k = s["logits"].float(), s["case"]["top"]
    top = raw.amax(-1, keepdim=True)
    d = raw - top
    e = torch.exp(d)
    total = e.sum(-1)
    log_total = torch.log(total)
    mine = torch.gather(raw, 1, s["ids"].long()[:, None])
    out = {"logprobs": (mine - top)[:, 0] - log_total,
           "ranks": (raw > mine).sum(-1).to(torch.int32),
           "entropy": log_total - (e * d.clamp(min=-200.0)).sum(-1) / total}
    if k:
        # descending values, ties to the lowest index, as one whole number each
        bits = (raw + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        key = (order << 32) + (2 ** 31 - torch.arange(raw.shape[1], device=raw.device))
        ids = 2 ** 31 - (torch.topk(key, k, -1).values & 0xFFFFFFFF)
        best = torch.gather(raw, 1, ids)
        out["top_ids"] = torch.where(best == -math.inf, -1, ids).to(torch.int32)
        out["top_logprobs"] = best - top - log_total[:, None]
    return out


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"norm": _norm_plain, "rope": _rope_plain, "pages": _pages_plain, "attend": _attend_plain,
                "logprobs": _logprobs_plain}[op](s)
    from block_quantized_weight_dot_gb300 import lean
    case = s["case"]
    if op == "norm":
        lean.lean_residual_norm(s["x"], s["h"], s["w"], s["h_out"], s["y"], eps=EPS, post_w=s["post_w"], gate=s["gate"],
                                res_scale=case["alpha"])
        return {"h": s["h_out"], "y": s["y"]}
    if op == "rope":
        lean.lean_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["turns"], s["q_out"], s["k_cache"],
                              s["v_cache"], rot_dim=case["rot"], interleaved=case["inter"], rot_scale=case["scale"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "pages":
        lean.lean_kv_pages(s["lens"], s["targets"], s["table"], s["ring"], s["ring_state"], case["page"], s["lens_out"],
                           s["ring_state_out"], s["status"], s["starts"], s["slots"], s["positions"], s["token_seqs"])
        return {"table": s["table"], "ring": s["ring"], "ring_state": s["ring_state_out"], "lens": s["lens_out"],
                "status": s["status"], "starts": s["starts"], "slots": s["slots"], "positions": s["positions"],
                "token_seqs": s["token_seqs"]}
    if op == "attend":
        if "workspace" not in s:  # zeroed once and kept, as a serving loop keeps it
            size = lean.lean_paged_attention_workspace_bytes(case["seqs"], case["q_heads"], case["kv_heads"], case["dim"])
            s["workspace"] = torch.zeros((size,), device="cuda", dtype=torch.uint8)
        lean.lean_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["out"],
                                  scale=1 / math.sqrt(case["dim"]), window=case["window"], lse=s["lse"],
                                  workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if "workspace" not in s:
        size = lean.lean_token_logprobs_workspace_bytes(case["tokens"], case["vocab"], case["top"])
        s["workspace"] = torch.zeros((size,), device="cuda", dtype=torch.uint8)
    lean.lean_token_logprobs(s["logits"], s["ids"], s["logprobs"], ranks=s["ranks"], entropy=s["entropy"],
                             top_ids=s["top_ids"], top_logprobs=s["top_logprobs"], workspace=s["workspace"])
    out = {"logprobs": s["logprobs"], "ranks": s["ranks"], "entropy": s["entropy"]}
    if case["top"]:
        out["top_ids"], out["top_logprobs"] = s["top_ids"], s["top_logprobs"]
    return out


# ---- the definitions in 64 bits --------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None
    s = prepare(case, seed)
    f8 = torch.float64
    if op == "norm":
        u = s["x"].to(f8)
        if case["post"]:
            u = u / torch.sqrt(u.pow(2).sum(1, keepdim=True) / case["width"] + EPS) * s["post_w"].to(f8)
        if case["gate"] != "none":
            u = u * s["gate"].to(f8)
        h = s["h"].to(f8) + u * case["alpha"]
        return {"h": h, "y": s["w"].to(f8) * h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["width"] + EPS)}
    if op == "rope":
        rot, page = case["rot"], case["page"]
        pair = torch.arange(rot // 2, dtype=f8, device="cuda")
        phi = s["positions"].to(f8)[:, None] * torch.pow(torch.tensor(1e6, dtype=f8, device="cuda"), -2 * pair / rot)[None]
        turn = torch.polar(torch.full_like(phi, case["scale"]), phi)[:, None]  # rotation as a complex factor

        def rotate(x):
            x = x.to(f8).clone()
            lo = torch.arange(rot // 2, device="cuda") * (2 if case["inter"] else 1)
            hi = lo + (1 if case["inter"] else rot // 2)
            z = torch.complex(x[..., lo], x[..., hi]) * turn
            x[..., lo], x[..., hi] = z.real, z.imag
            return x

        out = {"q": rotate(s["q"])}
        for name, rows in (("k_cache", rotate(s["k"])), ("v_cache", s["v"].to(f8))):
            c = s[name].to(f8)
            c[s["slots"].long() // page, s["slots"].long() % page] = rows
            out[name] = c
        return out
    if op == "attend":
        n, q, d = s["q"].shape
        page, kv = case["page"], case["kv_heads"]
        out, lse = torch.zeros((n, q, d), dtype=f8, device="cuda"), torch.full((n, q), -math.inf, dtype=f8, device="cuda")
        for i, length in enumerate(_lengths(case)):
            lo = max(0, length - case["window"]) if case["window"] else 0
            t = torch.arange(lo, length, device="cuda")
            rows = s["table"][i].long()[t // page], t % page
            keys, values = s["k_cache"][rows].to(f8), s["v_cache"][rows].to(f8)
            x = s["q"][i].to(f8).view(kv, q // kv, d).transpose(1, 2)
            z = torch.matmul(keys.transpose(0, 1), x).transpose(1, 2) * d ** -0.5  # [kv, group, keys]
            lse[i] = torch.logsumexp(z, -1).reshape(q)
            out[i] = torch.matmul(torch.softmax(z, -1), values.transpose(0, 1)).reshape(q, d)
        return {"out": out, "lse": lse}
    t, v, k = case["tokens"], case["vocab"], case["top"]
    lp, ent = torch.empty((t,), dtype=f8, device="cuda"), torch.empty((t,), dtype=f8, device="cuda")
    best = torch.empty((t, k), dtype=f8, device="cuda")
    for a in range(0, t, 256):
        x = torch.log_softmax(s["logits"][a:a + 256].to(f8), -1)
        lp[a:a + 256] = x[torch.arange(x.shape[0], device="cuda"), s["ids"][a:a + 256].long()]
        ent[a:a + 256] = -torch.special.xlogy(x.exp(), x.exp()).sum(-1)
        if k:
            best[a:a + 256] = torch.topk(x, k, -1).values
    out = {"logprobs": lp, "ranks": None, "entropy": ent}
    if k:
        out["top_ids"], out["top_logprobs"] = None, best
    return out
