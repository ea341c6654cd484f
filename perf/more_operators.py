"""Caches of keys and values in 8 bits, and attention to prefixes that sequences share, as they are measured.

Each case is one call (or the calls that belong together) at sizes from a single
new token to long prompts, long caches and whole serving batches:

  append  rotary positions of q and k, k and v quantised into the paged cache as
          they are written, and the tokens read back
  read    tokens of many sequences read back from the cache, as a prompt's next
          chunk needs its earlier ones
  attend  attention of one new token per sequence over the cache in 8 bits
  prefix  the same where many sequences begin with one long prefix, whose keys and
          values lie in the cache once

A cache in 8 bits holds, for each token and kv head, whole numbers c in -127..127
and one fp32 scale s = max |x| / 127, c = x / s to the nearest (halves away from 0).

With `own` false, run() computes them in elementary torch operations in 32 bits
(the quotients x / s in 64: they decide which whole number is nearest); with it
true, through this package.  exact() is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}


# ---- the cases -------------------------------------------------------------------

def listed():
    return [
        # four sequences' new tokens, fp32 from the linears
        {"name": "append_token", "op": "append", "tokens": 4, "q_heads": 15, "kv_heads": 5, "dim": 64, "rot": 64,
         "inter": False, "act": "f32", "page": 16, "start": 2000, "heads_first": True},
        # a long prompt, bf16, half of each head rotated
        {"name": "append_prompt", "op": "append", "tokens": 16384, "q_heads": 16, "kv_heads": 2, "dim": 128, "rot": 64,
         "inter": True, "act": "bf16", "page": 64, "start": 98304, "heads_first": True},
        # one short sequence back in fp32, the scales in the cache's own order
        {"name": "read_short", "op": "read", "tokens": 613, "kv_heads": 5, "dim": 64, "page": 16, "cache": "i8",
         "out": "f32", "heads_first": False},
        # all the earlier tokens of a long prompt, for its next chunk
        {"name": "read_prompt", "op": "read", "tokens": 131072, "kv_heads": 8, "dim": 128, "page": 64, "cache": "i8",
         "out": "bf16", "heads_first": True},
        # one sequence, a few pages: latency
        {"name": "attend_short", "op": "attend", "seqs": 1, "q_heads": 15, "kv_heads": 5, "dim": 64, "page": 16,
         "longest": 613, "ragged": False, "window": 0, "act": "f32", "heads_first": True},
        # one sequence with a long cache: the length has to be split over the GPU
        {"name": "attend_long", "op": "attend", "seqs": 1, "q_heads": 16, "kv_heads": 2, "dim": 128, "page": 64,
         "longest": 131072, "ragged": False, "window": 0, "act": "f32", "heads_first": True},
        # a serving batch of very different lengths
        {"name": "attend_batch", "op": "attend", "seqs": 384, "q_heads": 32, "kv_heads": 4, "dim": 64, "page": 16,
         "longest": 8192, "ragged": True, "window": 0, "act": "bf16", "heads_first": True},
        # four answers to one prompt: latency
        {"name": "prefix_few", "op": "prefix", "prefixes": 1, "seqs": 4, "q_heads": 15, "kv_heads": 5, "dim": 64, "page": 16,
         "longest": 2000, "tail": 100, "act": "f32", "cache": "bf16", "heads_first": True},
        # a batch of answers to one very long document
        {"name": "prefix_document", "op": "prefix", "prefixes": 1, "seqs": 96, "q_heads": 16, "kv_heads": 2, "dim": 128,
         "page": 64, "longest": 32768, "tail": 512, "act": "bf16", "cache": "bf16", "heads_first": True},
        # several prompts of different lengths with different numbers of answers, the cache in 8 bits
        {"name": "prefix_prompts", "op": "prefix", "prefixes": 12, "seqs": 240, "q_heads": 32, "kv_heads": 4, "dim": 64,
         "page": 16, "longest": 8192, "tail": 700, "act": "bf16", "cache": "i8", "heads_first": True},
        # one system prompt for a whole serving batch
        {"name": "prefix_system", "op": "prefix", "prefixes": 1, "seqs": 256, "q_heads": 32, "kv_heads": 4, "dim": 64,
         "page": 32, "longest": 16384, "tail": 300, "act": "f16", "cache": "f16", "heads_first": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "prefix"])
    act = rng.choice(["f32", "bf16", "f16"])
    kv = rng.choice([1, 2, 3, 4, 5, 8])
    q = kv * rng.choice([1, 2, 3, 4, 6, 8, 12])
    dim = rng.choice([64, 80, 96, 128, 128, 256])
    page = rng.choice([16, 16, 24, 32, 64, 128])
    heads_first = rng.random() < 0.7
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 16384 * 20 * 128 // ((q + 2 * kv) * dim)), "q_heads": q, "kv_heads": kv,
                "dim": dim, "rot": rng.choice([dim, dim // 2]), "inter": rng.random() < 0.5, "act": act, "page": page,
                "start": _log(rng, 1, 1000000), "heads_first": heads_first}
    if op == "read":
        cache = rng.choice(["i8", "i8", "bf16", "f16"])
        size = SIZE[cache] + SIZE[act]
        return {"op": op, "tokens": _log(rng, 1, 131072 * 8 * 128 * 3 // (kv * dim * size)), "kv_heads": kv, "dim": dim,
                "page": page, "cache": cache, "out": act, "heads_first": heads_first}
    if op == "attend":
        seqs = _log(rng, 1, 256)
        longest = _log(rng, 1, max(1, min(131072, 384 * 1024 * 4 * 64 // (seqs * kv * dim))))
        return {"op": op, "seqs": seqs, "q_heads": q, "kv_heads": kv, "dim": dim, "page": page, "longest": longest,
                "ragged": rng.random() < 0.6, "window": rng.choice([0, 0, 0, 1024]), "act": act,
                "heads_first": heads_first}
    dim = min(dim, 128)
    cache = rng.choice(["i8", act if act != "f32" else rng.choice(["bf16", "f16"])])
    seqs = _log(rng, 1, 256)
    longest = _log(rng, 1, max(1, min(32768, 256 * 32 * 16384 * 64 // (4 * seqs * q * dim))))
    return {"op": op, "prefixes": _log(rng, 1, max(1, min(16, seqs // 2))), "seqs": seqs, "q_heads": q, "kv_heads": kv, "dim": dim,
            "page": page, "longest": longest, "tail": _log(rng, 1, 512), "act": act, "cache": cache,
            "heads_first": heads_first}


def _spread(n, top):
    """n lengths from 1 to top, log-uniform in an order that mixes them: the same for every seed, so that the work is the case's."""
    return [int(round(top ** ((i * 0.6180339887) % 1.0))) if i else top for i in range(n)]


def _lengths(case):
    return _spread(case["seqs"], case["longest"]) if case["ragged"] else [case["longest"]] * case["seqs"]


def _attended(case):
    w = case["window"]
    return [min(x, w) if w else x for x in _lengths(case)]


def _prefixes(case):
    """(length, number of sequences) of each prefix: halves of the longest at least, shares that differ by up to 8 times."""
    n, seqs = case["prefixes"], case["seqs"]
    lens = [max(1, int(case["longest"] * (1 - 0.5 * ((i * 0.6180339887) % 1.0)))) for i in range(n)]
    weight = [8 ** ((0.3 + i * 0.7548776662) % 1.0) for i in range(n)]
    ends = [int(round(seqs * sum(weight[:i + 1]) / sum(weight))) for i in range(n)]
    return [(lens[i], ends[i] - (ends[i - 1] if i else 0)) for i in range(n)]


def work(case):
    op, d, kv = case["op"], case["dim"], case["kv_heads"]
    if op == "append":
        t, a, q = case["tokens"], SIZE[case["act"]], case["q_heads"]
        read = SIZE[_read_type(case)]
        # q in and out, k and v in, codes and scales written, read, and given back as values
        return {"bytes": t * d * (2 * q * a + 2 * kv * (a + 2 + read)) + 4 * t * (2 + 4 * kv) + 4 * case["rot"],
                "flops": t * d * (3 * (q + kv) + 8 * kv)}
    if op == "read":
        t, scales = case["tokens"], 4 if case["cache"] == "i8" else 0
        return {"bytes": 2 * t * kv * (d * (SIZE[case["cache"]] + SIZE[case["out"]]) + scales) + 4 * t, "flops": 2 * t * kv * d}
    q, act = case["q_heads"], SIZE[case["act"]]
    if op == "attend":
        keys, b = sum(_attended(case)), case["seqs"]
        return {"bytes": 2 * keys * kv * (d + 4) + 2 * b * q * d * act + 4 * sum(-(-x // case["page"]) for x in _attended(case))
                + 4 * b + 4 * b * q, "flops": 4 * keys * q * d}
    b, tails = case["seqs"], _spread(case["seqs"], case["tail"])
    keys = sum(x for x, _ in _prefixes(case)) + sum(tails)
    pairs = sum(x * n for x, n in _prefixes(case)) + sum(tails)
    row = d * SIZE[case["cache"]] + (4 if case["cache"] == "i8" else 0)
    return {"bytes": 2 * keys * kv * row + 2 * b * q * d * act + 4 * keys // case["page"] + 8 * b + 4 * b * q,
            "flops": 4 * pairs * q * d}


# ---- inputs ----------------------------------------------------------------------

def _read_type(case):
    return case["act"] if case["act"] != "f32" else "bf16"


def _turns(rot, base=1000000.0):
    """Turns per position of each rotated pair, in units of 2^-64."""
    at = torch.arange(0, rot, 2, dtype=torch.float64) / rot
    return (torch.pow(torch.tensor(base, dtype=torch.float64), -at) / (2 * math.pi) * 2.0 ** 64).to(torch.int64)


def _scales(case, pages, make):
    """[page, place, kv head], the places of a head beside one another or the heads of a place."""
    if case["heads_first"]:
        return make(pages, case["kv_heads"], case["page"]).transpose(1, 2)
    return make(pages, case["page"], case["kv_heads"])


def _quantised(x, scale):
    """x as whole numbers of scale, the nearest, halves away from 0."""
    ratio = x.double() / scale.double()[..., None]
    ratio = torch.where(scale[..., None] > 0, ratio, 0.0)
    return torch.trunc(ratio + torch.where(ratio < 0, -0.5, 0.5)).clamp(-127, 127).to(torch.int8)


def _fill(case, s, pool, cache, normal):
    """A cache of `pool` pages, in 8 bits from normal values whose tokens differ in size."""
    page, kv, d = case["page"], case["kv_heads"], case["dim"]
    for name in ("k", "v"):
        x = normal(pool, page, kv, d)
        if cache != "i8":
            s[name + "_cache"], s[name + "_scales"] = x.to(DTYPES[cache]), None
            continue
        x = x * torch.exp(0.3 * normal(pool, page, kv, 1))
        scale = x.abs().amax(-1) / 127
        s[name + "_cache"] = torch.empty((pool, page, kv, d), device="cuda", dtype=torch.int8)
        for a in range(0, pool, max(1, (1 << 26) // (page * kv * d))):  # (in pieces: the quotients take 8 bytes each)
            b = a + max(1, (1 << 26) // (page * kv * d))
            s[name + "_cache"][a:b] = _quantised(x[a:b], scale[a:b])
        s[name + "_scales"] = _scales(case, pool, lambda *n: torch.empty(n, device="cuda"))
        s[name + "_scales"].copy_(scale)


def _table(lens, page, order):
    """(pages of each sequence with -1 after them, pages left over) from a list of all pages."""
    need = [-(-x // page) for x in lens]
    dev = order.device
    first = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
    at = torch.arange(max(need), device=dev)
    have = at[None] < torch.tensor(need, device=dev)[:, None]
    return torch.where(have, order[torch.where(have, first[:, None] + at[None], 0)], -1).to(torch.int32), order[sum(need):]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    op, s = case["op"], {"case": case}
    d, kv, page = case["dim"], case["kv_heads"], case["page"]
    if op == "append":
        t, q, act = case["tokens"], case["q_heads"], DTYPES[case["act"]]
        s["q"], s["k"], s["v"] = normal(t, q, d, dtype=act), normal(t, kv, d, dtype=act), normal(t, kv, d, dtype=act)
        s["positions"] = torch.arange(t, device=dev, dtype=torch.int32) + case["start"]
        pages = -(-t // page) + 3
        order = torch.randperm(pages, generator=g, device=dev)
        at = torch.arange(t, device=dev)
        s["slots"] = (order[at // page] * page + at % page).to(torch.int32)
        s["turns"] = _turns(case["rot"]).to(dev)
        s["q_out"] = torch.empty_like(s["q"])
        for name in ("k", "v"):
            s[name + "_cache"] = torch.zeros((pages, page, kv, d), device=dev, dtype=torch.int8)
            s[name + "_scales"] = _scales(case, pages, lambda *n: torch.zeros(n, device=dev))
            s[name + "_out"] = torch.empty((t, kv, d), device=dev, dtype=DTYPES[_read_type(case)])
    elif op == "read":
        t = case["tokens"]
        pages = -(-t // page) + 3
        _fill(case, s, pages, case["cache"], normal)
        order = torch.randperm(pages, generator=g, device=dev)
        at = torch.arange(t, device=dev)
        s["slots"] = (order[at // page] * page + at % page).to(torch.int32)
        s["k_out"], s["v_out"] = (torch.empty((t, kv, d), device=dev, dtype=DTYPES[case["out"]]) for _ in range(2))
    elif op == "attend":
        n, q, lens = case["seqs"], case["q_heads"], _lengths(case)
        pool = sum(-(-x // page) for x in lens) + 5
        s["q"] = normal(n, q, d, dtype=DTYPES[case["act"]], std=2.0)
        _fill(case, s, pool, "i8", normal)
        s["table"], _ = _table(lens, page, torch.randperm(pool, generator=g, device=dev))
        s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
    else:
        n, q, prefixes, tails = case["seqs"], case["q_heads"], _prefixes(case), _spread(case["seqs"], case["tail"])
        pool = sum(-(-x // page) for x, _ in prefixes) + sum(-(-x // page) for x in tails) + 5
        s["q"] = normal(n, q, d, dtype=DTYPES[case["act"]], std=2.0)
        _fill(case, s, pool, case["cache"], normal)
        order = torch.randperm(pool, generator=g, device=dev)
        s["prefix_table"], order = _table([x for x, _ in prefixes], page, order)
        s["table"], _ = _table(tails, page, order)
        ints = lambda v: torch.tensor(v, device=dev, dtype=torch.int32)  # noqa: E731
        s["prefix_lens"], s["lens"] = ints([x for x, _ in prefixes]), ints(tails)
        starts = [0]
        for _, count in prefixes:
            starts.append(starts[-1] + count)
        s["seq_starts"] = ints(starts)
    if op in ("attend", "prefix"):
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((case["seqs"], case["q_heads"]), device=dev)
    return s


# ---- one pass --------------------------------------------------------------------

def _append_plain(s):
    case = s["case"]
    rot, page = case["rot"], case["page"]
    # whole turns drop out of the 64-bit product; the upper half is the angle
    turn = (s["positions"].long()[:, None] * s["turns"][None]) >> 32
    angle = turn.float() * (2 * math.pi / 2 ** 32)
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]

    def rotated(x):
        x = x.float()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        u, v = a * cos - b * sin, a * sin + b * cos
        both = torch.stack([u, v], -1).flatten(-2) if case["inter"] else torch.cat([u, v], -1)
        return torch.cat([both, x[..., rot:]], -1)

    at = s["slots"].long() // page, s["slots"].long() % page
    out = {"q": rotated(s["q"]).to(s["q"].dtype)}
    for name, x in (("k", rotated(s["k"])), ("v", s["v"].float())):
        scale = x.abs().amax(-1) / 127
        s[name + "_cache"][at], s[name + "_scales"][at] = _quantised(x, scale), scale
        out[name] = (s[name + "_cache"][at].float() * s[name + "_scales"][at][..., None]).to(s[name + "_out"].dtype)
        out[name + "_scales"] = s[name + "_scales"]
    return out


def _values(s, name, at):
    """Tokens of a cache as fp32."""
    x = s[name + "_cache"][at].float()
    return x if s[name + "_scales"] is None else x * s[name + "_scales"][at][..., None]


def _read_plain(s):
    page = s["case"]["page"]
    at = s["slots"].long() // page, s["slots"].long() % page
    return {name: _values(s, name, at).to(s[name + "_out"].dtype) for name in ("k", "v")}


def _places(table, page):
    """Page and place of each token of each row of a block table."""
    at = torch.arange(table.shape[1] * page, device=table.device)
    return table.long().clamp(min=0)[:, at // page], (at % page)[None].expand(table.shape[0], -1)


def _attend_plain(s):
    case = s["case"]
    n, q, d = s["q"].shape
    kv = case["kv_heads"]
    at = _places(s["table"], case["page"])
    x = s["q"].float().view(n, kv, q // kv, d) / math.sqrt(d)
    score = torch.einsum("ngrd,nlgd->ngrl", x, _values(s, "k", at))
    lens, token = s["lens"].long()[:, None], torch.arange(score.shape[-1], device=score.device)[None]
    seen = token < lens
    if case["window"]:
        seen = seen & (token >= lens - case["window"])
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    out = torch.einsum("ngrl,nlgd->ngrd", e, _values(s, "v", at)) / total
    return {"out": out.reshape(n, q, d).to(s["q"].dtype), "lse": (top + torch.log(total)).reshape(n, q)}


def _prefix_plain(s):
    case = s["case"]
    n, q, d = s["q"].shape
    kv, page, starts = case["kv_heads"], case["page"], s["seq_starts"].long()
    x = s["q"].float().view(n, kv, q // kv, d) / math.sqrt(d)
    # the sequences of each prefix side by side, as many places as the largest group has
    most = max(c for _, c in _prefixes(case))
    group = starts[:-1, None] + torch.arange(most, device=starts.device)[None]
    member = group < starts[1:, None]
    group = group.clamp(max=n - 1)
    seq = torch.arange(n, device=starts.device)
    mine = torch.searchsorted(starts[1:], seq, right=True)
    place = seq - starts[mine]
    at = _places(s["prefix_table"], page)
    score = torch.einsum("pcgrd,plgd->pcgrl", x[group], _values(s, "k", at))
    token = torch.arange(score.shape[-1], device=score.device)
    score = score.masked_fill((token[None] >= s["prefix_lens"].long()[:, None])[:, None, None, None], -math.inf)
    own_at = _places(s["table"], page)
    own_score = torch.einsum("ngrd,nlgd->ngrl", x, _values(s, "k", own_at))
    token = torch.arange(own_score.shape[-1], device=score.device)
    own_score = own_score.masked_fill((token[None] >= s["lens"].long()[:, None])[:, None, None], -math.inf)
    top = torch.maximum(score.amax(-1)[mine, place], own_score.amax(-1))
    shared_top = torch.zeros(score.shape[:-1], device=score.device)
    shared_top[mine, place] = top
    e = torch.exp(score - shared_top[..., None]).masked_fill(~member[:, :, None, None, None], 0.0)
    own_e = torch.exp(own_score - top[..., None])
    total = e.sum(-1)[mine, place] + own_e.sum(-1)
    out = torch.einsum("pcgrl,plgd->pcgrd", e, _values(s, "v", at))[mine, place]
    out = (out + torch.einsum("ngrl,nlgd->ngrd", own_e, _values(s, "v", own_at))) / total[..., None]
    return {"out": out.reshape(n, q, d).to(s["q"].dtype), "lse": (top + torch.log(total)).reshape(n, q)}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _append_plain, "read": _read_plain, "attend": _attend_plain, "prefix": _prefix_plain}[op](s)
    from block_quantized_weight_dot_gb300 import lean
    case = s["case"]
    scales = {"k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    if op == "append":
        lean.lean_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["turns"], s["q_out"], s["k_cache"],
                              s["v_cache"], rot_dim=case["rot"], interleaved=case["inter"], **scales)
        lean.lean_kv_read(s["k_cache"], s["v_cache"], s["slots"], s["k_out"], s["v_out"], **scales)
        return {"q": s["q_out"], "k": s["k_out"], "k_scales": s["k_scales"], "v": s["v_out"], "v_scales": s["v_scales"]}
    if op == "read":
        lean.lean_kv_read(s["k_cache"], s["v_cache"], s["slots"], s["k_out"], s["v_out"], **scales)
        return {"k": s["k_out"], "v": s["v_out"]}
    sizes = case["seqs"], case["q_heads"], case["kv_heads"], case["dim"]
    scale = 1 / math.sqrt(case["dim"])
    if op == "attend":
        if "workspace" not in s:  # allocated once and kept, as a serving loop keeps it
            s["workspace"] = torch.empty((lean.lean_paged_attention_workspace_bytes(*sizes),), device="cuda", dtype=torch.uint8)
        lean.lean_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["out"], scale=scale,
                                  window=case["window"], lse=s["lse"], workspace=s["workspace"], **scales)
    else:
        if "workspace" not in s:
            size = lean.lean_prefix_attention_workspace_bytes(*sizes, case["prefixes"])
            s["workspace"] = torch.empty((size,), device="cuda", dtype=torch.uint8)
        lean.lean_prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_lens"], s["seq_starts"],
                                   s["table"], s["lens"], s["out"], scale=scale, lse=s["lse"], workspace=s["workspace"],
                                   **scales)
    return {"out": s["out"], "lse": s["lse"]}


# ---- the definitions in 64 bits --------------------------------------------------

def exact(case, seed):
    op, d, kv, page = case["op"], case["dim"], case["kv_heads"], case["page"]
    s, f8 = prepare(case, seed), torch.float64

    def tokens(name, rows):
        x = s[name + "_cache"][rows].to(f8)
        return x if s[name + "_scales"] is None else x * s[name + "_scales"][rows].to(f8).unsqueeze(-1)

    if op == "append":
        rot = case["rot"]
        pair = torch.arange(rot // 2, dtype=f8, device="cuda")
        phi = s["positions"].to(f8)[:, None] * torch.pow(torch.tensor(1e6, dtype=f8, device="cuda"), -2 * pair / rot)[None]
        turn = torch.polar(torch.ones_like(phi), phi)[:, None]  # rotation as a complex factor

        def rotate(x):
            x = x.to(f8).clone()
            lo = torch.arange(rot // 2, device="cuda") * (2 if case["inter"] else 1)
            hi = lo + (1 if case["inter"] else rot // 2)
            z = torch.complex(x[..., lo], x[..., hi]) * turn
            x[..., lo], x[..., hi] = z.real, z.imag
            return x

        rows = s["slots"].long() // page, s["slots"].long() % page
        out = {"q": rotate(s["q"])}
        for name, x in (("k", rotate(s["k"])), ("v", s["v"].to(f8))):
            unit = torch.linalg.vector_norm(x, math.inf, -1) / 127
            out[name] = torch.round(x / unit[..., None]) * unit[..., None]
            full = s[name + "_scales"].to(f8)
            full[rows] = unit
            out[name + "_scales"] = full
        return out
    if op == "read":
        rows = s["slots"].long() // page, s["slots"].long() % page
        return {"k": tokens("k", rows), "v": tokens("v", rows)}
    n, q = case["seqs"], case["q_heads"]
    out, lse = torch.zeros((n, q, d), dtype=f8, device="cuda"), torch.zeros((n, q), dtype=f8, device="cuda")

    def gathered(table, lo, hi):
        t = torch.arange(lo, hi, device="cuda")
        rows = table.long()[t // page], t % page
        return tokens("k", rows), tokens("v", rows)

    def attended(i, keys, values):
        x = s["q"][i].to(f8).view(kv, q // kv, d).transpose(1, 2)
        z = torch.matmul(keys.transpose(0, 1), x).transpose(1, 2) * d ** -0.5  # [kv, group, keys]
        lse[i] = torch.logsumexp(z, -1).reshape(q)
        out[i] = torch.matmul(torch.softmax(z, -1), values.transpose(0, 1)).reshape(q, d)

    if op == "attend":
        for i, length in enumerate(_lengths(case)):
            attended(i, *gathered(s["table"][i], max(0, length - case["window"]) if case["window"] else 0, length))
    else:
        tails, i = _spread(n, case["tail"]), 0
        for p, (length, count) in enumerate(_prefixes(case)):
            keys, values = gathered(s["prefix_table"][p], 0, length)
            for i in range(i, i + count):
                mine = gathered(s["table"][i], 0, tails[i])
                attended(i, torch.cat([keys, mine[0]]), torch.cat([values, mine[1]]))
            i += count > 0
    return {"out": out, "lse": lse}
