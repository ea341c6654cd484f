"""Plain 64-bit forms of the cache in 8 bits and runners that call the library on
small inputs and compare.  U, HALF, TINY and the tolerances' reasoning: step_testlib."""
import math

import numpy as np

from lean_testlib import torch_cuda
from step_testlib import HALF, TINY, U, attend_ref, close, dtype, gen, normal, rotate_ref, strided


def codes_ref(x):
    """(codes, scales) of rows of fp32 x [..., dim] by the definition: s = max |x| / 127 rounded to fp32, c nearest to
    x / s, halves away from 0.  The quotient of two fp32 numbers is either half-way between whole numbers or further
    from it than the last place of a double, so that it may be taken in 64 bits."""
    torch = torch_cuda()
    x = x.float()
    top = x.abs().amax(-1)
    ok = torch.isfinite(x).all(-1)
    s = torch.where(ok, (torch.where(ok, top, 0.0).double() / 127).float(), math.nan)  # (two roundings: see below)
    r = x.double() / s.double()[..., None]
    r = torch.where(torch.isfinite(r), r, 0.0)
    c = torch.trunc(r + torch.where(r < 0, -0.5, 0.5)).clamp(-127, 127)
    return c.to(torch.int8), s


# (A quotient by 127 rounded to 53 and then to 24 bits is the one rounded to 24: its expansion in base 2 has period 7,
# so that no run of 29 equal digits, which a second rounding could turn over, follows the 24th place.)


def scales_like(cache, heads_first, fill=7.0):
    """[pages, page, kv heads] float32 beside a cache: the places of a head, or the heads of a place, next to one another."""
    torch = torch_cuda()
    p, n, h = cache.shape[:3]
    if heads_first:
        return torch.full((p, h, n), fill, device="cuda").transpose(1, 2)
    return torch.full((p, n, h), fill, device="cuda")


def make_cache8(pool, page, hkv, dim, seed, spread=0.5, heads_first=True):
    """Random codes and scales (log-normal) of a whole cache."""
    torch = torch_cuda()
    g = gen(7000 + seed)
    out = []
    for _ in range(2):
        c = torch.randint(-127, 128, (pool, page, hkv, dim), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
        s = scales_like(c, heads_first)
        s.copy_(torch.exp(spread * torch.randn((pool, page, hkv), generator=g, device="cuda")) / 73)
        out += [c, s]
    return out  # k, its scales, v, its scales


def run_append8(lean, tokens, hq, hkv, dim, rot, act="f32", inter=False, page=16, start=0, scale=1.0, seed=0, pad=0,
                in_place=False, k_out=False, padding=(), heads_first=True, cache_pad=0, flags=0, stream=None, x=None):
    torch = torch_cuda()
    g = gen(7100 + seed)
    q = normal(g, tokens, hq, dim, t=act) if hq else None
    k, v = (normal(g, tokens, hkv, dim, t=act) for _ in range(2)) if x is None else x
    freq = lean.lean_rope_frequencies(lean.LEAN_ROPE_PLAIN, rot, 10000.0) if rot else np.zeros(0)
    turns = torch.from_numpy(lean.lean_rope_turns(freq)).cuda() if rot else None
    pos = (torch.arange(tokens, device="cuda") * 7 + start).to(torch.int32)
    pages = -(-tokens // page) + 2
    order = torch.randperm(pages, generator=g, device="cuda")
    at = torch.arange(tokens, device="cuda")
    slots = (order[at // page] * page + at % page).to(torch.int32)
    for t in padding:
        slots[t] = -1
    kc, vc = (torch.full((pages, page, hkv, dim + cache_pad), 99, device="cuda", dtype=torch.int8)[..., :dim] for _ in range(2))
    ks, vs = (scales_like(kc, heads_first) for _ in range(2))
    # without a rotation x is what it is; with one, k errs as in step_testlib.run_rope
    rel = (4 + 2 * math.pi + 3) * U if rot else 0.0
    want_q = rotate_ref(q, pos, freq, rot, inter, scale) if hq else None
    want_k = rotate_ref(k, pos, freq, rot, inter, scale)
    size = lambda t: t.double().abs().amax(-1, keepdim=True) * 2 * abs(scale)  # noqa: E731
    qsize, ksize = size(q) if hq else None, size(k)
    k_is, v_is = k.float(), v.float()
    if pad:
        q, k, v = (strided(t, pad) if t is not None else None for t in (q, k, v))
    qo = None if not hq else q if in_place else torch.empty((tokens, hq, dim), device="cuda", dtype=dtype(act))
    ko = None if not k_out else k if in_place else torch.empty((tokens, hkv, dim), device="cuda", dtype=dtype(act))
    torch.cuda.synchronize()
    lean.lean_rope_append(q, k, v, pos, slots, turns, qo, kc, vc, rot_dim=rot, interleaved=inter, rot_scale=scale, k_out=ko,
                          flags=flags, stream=stream, k_scales=ks, v_scales=vs)
    torch.cuda.synchronize()
    what = "append8 %dx%d/%dx%d rot %d %s" % (tokens, hq, hkv, dim, rot, act)
    if hq:
        close(qo, want_q, rel * qsize + HALF[act] * (want_q.abs() + rel * qsize) + TINY[act], what + " q")
    if ko is not None:
        close(ko, want_k, rel * ksize + HALF[act] * (want_k.abs() + rel * ksize) + TINY[act], what + " k_out")
    kept = [t for t in range(tokens) if t not in set(padding)]
    s = slots[kept].long()
    where = s // page, s % page
    for name, is_x, codes, scales in (("v", v_is, vc, vs), ("k", k_is, kc, ks)):
        got_c, got_s = codes[where], scales[where]
        if name == "v" or not rot:
            want_c, want_s = codes_ref(is_x[kept])
            same = (got_s == want_s) | (torch.isnan(got_s) & torch.isnan(want_s))
            assert bool(same.all()), what + " %s scales: %r" % (name, (~same).nonzero()[:3])
            assert torch.equal(got_c, want_c), what + " %s codes: %r" % (name, (got_c != want_c).nonzero()[:3])
        else:
            err = (rel * ksize[kept])[..., 0]
            top = want_k[kept].abs().amax(-1)
            close(got_s, top / 127, err / 127 + U * (top + err) / 127, what + " k scales")
            # half a step, of the scale that was stored, and what x and the quotient by 127 err by
            close(got_c.double() * got_s.double()[..., None], want_k[kept],
                  (0.5 * (1 + 4 * U) * got_s.double() + 2 * err + 127 * U * got_s.double())[..., None], what + " k values")
            assert int(got_c.abs().amax()) == 127
    for codes, scales in ((kc, ks), (vc, vs)):  # every other place untouched
        codes[where], scales[where] = 99, 7.0
        assert bool((codes == 99).all()) and bool((scales == 7.0).all()), what + ": a write outside the slots"


def run_read(lean, tokens, hkv, dim, page=16, cache="i8", out="f32", pool=None, heads_first=True, pad=0, cache_pad=0,
             slots=None, which="kv", seed=0, flags=0, stream=None, heads_major=False):
    torch = torch_cuda()
    g = gen(7200 + seed)
    pool = pool or -(-tokens // page) + 2
    ks = vs = None
    if cache == "i8":
        kc, ks, vc, vs = make_cache8(pool, page, hkv, dim + cache_pad, seed, heads_first=heads_first)
        kc, vc = kc[..., :dim], vc[..., :dim]
    else:
        kc, vc = (normal(g, pool, page, hkv, dim + cache_pad, t=cache)[..., :dim] for _ in range(2))
    if slots is None:
        slots = torch.randint(0, pool * page, (tokens,), generator=g, device="cuda").tolist()  # some of them twice
    sd = torch.tensor(slots, dtype=torch.int32, device="cuda")

    def room():
        if heads_major:
            return torch.full((hkv, tokens, dim), 7.0, device="cuda", dtype=dtype(out)).transpose(0, 1)
        return strided(torch.full((tokens, hkv, dim), 7.0, device="cuda", dtype=dtype(out)), pad) if pad else \
            torch.full((tokens, hkv, dim), 7.0, device="cuda", dtype=dtype(out))
    ko, vo = room() if "k" in which else None, room() if "v" in which else None
    torch.cuda.synchronize()
    lean.lean_kv_read(kc if "k" in which else None, vc if "v" in which else None, sd, ko, vo,
                      k_scales=ks if "k" in which else None, v_scales=vs if "v" in which else None, flags=flags, stream=stream)
    torch.cuda.synchronize()
    s = sd.long()
    ok, none = (s >= 0) & (s < pool * page), s < 0
    at = torch.where(ok, s, 0)
    for name, got, c, sc in (("k", ko, kc, ks), ("v", vo, vc, vs)):
        if got is None:
            continue
        want = c[at // page, at % page].double()
        if sc is not None:  # (the product is exact in 64 bits; fp32, then the output's type)
            want = want * sc[at // page, at % page].double()[..., None]
        want = want.float().to(dtype(out))
        want[none] = 0
        want[~ok & ~none] = math.nan
        same = (got == want) | (torch.isnan(got) & torch.isnan(want))
        assert bool(same.all()), "read %s %s: %r" % (name, cache, (~same).nonzero()[:3])
        if pad and tokens > 1:
            flat = got.as_strided((tokens - 1, got.stride(0)), (got.stride(0), 1))[:, hkv * dim:]
            assert bool(torch.isnan(flat).all()), "a write between the rows"


def make_attend8(lens, hq, hkv, dim, page, act, seed=0, width=None, heads_first=True, spread=0.5, junk=math.nan):
    """q, caches with their scales and the table of a batch; scales that no sequence holds are junk, and table entries
    past a sequence's pages far outside the cache."""
    torch = torch_cuda()
    need = [-(-max(x, 0) // page) for x in lens]
    pool = sum(need) + 3
    width = width or max(1, max(need))
    kc, ks, vc, vs = make_cache8(pool, page, hkv, dim, seed, spread, heads_first)
    g = gen(7300 + seed)
    order = torch.randperm(pool, generator=g, device="cuda").tolist()
    table = torch.full((len(lens), width), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    held = torch.zeros((pool, page), dtype=torch.bool, device="cuda")
    for s, x in enumerate(lens):
        for j in range(need[s]):
            pg = order.pop()
            table[s, j] = pg
            held[pg, :min(page, x - j * page)] = True
    for t in (ks, vs):
        t[~held] = junk
    q = normal(g, len(lens), hq, dim, t=act, std=1.5)
    return q, kc, ks, vc, vs, table


def run_attend8(lean, lens, hq, hkv, dim, page=16, act="f32", window=0, seed=0, lse=True, pad=0, heads_first=True, width=None,
                flags=0, scale=None, stream=None, inputs=None, workspace=None, spread=0.5, junk=math.nan):
    torch = torch_cuda()
    q, kc, ks, vc, vs, table = inputs or make_attend8(lens, hq, hkv, dim, page, act, seed, width, heads_first, spread, junk)
    scale = 1 / math.sqrt(dim) if scale is None else scale
    if pad:
        q = strided(q, pad)
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full((len(lens), hq, dim), 7.0, device="cuda", dtype=dtype(act))
    ls = torch.full((len(lens), hq), 7.0, device="cuda") if lse else None
    ws = workspace
    if ws is None:
        ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(len(lens), hq, hkv, dim), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    lean.lean_paged_attention(q, kc, vc, table, ld, out, scale=scale, window=window, lse=ls, workspace=ws, flags=flags,
                              stream=stream, k_scales=ks, v_scales=vs)
    torch.cuda.synchronize()
    kd, vd = kc.double() * ks.double()[..., None], vc.double() * vs.double()[..., None]
    want, want_lse, size, reach = attend_ref(q, kd, vd, table, lens, scale, window)
    # as step_testlib.run_attend; codes are exact in the instruction's type, two more products by scales in fp32
    seen = max([1] + [min(x, window) if window else x for x in lens])
    rel = (2 * 2.0 ** -16 + 20 * U) * reach + 2.0 ** -16 + (seen / 8 + 68) * U
    what = "attend8 %s heads %d/%d dim %d page %d %s window %d" % (lens[:4], hq, hkv, dim, page, act, window)
    top = torch.where(torch.isfinite(vd), vd.abs(), 0.0).max()
    err = rel[..., None] * size + 2.0 ** -37 * top
    close(out, want, err + HALF[act] * (want.abs() + err) + TINY[act], what)
    if lse:
        close(ls, want_lse, rel + 4 * U * torch.where(want_lse.isinf(), 0.0, want_lse).abs(), what + " lse")
    return out, ls


# ---- shared prefixes ------------------------------------------------------------------------

def prefix_ref(q, kd, vd, prefix_table, prefix_lens, starts, table, lens, scale):
    """(out, lse, sum p |v|, the largest sum |q k| scale) in 64 bits; kd, vd: the caches' values as float64."""
    torch = torch_cuda()
    n, hq, d = q.shape
    page, hkv = kd.shape[1], kd.shape[2]
    out, size = (torch.zeros((n, hq, d), dtype=torch.float64, device="cuda") for _ in range(2))
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    reach = torch.zeros((n, hq), dtype=torch.float64, device="cuda")

    def rows(tab, length):
        length = min(max(length, 0), tab.shape[0] * page)
        t = torch.arange(length, device="cuda")
        at = tab.long()[t // page], t % page
        return kd[at], vd[at]
    for s in range(n):
        mine = [i for i in range(len(prefix_lens)) if starts[i] <= s < starts[i + 1]]
        parts = [rows(prefix_table[i], prefix_lens[i]) for i in mine] + [rows(table[s], lens[s])]
        k, v = torch.cat([x[0] for x in parts]), torch.cat([x[1] for x in parts])
        if not k.shape[0]:
            continue
        x = q[s].double().view(hkv, hq // hkv, d)
        z = scale * torch.einsum("grd,lgd->grl", x, k)
        p = torch.softmax(z, -1)
        lse[s] = torch.logsumexp(z, -1).view(-1)
        out[s] = torch.einsum("grl,lgd->grd", p, v).reshape(hq, d)
        size[s] = torch.einsum("grl,lgd->grd", p, v.abs()).reshape(hq, d)
        reach[s] = abs(scale) * torch.einsum("grd,lgd->grl", x.abs(), k.abs()).amax(-1).view(-1)
    return out, lse, size, reach


def make_prefix(prefix_lens, lens, hq, hkv, dim, page=16, act="f32", cache="bf16", seed=0, heads_first=True, spread=0.5,
                junk=math.nan, extra=0):
    """q, caches, scales, both tables; what nobody holds is junk (scales of it in 8 bits), and table entries past the
    pages that are held far outside the cache."""
    torch = torch_cuda()
    g = gen(7500 + seed)
    every = [max(x, 0) for x in list(prefix_lens) + list(lens)]
    need = [-(-x // page) for x in every]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").tolist()
    held = torch.zeros((pool, page), dtype=torch.bool)
    tables = []
    for part, ls in ((need[:len(prefix_lens)], every[:len(prefix_lens)]), (need[len(prefix_lens):], every[len(prefix_lens):])):
        tab = torch.full((len(part), max(1, max(part)) + extra), 2 ** 31 - 1, dtype=torch.int32)
        for s, x in enumerate(ls):
            for j in range(part[s]):
                tab[s, j] = order.pop()
                held[tab[s, j], :min(page, x - j * page)] = True
        tables.append(tab.cuda())
    held = held.cuda()
    if cache == "i8":
        kc, ks, vc, vs = make_cache8(pool, page, hkv, dim, seed, spread, heads_first)
        ks[~held], vs[~held] = junk, junk
    else:
        ks = vs = None
        shape = (pool, hkv, page, dim) if heads_first else (pool, page, hkv, dim)
        kc, vc = (normal(g, *shape, t=cache) for _ in range(2))
        if heads_first:
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        kc[~held], vc[~held] = junk, junk
    q = normal(g, len(lens), hq, dim, t=act, std=1.5)
    return q, kc, ks, vc, vs, tables[0], tables[1]


def run_prefix(lean, prefix_lens, starts, lens, hq, hkv, dim, page=16, act="f32", cache="bf16", seed=0, lse=True, pad=0,
               heads_first=True, flags=0, scale=None, stream=None, inputs=None, workspace=None, spread=0.5, junk=math.nan,
               extra=0):
    torch = torch_cuda()
    inputs = inputs or make_prefix(prefix_lens, lens, hq, hkv, dim, page, act, cache, seed, heads_first, spread, junk, extra)
    q, kc, ks, vc, vs, shared, table = inputs
    scale = 1 / math.sqrt(dim) if scale is None else scale
    if pad:
        q = strided(q, pad)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pl, st, ld = ints(prefix_lens), ints(starts), ints(lens)
    out = torch.full((len(lens), hq, dim), 7.0, device="cuda", dtype=dtype(act))
    if pad:
        out = strided(out, pad)
    ls = torch.full((len(lens), hq), 7.0, device="cuda") if lse else None
    ws = workspace
    if ws is None:  # (what it holds does not matter)
        size = lean.lean_prefix_attention_workspace_bytes(len(lens), hq, hkv, dim, len(prefix_lens))
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    lean.lean_prefix_attention(q, kc, vc, shared, pl, st, table, ld, out, scale=scale, lse=ls, workspace=ws, flags=flags,
                               stream=stream, k_scales=ks, v_scales=vs)
    torch.cuda.synchronize()
    kd, vd = (c.double() if s is None else c.double() * s.double()[..., None] for c, s in ((kc, ks), (vc, vs)))
    want, want_lse, size, reach = prefix_ref(q, kd, vd, shared, prefix_lens, starts, table, lens, scale)
    # a sequence's own part as step_testlib.run_attend: the parts of q and p, and fp32.  The prefix's: sums of scores and
    # of a tile's products are taken 16 terms at a time, each rounded towards zero (2 U), up to 24 times, and tiles of
    # 128 keys are added one by one; p in one part of the operands' type errs by half a step.  Joins: a few U.
    seen = max([1] + [max(x, 0) for x in prefix_lens] + [max(x, 0) for x in lens])
    one = HALF["bf16"] if cache == "bf16" else HALF["f16"]
    split = act == "f32" or (act == "f16" and cache == "bf16")
    rel = (2 * 2.0 ** -16 + 80 * U) * reach + 2.0 ** -16 + (seen / 8 + 200) * U
    what = "prefix %s %s own %s heads %d/%d dim %d page %d %s/%s" % (prefix_lens[:4], starts[:4], lens[:4], hq, hkv, dim, page, act, cache)
    top = torch.where(torch.isfinite(vd), vd.abs(), 0.0).max()
    # f16 operands lose what of p is below half their smallest step, 2^-25, of a p that lies 2^9 above its reference in
    # one part and 2^13 in more; the reference is no larger than the largest p, and that no larger than the sum: 2^-34 (or
    # 2^-38) of the sum for each of the keys, times the largest value
    lost = 0.0 if cache == "bf16" else seen * 2.0 ** (-38 if split else -34)
    err = (rel[..., None] + (0.0 if split else one)) * size + (lost + 2.0 ** -37) * top
    close(out, want, err + HALF[act] * (want.abs() + err) + TINY[act], what)
    if lse:
        close(ls, want_lse, rel + 4 * U * torch.where(want_lse.isinf(), 0.0, want_lse).abs(), what + " lse")
    if pad and len(lens) > 1:
        flat = out.as_strided((len(lens) - 1, out.stride(0)), (out.stride(0), 1))[:, hq * dim:]
        assert bool(torch.isnan(flat).all()), what + ": a write between the rows"
    return out, ls
