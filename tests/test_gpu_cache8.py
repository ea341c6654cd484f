"""Caches in 8 bits on the GPU: written by lean_rope_append, read back by
lean_kv_read, attended by lean_paged_attention, each against 64 bits."""
import math

import pytest

from cache_testlib import codes_ref, make_attend8, make_cache8, run_append8, run_attend8, run_read, scales_like
from lean_testlib import torch_cuda
from step_testlib import gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


@pytest.fixture(autouse=True)
def clean(lean):
    yield
    assert lean.lean_device_error(True) == 0


# ---- written -------------------------------------------------------------------------

@pytest.mark.parametrize("act", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (80, 40), (128, 64), (128, 0), (96, 96), (256, 256), (512, 64), (6, 4), (72, 24), (2, 2)])
def test_append(lean, dim, rot, inter, act):
    run_append8(lean, 19, 6, 3, dim, rot, act, inter=inter, page=5, padding=(2, 18), scale=1.07)
    run_append8(lean, 3, 4, 1, dim, rot, act, inter=inter, k_out=True, heads_first=False, start=100000, seed=1)


@pytest.mark.parametrize("tokens", [1, 2, 700, 5000])
def test_append_lengths(lean, tokens):
    run_append8(lean, tokens, 16, 2, 128, 64, "bf16", inter=True, page=64)
    run_append8(lean, tokens, 15, 5, 64, 64, "f32", in_place=True, k_out=True)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_append_odd_places(lean, act):
    """Rows and caches off every wide access; heads of k and v alone."""
    run_append8(lean, 23, 3, 2, 64, 32, act, pad=3, cache_pad=5, page=7)
    run_append8(lean, 23, 0, 2, 64, 32, act, pad=4, cache_pad=4, page=7)
    run_append8(lean, 23, 0, 2, 128, 0, act, cache_pad=16)


@pytest.mark.parametrize("dim", [16, 64, 128, 130])
def test_append_rows_that_are_hard(lean, dim):
    """Zeros, halves between whole numbers, one large element, numbers that are subnormal or near the largest, infinities
    and NaN: codes and scales to the bit."""
    torch = torch_cuda()
    rows = []
    tie = torch.arange(dim, device="cuda").float() - dim // 2 + 0.5  # halves, with 127 among them: s is 1
    tie[0] = 127.0
    rows += [torch.zeros(dim, device="cuda"), tie.clamp(-126.5, 127), -tie.clamp(-126.5, 127)]
    for size in (1e-45, 2e-43, 1e-38, 2e-25, 1e-18, 1e-3, 1e4, 3e37):
        x = normal(gen(int(-math.log10(size)) + 50), dim) * size
        rows += [x, torch.where(torch.arange(dim, device="cuda") == 3, x * 0 + 9 * size, x * 0)]
    wide = normal(gen(9), dim)
    wide[5] = 3e5
    rows.append(wide)
    for bad in (math.inf, -math.inf, math.nan):
        x = normal(gen(10), dim)
        x[dim - 1] = bad
        rows.append(x)
    x = torch.stack(rows)[:, None]
    run_append8(lean, len(rows), 0, 1, dim, 0, "f32", x=(x, x.flip(0).contiguous()))


def test_append_all_half_ways(lean):
    """Every half-way point and its two neighbours, for scales with few and with many bits."""
    torch = torch_cuda()
    half = torch.arange(-126, 127, device="cuda").double() + 0.5
    rows = []
    for s in (1.0, 0.75, 2.0 ** -20, 1 / 127, 0.0123456, 1.9999999):
        s32 = torch.tensor(127 * s, dtype=torch.float32, device="cuda")
        mid = (half * float((s32.double() / 127).float())).float()
        up, down = torch.nextafter(mid, mid * 4), torch.nextafter(mid, mid * 0)
        rows += [torch.cat([s32[None], t, s32.new_zeros(2)]) for t in (mid, up, down)]
    x = torch.stack(rows)[:, None]
    run_append8(lean, len(rows), 0, 1, 256, 0, "f32", x=(x, -x))


def test_append_bad_slots(lean):
    torch = torch_cuda()
    g = gen(4)
    k, v = normal(g, 4, 2, 64), normal(g, 4, 2, 64)
    kc, vc = (torch.full((3, 16, 2, 64), 99, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (scales_like(kc, True) for _ in range(2))
    slots = torch.tensor([48, -5, 2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    lean.lean_rope_append(None, k, v, pos, slots, None, None, kc, vc, rot_dim=0, k_scales=ks, v_scales=vs)
    assert lean.lean_device_error(True) == 64
    for c, s, x in ((kc, ks, k), (vc, vs, v)):
        want_c, want_s = codes_ref(x[3])
        assert torch.equal(c[0, 7], want_c) and torch.equal(s[0, 7], want_s)
        c[0, 7], s[0, 7] = 99, 7.0
        assert bool((c == 99).all()) and bool((s == 7.0).all())


# ---- read back -------------------------------------------------------------------------

@pytest.mark.parametrize("cache", ["i8", "bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 80, 128, 130, 7, 512])
def test_read(lean, dim, out, cache):
    run_read(lean, 37, 3, dim, page=5, cache=cache, out=out)
    run_read(lean, 9, 1, dim, page=16, cache=cache, out=out, heads_first=False, which="k", pad=3)
    run_read(lean, 9, 2, dim, page=16, cache=cache, out=out, which="v", cache_pad=8, pad=8)
    run_read(lean, 11, 2, dim, page=16, cache=cache, out=out, cache_pad=1, heads_major=True)


@pytest.mark.parametrize("tokens", [1, 613, 20000])
def test_read_lengths(lean, tokens):
    run_read(lean, tokens, 5, 64, out="bf16")
    run_read(lean, tokens, 8, 128, page=64, out="f32")


def test_read_padding_and_bad_slots(lean):
    run_read(lean, 5, 2, 64, slots=[-1, 3, -2 ** 31, 0, 31], pool=2)
    assert lean.lean_device_error(True) == 0
    run_read(lean, 4, 2, 64, slots=[32, 3, 2 ** 31 - 1, -1], pool=2)
    assert lean.lean_device_error(True) == 64
    run_read(lean, 3, 2, 64, slots=[32, 3, -1], pool=2, cache="bf16", out="bf16")
    assert lean.lean_device_error(True) == 64


def test_read_infinite_scales(lean):
    """A scale that is NaN or infinite, and codes of 0 under it."""
    torch = torch_cuda()
    kc, ks, vc, vs = make_cache8(1, 4, 1, 16, 3)
    ks[0, 1], ks[0, 2] = math.nan, math.inf
    kc[0, 2, 0, 5] = 0
    out = torch.zeros((4, 1, 16), device="cuda")
    lean.lean_kv_read(kc, None, torch.arange(4, dtype=torch.int32, device="cuda"), out, None, k_scales=ks)
    want = kc[0].float() * ks[0][..., None]
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and bool(torch.isnan(out[2, 0, 5]))
    assert torch.equal(out[torch.isfinite(want)], want[torch.isfinite(want)])


# ---- attended ----------------------------------------------------------------------------

RAGGED = [0, 1, 15, 16, 17, 31, 32, 33, 130, 700]


@pytest.mark.parametrize("act", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 176, 256])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (6, 2), (8, 1), (9, 1), (34, 2)])
def test_attend(lean, hq, hkv, dim, act):
    run_attend8(lean, RAGGED, hq, hkv, dim, act=act)


@pytest.mark.parametrize("page", [1, 5, 16, 24, 64, 200])
def test_attend_pages(lean, page):
    for window in (0, 1, 40):
        run_attend8(lean, [0, 3, 61, 500], 6, 2, 64, page=page, window=window, heads_first=page % 2 == 0)
    run_attend8(lean, [77, 300], 9, 1, 128, page=page, act="bf16", pad=8)


@pytest.mark.parametrize("dim,hq,hkv", [(64, 15, 5), (128, 16, 2), (256, 16, 2), (128, 32, 2)])
def test_attend_long(lean, dim, hq, hkv):
    """Sequences that many warps and blocks share, beside short ones."""
    run_attend8(lean, [9000, 3, 0, 700, 40], hq, hkv, dim)
    run_attend8(lean, [20000], hq, hkv, dim, act="bf16", page=24, window=15000)


@pytest.mark.parametrize("dim,hq", [(64, 4), (128, 16)])
def test_attend_folded(lean, dim, hq):
    """Sequences of more than 64 units in one warp's run, sizes of values that grow and shrink along them."""
    torch = torch_cuda()
    n, seqs = 2100, 2500
    kc, ks, vc, vs = make_cache8(17, 128, 1, dim, 5)
    vc.fill_(64)
    size = torch.exp2(torch.linspace(-12, 12, 17 * 128, device="cuda").sin() * 9).view(17, 128, 1)
    vs.copy_(size)
    q = normal(gen(hq), 1, hq, dim).repeat(seqs, 1, 1)
    table = torch.arange(17, device="cuda", dtype=torch.int32)[None].repeat(seqs, 1).contiguous()
    lens = torch.full((seqs,), n, device="cuda", dtype=torch.int32)
    out, lse = torch.zeros_like(q), torch.zeros((seqs, hq), device="cuda")
    ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(seqs, hq, 1, dim), dtype=torch.uint8, device="cuda")
    lean.lean_paged_attention(q, kc, vc, table, lens, out, scale=dim ** -0.5, lse=lse, workspace=ws, k_scales=ks, v_scales=vs)
    z = (q[0].double() @ (kc.double() * ks.double()[..., None]).view(-1, dim)[:n].T) * dim ** -0.5
    want = torch.softmax(z, -1) @ (vc.double() * vs.double()[..., None]).view(-1, dim)[:n]
    # every value is positive: sum p |v| is the output itself (step_testlib.run_attend's terms)
    reach = (q[0].double().abs() @ (kc.double() * ks.double()[..., None]).abs().view(-1, dim)[:n].T).amax(-1) * dim ** -0.5
    rel = (2.0 ** -15 + 20 * 2.0 ** -24) * reach + 2.0 ** -16 + (n / 8 + 68) * 2.0 ** -24
    assert bool(((out.double() - want[None]).abs() <= rel[:, None] * want + 2.0 ** -37 * 64 * float(vs.max())).all())
    assert bool(((lse.double() - torch.logsumexp(z, -1)).abs() <= rel + 1e-5).all())


@pytest.mark.parametrize("spread", [0.0, 3.0, 8.0])
def test_attend_scales_far_apart(lean, spread):
    """Tokens whose scales differ by up to e^30."""
    run_attend8(lean, [1, 40, 900], 6, 2, 64, spread=spread, scale=1e-3 if spread > 1 else None)
    run_attend8(lean, [300], 10, 1, 128, spread=spread, scale=1e-6, act="bf16")


def test_attend_zero_and_tiny_scales(lean):
    torch = torch_cuda()
    for size in (0.0, 1e-44, 1e-36, 1e30):
        inputs = list(make_attend8([5, 200], 4, 2, 64, 16, "f32"))
        fine = torch.isfinite(inputs[4])
        inputs[4] = torch.where(fine, size, inputs[4])
        run_attend8(lean, [5, 200], 4, 2, 64, inputs=inputs)


def test_attend_not_finite(lean):
    """A NaN or infinite scale reaches its sequence and kv head and no other."""
    torch = torch_cuda()
    for which, bad in ((2, math.nan), (4, math.nan), (4, math.inf), (2, math.inf), (2, -math.inf)):
        lens = [40, 70, 33]
        inputs = list(make_attend8(lens, 4, 2, 64, 16, "f32"))
        clean, _ = run_attend8(lean, lens, 4, 2, 64, inputs=inputs)
        page = int(inputs[5][1, 2])
        inputs[which] = inputs[which].clone()
        inputs[which][page, 3, 1] = bad
        q, kc, ks, vc, vs, table = inputs
        out = torch.zeros_like(q)
        ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(3, 4, 2, 64), dtype=torch.uint8, device="cuda")
        lean.lean_paged_attention(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, scale=0.125,
                                  workspace=ws, k_scales=ks, v_scales=vs)
        assert not bool(torch.isfinite(out[1, 2:]).any())
        assert torch.equal(out[1, :2], clean[1, :2]) and torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])


def test_attend_bad_pages(lean):
    torch = torch_cuda()
    lens = [40, 70, 33]
    for page in (16, 5):
        inputs = list(make_attend8(lens, 4, 2, 64, page, "f32"))
        clean, _ = run_attend8(lean, lens, 4, 2, 64, page=page, inputs=inputs)
        for bad in (-1, inputs[1].shape[0], 2 ** 31 - 1):
            q, kc, ks, vc, vs, table = inputs
            table = table.clone()
            table[1, 1] = bad
            out, lse = torch.zeros_like(q), torch.zeros((3, 4), device="cuda")
            ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(3, 4, 2, 64), dtype=torch.uint8, device="cuda")
            lean.lean_paged_attention(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, scale=0.125,
                                      workspace=ws, lse=lse, k_scales=ks, v_scales=vs)
            assert lean.lean_device_error(True) == 64
            assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())
            assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])


def test_append_attend_read_in_a_graph(lean):
    """A step as it is used, recorded and replayed: written in 8 bits, attended, read back; the lengths on the device."""
    torch = torch_cuda()
    n, hq, hkv, dim, page, width = 3, 6, 2, 64, 16, 4
    g = gen(77)
    kc, vc = (torch.zeros((n * width, page, hkv, dim), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (scales_like(kc, True, 0.0) for _ in range(2))
    table = torch.arange(n * width, dtype=torch.int32, device="cuda").view(n, width)
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    q, k, v = normal(g, n, hq, dim), normal(g, n, hkv, dim), normal(g, n, hkv, dim)
    slots, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    turns = torch.from_numpy(lean.lean_rope_turns(lean.lean_rope_frequencies(0, dim, 1e4))).cuda()
    q_out, out, k_back, v_back = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(lean.lean_paged_attention_workspace_bytes(n, hq, hkv, dim), dtype=torch.uint8, device="cuda")
    scales = dict(k_scales=ks, v_scales=vs)

    def step():
        lean.lean_rope_append(q, k, v, pos, slots, turns, q_out, kc, vc, rot_dim=dim, **scales)
        lean.lean_paged_attention(q_out, kc, vc, table, lens, out, scale=dim ** -0.5, workspace=ws, **scales)
        lean.lean_kv_read(kc, vc, slots, k_back, v_back, **scales)

    step()  # what a first call sets up
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for t in range(50):
        q.copy_(normal(g, n, hq, dim)), k.copy_(normal(g, n, hkv, dim)), v.copy_(normal(g, n, hkv, dim))
        lens.fill_(t + 1)
        pos.fill_(t)
        slots.copy_(table[:, t // page] * page + t % page)
        graph.replay()
    torch.cuda.synchronize()
    kd, vd = kc.double() * ks.double()[..., None], vc.double() * vs.double()[..., None]
    for s in range(n):
        keys, values = kd[s * width:(s + 1) * width].reshape(-1, hkv, dim)[:50], vd[s * width:(s + 1) * width].reshape(-1, hkv, dim)[:50]
        for h in range(hq):
            z = keys[:, h // 3] @ q_out[s, h].double() * dim ** -0.5
            want = torch.softmax(z, 0) @ values[:, h // 3]
            assert float((out[s, h].double() - want).abs().max()) < 1e-4 * float(values.abs().max())
        assert torch.equal(k_back[s], keys[49].float()) and torch.equal(v_back[s], values[49].float())


def test_on_another_stream(lean):
    torch = torch_cuda()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run_append8(lean, 40, 4, 2, 64, 64, "bf16")
        run_attend8(lean, [30, 200], 4, 2, 64, act="bf16", flags=lean.LEAN_FLAG_EARLY_WEIGHTS)
        run_read(lean, 40, 2, 64, flags=lean.LEAN_FLAG_EARLY_WEIGHTS)
    run_attend8(lean, [30, 200], 4, 2, 64, stream=side)


def test_same_every_time(lean):
    torch = torch_cuda()
    inputs = make_attend8([5000, 40, 900], 16, 2, 128, 16, "f32")
    first = run_attend8(lean, [5000, 40, 900], 16, 2, 128, inputs=inputs)
    for _ in range(3):
        again = run_attend8(lean, [5000, 40, 900], 16, 2, 128, inputs=inputs)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
