"""lean_prefix_attention: sequences that share prefixes, against 64 bits."""
import math

import pytest

from cache_testlib import make_prefix, run_prefix
from lean_testlib import torch_cuda

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


def starts_of(counts, first=0):
    out = [first]
    for c in counts:
        out.append(out[-1] + c)
    return out


TYPES = [("f32", "bf16"), ("f32", "f16"), ("f32", "i8"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "i8"), ("f16", "bf16"),
         ("bf16", "f16"), ("f16", "i8")]


@pytest.mark.parametrize("act,cache", TYPES)
def test_smallest(lean, act, cache):
    """One prefix and one sequence."""
    run_prefix(lean, [1], [0, 1], [1], 1, 1, 64, act=act, cache=cache)
    run_prefix(lean, [40], [0, 2], [3, 1], 4, 2, 64, act=act, cache=cache)
    run_prefix(lean, [130], [0, 2], [3, 1], 4, 2, 128, act=act, cache=cache)


@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("hq,hkv,dim", [(4, 4, 64), (6, 2, 80), (8, 1, 128), (34, 2, 64), (15, 5, 96), (2, 1, 16), (3, 1, 112)])
def test_types_and_heads(lean, hq, hkv, dim, act, cache):
    """Prefixes of no, of few and of some hundred tokens; of no sequence; sequences without a prefix, without own tokens,
    and without any."""
    run_prefix(lean, [0, 1, 128, 300, 129], starts_of([2, 1, 0, 4, 2], 1), [5, 0, 17, 40, 1, 0, 16, 200, 33, 3, 0, 9],
               hq, hkv, dim, act=act, cache=cache)


@pytest.mark.parametrize("act,cache", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "i8")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length", [127, 128, 129, 255, 257, 1000])
def test_two_tiles_of_rows(lean, length, dim, act, cache):
    """More than 128 and more than 256 rows of a kv head; the last tile and the second half of the first nearly empty."""
    for seqs, hq, hkv in ((17, 8, 1), (33, 16, 2), (65, 4, 1)):
        run_prefix(lean, [length], [0, seqs], [1 + i % 5 for i in range(seqs)], hq, hkv, dim, act=act, cache=cache)


@pytest.mark.parametrize("act,cache", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "i8"), ("f32", "i8")])
@pytest.mark.parametrize("dim", [64, 128])
def test_long(lean, dim, act, cache):
    """Runs of many tiles; parts of one prefix in every block; long and short prefixes in a block's run."""
    run_prefix(lean, [40000], [0, 3], [1, 100, 0], 8, 4, dim, act=act, cache=cache, page=64)
    run_prefix(lean, [30000, 77, 12000, 128], starts_of([20, 3, 50, 1]), [i % 40 for i in range(74)], 8, 2, dim, act=act,
               cache=cache, page=64)


@pytest.mark.parametrize("act,cache", [("f32", "bf16"), ("bf16", "bf16"), ("bf16", "i8")])
def test_many_prefixes(lean, act, cache):
    """More prefixes than a block has threads, most of them short."""
    lens = [(37 * i) % 300 for i in range(700)]
    counts = [1 + i % 2 for i in range(700)]
    run_prefix(lean, lens, starts_of(counts), [1 + i % 3 for i in range(sum(counts))], 4, 2, 64, act=act, cache=cache)


@pytest.mark.parametrize("cache", ["bf16", "i8"])
@pytest.mark.parametrize("page", [1, 5, 16, 24, 64, 200])
def test_pages(lean, page, cache):
    for heads_first in (True, False):
        run_prefix(lean, [61, 500], [0, 2, 5], [3, 0, 30, 100, 1], 6, 2, 64, page=page, cache=cache, heads_first=heads_first,
                   extra=2)
    run_prefix(lean, [700], [0, 40], [3] * 40, 8, 2, 128, page=page, cache=cache, act="bf16", pad=8)


def test_lengths_past_the_table(lean):
    """Lengths below 0 count as 0, past the table as all of it."""
    torch = torch_cuda()
    inputs = make_prefix([64, 32], [16, 16, 16], 4, 2, 64)
    inputs = list(inputs)
    q, kc, ks, vc, vs, shared, table = inputs
    shared = shared.clone()
    shared[1, 2:] = shared[0, 2:]
    whole, _ = run_prefix(lean, [64, 64], [0, 2, 3], [16, 0, 16], 4, 2, 64, inputs=(q, kc, ks, vc, vs, shared, table))
    out = torch.zeros_like(q)
    ws = torch.empty(lean.lean_prefix_attention_workspace_bytes(3, 4, 2, 64, 2), dtype=torch.uint8, device="cuda")
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lean.lean_prefix_attention(q, kc, vc, shared, ints([2 ** 31 - 1, 65]), ints([0, 2, 3]), table, ints([99, -7, 2 ** 31 - 1]),
                               out, scale=0.125, workspace=ws)
    assert torch.equal(out, whole)


def test_nothing_at_all(lean):
    out, lse = run_prefix(lean, [0], [0, 2], [0, 0, 0], 4, 2, 64)
    assert not bool(out.any()) and bool((lse == -math.inf).all())


def test_starts_that_do_not_ascend(lean):
    """Sequences that no such prefix concerns are right; nothing is read or written outside."""
    torch = torch_cuda()
    inputs = make_prefix([200, 300, 100], [5, 6, 7, 8, 9, 10], 4, 2, 64)
    q, kc, ks, vc, vs, shared, table = inputs
    right, _ = run_prefix(lean, [200, 300, 100], [0, 2, 4, 6], [5, 6, 7, 8, 9, 10], 4, 2, 64, inputs=inputs)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(lean.lean_prefix_attention_workspace_bytes(6, 4, 2, 64, 3), dtype=torch.uint8, device="cuda")
    for starts, fine in (([0, 2, 1, 1], [0, 1]), ([-5, 2, 4, 99], [0, 1, 2, 3, 4, 5]), ([4, 0, 2 ** 31 - 1, -2 ** 31], []),
                         ([9, 9, 9, 9], [])):
        out = torch.zeros_like(q)
        lean.lean_prefix_attention(q, kc, vc, shared, ints([200, 300, 100]), ints(starts), table, ints([5, 6, 7, 8, 9, 10]), out,
                                   scale=0.125, workspace=ws)
        for s in fine:
            if starts[0] != 0 or s < 1:  # (where prefixes overlap, which one counts is open)
                assert torch.equal(out[s], right[s]), (starts, s)
    assert lean.lean_device_error(True) == 0


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, 1e-30])
@pytest.mark.parametrize("act,cache", [("f32", "bf16"), ("bf16", "i8"), ("f16", "f16")])
def test_scales_of_scores(lean, scale, act, cache):
    run_prefix(lean, [200, 129], [0, 2, 45], [i % 7 for i in range(45)], 8, 2, 64, act=act, cache=cache, scale=scale)


@pytest.mark.parametrize("spread", [3.0, 8.0])
def test_scales_far_apart(lean, spread):
    """Tokens in 8 bits whose scales differ by up to e^30."""
    for act in ("f32", "bf16"):
        run_prefix(lean, [500, 40], [0, 2, 45], [i % 7 for i in range(45)], 8, 2, 64, act=act, cache="i8", spread=spread, scale=1e-5)


def test_values_of_zero_beside_large_ones(lean):
    """Whole tiles of values that are 0 or tiny after and before large ones: p keeps counting in the sum."""
    torch = torch_cuda()
    inputs = list(make_prefix([1024], [3] * 20, 8, 1, 64, page=128, act="bf16", cache="i8"))
    vs = inputs[4]
    shared = inputs[5][0].long()
    for tile, size in zip(range(8), (0.0, 1e25, 0.0, 1e-25, 1.0, 1e30, 0.0, 1e-44)):
        vs[shared[tile]] = size
    run_prefix(lean, [1024], [0, 20], [3] * 20, 8, 1, 64, page=128, act="bf16", cache="i8", inputs=inputs)
    run_prefix(lean, [1024], [0, 2], [3] * 20, 8, 1, 64, page=128, act="bf16", cache="i8", inputs=inputs)


def test_one_key_far_above_many(lean):
    """What many small probabilities give beside one large one: 4000 keys 12 nats below it."""
    torch = torch_cuda()
    for act, cache in (("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16")):
        inputs = list(make_prefix([4096], [0, 0], 2, 1, 64, page=64, act=act, cache=cache))
        q, kc, vc, shared = inputs[0], inputs[1], inputs[3], inputs[5][0].long()
        q.zero_()
        q[..., 0] = 1.0
        kc[shared] = 0
        kc[shared[3], 5, 0, 0] = 12.0
        vc[shared] = 1.0
        vc[shared[3], 5] = 0.0
        run_prefix(lean, [4096], [0, 2], [0, 0], 2, 1, 64, page=64, act=act, cache=cache, scale=1.0, inputs=inputs)


@pytest.mark.parametrize("cache", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_bad_pages(lean, act, cache):
    """A page outside the cache: NaN for the sequences of its prefix, or for its sequence, and for no other."""
    torch = torch_cuda()
    starts, lens = [0, 2, 40], [5 + i % 40 for i in range(42)]
    inputs = make_prefix([200, 300], lens, 8, 2, 64, act=act, cache=cache)
    right, _ = run_prefix(lean, [200, 300], starts, lens, 8, 2, 64, act=act, cache=cache, inputs=inputs)
    q, kc, ks, vc, vs, shared, table = inputs
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(lean.lean_prefix_attention_workspace_bytes(42, 8, 2, 64, 2), dtype=torch.uint8, device="cuda")
    for bad in (-1, kc.shape[0], 2 ** 31 - 1):
        for which, hurt in (((0, 0, 3), [0, 1]), ((0, 1, 18), list(range(2, 40))), ((1, 41, 0), [41])):
            sh, tab = shared.clone(), table.clone()
            (tab if which[0] else sh)[which[1], which[2]] = bad
            out, lse = torch.zeros_like(q), torch.zeros((42, 8), device="cuda")
            lean.lean_prefix_attention(q, kc, vc, sh, ints([200, 300]), ints(starts), tab, ints(lens), out, scale=0.125, lse=lse,
                                       workspace=ws, k_scales=ks, v_scales=vs)
            assert lean.lean_device_error(True) == 64
            for s in range(42):
                if s in hurt:
                    assert bool(torch.isnan(out[s]).all()) and bool(torch.isnan(lse[s]).all()), (which, s)
                else:
                    assert torch.equal(out[s], right[s]), (which, s)


@pytest.mark.parametrize("cache", ["bf16", "i8"])
def test_not_finite(lean, cache):
    """A NaN or infinity in a prefix reaches the sequences that share it, of its kv head."""
    torch = torch_cuda()
    lens = [4] * 24
    inputs = make_prefix([200, 300], lens, 8, 2, 64, act="bf16", cache=cache)
    right, _ = run_prefix(lean, [200, 300], [0, 20, 24], lens, 8, 2, 64, act="bf16", cache=cache, inputs=inputs)
    for which, bad in ((1, math.nan), (3, math.nan), (3, math.inf), (1, math.inf)):
        x = list(inputs)
        at = which + (1 if cache == "i8" else 0)
        x[at] = x[at].clone()
        x[at][int(x[5][0, 7]), 3, 1] = bad
        q, kc, ks, vc, vs, shared, table = x
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        out = torch.zeros_like(q)
        ws = torch.zeros(lean.lean_prefix_attention_workspace_bytes(24, 8, 2, 64, 2), dtype=torch.uint8, device="cuda")
        lean.lean_prefix_attention(q, kc, vc, shared, ints([200, 300]), ints([0, 20, 24]), table, ints(lens), out, scale=0.125,
                                   workspace=ws, k_scales=ks, v_scales=vs)
        assert not bool(torch.isfinite(out[:20, 4:]).any())
        assert torch.equal(out[:20, :4], right[:20, :4]) and torch.equal(out[20:], right[20:])


def test_same_as_attention_over_joined_tables(lean):
    """Sequences whose block tables begin with the prefix's pages give the same through lean_paged_attention."""
    torch = torch_cuda()
    n, hq, hkv, dim, page = 20, 8, 2, 128, 16
    lens = [1 + 3 * i for i in range(n)]
    q, kc, ks, vc, vs, shared, table = make_prefix([480], lens, hq, hkv, dim, page=page)
    out, lse = run_prefix(lean, [480], [0, n], lens, hq, hkv, dim, page=page, inputs=(q, kc, ks, vc, vs, shared, table))
    joined = torch.cat([shared.expand(n, -1), table], 1).contiguous()
    other, other_lse = torch.zeros_like(q), torch.zeros((n, hq), device="cuda")
    ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(n, hq, hkv, dim), dtype=torch.uint8, device="cuda")
    lean.lean_paged_attention(q, kc, vc, joined, torch.tensor([480 + x for x in lens], dtype=torch.int32, device="cuda"), other,
                              scale=dim ** -0.5, lse=other_lse, workspace=ws)
    assert float((out - other).abs().max()) < 1e-4 and float((lse - other_lse).abs().max()) < 1e-4


def test_in_a_graph_and_on_another_stream(lean):
    torch = torch_cuda()
    lens = [3 + i for i in range(30)]
    inputs = make_prefix([1000, 200], lens, 8, 2, 64, act="bf16")
    right, right_lse = run_prefix(lean, [1000, 200], [0, 25, 30], lens, 8, 2, 64, act="bf16", inputs=inputs)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out, lse = run_prefix(lean, [1000, 200], [0, 25, 30], lens, 8, 2, 64, act="bf16", inputs=inputs,
                              flags=lean.LEAN_FLAG_EARLY_WEIGHTS)
    assert torch.equal(out, right) and torch.equal(lse, right_lse)
    q, kc, ks, vc, vs, shared, table = inputs
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pl, st, ld = ints([1000, 200]), ints([0, 25, 30]), ints(lens)
    out = torch.zeros_like(q)
    ws = torch.empty(lean.lean_prefix_attention_workspace_bytes(30, 8, 2, 64, 2), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        for _ in range(2):
            lean.lean_prefix_attention(q, kc, vc, shared, pl, st, table, ld, out, scale=0.125, workspace=ws,
                                       flags=lean.LEAN_FLAG_EARLY_WEIGHTS)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, right)
    # other lengths, read when it is replayed
    pl.copy_(ints([777, 1]))
    ld.copy_(ints([1] * 30))
    graph.replay()
    torch.cuda.synchronize()
    other, _ = run_prefix(lean, [777, 1], [0, 25, 30], [1] * 30, 8, 2, 64, act="bf16", inputs=inputs)
    assert torch.equal(out, other)


def test_same_every_time(lean):
    torch = torch_cuda()
    for act, cache in (("f32", "bf16"), ("bf16", "i8")):
        lens = [3 + i for i in range(30)]
        inputs = make_prefix([5000, 200], lens, 8, 2, 64, act=act, cache=cache)
        first = run_prefix(lean, [5000, 200], [0, 25, 30], lens, 8, 2, 64, act=act, cache=cache, inputs=inputs)
        for _ in range(3):
            again = run_prefix(lean, [5000, 200], [0, 25, 30], lens, 8, 2, 64, act=act, cache=cache, inputs=inputs)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
