"""lean_kv_pages against plain lists: growth, shrinking and ends over many
sequences, the ring's wrap, every failure, odd page sizes, strides, and a random
walk of many steps that must neither lose nor double a page."""
import random

import pytest

from lean_testlib import torch_cuda
from step_testlib import run_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


def pool(lens, page, width, spare, head=0, seed=0):
    """(table, ring, state) in which sequence s owns ceil(lens[s] / page) pages."""
    r = random.Random(seed)
    ids = list(range(sum(-(-max(x, 0) // page) for x in lens) + spare))
    size = len(ids)
    r.shuffle(ids)
    table = [[-1] * width for _ in lens]
    for s, x in enumerate(lens):
        for j in range(min(width, -(-max(x, 0) // page))):
            table[s][j] = ids.pop()
    ring = [-5] * size
    for i, pg in enumerate(ids):
        ring[(head + i) % size] = pg
    return table, ring, [head, len(ids)]


@pytest.mark.parametrize("n", [1, 2, 31, 511, 512, 513, 1100])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_mixed(lean, n, page):
    r = random.Random(n * 100 + page)
    lens = [r.choice([0, 1, page, page + 1, r.randrange(0, 200)]) for _ in range(n)]
    targets = [r.choice([0, x, x + 1, x + r.randrange(0, 100), r.randrange(0, x + 1)]) for x in lens]
    width = max(-(-max(a, b) // page) for a, b in zip(lens, targets)) + 1
    need = sum(max(0, -(-b // page) - -(-a // page)) for a, b in zip(lens, targets))
    table, ring, state = pool(lens, page, width, need + 5, head=3, seed=n)
    total = sum(max(0, b - a) for a, b in zip(lens, targets))
    run_pages(lean, lens, targets, table, ring, state, page, total + 7)
    run_pages(lean, lens, targets, table, ring, state, page, total, pad=3)


@pytest.mark.parametrize("head", [0, 1, 9, 19])
def test_ring_wraps(lean, head):
    lens, targets = [16, 40, 0, 100], [40, 0, 33, 100]
    table, ring, state = pool(lens, 16, 8, 9, head=head)
    run_pages(lean, lens, targets, table, ring, state, 16, 64)


def test_decode_steps(lean):
    """Every sequence one more token; and nothing to do at all."""
    lens = list(range(40))
    table, ring, state = pool(lens, 16, 4, 40)
    run_pages(lean, lens, [x + 1 for x in lens], table, ring, state, 16, 40)
    run_pages(lean, lens, lens, table, ring, state, 16, 0)
    run_pages(lean, lens, lens, table, ring, state, 16, 5)


def test_out_of_pages(lean):
    """From the first sequence that finds too few pages on, those that need any fail; the others go on."""
    lens, targets = [10, 16, 5, 16, 16, 48], [20, 17, 6, 80, 17, 16]
    table, ring, state = pool(lens, 16, 8, 3)
    got = run_pages(lean, lens, targets, table, ring, state, 16, 200)
    assert got[4].tolist() == [0, 0, 0, 1, 1, 0]
    table, ring, state = pool(lens, 16, 8, 0)
    run_pages(lean, lens, targets, table, ring, state, 16, 200)


def test_failures(lean):
    lens, targets = [16, 0, 100, -3, 5, 4], [100, 3, 4, 5, -1, 6]
    table, ring, state = pool(lens, 16, 6, 8)
    got = run_pages(lean, lens, targets, table, ring, state, 16, 200)
    assert got[4].tolist() == [2, 0, 2, 4, 4, 0]
    # the batch is too small: tokens past its end are not written
    lens, targets = [0, 0, 0, 7], [10, 10, 10, 7]
    table, ring, state = pool(lens, 4, 6, 12)
    got = run_pages(lean, lens, targets, table, ring, state, 4, 15)
    assert got[4].tolist() == [0, 3, 3, 0] and got[5].tolist() == [0, 10, 20, 30, 30]
    # a state outside the ring
    for bad in ([-1, 2], [12, 2], [0, 13], [3, -1]):
        table, ring, _ = pool([4, 4], 4, 6, 10)
        got = run_pages(lean, [4, 4], [8, 0], table, ring, bad, 4, 15)
        assert got[4].tolist() == [4, 4]
    # more pages come back than the ring can hold
    table, ring, state = pool([16, 16], 4, 6, 2)
    ring, state = ring[:5], [1, 2]
    got = run_pages(lean, [16, 4], [4, 0], table, ring, state, 4, 15)
    assert got[4].tolist() == [0, 4]


def test_large_lengths(lean):
    """Lengths near 2^31 - 1 are sequences like others (their pages do not fit a table here)."""
    top = 2 ** 31 - 1
    table, ring, state = pool([0, 5, 0], 1 << 20, 2048, 3000)
    run_pages(lean, [0, 5, 0], [top, 5, 12], table, ring, state, 1 << 20, 50)
    table, ring, state = pool([0, 0, 0], 16, 4, 10)
    run_pages(lean, [0, 0, 0], [top, top, 12], table, ring, state, 16, 50)


def test_parts_left_out(lean):
    lens, targets = [3, 20], [9, 40]
    for outputs in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        table, ring, state = pool(lens, 16, 4, 9)
        run_pages(lean, lens, targets, table, ring, state, 16, 26 if any(outputs) else 0, outputs=outputs)


def test_long_prompts(lean):
    """Far more tokens than one pass of the grid."""
    r = random.Random(5)
    lens = [r.randrange(0, 3000) for _ in range(300)]
    targets = [x + r.randrange(0, 2500) for x in lens]
    need = sum(-(-b // 16) - -(-a // 16) for a, b in zip(lens, targets))
    table, ring, state = pool(lens, 16, 400, need, head=77)
    total = sum(b - a for a, b in zip(lens, targets))
    assert total > 152 * 512
    run_pages(lean, lens, targets, table, ring, state, 16, total + 1000)


def test_random_walk(lean):
    """Many steps in a row, on the device's own outputs: pages are conserved and no two sequences share one."""
    torch = torch_cuda()
    r = random.Random(6)
    n, page, width, pages = 37, 8, 12, 200
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table = ints([[-1] * width] * n)
    ring, state = ints(list(range(pages))), [ints([0, pages]), ints([0, 0])]
    lens = [ints([0] * n), ints([0] * n)]
    status, starts = ints([0] * n), ints([0] * (n + 1))
    for step in range(60):
        a, b = step % 2, 1 - step % 2
        now = lens[a].tolist()
        want = [0 if r.random() < 0.1 else min(width * page, x + r.choice([1, 1, 1, 20])) if r.random() < 0.9 else x // 2
                for x in now]
        lean.lean_kv_pages(lens[a], ints(want), table, ring, state[a], page, lens[b], state[b], status, starts)
        got, st = lens[b].tolist(), status.tolist()
        assert all(g == (w if s == 0 else o) for g, w, s, o in zip(got, want, st, now))
        rows, (head, count), q = table.tolist(), state[b].tolist(), ring.tolist()
        held = [rows[s][j] for s in range(n) for j in range(-(-got[s] // page))]
        free = [q[(head + i) % pages] for i in range(count)]
        assert sorted(held + free) == list(range(pages)), step


def test_captured(lean):
    """A step recorded into a graph, replayed from a changed state."""
    torch = torch_cuda()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    lens, targets, table = ints([4, 0]), ints([5, 3]), ints([[7, -1], [-1, -1]])
    ring, state, lo, so, st, starts, slots = ints([3, 4, 5, 6]), ints([0, 4]), ints([0, 0]), ints([0, 0]), ints([0, 0]), ints([0] * 3), ints([0] * 6)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        lean.lean_kv_pages(lens, targets, table, ring, state, 4, lo, so, st, starts, slots, flags=lean.LEAN_FLAG_EARLY_WEIGHTS)
    g.replay()
    torch.cuda.synchronize()
    assert table.tolist() == [[7, 3], [4, -1]] and slots.tolist() == [12, 16, 17, 18, -1, -1] and so.tolist() == [2, 2]
    state.copy_(ints([3, 1]))
    g.replay()
    torch.cuda.synchronize()
    assert table.tolist() == [[7, 6], [4, -1]] and st.tolist() == [0, 1] and so.tolist() == [0, 0]
