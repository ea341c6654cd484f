"""lean_kv_pages over many steps on its own outputs, with and without slot maps:
sequences grow, shrink and end, the ring goes around, and pages are neither lost
nor doubled; each step against plain lists."""
import random

import pytest

from lean_testlib import torch_cuda
from step_testlib import pages_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


@pytest.mark.parametrize("maps", [(), ("slots",), ("positions", "token_seqs"), ("slots", "positions", "token_seqs")])
@pytest.mark.parametrize("limit", [150, 2 ** 31 - 1])
def test_walk(lean, maps, limit):
    torch = torch_cuda()
    if maps and limit > 150:
        limit = 1 << 12  # the maps have that many entries
    r = random.Random(6)
    n, page, width, pages = 37, 8, 12, 110
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, ring = ints([[-1] * width] * n), ints(list(range(pages)))
    state, lens = [ints([0, pages]), ints([0, 0])], [ints([0] * n), ints([0] * n)]
    status, starts = ints([0] * n), ints([0] * (n + 1))
    out = {name: ints([-9] * limit) for name in maps}
    names = ("lens", "table", "ring", "state", "status", "starts", "slots", "positions", "token_seqs")
    grown = shrunk = turns = 0
    seen = set()
    for step in range(60):
        a, b = step % 2, 1 - step % 2
        now = lens[a].tolist()
        want = [0 if r.random() < 0.1 else min(width * page, x + r.choice([1, 1, 1, 20])) if r.random() < 0.9 else x // 2
                for x in now]
        before = state[a].tolist()
        ref = dict(zip(names, pages_ref(now, want, table.tolist(), ring.tolist(), before, page, min(limit, 1 << 12))))
        lean.lean_kv_pages(lens[a], ints(want), table, ring, state[a], page, lens[b], state[b], status, starts,
                           max_tokens=limit, **out)
        got = dict(lens=lens[b], table=table, ring=ring, state=state[b], status=status, starts=starts, **out)
        for name, t in got.items():
            assert t.tolist() == ref[name], (step, name)
        held = [table[s, j].item() for s in range(n) for j in range(-(-ref["lens"][s] // page))]
        head, count = ref["state"]
        free = [ref["ring"][(head + i) % pages] for i in range(count)]
        assert sorted(held + free) == list(range(pages)), step
        grown += sum(g > x for g, x in zip(ref["lens"], now))
        shrunk += sum(g < x for g, x in zip(ref["lens"], now))
        turns += head < before[0]
        seen |= set(ref["status"])
    # the walk has gone through what it is for: growth, shrinking, the ring's end, and sequences that found no page or no room
    assert grown > 500 and shrunk > 100 and turns >= 1 and seen == ({0, 1, 3} if limit == 150 else {0, 1})


def test_limit_is_the_callers(lean):
    """max_tokens without maps, at the batch's size and one below; a limit that the maps do not have."""
    torch = torch_cuda()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")

    def call(**kw):
        table, ring, state = ints([[-1] * 4] * 2), ints(list(range(8))), ints([0, 8])
        lens_out, st, starts, so = ints([9, 9]), ints([9, 9]), ints([9] * 3), ints([9, 9])
        lean.lean_kv_pages(ints([0, 0]), ints([10, 7]), table, ring, state, 16, lens_out, so, st, starts, **kw)
        return lens_out.tolist(), st.tolist(), so.tolist(), starts.tolist()

    assert call(max_tokens=17) == ([10, 7], [0, 0], [2, 6], [0, 10, 17])
    assert call(max_tokens=2 ** 31 - 1) == ([10, 7], [0, 0], [2, 6], [0, 10, 17])
    assert call(max_tokens=16) == ([10, 0], [0, 3], [1, 7], [0, 10, 17])
    assert call(slots=ints([0] * 17)) == ([10, 7], [0, 0], [2, 6], [0, 10, 17])
    with pytest.raises(ValueError):
        call(max_tokens=18, slots=ints([0] * 17))
    with pytest.raises(lean.LeanError):
        call(max_tokens=-1)
