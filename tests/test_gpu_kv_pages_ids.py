"""lean_kv_pages on tables and rings that hold what is no page: such tokens get no
slot, bit 64 of the error word is set, and nothing else changes."""
import pytest

from lean_testlib import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    assert L.lean_device_error(True) == 0
    return L


def step(lean, page, in_table, in_ring):
    """Two sequences: the first grows inside its last page (in_table) and into one from the ring (in_ring), the second
    begins in a sound page, 5."""
    torch = torch_cuda()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, ring, state = ints([[in_table, -9], [-9, -9]]), ints([in_ring, 5, 6]), ints([0, 3])
    lens_out, so, st, starts = ints([0, 0]), ints([0, 0]), ints([9, 9]), ints([9] * 3)
    slots, pos, seqs = ints([-7] * 6), ints([-7] * 6), ints([-7] * 6)
    lean.lean_kv_pages(ints([page - 2, 0]), ints([page + 2, 1]), table, ring, state, page, lens_out, so, st, starts, slots,
                       pos, seqs)
    err = lean.lean_device_error(True)
    assert st.tolist() == [0, 0] and starts.tolist() == [0, 4, 5] and so.tolist() == [2, 1]
    assert table.tolist() == [[in_table, in_ring], [5, -9]] and lens_out.tolist() == [page + 2, 1]
    assert pos.tolist() == [page - 2, page - 1, page, page + 1, 0, 0] and seqs.tolist() == [0, 0, 0, 0, 1, -1]
    return slots.tolist(), err


@pytest.mark.parametrize("page", [4, 16, 1 << 20])
def test_what_is_no_page(lean, page):
    last = (2 ** 31 - 1) // page - 1  # the last page all of whose slots fit
    good = lambda a, b: [a * page + page - 2, a * page + page - 1, b * page, b * page + 1, 5 * page, -1]
    assert step(lean, page, 1, 2) == (good(1, 2), 0)
    assert step(lean, page, last, last) == (good(last, last), 0)
    for bad in (-1, -(2 ** 31), 2 ** 32 // page, 2 ** 31 // page, 2 ** 31 - 1):
        if bad >= 2 ** 31:
            continue
        g = good(1, 2)
        assert step(lean, page, bad, 2) == ([-1, -1] + g[2:], 64), bad
        assert step(lean, page, 1, bad) == (g[:2] + [-1, -1] + g[4:], 64), bad


def test_end_of_31_bits(lean):
    """A page that begins within 31 bits and ends past them: the slots that fit are slots."""
    page = 48
    edge = (2 ** 31 - 1) // page  # 31 of its places are below 2^31 - 1
    slots, err = step(lean, page, 3, edge)
    assert err == 0 and slots[2:4] == [edge * page, edge * page + 1]
    slots, err = step(lean, page, edge, 3)
    assert err == 64 and slots[:2] == [-1, -1] and slots[2:4] == [144, 145]
