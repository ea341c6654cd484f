"""GPU parity of lean_paged_attention with its definition in 64 bits: lengths from
none to many pages, windows, shared heads, head sizes, page sizes that do not
divide anything, types, layouts; what must not be read holds NaN throughout."""
import math

import pytest

from lean_testlib import torch_cuda
from step_testlib import attend_ref, close, dtype, gen, make_attend, normal, run_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


@pytest.mark.parametrize("length", [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 127, 128, 129, 500, 2049])
@pytest.mark.parametrize("dim", [64, 128])
def test_lengths(lean, length, dim):
    run_attend(lean, [length], 6, 2, dim, seed=length)


def test_ragged_batch(lean):
    run_attend(lean, [5, 0, 1000, 17, 1, 0, 333, 16, 64, 2500, 0], 15, 5, 64)
    run_attend(lean, [0, 0, 0], 8, 1, 128)
    run_attend(lean, [1] * 300, 4, 2, 64)
    run_attend(lean, [3, 700, 12] * 40, 8, 2, 128, act="bf16")


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (8, 1), (9, 1), (12, 1), (16, 1), (17, 1), (40, 1), (71, 1),
                                    (8, 8), (15, 5), (32, 4), (16, 2), (24, 2), (128, 8)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_shared_heads(lean, hq, hkv, dim):
    run_attend(lean, [130, 9, 0, 411], hq, hkv, dim, seed=hq)


@pytest.mark.parametrize("dim", [8, 16, 24, 40, 64, 72, 80, 96, 104, 128, 136, 192, 200, 248, 256])
@pytest.mark.parametrize("act,cache", [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16"), ("f16", "bf16")])
def test_head_sizes(lean, dim, act, cache):
    run_attend(lean, [100, 3, 257], 6, 3, dim, act=act, cache=cache, seed=dim)


@pytest.mark.parametrize("page", [1, 2, 5, 8, 15, 16, 17, 24, 32, 48, 64, 100, 128, 256])
def test_page_sizes(lean, page):
    run_attend(lean, [300, page, page + 1, max(0, page - 1), 3 * page, 1], 4, 2, 64, page=page, seed=page)
    run_attend(lean, [300, 2 * page + 3], 16, 2, 128, page=page, window=70, seed=page)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 1000, 2 ** 31 - 1])
def test_windows(lean, window):
    run_attend(lean, [0, 1, 16, 17, 99, 100, 101, 117, 1500], 6, 2, 64, window=window, seed=window % 1000)


@pytest.mark.parametrize("kw", [dict(heads_first=True), dict(pad=8), dict(lse=False), dict(spare="inf"), dict(width=200),
                                dict(scale=1.0), dict(scale=-0.3), dict(scale=0.0)])
def test_layouts(lean, kw):
    run_attend(lean, [77, 300, 0, 5], 6, 2, 64, seed=1, **kw)
    run_attend(lean, [77, 300, 0, 5], 16, 2, 128, act="bf16", seed=2, **kw)


def test_lengths_out_of_range(lean):
    """A length below 0 counts as 0, one past the table as all of the table."""
    torch = torch_cuda()
    q, kc, vc, table = make_attend([32, 32, 16], 4, 2, 64, 16, "f32", "bf16", seed=3)
    table[2, 1] = table[0, 0]  # a page for the third sequence too
    run_attend(lean, [-5, 1 << 30, 2 ** 31 - 1], 4, 2, 64, inputs=(q, kc, vc, table))
    assert lean.lean_device_error(True) == 0
    assert torch.cuda.is_available()


@pytest.mark.parametrize("big", [30.0, 300.0, 3e4])
@pytest.mark.parametrize("cache", ["bf16", "f16"])
def test_sharp_scores(lean, big, cache):
    """Scores far apart: one key takes all, and the maximum moves late or early."""
    torch = torch_cuda()
    q, kc, vc, table = make_attend([513, 513], 4, 1, 64, 16, "f32", cache, seed=4)
    q[:] = 0
    q[:, :, 0] = big
    lens = [513, 513]
    for s in range(2):
        t = torch.arange(513, device="cuda")
        rows = table[s].long()[t // 16], t % 16
        ramp = torch.linspace(-1, 1, 513, device="cuda")
        kc[rows[0], rows[1], 0, 0] = (ramp if s == 0 else -ramp).to(kc.dtype)
    run_attend(lean, lens, 4, 1, 64, cache=cache, inputs=(q, kc, vc, table))


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e6, 1e30])
@pytest.mark.parametrize("cache", ["bf16", "f16"])
def test_query_sizes(lean, size, cache):
    """q of any size against keys scaled to meet it: no part of q may overflow or vanish in the cache's type."""
    q, kc, vc, table = make_attend([200], 4, 2, 64, 16, "f32", cache, seed=5)
    q *= size
    run_attend(lean, [200], 4, 2, 64, cache=cache, inputs=(q, kc, vc, table), scale=0.125 / size if size < 1e20 else 0.125e-30)


def test_values_not_finite(lean):
    """An infinite key or value that is attended shows; one that is not does not."""
    torch = torch_cuda()
    q, kc, vc, table = make_attend([40, 40], 2, 1, 64, 16, "f32", "bf16", seed=6)
    vc[int(table[0, 1]), 3, 0, 5] = float("inf")
    vc[int(table[1, 0]), 3, 0, 5] = float("nan")  # position 3: before the window of 30
    size = lean.lean_paged_attention_workspace_bytes(2, 2, 1, 64)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    out = torch.empty((2, 2, 64), device="cuda")
    lens = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    lean.lean_paged_attention(q, kc, vc, table, lens, out, scale=0.125, window=30, workspace=ws)
    assert not bool(torch.isfinite(out[0, :, 5]).any())
    keep = [d for d in range(64) if d != 5]
    assert bool(torch.isfinite(out[0][:, keep]).all()) and bool(torch.isfinite(out[1]).all())


def test_bad_pages(lean):
    """A page outside the cache: its sequence is NaN, bit 64 is set, the others are right, and the workspace stays fit
    for the next call."""
    torch = torch_cuda()
    assert lean.lean_device_error(True) == 0
    for dim, hq in ((64, 4), (128, 24)):
        lens = [700, 700, 700]
        q, kc, vc, table = make_attend(lens, hq, 2, dim, 16, "f32", "bf16", seed=7)
        want, want_lse, size, _ = attend_ref(q, kc, vc, table, lens, 0.125, 0)
        good = table.clone()
        ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(3, hq, 2, dim), dtype=torch.uint8, device="cuda")
        ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for bad in (-1, kc.shape[0], 2 ** 31 - 1):
            table[1, 20] = bad
            out, lse = torch.zeros((3, hq, dim), device="cuda"), torch.zeros((3, hq), device="cuda")
            lean.lean_paged_attention(q, kc, vc, table, ld, out, scale=0.125, lse=lse, workspace=ws)
            assert lean.lean_device_error(True) == 64
            assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())
            for s in (0, 2):
                close(out[s], want[s], 1e-3 * size[s], "beside a bad page")
            lean.lean_paged_attention(q, kc, vc, good, ld, out, scale=0.125, lse=lse, workspace=ws)
            close(out, want, 1e-3 * size, "after a bad page")
        # past the length nothing looks at the table
        table[1, 20] = good[1, 20]
        assert lean.lean_device_error(True) == 0


@pytest.mark.parametrize("page", [5, 17, 20, 24])
def test_pages_that_end_inside_a_unit(lean, page):
    """Windows that begin at every place of a page; table entries of no attended token may be anything, the entry of
    one attended token may not."""
    torch = torch_cuda()
    assert lean.lean_device_error(True) == 0
    for window in range(60, 60 + page):
        run_attend(lean, [0, 59, 200, 3 * page], 4, 2, 64, page=page, window=window, seed=window)
    length, window = 10 * page + 1, 2 * page + 1  # the last three pages, one token of the last
    q, kc, vc, table = make_attend([length] * 2, 4, 2, 64, page, "f32", "bf16", seed=page, width=13)
    want, _, size, _ = attend_ref(q, kc, vc, table, [length] * 2, 0.125, window)
    ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(2, 4, 2, 64), dtype=torch.uint8, device="cuda")
    ld = torch.tensor([length] * 2, dtype=torch.int32, device="cuda")
    out = torch.zeros((2, 4, 64), device="cuda")
    table[:, :8] = -1
    lean.lean_paged_attention(q, kc, vc, table, ld, out, scale=0.125, window=window, workspace=ws)
    assert lean.lean_device_error(True) == 0
    close(out, want, 1e-3 * size, "entries of no attended token")
    for entry in (8, 10):
        bad = table.clone()
        bad[0, entry] = kc.shape[0]
        lean.lean_paged_attention(q, kc, vc, bad, ld, out, scale=0.125, window=window, workspace=ws)
        assert lean.lean_device_error(True) == 64
        assert bool(torch.isnan(out[0]).all())
        close(out[1], want[1], 1e-3 * size[1], "beside a bad page")


def test_lse_joins_two_caches(lean):
    """Attention over two halves, joined by their lse, is attention over the whole."""
    torch = torch_cuda()
    q, kc, vc, table = make_attend([640], 4, 2, 64, 16, "f32", "f16", seed=8)
    whole, wl = run_attend(lean, [640], 4, 2, 64, cache="f16", inputs=(q, kc, vc, table))
    a, al = run_attend(lean, [320], 4, 2, 64, cache="f16", inputs=(q, kc, vc, table))
    b, bl = run_attend(lean, [320], 4, 2, 64, cache="f16", inputs=(q, kc, vc, table[:, 20:].contiguous()))
    both = torch.logaddexp(al.double(), bl.double())
    joined = a.double() * (al - both).exp()[..., None] + b.double() * (bl - both).exp()[..., None]
    close(wl, both, 1e-5, "lse")
    close(whole, joined, 2e-5, "out")


def test_deterministic_and_workspace_reused(lean):
    """The same call gives the same bits, and one workspace serves calls of other lengths in turn."""
    torch = torch_cuda()
    hq, hkv, dim = 16, 2, 128
    ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(4, hq, hkv, dim), dtype=torch.uint8, device="cuda")
    seen = {}
    for lens in ([4000, 3, 900, 0], [1, 1, 1, 1], [9000, 9000, 9000, 9000], [4000, 3, 900, 0], [0, 0, 0, 5000],
                 [9000, 9000, 9000, 9000]):
        out, lse = run_attend(lean, lens, hq, hkv, dim, seed=9, workspace=ws)
        key = tuple(lens)
        if key in seen:
            assert torch.equal(out, seen[key][0]) and torch.equal(lse, seen[key][1])
        seen[key] = out, lse


def test_long_cache(lean):
    """A long sequence alone, and next to short ones; types as a serving step has them."""
    run_attend(lean, [40001], 15, 5, 64, seed=10)
    run_attend(lean, [30000, 12, 0, 2000], 16, 2, 128, act="bf16", page=64, seed=11)


def test_far_pages(lean):
    """Offsets past 2^31 elements in a large cache."""
    torch = torch_cuda()
    pages, page, heads, dim = 70000, 128, 2, 128
    kc = torch.zeros((pages, page, heads, dim), device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    g = gen(12)
    table = torch.tensor([[pages - 1, 3, 68001]], dtype=torch.int32, device="cuda")
    for p in table[0].tolist():
        kc[p], vc[p] = normal(g, page, heads, dim, t="bf16"), normal(g, page, heads, dim, t="bf16")
    q = normal(g, 1, 8, dim)
    run_attend(lean, [300], 8, 2, dim, page=128, inputs=(q, kc, vc, table))


def test_stream_graph_flag(lean):
    torch = torch_cuda()
    run_attend(lean, [100, 2000], 8, 2, 64, stream=torch.cuda.Stream(), seed=13)
    lens = [1200, 77]
    q, kc, vc, table = make_attend(lens, 8, 2, 64, 16, "f32", "bf16", seed=14)
    want, _, size, _ = attend_ref(q, kc, vc, table, lens, 0.125, 0)
    ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(2, 8, 2, 64), dtype=torch.uint8, device="cuda")
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.empty((2, 8, 64), device="cuda")
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        for _ in range(5):
            lean.lean_paged_attention(q, kc, vc, table, ld, out, scale=0.125, workspace=ws,
                                      flags=lean.LEAN_FLAG_EARLY_WEIGHTS)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        close(out, want, 1e-3 * size, "graph")


def test_binding_refusals(lean):
    torch = torch_cuda()
    q, kc, vc, table = make_attend([20], 4, 2, 64, 16, "f32", "bf16")
    ld = torch.tensor([20], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(1, 4, 2, 64), dtype=torch.uint8, device="cuda")
    ok = dict(scale=0.125, workspace=ws)
    lean.lean_paged_attention(q, kc, vc, table, ld, out, **ok)
    for bad in (dict(q=q[:, :, :32]), dict(vc=vc.transpose(1, 2)), dict(vc=vc.float()), dict(ld=ld.long()),
                dict(table=table[0]), dict(out=out.bfloat16()), dict(lse=torch.zeros(3, device="cuda"))):
        a = dict(q=q, kc=kc, vc=vc, table=table, ld=ld, out=out, lse=None, **{})
        a.update(bad)
        with pytest.raises(ValueError):
            lean.lean_paged_attention(a["q"], a["kc"], a["vc"], a["table"], a["ld"], a["out"], lse=a["lse"], **ok)
    with pytest.raises(lean.LeanError):
        lean.lean_paged_attention(q, kc, vc, table, ld, out, scale=0.125, workspace=None)
    with pytest.raises(lean.LeanError):
        lean.lean_paged_attention(q, kc.float(), vc.float(), table, ld, out, **ok)
    assert math.isfinite(float(out.sum())) and dtype("f32") == torch.float32
