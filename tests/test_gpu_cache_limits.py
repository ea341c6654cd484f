"""Caches past 2^32 elements, pages longer than a tile, calls at the same time: what the calls of the cache allow and
ordinary sizes do not reach."""
import pytest

from cache_testlib import make_prefix, run_append8, run_attend8, run_prefix, run_read
from lean_testlib import torch_cuda
from step_testlib import dtype, gen, normal

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


@pytest.mark.parametrize("act,cache", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "i8"), ("f32", "i8")])
def test_pages_past_32_bits(lean, act, cache):
    """The same pages near both ends of a cache of more than 2^32 elements and in a small one: the same results."""
    torch = torch_cuda()
    n, hq, hkv, dim, page, pages = 6, 4, 2, 128, 64, 270000
    assert pages * page * hkv * dim > 2 ** 32
    lens, plens, starts = [40, 0, 200, 1, 64, 130], [700, 129], [0, 4, 6]
    q, kc, ks, vc, vs, shared, table = make_prefix(plens, lens, hq, hkv, dim, page=page, act=act, cache=cache)
    small = kc.shape[0]
    far = torch.tensor([i if i % 3 == 0 else pages - 1 - i for i in range(small)], device="cuda")  # where each page goes
    i8 = cache == "i8"
    big = [torch.empty((pages, hkv, page, dim), dtype=kc.dtype, device="cuda").transpose(1, 2) for _ in range(2)]
    scales = [torch.empty((pages, hkv, page), device="cuda").transpose(1, 2) for _ in range(2)] if i8 else [None, None]
    for b, c in zip(big, (kc, vc)):
        b[far] = c
    for b, c in zip(scales, (ks, vs)):
        if i8:
            b[far] = c
    moved = [torch.where((t >= 0) & (t < small), far[t.long().clamp(0, small - 1)], t.long()).to(torch.int32) for t in (shared, table)]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.empty(lean.lean_prefix_attention_workspace_bytes(n, hq, hkv, dim, 2), dtype=torch.uint8, device="cuda")
    out = [torch.zeros((n, hq, dim), device="cuda", dtype=dtype(act)) for _ in range(4)]
    for i, (k, v, s, t) in enumerate((((kc, vc, (ks, vs), (shared, table))), (*big, scales, moved))):
        lean.lean_prefix_attention(q, k, v, t[0], ints(plens), ints(starts), t[1], ints(lens), out[i], scale=0.09, workspace=ws,
                                   k_scales=s[0], v_scales=s[1])
        lean.lean_paged_attention(q, k, v, t[1], ints(lens), out[2 + i], scale=0.09, workspace=ws, k_scales=s[0], v_scales=s[1])
    assert torch.equal(out[0], out[1]) and torch.equal(out[2], out[3]) and bool(torch.isfinite(out[0]).all())
    # written and read back at the far end
    slots = ints([(pages - 1) * page + 5, 7, (pages - 70) * page])
    rows = [normal(gen(i), 3, hkv, dim, t=act) for i in (1, 2)]
    lean.lean_rope_append(None, *rows, ints([0, 0, 0]), slots, None, None, *big, rot_dim=0,
                          **(dict(k_scales=scales[0], v_scales=scales[1]) if i8 else {}))
    back = [torch.empty_like(rows[0], dtype=torch.float32) for _ in range(2)]
    lean.lean_kv_read(*big, slots, *back, k_scales=scales[0], v_scales=scales[1])
    at = slots.long() // page, slots.long() % page
    for b, c, s, x in zip(back, big, scales, rows):
        assert torch.equal(b, c[at].float() * s[at][..., None] if i8 else c[at].float())
        assert float((b - x.float()).abs().max()) <= float(x.float().abs().max()) / 200


@pytest.mark.parametrize("cache", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("page", [128, 384, 1024])
def test_long_pages(lean, page, cache):
    act = "f16" if cache == "f16" else "bf16"
    for dim in (64, 128):
        run_prefix(lean, [page + 130, 2 * page, 60], [0, 3, 20, 24], [(13 * i) % 70 for i in range(25)], 16, 2, dim, page=page, act=act,
                   cache=cache)


def test_two_calls_at_once(lean):
    """Calls with workspaces of their own on two streams, again and again: each as it is alone."""
    torch = torch_cuda()
    jobs = []
    for act, cache, dim in (("bf16", "bf16", 128), ("f32", "i8", 64)):
        lens = [5 + i for i in range(40)]
        inputs = make_prefix([3000, 777], lens, 8, 2, dim, act=act, cache=cache)
        alone, _ = run_prefix(lean, [3000, 777], [0, 30, 40], lens, 8, 2, dim, act=act, cache=cache, inputs=inputs)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        q, kc, ks, vc, vs, shared, table = inputs
        ws = torch.empty(lean.lean_prefix_attention_workspace_bytes(40, 8, 2, dim, 2), dtype=torch.uint8, device="cuda")
        outs = [torch.zeros_like(q) for _ in range(8)]
        args = (q, kc, vc, shared, ints([3000, 777]), ints([0, 30, 40]), table, ints(lens))
        jobs.append((alone, outs, args, dict(scale=dim ** -0.5, workspace=ws, k_scales=ks, v_scales=vs), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(8):
        for alone, outs, args, more, stream in jobs:
            lean.lean_prefix_attention(*args, outs[i], stream=stream, flags=lean.LEAN_FLAG_EARLY_WEIGHTS * (i % 2), **more)
    torch.cuda.synchronize()
    for alone, outs, *_ in jobs:
        assert all(torch.equal(o, alone) for o in outs)


def test_the_same_slot_read_twice_and_calls_in_a_row(lean):
    """Early launches one after the other: each call sees what the one before it wrote."""
    flags = lean.LEAN_FLAG_EARLY_WEIGHTS
    for _ in range(3):
        run_append8(lean, 300, 8, 2, 128, 128, "bf16", flags=flags)
        run_read(lean, 40, 2, 64, slots=[5] * 20 + [-1] * 3 + [17] * 17, pool=4, flags=flags)
        run_attend8(lean, [30, 0, 200], 4, 2, 64, act="bf16", flags=flags)
        run_prefix(lean, [300], [1, 3], [30, 0, 20], 4, 2, 64, act="bf16", cache="i8", flags=flags)
