"""lean_prefix_attention in three parts of q and p (fp32 out, and f16 out of bf16
caches): what they leave of fp32's precision, over prefixes alone, where two parts
would not do.  Tolerances come from the kernel's arithmetic, derived beside each test
as in test_gpu_attend_precision."""
import math

import pytest

from lean_testlib import torch_cuda
from step_testlib import HALF, U, close, dtype, gen, normal

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


def caches(cache, pages, page, dim):
    """Zeros, and scales of 1 in 8 bits."""
    torch = torch_cuda()
    kc, vc = (torch.zeros((pages, page, 1, dim), device="cuda", dtype=torch.int8 if cache == "i8" else dtype(cache)) for _ in range(2))
    ks, vs = (torch.ones((pages, page, 1), device="cuda") if cache == "i8" else None for _ in range(2))
    return kc, ks, vc, vs


def attend(lean, q, kc, ks, vc, vs, table, length, starts):
    """(out, lse); sequences have no tokens of their own."""
    torch = torch_cuda()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    n, hq, dim = q.shape
    out, lse = torch.full_like(q, 7.0), torch.full((n, hq), 7.0, device="cuda")
    ws = torch.full((lean.lean_prefix_attention_workspace_bytes(n, hq, 1, dim, len(starts) - 1),), 255, dtype=torch.uint8, device="cuda")
    lean.lean_prefix_attention(q, kc, vc, table, ints([length] * (len(starts) - 1)), ints(starts), ints([[0]] * n), ints([0] * n),
                               out, scale=1.0, lse=lse, workspace=ws, k_scales=ks, v_scales=vs)
    return out, lse


def run_lone_keys(lean, act, cache, outlier, hq, dim):
    """Sequence s has a prefix of one key, 1 in dimension s + 1: its lse is that element of q, whatever the size of
    element 0."""
    torch = torch_cuda()
    n = dim - 1
    kc, ks, vc, vs = caches(cache, n, 16, dim)
    kc[torch.arange(n), 0, 0, torch.arange(n) + 1] = 1
    vc.fill_(1)
    q = normal(gen(dim + hq), n, hq, dim)
    q[:, :, 0] = outlier
    q = q.to(dtype(act))
    table = torch.arange(n, device="cuda", dtype=torch.int32)[:, None].contiguous()
    out, lse = attend(lean, q, kc, ks, vc, vs, table, 1, list(range(n + 1)))
    want = q[torch.arange(n), :, torch.arange(n) + 1].double()
    # as test_gpu_attend_precision.run_lone_keys: 8 U; and the power of two of what the maximum's rounding leaves, 2^-22.
    # f16 operands: p is lifted by 13 binary places, whose sum with the score rounds; elements of q are held to 2^-38 of
    # the largest
    tol = 8 * U * want.abs() + 2.0 ** -22
    if cache != "bf16":
        tol = tol + (13 + 1.5 * want.abs()) * U + 2.0 ** -38 * q.double().abs().amax(-1)
    what = "lone keys %s/%s outlier %g hq %d dim %d" % (act, cache, outlier, hq, dim)
    close(lse, want, tol, what)
    # the one value: a few roundings, and of f16 out one more
    close(out, torch.ones_like(out).double(), 8 * U + 2.0 ** -21 + HALF[act], what + " out")
    return want, tol


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_third_part_of_q(lean, dim, hq):
    want, tol = run_lone_keys(lean, "f32", "bf16", 1.0, hq, dim)
    two = want.bfloat16().double()
    two = two + (want - two).bfloat16().double()
    assert bool(((two - want).abs() > tol).any())  # two parts would not do


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("act,cache,outlier", [("f32", "bf16", 4096.0), ("f32", "f16", 1.0), ("f32", "f16", -4096.0),
                                               ("f32", "f16", 60000.0), ("f32", "i8", 1.0), ("f32", "i8", 60000.0),
                                               ("f16", "bf16", 1.0), ("f16", "bf16", -4096.0)])
def test_one_large_element_of_q(lean, act, cache, outlier, dim, hq):
    """An element of q that is far larger than the others must not cost them their lower bits."""
    run_lone_keys(lean, act, cache, outlier, hq, dim)


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("cache", ["bf16", "f16", "i8"])
def test_third_part_of_p(lean, cache, dim, hq):
    """Key and value j are 1 in dimension j alone: out is the softmax of q."""
    torch = torch_cuda()
    n, seqs = 48, 64
    kc, ks, vc, vs = caches(cache, 3, 16, dim)
    for c in (kc, vc):
        c.view(48, dim)[torch.arange(n), torch.arange(n)] = 1
    q = torch.zeros((seqs, hq, dim), device="cuda")
    q[:, :, :n] = -0.5 * torch.rand((seqs, hq, n), generator=gen(7), device="cuda")
    out, lse = attend(lean, q, kc, ks, vc, vs, torch.arange(3, device="cuda", dtype=torch.int32)[None], n, [0, seqs])
    want = torch.softmax(q[:, :, :n].double(), -1)
    # a score of half a nat at most is cut off and rounds twice (2 U), its power is good to 2^-22, in f16 after a sum with
    # 13, which rounds by 8 U / 1.44: in p and in the sum of all.  That has chains of 16, then 3; the parts' products are
    # cut off when they are added (2 U each); the sum, its quotient and the product with that
    power = 6 + (6 if cache != "bf16" else 0)
    tol = (2 * power + 20 + 4 + 4) * U * want
    close(out[:, :, :n], want, tol, "softmax as output")
    assert not bool(out[:, :, n:].any())
    if cache == "bf16":
        p = torch.exp(q[:, :, :n].double() - q[:, :, :n].double().amax(-1, keepdim=True))
        two = p.bfloat16().double()
        two = two + (p - two).bfloat16().double()
        assert bool(((two - p).abs() * (want / p) > tol).any())  # two parts would not do


@pytest.mark.parametrize("place", ["first", "middle", "last"])
@pytest.mark.parametrize("dim,hq", [(64, 4), (128, 16)])
@pytest.mark.parametrize("gap", [10.0, 14.0, 17.375])
@pytest.mark.parametrize("n", [1000, 8192, 60001])
@pytest.mark.parametrize("cache", ["bf16", "f16", "i8"])
def test_one_key_outweighs_many(lean, cache, n, gap, dim, hq, place):
    """One key `gap` nats above n - 1 equal ones, values 1, and in the second half of the dimensions 0 for the one."""
    torch = torch_cuda()
    page, seqs = 128, 9
    kc, ks, vc, vs = caches(cache, -(-n // page), page, dim)
    vc.view(-1, dim)[:n] = 1
    at = {"first": 0, "middle": n // 2, "last": n - 1}[place]
    kc.view(-1, dim)[at, 0] = 1 if cache == "i8" else gap
    if cache == "i8":
        ks.view(-1)[at] = gap
    vc.view(-1, dim)[at, dim // 2:] = 0
    q = torch.zeros((seqs, hq, dim), device="cuda")
    q[:, :, 0] = 1
    table = torch.arange(kc.shape[0], device="cuda", dtype=torch.int32)[None]
    out, lse = attend(lean, q, kc, ks, vc, vs, table, n, [0, seqs])
    tail = (n - 1) * math.exp(-gap)
    want = torch.ones((dim,), dtype=torch.float64, device="cuda")
    want[dim // 2:] = tail / (1 + tail)
    # the n / 64 halves of tiles, of two tiles of rows at most, are shared by more than 100 blocks, which add theirs in a
    # chain; a half's 64 products come in 12 instructions whose sums are cut off (2 U), its powers in chains of 16 and 3;
    # then up to 152 blocks' parts in a chain
    chain = (2 * n / 64 / 100 + 1 + 24 + 19 + 152 + 8) * U
    # e^(z - m): three roundings of an argument of `gap` nats, and of f16 one with 13 more; the power itself, 2^-22
    power = 3 * U * gap + 2.0 ** -22 + (6 * U if cache != "bf16" else 0)
    tol = torch.full((dim,), 2 * chain + 4 * U + 2 * power, dtype=torch.float64, device="cuda")
    tol[dim // 2:] = want[dim // 2:] * (2 * chain + 4 * power + 4 * U)
    if cache != "bf16":  # a probability is held to 2^-38 of a reference that is the largest one or up to 4 times smaller
        tol += n * 2.0 ** -38
    what = "%s n %d gap %g %s hq %d dim %d" % (cache, n, gap, place, hq, dim)
    close(out, want.expand_as(out), tol.expand_as(out), what)
    want_lse = torch.full((1,), gap + math.log1p(tail), dtype=torch.float64, device="cuda")
    close(lse, want_lse.expand_as(lse), chain + power + 4 * U * (1 + gap), what + " lse")
