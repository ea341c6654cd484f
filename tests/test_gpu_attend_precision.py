"""lean_paged_attention where few keys outweigh very many: what the many give has
to arrive in the output as it does in 64 bits.  Tolerances come from the kernel's
arithmetic and are derived here, beside each test."""
import math

import pytest

from lean_testlib import torch_cuda
from step_testlib import U, close, dtype, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


def attend(lean, q, kc, vc, length, scale=1.0):
    """The same pages for every sequence; (out, lse)."""
    torch = torch_cuda()
    n, hq, dim = q.shape
    hkv = kc.shape[2]
    table = torch.arange(kc.shape[0], device="cuda", dtype=torch.int32)[None].repeat(n, 1).contiguous()
    lens = torch.full((n,), length, device="cuda", dtype=torch.int32)
    out, lse = torch.full_like(q, 7.0), torch.full((n, hq), 7.0, device="cuda")
    ws = torch.full((lean.lean_paged_attention_workspace_bytes(n, hq, hkv, dim),), 255, dtype=torch.uint8, device="cuda")
    lean.lean_paged_attention(q, kc, vc, table, lens, out, scale=scale, lse=lse, workspace=ws)
    return out, lse


def run_one_key_outweighs(lean, cache, n, gap, place, hq, dim, seqs=2500):
    """One key `gap` nats above n - 1 equal ones, in so many sequences that single warps walk whole ones (with 2500, every
    warp's run has one).  Values: 1 for all keys in the first half of the dimensions; in the second 1 for the many and 0
    for the one."""
    torch = torch_cuda()
    page = 128
    kc = torch.zeros((-(-n // page), page, 1, dim), device="cuda", dtype=dtype(cache))
    vc = torch.full_like(kc, float("nan"))
    vc.view(-1, dim)[:n] = 1
    at = {"first": 0, "middle": n // 2, "last": n - 1}[place]
    kc.view(-1, dim)[at, 0] = gap
    vc.view(-1, dim)[at, dim // 2:] = 0
    q = torch.zeros((seqs, hq, dim), device="cuda")
    q[:, :, 0] = 1
    out, lse = attend(lean, q, kc, vc, n)
    tail = (n - 1) * math.exp(-gap)
    want = torch.ones((dim,), dtype=torch.float64, device="cuda")
    want[dim // 2:] = tail / (1 + tail)
    # A warp adds its units of 16 tokens in chains of 64, and the chains' sums in a chain of their own, half an ulp each;
    # a unit's 16 products are cut off at 2^-24 of the largest of them or below
    units = -(-n // 16)
    chain = (min(64, units) + units / 64 + 2) * U + 16 * U
    # e^(z - m): three roundings of an argument of `gap` nats, and the power of two itself, 2^-22
    power = 3 * U * gap + 2.0 ** -22
    tol = torch.full((dim,), 2 * chain + 4 * U, dtype=torch.float64, device="cuda")  # sum and normaliser
    tol[dim // 2:] = want[dim // 2:] * (2 * chain + 2 * power + 4 * U)
    if cache == "f16":  # a probability is held to 2^-38 of a reference that is the largest one or up to 4 times smaller
        tol += n * 2.0 ** -38
    what = "%s n %d gap %g %s hq %d dim %d" % (cache, n, gap, place, hq, dim)
    close(out, want.expand_as(out), tol.expand_as(out), what)
    want_lse = torch.full((1,), gap + math.log1p(tail), dtype=torch.float64, device="cuda")
    close(lse, want_lse.expand_as(lse), chain + power + 4 * U * (1 + gap), what + " lse")


@pytest.mark.parametrize("gap", [10.0, 14.0, 17.375])
@pytest.mark.parametrize("n", [1008, 1024, 1025, 2048, 8192, 131072])
def test_one_key_outweighs_many_bf16(lean, n, gap):
    run_one_key_outweighs(lean, "bf16", n, gap, "first", 4, 64)


@pytest.mark.parametrize("place", ["first", "middle", "last"])
@pytest.mark.parametrize("hq", [1, 8, 9, 16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_key_outweighs_many_bf16_everywhere(lean, dim, hq, place):
    run_one_key_outweighs(lean, "bf16", 8192, 17.375, place, hq, dim)
    run_one_key_outweighs(lean, "bf16", 8192, 17.375, place, hq, dim, seqs=1)


@pytest.mark.parametrize("gap", [10.0, 14.0, 17.375])
@pytest.mark.parametrize("n", [1008, 1025, 8192, 131072])
def test_one_key_outweighs_many_f16(lean, n, gap):
    """f16 holds nothing below 2^-24: e^-17.4 is 2^-25."""
    run_one_key_outweighs(lean, "f16", n, gap, "first", 4, 64)


@pytest.mark.parametrize("place", ["middle", "last"])
@pytest.mark.parametrize("hq", [8, 16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_key_outweighs_many_f16_everywhere(lean, dim, hq, place):
    run_one_key_outweighs(lean, "f16", 8192, 17.375, place, hq, dim)
    run_one_key_outweighs(lean, "f16", 8192, 17.375, place, hq, dim, seqs=1)


@pytest.mark.parametrize("cache", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [3e5, 5e7, 2e9])
def test_large_scores(lean, cache, scale):
    """Scores so large that a reference below the maximum, or a sum with the slack, would round past it: rising and
    falling ones, and ties of the largest, whose values' mean is the output."""
    torch = torch_cuda()
    n, dim = 512, 64
    kc, vc = (torch.zeros((4, 128, 1, dim), device="cuda", dtype=dtype(cache)) for _ in range(2))
    steps = torch.arange(n, device="cuda").float() / 512  # exact in both types up to 256 / 512
    kc.view(-1, dim)[:, 0] = steps.to(kc.dtype)
    vc.view(-1, dim)[:, 0] = (torch.arange(n, device="cuda") % 8).to(vc.dtype)
    q = torch.zeros((2, 4, dim), device="cuda")
    q[0, :, 0], q[1, :, 0] = 1, -1
    out, lse = attend(lean, q, kc, vc, n, scale=scale)
    k = kc.view(-1, dim)[:, 0].double()
    for s, best in ((0, k.max()), (1, k.min())):
        z = scale * best * (1 if s == 0 else -1)
        want = vc.view(-1, dim)[:, 0].double()[k == best].mean()
        close(out[s, :, 0], want.expand(4), 4 * U * want.abs(), "large scores")
        ties = math.log(int((k == best).sum()))
        close(lse[s], (z + ties).expand(4), 8 * U * (z.abs() + ties), "large scores lse")


def run_lone_keys(lean, cache, outlier, hq, dim):
    """Sequence s has one key, 1 in dimension s + 1: its lse is that element of q, whatever the size of element 0."""
    torch = torch_cuda()
    n = dim - 1
    kc = torch.zeros((n, 16, 1, dim), device="cuda", dtype=dtype(cache))
    kc[torch.arange(n), 0, 0, torch.arange(n) + 1] = 1
    vc = torch.ones_like(kc)
    q = normal(gen(dim + hq), n, hq, dim)
    q[:, :, 0] = outlier
    table = torch.arange(n, device="cuda", dtype=torch.int32)[:, None].contiguous()
    lens = torch.ones((n,), device="cuda", dtype=torch.int32)
    out, lse = torch.empty_like(q), torch.empty((n, hq), device="cuda")
    ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(n, hq, 1, dim), dtype=torch.uint8, device="cuda")
    lean.lean_paged_attention(q, kc, vc, table, lens, out, scale=1.0, lse=lse, workspace=ws)
    want = q[torch.arange(n), :, torch.arange(n) + 1].double()
    # three parts leave less than U of an element; f16 has steps of 2^-24, which scaling the largest element to 2^14 or
    # more makes 2^-38 of it; scale * log2 e, the product with it, the product with ln 2 and the results round
    tol = 8 * U * want.abs() + (2.0 ** -38 * q.abs().amax(-1).double() if cache == "f16" else 0)
    close(lse, want, tol, "lone keys %s outlier %g hq %d dim %d" % (cache, outlier, hq, dim))
    return q, want, tol


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_third_part_of_q(lean, dim, hq):
    q, want, tol = run_lone_keys(lean, "bf16", 1.0, hq, dim)
    two = want.bfloat16().double()
    two = two + (want - two).bfloat16().double()
    assert bool(((two - want).abs() > tol).any())  # two parts would not do


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("cache,outlier", [("bf16", 4096.0), ("f16", 1.0), ("f16", 300.0), ("f16", -4096.0), ("f16", 60000.0)])
def test_one_large_element_of_q(lean, cache, outlier, dim, hq):
    """An element of q that is far larger than the others must not cost them their lower bits."""
    run_lone_keys(lean, cache, outlier, hq, dim)


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("cache", ["bf16", "f16"])
def test_third_part_of_p(lean, cache, dim, hq):
    """Key and value j are 1 in dimension j alone: out is the softmax of q."""
    torch = torch_cuda()
    n, seqs = 48, 64
    kc = torch.zeros((3, 16, 1, dim), device="cuda", dtype=dtype(cache))
    kc.view(48, dim)[torch.arange(n), torch.arange(n)] = 1
    q = torch.zeros((seqs, hq, dim), device="cuda")
    q[:, :, :n] = -0.5 * torch.rand((seqs, hq, n), generator=gen(7), device="cuda")
    out, lse = attend(lean, q, kc, kc.clone(), n)
    want = torch.softmax(q[:, :, :n].double(), -1)
    # a score of half a nat at most rounds three times, its power is good to 2^-22; the sum has 48 terms in chains of
    # 12 and 3; then the parts' products, their sum and the quotient
    tol = (2 * (3 * 0.5 + 4) + 16 + 4) * U * want
    close(out[:, :, :n], want, tol, "softmax as output")
    assert not bool(out[:, :, n:].any())
    if cache == "bf16":
        p = torch.exp(q[:, :, :n].double() - q[:, :, :n].double().amax(-1, keepdim=True))
        two = p.bfloat16().double()
        two = two + (p - two).bfloat16().double()
        assert bool(((two - p).abs() * (want / p) > tol).any())  # two parts would not do
