"""lean_prefix_attention where scores climb along a prefix, so that the reference of
the exponentials has to move while outputs are being summed: by a little and by a
lot, before and after outputs go to the workspace, in some rows of a warp and not in
others, with values of every size whose sums fp32 holds."""
import math

import pytest

from cache_testlib import scales_like
from lean_testlib import torch_cuda
from step_testlib import HALF, TINY, U, close, dtype, gen, normal

pytestmark = pytest.mark.gpu

LENGTH, PAGE = 4500, 60  # 36 tiles of keys, the last one with 20: outputs are folded every 32 halves of tiles
# tokens from which scores are one step higher: in a first half, in neighbouring tokens, next to the ends of tiles and folds
CLIMBS = (70, 200, 201, 640, 2047, 2048, 2050, 2500, 4090, 4100)


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


@pytest.fixture(autouse=True)
def clean(lean):
    yield
    assert lean.lean_device_error(True) == 0


def run_climb(lean, act, cache, dim, seqs_each, step, size, hkv=4, group=4, prefixes=48):
    """So many prefixes (all of the same pages) that blocks have whole ones; scores of rows climb by step nats times a
    factor of the row's own, 1 to -1."""
    torch = torch_cuda()
    g = gen(8200 + dim + seqs_each)
    pages = -(-LENGTH // PAGE)
    n, hq = prefixes * seqs_each, hkv * group
    climb = torch.zeros(pages * PAGE, device="cuda")
    for t in CLIMBS:
        climb[t:] += step
    climb = climb.view(pages, PAGE, 1)
    ks = vs = None
    if cache == "i8":  # the climb is the keys' scales'
        kc, vc = (torch.zeros((pages, PAGE, hkv, dim), device="cuda", dtype=torch.int8) for _ in range(2))
        kc[..., 0] = 127
        vc.copy_(torch.randint(-127, 128, vc.shape, generator=g, device="cuda", dtype=torch.int32))
        ks, vs = (scales_like(kc, True) for _ in range(2))
        ks.copy_((climb / 127).expand(ks.shape))
        vs.copy_(size / 73 * torch.exp(0.5 * torch.randn(vs.shape, generator=g, device="cuda")))
    else:
        kc, vc = (normal(g, pages, PAGE, hkv, dim) for _ in range(2))
        kc = 0.25 * kc
        kc[..., 0] = climb
        kc, vc = kc.to(dtype(cache)), (vc * size).to(dtype(cache))
    q = normal(g, n, hq, dim, std=0.5)
    factors = torch.tensor([1.0, 0.5, 0.25, 0.125, 0.0, -0.5, -1.0], device="cuda")
    q[..., 0] = factors[torch.randint(0, 7, (n, hq), generator=g, device="cuda")]
    q = q.to(dtype(act))
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None].repeat(prefixes, 1).contiguous()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = torch.full_like(q, 7.0), torch.full((n, hq), 7.0, device="cuda")
    ws = torch.full((lean.lean_prefix_attention_workspace_bytes(n, hq, hkv, dim, prefixes),), 255, dtype=torch.uint8, device="cuda")
    none = torch.full((n, 1), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    lean.lean_prefix_attention(q, kc, vc, table, ints([LENGTH] * prefixes), ints([seqs_each * i for i in range(prefixes + 1)]), none,
                               ints([0] * n), out, scale=1.0, lse=lse, workspace=ws, k_scales=ks, v_scales=vs)
    kd, vd = (c.double() if s is None else c.double() * s.double()[..., None] for c, s in ((kc, ks), (vc, vs)))
    kd, vd = (x.reshape(-1, hkv, dim)[:LENGTH] for x in (kd, vd))
    one = HALF["bf16"] if cache == "bf16" else HALF["f16"]
    split = act == "f32" or (act == "f16" and cache == "bf16")
    for a in range(0, n, 128):
        x = q[a:a + 128].double().view(-1, hkv, group, dim)
        m = x.shape[0]
        z = torch.einsum("sgrd,lgd->sgrl", x, kd)
        want_lse = torch.logsumexp(z, -1).view(m, hq)
        reach = torch.einsum("sgrd,lgd->sgrl", x.abs(), kd.abs()).amax(-1).view(m, hq)
        z = torch.softmax(z, -1)
        want = torch.einsum("sgrl,lgd->sgrd", z, vd).reshape(m, hq, dim)
        weight = torch.einsum("sgrl,lgd->sgrd", z, vd.abs()).reshape(m, hq, dim)
        # scores: up to 24 sums of 16 terms, each rounded towards zero (2 U), and four roundings in 32 bits; a power of
        # two, 2^-22; sums of keys and of tiles as in cache_testlib.run_prefix; each move of a reference rescales, a
        # power and two roundings.  The scores' error counts in p and in the sum of all p.
        rel = 52 * U * reach + (len(CLIMBS) + 1) * 2.0 ** -21 + (LENGTH / 8 + 200) * U
        # what f16 operands lose of small p: as in cache_testlib.run_prefix
        lost = 0.0 if cache == "bf16" else LENGTH * 2.0 ** (-38 if split else -34)
        err = (2 * rel[..., None] + (0.0 if split else one)) * weight + (lost + 2.0 ** -37) * vd.abs().max()
        what = "climb by %g %s/%s dim %d, %d sequences a prefix, values of %g" % (step, act, cache, dim, seqs_each, size)
        close(out[a:a + 128], want, err + HALF[act] * (want.abs() + err) + TINY[act], what)
        close(lse[a:a + 128], want_lse, rel + 4 * U * want_lse.abs(), what + " lse")


@pytest.mark.parametrize("seqs_each", [5, 40])  # one tile of rows, two
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("step", [4.0, 10.0, 24.0])
@pytest.mark.parametrize("act,cache", [("bf16", "bf16"), ("bf16", "f16"), ("f16", "f16"), ("bf16", "i8"), ("f32", "bf16")])
def test_climbing_scores(lean, act, cache, step, dim, seqs_each):
    run_climb(lean, act, cache, dim, seqs_each, step, 1.0)


@pytest.mark.parametrize("seqs_each", [5, 40])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("step", [5.0, 24.0])  # (24 nats: 32 p are just below 2^40)
@pytest.mark.parametrize("act,cache,size", [("bf16", "bf16", 1e30), ("f32", "bf16", 1e30), ("f16", "i8", 1e30), ("bf16", "i8", 1e30)])
def test_large_values(lean, act, cache, size, step, dim, seqs_each):
    """Values up to 2^120 / keys: what comes out is finite, and so is every sum on the way."""
    if act == "f16":
        size = 1e4  # (what f16 out holds)
    run_climb(lean, act, cache, dim, seqs_each, step, size)
