"""More paths of the step operators through the LEAN_DEBUG build: the parts that
go through a workspace, rows that warps share, rows too long for registers, every
width of access, maps left out.  Each leaves a clean device status.  Nothing here
plants a bad index."""
import random

import pytest

from lean_testlib import torch_cuda
from step_testlib import gen, normal, run_attend, run_logprobs, run_norm, run_pages, run_rope, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import build
    from block_quantized_weight_dot_gb300 import lean as L
    prev = L.use_library(L.open_library(build.build(debug=True)))
    assert L.lean_debug_build() == 1 and L.lean_device_status(True) == L.LEAN_OK
    yield L
    L.use_library(prev)


@pytest.fixture(autouse=True)
def clean(lean):
    yield
    assert lean.lean_device_status(True) == lean.LEAN_OK


@pytest.mark.parametrize("hq,hkv", [(4, 1), (16, 1), (40, 2)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_shared_by_blocks(lean, dim, hq, hkv):
    """Long sequences beside short ones: parts of warps and of blocks."""
    run_attend(lean, [9000, 3, 0, 700, 40], hq, hkv, dim)
    run_attend(lean, [5000, 17], hq, hkv, dim, act="bf16", cache="f16", page=24, window=3000)


@pytest.mark.parametrize("dim,hq", [(64, 4), (64, 16), (128, 16), (256, 16)])
def test_attend_folded(lean, dim, hq):
    """Sequences of more than 64 units in one warp's run."""
    torch = torch_cuda()
    n, seqs = 2100, 2500
    kc = normal(gen(dim), 17, 128, 1, dim, t="bf16")
    vc = torch.full_like(kc, 0.5)
    q = normal(gen(hq), 1, hq, dim).repeat(seqs, 1, 1)
    table = torch.arange(17, device="cuda", dtype=torch.int32)[None].repeat(seqs, 1).contiguous()
    lens = torch.full((seqs,), n, device="cuda", dtype=torch.int32)
    out, lse = torch.zeros_like(q), torch.zeros((seqs, hq), device="cuda")
    ws = torch.zeros(lean.lean_paged_attention_workspace_bytes(seqs, hq, 1, dim), dtype=torch.uint8, device="cuda")
    lean.lean_paged_attention(q, kc, vc, table, lens, out, scale=dim ** -0.5, lse=lse, workspace=ws)
    assert float((out - 0.5).abs().max()) < 1e-5
    assert float((lse - lse[:1]).abs().max()) < 1e-4


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16", "f16"])
def test_rope_accesses(lean, act, inter):
    for dim, rot, pad in ((128, 128, 0), (80, 40, 4), (72, 24, 3), (6, 4, 1), (512, 0, 0)):
        run_rope(lean, 37, 7, 2, dim, rot, act, "bf16", inter=inter, pad=pad, k_out=True, padding=(0, 36))
    run_rope(lean, 1500, 3, 1, 64, 32, act, "f16", inter=inter, in_place=True)
    run_rope(lean, 5, 3, 0, 64, 64, act, inter=inter)


@pytest.mark.parametrize("act,res", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("width", [2049, 5001, 16392, 17001])
def test_norm_odd_and_long(lean, width, act, res):
    run_norm(lean, 5, width, act, res, post=True, gate="row")
    run_norm(lean, 5, width, act, res, post=True, gate="all", pad=1)
    run_norm(lean, 3, width, act, res, with_x=False, h_out=False)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_logprobs_shared_and_many(lean, t):
    """Rows over many warps, warps over many rows, a warp per row at the end; with and without alternatives."""
    for rows, vocab, k in ((1, 151936, 20), (3, 60000, 0), (700, 1100, 0), (700, 1100, 5), (900, 5003, 1), (2, 9, 64)):
        x = normal(gen(rows), rows, vocab, t=t)
        run_logprobs(lean, x if vocab > 60000 else strided(x, 5), [(13 * i) % vocab for i in range(rows)], k=k)


def test_pages_around_the_ring(lean):
    r = random.Random(2)
    lens = [r.randrange(0, 300) for _ in range(700)]
    targets = [r.choice([0, x, x + r.randrange(0, 200)]) for x in lens]
    width = max(-(-max(a, b) // 8) for a, b in zip(lens, targets))
    ids = list(range(60000))
    table = [[ids.pop() for _ in range(width)] for _ in lens]
    ring = [60000 + i for i in range(70000)]
    for maps in ((True, True, True), (False, True, False)):
        run_pages(lean, lens, targets, table, ring, [69990, 40000], 8, 1 << 17, pad=1, outputs=maps)
    run_pages(lean, lens, targets, table, ring, [69990, 300], 8, 1000)
