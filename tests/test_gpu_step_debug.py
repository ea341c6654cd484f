"""The step operators through the LEAN_DEBUG build, whose kernels check each
global-memory index against the buffers their arguments describe: small odd
shapes of every path, parity as elsewhere and a clean device status after each."""
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


@pytest.mark.parametrize("width", [1, 33, 960, 2048, 4097, 20001])
def test_norm(lean, width):
    run_norm(lean, 3, width, "bf16", "f32", post=True, gate="all", pad=8)
    run_norm(lean, 2, width, "f32", "f32", gate="row", in_place=True)


@pytest.mark.parametrize("dim,rot", [(64, 64), (80, 40), (128, 64), (6, 4)])
def test_rope(lean, dim, rot):
    for inter in (False, True):
        run_rope(lean, 19, 6, 3, dim, rot, "f32", "bf16", inter=inter, page=5, padding=(2,))
        run_rope(lean, 19, 6, 3, dim, rot, "bf16", "bf16", inter=inter, cache_heads_first=True, k_out=True)


def test_pages(lean):
    r = random.Random(1)
    lens = [r.randrange(0, 60) for _ in range(40)]
    targets = [r.randrange(0, 90) for _ in lens]
    ids = list(range(40 * 12))
    table = [[ids.pop() for _ in range(12)] for _ in lens]
    ring = [900 + i for i in range(600)]
    run_pages(lean, lens, targets, table, ring, [590, 500], 8, 1500, pad=2)
    run_pages(lean, lens, targets, table, ring, [590, 20], 8, 300)


@pytest.mark.parametrize("dim", [8, 64, 80, 128, 256])
@pytest.mark.parametrize("page", [1, 13, 16, 64])
def test_attend(lean, dim, page):
    run_attend(lean, [0, 1, 15, 16, 17, 130, 700], 6, 2, dim, page=page)
    run_attend(lean, [33, 200], 17, 1, dim, page=page, window=40, act="bf16", heads_first=True)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 9, 1000, 8193, 32003])
def test_logprobs(lean, vocab, t):
    run_logprobs(lean, strided(normal(gen(vocab), 5, vocab, t=t), 3), [(7 * i) % vocab for i in range(5)], k=8)
    run_logprobs(lean, normal(gen(vocab), 1, vocab, t=t), [0], k=64)
