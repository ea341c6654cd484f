"""Caches in 8 bits, tokens read back and shared prefixes through the LEAN_DEBUG
build, whose kernels check each global-memory index against the buffers their
arguments describe: parity as elsewhere and a clean device status after each."""
import pytest

from cache_testlib import run_append8, run_attend8, run_prefix, run_read
from lean_testlib import torch_cuda

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


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("dim,rot", [(64, 64), (80, 40), (128, 64), (6, 4), (512, 0), (256, 256)])
def test_append(lean, dim, rot, act):
    for inter in (False, True):
        run_append8(lean, 19, 6, 3, dim, rot, act, inter=inter, page=5, padding=(2,))
        run_append8(lean, 19, 0, 3, dim, rot, act, inter=inter, k_out=True, heads_first=False, pad=3, cache_pad=1)
    run_append8(lean, 1500, 3, 1, dim, rot, act)


@pytest.mark.parametrize("cache", ["i8", "bf16"])
@pytest.mark.parametrize("dim", [64, 80, 7])
def test_read(lean, dim, cache):
    run_read(lean, 37, 3, dim, page=5, cache=cache, out="bf16", slots=[-1] + [(i * 7) % 180 for i in range(36)], pool=36)
    run_read(lean, 2000, 3, dim, cache=cache, out="f32", pad=3)


@pytest.mark.parametrize("dim", [16, 64, 80, 128, 256])
@pytest.mark.parametrize("page", [1, 13, 16, 64])
def test_attend(lean, dim, page):
    run_attend8(lean, [0, 1, 15, 16, 17, 130, 700], 6, 2, dim, page=page)
    run_attend8(lean, [33, 200], 17, 1, dim, page=page, window=40, act="bf16", heads_first=False)
    run_attend8(lean, [5000, 3, 40], 4, 1, dim, page=page)


@pytest.mark.parametrize("act,cache", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "i8"), ("f32", "i8")])
@pytest.mark.parametrize("dim", [16, 64, 80, 128])
@pytest.mark.parametrize("page", [5, 16, 128])
def test_prefix(lean, page, dim, act, cache):
    run_prefix(lean, [0, 1, 128, 300, 129], [1, 3, 4, 4, 8, 9], [5, 0, 17, 40, 1, 0, 16, 200, 33, 3, 0, 9], 6, 2, dim, page=page,
               act=act, cache=cache)
    run_prefix(lean, [5000], [0, 40], [i % 9 for i in range(40)], 8, 2, dim, page=page, act=act, cache=cache, pad=8)
