"""lean_prefix_attention where more than eight query heads share a kv head and sequences
have many tokens of their own: both kernels of a call are at work on their SMs, and
items of both are shared by blocks."""
import pytest

from cache_testlib import run_prefix
from lean_testlib import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    yield L
    assert L.lean_device_error(True) == 0


@pytest.mark.parametrize("act,cache", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "i8"), ("f32", "i8")])
@pytest.mark.parametrize("hq,hkv,dim", [(48, 4, 64), (24, 2, 128), (40, 2, 80)])
def test_wide_groups_with_own_tokens(lean, hq, hkv, dim, act, cache):
    for plens, tail in (([9000, 700], 300), ([40, 1], 2500)):
        lens = [tail - 97 * i % tail for i in range(30)]
        run_prefix(lean, plens, [0, 21, 29], lens, hq, hkv, dim, act=act, cache=cache)
