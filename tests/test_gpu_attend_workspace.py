"""What every warp of the largest grid folds and leaves in lean_paged_attention's
workspace stays inside it: long runs through the build that checks every index,
with what lies behind the workspace left as it was."""
import pytest

from cache_testlib import make_cache8
from lean_testlib import torch_cuda
from step_testlib import U, attend_ref, close, dtype, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", params=["plain", "checked"])
def lean(request):
    torch_cuda()
    from block_quantized_weight_dot_gb300 import build
    from block_quantized_weight_dot_gb300 import lean as L
    if request.param == "plain":
        yield L
        return
    prev = L.use_library(L.open_library(build.build(debug=True)))
    assert L.lean_debug_build() == 1 and L.lean_device_status(True) == L.LEAN_OK
    yield L
    L.use_library(prev)


@pytest.mark.parametrize("cache", ["i8", "bf16"])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 4, 64), (36, 4, 64), (8, 4, 128), (36, 4, 128), (4, 2, 256)])
def test_folds_of_every_warp(lean, hq, hkv, dim, cache):
    """600 sequences of up to 9000 tokens, the same pages for all: hundreds of units for every warp of 160 blocks of 16."""
    torch = torch_cuda()
    page, longest, n = 100, 9000, 600
    lens = [longest - 7 * (i % 50) for i in range(n)]
    pages = longest // page
    if cache == "i8":
        kc, ks, vc, vs = make_cache8(pages, page, hkv, dim, 3)
    else:
        kc, vc = (normal(gen(30 + i), pages, page, hkv, dim, t=cache) for i in range(2))
        ks = vs = None
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None].repeat(n, 1).contiguous()
    q = normal(gen(33), 4, hq, dim).repeat(n // 4, 1, 1).contiguous()
    out = torch.empty_like(q)
    size = lean.lean_paged_attention_workspace_bytes(n, hq, hkv, dim)
    room = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    lean.lean_paged_attention(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, scale=dim ** -0.5,
                              workspace=room[:size], k_scales=ks, v_scales=vs)
    assert lean.lean_device_status(True) == lean.LEAN_OK
    assert bool((room[size:] == 255).all())
    some = list(range(0, n, 37))
    kd, vd = (c.double() if s is None else c.double() * s.double()[..., None] for c, s in ((kc, ks), (vc, vs)))
    want, _, weight, reach = attend_ref(q[some], kd, vd, table[some], [lens[s] for s in some], dim ** -0.5, 0)
    rel = (2 * 2.0 ** -16 + 20 * U) * reach + 2.0 ** -16 + (longest / 8 + 68) * U  # as step_testlib.run_attend
    close(out[some], want, rel[..., None] * weight + 2.0 ** -37 * vd.abs().max(), "folds %d/%d of %d %s" % (hq, hkv, dim, cache))
    # (sequences of one length and q have the same answer, wherever their runs were cut, but for its rounding)
    same = [s for s in range(n) if lens[s] == lens[0] and s % 4 == 0]
    assert float((out[same] - out[same[0]]).abs().max()) <= float(2 * (rel[0].max() * weight[0].max()))
