"""lean_paged_attention over caches in 8 bits whose values are large: sums of many
keys that fp32 holds come out finite."""
import pytest

from lean_testlib import torch_cuda
from step_testlib import HALF, U, close, dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("dim,hq", [(64, 4), (64, 12), (128, 4), (256, 4), (256, 12)])
@pytest.mark.parametrize("scale", [1.0, 1e25, 1e30])
@pytest.mark.parametrize("n", [1024, 8192])
def test_large_scales(lean, n, scale, dim, hq, act):
    """Keys that count alike, in so many sequences that single warps walk whole ones and fold their sums: the mean of the
    values comes out."""
    torch = torch_cuda()
    seqs, page = 2500, 128
    kc = torch.zeros((n // page, page, 1, dim), dtype=torch.int8, device="cuda")
    vc = torch.full_like(kc, 100)
    vc[:, ::2] = -27
    ks = torch.ones((n // page, page, 1), device="cuda")
    vs = torch.full_like(ks, scale)
    q = torch.zeros((seqs, hq, dim), device="cuda", dtype=dtype(act))
    out = torch.zeros_like(q)
    table = torch.arange(n // page, device="cuda", dtype=torch.int32)[None].repeat(seqs, 1).contiguous()
    lens = torch.full((seqs,), n, device="cuda", dtype=torch.int32)
    ws = torch.full((lean.lean_paged_attention_workspace_bytes(seqs, hq, 1, dim),), 255, dtype=torch.uint8, device="cuda")
    lean.lean_paged_attention(q, kc, vc, table, lens, out, scale=1.0, workspace=ws, k_scales=ks, v_scales=vs)
    want = torch.full(out.shape, 36.5, dtype=torch.float64, device="cuda") * vs[0, 0, 0].double()
    # chains of 64 units and of folds, a unit's 16 products cut off below 2^-24 of the largest; of terms of 63.5 on average
    tol = 2 * (64 + n / 1024 + 20) * U * 63.5 / 36.5 * want
    close(out, want, tol + HALF[act] * want, "values of %g x 100, %d keys" % (scale, n))
