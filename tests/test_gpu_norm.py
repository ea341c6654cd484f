"""GPU parity of lean_residual_norm with its definition in 64 bits: every type
pair, widths of one element, odd widths, vector and scalar rows, rows longer than
a block's registers, each optional part, strides, buffers used in place, streams,
and magnitudes at the ends of fp32."""
import pytest

from lean_testlib import torch_cuda
from step_testlib import close, dtype, norm_ref, normal, gen, run_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")]
# one element; below a warp; odd; vectors with a part of a block; the scalar and vector limits of a block and past them
WIDTHS = [1, 2, 7, 8, 31, 33, 64, 96, 257, 576, 960, 1000, 2048, 4096, 4097, 8192, 11008, 16384, 16392, 20001]


@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(lean, width, act, res):
    run_norm(lean, 3, width, act, res, post=True, gate="all", seed=width)
    run_norm(lean, 1, width, act, res, seed=width + 1)


@pytest.mark.parametrize("rows", [1, 2, 5, 64, 303, 305, 1025])
@pytest.mark.parametrize("width", [96, 960, 2048])
def test_rows(lean, rows, width):
    run_norm(lean, rows, width, "bf16", "f32", post=True, gate="row", seed=rows)
    run_norm(lean, rows, width, "f32", "f32", seed=rows)


@pytest.mark.parametrize("width", [200, 2048, 4099, 20480])
@pytest.mark.parametrize("with_x,with_h,with_w,post,gate,h_out,y", [
    (True, True, True, False, "none", True, True), (False, True, True, False, "none", False, True),
    (False, True, True, False, "none", True, True), (True, False, True, True, "row", True, True),
    (True, True, False, True, "all", True, True), (True, True, True, False, "row", True, False),
    (True, True, False, True, "none", False, True), (True, True, True, False, "all", False, True)])
def test_parts(lean, width, with_x, with_h, with_w, post, gate, h_out, y):
    run_norm(lean, 4, width, "bf16", "f32", post=post, gate=gate, with_x=with_x, with_h=with_h, with_w=with_w,
             h_out=h_out, y=y, seed=7)


@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("width,pad", [(960, 8), (960, 3), (333, 1), (2048, 64), (17000, 5), (20480, 8)])
def test_strides(lean, width, pad, act, res):
    run_norm(lean, 5, width, act, res, post=True, gate="all", pad=pad, seed=3)


@pytest.mark.parametrize("width", [1, 960, 2048, 4097, 16400])
def test_in_place(lean, width):
    for act, res in TYPES:
        run_norm(lean, 6, width, act, res, post=True, gate="all", in_place=True, seed=4)


def test_unaligned_base(lean):
    """Rows that begin off 16 bytes take the scalar form."""
    torch = torch_cuda()
    g = gen(9)
    flat = normal(g, 3 * 512 + 1, t="bf16")
    x = flat[1:].view(3, 512)
    y = torch.empty((3, 512), device="cuda", dtype=torch.bfloat16)
    lean.lean_residual_norm(x, None, None, None, y, eps=1e-6)
    _, want, _, _ = norm_ref(x, None, None, None, None, 1.0, 1e-6)
    close(y, want, 2.0 ** -8 * want.abs() + 1e-6, "unaligned")


@pytest.mark.parametrize("std", [1e-12, 1e-3, 1e6, 1e17])
def test_magnitudes(lean, std):
    """Small rows are ruled by eps, large ones by the squares (below their overflow at 2^64)."""
    run_norm(lean, 4, 768, "f32", "f32", post=True, std=std, seed=5)
    run_norm(lean, 4, 770, "f32", "f32", std=std, seed=6)


def test_zero_row_and_not_finite(lean):
    torch = torch_cuda()
    x = torch.zeros((3, 64), device="cuda")
    x[1, 5] = float("nan")
    x[2] = 1
    y = torch.empty_like(x)
    lean.lean_residual_norm(x, None, None, None, y, eps=1e-6)
    assert y[0].tolist() == [0.0] * 64 and bool(torch.isnan(y[1]).all())
    close(y[2], torch.full((64,), 1 / (1 + 1e-6) ** 0.5, dtype=torch.float64, device="cuda"), 4e-7, "ones")


def test_stream_graph_and_flag(lean):
    """Another stream than the current one, a captured graph, and a chain of calls launched early."""
    torch = torch_cuda()
    s = torch.cuda.Stream()
    run_norm(lean, 7, 960, "bf16", "f32", post=True, stream=s, seed=8)
    g = gen(10)
    h = normal(g, 4, 2048)
    w = 1 + normal(g, 2048, std=0.1)
    x = normal(g, 4, 2048)
    want = h.double()
    for _ in range(20):
        want, wy, _, _ = norm_ref(x, want, w, None, None, 0.5, 1e-5)
    h0, y = h.clone(), torch.empty_like(h)
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for _ in range(20):
            lean.lean_residual_norm(x, h, w, h, y, eps=1e-5, res_scale=0.5, flags=lean.LEAN_FLAG_EARLY_WEIGHTS)
    h.copy_(h0)
    graph.replay()
    torch.cuda.synchronize()
    close(h, want, 1e-5 * want.abs() + 2e-5, "chain h")
    close(y, wy, 1e-5 * wy.abs() + 2e-5, "chain y")


def test_binding_refusals(lean):
    torch = torch_cuda()
    x = torch.zeros((2, 64), device="cuda")
    with pytest.raises(ValueError):
        lean.lean_residual_norm(x, torch.zeros((2, 63), device="cuda"), None, None, x)
    with pytest.raises(ValueError):
        lean.lean_residual_norm(x, None, torch.zeros(63, device="cuda"), None, x)
    with pytest.raises(ValueError):
        lean.lean_residual_norm(x.t(), None, None, None, torch.zeros((64, 2), device="cuda"))
    with pytest.raises(lean.LeanError):
        lean.lean_residual_norm(x, None, None, None, None)
    with pytest.raises(lean.LeanError):
        lean.lean_residual_norm(x.half(), torch.zeros((2, 64), device="cuda", dtype=torch.bfloat16), None, None, x.half())
    assert dtype("f32") == torch.float32
