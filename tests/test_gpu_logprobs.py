"""GPU parity of lean_token_logprobs with its definition in 64 bits: vocabularies
from one token up, odd sizes and strides, every type, ties, masks, rows that are
all masked, values that are not finite, bad ids, parts left out."""
import math

import pytest

from lean_testlib import torch_cuda
from step_testlib import U, close, dtype, gen, logprobs_ref, normal, run_logprobs, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


def ids_of(rows, vocab, seed=0):
    return [(i * 7919 + seed) % vocab for i in range(rows)]


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 63, 255, 256, 257, 511, 1000, 1024, 1025, 4096, 8191, 8192, 8193, 32000,
                                   32003, 151936])
def test_vocabularies(lean, vocab, t):
    x = normal(gen(vocab), 3, vocab, t=t, std=3.0)
    run_logprobs(lean, x, ids_of(3, vocab), k=min(5, 64))
    run_logprobs(lean, x[:1], ids_of(1, vocab, 5), k=20)


@pytest.mark.parametrize("rows", [1, 2, 5, 37, 151, 153, 700])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_rows(lean, rows, t):
    x = normal(gen(rows), rows, 5003, t=t, std=2.0)
    run_logprobs(lean, x, ids_of(rows, 5003), k=4)


@pytest.mark.parametrize("k", [0, 1, 2, 31, 32, 33, 64])
@pytest.mark.parametrize("t", ["f32", "f16"])
def test_top_counts(lean, k, t):
    run_logprobs(lean, normal(gen(k), 3, 20011, t=t, std=2.0), ids_of(3, 20011), k=k)
    run_logprobs(lean, normal(gen(k), 2, 40, t=t, std=2.0), ids_of(2, 40), k=k)  # more places than tokens for 64


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad", [1, 2, 3, 5, 8, 64])
def test_strides(lean, t, pad):
    """Rows that begin anywhere: NaN between them must not be seen."""
    run_logprobs(lean, strided(normal(gen(pad), 9, 4001, t=t), pad), ids_of(9, 4001), k=6)
    run_logprobs(lean, strided(normal(gen(pad), 4, 4096, t=t), pad), ids_of(4, 4096), k=6)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_unaligned_base(lean, t):
    for off in (1, 2, 3, 7):
        flat = normal(gen(off), off + 2 * 3000, t=t)
        run_logprobs(lean, flat[off:].view(2, 3000), ids_of(2, 3000), k=3)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_ties(lean, t):
    """Equal logits: the lowest ids first, whatever the order in which they are met."""
    torch = torch_cuda()
    run_logprobs(lean, torch.full((2, 30000), 1.5, device="cuda", dtype=dtype(t)), [29999, 0], k=64)
    x = torch.zeros((3, 50000), device="cuda", dtype=dtype(t))
    x[0, 100::1000] = 2
    x[1, 49000:] = 2
    x[2] = (torch.arange(50000, device="cuda") // 5000).to(dtype(t))
    run_logprobs(lean, x, [100, 49001, 7], k=60)
    x = torch.round(normal(gen(4), 8, 9000) * 2).to(dtype(t))
    run_logprobs(lean, x, ids_of(8, 9000), k=33)
    run_logprobs(lean, torch.where(x > 0, 0.0, -0.0).to(dtype(t)), ids_of(8, 9000), k=20)  # zeros of both signs are equal


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_sorted_rows(lean, order):
    """Every new logit beats all before it, or none does."""
    torch = torch_cuda()
    x = torch.linspace(-20, 5, 60000, device="cuda")
    x = (x if order == "rising" else x.flip(0)).repeat(3, 1)
    run_logprobs(lean, x, [0, 59999, 30000], k=40)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_masks(lean, t):
    """Masked tokens, rows with few or no tokens left, and masks of the type's lowest value."""
    torch = torch_cuda()
    x = normal(gen(5), 8, 7001, t=t, std=2.0)
    x[0, ::2] = -math.inf
    x[1, 3:] = -math.inf
    x[2] = -math.inf
    x[3] = -math.inf
    x[3, 6999] = 1
    x[4, :7000] = -math.inf
    x[5, ::3] = torch.finfo(dtype(t)).min
    x[6] = torch.finfo(dtype(t)).min
    x[7] = torch.finfo(dtype(t)).min
    x[7, 17] = 0
    run_logprobs(lean, x, [2, 3000, 5, 6999, 7000, 3, 9, 18], k=5)


def test_not_finite(lean):
    """NaN or +inf in a row gives NaN there and nowhere else; the top ids are the largest that are not NaN."""
    torch = torch_cuda()
    x = normal(gen(6), 6, 6000)
    x[1, 77] = math.nan
    x[3, 5000] = math.inf
    x[4] = math.nan
    run_logprobs(lean, x, [1, 2, 3, 4, 5, 6], k=3)
    assert torch.cuda.is_available()


@pytest.mark.parametrize("scale", [0.01, 0.7, 1.0, 3.0, 50.0])
def test_scales(lean, scale):
    run_logprobs(lean, normal(gen(7), 5, 9973, std=2.0), ids_of(5, 9973), k=7, scale=scale)


@pytest.mark.parametrize("shift", [-1e4, -300.0, 300.0, 1e4])
def test_shifted_logits(lean, shift):
    """A constant added to all logits changes nothing but their own rounding."""
    run_logprobs(lean, normal(gen(8), 3, 5000, std=2.0) + shift, ids_of(3, 5000), k=4)


@pytest.mark.parametrize("t,vocab,k,rows", [("f16", 1100, 32, 700), ("bf16", 16400, 32, 4900), ("f32", 600, 20, 1300),
                                            ("f32", 5003, 8, 2500), ("bf16", 32003, 1, 170), ("f16", 5003, 5, 800),
                                            ("bf16", 7, 3, 400), ("f32", 32003, 2, 700)])
def test_many_rows(lean, t, vocab, k, rows):
    """The rows that can go wrong, over and over: ties, orders, masks, NaN and infinities."""
    torch = torch_cuda()
    x = normal(gen(vocab), 13, vocab, t=t, std=2.0)
    x[1] = torch.round(x[1] * 2)
    x[2] = 1.5
    x[3] = torch.where(x[3] > 0, 0.0, -0.0).to(x.dtype)
    x[4] = torch.linspace(-20, 5, vocab, device="cuda").to(x.dtype)
    x[5] = x[4].flip(0)
    x[6, ::2] = -math.inf
    x[7] = -math.inf
    x[8, 1:] = -math.inf
    x[9, vocab // 2] = math.nan
    x[10] = math.nan
    x[11, vocab - 1] = math.inf
    x[12] = torch.finfo(x.dtype).min
    x[12, 3] = 0
    n = -(-rows // 13)
    ids = [(5 * r) % vocab for r in range(13)]
    want_lp, want_rk, want_en, want_ti, want_tl = logprobs_ref(x, ids, 1.0, k)
    idd = torch.tensor(ids * n, dtype=torch.int32, device="cuda")
    lp, en = torch.full((13 * n,), 7.0, device="cuda"), torch.full((13 * n,), 7.0, device="cuda")
    rk, ti = idd.clone(), torch.full((13 * n, k), 7, dtype=torch.int32, device="cuda")
    tl = torch.full((13 * n, k), 7.0, device="cuda")
    ws = torch.zeros(lean.lean_token_logprobs_workspace_bytes(13 * n, vocab, k), dtype=torch.uint8, device="cuda")
    lean.lean_token_logprobs(x.repeat(n, 1), idd, lp, ranks=rk, entropy=en, top_ids=ti, top_logprobs=tl, workspace=ws)
    rel = (vocab / 128 + 128) * U  # (as in run_logprobs)
    fin = lambda v: torch.where(torch.isfinite(v), v, 0.0).abs()
    assert rk.tolist() == want_rk * n
    assert ti.tolist() == want_ti * n
    close(lp, want_lp.repeat(n), rel + 4 * U * fin(want_lp).repeat(n), "logprobs")
    close(en, want_en.repeat(n), rel * (2 + fin(want_en).repeat(n)), "entropy")
    close(tl, want_tl.repeat(n, 1), rel + 4 * U * fin(want_tl).repeat(n, 1), "top logprobs")


def test_bad_ids(lean):
    assert lean.lean_device_error(True) == 0
    x = normal(gen(9), 5, 3001)
    run_logprobs(lean, x, [4, -1, 3001, 2 ** 31 - 1, 3000], k=2)
    assert lean.lean_device_error(True) == 256 and lean.lean_device_error(True) == 0


@pytest.mark.parametrize("outputs", [(True, False, False), (False, True, False), (False, False, True), (False, False, False)])
def test_parts(lean, outputs):
    x = normal(gen(10), 3, 3001)
    run_logprobs(lean, x, ids_of(3, 3001), k=3, outputs=outputs)
    run_logprobs(lean, x, None, k=3, outputs=outputs)
    run_logprobs(lean, x, ids_of(3, 3001), k=0, outputs=outputs)


def test_largest_vocabulary(lean):
    run_logprobs(lean, normal(gen(11), 2, 1 << 20, t="bf16", std=2.0), [0, (1 << 20) - 1], k=10)
    run_logprobs(lean, normal(gen(11), 1, 1 << 20, std=2.0), [12345], k=10)


def test_far_rows(lean):
    """Offsets past 2^31 elements: the last rows of a large batch."""
    torch = torch_cuda()
    rows, vocab = 15000, 151936
    x = torch.zeros((rows, vocab), device="cuda", dtype=torch.bfloat16)
    for r in (0, 14134, 14135, rows - 1):
        x[r] = normal(gen(r), vocab, t="bf16", std=2.0)
    ids = torch.arange(rows, dtype=torch.int32, device="cuda")
    lp, en = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ti, tl = torch.empty((rows, 2), dtype=torch.int32, device="cuda"), torch.empty((rows, 2), device="cuda")
    ws = torch.zeros(lean.lean_token_logprobs_workspace_bytes(rows, vocab, 2), dtype=torch.uint8, device="cuda")
    lean.lean_token_logprobs(x, ids, lp, entropy=en, top_ids=ti, top_logprobs=tl, workspace=ws)
    for r in (0, 14134, 14135, rows - 1):
        want = logprobs_ref(x[r:r + 1], [r], 1.0, 2)
        close(lp[r:r + 1], want[0], 2e-4, "far row")
        assert ti[r].tolist() == want[3][0]
    flat = torch.full((1,), -math.log(vocab), dtype=torch.float64, device="cuda")
    close(lp[700:701], flat, 1e-4, "flat row")
    assert ti[700].tolist() == [0, 1]


def test_deterministic_and_workspace_reused(lean):
    torch = torch_cuda()
    ws = torch.zeros(max(lean.lean_token_logprobs_workspace_bytes(r, v, 20) for r, v in ((1, 151936), (37, 32003), (300, 999))),
                     dtype=torch.uint8, device="cuda")
    seen = {}
    for rows, vocab in ((1, 151936), (37, 32003), (300, 999), (1, 151936), (300, 999), (37, 32003)):
        got = run_logprobs(lean, normal(gen(vocab), rows, vocab), ids_of(rows, vocab), k=20, workspace=ws)
        if vocab in seen:
            assert all(torch.equal(a, b) for a, b in zip(got, seen[vocab]))
        seen[vocab] = got


def test_stream_and_flag(lean):
    torch = torch_cuda()
    x = normal(gen(13), 4, 9001, t="bf16")
    torch.cuda.synchronize()
    run_logprobs(lean, x, ids_of(4, 9001), stream=torch.cuda.Stream(), flags=lean.LEAN_FLAG_EARLY_WEIGHTS)


def test_binding_refusals(lean):
    torch = torch_cuda()
    x = torch.zeros((2, 100), device="cuda")
    ids, lp = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, device="cuda")
    ws = torch.zeros(lean.lean_token_logprobs_workspace_bytes(2, 100, 4), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        lean.lean_token_logprobs(x, ids.long(), lp, workspace=ws)
    with pytest.raises(ValueError):
        lean.lean_token_logprobs(x, ids, lp[:1], workspace=ws)
    with pytest.raises(lean.LeanError):
        lean.lean_token_logprobs(x, None, lp, workspace=ws)
    with pytest.raises(lean.LeanError):
        lean.lean_token_logprobs(x, ids, lp)
    with pytest.raises(lean.LeanError):
        lean.lean_token_logprobs(x, ids, lp, scale=-1.0, workspace=ws)
    with pytest.raises(lean.LeanError):
        lean.lean_token_logprobs(x, ids, lp, workspace=ws[:16])
