"""GPU parity of lean_rope_append with its definition in 64 bits: both pairings,
part of the head, every type, odd head sizes, far and negative positions, cache
layouts, padding tokens, parts left out, in place, slots outside the cache."""
import math

import numpy as np
import pytest

from lean_testlib import torch_cuda
from step_testlib import close, gen, normal, rotate_ref, run_rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


@pytest.mark.parametrize("act,cache", [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16")])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 128), (128, 64), (96, 32), (80, 80), (80, 40), (64, 0), (2, 2), (6, 4),
                                     (256, 256), (512, 512), (72, 18)])
def test_heads(lean, dim, rot, inter, act, cache):
    run_rope(lean, 5, 4, 2, dim, rot, act, cache, inter, seed=dim + rot)


@pytest.mark.parametrize("tokens", [1, 2, 17, 300, 1111])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (15, 5), (32, 4), (8, 8)])
def test_tokens_and_heads(lean, tokens, hq, hkv):
    run_rope(lean, tokens, hq, hkv, 64, 64, "f32", "bf16", seed=tokens)
    run_rope(lean, tokens, hq, hkv, 64, 32, "bf16", "bf16", inter=True, page=24, seed=tokens)


@pytest.mark.parametrize("start", [0, 100000, 1 << 20, (1 << 31) - 100, -5000])
def test_positions(lean, start):
    """The angle stays exact at any position; negative positions turn backwards."""
    run_rope(lean, 9, 2, 1, 128, 128, "f32", "f16", start=start, scale=1.25, seed=1)


@pytest.mark.parametrize("kw", [
    dict(pad=8), dict(pad=6), dict(pad=1), dict(in_place=True), dict(k_out=True), dict(k_out=True, in_place=True),
    dict(cache_heads_first=True), dict(padding=(0, 3, 11)), dict(padding=tuple(range(12))),
    dict(k_out=True, with_cache=False)])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_layouts(lean, act, kw):
    run_rope(lean, 12, 6, 3, 64, 48, act, "bf16", page=16, seed=2, **kw)


@pytest.mark.parametrize("dim,rot", [(80, 40), (72, 24), (64, 24), (64, 8), (16, 8), (48, 20), (64, 4)])
@pytest.mark.parametrize("kw", [dict(), dict(pad=4), dict(pad=8, k_out=True), dict(pad=4, in_place=True), dict(pad=2)])
@pytest.mark.parametrize("inter", [False, True])
def test_run_widths(lean, dim, rot, kw, inter):
    """Heads and strides that allow 16, 8 or 2 bytes at a time, the rotated part ending inside a wider run."""
    for act in ("f32", "bf16", "f16"):
        run_rope(lean, 7, 5, 2, dim, rot, act, "bf16", inter, page=16, seed=dim + rot, **kw)


def test_q_or_kv_alone(lean):
    run_rope(lean, 4, 3, 0, 64, 64)
    run_rope(lean, 4, 0, 3, 64, 64, k_out=True)


def test_scaled_frequencies(lean):
    """Frequencies from the long-context rules give the rotation by their own angles."""
    torch = torch_cuda()
    for kind in (lean.LEAN_ROPE_LINEAR, lean.LEAN_ROPE_BASE, lean.LEAN_ROPE_RAMP, lean.LEAN_ROPE_BANDS):
        freq = lean.lean_rope_frequencies(kind, 64, 10000.0, 8.0, 2048.0, 1.0, 4.0)
        turns = torch.from_numpy(lean.lean_rope_turns(freq)).cuda()
        q = normal(gen(kind), 8, 2, 64)
        pos = torch.tensor([0, 1, 2047, 2048, 9999, 16383, 50000, 131071], dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)
        lean.lean_rope_append(q, None, None, pos, None, turns, out, None, None, rot_dim=64)
        close(out, rotate_ref(q, pos, freq, 64, False, 1.0), 3e-6 * q.abs().max().double(), "kind %d" % kind)


def test_rotation_is_relative(lean):
    """q at position a against k at position b depends on a - b alone."""
    torch = torch_cuda()
    freq = lean.lean_rope_frequencies(lean.LEAN_ROPE_PLAIN, 128, 1e6)
    turns = torch.from_numpy(lean.lean_rope_turns(freq)).cuda()
    x = normal(gen(3), 1, 2, 128)

    def at(p):
        out = torch.empty_like(x)
        lean.lean_rope_append(x, None, None, torch.tensor([p], dtype=torch.int32, device="cuda"), None, turns, out, None,
                              None, rot_dim=128)
        return out.double()

    near = [float((at(a)[0, 0] * at(a - 37)[0, 1]).sum()) for a in (37, 5000, 900000, 100000000)]
    for v in near[1:]:
        assert abs(v - near[0]) <= 20 * 2.0 ** -24 * float(x[0, 0].double().norm() * x[0, 1].double().norm()), near


def test_slot_outside_the_cache(lean):
    torch = torch_cuda()
    assert lean.lean_device_error(True) == 0
    g = gen(5)
    k, v = normal(g, 3, 2, 64), normal(g, 3, 2, 64)
    kc = torch.full((2, 16, 2, 64), float("nan"), device="cuda", dtype=torch.bfloat16)
    vc = kc.clone()
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    slots = torch.tensor([31, 32, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    lean.lean_rope_append(None, k, v, pos, slots, None, None, kc, vc, rot_dim=0)
    assert lean.lean_device_error(True) == 64 and lean.lean_device_error(True) == 0
    assert torch.equal(kc[1, 15], k[0].bfloat16()) and torch.equal(vc[1, 15], v[0].bfloat16())
    kc[1, 15] = float("nan")
    assert bool(torch.isnan(kc).all())


def test_far_slots(lean):
    """Element offsets past 2^31 in a large cache."""
    torch = torch_cuda()
    pages, page, heads, dim = 70000, 128, 2, 128  # 2.3e9 elements, 4.6 GB a cache
    kc = torch.empty((pages, page, heads, dim), device="cuda", dtype=torch.bfloat16)
    vc = torch.empty_like(kc)
    g = gen(6)
    k, v = normal(g, 2, heads, dim, t="bf16"), normal(g, 2, heads, dim, t="bf16")
    slots = torch.tensor([pages * page - 1, 69000 * page + 5], dtype=torch.int32, device="cuda")
    lean.lean_rope_append(None, k, v, torch.zeros(2, dtype=torch.int32, device="cuda"), slots, None, None, kc, vc, rot_dim=0)
    assert torch.equal(kc[-1, -1], k[0]) and torch.equal(vc[69000, 5], v[1])
    assert lean.lean_device_error(True) == 0


def test_stream_and_flag(lean):
    torch = torch_cuda()
    run_rope(lean, 33, 4, 2, 64, 64, stream=torch.cuda.Stream(), flags=lean.LEAN_FLAG_EARLY_WEIGHTS, seed=11)
    assert math.isfinite(float(np.float32(1)))
