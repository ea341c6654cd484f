"""The cache's operators together, as answers to shared prompts use them: prompts and
answers are rows of one block table, pages are handed out on the GPU, keys and values
are written as they come, attended over prompt and answer, and read back."""
import importlib.util
import os

import pytest

from cache_testlib import run_prefix, scales_like
from lean_testlib import torch_cuda
from step_testlib import HALF, U, dtype, gen, normal, rotate_ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lean():
    torch_cuda()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


@pytest.mark.parametrize("act,cache", [("bf16", "i8"), ("f32", "i8"), ("f32", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("hq,hkv,dim,page", [(8, 2, 64, 16), (6, 1, 128, 24), (4, 2, 96, 5)])
def test_answers_to_shared_prompts(lean, hq, hkv, dim, page, act, cache):
    torch = torch_cuda()
    prompts, starts, answers, steps = [300, 130], [0, 5, 7], 8, 12  # (the last answer has no prompt)
    rows, width = len(prompts) + answers, -(-300 // page)
    pages = sum(-(-n // page) for n in prompts) + answers * -(-steps // page)
    ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    table, ring = ints(rows, width), torch.arange(pages, dtype=torch.int32, device="cuda").flip(0).contiguous()
    lens, state = [ints(rows), ints(rows)], [torch.tensor([0, pages], dtype=torch.int32, device="cuda"), ints(2)]
    status, token_starts = ints(rows), ints(rows + 1)
    kc, vc = (torch.zeros((pages, page, hkv, dim), dtype=torch.int8 if cache == "i8" else dtype(cache), device="cuda")
              for _ in range(2))
    ks, vs = (scales_like(kc, True, 0.0), scales_like(kc, True, 0.0)) if cache == "i8" else (None, None)
    scales = dict(k_scales=ks, v_scales=vs)
    freq = lean.lean_rope_frequencies(lean.LEAN_ROPE_PLAIN, dim, 10000.0)
    turns = torch.from_numpy(lean.lean_rope_turns(freq)).cuda()
    begin = torch.tensor([0, 0] + [300] * 5 + [130] * 2 + [0], dtype=torch.int32, device="cuda")  # a row's first position
    ws = torch.empty(lean.lean_prefix_attention_workspace_bytes(answers, hq, hkv, dim, 2), dtype=torch.uint8, device="cuda")
    g, exact = gen(91), {}
    for t in range(steps + 1):
        a, b = t % 2, 1 - t % 2
        targets = torch.tensor(prompts + [t] * answers, dtype=torch.int32, device="cuda")
        new = sum(prompts) if t == 0 else answers
        slots, positions, seqs = ints(new), ints(new), ints(new)
        lean.lean_kv_pages(lens[a], targets, table, ring, state[a], page, lens[b], state[b], status, token_starts, slots,
                           positions, seqs)
        assert not status.any()
        positions += begin[seqs.long()]
        q, k, v = normal(g, new, hq, dim, t=act, std=1.5), normal(g, new, hkv, dim, t=act), normal(g, new, hkv, dim, t=act)
        q_out = torch.empty_like(q)
        lean.lean_rope_append(q, k, v, positions, slots, turns, q_out, kc, vc, rot_dim=dim, **scales)
        k_back, v_back = torch.empty((2, new, hkv, dim), device="cuda").unbind(0)
        lean.lean_kv_read(kc, vc, slots, k_back, v_back, **scales)
        for got, want in ((k_back, rotate_ref(k, positions, freq, dim, False, 1.0)), (v_back, v.double())):
            # half a step of the cache's type, and a rotation in fp32 (an angle within 2^-22 of a turn, products, a sum)
            size = want.abs().amax(-1, keepdim=True)
            step = size / 254 if cache == "i8" else HALF[cache] * want.abs()
            assert bool(((got.double() - want).abs() <= step * (1 + 2.0 ** -7) + 64 * U * size).all())
        for i, slot in enumerate(slots.tolist()):
            assert slot not in exact
            exact[slot] = k_back[i]
        if t:
            run_prefix(lean, prompts, starts, [t] * answers, hq, hkv, dim, act=act, cache=cache, workspace=ws, seed=t,
                       inputs=(q_out, kc, ks, vc, vs, table[:2], table[2:]))
    # a prompt as contiguous rows, in the order of its tokens
    token = torch.arange(300, device="cuda")
    slots = (table[0].long()[token // page] * page + token % page).to(torch.int32)
    k_back = torch.empty((300, hkv, dim), device="cuda")
    lean.lean_kv_read(kc, None, slots, k_back, None, **scales)
    assert torch.equal(k_back, torch.stack([exact[s] for s in slots.tolist()]))
    assert lean.lean_device_error(True) == 0


def test_the_example_with_a_cache_in_8_bits():
    """Steps one by one and steps recorded into a graph run and give the same tokens."""
    torch = torch_cuda()
    spec = importlib.util.spec_from_file_location("decode_example", os.path.join(ROOT, "examples", "decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    cfg = example.Config(layers=2, hidden=256, q_heads=4, kv_heads=2, ffn=512, vocab=500, cache_bits=8)
    weights = example.Weights(cfg, seed=3)
    runs = []
    for recorded in (False, True):
        dec, out = example.Decoder(cfg, weights, 3, 40), []
        dec.ids.copy_(torch.tensor([1, 2, 3]))
        for _ in range(2):
            dec.step()
            out.append(dec.ids.tolist())
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        if recorded:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.graph(graph, stream=side):
                dec.step()
                first = dec.ids.clone()
                dec.step()
        for _ in range(10):
            if recorded:
                graph.replay()
                out += [first.tolist(), dec.ids.tolist()]
            else:
                for _ in range(2):
                    dec.step()
                    out.append(dec.ids.tolist())
        assert bool(torch.isfinite(dec.logits).all()) and dec.lens[dec.turn].tolist() == [22] * 3
        runs.append(out)
    assert runs[0] == runs[1] and example.lean.lean_device_error(True) == 0
