"""The example's decode steps, every operator in its place, against the same model
in 64 bits (oracle weights, attention over the whole prefix without a cache)."""
import importlib.util
import math
import os

import numpy as np
import pytest

import oracle
from block_quantized_weight_dot_gb300 import synthetic as syn
from lean_testlib import torch_cuda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    torch_cuda()
    spec = importlib.util.spec_from_file_location("decode_example", os.path.join(ROOT, "examples", "decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(cfg, weights, tokens):
    """Logits after every token of one sequence, 64 bits; k and v rounded to bf16 as the cache holds them."""
    torch = torch_cuda()
    w = {name: torch.from_numpy(oracle.dequant(weights.fmt[name], weights.canon[name].reshape(shape[0], -1), *shape)).cuda()
         for name, shape in weights.shape.items()}
    norms = weights.norms.double()
    norm = lambda x, g: x / (x.square().mean(-1, keepdim=True) + cfg.eps).sqrt() * g
    n, hd, group = len(tokens), cfg.head_dim, cfg.q_heads // cfg.kv_heads
    h = w["embed"][tokens]
    pos = torch.arange(n, dtype=torch.float64, device="cuda")
    ang = pos[:, None] * cfg.rope_base ** (-torch.arange(0, hd, 2, dtype=torch.float64, device="cuda") / hd)
    c, s = ang.cos()[:, None], ang.sin()[:, None]

    def rope(x):
        a, b = x[..., :hd // 2], x[..., hd // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    mask = torch.ones((n, n), device="cuda").tril().bool()
    for i in range(cfg.layers):
        x = norm(h, norms[2 * i])
        q = rope((x @ w[(i, "q")].T).view(n, cfg.q_heads, hd))
        k = rope((x @ w[(i, "k")].T).view(n, cfg.kv_heads, hd)).bfloat16().double()
        v = (x @ w[(i, "v")].T).view(n, cfg.kv_heads, hd).bfloat16().double()
        z = torch.einsum("thd,shd->hts", q, k.repeat_interleave(group, 1)) * hd ** -0.5
        p = torch.softmax(z.masked_fill(~mask, -math.inf), -1)
        a = torch.einsum("hts,shd->thd", p, v.repeat_interleave(group, 1)).reshape(n, -1)
        h = h + a @ w[(i, "o")].T
        x = norm(h, norms[2 * i + 1])
        h = h + (torch.nn.functional.silu(x @ w[(i, "gate")].T) * (x @ w[(i, "up")].T)) @ w[(i, "down")].T
    return norm(h, norms[-1]) @ w["lm_head"].T


@pytest.mark.parametrize("linear,table,heads", [(syn.Q4_0, syn.Q8_0, (6, 2)), (syn.Q8_0, syn.Q4_0, (4, 4))])
def test_steps_match_64_bits(example, linear, table, heads):
    torch = torch_cuda()
    lean = example.lean
    cfg = example.Config(layers=3, hidden=256, q_heads=heads[0], kv_heads=heads[1], ffn=512, vocab=1003, linear=linear,
                         table=table)
    weights = example.Weights(cfg, seed=1)
    prompts = np.random.default_rng(2).integers(0, cfg.vocab, (3, 37))
    dec = example.Decoder(cfg, weights, 3, 48)
    want = [reference(cfg, weights, torch.from_numpy(p).cuda()) for p in prompts]
    for t in range(37):
        dec.ids.copy_(torch.from_numpy(prompts[:, t].astype(np.int32)))
        dec.given.copy_(torch.from_numpy(prompts[:, min(t + 1, 36)].astype(np.int32)))
        dec.step()
        for s in range(3):
            # A key or value near the middle of two bf16 numbers may be rounded the other way: 2^-8 of it, in some of the
            # prefix's elements and layers; 2% of the largest logit is several times what all of them together can do.
            ref = want[s][t]
            assert float((dec.logits[s].double() - ref).abs().max()) <= 0.02 * float(ref.abs().max()), (t, s)
            lp = torch.log_softmax(dec.logits[s].double(), 0)
            assert abs(float(dec.logprobs[s]) - float(lp[int(dec.given[s])])) < 1e-4
            assert int(dec.top_ids[s, 0]) == int(dec.logits[s].argmax()) == int(dec.ids[s])
            assert abs(float(dec.entropy[s]) + float((lp.exp() * lp).sum())) < 1e-4
    assert dec.lens[dec.turn].tolist() == [37] * 3 and dec.status.tolist() == [0] * 3
    assert lean.lean_device_error(True) == 0


def test_graph_gives_the_same_tokens(example):
    """Two steps recorded into a graph and replayed decode what steps one by one do."""
    torch = torch_cuda()
    cfg = example.Config(layers=2, hidden=256, q_heads=4, kv_heads=2, ffn=512, vocab=500)
    weights = example.Weights(cfg, seed=3)
    runs = []
    for use_graph in (False, True):
        dec = example.Decoder(cfg, weights, 2, 40)
        dec.ids.copy_(torch.tensor([5, 9]))
        out = []
        for _ in range(2):
            dec.step()
            out.append(dec.ids.tolist())
        if use_graph:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                dec.step()
                first = dec.ids.clone()
                dec.step()
            for _ in range(10):
                graph.replay()
                out += [first.tolist(), dec.ids.tolist()]
        else:
            for _ in range(20):
                dec.step()
                out.append(dec.ids.tolist())
        runs.append(out)
    assert runs[0] == runs[1]
