"""A whole decode step from this library's calls: a small gated-FFN transformer
with quantized linears, a paged key-value cache and greedy decoding, all on the
GPU (no value comes back to the host between steps).

    python examples/decode.py [--layers 32] [--tokens 32] [--sequences 2] [--graph] [--cache-bits 8]

Weights are random, in the shapes of SmolLM2-360M (hidden 960, 15 query and 5 kv
heads of 64, FFN 2560); the linears are Q4_0, the embedding and lm_head Q8_0.
Each step, for every sequence at once:

    lean_kv_pages          one more token each: pages, slot, position
    lean_embed_rows        the tokens' rows of the embedding
    per layer
      lean_qmatmul         q, k, v
      lean_rope_append     rotary positions, k and v into the cache
      lean_paged_attention
      lean_qmatmul         o
      lean_residual_norm   h += o, the norm before the FFN
      lean_qmatmul_swiglu  silu(gate) * up, per sequence
      lean_qmatmul         down
      lean_residual_norm   h += down, the norm before the next layer
    lean_qmatmul           logits
    lean_token_logprobs    the likeliest tokens with their log probabilities, the
                           entropy, and the log probability of a given next token
"""
import argparse
import os
import sys
import time
from dataclasses import dataclass

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from block_quantized_weight_dot_gb300 import lean  # noqa: E402
from block_quantized_weight_dot_gb300 import synthetic as syn  # noqa: E402


@dataclass
class Config:
    layers: int = 32
    hidden: int = 960
    q_heads: int = 15
    kv_heads: int = 5
    head_dim: int = 64
    ffn: int = 2560
    vocab: int = 49152
    linear: int = syn.Q4_0    # format of the layers' linears
    table: int = syn.Q8_0     # of the embedding and the lm_head
    rope_base: float = 100000.0
    eps: float = 1e-5
    page_size: int = 16
    cache_bits: int = 16      # 16: bf16; 8: whole numbers with a scale for each token and kv head
    top: int = 5


class Weights:
    """Random weights: canonical blocks on the host (canon) and packed on the GPU."""

    def __init__(self, cfg, seed=0):
        rng = np.random.default_rng(seed)
        self.canon, self.packed, self.shape, self.fmt = {}, {}, {}, {}
        d, q, kv = cfg.hidden, cfg.q_heads * cfg.head_dim, cfg.kv_heads * cfg.head_dim
        shapes = {"q": (q, d), "k": (kv, d), "v": (kv, d), "o": (d, q), "gate": (cfg.ffn, d), "up": (cfg.ffn, d),
                  "down": (d, cfg.ffn)}
        for layer in range(cfg.layers):
            for name, (n, k) in shapes.items():
                self.add((layer, name), cfg.linear, n, k, rng.standard_normal((n, k), dtype=np.float32) / np.sqrt(k))
        self.add("embed", cfg.table, cfg.vocab, d, rng.standard_normal((cfg.vocab, d), dtype=np.float32))
        self.add("lm_head", cfg.table, cfg.vocab, d, 2 * rng.standard_normal((cfg.vocab, d), dtype=np.float32) / np.sqrt(d))
        self.norms = torch.from_numpy(1 + 0.1 * rng.standard_normal((2 * cfg.layers + 1, d), dtype=np.float32)).cuda()

    def add(self, name, fmt, n, k, w):
        self.canon[name] = lean.lean_quantize(fmt, w, n, k)
        self.packed[name] = lean.upload_packed(fmt, self.canon[name], n, k)
        self.shape[name], self.fmt[name] = (n, k), fmt


class Decoder:
    """Sequences that grow by a token a step.  ids, given: int32 [sequences] on the GPU; step() reads the tokens in ids
    and leaves the likeliest next ones there, with top_ids, top_logprobs, entropy, and logprobs of the tokens in given."""

    def __init__(self, cfg, weights, sequences, max_tokens):
        self.cfg, self.w, self.n = cfg, weights, sequences
        dev, n, d, page = "cuda", sequences, cfg.hidden, cfg.page_size
        q, kv, hd = cfg.q_heads, cfg.kv_heads, cfg.head_dim
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
        floats = lambda *s: torch.empty(s, device=dev)
        width = -(-max_tokens // page)
        pages = n * width
        cache = torch.int8 if cfg.cache_bits == 8 else torch.bfloat16
        self.k_cache = torch.zeros((cfg.layers, pages, page, kv, hd), dtype=cache, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.scales = [{} for _ in range(cfg.layers)]
        if cfg.cache_bits == 8:
            self.scales = [dict(k_scales=floats(pages, page, kv), v_scales=floats(pages, page, kv)) for _ in range(cfg.layers)]
        self.table, self.ring = ints(n, width), torch.arange(pages, dtype=torch.int32, device=dev)
        # two sets in turn: lean_kv_pages writes its results beside its inputs
        self.lens, self.ring_state = [ints(n), ints(n)], [torch.tensor([0, pages], dtype=torch.int32, device=dev), ints(2)]
        self.status, self.starts, self.slots, self.positions = ints(n), ints(n + 1), ints(n), ints(n)
        self.turn = 0
        freq = lean.lean_rope_frequencies(lean.LEAN_ROPE_PLAIN, hd, cfg.rope_base)
        self.turns = torch.from_numpy(lean.lean_rope_turns(freq)).to(dev)
        self.ids, self.given = ints(n), ints(n)
        self.h, self.x = floats(n, d), floats(n, d)
        self.q, self.q_rot, self.att = (floats(n, q, hd) for _ in range(3))
        self.k, self.v = floats(n, kv, hd), floats(n, kv, hd)
        self.block, self.ffn = floats(n, d), floats(n, cfg.ffn)
        self.logits = floats(n, cfg.vocab)
        self.logprobs, self.entropy = floats(n), floats(n)
        self.top_ids, self.top_logprobs = ints(n, cfg.top), floats(n, cfg.top)
        size = lean.lean_paged_attention_workspace_bytes(n, q, kv, hd)
        self.att_ws = torch.zeros(size, dtype=torch.uint8, device=dev)
        size = lean.lean_token_logprobs_workspace_bytes(n, cfg.vocab, cfg.top)
        self.lp_ws = torch.zeros(size, dtype=torch.uint8, device=dev)

    def linear(self, name, x, y):
        n, k = self.w.shape[name]
        lean.lean_qmatmul(self.w.fmt[name], self.w.packed[name], x, y, n, k, self.n)

    def step(self):
        cfg, a, b = self.cfg, self.turn, 1 - self.turn
        self.turn = b
        lens = self.lens[b]
        lean.lean_kv_pages(self.lens[a], self.lens[a] + 1, self.table, self.ring, self.ring_state[a], cfg.page_size, lens,
                           self.ring_state[b], self.status, self.starts, self.slots, self.positions)
        lean.lean_embed_rows(cfg.table, self.w.packed["embed"], self.ids, self.h, self.n, cfg.vocab, cfg.hidden)
        norms = self.w.norms
        lean.lean_residual_norm(None, self.h, norms[0], None, self.x, eps=cfg.eps)
        for i in range(cfg.layers):
            for name, y in (("q", self.q), ("k", self.k), ("v", self.v)):
                self.linear((i, name), self.x, y)
            lean.lean_rope_append(self.q, self.k, self.v, self.positions, self.slots, self.turns, self.q_rot,
                                  self.k_cache[i], self.v_cache[i], rot_dim=cfg.head_dim, **self.scales[i])
            lean.lean_paged_attention(self.q_rot, self.k_cache[i], self.v_cache[i], self.table, lens, self.att,
                                      scale=cfg.head_dim ** -0.5, workspace=self.att_ws, **self.scales[i])
            self.linear((i, "o"), self.att, self.block)
            lean.lean_residual_norm(self.block, self.h, norms[2 * i + 1], self.h, self.x, eps=cfg.eps)
            gate, up = self.w.packed[(i, "gate")], self.w.packed[(i, "up")]
            for s in range(self.n):
                lean.lean_qmatmul_swiglu(cfg.linear, gate, up, self.x[s], self.ffn[s], cfg.ffn, cfg.hidden)
            self.linear((i, "down"), self.ffn, self.block)
            lean.lean_residual_norm(self.block, self.h, norms[2 * i + 2], self.h, self.x, eps=cfg.eps)
        self.linear("lm_head", self.x, self.logits)
        lean.lean_token_logprobs(self.logits, self.given, self.logprobs, entropy=self.entropy, top_ids=self.top_ids,
                                 top_logprobs=self.top_logprobs, workspace=self.lp_ws)
        self.ids.copy_(self.top_ids[:, 0])


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--layers", type=int, default=32)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--sequences", type=int, default=1)
    ap.add_argument("--graph", action="store_true", help="two steps recorded into a CUDA graph")
    ap.add_argument("--cache-bits", type=int, choices=(8, 16), default=16)
    args = ap.parse_args()
    cfg = Config(layers=args.layers, cache_bits=args.cache_bits)
    dec = Decoder(cfg, Weights(cfg), args.sequences, args.tokens + 8)
    dec.ids.copy_(torch.arange(args.sequences) + 1)
    out = []
    for _ in range(2):  # the first two tokens, and what a first call sets up
        dec.step()
        out.append(dec.ids.clone())
    pairs = (args.tokens - 2) // 2
    if args.graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            dec.step()
            first = dec.ids.clone()
            dec.step()
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(pairs):
        if args.graph:
            graph.replay()
            out += [first.clone(), dec.ids.clone()]
        else:
            for _ in range(2):
                dec.step()
                out.append(dec.ids.clone())
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    assert lean.lean_device_error(True) == 0 and not dec.status.any()
    for s in range(args.sequences):
        print("sequence %d: %s" % (s, " ".join(str(int(t[s])) for t in out)))
    print("last token: log probability %.3f, entropy %.3f" % (float(dec.top_logprobs[0, 0]), float(dec.entropy[0])))
    if pairs:
        print("%d layers, %d sequences: %.3f ms a step" % (args.layers, args.sequences, took / (2 * pairs) * 1e3))


if __name__ == "__main__":
    main()
