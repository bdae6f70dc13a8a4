"""An attention sublayer between the seam's two halves, over a paged 8-bit cache.

One decoder layer's attention: ``mhc.pre_delayed`` collapses the streams into
the layer's input, a projection forms queries, keys and values in one product,
``mhc.kv_append`` rotates them and writes the cache, ``mhc.kv_attend`` reads
it, and ``mhc.post`` mixes the projected result back into the streams.

``run()`` feeds three prompts of different lengths in one ragged call and then
decodes one token a sequence, a CUDA graph replayed for each step.  It repeats
the whole as single ragged calls over all tokens, and returns both results.

    python examples/attention_decode.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mhc_hyper_connection_pre_gb300 as mhc
from workloads import seam_inputs


class AttentionSublayer:
    """Random weights, and one layer's cache, for up to ``max_tokens`` tokens a sequence."""

    def __init__(self, sequences, max_tokens, *, C=5120, q_heads=40, heads=8, head_dim=128, page_tokens=64, seed=0):
        p = seam_inputs(1, C=C, seed=seed, fold=True)
        self.fn, self.bias, self.alpha, self.norm_w = (p[k].cuda() for k in ("fn", "bias", "alpha", "norm_w"))
        self.q_heads, self.heads, self.head_dim = q_heads, heads, head_dim
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5).bfloat16()

        self.w_qkv = weight((q_heads + 2 * heads) * head_dim, C)
        self.w_out = weight(C, q_heads * head_dim)
        turns = torch.outer(torch.arange(max_tokens, device="cuda"),
                            10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda") / head_dim))
        self.cos, self.sin = turns.cos(), turns.sin()
        pages = -(-max_tokens // page_tokens)
        self.cache = mhc.kv_cache(sequences * pages, heads, page_tokens, head_dim)
        # a real server hands out pages as sequences grow; here each sequence owns some, in no order
        self.block_table = torch.randperm(sequences * pages, generator=g, device="cuda").int().view(sequences, pages)

    def __call__(self, x, pre_in, seq_lens, cu_q=None):
        """x [T, n, C], the new tokens of all sequences; seq_lens with them.  Returns (next x, next pre_in)."""
        seam = mhc.pre_delayed(x, pre_in, self.fn, self.bias, self.alpha, self.norm_w)
        qkv = (seam["layer_input"] @ self.w_qkv.T).view(-1, self.q_heads + 2 * self.heads, self.head_dim)
        q, k, v = qkv.split([self.q_heads, self.heads, self.heads], dim=1)      # slices, not copies
        q = mhc.kv_append(self.cache, k, v, self.block_table, seq_lens, cu_q, q=q, cos=self.cos, sin=self.sin)
        o = mhc.kv_attend(q, self.cache, self.block_table, seq_lens, cu_q)["out"]
        y = o.flatten(1) @ self.w_out.T
        return mhc.post(x, y, seam["comb"], seam["post"]), seam["pre"]


def ragged(lengths):
    """(seq_lens, cu_q) of sequences that begin here."""
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return lens, torch.cat([lens.new_zeros(1), lens.cumsum(0, dtype=torch.int32)])


def run(prompts=(130, 5, 77), steps=4):
    """(stepped, at_once): x of the decoded tokens [sequences, steps, n, C], prompt first and then token by
    token, and all tokens in one call."""
    B, lengths = len(prompts), [n + steps for n in prompts]
    d = seam_inputs(sum(lengths), seed=1)
    every = {k: d[k].cuda().split(lengths) for k in ("x", "pre_in")}            # by sequence

    def tokens(key, begin, end):
        return torch.cat([t[b:e] for t, b, e in zip(every[key], begin, end)])

    layer = AttentionSublayer(B, max(lengths))
    lens, cu_q = ragged(lengths)
    x, _ = layer(tokens("x", [0] * B, lengths), tokens("pre_in", [0] * B, lengths), lens, cu_q)
    at_once = torch.stack([t[-steps:] for t in x.split(lengths)])

    layer = AttentionSublayer(B, max(lengths))
    lens, cu_q = ragged(prompts)
    layer(tokens("x", [0] * B, prompts), tokens("pre_in", [0] * B, prompts), lens, cu_q)
    x_in, pre_in = torch.empty_like(at_once[:, 0]), torch.empty_like(tokens("pre_in", [0] * B, [1] * B))

    def step():
        lens.add_(1)
        return layer(x_in, pre_in, lens)[0]

    def load(i):
        at = [n + i for n in prompts]
        x_in.copy_(tokens("x", at, [a + 1 for a in at]))
        pre_in.copy_(tokens("pre_in", at, [a + 1 for a in at]))

    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):               # the first step as it is: what is set up on first use is set up here
        out = [step().clone()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            x_out = step()
        for i in range(1, steps):
            load(i)
            graph.replay()
            out.append(x_out.clone())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    if mhc.device_status():
        raise RuntimeError("a call met a bad page or length")
    return torch.stack(out, dim=1), at_once


if __name__ == "__main__":
    stepped, at_once = run()
    error = (stepped.float() - at_once.float()).norm() / at_once.float().norm()
    print(f"{stepped.shape[1]} tokens of {stepped.shape[0]} sequences, token by token and at once: "
          f"relative difference {error:.2e}")
