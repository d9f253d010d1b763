"""The attention block of a decoder layer on quantized weights and a paged cache.

One layer shaped like Qwen3-0.6B's (hidden 1024, 16 query and 8 key heads of 128): the q|k|v
weights are one 4-bit matrix, so a step is

    qlinear_gemm / qlinear_gemv   x -> q|k|v, one product
    qlinear_kv_append             norms and rotation of q and k, k and v into the cache's pages
    qlinear_paged_attention       the new tokens over everything cached
    qlinear_gemm / qlinear_gemv   heads -> hidden

Run on a GPU: ``python examples/attention_block.py`` prefills four prompts in chunks, those that are
through decoding next to the chunks of the others, then decodes all of them from one captured graph,
and checks that the outputs equal those of each whole sequence in a single call.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_affine_amd as ql  # noqa: E402

BITS, GROUP = 4, 64


def rope_table(max_pos: int, rot: int, theta: float = 1.0e6, device="cuda"):
    """fp32 [max_pos, rot]: cosines, then sines, of position * theta^(-2i/rot); angles in 64 bits."""
    inv = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv[None]
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


class PagedCache:
    """Pages of one layer, and for each sequence its pages and length."""

    def __init__(self, n_pages, page_size, heads, d, max_seqs, max_pages, dtype=torch.bfloat16, device="cuda"):
        shape = (n_pages, page_size, heads, d)
        self.k, self.v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        self.page_size = page_size
        self.free = list(range(n_pages))
        self.pages = [[] for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.block_table = torch.zeros((max_seqs, max_pages), dtype=torch.int32, device=device)
        self.kv_lens = torch.zeros(max_seqs, dtype=torch.int32, device=device)

    def extend(self, counts):
        """Room for counts[s] new tokens of each sequence -> (positions, slots, cu_q) of the batch."""
        positions, slots, cu = [], [], [0]
        for s, n in enumerate(counts):
            while len(self.pages[s]) * self.page_size < self.lens[s] + n:
                self.block_table[s, len(self.pages[s])] = self.free[-1]
                self.pages[s].append(self.free.pop())
            for p in range(self.lens[s], self.lens[s] + n):
                positions.append(p)
                slots.append(self.pages[s][p // self.page_size] * self.page_size + p % self.page_size)
            self.lens[s] += n
            cu.append(cu[-1] + n)
        device = self.k.device
        self.kv_lens.copy_(torch.tensor(self.lens, dtype=torch.int32))
        return (torch.tensor(positions, device=device), torch.tensor(slots, device=device),
                torch.tensor(cu, dtype=torch.int32, device=device))


class AttentionBlock:
    def __init__(self, hidden=1024, hq=16, hk=8, d=128, max_pos=4096, eps=1e-6, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        weight = lambda n, k: torch.randn((n, k), generator=g, device=device) * k ** -0.5  # noqa: E731
        self.hq, self.hk, self.d, self.eps = hq, hk, d, eps
        self.w_qkv = ql.qlinear_quantize(weight((hq + 2 * hk) * d, hidden), BITS, GROUP)
        self.w_out = ql.qlinear_quantize(weight(hidden, hq * d), BITS, GROUP)
        self.q_norm, self.k_norm = ((1 + 0.2 * torch.randn(d, generator=g, device=device)).bfloat16() for _ in range(2))
        self.cos_sin = rope_table(max_pos, d, device=device)

    @staticmethod
    def linear(x, w):
        product = ql.qlinear_gemv if x.shape[0] <= 8 else ql.qlinear_gemm
        return product(x, *w, bits=BITS, group_size=GROUP)

    def __call__(self, x, cache, positions, slots, cu_q, max_q):
        """x [t, hidden], the new tokens of the cache's sequences -> [t, hidden]."""
        t, hq, hk, d = x.shape[0], self.hq, self.hk, self.d
        q, k, v = self.linear(x, self.w_qkv).view(t, hq + 2 * hk, d).split([hq, hk, hk], dim=1)
        q = ql.qlinear_kv_append(k, v, cache.k, cache.v, slots, q=q, q_out=q, q_weight=self.q_norm, k_weight=self.k_norm,
                                 eps=self.eps, positions=positions, cos_sin=self.cos_sin)
        out = ql.qlinear_paged_attention(q, cache.k, cache.v, cache.block_table, cu_q, cache.kv_lens, max_q=max_q)
        out = out if out.is_contiguous() else out.contiguous()
        return self.linear(out.view(t, hq * d), self.w_out)


def main(prompts=(300, 41, 130, 7), chunk=128, steps=6, seed=1):
    block = AttentionBlock()
    n_seqs, rounds = len(prompts), max(-(-p // chunk) for p in prompts)
    # a prompt that takes fewer chunks than the longest decodes a token in each round that is left
    first = [p + rounds - -(-p // chunk) for p in prompts]
    total = [n + steps for n in first]
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = [torch.randn((n, 1024), generator=g, device="cuda").bfloat16() for n in total]

    def new_cache():
        return PagedCache(64, 16, block.hk, block.d, n_seqs, 64)

    # each sequence whole, in one call
    whole = []
    for s, x in enumerate(tokens):
        cache = new_cache()
        whole.append(block(x, cache, *cache.extend([x.shape[0] if i == s else 0 for i in range(n_seqs)]), x.shape[0]))

    # prompts in chunks, all sequences in one batch; those whose prompt is through decode
    cache, got = new_cache(), [[] for _ in prompts]
    for _ in range(rounds):
        counts = [min(chunk, p - cache.lens[s]) if cache.lens[s] < p else 1 for s, p in enumerate(prompts)]
        x = torch.cat([tokens[s][cache.lens[s]:cache.lens[s] + n] for s, n in enumerate(counts)])
        y = block(x, cache, *cache.extend(counts), max(counts))
        for s, part in enumerate(y.split(counts)):
            got[s].append(part)

    # decode: one graph, its inputs copied in before each replay
    x = torch.empty((n_seqs, 1024), dtype=torch.bfloat16, device="cuda")
    step, graph, y = None, None, None
    for i in range(steps):
        new = cache.extend([1] * n_seqs)
        x.copy_(torch.stack([tokens[s][n + i] for s, n in enumerate(first)]))
        if graph is None:
            step = new
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):  # warm up; the same slots are written again by the replay
                block(x, cache, *step, 1)
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = block(x, cache, *step, 1)
        for a, b in zip(step, new):
            a.copy_(b)
        graph.replay()
        for s in range(n_seqs):
            got[s].append(y[s:s + 1].clone())
    # the 4-bit products round differently in the GEMV and the GEMM: compare by norm
    worst = max(float(((torch.cat(a) - b).float().norm(dim=1) / b.float().norm(dim=1)).max()) for a, b in zip(got, whole))
    print(f"{n_seqs} sequences, {sum(total)} tokens: chunks and single tokens against whole sequences, worst row {worst:.2e}")
    return worst


if __name__ == "__main__":
    sys.exit(main() > 2e-2)
