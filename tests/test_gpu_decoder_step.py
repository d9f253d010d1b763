"""One step of a decoder layer as a server runs it, every part on the device: the batch's tables, the append
into a cache in 4 bits, the attention over it, the choice of experts, the experts, the combination.

Each part is compared with the 64-bit oracle over what the part before it gave, with the tolerances of its
own tests; whole numbers are equal.
"""
import numpy as np
import pytest
import torch

import weight_only_quantized_affine_amd as q
from oracle import decoder_oracle as D
from test_gpu_paged_attention_4bit import Problem, close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
U = 2.0 ** -24
I32 = dict(dtype=torch.int32, device=DEV)


class Layer:
    hq, hk, d, group, page, e, k = 4, 2, 64, 32, 8, 16, 3

    def __init__(self, n_seqs, rows, n_pages, width, seed):
        self.rows, self.dim = rows, self.hq * self.d
        g = self.g = torch.Generator(device=DEV).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.cache = q.qlinear_paged_cache_4bit(n_pages, self.page, self.hk, self.d, self.group)
        self.counts, self.lens = torch.zeros(n_seqs, **I32), torch.zeros(n_seqs, **I32)
        self.table = torch.full((n_seqs, width), -1, **I32)
        self.free, self.free_count = torch.randperm(n_pages, generator=g, device=DEV).int(), torch.tensor([n_pages], **I32)
        self.cu, self.info = torch.zeros(n_seqs + 1, **I32), torch.zeros(4, **I32)
        self.pos, self.slots = (torch.zeros(rows, dtype=torch.int64, device=DEV) for _ in range(2))
        self.x = rand(rows, self.dim).to(BF)
        self.qkv = rand(rows, self.hq + 2 * self.hk, self.d).to(BF)
        angle = torch.arange(width * self.page, device=DEV)[:, None] * 10.0 ** -torch.arange(0, 2, 4 / self.d, device=DEV)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        self.q_rows, self.att = torch.empty(rows, self.hq, self.d, dtype=BF, device=DEV), torch.empty(rows, self.hq, self.d, dtype=BF, device=DEV)
        need = q.qlinear_paged_attention_4bit_workspace_size(self.q_rows, self.cache, self.table, max_q=rows)
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        self.router, self.logits = q.qlinear_quantize(rand(self.e, self.dim), 8, 64), torch.empty(rows, self.e, dtype=BF, device=DEV)
        self.codes = torch.randint(0, 256, (self.e, self.dim, self.dim // 2), generator=g, device=DEV).to(torch.uint8)
        self.scales = torch.randint(116, 122, (self.e, self.dim, self.dim // 32), generator=g, device=DEV).to(torch.uint8)
        self.ids, self.w = torch.empty(rows, self.k, dtype=torch.int64, device=DEV), torch.empty(rows, self.k, device=DEV)
        self.y, self.out = torch.empty(rows * self.k, self.dim, dtype=BF, device=DEV), torch.empty(rows, self.dim, dtype=BF, device=DEV)
        self.experts_ws = torch.empty(q.qlinear_apply_experts_workspace_size(rows * self.k, self.e), dtype=torch.uint8, device=DEV)

    def state(self):
        return [*self.cache, self.lens, self.table, self.free, self.free_count]

    def step(self):
        q.qlinear_kv_extend(self.counts, self.lens, self.table, page_size=self.page, rows=self.rows, free_pages=self.free,
                            free_count=self.free_count, cu_q=self.cu, positions=self.pos, slots=self.slots, info=self.info)
        xq, xk, xv = self.qkv.split([self.hq, self.hk, self.hk], dim=1)
        q.qlinear_kv_append_4bit(xk, xv, self.cache, self.slots, q=xq, q_out=self.q_rows, positions=self.pos, cos_sin=self.cos_sin)
        q.qlinear_paged_attention_4bit(self.q_rows, self.cache, self.table, self.cu, self.lens, max_q=self.rows, out=self.att,
                                       workspace=self.ws)
        q.qlinear_gemm(self.att.view(self.rows, self.dim), *self.router, bits=8, group_size=64, y=self.logits)
        q.qlinear_select_experts(self.logits, self.k, ids=self.ids, weights=self.w, n_rows=self.info[:1])
        q.qlinear_apply_experts(q.QL_MXFP4, self.codes, self.scales, self.ids.view(-1), self.x, n=self.dim, k=self.dim,
                                pos_per_row=self.k, y=self.y, workspace=self.experts_ws)
        q.qlinear_combine_experts(self.y, self.w, ids=self.ids, e=self.e, residual=self.x, out=self.out)

    def fresh(self, counts):
        self.counts.copy_(torch.tensor(counts, **I32))
        self.x.normal_(generator=self.g)
        self.qkv.normal_(generator=self.g)
        self.att.fill_(7)


def f64(t):
    return t.double().cpu().numpy()


STEPS = [[5, 1, 3, 0, 2], [1, 1, 1, 1, 1], [-1, 1, 1, 9, 1], [0, 1, 20, 1, 1], [3, -1, -1, 0, 8], [0, 0, 0, 0, 0], [12, 0, 0, 0, 0], [1, 1, 1, 1, 1]]


def test_a_captured_layer_follows_its_sequences():
    m = Layer(n_seqs=5, rows=14, n_pages=13, width=6, seed=3)
    lens, table = m.lens.tolist(), m.table.tolist()
    free = (m.free.tolist(), 13)
    m.fresh([0] * 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step()  # nothing but padding
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step()
    refused = 0
    for counts in STEPS:
        m.fresh(counts)
        before = [x.clone() for x in m.state()]
        graph.replay()
        torch.cuda.synchronize()
        cu, pos, slots, lens, table, stack, info = D.kv_extend(counts, lens, table, m.page, m.rows, free)
        free = (stack, 13)
        assert m.cu.tolist() == cu and m.pos.tolist() == pos and m.slots.tolist() == slots
        assert m.lens.tolist() == lens and m.table.tolist() == table and m.info.tolist() == info
        assert m.free[:len(stack)].tolist() == stack and int(m.free_count) == len(stack)
        t = info[0]
        refused += info[2] != 0
        # what was stored, and nothing else
        want = D.quantize_rows(f64(m.qkv[:t, -m.hk:]).astype(np.float32), m.group)
        flat = [x.transpose(1, 2).contiguous().transpose(1, 2).cpu().numpy() for x in m.cache[2:]]
        for i, s in enumerate(slots[:t]):
            assert (flat[0][s // m.page, s % m.page].view(np.uint32) == want[0][i]).all()
            assert (flat[1][s // m.page, s % m.page] == want[1][i]).all()
        kept = torch.ones(13 * m.page, dtype=torch.bool, device=DEV)
        kept[m.slots[:t]] = False
        for a, b in zip(m.cache, before):
            assert torch.equal(a.reshape(13 * m.page, -1)[kept], b.reshape(13 * m.page, -1)[kept])
        # the attention of the new tokens over it
        p = Problem.__new__(Problem)
        p.dtype, p.cache, p.q, p.lens = BF, list(m.cache), m.q_rows[:t], [(n, kv) for n, kv in zip(np.diff(cu).tolist(), lens)]
        p.table, p.cu = m.table.cpu(), np.array(cu, dtype=np.int32)
        if t:
            close(p, m.att[:t], p.oracle())
        assert (m.att[t:] == 7).all()
        # the choice and the combination
        ids, w = D.select_experts(f64(m.logits[:t]), m.k) if t else (np.zeros((0, m.k)), np.zeros((0, m.k)))
        assert (m.ids[:t].cpu().numpy() == ids).all() and (m.ids[t:] == -1).all() and (m.w[t:] == 0).all()
        assert (np.abs(f64(m.w[:t]) - w) <= U * (1 + 1e-6) * w).all()
        want, mag = D.combine_experts(f64(m.y), f64(m.w), m.ids.cpu().numpy(), m.e, f64(m.x))
        h = 2.0 ** -8
        assert (np.abs(f64(m.out) - want) <= (m.k + 2) * U * mag * (1 + h) + h * np.abs(want)).all()
        assert torch.equal(m.out[t:], m.x[t:])
        # eager, from the same state: the same bits
        after, out = [x.clone() for x in m.state()], m.out.clone()
        for a, b in zip(m.state(), before):
            a.copy_(b)
        m.att.fill_(7)
        m.step()
        assert torch.equal(m.out, out)
        for a, b in zip(m.state(), after):
            assert torch.equal(a, b)
    assert refused == 1  # 23 tokens in 14 rows


def test_two_layers_at_once_on_two_streams():
    """Nothing is shared between calls: two layers, each on its own stream, give what they give one after the other."""
    layers = [Layer(n_seqs=5, rows=14, n_pages=13, width=6, seed=s) for s in (8, 9)]
    steps = [c for c in STEPS if sum(max(x, 0) for x in c) <= 14]
    first = [[x.clone() for x in m.state()] for m in layers]
    inputs, want = [], []
    for m in layers:
        mine, outs = [], []
        for counts in steps:
            m.fresh(counts)
            mine.append((m.x.clone(), m.qkv.clone()))
            m.step()
            outs.append(m.out.clone())
        inputs.append(mine)
        want.append(outs)
    ends = [[x.clone() for x in m.state()] for m in layers]
    for m, s in zip(layers, first):
        for a, b in zip(m.state(), s):
            a.copy_(b)
    got = [[torch.empty_like(m.out) for _ in steps] for m in layers]
    plans = [torch.tensor(c, **I32) for c in steps]
    streams = [torch.cuda.Stream() for _ in layers]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(len(steps)):
        for n, (m, s) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(s):
                m.counts.copy_(plans[i])
                m.x.copy_(inputs[n][i][0])
                m.qkv.copy_(inputs[n][i][1])
                m.att.fill_(7)
                m.step()
                got[n][i].copy_(m.out)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for n, m in enumerate(layers):
        for a, b in zip(got[n], want[n]):
            assert torch.equal(a, b)
        for a, b in zip(m.state(), ends[n]):
            assert torch.equal(a, b)
