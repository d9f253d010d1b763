"""Cases of the attention-side operators, timed and checked one pass at a time.

Three operators sit between the q|k|v products of a layer and its output product:

  norm_rope   per-head RMS norms of q and k with the position rotation, into tensors
  append      the same on the way into a paged cache, with v stored beside k
  attention   causal attention of each sequence's new tokens over its pages of the cache

`run` computes them in elementary torch operations in 32 bits, rounded once at the end, or (`own`)
by the calls of weight_only_quantized_affine_amd.  `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
THETA = 1.0e6


def listed():
    return [
        # One token of a 0.6B-class decoder (16 query and 8 key heads of 128): a launch's latency.
        dict(name="norm_rope_1tok", op="norm_rope", dtype="bf16", tokens=1, hq=16, hk=8, d=128, rot=128,
             interleaved=False, fused=True, max_pos=40960),
        # A prefill chunk of a 9B-class layer (q 4096, k and v 1024 wide), read out of one q|k|v product.
        dict(name="norm_rope_8192tok", op="norm_rope", dtype="bf16", tokens=8192, hq=32, hk=8, d=128, rot=128,
             interleaved=False, fused=True, max_pos=131072),
        # A ragged fp16 chunk with small heads, half of each rotated in neighbouring pairs.
        dict(name="norm_rope_777tok_pairs", op="norm_rope", dtype="f16", tokens=777, hq=24, hk=6, d=64, rot=32,
             interleaved=True, fused=False, max_pos=8192),
        # One decode step of 60 sequences padded to a captured batch of 64, pages of 16 tokens.
        dict(name="append_decode_64", op="append", dtype="bf16", tokens=64, padding=4, hq=16, hk=8, d=128, rot=128,
             interleaved=False, max_pos=40960, page=16, n_pages=512, heads_first=False, chunk=False),
        # A prefill chunk of a 9B-class layer into head-major pages.
        dict(name="append_chunk_4096", op="append", dtype="bf16", tokens=4096, padding=0, hq=32, hk=8, d=128, rot=128,
             interleaved=False, max_pos=131072, page=64, n_pages=80, heads_first=True, chunk=True),
        # One sequence of a 0.6B-class decoder, a short chat's length.
        dict(name="attn_decode_1x1025", op="attention", dtype="bf16", n_seqs=1, q_min=1, q_max=1, kv_min=1025,
             kv_max=1025, lens_seed=0, hq=16, hk=8, d=128, page=16, window=0, sinks=False, heads_first=False),
        # One sequence at the end of a long context.
        dict(name="attn_decode_1x131071", op="attention", dtype="bf16", n_seqs=1, q_min=1, q_max=1, kv_min=131071,
             kv_max=131071, lens_seed=0, hq=32, hk=8, d=128, page=64, window=0, sinks=False, heads_first=False),
        # A serving batch: 64 sequences of all lengths, one token each.
        dict(name="attn_decode_64_ragged", op="attention", dtype="bf16", n_seqs=64, q_min=1, q_max=1, kv_min=100,
             kv_max=16000, lens_seed=7, hq=32, hk=8, d=128, page=16, window=0, sinks=False, heads_first=False),
        # Checking drafted tokens: 5 a sequence, fp16 heads of 64 with a window and sinks, odd pages.
        dict(name="attn_draft_16x5_window", op="attention", dtype="f16", n_seqs=16, q_min=5, q_max=5, kv_min=300,
             kv_max=9000, lens_seed=3, hq=32, hk=8, d=64, page=24, window=2000, sinks=True, heads_first=True),
        # The first chunk of a prompt: a 9B-class layer, nothing cached before it.
        dict(name="attn_prefill_4096", op="attention", dtype="bf16", n_seqs=1, q_min=4096, q_max=4096, kv_min=4096,
             kv_max=4096, lens_seed=0, hq=32, hk=8, d=128, page=64, window=0, sinks=False, heads_first=False),
        # A later chunk of a long prompt, its length odd.
        dict(name="attn_chunk_1000_at_32k", op="attention", dtype="bf16", n_seqs=1, q_min=1000, q_max=1000,
             kv_min=32767, kv_max=32767, lens_seed=0, hq=32, hk=8, d=128, page=16, window=0, sinks=False,
             heads_first=False),
        # Continuous batching: sequences that decode next to sequences that prefill.
        dict(name="attn_mixed_12", op="attention", dtype="bf16", n_seqs=12, q_min=1, q_max=700, kv_min=700,
             kv_max=9000, lens_seed=11, hq=16, hk=8, d=128, page=16, window=0, sinks=False, heads_first=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attention", "attention"])
    d = rng.choice([64, 128, 128, 256])
    hk = rng.choice([1, 2, 3, 4, 6, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 5, 7, 8])
    dtype = rng.choice(["bf16", "f16"])
    if op == "attention":
        n_seqs = _log(rng, 1, 64)
        kind = rng.choice(["decode", "draft", "chunk", "mixed"])
        q_min, q_max = {"decode": (1, 1), "draft": (2, 8), "chunk": (9, 4000), "mixed": (1, 700)}[kind]
        if kind in ("chunk", "mixed"):
            n_seqs = min(n_seqs, 8)
        if kind == "chunk":
            q_min = q_max = _log(rng, 9, 4000 // n_seqs)
        if kind == "draft":
            q_min = q_max = rng.randint(2, 8)
        kv_max = _log(rng, max(16, q_max), {"decode": 16000, "draft": 12000, "chunk": 16000, "mixed": 9000}[kind])
        kv_min = rng.randint(max(1, q_max), kv_max)
        # the heads shrink until the work is within that of the listed cases
        while True:
            c = dict(op=op, dtype=dtype, n_seqs=n_seqs, q_min=q_min, q_max=q_max, kv_min=kv_min, kv_max=kv_max,
                     lens_seed=rng.randint(0, 1 << 20), hq=hq, hk=hk, d=d, page=rng.choice([1, 8, 16, 24, 37, 64, 128]),
                     window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), sinks=rng.random() < 0.3,
                     heads_first=rng.random() < 0.3)
            w = work(c)
            if (w["flops"] < 2.5e11 and w["bytes"] < 6e8) or hk == 1:
                return c
            hk, hq = 1, hq // hk
    tokens = _log(rng, 1, 4096)
    rot = rng.choice([d, d, d // 2, d // 4, 0])
    c = dict(op=op, dtype=dtype, tokens=tokens, hq=hq, hk=hk, d=d, rot=rot, interleaved=rng.random() < 0.4,
             max_pos=rng.choice([8192, 40960, 131072]))
    if op == "norm_rope":
        c["fused"] = rng.random() < 0.5
        return c
    c["padding"] = rng.choice([0, 0, tokens // 5])
    c["page"] = rng.choice([1, 8, 16, 24, 37, 64, 128])
    c["n_pages"] = -(-tokens // c["page"]) + rng.randint(1, 9)
    c["heads_first"] = rng.random() < 0.5
    c["chunk"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs


def _lens(case):
    """The (new tokens, cached tokens with them) of each sequence: log-uniform in the case's ranges."""
    rng = random.Random(case["lens_seed"])
    out = []
    for i in range(case["n_seqs"]):
        nq = case["q_max"] if i == 0 else _log(rng, case["q_min"], case["q_max"])
        if case["q_min"] == 1 and case["q_max"] > 8 and i % 3:  # a mixed batch: two of three decode
            nq = 1
        nkv = case["kv_max"] if i == 0 else _log(rng, case["kv_min"], case["kv_max"])
        out.append((nq, max(nkv, nq)))
    return out


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dt, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


def _table(max_pos, rot):
    """cos then sin of position * theta^(-2i/rot), angles in 64 bits, stored in 32."""
    i = torch.arange(0, rot, 2, device=DEV, dtype=torch.float64)
    ang = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * THETA ** (-i / rot)[None, :]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def _cache(g, case, n_pages, dt):
    hk, d, page = case["hk"], case["d"], case["page"]
    if case["heads_first"]:
        return [_randn(g, (n_pages, hk, page, d), dt).transpose(1, 2) for _ in range(2)]
    return [_randn(g, (n_pages, page, hk, d), dt) for _ in range(2)]


def prepare(case, seed):
    g = _gen(seed)
    dt = DT[case["dtype"]]
    hq, hk, d = case["hq"], case["hk"], case["d"]
    st = dict(case=case)
    if case["op"] == "attention":
        lens = _lens(case)
        page = case["page"]
        pages = [-(-nkv // page) for _, nkv in lens]
        n_pages = sum(pages) + 1
        st["k_cache"], st["v_cache"] = _cache(g, case, n_pages, dt)
        order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros((len(lens), max(pages)), dtype=torch.int32, device=DEV)
        at, cu = 0, [0]
        for s, (nq, _) in enumerate(lens):
            table[s, :pages[s]] = order[at:at + pages[s]]
            at += pages[s]
            cu.append(cu[-1] + nq)
        st.update(lens=lens, cu=cu, block_table=table, max_q=max(n for n, _ in lens),
                  cu_q=torch.tensor(cu, dtype=torch.int32, device=DEV),
                  kv_lens=torch.tensor([n for _, n in lens], dtype=torch.int32, device=DEV))
        st["q"] = _randn(g, (cu[-1], hq, d), dt, 2.0)
        st["sinks"] = torch.randn(hq, generator=g, device=DEV) * 2 if case["sinks"] else None
        if own:
            import weight_only_quantized_affine_amd as ql
            n = ql.qlinear_paged_attention_workspace_size(st["q"], st["k_cache"], st["block_table"], max_q=st["max_q"],
                                                          window=case["window"])
            st["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        return st
    t = case["tokens"]
    if case.get("fused", True):
        qkv = _randn(g, (t, (hq + 2 * hk) * d), dt)
        st["q"] = qkv[:, :hq * d].view(t, hq, d)
        st["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        st["v"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
    else:
        st["q"], st["k"] = _randn(g, (t, hq, d), dt), _randn(g, (t, hk, d), dt)
    st["q_weight"] = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(dt)
    st["k_weight"] = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(dt)
    st["cos_sin"] = _table(case["max_pos"], case["rot"]) if case["rot"] else None
    if case.get("chunk", True):
        first = int(torch.randint(0, case["max_pos"] - t + 1, (1,), generator=g, device=DEV))
        pos = torch.arange(first, first + t, device=DEV)
    else:
        pos = torch.randint(0, case["max_pos"], (t,), generator=g, device=DEV)
    st["positions"] = pos.to(torch.int64)
    if case["op"] == "append":
        page, n_pages, valid = case["page"], case["n_pages"], t - case["padding"]
        st["k_cache"], st["v_cache"] = _cache(g, case, n_pages, dt)
        slots = torch.full((t,), -1, dtype=torch.int64, device=DEV)
        if case["chunk"]:
            order = torch.randperm(n_pages, generator=g, device=DEV)
            j = torch.arange(valid, device=DEV)
            slots[:valid] = order[j // page] * page + j % page
        else:
            slots[:valid] = torch.randperm(n_pages * page, generator=g, device=DEV)[:valid]
        st.update(slots=slots, valid=valid)
        st["q_out"] = torch.empty((t, hq, d), dtype=dt, device=DEV)
    else:
        st["q_out"] = torch.empty((t, hq, d), dtype=dt, device=DEV)
        st["k_out"] = torch.empty((t, hk, d), dtype=dt, device=DEV)
    return st


# ---------------------------------------------------------------- one pass


def _plain_norm_rope(x, weight, st):
    case = st["case"]
    rot = case["rot"]
    v = x.float()
    v = v * torch.rsqrt((v * v).mean(dim=-1, keepdim=True) + EPS) * weight.float()
    if rot:
        cs = st["cos_sin"][st["positions"]]
        c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
        if case["interleaved"]:
            a, b = v[..., 0:rot:2], v[..., 1:rot:2]
            r = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
        else:
            a, b = v[..., :rot // 2], v[..., rot // 2:rot]
            r = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
        v = torch.cat([r, v[..., rot:]], dim=-1)
    return v.to(x.dtype)


def _plain_attention(st):
    case = st["case"]
    hq, hk, d, page, window = case["hq"], case["hk"], case["d"], case["page"], case["window"]
    rep = hq // hk
    out = torch.empty_like(st["q"])
    for s, (nq, nkv) in enumerate(st["lens"]):
        j = torch.arange(nkv, device=DEV)
        pg = st["block_table"][s][j // page].long()
        k = st["k_cache"][pg, j % page].float()
        v = st["v_cache"][pg, j % page].float()
        q = st["q"][st["cu"][s]:st["cu"][s + 1]].float().view(nq, hk, rep, d)
        p = torch.arange(nkv - nq, nkv, device=DEV)[:, None]
        see = j[None, :] <= p
        if window:
            see = see & (j[None, :] > p - window)
        see = see[:, None, :].expand(nq, rep, nkv).reshape(nq * rep, nkv)
        for h in range(hk):
            x = q[:, h].reshape(nq * rep, d) @ k[:, h].t().contiguous()
            x = (x * d ** -0.5).masked_fill(~see, -math.inf)
            m = x.max(dim=1, keepdim=True).values
            if st["sinks"] is not None:
                sink = st["sinks"][h * rep:(h + 1) * rep].repeat(nq)[:, None]
                m = torch.maximum(m, sink)
            e = torch.exp(x - m)
            z = e.sum(dim=1, keepdim=True)
            if st["sinks"] is not None:
                z = z + torch.exp(sink - m)
            o = (e @ v[:, h].contiguous()) / z
            out[st["cu"][s]:st["cu"][s + 1], h * rep:(h + 1) * rep] = o.view(nq, rep, d).to(out.dtype)
    return out


def run(state):
    st = state
    case = st["case"]
    if own:
        import weight_only_quantized_affine_amd as ql
        if case["op"] == "attention":
            return ql.qlinear_paged_attention(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["cu_q"],
                                              st["kv_lens"], max_q=st["max_q"], window=case["window"],
                                              sinks=st["sinks"], workspace=st["workspace"])
        if case["op"] == "append":
            ql.qlinear_kv_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"], q=st["q"],
                                 q_out=st["q_out"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                                 positions=st["positions"], cos_sin=st["cos_sin"], interleaved=case["interleaved"])
            return st["q_out"], st["k_cache"], st["v_cache"]
        return ql.qlinear_qk_norm_rope(st["q"], st["k"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                                       positions=st["positions"], cos_sin=st["cos_sin"],
                                       interleaved=case["interleaved"], q_out=st["q_out"], k_out=st["k_out"])
    if case["op"] == "attention":
        return _plain_attention(st)
    st["q_out"].copy_(_plain_norm_rope(st["q"], st["q_weight"], st))
    k = _plain_norm_rope(st["k"], st["k_weight"], st)
    if case["op"] == "append":
        n, page = st["valid"], case["page"]
        pg, at = st["slots"][:n] // page, st["slots"][:n] % page
        st["k_cache"][pg, at] = k[:n]
        st["v_cache"][pg, at] = st["v"][:n]
        return st["q_out"], st["k_cache"], st["v_cache"]
    st["k_out"].copy_(k)
    return st["q_out"], st["k_out"]


# ---------------------------------------------------------------- work and the definition in 64 bits


def work(case):
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "attention":
        pairs = read = toks = 0
        w = case["window"]
        for nq, nkv in _lens(case):
            toks += nq
            first = nkv - nq  # the first query's position
            read += min(nkv, nq - 1 + w) if w else nkv
            for p in range(first, nkv):
                pairs += min(p + 1, w) if w else p + 1
        return dict(bytes=read * hk * d * 2 * 2 + 2 * toks * hq * d * 2, flops=4 * pairs * hq * d)
    t = case["tokens"]
    rows = t * (hq + hk)
    b = 2 * rows * d * 2 + t * case["rot"] * 4 + t * 8 + 2 * d * 2
    if case["op"] == "append":
        n = t - case["padding"]
        b += 2 * n * hk * d * 2 + t * 8 - case["padding"] * hk * d * 2 * 2
    return dict(bytes=b, flops=rows * (4 * d + 3 * case["rot"]))


def _exact_heads(x, weight, table, positions, rot, interleaved):
    y = x.double().clone()
    rms = torch.sqrt((y.pow(2).sum(-1) / y.shape[-1] + EPS))
    y = y / rms.unsqueeze(-1) * weight.double()
    if rot:
        z = y.clone()
        cs = table[positions].double()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = cs[:, i, None], cs[:, rot // 2 + i, None]
            z[..., a] = y[..., a] * c - y[..., b] * s
            z[..., b] = y[..., a] * s + y[..., b] * c
        y = z
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] != "attention":
        args = (st["cos_sin"], st["positions"], case["rot"], case["interleaved"])
        q = _exact_heads(st["q"], st["q_weight"], *args)
        k = _exact_heads(st["k"], st["k_weight"], *args)
        if case["op"] == "norm_rope":
            return q, k
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        keep = st["slots"] >= 0
        pg = torch.div(st["slots"][keep], case["page"], rounding_mode="floor")
        at = st["slots"][keep] - pg * case["page"]
        kc[pg, at] = k[keep]
        vc[pg, at] = st["v"].double()[keep]
        return q, kc, vc
    rep, page, w, d = case["hq"] // case["hk"], case["page"], case["window"], case["d"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for s in range(case["n_seqs"]):
        q0, q1 = int(st["cu_q"][s]), int(st["cu_q"][s + 1])
        n = int(st["kv_lens"][s])
        pages = st["block_table"][s, :(n + page - 1) // page].long()
        for h in range(case["hk"]):
            k = st["k_cache"][pages, :, h].reshape(-1, d)[:n].double()
            v = st["v_cache"][pages, :, h].reshape(-1, d)[:n].double()
            for g in range(rep):
                head = h * rep + g
                for a in range(q0, q1, 2048):
                    b = min(q1, a + 2048)
                    x = torch.matmul(st["q"][a:b, head].double(), k.t().contiguous()) / math.sqrt(d)
                    at = n - (q1 - torch.arange(a, b, device=DEV))[:, None]
                    j = torch.arange(n, device=DEV)[None, :]
                    hide = j > at
                    if w:
                        hide = hide | (j <= at - w)
                    x[hide] = -math.inf
                    if st["sinks"] is not None:
                        col = st["sinks"][head].double().expand(b - a, 1)
                        p = torch.softmax(torch.cat([x, col], dim=1), dim=1)[:, :n]
                    else:
                        p = torch.softmax(x, dim=1)
                    out[a:b, head] = torch.matmul(p, v)
    return out
