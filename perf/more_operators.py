"""Cases of a decoder layer's operators around a cache in 4 bits and around routed experts.

  extend     lengths, block table, positions and slots of a batch from its token counts, pages taken
             from and given back to a list of free ones
  append     norm and rotation of new keys, then k and v quantized to 4 bits in the pages of a cache,
             and the stored rows read back as the values they stand for
  attention  causal attention of each sequence's new tokens over its pages of such a cache
  select     the experts of each token and their weights from a router's logits
  combine    the weighted sum of a token's expert outputs and its residual

`run` computes them in elementary torch operations, or (`own`) by the calls of
weight_only_quantized_affine_amd.  `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
THETA = 1.0e6


def listed():
    return [
        # One decode step of 60 sequences in a captured batch of 64: some begin a page, four are padding.
        dict(name="extend_decode_64", op="extend", n_seqs=64, rows=64, count_max=1, release=0, len_max=16000, page=16,
             max_pages=1024, spare=64, lens_seed=5),
        # A step that admits prompts: 300 sequences, two of three decode, the others bring chunks of up
        # to 1000 tokens, and 20 are through and give their pages back.
        dict(name="extend_mixed_300", op="extend", n_seqs=300, rows=65536, count_max=1000, release=20, len_max=30000,
             page=16, max_pages=2048, spare=8000, lens_seed=6),
        # One decode step of 60 sequences padded to a captured batch of 64 (a 0.6B-class decoder).
        dict(name="append_decode_64", op="append", dtype="bf16", tokens=64, padding=4, hq=16, hk=8, d=128, group=64,
             rot=128, interleaved=False, max_pos=40960, page=16, n_pages=512, heads_first=True, chunk=False),
        # A prefill chunk of a 9B-class layer.
        dict(name="append_chunk_4096", op="append", dtype="bf16", tokens=4096, padding=0, hq=32, hk=8, d=128, group=64,
             rot=128, interleaved=False, max_pos=131072, page=64, n_pages=80, heads_first=True, chunk=True),
        # One sequence of a 0.6B-class decoder, a short chat's length.
        dict(name="attn_decode_1x1025", op="attention", dtype="bf16", n_seqs=1, q_min=1, q_max=1, kv_min=1025,
             kv_max=1025, lens_seed=0, hq=16, hk=8, d=128, group=64, page=16, window=0, sinks=False, heads_first=True),
        # A serving batch: 64 sequences of all lengths, one token each.
        dict(name="attn_decode_64_ragged", op="attention", dtype="bf16", n_seqs=64, q_min=1, q_max=1, kv_min=100,
             kv_max=16000, lens_seed=7, hq=32, hk=8, d=128, group=64, page=16, window=0, sinks=False, heads_first=True),
        # Checking drafted tokens: 5 a sequence, fp16 heads of 64 with a window and sinks, odd token-major pages.
        dict(name="attn_draft_16x5_window", op="attention", dtype="f16", n_seqs=16, q_min=5, q_max=5, kv_min=300,
             kv_max=9000, lens_seed=3, hq=32, hk=8, d=64, group=32, page=24, window=2000, sinks=True,
             heads_first=False),
        # A later chunk of a long prompt, its length odd.
        dict(name="attn_chunk_1000_at_32k", op="attention", dtype="bf16", n_seqs=1, q_min=1000, q_max=1000,
             kv_min=32767, kv_max=32767, lens_seed=0, hq=32, hk=8, d=128, group=64, page=16, window=0, sinks=False,
             heads_first=True),
        # One token, softmax over 128 experts, the best 8 renormalised.
        dict(name="select_1tok_128", op="select", dtype="bf16", tokens=1, padding=0, e=128, k=8, sigmoid=False,
             bias=False, n_groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0),
        # A prefill chunk: sigmoid scores of 256 experts with a balancing bias, 4 groups of 8, 8 experts.
        dict(name="select_8192tok_256_groups", op="select", dtype="f32", tokens=8192, padding=0, e=256, k=8,
             sigmoid=True, bias=True, n_groups=8, top_groups=4, group_top=2, renormalize=True, scale=2.5),
        # A small decode batch, four experts each, outputs of 2880 values.
        dict(name="combine_16tok_4", op="combine", dtype="bf16", tokens=16, k=4, e=32, n=2880, residual=True,
             dropped=False),
        # A prefill chunk, eight experts each, a few positions routed nowhere.
        dict(name="combine_4096tok_8", op="combine", dtype="bf16", tokens=4096, k=8, e=256, n=4096, residual=True,
             dropped=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["extend", "append", "attention", "attention", "select", "combine"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "extend":
        n = _log(rng, 1, 600)
        count_max = rng.choice([1, 1, 8, 1000])
        return dict(op=op, n_seqs=n, rows=n * (1 if count_max == 1 else min(count_max, 220)) + rng.randint(0, 9),
                    count_max=count_max, release=rng.choice([0, n // 9]), len_max=_log(rng, 20, 15000),
                    page=rng.choice([1, 8, 16, 24, 37, 64, 128]), max_pages=0, spare=rng.choice([0, 100, 20000]),
                    lens_seed=rng.randint(0, 1 << 20))
    d = rng.choice([64, 128, 128, 256])
    group = rng.choice([32, 64, 64] if d == 64 else [32, 64, 64, 128])
    hk = rng.choice([1, 2, 3, 4, 6, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 5, 7, 8])
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
                     lens_seed=rng.randint(0, 1 << 20), hq=hq, hk=hk, d=d, group=group,
                     page=rng.choice([1, 8, 16, 24, 37, 64, 128]), window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]),
                     sinks=rng.random() < 0.3, heads_first=rng.random() < 0.7)
            w = work(c)
            if (w["flops"] < 2.5e11 and w["bytes"] < 2.2e8) or hk == 1:
                return c
            hk, hq = 1, hq // hk
    if op == "append":
        tokens = _log(rng, 1, 4096)
        page = rng.choice([1, 8, 16, 24, 37, 64, 128])
        return dict(op=op, dtype=dtype, tokens=tokens, padding=rng.choice([0, 0, tokens // 5]), hq=hq, hk=hk, d=d,
                    group=group, rot=rng.choice([d, d, d // 2, d // 4, 0]), interleaved=rng.random() < 0.4,
                    max_pos=rng.choice([8192, 40960, 131072]), page=page, n_pages=-(-tokens // page) + rng.randint(1, 9),
                    heads_first=rng.random() < 0.7, chunk=rng.random() < 0.5)
    tokens = _log(rng, 1, 8192)
    if op == "select":
        n_groups = rng.choice([1, 1, 1, 2, 4, 8])
        e = n_groups * _log(rng, 4, 512 // n_groups)
        top_groups = rng.randint(1, n_groups)
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), tokens=tokens, padding=rng.choice([0, tokens // 4]),
                    e=e, k=rng.randint(1, min(10, top_groups * (e // n_groups))), sigmoid=rng.random() < 0.5,
                    bias=rng.random() < 0.5, n_groups=n_groups, top_groups=top_groups, group_top=rng.choice([1, 2]),
                    renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 1.0, 2.5]))
    k, dtype = rng.choice([1, 2, 4, 6, 8]), rng.choice(["bf16", "f16", "f32"])
    n = rng.choice([_log(rng, 64, 2000), 1024, 2880, 4096])
    tokens = min(tokens, (1 << 27) // (k * n * (2 if dtype == "f32" else 1)), 4096)
    return dict(op=op, dtype=dtype, tokens=tokens, k=k, e=rng.choice([8, 32, 256]), n=n, residual=rng.random() < 0.6,
                dropped=rng.random() < 0.4)


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


def _quantize(x, group):
    """Rows of 16-bit values -> (words [.., d/8] int32, params [.., d/group, 2] fp16): per group the scale
    (max - min) / 15 and the bias min in fp16, the codes the nearest levels of those."""
    v = x.float().unflatten(-1, (-1, group))
    lo, hi = v.amin(-1), v.amax(-1)
    s, b = ((hi - lo) / 15).half(), lo.half()
    c = torch.round((v - b.float()[..., None]) / s.float()[..., None]).clamp(0, 15)
    c = torch.where(s[..., None] == 0, torch.zeros_like(c), c).to(torch.int64).flatten(-2).unflatten(-1, (-1, 8))
    w = (c << (4 * torch.arange(8, device=x.device))).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32), torch.stack([s, b], dim=-1)


def _dequantize(words, params):
    """The values of rows, in the type of 64 or 32 bits that `params` has."""
    c = (words[..., None] >> (4 * torch.arange(8, device=words.device, dtype=torch.int32))) & 15
    c = c.flatten(-2).unflatten(-1, (params.shape[-2], -1)).to(params.dtype)
    return (c * params[..., 0:1] + params[..., 1:2]).flatten(-2)


def _cache(g, case, n_pages, dt):
    """(k_codes, k_params, v_codes, v_params), [n_pages, page, hk, ...], head-major pages or token-major ones."""
    hk, d, page, group = case["hk"], case["d"], case["page"], case["group"]
    shape = (n_pages, hk, page, d) if case["heads_first"] else (n_pages, page, hk, d)
    out = []
    for _ in range(2):
        words = torch.empty(shape[:3] + (d // 8,), dtype=torch.int32, device=DEV)
        params = torch.empty(shape[:3] + (d // group, 2), dtype=torch.float16, device=DEV)
        step = max(1, (1 << 25) // (hk * page * d))
        for a in range(0, n_pages, step):
            b = min(n_pages, a + step)
            words[a:b], params[a:b] = _quantize(_randn(g, (b - a,) + shape[1:], dt), group)
        out += [x.transpose(1, 2) if case["heads_first"] else x for x in (words, params)]
    return out


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "extend":
        return _prepare_extend(case, seed, st)
    dt = DT[case["dtype"]]
    if case["op"] == "select":
        t, e = case["tokens"], case["e"]
        st["logits"] = _randn(g, (t, e), dt, 1.5)
        st["bias"] = torch.randn(e, generator=g, device=DEV) * 0.1 if case["bias"] else None
        st["n_rows"] = torch.tensor([t - case["padding"]], dtype=torch.int32, device=DEV) if case["padding"] else None
        return st
    if case["op"] == "combine":
        t, k, e, n = case["tokens"], case["k"], case["e"], case["n"]
        st["y"] = _randn(g, (t * k, n), dt)
        w = torch.rand((t, k), generator=g, device=DEV) + 0.05
        st["weights"] = w / w.sum(dim=1, keepdim=True)
        st["ids"] = torch.randint(0, e, (t, k), generator=g, device=DEV)
        if case["dropped"]:
            st["ids"][torch.rand((t, k), generator=g, device=DEV) < 0.02] = -1
        st["residual"] = _randn(g, (t, n), dt) if case["residual"] else None
        return st
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "attention":
        lens, page = _lens(case), case["page"]
        pages = [-(-nkv // page) for _, nkv in lens]
        n_pages = sum(pages) + 1
        st["cache"] = _cache(g, case, n_pages, dt)
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
            n = ql.qlinear_paged_attention_4bit_workspace_size(st["q"], st["cache"], st["block_table"],
                                                               max_q=st["max_q"], window=case["window"])
            st["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        return st
    t, page, n_pages, valid = case["tokens"], case["page"], case["n_pages"], case["tokens"] - case["padding"]
    qkv = _randn(g, (t, (hq + 2 * hk) * d), dt)
    st["q"] = qkv[:, :hq * d].view(t, hq, d)
    st["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
    st["v"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
    st["q_weight"] = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(dt)
    st["k_weight"] = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(dt)
    st["cos_sin"] = _table(case["max_pos"], case["rot"]) if case["rot"] else None
    st["cache"] = _cache(g, case, n_pages, dt)
    slots = torch.full((t,), -1, dtype=torch.int64, device=DEV)
    if case["chunk"]:
        first = int(torch.randint(0, case["max_pos"] - t + 1, (1,), generator=g, device=DEV))
        pos = torch.arange(first, first + t, device=DEV)
        order = torch.randperm(n_pages, generator=g, device=DEV)
        j = torch.arange(valid, device=DEV)
        slots[:valid] = order[j // page] * page + j % page
    else:
        pos = torch.randint(0, case["max_pos"], (t,), generator=g, device=DEV)
        slots[:valid] = torch.randperm(n_pages * page, generator=g, device=DEV)[:valid]
    st.update(positions=pos.to(torch.int64), slots=slots, q_out=torch.empty((t, hq, d), dtype=dt, device=DEV))
    st["k_back"], st["v_back"] = (torch.empty((t, hk, d), dtype=dt, device=DEV) for _ in range(2))
    return st


def _prepare_extend(case, seed, st):
    """Sequences of all lengths with their pages, and a list of free ones that holds `spare` more than the
    step needs."""
    rng = random.Random(case["lens_seed"])
    n, page = case["n_seqs"], case["page"]
    lens = [_log(rng, 1, case["len_max"]) for _ in range(n)]
    gone = set(rng.sample(range(n), case["release"]))
    counts, left = [], case["rows"]
    for s in range(n):
        c = 1 if case["count_max"] == 1 or s % 3 else _log(rng, 1, case["count_max"])
        if case["count_max"] == 1 and s % 16 == 15:  # a place of the captured batch that holds no sequence
            c = 0
        c = -1 if s in gone else min(c, left - (n - 1 - s))
        left -= max(c, 0)
        counts.append(c)
    have = [-(-x // page) for x in lens]
    after = [-(-(x + max(c, 0)) // page) for x, c in zip(lens, counts)]
    order = list(range(sum(after) + case["spare"]))
    random.Random(seed).shuffle(order)
    table = torch.full((n, max(case["max_pages"], max(after))), -1, dtype=torch.int32)
    at = 0
    for s in range(n):
        table[s, :have[s]] = torch.tensor(order[at:at + have[s]], dtype=torch.int32)
        at += have[s]
    free = order[at:]
    st["free_pages"] = torch.full((len(order),), -1, dtype=torch.int32)
    st["free_pages"][:len(free)] = torch.tensor(free, dtype=torch.int32)
    st["free_count"] = torch.tensor([len(free)], dtype=torch.int32)
    st.update(counts=torch.tensor(counts, dtype=torch.int32), lens=torch.tensor(lens, dtype=torch.int32), block_table=table)
    st = {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in st.items()}
    i32 = dict(dtype=torch.int32, device=DEV)
    st.update(new_lens=torch.empty(n, **i32), new_count=torch.empty(1, **i32))
    return st


# ---------------------------------------------------------------- one pass


def _plain_extend(st):
    case = st["case"]
    page, rows = case["page"], case["rows"]
    counts, lens, table, free = st["counts"].long(), st["lens"].long(), st["block_table"], st["free_pages"]
    n, width = table.shape
    gone = counts < 0
    new = counts.clamp(min=0)
    old = torch.where(gone, torch.zeros_like(lens), lens)
    had = (lens + page - 1) // page
    have, after = (old + page - 1) // page, (old + new + page - 1) // page
    back, need = had - have, after - have
    f0 = st["free_count"].long()
    total, n_back, n_need = new.sum(), back.sum(), need.sum()
    why = ((total > rows).int() + 2 * (n_need > f0 + n_back).int()
           + 4 * ((lens < 0) | (old + new > width * page)).any().int()
           + 8 * ((f0 < 0) | (f0 + n_back > free.shape[0])).int())
    ok = why == 0
    # pages that come back, in order, on top of the list
    j = torch.arange(width, device=DEV)[None, :]
    given = (j < had[:, None]) & gone[:, None] & ok
    at = f0 + (torch.cumsum(back, 0) - back)[:, None] + j
    free = torch.cat([free, free.new_zeros(1)])  # the last place takes what is not given
    free.scatter_(0, torch.where(given, at, free.shape[0] - 1).flatten(), table.flatten())
    free = free[:-1]
    # pages that are taken, from the top down
    taken = (j >= have[:, None]) & (j < after[:, None]) & ok
    at = f0 + n_back - 1 - ((torch.cumsum(need, 0) - need)[:, None] + j - have[:, None])
    table = torch.where(taken, free[at.clamp(0, free.shape[0] - 1)], table)
    cu = torch.cat([total.new_zeros(1), torch.cumsum(new, 0)]) * ok
    i = torch.arange(rows, device=DEV)
    s = torch.searchsorted(cu[1:].contiguous(), i, right=True).clamp(max=n - 1)
    inside = i < cu[-1]
    pos = torch.where(inside, old[s] + i - cu[s], torch.zeros_like(i))
    slot = torch.where(inside, table[s, (pos // page).clamp(max=width - 1)].long() * page + pos % page, -torch.ones_like(i))
    st["new_lens"].copy_(torch.where(ok, old + new, lens))
    st["new_count"].copy_(torch.where(ok, f0 + n_back - n_need, f0))
    st["block_table"].copy_(table)
    st["free_pages"].copy_(free)
    info = torch.stack([cu[-1], (n_need * ok)[0], why[0].long(), st["new_count"][0].long()]).int()
    return cu.int(), pos, slot, st["new_lens"], st["block_table"], st["free_pages"], st["new_count"], info


def _plain_norm_rope(x, weight, st, wide):
    """In 64 bits where a value decides a code."""
    case = st["case"]
    rot, dt = case["rot"], torch.float64 if wide else torch.float32
    v = x.to(dt)
    v = v * torch.rsqrt((v * v).mean(dim=-1, keepdim=True) + EPS) * weight.to(dt)
    if rot:
        cs = st["cos_sin"][st["positions"]].to(dt)
        c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
        if case["interleaved"]:
            a, b = v[..., 0:rot:2], v[..., 1:rot:2]
            r = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
        else:
            a, b = v[..., :rot // 2], v[..., rot // 2:rot]
            r = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
        v = torch.cat([r, v[..., rot:]], dim=-1)
    return v.to(x.dtype)


def _plain_append(st):
    case = st["case"]
    page, t = case["page"], case["tokens"]
    n = t - case["padding"]
    st["q_out"].copy_(_plain_norm_rope(st["q"], st["q_weight"], st, False))
    k = _plain_norm_rope(st["k"], st["k_weight"], st, True)
    pg, at = st["slots"][:n] // page, st["slots"][:n] % page
    back = []
    for x, words, params in ((k, *st["cache"][:2]), (st["v"], *st["cache"][2:])):
        words[pg, at], params[pg, at] = _quantize(x[:n], case["group"])
        y = torch.zeros_like(x, memory_format=torch.contiguous_format)
        y[:n] = _dequantize(words[pg, at], params[pg, at].float()).to(x.dtype)
        back.append(y)
    return st["q_out"], *back


def _plain_attention(st):
    case = st["case"]
    hq, hk, d, page, window = case["hq"], case["hk"], case["d"], case["page"], case["window"]
    rep = hq // hk
    out = torch.empty_like(st["q"])
    kc, kp, vc, vp = st["cache"]
    for s, (nq, nkv) in enumerate(st["lens"]):
        j = torch.arange(nkv, device=DEV)
        pg, at = st["block_table"][s][j // page].long(), j % page
        k = _dequantize(kc[pg, at], kp[pg, at].float())
        v = _dequantize(vc[pg, at], vp[pg, at].float())
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


def _plain_select(st):
    case = st["case"]
    t, e, k, n_groups = case["tokens"], case["e"], case["k"], case["n_groups"]
    x = st["logits"].double()  # near ties: what is chosen hangs on the last bits
    if case["sigmoid"]:
        p = 1 / (1 + torch.exp(-x))
    else:
        p = torch.exp(x - x.max(dim=1, keepdim=True).values)
        p = p / p.sum(dim=1, keepdim=True)
    c = p if st["bias"] is None else p + st["bias"].double()
    if n_groups > 1:
        g = c.view(t, n_groups, -1).sort(dim=2, descending=True).values[:, :, :case["group_top"]].sum(dim=2)
        order = g.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        keep = torch.zeros_like(g, dtype=torch.bool).scatter_(1, order, True)
        c = c.masked_fill(~keep.repeat_interleave(e // n_groups, dim=1), -math.inf)
    ids = c.sort(dim=1, descending=True, stable=True).indices[:, :k].contiguous()
    w = p.gather(1, ids)
    if case["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = (w * case["scale"]).float()
    if st["n_rows"] is not None:
        dead = torch.arange(t, device=DEV)[:, None] >= st["n_rows"]
        ids, w = ids.masked_fill(dead, -1), w.masked_fill(dead, 0)
    return ids, w


def _plain_combine(st):
    case = st["case"]
    on = (st["ids"] >= 0) & (st["ids"] < case["e"])
    y = st["y"].float().view(case["tokens"], case["k"], case["n"]) * st["weights"][:, :, None]
    out = y.masked_fill(~on[:, :, None], 0).sum(dim=1)
    if st["residual"] is not None:
        out = out + st["residual"].float()
    return out.to(st["y"].dtype)


def run(state):
    st = state
    case = st["case"]
    if not own:
        return {"extend": _plain_extend, "append": _plain_append, "attention": _plain_attention,
                "select": _plain_select, "combine": _plain_combine}[case["op"]](st)
    import weight_only_quantized_affine_amd as ql
    if case["op"] == "extend":
        cu_q, positions, slots, info = ql.qlinear_kv_extend(
            st["counts"], st["lens"], st["block_table"], page_size=case["page"], rows=case["rows"],
            free_pages=st["free_pages"], free_count=st["free_count"], lens_out=st["new_lens"],
            free_count_out=st["new_count"])
        return cu_q, positions, slots, st["new_lens"], st["block_table"], st["free_pages"], st["new_count"], info
    if case["op"] == "append":
        ql.qlinear_kv_append_4bit(st["k"], st["v"], st["cache"], st["slots"], q=st["q"], q_out=st["q_out"],
                                  q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS, positions=st["positions"],
                                  cos_sin=st["cos_sin"], interleaved=case["interleaved"])
        ql.qlinear_kv_read_4bit(st["cache"], st["slots"], k_out=st["k_back"], v_out=st["v_back"])
        return st["q_out"], st["k_back"], st["v_back"]
    if case["op"] == "attention":
        return ql.qlinear_paged_attention_4bit(st["q"], st["cache"], st["block_table"], st["cu_q"], st["kv_lens"],
                                               max_q=st["max_q"], window=case["window"], sinks=st["sinks"],
                                               workspace=st["workspace"])
    if case["op"] == "select":
        return ql.qlinear_select_experts(st["logits"], case["k"], sigmoid=case["sigmoid"], bias=st["bias"],
                                         n_groups=case["n_groups"], top_groups=case["top_groups"],
                                         group_top=case["group_top"], renormalize=case["renormalize"],
                                         scale=case["scale"], n_rows=st["n_rows"])
    return ql.qlinear_combine_experts(st["y"], st["weights"], ids=st["ids"], e=case["e"], residual=st["residual"])


# ---------------------------------------------------------------- work and the definition in 64 bits


def work(case):
    if case["op"] == "extend":
        n = case["n_seqs"]
        return dict(bytes=16 * case["rows"] + 16 * n, flops=4 * case["rows"] + 20 * n)
    size = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    if case["op"] == "select":
        t, e, k = case["tokens"], case["e"], case["k"]
        return dict(bytes=size * t * e + 12 * t * k + (4 * e if case["bias"] else 0), flops=t * e * 20)
    if case["op"] == "combine":
        t, k, n = case["tokens"], case["k"], case["n"]
        return dict(bytes=size * t * n * (k + 1 + bool(case["residual"])) + 12 * t * k, flops=2 * t * k * n)
    hq, hk, d = case["hq"], case["hk"], case["d"]
    row = d // 2 + 4 * (d // case["group"])  # a cached row of k or v
    if case["op"] == "attention":
        pairs = read = toks = 0
        w = case["window"]
        for nq, nkv in _lens(case):
            toks += nq
            first = nkv - nq  # the first query's position
            read += min(nkv, nq - 1 + w) if w else nkv
            a, b = first + 1, nkv  # keys that the first and the last query see
            if w and b > w:
                c = max(a, w)
                pairs += (b - c + 1) * w + ((a + c - 1) * (c - a) // 2)
            else:
                pairs += (a + b) * nq // 2
        return dict(bytes=read * hk * row * 2 + 2 * toks * hq * d * 2, flops=4 * pairs * hq * d)
    t, n = case["tokens"], case["tokens"] - case["padding"]
    b = 2 * t * hq * d * 2 + t * case["rot"] * 4 + t * 16 + 2 * d * 2
    b += 2 * n * hk * (d * 2 + row)  # appended
    b += 2 * hk * (n * row + t * d * 2)  # read back
    return dict(bytes=b, flops=t * (hq + hk) * (4 * d + 3 * case["rot"]) + 2 * n * hk * d * 8)


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


def _exact_stored(rows, group):
    """The values that 16-bit rows [n, hk, d] keep in 4 bits, group by group."""
    out = torch.zeros(rows.shape, dtype=torch.float64, device=DEV)
    for a in range(0, rows.shape[-1], group):
        x = rows[..., a:a + group].double()
        lo = x.min(dim=-1, keepdim=True).values
        scale = ((x.max(dim=-1, keepdim=True).values - lo).float() / 15.0).half().double()
        bias = lo.half().double()
        level = ((x - bias) / scale).round().clamp(0, 15)
        out[..., a:a + group] = torch.where(scale == 0, bias, level * scale + bias)
    return out


def _exact_values(words, params, n, d):
    """Rows [n, d/8] of codes and [n, groups, 2] of parameters, one code place at a time."""
    out = torch.empty((n, d), dtype=torch.float64, device=DEV)
    per = d // params.shape[1]
    for i in range(8):
        code = torch.bitwise_and(torch.bitwise_right_shift(words, 4 * i), 15).double()
        grp = torch.arange(i, d, 8, device=DEV) // per
        out[:, i::8] = code * params[:, grp, 0].double() + params[:, grp, 1].double()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "extend":
        return _exact_extend(case, st)
    if case["op"] == "select":
        return _exact_select(case, st)
    if case["op"] == "combine":
        out = torch.zeros((case["tokens"], case["n"]), dtype=torch.float64, device=DEV)
        if st["residual"] is not None:
            out += st["residual"]
        for j in range(case["k"]):
            i = st["ids"][:, j]
            w = torch.where((i >= 0) & (i < case["e"]), st["weights"][:, j].double(), 0.0)
            out += w[:, None] * st["y"][j::case["k"]].double()
        return out
    if case["op"] == "append":
        args = (st["cos_sin"], st["positions"], case["rot"], case["interleaved"])
        q = _exact_heads(st["q"], st["q_weight"], *args)
        k = _exact_heads(st["k"], st["k_weight"], *args).to(st["k"].dtype)
        keep = (st["slots"] >= 0)[:, None, None]
        return q, *(torch.where(keep, _exact_stored(x, case["group"]), 0.0) for x in (k, st["v"]))
    rep, page, w, d = case["hq"] // case["hk"], case["page"], case["window"], case["d"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for s in range(case["n_seqs"]):
        q0, q1 = int(st["cu_q"][s]), int(st["cu_q"][s + 1])
        n = int(st["kv_lens"][s])
        pages = st["block_table"][s, :(n + page - 1) // page].long()
        for h in range(case["hk"]):
            kc, kp, vc, vp = (x[pages, :, h].flatten(0, 1)[:n] for x in st["cache"])
            k, v = _exact_values(kc, kp, n, d), _exact_values(vc, vp, n, d)
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


def _exact_select(case, st):
    """Expert by expert chosen: the best of what is left."""
    t, e, m = case["tokens"], case["e"], case["e"] // case["n_groups"]
    x = st["logits"].double()
    p = torch.sigmoid(x) if case["sigmoid"] else torch.softmax(x, dim=1)
    c = p.clone()
    if st["bias"] is not None:
        c += st["bias"]
    if case["n_groups"] > 1:
        best = []
        for g in range(case["n_groups"]):
            part = c[:, g * m:(g + 1) * m]
            top = part.max(dim=1).values
            if case["group_top"] == 2 and m > 1:
                second = part.scatter(1, part.argmax(dim=1, keepdim=True), -math.inf).max(dim=1).values
                top = top + second
            best.append(top)
        best = torch.stack(best, dim=1)
        for g in range(case["n_groups"]):
            ahead = (best > best[:, g:g + 1]).sum(dim=1) + (best[:, :g] == best[:, g:g + 1]).sum(dim=1)
            c[:, g * m:(g + 1) * m][ahead >= case["top_groups"]] = -math.inf
    ids, w = [], []
    index = torch.arange(e, device=DEV)
    for _ in range(case["k"]):
        top = c.max(dim=1, keepdim=True).values
        i = torch.where(c == top, index, e).min(dim=1, keepdim=True).values
        ids.append(i)
        w.append(p.gather(1, i))
        c.scatter_(1, i, -math.inf)
    ids, w = torch.cat(ids, dim=1), torch.cat(w, dim=1)
    if case["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = w * case["scale"]
    if case["padding"]:
        ids[t - case["padding"]:] = -1
        w[t - case["padding"]:] = 0
    return ids, w


def _exact_extend(case, st):
    """On the host, one sequence at a time, a list of free pages as a list."""
    page, rows = case["page"], case["rows"]
    counts, lens, table = st["counts"].tolist(), st["lens"].tolist(), st["block_table"].tolist()
    store = st["free_pages"].tolist()
    top = int(st["free_count"])
    for s, c in enumerate(counts):
        if c < 0:
            for j in range(-(-lens[s] // page)):
                store[top] = table[s][j]
                top += 1
            lens[s] = 0
    cu, pos, slots, taken = [0], [], [], 0
    for s, c in enumerate(counts):
        for p in range(lens[s], lens[s] + max(c, 0)):
            if p % page == 0:
                top -= 1
                taken += 1
                table[s][p // page] = store[top]
            pos.append(p)
            slots.append(table[s][p // page] * page + p % page)
        lens[s] += max(c, 0)
        cu.append(len(pos))
    info = [len(pos), taken, 0, top]
    fill = rows - len(pos)
    i32 = dict(dtype=torch.int32, device=DEV)
    return (torch.tensor(cu, **i32), torch.tensor(pos + [0] * fill, device=DEV),
            torch.tensor(slots + [-1] * fill, device=DEV), torch.tensor(lens, **i32), torch.tensor(table, **i32),
            torch.tensor(store, **i32), torch.tensor([top], **i32), torch.tensor(info, **i32))
