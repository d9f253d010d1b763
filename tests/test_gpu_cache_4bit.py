"""Append to a cache in 4 bits and the reading back of its rows, against the 64-bit oracle: codes, scales and
biases bit for bit (a row of k is worked out in 64 bits on both sides before its one rounding), q_out as
qlinear_kv_append gives it."""
import numpy as np
import pytest
import torch

import weight_only_quantized_affine_amd as q
from gpu_helpers import dev_to_bits
from oracle import decoder_oracle as D
from oracle import qlinear_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
NAME = {BF: "bf16", HF: "f16"}


def f64(t):
    return t.double().cpu().numpy()


def table(max_pos, rot, seed=0):
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)[None]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float().to(DEV)


def new_cache(n_pages, page, hk, d, group, layout, seed=0):
    """A cache of random bits: head-major pages, token-major ones, or rows that are parts of a larger array."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, dtype=torch.int64).int().to(DEV)  # noqa: E731
    out = []
    for _ in range(2):
        w, r = d // 8, d // group
        if layout == "heads":
            pair = [rnd(n_pages, hk, page, w).transpose(1, 2), rnd(n_pages, hk, page, r).transpose(1, 2)]
        elif layout == "tokens":
            pair = [rnd(n_pages, page, hk, w), rnd(n_pages, page, hk, r)]
        else:
            pair = [rnd(n_pages + 1, page, hk + 1, w + 8)[1:, :, 1:, 4:w + 4], rnd(n_pages + 2, page, hk + 1, r + 3)[:-2, :, :-1, 1:r + 1]]
        out += [pair[0], pair[1][..., None].view(torch.float16)]
    return tuple(out)


def host(cache):
    return [dev_to_bits(x).view(np.float16) if x.dtype == HF else x.cpu().contiguous().numpy().view(np.uint32) for x in cache]


def same(a, b):
    a, b = (x.view(np.uint16) if x.dtype == np.float16 else x for x in (a, b))
    return np.array_equal(a, b)


def check(x, cache, before, slots, rows_k, rows_v, group):
    page = cache[0].shape[1]
    want = [w.copy() for w in before]
    for rows, at in ((rows_k, 0), (rows_v, 2)):
        codes, groups = D.quantize_rows(rows, group)
        for i, s in enumerate(slots):
            if 0 <= s < cache[0].shape[0] * page:
                want[at][s // page, s % page] = codes[i]
                want[at + 1][s // page, s % page] = groups[i]
    got = host(cache)
    for name, g, w in zip(("k codes", "k groups", "v codes", "v groups"), got, want):
        if g.dtype == np.float16:  # a NaN bias is a NaN, whatever its bits
            nan = np.isnan(g) & np.isnan(w)
            g, w = np.where(nan, np.float16(0), g), np.where(nan, np.float16(0), w)
        assert same(g, w), (x, name)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hk,d,group,rot,inter,page,layout", [
    (4, 2, 128, 64, 128, False, 16, "heads"), (0, 3, 64, 32, 32, True, 7, "tokens"), (6, 1, 128, 32, 64, False, 1, "parts"),
    (3, 3, 256, 128, 256, False, 24, "parts"), (2, 2, 128, 128, 128, True, 64, "tokens"), (5, 5, 64, 64, 0, False, 16, "heads"),
    (1, 1, 512, 64, 128, False, 5, "heads"), (2, 1, 96, 32, 96, False, 16, "tokens"), (1, 2, 32, 32, 16, True, 3, "parts")])
@pytest.mark.parametrize("t", [1, 37])
def test_append(dtype, hq, hk, d, group, rot, inter, page, layout, t):
    g = torch.Generator().manual_seed(t + d)
    n_pages = 40 // page + 3
    cache = new_cache(n_pages, page, hk, d, group, layout)
    before = host(cache)
    qkv = torch.randn(t, hq + 2 * hk, d, generator=g).to(dtype).to(DEV)
    x, k, v = qkv.split([hq, hk, hk], dim=1)
    slots = torch.randperm(n_pages * page, generator=g)[:t]
    slots[t // 3::7] = torch.tensor([-1, n_pages * page, -2 ** 62, 2 ** 62])[torch.arange(len(slots[t // 3::7])) % 4]
    pos = torch.randint(0, 64, (t,), generator=g)
    if t > 5 and rot:
        pos[3], pos[4] = -1, 64  # zero rows
    w = (1 + 0.3 * torch.randn(2, d, generator=g)).to(DEV)
    cs = table(64, rot) if rot else None
    kw = dict(q_weight=w[0], k_weight=w[1], positions=pos.to(DEV) if rot else None, cos_sin=cs, interleaved=inter)
    out = q.qlinear_kv_append_4bit(k, v, cache, slots.to(DEV), q=x if hq else None, **kw)
    rows = D.stored_rows(f64(k), f64(w[1]), float(np.float32(1e-6)), pos.numpy(), f64(cs) if rot else None, inter, NAME[dtype])
    check((t, d), cache, before, slots.tolist(), rows, f64(v).astype(np.float32), group)
    if hq:
        plain = torch.empty(n_pages, page, hk, d, dtype=dtype, device=DEV)
        want = q.qlinear_kv_append(k, v, plain, plain.clone(), slots.to(DEV), q=x, **kw)
        assert torch.equal(out, want)
    # and what is read back
    kb, vb = q.qlinear_kv_read_4bit(cache, slots.to(DEV), dtype=dtype)
    now = host(cache)
    for got, at in ((kb, 0), (vb, 2)):
        vals = np.zeros((t, hk, d))
        for i, s in enumerate(slots.tolist()):
            if 0 <= s < n_pages * page:
                vals[i] = D.row_values(now[at][s // page, s % page], now[at + 1][s // page, s % page])
        assert np.array_equal(dev_to_bits(got), O.to_bits(NAME[dtype], vals.astype(np.float32)))


@pytest.mark.parametrize("t", [300, 700, 2100])
def test_every_row_count_of_a_lane(t):
    """Launches whose lanes hold one, two and four rows, without norm or rotation and with both."""
    hq, hk, d, page = 8, 8, 128, 16
    g = torch.Generator(device=DEV).manual_seed(t)
    qkv = torch.randn(t, hq + 2 * hk, d, generator=g, device=DEV).to(BF)
    x, k, v = qkv.split([hq, hk, hk], dim=1)
    slots = torch.randperm(t + 20, generator=g, device=DEV)[:t]
    w = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(BF)
    kw = dict(q=x, q_weight=w, k_weight=w, positions=torch.arange(t, device=DEV), cos_sin=table(t, d))
    for kw in (kw, {}):
        cache = new_cache(-(-(t + 20) // page), page, hk, d, 64, "heads")
        few = tuple(c.clone(memory_format=torch.preserve_format) for c in cache)
        q.qlinear_kv_append_4bit(k, v, cache, slots, **kw)
        for a in range(0, t, 100):  # calls whose lanes hold one row
            b = min(a + 100, t)
            part = {n: z[a:b] if n in ("q", "positions") else z for n, z in kw.items()}
            q.qlinear_kv_append_4bit(k[a:b], v[a:b], few, slots[a:b], **part)
        assert all(same(a, b) for a, b in zip(host(cache), host(few)))


def test_magnitudes():
    """Groups of one value, of zeros of both signs, of the largest magnitudes that are held, past those, of
    infinities and of NaN; tiny values; and fp16's borders."""
    t, d = 12, 64
    for dtype in (BF, HF):
        v = torch.randn(t, 1, d, generator=torch.Generator().manual_seed(3))
        v[0] = 3.0
        v[1, 0, ::2], v[1, 0, 1::2] = 0.0, -0.0
        v[2, 0, 0], v[2, 0, 40] = 32768, -32768
        v[3, 0, 0], v[3, 0, 40] = 33280, -33280
        v[4, 0, 5], v[5, 0, 6], v[6, 0, 7] = float("inf"), -float("inf"), float("nan")
        v[7] *= 1e-5
        v[8] *= 1e-7
        v[9] = 1000 + torch.arange(d) % 3
        v[10, 0, 32:] = torch.tensor([-1.0, 1.0]).repeat(16)
        v[11] *= 2.0 ** 11
        v = v.to(dtype).to(DEV)
        cache = new_cache(1, 16, 1, d, 32, "heads")
        before = host(cache)
        slots = torch.arange(t, device=DEV)
        q.qlinear_kv_append_4bit(v, v, cache, slots)
        rows = f64(v).astype(np.float32)
        check("magnitudes", cache, before, range(t), rows, rows, 32)
        kb, vb = q.qlinear_kv_read_4bit(cache, slots, dtype=dtype)
        odd = torch.isnan(vb).view(t, 2, 32).all(dim=2)
        assert torch.equal(torch.isnan(vb).view(t, 2, 32).any(dim=2), odd)
        want = torch.zeros(t, 2, dtype=torch.bool, device=DEV)
        want[3, 0] = want[3, 1] = want[4, 0] = want[5, 0] = want[6, 0] = True
        assert torch.equal(odd, want)
        assert (vb[0] == 3).all() and (vb[1] == 0).all()


def test_ties_go_to_even():
    """Values half way between two levels, from both sides of zero."""
    d = 64
    v = torch.zeros(4, 1, d)
    for r, (lo, step) in enumerate(((0.0, 1.0), (-7.5, 1.0), (-16.0, 2.0), (3.0, 0.5))):
        v[r, 0] = lo + step * (torch.arange(d) % 31) / 2
    v = v.to(HF).to(DEV)
    cache = new_cache(1, 4, 1, d, 64, "tokens")
    before = host(cache)
    q.qlinear_kv_append_4bit(v, v, cache, torch.arange(4, device=DEV))
    check("ties", cache, before, range(4), f64(v).astype(np.float32), f64(v).astype(np.float32), 64)


def test_another_stream_repeated_slots_and_a_graph():
    t, hk, d = 8, 2, 128
    cache = new_cache(3, 16, hk, d, 64, "heads")
    k, v = (torch.randn(t, hk, d, device=DEV).to(BF) for _ in range(2))
    slots = torch.randperm(48, device=DEV)[:t]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.qlinear_kv_append_4bit(k, v, cache, slots)
        got = q.qlinear_kv_read_4bit(cache, slots[torch.tensor([0, 0, 3, 0], device=DEV)], dtype=BF)
    side.synchronize()
    one = q.qlinear_kv_read_4bit(cache, slots, dtype=BF)
    for g, o in zip(got, one):
        assert torch.equal(g, o[[0, 0, 3, 0]])
    graph, ko, vo = torch.cuda.CUDAGraph(), torch.empty_like(k), torch.empty_like(v)
    with torch.cuda.graph(graph):
        q.qlinear_kv_append_4bit(k, v, cache, slots)
        q.qlinear_kv_read_4bit(cache, slots, k_out=ko, v_out=vo)
    for i in range(3):
        k.normal_()
        v.normal_()
        slots.copy_(torch.randperm(48, device=DEV)[:t])
        graph.replay()
        torch.cuda.synchronize()
        got = ko.clone(), vo.clone()
        other = new_cache(3, 16, hk, d, 64, "tokens")
        q.qlinear_kv_append_4bit(k, v, other, slots)
        for g, o in zip(got, q.qlinear_kv_read_4bit(other, slots, dtype=BF)):
            assert torch.equal(g, o)


def test_offsets_past_32_bits():
    page, hk, d, n_pages = 128, 8, 128, 70000  # 4.6 GB of codes
    codes = [torch.zeros(n_pages, hk, page, d // 8, dtype=torch.int32, device=DEV).transpose(1, 2) for _ in range(2)]
    groups = [torch.zeros(n_pages, hk, page, d // 32, 2, dtype=HF, device=DEV).transpose(1, 2) for _ in range(2)]
    cache = (codes[0], groups[0], codes[1], groups[1])
    small = new_cache(1, 4, hk, d, 32, "heads")
    k, v = (torch.randn(4, hk, d, device=DEV).to(BF) for _ in range(2))
    far = torch.tensor([n_pages * page - 1, n_pages * page - 130, (1 << 22) * 2 + 5, 7], device=DEV)
    q.qlinear_kv_append_4bit(k, v, cache, far)
    q.qlinear_kv_append_4bit(k, v, small, torch.arange(4, device=DEV))
    for a, b in zip(q.qlinear_kv_read_4bit(cache, far, dtype=BF), q.qlinear_kv_read_4bit(small, torch.arange(4, device=DEV), dtype=BF)):
        assert torch.equal(a, b) and a.abs().sum() > 0


def test_nothing_to_do():
    cache = new_cache(2, 4, 2, 64, 32, "heads")
    before = host(cache)
    e = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    q.qlinear_kv_append_4bit(e, e, cache, none)
    assert q.qlinear_kv_read_4bit(cache, none)[0].shape == (0, 2, 64)
    assert all(same(a, b) for a, b in zip(host(cache), before))
    empty = tuple(c[:0] for c in cache)
    x = torch.ones(3, 2, 64, dtype=BF, device=DEV)
    s = torch.arange(3, device=DEV)
    q.qlinear_kv_append_4bit(x, x, empty, s)
    assert (q.qlinear_kv_read_4bit(empty, s)[1] == 0).all()


@pytest.mark.parametrize("magnitude,eps", [(1e25, 1e-6), (3e37, 0.0), (1e-25, 0.0), (1e-25, 1e-6), (1e-38, 0.0), (2.0 ** -126, 1e-30)])
@pytest.mark.parametrize("rot", [0, 128])
def test_norm_of_rows_whose_squares_leave_fp32(magnitude, eps, rot):
    """bf16 rows of k with squares past fp32's range on either side: in 64 bits they are ordinary rows."""
    t, hk, d, group = 9, 2, 128, 64
    g = torch.Generator().manual_seed(17)
    k = (torch.randn(t, hk, d, generator=g).double() * magnitude).to(BF)
    k[1, :, 1:] = 0  # one value alone
    k[2, :, ::2] = k[2, :, ::2] * 2.0 ** -8
    k, v = k.to(DEV), torch.randn(t, hk, d, generator=g).to(BF).to(DEV)
    w, cs = (1 + 0.3 * torch.randn(d, generator=g)).to(DEV), table(16, rot) if rot else None
    slots, pos = torch.arange(t, device=DEV), torch.arange(t, device=DEV) if rot else None
    cache = new_cache(1, 16, hk, d, group, "heads")
    before = host(cache)
    q.qlinear_kv_append_4bit(k, v, cache, slots, k_weight=w, eps=eps, positions=pos, cos_sin=cs)
    rows = D.stored_rows(f64(k), f64(w), float(np.float32(eps)), np.arange(t), f64(cs) if rot else None, False, "bf16")
    assert np.isfinite(rows).all() and np.abs(rows).max() < 32
    check((magnitude, eps), cache, before, range(t), rows, f64(v).astype(np.float32), group)


def test_more_heads_than_tokens_have_room_for():
    """One token of very many heads: 2^31 chunks of 8 values are the limit, not heads."""
    t, hk, d = 2, 70000, 512
    g = torch.Generator(device=DEV).manual_seed(2)
    k = torch.randn(t, hk, d, generator=g, device=DEV).to(BF)
    cache = q.qlinear_paged_cache_4bit(1, 3, hk, d, 128)
    few = q.qlinear_paged_cache_4bit(1, 3, 7, d, 128)
    q.qlinear_kv_append_4bit(k, k, cache, torch.tensor([2, 0], device=DEV))
    q.qlinear_kv_append_4bit(k[:, -7:], k[:, -7:], few, torch.tensor([2, 0], device=DEV))
    slots = torch.tensor([0, 1, 2], device=DEV)
    for a, b in zip(q.qlinear_kv_read_4bit(cache, slots), q.qlinear_kv_read_4bit(few, slots)):
        assert torch.equal(a[:, -7:], b) and b[0].abs().sum() > 0
