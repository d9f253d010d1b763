"""qlinear_qk_norm_rope and qlinear_kv_append against the 64-bit oracle.

Tolerance of a normed and rotated value y = y_a c -+ y_b s: the sum of squares takes at most 8
products in a lane and 6 additions across lanes, the mean, eps, root and quotient one rounding
each (the root halves what came before), then x r w and the rotation's products and sum: fewer
than 16 roundings of 2^-24 relative to |y_a c| + |y_b s|, and half a step of the output type.
"""
import numpy as np
import pytest
import torch

import weight_only_quantized_affine_amd as q
from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def table(max_pos, rot, theta=1e6):
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * theta ** (-torch.arange(0, rot, 2).double() / rot)[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)


def close(got, want, mag):
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2  # half a subnormal step
    tol = torch.finfo(got.dtype).eps / 2 * np.abs(want) * (1 + 2.0 ** -10) + 16 * 2.0 ** -24 * mag + tiny
    bad = np.abs(f64(got) - want) > tol
    assert not bad.any(), (bad.sum(), np.abs(f64(got) - want).max(), np.argwhere(bad)[:4])


def randn(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


CASES = [
    # dtype, tokens, hq, hk, d, rot, interleaved, weights
    (BF, 1, 16, 8, 128, 128, False, BF),
    (HF, 1, 1, 1, 64, 64, True, HF),
    (BF, 7, 5, 1, 128, 64, False, torch.float32),
    (HF, 33, 3, 3, 256, 256, False, BF),
    (BF, 2, 4, 2, 8, 0, False, BF),
    (BF, 5, 4, 2, 24, 16, True, BF),
    (HF, 9, 2, 1, 72, 32, False, torch.float32),
    (BF, 6, 2, 2, 512, 512, True, HF),
    (BF, 130, 7, 1, 80, 80, False, None),
    (HF, 17, 0, 4, 128, 16, False, HF),
    (BF, 17, 4, 0, 128, 128, True, None),
    (BF, 3, 3, 2, 264, 128, False, BF),
]


@pytest.mark.parametrize("dtype,t,hq,hk,d,rot,inter,wdt", CASES)
def test_norm_rope_matches_the_oracle(dtype, t, hq, hk, d, rot, inter, wdt):
    g = torch.Generator().manual_seed(t * 1000 + d)
    scale = torch.exp(torch.randn(t, 1, 1, generator=g) * 2).to(DEV)  # rows of very different size
    x = {n: (randn(g, t, h, d, dtype=torch.float32) * scale).to(dtype) if h else None for n, h in (("q", hq), ("k", hk))}
    w = {n: None if wdt is None else randn(g, d, dtype=wdt, scale=2.0) for n in "qk"}
    max_pos = 1000
    cs = table(max_pos, rot) if rot else None
    pos = torch.randint(0, max_pos, (t,), generator=g)
    if t > 4:
        pos[1], pos[3] = -1, max_pos  # outside the table: zero rows
    qo, ko = q.qlinear_qk_norm_rope(x["q"], x["k"], q_weight=w["q"], k_weight=w["k"], eps=1e-5, positions=pos.to(DEV),
                                    cos_sin=cs, interleaved=inter)
    for n, out in (("q", qo), ("k", ko)):
        if x[n] is None:
            assert out is None
            continue
        want, mag = A.norm_rope(f64(x[n]), f64(w[n]), 1e-5, pos.numpy(), f64(cs), inter)
        close(out, want, mag)
    again = q.qlinear_qk_norm_rope(x["q"], x["k"], q_weight=w["q"], k_weight=w["k"], eps=1e-5, positions=pos.to(DEV),
                                   cos_sin=cs, interleaved=inter)
    for a, b in zip((qo, ko), again):
        assert a is None or torch.equal(a, b)


def test_norm_rope_strided_in_place_and_guarded():
    g = torch.Generator().manual_seed(5)
    t, hq, hk, d = 11, 6, 2, 128
    qkv = randn(g, t + 2, (hq + 2 * hk) * d)
    before = qkv.clone()
    x = qkv[1:-1]
    qv, kv = x[:, :hq * d].view(t, hq, d), x[:, hq * d:(hq + hk) * d].view(t, hk, d)
    w, cs, pos = randn(g, d), table(64, d), torch.arange(t, device=DEV)
    want = [A.norm_rope(f64(v), f64(w), 1e-6, pos.cpu().numpy(), f64(cs), False) for v in (qv, kv)]
    k_out = torch.full((hk, t + 2, d), 7.0, dtype=BF, device=DEV)  # head-major output inside a guard
    q.qlinear_qk_norm_rope(qv, kv, q_weight=w, k_weight=w, positions=pos, cos_sin=cs, q_out=qv,
                           k_out=k_out[:, 1:-1].transpose(0, 1))
    close(qv, *want[0])
    close(k_out[:, 1:-1].transpose(0, 1), *want[1])
    assert (k_out[:, 0] == 7).all() and (k_out[:, -1] == 7).all()
    assert torch.equal(qkv[0], before[0]) and torch.equal(qkv[-1], before[-1])
    assert torch.equal(qkv[1:-1, hq * d:], before[1:-1, hq * d:])


def test_norm_rope_empty_and_non_finite_rows():
    w = torch.ones(64, dtype=BF, device=DEV)
    e = torch.empty(0, 4, 64, dtype=BF, device=DEV)
    a, b = q.qlinear_qk_norm_rope(e, e, q_weight=w, k_weight=w)
    assert a.shape == e.shape and b.shape == e.shape
    x = torch.ones(3, 1, 64, dtype=BF, device=DEV)
    x[1, 0, 5] = float("nan")
    y, _ = q.qlinear_qk_norm_rope(x, None, q_weight=w)
    assert torch.isnan(y[1]).all() and (y[0] == 1).all() and (y[2] == 1).all()
    z, _ = q.qlinear_qk_norm_rope(torch.zeros_like(x), None, q_weight=w, eps=1e-6)
    assert (z == 0).all()


@pytest.mark.parametrize("page,heads_first,dtype,d,rot", [(16, False, BF, 128, 128), (1, True, HF, 64, 32), (37, True, BF, 256, 0),
                                                          (24, False, HF, 80, 80)])
@pytest.mark.parametrize("with_q", [True, False])
def test_append_matches_the_oracle(page, heads_first, dtype, d, rot, with_q):
    g = torch.Generator().manual_seed(page)
    t, hq, hk, n_pages = 29, 6, 3, 90 // page + 2
    x = randn(g, t, hq + 2 * hk, d, dtype=dtype)
    qx, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    shape = (n_pages + 2, hk, page, d) if heads_first else (n_pages + 2, page, hk, d)
    full = [randn(g, *shape, dtype=dtype) for _ in range(2)]
    old = [c.clone() for c in full]
    caches = [c[1:-1].transpose(1, 2) if heads_first else c[1:-1] for c in full]
    slots = torch.randperm(n_pages * page, generator=g)[:t]
    slots[3], slots[8], slots[9] = -1, n_pages * page, 1 << 40
    wq, wk = randn(g, d, dtype=dtype), randn(g, d, dtype=dtype)
    pos = torch.randint(0, 500, (t,), generator=g)
    cs = table(500, rot) if rot else None
    before = [f64(c) for c in caches]
    out = q.qlinear_kv_append(k, v, *caches, slots.to(DEV), q=qx if with_q else None, q_weight=wq, k_weight=wk,
                              positions=pos.to(DEV), cos_sin=cs)
    kw, km = A.norm_rope(f64(k), f64(wk), 1e-6, pos.numpy(), f64(cs), False)
    close(caches[0], A.kv_append(before[0], kw, slots.numpy()), A.kv_append(np.zeros_like(before[0]), km, slots.numpy()))
    assert np.array_equal(f64(caches[1]), A.kv_append(before[1], f64(v), slots.numpy()))  # bytes as they are
    for c, o in zip(full, old):  # the pages around the cache are untouched
        assert torch.equal(c[0], o[0]) and torch.equal(c[-1], o[-1])
    if with_q:
        close(out, *A.norm_rope(f64(qx), f64(wq), 1e-6, pos.numpy(), f64(cs), False))
    else:
        assert out is None


def test_append_copies_any_bits_and_zeroes_unknown_positions():
    d, hk = 64, 2
    raw = torch.arange(3 * hk * d, dtype=torch.int32).mul(331).to(torch.int16).view(3, hk, d).to(DEV)
    v = raw.view(BF)
    k = torch.ones(3, hk, d, dtype=BF, device=DEV)
    kc, vc = torch.full((2, 4, hk, d), 5.0, dtype=BF, device=DEV), torch.full((2, 4, hk, d), 5.0, dtype=BF, device=DEV)
    q.qlinear_kv_append(k, v, kc, vc, torch.tensor([0, 7, 2], device=DEV), positions=torch.tensor([0, 10, -3], device=DEV),
                        cos_sin=table(10, d))
    assert torch.equal(vc.view(8, hk, d)[[0, 7, 2]].view(torch.int16), raw)
    assert (kc.view(8, hk, d)[0] == 1).all() and (kc.view(8, hk, d)[[7, 2]] == 0).all()
    assert (kc.view(8, hk, d)[[1, 3, 4, 5, 6]] == 5).all()


def test_append_past_32_bit_offsets():
    hk, d, page, n_pages = 8, 128, 128, 9000  # 2.36 GB of each, offsets up to 2.36e9 bytes and past 2^31
    kc = torch.zeros(n_pages, page, hk, d, dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    k = torch.full((2, hk, d), 2.0, dtype=BF, device=DEV)
    q.qlinear_kv_append(k, k * 2, kc, vc, torch.tensor([n_pages * page - 1, 0], device=DEV))
    assert (kc[-1, -1] == 2).all() and (vc[-1, -1] == 4).all() and (kc[0, 0] == 2).all()
    assert int((kc != 0).sum()) == 2 * hk * d and int((vc != 0).sum()) == 2 * hk * d


def test_append_in_a_graph_and_on_another_stream():
    g = torch.Generator().manual_seed(9)
    t, hk, d = 5, 2, 128
    k, v = randn(g, t, hk, d), randn(g, t, hk, d)
    w, cs, pos = randn(g, d), table(64, d), torch.arange(t, device=DEV)
    slots = torch.arange(t, device=DEV)
    caches = [torch.zeros(2, 4, hk, d, dtype=BF, device=DEV) for _ in range(2)]
    run = lambda c: q.qlinear_kv_append(k, v, *c, slots, k_weight=w, positions=pos, cos_sin=cs)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(caches)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(caches)
    for i in range(3):
        k.copy_(randn(g, t, hk, d))
        eager = [torch.zeros_like(c) for c in caches]
        run(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(caches, eager))


@pytest.mark.parametrize("t,hq,hk,d,dtype,inter", [(900, 21, 5, 128, BF, False), (3000, 21, 5, 128, HF, True),
                                                   (3000, 13, 3, 256, BF, False), (5000, 26, 5, 64, BF, False)])
def test_large_launches_match_small_ones(t, hq, hk, d, dtype, inter):
    """Every number of rows a lane holds: bit for bit what calls of a few tokens give, which the oracle checks."""
    g = torch.Generator().manual_seed(t + d)
    page, n_pages = 16, t // 16 + 3
    x, w, cs = randn(g, t, hq + 2 * hk, d, dtype=dtype), [randn(g, d, dtype=dtype) for _ in range(2)], table(6000, d // 2)
    pos = torch.arange(t, device=DEV)
    slots = torch.randperm(n_pages * page, generator=g)[:t].to(DEV)
    caches = [[torch.zeros(n_pages, page, hk, d, dtype=dtype, device=DEV) for _ in range(2)] for _ in range(2)]
    outs = [torch.empty(t, hq, d, dtype=dtype, device=DEV) for _ in range(3)]
    k_out = torch.empty(t, hk, d, dtype=dtype, device=DEV)
    for c, out, step in ((caches[0], outs[0], t), (caches[1], outs[1], 37)):
        for i in range(0, t, step):
            j = slice(i, i + step)
            q.qlinear_kv_append(x[j, hq:hq + hk], x[j, hq + hk:], *c, slots[j], q=x[j, :hq], q_out=out[j], q_weight=w[0],
                                k_weight=w[1], positions=pos[j], cos_sin=cs, interleaved=inter)
    assert torch.equal(outs[0], outs[1])
    assert all(torch.equal(a, b) for a, b in zip(*caches))
    q.qlinear_qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], q_weight=w[0], k_weight=w[1], positions=pos, cos_sin=cs,
                           interleaved=inter, q_out=outs[2], k_out=k_out)
    assert torch.equal(outs[2], outs[1])
    assert torch.equal(caches[1][0].view(-1, hk, d)[slots], k_out)
