"""How exact the few-row 4-bit attention is, against the definition in 64 bits: its root mean square error over many
outputs is that of its stated roundings, so that a sum which loses more shows, however far below the largest
error that the roundings allow.

With weights w_j (they sum to one), v_j = s_j (c_j - 8) + m_j, m_j = b_j + 8 s_j, f = 2^-11 and h half a step of out's
type relative to the value, an output o errs by
  w_j s_j    rounds once to fp16 in its product with c_j - 8:                f w_j |s_j (c_j - 8)|
  w_j        rounds once to fp16 in its product with m_j and in the sum of the weights:       f w_j |m_j - o|
  o          rounds once:                                                    h |o|
each at most so, independent of the others, and spread evenly over their range: a third of the squares on average.
Sums: a product of the matrix cores takes a subnormal half as if its exponent were that of the smallest normal one, 2^-14,
and drops what lies below 2^-24 of the largest term so taken.  Codes are subnormal, c 2^-24, so that a product over 32
keys loses at most 2^-24 2^10 of its largest w_j s_j: the sum of these is counted whole, and the same, of
|q_i| s_j, for each of a row's d / 32 products of a score.
"""
import numpy as np
import pytest
import torch

import weight_only_quantized_affine_amd as q
from test_gpu_paged_attention_4bit import LENS, Problem

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
F = 2.0 ** -11
LOST = 2.0 ** -14


def parts(words, params):
    """Codes, scales and biases of rows [.., d / 8], each [.., d] in 64 bits."""
    c = ((words[..., None] >> (4 * torch.arange(8, device=DEV))) & 15).flatten(-2).double()
    s, b = (params[..., i].double().repeat_interleave(c.shape[-1] // params.shape[-2], -1) for i in (0, 1))
    return c, s, b


def row(p, cache, pages, n, scale):
    """One kv head's n positions and its query rows p [rows, d] -> outputs and their mean square error."""
    kc, ks, kb = (x.flatten(0, 1)[:n] for x in parts(cache[0][pages], cache[1][pages]))
    c, s, b = (x.flatten(0, 1)[:n] for x in parts(cache[2][pages], cache[3][pages]))
    x = p @ (kc * ks + kb).T * scale
    w = x.softmax(-1)
    o = w @ (c * s + b)
    e = scale * LOST * p.abs().amax(-1, keepdim=True) * ks.amax() * (p.shape[1] // 32) + 64 * 2.0 ** -24 * x.abs().amax(-1, keepdim=True)
    m = b + 8 * s
    w2 = w * w
    spread = lambda y: w2 @ (y * y) - 2 * (w2 @ y) * o + w2.sum(-1, keepdim=True) * o * o  # noqa: E731  sum w^2 (y - o)^2
    var = F * F / 3 * (w2 @ (s * (c - 8)) ** 2 + spread(m)) + e * e * spread(c * s + b)
    pad = torch.nn.functional.pad(w, (0, -n % 32)).unflatten(-1, (-1, 32)).amax(-1)  # 32 keys' largest weight
    return o, var, LOST * s.amax() * pad.sum(-1, keepdim=True).expand_as(o)


@pytest.mark.parametrize("d,group,tokens,q_scale", [(128, 64, 1, 1.0), (128, 64, 1, 4.0), (64, 32, 1, 1.0), (128, 128, 1, 1.0), (64, 64, 1, 1.0),
                                                    (256, 128, 1, 1.0), (256, 32, 1, 1.0), (128, 32, 1, 1.0), (128, 64, 5, 1.0)])
@pytest.mark.parametrize("n", [500, 16000])
def test_errors_are_those_of_the_roundings(d, group, tokens, q_scale, n):
    seqs, hk, g, page, scale = 4, 4, 4, 16, d ** -0.5
    gen = torch.Generator(device=DEV).manual_seed(n + d)
    per = -(-n // page)
    cache = q.qlinear_paged_cache_4bit(per * seqs, page, hk, d, group)
    k, v = (torch.randn(per * seqs * page, hk, d, generator=gen, device=DEV).to(HF) for _ in range(2))
    q.qlinear_kv_append_4bit(k, v, cache, torch.arange(per * seqs * page, device=DEV))
    table = torch.arange(per * seqs, device=DEV, dtype=torch.int32).view(seqs, per)
    cu = torch.arange(seqs + 1, device=DEV, dtype=torch.int32) * tokens
    x = (torch.randn(seqs * tokens, hk * g, d, generator=gen, device=DEV) * q_scale).to(HF)
    out = q.qlinear_paged_attention_4bit(x, cache, table, cu, torch.full((seqs,), n, device=DEV, dtype=torch.int32), max_q=tokens)
    err = stat = lost = 0.0
    for s in range(seqs):
        for i in range(tokens):
            for h in range(hk):
                rows = x[s * tokens + i, h * g:(h + 1) * g].double()
                o, var, low = row(rows, [y[:, :, h] for y in cache], table[s].long(), n - tokens + i + 1, scale)
                got = out[s * tokens + i, h * g:(h + 1) * g].double()
                err += float((got - o).pow(2).sum())
                stat += float((var + (torch.finfo(HF).eps / 2) ** 2 / 3 * o * o).sum())
                lost += float(low.pow(2).sum())
    # thousands of outputs: their mean square is within a tenth of its expectation
    assert np.sqrt(err) <= 1.1 * np.sqrt(stat) + np.sqrt(lost), (np.sqrt(err), np.sqrt(stat), np.sqrt(lost))


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("tokens,n", [(1, 700), (4, 300), (40, 300)])
@pytest.mark.parametrize("large", [64.0, 4096.0])
def test_biases_meet_the_whole_sum_of_a_row(d, group, tokens, n, large):
    """Queries whose values nearly cancel in each group, over keys that are their biases alone (scale 0): a score is a
    small sum of large values times a bias, every term and partial sum of it exact in fp32.  What is left is the scores' own
    scaling and exponential, |score| (2^-22 + 2^-24) and 2^-22, and the roundings of weights, values and output."""
    hk, g, page, scale = 2, 2, 16, 0.25
    gen = torch.Generator(device=DEV).manual_seed(d + group + n)
    per = -(-n // page)
    cache = q.qlinear_paged_cache_4bit(per, page, hk, d, group)
    k, v = torch.zeros(per * page, hk, d, device=DEV), torch.randn(per * page, hk, d, generator=gen, device=DEV)
    bias = torch.randint(-48, 49, (per * page, hk, d // group, 1), generator=gen, device=DEV) / 8
    k = (k.unflatten(-1, (-1, group)) + bias).flatten(-2).to(BF)  # exact
    q.qlinear_kv_append_4bit(k, v.to(BF), cache, torch.arange(per * page, device=DEV))
    assert torch.equal(cache[1][..., 0], torch.zeros_like(cache[1][..., 0]))
    sign = torch.tensor([1.0, -1.0], device=DEV).repeat(group // 2)
    x = torch.zeros(tokens, hk * g, d // group, group, device=DEV) + large * sign
    # one pair of a group holds other values: what the group sums to
    x[..., 6] = torch.randint(64, 255, x.shape[:3], generator=gen, device=DEV) / 128
    x[..., 11] = torch.randint(-255, -64, x.shape[:3], generator=gen, device=DEV) / 256
    x = x.flatten(-2).to(BF)
    table = torch.arange(per, device=DEV, dtype=torch.int32)[None]
    cu, lens = (torch.tensor(y, device=DEV, dtype=torch.int32) for y in ([0, tokens], [n]))
    out = q.qlinear_paged_attention_4bit(x, cache, table, cu, lens, max_q=tokens, scale=scale)
    for i in range(tokens):
        m = n - tokens + i + 1
        for h in range(hk):
            kc, ks, kb = (y.flatten(0, 1)[:m] for y in parts(cache[0][:, :, h], cache[1][:, :, h]))
            c, s, b = (y.flatten(0, 1)[:m] for y in parts(cache[2][:, :, h], cache[3][:, :, h]))
            sc = x[i, h * g:(h + 1) * g].double() @ kb.T * scale
            w = sc.softmax(-1)
            o, big = w @ (c * s + b), w @ (c * s + b).abs()
            e = sc.abs().amax(-1, keepdim=True) * (2.0 ** -22 + 2.0 ** -24) * 2 + 2.0 ** -22
            # 16-bit roundings: a weight and a value (or w s and w), the sum's weights; a code's sum, a third as much
            tol = 3 * F * (big + 8 * (w @ s)) * (1 + F) + (F + torch.finfo(BF).eps / 2) * o.abs() + 2 * e * big + 2 * (m + 8) * 2.0 ** -24 * big + 2.0 ** -24
            bad = (out[i, h * g:(h + 1) * g].double() - o).abs() > tol
            assert not bad.any(), (i, h, float((out[i, h * g:(h + 1) * g].double() - o).abs().max()), float(tol.max()))


def few_rows_tolerance(p, x, n, first, last, cache, scale, sink):
    """Query rows x [rows, d] that see the positions [first, last) of `cache` (codes and parameters of one kv head, n rows) ->
    outputs and what each may be off by: every rounding above at its largest, and
      a weight's relative error e (numerator and sum): what a product over codes drops, d / 32 times LOST max|q| s; the
                 fp32 sums, (d + 8) u of g = sum |q| (15 s + |b|) (u = 2^-24), and the two halves of the sums of q, 4 u
                 of it; its scaling and difference, 8 u |score|; the exponential, 2 u
      2 (n + 8) u sum w (24 s + |b|)    the fp32 sums over the keys and the quotient
      LOST sum w s                      what the products over codes drop
      2^-25 |v| a key                   weights below 2^-14, where the largest weighs 2^-8 at least."""
    u = 2.0 ** -24
    kc, ks, kb = (y[first:last] for y in parts(cache[0], cache[1]))
    c, s, b = (y[first:last] for y in parts(cache[2], cache[3]))
    sc = x @ (kc * ks + kb).T * scale
    top = sc.amax(-1, keepdim=True)
    ex = (sc - top).exp()
    z = ex.sum(-1, keepdim=True) + (0 if sink is None else (sink[:, None] - top).exp())
    w = ex / z
    o = w @ (c * s + b)
    g = (x.abs() @ (15 * ks + kb.abs()).T * scale).amax(-1, keepdim=True)
    e = scale * LOST * x.abs().amax(-1, keepdim=True) * ks.amax() * (x.shape[1] / 32) + (x.shape[1] + 12) * u * g + 8 * u * sc.abs().amax(-1, keepdim=True) + 2 * u
    count = last - first
    tol = F * (1 + F) * (w @ (s * (c - 8)).abs() + w @ (b + 8 * s).abs()) + (F + torch.finfo(p.dtype).eps / 2) * o.abs()
    tol = tol + 2 * e * (w @ (c * s + b).abs()) + 2 * (count + 8) * u * (w @ (24 * s + b.abs())) + LOST * (w @ s)
    tol = tol + 2.0 ** -25 * count * (c * s + b).abs().amax() / (ex.sum(-1, keepdim=True) * 2.0 ** -8).clamp(min=1) + 2.0 ** -25
    return o, tol * (1 + 2.0 ** -6)


def check_few(p, got, scale=None, window=0, sinks=None):
    hk, page, d = p.cache[0].shape[2], p.cache[0].shape[1], p.q.shape[2]
    g = p.q.shape[1] // hk
    for s, (n, kv) in enumerate(p.lens):
        pages = p.table[s, :-(-kv // page)].long().to(DEV)
        for h in range(hk):
            cache = [y[pages, :, h].flatten(0, 1)[:kv] for y in p.cache]
            for i in range(n):
                at, last = int(p.cu[s]) + i, kv - n + i + 1
                first = max(0, last - window) if window else 0
                out = got[at, h * g:(h + 1) * g].double()
                if last <= first:
                    assert (out == 0).all()
                    continue
                o, tol = few_rows_tolerance(p, p.q[at, h * g:(h + 1) * g].double(), n, first, last, cache, d ** -0.5 if scale is None else scale,
                                            None if sinks is None else sinks[h * g:(h + 1) * g].double())
                bad = ~((out - o).abs() <= tol)
                assert not bad.any(), (s, i, h, float((out - o).abs().max()), float(tol.max()), torch.argwhere(bad)[:4].tolist())


@pytest.mark.parametrize("lens", ["tokens", "one", "drafts", "empty"])
@pytest.mark.parametrize("dtype,hq,hk,d,group,page,heads_first", [
    (BF, 8, 4, 128, 64, 16, True), (HF, 6, 2, 64, 32, 7, False), (BF, 4, 1, 256, 128, 64, True), (HF, 3, 3, 128, 128, 1, False),
    (BF, 8, 2, 64, 64, 200, False), (HF, 8, 2, 256, 32, 48, False), (BF, 4, 4, 128, 32, 24, True), (HF, 4, 2, 256, 64, 16, True),
    (HF, 16, 2, 128, 64, 16, True), (BF, 16, 2, 64, 32, 48, True), (HF, 14, 2, 128, 32, 5, False)])
def test_every_output_is_within_the_few_row_kernels_own_roundings(lens, dtype, hq, hk, d, group, page, heads_first):
    """Four tokens of at most eight heads a kv head (four at 256 values) are the few-row kernel's: nothing is allowed for
    values or keys that round."""
    p = Problem(LENS[lens], hq, hk, d, group, page, dtype, heads_first=heads_first, seed=31)
    check_few(p, p.run())
    check_few(p, p.run(window=60, sinks=p.sinks, scale=0.15), 0.15, 60, p.sinks)


@pytest.mark.parametrize("magnitude", [0.02, 1.0, 12.0])
def test_keys_with_large_biases(magnitude):
    """Channels of k far from zero, as keys have them: a group's bias is many times its scale."""
    p = Problem([(1, 900), (4, 350), (2, 64), (1, 1)], 8, 2, 128, 64, 16, BF, seed=32)
    p.cache[1][..., 1] += torch.randn(p.cache[1].shape[2:4], device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(HF) * 20
    p.q *= magnitude
    check_few(p, p.run())
