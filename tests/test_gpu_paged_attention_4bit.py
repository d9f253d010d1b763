"""qlinear_paged_attention_4bit against the 64-bit oracle over the values that the cache stands for.

Tolerance of an output o = sum w_j v_j with A = sum w_j |v_j| and v_j = s_j (c_j - 8) + m_j, B = sum w_j |s_j (c_j - 8)|
(u = 2^-24, f = 2^-11, half a step of fp16, h half a step of out's type, relative to the value):
  many rows: 2 f A (1 + f)  each weight rounds once to fp16 in the product and each value of v once;  f |o|  the
                 weight rounds in the sum too
  few rows:  f B  each product of a weight and a scale rounds once to fp16, and takes part with c_j - 8
  (which sequences are which is the kernels' business: the sum of both is allowed)
  h |o|          the output rounds once
  2 E A          E bounds the relative error of an unnormalised weight (numerator and sum): each value of k rounds
                 once to fp16, f sum|q k| scale; the score's fp32 sum of d products, d u sum|q k| scale, its scaling
                 and difference, 4 u (|s| + |max|); the exponential, 2 u
  2 (n + 8) u A  the fp32 sums over n keys, the rescalings and the quotient
  below 2^-14    fp16 keeps an absolute 2^-25: of each value of v (weights that sum to one), 2^-25; of each value
                 of k, 2^-25 sum|q| scale in E; of a weight, whose reference weighs at least 1,
                 2^-25 sum|v| / max(1, 2^-8 sum e^(s - max))
q enters exactly: bf16 values after a scaling by a power of two keep 2^-39 of the row's largest.
"""
import numpy as np
import pytest
import torch

import weight_only_quantized_affine_amd as q
from oracle import attention_oracle as A
from oracle import decoder_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
U, F = 2.0 ** -24, 2.0 ** -11


def f64(t):
    return t.double().cpu().numpy()


def quantize(rows, group):
    """The same rule as the append's, on the GPU (what the codes are does not matter here)."""
    v = rows.float().unflatten(-1, (-1, group))
    lo = v.amin(-1)
    s, b = ((v.amax(-1) - lo) / 15).half(), lo.half()
    c = torch.nan_to_num(((v - b.float()[..., None]) / s.float()[..., None]).round()).clamp(0, 15).long().flatten(-2).unflatten(-1, (-1, 8))
    w = (c << (4 * torch.arange(8, device=c.device))).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int(), torch.stack([s, b], dim=-1)


class Problem:
    """Sequences of (new tokens, cached tokens), shuffled pages, and slots past the lengths that stand for NaN and
    infinities."""

    def __init__(self, lens, hq, hk, d, group, page, dtype, seed=0, heads_first=True, extra=1, q_scale=2.0, odd=True):
        g = torch.Generator(device=DEV).manual_seed(seed)
        c = torch.Generator().manual_seed(seed)
        self.lens, self.dtype = lens, dtype
        need = [-(-kv // page) for _, kv in lens]
        n_pages = sum(need) + extra
        order = torch.randperm(n_pages, generator=c).int()
        self.table = torch.full((len(lens), max(max(need), 1)), -7, dtype=torch.int32)
        at, used = 0, torch.zeros(n_pages, page, dtype=torch.bool)
        for s, (_, kv) in enumerate(lens):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
            for j in range(need[s]):
                used[self.table[s, j], :min(page, kv - j * page)] = True
        used = used.to(DEV)
        self.cache = []
        for _ in range(2):
            codes, groups = quantize(torch.randn(n_pages, page, hk, d, generator=g, device=DEV), group)
            if odd:
                groups[~used] = torch.tensor([float("inf"), float("nan")], dtype=HF, device=DEV)
            if heads_first:
                codes, groups = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (codes, groups))
            self.cache += [codes, groups]
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.q = (torch.randn(int(self.cu[-1]), hq, d, generator=g, device=DEV) * q_scale).to(dtype)
        self.sinks = torch.randn(hq, generator=g, device=DEV)

    def args(self):
        return (self.q, tuple(self.cache), self.table.to(DEV), torch.from_numpy(self.cu).to(DEV),
                torch.tensor([kv for _, kv in self.lens], dtype=torch.int32, device=DEV))

    def run(self, **kw):
        kw.setdefault("max_q", max(max(n for n, _ in self.lens), 1))
        return q.qlinear_paged_attention_4bit(*self.args(), **kw)

    def oracle(self, scale=None, window=0, sinks=None):
        d = self.q.shape[2]
        kc, kg, vc, vg = (x.cpu().contiguous().numpy() for x in self.cache)
        with np.errstate(all="ignore"):
            k, v = (np.nan_to_num(D.row_values(a.view(np.uint32), b), nan=1e300, posinf=1e300, neginf=1e300) for a, b in ((kc, kg), (vc, vg)))
            step = vg.astype(np.float64).copy()
            step[..., 1] = -8 * step[..., 0]
            parts = np.nan_to_num(D.row_values(vc.view(np.uint32), step), nan=1e300, posinf=1e300, neginf=1e300)
            args = (self.table.numpy(), self.cu, [kv for _, kv in self.lens], d ** -0.5 if scale is None else scale, window,
                    None if sinks is None else f64(sinks))
            return *A.paged_attention(f64(self.q), k, v, *args), A.paged_attention(f64(self.q), k, parts, *args)[1]

    def place(self, s, j):
        page = self.cache[0].shape[1]
        return int(self.table[s, j // page]), j % page


def close(p, got, want, scale=None, q_rows=None):
    out, a, info, b = want
    d, dtype = p.q.shape[2], p.dtype
    h = torch.finfo(dtype).eps / 2
    qk, s, n, z = (info[..., i:i + 1] for i in range(4))
    sq = np.abs(f64(p.q if q_rows is None else q_rows)).sum(axis=-1, keepdims=True) * (d ** -0.5 if scale is None else scale)
    e = (F + d * U) * qk + 2.0 ** -25 * sq + 8 * U * s + 2 * U
    tol = (2 * F * (1 + F) * a + F * b + (F + h) * np.abs(out) + 2 * e * a + 2 * (n + 8) * U * a) * (1 + 2.0 ** -6)
    tol += torch.finfo(dtype).smallest_normal * h + 2.0 ** -25 * (n > 0)
    tol += 2.0 ** -25 * n * 8.0 / np.maximum(1.0, z * 2.0 ** -8)  # |v| < 8
    g = f64(got)
    assert np.isfinite(g).all()
    bad = np.abs(g - out) > tol
    assert not bad.any(), (int(bad.sum()), float(np.abs(g - out).max()), np.argwhere(bad)[:4].tolist())


LENS = {
    "tokens": [(1, 1), (1, 2), (1, 63), (1, 65), (1, 256), (1, 257), (1, 700)],
    "one": [(1, 1500)],
    "drafts": [(3, 3), (4, 300), (2, 65), (4, 129), (1, 40)],
    "empty": [(0, 10), (1, 0), (4, 2), (0, 0), (1, 5)],
    "chunk": [(200, 517)],
    "chunks": [(130, 130), (64, 64), (33, 700), (65, 66)],
    "mixed": [(1, 300), (90, 90), (1, 1), (0, 3), (40, 555), (5, 3), (1, 64)],
}


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dtype,hq,hk,d,group,page,heads_first", [
    (BF, 8, 4, 128, 64, 16, True), (HF, 6, 2, 64, 32, 7, False), (BF, 5, 1, 256, 128, 64, True), (HF, 3, 3, 128, 128, 1, False),
    (BF, 32, 2, 64, 64, 200, False), (HF, 8, 2, 256, 32, 48, False), (BF, 4, 4, 128, 32, 24, True), (HF, 4, 2, 256, 64, 16, True)])
def test_matches_the_oracle(lens, dtype, hq, hk, d, group, page, heads_first):
    p = Problem(LENS[lens], hq, hk, d, group, page, dtype, heads_first=heads_first)
    close(p, p.run(), p.oracle())


@pytest.mark.parametrize("lens", ["tokens", "drafts", "chunks", "mixed", "empty"])
@pytest.mark.parametrize("window", [1, 50, 200, 1 << 40])
@pytest.mark.parametrize("dtype,hq,hk,d,page", [(BF, 8, 2, 64, 24), (HF, 4, 4, 128, 16)])
def test_window_and_sinks(lens, window, dtype, hq, hk, d, page):
    p = Problem(LENS[lens], hq, hk, d, 64, page, dtype, seed=window % 97)
    close(p, p.run(window=window, sinks=p.sinks, scale=0.2), p.oracle(0.2, window, p.sinks), 0.2)


@pytest.mark.parametrize("lens", ["tokens", "drafts", "chunk", "mixed"])
def test_scores_that_grow_and_fall(lens):
    """Keys whose scores rise by hundreds, then fall: the running maximum moves, small weights vanish."""
    p = Problem(LENS[lens], 4, 2, 64, 32, 16, BF, seed=3, q_scale=8.0)
    p.cache[1].mul_(torch.linspace(0.1, 6, p.cache[1].shape[0], device=DEV)[:, None, None, None, None].to(HF))
    close(p, p.run(), p.oracle())


@pytest.mark.parametrize("lens", ["tokens", "drafts", "chunks"])
@pytest.mark.parametrize("magnitude", [1e-30, 1e-6, 1e4, 1e30])
def test_queries_of_any_magnitude(lens, magnitude):
    """bf16 queries far outside fp16's range, a row of zeros and rows whose values differ by 2^20; the scale makes up
    for the magnitude."""
    p = Problem(LENS[lens], 4, 2, 128, 64, 16, BF, seed=5)
    p.q[..., ::7] *= 2.0 ** -20
    p.q[0, 0] = 0
    p.q = (p.q.double() * magnitude).to(BF)
    close(p, p.run(scale=0.08 / magnitude), p.oracle(0.08 / magnitude), 0.08 / magnitude)


@pytest.mark.parametrize("lens", ["drafts", "chunk", "chunks"])
@pytest.mark.parametrize("d,group", [(64, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("bias,scale", [(float("nan"), 0.0), (float("inf"), 0.0), (1.0, float("-inf")), (60000.0, 4000.0)])
def test_groups_that_are_not_finite_reach_only_rows_that_see_them(lens, d, group, bias, scale):
    p = Problem(LENS[lens], 4, 2, d, group, 16, BF, seed=4)
    want = p.run()
    hit, last = [], d // group - 1
    for s, (n, kv) in enumerate(LENS[lens]):
        if n > 1:
            j = kv - 1 - (n - 1) // 2  # a new token: the rows before it do not see it
            at = p.place(s, j)
            p.cache[3][at][0, last] = torch.tensor([scale, bias], dtype=HF)  # v of head 0: one group
            p.cache[2][at][0, -1] = -1  # code 15 in its last word
            p.cache[1][at][1] = torch.tensor([0.0, float("nan")], dtype=HF)  # k of head 1
            hit.append((int(p.cu[s]) + j - (kv - n), int(p.cu[s + 1])))
    got = p.run()
    rows = torch.ones(p.q.shape[0], dtype=torch.bool, device=DEV)
    for a, b in hit:
        rows[a:b] = False
    assert torch.equal(got[rows], want[rows])
    for a, b in hit:
        assert torch.isnan(got[a:b, 2:]).all()
        assert torch.equal(got[a:b, :2, :last * group], want[a:b, :2, :last * group])
        if bias != 60000.0:  # (values past fp16's range may be taken as infinite)
            assert not torch.isfinite(got[a, :2, d - 8:]).any()


def test_pages_outside_the_cache_are_not_seen():
    for lens in ("tokens", "chunk", "mixed"):
        for page in (16, 24):
            p = Problem(LENS[lens], 4, 2, 128, 64, page, BF, seed=6)
            bad = torch.rand(p.table.shape, generator=torch.Generator().manual_seed(1)) < 0.3
            p.table[bad] = torch.where(torch.rand(int(bad.sum())) < 0.5, torch.tensor(-1), torch.tensor(p.cache[0].shape[0])).int()
            close(p, p.run(), p.oracle())
            p.table.fill_(2 ** 31 - 1)
            assert (p.run() == 0).all()


def test_device_lengths_past_the_arrays_are_cut():
    """Lengths and offsets that the host could not check: nothing outside the arrays is touched."""
    p = Problem([(1, 40), (3, 20)], 4, 2, 64, 32, 16, BF, odd=False)
    qq, cache, table, cu, kv = p.args()
    guard = torch.full((8, 4, 64), 9.0, dtype=BF, device=DEV)
    out = guard[2:6]
    big = torch.tensor([10 ** 6, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    q.qlinear_paged_attention_4bit(qq, cache, table, cu, big, max_q=3, out=out)
    for c in ([0, 10 ** 6, 10 ** 6 + 5], [-5, 2, 1], [3, 1, 2 ** 31 - 1]):
        c = torch.tensor(c, dtype=torch.int32, device=DEV)
        q.qlinear_paged_attention_4bit(qq, cache, table, c, kv, max_q=3, out=out)
        q.qlinear_paged_attention_4bit(qq, cache, table, c, -kv, max_q=100, out=out)
    torch.cuda.synchronize()
    assert (guard[:2] == 9).all() and (guard[6:] == 9).all()


def test_strided_queries_caches_and_guarded_output():
    for lens, hq, hk, d in ((LENS["tokens"], 4, 2, 128), (LENS["chunks"], 4, 2, 64)):
        p = Problem(lens, hq, hk, d, 32, 16, BF, seed=7)
        want = p.run()
        t = p.q.shape[0]
        qkv = torch.full((t, (hq + 2 * hk) * d), float("nan"), dtype=BF, device=DEV)
        qkv[:, :hq * d] = p.q.reshape(t, hq * d)
        p.q = qkv[:, :hq * d].view(t, hq, d)
        out = torch.full((hq, t + 2, d), 3.0, dtype=BF, device=DEV)
        p.run(out=out[:, 1:-1].transpose(0, 1))
        assert torch.equal(out[:, 1:-1].transpose(0, 1), want)
        assert (out[:, 0] == 3).all() and (out[:, -1] == 3).all()
        for i, x in enumerate(p.cache):  # rows that are parts of a larger array
            pad = (4,) if i % 2 == 0 else (3, 0)
            big = torch.zeros([n + 1 for n in x.shape[:3]] + [n + m for n, m in zip(x.shape[3:], pad)], dtype=x.dtype, device=DEV)
            if i % 2:
                big.fill_(float("nan"))
            part = big[1:, :-1, 1:, :x.shape[3]]
            part.copy_(x)
            p.cache[i] = part
        assert torch.equal(p.run(), want)


def test_many_sequences():
    """More sequences than the workgroups' scans take at once, and lengths that cut items anywhere."""
    r = np.random.default_rng(8)
    lens = [(int(r.integers(0, 3)), int(kv)) for kv in r.integers(0, 400, 600)]
    p = Problem(lens, 2, 1, 64, 64, 16, BF, seed=8)
    close(p, p.run(), p.oracle())
    lens = [(int(n), int(n + e)) for n, e in zip(r.integers(0, 40, 300), r.integers(0, 90, 300))]
    p = Problem(lens, 2, 1, 64, 32, 16, BF, seed=9)
    close(p, p.run(), p.oracle())


def sampled(p, got, places, **kw):
    """Rows (sequence, token, head) of got against the oracle, each as one token of its own."""
    for s, i, h in places:
        n, kv = p.lens[s]
        row, kh, page = int(p.cu[s]) + i, h // (p.q.shape[1] // p.cache[0].shape[2]), p.cache[0].shape[1]
        seen = kv - n + i + 1
        one = Problem.__new__(Problem)
        one.lens, one.dtype, one.cu = [(1, seen)], p.dtype, np.array([0, 1], dtype=np.int32)
        one.q, pages = p.q[row:row + 1, h:h + 1], p.table[s, :-(-seen // page)].long().to(DEV)
        one.cache, one.table = [x[pages, :, kh:kh + 1] for x in p.cache], torch.arange(len(pages))[None]
        kw_one = dict(kw, sinks=kw["sinks"][h:h + 1]) if kw.get("sinks") is not None else kw
        try:
            close(one, got[row:row + 1, h:h + 1], one.oracle(**kw_one))
        except AssertionError as e:
            raise AssertionError(f"sequence {s}, token {i}, head {h}: {e}") from None


@pytest.mark.parametrize("d,group", [(64, 32), (128, 64), (256, 128), (256, 32)])
@pytest.mark.parametrize("dtype,page,window,sinks", [(BF, 16, 0, False), (HF, 24, 500, True), (BF, 1, 70, True), (HF, 128, 0, True)])
def test_whole_row_tiles(d, group, dtype, page, window, sinks):
    """Row tiles of two query heads a kv head, none split, with sequences that are short, empty or before their first
    position among them; then a group of v that is not finite, at a position that some of a tile's rows see."""
    p = Problem([(2500, 2600), (1, 700), (0, 5), (1700, 1700), (1, 1), (60, 30), (0, 0), (3, 9)], 32, 16, d, group, page, dtype, seed=19)
    kw = dict(window=window, sinks=p.sinks if sinks else None)
    got = p.run(**kw)
    rows = [(0, i, (i // 16) % 32) for i in (0, 1, 63, 64, 127, 128, 255, 999, 1791, 2432, 2498, 2499)]
    rows += [(3, i, (7 * i) % 32) for i in (0, 1, 2, 69, 70, 500, 1600, 1664, 1699)]
    rows += [(1, 0, 3), (4, 0, 31), (5, 30, 8), (5, 59, 9), (7, 0, 1), (7, 2, 30)]
    sampled(p, got, rows, **kw)
    at = int(p.cu[5])
    assert (got[at:at + 30] == 0).all()
    first, end = 2500 - 1 - 1200, min(2500, 2500 - 1 - 1200 + (window or 2500))
    where = p.place(0, 2600 - 1 - 1200)
    p.cache[3][where][3, 0] = torch.tensor([0.0, float("nan")], dtype=HF)
    odd = p.run(**kw)
    mask = torch.ones_like(got, dtype=torch.bool)
    mask[first:end, 6:8, :group] = False
    assert torch.equal(odd[mask], got[mask])
    assert not torch.isfinite(odd[first, 6:8, :group]).any()


@pytest.mark.parametrize("hk", [4, 16], ids=["cut into runs", "whole items"])
def test_long_chunks_of_256_values(hk):
    p = Problem([(2010, 4500), (70, 2000)], 2 * hk, hk, 256, 64, 64, BF, seed=15)
    want = p.run()
    places = [(0, i, h) for i, h in zip((0, 1, 777, 1983, 1984, 1990, 2008, 2009, 2009), (0, 1, 5, 0, 3, 6, 7, 2, 2 * hk - 1))]
    sampled(p, want, places + [(1, 0, 0), (1, 69, 2 * hk - 1)])
    for _ in range(5):  # the same bits with the keys in the caches
        assert torch.equal(p.run(), want)


@pytest.mark.parametrize("n_seqs,hk,d,group,dtype", [(64, 8, 64, 32, BF), (100, 8, 128, 64, HF), (300, 3, 64, 64, HF), (60, 4, 256, 64, BF), (400, 1, 128, 128, BF)])
def test_long_runs_of_few_rows(n_seqs, hk, d, group, dtype):
    """So many key tiles (20 a workgroup and more) that an item's start and end are counted in the division: pieces
    recorded by item (up to as many as workgroups) and by workgroup, up to 256 sequences and more."""
    r = np.random.default_rng(n_seqs)
    workgroups = 256 if d == 256 else 512
    tiles = 20 * workgroups * 1.3 / hk / n_seqs
    lens = [(1 + (s % 7 == 3), int(256 * tiles * x) + 1) for s, x in enumerate(r.uniform(0.3, 1.7, n_seqs))]
    lens[1], lens[n_seqs // 2], lens[-1] = (1, 1), (0, 900), (2, 1)
    assert sum(-(-kv // 256) for n, kv in lens if n) * hk >= 20 * workgroups
    p = Problem(lens, 2 * hk, hk, d, group, 16, dtype, seed=18)
    got = p.run()
    assert torch.isfinite(got).all()
    seqs = sorted(set(range(0, n_seqs, max(1, n_seqs // 20))) | {n_seqs - 2})
    sampled(p, got, [(s, lens[s][0] - 1, (5 * s) % (2 * hk)) for s in seqs if lens[s][0] and lens[s][1] >= lens[s][0]])
    assert (got[int(p.cu[-1]) - 2] == 0).all()  # two tokens, one position: the first sees nothing


@pytest.mark.parametrize("lens", ["empty", "drafts", "chunks", "mixed", "one", "long chunk"])
@pytest.mark.parametrize("dtype,d", [(BF, 64), (HF, 128), (BF, 256)])
def test_infinite_sinks(lens, dtype, d):
    """-inf is no term, +inf takes all the weight; a row that sees nothing is zero either way."""
    p = Problem({**LENS, "long chunk": [(40, 3000), (0, 0), (50, 7)]}[lens], 4, 2, d, 64, 16, dtype, seed=16)
    inf = float("inf")
    for sinks in ([-inf, 0.5, inf, -inf], [-inf] * 4):
        sinks = torch.tensor(sinks, device=DEV)
        close(p, p.run(sinks=sinks), p.oracle(sinks=sinks))
    assert torch.equal(p.run(sinks=torch.full((4,), -inf, device=DEV)), p.run())


def test_same_bits_every_time_in_any_workspace_that_is_not_overrun():
    for lens in ("tokens", "one", "drafts", "chunks", "mixed"):
        p = Problem(LENS[lens], 4, 2, 128, 64, 16, BF, seed=11)
        want = p.run()
        n = q.qlinear_paged_attention_4bit_workspace_size(p.q, p.cache, p.table, max_q=max(a for a, _ in p.lens))
        for fill in (0, 171, 255):
            ws = torch.full((n + 4096,), fill, dtype=torch.uint8, device=DEV)
            assert torch.equal(p.run(workspace=ws[:n]), want)
            assert (ws[n:] == fill).all()


def test_graph_replays_follow_the_device_lengths():
    p = Problem([(1, 200), (1, 37), (2, 90)], 4, 2, 64, 32, 16, BF, seed=13, extra=3)
    qq, cache, table, cu, kv = p.args()
    out = torch.empty_like(qq)
    n = q.qlinear_paged_attention_4bit_workspace_size(qq, cache, table, max_q=2)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    run = lambda o: q.qlinear_paged_attention_4bit(qq, cache, table, cu, kv, max_q=2, out=o, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    for i in range(4):
        kv.copy_(torch.tensor([200 - 60 * i, 37 - i, 90 - 20 * i], dtype=torch.int32))
        qq.mul_(0.9)
        want = torch.empty_like(out)
        run(want)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_cache_past_32_bit_offsets():
    hk, d, page, n_pages = 8, 128, 128, 70000  # 4.6 GB of codes of k
    codes = [torch.zeros(n_pages, hk, page, d // 8, dtype=torch.int32, device=DEV).transpose(1, 2) for _ in range(2)]
    groups = [torch.zeros(n_pages, hk, page, d // 32, 2, dtype=HF, device=DEV).transpose(1, 2) for _ in range(2)]
    small = Problem([(1, 300), (70, 290)], 16, hk, d, 32, page, BF, seed=14)
    big, moved = [codes[0], groups[0], codes[1], groups[1]], small.table.clone()
    for s in range(2):
        for j in range(3):
            moved[s, j] = n_pages - 1 - 5 * (3 * s + j)
            for x, y in zip(big, small.cache):
                x[moved[s, j]] = y[small.table[s, j]]
    want = small.run()
    small.cache, small.table = big, moved
    assert torch.equal(small.run(), want)


def test_groups_of_a_page_past_32_bits():
    """The words of a page's 16 slots 300 MB apart (pages and heads next to each other)."""
    hk, d, page = 2, 128, 16
    small = Problem([(1, 300), (70, 290), (3, 40)], 8, hk, d, 32, page, BF, seed=15)
    n_pages, per = small.cache[0].shape[0], 2 * d // 32
    token, far = 150_000_006, []
    assert n_pages * hk * per < token and 2 * 15 * token > 1 << 32
    for x in small.cache[1::2]:
        buf = torch.empty(15 * token + n_pages * hk * per, dtype=HF, device=DEV)
        far.append(buf.as_strided(x.shape, (hk * per, token, per, 2, 1)))
        far[-1].copy_(x)
    want = small.run()
    small.cache[1::2] = far
    assert torch.equal(small.run(), want)


def test_no_sequences_no_tokens_no_pages():
    cache = q.qlinear_paged_cache_4bit(2, 4, 2, 64, 32)
    i32 = dict(dtype=torch.int32, device=DEV)
    e = torch.empty(0, 4, 64, dtype=BF, device=DEV)
    assert q.qlinear_paged_attention_4bit(e, cache, torch.zeros(1, 2, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32),
                                          max_q=1).shape == e.shape
    x = torch.ones(2, 4, 64, dtype=BF, device=DEV)
    out = q.qlinear_paged_attention_4bit(x, cache, torch.zeros(2, 0, **i32), torch.arange(3, **i32), torch.ones(2, **i32), max_q=1)
    assert (out == 0).all()
    none = tuple(c[:0] for c in cache)
    out = q.qlinear_paged_attention_4bit(x, none, torch.zeros(2, 1, **i32), torch.arange(3, **i32), torch.ones(2, **i32), max_q=1)
    assert (out == 0).all()


@pytest.mark.parametrize("lens", [[(1, 40000)], [(3, 20000), (1, 100)], [(40, 40000)]])
def test_weights_below_the_normal_range_count(lens):
    """One key of weight 1 with v = 0 and many of weight 2^-17 with v = 1: the sum of the small ones, which are exact in
    fp16, is a share of it all."""
    p = Problem(lens, 2, 1, 64, 64, 16, HF, seed=22, odd=False)
    p.q.zero_()
    p.q[..., 0] = 1
    for i in (0, 2):
        p.cache[i].zero_()
    p.cache[1].zero_()
    p.cache[3].zero_()
    p.cache[3][..., 1] = 1.0
    for s in range(len(lens)):
        at = p.place(s, 0)
        p.cache[0][at][0, 0], p.cache[1][at][0, 0, 0] = 1, 17.0  # code 1 of the first value
        p.cache[3][at] = 0
    got = f64(p.run(scale=float(np.log(2.0))))
    for s, (n, kv) in enumerate(lens):
        for i in range(n):
            small = (kv - n + i) * 2.0 ** -17
            o = small / (1 + small)
            assert np.abs(got[int(p.cu[s]) + i] - o).max() <= (2 ** -11 + 2 ** -16) * o


def test_after_an_append_it_is_the_attention_of_the_values_that_are_stored():
    """Append, read back, and the 16-bit attention over what was read: the same up to both kernels' roundings."""
    t, hq, hk, d, page = 300, 8, 2, 128, 16
    x, k, v = (torch.randn(t, h, d, device=DEV).to(HF) for h in (hq, hk, hk))
    cache, slots = q.qlinear_paged_cache_4bit(20, page, hk, d), torch.arange(t, device=DEV)
    q.qlinear_kv_append_4bit(k, v, cache, slots)
    kb, vb = q.qlinear_kv_read_4bit(cache, torch.arange(320, device=DEV), dtype=HF)
    i32 = dict(dtype=torch.int32, device=DEV)
    table, cu, lens = torch.arange(20, **i32)[None], torch.tensor([0, t], **i32), torch.tensor([t], **i32)
    got = q.qlinear_paged_attention_4bit(x, cache, table, cu, lens, max_q=t)
    want = q.qlinear_paged_attention(x, kb.view(20, page, hk, d), vb.view(20, page, hk, d), table, cu, lens, max_q=t)
    # both take the same fp16 keys and values; the references of the weights differ: weights round twice (2^-11
    # each, on values below 5), outputs once each
    assert ((got.float() - want.float()).abs() <= 2 * 2.0 ** -11 * 5 + 2 * 2.0 ** -11 * want.float().abs()).all()


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("page,heads_first", [(16, True), (64, False), (24, True)])
def test_more_than_sixteen_rows(d, group, page, heads_first):
    """Sequences whose rows fill two column tiles of the few-row kernel (5 tokens of 4 heads and others), whole tiles, cut
    ones and tails, in several pieces."""
    p = Problem([(5, 5), (5, 64), (5, 700), (8, 2049), (1, 1), (3, 9000), (5, 130), (0, 4)], 16, 4, d, group, page, BF, seed=23, heads_first=heads_first)
    got = p.run()
    places = [(0, 0, 0), (0, 4, 15), (1, 0, 3), (1, 4, 8), (2, 0, 1), (2, 4, 14), (3, 0, 0), (3, 7, 15), (3, 3, 9), (4, 0, 5), (5, 0, 2), (5, 2, 13), (6, 2, 7)]
    sampled(p, got, places)
    kw = dict(window=100, sinks=p.sinks)
    sampled(p, p.run(**kw), places, **kw)
