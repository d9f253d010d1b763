"""qlinear_paged_attention against the 64-bit oracle.

Tolerance of an output o = sum w_j v_j with A = sum w_j |v_j| (u = 2^-24, h = half a step of the
16-bit type relative to the value):
  h (A + |o|)   each weight rounds once, in the product and in the sum;   h |o|   the output rounds once
  2 E A         E bounds the relative error of an unnormalised weight (numerator and sum): the
                score's fp32 sum of d products, d u sum|q k| scale, its scaling and difference,
                4 u (|s| + |max|), and the exponential, 2 u
  2 (n + 8) u A the fp32 sums over n keys, the rescalings and the quotient
  fp16 only: weights below 2^-14 of the reference keep an absolute 2^-25 each, and the reference
  weighs at least 1, so 2^-25 sum|v| / max(1, 2^-8 sum e^(s - max)) more.
"""
import numpy as np
import pytest
import torch

import weight_only_quantized_affine_amd as q
from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
U = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


class Problem:
    """Sequences of (new tokens, cached tokens), shuffled pages, and slots past the lengths that hold
    infinities and NaN."""

    def __init__(self, lens, hq, hk, d, page, dtype, seed=0, heads_first=False, fill=float("nan"), extra=1, q_scale=2.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.dtype = lens, dtype
        need = [-(-kv // page) for _, kv in lens]
        n_pages = sum(need) + extra
        order = torch.randperm(n_pages, generator=g).int()
        self.table = torch.full((len(lens), max(max(need), 1)), -7, dtype=torch.int32)
        at = 0
        caches = [torch.full((n_pages, page, hk, d), fill, dtype=torch.float32) for _ in range(2)]
        for s, (n, kv) in enumerate(lens):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
            for j in range(need[s]):
                m = min(page, kv - j * page)
                for c in caches:
                    c[self.table[s, j], :m] = torch.randn(m, hk, d, generator=g)
        self.k, self.v = (c.to(dtype).to(DEV) for c in caches)
        if heads_first:
            self.k, self.v = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (self.k, self.v))
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.q = (torch.randn(int(self.cu[-1]), hq, d, generator=g) * q_scale).to(dtype).to(DEV)
        self.sinks = torch.randn(hq, generator=g).to(DEV)

    def args(self):
        return (self.q, self.k, self.v, self.table.to(DEV), torch.from_numpy(self.cu).to(DEV),
                torch.tensor([kv for _, kv in self.lens], dtype=torch.int32, device=DEV))

    def run(self, **kw):
        kw.setdefault("max_q", max(max(n for n, _ in self.lens), 1))
        return q.qlinear_paged_attention(*self.args(), **kw)

    def oracle(self, scale=None, window=0, sinks=None):
        d = self.q.shape[2]
        clean = lambda c: np.nan_to_num(f64(c), nan=1e300)  # noqa: E731  (what must not be read shows)
        return A.paged_attention(f64(self.q), clean(self.k), clean(self.v), self.table.numpy(), self.cu,
                                 [kv for _, kv in self.lens], d ** -0.5 if scale is None else scale, window,
                                 None if sinks is None else f64(sinks))


def close(got, want, scale_d, dtype):
    out, a, info = want
    h = torch.finfo(dtype).eps / 2
    qk, s, n, z = (info[..., i:i + 1] for i in range(4))
    e = scale_d * U * qk + 8 * U * s + 2 * U
    tol = (h * a + 2 * h * np.abs(out) + 2 * e * a + 2 * (n + 8) * U * a) * (1 + 2.0 ** -6)
    tol += torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    if dtype == HF:
        tol += 2.0 ** -25 * n * 6.0 / np.maximum(1.0, z * 2.0 ** -8)  # |v| < 6
    g = f64(got)
    assert np.isfinite(g).all()
    bad = np.abs(g - out) > tol
    assert not bad.any(), (int(bad.sum()), float(np.abs(g - out).max()), np.argwhere(bad)[:4].tolist())


FEW = [(1, 1), (1, 2), (1, 31), (1, 33), (1, 128), (1, 129), (1, 700)]
LENS = {
    "tokens": FEW,
    "one": [(1, 1500)],
    "drafts": [(3, 3), (4, 300), (2, 65), (4, 129), (1, 40)],
    "empty": [(0, 10), (1, 0), (4, 2), (0, 0), (1, 5)],
    "chunk": [(200, 517)],
    "chunks": [(130, 130), (64, 64), (33, 700), (65, 66)],
    "mixed": [(1, 300), (90, 90), (1, 1), (0, 3), (40, 555), (5, 3), (1, 64)],
}


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dtype,hq,hk,d,page,heads_first", [(BF, 8, 4, 128, 16, False), (HF, 6, 2, 64, 7, True),
                                                            (BF, 5, 1, 256, 64, False), (HF, 3, 3, 128, 1, False),
                                                            (BF, 32, 2, 64, 200, True)])
def test_matches_the_oracle(lens, dtype, hq, hk, d, page, heads_first):
    p = Problem(LENS[lens], hq, hk, d, page, dtype, heads_first=heads_first)
    close(p.run(), p.oracle(), d, dtype)


@pytest.mark.parametrize("lens", ["tokens", "drafts", "chunks", "mixed", "empty"])
@pytest.mark.parametrize("window", [1, 50, 200, 1 << 40])
@pytest.mark.parametrize("dtype,hq,hk,d", [(BF, 8, 2, 64), (HF, 4, 4, 128)])
def test_window_and_sinks(lens, window, dtype, hq, hk, d):
    p = Problem(LENS[lens], hq, hk, d, 24, dtype, seed=window % 97)
    close(p.run(window=window, sinks=p.sinks, scale=0.2), p.oracle(0.2, window, p.sinks), d, dtype)


@pytest.mark.parametrize("lens", ["tokens", "drafts", "chunk", "mixed"])
def test_scores_that_grow_and_fall(lens):
    """Keys whose scores rise by hundreds, then fall: the running maximum moves, small weights vanish."""
    p = Problem(LENS[lens], 4, 2, 64, 16, BF, seed=3, q_scale=8.0)
    p.k.mul_(torch.linspace(0.1, 6, p.k.shape[0], device=DEV)[:, None, None, None].to(BF))
    close(p.run(), p.oracle(), 64, BF)


@pytest.mark.parametrize("lens", ["drafts", "chunk", "chunks"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_non_finite_keys_and_values_reach_only_rows_that_see_them(lens, d, value):
    p = Problem(LENS[lens], 4, 2, d, 16, BF, seed=4)
    want = p.run()
    hit = []
    for s, (n, kv) in enumerate(LENS[lens]):
        if n > 1:
            j = kv - 1 - (n - 1) // 2  # a new token: the rows before it do not see it
            page, place = int(p.table[s, j // 16]), j % 16
            p.v[page, place, 0, 3] = value
            p.k[page, place, 1, :] = value
            hit.append((int(p.cu[s]) + j - (kv - n), int(p.cu[s + 1])))
    got = p.run()
    rows = np.ones(p.q.shape[0], dtype=bool)
    for a, b in hit:
        rows[a:b] = False
    r = torch.from_numpy(rows).to(DEV)
    assert torch.equal(got[r], want[r])
    # rows that see the value: heads 0, 1 read it in one place of v, heads 2, 3 in all of k
    for a, b in hit:
        if value != value:
            assert torch.isnan(got[a:b, :2, 3]).all()
        else:
            # the weight of that key may be zero in fp32 (then 0 * inf)
            assert (~torch.isfinite(got[a:b, :2, 3])).all() or (got[a:b, :2, 3] == value).any()
        assert torch.equal(got[a:b, :2, :3], want[a:b, :2, :3]) and torch.equal(got[a:b, :2, 4:], want[a:b, :2, 4:])


def test_pages_outside_the_cache_are_not_seen():
    for lens in ("tokens", "chunk", "mixed"):
        p = Problem(LENS[lens], 4, 2, 128, 16, BF, seed=6)
        bad = torch.rand(p.table.shape, generator=torch.Generator().manual_seed(1)) < 0.3
        p.table[bad] = torch.where(torch.rand(int(bad.sum())) < 0.5, torch.tensor(-1), torch.tensor(p.k.shape[0])).int()
        close(p.run(), p.oracle(), 128, BF)
        p.table.fill_(2 ** 31 - 1)
        assert (p.run() == 0).all()


def test_device_lengths_past_the_arrays_are_cut():
    """Lengths and offsets that the host could not check: nothing outside the arrays is touched."""
    p = Problem([(1, 40), (3, 20)], 4, 2, 64, 16, BF, fill=0.0)
    qq, k, v, table, cu, kv = p.args()
    guard = torch.full((8, 4, 64), 9.0, dtype=BF, device=DEV)
    out = guard[2:6]
    big = torch.tensor([10 ** 6, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    q.qlinear_paged_attention(qq, k, v, table, cu, big, max_q=3, out=out)
    for c in ([0, 10 ** 6, 10 ** 6 + 5], [-5, 2, 1], [3, 1, 2 ** 31 - 1]):
        q.qlinear_paged_attention(qq, k, v, table, torch.tensor(c, dtype=torch.int32, device=DEV), kv, max_q=3, out=out)
        q.qlinear_paged_attention(qq, k, v, table, torch.tensor(c, dtype=torch.int32, device=DEV), -kv, max_q=100, out=out)
    torch.cuda.synchronize()
    assert (guard[:2] == 9).all() and (guard[6:] == 9).all()


def test_strided_queries_and_guarded_output():
    for lens, hq, hk, d in ((LENS["tokens"], 4, 2, 128), (LENS["chunks"], 4, 2, 64)):
        p = Problem(lens, hq, hk, d, 16, BF, seed=7)
        want = p.run()
        t = p.q.shape[0]
        qkv = torch.full((t, (hq + 2 * hk) * d), float("nan"), dtype=BF, device=DEV)
        qkv[:, :hq * d] = p.q.reshape(t, hq * d)
        p.q = qkv[:, :hq * d].view(t, hq, d)
        out = torch.full((hq, t + 2, d), 3.0, dtype=BF, device=DEV)
        p.run(out=out[:, 1:-1].transpose(0, 1))
        assert torch.equal(out[:, 1:-1].transpose(0, 1), want)
        assert (out[:, 0] == 3).all() and (out[:, -1] == 3).all()


def test_many_sequences():
    """More sequences than the workgroups' scans take at once, and lengths that cut items anywhere."""
    r = np.random.default_rng(8)
    lens = [(int(r.integers(0, 3)), int(kv)) for kv in r.integers(0, 400, 600)]
    p = Problem(lens, 2, 1, 64, 16, BF, seed=8)
    close(p.run(), p.oracle(), 64, BF)
    lens = [(int(n), int(n + e)) for n, e in zip(r.integers(0, 40, 300), r.integers(0, 90, 300))]
    p = Problem(lens, 2, 1, 64, 16, BF, seed=9)
    close(p.run(), p.oracle(), 64, BF)


def test_one_workgroup_per_row_tile():
    """Enough row tiles that none is split: 4300 tokens x 32 heads, checked at rows of every tile."""
    lens = [(4000, 4100), (300, 300)]
    p = Problem(lens, 32, 32, 64, 64, BF, seed=10)
    got = p.run()
    rows = list(range(0, 4300, 97)) + [3999, 4000, 4299]
    for i in rows:
        s = int(i >= 4000)
        n, kv = lens[s]
        seen = kv - n + (i - int(p.cu[s])) + 1
        one = Problem.__new__(Problem)
        one.lens, one.dtype, one.cu = [(1, seen)], BF, np.array([0, 1], dtype=np.int32)
        one.q, one.k, one.v, one.table = p.q[i:i + 1], p.k, p.v, p.table[s:s + 1]
        h = i % 32
        one.q = one.q[:, h:h + 1]
        one.k, one.v = p.k[:, :, h:h + 1], p.v[:, :, h:h + 1]
        close(got[i:i + 1, h:h + 1], one.oracle(), 64, BF)


def test_same_bits_every_time_and_any_workspace():
    for lens in ("tokens", "chunks", "mixed"):
        p = Problem(LENS[lens], 4, 2, 128, 16, BF, seed=11)
        want = p.run()
        n = q.qlinear_paged_attention_workspace_size(p.q, p.k, p.table, max_q=max(a for a, _ in p.lens))
        for fill in (0, 255):
            ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
            assert torch.equal(p.run(workspace=ws), want)


def test_workspace_is_not_overrun():
    for lens in ("one", "drafts", "chunks", "mixed"):
        p = Problem(LENS[lens], 8, 2, 64, 16, BF, seed=12)
        n = q.qlinear_paged_attention_workspace_size(p.q, p.k, p.table, max_q=max(a for a, _ in p.lens))
        ws = torch.full((n + 4096,), 171, dtype=torch.uint8, device=DEV)
        p.run(workspace=ws[:n])
        assert (ws[n:] == 171).all()


def test_graph_replays_follow_the_device_lengths():
    p = Problem([(1, 200), (1, 37), (2, 90)], 4, 2, 64, 16, BF, seed=13, extra=3)
    qq, k, v, table, cu, kv = p.args()
    out = torch.empty_like(qq)
    n = q.qlinear_paged_attention_workspace_size(qq, k, table, max_q=2)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    run = lambda o: q.qlinear_paged_attention(qq, k, v, table, cu, kv, max_q=2, out=o, workspace=ws)  # noqa: E731
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
    hk, d, page, n_pages = 8, 128, 128, 17000  # 4.46 GB of keys: offsets past 2^32 bytes
    k = torch.zeros(n_pages, page, hk, d, dtype=BF, device=DEV)
    v = torch.zeros_like(k)
    small = Problem([(1, 300), (70, 290)], 16, hk, d, page, BF, seed=14)
    moved = small.table.clone()
    for s in range(2):
        for j in range(3):
            moved[s, j] = n_pages - 1 - 5 * (3 * s + j)
            k[moved[s, j]] = small.k[small.table[s, j]]
            v[moved[s, j]] = small.v[small.table[s, j]]
    want = small.run()
    small.k, small.v, small.table = k, v, moved
    assert torch.equal(small.run(), want)


def test_no_sequences_no_tokens_no_pages():
    k = torch.zeros(2, 4, 2, 64, dtype=BF, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    e = torch.empty(0, 4, 64, dtype=BF, device=DEV)
    assert q.qlinear_paged_attention(e, k, k, torch.zeros(1, 2, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32),
                                     max_q=1).shape == e.shape
    x = torch.ones(2, 4, 64, dtype=BF, device=DEV)
    out = q.qlinear_paged_attention(x, k, k, torch.zeros(2, 0, **i32), torch.arange(3, **i32), torch.ones(2, **i32), max_q=1)
    assert (out == 0).all()
    none = k[:0]
    out = q.qlinear_paged_attention(x, none, none, torch.zeros(2, 1, **i32), torch.arange(3, **i32), torch.ones(2, **i32),
                                    max_q=1)
    assert (out == 0).all()


def sampled(p, got, places, **kw):
    """Rows (sequence, token, head) of got against the oracle, each as one token of its own."""
    for s, i, h in places:
        n, kv = p.lens[s]
        row, kh, page = int(p.cu[s]) + i, h // (p.q.shape[1] // p.k.shape[2]), p.k.shape[1]
        seen = kv - n + i + 1
        one = Problem.__new__(Problem)
        one.lens, one.dtype, one.cu = [(1, seen)], p.dtype, np.array([0, 1], dtype=np.int32)
        one.q, pages = p.q[row:row + 1, h:h + 1], p.table[s, :-(-seen // page)].long().to(DEV)
        one.k, one.v, one.table = p.k[pages, :, kh:kh + 1], p.v[pages, :, kh:kh + 1], torch.arange(len(pages))[None]
        kw_one = dict(kw, sinks=kw["sinks"][h:h + 1]) if kw.get("sinks") is not None else kw
        try:
            close(got[row:row + 1, h:h + 1], one.oracle(**kw_one), p.q.shape[2], p.dtype)
        except AssertionError as e:
            raise AssertionError(f"sequence {s}, token {i}, head {h}: {e}") from None


@pytest.mark.parametrize("hk", [4, 16], ids=["cut into runs", "whole items"])
def test_long_chunks_of_256_values(hk):
    """Row tiles of 128 rows over many key tiles whose last row tile leaves waves without rows (2010 x 2
    rows: 52 in the last): every key tile's scores are of that tile, in every call."""
    p = Problem([(2010, 4500), (70, 2000)], 2 * hk, hk, 256, 64, BF, seed=15)
    want = p.run()
    places = [(0, i, h) for i, h in zip((0, 1, 777, 1983, 1984, 1990, 2008, 2009, 2009), (0, 1, 5, 0, 3, 6, 7, 2, 2 * hk - 1))]
    sampled(p, want, places + [(1, 0, 0), (1, 69, 2 * hk - 1)])
    for _ in range(5):  # the same bits with the keys in the caches
        assert torch.equal(p.run(), want)


@pytest.mark.parametrize("lens", ["empty", "drafts", "chunks", "mixed", "one", "long chunk"])
@pytest.mark.parametrize("dtype,d", [(BF, 64), (HF, 128), (BF, 256)])
def test_infinite_sinks(lens, dtype, d):
    """-inf is no term, +inf takes all the weight; a row that sees nothing is zero either way.  In every
    epilogue: whole items and cut ones of few and of many rows."""
    p = Problem({**LENS, "long chunk": [(40, 3000), (0, 0), (50, 7)]}[lens], 4, 2, d, 16, dtype, seed=16)
    inf = float("inf")
    for sinks in ([-inf, 0.5, inf, -inf], [-inf] * 4):
        sinks = torch.tensor(sinks, device=DEV)
        close(p.run(sinks=sinks), p.oracle(sinks=sinks), d, dtype)
    assert torch.equal(p.run(sinks=torch.full((4,), -inf, device=DEV)), p.run())


def test_infinite_sinks_of_whole_row_tiles():
    """Row tiles that are not split, and rows before the first cached position."""
    p = Problem([(2200, 1900), (2100, 2100)], 32, 32, 64, 64, BF, seed=17)
    sinks = torch.zeros(32, device=DEV)
    sinks[::3], sinks[1::3] = -float("inf"), float("inf")
    got = p.run(sinks=sinks)
    assert (got[:300] == 0).all() and (got[:, 1::3] == 0).all()
    assert torch.equal(got[:, ::3], p.run()[:, ::3])
    sampled(p, got, [(0, 300, 0), (0, 2199, 3), (1, 0, 6), (1, 1000, 2), (1, 2099, 31)], sinks=sinks)


class Large(Problem):
    """As Problem, with caches of finite values made on the GPU."""

    def __init__(self, lens, hq, hk, d, page, dtype, seed=0):
        g, c = torch.Generator(device=DEV).manual_seed(seed), torch.Generator().manual_seed(seed)
        self.lens, self.dtype = lens, dtype
        need = [-(-kv // page) for _, kv in lens]
        self.table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
        order, at = torch.randperm(sum(need), generator=c).int(), 0
        for s, m in enumerate(need):
            self.table[s, :m] = order[at:at + m]
            at += m
        self.k, self.v = (torch.randn(sum(need), page, hk, d, generator=g, device=DEV).to(dtype) for _ in range(2))
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.q = (torch.randn(int(self.cu[-1]), hq, d, generator=g, device=DEV) * 2).to(dtype)
        self.sinks = torch.randn(hq, generator=c).to(DEV)


@pytest.mark.parametrize("n_seqs,hk,d,dtype", [(64, 8, 64, BF), (100, 8, 128, HF), (300, 3, 64, HF), (60, 4, 256, BF), (400, 1, 128, BF)])
def test_long_runs_of_few_rows(n_seqs, hk, d, dtype):
    """So many key tiles (20 a workgroup and more) that an item's start and end are counted in the division:
    pieces recorded by item (up to as many as workgroups) and by workgroup, up to 256 sequences and more."""
    r = np.random.default_rng(n_seqs)
    tiles = 20 * (256 if d == 256 else 512) * 1.3 / hk / n_seqs
    lens = [(1 + (s % 7 == 3), int(128 * tiles * x) + 1) for s, x in enumerate(r.uniform(0.3, 1.7, n_seqs))]
    lens[1], lens[n_seqs // 2], lens[-1] = (1, 1), (0, 900), (2, 1)
    assert sum(-(-kv // 128) for n, kv in lens if n) * hk >= 20 * (256 if d == 256 else 512)
    p = Large(lens, 2 * hk, hk, d, 16, dtype, seed=18)
    got = p.run()
    assert torch.isfinite(got).all()
    seqs = sorted(set(range(0, n_seqs, max(1, n_seqs // 40))) | {n_seqs - 2})
    sampled(p, got, [(s, lens[s][0] - 1, (5 * s) % (2 * hk)) for s in seqs if lens[s][0] and lens[s][1] >= lens[s][0]])
    assert (got[int(p.cu[-1]) - 2] == 0).all()  # two tokens, one position: the first sees nothing
    # every (token, head) against the same sequence by itself, which is divided otherwise
    for s in seqs[::8]:
        if lens[s][0]:
            a, b = int(p.cu[s]), int(p.cu[s + 1])
            one = q.qlinear_paged_attention(p.q[a:b], p.k, p.v, p.table[s:s + 1].to(DEV), torch.tensor([0, b - a], dtype=torch.int32, device=DEV),
                                            torch.tensor([lens[s][1]], dtype=torch.int32, device=DEV), max_q=b - a)
            # weights rounded under two references (half a step each), then both outputs
            assert ((one.float() - got[a:b].float()).abs() <= 4 * torch.finfo(dtype).eps).all()


WHOLE = [(2500, 2600), (1, 700), (0, 5), (1700, 1700), (1, 1), (60, 30), (0, 0), (3, 9)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,page,window,sinks", [(BF, 16, 0, False), (HF, 24, 500, True), (BF, 1, 70, True), (HF, 128, 0, True)])
def test_whole_row_tiles(d, dtype, page, window, sinks):
    """Row tiles of two query heads a kv head, none split, with sequences that are short, empty or before
    their first position among them, and more workgroups than row tiles."""
    p = Problem(WHOLE, 32, 16, d, page, dtype, seed=19)
    kw = dict(window=window, sinks=p.sinks if sinks else None)
    got = p.run(**kw)
    rows = [(0, i, (i // 16) % 32) for i in (0, 1, 63, 64, 127, 128, 255, 999, 1791, 2432, 2498, 2499)]
    rows += [(3, i, (7 * i) % 32) for i in (0, 1, 2, 69, 70, 500, 1600, 1664, 1699)]
    rows += [(1, 0, 3), (4, 0, 31), (5, 30, 8), (5, 59, 9), (7, 0, 1), (7, 2, 30)]
    sampled(p, got, rows, **kw)
    at = int(p.cu[5])
    assert (got[at:at + 30] == 0).all()
    # a NaN, then an infinity, in V of a position that is new: the rows before it do not see it
    j = 2600 - 1 - 1200
    where = (int(p.table[0, j // page]), j % page, 3, 5)
    first, end = 2500 - 1 - 1200, min(2500, 2500 - 1 - 1200 + (window or 2500))
    for value in (float("nan"), float("inf")):
        p.v[where] = value
        odd = p.run(**kw)
        mask = torch.ones_like(got, dtype=torch.bool)
        mask[first:end, 6:8, 5] = False
        assert torch.equal(odd[mask], got[mask])
        assert not torch.isfinite(odd[first, 6:8, 5]).any()


def test_more_sequences_than_a_plan_holds():
    r = np.random.default_rng(20)
    lens = [(20, int(20 + e)) for e in r.integers(0, 60, 4100)]
    lens[7], lens[4099] = (0, 3), (19, 30)
    p = Large(lens, 1, 1, 64, 16, BF, seed=20)
    got = p.run()
    sampled(p, got, [(s, i, 0) for s, i in zip([*range(0, 4100, 205), 4098, 4099], [*range(20), 19, 18]) if lens[s][0] > i])
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("lens", [[(1, 5000)], [(3, 900), (2, 66)], [(200, 517)], [(70, 3000), (1, 400)], [(300, 300), (40, 5000)]])
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, HF), (256, BF)])
def test_keys_that_are_not_finite_reach_every_row_that_sees_them(lens, d, dtype):
    p = Problem(lens, 4, 2, d, 16, dtype, seed=21)
    want = p.run()
    s, (n, kv) = len(lens) - 1, lens[-1]
    j = kv - 1 - (n - 1) // 2
    first = int(p.cu[s]) + j - (kv - n)  # first row that sees j
    keep = p.k.clone()
    # a whole row: q.k is NaN, since q has values of both signs
    for value in (float("nan"), float("inf"), float("-inf")):
        p.k[int(p.table[s, j // 16]), j % 16, 1] = value
        got = p.run()
        assert torch.isnan(got[first:int(p.cu[s + 1]), 2:]).all()
        assert torch.equal(got[:, :2], want[:, :2]) and torch.equal(got[:first, 2:], want[:first, 2:])
    # one infinite value: a score of +-infinity, NaN or no weight
    p.k.copy_(keep)
    p.k[int(p.table[s, j // 16]), j % 16, 1, 3] = float("inf")
    got = p.run()
    q3 = p.q[first:int(p.cu[s + 1]), 2:, 3]
    rows = got[first:int(p.cu[s + 1]), 2:]
    assert torch.isnan(rows[q3 > 0]).all() and torch.isfinite(rows[q3 < 0]).all()
    for i in range(first - int(p.cu[s]), n, max(1, n // 9)):
        for h in (2, 3):
            if float(p.q[int(p.cu[s]) + i, h, 3]) < 0:
                sampled(p, got, [(s, i, h)])
    # every score NaN, in every piece
    p.k.fill_(float("nan"))
    got = p.run()
    sees = torch.cat([torch.arange(a) >= a - b for a, b in lens]).to(DEV)
    assert torch.isnan(got[sees]).all() and (got[~sees] == 0).all()


@pytest.mark.parametrize("lens", [[(1, 40000)], [(3, 20000), (1, 100)], [(40, 40000)]])
def test_fp16_weights_below_the_normal_range_count(lens):
    """One key of weight 1 with v = 0 and many of weight 2^-17 with v = 1: the sum of the small ones, which
    are exact in fp16, is a share of it all."""
    p = Problem(lens, 2, 1, 64, 16, HF, seed=22)
    p.q.zero_()
    p.q[..., 0] = 1
    p.k.zero_()
    p.v.fill_(1.0)
    for s in range(len(lens)):
        p.k[int(p.table[s, 0]), 0, 0, 0] = 17.0
        p.v[int(p.table[s, 0]), 0] = 0.0
    got = f64(p.run(scale=float(np.log(2.0))))
    for s, (n, kv) in enumerate(lens):
        for i in range(n):
            small = (kv - n + i) * 2.0 ** -17
            o = small / (1 + small)
            assert np.abs(got[int(p.cu[s]) + i] - o).max() <= (2 ** -11 + 2 ** -16) * o
