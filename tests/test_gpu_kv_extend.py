"""qlinear_kv_extend against the oracle: every number equal."""
import numpy as np
import pytest
import torch

import weight_only_quantized_affine_amd as q
from oracle import decoder_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Step:
    def __init__(self, counts, lens, page, rows, spare=3, extra=None, seed=0, short=0, width=None):
        r = np.random.default_rng(seed)
        self.counts, self.lens, self.page, self.rows = counts, lens, page, rows
        had = [-(-x // page) for x in lens]
        after = [-(-(x + max(c, 0)) // page) for c, x in zip(counts, lens)]
        self.width = max(after + [1]) + 1 if width is None else width
        n = sum(after) + spare
        order = r.permutation(n).tolist()
        self.table = np.full((len(lens), self.width), -5, dtype=np.int64)
        at = 0
        for s, h in enumerate(had):
            self.table[s, :h] = order[at:at + h]
            at += h
        self.free = order[at:len(order) - short]
        self.cap = n if extra is None else len(self.free) + extra  # room for every page

    def run(self, in_place=False, with_list=True, stride=0):
        n = len(self.lens)
        wide = torch.full((n, self.width + stride), -9, dtype=torch.int32, device=DEV)
        table = wide[:, :self.width]
        table.copy_(torch.from_numpy(self.table).int())
        counts, lens = i32(self.counts), i32(self.lens)
        free = torch.full((self.cap,), -3, dtype=torch.int32, device=DEV)
        free[:len(self.free)] = i32(self.free)
        fc = i32([len(self.free)])
        kw = dict(free_pages=free, free_count=fc) if with_list else {}
        lens_out, fc_out = (lens, fc) if in_place else (torch.empty_like(lens), torch.empty_like(fc))
        if not in_place:
            kw["lens_out"] = lens_out
            if with_list:
                kw["free_count_out"] = fc_out
        cu, pos, slots, info = q.qlinear_kv_extend(counts, lens, table, page_size=self.page, rows=self.rows, **kw)
        want = D.kv_extend(self.counts, self.lens, self.table.tolist(), self.page, self.rows, (self.free, self.cap) if with_list else None)
        got = [x.tolist() for x in (cu, pos, slots, lens_out, table)]
        for name, g, w in zip(("cu_q", "positions", "slots", "lens", "table"), got, want):
            assert g == w, (name, info.tolist())
        assert info.tolist() == want[6]
        if with_list:
            assert int(fc_out) == len(want[5]) and free[:len(want[5])].tolist() == want[5]
        if not in_place:
            assert lens.tolist() == list(self.lens) and int(fc) == len(self.free)
        assert counts.tolist() == list(self.counts)
        assert (wide[:, self.width:] == -9).all()
        return info.tolist()


RNG = np.random.default_rng(1)
STEPS = {
    "one": ([1], [0], 16, 1), "rest": ([0, 0], [5, 0], 4, 3), "decode": ([1] * 60 + [0] * 4, [int(x) for x in RNG.integers(1, 900, 64)], 16, 64),
    "page of one": ([3, 1, 0, 7], [0, 9, 2, 1], 1, 20), "chunks": ([100, 1, 333, 0, 64], [0, 17, 40, 8, 64], 24, 700),
    "through": ([-1, 2, -7, 1, -2 ** 31], [33, 8, 0, 15, 100], 8, 9), "all through": ([-1] * 5, [20, 300, 1, 0, 64], 16, 0),
    "many": ([int(x) for x in RNG.integers(-1, 4, 2500)], [int(x) for x in RNG.integers(0, 90, 2500)], 7, 6000),
    "many rows": ([int(x) for x in RNG.integers(0, 60, 300)], [int(x) for x in RNG.integers(0, 500, 300)], 16, 20000),
    "1024": ([1] * 1024, list(range(1024)), 16, 1024), "1025": ([2] * 1025, list(range(1025)), 16, 4100),
    "long rows": ([5000, -1, 3000], [10, 9000, 0], 2, 8500),
}


@pytest.mark.parametrize("name", list(STEPS))
@pytest.mark.parametrize("in_place", [False, True])
def test_steps(name, in_place):
    info = Step(*STEPS[name]).run(in_place, stride=3)
    assert info[2] == 0


@pytest.mark.parametrize("name", list(STEPS))
def test_steps_without_a_list(name):
    counts, lens, page, rows = STEPS[name]
    s = Step(counts, lens, page, rows)
    s.table[s.table < 0] = 11
    assert s.run(with_list=False)[:3] == [sum(max(c, 0) for c in counts), 0, 0]


@pytest.mark.parametrize("spare,short", [(0, 0), (5, 5)])
def test_the_last_page_is_taken(spare, short):
    assert Step([17, 1, 16], [0, 16, 5], 16, 40, spare=spare, short=short, extra=0).run()[2:] == [0, 0]


def test_refusals_change_nothing():
    assert Step([17, 1], [0, 16], 16, 17).run()[2] == 1
    assert Step([17, 1], [0, 16], 16, 18, spare=0, short=1).run(in_place=True)[2] == 2
    assert Step([17, 1], [0, 16], 16, 18, width=1).run()[2] == 4
    assert Step([1, -1], [4, 40], 16, 18, extra=2).run()[2] == 8
    assert Step([9, -1], [4, 40], 16, 3, extra=2).run()[2] == 9
    s = Step([1, 1], [0, 16], 16, 18)
    s.lens = [-1, 16]
    s.counts = [1, 1]
    want = [0, 0, 4, len(s.free)]
    assert s.run() == want
    s.counts = [-1, 1]
    assert s.run() == want
    s.counts, s.lens = [2 ** 31 - 1, 2 ** 31 - 1], [2 ** 31 - 1, 16]
    assert s.run()[2] & 4
    for with_list in (False, True):
        big = Step([3000] * 2, [0, 0], 16, 5999)
        assert big.run(with_list=with_list)[2] == 1


@pytest.mark.parametrize("count,cap", [(-1, 8), (9, 8), (2 ** 31 - 1, 8)])
def test_a_count_of_free_pages_that_cannot_be(count, cap):
    table, free = torch.full((1, 4), 3, dtype=torch.int32, device=DEV), torch.arange(cap, dtype=torch.int32, device=DEV)
    lens, fc = i32([4]), i32([count])
    cu, pos, slots, info = q.qlinear_kv_extend(i32([1]), lens, table, page_size=4, rows=2, free_pages=free, free_count=fc)
    assert info.tolist()[:2] == [0, 0] and info.tolist()[2] & 8 and info.tolist()[3] == count
    assert cu.tolist() == [0, 0] and slots.tolist() == [-1, -1] and pos.tolist() == [0, 0]
    assert lens.tolist() == [4] and int(fc) == count and (table == 3).all() and free.tolist() == list(range(cap))


def test_no_sequences_and_no_pages():
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    cu, pos, slots, info = q.qlinear_kv_extend(z, z, torch.zeros(0, 3, dtype=torch.int32, device=DEV), page_size=4, rows=3)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 3 and info.tolist() == [0, 0, 0, 0]
    one = i32([0])
    cu, pos, slots, info = q.qlinear_kv_extend(one, one, torch.zeros(1, 0, dtype=torch.int32, device=DEV), page_size=4, rows=0)
    assert cu.tolist() == [0, 0] and info.tolist() == [0, 0, 0, 0]
    assert q.qlinear_kv_extend(i32([1]), one, torch.zeros(1, 0, dtype=torch.int32, device=DEV), page_size=4, rows=2)[3].tolist() == [0, 0, 4, 0]


def test_outputs_end_where_they_end():
    s = Step(*STEPS["chunks"])
    n, rows = len(s.lens), s.rows
    buf = {k: torch.full((m + 8,), 77, dtype=t, device=DEV)
           for k, m, t in (("cu_q", n + 1, torch.int32), ("positions", rows, torch.int64), ("slots", rows, torch.int64), ("info", 4, torch.int32), ("lens_out", n, torch.int32))}
    free = torch.full((s.cap + 8,), 77, dtype=torch.int32, device=DEV)
    free[:len(s.free)] = i32(s.free)
    table = torch.full((n + 2, s.width), 77, dtype=torch.int32, device=DEV)
    table[:n] = torch.from_numpy(s.table).int()
    q.qlinear_kv_extend(i32(s.counts), i32(s.lens), table[:n], page_size=s.page, rows=rows, free_pages=free[:s.cap], free_count=i32([len(s.free)]),
                        **{k: b[:-8] for k, b in buf.items()})
    assert all((b[-8:] == 77).all() for b in buf.values()) and (free[s.cap:] == 77).all() and (table[n:] == 77).all()


def test_a_captured_step_runs_on():
    """One graph, in place: lengths, tables and the list move from replay to replay as on the host."""
    page, n = 4, 6
    table = torch.full((n, 30), -1, dtype=torch.int32, device=DEV)
    free, fc, lens, counts = torch.arange(200, dtype=torch.int32, device=DEV), i32([120]), i32([0] * n), i32([0] * n)
    host = (list(range(120)), 200)
    state = [[0] * n, table.tolist()]
    graph = torch.cuda.CUDAGraph()
    bufs = dict(cu_q=torch.empty(n + 1, dtype=torch.int32, device=DEV), info=torch.empty(4, dtype=torch.int32, device=DEV),
                positions=torch.empty(50, dtype=torch.int64, device=DEV), slots=torch.empty(50, dtype=torch.int64, device=DEV))
    with torch.cuda.graph(graph):
        q.qlinear_kv_extend(counts, lens, table, page_size=page, rows=50, free_pages=free, free_count=fc, **bufs)
    r = np.random.default_rng(3)
    for i in range(12):
        c = [int(x) for x in r.integers(-1, 9, n)]
        counts.copy_(i32(c))
        graph.replay()
        cu, pos, slots, state[0], state[1], stack, info = D.kv_extend(c, state[0], state[1], page, 50, host)
        host = (stack, 200)
        got = [x.tolist() for x in (bufs["cu_q"], bufs["positions"], bufs["slots"], lens, table, bufs["info"])]
        assert got == [cu, pos, slots, state[0], state[1], info] and free[:int(fc)].tolist() == stack


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows", [4000, 30000])
def test_more_sequences_than_shared_memory_holds(in_place, rows):
    r = np.random.default_rng(5)
    counts = [int(x) for x in r.integers(-1, 2 if rows == 4000 else 6, 6001)]
    if rows == 4000:
        counts = [c if i % 3 else min(c, 0) for i, c in enumerate(counts)]
    info = Step(counts, [int(x) for x in r.integers(0, 40, 6001)], 8, rows).run(in_place)
    assert info[2] == 0 and info[0] > rows // 4


def test_a_list_without_entries():
    """An empty tensor of free pages is a list that gives nothing and takes nothing, not the absence of one."""
    for counts, lens, why in (([1, 0], [3, 4], 0), ([1, 0], [4, 4], 2), ([-1, 0], [0, 4], 0), ([-1, 0], [3, 4], 8)):
        step = Step(counts, lens, 4, 2, spare=0)
        step.free, step.cap = [], 0
        assert step.run()[2] == why and step.run(in_place=True)[2] == why
    table, free = i32([[0, 1]]), i32([])
    for kw in (dict(free_pages=free), dict(free_pages=i32([5])), dict(free_count=i32([0]))):
        with pytest.raises(q.QLError, match="free_pages and free_count"):
            q.qlinear_kv_extend(i32([1]), i32([1]), table, page_size=4, rows=1, **kw)
    with pytest.raises(q.QLError):
        q.qlinear_kv_extend(i32([1]), i32([1]), table, page_size=4, rows=1, free_count_out=i32([0]))
