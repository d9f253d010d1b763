"""qlinear_select_experts and qlinear_combine_experts against the 64-bit oracle.

The chosen experts are equal (both sides choose in 64 bits); a weight is off by its rounding to fp32, 2^-24
of it, and by 64-bit errors far below.  A combined value is off by its fp32 sums, (k + 2) 2^-24 of the sum of
its terms' magnitudes, and by its rounding, half a step of its type relative to the value.
"""
import numpy as np
import pytest
import torch

import weight_only_quantized_affine_amd as q
from oracle import decoder_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def check(x, k, bias=None, **kw):
    ids, w = q.qlinear_select_experts(x, k, bias=bias, **kw)
    want, ww = D.select_experts(f64(x), k, bias=None if bias is None else f64(bias), **kw)
    assert ids.tolist() == want.tolist()
    assert ids.dtype == torch.int64 and w.dtype == FP
    assert (np.abs(f64(w) - ww) <= U * (1 + 1e-6) * np.abs(ww) + 2.0 ** -150).all()
    return ids, w


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 128, 8), (5, 7, 7), (3, 64, 4), (9, 65, 2), (33, 32, 4), (2, 1024, 64), (7, 300, 10),
                                   (4, 513, 1), (200, 256, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_choice(dtype, t, e, k, sigmoid):
    g = torch.Generator().manual_seed(e + k)
    x = (torch.randn(t, e, generator=g) * 2).to(dtype).to(DEV)
    b = (torch.randn(e, generator=g) * 0.2).to(DEV)
    for bias in (None, b):
        check(x, k, bias, sigmoid=sigmoid, renormalize=True, scale=1.0)
        check(x, k, bias, sigmoid=sigmoid, renormalize=False, scale=2.5)


@pytest.mark.parametrize("e,n_groups,top,group_top,k", [(256, 8, 4, 2, 8), (160, 8, 3, 1, 6), (64, 64, 5, 2, 5), (60, 3, 2, 2, 40), (18, 6, 6, 2, 4),
                                                        (640, 5, 1, 2, 64), (1024, 16, 3, 1, 9), (36, 12, 1, 1, 3), (512, 33 - 1, 8, 2, 8), (66, 33, 20, 2, 7)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups(e, n_groups, top, group_top, k, sigmoid):
    g = torch.Generator().manual_seed(e)
    x = (torch.randn(50, e, generator=g) * 1.5).to(DEV)
    b = (torch.randn(e, generator=g) * 0.1).to(DEV)
    for bias in (None, b):
        check(x, k, bias, sigmoid=sigmoid, n_groups=n_groups, top_groups=top, group_top=group_top, renormalize=True, scale=2.5)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_ties_go_to_the_lowest_index(dtype):
    r = np.random.default_rng(0)
    x = torch.from_numpy(r.integers(-2, 3, (64, 256))).to(dtype).to(DEV)  # five values
    bias = torch.zeros(256, device=DEV)
    for kw in (dict(), dict(sigmoid=True), dict(n_groups=16, top_groups=4, group_top=2), dict(n_groups=8, top_groups=8, group_top=1)):
        check(x, 8, **kw)
        check(x, 8, bias, **kw)
    assert check(torch.zeros(3, 100, dtype=dtype, device=DEV), 5)[0].tolist() == [[0, 1, 2, 3, 4]] * 3


def test_values_next_to_each_other():
    """Scores that differ in the last bits of fp32 logits, and biases that nearly make up for it."""
    base = torch.full((1, 256), 0.7)
    step = torch.arange(256).flip(0)[None] * 2.0 ** -23
    x = (base + step[:, torch.randperm(256, generator=torch.Generator().manual_seed(1))]).to(DEV)
    for kw in (dict(), dict(sigmoid=True)):
        check(x, 64, **kw)
        check(x, 64, -torch.sigmoid(x[0]), **kw)


def test_values_that_are_not_finite():
    inf, nan = float("inf"), float("nan")
    x = torch.randn(8, 40, generator=torch.Generator().manual_seed(2))
    x[0, 3], x[1, 5:9], x[2] = inf, inf, -inf
    x[3], x[4, 0], x[5, ::2], x[6, 7], x[7, 1:] = nan, -inf, nan, -1e30, -inf
    for dtype in (FP, BF, HF):
        y = x.to(dtype).to(DEV)
        for kw in (dict(), dict(renormalize=False), dict(sigmoid=True), dict(n_groups=4, top_groups=2, group_top=2)):
            check(y, 6, **kw)
    bias = torch.zeros(40, device=DEV)
    bias[4], bias[9], bias[20] = -inf, inf, nan
    finite = torch.randn(8, 40, generator=torch.Generator().manual_seed(3)).to(DEV)
    for kw in (dict(), dict(sigmoid=True)):
        check(finite, 40, bias, **kw)
        check(finite, 3, bias, **kw)


def test_large_logits():
    x = torch.tensor([[3e38, -3e38, 1e3, 0.0], [800.0, 1.0, 799.0, 0.0], [-800.0, -801.0, -1e4, -3e38]], device=DEV)
    for kw in (dict(), dict(sigmoid=True), dict(renormalize=False)):
        check(x, 4, **kw)


def test_strided_rows_padding_and_guards():
    x = torch.randn(20, 300, generator=torch.Generator().manual_seed(4)).to(DEV)
    part = x[::2, 17:145]
    want = q.qlinear_select_experts(part.contiguous(), 8)
    for g, w in zip(q.qlinear_select_experts(part, 8), want):
        assert torch.equal(g, w)
    half = x.to(BF)[:, 1:]  # rows that begin at two bytes
    for g, w in zip(q.qlinear_select_experts(half, 3), q.qlinear_select_experts(half.contiguous(), 3)):
        assert torch.equal(g, w)
    for n in (0, 1, 7, 10, 99, -5):
        ids, w = torch.full((12, 8), 55, device=DEV), torch.full((12, 8), 5.0, device=DEV)
        q.qlinear_select_experts(part, 8, ids=ids[1:-1], weights=w[1:-1], n_rows=torch.tensor([n], dtype=torch.int32, device=DEV))
        m = min(max(n, 0), 10)
        assert torch.equal(ids[1:1 + m], want[0][:m]) and torch.equal(w[1:1 + m], want[1][:m])
        assert (ids[1 + m:-1] == -1).all() and (w[1 + m:-1] == 0).all()
        assert (ids[[0, -1]] == 55).all() and (w[[0, -1]] == 5).all()
    assert q.qlinear_select_experts(x[:0], 4)[0].shape == (0, 4)


def test_many_tokens():
    x = torch.randn(5000, 128, generator=torch.Generator().manual_seed(5)).to(DEV)
    ids, w = q.qlinear_select_experts(x, 8)
    p = torch.softmax(x.double(), dim=1)
    top = p.sort(dim=1, descending=True, stable=True)
    assert torch.equal(ids, top.indices[:, :8])
    ref = top.values[:, :8] / top.values[:, :8].sum(dim=1, keepdim=True)
    assert ((w.double() - ref).abs() <= U * (1 + 1e-6) * ref).all()


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("t,k,n", [(1, 1, 1), (3, 4, 2880), (17, 8, 129), (5, 2, 8), (9, 13, 100), (2, 64, 40), (300, 8, 256), (1, 6, 4096), (40, 3, 12)])
@pytest.mark.parametrize("residual", [False, True])
def test_combination(dtype, t, k, n, residual):
    g = torch.Generator().manual_seed(t * k + n)
    y, r = torch.randn(t * k, n, generator=g).to(dtype), torch.randn(t, n, generator=g).to(dtype)
    w = torch.randn(t, k, generator=g)
    ids = torch.randint(-2, 10, (t, k), generator=g)
    gone = ((ids < 0) | (ids >= 8)).view(-1)
    for use in (False, True):
        z = y.clone()
        if use:
            z[gone] = float("nan")  # not looked at
        kw = dict(ids=ids.to(DEV), e=8) if use else {}
        out = torch.full((t + 2, n), 7.0, dtype=dtype, device=DEV)
        got = q.qlinear_combine_experts(z.to(DEV), w.to(DEV), residual=r.to(DEV) if residual else None, out=out[1:-1], **kw)
        want, mag = D.combine_experts(f64(z), f64(w), ids.numpy() if use else None, 8, f64(r) if residual else None)
        h = torch.finfo(dtype).eps / 2
        tol = (k + 2) * U * mag * (1 + h) + h * np.abs(want) + torch.finfo(dtype).smallest_normal * h
        assert (np.abs(f64(got) - want) <= tol).all()
        assert (out[[0, -1]] == 7).all()


def test_combination_into_its_residual_at_any_alignment():
    for dtype in (BF, FP):
        t, k, n = 6, 4, 64
        y = torch.randn(t * k * n + 9, device=DEV).to(dtype)
        w, r = torch.rand(t, k, device=DEV), torch.randn(t * n + 9, device=DEV).to(dtype)
        want = q.qlinear_combine_experts(y[8:-1].view(t * k, n).clone(), w, residual=r[8:-1].view(t, n).clone())
        for shift in (1, 3, 8):
            yy, rr = y.clone(), r.clone()
            yy[shift:shift + t * k * n], rr[shift:shift + t * n] = y[8:-1], r[8:-1]
            rows = rr[shift:shift + t * n].view(t, n)
            got = q.qlinear_combine_experts(yy[shift:shift + t * k * n].view(t * k, n), w, residual=rows, out=rows)
            assert torch.equal(got, want)


def test_combination_of_infinities():
    inf, nan = float("inf"), float("nan")
    y = torch.tensor([[inf, 1.0, -inf, 3e38], [inf, nan, 2.0, 3e38]], device=DEV)
    got = q.qlinear_combine_experts(y, torch.tensor([[1.0, 1.0]], device=DEV))[0].tolist()
    assert got[0] == inf and got[1] != got[1] and got[2] == -inf and got[3] == inf
    got = q.qlinear_combine_experts(y, torch.tensor([[1.0, 0.0]], device=DEV))[0].tolist()
    assert got[0] != got[0] and got[2] == -inf and got[3] == np.float32(3e38)


def test_captured_with_the_routed_experts():
    """Router, experts and combination as one layer runs them, from one graph, padding included."""
    e, k, n, dim, t = 8, 2, 64, 256, 12
    g = torch.Generator(device=DEV).manual_seed(6)
    codes = torch.randint(0, 256, (e, n, dim // 2), generator=g, device=DEV).to(torch.uint8)
    scales = torch.randint(118, 126, (e, n, dim // 32), generator=g, device=DEV).to(torch.uint8)
    x, logits = torch.randn(t, dim, generator=g, device=DEV).to(BF), torch.randn(t, e, generator=g, device=DEV)
    res, rows = torch.randn(t, n, generator=g, device=DEV).to(BF), torch.tensor([t], dtype=torch.int32, device=DEV)
    ids, w, out = torch.empty(t, k, dtype=torch.int64, device=DEV), torch.empty(t, k, device=DEV), torch.empty(t, n, dtype=BF, device=DEV)
    y, ws = torch.empty(t * k, n, dtype=BF, device=DEV), torch.empty(q.qlinear_apply_experts_workspace_size(t * k, e), dtype=torch.uint8, device=DEV)

    def layer():
        q.qlinear_select_experts(logits, k, ids=ids, weights=w, n_rows=rows)
        q.qlinear_apply_experts(q.QL_MXFP4, codes, scales, ids.view(-1), x, n=n, k=dim, pos_per_row=k, y=y, workspace=ws)
        q.qlinear_combine_experts(y, w, ids=ids, e=e, residual=res, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    dense = q.qlinear_dequant(q.QL_MXFP4, codes, scales, rows=e * n, k=dim).view(e, n, dim)
    for m in (t, 5, 0, t):
        logits.normal_(generator=g)
        x.normal_(generator=g)
        rows.fill_(m)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        p = torch.softmax(logits.double(), dim=1).topk(k, dim=1)
        assert torch.equal(ids[:m], p.indices[:m]) and (ids[m:] == -1).all()
        weight = p.values / p.values.sum(dim=1, keepdim=True)
        for i in range(t):
            want, mag = res[i].double(), res[i].double().abs()
            for j in range(k if i < m else 0):
                row = dense[p.indices[i, j]].double() @ x[i].double()
                want, mag = want + weight[i, j] * row, mag + weight[i, j] * (dense[p.indices[i, j]].double().abs() @ x[i].double().abs())
            # the experts' fp32 sums (dim terms) and rounding to bf16, then this sum and its rounding
            assert ((got[i].double() - want).abs() <= 2.0 ** -7 * mag + 2.0 ** -8 * want.abs()).all()
        layer()
        assert torch.equal(out, got)


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("low", [-700.0, -709.0, -709.75, -720.0, -740.0])
def test_sigmoids_next_to_the_smallest_numbers(low, renormalize):
    """Logits whose sigmoid, e^x there, lies around and below the smallest normal number of 64 bits: they are still in
    order, and the k largest of a row of nothing else share the weight by their ratios."""
    x = (low - torch.arange(9.0) / 4)[None, [3, 0, 7, 5, 1, 8, 2, 6, 4]]
    ids, w = q.qlinear_select_experts(x.to(DEV), 4, sigmoid=True, renormalize=renormalize, scale=2.0)
    order = [1, 4, 6, 0]
    assert ids.tolist() == [order]
    if renormalize:
        e = np.exp(f64(x[0, order]) - low)
        # a p is off by the smallest number, 2^-1074, which is up to 2^-1074 / e^x of it; twice for its share
        off = 2.0 ** -23 + 4 * np.exp(-1074 * np.log(2.0) - f64(x[0, order]).min())
        assert (np.abs(f64(w[0]) - 2 * e / e.sum()) <= off * 2).all()
    else:
        assert (w == 0).all()
