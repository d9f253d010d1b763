"""Refusals of the entry points around a cache in 4 bits and around routed experts, on the host before any
launch (no GPU)."""
import ctypes
import os
import re

import pytest
import torch

import weight_only_quantized_affine_amd as q

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE = range(7)
F32, F16, BF16 = 0, 1, 2
FAKE = 0x100000  # a 16-byte aligned non-NULL address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(q.lib_path()):
        import __graft_entry__

        __graft_entry__.build()
    return q.load_library()


def heads(p=FAKE, n=8, ts=1024, hs=128):
    return q._Heads(p, n, ts, hs)


def cache(**kw):
    a = dict(k_codes=FAKE, v_codes=FAKE, k_groups=FAKE, v_groups=FAKE, n_pages=4, page_size=16, hk=8, d=128, group_size=64,
             page_stride=8192, token_stride=64, head_stride=1024, group_page_stride=256, group_token_stride=2,
             group_head_stride=32)
    a.update(kw)
    return q._PagedCache4(**a)


def nrope(**kw):
    a = dict(q_weight=FAKE, k_weight=FAKE, w_dtype=BF16, eps=1e-6, positions=FAKE, cos_sin=FAKE, max_pos=64, rot=128,
             interleaved=0)
    a.update(kw)
    return q._NormRope(**a)


def ref(s):
    return None if s is None else ctypes.addressof(s)


BAD_CACHES = ((dict(k_codes=None), NULL), (dict(v_groups=None), NULL), (dict(v_codes=FAKE + 8), ALIGN),
              (dict(k_groups=FAKE + 2), ALIGN), (dict(page_size=0), SHAPE), (dict(n_pages=-1), SHAPE), (dict(hk=0), SHAPE),
              (dict(token_stride=40), ALIGN), (dict(page_stride=-16), ALIGN), (dict(group_token_stride=-1), SHAPE),
              (dict(group_head_stride=1 << 38), SHAPE), (dict(n_pages=1 << 28), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
              (dict(d=0), UNSUPPORTED), (dict(d=576), UNSUPPORTED), (dict(group_size=16), UNSUPPORTED),
              (dict(group_size=0), UNSUPPORTED), (dict(group_size=256, d=256), UNSUPPORTED))


def append(lib, qh=None, qo=None, k=None, v=None, c=None, slots=FAKE, dtype=BF16, t=2, nr=None):
    return lib.qlinear_kv_append_4bit(ref(qh), ref(qo), ref(k), ref(v), ref(c), slots, dtype, t, ref(nr), None)


def test_append_refusals(lib):
    h, n, c = heads(), nrope(), cache()
    assert append(lib, k=h, v=h, c=c, dtype=F32, nr=n) == DTYPE
    assert append(lib, k=h, v=h, c=None, nr=n) == NULL
    assert append(lib, k=None, v=h, c=c, nr=n) == NULL
    assert append(lib, k=h, v=None, c=c, nr=n) == NULL
    assert append(lib, k=h, v=h, c=c, nr=None) == NULL
    assert append(lib, k=h, v=h, c=c, slots=None, nr=n) == NULL
    assert append(lib, k=h, v=h, c=c, slots=FAKE + 4, nr=n) == ALIGN
    assert append(lib, k=heads(n=4), v=h, c=c, nr=n) == SHAPE
    assert append(lib, k=h, v=heads(n=4), c=c, nr=n) == SHAPE
    assert append(lib, qh=h, qo=None, k=h, v=h, c=c, nr=n) == NULL
    assert append(lib, k=h, v=h, c=c, t=-1, nr=n) == SHAPE
    assert append(lib, k=h, v=h, c=c, t=1 << 31, nr=n) == UNSUPPORTED
    for bad, st in BAD_CACHES:
        assert append(lib, k=h, v=h, c=cache(**bad), nr=n) == st, bad
    assert append(lib, k=h, v=h, c=c, t=0, slots=None, nr=n) == OK
    assert lib.qlinear_last_error() == b""


def test_read_refusals(lib):
    def read(c=cache(), slots=FAKE, t=2, k=heads(), v=heads(), dtype=BF16):
        return lib.qlinear_kv_read_4bit(ref(c), slots, t, ref(k), ref(v), dtype, None)

    for bad, st in ((dict(c=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=heads(n=4)), SHAPE),
                    (dict(slots=None), NULL), (dict(slots=FAKE + 4), ALIGN), (dict(t=-1), SHAPE), (dict(dtype=F32), DTYPE),
                    (dict(v=heads(p=None)), NULL), (dict(k=heads(ts=4)), ALIGN), (dict(t=1 << 24), UNSUPPORTED)):
        assert read(**bad) == st, bad
    for bad, st in BAD_CACHES:
        assert read(c=cache(**bad)) == st, bad
    assert read(t=0, slots=None) == OK


def attend(lib, qh=None, out=None, dtype=BF16, t=2, c=None, table=FAKE, stride=4, pages=4, cu=FAKE, lens=FAKE, n=1,
           max_q=2, scale=0.1, window=0, sinks=None, ws=FAKE, ws_bytes=1 << 40):
    return lib.qlinear_paged_attention_4bit(ref(qh), ref(out), dtype, t, ref(c), table, stride, pages, cu, lens, n, max_q,
                                            scale, window, sinks, ws, ws_bytes, None)


def test_attention_refusals(lib):
    h, c = heads(n=16, ts=2048), cache()
    ok = dict(qh=h, out=h, c=c)
    for bad, st in ((dict(dtype=F32), DTYPE), (dict(c=None), NULL), (dict(qh=None), NULL), (dict(out=None), NULL),
                    (dict(c=cache(d=192)), UNSUPPORTED), (dict(c=cache(d=512)), UNSUPPORTED), (dict(qh=heads(n=12)), SHAPE),
                    (dict(out=heads(n=8)), SHAPE), (dict(t=-1), SHAPE), (dict(n=-1), SHAPE), (dict(max_q=-1), SHAPE),
                    (dict(pages=-1), SHAPE), (dict(stride=-1), SHAPE), (dict(scale=0.0), SHAPE),
                    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(window=-1), SHAPE),
                    (dict(cu=None), NULL), (dict(lens=None), NULL), (dict(table=None), NULL), (dict(cu=FAKE + 2), ALIGN),
                    (dict(sinks=FAKE + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws_bytes=64), WORKSPACE),
                    (dict(ws=FAKE + 4), ALIGN), (dict(pages=1 << 28), UNSUPPORTED), (dict(t=1 << 30), UNSUPPORTED),
                    (dict(qh=heads(p=None, n=16)), NULL), (dict(qh=heads(n=16, ts=4)), ALIGN)):
        assert attend(lib, **{**ok, **bad}) == st, bad
    for bad, st in BAD_CACHES:
        assert attend(lib, **{**ok, "c": cache(**bad)}) == st, bad
    for nothing in (dict(t=0), dict(n=0), dict(max_q=0)):
        assert attend(lib, **{**ok, **nothing, "ws": None}) == OK


def test_attention_workspace_size(lib):
    size = lib.qlinear_paged_attention_4bit_workspace_size
    assert size(0, 1, 16, 8, 128, 1, 4, 16, 0) == 0
    assert size(1, 1, 16, 5, 128, 1, 4, 16, 0) == 0
    few, many = size(4, 4, 16, 8, 128, 1, 64, 16, 0), size(300, 1, 16, 8, 128, 300, 64, 16, 0)
    assert 0 < few < many
    h = heads(n=16, ts=2048)
    assert attend(lib, qh=h, out=h, c=cache(), t=4, n=4, max_q=1, pages=64, ws_bytes=few - 1) == WORKSPACE
    big = (1 << 63) - 1
    for window in (64 * 16, 1 << 40, big):
        assert size(80, 16, 32, 8, 128, 5, 64, 16, window) == size(80, 16, 32, 8, 128, 5, 64, 16, 0)


def test_extend_refusals(lib):
    names = ("counts lens n_seqs block_table table_stride max_pages page_size free_pages free_cap free_count lens_out "
             "free_count_out cu_q positions slots rows info").split()
    base = dict(counts=FAKE, lens=FAKE, n_seqs=3, block_table=FAKE, table_stride=8, max_pages=8, page_size=16,
                free_pages=FAKE, free_cap=9, free_count=FAKE, lens_out=FAKE, free_count_out=FAKE, cu_q=FAKE,
                positions=FAKE, slots=FAKE, rows=4, info=FAKE)

    def extend(**kw):
        a = {**base, **kw}
        return lib.qlinear_kv_extend(*[a[n] for n in names], None)

    for n in ("n_seqs", "rows", "max_pages", "table_stride", "free_cap"):
        assert extend(**{n: -1}) == SHAPE, n
    for n in ("counts", "lens", "lens_out", "block_table", "cu_q", "info", "positions", "slots", "free_count", "free_count_out"):
        assert extend(**{n: None}) == NULL, n
    for n in ("counts", "lens", "lens_out", "block_table", "cu_q", "info", "free_pages", "free_count", "free_count_out"):
        assert extend(**{n: FAKE + 2}) == ALIGN, n
    for n in ("positions", "slots"):
        assert extend(**{n: FAKE + 4}) == ALIGN, n
    for bad, st in ((dict(page_size=0), SHAPE), (dict(table_stride=7), SHAPE), (dict(free_pages=None), NULL),
                    (dict(free_pages=None, free_cap=0), NULL), (dict(free_pages=None, free_count=None, free_count_out=None), NULL),
                    (dict(n_seqs=1 << 24), UNSUPPORTED), (dict(rows=(1 << 31) - 1), UNSUPPORTED),
                    (dict(free_cap=1 << 31), UNSUPPORTED), (dict(max_pages=1 << 27, table_stride=1 << 27), UNSUPPORTED),
                    (dict(table_stride=1 << 38), SHAPE)):
        assert extend(**bad) == st, bad


def test_select_refusals(lib):
    names = ("logits dtype t e row_stride bias sigmoid n_groups top_groups group_top k renormalize scale n_rows ids "
             "weights").split()
    base = dict(logits=FAKE, dtype=F32, t=3, e=64, row_stride=64, bias=None, sigmoid=0, n_groups=8, top_groups=2,
                group_top=2, k=4, renormalize=1, scale=1.0, n_rows=None, ids=FAKE, weights=FAKE)

    def select(**kw):
        a = {**base, **kw}
        return lib.qlinear_select_experts(*[a[n] for n in names], None)

    for bad, st in ((dict(dtype=7), DTYPE), (dict(t=-1), SHAPE), (dict(t=1 << 31), SHAPE), (dict(e=0), UNSUPPORTED),
                    (dict(e=1025, n_groups=1, top_groups=1), UNSUPPORTED), (dict(n_groups=0), SHAPE), (dict(n_groups=7), SHAPE),
                    (dict(e=130, n_groups=65), SHAPE), (dict(top_groups=0), SHAPE), (dict(top_groups=9), SHAPE),
                    (dict(group_top=0), SHAPE), (dict(group_top=3), SHAPE), (dict(k=0), SHAPE), (dict(k=17), SHAPE),
                    (dict(k=65, e=512), SHAPE), (dict(row_stride=-1), SHAPE), (dict(scale=float("nan")), SHAPE),
                    (dict(scale=float("inf")), SHAPE), (dict(logits=None), NULL), (dict(ids=None), NULL),
                    (dict(weights=None), NULL), (dict(logits=FAKE + 2), ALIGN), (dict(ids=FAKE + 4), ALIGN),
                    (dict(weights=FAKE + 2), ALIGN), (dict(bias=FAKE + 2), ALIGN), (dict(n_rows=FAKE + 2), ALIGN)):
        assert select(**bad) == st, bad
    assert select(t=0, logits=None) == OK


def test_combine_refusals(lib):
    names = "y dtype weights ids e residual t k n out".split()
    base = dict(y=FAKE, dtype=BF16, weights=FAKE, ids=FAKE, e=8, residual=FAKE, t=3, k=2, n=64, out=FAKE)

    def combine(**kw):
        a = {**base, **kw}
        return lib.qlinear_combine_experts(*[a[n] for n in names], None)

    for bad, st in ((dict(dtype=5), DTYPE), (dict(t=-1), SHAPE), (dict(n=-1), SHAPE), (dict(e=-1), SHAPE), (dict(k=0), SHAPE),
                    (dict(k=65), SHAPE), (dict(t=1 << 20, n=1 << 11), UNSUPPORTED), (dict(y=None), NULL),
                    (dict(weights=None), NULL), (dict(out=None), NULL), (dict(y=FAKE + 1), ALIGN),
                    (dict(residual=FAKE + 1), ALIGN), (dict(out=FAKE + 1), ALIGN), (dict(weights=FAKE + 2), ALIGN),
                    (dict(ids=FAKE + 4), ALIGN), (dict(dtype=F32, y=FAKE + 2), ALIGN)):
        assert combine(**bad) == st, bad
    assert combine(t=0, y=None) == OK and combine(n=0, out=None) == OK


def test_launches_of_2_32_threads_are_refused(lib):
    """The largest launch has 2^32 - 1 threads: 64 a token of a choice, 8 to 64 a row of an append."""
    for t in ((1 << 26) - 3, 1 << 26, (1 << 31) - 1):
        assert lib.qlinear_select_experts(FAKE, F32, t, 8, 8, None, 0, 1, 1, 1, 2, 1, 1.0, None, FAKE, FAKE, None) == UNSUPPORTED
        assert b"2^26" in lib.qlinear_last_error()
    # 8 + 8 rows of 16 lanes a token, and with 8 heads of q, four a lane, two more; 64 lanes at 512 values
    for t, d, qh in ((1 << 24, 128, None), (1 << 24, 128, heads()), (15_000_000, 128, heads()), (1 << 22, 512, None)):
        n, c, k = nrope(), cache(d=d, group_size=64), heads()
        assert append(lib, qh=qh, qo=qh, k=k, v=k, c=c, t=t, nr=n) == UNSUPPORTED, (t, d)
        assert b"threads" in lib.qlinear_last_error()


def test_combine_takes_ids_only_with_their_number(lib):
    """Without e every id would lie outside [0, e) and no expert be counted."""
    args = lambda ids, e, t=3, n=64: (FAKE, BF16, FAKE, ids, e, None, t, 2, n, FAKE, None)  # noqa: E731
    for t, n in ((3, 64), (0, 64), (3, 0)):
        assert lib.qlinear_combine_experts(*args(FAKE, 0, t, n)) == SHAPE
        assert b"e must be >= 1" in lib.qlinear_last_error()
    assert lib.qlinear_combine_experts(*args(None, 0, 0)) == OK
    assert lib.qlinear_combine_experts(*args(FAKE, 1, 0)) == OK
    for t in (0, 2):
        y, w, ids = torch.zeros(t * 2, 8), torch.zeros(t, 2), torch.zeros(t, 2, dtype=torch.int64)
        with pytest.raises(q.QLError, match="must be given with ids"):
            q.qlinear_combine_experts(y, w, ids=ids, residual=torch.zeros(t, 8))


def test_binding_refuses_wrong_tensors():
    bf, i32 = torch.bfloat16, dict(dtype=torch.int32)
    k = torch.zeros(2, 4, 64, dtype=bf)
    c = q.qlinear_paged_cache_4bit(3, 8, 4, 64, 32, device="cpu")
    slots = torch.zeros(2, dtype=torch.int64)
    table, cu, lens = torch.zeros(1, 3, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)
    attend = lambda c=c, **kw: q.qlinear_paged_attention_4bit(k, c, table, cu, lens, max_q=2, **kw)  # noqa: E731
    bad = [lambda: q.qlinear_paged_cache_4bit(3, 8, 4, 64, 128, device="cpu"), lambda: q.qlinear_paged_cache_4bit(3, 8, 4, 64, 16, device="cpu"),
           lambda: attend(out=k[:1]), lambda: attend(sinks=torch.zeros(3)), lambda: q.qlinear_kv_append_4bit(k, k[:1], c, slots),
           lambda: q.qlinear_kv_append_4bit(k, k, c, slots.int()), lambda: q.qlinear_kv_append_4bit(k, k.half(), c, slots),
           lambda: q.qlinear_kv_read_4bit(c, slots, k_out=k.half(), v_out=k), lambda: q.qlinear_kv_read_4bit(c, slots.int())]
    wide = q.qlinear_paged_cache_4bit(3, 8, 4, 128, 32, device="cpu")
    odd = [c[:3], (c[0].float(), *c[1:]), (c[0], c[1].float(), *c[2:]), (c[0][:2], *c[1:]), (c[0], c[1][..., :1], *c[2:]),
           (c[0], c[1][:, :4], *c[2:]), (c[0].contiguous(), *c[1:]), wide]
    for x in odd:
        bad += [lambda x=x: q.qlinear_kv_append_4bit(k, k, x, slots), lambda x=x: attend(x)]
    step = dict(page_size=8, rows=4)
    bad += [lambda: q.qlinear_kv_extend(lens.long(), lens, table, **step), lambda: q.qlinear_kv_extend(lens, cu, table, **step),
            lambda: q.qlinear_kv_extend(lens, lens, table.long(), **step), lambda: q.qlinear_kv_extend(lens, lens, table, free_pages=cu, free_count=cu, **step),
            lambda: q.qlinear_kv_extend(lens, lens, table, positions=torch.zeros(3, dtype=torch.int64), **step)]
    x = torch.zeros(2, 8)
    bad += [lambda: q.qlinear_select_experts(x[0], 2), lambda: q.qlinear_select_experts(x.t(), 2), lambda: q.qlinear_select_experts(x.double(), 2),
            lambda: q.qlinear_select_experts(x, 2, bias=x[0, :4]), lambda: q.qlinear_select_experts(x, 2, ids=torch.zeros(2, 2, **i32)),
            lambda: q.qlinear_combine_experts(x, x[:, :2]), lambda: q.qlinear_combine_experts(x, torch.zeros(1, 2), residual=x),
            lambda: q.qlinear_combine_experts(x, torch.zeros(1, 2).double()), lambda: q.qlinear_combine_experts(x, torch.zeros(1, 2), out=torch.zeros(1, 8).half())]
    for i, f in enumerate(bad):
        with pytest.raises(q.QLError) as e:
            f()
        assert "one GPU" not in str(e.value), i


def test_binding_refuses_host_memory():
    k, i32 = torch.zeros(2, 4, 64, dtype=torch.bfloat16), dict(dtype=torch.int32)
    c, slots = q.qlinear_paged_cache_4bit(3, 8, 4, 64, 32, device="cpu"), torch.zeros(2, dtype=torch.int64)
    for bad in (lambda: q.qlinear_kv_append_4bit(k, k, c, slots), lambda: q.qlinear_kv_read_4bit(c, slots),
                lambda: q.qlinear_paged_attention_4bit(k, c, torch.zeros(1, 3, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32), max_q=2),
                lambda: q.qlinear_kv_extend(torch.zeros(1, **i32), torch.zeros(1, **i32), torch.zeros(1, 3, **i32), page_size=8, rows=2),
                lambda: q.qlinear_select_experts(torch.zeros(2, 8), 2), lambda: q.qlinear_combine_experts(torch.zeros(4, 8), torch.zeros(2, 2))):
        with pytest.raises(q.QLError, match="one GPU"):
            bad()


def test_matrix_results_are_first_read_by_the_compilers_own_instruction():
    """The running maximum over scores (inline max3) begins with fmaxf of a value of each product, which the
    compiler waits for, and every step depends on it."""
    with open(os.path.join(os.path.dirname(q.lib_path()), "..", "csrc", "attn_few4.hip")) as f:
        text = f.read()
    first = re.findall(r"float mx = (.*);", text)
    assert len(first) == 1 and first[0].startswith("fmaxf(") and all(f"sc[n][{i}]" in first[0] for i in range(4)), first
    steps = [m for m in re.findall(r"max3\(([^;]*);", text) if "sc[" in m]
    assert steps and all(m.startswith(("mx,", "max3(mx,")) for m in steps), steps
    assert not re.search(r"asm[^;]*\bsc\[", text)
