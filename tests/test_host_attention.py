"""Refusals of the attention-side entry points, on the host before any launch (no GPU)."""
import ctypes
import os

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
    a = dict(k=FAKE, v=FAKE, n_pages=4, page_size=16, hk=8, d=128, page_stride=16 * 1024, token_stride=1024,
             head_stride=128)
    a.update(kw)
    return q._PagedCache(**a)


def nrope(**kw):
    a = dict(q_weight=FAKE, k_weight=FAKE, w_dtype=BF16, eps=1e-6, positions=FAKE, cos_sin=FAKE, max_pos=64, rot=128,
             interleaved=0)
    a.update(kw)
    return q._NormRope(**a)


def ref(s):
    return None if s is None else ctypes.addressof(s)


def norm(lib, qh=None, qo=None, k=None, ko=None, dtype=BF16, t=2, d=128, nr=None):
    return lib.qlinear_qk_norm_rope(ref(qh), ref(qo), ref(k), ref(ko), dtype, t, d, ref(nr), None)


def test_norm_rope_refusals(lib):
    h, n = heads(), nrope()
    assert norm(lib, h, h, h, h, dtype=F32, nr=n) == DTYPE
    assert norm(lib, h, h, h, h, nr=None) == NULL
    assert norm(lib, h, None, h, h, nr=n) == NULL
    assert b"q_out" in lib.qlinear_last_error()
    assert norm(lib, h, h, h, None, nr=n) == NULL
    assert norm(lib, heads(p=None), h, h, h, nr=n) == NULL
    assert norm(lib, heads(p=FAKE + 8), h, h, h, nr=n) == ALIGN
    assert norm(lib, heads(ts=1028), h, h, h, nr=n) == ALIGN
    assert norm(lib, heads(hs=-128), h, h, h, nr=n) == ALIGN
    assert norm(lib, h, heads(n=4), h, h, nr=n) == SHAPE
    assert norm(lib, h, h, heads(n=-1), h, nr=n) == SHAPE
    assert norm(lib, h, h, h, h, t=-1, nr=n) == SHAPE
    for d in (0, 12, 520, -8):
        assert norm(lib, h, h, h, h, d=d, nr=n) == UNSUPPORTED
    for bad in (dict(rot=8), dict(rot=144), dict(rot=-16), dict(max_pos=0), dict(max_pos=-1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf"))):
        assert norm(lib, h, h, h, h, nr=nrope(**bad)) == SHAPE, bad
    assert norm(lib, h, h, h, h, nr=nrope(w_dtype=7)) == DTYPE
    assert norm(lib, h, h, h, h, nr=nrope(q_weight=FAKE + 2)) == ALIGN
    assert norm(lib, h, h, h, h, nr=nrope(positions=FAKE + 4)) == ALIGN
    assert norm(lib, h, h, h, h, nr=nrope(cos_sin=FAKE + 4)) == ALIGN
    assert norm(lib, h, h, h, h, nr=nrope(positions=None)) == NULL
    assert norm(lib, h, h, h, h, nr=nrope(cos_sin=None)) == NULL
    assert norm(lib, h, h, h, h, t=(1 << 31), nr=n) == UNSUPPORTED


def test_norm_rope_nothing_to_do(lib):
    h = heads()
    assert norm(lib, h, h, h, h, t=0, nr=nrope(positions=None, cos_sin=None)) == OK
    assert norm(lib, None, None, None, None, nr=nrope()) == OK
    assert norm(lib, heads(n=0), None, heads(n=0, p=None), None, nr=nrope()) == OK
    assert lib.qlinear_last_error() == b""


def append(lib, qh=None, qo=None, k=None, v=None, c=None, slots=FAKE, dtype=BF16, t=2, nr=None):
    return lib.qlinear_kv_append(ref(qh), ref(qo), ref(k), ref(v), ref(c), slots, dtype, t, ref(nr), None)


def test_kv_append_refusals(lib):
    h, n, c = heads(), nrope(), cache()
    assert append(lib, k=h, v=h, c=c, dtype=F32, nr=n) == DTYPE
    assert append(lib, k=h, v=h, c=None, nr=n) == NULL
    assert append(lib, k=None, v=h, c=c, nr=n) == NULL
    assert append(lib, k=h, v=None, c=c, nr=n) == NULL
    assert append(lib, k=h, v=h, c=c, slots=None, nr=n) == NULL
    assert append(lib, k=h, v=h, c=c, slots=FAKE + 4, nr=n) == ALIGN
    assert append(lib, k=heads(n=4), v=h, c=c, nr=n) == SHAPE
    assert append(lib, k=h, v=heads(n=4), c=c, nr=n) == SHAPE
    assert append(lib, qh=h, qo=None, k=h, v=h, c=c, nr=n) == NULL
    for bad, st in ((dict(k=None), NULL), (dict(v=FAKE + 2), ALIGN), (dict(page_size=0), SHAPE), (dict(n_pages=-1), SHAPE),
                    (dict(hk=0), SHAPE), (dict(token_stride=4), ALIGN), (dict(page_stride=-8), ALIGN),
                    (dict(n_pages=1 << 28), UNSUPPORTED), (dict(d=100), UNSUPPORTED)):
        assert append(lib, k=h, v=h, c=cache(**bad), nr=n) == st, bad
    assert append(lib, k=h, v=h, c=c, t=0, slots=None, nr=n) == OK


def attend(lib, qh=None, out=None, dtype=BF16, t=2, c=None, table=FAKE, stride=4, pages=4, cu=FAKE, lens=FAKE, n=1,
           max_q=2, scale=0.1, window=0, sinks=None, ws=FAKE, ws_bytes=1 << 40):
    return lib.qlinear_paged_attention(ref(qh), ref(out), dtype, t, ref(c), table, stride, pages, cu, lens, n, max_q,
                                       scale, window, sinks, ws, ws_bytes, None)


def test_paged_attention_refusals(lib):
    h, c = heads(n=16, ts=2048), cache()
    ok = dict(qh=h, out=h, c=c)
    for bad, st in ((dict(dtype=F32), DTYPE), (dict(c=None), NULL), (dict(qh=None), NULL), (dict(out=None), NULL),
                    (dict(c=cache(d=96)), UNSUPPORTED), (dict(qh=heads(n=12)), SHAPE), (dict(out=heads(n=8)), SHAPE),
                    (dict(t=-1), SHAPE), (dict(n=-1), SHAPE), (dict(max_q=-1), SHAPE), (dict(pages=-1), SHAPE),
                    (dict(stride=-1), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE),
                    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(window=-1), SHAPE),
                    (dict(cu=None), NULL), (dict(lens=None), NULL), (dict(table=None), NULL), (dict(cu=FAKE + 2), ALIGN),
                    (dict(sinks=FAKE + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws_bytes=64), WORKSPACE),
                    (dict(ws=FAKE + 4), ALIGN), (dict(pages=1 << 28), UNSUPPORTED), (dict(t=1 << 30), UNSUPPORTED),
                    (dict(qh=heads(p=None, n=16)), NULL), (dict(qh=heads(n=16, ts=4)), ALIGN)):
        assert attend(lib, **{**ok, **bad}) == st, bad
    for nothing in (dict(t=0), dict(n=0), dict(max_q=0)):
        assert attend(lib, **{**ok, **nothing, "ws": None}) == OK


def test_paged_attention_workspace_size(lib):
    size = lib.qlinear_paged_attention_workspace_size
    assert size(0, 1, 16, 8, 128, 1, 4, 16, 0) == 0
    assert size(1, 1, 16, 5, 128, 1, 4, 16, 0) == 0
    few, many = size(4, 4, 16, 8, 128, 1, 64, 16, 0), size(300, 1, 16, 8, 128, 300, 64, 16, 0)
    assert 0 < few < many
    h = heads(n=16, ts=2048)
    assert attend(lib, qh=h, out=h, c=cache(), t=4, n=4, max_q=1, pages=64, ws_bytes=few - 1) == WORKSPACE


def test_binding_refuses_wrong_tensors():
    bf = torch.bfloat16
    k = torch.zeros(2, 4, 64, dtype=bf)
    kc = torch.zeros(3, 8, 4, 64, dtype=bf)
    slots = torch.zeros(2, dtype=torch.int64)
    for bad in (lambda: q.qlinear_kv_append(k, k, kc, kc.half(), slots), lambda: q.qlinear_kv_append(k, k, kc.half(), kc.half(), slots),
                lambda: q.qlinear_kv_append(k, k, kc, kc.transpose(1, 2).contiguous().transpose(1, 2), slots),
                lambda: q.qlinear_kv_append(k, k[:1], kc, kc, slots), lambda: q.qlinear_kv_append(k, k, kc, kc, slots.int()),
                lambda: q.qlinear_kv_append(k, k, kc, kc, slots[:1]),
                lambda: q.qlinear_kv_append(k, k, kc, kc, slots, q_weight=torch.zeros(32, dtype=bf)),
                lambda: q.qlinear_kv_append(k, k, kc, kc, slots, cos_sin=torch.zeros(4, 64).double()),
                lambda: q.qlinear_kv_append(k.transpose(1, 2), k, kc, kc, slots),
                lambda: q.qlinear_qk_norm_rope(k, k.half()), lambda: q.qlinear_qk_norm_rope(None, None),
                lambda: q.qlinear_qk_norm_rope(k, None, q_out=torch.zeros(1, 4, 64, dtype=bf))):
        with pytest.raises(q.QLError):
            bad()
    table, cu, lens = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for bad in (lambda: q.qlinear_paged_attention(k, kc, kc, table.long(), cu, lens, max_q=2),
                lambda: q.qlinear_paged_attention(k, kc, kc, table, cu[:1], lens, max_q=2),
                lambda: q.qlinear_paged_attention(k, kc, kc, table, cu, lens.long(), max_q=2),
                lambda: q.qlinear_paged_attention(k, kc, kc, table, cu, lens, max_q=2, sinks=torch.zeros(3)),
                lambda: q.qlinear_paged_attention(k, kc, kc, table, cu, lens, max_q=2, out=k[:1]),
                lambda: q.qlinear_paged_attention(k.half(), kc, kc, table, cu, lens, max_q=2)):
        with pytest.raises(q.QLError):
            bad()


def test_binding_refuses_host_memory():
    k, kc = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 8, 4, 64, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    for bad in (lambda: q.qlinear_qk_norm_rope(k, k), lambda: q.qlinear_kv_append(k, k, kc, kc, torch.zeros(2, dtype=torch.int64)),
                lambda: q.qlinear_paged_attention(k, kc, kc, torch.zeros(1, 3, **i32), torch.zeros(2, **i32),
                                                  torch.zeros(1, **i32), max_q=2)):
        with pytest.raises(q.QLError, match="one GPU"):
            bad()


def test_work_past_64_bits_is_refused_and_any_window_is_planned(lib):
    size = lib.qlinear_paged_attention_workspace_size
    big = (1 << 63) - 1
    for args in ((2, 1, 16, 8, 128, 2), (80, 16, 32, 8, 128, 5), (4000, 3, 8, 8, 256, 4000), (9, 9, 4, 4, 64, 1)):
        none = size(*args, 64, 16, 0)
        assert none > 0
        for window in (64 * 16, 1 << 40, big - 1, big):  # windows over the whole cache
            assert size(*args, 64, 16, window) == none, (args, window)
    # units of work past 2^31, 2^63 and 2^64: refused, whatever the products wrap to
    h = heads(n=1 << 19, ts=1 << 26)
    c = cache(n_pages=0, k=None, v=None, hk=1 << 19, page_size=1)
    for n in ((1 << 13), (1 << 20), (1 << 24) + 1, (1 << 26), (1 << 29)):
        for pages in (1 << 12, 1 << 21, (1 << 30) - 1):
            for t, max_q in ((n, 1), (min(4 * n, (1 << 30) - 1), 100)):
                assert attend(lib, qh=h, out=h, c=c, t=t, n=n, max_q=max_q, pages=pages, ws_bytes=(1 << 63)) == UNSUPPORTED, (n, pages, t)
                assert size(t, n, 1 << 19, 1 << 19, 128, max_q, pages, 1, 0) < (1 << 40)


def test_matrix_results_are_first_read_by_the_compilers_own_instruction():
    """The wait between a matrix product and the reader of its result is put in for instructions that the
    compiler knows, not for inline ones.  Each running maximum over the scores (inline max3) therefore
    begins with fmaxf of a value of the first and of the last product, and every step depends on it."""
    import re

    csrc = os.path.join(os.path.dirname(q.lib_path()), "..", "csrc")
    for name, last in (("attn_few.hip", "sc[n][1]"), ("attn_tile.hip", "sc[NK - 1]")):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        first = re.findall(r"float mx = (.*);", text)
        assert len(first) == 1 and first[0].startswith("fmaxf(sc") and last in first[0], (name, first)
        steps = [m for m in re.findall(r"max3\(([^;]*);", text) if "sc[" in m]
        assert steps and all(m.startswith("mx,") for m in steps), (name, steps)
        assert not re.search(r"asm[^;]*\bsc\[", text)
