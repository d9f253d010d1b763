"""Pins of the oracle of the 4-bit cache's and the experts' operators: small cases worked out by hand."""
import numpy as np

from oracle import decoder_oracle as D
from oracle import qlinear_oracle as O


def test_a_group_of_levels_is_kept_exactly():
    row = np.full((1, 32), 2.0, dtype=np.float32)
    row[0, :16] = 2.0 + 0.25 * np.arange(16)
    words, groups = D.quantize_rows(row, 32)
    assert groups.tolist() == [[[0.25, 2.0]]]
    assert words[0, 0] == 0x76543210 and words[0, 1] == 0xFEDCBA98 and (words[0, 2:] == 0).all()
    assert np.array_equal(D.row_values(words, groups), row)


def test_groups_are_those_of_the_weights_quantizer():
    rows = np.random.default_rng(0).standard_normal((3, 2, 128)).astype(np.float32)
    words, groups = D.quantize_rows(rows, 64)
    w, s, b = O.affine_quantize(rows.reshape(6, 128), 4, 64, "f16")
    assert np.array_equal(words.reshape(6, 16), w)
    assert np.array_equal(groups.reshape(6, 2, 2)[..., 0].view(np.uint16), s)
    assert np.array_equal(groups.reshape(6, 2, 2)[..., 1].view(np.uint16), b)
    assert np.array_equal(D.row_values(words, groups).reshape(6, 128).astype(np.float32), O.affine_dequant_f32(w, s, b, 4, 64, "f16", 128))


def test_magnitudes_that_are_not_held():
    row = np.zeros((4, 64), dtype=np.float32)
    row[0, 3], row[1, 40], row[2, 0], row[3, 0] = np.nan, np.inf, 32769, -32768
    words, groups = D.quantize_rows(row, 32)
    assert np.isnan(groups[:3, :, 1]).tolist() == [[True, False], [False, True], [True, False]]
    assert (groups[:3, :, 0] == 0).all() and (words[:3] == 0).all()
    assert groups[3, 0].tolist() == [2184.0, -32768.0] and D.row_values(words, groups)[3, 1] == -8.0


def test_extend_by_hand():
    # pages of 4: 3 tokens and one page; through with two pages; empty
    cu, pos, slots, lens, table, stack, info = D.kv_extend([2, -1, 1], [3, 5, 0], [[7, -1], [8, 9], [-1, -1]], 4, 5, ([1, 2], 6))
    assert cu == [0, 2, 2, 3] and pos == [3, 4, 0, 0, 0] and slots == [31, 36, 32, -1, -1]
    assert lens == [5, 0, 1] and table == [[7, 9], [8, 9], [8, -1]] and stack == [1, 2] and info == [3, 2, 0, 2]


def test_extend_refused_by_hand():
    base = dict(counts=[2], lens=[3], table=[[7, -1]], page=4, rows=5)
    assert D.kv_extend(**base, free=([], 4))[6] == [0, 0, 2, 0]
    assert D.kv_extend(**{**base, "rows": 1}, free=([1], 4))[6] == [0, 0, 1, 1]
    assert D.kv_extend(**{**base, "counts": [6]}, free=([1], 4))[6] == [0, 0, 4, 1]
    assert D.kv_extend([-1], [8], [[7, 8]], 4, 5, ([1], 2))[6] == [0, 0, 8, 1]
    assert D.kv_extend(**base)[6] == [2, 0, 0, 0]


def test_select_by_hand():
    x = np.log(np.array([[1.0, 4.0, 2.0, 4.0, 1.0, 4.0]]))
    ids, w = D.select_experts(x, 3)
    assert ids.tolist() == [[1, 3, 5]] and np.allclose(w, 1 / 3)
    ids, w = D.select_experts(x, 2, n_groups=3, top_groups=1, group_top=2, renormalize=False, scale=2.0)
    assert ids.tolist() == [[3, 2]] and np.allclose(w, [[0.5, 0.25]])
    ids, w = D.select_experts(x, 1, sigmoid=True, bias=np.array([0, 0, 0.5, 0, 0, 0]), renormalize=False)
    assert ids.tolist() == [[2]] and np.allclose(w, 2 / 3)
    inf = np.inf
    ids, w = D.select_experts(np.array([[-inf, np.nan, -inf], [0, inf, inf]]), 2)
    assert ids.tolist() == [[0, 1], [1, 2]] and w.tolist() == [[0, 0], [0.5, 0.5]]


def test_combine_by_hand():
    y = np.array([[1.0, 2.0], [np.nan, 3.0], [5.0, 6.0], [7.0, 8.0]])
    out, mag = D.combine_experts(y, np.array([[2.0, 9.0], [1.0, -1.0]]), np.array([[0, -1], [1, 0]]), 2, np.array([[1.0, 1.0], [0.0, 0.0]]))
    assert out.tolist() == [[3.0, 5.0], [-2.0, -2.0]] and mag.tolist() == [[3.0, 5.0], [12.0, 14.0]]
