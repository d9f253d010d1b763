"""The oracle of the attention-side operators against closed forms (no GPU)."""
import numpy as np
import pytest

from oracle import attention_oracle as A


def test_norm_alone_gives_unit_mean_square():
    x = np.random.default_rng(1).normal(size=(3, 2, 16))
    y, _ = A.norm_rope(x, np.ones(16), 0.0, None, None, False)
    assert np.allclose((y * y).mean(-1), 1.0)
    w = np.linspace(-1, 1, 16)
    assert np.allclose(A.norm_rope(x, w, 0.0, None, None, False)[0], y * w)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    r = np.random.default_rng(2)
    t, d, rot = 5, 24, 16
    x = r.normal(size=(t, 1, d))
    pos = np.array([0, 3, 7, 1, 2])
    ang = np.arange(8)[:, None] * 0.37 ** np.arange(rot // 2)[None]
    tab = np.concatenate([np.cos(ang), np.sin(ang)], axis=1)
    y, _ = A.norm_rope(x, None, 0.0, pos, tab, interleaved)
    pair = (lambda z: z[..., 0:rot:2] + 1j * z[..., 1:rot:2]) if interleaved else (
        lambda z: z[..., :rot // 2] + 1j * z[..., rot // 2:rot])
    assert np.allclose(pair(y[:, 0]), pair(x[:, 0]) * np.exp(1j * ang[pos]))
    assert np.array_equal(y[..., rot:], x[..., rot:])


def test_positions_outside_the_table_give_zero_rows():
    x = np.ones((3, 1, 16))
    tab = np.concatenate([np.ones((4, 8)), np.zeros((4, 8))], axis=1)
    y, _ = A.norm_rope(x, None, 0.0, np.array([-1, 3, 4]), tab, False)
    assert (y[0] == 0).all() and (y[1] == 1).all() and (y[2] == 0).all()


def test_attention_equal_scores_average_what_is_seen():
    kv, page = 11, 4
    kc, vc = np.zeros((3, page, 1, 2)), np.arange(24.0).reshape(3, page, 1, 2)
    table = np.array([[2, 0, 1]])
    seq = np.concatenate([vc[2, :, 0], vc[0, :, 0], vc[1, :, 0]])[:kv]
    q = np.random.default_rng(0).normal(size=(3, 1, 2))
    out, _, _ = A.paged_attention(q, kc, vc, table, [0, 3], [kv], 1.0)
    for i in range(3):
        assert np.allclose(out[i, 0], seq[:kv - 2 + i].mean(0))
    out, _, _ = A.paged_attention(q, kc, vc, table, [0, 3], [kv], 1.0, window=2)
    for i in range(3):
        assert np.allclose(out[i, 0], seq[kv - 4 + i:kv - 2 + i].mean(0))
    out, _, _ = A.paged_attention(q, kc, vc, table, [0, 3], [kv], 1.0, sinks=np.array([np.log(5.0)]))
    assert np.allclose(out[0, 0], seq[:kv - 2].sum(0) / (kv - 2 + 5))


def test_attention_rows_that_see_nothing_are_zero():
    kc = vc = np.ones((2, 4, 1, 2))
    q = np.ones((4, 1, 2))
    out, _, _ = A.paged_attention(q, kc, vc, np.array([[0], [-1]]), [0, 3, 4], [1, 3], 1.0)
    assert (out[:2] == 0).all() and (out[2] == 1).all() and (out[3] == 0).all()


def test_append_skips_slots_out_of_range():
    cache = np.zeros((2, 3, 1, 1))
    out = A.kv_append(cache, np.arange(1.0, 5.0).reshape(4, 1, 1), [4, -1, 6, 0])
    assert out.reshape(-1).tolist() == [4, 0, 0, 0, 1, 0]


def test_infinite_sinks_are_no_term_and_no_weight():
    r = np.random.default_rng(4)
    kc, vc = r.normal(size=(2, 4, 1, 2)), r.normal(size=(2, 4, 1, 2))
    q = r.normal(size=(3, 2, 2))
    args = (q, kc, vc, np.array([[1, 0]]), [0, 3], [6], 0.7)
    out, _, _ = A.paged_attention(*args, sinks=np.array([-np.inf, np.inf]))
    assert np.array_equal(out[:, 0], A.paged_attention(*args)[0][:, 0]) and (out[:, 1] == 0).all()
