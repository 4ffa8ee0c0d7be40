"""Pins of the oracle's encoder-state operators: hand-worked rotations and weights, closed
forms, and agreement with the oracles of the other paths."""
import numpy as np
import pytest

import oracle


def test_rotation_by_hand():
    half_pi = np.float32(np.pi / 2)
    pos = np.array([[1, 0], [0, 2]])
    x = np.array([1.0, 2, 3, 4, 5]).reshape(1, 1, 5).repeat(2, 0)
    freq, axis = np.array([half_pi, half_pi]), [0, 1]
    got = oracle.rope_axes(x, pos, freq, axis, False)  # pairs (1, 3) by axis 0, (2, 4) by axis 1
    assert np.allclose(got[0, 0], [-3, 2, 1, 4, 5], atol=1e-6)   # a quarter, nothing
    assert np.allclose(got[1, 0], [1, -2, 3, -4, 5], atol=1e-6)  # nothing, a half
    got = oracle.rope_axes(x, pos, freq, axis, True)  # pairs (1, 2), (3, 4)
    assert np.allclose(got[0, 0], [-2, 1, 3, 4, 5], atol=1e-6)
    assert np.allclose(got[1, 0], [1, 2, -3, -4, 5], atol=1e-6)
    back = oracle.rope_axes(got, pos, freq, axis, True, inverse=True)
    assert np.allclose(back, x, atol=1e-12)


def test_rotation_with_one_axis_is_the_table_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, 2, 16))
    pos = rng.integers(0, 1000, 6)
    freq = (10000.0 ** (-np.arange(6) / 6)).astype(np.float32)
    ang = np.arange(1000)[:, None] * freq.astype(np.float64)
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for inter in (False, True):
        want = oracle.rotate(x, table, pos, inter)
        assert np.allclose(oracle.rope_axes(x, pos[None], freq, [0] * 6, inter), want, atol=1e-12)


def test_rotation_of_far_positions_is_exact():
    # angle p f mod 2 pi against the sum of doublings: e^(i 2a) = (e^(i a))^2
    f = np.float32(0.7390851)
    x = np.zeros((1, 1, 2))
    x[..., 0] = 1.0
    z = complex(np.cos(float(f)), np.sin(float(f)))
    for e in range(1, 21):
        z = z * z
        z /= abs(z)
        got = oracle.rope_axes(x, np.array([[2 ** e]]), [f], [0], False)[0, 0]
        assert abs(complex(*got) - z) < 1e-9


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_cross_attention_is_the_window_oracle_where_lengths_agree(mode):
    rng = np.random.default_rng(mode)
    cu, H, Hkv, d = np.array([0, 5, 12, 12, 13], np.int32), 4, 2, 64
    q, k, v = (rng.standard_normal((13, h, d)).astype(np.float32) for h in (H, Hkv, Hkv))
    sinks = rng.standard_normal(H).astype(np.float32)
    wo, wl = oracle.window(q, k, v, cu, H, Hkv, d, -1, -1, 0, sinks if mode else None, mode, 0.125)
    o, lse = oracle.cross_attend(q, k, v, cu, cu[:-1], np.diff(cu), sinks, mode, 0.125)
    assert np.allclose(o, wo.reshape(o.shape), atol=1e-12)
    assert np.allclose(lse, wl.reshape(lse.shape), atol=1e-12)


def test_cross_attention_counts_states():
    # q = 0: the mean of the values, lse = ln of their number, whatever the query count
    rng = np.random.default_rng(3)
    v = rng.standard_normal((9, 1, 4))
    o, lse = oracle.cross_attend(np.zeros((3, 2, 4)), np.ones((9, 1, 4)), v, [0, 2, 3, 3],
                                 [4, 0, 0], [5, 0, 3], [0.0, 1.0], 2, 1.0)
    assert np.allclose(o[0, 0], v[4:9, 0].sum(0) / 6) and np.allclose(lse[0, 0], np.log(6))
    assert np.allclose(lse[1, 1], np.log(5 + np.e))
    assert np.all(o[2] == 0) and np.allclose(lse[2], [0.0, 1.0])  # no states: the sink alone
    o, lse = oracle.cross_attend(np.zeros((1, 1, 4)), v, v, [0, 1], [0], [0], None, 0, 1.0)
    assert np.all(o == 0) and np.isneginf(lse).all()


def test_key_weights_add_up_to_the_rows():
    rng = np.random.default_rng(4)
    H, Hkv, d = 6, 2, 8
    q, k = rng.standard_normal((7, H, d)), rng.standard_normal((20, Hkv, d))
    cu, st, ln = [0, 3, 3, 7], [0, 6, 11], [6, 5, 9]
    _, lse = oracle.cross_attend(q, k, k, cu, st, ln, None, 0, 0.3)
    w = oracle.cross_key_weights(q, k, lse, cu, st, ln, np.full((Hkv, 20), 2.0), False, None, 0, 0.3)
    for b in range(3):
        n = cu[b + 1] - cu[b]
        assert np.allclose(w[:, st[b]:st[b] + ln[b]].sum(1), n * H // Hkv)
    twice = oracle.cross_key_weights(q, k, lse, cu, st, ln, w, True, None, 0, 0.3)
    assert np.allclose(twice, 2 * w)


def test_key_weights_with_sinks():
    # q = 0, 3 keys: weight 1 / (3 + e^s) each with a null logit; key 0 e^s times the others'
    q, k, s = np.zeros((1, 1, 4)), np.ones((3, 1, 4)), 0.7
    _, lse = oracle.cross_attend(q, k, k, [0, 1], [0], [3], [s], 2, 1.0)
    w = oracle.cross_key_weights(q, k, lse, [0, 1], [0], [3], np.zeros((1, 3)), False, [s], 2, 1.0)
    assert np.allclose(w, 1 / (3 + np.exp(s)))
    _, lse = oracle.cross_attend(q, k, k, [0, 1], [0], [3], [s], 1, 1.0)
    w = oracle.cross_key_weights(q, k, lse, [0, 1], [0], [3], np.zeros((1, 3)), False, [s], 1, 1.0)
    assert np.allclose(w, np.array([[np.exp(s), 1, 1]]) / (2 + np.exp(s)))


def test_eviction_by_hand():
    w = np.array([[0.1, 5, 2, 2, 0, 3, 2, np.nan, -1, 9]])
    assert oracle.evict_keys(w, [0], [10], 4, 0, 0).tolist() == [[1, 2, 5, 9]]   # 2 ties: lowest
    assert oracle.evict_keys(w, [0], [10], 4, 1, 2).tolist() == [[0, 1, 8, 9]]   # protected ends
    assert oracle.evict_keys(w, [0], [10], 9, 0, 0).tolist() == [[0, 1, 2, 3, 4, 5, 6, 7, 9]]
    assert oracle.evict_keys(w, [2, 0], [3, 0], 4, 1, 1).tolist() == [[0, 1, 2] + [-1] * 5]
