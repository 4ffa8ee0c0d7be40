"""Pins of the oracle's paged FP8 cache: hand-worked scales and rotations, the
append against one-shot quantisation and its recoding rule, the attention
against closed forms and the window oracle."""
import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("amax,s", [
    (0.0, 2.0 ** -64), (448.0, 1.0), (448.1, 2.0), (224.0, 0.5), (3.5, 2.0 ** -7),
    (3.6, 2.0 ** -6), (1e-30, 2.0 ** -64), (float("inf"), 2.0 ** 120)])
def test_scale_by_hand(amax, s):
    assert float(oracle.pow2_scale(amax)) == s


def test_rotation_by_hand():
    cs = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 0.6, 1.0, 0.8]])  # angles 0; pi/2 and 0.6/0.8
    x = np.arange(1.0, 6.0).reshape(1, 1, 5)
    assert np.array_equal(oracle.rotate(x, cs, np.array([0]), False), x)
    half = oracle.rotate(x, cs, np.array([1]), False)[0, 0]  # pairs (1, 3), (2, 4)
    assert np.allclose(half, [-3, 2 * 0.6 - 4 * 0.8, 1, 4 * 0.6 + 2 * 0.8, 5])
    inter = oracle.rotate(x, cs, np.array([1]), True)[0, 0]  # pairs (1, 2), (3, 4)
    assert np.allclose(inter, [-2, 1, 3 * 0.6 - 4 * 0.8, 4 * 0.6 + 3 * 0.8, 5])


def test_rotation_keeps_relative_angles():
    rng = np.random.default_rng(0)
    ang = np.arange(40)[:, None] * np.array([[1.0, 0.1, 0.01, 0.001]])
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    q, k = rng.standard_normal((2, 1, 1, 8))
    for inter in (False, True):
        a = np.sum(oracle.rotate(q, cs, np.array([30]), inter)
                   * oracle.rotate(k, cs, np.array([25]), inter))
        b = np.sum(oracle.rotate(q, cs, np.array([7]), inter)
                   * oracle.rotate(k, cs, np.array([2]), inter))
        assert abs(a - b) < 1e-12


def _cache(pages, Hkv, page, d):
    return np.full((pages, Hkv, page, d), 0x55, np.uint8), np.full((pages, Hkv), 7.0, np.float32)


def test_append_a_prompt_page_by_page():
    rng = np.random.default_rng(1)
    page, d = 4, 8
    x = rng.standard_normal((6, 2, d)) * 30
    codes, scale = _cache(3, 2, page, d)
    c, s = oracle.paged_append(x, codes, scale, [[2, 0]], [0, 6], [6])
    for j, pid, m in ((0, 2, 4), (1, 0, 2)):
        for h in range(2):
            part = x[j * page: j * page + m, h]
            want = float(oracle.pow2_scale(np.abs(part).max()))
            assert s[pid, h] == want
            err = np.abs(oracle.e4m3_decode(c[pid, h, :m]) * want - part)
            assert np.all(err <= 2.0 ** -4 * np.abs(part) + 2.0 ** -10 * want)
    assert np.array_equal(c[0, :, 2:], codes[0, :, 2:])  # rows behind the last token
    assert np.array_equal(c[1], codes[1]) and np.array_equal(s[1], scale[1])


def test_later_tokens_recode_the_page():
    page, d = 4, 2
    codes, scale = _cache(1, 1, page, d)
    a = np.array([[[448.0, 1.0]]])
    b = np.array([[[-3584.0, 0.0]]])  # 8 times the first row's largest value
    c, s = oracle.paged_append(a, codes, scale, [[0]], [0, 1], [1])
    assert s[0, 0] == 1.0 and list(oracle.e4m3_decode(c[0, 0, 0])) == [448.0, 1.0]
    c, s = oracle.paged_append(b, c, s, [[0]], [0, 1], [2])
    assert s[0, 0] == 8.0
    assert list(oracle.e4m3_decode(c[0, 0, 0])) == [56.0, 0.125]
    assert list(oracle.e4m3_decode(c[0, 0, 1])) == [-448.0, 0.0]
    c2, s2 = oracle.paged_append(b, c, s, [[0]], [0, 1], [2])  # again: nothing changes
    assert np.array_equal(c, c2) and np.array_equal(s, s2)
    c3, s3 = oracle.paged_append(a / 1024, c, s, [[0]], [0, 1], [3])  # smaller: scale kept
    assert s3[0, 0] == 8.0 and np.array_equal(c3[0, 0, :2], c[0, 0, :2])


def test_attention_with_equal_logits_counts_the_visible_keys():
    rng = np.random.default_rng(2)
    page, d, L, n = 4, 4, 11, 3
    kc = oracle.e4m3_encode(rng.standard_normal((3, 1, page, d)))
    vc = oracle.e4m3_encode(rng.standard_normal((3, 1, page, d)))
    ks, vs = np.ones((3, 1), np.float32), np.array([[1.0], [2.0], [0.5]], np.float32)
    table = [[1, 2, 0]]
    v = np.concatenate([oracle.e4m3_decode(vc[p, 0]) * vs[p, 0] for p in table[0]])
    q = np.zeros((n + 1, 2, d))
    for w in (-1, 2):
        o, lse = oracle.paged_attend(q, kc, vc, ks, vs, table, [0, n], [L], 1, w, None, 0, 0.5)
        for i in range(n):
            lo = 0 if w < 0 else max(0, L - n + i - w)
            rows = v[lo: L - n + i + 1]
            assert np.allclose(o[i], rows.mean(0)) and np.allclose(lse[i], np.log(len(rows)))
    assert np.all(np.isnan(o[n]))  # behind the last sequence
    s = np.array([0.3, -1.0])
    o2, lse2 = oracle.paged_attend(q, kc, vc, ks, vs, table, [0, n], [L], 1, -1, s, 2, 0.5)
    assert np.allclose(np.exp(lse2[:n]), 9 + np.arange(n)[:, None] + np.exp(s)[None])
    o1, lse1 = oracle.paged_attend(q, kc, vc, ks, vs, table, [0, n], [L], 1, -1, s, 1, 0.5)
    assert np.allclose(np.exp(lse1[:n]), 8 + np.arange(n)[:, None] + np.exp(s)[None])


def test_attention_matches_the_window_oracle():
    """One sequence, all of it new, unit scales: the windowed oracle on the decoded rows."""
    rng = np.random.default_rng(3)
    page, d, L, H, Hkv = 16, 64, 37, 4, 2
    kc = oracle.e4m3_encode(rng.standard_normal((3, Hkv, page, d)))
    vc = oracle.e4m3_encode(rng.standard_normal((3, Hkv, page, d)))
    one = np.ones((3, Hkv), np.float32)
    table = [[2, 0, 1]]
    dense = [np.concatenate([oracle.e4m3_decode(c[p]).transpose(1, 0, 2) for p in table[0]])[:L]
             .astype(np.float32) for c in (kc, vc)]
    q = rng.standard_normal((L, H, d)).astype(np.float32)
    sinks = rng.standard_normal(H).astype(np.float32)
    for mode in (0, 1, 2):
        for w in (-1, 9):
            o, lse = oracle.paged_attend(q, kc, vc, one, one, table, [0, L], [L], 1, w, sinks, mode,
                                         0.125)
            ro, rl = oracle.window(q, dense[0], dense[1], np.array([0, L], np.int32), H, Hkv, d, w,
                                   -1, 1, sinks if mode else None, mode, 0.125)
            assert np.abs(o - np.asarray(ro).reshape(o.shape)).max() < 1e-9
            assert np.abs(lse - np.asarray(rl).reshape(lse.shape)).max() < 1e-9


def test_rows_that_see_nothing():
    kc = np.zeros((1, 1, 16, 64), np.uint8)
    one = np.ones((1, 1), np.float32)
    q = np.ones((3, 1, 64))
    # three queries over one cached position: the first two lie before position 0
    o, lse = oracle.paged_attend(q, kc, kc, one, one, [[0]], [0, 3], [1], 1, -1, None, 0, 1.0)
    assert np.all(o == 0) and list(np.isneginf(lse[:, 0])) == [True, True, False]
    o, lse = oracle.paged_attend(q, kc, kc, one, one, [[0]], [0, 3], [0], 0, -1, [0.5], 2, 1.0)
    assert np.all(o == 0) and np.allclose(lse, 0.5)
