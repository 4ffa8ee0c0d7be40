"""GPU parity of the encoder-state operators with the fp64 oracle.

Tolerances, with A = sum p |v| / z of a row and E the largest sum |q_c k_c| scale of its
keys. A logit is a sum of d exact products (bf16) or rounded ones (fp32) in fp32, kept in
units of log 2: off by eps = 2^-17 E at most (d 2^-24 E for the sum, in any order and with
truncation twice that, and a few roundings of the result). A probability is then off by eps and the
exponential's 2^-21 relative. o: 2 (eps + 2^-21) A, plus for bf16 half a step of p, 2^-8 A, and
of o, 2^-8 |o|. lse: eps + 2^-21 + 2^-22 |lse|. A key's weight w, a sum of r such
exponentials of numbers up to |lse|: (2 eps + 2^-20 + 2^-22 |lse| + r 2^-24) w."""
import numpy as np
import pytest
import torch

import oracle
import windowed_attention_sinks_gb300 as sa

from gpu_helpers import PARITY_LOG  # noqa: F401

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def cuda(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


class Case:
    """Sequences given as (queries, states). Rows of k and v outside them are NaN."""

    def __init__(self, lens, H, Hkv, d, dtype="bf16", seed=0, gap=3, tail=2, spread=1.0):
        rng = np.random.default_rng(seed)
        self.H, self.Hkv, self.d, self.dtype = H, Hkv, d, dtype
        self.n = np.array([a for a, _ in lens], np.int64)
        self.len = np.array([b for _, b in lens], np.int32)
        self.cu = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        order = rng.permutation(len(lens))  # the states lie in another order, with gaps
        self.start = np.zeros(len(lens), np.int32)
        at = 1
        for b in order:
            self.start[b] = at
            at += self.len[b] + gap
        self.T, self.S = int(self.cu[-1]) + tail, at
        q = rng.standard_normal((self.T, H, d)) * spread
        kv = rng.standard_normal((self.S, 2 * Hkv, d))
        dead = np.ones(self.S, bool)
        for s, l in zip(self.start, self.len):
            dead[s:s + l] = False
        kv[dead] = np.nan
        self.q, self.kv = q.astype(np.float32), kv.astype(np.float32)
        if dtype == "bf16":
            self.q = oracle.bf16_round(self.q)
            self.kv[~dead] = oracle.bf16_round(self.kv[~dead])
        self.k, self.v = self.kv[:, :Hkv], self.kv[:, Hkv:]
        self.sinks = rng.standard_normal(H).astype(np.float32)
        self.scale = d ** -0.5

    def tensors(self):
        kv = cuda(self.kv, DT[self.dtype])  # one projection's output
        return cuda(self.q, DT[self.dtype]), kv[:, :self.Hkv], kv[:, self.Hkv:]

    def ranges(self):
        return cuda(self.cu), cuda(self.start), cuda(self.len)

    def of_rows(self, f):
        """f(q, k, v) for every sequence and head -> [T, H] (0 for rows of no sequence)."""
        out = np.zeros((self.T, self.H))
        for b in range(len(self.len)):
            r, s = slice(self.cu[b], self.cu[b + 1]), slice(self.start[b], self.start[b] + self.len[b])
            for h in range(self.H):
                g = h // (self.H // self.Hkv)
                if self.len[b]:
                    out[r, h] = f(self.q[r, h], self.k[s, g], self.v[s, g])
        return out

    def eps(self):
        return 2.0 ** -17 * self.scale * self.of_rows(
            lambda q, k, v: (np.abs(q) @ np.abs(k).T).max(1))

    def spread_of(self, mode):
        """A of every row and column: the attention over |v|."""
        sinks = self.sinks if mode else None
        return oracle.cross_attend(self.q, self.k, np.abs(self.v), self.cu, self.start, self.len,
                                   sinks, mode, self.scale)[0][:self.cu[-1]]

    def check(self, o, lse, mode, sinks=None):
        live = int(self.cu[-1])
        wo, wl = oracle.cross_attend(self.q, self.k, self.v, self.cu, self.start, self.len,
                                     self.sinks if sinks is None else sinks, mode, self.scale)
        wo, wl = wo[:live], wl[:live]
        eps = self.eps()[:live]
        go, gl = o[:live].float().cpu().numpy(), lse[:live].cpu().numpy()
        tol = 2 * (eps + 2.0 ** -21)[..., None] * self.spread_of(mode)
        if self.dtype == "bf16":
            tol += 2.0 ** -8 * self.spread_of(mode) + 2.0 ** -8 * np.abs(wo)
        assert np.all(np.abs(go - wo) <= tol + 1e-30), np.abs(go - wo).max()
        assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
        fin = ~np.isneginf(wl)
        bound = eps + 2.0 ** -21 + 2.0 ** -22 * np.abs(np.where(fin, wl, 0.0))
        assert np.all(np.abs(gl[fin] - wl[fin]) <= bound[fin])
        return wl

    def check_weights(self, got, lse, before, add, mode):
        want = oracle.cross_key_weights(self.q, self.k, lse, self.cu, self.start, self.len, before,
                                        add, self.sinks, mode, self.scale)
        add_ = want - (before if add else 0.0)
        top = np.abs(lse[np.isfinite(lse)]).max(initial=0.0)
        rows = self.n.max(initial=0) * (self.H // self.Hkv)
        rel = 2 * self.eps().max() + 2.0 ** -20 + 2.0 ** -22 * top + rows * 2.0 ** -24
        tol = rel * np.abs(add_) + 2.0 ** -23 * np.abs(want)
        touched = np.zeros(self.S, bool)
        for s, l in zip(self.start, self.len):
            touched[s:s + l] = True
        assert np.array_equal(got[:, ~touched], before[:, ~touched].astype(np.float32))
        assert np.all(np.abs(got - want)[:, touched] <= tol[:, touched] + 1e-37)


LENS = {
    "one": [(1, 1)],
    "tokens": [(1, 5), (1, 0), (1, 128), (1, 129), (1, 700), (1, 127), (1, 1)],
    "beams": [(5, 331), (0, 40), (5, 64), (3, 1)],
    "ragged": [(7, 300), (0, 0), (130, 65), (33, 0), (1, 513), (257, 128), (2, 2)],
    "long": [(3, 5000), (140, 1111)],
}
HEADS = [(8, 2, 128), (8, 8, 64), (5, 1, 128), (6, 2, 64), (14, 2, 128), (40, 1, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("lens", list(LENS))
def test_cross_attention(lens, H, Hkv, d, dtype):
    c = Case(LENS[lens], H, Hkv, d, dtype, seed=H + d)
    mode = (H + len(lens)) % 3
    q, k, v = c.tensors()
    o = torch.full_like(q, 77.0)
    lse = torch.full((c.T, H), 77.0, device="cuda")
    got = sa.cross_fwd(q, k, v, *c.ranges(), max_q_len=int(c.n.max()),
                       sinks=cuda(c.sinks) if mode else None, sink_mode=mode, o=o, lse=lse)
    sa.check_device()
    assert got[0] is o and got[1] is lse
    c.check(o, lse, mode)
    assert torch.all(o[c.cu[-1]:] == 77.0) and torch.all(lse[c.cu[-1]:] == 77.0)


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("hint", [None, 1, 4000])
@pytest.mark.parametrize("lens", ["tokens", "ragged"])
def test_cross_attention_with_any_hint_and_without_a_workspace(lens, hint, mode):
    c = Case(LENS[lens], 8, 2, 128, seed=5)
    q, k, v = c.tensors()
    sinks = cuda(c.sinks) if mode else None
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for ws in (None, small):
        o, lse = sa.cross_fwd(q, k, v, *c.ranges(), max_q_len=hint, sinks=sinks, sink_mode=mode,
                              workspace=ws)
        sa.check_device()
        c.check(o, lse, mode)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("lens", list(LENS))
def test_key_weights(lens, H, Hkv, d, dtype, accumulate):
    c = Case(LENS[lens], H, Hkv, d, dtype, seed=H + d + 1)
    mode = (H + len(lens)) % 3
    q, k, v = c.tensors()
    _, lse = oracle.cross_attend(c.q, c.k, np.zeros_like(c.k), c.cu, c.start, c.len, c.sinks, mode,
                                 c.scale)
    lse = np.where(np.isnan(lse), 0.0, lse).astype(np.float32)
    before = np.random.default_rng(1).random((Hkv, c.S)).astype(np.float32)
    w = cuda(before)
    got = sa.cross_key_weights(q, k, cuda(lse), *c.ranges(), w, max_q_len=int(c.n.max()),
                               accumulate=accumulate, sinks=cuda(c.sinks) if mode else None,
                               sink_mode=mode)
    sa.check_device()
    assert got is w
    c.check_weights(w.cpu().numpy(), lse, before, accumulate, mode)


# ------------------------------------------------------------------ rotation

AXES = {
    "video": (3, lambda half: np.where(np.arange(half) < half // 4, 0, 1 + np.arange(half) % 2)),
    "image": (2, lambda half: (np.arange(half) >= half // 2).astype(int)),
    "text": (1, lambda half: np.zeros(half, int)),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rd,inter", [(128, 128, False), (128, 64, True), (64, 48, True),
                                        (80, 80, False), (72, 64, False), (256, 256, False),
                                        (64, 16, False), (24, 16, True)])
@pytest.mark.parametrize("kind", list(AXES))
def test_rope_axes(kind, d, rd, inter, dtype):
    rng = np.random.default_rng(d + rd)
    T, H, Hkv = 37, 5, 2
    axes, of = AXES[kind]
    axis = of(rd // 2).astype(np.uint8)
    pos = rng.integers(-70000, 300000, (axes, T)).astype(np.int32)
    pos[:, :3] = [[0, 2 ** 31 - 1, -2 ** 31]]
    freq = (10000.0 ** (-np.arange(rd // 2) / (rd // 2))).astype(np.float32)
    x = rng.standard_normal((T, H + 2 * Hkv, d)).astype(np.float32)
    if dtype == "bf16":
        x = oracle.bf16_round(x)
    qkv = cuda(x, DT[dtype])
    before = qkv.clone()
    args = cuda(pos), cuda(freq), cuda(axis)
    for inverse in (False, True):
        q, k = sa.rope_axes(qkv[:, :H], qkv[:, H:H + Hkv], *args, interleaved=inter,
                            inverse=inverse)
        sa.check_device()
        assert torch.equal(qkv, before)
        want = oracle.rope_axes(x[:, :H + Hkv], pos, freq, axis, inter, inverse)
        # fp32: the angle is off by 2^-25 turns, cosine and sine by 2^-23, products by 2^-23
        pair = np.abs(x[:, :H + Hkv]).max()
        got = torch.cat([q, k], 1).float().cpu().numpy()
        tol = 2 * pair * (2 * np.pi * 2.0 ** -25 + 2.0 ** -22)
        tol = tol + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
        assert np.all(np.abs(got - want) <= tol)
        assert np.array_equal(got[:, :, rd:], x[:, :H + Hkv, rd:])
    # in place, on the slices, to the same bits; v stays
    q, k = sa.rope_axes(qkv[:, :H], qkv[:, H:H + Hkv], *args, interleaved=inter)
    qi, ki = qkv[:, :H], qkv[:, H:H + Hkv]
    sa.rope_axes(qi, ki, *args, interleaved=inter, q_out=qi, k_out=ki)
    assert torch.equal(qi, q) and torch.equal(ki, k)
    assert torch.equal(qkv[:, H + Hkv:], before[:, H + Hkv:])
    alone, none = sa.rope_axes(before[:, :H], None, *args, interleaved=inter)
    assert none is None and torch.equal(alone, q)


@pytest.mark.parametrize("T", [0, 1, 3, 1000, 4099])
def test_rope_axes_of_many_tokens(T):
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, 3, 64)).astype(np.float32)
    pos = rng.integers(0, 5000, (2, T)).astype(np.int32)
    freq, axis = np.array([1.0, 0.1] * 8, np.float32), np.array([0, 1] * 8, np.uint8)
    q, _ = sa.rope_axes(cuda(x), None, cuda(pos), cuda(freq), cuda(axis))
    want = oracle.rope_axes(x, pos, freq, axis, False)
    assert np.all(np.abs(q.cpu().numpy() - want) <= 2 * np.abs(x).max(initial=0) * 2.0 ** -21)


def test_rope_axes_gradient_is_the_inverse():
    """d <rope(x), y> / dx = rope^-1(y), against differences in both arguments."""
    rng = np.random.default_rng(2)
    T, H, d, rd = 9, 3, 64, 48
    x, y, dx = (cuda(rng.standard_normal((T, H, d)).astype(np.float32)) for _ in range(3))
    pos = cuda(rng.integers(0, 900, (3, T)).astype(np.int32))
    freq = cuda((100.0 ** (-np.arange(rd // 2) / 24)).astype(np.float32))
    axis = cuda((np.arange(rd // 2) % 3).astype(np.uint8))

    def f(t, **kw):
        return sa.rope_axes(t, None, pos, freq, axis, **kw)[0].double()

    # the map is linear: the difference over a step of any size is the derivative. Each
    # side sums T H d = 1728 products, each off by 2^-21 of its factors
    change = ((f(x + dx) - f(x)) * y.double()).sum().item()
    grad = (f(y, inverse=True) * dx.double()).sum().item()
    size = (f(x).abs() * y.double().abs()).sum().item() + (dx.abs() * y.abs()).sum().item()
    assert abs(change - grad) <= 8 * 2.0 ** -21 * size


def test_an_axis_that_is_not_there_is_reported():
    x = torch.randn(4, 2, 64, device="cuda")
    pos = torch.ones(2, 4, dtype=torch.int32, device="cuda")
    axis = torch.tensor([0, 1, 2, 255, 0, 0, 0, 0], dtype=torch.uint8, device="cuda")
    freq = torch.full((8,), 0.5, device="cuda")
    freq[5] = float("nan")
    q, _ = sa.rope_axes(x, None, pos, freq, axis)
    with pytest.raises(sa.SattnError) as e:
        sa.check_device()
    assert e.value.code == 4
    for i in (2, 3):  # the pair stays
        assert torch.equal(q[..., [i, i + 8]], x[..., [i, i + 8]])
    assert torch.isnan(q[..., [5, 13]]).all() and not torch.isnan(q[..., [4, 12]]).any()


# ------------------------------------------------------------------ eviction

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,d", [(2, 128), (3, 64), (1, 128)])
@pytest.mark.parametrize("keep,first,last", [(1, 0, 0), (4, 2, 2), (100, 3, 17), (1000, 0, 1),
                                             (2100, 0, 0)])
def test_evict(keep, first, last, Hkv, d, dtype):
    lens = [(1, 1), (1, 0), (1, 5), (1, 99), (1, 100), (1, 101), (1, 1500), (1, 2099)]
    c = Case(lens, Hkv, Hkv, d, dtype, seed=keep)
    rng = np.random.default_rng(keep)
    w = np.exp(rng.standard_normal((Hkv, c.S)) * 4).astype(np.float32)
    w[rng.random((Hkv, c.S)) < 0.3] = 0.0  # many ties
    w[rng.random((Hkv, c.S)) < 0.2] = 2.5
    w[:, 7::50] = np.nan
    w[:, 9::50] = -1.0
    w[:, 11::50] = np.inf
    _, k, v = c.tensors()
    _, start, len_ = c.ranges()
    ko, vo, wo, rows, starts, kept = sa.evict_keys(k, v, cuda(w), start, len_, keep, first, last)
    sa.check_device()
    want = oracle.evict_keys(w, c.start, c.len, keep, first, last)
    assert np.array_equal(rows.cpu().numpy(), want)
    B = len(lens)
    assert np.array_equal(starts.cpu().numpy(), np.arange(B) * keep)
    assert np.array_equal(kept.cpu().numpy(), np.minimum(c.len, keep))
    at = np.repeat(c.start, keep)[None] + want
    for h in range(Hkv):
        live = want[h] >= 0
        for got, src in ((ko, c.k), (vo, c.v)):
            g = got[:, h].float().cpu().numpy()
            assert np.array_equal(g[live], src[at[h][live], h]) and np.all(g[~live] == 0)
        g = wo[h].cpu().numpy()
        assert np.array_equal(g[live], w[h][at[h][live]], equal_nan=True) and np.all(g[~live] == 0)


@pytest.mark.parametrize("L,keep", [(16384, 5000), (16385, 16384), (40000, 777)])
def test_evict_of_long_sequences(L, keep):
    rng = np.random.default_rng(L)
    S = L + 10
    w = np.round(np.exp(rng.standard_normal((1, S))), 1).astype(np.float32)
    k = torch.randn(S, 1, 64, device="cuda")
    start, len_ = cuda(np.array([5], np.int32)), cuda(np.array([L], np.int32))
    ko, vo, wo, rows, _, _ = sa.evict_keys(k, k + 1, cuda(w), start, len_, keep, 10, 20)
    want = oracle.evict_keys(w, [5], [L], keep, 10, 20)
    assert np.array_equal(rows.cpu().numpy(), want)
    assert torch.equal(ko, k[5 + cuda(want[0]).long()])


# ------------------------------------------------------------------ together

def test_rotate_attend_weigh_evict_attend():
    """A serving loop: states rotated and stored, prompts and then single tokens attend,
    the weights add up, the light rows leave, and tokens attend to what is left."""
    H, Hkv, d = 8, 2, 128
    c = Case([(20, 700), (3, 150), (9, 1), (1, 400)], H, Hkv, d, seed=3, tail=0)
    live = np.concatenate([np.arange(s, s + l) for s, l in zip(c.start, c.len)])
    rng = np.random.default_rng(9)
    pos = rng.integers(0, 64, (3, c.S)).astype(np.int32)
    freq = (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
    axis = (np.arange(64) % 3).astype(np.uint8)
    q, k, v = c.tensors()
    k, _ = sa.rope_axes(k, None, cuda(pos), cuda(freq), cuda(axis), q_out=k)
    turned = k.float().cpu().numpy()
    err = np.abs(turned[live] - oracle.rope_axes(c.k[live], pos[:, live], freq, axis, False))
    assert err.max() <= 2.0 ** -8 * np.abs(turned[live]).max() + 1e-5
    c.kv = np.concatenate([turned, c.v], 1)
    c.k, c.v = c.kv[:, :Hkv], c.kv[:, Hkv:]
    weights = torch.zeros(Hkv, c.S, device="cuda")
    before = np.zeros((Hkv, c.S), np.float32)
    ranges = c.ranges()
    for step in range(3):
        if step:  # single tokens from now on
            q = torch.randn(4, H, d, device="cuda").bfloat16()
            c.n, c.cu, c.T = np.ones(4, np.int64), np.arange(5, dtype=np.int32), 4
            c.q = q.float().cpu().numpy()
            ranges = c.ranges()
        n = int(c.n.max())
        o, lse = sa.cross_fwd(q, k, v, *ranges, max_q_len=n)
        sa.cross_key_weights(q, k, lse, *ranges, weights, max_q_len=n, accumulate=True)
        sa.check_device()
        c.check(o, lse, 0)
        after = weights.cpu().numpy()
        c.check_weights(after, lse.cpu().numpy(), before, True, 0)
        before = after
    k2, v2, w2, rows, starts, lens = sa.evict_keys(k, v, weights, ranges[1], ranges[2], 128, 4, 16)
    want = oracle.evict_keys(before, c.start, c.len, 128, 4, 16)
    assert np.array_equal(rows.cpu().numpy(), want)
    o, lse = sa.cross_fwd(q, k2, v2, ranges[0], starts, lens, max_q_len=1)
    c.start, c.len, c.S = starts.cpu().numpy(), lens.cpu().numpy(), 4 * 128
    c.k, c.v = k2.float().cpu().numpy(), v2.float().cpu().numpy()
    c.check(o, lse, 0)
    sa.cross_key_weights(q, k2, lse, ranges[0], starts, lens, w2, accumulate=True)
    sa.check_device()
