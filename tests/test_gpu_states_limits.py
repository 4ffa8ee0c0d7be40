"""Encoder-state operators at the limits of what their numbers may be. Tolerances are those of
test_gpu_states."""
import numpy as np
import pytest
import torch

import oracle
import windowed_attention_sinks_gb300 as sa

from test_gpu_states import DT, LENS, Case, cuda

pytestmark = pytest.mark.gpu

DTYPES = list(DT)


def attend(c, mode=0, hint=None, **kw):
    q, k, v = c.tensors()
    o, lse = sa.cross_fwd(q, k, v, *c.ranges(), max_q_len=hint or int(c.n.max()),
                          sinks=cuda(c.sinks) if mode else None, sink_mode=mode, **kw)
    sa.check_device()
    return o, lse


def reported():
    with pytest.raises(sa.SattnError) as e:
        sa.check_device()
    assert e.value.code == 4


# ------------------------------------------------------------------ large logits

@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("spread", [1e6, 1e8, 1e12, 1e30])
@pytest.mark.parametrize("n", [1, 12, 20, 90])
def test_logits_so_large_that_one_key_has_it_all(n, spread, dtype, mode):
    """Logits up to 10^31, behind which a step of fp32 is far above 1: the value of the
    largest one comes out."""
    H, Hkv, d = 4, 2, 64
    c = Case([(n, 300), (n, 33), (n, 700)], H, Hkv, d, dtype, seed=n, tail=0, spread=spread)
    c.sinks = (c.sinks * spread).astype(np.float32)
    o, lse = attend(c, mode)
    sinks = c.sinks.astype(np.float64)
    wo, wl = oracle.cross_attend(c.q, c.k, c.v, c.cu, c.start, c.len, sinks, mode, c.scale)
    # off by the logits' own error and two roundings of lse, for the few near ties too
    eps = c.eps()
    assert np.all(np.abs(lse.cpu().numpy() - wl) <= eps + 2.0 ** -21 + 2.0 ** -22 * np.abs(wl))
    # rows whose largest logit is further from the next than both can be off
    clear = np.zeros((c.T, H), bool)
    for b in range(3):
        for h in range(H):
            for t in range(c.cu[b], c.cu[b + 1]):
                s = slice(c.start[b], c.start[b] + c.len[b])
                x = c.k[s, h // 2].astype(np.float64) @ c.q[t, h] * c.scale
                if mode == 1:
                    x[0] += sinks[h]
                x = np.sort(np.append(x, sinks[h]) if mode == 2 else x)
                clear[t, h] = x[-1] - x[-2] > 4 * eps[t, h] + 2.0 ** -20 * np.abs(sinks[h]) + 200
    assert clear.mean() > 0.5
    # p, which is not always 1 (m may be off by its rounding), and o are rounded to bf16
    rel = 2 * 2.0 ** -8 if dtype == "bf16" else 2.0 ** -20
    got = o.float().cpu().numpy()
    assert np.all(np.abs(got[clear] - wo[clear]) <= rel * np.abs(wo[clear]))


# ------------------------------------------------------------------ maxima that move

@pytest.mark.parametrize("G", [1, 6])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 8, 20, 150])
def test_a_maximum_that_rises_in_every_step(n, d, G):
    """Keys whose logits climb by 20 every 32 keys, for every other row down instead of up: each
    step's probabilities are taken twice, and what is kept is in the last maximum's terms."""
    c = Case([(n, 1111), (n, 640), (n, 64)], 2 * G, 2, d, seed=n + d, tail=0)
    climb = np.zeros((c.S, 2, 1), np.float32)
    for s, l in zip(c.start, c.len):
        climb[s:s + l, :, 0] = (np.arange(l) // 32 * 20.0)[:, None]
    side = np.where(np.arange(c.T) % 2, 1.0, -1.0)[:, None]
    c.q[..., 0] = oracle.bf16_round((side * np.ones((1, 2 * G))).astype(np.float32))
    live = ~np.isnan(c.k[..., :1])
    c.k[..., :1] = np.where(live, oracle.bf16_round((climb / c.scale).astype(np.float32)), np.nan)
    o, lse = attend(c)
    c.check(o, lse, 0)


# ------------------------------------------------------------------ malformed sequences

@pytest.mark.parametrize("bad", ["in front", "behind", "negative"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_bad_range_of_a_sequence_without_queries_is_reported(dtype, bad):
    c = Case([(3, 100), (0, 50), (2, 64)], 4, 2, 64, dtype, seed=1)
    q, k, v = c.tensors()
    cu, start, lens = c.ranges()
    if bad == "in front":
        start[1] = -1
    else:
        lens[1] = c.S if bad == "behind" else -1
    o = torch.full_like(q, 77.0)
    lse = torch.full((c.T, 4), 77.0, device="cuda")
    sa.cross_fwd(q, k, v, cu, start, lens, max_q_len=3, o=o, lse=lse)
    reported()
    c.check(o, lse, 0)  # the others are right
    assert torch.all(o[5:] == 77.0) and torch.all(lse[5:] == 77.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_bad_range_where_there_are_no_states_is_reported(dtype):
    q = torch.randn(4, 4, 64, device="cuda").to(DT[dtype])
    none = torch.empty(0, 2, 64, device="cuda", dtype=DT[dtype])
    cu, start, lens = (cuda(np.array(x, np.int32)) for x in ([0, 3, 3], [0, 0], [0, 5]))
    o, lse = torch.full_like(q, 77.0), torch.full((4, 4), 77.0, device="cuda")
    sa.cross_fwd(q, none, none, cu, start, lens, o=o, lse=lse)
    reported()
    assert torch.all(o[:3] == 0) and torch.isneginf(lse[:3]).all()
    assert torch.all(o[3:] == 77.0) and torch.all(lse[3:] == 77.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_malformed_sequences_are_skipped_and_reported(dtype):
    n, H, Hkv, d = 3, 4, 2, 64
    c = Case([(n, 100), (n, 50), (n, 80), (n, 64)], H, Hkv, d, dtype, seed=n, tail=0)
    q, k, v = c.tensors()
    cu, start, lens = c.ranges()
    start[1], lens[2] = -1, c.S
    o, lse = torch.full_like(q, 77.0), torch.full((c.T, H), 77.0, device="cuda")
    w = torch.full((Hkv, c.S), 7.0, device="cuda")
    sa.cross_fwd(q, k, v, cu, start, lens, max_q_len=n, o=o, lse=lse)
    reported()
    assert torch.all(o[n:3 * n] == 77.0) and torch.all(lse[n:3 * n] == 77.0)
    ok, wl = attend(c)
    good = [*range(n), *range(3 * n, 4 * n)]
    assert torch.equal(o[good], ok[good]) and torch.equal(lse[good], wl[good])
    sa.cross_key_weights(q, k, wl, cu, start, lens, w, max_q_len=n)
    reported()
    for b in (1, 2):
        assert torch.all(w[:, c.start[b]:c.start[b] + c.len[b]] == 7.0)
    sa.evict_keys(k, v, w, start, lens, 16)
    reported()


@pytest.mark.parametrize("dtype", DTYPES)
def test_cu_seqlens_that_fall_leave_the_others_their_rows(dtype):
    # sequence 0 has rows 0 .. 4, 1 is malformed, 2 claims row 3 as well, 3 has none
    c = Case([(5, 90), (0, 40), (0, 130), (0, 20)], 4, 2, 64, dtype, seed=4, tail=1)
    q, k, v = c.tensors()
    o, lse = torch.full_like(q, 77.0), torch.full((c.T, 4), 77.0, device="cuda")
    cu = cuda(np.array([0, 5, 3, 4, 4], np.int32))
    sa.cross_fwd(q, k, v, cu, *c.ranges()[1:], max_q_len=5, o=o, lse=lse)
    reported()
    assert torch.all(o[5:] == 77.0) and torch.all(lse[5:] == 77.0)
    want, wl = attend(c)
    rows = [0, 1, 2, 4]
    assert torch.equal(o[rows], want[rows]) and torch.equal(lse[rows], wl[rows])
    for bad in ([1, 2, 3, 4, 4], [0, 1, 2, 3, c.T + 1]):
        sa.cross_fwd(q, k, v, cuda(np.array(bad, np.int32)), *c.ranges()[1:], max_q_len=5)
        reported()


# ------------------------------------------------------------------ rows without a denominator

@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 12, 60, 130])
def test_a_row_with_an_infinite_lse_weighs_nothing(n, dtype, mode, value):
    """Whatever its query holds: rows that a caller masks by their lse are often padding."""
    H, Hkv, d = 8, 4, 64
    c = Case([(n, 300), (n + 1, 77), (n, 520)], H, Hkv, d, dtype, seed=n)
    _, wl = oracle.cross_attend(c.q, c.k, np.zeros_like(c.k), c.cu, c.start, c.len, c.sinks, mode,
                                c.scale)
    lse = np.where(np.isnan(wl), 0.0, wl).astype(np.float32)
    rng = np.random.default_rng(n)
    out = rng.random((c.T, H)) < 0.3
    out[0, :3], out[n, 1] = True, True
    lse[out] = np.where(rng.random(out.sum()) < 0.5, np.inf, -np.inf)
    q, k, _ = c.tensors()
    poison = q.clone()
    poison[cuda(out)] = float(value)
    before = rng.random((Hkv, c.S)).astype(np.float32)
    w = cuda(before)
    sa.cross_key_weights(poison, k, cuda(lse), *c.ranges(), w, max_q_len=n + 1, accumulate=True,
                         sinks=cuda(c.sinks) if mode else None, sink_mode=mode)
    sa.check_device()
    c.check_weights(w.cpu().numpy(), lse, before, True, mode)


# ------------------------------------------------------------------ large sinks and logits

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 20, 90])
def test_key_weights_with_extreme_sinks(n, dtype):
    """A sink so large that the logits are lost in it leaves key 0 everything, one so low nothing
    where there are other keys; the only key of a sequence has it all in both cases."""
    H, Hkv, d = 8, 2, 64
    c = Case([(n, 150), (n, 1), (n, 0), (1, 700)], H, Hkv, d, dtype, seed=n, tail=0)
    c.sinks = np.array([-3.4e38, -1e30, -np.inf, 40.0, 3.4e38, 1e30, 2.1e38, -3.0], np.float32)
    _, lse = attend(c, 1)
    before = np.zeros((Hkv, c.S), np.float32)
    w = torch.zeros(Hkv, c.S, device="cuda")
    q, k, _ = c.tensors()
    sa.cross_key_weights(q, k, lse, *c.ranges(), w, max_q_len=n, sinks=cuda(c.sinks), sink_mode=1)
    sa.check_device()
    got = w.cpu().numpy()
    most = 3e38 * np.log(2)
    sinks = np.clip(c.sinks.astype(np.float64), -most, most)
    sinks[2] = -np.inf
    _, wl = oracle.cross_attend(c.q, c.k, np.zeros_like(c.k), c.cu, c.start, c.len, sinks, 1, c.scale)
    want = oracle.cross_key_weights(c.q, c.k, wl, c.cu, c.start, c.len, before, False, sinks, 1,
                                    c.scale)
    # a weight's and its lse's own error, the largest lse that is not a sink's below 64
    rel = 3 * c.eps().max() + 2.0 ** -20 + 2.0 ** -21 + 2.0 ** -21 * 64 + 4 * n * 2.0 ** -24
    assert np.all(np.abs(got - want) <= rel * want + 1e-30)


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 70])
def test_key_weights_of_huge_logits_stay_shares(n, dtype, mode):
    """Logits up to 10^12, of which an fp32 lse is off by thousands: a weight is then no more than
    its formula says of that lse, and never above 1 a row."""
    H, Hkv, d = 4, 2, 64
    c = Case([(n, 300), (n, 33)], H, Hkv, d, dtype, seed=n, tail=0, spread=1e12)
    c.sinks = np.array([1e10, -1e10, 1e9, 0.0], np.float32)
    _, lse = attend(c, mode)
    assert torch.isfinite(lse).all()
    w = torch.zeros(Hkv, c.S, device="cuda")
    q, k, _ = c.tensors()
    sa.cross_key_weights(q, k, lse, *c.ranges(), w, max_q_len=n,
                         sinks=cuda(c.sinks) if mode else None, sink_mode=mode)
    sa.check_device()
    assert torch.isfinite(w).all() and w.max().item() <= 2 * n * (1 + 2 * n * 2.0 ** -24)


# ------------------------------------------------------------------ other forms of the calls

@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("hint", [1, 4000])
@pytest.mark.parametrize("lens", ["tokens", "ragged", "long"])
@pytest.mark.parametrize("d", [64, 128])
def test_key_weights_without_a_workspace(d, lens, hint, mode):
    c = Case(LENS[lens], 8, 2, d, seed=5)
    _, wl = oracle.cross_attend(c.q, c.k, np.zeros_like(c.k), c.cu, c.start, c.len, c.sinks, mode,
                                c.scale)
    lse = np.where(np.isnan(wl), 0.0, wl).astype(np.float32)
    before = np.random.default_rng(1).random((2, c.S)).astype(np.float32)
    q, k, _ = c.tensors()
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for add in (False, True):
        w = cuda(before)
        sa.cross_key_weights(q, k, cuda(lse), *c.ranges(), w, max_q_len=hint, accumulate=add,
                             sinks=cuda(c.sinks) if mode else None, sink_mode=mode,
                             workspace=small)
        sa.check_device()
        c.check_weights(w.cpu().numpy(), lse, before, add, mode)


@pytest.mark.parametrize("B", [33, 700])
def test_many_sequences_fp32(B):
    rng = np.random.default_rng(B)
    c = Case([(int(rng.integers(0, 3)), int(rng.integers(0, 100))) for _ in range(B)], 2, 1, 64,
             "f32", seed=B)
    o, lse = attend(c, 1)
    wl = c.check(o, lse, 1)
    full = np.zeros((c.T, 2), np.float32)
    full[:len(wl)] = wl
    w = torch.zeros(1, c.S, device="cuda")
    q, k, _ = c.tensors()
    sa.cross_key_weights(q, k, cuda(full), *c.ranges(), w, sinks=cuda(c.sinks), sink_mode=1)
    sa.check_device()
    c.check_weights(w.cpu().numpy(), full, np.zeros((1, c.S), np.float32), False, 1)


def test_sequences_share_states_fp32():
    H, Hkv, d = 8, 4, 128
    c = Case([(5, 700)], H, Hkv, d, "f32", seed=1, tail=0)
    q, k, v = c.tensors()
    c.n, c.cu = np.ones(5, np.int64), np.arange(6, dtype=np.int32)
    c.start = c.start[0] + np.array([0, 0, 0, 130, 0], np.int32)
    c.len = np.array([700, 700, 1, 129, 700], np.int32)
    o, lse = sa.cross_fwd(q, k, v, *c.ranges(), max_q_len=1)
    sa.check_device()
    c.check(o, lse, 0)


def test_far_states_fp32():
    """Rows whose elements lie behind 2^31 elements."""
    H, Hkv, d, S = 4, 4, 128, 2_110_000
    kv = torch.empty(S, 2 * Hkv, d, device="cuda")
    lens, starts = [133, 50], [S - 133, 2_100_000]
    for s, l in zip(starts, lens):
        kv[s:s + l] = torch.randn(l, 2 * Hkv, d, device="cuda")
    c = Case([(3, 133), (3, 50)], H, Hkv, d, "f32", tail=0)
    c.kv = torch.cat([kv[s:s + l] for s, l in zip(starts, lens)]).cpu().numpy()
    c.k, c.v, c.S = c.kv[:, :Hkv], c.kv[:, Hkv:], 183
    c.start, c.len = np.array([0, 133], np.int32), np.array(lens, np.int32)
    at = cuda(c.cu), cuda(np.array(starts, np.int32)), cuda(c.len)
    q, k, v = cuda(c.q), kv[:, :Hkv], kv[:, Hkv:]
    o, lse = sa.cross_fwd(q, k, v, *at)
    sa.check_device()
    wl = c.check(o, lse, 0)
    w = torch.zeros(Hkv, S, device="cuda")
    sa.cross_key_weights(q, k, lse, *at, w)
    sa.check_device()
    near = np.concatenate([w[:, s:s + l].cpu().numpy() for s, l in zip(starts, lens)], 1)
    c.check_weights(near, wl.astype(np.float32), np.zeros_like(near), False, 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", [0, 2])
@pytest.mark.parametrize("n", [1, 14, 130])
def test_cross_attention_without_lse(n, mode, dtype):
    """lse = NULL in C; the binding always makes one."""
    H, Hkv, d = 8, 2, 128
    c = Case([(n, 900), (1, 64), (n, 0)], H, Hkv, d, dtype, seed=n)
    want, _ = attend(c, mode)
    q, k, v = c.tensors()
    cu, start, lens = c.ranges()
    o = torch.full_like(q, 77.0)
    sinks = cuda(c.sinks)
    nb = sa.cross_workspace_bytes(n, H, Hkv, d)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    rc = sa.lib().sattn_cross_fwd(
        q.data_ptr(), H * d, k.data_ptr(), 2 * Hkv * d, v.data_ptr(), 2 * Hkv * d, cu.data_ptr(),
        start.data_ptr(), lens.data_ptr(), 3, c.T, c.S, n, H, Hkv, d, sinks.data_ptr(), mode,
        c.scale, o.data_ptr(), None, ws.data_ptr(), nb, 1 if dtype == "bf16" else 0,
        torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    sa.check_device()
    live = int(c.cu[-1])
    assert torch.equal(o[:live], want[:live]) and torch.all(o[live:] == 77.0)


def test_evict_of_shared_and_of_no_states():
    Hkv, d, keep = 2, 64, 40
    rng = np.random.default_rng(0)
    k = torch.randn(300, 2 * Hkv, d, device="cuda").bfloat16()
    w = rng.random((Hkv, 300)).astype(np.float32)
    start, lens = [0, 0, 100, 299, 7, 300], [300, 300, 150, 1, 0, 0]
    got = sa.evict_keys(k[:, :Hkv], k[:, Hkv:], cuda(w), cuda(np.array(start, np.int32)),
                        cuda(np.array(lens, np.int32)), keep, 3, 5)
    sa.check_device()
    want = oracle.evict_keys(w, start, lens, keep, 3, 5)
    assert np.array_equal(got[3].cpu().numpy(), want)
    at = np.repeat(np.array(start), keep)[None] + want
    for h in range(Hkv):
        live = want[h] >= 0
        rows = cuda(at[h][live].astype(np.int64))
        assert torch.equal(got[0][cuda(live), h], k[rows, h])
        assert torch.equal(got[1][cuda(live), h], k[rows, Hkv + h])
    none = torch.empty(0, Hkv, d, device="cuda").bfloat16()
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    ko, vo, wo, rows, at, kept = sa.evict_keys(none, none, torch.empty(Hkv, 0, device="cuda"),
                                               zero, zero, 3)
    sa.check_device()
    assert torch.all(ko == 0) and torch.all(vo == 0) and torch.all(wo == 0)
    assert torch.all(rows == -1) and kept.tolist() == [0, 0] and at.tolist() == [0, 3]
