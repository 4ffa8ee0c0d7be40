"""Encoder-state operators where they can go wrong: many sequences, wide groups, shared and far
states, NaN and infinities, extreme sinks and logits, streams, graphs, timeouts, repeated
calls. Tolerances are those of test_gpu_states."""
import numpy as np
import pytest
import torch

import oracle
import windowed_attention_sinks_gb300 as sa

from test_gpu_states import DT, Case, cuda

pytestmark = pytest.mark.gpu


def attend(c, mode=0, hint=None, **kw):
    q, k, v = c.tensors()
    o, lse = sa.cross_fwd(q, k, v, *c.ranges(), max_q_len=hint or int(c.n.max()),
                          sinks=cuda(c.sinks) if mode else None, sink_mode=mode, **kw)
    sa.check_device()
    return o, lse


@pytest.mark.parametrize("B", [33, 128, 129, 700])
@pytest.mark.parametrize("n", [1, 70])
def test_many_sequences(B, n):
    rng = np.random.default_rng(B)
    lens = [(int(rng.integers(0, n + 1)), int(rng.integers(0, 200))) for _ in range(B)]
    if n == 70:
        lens = [(a if i % 9 == 0 else a % 2, b) for i, (a, b) in enumerate(lens)]
    c = Case(lens, 2, 1, 64, seed=B)
    o, lse = attend(c, 2, n)
    wl = c.check(o, lse, 2)
    w = torch.zeros(1, c.S, device="cuda")
    q, k, _ = c.tensors()
    full = np.zeros((c.T, 2), np.float32)
    full[:len(wl)] = wl
    sa.cross_key_weights(q, k, cuda(full), *c.ranges(), w, max_q_len=n, sinks=cuda(c.sinks),
                         sink_mode=2)
    sa.check_device()
    c.check_weights(w.cpu().numpy(), full, np.zeros((1, c.S), np.float32), False, 2)


@pytest.mark.parametrize("G", [3, 7, 31, 33, 64, 65, 96, 127, 128])
@pytest.mark.parametrize("n", [1, 3])
def test_wide_groups(G, n):
    c = Case([(n, 300), (1, 77), (n, 129)], 2 * G, 2, 64, seed=G)
    o, lse = attend(c, 1)
    wl = c.check(o, lse, 1)
    full = np.zeros((c.T, 2 * G), np.float32)
    full[:len(wl)] = wl
    q, k, _ = c.tensors()
    before = np.random.default_rng(G).random((2, c.S)).astype(np.float32)
    w = cuda(before)
    sa.cross_key_weights(q, k, cuda(full), *c.ranges(), w, max_q_len=n, accumulate=True,
                         sinks=cuda(c.sinks), sink_mode=1)
    sa.check_device()
    c.check_weights(w.cpu().numpy(), full, before, True, 1)


def test_sequences_may_share_states():
    """Hypotheses over the same states, as sequences of their own and as one's queries."""
    H, Hkv, d = 8, 4, 128
    c = Case([(5, 700)], H, Hkv, d, seed=1, tail=0)
    q, k, v = c.tensors()
    o, lse = sa.cross_fwd(q, k, v, *c.ranges(), max_q_len=5)
    c.check(o, lse, 0)
    cu = torch.arange(6, dtype=torch.int32, device="cuda")
    start = torch.full((5,), int(c.start[0]), dtype=torch.int32, device="cuda")
    lens = torch.full((5,), 700, dtype=torch.int32, device="cuda")
    o2, lse2 = sa.cross_fwd(q, k, v, cu, start, lens, max_q_len=1)
    sa.check_device()
    c.check(o2, lse2, 0)
    lens[2:4] = torch.tensor([1, 129], dtype=torch.int32, device="cuda")  # and part of them
    start[3] += 130
    o3, lse3 = sa.cross_fwd(q, k, v, cu, start, lens, max_q_len=1)
    part = Case([(1, 700), (1, 700), (1, 1), (1, 129), (1, 700)], H, Hkv, d, tail=0)
    part.q, part.kv, part.k, part.v, part.S = c.q, c.kv, c.k, c.v, c.S
    part.start, part.len = start.cpu().numpy(), lens.cpu().numpy()
    part.check(o3, lse3, 0)


@pytest.mark.parametrize("n", [1, 40])
def test_far_states(n):
    """Rows whose elements lie behind 2^32 bytes, and 2^31 elements."""
    H, Hkv, d, S = 4, 8, 128, 1_060_000
    H = 8
    kv = torch.empty(S, 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")
    lens, starts = [333, 200], [S - 333, 1_050_000]
    for s, l in zip(starts, lens):
        kv[s:s + l] = torch.randn(l, 2 * Hkv, d, device="cuda").bfloat16()
    c = Case([(n, 333), (n, 200)], H, Hkv, d, tail=0)
    small = torch.cat([kv[s:s + l] for s, l in zip(starts, lens)])
    c.kv = small.float().cpu().numpy()
    c.k, c.v, c.S = c.kv[:, :Hkv], c.kv[:, Hkv:], 533
    c.start, c.len = np.array([0, 333], np.int32), np.array(lens, np.int32)
    q = cuda(c.q, torch.bfloat16)
    cu = cuda(c.cu)
    at = cuda(np.array(starts, np.int32)), cuda(c.len)
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    o, lse = sa.cross_fwd(q, k, v, cu, *at, max_q_len=n)
    sa.check_device()
    wl = c.check(o, lse, 0)
    w = torch.zeros(Hkv, S, device="cuda")
    sa.cross_key_weights(q, k, lse, cu, *at, w, max_q_len=n)
    near = np.concatenate([w[:, s:s + l].cpu().numpy() for s, l in zip(starts, lens)], 1)
    c.check_weights(near, wl.astype(np.float32), np.zeros_like(near), False, 0)
    k2, v2, w2, rows, _, _ = sa.evict_keys(k, v, w, *at, 100, 2, 3)
    sa.check_device()
    want = oracle.evict_keys(near, [0, 333], lens, 100, 2, 3)
    assert np.array_equal(rows.cpu().numpy(), want)
    src = np.repeat(np.array(starts), 100)[None] + want
    for h in (0, Hkv - 1):
        assert torch.equal(k2[:, h], k[cuda(src[h]).long(), h])
        assert torch.equal(v2[:, h], v[cuda(src[h]).long(), h])


@pytest.mark.parametrize("n", [1, 12, 100])
def test_nan_reaches_what_it_belongs_to(n):
    H, Hkv, d = 8, 2, 128
    lens = [(n, 200), (n, 300), (n, 130)]
    c = Case(lens, H, Hkv, d, seed=n, tail=0)
    q, k, v = (t.clone() for t in c.tensors())
    s0, s1 = int(c.start[0]), int(c.start[1])
    q[0, 3] = float("nan")                # a query row
    k[s1 + 7, 1, 5] = float("nan")        # a key: every row of its sequence's heads
    v[s0 + 199, 0, 11] = float("nan")     # a value: its column
    o, lse = sa.cross_fwd(q, k, v, *c.ranges(), max_q_len=n)
    sa.check_device()
    bad = np.zeros((c.T, H, d), bool)
    bad[0, 3] = True
    bad[n:2 * n, 4:] = True
    bad[:n, :4, 11] = True
    assert np.array_equal(torch.isnan(o).cpu().numpy(), bad)
    rows = np.zeros((c.T, H), bool)
    rows[0, 3] = True
    rows[n:2 * n, 4:] = True
    assert np.array_equal(torch.isnan(lse).cpu().numpy(), rows)
    # The others are right all the same. (Not the same bits as without: which m a row's
    # probabilities are taken in terms of is decided for 32 rows at once, and any m gives the
    # same quotient before P's rounding, which `check` allows for.)
    o0, lse0 = sa.cross_fwd(*c.tensors(), *c.ranges(), max_q_len=n)
    bad, rows = torch.from_numpy(bad).cuda(), torch.from_numpy(rows).cuda()
    c.check(torch.where(bad, o0, o), torch.where(rows, lse0, lse), 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("n", [1, 90])
def test_extreme_sinks(n, mode, dtype):
    c = Case([(n, 150), (n, 1), (n, 0)], 6, 2, 64, dtype, seed=mode, tail=0)
    c.sinks = np.array([-3.4e38, 3.4e38, -np.inf, 60.0, -60.0, 0.0], np.float32)
    o, lse = attend(c, mode)
    most = 3e38 * np.log(2)  # a finite sink in log2 units is kept below 3e38
    sink = np.clip(c.sinks.astype(np.float64), -most, most)
    sink[2] = -np.inf
    c.sinks = sink
    wo, wl = oracle.cross_attend(c.q, c.k, c.v, c.cu, c.start, c.len, sink, mode, c.scale)
    rel = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -14  # of sums of |v| below 5
    got = o.float().cpu().numpy()
    assert np.all(np.abs(got - wo) <= rel * 5)
    gl = lse.cpu().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
    fin = np.isfinite(wl)
    assert np.all(np.abs(gl[fin] - wl[fin]) <= 1e-3 + 2.0 ** -20 * np.abs(wl[fin]))


@pytest.mark.parametrize("n", [1, 7, 100])
def test_large_logits(n):
    """Logits in the thousands: one key takes it all, wherever it stands; the maximum moves."""
    H, Hkv, d = 4, 2, 64
    c = Case([(n, 700), (n, 333)], H, Hkv, d, seed=n, tail=0, spread=60.0)
    o, lse = attend(c)
    c.check(o, lse, 0)


@pytest.mark.parametrize("n", [1, 100])
def test_equal_logits_count_the_states(n):
    c = Case([(n, 1), (n, 127), (n, 128), (n, 129), (n, 1000)], 4, 2, 128, tail=0)
    c.q[:] = 0
    c.kv[~np.isnan(c.kv)] = 1.0
    o, lse = attend(c)
    want = np.repeat(np.log(c.len.astype(np.float64)), n)[:, None]
    assert np.abs(lse.cpu().numpy() - want).max() <= 2.0 ** -20
    assert torch.all(o == 1.0)
    w = torch.full((2, c.S), 7.0, device="cuda")
    q, k, _ = c.tensors()
    sa.cross_key_weights(q, k, lse, *c.ranges(), w, max_q_len=n)
    for s, l in zip(c.start, c.len):
        assert (w[:, s:s + l] - 2 * n / l).abs().max().item() <= 2 * n / l * (2.0 ** -19 + 2 * n * 2.0 ** -24)


@pytest.mark.parametrize("n", [1, 6, 40, 300])
def test_output_on_a_16_byte_boundary_and_padded_strides(n):
    H, Hkv, d = 8, 2, 64
    c = Case([(n, 400), (n, 65)], H, Hkv, d, seed=n)
    buf = torch.empty(c.T * H * d + 8, dtype=torch.bfloat16, device="cuda")
    o = buf[8:].view(c.T, H, d)
    q, k, v = c.tensors()
    qw = torch.empty(c.T, H * d + 24, dtype=torch.bfloat16, device="cuda")  # odd token strides
    qw[:, 16:16 + H * d] = q.reshape(c.T, -1)
    kw = torch.empty(c.S, Hkv * d + 8, dtype=torch.bfloat16, device="cuda")
    kw[:, :Hkv * d] = k.reshape(c.S, -1)
    lse = torch.empty(c.T, H, device="cuda")
    sa.cross_fwd(qw[:, 16:16 + H * d].view(c.T, H, d), kw[:, :Hkv * d].view(c.S, Hkv, d), v,
                 *c.ranges(), max_q_len=n, o=o, lse=lse)
    sa.check_device()
    c.check(o, lse, 0)


def test_malformed_sequences_are_skipped_and_reported():
    H, Hkv, d = 4, 2, 64
    for n in (1, 60):
        c = Case([(n, 100), (n, 50), (n, 80), (n, 64)], H, Hkv, d, seed=n, tail=0)
        q, k, v = c.tensors()
        cu, start, lens = c.ranges()
        start[1], lens[2] = -1, c.S  # in front of the states, and behind them
        o = torch.full_like(q, 77.0)
        w = torch.full((Hkv, c.S), 7.0, device="cuda")
        lse = torch.full((c.T, H), 77.0, device="cuda")
        sa.cross_fwd(q, k, v, cu, start, lens, max_q_len=n, o=o, lse=lse)
        with pytest.raises(sa.SattnError) as e:
            sa.check_device()
        assert e.value.code == 4
        assert torch.all(o[n:3 * n] == 77.0) and torch.all(lse[n:3 * n] == 77.0)
        sa.cross_key_weights(q, k, lse, cu, start, lens, w, max_q_len=n)
        with pytest.raises(sa.SattnError):
            sa.check_device()
        for b in (1, 2):
            assert torch.all(w[:, c.start[b]:c.start[b] + c.len[b]] == 7.0)
        ko, _, _, rows, _, kept = sa.evict_keys(k, v, w, start, lens, 16)
        with pytest.raises(sa.SattnError):
            sa.check_device()
        assert kept.tolist() == [16, 0, 0, 16]
        assert torch.all(ko[16:48] == 0) and torch.all(rows[:, 16:48] == -1)
        good = np.array([0, 3])
        wo, _ = oracle.cross_attend(c.q, c.k, c.v, c.cu, c.start, c.len, None, 0, c.scale)
        for b in good:
            err = np.abs(o[b * n:(b + 1) * n].float().cpu().numpy() - wo[b * n:(b + 1) * n])
            assert err.max() <= 0.05
        # cu_seqlens that fall, or reach behind T
        for bad in ([0, 5, 3, 4, 4], [1, 2, 3, 4, 4], [0, 1, 2, 3, c.T + 1]):
            sa.cross_fwd(q, k, v, cuda(np.array(bad, np.int32)), *c.ranges()[1:], max_q_len=n)
            with pytest.raises(sa.SattnError):
                sa.check_device()


@pytest.mark.parametrize("n", [1, 50])
def test_a_batch_without_queries(n):
    c = Case([(0, 100), (0, 3)], 4, 2, 64, tail=5)
    q, k, v = c.tensors()
    o, lse = torch.full_like(q, 77.0), torch.full((5, 4), 77.0, device="cuda")
    sa.cross_fwd(q, k, v, *c.ranges(), max_q_len=n, o=o, lse=lse)
    w = torch.full((2, c.S), 77.0, device="cuda")
    sa.cross_key_weights(q, k, lse, *c.ranges(), w, max_q_len=n)
    sa.check_device()
    assert torch.all(o == 77.0) and torch.all(lse == 77.0)
    for s, l in zip(c.start, c.len):
        assert torch.all(w[:, s:s + l] == 0.0)
    assert (w == 77.0).sum().item() == 2 * (c.S - 103)


def test_no_states_and_no_queries():
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    none = torch.empty(0, 2, 64, device="cuda").bfloat16()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    sinks = torch.randn(4, device="cuda")
    o, lse = sa.cross_fwd(q, none, none, cu, zero, zero, sinks=sinks, sink_mode=2)
    sa.check_device()
    assert torch.all(o == 0) and (lse - sinks).abs().max() < 1e-6
    kv = torch.randn(10, 2, 64, device="cuda").bfloat16()
    ten = torch.tensor([10], dtype=torch.int32, device="cuda")
    w = torch.full((2, 10), 3.0, device="cuda")
    args = q[:0], kv, torch.empty(0, 4, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    sa.cross_key_weights(*args, zero, ten, w, accumulate=True)
    assert torch.all(w == 3.0)
    sa.cross_key_weights(*args, zero, ten, w)
    assert torch.all(w == 0.0)
    sa.check_device()


class Job:
    """The four calls on one stream, with workspaces of their own, to the same outputs."""

    def __init__(self, lens, seed, H=8, Hkv=2, d=128):
        self.c = c = Case(lens, H, Hkv, d, seed=seed, tail=0)
        self.q, self.k, self.v = c.tensors()
        self.n = int(c.n.max())
        self.r = c.ranges()
        self.ws = torch.full((sa.cross_workspace_bytes(self.n, H, Hkv, d),), 0xFF,
                             dtype=torch.uint8, device="cuda")
        self.ws2 = torch.full((4 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
        self.o = torch.empty_like(self.q)
        self.lse = torch.empty(c.T, H, device="cuda")
        self.w = torch.full((Hkv, c.S), 77.0, device="cuda")  # (rows of no sequence keep it)
        B = len(lens)
        self.kept = [torch.empty(B * 64, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        self.kept += [torch.empty(Hkv, B * 64, device="cuda")]
        self.kept += [torch.empty(s, dtype=torch.int32, device="cuda") for s in ((Hkv, B * 64), B, B)]

    def run(self, stream=None):
        sa.cross_fwd(self.q, self.k, self.v, *self.r, max_q_len=self.n, o=self.o, lse=self.lse,
                     workspace=self.ws, stream=stream)
        sa.cross_key_weights(self.q, self.k, self.lse, *self.r, self.w, max_q_len=self.n,
                             workspace=self.ws2, stream=stream)
        sa.evict_keys(self.k, self.v, self.w, *self.r[1:], 64, 0, 0, *self.kept, stream=stream)

    def outs(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.o, self.lse, self.w, *self.kept)]

    def spoil(self):
        for t in (self.o, self.lse, self.w, *self.kept):
            t.fill_(77)
        self.ws.fill_(0xFF), self.ws2.fill_(0xFF)


LENS = {"few": [(1, 3000), (1, 70), (1, 5000), (2, 900)],
        "some": [(12, 2000), (9, 333)],
        "many": [(200, 1500), (77, 4000), (3, 130)]}


@pytest.mark.parametrize("a,b", [("few", "few"), ("many", "few"), ("many", "many"), ("some", "few")])
def test_two_streams_at_once(a, b):
    jobs = [Job(LENS[a], 1), Job(LENS[b], 2)]
    want = []
    for j in jobs:
        j.run()
        want.append(j.outs())
        sa.check_device()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for j in jobs:
            j.spoil()
        torch.cuda.synchronize()
        for _ in range(3):
            for j, s in zip(jobs, streams):
                j.run(s)
        for j, w in zip(jobs, want):
            assert all(torch.equal(x, y) for x, y in zip(j.outs(), w))  # bit for bit
    sa.check_device()


@pytest.mark.parametrize("kind", list(LENS))
def test_captured_calls_replay_with_other_lengths(kind):
    j = Job(LENS[kind], 3)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        j.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            j.run()
    first = [t.clone() for t in j.r]
    for other in (False, True, False):
        if other:  # fewer states, an empty sequence, fewer queries
            j.r[2].copy_(torch.tensor([max(0, int(x) - 61) for x in first[2][:-1]] + [0],
                                      dtype=torch.int32))
            j.r[0].copy_((first[0] // 2).int())
        else:
            for t, f in zip(j.r, first):
                t.copy_(f)
        j.spoil()
        g.replay()
        got = j.outs()
        j.spoil()
        j.run()
        live = int(j.r[0][-1])
        assert torch.equal(got[0][:live], j.o[:live]) and torch.equal(got[1][:live], j.lse[:live])
        assert all(torch.equal(x, y) for x, y in zip(got[2:], j.outs()[2:]))
        sa.check_device()


@pytest.mark.parametrize("what", ["cross", "weights"])
@pytest.mark.parametrize("kind", list(LENS))
def test_a_wait_that_runs_out_is_reported(kind, what):
    j = Job(LENS[kind], 4)
    j.run()
    want = j.outs()
    sa.set_test_wait_stall(True)
    sa.set_wait_limit_ns(2_000_000)
    try:
        if what == "cross":
            sa.cross_fwd(j.q, j.k, j.v, *j.r, max_q_len=j.n, workspace=j.ws)
        else:
            sa.cross_key_weights(j.q, j.k, j.lse, *j.r, j.w.clone(), max_q_len=j.n,
                                 workspace=j.ws2)
        with pytest.raises(sa.SattnError) as e:
            sa.check_device()
        assert e.value.code == 5
    finally:
        sa.set_test_wait_stall(False)
        sa.set_wait_limit_ns(0)
    j.spoil()
    j.run()
    sa.check_device()
    assert all(torch.equal(x, y) for x, y in zip(j.outs(), want))


def test_outputs_made_on_a_side_stream_belong_to_it():
    j = Job(LENS["few"], 5)
    j.run()
    want = j.outs()
    s = torch.cuda.Stream()
    for _ in range(30):
        torch.cuda._sleep(200_000)  # the current stream is behind
        o, lse = sa.cross_fwd(j.q, j.k, j.v, *j.r, max_q_len=j.n, stream=s)
        del o, lse
        o, lse = sa.cross_fwd(j.q, j.k, j.v, *j.r, max_q_len=j.n, stream=s)
        junk = torch.full_like(o, 3.0)  # on the current stream
        s.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        del junk
    sa.check_device()


def test_argument_checks():
    c = Case([(2, 30)], 4, 2, 64, tail=0)
    q, k, v = c.tensors()
    cu, start, lens = c.ranges()
    lse, w = torch.zeros(2, 4, device="cuda"), torch.zeros(2, c.S, device="cuda")
    bad = [dict(q=q.float()), dict(q=q.cpu()), dict(k=k[:, :, :32]), dict(v=v[1:]),
           dict(v=v.transpose(1, 2)), dict(cu=cu.long()), dict(cu=cu[:1]), dict(start=start.cpu()),
           dict(lens=lens[:0])]
    for kw in bad:
        a = dict(q=q, k=k, v=v, cu=cu, start=start, lens=lens)
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            sa.cross_fwd(*a.values())
    with pytest.raises(ValueError):
        sa.cross_fwd(q, k, v, cu, start, lens, sinks=torch.zeros(3, device="cuda"), sink_mode=1)
    with pytest.raises(ValueError):
        sa.cross_fwd(q, k, v, cu, start, lens, o=torch.empty(2, 4, 64, device="cuda"))
    for kw in (dict(lse=lse[:1]), dict(w=w[:1]), dict(w=None), dict(lse=None), dict(w=w.double())):
        a = dict(q=q, k=k, lse=lse, cu=cu, start=start, lens=lens, w=w)
        a.update(kw)
        with pytest.raises(ValueError):
            sa.cross_key_weights(*a.values())
    for kw in (dict(w=w[:, 1:]), dict(w=None), dict(keep=0), dict(v=v[:-1])):
        a = dict(k=k, v=v, w=w, start=start, lens=lens, keep=4)
        a.update(kw)
        with pytest.raises(ValueError):
            sa.evict_keys(*a.values())
    with pytest.raises(sa.SattnError):
        sa.evict_keys(k, v, w, start, lens, 4, first=3, last=2)
    pos = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    f, ax = torch.ones(16, device="cuda"), torch.zeros(16, dtype=torch.uint8, device="cuda")
    for kw in (dict(pos=pos.long()), dict(pos=pos[:, :1]), dict(f=f[:8]), dict(ax=ax.int()),
               dict(q=q.half()), dict(k=k)):
        a = dict(q=q, k=None, pos=pos, f=f, ax=ax)
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            sa.rope_axes(*a.values())
    with pytest.raises(sa.SattnError):  # rd is 8
        sa.rope_axes(q, None, pos, f[:4], ax[:4])


def test_calls_repeat_bit_for_bit():
    for kind in LENS:
        j = Job(LENS[kind], 6)
        j.run()
        want = j.outs()
        for _ in range(12):
            j.spoil()
            j.run()
            assert all(torch.equal(x, y) for x, y in zip(j.outs(), want))


@pytest.mark.parametrize("dtype", list(DT))
def test_rope_axes_captured_and_on_a_side_stream(dtype):
    T, H, d = 300, 4, 128
    x = torch.randn(T, H, d, device="cuda").to(DT[dtype])
    pos = torch.randint(0, 1000, (3, T), dtype=torch.int32, device="cuda")
    f = torch.rand(64, device="cuda")
    ax = (torch.arange(64, device="cuda") % 3).to(torch.uint8)
    want = sa.rope_axes(x, None, pos, f, ax)[0]
    s, y = torch.cuda.Stream(), torch.empty_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        sa.rope_axes(x, None, pos, f, ax, q_out=y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    got = sa.rope_axes(x, None, pos, f, ax, stream=s)[0]
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("n,G,d", [(1, 8, 128), (6, 1, 64), (6, 5, 128), (15, 4, 64), (8, 8, 128),
                                   (100, 2, 64)])
def test_one_sequence_in_more_pieces_than_a_warp_has_lanes(n, G, d, mode):
    # 129 tiles of keys: a piece each on up to 152 SMs
    c = Case([(n, 16411)], G, 1, d, seed=n)
    c.check(*attend(c, mode), mode)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,Hkv", [(1, 2), (9, 2), (3, 3), (2, 4)])
def test_heads_side_by_side_in_many_pieces(n, Hkv, d):
    # an even number of KV heads goes by pairs; a unit's pieces are then every other CTA's
    c = Case([(n, 16411), (n, 3)], 3 * Hkv, Hkv, d, seed=Hkv)
    c.check(*attend(c, 2), 2)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("Hkv,d", [(2, 64), (2, 128), (3, 64)])
def test_key_weights_of_more_queries_than_the_hint_says(Hkv, d, accumulate):
    # the form of few rows with many steps a unit: its units are cut between CTAs
    c = Case([(700, 513), (1, 4), (33, 90)], 2 * Hkv, Hkv, d, seed=d)
    lse = c.check(*attend(c, 1), 1)
    full = np.zeros((c.T, 2 * Hkv), np.float32)
    full[:len(lse)] = lse
    before = np.random.default_rng(1).random((Hkv, c.S)).astype(np.float32)
    w = cuda(before)
    q, k, _ = c.tensors()
    sa.cross_key_weights(q, k, cuda(full), *c.ranges(), w, max_q_len=1, accumulate=accumulate,
                         sinks=cuda(c.sinks), sink_mode=1)
    sa.check_device()
    c.check_weights(w.cpu().numpy(), full, before, accumulate, 1)
