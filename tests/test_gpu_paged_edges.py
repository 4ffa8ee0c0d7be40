"""The paged FP8 cache at its edges: NaN in places that only some rows see,
queries and sinks of extreme size, many short sequences, odd head layouts, calls
that run at once, waits that run out, and the binding's refusals.

Tolerances are those of the plain cases (1e-2 and o's own rounding for bf16
queries, 1e-4 for fp32 ones): every case is compared with the fp64 oracle on the
same codes."""
import numpy as np
import pytest
import torch

import oracle
import windowed_attention_sinks_gb300 as sa

from gpu_helpers import TOL_BF16_O, TOL_F32_O, compare
from test_gpu_paged import DT, Batch, attend, cuda, filled

pytestmark = pytest.mark.gpu

TOL = {"bf16": TOL_BF16_O, "f32": TOL_F32_O}


def seen(b, window, causal):
    """For each sequence the [n, L] mask of what its rows see."""
    out = []
    for n, L in zip(b.n, b.kv_lens):
        pos, j = (L - n + np.arange(n))[:, None], np.arange(L)[None]
        m = j <= pos if causal else np.ones((n, L), bool)
        out.append(m & (j >= pos - window) if window >= 0 else m)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("lens", [[(500, 4), (3, 4), (0, 1)], [(200, 8), (127, 5)],
                                  [(300, 150), (0, 70)], [(6000, 4)], [(6000, 40)]])
@pytest.mark.parametrize("window", [-1, 30])
def test_nan_codes_reach_the_rows_that_see_them(window, lens, d, page, dtype):
    """A NaN value spoils its column of the rows that see its key, a NaN key the
    whole of them; every other number is as without."""
    rng = np.random.default_rng(page)
    b = Batch(lens, page)
    H, Hkv = 4, 2
    kc, ks = filled(rng, b, Hkv, d)
    vc, vs = filled(rng, b, Hkv, d)
    q = rng.standard_normal((b.T, H, d)).astype(np.float32)
    if dtype == "bf16":
        q = oracle.bf16_round(q)
    ro, rl = oracle.paged_attend(q, *(np.where(c & 0x7F == 0x7F, 0, c).astype(np.uint8)
                                      for c in (kc, vc)), ks, vs, b.table, b.cu, b.kv_lens, 1,
                                 window, None, 0, d ** -0.5)
    bad_o, bad_row = np.zeros(ro.shape, bool), np.zeros(rl.shape, bool)
    for i, m in enumerate(seen(b, window, True)):
        n, L = m.shape
        # values: one column of a new key of head 0, all of another of head 1
        for g, key, cols in ((0, L - 1, slice(3, 4)), (1, max(0, L - 2), slice(0, d)),
                             (0, max(0, L - n // 2 - 1), slice(d - 1, d))):
            vc[b.table[i, key // page], g, key % page, cols] = 0xFF if g else 0x7F
            rows = b.cu[i] + np.nonzero(m[:, key])[0]
            for h in range(g * 2, g * 2 + 2):
                bad_o[rows, h, cols] = True
    if len(b.n) > 1:  # a key, in the second sequence
        m = seen(b, window, True)[1]
        key = m.shape[1] - 1 - m.shape[0] // 3
        kc[b.table[1, key // page], 1, key % page, 5] = 0x7F
        bad_row[b.cu[1] + np.nonzero(m[:, key])[0], 2:] = True
        bad_o[bad_row] = True
    o, lse = sa.paged_fp8_fwd(cuda(q, DT[dtype]), cuda(kc), cuda(vc), cuda(ks), cuda(vs),
                              *b.tensors(), max_q_len=int(b.n.max()), window_left=window)
    sa.check_device()
    got = o.float().cpu().numpy()
    assert np.array_equal(np.isnan(got), bad_o)
    assert np.array_equal(np.isnan(lse.cpu().numpy()), bad_row)
    fix = torch.from_numpy(bad_o).cuda()
    o[fix] = torch.from_numpy(ro).to(o.dtype).cuda()[fix]
    rows = torch.from_numpy(bad_row).cuda()
    lse[rows] = torch.from_numpy(rl).float().cuda()[rows]
    compare(o, lse, ro, rl, TOL[dtype])


@pytest.mark.parametrize("n", [1, 4, 70])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_spoilt_query_spoils_its_own_row(value, n):
    rng = np.random.default_rng(n)
    b = Batch([(400, n), (30, n)], 64)
    kc, ks = filled(rng, b, 1, 128)
    vc, vs = filled(rng, b, 1, 128)
    q = oracle.bf16_round(rng.standard_normal((b.T, 8, 128)).astype(np.float32))
    args = (cuda(kc), cuda(vc), cuda(ks), cuda(vs), *b.tensors())
    want, wl = sa.paged_fp8_fwd(cuda(q, torch.bfloat16), *args, max_q_len=n)
    q[n, 3, 77] = value
    o, lse = sa.paged_fp8_fwd(cuda(q, torch.bfloat16), *args, max_q_len=n)
    sa.check_device()
    assert torch.isnan(o[n, 3]).all() and torch.isnan(lse[n, 3])
    o[n, 3], lse[n, 3] = want[n, 3], wl[n, 3]
    # the other rows' maxima may move at other keys: both are within the tolerance
    # of the exact result, of which probabilities take up to half
    assert torch.allclose(o.float(), want.float(), rtol=2.0 ** -7, atol=TOL_BF16_O)
    assert torch.allclose(lse, wl, rtol=0, atol=1e-3)


@pytest.mark.parametrize("n", [1, 4, 70])
def test_rows_of_very_different_sizes(n):
    """Rows of a KV group that are 2^40 apart keep their own precision: the large
    ones meet zeros in every key's first column, the small ones are scaled up by
    the softmax's scale."""
    rng = np.random.default_rng(n)
    b = Batch([(700, n), (30, n)], 64)
    kc, ks = filled(rng, b, 1, 128)
    kc[..., 0] = 0
    vc, vs = filled(rng, b, 1, 128)
    q = np.zeros((b.T, 8, 128), np.float32)
    q[:, ::2, 0] = 2.0 ** 20
    q[:, 1::2] = rng.standard_normal((b.T, 4, 128)) * 2.0 ** -20
    q = oracle.bf16_round(q)
    scale = 128 ** -0.5 * 2.0 ** 20
    o, lse = sa.paged_fp8_fwd(cuda(q, torch.bfloat16), cuda(kc), cuda(vc), cuda(ks), cuda(vs),
                              *b.tensors(), max_q_len=n, scale=scale)
    sa.check_device()
    kc[kc == 0x7F], vc[vc == 0x7F] = 0, 0
    ro, rl = oracle.paged_attend(q, kc, vc, ks, vs, b.table, b.cu, b.kv_lens, 1, -1, None, 0, scale)
    compare(o, lse, ro, rl, TOL_BF16_O)


@pytest.mark.parametrize("n", [1, 4, 70])
@pytest.mark.parametrize("scale", [1.0, 1e5, 1e8, 1e20, 1e33])
def test_logits_of_any_size(scale, n):
    """Keys with one 1 each and queries of distinct integers: every logit is exact,
    and from some size on a row is the mean of the values of its largest ones. (A
    logit is at most 128 * 128 scale, in fp32's range for each scale here.)"""
    rng = np.random.default_rng(n)
    b = Batch([(700, n), (30, n), (0, n)], 64)
    kc = np.zeros((b.pages, 1, 64, 128), np.uint8)
    kc[:, 0, np.arange(64), rng.integers(0, 128, (b.pages, 64))] = 0x38  # 1.0
    vc, _ = filled(rng, b, 1, 128)
    ks, vs = np.ones((b.pages, 1), np.float32), np.full((b.pages, 1), 2.0 ** -7, np.float32)
    q = np.stack([rng.permutation(128) + 1 for _ in range(b.T * 8)]).reshape(b.T, 8, 128)
    q = (q * np.where(rng.random((b.T, 8, 1)) < 0.5, 1, -1)).astype(np.float32)
    o, lse = sa.paged_fp8_fwd(cuda(q, torch.bfloat16), cuda(kc), cuda(vc), cuda(ks), cuda(vs),
                              *b.tensors(), max_q_len=n, scale=scale)
    sa.check_device()
    vc[vc == 0x7F] = 0
    ro, rl = oracle.paged_attend(q, kc, vc, ks, vs, b.table, b.cu, b.kv_lens, 1, -1, None, 0, scale)
    assert np.allclose(lse.cpu().numpy(), rl, rtol=1e-6, atol=1e-3)
    compare(o, None, ro, rl, TOL_BF16_O)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 4, 70])
@pytest.mark.parametrize("mode", [1, 2])
def test_sinks_of_extreme_size(mode, n, dtype):
    """The largest finite values and infinities. A bias of the lowest value leaves
    key 0 to the rows that see nothing else."""
    rng = np.random.default_rng(n)
    big = float(np.finfo(np.float32).max)
    sinks = np.array([-big, -np.inf, -1e30, 1e30, -3e4, 3e4, 0.5, big], np.float32)
    b = Batch([(0, n), (150, n), (1, n)], 32)
    kc, ks = filled(rng, b, 2, 64)
    vc, vs = filled(rng, b, 2, 64)
    q = oracle.bf16_round(rng.standard_normal((b.T, 8, 64)).astype(np.float32))
    o, lse = sa.paged_fp8_fwd(cuda(q, DT[dtype]), cuda(kc), cuda(vc), cuda(ks), cuda(vs),
                              *b.tensors(), max_q_len=n, sinks=cuda(sinks), sink_mode=mode)
    sa.check_device()
    kc[kc == 0x7F], vc[vc == 0x7F] = 0, 0
    ro, rl = oracle.paged_attend(q, kc, vc, ks, vs, b.table, b.cu, b.kv_lens, 1, -1, sinks, mode,
                                 64 ** -0.5)
    far = np.abs(rl) > 1e4  # of the size of the sink: to fp32's precision, within its clamp
    got = lse.cpu().numpy()
    far &= ~np.isinf(rl)
    assert np.allclose(got[far & (np.abs(rl) < 2e38)], rl[far & (np.abs(rl) < 2e38)], rtol=1e-6)
    assert np.all(np.abs(got[far & (np.abs(rl) > 2e38)]) > 2e38)
    lse[torch.from_numpy(far).cuda()] = 0.0
    rl[far] = 0.0
    compare(o, lse, ro, rl, TOL[dtype])


@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_window_is_none(n, dtype):
    b = Batch([(0, n), (300, n), (0, n)], 32)
    b.kv_lens[2] = max(0, n - 3)  # rows in front of position 0
    for window in (2 ** 30, 2 ** 31 - 1):
        attend(b, 4, 2, 64, dtype, window=window)
        attend(b, 4, 2, 64, dtype, causal=False, window=window)


@pytest.mark.parametrize("H,Hkv,window,B", [(8, 2, -1, 150), (4, 4, 20, 150), (8, 1, 300, 450)])
def test_many_sequences_of_single_tokens(H, Hkv, window, B):
    """Units of one or two tiles, which the kernel's halves take by themselves, among
    longer ones, with empty sequences between them."""
    rng = np.random.default_rng(B)
    lens = [(int(rng.integers(0, 200 if i % 9 else 2500)), int(i % 7 != 3)) for i in range(B)]
    attend(Batch(lens, 32), H, Hkv, 64, window=window, mode=2)


@pytest.mark.parametrize("window", [-1, 40])
def test_many_prompts(window):
    rng = np.random.default_rng(3)
    lens = [(int(rng.integers(0, 300)), int(rng.integers(0, 40))) for _ in range(90)]
    attend(Batch(lens, 16), 6, 2, 64, window=window, mode=1)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (5, 1), (17, 1), (64, 1), (130, 1), (260, 2), (9, 3)])
def test_prompts_of_odd_head_layouts(H, Hkv):
    attend(Batch([(300, 40), (0, 3), (77, 1), (5, 131)], 32), H, Hkv, 128, mode=2)


@pytest.mark.parametrize("n", [1, 70])
def test_calls_at_once(n):
    """Two streams, each with its own workspace; and a captured call replayed
    beside several rings' worth of eager ones."""
    torch.manual_seed(0)
    rng = np.random.default_rng(0)
    H, Hkv, d = 8, 2, 128
    jobs = []
    for seed, lens in enumerate(([(9000, n), (300, n)], [(4000, n), (5000, n), (1, n)])):
        b = Batch(lens, 64, seed)
        pool = [cuda(x) for x in (*filled(rng, b, Hkv, d), *filled(rng, b, Hkv, d))]
        q = torch.randn(b.T, H, d, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(sa.paged_fp8_workspace_bytes(n, H, Hkv, d), dtype=torch.uint8,
                         device="cuda")
        jobs.append((q, pool, b.tensors(), ws))

    def run(job, o=None, lse=None):
        q, (kc, ks, vc, vs), where, ws = job
        return sa.paged_fp8_fwd(q, kc, vc, ks, vs, *where, max_q_len=n, workspace=ws, o=o, lse=lse)

    want = [[t.clone() for t in run(j)] for j in jobs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(jobs[0])
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(t) for t in w] for w in want]
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(300):
        with torch.cuda.stream(sides[0]):
            graph.replay()
            bad0 = sum((x != y).sum() for x, y in zip(held, want[0]))
            bad += bad0
        with torch.cuda.stream(sides[1]):
            run(jobs[1], *outs[1])
    torch.cuda.synchronize()
    sa.check_device()
    assert bad.item() == 0
    assert all(torch.equal(x, y) for x, y in zip(outs[1], want[1]))


@pytest.mark.parametrize("n", [1, 4, 70])
def test_a_wait_that_runs_out(n):
    """The issuing threads wait for what nothing completes (2 ms); the call reports
    it, and the next one is right."""
    b = Batch([(5000, n), (64, n), (900, n)], 64)
    want = attend(b, 8, 2, 128)
    pool = [cuda(x) for x in filled(np.random.default_rng(0), b, 2, 128)]
    q = torch.zeros(b.T, 8, 128, dtype=torch.bfloat16, device="cuda")
    sa.set_test_wait_stall(True)
    sa.set_wait_limit_ns(2_000_000)
    try:
        sa.paged_fp8_fwd(q, pool[0], pool[0], pool[1], pool[1], *b.tensors(), max_q_len=n)
        with pytest.raises(sa.SattnError) as err:
            sa.check_device()
    finally:
        sa.set_test_wait_stall(False)
        sa.set_wait_limit_ns(0)
    assert err.value.code == 5
    for _ in range(2):
        got = attend(b, 8, 2, 128)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_refusals():
    b = Batch([(5, 2), (0, 3)], 16)
    rng = np.random.default_rng(0)
    kc, ks = (cuda(x) for x in filled(rng, b, 2, 64))
    q = torch.zeros(b.T, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(b.T, 2, 64, dtype=torch.bfloat16, device="cuda")
    table, cu, lens = b.tensors()
    good = dict(k_cache=kc, v_cache=kc.clone(), k_scale=ks, v_scale=ks.clone(), page_table=table,
                cu_seqlens=cu, kv_lens=lens)
    cs = torch.zeros(32, 64, device="cuda")
    sa.paged_fp8_fwd(q, **good)
    sa.paged_fp8_append(k, k, **good, cos_sin=cs, q=q)
    bad_cache = (dict(k_cache=kc.cpu()), dict(k_cache=kc.float()), dict(v_cache=kc[:, :1]),
                 dict(k_scale=ks.double()), dict(v_scale=ks[:, :1]), dict(page_table=table.long()),
                 dict(page_table=table[0]), dict(cu_seqlens=cu[:-1]), dict(kv_lens=lens[:-1]),
                 dict(kv_lens=lens.cpu()), dict(k_cache=kc.transpose(1, 2)))
    for bad in bad_cache:
        with pytest.raises(ValueError):
            sa.paged_fp8_fwd(q, **{**good, **bad})
        with pytest.raises(ValueError):
            sa.paged_fp8_append(k, k, **{**good, **bad})
    with pytest.raises(TypeError):
        sa.paged_fp8_fwd(q.half(), **good)
    for bad in (dict(q=q[..., :32]), dict(q=q.transpose(0, 1)),
                dict(q=q.cpu()), dict(sinks=torch.zeros(3, device="cuda")),
                dict(o=torch.empty(b.T, 4, 64, device="cuda")), dict(lse=q[..., 0]),
                dict(workspace=torch.empty(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            sa.paged_fp8_fwd(**{**good, "q": q, **bad})
    for bad in (dict(v=k[:, :1]), dict(v=k.float()), dict(q=q.float()), dict(q_out=q),
                dict(cos_sin=cs.double()), dict(cos_sin=cs[:, ::2]), dict(q=q, q_out=q[:-1])):
        with pytest.raises(ValueError):
            sa.paged_fp8_append(**{**good, "k": k, "v": k, **bad})
    for bad in (dict(q=q[:, :3]), dict(sink_mode=1), dict(scale=0.0), dict(causal=True, scale=-1.0)):
        with pytest.raises((sa.SattnError, ValueError)):
            sa.paged_fp8_fwd(**{**good, "q": q, **bad})
    with pytest.raises((sa.SattnError, ValueError)):
        sa.paged_fp8_append(k, k, **good, q=q)  # nothing to rotate them by
    sa.check_device()
