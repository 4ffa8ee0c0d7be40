"""GPU parity of the paged FP8 cache: the append against the oracle's coding
rules, the attention against the fp64 oracle on the same codes, and the two run
one after the other as a serving loop does.

Tolerances. Codes and scales of unrotated rows are exact: scales are powers of
two, so x / s is exact and rounded once. A rotated key is computed in fp32
(error below 2^-22 (|a| + |b|)) and rounded to e4m3: within half a step, at most
2^-4 |x|, or 2^-10 s below the normal range. Rotated bf16 queries are off by
their rounding, 2^-8 |x|. Attention: the bounds of the other bf16 kernels (1e-2
and o's own rounding; probabilities keep 8 significant bits, so their share is
below 2^-8 sum p |v|, under 5e-3 here), 1e-4 for fp32 queries."""
import numpy as np
import pytest
import torch

import oracle
import windowed_attention_sinks_gb300 as sa

from gpu_helpers import TOL_BF16_O, TOL_F32_O, compare

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def cuda(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


class Batch:
    """Sequences given as (cached, new) and pages that lie anywhere in a pool."""

    def __init__(self, lens, page, seed=0, spare=2, width=None):
        rng = np.random.default_rng(seed)
        self.page = page
        self.n = np.array([n for _, n in lens])
        self.kv_lens = np.array([kv + n for kv, n in lens], np.int32)
        self.cu = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.T = int(self.cu[-1])
        used = -(-self.kv_lens // page)
        self.pages = int(used.sum()) + spare
        width = width or max(1, int(used.max(initial=0)))
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(lens), width), -1, np.int32)  # unused entries are no pages
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at: at + u]
            at += u

    def tensors(self):
        return cuda(self.table), cuda(self.cu), cuda(self.kv_lens)


def filled(rng, b, Hkv, d):
    """A pool with codes in every row (random scales a page), NaN codes in the
    rows that hold no position."""
    codes = oracle.e4m3_encode(rng.standard_normal((b.pages, Hkv, b.page, d)) * 100)
    scale = (2.0 ** rng.integers(-9, -5, (b.pages, Hkv))).astype(np.float32)
    live = np.zeros((b.pages, b.page), bool)
    for row, L in zip(b.table, b.kv_lens):
        for p in range(L):
            live[row[p // b.page], p % b.page] = True
    codes[np.broadcast_to(~live[:, None, :, None], codes.shape)] = 0x7F
    return codes, scale


def rope_table(rows, rd):
    ang = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, rd, 2) / rd)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


# ------------------------------------------------------------------ append

LENS = {
    "one": [(0, 1)],
    "decode": [(5, 1), (0, 1), (15, 1), (16, 1), (63, 1), (64, 1), (200, 1), (127, 1), (128, 1)],
    "ragged": [(0, 7), (3, 40), (16, 0), (0, 0), (31, 33), (64, 129), (130, 1), (0, 300)],
    "many": [(i % 37, 1 + i % 3) for i in range(70)],
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,d,Hkv", [(16, 64, 3), (64, 128, 2), (128, 128, 1), (32, 64, 8)])
@pytest.mark.parametrize("lens", list(LENS))
def test_append_without_rotation_is_exact(lens, page, d, Hkv, dtype):
    rng = np.random.default_rng(page + d)
    b = Batch(LENS[lens], page)
    codes, scale = filled(rng, b, Hkv, d)
    x = (rng.standard_normal((2, b.T, Hkv, d)) * np.exp(rng.standard_normal((2, b.T, 1, 1)) * 2)
         ).astype(np.float32)
    if dtype == "bf16":
        x = oracle.bf16_round(x)
    kc, vc, ks, vs = cuda(codes), cuda(codes), cuda(scale), cuda(scale)
    k, v = cuda(x[0], DT[dtype]), cuda(x[1], DT[dtype])
    for _ in range(2):  # the second call changes nothing
        sa.paged_fp8_append(k, v, kc, vc, ks, vs, *b.tensors())
        sa.check_device()
        for name, c, s, rows in (("k", kc, ks, x[0]), ("v", vc, vs, x[1])):
            wc, ws = oracle.paged_append(rows, codes, scale, b.table, b.cu, b.kv_lens)
            assert np.array_equal(s.cpu().numpy(), ws), name
            assert np.array_equal(c.cpu().numpy(), wc), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rd,inter", [(128, 128, False), (128, 128, True), (128, 64, False),
                                        (64, 16, True), (64, 64, False), (128, 48, True)])
@pytest.mark.parametrize("lens", ["decode", "ragged"])
def test_append_rotates_keys_and_queries(lens, d, rd, inter, dtype):
    rng = np.random.default_rng(rd + d)
    page, Hkv, H = 64, 2, 6
    b = Batch(LENS[lens], page)
    codes, scale = filled(rng, b, Hkv, d)
    x = rng.standard_normal((b.T + 3, H + 2 * Hkv, d)).astype(np.float32)
    if dtype == "bf16":
        x = oracle.bf16_round(x)
    cs = rope_table(512, rd)
    qkv = cuda(x, DT[dtype])  # one projection's output: q, k and v are slices of it
    kc, vc, ks, vs = cuda(codes), cuda(codes), cuda(scale), cuda(scale)
    q_out = torch.full((b.T + 3, H, d), 77.0, dtype=DT[dtype], device="cuda")
    got = sa.paged_fp8_append(qkv[:, H:H + Hkv], qkv[:, H + Hkv:], kc, vc, ks, vs, *b.tensors(),
                              cos_sin=cuda(cs), interleaved=inter, q=qkv[:, :H], q_out=q_out)
    sa.check_device()
    assert got is q_out
    pos = np.concatenate([np.arange(L - n, L) for L, n in zip(b.kv_lens, b.n)]).astype(int)
    wq = oracle.rotate(x[:b.T, :H], cs, pos, inter)
    err = np.abs(q_out[:b.T].float().cpu().numpy() - wq)
    near = np.abs(x).max() * 2.0 ** -21
    assert np.all(err <= (2.0 ** -8 * np.abs(wq) if dtype == "bf16" else 0) + near)
    assert torch.all(q_out[b.T:] == 77.0)  # behind the last sequence
    wk = oracle.rotate(x[:b.T, H:H + Hkv], cs, pos, inter)
    wc, ws = oracle.paged_append(wk, codes, scale, b.table, b.cu, b.kv_lens)
    gs, gc = ks.cpu().numpy(), kc.cpu().numpy()
    assert np.array_equal(gs, ws)
    fresh = 0
    for q_row, (L, n) in enumerate(zip(b.kv_lens, b.n)):
        for p in range(L - n, L):
            pid = b.table[q_row, p // page]
            val = oracle.e4m3_decode(gc[pid, :, p % page]) * gs[pid][:, None]
            want = wk[fresh]
            fresh += 1
            tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * gs[pid][:, None]) + near
            assert np.all(np.abs(val - want) <= tol)
    # everything but the new rows is as the oracle has it, bit for bit
    new = np.zeros((b.pages, page), bool)
    for row, L, n in zip(b.table, b.kv_lens, b.n):
        for p in range(L - n, L):
            new[row[p // page], p % page] = True
    keep = np.broadcast_to(~new[:, None, :, None], gc.shape)
    assert np.array_equal(gc[keep], wc[keep])
    wv, wvs = oracle.paged_append(x[:b.T, H + Hkv:], codes, scale, b.table, b.cu, b.kv_lens)
    assert np.array_equal(vc.cpu().numpy(), wv) and np.array_equal(vs.cpu().numpy(), wvs)


def test_append_special_values():
    """NaN is stored and sets no scale, infinities are stored as the largest
    value, zeros take the least scale, -0 keeps its sign."""
    page, d = 16, 64
    b = Batch([(0, 3), (0, 1), (0, 2), (0, 1)], page, spare=0)
    x = np.zeros((b.T, 1, d), np.float32)
    x[0], x[1, 0, 5], x[2, 0, 0] = 1.0, np.nan, 2.0
    x[3, 0, 1] = -0.0
    x[4, 0, :3] = [np.inf, -np.inf, 1.0]
    x[6] = 1e-30
    kc = torch.full((b.pages, 1, page, d), 0x11, dtype=torch.uint8, device="cuda")
    ks = torch.full((b.pages, 1), 3.0, device="cuda")
    vc, vs = kc.clone(), ks.clone()
    sa.paged_fp8_append(cuda(x), cuda(x), kc, vc, ks, vs, *b.tensors())
    sa.check_device()
    wc, ws = oracle.paged_append(x, np.full((b.pages, 1, page, d), 0x11, np.uint8),
                                 np.full((b.pages, 1), 3.0, np.float32), b.table, b.cu, b.kv_lens)
    assert np.array_equal(ks.cpu().numpy(), ws) and np.array_equal(kc.cpu().numpy(), wc)
    assert ws[b.table[0, 0], 0] == 2.0 ** -7 and ws[b.table[1, 0], 0] == 2.0 ** -64
    assert kc[b.table[0, 0], 0, 1, 5] == 0x7F


def test_append_queries_in_place_and_empty_calls():
    b = Batch([(4, 2), (0, 3)], 16)
    rng = np.random.default_rng(0)
    q = cuda(rng.standard_normal((b.T, 4, 64)).astype(np.float32))
    k = cuda(rng.standard_normal((b.T, 2, 64)).astype(np.float32))
    cs = cuda(rope_table(32, 64))

    def pool():
        return [torch.zeros(b.pages, 2, 16, 64, dtype=torch.uint8, device="cuda") for _ in "kv"] + [
            torch.ones(b.pages, 2, device="cuda") for _ in "kv"]

    want = sa.paged_fp8_append(k, k, *pool(), *b.tensors(), cos_sin=cs, q=q)
    got = sa.paged_fp8_append(k, k, *pool(), *b.tensors(), cos_sin=cs, q=q, q_out=q)
    assert got is q and torch.equal(got, want)
    none = sa.paged_fp8_append(k[:0], k[:0], *pool(), *b.tensors())
    assert none is None
    sa.check_device()


def test_append_reports_what_it_skips():
    """A sequence that does not fit and a table entry that is no page are
    reported; the others are stored."""
    page, d = 16, 64
    rng = np.random.default_rng(4)
    x = rng.standard_normal((12, 1, d)).astype(np.float32)
    good = Batch([(0, 4), (3, 4), (0, 4)], page, spare=0)
    for what in ("short", "table", "page", "rope", "cu"):
        kc = torch.full((good.pages, 1, page, d), 0x11, dtype=torch.uint8, device="cuda")
        ks = torch.ones(good.pages, 1, device="cuda")
        lens, table, cu = good.kv_lens.copy(), good.table.copy(), good.cu.copy()
        cos_sin = None
        if what == "short":
            lens[1] = 3
        elif what == "table":
            lens[1] = 2 * page
        elif what == "page":
            table[1, 0] = good.pages
        elif what == "rope":
            cos_sin = cuda(rope_table(6, 16))
        else:
            cu[2] = 100
        sa.paged_fp8_append(cuda(x), cuda(x), kc, kc.clone(), ks, ks.clone(), cuda(table), cuda(cu),
                            cuda(lens), cos_sin=cos_sin)
        with pytest.raises(sa.SattnError):
            sa.check_device()
        sa.check_device()  # cleared
        assert torch.all(kc[good.table[1, 0]] == 0x11), what
        assert not torch.all(kc[good.table[0, 0], :, :4] == 0x11), what


def test_append_and_attend_beyond_32_bit_offsets():
    page, Hkv, d, H = 128, 8, 128, 8
    pages = (1 << 32) // (page * Hkv * d) + 40
    b = Batch([(130, 1), (0, 40)], page)
    b.table += pages - b.pages  # the pool's last pages, beyond 4 GiB
    b.table[b.table < pages - b.pages] = -1
    kc = torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device="cuda")
    ks, vs = torch.ones(pages, Hkv, device="cuda"), torch.ones(pages, Hkv, device="cuda")
    rng = np.random.default_rng(6)
    x = oracle.bf16_round(rng.standard_normal((3, b.T, Hkv, d)).astype(np.float32))
    k, v, q = (cuda(y, torch.bfloat16) for y in x)
    sa.paged_fp8_append(k, v, kc, vc, ks, vs, *b.tensors())
    o, lse = sa.paged_fp8_fwd(q, kc, vc, ks, vs, *b.tensors(), max_q_len=40)
    sa.check_device()
    first = pages - b.pages
    small = [t[first:].cpu().numpy() for t in (kc, vc, ks, vs)]
    assert not kc[:first].any()
    table = np.where(b.table < 0, -1, b.table - first)
    want, _ = oracle.paged_append(x[0], np.zeros(small[0].shape, np.uint8),
                                  np.ones(small[2].shape, np.float32), table, b.cu, b.kv_lens)
    assert np.array_equal(small[0], want)
    ro, rl = oracle.paged_attend(x[2], *small, table, b.cu, b.kv_lens, 1, -1, None, 0, d ** -0.5)
    compare(o, lse, ro, rl, TOL_BF16_O)


# ------------------------------------------------------------------ attention

def attend(b, H, Hkv, d, dtype="bf16", causal=True, window=-1, mode=0, seed=0, hint=None,
           pool=None, workspace=None, extra=2, scale=None):
    rng = np.random.default_rng(seed + 1000)
    kc, ks = pool[:2] if pool else filled(rng, b, Hkv, d)
    vc, vs = pool[2:] if pool else filled(rng, b, Hkv, d)
    q = rng.standard_normal((b.T + extra, H, d)).astype(np.float32)
    if dtype == "bf16":
        q = oracle.bf16_round(q)
    sinks = rng.standard_normal(H).astype(np.float32)
    scale = d ** -0.5 if scale is None else scale
    o = torch.full((b.T + extra, H, d), 5.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((b.T + extra, H), 5.0, device="cuda")
    sa.paged_fp8_fwd(cuda(q, DT[dtype]), cuda(kc), cuda(vc), cuda(ks), cuda(vs), *b.tensors(),
                     max_q_len=int(b.n.max(initial=0)) if hint is None else hint, causal=causal,
                     window_left=window, sinks=cuda(sinks) if mode else None, sink_mode=mode,
                     scale=scale, o=o, lse=lse, workspace=workspace)
    sa.check_device()
    assert torch.all(o[b.T:] == 5.0) and torch.all(lse[b.T:] == 5.0)  # behind the last sequence
    ro, rl = oracle.paged_attend(q[:b.T], kc, vc, ks, vs, b.table, b.cu, b.kv_lens, int(causal),
                                 window, sinks, mode, scale)
    compare(o[:b.T], lse[:b.T], ro, rl, TOL_BF16_O if dtype == "bf16" else TOL_F32_O)
    return o, lse


DECODE = [(0, 1), (1, 1), (14, 1), (15, 1), (16, 1), (126, 1), (127, 1), (128, 1), (129, 1),
          (511, 1), (700, 1), (0, 0), (2000, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(128, 64), (128, 16), (64, 32), (64, 128), (128, 128)])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (5, 1), (4, 4)])
def test_single_tokens(H, Hkv, d, page, dtype):
    attend(Batch(DECODE, page), H, Hkv, d, dtype)


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("window", [-1, 0, 1, 127, 300])
@pytest.mark.parametrize("d,page", [(128, 64), (64, 16)])
def test_single_tokens_with_window_and_sinks(d, page, window, mode):
    attend(Batch(DECODE, page), 16, 2, d, window=window, mode=mode)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 1), (16, 1), (17, 1), (32, 1), (40, 2), (64, 1),
                                   (128, 1), (130, 2)])
def test_head_layouts(H, Hkv):
    attend(Batch([(300, 1), (77, 2), (0, 3)], 32), H, Hkv, 128, mode=2)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [2, 3, 5, 8])
def test_a_few_tokens_a_sequence(n, causal):
    b = Batch([(500, n), (0, n), (127, n), (1, 1), (250, max(1, n - 1))], 64)
    attend(b, 8, 2, 128, causal=causal, mode=2)
    attend(b, 8, 1, 64, causal=causal, window=130)


PROMPTS = [(0, 1), (0, 130), (5, 257), (300, 64), (0, 0), (129, 100), (0, 33), (1000, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(128, 64), (64, 16), (128, 128), (64, 32)])
@pytest.mark.parametrize("H,Hkv", [(4, 1), (6, 2)])
def test_prompts(H, Hkv, d, page, dtype):
    attend(Batch(PROMPTS, page), H, Hkv, d, dtype)


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (True, 200), (False, -1),
                                           (False, 70)])
def test_prompts_with_window_and_sinks(causal, window, mode):
    attend(Batch(PROMPTS, 32), 10, 2, 128, causal=causal, window=window, mode=mode)


@pytest.mark.parametrize("hint", [1, 4, 64, 100000])
def test_the_length_hint_changes_no_result(hint):
    attend(Batch(PROMPTS, 64), 8, 2, 128, hint=hint, mode=1)


@pytest.mark.parametrize("n", [1, 4, 90])
def test_rows_that_see_nothing(n):
    """More queries than cached positions: the first rows lie before position 0."""
    b = Batch([(0, n), (40, n), (0, n)], 16)
    b.kv_lens[:] = [max(0, n - 1), 40 + n, 0]
    for mode in (0, 1, 2):
        attend(b, 4, 2, 64, mode=mode)
        attend(b, 4, 2, 128, causal=False, mode=mode)


@pytest.mark.parametrize("n", [1, 70])
def test_large_and_uneven_scales(n):
    """Scales from 2^-20 to 2^6 a page, zeros in some, not powers of two."""
    rng = np.random.default_rng(n)
    b = Batch([(1500, n), (333, n)], 64)
    kc, _ = filled(rng, b, 2, 128)
    vc, _ = filled(rng, b, 2, 128)
    ks = rng.uniform(0.5, 1.5, (b.pages, 2)).astype(np.float32) / 200
    vs = (rng.uniform(0.5, 1.5, (b.pages, 2)) * 2.0 ** rng.integers(-20, -6, (b.pages, 2))
          ).astype(np.float32)
    vs[b.table[0, 3]] = 0.0
    attend(b, 8, 2, 128, pool=(kc, ks, vc, vs))


@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("scale", [1e-6, 1.0, 4.0])
def test_flat_and_peaked_softmax(scale, n):
    attend(Batch([(3000, n), (40, n)], 64), 4, 1, 128, scale=scale)


@pytest.mark.parametrize("n", [1, 70])
def test_hidden_keys_may_hold_anything(n):
    """NaN codes in front of the window and behind the last position reach no row."""
    rng = np.random.default_rng(9)
    b = Batch([(700, n)], 64)
    kc, ks = filled(rng, b, 1, 128)
    vc, vs = filled(rng, b, 1, 128)
    for p in range(500):
        kc[b.table[0, p // 64], :, p % 64] = 0x7F
        vc[b.table[0, p // 64], :, p % 64] = 0xFF
    q = oracle.bf16_round(rng.standard_normal((n, 4, 128)).astype(np.float32))
    o, lse = sa.paged_fp8_fwd(cuda(q, torch.bfloat16), cuda(kc), cuda(vc), cuda(ks), cuda(vs),
                              *b.tensors(), max_q_len=n, window_left=200)
    sa.check_device()
    kc[kc == 0x7F], vc[vc == 0xFF] = 0, 0
    ro, rl = oracle.paged_attend(q, kc, vc, ks, vs, b.table, b.cu, b.kv_lens, 1, 200, None, 0,
                                 128 ** -0.5)
    compare(o, lse, ro, rl, TOL_BF16_O)


@pytest.mark.parametrize("n", [1, 70])
def test_skipped_sequences_and_pages(n):
    rng = np.random.default_rng(10)
    b = Batch([(200, n), (300, n), (90, n)], 64)
    pool = [*filled(rng, b, 2, 128), *filled(rng, b, 2, 128)]
    kc, ks, vc, vs = (cuda(t) for t in pool)
    q = cuda(oracle.bf16_round(rng.standard_normal((b.T, 4, 128)).astype(np.float32)),
             torch.bfloat16)

    def call(table, cu, lens):
        o = torch.full((b.T, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        _, lse = sa.paged_fp8_fwd(q, kc, vc, ks, vs, cuda(table), cuda(cu), cuda(lens),
                                  max_q_len=n, o=o)
        return o, lse

    want, wl = call(b.table, b.cu, b.kv_lens)
    sa.check_device()
    lens = b.kv_lens.copy()
    lens[1] = 64 * b.table.shape[1] + 1  # more than the table holds
    o, _ = call(b.table, b.cu, lens)
    with pytest.raises(sa.SattnError):
        sa.check_device()
    assert torch.all(o[n:2 * n] == 5.0)
    assert torch.equal(o[:n], want[:n]) and torch.equal(o[2 * n:], want[2 * n:])
    table = b.table.copy()
    table[1, 1] = b.pages  # 64 positions of the second sequence are in no page
    o, lse = call(table, b.cu, b.kv_lens)
    with pytest.raises(sa.SattnError):
        sa.check_device()
    assert torch.equal(o[:n], want[:n]) and torch.equal(o[2 * n:], want[2 * n:])
    assert torch.isfinite(o.float()).all() and torch.all(lse[n:2 * n] < wl[n:2 * n])


@pytest.mark.parametrize("n", [1, 3, 100])
def test_workspace_and_repeats_change_nothing(n):
    b = Batch([(5000, n), (64, n), (900, n)], 64)
    ws = torch.full((max(256, sa.paged_fp8_workspace_bytes(n, 8, 2, 128)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    runs = [attend(b, 8, 2, 128, workspace=ws) for _ in range(3)]
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])
    tiny = torch.empty(256, dtype=torch.uint8, device="cuda")
    attend(b, 8, 2, 128, workspace=tiny)  # too small to split: same operation


@pytest.mark.parametrize("n", [1, 40])
def test_captured_calls_and_other_streams(n):
    """A captured append and attention, replayed with new inputs in the same
    buffers; and the same on a side stream."""
    rng = np.random.default_rng(11)
    H, Hkv, d, page = 8, 2, 128, 64
    b = Batch([(100, n), (1000, n), (0, n)], page)
    table, cu, lens = b.tensors()
    cs = cuda(rope_table(2048, d))
    pool = [cuda(x) for x in (*filled(rng, b, Hkv, d), *filled(rng, b, Hkv, d))]
    qkv = torch.empty(b.T, H + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(256, sa.paged_fp8_workspace_bytes(n, H, Hkv, d)), dtype=torch.uint8,
                     device="cuda")

    def step(kc, ks, vc, vs):
        q = sa.paged_fp8_append(qkv[:, H:H + Hkv], qkv[:, H + Hkv:], kc, vc, ks, vs, table, cu,
                                lens, cos_sin=cs, q=qkv[:, :H])
        return sa.paged_fp8_fwd(q, kc, vc, ks, vs, table, cu, lens, max_q_len=n, workspace=ws)

    work = [t.clone() for t in pool]
    qkv.normal_()
    step(*work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*work)
    for seed in range(3):
        torch.manual_seed(seed)
        qkv.normal_()
        for w, p in zip(work, pool):
            w.copy_(p)
        graph.replay()
        got = [t.clone() for t in out]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = [t.clone() for t in pool]
            want = step(*again)
        torch.cuda.current_stream().wait_stream(side)
        sa.check_device()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        for x, y in zip(work, again):
            assert torch.equal(x, y)


@pytest.mark.parametrize("window,mode", [(-1, 0), (100, 2)])
def test_a_conversation(window, mode):
    """Prompt, then single tokens, then drafted tokens: each step appends and
    attends; every step is compared with the oracle on the cache so far, and the
    cached keys with the rotation of what went in."""
    rng = np.random.default_rng(12)
    H, Hkv, d, page, B = 8, 2, 128, 16, 3
    width, pages = 20, 3 * 20
    table = rng.permutation(pages).astype(np.int32).reshape(B, width)
    cs = rope_table(width * page, d)
    kc = torch.full((pages, Hkv, page, d), 0x7F, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    ks = torch.full((pages, Hkv), float("nan"), device="cuda")
    vs = ks.clone()
    sinks = rng.standard_normal(H).astype(np.float32)
    have = np.zeros(B, np.int64)
    keys = [[] for _ in range(B)]
    for n in ([37, 150, 1], [1, 1, 1], [1, 0, 1], [1, 1, 1], [4, 4, 4], [0, 70, 16], [1, 1, 1]):
        n = np.array(n)
        have += n
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        T = int(cu[-1])
        x = oracle.bf16_round(rng.standard_normal((T, H + 2 * Hkv, d)).astype(np.float32) * 2)
        t = cuda(x, torch.bfloat16)
        args = (cuda(table), cuda(cu), cuda(have.astype(np.int32)))
        q = sa.paged_fp8_append(t[:, H:H + Hkv], t[:, H + Hkv:], kc, vc, ks, vs, *args,
                                cos_sin=cuda(cs), q=t[:, :H])
        o, lse = sa.paged_fp8_fwd(q, kc, vc, ks, vs, *args, max_q_len=int(n.max()),
                                  window_left=window, sinks=cuda(sinks) if mode else None,
                                  sink_mode=mode)
        sa.check_device()
        pool = [y.cpu().numpy() for y in (kc, vc, ks, vs)]
        ro, rl = oracle.paged_attend(q.float().cpu().numpy(), *pool, table, cu, have, 1, window,
                                     sinks, mode, d ** -0.5)
        compare(o, lse, ro, rl, TOL_BF16_O)
        pos = np.concatenate([np.arange(h - m, h) for h, m in zip(have, n)]).astype(int)
        turned = oracle.rotate(x[:, H:H + Hkv], cs, pos, False)
        for i in range(B):
            keys[i].extend(turned[cu[i]:cu[i + 1]])
            for p, want in enumerate(keys[i]):
                pid = table[i, p // page]
                s = pool[2][pid][:, None]
                got = oracle.e4m3_decode(pool[0][pid, :, p % page]) * s
                # recoding below the normal range adds half a step of it each time
                assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -9 * s)
