"""Value scales of any size over the paged FP8 cache, and far apart within one sequence.

Tolerances. A row's error counts against the mean of |v| under its own weights, A =
sum p |v|: probabilities keep 9 significant bits (2^-9 A), the exponents' and sums'
fp32 errors stay below 2^-12 A, and the output is rounded to bf16 (2^-8 |o|); fp32 queries
1e-4 A. A probability times its scale may be off by 2^-32 of the row's largest such product
(the header's bound, a scale of 0 counting as 2^-64), that is by 2^-32 * 1.875 L sum p s over L keys. Half of the output's least step, 2^-134 or 2^-150, is added, twice for fp32 where the
row is scaled once more. Logits are below 16, lse within the 1e-3 of the other cases."""
import numpy as np
import pytest
import torch

import oracle
import windowed_attention_sinks_gb300 as sa

from gpu_helpers import TOL_LSE
from test_gpu_paged import DT, Batch, cuda, filled
from test_gpu_paged_edges import seen

pytestmark = pytest.mark.gpu

LEAST, LARGEST = 2.0 ** -149, float(np.finfo(np.float32).max)


def run(b, H, Hkv, d, vs, dtype="bf16", window=-1, causal=True, mode=0, equal=False, nan=()):
    """nan: (sequence, KV head, key, column) of NaN value codes."""
    rng = np.random.default_rng(b.T)
    kc, ks = filled(rng, b, Hkv, d)
    # values up to 1.875: with the largest scale they stay in fp32's range
    vc = oracle.e4m3_encode(rng.uniform(-1.875, 1.875, kc.shape))
    vc[kc == 0x7F] = 0x7F
    vs = vs.astype(np.float32)
    big = np.broadcast_to((vs > 2.0 ** 126)[:, :, None, None], vc.shape) & (vc != 0x7F)
    vc[big] &= 0x80 | 0x37  # below 1
    q = rng.standard_normal((b.T, H, d)).astype(np.float32)
    q = np.zeros_like(q) if equal else oracle.bf16_round(q)
    sinks = rng.standard_normal(H).astype(np.float32)
    where = (b.table, b.cu, b.kv_lens, int(causal), window, sinks, mode, d ** -0.5)
    ro, rl = oracle.paged_attend(q, kc, vc, ks, vs, *where)
    mean, _ = oracle.paged_attend(q, kc, vc & 0x7F, ks, vs, *where)
    ones = np.full_like(vc, 0x38)
    floor, _ = oracle.paged_attend(q, kc, ones, ks, np.where(vs == 0, 2.0 ** -64, vs), *where)
    floor *= 2.0 ** -32 * 1.875 * b.kv_lens.max()
    held = vc.copy()
    spoilt = np.zeros(ro.shape, bool)
    masks = seen(b, window, causal)
    for i, g, key, col in nan:
        held[b.table[i, key // b.page], g, key % b.page, col] = 0x7F
        rows = b.cu[i] + np.nonzero(masks[i][:, key])[0]
        spoilt[rows, g * (H // Hkv):(g + 1) * (H // Hkv), col] = True
    o, lse = sa.paged_fp8_fwd(cuda(q, DT[dtype]), cuda(kc), cuda(held), cuda(ks), cuda(vs),
                              *b.tensors(), max_q_len=int(b.n.max()), window_left=window,
                              causal=causal, sinks=cuda(sinks) if mode else None, sink_mode=mode)
    sa.check_device()
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), spoilt)
    got[spoilt] = ro[spoilt]
    assert np.isfinite(got).all()
    part = 2.0 ** -9 + 2.0 ** -12 if dtype == "bf16" else 1e-4
    tol = part * mean + floor + (2.0 ** -8 * np.abs(ro) + 2.0 ** -134 if dtype == "bf16" else 2.0 ** -149)
    assert (np.abs(got - ro) <= tol).all(), (np.abs(got - ro) / np.maximum(tol, 1e-300)).max()
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), none)
    assert np.abs(gl[~none] - rl[~none]).max(initial=0) <= TOL_LSE


def batch(n, page=64):
    return Batch([(1500, n), (33, n), (0, n), (700, n)], page)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 4, 70])
@pytest.mark.parametrize("power", [-149, -140, -130, -127, -126, -100, -65, -64, -30, 24, 25, 60,
                                   100, 120, 126, 127])
def test_scales_of_one_size(power, n, dtype):
    b = batch(n)
    run(b, 8, 2, 128, np.full((b.pages, 2), 2.0 ** power), dtype)


@pytest.mark.parametrize("equal", [True, False])
@pytest.mark.parametrize("n", [1, 4, 70])
@pytest.mark.parametrize("small,large", [(0.0, 2.0 ** 24), (0.0, 2.0 ** 70), (0.0, 2.0 ** 120),
                                         (2.0 ** -64, 2.0 ** 24), (2.0 ** -64, 2.0 ** 66),
                                         (2.0 ** -64, 2.0 ** 120), (LEAST, 1.0), (LEAST, 2.0 ** 127),
                                         (2.0 ** -120, 2.0 ** 20), (0.0, LEAST), (1.0, 2.0 ** 100)])
def test_scales_far_apart(small, large, n, equal):
    """Every arrangement of the two among neighbouring pages: small first, large first, in turn."""
    for order in ("up", "down", "turn", "one large", "one small"):
        b = batch(n)
        vs = np.full((b.pages, 2), small)
        for row in b.table:
            ids = row[row >= 0]
            k = len(ids)
            if order == "up":
                vs[ids[k // 2:]] = large
            elif order == "down":
                vs[ids[: (k + 1) // 2]] = large
            elif order == "turn":
                vs[ids[::2], 0], vs[ids[1::2], 1] = large, large
            elif order == "one large":
                vs[ids[k // 3]] = large
            else:
                vs[ids] = large
                vs[ids[2 * k // 3]] = small
        run(b, 8, 2, 128, vs, equal=equal, mode=2 if order == "turn" else 0)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (64, 128)])
@pytest.mark.parametrize("n", [1, 4, 70])
@pytest.mark.parametrize("window,causal,mode", [(-1, True, 1), (100, True, 2), (-1, False, 2)])
def test_scales_of_every_size_at_once(window, causal, mode, n, d, page):
    rng = np.random.default_rng(page)
    b = batch(n, page)
    vs = 2.0 ** rng.uniform(-149, 126, (b.pages, 2))
    vs[rng.random(vs.shape) < 0.1] = 0.0
    run(b, 6, 2, d, vs, window=window, causal=causal, mode=mode)


@pytest.mark.parametrize("n,H", [(1, 64), (4, 16), (5, 12)])
def test_scales_of_every_size_with_many_rows_of_few_tokens(n, H):
    rng = np.random.default_rng(H)
    b = batch(n)
    vs = 2.0 ** rng.uniform(-149, 126, (b.pages, 2))
    run(b, H, 2, 128, vs, mode=2)
    run(b, H, 2, 128, np.where(rng.random(vs.shape) < 0.1, vs, 2.0 ** -5), window=300)


@pytest.mark.parametrize("n", [1, 4, 70])
@pytest.mark.parametrize("keys", [20000, 9000])
def test_one_far_page_in_a_long_sequence(keys, n):
    """Pieces with and without such a page, joined."""
    b = Batch([(keys, n), (500, n)], 64)
    for at, scale in ((0, 2.0 ** 90), (140, 2.0 ** 90), (70, 2.0 ** -110)):
        vs = np.full((b.pages, 2), 2.0 ** -3)
        vs[b.table[0, at]] = scale
        run(b, 8, 2, 128, vs)
        vs[b.table[0, at - 1 if at else 1]] = 0.0
        run(b, 8, 2, 128, vs, equal=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 4, 70])
@pytest.mark.parametrize("window", [-1, 150])
def test_nan_values_under_a_zero_scale(window, n, dtype):
    """NaN times 0 is NaN: to the rows that see it, whatever the page's scale."""
    b = batch(n)
    vs = np.full((b.pages, 2), 0.25)
    nan = []
    for i, length in enumerate(b.kv_lens):
        for g, key, col in ((0, int(length) // 2, 7), (1, int(length) - 1, 100)):
            vs[b.table[i, key // 64], g] = 0.0
            nan.append((i, g, key, col))
    run(b, 8, 2, 128, vs, dtype, window=window, nan=nan)


@pytest.mark.parametrize("n", [1, 4, 40])
def test_nan_values_under_a_zero_scale_of_a_long_sequence(n):
    """Found again at the unit's end among 200000 keys of one piece, in ordinary and in far units:
    within the limit of a wait."""
    keys, d = 200000, 64
    b = Batch([(keys, n)], 128)
    kc = np.zeros((b.pages, 1, 128, d), np.uint8)
    vc = np.full(kc.shape, 0x38, np.uint8)  # 1.0
    q = torch.zeros(b.T, 2, d, dtype=torch.bfloat16, device="cuda")
    for far in (0.25, 2.0 ** 40):
        vs = np.full((b.pages, 1), 0.25, np.float32)
        vs[b.table[0, 700]] = far
        vs[b.table[0, 90]] = 0.0
        spoilt = vc.copy()
        spoilt[b.table[0, 90], 0, 17, 5] = 0x7F
        o, lse = sa.paged_fp8_fwd(q, cuda(kc), cuda(spoilt), cuda(np.ones_like(vs)), cuda(vs),
                                  *b.tensors(), max_q_len=n,
                                  workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
        sa.check_device()
        o = o.float().cpu().numpy()
        assert np.isnan(o[..., 5]).all() and np.isnan(o).sum() == o[..., 5].size
        L = keys + 1 + np.arange(n)  # keys that a row sees, all alike
        want = (0.25 * (L - 256) + 128 * far) / L
        assert np.abs(o[..., 0] / want[:, None] - 1).max() <= 2.0 ** -7
        assert np.abs(lse.cpu().numpy() - np.log(L)[:, None]).max() <= TOL_LSE
