"""One dominating key before a long flat tail of lighter ones, over the paged FP8 cache.

The tail's keys are each below any share of the largest weight that a test of
random logits reaches, and together they weigh as much as the large one; the values'
mean is not 0, so what is lost of them does not average out.

Tolerance: a probability keeps 9 significant bits (2^-9 of itself at most, the same
way for equal logits), values are at most 1.5 in size, so the weighted mean is off by
1.5 * 2^-9 = 0.003 at most, and what lies below the kernels' floors (2^-32 of the largest
weight a key, 2^18 keys) by 1.5 * 2^-14: within the 1e-2 of the other bf16 cases."""
import numpy as np
import pytest
import torch

import oracle
import windowed_attention_sinks_gb300 as sa

from gpu_helpers import TOL_BF16_O, compare
from test_gpu_paged import Batch, cuda

pytestmark = pytest.mark.gpu

# queries a sequence, heads, KV heads: 4, 8, 16, 20, 32 and 160 rows a KV head
ROWS = {4: (1, 4, 1), 8: (1, 16, 2), 16: (4, 4, 1), 20: (5, 8, 2), 32: (4, 8, 1), 160: (40, 4, 1)}


def tail(gap, keys, rows, d, by, spread, split, place, page=64, value=0.0):
    n, H, Hkv = ROWS[rows]
    rng = np.random.default_rng(int(gap) + rows)
    b = Batch([(keys, n), (70, n)], page)
    kc = np.zeros((b.pages, Hkv, page, d), np.uint8)
    kc[..., 1] = oracle.e4m3_encode(rng.standard_normal(kc.shape[:3]) * spread)
    ks, vs = np.ones((b.pages, Hkv), np.float32), np.full((b.pages, Hkv), 0.5, np.float32)
    vc = oracle.e4m3_encode(rng.choice([1.0, 2.0, 3.0], (b.pages, Hkv, page, d)))  # mean 1
    pid, row = b.table[0, place // page], place % page
    vc[pid, :, row] = oracle.e4m3_encode(np.float64(value))  # the large key's
    q = np.zeros((b.T, H, d), np.float32)
    q[..., 1] = 1.0
    sinks, mode = None, 0
    if by == "logit":
        kc[pid, :, row, 0] = oracle.e4m3_encode(np.float64(gap))
        q[..., 0] = 1.0
    else:
        sinks, mode = np.full(H, gap, np.float32), 1
    ws = None if split else torch.empty(256, dtype=torch.uint8, device="cuda")
    o, lse = sa.paged_fp8_fwd(cuda(q, torch.bfloat16), cuda(kc), cuda(vc), cuda(ks), cuda(vs),
                              *b.tensors(), max_q_len=n, scale=1.0, workspace=ws, sink_mode=mode,
                              sinks=cuda(sinks) if mode else None)
    sa.check_device()
    ro, rl = oracle.paged_attend(q, kc, vc, ks, vs, b.table, b.cu, b.kv_lens, 1, -1, sinks, mode,
                                 1.0)
    compare(o, lse, ro, rl, TOL_BF16_O)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("gap", [11.0, 12.0, 13.0, 14.0, 15.0])
@pytest.mark.parametrize("by", ["logit", "bias"])
def test_a_large_first_key_and_a_flat_tail(by, gap, rows, d):
    tail(gap, 32768, rows, d, by, 0.0, False, 0)
    if gap == 13.0:
        tail(gap, 32768, rows, d, by, 0.0, False, 0, value=-2.0)  # -1, against the tail's 1


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("place", [0, 9000, 32700])
def test_a_large_key_anywhere_in_an_uneven_tail(place, rows, split):
    """The tail's logits are normal (of deviation 0.5), the large key first, inside or last."""
    tail(13.0, 32768, rows, 128, "logit", 0.5, split, place)


@pytest.mark.parametrize("rows", [4, 32, 160])
@pytest.mark.parametrize("gap", [9.0, 18.0])
def test_a_tail_of_262144_keys(gap, rows):
    tail(gap, 262144, rows, 64, "bias", 0.25, False, 0, page=128)
