"""Encoder-state operators at the limits of what their numbers may be. Tolerances are those of
test_gpu_states."""
import numpy as np
import pytest
import torch

import oracle
import windowed_attention_sinks_gb300 as sa

from test_gpu_states import DT, Case, cuda

pytestmark = pytest.mark.gpu

DTYPES = list(DT)


def attend(c, mode=0, hint=None, **kw):
    q, k, v = c.tensors()
    o, lse = sa.cross_fwd(q, k, v, *c.ranges(), max_q_len=hint or int(c.n.max()),
                          sinks=cuda(c.sinks) if mode else None, sink_mode=mode, **kw)
    sa.check_device()
    return o, lse


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
