"""Outputs that a call makes itself belong to the stream that the call runs on: they are
not memory that the current stream has freed (work queued there may still use it), and
what is zeroed first is zeroed on that stream."""
import numpy as np
import pytest
import torch

import windowed_attention_sinks_gb300 as sa

pytestmark = pytest.mark.gpu


def randn(*shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device="cuda").to(dtype)


def calls():
    torch.manual_seed(0)
    q, k, v = randn(300, 8, 128), randn(300, 4, 128), randn(300, 4, 128)
    cu = torch.tensor([0, 130, 300], dtype=torch.int32, device="cuda")
    qs, cache = randn(2, 3, 32, 128), randn(2, 400, 128)
    idx = torch.randint(0, 400, (2, 3, 128), device="cuda", dtype=torch.int32)
    nope, rope, scl = sa.quantize_kv_fp8(cache, 64)
    xq, xk = randn(256, 4, 128), randn(512, 2, 128)
    mask = torch.ones(4, 2, 4, dtype=torch.uint8, device="cuda")
    op, lp = sa.block_sparse_chunks_fwd(xq, xk, xk, mask, 256, 0, 512, 256)
    m, l = sa.xattn_partial_stats(xq, xk, 256, 0, 512, True)
    sums = sa.xattn_block_sum(xq, xk, m, l, 256, 0, 512, True)
    ms, ls = torch.stack([m, m]), torch.stack([l, l])
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    kv, score, ape = randn(2, 64, 256), randn(2, 64, 256), randn(4, 256, dtype=torch.float32)
    return {
        "window_fwd": lambda s: sa.window_fwd(q, k, v, cu, 170, 64, 0, stream=s),
        "sparse_fwd": lambda s: sa.sparse_fwd(qs, cache, idx, stream=s),
        "quantize_kv_fp8": lambda s: sa.quantize_kv_fp8(cache, 64, stream=s),
        "sparse_fp8_fwd": lambda s: sa.sparse_fp8_fwd(qs, nope, rope, scl, idx, stream=s),
        "block_sparse_fwd": lambda s: sa.block_sparse_fwd(xq, xk, xk, mask, 256, 0, 512, stream=s),
        "block_sparse_chunks_fwd":
            lambda s: sa.block_sparse_chunks_fwd(xq, xk, xk, mask, 256, 0, 512, 256, stream=s),
        "merge_lse": lambda s: sa.merge_lse(op.view(2, -1, 128), lp.view(2, -1), 4, stream=s),
        "build_topk_idxs": lambda s: (sa.build_topk_idxs(pos, 50, 64, 32, 4, stream=s),),
        "compress_kv": lambda s: (sa.compress_kv(kv, score, ape, 4, True, stream=s),),
        "xattn_partial_stats": lambda s: sa.xattn_partial_stats(xq, xk, 256, 0, 512, True, stream=s),
        "xattn_merge_stats": lambda s: sa.xattn_merge_stats(ms, ls, stream=s),
        "xattn_block_sum": lambda s: (sa.xattn_block_sum(xq, xk, m, l, 256, 0, 512, True, stream=s),),
        "xattn_find_blocks": lambda s: (sa.xattn_find_blocks(sums, 0.9, stream=s),),
        "xattn_select_blocks": lambda s: sa.xattn_select_blocks(xq, xk, 256, True, 0.9, stream=s),
    }


NAMES = ["window_fwd", "sparse_fwd", "quantize_kv_fp8", "sparse_fp8_fwd", "block_sparse_fwd",
         "block_sparse_chunks_fwd", "merge_lse", "build_topk_idxs", "compress_kv",
         "xattn_partial_stats", "xattn_merge_stats", "xattn_block_sum", "xattn_find_blocks",
         "xattn_select_blocks"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_belong_to_the_calls_stream(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    freed = [torch.empty_like(t) for _ in range(8) for t in want]
    addresses = {t.data_ptr() for t in freed}
    del freed
    got = call(side)
    side.synchronize()
    sa.check_device(side)
    assert all(t.data_ptr() not in addresses for t in got)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_call_does_not_wait_for_the_current_stream():
    """Its zeros are its own stream's: they are there although the current stream is busy."""
    call = calls()["xattn_block_sum"]
    want = call(None)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # some 10 ms
    got = call(side)[0]
    side.synchronize()
    early = got.cpu() if not torch.cuda.current_stream().query() else None
    torch.cuda.synchronize()
    sa.check_device(side)
    assert torch.equal(got, want)
    assert early is None or np.array_equal(early.numpy(), want.cpu().numpy())
