"""Paged FP8 calls on several streams: calls far apart in issue order, and a timeout that
is taken note of on one stream while a call runs on another. Every call has its own
workspace (filled with ones before: the call depends on nothing in it). And what the
binding chooses by itself: memory for outputs, the kernel."""
import numpy as np
import pytest
import torch

import windowed_attention_sinks_gb300 as sa

from test_gpu_paged import Batch, cuda

pytestmark = pytest.mark.gpu


class Job:
    """A call with few rows a sequence, so that units cut between CTAs are joined."""

    def __init__(self, lens, seed, H=8, Hkv=2, d=128):
        rng = np.random.default_rng(seed)
        self.b = Batch(lens, 64, seed)
        shape = (self.b.pages, Hkv, 64, d)
        self.cache = [(torch.randn(shape, device="cuda") * 8).to(torch.float8_e4m3fn)
                      .view(torch.uint8) for _ in "kv"]
        self.cache += [torch.full(shape[:2], 2.0 ** -6, device="cuda") for _ in "kv"]
        self.cache += self.b.tensors()
        self.q = cuda(rng.standard_normal((self.b.T, H, d)).astype(np.float32), torch.bfloat16)
        self.n = int(self.b.n.max())
        bytes_ = sa.paged_fp8_workspace_bytes(self.n, H, Hkv, d)
        self.ws = torch.full((bytes_,), 0xFF, dtype=torch.uint8, device="cuda")
        self.o = torch.empty_like(self.q)
        self.lse = torch.empty(self.b.T, H, device="cuda")

    def run(self, stream=None, o=None, lse=None):
        return sa.paged_fp8_fwd(self.q, *self.cache, max_q_len=self.n, workspace=self.ws,
                                o=self.o if o is None else o, lse=self.lse if lse is None else lse,
                                stream=stream)

    def want(self):
        out = [t.clone() for t in self.run()]
        torch.cuda.synchronize()
        sa.check_device()
        return out

    def spoil(self):
        self.o.fill_(77.0)
        self.lse.fill_(77.0)
        self.ws.fill_(0xFF)


LONG = [(int(x), 1) for x in np.linspace(20000, 60000, 40)]


@pytest.mark.parametrize("n", [1, 4])
def test_a_timeout_on_one_stream_leaves_a_call_on_another_alone(n):
    long = Job([(kv, n) for kv, _ in LONG], 0)
    small = Job([(900, n)], 1)
    want = long.want()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(torch.empty_like(long.o), torch.empty_like(long.lse)) for _ in range(40)]
    for _ in range(8):
        long.spoil()
        for o, lse in outs:
            o.fill_(77.0), lse.fill_(77.0)
        torch.cuda.synchronize()
        sa.set_test_wait_stall(True)
        sa.set_wait_limit_ns(1_000_000)
        try:
            small.run(b)
        finally:
            sa.set_test_wait_stall(False)
            sa.set_wait_limit_ns(0)
        for o, lse in outs:  # some of these run while the timeout is read and cleared
            long.run(a, o, lse)
        with pytest.raises(sa.SattnError) as err:
            sa.check_device(b)
        assert err.value.code == 5
        torch.cuda.synchronize()
        sa.check_device(a)
        assert all(torch.equal(o, want[0]) and torch.equal(lse, want[1]) for o, lse in outs)


def test_calls_hundreds_apart_on_two_streams():
    """A long call and many short ones enqueued behind it elsewhere."""
    long, small = Job(LONG, 2), Job([(300, 1), (2500, 1), (0, 1)], 3)
    want, wants = long.want(), small.want()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    long.spoil()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(4):
            long.run(a)
        for _ in range(600):
            small.run(b)
            with torch.cuda.stream(b):
                bad += (small.o != wants[0]).sum()
        with torch.cuda.stream(a):
            bad2 = (long.o != want[0]).sum() + (long.lse != want[1]).sum()
        torch.cuda.synchronize()
        assert bad.item() == 0 and bad2.item() == 0
    sa.check_device()


def test_two_graphs_and_eager_calls_at_once():
    jobs = [Job([(9000, 1), (300, 1)], 4), Job([(4000, 2), (7000, 2)], 5), Job([(12000, 1)], 6)]
    want = [j.want() for j in jobs]
    graphs = []
    for j in jobs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            j.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in jobs]
    for j in jobs:
        j.spoil()
    torch.cuda.synchronize()
    bad = [torch.zeros((), dtype=torch.int64, device="cuda") for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(300):
        for i, (j, s) in enumerate(zip(jobs, streams)):
            with torch.cuda.stream(s):
                if i < 2:
                    graphs[i].replay()
                else:
                    j.run()
                bad[i] += (j.o != want[i][0]).sum() + (j.lse != want[i][1]).sum()
    torch.cuda.synchronize()
    sa.check_device()
    assert [x.item() for x in bad] == [0, 0, 0]


def test_outputs_that_a_call_makes_are_its_streams():
    """Not in memory that the current stream has freed (and may still use there)."""
    torch.manual_seed(0)
    job = Job([(500, 3), (90, 2)], 7)
    T, H, d = job.q.shape
    k = torch.randn(T, 2, d, device="cuda").bfloat16()
    cs = torch.randn(1024, d, device="cuda")
    side = torch.cuda.Stream()

    def calls(stream):
        q = sa.paged_fp8_append(k, k, *job.cache, cos_sin=cs, q=job.q, stream=stream)
        o, lse = sa.paged_fp8_fwd(job.q, *job.cache, max_q_len=3, stream=stream)
        return q, o, lse

    want = [t.clone() for t in calls(None)]
    torch.cuda.synchronize()
    freed = [torch.empty_like(t) for _ in range(8) for t in want]
    addresses = {t.data_ptr() for t in freed}
    del freed
    got = calls(side)
    side.synchronize()
    sa.check_device(side)
    assert all(t.data_ptr() not in addresses for t in got)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("n", [1, 4, 40])
def test_without_a_hint_the_kernel_is_chosen_by_the_mean_length(n):
    """The kernels round differently: the same bits are the same kernel's."""
    job = Job([(int(x), n) for x in np.linspace(500, 5000, 20)], 8)
    o, lse = job.want()
    other = sa.paged_fp8_fwd(job.q, *job.cache, max_q_len=100 if n < 40 else 1)[0]
    got = sa.paged_fp8_fwd(job.q, *job.cache)
    sa.check_device()
    assert torch.equal(got[0], o) and torch.equal(got[1], lse)
    assert not torch.equal(other, o)
