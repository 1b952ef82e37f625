"""Captured calls of the paged attention whose units are drawn from a counter:
its reset is a node of the graph in front of the kernel, and every replay draws
all units anew."""

import pytest
import torch

import exact_tiled_attention_18_gb300 as fa
from tests.test_paged_gpu import make_batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Hq,Hkv,Nq,d,page,prefix,lens", [
    (1, 20, 20, 4096, 64, 64, 0, [4096]),                                   # all drawn
    (38, 20, 20, 257, 64, 64, 0, [700 + 10 * i for i in range(38)]),        # behind a line
    (170, 4, 2, 40, 128, 16, 0, [60 + i for i in range(170)]),              # two row tiles on the same rows
    (300, 4, 2, 128, 64, 16, 64, [192 + i % 50 for i in range(300)]),       # of the prefix and of the sequences
])
def test_captured_calls_draw_all_units_at_every_replay(B, Hq, Hkv, Nq, d, page, prefix, lens):
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=B)
    n = prefix // page
    table[:, :n] = table[0, :n].clone()
    q, kp, vp, table = (t.cuda() for t in (q, kp, vp, table))
    lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lq = torch.full((B,), Nq, dtype=torch.int32, device="cuda")
    first = table[0, :n].contiguous()

    def call(out=None):
        if prefix:
            return fa.forward_shared_prefix(q, kp, vp, first, prefix, table, lk, lq, out=out)
        return fa.forward_paged(q, kp, vp, table, lk, lq, out=out)

    out = call()
    fa.sync_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
        call(out)  # two in a row: the second's reset behind the first's kernels
    g = torch.Generator().manual_seed(B)
    for step in range(4):
        if step:  # other lengths, among them empty sequences
            lk.copy_(torch.tensor([int(torch.randint(0, m + 1, (1,), generator=g)) for m in lens], dtype=torch.int32))
            lq.copy_(torch.randint(0, Nq + 1, (B,), generator=g).to(torch.int32))
        q.copy_(torch.randn(q.shape, generator=g).to(torch.bfloat16))
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        fa.sync_status()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), step
        assert not torch.isnan(out[0]).any() and not torch.isnan(out[1]).any()
