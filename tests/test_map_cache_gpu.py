"""Tensor maps are encoded once: a loop over many layers' caches and the calls
beside it find theirs again."""

import pytest
import torch

import exact_tiled_attention_18_gb300 as fa
from tests.test_paged_gpu import make_batch

pytestmark = pytest.mark.gpu

LAYERS = 48


def test_a_loop_over_many_layers_encodes_no_map_twice():
    """A decoding step of 48 layers, each with a cache of its own and both
    paged calls on it (six maps a layer), and a training call's maps beside
    them: from the second step on nothing is encoded, and the results stay."""
    B, Hq, Hkv, d, page = 2, 8, 2, 128, 64
    lens = [200, 130]
    q, kp, vp, table = make_batch(B, Hq, Hkv, 1, d, page, lens)
    table[1, :1] = table[0, :1]
    q, table = q.cuda(), table.cuda()
    lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
    prefix = table[0, :1].contiguous()
    caches = [(kp.cuda(), vp.cuda()) for _ in range(LAYERS)]
    outs = [(torch.empty(B, Hq, 1, d, device="cuda"), torch.empty(B, Hq, 1, device="cuda")) for _ in range(2)]
    square = [torch.randn(1, 2, 300, d).to(torch.bfloat16).cuda() for _ in range(3)]
    square_out = torch.empty(1, 2, 300, d, device="cuda"), torch.empty(1, 2, 300, device="cuda")

    def step():
        fa.forward(*square, out=square_out)
        for k, v in caches:
            fa.forward_paged(q, k, v, table, lk, out=outs[0])
            fa.forward_shared_prefix(q, k, v, prefix, page, table, lk, out=outs[1])

    step()
    fa.sync_status()
    want = [o.clone() for o in outs[0] + outs[1]]
    before = fa.fa_test_map_encodes()
    for _ in range(3):
        step()
    fa.sync_status()
    assert fa.fa_test_map_encodes() == before
    assert all(torch.equal(a, b) for a, b in zip(outs[0] + outs[1], want))
    other = [torch.zeros_like(t) for t in square]  # (kept alive: other addresses, other maps)
    fa.forward(*other, out=square_out)
    fa.sync_status()
    assert fa.fa_test_map_encodes() > before


def test_more_maps_than_the_cache_holds():
    """Calls on more tensors than there is room for: maps are encoded again and
    are the right ones."""
    d, n = 64, 128
    rows = 4200 * n
    pool = torch.randn(1, 1, rows, d).to(torch.bfloat16).cuda()
    for i in list(range(0, 4200)) + [0, 17, 4199]:
        x = pool[:, :, i * n:(i + 1) * n]
        o, lse = fa.forward(x, x, x, scale=0.5)
        if i % 600 == 17 or i == 4199 or i == 0:
            s = 0.5 * x.double() @ x.double().transpose(2, 3)
            assert (lse - torch.logsumexp(s, -1)).abs().max() <= 1e-3
    fa.sync_status()
