"""The append into E4M3 pages whose heads lie 2^31 bytes and more apart."""

import pytest
import torch

import exact_tiled_attention_18_gb300 as fa

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("page", [2 ** 24, 2 ** 24 + 16])
def test_a_page_of_2_24_tokens(page):
    """One page of 2^24 tokens and more, three heads, so many new tokens that a
    thread takes several heads: the bytes and scales are those of small pages."""
    H, d, n = 3, 128, 30000
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(1, H, n, d, generator=g).to(BF16).cuda() for _ in range(2))
    turns = fa.rope_turns(d, device="cuda")

    def cache(pages, size):
        return [torch.empty(pages, H, size, d, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)] + [
            torch.empty(pages, H, size // 16, device="cuda") for _ in range(2)]

    small = cache(-(-n // 64), 64)
    table = torch.arange(small[0].shape[0], dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    fa.kv_append_fp8(k, v, *small, table, lens, turns=turns)
    want = [x.transpose(0, 1).reshape(H, -1, d)[:, :n] for x in (t.view(torch.uint8) for t in small[:2])]
    scales = [x.transpose(0, 1).reshape(H, -1)[:, :n // 16] for x in small[2:]]
    large = cache(1, page)
    fa.kv_append_fp8(k, v, *large, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), lens, turns=turns)
    fa.sync_status()
    for h in range(H):
        for got, x in zip(large[:2], want):
            assert torch.equal(got.view(torch.uint8)[0, h, :n], x[h])
        for got, x in zip(large[2:], scales):
            assert torch.equal(got[0, h, :n // 16], x[h])
    for Nq in (1, 60):
        q = torch.randn(1, H, Nq, d, generator=g).to(BF16).cuda()
        a = fa.forward_paged_fp8(q, *large, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), lens)
        b = fa.forward_paged_fp8(q, *small, table, lens)
        fa.sync_status()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
