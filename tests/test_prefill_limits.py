"""The largest batch of the prefill calls: refused above it before a GPU is touched."""

import pytest
import torch

MOST = 1 << 24


@pytest.mark.parametrize("batch", [MOST + 1, (1 << 31) - 1, (1 << 31) - 100])
def test_batch_beyond_the_limit_is_refused(libmla, batch):
    d = libmla.make_read_desc(batch=batch, max_pages_per_seq=4, num_pages=8, num_rows=100)
    for fn in (libmla.mlap_cache_read, libmla.mlap_cache_read_fp8):
        assert fn(d, 16, 16, 16, 16, 16, None, None) == libmla.MLA_ERR_UNSUPPORTED
    d = libmla.make_attention_desc(batch=batch, num_heads=8, num_q=10, num_k=20)
    assert libmla.mlap_attention_workspace_bytes(d) == 0
    assert libmla.mlap_attention(d, *([32] * 8), 1 << 40, None, None) == libmla.MLA_ERR_UNSUPPORTED


@pytest.mark.gpu
def test_one_sequence_among_a_million_empty_ones(libmla):
    from mla_latent_kv_26_b200.prefill import cache_read, prefill_attention

    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator().manual_seed(241)
    batch, at, n, L = 1 << 20, 654321, 100, 300
    cu_q, cu_k = (torch.zeros(batch + 1, dtype=torch.int32, device=dev) for _ in range(2))
    cu_q[at + 1:], cu_k[at + 1:] = n, L
    q, kv, pe = (torch.randn(*s, generator=g).to(torch.bfloat16).to(dev) for s in ((n, 2, 192), (L, 2, 256), (L, 64)))
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = prefill_attention(q, kv, pe, cu_q, cu_k, error_word=err)
    alone = prefill_attention(q, kv, pe, cu_q[at:at + 2].contiguous(), cu_k[at:at + 2].contiguous())
    assert torch.equal(out, alone[0]) and torch.equal(lse, alone[1])
    cache = torch.randn(5, 64, 576, generator=g).to(torch.bfloat16).to(dev)
    table = torch.full((batch, 5), -1, dtype=torch.int32, device=dev)
    table[at] = torch.tensor([4, 0, 3, 1, 2], dtype=torch.int32, device=dev)
    rows = cache_read(cache, table, cu_k, num_rows=L, error_word=err)
    assert torch.equal(rows, cache[table[at].long()].view(-1, 576)[:L]) and int(err.item()) == 0
