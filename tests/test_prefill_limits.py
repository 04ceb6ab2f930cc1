"""The largest batch of the prefill calls: refused above it before a GPU is touched."""

import pytest
import torch

MOST = 1 << 22


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


@pytest.mark.gpu
@pytest.mark.parametrize("n,L,heads,num_sms", [(100, 300, 2, 2), (1100, 8200, 16, 4)])
def test_two_sequences_at_the_ends_of_a_long_list(libmla, n, L, heads, num_sms):
    """A worker goes from one to the other past 2^18 empty sequences, in runs and in rounds."""
    from mla_latent_kv_26_b200.prefill import prefill_attention

    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(242)
    q, kv, pe = (torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)
                 for s in ((2 * n, heads, 192), (2 * L, heads, 256), (2 * L, 64)))
    batch, err = 1 << 18, torch.zeros(1, dtype=torch.int32, device=dev)
    results = []
    for b in (2, batch):
        cu_q, cu_k = (torch.full((b + 1,), x, dtype=torch.int32, device=dev) for x in (n, L))
        cu_q[0], cu_k[0], cu_q[-1], cu_k[-1] = 0, 0, 2 * n, 2 * L
        results.append(prefill_attention(q, kv, pe, cu_q, cu_k, num_sms=num_sms, error_word=err))
    assert int(err.item()) == 0
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
