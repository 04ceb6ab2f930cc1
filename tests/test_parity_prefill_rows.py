"""Rows around those that a prefill call owns: left as they were, in MlaPrefill's
own buffers and in memory around buffers of a smaller capacity."""

import math

import pytest
import torch

import oracle
from test_parity_prefill import _check_chunk, _chunk, dev  # noqa: F401  (dev: a fixture)

pytestmark = pytest.mark.gpu


def test_rows_without_a_sequence_keep_what_they_held(dev):
    """0 and -inf in a new object whatever its memory held before, later an earlier call's rows."""
    from mla_latent_kv_26_b200.prefill import MlaPrefill

    H, cap = 2, 200
    junk = [torch.full((cap, H, 128), math.nan, dtype=torch.bfloat16, device=dev) for _ in range(4)]
    junk += [torch.full((cap, H), math.nan, device=dev) for _ in range(4)]
    del junk
    pre = MlaPrefill(max_queries=cap, max_keys=500, num_heads=H, device=dev)
    q_all = torch.zeros(cap, H, 192, dtype=torch.bfloat16, device=dev)

    def call(seqs, seed):
        cache, bt, q, w, cu_q, cu_k = _chunk(seqs, H, seed, False)
        q_all[:q.shape[0]] = q.to(dev)
        pre(q_all, w.to(dev), cache.to(dev), bt.to(dev), cu_q.to(dev), cu_k.to(dev))
        assert int(pre.error_word.item()) == 0
        n = q.shape[0]
        _check_chunk(pre.out[:n], pre.lse[:n], cache, bt, q, w, cu_q, cu_k)
        return n

    n = call([(90, 200), (40, 41)], 231)
    assert torch.all(pre.out[n:] == 0) and torch.all(torch.isneginf(pre.lse[n:]))
    out, lse = pre.out.clone(), pre.lse.clone()
    m = call([(17, 300)], 232)
    assert torch.equal(pre.out[m:], out[m:]) and torch.equal(pre.lse[m:], lse[m:])
