"""NaN and infinities in owned query rows of the prefill attention, whole and
split over workers, and in the parts of a merge.

A score with a NaN or an infinity in it has no finite softmax: the row and head
it belongs to get NaN in ``out`` and ``lse``, however the work was cut; all
others are untouched. (0, -inf) stands for a row without a visible key alone.
"""

import math

import pytest
import torch

import oracle
from test_parity_prefill import _attention_inputs, _check_attention, dev  # noqa: F401  (dev: a fixture)

pytestmark = pytest.mark.gpu


def _run(dev, q, kv, pe, cu_q, cu_k, causal, num_sms=0):
    from mla_latent_kv_26_b200.prefill import prefill_attention

    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = prefill_attention(q.to(dev), kv.to(dev), pe.to(dev), cu_q.to(dev), cu_k.to(dev), causal=causal,
                                 num_sms=num_sms, error_word=err)
    assert int(err.item()) == 0
    return out.double().cpu(), lse.double().cpu()


def _check_rows(out, lse, bad, q, kv, pe, cu_q, cu_k, causal):
    """NaN in the rows and heads ``bad``, every other one as the oracle has it."""
    clean = torch.where(torch.isfinite(q.float()), q.float(), torch.zeros(())).to(torch.bfloat16)
    ref, rl = oracle.prefill.prefill_attention(clean, kv, pe, cu_q, cu_k, causal=causal)
    for r, h in bad:
        assert torch.isnan(out[r, h]).all() and torch.isnan(lse[r, h]), (r, h)
        out[r, h], lse[r, h] = ref[r, h], rl[r, h]
    _check_attention(out, lse, clean, kv, pe, cu_q, cu_k, causal, oracle.DEFAULT_SOFTMAX_SCALE)


# num_sms 2: one worker, every item whole; 0: every item split over many workers
@pytest.mark.parametrize("num_sms", [2, 0, 10])
@pytest.mark.parametrize("causal", [True, False])
def test_nonfinite_queries(dev, causal, num_sms):
    q, kv, pe, cu_q, cu_k = _attention_inputs(2, [(256, 1500), (3, 40), (1, 1)], 201)
    bad = [(5, 0, 3, math.nan), (5, 1, 191, math.nan), (100, 1, 0, math.inf), (130, 0, 127, -math.inf),
           (255, 0, 150, math.nan), (257, 1, 64, math.inf), (258, 0, 190, math.nan)]
    for r, h, d, x in bad:
        q[r, h, d] = x
    q[259, 1] = math.nan                                 # a row that sees one key
    where = [b[:2] for b in bad] + [(259, 1)]
    out, lse = _run(dev, q, kv, pe, cu_q, cu_k, causal, num_sms)
    _check_rows(out, lse, where, q, kv, pe, cu_q, cu_k, causal)


@pytest.mark.parametrize("num_sms", [2, 0])
def test_infinite_query_against_keys_of_one_sign(dev, num_sms):
    """Every score of the row is -inf (or +inf): still no row without keys."""
    q, kv, pe, cu_q, cu_k = _attention_inputs(2, [(200, 900)], 202)
    kv[..., 0] = -(kv[..., 0].abs() + 0.5)
    q[7, 0, 0], q[140, 1, 0] = math.inf, -math.inf
    for causal in (True, False):
        out, lse = _run(dev, q, kv, pe, cu_q, cu_k, causal, num_sms)
        _check_rows(out, lse, [(7, 0), (140, 1)], q, kv, pe, cu_q, cu_k, causal)


@pytest.mark.parametrize("num_sms", [2, 0])
def test_nonfinite_query_without_keys(dev, num_sms):
    """More queries than keys: the first rows see none, whatever they hold."""
    q, kv, pe, cu_q, cu_k = _attention_inputs(2, [(300, 200), (4, 0)], 203)
    q[3], q[99, 1], q[301] = math.nan, math.inf, math.nan
    q[100, 0] = math.nan                                 # the first row with a key
    out, lse = _run(dev, q, kv, pe, cu_q, cu_k, True, num_sms)
    _check_rows(out, lse, [(100, 0)], q, kv, pe, cu_q, cu_k, True)
    assert torch.all(out[:100] == 0) and torch.all(torch.isneginf(lse[300:]))
