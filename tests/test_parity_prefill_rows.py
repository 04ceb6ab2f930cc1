"""Rows around those that a prefill call owns: left as they were, in MlaPrefill's
own buffers and in memory around buffers of a smaller capacity."""

import math

import pytest
import torch

import oracle
from test_parity_prefill import (_attention_inputs, _check_attention, _check_chunk, _chunk,  # noqa: F401
                                 dev)

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


class _Guarded:
    """A tensor in the middle of a larger one, whose other values have to stay."""

    def __init__(self, like, pad=64):
        self.all = torch.full((like.shape[0] + 2 * pad, *like.shape[1:]), 7, dtype=like.dtype, device=like.device)
        self.pad, self.view = pad, self.all[pad:pad + like.shape[0]]
        assert self.view.data_ptr() % 32 == 0

    def intact(self):
        return bool((self.all[:self.pad] == 7).all() and (self.all[self.pad + self.view.shape[0]:] == 7).all())


def test_more_keys_than_capacity_stay_inside_the_buffers(dev, libmla):
    """Keys beyond ``max_keys`` are cut off: nothing around the buffers changes, the
    result is that of the offsets clipped to the capacity, and the error word says so."""
    from mla_latent_kv_26_b200.prefill import MlaPrefill

    cache, bt, q, w, cu_q, cu_k = _chunk([(40, 200), (30, 90)], 2, 233, False)
    pre = MlaPrefill(max_queries=70, max_keys=150, num_heads=2, device=dev)
    guards = {n: _Guarded(getattr(pre, n)) for n in ("rows", "kv", "out", "lse", "workspace")}
    for n, g in guards.items():
        setattr(pre, n, g.view)
    pre(*(t.to(dev) for t in (q, w, cache, bt, cu_q, cu_k)))
    torch.cuda.synchronize(dev)
    assert int(pre.error_word.item()) == libmla.MLA_DEVERR_SEQ_LEN
    assert all(g.intact() for g in guards.values()), [n for n, g in guards.items() if not g.intact()]
    clipped = torch.tensor([0, 150], dtype=torch.int32)
    _check_chunk(pre.out[:40], pre.lse[:40], cache, bt, q[:40], w, cu_q[:2], clipped)
    assert torch.all(pre.out[40:] == 0) and torch.all(torch.isneginf(pre.lse[40:]))  # no keys are left for them


@pytest.mark.parametrize("num_sms", [0, 2])
@pytest.mark.parametrize("cu_q,cu_k,clip_q,clip_k", [
    ([0, 60, 500], [0, 80, 150], [0, 60, 100], [0, 80, 150]), ([0, 60, 100], [0, 90, 5000], [0, 60, 100], [0, 90, 150]),
    ([0, 70, 40], [0, 50, 90], [0, 70, 70], [0, 50, 90]), ([-4, 60, 100], [-9, 80, 150], [0, 60, 100], [0, 80, 150]),
])
def test_bad_offsets_stay_inside_and_give_the_clipped_result(dev, libmla, cu_q, cu_k, clip_q, clip_k, num_sms):
    from mla_latent_kv_26_b200.prefill import attention_workspace_bytes, prefill_attention

    q, kv, pe, _, _ = _attention_inputs(2, [(100, 150)], 234)
    out, lse = (_Guarded(torch.empty(100, 2, *s, dtype=t, device=dev)) for s, t in (((128,), torch.bfloat16),
                                                                                  ((), torch.float32)))
    ws = _Guarded(torch.empty(attention_workspace_bytes(100, 2, 150, batch=2, num_sms=num_sms), dtype=torch.uint8,
                              device=dev))
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out.view.fill_(7)
    lse.view.fill_(7)
    prefill_attention(q.to(dev), kv.to(dev), pe.to(dev), *(torch.tensor(c, dtype=torch.int32, device=dev)
                                                          for c in (cu_q, cu_k)),
                      out=out.view, lse=lse.view, workspace=ws.view, num_sms=num_sms, error_word=err)
    torch.cuda.synchronize(dev)
    assert int(err.item()) == libmla.MLA_DEVERR_SEQ_LEN and out.intact() and lse.intact() and ws.intact()
    _check_attention(out.view, lse.view, q, kv, pe, clip_q, clip_k, True, oracle.DEFAULT_SOFTMAX_SCALE)
    rest = slice(clip_q[-1], None)
    assert torch.all(out.view[rest] == 7) and torch.all(lse.view[rest] == 7)


@pytest.mark.parametrize("fp8", [False, True])
def test_context_in_parts_through_the_cache(dev, fp8):
    """A context too long for one expansion: its parts read back by ``starts``, the
    older ones without a mask, the last one causal, merged by their log-sum-exp.
    On top of the chain's bound each part's output is rounded to bf16 before the
    merge, another 2^-8 of sum p|v|."""
    from mla_latent_kv_26_b200.prefill import MlaPrefill, merge_parts

    H, seqs = 3, [(70, 900), (130, 333), (1, 64)]
    cache, bt, q, w, cu_q, cu_k = _chunk(seqs, H, 235, fp8)
    # tokens of every part of every sequence; the last ones hold all new tokens
    parts = [[400, 100, 0], [300, 0, 63], [200, 233, 1]]
    g = [t.to(dev) for t in (q, w, cache, bt)]
    pre = MlaPrefill(max_queries=q.shape[0], max_keys=500, num_heads=H, device=dev)
    outs, lses = [], []
    for i, lens in enumerate(parts):
        first = torch.tensor([sum(p[b] for p in parts[:i]) for b in range(len(seqs))], dtype=torch.int32, device=dev)
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev)
        o = pre(*g, cu_q.to(dev), cu, starts=first, causal=i == len(parts) - 1)
        outs.append(o.clone())
        lses.append(pre.lse.clone())
    assert int(pre.error_word.item()) == 0
    assert torch.all(torch.isneginf(lses[0][-1])) and torch.all(outs[0][-1] == 0)     # an empty part
    out, lse = merge_parts(torch.stack(outs), torch.stack(lses))
    rows = oracle.prefill.cache_read(cache, bt, cu_k, None, torch.zeros(int(cu_k[-1]), 576))
    kv = oracle.prefill.expand_kv(rows, w).to(torch.bfloat16)
    ref, rl, mag, _, _ = oracle.prefill.prefill_attention(q, kv, rows[:, 512:], cu_q, cu_k, absolute=True)
    o, l = out.double().cpu(), lse.double().cpu()
    assert ((o - ref).abs() <= 2.0 ** -8 * ref.abs() + (3 * 2.0 ** -8 + 2.0 ** -10) * mag).all()
    assert ((l - rl).abs() <= 1e-3).all()
