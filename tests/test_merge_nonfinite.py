"""NaN parts in ``mla_merge``: a part whose lse is NaN makes the merged row NaN,
a part with lse -inf weighs nothing whatever its row holds."""

import math

import pytest
import torch

import oracle
from test_parity_prefill import _attention_inputs, dev  # noqa: F401  (dev: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("parts", [1, 3])
@pytest.mark.parametrize("width", [128, 512])
def test_merge_of_nan_parts(dev, libmla, width, parts):
    rows = 37
    g = torch.Generator().manual_seed(width + parts)
    po = torch.randn(parts, rows, width, generator=g).to(torch.bfloat16)
    pl = torch.randn(parts, rows, generator=g) * 3
    po[0, 2], pl[0, 2] = math.nan, math.nan              # NaN in one part
    po[:, 5], pl[:, 5] = math.nan, math.nan              # in every part
    po[-1, 9], pl[-1, 9] = math.nan, -math.inf           # an empty part, its row undefined
    pl[:, 11] = -math.inf                                # empty everywhere
    pl[0, 20] = math.nan                                 # lse alone
    out = torch.empty(rows, width, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(rows, device=dev)
    desc = libmla.make_merge_desc(parts=parts, rows=rows, d_latent=width)
    libmla.check(libmla.mla_merge(desc, po.to(dev), pl.to(dev), out, lse), "mla_merge")
    out, lse = out.double().cpu(), lse.double().cpu()
    nan = [2, 5, 20]
    assert torch.isnan(out[nan]).all() and torch.isnan(lse[nan]).all()
    assert torch.all(out[11] == 0) and lse[11] == -math.inf
    if parts == 1:
        assert torch.all(out[9] == 0) and lse[9] == -math.inf
    rest = [r for r in range(rows) if r not in nan]
    po[-1, 9] = 0
    mo, ml = oracle.lse_merge(po[:, rest], pl[:, rest])
    assert ((out[rest] - mo).abs() <= 2.0 ** -8 * mo.abs() + 2.0 ** -16).all()
    live = ~torch.isinf(ml)
    assert ((lse[rest] - ml).abs()[live] <= 2.0 ** -20).all() and torch.equal(torch.isneginf(lse[rest]), ~live)


def test_context_in_parts_keeps_a_nan_query(dev):
    from mla_latent_kv_26_b200.prefill import merge_parts, prefill_attention

    n, L, cut = 150, 1000, 600
    q, kv, pe, cu_q, _ = _attention_inputs(3, [(n, L)], 211)
    q[4, 1, 17], q[149, 0, 150] = math.nan, math.inf
    qg, kg, pg, cq = q.to(dev), kv.to(dev), pe.to(dev), cu_q.to(dev)
    parts = [prefill_attention(qg, kg[a:b], pg[a:b], cq, torch.tensor([0, b - a], dtype=torch.int32, device=dev),
                               causal=c) for a, b, c in ((0, cut, False), (cut, L, True))]
    out, lse = merge_parts(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]))
    hit = torch.zeros(n, 3, dtype=torch.bool)
    hit[4, 1] = hit[149, 0] = True
    assert torch.equal(torch.isnan(lse).cpu(), hit)
    assert torch.equal(torch.isnan(out).all(-1).cpu(), hit) and torch.equal(torch.isnan(out).any(-1).cpu(), hit)
