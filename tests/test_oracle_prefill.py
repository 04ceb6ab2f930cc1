"""Pins of the prefill oracle: against the naive per-head attention of the
decode oracle, decode's own causal rule, and brute force on tiny shapes."""

import math

import torch

import oracle


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_one_query_is_the_unabsorbed_attention():
    H, L = 3, 17
    w, rows, q = _rand(H, 256, 512, seed=1) * 0.05, _rand(L, 576, seed=2), _rand(1, H, 192, seed=3)
    kv = oracle.prefill.expand_kv(rows, w)
    out, _ = oracle.prefill.prefill_attention(q, kv, rows[:, 512:], [0, 1], [0, L])
    ref = oracle.unabsorbed_attention(q[0, :, :128], q[0, :, 128:], w[:, :128], w[:, 128:], rows[:, :512], rows[:, 512:])
    assert torch.allclose(out[0], ref, rtol=0, atol=1e-12)


def test_causal_rule_is_decodes():
    """Query i of n over L keys: decode's visible tokens."""
    H, n, L = 2, 5, 9
    q, kv, pe = _rand(n, H, 192, seed=4), _rand(L, H, 256, seed=5), _rand(L, 64, seed=6)
    out, lse = oracle.prefill.prefill_attention(q, kv, pe, [0, n], [0, L])
    for i in range(n):
        t = oracle.visible_tokens(L, n, i, True, None)
        o, l = oracle.prefill.prefill_attention(q[i:i + 1], kv[t], pe[t], [0, 1], [0, len(t)], causal=False)
        assert torch.allclose(out[i], o[0], atol=1e-12) and torch.allclose(lse[i], l[0], atol=1e-12)


def test_brute_force_ragged():
    H, ns, Ls = 2, [3, 0, 2], [4, 2, 1]
    cu_q, cu_k = [0, 3, 3, 5], [0, 4, 6, 7]
    q, kv, pe = _rand(5, H, 192, seed=7), _rand(7, H, 256, seed=8), _rand(7, 64, seed=9)
    out, lse, mag, smag, smax = oracle.prefill.prefill_attention(q, kv, pe, cu_q, cu_k, softmax_scale=0.1, absolute=True)
    for b in range(3):
        for i in range(ns[b]):
            for h in range(H):
                seen = [t for t in range(Ls[b]) if t <= Ls[b] - ns[b] + i]
                r, ks = cu_q[b] + i, [cu_k[b] + t for t in seen]
                if not ks:
                    assert torch.all(out[r, h] == 0) and lse[r, h] == -math.inf and smax[r, h] == 0
                    continue
                terms = [[float(q[r, h, d]) * float(kv[t, h, d] if d < 128 else pe[t, d - 128]) for d in range(192)]
                         for t in ks]
                s = [0.1 * sum(x) for x in terms]
                z = sum(math.exp(x) for x in s)
                assert abs(float(lse[r, h]) - math.log(z)) < 1e-12
                assert abs(float(smag[r, h]) - max(0.1 * sum(abs(y) for y in x) for x in terms)) < 1e-10
                assert abs(float(smax[r, h]) - max(abs(x) for x in s)) < 1e-12
                for j in (0, 77, 127):
                    v = [float(kv[t, h, 128 + j]) for t in ks]
                    assert abs(float(out[r, h, j]) - sum(math.exp(x) / z * y for x, y in zip(s, v))) < 1e-12
                    assert abs(float(mag[r, h, j]) - sum(math.exp(x) / z * abs(y) for x, y in zip(s, v))) < 1e-12


def test_parts_merge_to_the_whole():
    H, n, L = 2, 4, 30
    q, kv, pe = _rand(n, H, 192, seed=10), _rand(L, H, 256, seed=11), _rand(L, 64, seed=12)
    whole = oracle.prefill.prefill_attention(q, kv, pe, [0, n], [0, L])
    parts = [oracle.prefill.prefill_attention(q, kv[a:b], pe[a:b], [0, n], [0, b - a], causal=c)
             for a, b, c in ((0, 11, False), (11, 20, False), (20, 30, True))]
    out, lse = oracle.lse_merge(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]))
    assert torch.allclose(out, whole[0], atol=1e-12) and torch.allclose(lse, whole[1], atol=1e-12)


def test_cache_read_values():
    cache = torch.arange(3 * 64, dtype=torch.float64).view(3, 64, 1).expand(3, 64, 576).contiguous()
    table = torch.tensor([[2, 0], [1, 9]], dtype=torch.int32)
    out = oracle.prefill.cache_read(cache, table, [1, 4, 8], [62, 63], torch.full((10, 576), -5.0))
    # sequence 0: page 2 rows 62, 63, page 0 row 0; sequence 1: page 1 row 63, then a page that does not exist
    assert out[:, 0].tolist() == [-5.0, 190.0, 191.0, 0.0, 127.0, 0.0, 0.0, 0.0, -5.0, -5.0]
    gone = oracle.prefill.cache_read(cache, table, [0, 2, 2], [127, 0], torch.full((2, 576), -5.0))
    assert gone[:, 0].tolist() == [63.0, 0.0]
