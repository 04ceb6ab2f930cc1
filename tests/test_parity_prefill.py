"""GPU parity of the prefill operators (cache read-back, key / value expansion,
ragged attention) and of the three together against the float64 oracle.

Tolerances, from the arithmetic (a rounding to bf16 is off by at most 2^-8 of
the value, to float32 by 2^-24):

* read-back: exact.
* expansion: one bf16 rounding of a float32 sum of 512 products:
  2^-8 |ref| + 512 * 2^-24 * sum |terms| (2^-14 of it allowed).
* attention: with A = scale * sum_d |q_d k_d|, a score is off by at most
  196 * 2^-24 * A (192 products summed in float32), its exponent's argument by
  2^-22 |s| more, the exponential by 2^-21: every p is off by the relative
  e = 196 * 2^-24 * A + 2^-22 |s| + 2^-20, and rounded to bf16 for the product:
  |out - ref| <= 2^-8 |ref| + (2^-8 + 2 e + 2^-12) * sum_t p_t |v_t|,
  |lse - ref| <= e + L * 2^-24 + 2^-21 |ref| + 2^-20.
"""

import math

import pytest
import torch

import oracle
from mla_latent_kv_26_b200.workloads import make_fp8_cache, small

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(libmla):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda", torch.cuda.current_device())


def _offsets(counts, first=0):
    return torch.tensor([first] + counts, dtype=torch.int64).cumsum(0).to(torch.int32)


# ---------------------------------------------------------------- read-back


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,starts,first", [
    ([1], None, 0), ([64, 65, 1, 700], None, 0), ([3, 0, 130, 0, 0, 66, 257], [5, 0, 63, 1, 0, 64, 100], 7),
    ([2] * 40 + [33], [1] * 41, 0),
])
def test_cache_read(dev, fp8, lens, starts, first):
    from mla_latent_kv_26_b200.prefill import cache_read

    total = [max(n + (starts[i] if starts else 0), 1) for i, n in enumerate(lens)]
    d = small(batch=len(lens), heads=1, lens=total, seed=len(lens), nan_tail=True)
    cache = make_fp8_cache(d, nan_tail=True) if fp8 else d["cache"]
    off = _offsets(lens, first)
    M = int(off[-1]) + 9
    out = torch.full((M, 576), 7.0, dtype=torch.bfloat16, device=dev)
    st = torch.tensor(starts, dtype=torch.int32) if starts else None
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    got = cache_read(cache.to(dev), d["block_table"].to(dev), off.to(dev), starts=st.to(dev) if starts else None,
                     out=out, error_word=err)
    assert got is out and int(err.item()) == 0
    ref = oracle.prefill.cache_read(cache, d["block_table"], off, st, torch.full((M, 576), 7.0))
    assert torch.equal(got.double().cpu(), ref)


def test_cache_read_bad_positions_pages_and_offsets(dev, libmla):
    from mla_latent_kv_26_b200.prefill import cache_read

    d = small(batch=3, heads=1, lens=[130, 64, 200], seed=5)
    bt = d["block_table"].clone()
    bt[2, 1] = d["num_pages"] + 4
    cache, bt_g = d["cache"].to(dev), bt.to(dev)

    def run(off, starts, rows):
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        out = torch.full((rows, 576), 7.0, dtype=torch.bfloat16, device=dev)
        cache_read(cache, bt_g, torch.tensor(off, dtype=torch.int32, device=dev),
                   starts=torch.tensor(starts, dtype=torch.int32, device=dev), out=out, error_word=err)
        return out.double().cpu(), int(err.item())

    off, starts = [0, 20, 84, 284], [-3, 0, 0]   # three rows before position 0; page 1 of sequence 2 does not exist
    out, err = run(off, starts, 300)
    assert err == libmla.MLA_DEVERR_POSITION | libmla.MLA_DEVERR_PAGE_ID
    ref = oracle.prefill.cache_read(d["cache"], bt, off, starts, torch.full((300, 576), 7.0))
    assert torch.equal(out, ref) and torch.all(out[:3] == 0) and torch.all(out[84 + 64:84 + 128] == 0)
    # more rows than the matrix holds: clipped and reported
    out, err = run([0, 20, 84, 148], [0, 0, 0], 100)
    assert err & libmla.MLA_DEVERR_SEQ_LEN and torch.equal(out, ref_rows(d, bt, [0, 20, 84, 148], 100))
    # offsets out of order touch nothing outside the matrix
    out, err = run([0, 50, 20, 60], [0, 0, 0], 64)
    assert err & libmla.MLA_DEVERR_SEQ_LEN and torch.all(out[60:] == 7.0)


def ref_rows(d, bt, off, rows):
    return oracle.prefill.cache_read(d["cache"], bt, off, None, torch.full((rows, 576), 7.0))


# ---------------------------------------------------------------- expansion


@pytest.mark.parametrize("rows,heads,stride", [(1, 1, 576), (127, 3, 512), (128, 128, 576), (129, 16, 640),
                                               (1000, 5, 576), (257, 40, 576)])
def test_expand_kv(dev, rows, heads, stride):
    from mla_latent_kv_26_b200.prefill import expand_kv

    g = torch.Generator().manual_seed(rows + heads)
    x = torch.randn(rows, stride, generator=g).to(torch.bfloat16)
    w = (torch.randn(heads, 256, 512, generator=g) * 0.05).to(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    got = expand_kv(x.to(dev), w.to(dev), error_word=err).double().cpu()
    assert int(err.item()) == 0
    ref, mag = oracle.prefill.expand_kv(x, w), oracle.prefill.expand_kv(x.abs(), w.abs())
    assert ((got - ref).abs() <= ref.abs() * 2.0 ** -8 + mag * 2.0 ** -14).all()


@pytest.mark.parametrize("rows,count", [(300, 0), (300, 1), (300, 128), (300, 200), (300, 300), (300, 999), (40, -5)])
def test_expand_kv_row_count(dev, rows, count):
    """Rows at or behind the device-side count are neither read (NaN here) nor written."""
    from mla_latent_kv_26_b200.prefill import expand_kv

    g = torch.Generator().manual_seed(3)
    x = torch.randn(rows, 576, generator=g).to(torch.bfloat16)
    live = max(min(rows, count), 0)
    x[live:] = math.nan
    w = (torch.randn(7, 256, 512, generator=g) * 0.05).to(torch.bfloat16)
    out = torch.full((rows, 7, 256), 7.0, dtype=torch.bfloat16, device=dev)
    expand_kv(x.to(dev), w.to(dev), out=out, row_count=torch.tensor([count], dtype=torch.int32, device=dev))
    got = out.double().cpu()
    ref, mag = oracle.prefill.expand_kv(x[:live], w), oracle.prefill.expand_kv(x[:live].abs(), w.abs())
    assert ((got[:live] - ref).abs() <= ref.abs() * 2.0 ** -8 + mag * 2.0 ** -14).all()
    assert torch.all(got[live:] == 7.0)


# ---------------------------------------------------------------- attention


def _attention_inputs(heads, seqs, seed, *, q_std=1.0, pad=0):
    """Ragged inputs with ``pad`` unowned rows before, and after, the sequences' (NaN in kv and k_pe)."""
    g = torch.Generator().manual_seed(seed)
    n, L = [s[0] for s in seqs], [s[1] for s in seqs]
    cu_q, cu_k = _offsets(n, pad), _offsets(L, pad)
    Nq, Nk = int(cu_q[-1]) + pad, int(cu_k[-1]) + pad
    q = (torch.randn(Nq, heads, 192, generator=g) * q_std).to(torch.bfloat16)
    kv = torch.randn(Nk, heads, 256, generator=g).to(torch.bfloat16)
    pe = torch.randn(Nk, 64, generator=g).to(torch.bfloat16)
    if pad:
        for t in (kv, pe):
            t[:pad] = math.nan
            t[-pad:] = math.nan
        q[:pad] = math.nan
        q[-pad:] = math.inf
    return q, kv, pe, cu_q, cu_k


def _check_attention(out, lse, q, kv, pe, cu_q, cu_k, causal, scale, where=""):
    out, lse = out.double().cpu(), lse.double().cpu()
    ref, rl, mag, smag, smax = oracle.prefill.prefill_attention(q, kv, pe, cu_q, cu_k, causal=causal,
                                                                softmax_scale=scale, absolute=True)
    own = slice(int(cu_q[0]), int(cu_q[-1]))
    out, lse, ref, rl, mag, smag, smax = (t[own] for t in (out, lse, ref, rl, mag, smag, smax))
    e = 196 * 2.0 ** -24 * smag + 2.0 ** -22 * smax + 2.0 ** -20
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * e + 2.0 ** -12)[..., None] * mag
    bad = ~((out - ref).abs() <= bound)
    assert not bad.any(), f"{where}: {int(bad.sum())} of {bad.numel()} outputs out of bound"
    empty = torch.isinf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    L = max(int(kv.shape[0]), 1)
    lb = e + L * 2.0 ** -24 + 2.0 ** -21 * rl.abs() + 2.0 ** -20
    assert ((lse - rl).abs() <= lb)[~empty].all(), where


ATTENTION = [
    (1, [(1, 1)], True),
    (3, [(1, 64), (5, 5), (0, 70), (7, 0), (128, 128)], True),
    (2, [(129, 129), (0, 0), (256, 300), (257, 1000)], True),
    (2, [(300, 200), (40, 7), (1, 130)], True),          # more queries than keys: the first rows see none
    (2, [(130, 127), (1, 0), (200, 513)], False),
    (16, [(64, 3000)], True),                            # few queries, long keys: split along the keys
    (5, [(700, 700)], True),
    (1, [(1, 5000), (2, 4097)], False),
    (1, [(2, 2)] * 70 + [(130, 140)], True),             # more sequences than a warp scans at once
]


@pytest.mark.parametrize("num_sms", [0, 1, 5])
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention(dev, case, num_sms):
    from mla_latent_kv_26_b200.prefill import prefill_attention

    heads, seqs, causal = ATTENTION[case]
    q, kv, pe, cu_q, cu_k = _attention_inputs(heads, seqs, 100 + case)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = prefill_attention(q.to(dev), kv.to(dev), pe.to(dev), cu_q.to(dev), cu_k.to(dev), causal=causal,
                                 num_sms=num_sms, error_word=err)
    assert int(err.item()) == 0
    _check_attention(out, lse, q, kv, pe, cu_q, cu_k, causal, oracle.DEFAULT_SOFTMAX_SCALE)


@pytest.mark.parametrize("q_std,scale", [(10.0, oracle.DEFAULT_SOFTMAX_SCALE), (0.0, 1.0), (3.0, 0.5)])
def test_attention_large_and_equal_scores(dev, q_std, scale):
    """Maxima that grow by hundreds between tiles (O and l rescaled), and equal scores."""
    from mla_latent_kv_26_b200.prefill import prefill_attention

    q, kv, pe, cu_q, cu_k = _attention_inputs(2, [(200, 900), (33, 640)], 7, q_std=q_std)
    for causal in (True, False):
        out, lse = prefill_attention(q.to(dev), kv.to(dev), pe.to(dev), cu_q.to(dev), cu_k.to(dev), causal=causal,
                                     softmax_scale=scale)
        _check_attention(out, lse, q, kv, pe, cu_q, cu_k, causal, scale, f"causal={causal}")


def test_attention_growing_maximum(dev):
    """Every key tile holds a larger maximum than the one before, in some rows only."""
    from mla_latent_kv_26_b200.prefill import prefill_attention

    q, kv, pe, cu_q, cu_k = _attention_inputs(2, [(256, 1500)], 8)
    q[::3] = 1.0
    kv[..., :128] = (torch.arange(1500) / 128).floor()[:, None, None] * 0.5
    out, lse = prefill_attention(q.to(dev), kv.to(dev), pe.to(dev), cu_q.to(dev), cu_k.to(dev))
    _check_attention(out, lse, q, kv, pe, cu_q, cu_k, True, oracle.DEFAULT_SOFTMAX_SCALE)


@pytest.mark.parametrize("num_sms", [0, 2])
def test_attention_unowned_rows(dev, num_sms):
    """NaN and infinities in rows no sequence owns, before, behind and inside the
    last tiles, change nothing; unowned output rows stay as they were. k_pe is a
    strided view."""
    from mla_latent_kv_26_b200.prefill import prefill_attention

    q, kv, pe, cu_q, cu_k = _attention_inputs(3, [(70, 90), (0, 0), (129, 200)], 9, pad=11)
    wide = torch.full((pe.shape[0], 576), math.nan, dtype=torch.bfloat16)
    wide[:, 512:] = pe
    out = torch.full((q.shape[0], 3, 128), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((q.shape[0], 3), 7.0, device=dev)
    prefill_attention(q.to(dev), kv.to(dev), wide.to(dev)[:, 512:], cu_q.to(dev), cu_k.to(dev), out=out, lse=lse,
                      num_sms=num_sms)
    _check_attention(out, lse, q, kv, pe, cu_q, cu_k, True, oracle.DEFAULT_SOFTMAX_SCALE)
    for t in (out, lse):
        assert torch.all(t[:11] == 7.0) and torch.all(t[-11:] == 7.0)


def test_attention_next_sequence_nan(dev):
    """A sequence's last key tile holds the next sequence's rows: their NaN stays theirs."""
    from mla_latent_kv_26_b200.prefill import prefill_attention

    q, kv, pe, cu_q, cu_k = _attention_inputs(2, [(50, 50), (20, 40)], 10)
    kv[50:], pe[50:] = math.nan, math.nan
    out, lse = prefill_attention(q.to(dev), kv.to(dev), pe.to(dev), cu_q.to(dev), cu_k.to(dev))
    _check_attention(out[:50], lse[:50], q[:50], kv[:50], pe[:50], cu_q[:2], cu_k[:2], True,
                     oracle.DEFAULT_SOFTMAX_SCALE)
    assert torch.isnan(out[50:]).any()


def test_attention_no_keys_at_all(dev):
    from mla_latent_kv_26_b200.prefill import prefill_attention

    q, kv, pe, cu_q, cu_k = _attention_inputs(2, [(5, 0), (300, 0)], 11)
    out, lse = prefill_attention(q.to(dev), kv.to(dev), pe.to(dev), cu_q.to(dev), cu_k.to(dev))
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


def test_attention_bad_offsets_are_clipped_and_reported(dev, libmla):
    from mla_latent_kv_26_b200.prefill import prefill_attention

    q, kv, pe, _, _ = _attention_inputs(2, [(100, 150)], 12)
    for cu_q, cu_k in (([0, 60, 500], [0, 80, 150]), ([0, 60, 100], [0, 90, 5000]), ([0, 70, 40], [0, 50, 90]),
                       ([-4, 60, 100], [0, 80, 150])):
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        prefill_attention(q.to(dev), kv.to(dev), pe.to(dev), torch.tensor(cu_q, dtype=torch.int32, device=dev),
                          torch.tensor(cu_k, dtype=torch.int32, device=dev), error_word=err)
        assert int(err.item()) == libmla.MLA_DEVERR_SEQ_LEN, (cu_q, cu_k)


@pytest.mark.parametrize("cuts", [[0, 400, 1000], [0, 64, 65, 640, 1000]])
def test_parts_of_a_context_merge(dev, cuts):
    """The older context in parts, seen by every new token, and the new tokens'
    own causal part, merged by their log-sum-exp: the whole attention. Each
    part's output is rounded to bf16 before the merge: another 2^-8 of sum p|v|."""
    from mla_latent_kv_26_b200.prefill import merge_parts, prefill_attention

    H, n, L = 4, 150, 1150
    q, kv, pe, cu_q, cu_k = _attention_inputs(H, [(n, L)], 13)
    qg, kg, pg, cq = q.to(dev), kv.to(dev), pe.to(dev), cu_q.to(dev)
    parts = [(a, b, False) for a, b in zip(cuts, cuts[1:])] + [(cuts[-1], L, True)]
    outs, lses = [], []
    for a, b, causal in parts:
        o, l = prefill_attention(qg, kg[a:b], pg[a:b], cq, torch.tensor([0, b - a], dtype=torch.int32, device=dev),
                                 causal=causal)
        outs.append(o)
        lses.append(l)
    out, lse = merge_parts(torch.stack(outs), torch.stack(lses))
    ref, rl, mag, _, _ = oracle.prefill.prefill_attention(q, kv, pe, cu_q, cu_k, absolute=True)
    assert ((out.double().cpu() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -7 + 2.0 ** -11) * mag).all()
    assert ((lse.double().cpu() - rl).abs() <= 2.0 ** -14).all()
    mo, ml = oracle.lse_merge(torch.stack(outs).cpu(), torch.stack(lses).cpu())
    assert ((out.double().cpu() - mo).abs() <= 2.0 ** -8 * mo.abs() + 2.0 ** -16).all()


# ---------------------------------------------------------------- the three together


def _chunk(seqs, heads, seed, fp8):
    """A cache that already holds every sequence's L tokens, n of them the chunk's."""
    L = [s[1] for s in seqs]
    d = small(batch=len(seqs), heads=1, lens=[max(x, 1) for x in L], seed=seed, nan_tail=True)
    cache = make_fp8_cache(d, nan_tail=True) if fp8 else d["cache"]
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(sum(s[0] for s in seqs), heads, 192, generator=g).to(torch.bfloat16)
    w = (torch.randn(heads, 256, 512, generator=g) * 0.05).to(torch.bfloat16)
    return cache, d["block_table"], q, w, _offsets([s[0] for s in seqs]), _offsets(L)


def _check_chunk(out, lse, cache, bt, q, w, cu_q, cu_k):
    """Against the chain in float64 with the keys and values rounded to bf16 once,
    as the operator defines them. A key or value whose float32 sum lies next to a
    rounding border may go to the other neighbour (2^-7 of the value at most);
    few do, and they move an output by far less than the bound on average: the
    elementwise bound below adds 2^-8 of sum p|v| for them."""
    rows = oracle.prefill.cache_read(cache, bt, cu_k, None, torch.zeros(int(cu_k[-1]), 576))
    kv = oracle.prefill.expand_kv(rows, w).to(torch.bfloat16)
    ref, rl, mag, _, _ = oracle.prefill.prefill_attention(q, kv, rows[:, 512:], cu_q, cu_k, absolute=True)
    o, l = out.double().cpu(), lse.double().cpu()
    assert ((o - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -7 + 2.0 ** -10) * mag).all()
    assert float((o - ref).norm() / ref.norm()) <= 5e-3
    assert ((l - rl).abs() <= 1e-3).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,seqs", [(3, [(1, 1)]), (4, [(70, 200), (1, 65), (129, 129)]), (16, [(33, 1200)])])
def test_chunk_over_the_paged_cache(dev, fp8, heads, seqs):
    from mla_latent_kv_26_b200.prefill import MlaPrefill

    cache, bt, q, w, cu_q, cu_k = _chunk(seqs, heads, 20 + heads, fp8)
    pre = MlaPrefill(max_queries=q.shape[0] + 5, max_keys=int(cu_k[-1]) + 70, num_heads=heads, device=dev)
    out = pre(q.to(dev), w.to(dev), cache.to(dev), bt.to(dev), cu_q.to(dev), cu_k.to(dev))
    assert int(pre.error_word.item()) == 0
    _check_chunk(out, pre.lse[:q.shape[0]], cache, bt, q, w, cu_q, cu_k)


def test_chunk_agrees_with_decode(dev):
    """The chunk's last tokens through both branches: expanded attention, and
    absorb -> latent decode -> un-absorb (which rounds the absorbed query, the
    latent output and the result to bf16): relative 2-norm below 1e-2, the
    bound the decode chain is held to."""
    from mla_latent_kv_26_b200.decoder import MlaDecoder, absorb_query, unabsorb_output
    from mla_latent_kv_26_b200.prefill import MlaPrefill

    H, seqs = 16, [(2, 300), (2, 77)]
    cache, bt, q, w, cu_q, cu_k = _chunk(seqs, H, 31, False)
    g = [t.to(dev) for t in (cache, bt, q, w, cu_q, cu_k)]
    out = MlaPrefill(max_queries=4, max_keys=377, num_heads=H, device=dev)(g[2], g[3], g[0], g[1], g[4], g[5])
    dec = MlaDecoder(batch=2, q_len=2, num_heads=H, num_pages=cache.shape[0], max_pages_per_seq=bt.shape[1],
                     causal=True, device=dev)
    lens = torch.tensor([300, 77], dtype=torch.int32, device=dev)
    o_lat, _ = dec(absorb_query(g[2], g[3]).view(2, 2, H, 576), g[0], g[1], lens)
    got = unabsorb_output(o_lat.view(4, H, 512), g[3])
    assert float((got.double() - out.double()).norm() / out.double().norm()) <= 1e-2


def test_chunk_inserted_then_read(dev):
    """New tokens inserted into an fp8 cache, then the chunk's attention over it."""
    from mla_latent_kv_26_b200.decoder import cache_insert
    from mla_latent_kv_26_b200.prefill import MlaPrefill
    from mla_latent_kv_26_b200.workloads import insert_inputs

    H, lens, new = 2, [150, 40], [90, 40]
    d = insert_inputs(lens=lens, new_tokens=new, seed=3)
    g = {k: (v.to(dev) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    cache = torch.zeros(d["num_pages"], 64, 656, dtype=torch.uint8, device=dev)
    ids = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(lens)]).to(dev)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).to(dev)
    gen = torch.Generator().manual_seed(4)
    kv = torch.randn(sum(lens), 576, generator=gen).to(torch.bfloat16).to(dev)
    cache_insert(kv, g["weight"], g["cos"], g["sin"], ids, pos, g["block_table"], cache)
    q = torch.randn(sum(new), H, 192, generator=gen).to(torch.bfloat16)
    w = (torch.randn(H, 256, 512, generator=gen) * 0.05).to(torch.bfloat16)
    cu_q, cu_k = _offsets(new), _offsets(lens)
    pre = MlaPrefill(max_queries=sum(new), max_keys=sum(lens), num_heads=H, device=dev)
    out = pre(q.to(dev), w.to(dev), cache, g["block_table"], cu_q.to(dev), cu_k.to(dev))
    _check_chunk(out, pre.lse, cache.cpu(), d["block_table"], q, w, cu_q, cu_k)


def test_captured_chunk_replays_with_other_lengths(dev):
    """One graph of the three calls (and a second graph of its own), replayed
    after the offsets, block table and queries changed in place; results equal
    the eager calls' bit for bit."""
    from mla_latent_kv_26_b200.prefill import MlaPrefill

    H, cap_q, cap_k = 4, 300, 900
    first = _chunk([(100, 260), (50, 51)], H, 41, True)
    second = _chunk([(1, 500), (180, 300)], H, 42, True)
    pages = max(first[0].shape[0], second[0].shape[0])
    width = max(first[1].shape[1], second[1].shape[1])
    cache = torch.zeros(pages, 64, 656, dtype=torch.uint8, device=dev)
    bt = torch.zeros(2, width, dtype=torch.int32, device=dev)
    q = torch.zeros(cap_q, H, 192, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(H, 256, 512, dtype=torch.bfloat16, device=dev)
    cu_q, cu_k = (torch.zeros(3, dtype=torch.int32, device=dev) for _ in range(2))

    def put(case):
        cache[:case[0].shape[0]] = case[0].to(dev)
        bt[:, :case[1].shape[1]] = case[1].to(dev)
        q[:case[2].shape[0]] = case[2].to(dev)
        w.copy_(case[3].to(dev))
        cu_q.copy_(case[4].to(dev))
        cu_k.copy_(case[5].to(dev))

    a, b = (MlaPrefill(max_queries=cap_q, max_keys=cap_k, num_heads=H, device=dev) for _ in range(2))
    eager = MlaPrefill(max_queries=cap_q, max_keys=cap_k, num_heads=H, device=dev)
    put(first)
    for pre in (a, b):
        pre(q, w, cache, bt, cu_q, cu_k)
    torch.cuda.synchronize(dev)
    graphs = []
    for pre in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pre(q, w, cache, bt, cu_q, cu_k)
        graphs.append(graph)
    for case in (second, first, second):
        put(case)
        n = case[2].shape[0]
        for graph in graphs:
            graph.replay()
        want = eager(q, w, cache, bt, cu_q, cu_k)[:n].clone()
        for pre in (a, b):
            assert torch.equal(pre.out[:n], want) and torch.equal(pre.lse[:n], eager.lse[:n])
        _check_chunk(want, eager.lse[:n], *case)


def test_two_streams_at_once(dev):
    """Two calls with their own buffers on two streams give what each gives alone."""
    from mla_latent_kv_26_b200.prefill import MlaPrefill

    cases = [_chunk([(300, 700)], 16, 51, False), _chunk([(40, 900), (200, 400)], 16, 52, True)]
    dev_cases = [[t.to(dev) for t in c] for c in cases]
    pres = [MlaPrefill(max_queries=300, max_keys=1300, num_heads=16, device=dev) for _ in cases]
    want = [p(c[2], c[3], c[0], c[1], c[4], c[5]).clone() for p, c in zip(pres, dev_cases)]
    streams = [torch.cuda.Stream(dev) for _ in cases]
    torch.cuda.synchronize(dev)
    for p in pres:
        p.out.zero_()
    torch.cuda.synchronize(dev)
    for _ in range(3):
        for p, c, s in zip(pres, dev_cases, streams):
            p(c[2], c[3], c[0], c[1], c[4], c[5], stream=s)
    torch.cuda.synchronize(dev)
    for p, x in zip(pres, want):
        assert torch.equal(p.out[:x.shape[0]], x)


def test_more_tokens_than_capacity_is_clipped_and_reported(dev, libmla):
    """Offsets beyond MlaPrefill's buffers touch nothing outside them; the error word says so."""
    from mla_latent_kv_26_b200.prefill import MlaPrefill

    cache, bt, q, w, cu_q, cu_k = _chunk([(40, 200), (30, 90)], 2, 61, False)
    g = [t.to(dev) for t in (q, w, cache, bt, cu_q, cu_k)]
    pre = MlaPrefill(max_queries=70, max_keys=150, num_heads=2, device=dev)
    pre(*g)
    assert int(pre.error_word.item()) == libmla.MLA_DEVERR_SEQ_LEN
    with pytest.raises(ValueError):
        MlaPrefill(max_queries=69, max_keys=290, num_heads=2, device=dev)(*g)
    # within its capacity the same object is fine afterwards
    pre.error_word.zero_()
    cache, bt, q, w, cu_q, cu_k = _chunk([(40, 100), (30, 50)], 2, 62, False)
    out = pre(q.to(dev), w.to(dev), cache.to(dev), bt.to(dev), cu_q.to(dev), cu_k.to(dev))
    assert int(pre.error_word.item()) == 0
    _check_chunk(out, pre.lse[:70], cache, bt, q, w, cu_q, cu_k)


# ---------------------------------------------------------------- far rows


def test_rows_beyond_four_gigabytes(dev):
    """Cache pages, rows, keys / values and queries whose byte offsets pass 2^32."""
    from mla_latent_kv_26_b200.prefill import cache_read, expand_kv, prefill_attention

    g = torch.Generator().manual_seed(71)
    pages = 60000                                        # 4.4 GB of cache
    cache = torch.empty(pages, 64, 576, dtype=torch.bfloat16, device=dev)
    last = torch.randn(2, 64, 576, generator=g).to(torch.bfloat16)
    cache[-2:] = last.to(dev)
    bt = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=dev)
    rows = cache_read(cache, bt, torch.tensor([0, 128], dtype=torch.int32, device=dev), num_rows=128)
    assert torch.equal(rows.cpu(), torch.cat([last[1], last[0]]))
    del cache

    H, M = 128, 66000                                    # 4.3 GB of keys and values, 3.2 GB of queries
    x = torch.zeros(M, 576, dtype=torch.bfloat16, device=dev)
    x[-128:] = rows
    w = (torch.randn(H, 256, 512, generator=g) * 0.05).to(torch.bfloat16)
    kv = expand_kv(x, w.to(dev))
    tail = kv[-128:].double().cpu()
    ref = oracle.prefill.expand_kv(rows.cpu(), w)
    mag = oracle.prefill.expand_kv(rows.cpu().abs(), w.abs())
    assert ((tail - ref).abs() <= ref.abs() * 2.0 ** -8 + mag * 2.0 ** -14).all()
    assert torch.all(kv[:M - 128] == 0)

    nq = 90000                                           # 4.4 GB of queries
    q = torch.zeros(nq, H, 192, dtype=torch.bfloat16, device=dev)
    some = torch.randn(70, H, 192, generator=g).to(torch.bfloat16)
    q[-70:] = some.to(dev)
    cu_q = torch.tensor([nq - 70, nq], dtype=torch.int32, device=dev)
    cu_k = torch.tensor([M - 128, M], dtype=torch.int32, device=dev)
    out, lse = prefill_attention(q, kv, x[:, 512:], cu_q, cu_k)
    _check_attention(out[-70:, :4], lse[-70:, :4], some[:, :4], kv[-128:, :4].cpu(), x[-128:, 512:].cpu(),
                     torch.tensor([0, 70]), torch.tensor([0, 128]), True, oracle.DEFAULT_SOFTMAX_SCALE)


@pytest.mark.parametrize("heads,seqs,causal", [(128, [(300, 2300), (513, 1100)], True), (40, [(1030, 1030)], True),
                                               (24, [(257, 3000)], False)])
def test_attention_sampled_heads_of_larger_calls(dev, heads, seqs, causal):
    """Calls large enough for runs of many items and groups of heads; a few heads against the oracle."""
    from mla_latent_kv_26_b200.prefill import prefill_attention

    q, kv, pe, cu_q, cu_k = _attention_inputs(heads, seqs, 81)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = prefill_attention(q.to(dev), kv.to(dev), pe.to(dev), cu_q.to(dev), cu_k.to(dev), causal=causal,
                                 error_word=err)
    assert int(err.item()) == 0
    pick = sorted({0, heads // 2 + 1, heads - 1})
    _check_attention(out[:, pick], lse[:, pick], q[:, pick], kv[:, pick], pe, cu_q, cu_k, causal,
                     oracle.DEFAULT_SOFTMAX_SCALE)


def test_calls_on_a_stream_of_their_own(dev):
    """Buffers allocated by the call itself, on the stream it was given."""
    from mla_latent_kv_26_b200.prefill import cache_read, expand_kv, prefill_attention

    cache, bt, q, w, cu_q, cu_k = _chunk([(100, 300)], 4, 91, True)
    s = torch.cuda.Stream(dev)
    with torch.cuda.stream(s):
        c, b, qg, wg, cq, ck = (t.to(dev) for t in (cache, bt, q, w, cu_q, cu_k))
        rows = cache_read(c, b, ck, num_rows=300)
        kv = expand_kv(rows, wg)
        out, lse = prefill_attention(qg, kv, rows[:, 512:], cq, ck)
    s.synchronize()
    _check_chunk(out, lse, cache, bt, q, w, cu_q, cu_k)


def test_stream_argument_as_object_and_as_handle(dev):
    from mla_latent_kv_26_b200.prefill import cache_read, expand_kv, merge_parts, prefill_attention

    cache, bt, q, w, cu_q, cu_k = _chunk([(60, 150)], 2, 92, False)
    g = [t.to(dev) for t in (cache, bt, q, w, cu_q, cu_k)]
    s = torch.cuda.Stream(dev)
    torch.cuda.synchronize(dev)
    for stream in (s, s.cuda_stream):
        rows = cache_read(g[0], g[1], g[5], num_rows=150, stream=stream)
        kv = expand_kv(rows, g[3], stream=stream)
        out, lse = prefill_attention(g[2], kv, rows[:, 512:], g[4], g[5], stream=stream)
        s.synchronize()
        _check_chunk(out, lse, cache, bt, q, w, cu_q, cu_k)
        merged, mlse = merge_parts(out[None].contiguous(), lse[None].contiguous(), stream=stream)
        s.synchronize()
        assert torch.equal(merged, out) and torch.allclose(mlse, lse, atol=1e-6)


# Keys and values of 64 MiB, from four blocks of queries on: such a sequence's
# blocks go to the workers in rounds, two heads at a time, the rest in runs.
ROUNDS = [
    (33, [(1153, 4100), (0, 50), (700, 700), (2305, 4300)], True, 0),
    (17, [(1025, 7800), (300, 9000), (1300, 7711)], False, 9),
    (16, [(1024, 8192)], True, 2),          # one worker: nothing is left over
    (16, [(900, 8192), (40, 60)], True, 6),
    (128, [(1537, 1100), (1, 1)], True, 0),  # more queries than keys
]


@pytest.mark.parametrize("heads,seqs,causal,num_sms", ROUNDS)
def test_attention_in_rounds(dev, heads, seqs, causal, num_sms):
    """Every head of calls whose blocks share keys; heads repeat three heads' inputs."""
    from mla_latent_kv_26_b200.prefill import prefill_attention

    q, kv, pe, cu_q, cu_k = _attention_inputs(3, seqs, 101)
    pick = [h % 3 for h in range(heads)]
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = torch.full((q.shape[0], heads, 128), math.nan, dtype=torch.bfloat16, device=dev)
    lse = torch.full((q.shape[0], heads), math.nan, device=dev)
    prefill_attention(q.to(dev)[:, pick], kv.to(dev)[:, pick], pe.to(dev), cu_q.to(dev), cu_k.to(dev), causal=causal,
                      num_sms=num_sms, out=out, lse=lse, error_word=err)
    assert int(err.item()) == 0
    out, lse = out.cpu(), lse.cpu()
    for first in range(0, heads, 3):
        heads3 = list(range(first, min(first + 3, heads)))
        some = [h % 3 for h in heads3]
        _check_attention(out[:, heads3], lse[:, heads3], q[:, some], kv[:, some], pe, cu_q, cu_k, causal,
                         oracle.DEFAULT_SOFTMAX_SCALE, where=f"heads {heads3}")


def test_default_stream_by_its_handle(dev):
    """Handle 0 is the default stream, whatever the current one is."""
    from mla_latent_kv_26_b200.prefill import cache_read, expand_kv, prefill_attention

    cache, bt, q, w, cu_q, cu_k = _chunk([(60, 150)], 2, 93, False)
    g = [t.to(dev) for t in (cache, bt, q, w, cu_q, cu_k)]
    torch.cuda.synchronize(dev)
    with torch.cuda.stream(torch.cuda.Stream(dev)):
        rows = cache_read(g[0], g[1], g[5], num_rows=150, stream=0)
        kv = expand_kv(rows, g[3], stream=0)
        out, lse = prefill_attention(g[2], kv, rows[:, 512:], g[4], g[5], stream=0)
    torch.cuda.default_stream(dev).synchronize()
    _check_chunk(out, lse, cache, bt, q, w, cu_q, cu_k)


def test_rounds_between_many_short_sequences(dev):
    """Sequences with rounds at both ends of a list longer than a warp scans at once."""
    from mla_latent_kv_26_b200.prefill import prefill_attention

    seqs = [(1030, 8200)] + [(i % 4, 3 * i) for i in range(60)] + [(0, 0), (1300, 8192), (7, 9)]
    q, kv, pe, cu_q, cu_k = _attention_inputs(2, seqs, 102)
    pick = [h % 2 for h in range(16)]
    for num_sms in (0, 14):
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        out, lse = prefill_attention(q.to(dev)[:, pick], kv.to(dev)[:, pick], pe.to(dev), cu_q.to(dev), cu_k.to(dev),
                                     num_sms=num_sms, error_word=err)
        assert int(err.item()) == 0
        for h in range(0, 16, 2):
            _check_attention(out[:, h:h + 2], lse[:, h:h + 2], q, kv, pe, cu_q, cu_k, True,
                             oracle.DEFAULT_SOFTMAX_SCALE, where=f"heads {h}, {h + 1}, num_sms {num_sms}")
