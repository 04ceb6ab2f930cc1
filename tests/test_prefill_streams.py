"""Prefill calls on streams other than the one their buffers were made
on, without a synchronise in between."""

import pytest
import torch

from test_parity_prefill import _check_chunk, _chunk, dev  # noqa: F401  (dev: a fixture)

pytestmark = pytest.mark.gpu

_LONG = 400_000_000  # clock cycles of a delay on a stream: about 0.2 s


def test_new_object_called_on_a_side_stream(dev, libmla):
    """The constructor's fills lie behind work on the stream it ran on; a call on
    another stream neither loses its rows nor its error bits to them."""
    from mla_latent_kv_26_b200.prefill import MlaPrefill

    cache, bt, q, w, cu_q, cu_k = _chunk([(60, 150)], 2, 221, False)
    bt_bad = bt.clone()
    bt_bad[0, 0] = -1                                    # position 0 to 63 have no page
    g = [t.to(dev) for t in (q, w, cache, bt_bad, cu_q, cu_k)]
    bt_g = bt.to(dev)
    s = torch.cuda.Stream(dev)
    for _ in range(2):  # kernels loaded and memory at hand: what follows allocates without waiting
        MlaPrefill(max_queries=60, max_keys=150, num_heads=2, device=dev)(*g)
        torch.cuda.synchronize(dev)
    torch.cuda._sleep(_LONG)
    pre = MlaPrefill(max_queries=60, max_keys=150, num_heads=2, device=dev)
    pre(*g, stream=s)
    torch.cuda.synchronize(dev)
    assert int(pre.error_word.item()) == libmla.MLA_DEVERR_PAGE_ID
    assert torch.all(pre.rows[:64] == 0) and torch.all(pre.rows[64:].float().abs().sum(1) > 0)
    pre.error_word.zero_()
    torch.cuda._sleep(_LONG)
    pre = MlaPrefill(max_queries=60, max_keys=150, num_heads=2, device=dev)
    g[3] = bt_g
    with torch.cuda.stream(s):
        out = pre(*g)
    torch.cuda.synchronize(dev)
    _check_chunk(out, pre.lse, cache, bt, q, w, cu_q, cu_k)


def test_buffers_stay_with_a_stream_given(dev):
    """An object that goes away while its call still waits on the given stream
    leaves its buffers to that call."""
    from mla_latent_kv_26_b200.prefill import MlaPrefill

    cache, bt, q, w, cu_q, cu_k = _chunk([(60, 150)], 2, 222, False)
    g = [t.to(dev) for t in (q, w, cache, bt, cu_q, cu_k)]
    s = torch.cuda.Stream(dev)
    pre = MlaPrefill(max_queries=60, max_keys=5000, num_heads=2, device=dev)
    torch.cuda.synchronize(dev)
    with torch.cuda.stream(s):
        torch.cuda._sleep(_LONG)
    out, lse = pre(*g, stream=s), pre.lse
    kept = [(t.data_ptr(), t.shape, t.dtype) for t in (pre.rows, pre.kv, pre.workspace)]
    del pre
    other = [torch.empty(shape, dtype=dtype, device=dev) for _, shape, dtype in kept]
    assert not s.query(), "the delay was too short for this test"
    assert not {t.data_ptr() for t in other} & {p for p, _, _ in kept}
    torch.cuda.synchronize(dev)
    _check_chunk(out, lse, cache, bt, q, w, cu_q, cu_k)


def test_object_made_inside_a_capture(dev):
    """Its buffers are the graph's; nothing waits, and the replay gives the call's result."""
    from mla_latent_kv_26_b200.prefill import MlaPrefill

    cache, bt, q, w, cu_q, cu_k = _chunk([(60, 150), (3, 90)], 2, 223, True)
    g = [t.to(dev) for t in (q, w, cache, bt, cu_q, cu_k)]
    MlaPrefill(max_queries=63, max_keys=240, num_heads=2, device=dev)(*g)
    torch.cuda.synchronize(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pre = MlaPrefill(max_queries=63, max_keys=240, num_heads=2, device=dev)
        out = pre(*g)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize(dev)
    assert int(pre.error_word.item()) == 0
    _check_chunk(out, pre.lse, cache, bt, q, w, cu_q, cu_k)


def test_streams_as_handles_and_external_objects(dev):
    """Raw handles and external streams are used as they are, the buffers not recorded on them."""
    from mla_latent_kv_26_b200.prefill import MlaPrefill

    cache, bt, q, w, cu_q, cu_k = _chunk([(60, 150)], 2, 224, False)
    g = [t.to(dev) for t in (q, w, cache, bt, cu_q, cu_k)]
    s = torch.cuda.Stream(dev)
    pre = MlaPrefill(max_queries=60, max_keys=150, num_heads=2, device=dev)
    for stream in (s.cuda_stream, torch.cuda.ExternalStream(s.cuda_stream, device=dev), s, s):
        pre.out.zero_()
        torch.cuda.synchronize(dev)
        out = pre(*g, stream=stream)
        s.synchronize()
        _check_chunk(out, pre.lse, cache, bt, q, w, cu_q, cu_k)
