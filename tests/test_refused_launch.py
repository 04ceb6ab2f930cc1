"""Calls after a launch that the runtime refused: its error belongs to the call
that made it."""

import ctypes

import pytest
import torch

from test_parity_prefill import dev  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


class _RefusingStream:
    """A stream whose capture was ended by a call that is not allowed in one: the
    runtime refuses every launch on it, and nothing reaches the GPU."""

    def __enter__(self):
        self.rt = ctypes.CDLL("libcudart.so.12")
        self.handle = ctypes.c_void_p()
        assert self.rt.cudaStreamCreateWithFlags(ctypes.byref(self.handle), 1) == 0    # non-blocking
        assert self.rt.cudaStreamBeginCapture(self.handle, 2) == 0                     # relaxed
        assert self.rt.cudaStreamSynchronize(self.handle) != 0
        self.rt.cudaGetLastError()
        return self.handle.value

    def __exit__(self, *exc):
        graph = ctypes.c_void_p()
        self.rt.cudaStreamEndCapture(self.handle, ctypes.byref(graph))
        self.rt.cudaGetLastError()
        assert self.rt.cudaStreamDestroy(self.handle) == 0


def _merge_works(dev, libmla):
    po, pl = torch.ones(2, 4, 128, dtype=torch.bfloat16, device=dev), torch.zeros(2, 4, device=dev)
    out, lse = torch.zeros(4, 128, dtype=torch.bfloat16, device=dev), torch.zeros(4, device=dev)
    st = libmla.mla_merge(libmla.make_merge_desc(parts=2, rows=4, d_latent=128), po, pl, out, lse)
    torch.cuda.synchronize(dev)
    assert st == libmla.MLA_OK and torch.all(out == 1)


@pytest.mark.parametrize("call", ["read", "expand", "attention"])
def test_refused_launch_is_not_reported_again(dev, libmla, call):
    """MLA_ERR_CUDA for the call whose launch was refused, and for no later one."""
    i32 = torch.zeros(2, dtype=torch.int32, device=dev)
    x = torch.zeros(1 << 20, dtype=torch.bfloat16, device=dev)
    ad = libmla.make_attention_desc(batch=1, num_heads=1, num_q=4, num_k=4, pe_stride=64, num_sms=2)
    ws = torch.zeros(libmla.mlap_attention_workspace_bytes(ad), dtype=torch.uint8, device=dev)
    torch.cuda.synchronize(dev)
    _merge_works(dev, libmla)
    with _RefusingStream() as s:
        if call == "read":
            d = libmla.make_read_desc(batch=1, max_pages_per_seq=1, num_pages=1, num_rows=4)
            st = libmla.mlap_cache_read(d, x, i32, i32, None, x, None, s)
        elif call == "expand":
            st = libmla.mlap_expand_kv(libmla.make_expand_desc(num_rows=4, num_heads=1), x, x, None, x, None, s)
        else:
            st = libmla.mlap_attention(ad, x, x, x, i32, i32, x, x, ws, ws.numel(), None, s)
    assert st == libmla.MLA_ERR_CUDA
    _merge_works(dev, libmla)


@pytest.mark.parametrize("call", ["decode", "combine", "get_error", "topk"])
def test_refused_decode_calls_are_not_reported_again(dev, libmla, call):
    from mla_latent_kv_26_b200.decoder import decoder_for
    from mla_latent_kv_26_b200.workloads import small

    d = small(batch=1, heads=2, lens=[70], seed=1)
    dec = decoder_for(d, device=dev)
    q, cache, bt, lens = (d[k].to(dev) for k in ("q", "cache", "block_table", "seq_lens"))
    dec(q, cache, bt, lens)
    x = torch.zeros(64, dtype=torch.int32, device=dev)
    libmla.check(libmla.mla_topk(libmla.make_topk_desc(rows=1, num_keys=8, k=4), x, None, x[32:]), "mla_topk")
    torch.cuda.synchronize(dev)
    _merge_works(dev, libmla)
    with _RefusingStream() as s:
        if call == "topk":
            st = libmla.mla_topk(libmla.make_topk_desc(rows=1, num_keys=8, k=4), x, None, x[32:], s)
        elif call == "get_error":
            st = libmla.mla_get_error(dec.plan, s)[0]
        else:
            with pytest.raises(libmla.MlaError) as e:
                if call == "decode":
                    dec.decode_step(q, cache, bt, lens, stream=s)
                else:
                    dec.combine_step(s)
            st = e.value.status
    assert st == libmla.MLA_ERR_CUDA
    _merge_works(dev, libmla)
    dec(q, cache, bt, lens)
    assert dec.error()[0] == libmla.MLA_OK
