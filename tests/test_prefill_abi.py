"""CPU-side checks of the prefill part of the C ABI (include/mla_prefill.h):
every declared function is exported, and bad arguments are rejected before a
GPU is touched. The Python wrappers refuse tensors they cannot pass on."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_header_library_and_binding_agree(libmla):
    text = open(os.path.join(ROOT, "include", "mla_prefill.h")).read()
    declared = set(re.findall(r"MLA_API\s+[\w\s\*]+?\b(mlap_\w+)\s*\(", text))
    assert declared == set(libmla.EXPORTED_PREFILL)
    out = subprocess.run(["nm", "-D", "--defined-only", libmla.LIB_PATH], capture_output=True, text=True).stdout
    assert set(re.findall(r" T (mlap_\w+)", out)) == declared
    lib = ctypes.CDLL(libmla.LIB_PATH)
    assert all(hasattr(lib, n) for n in declared)


# ---------------------------------------------------------------- read-back


def _read(libmla, **kw):
    return libmla.make_read_desc(**dict(dict(batch=2, max_pages_per_seq=4, num_pages=8, num_rows=100), **kw))


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(max_pages_per_seq=0), 1), (dict(num_pages=0), 1), (dict(num_rows=-1), 1),
    (dict(d_latent=256), 2), (dict(d_rope=32), 2), (dict(page_size=16), 2), (dict(num_pages=(1 << 25) + 1), 2),
    (dict(max_pages_per_seq=(1 << 25) + 1), 2), (dict(num_rows=(1 << 31) - 1), 2),
])
def test_read_bad_descriptors_rejected(libmla, kw, status):
    for fn in (libmla.mlap_cache_read, libmla.mlap_cache_read_fp8):
        assert fn(_read(libmla, **kw), 16, 16, 16, 16, 16, None, None) == status


def test_read_null_misaligned_and_empty(libmla):
    INV = libmla.MLA_ERR_INVALID_ARG
    for fn in (libmla.mlap_cache_read, libmla.mlap_cache_read_fp8):
        for i in (0, 1, 2, 4):                       # starts may be NULL
            a = [16] * 5
            a[i] = None
            assert fn(_read(libmla), *a, None, None) == INV, i
        for i, off in ((0, 8), (1, 2), (2, 2), (3, 2), (4, 8)):
            a = [16] * 5
            a[i] += off
            assert fn(_read(libmla), *a, None, None) == INV, i
        assert fn(_read(libmla), 16, 16, 16, 16, 16, 18, None) == INV
        for kw in (dict(batch=0), dict(num_rows=0)):
            assert fn(_read(libmla, **kw), None, None, None, None, None, None, None) == libmla.MLA_OK


# ---------------------------------------------------------------- expansion


def _expand(libmla, **kw):
    return libmla.make_expand_desc(**dict(dict(num_rows=100, num_heads=8), **kw))


@pytest.mark.parametrize("kw,status", [
    (dict(num_rows=-1), 1), (dict(num_heads=0), 1), (dict(row_stride=504), 1), (dict(num_heads=129), 2),
    (dict(row_stride=577), 2), (dict(d_nope=64), 2), (dict(d_v=64), 2), (dict(d_latent=256), 2),
    (dict(num_rows=(1 << 31) - 1), 2),
])
def test_expand_bad_descriptors_rejected(libmla, kw, status):
    assert libmla.mlap_expand_kv(_expand(libmla, **kw), 16, 16, 16, 16, None, None) == status


def test_expand_null_misaligned_and_empty(libmla):
    INV = libmla.MLA_ERR_INVALID_ARG
    for i in (0, 1, 3):                              # row_count may be NULL
        a = [16] * 4
        a[i] = None
        assert libmla.mlap_expand_kv(_expand(libmla), *a, None, None) == INV, i
    for i, off in ((0, 8), (1, 8), (2, 2), (3, 8)):
        a = [16] * 4
        a[i] += off
        assert libmla.mlap_expand_kv(_expand(libmla), *a, None, None) == INV, i
    assert libmla.mlap_expand_kv(_expand(libmla), 16, 16, 16, 16, 18, None) == INV
    assert libmla.mlap_expand_kv(_expand(libmla, num_rows=0), None, None, None, None, None, None) == libmla.MLA_OK


# ---------------------------------------------------------------- attention


def _attn(libmla, **kw):
    return libmla.make_attention_desc(**dict(dict(batch=2, num_heads=8, num_q=10, num_k=20), **kw))


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(num_heads=0), 1), (dict(num_q=-1), 1), (dict(num_k=-1), 1), (dict(num_sms=-1), 1),
    (dict(softmax_scale=0.0), 1), (dict(softmax_scale=-1.0), 1), (dict(softmax_scale=float("nan")), 1),
    (dict(softmax_scale=float("inf")), 1), (dict(pe_stride=56), 1), (dict(pe_stride=68), 2), (dict(num_heads=129), 2),
    (dict(d_nope=64), 2), (dict(d_rope=32), 2), (dict(d_v=64), 2), (dict(num_q=(1 << 31) - 1), 2),
    (dict(num_k=(1 << 31) - 1), 2),
])
def test_attention_bad_descriptors_rejected(libmla, kw, status):
    d = _attn(libmla, **kw)
    assert libmla.mlap_attention_workspace_bytes(d) == 0
    assert libmla.mlap_attention(d, *([32] * 8), 1 << 40, None, None) == status


def test_attention_null_misaligned_and_empty(libmla):
    INV = libmla.MLA_ERR_INVALID_ARG
    for i in range(8):
        a = [32] * 8
        a[i] = None
        assert libmla.mlap_attention(_attn(libmla), *a, 1 << 40, None, None) == INV, i
    for i, off in enumerate((8, 8, 8, 2, 2, 16, 2, 16)):
        a = [32] * 8
        a[i] += off
        assert libmla.mlap_attention(_attn(libmla), *a, 1 << 40, None, None) == INV, i
    assert libmla.mlap_attention(_attn(libmla), *([32] * 8), 1 << 40, 18, None) == INV
    for kw in (dict(batch=0), dict(num_q=0)):
        assert libmla.mlap_attention(_attn(libmla, **kw), *([None] * 8), 0, None, None) == libmla.MLA_OK


def test_attention_causal_flag_outside_0_1_rejected(libmla):
    d = _attn(libmla)
    d.causal = 2
    assert libmla.mlap_attention(d, *([32] * 8), 1 << 40, None, None) == libmla.MLA_ERR_INVALID_ARG


def test_merge_takes_both_widths(libmla):
    mk = libmla.make_merge_desc
    for width in (128, 512):
        assert libmla.mla_merge(mk(parts=2, rows=0, d_latent=width), None, None, None, None, None) == libmla.MLA_OK
    assert libmla.mla_merge(mk(parts=2, rows=4, d_latent=64), 16, 16, 16, 16, None) == libmla.MLA_ERR_UNSUPPORTED


# ---------------------------------------------------------------- Python wrappers


def test_wrappers_refuse_host_tensors(libmla):
    from mla_latent_kv_26_b200 import prefill

    i32 = torch.zeros(2, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        prefill.cache_read(bf(1, 64, 576), i32[None], i32, num_rows=4)
    with pytest.raises(ValueError):
        prefill.expand_kv(bf(4, 576), bf(1, 256, 512))
    with pytest.raises(ValueError):
        prefill.prefill_attention(bf(4, 1, 192), bf(4, 1, 256), bf(4, 64), i32, i32)
    with pytest.raises(ValueError):
        prefill.merge_parts(bf(2, 4, 128), torch.zeros(2, 4))


def _on(name, shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=name)


@pytest.mark.gpu
def test_wrappers_refuse_wrong_shapes_types_and_strides(libmla):
    from mla_latent_kv_26_b200 import prefill

    d, i32 = "cuda", torch.int32
    ok = dict(q=_on(d, (4, 2, 192)), kv=_on(d, (6, 2, 256)), k_pe=_on(d, (6, 64)),
              cu_q=torch.tensor([0, 4], dtype=i32, device=d), cu_k=torch.tensor([0, 6], dtype=i32, device=d))
    for kw in (dict(q=_on(d, (4, 2, 128))), dict(q=_on(d, (4, 2, 192), torch.float16)), dict(kv=_on(d, (6, 3, 256))),
               dict(k_pe=_on(d, (5, 64))), dict(k_pe=_on(d, (6, 65))), dict(k_pe=_on(d, (6, 68))[:, :64]),
               dict(k_pe=_on(d, (64, 6)).t()), dict(k_pe=_on(d, (6, 576))[:, 4:68]),
               dict(cu_q=torch.tensor([0, 4], device=d)), dict(cu_k=torch.tensor([0, 3, 6], dtype=i32, device=d)),
               dict(cu_q=torch.zeros(0, dtype=i32, device=d), cu_k=torch.zeros(0, dtype=i32, device=d)),
               dict(out=_on(d, (4, 2, 192))), dict(lse=_on(d, (4, 2))), dict(workspace=_on(d, (64,))),
               dict(error_word=torch.zeros(1, device=d))):
        with pytest.raises(ValueError):
            prefill.prefill_attention(**dict(ok, **kw))
    with pytest.raises(libmla.MlaError) as e:
        prefill.prefill_attention(**ok, workspace=torch.empty(64, dtype=torch.uint8, device=d))
    assert e.value.status == libmla.MLA_ERR_WORKSPACE_TOO_SMALL
    w = _on(d, (2, 256, 512))
    for rows, kw in ((_on(d, (4, 500)), {}), (_on(d, (4, 580)), {}), (_on(d, (4, 1152))[:, ::2], {}),
                     (_on(d, (4, 576)), dict(out=_on(d, (4, 3, 256)))),
                     (_on(d, (4, 576)), dict(row_count=torch.zeros(1, device=d)))):
        with pytest.raises(ValueError):
            prefill.expand_kv(rows, w, **kw)
    table, off = torch.zeros(1, 1, dtype=i32, device=d), torch.tensor([0, 4], dtype=i32, device=d)
    for cache, kw in ((_on(d, (2, 64, 575)), {}), (_on(d, (2, 64, 576), torch.uint8), {}), (_on(d, (0, 64, 576)), {}),
                      (_on(d, (2, 64, 576)), dict(out=_on(d, (4, 512)))),
                      (_on(d, (2, 64, 576)), dict(starts=torch.zeros(2, dtype=i32, device=d)))):
        with pytest.raises(ValueError):
            prefill.cache_read(cache, table, off, **dict(dict(num_rows=4), **kw))
    with pytest.raises(ValueError):
        prefill.cache_read(_on(d, (2, 64, 576)), table, off)


@pytest.mark.gpu
def test_cache_read_refuses_an_out_that_is_no_tensor(libmla):
    from mla_latent_kv_26_b200 import prefill

    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        prefill.cache_read(_on("cuda", (2, 64, 576)), off[None].contiguous(), off, out=[0.0] * 4)
