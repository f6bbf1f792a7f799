"""The C ABI of the operators that take in a prompt without a GPU: exports,
struct layouts, and refusals that come before any device work."""
import ctypes
import os
import re

import pytest

import epilogue_tcgen05_tmem_gb300 as eg
from epilogue_tcgen05_tmem_gb300 import _build, prompt

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "eg_prompt.h")
BAD, NOT = eg.EG_ERR_INVALID_ARG, eg.EG_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    _build.build()
    return eg.lib()


def _source():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_exports_every_declared_function(L):
    names = set(re.findall(r"EG_API\s+[\w\s\*]+?\b(eg_\w+)\s*\(", _source()))
    assert names == set(prompt.EXPORTED)
    for n in names:
        assert hasattr(L, n), n


def _struct_names():
    return re.findall(r"typedef struct \{[^}]*\}\s*(eg_\w+);", _source())


@pytest.mark.parametrize("name", _struct_names())
def test_binding_structs_match_header(name):
    body = re.search(r"typedef struct \{([^}]*)\}\s*" + name + ";", _source()).group(1)
    fields = []
    for decl in body.split(";"):
        decl = decl.strip()
        if decl:
            decl = re.sub(r"^const\s+", "", decl)
            fields += [f.strip().lstrip("*") for f in decl.split(None, 1)[1].split(",")]
    assert [f for f, _ in getattr(prompt, name)._fields_] == fields


def _set(a, kw):
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def _norm(**kw):
    return _set(prompt.eg_norm_args(rows=4, width=256, dtype=0, quant=1, eps=1e-6, x=16, residual=16, weight=16, x_row=256, residual_row=256,
                                    sum=16, out=16, sum_row=256, out_row=256, codes=16, codes_row=256, scales=16), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(width=-1), BAD), (dict(width=0), NOT), (dict(width=65537), NOT), (dict(rows=1 << 25), NOT), (dict(dtype=3), BAD),
    (dict(dtype=-1), BAD), (dict(quant=4), BAD), (dict(quant=-1), BAD), (dict(quant=3, width=200), NOT), (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(x=None), BAD), (dict(x=17), BAD), (dict(weight=None), BAD), (dict(weight=1), BAD), (dict(x_row=255), BAD),
    (dict(residual_row=3), BAD), (dict(residual=17), BAD), (dict(sum=None), BAD), (dict(sum_row=0), BAD), (dict(out=None, quant=0), BAD), (dict(out=15), BAD),
    (dict(out_row=128), BAD), (dict(codes=None), BAD), (dict(codes_row=255), BAD), (dict(scales=None), BAD), (dict(scales=18), BAD)])
def test_norm_refusals_before_device(L, kw, status):
    assert L.eg_add_rms_norm(ctypes.addressof(_norm(**kw)), None) == status
    assert eg.last_error_detail()


def _norm_grads(**kw):
    return _set(prompt.eg_norm_grads(rows=4, width=256, dtype=0, eps=1e-6, d_out=16, sum=16, weight=16, d_sum=16, d_out_row=256, sum_row=256,
                                     d_sum_row=256, dx=16, dx_row=256, d_weight=16, workspace=16, workspace_bytes=1 << 30), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(width=0), NOT), (dict(dtype=5), BAD), (dict(eps=-1.0), BAD), (dict(d_out=None), BAD), (dict(sum=None), BAD),
    (dict(weight=None), BAD), (dict(d_sum=17), BAD), (dict(d_sum_row=5), BAD), (dict(dx=None), BAD), (dict(dx_row=0), BAD), (dict(d_weight=2), BAD)])
def test_norm_gradient_refusals_before_device(L, kw, status):
    assert L.eg_add_rms_norm_backward(ctypes.addressof(_norm_grads(**kw)), None) == status
    assert eg.last_error_detail()


def test_null_arguments(L):
    assert L.eg_add_rms_norm(None, None) == BAD
    assert L.eg_add_rms_norm_backward(None, None) == BAD
    assert L.eg_add_rms_norm_workspace_bytes(None, None) == BAD
    assert L.eg_add_rms_norm_workspace_bytes(ctypes.addressof(_norm_grads()), None) == BAD


def test_no_rows_is_no_work(L):
    assert L.eg_add_rms_norm(ctypes.addressof(_norm(rows=0, x=None, sum=None, out=None, codes=None, scales=None)), None) == eg.EG_OK


def _chunk_problem(**kw):
    return _set(prompt.eg_chunk_problem(q_heads=4, kv_heads=2, head_dim=64, dtype=0, page_size=16, max_batch=1, max_chunk=1), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(q_heads=0), BAD), (dict(q_heads=5), BAD), (dict(head_dim=0), NOT), (dict(head_dim=132), NOT), (dict(dtype=2), NOT), (dict(dtype=-1), BAD),
    (dict(page_size=20), NOT), (dict(max_batch=0), NOT), (dict(max_batch=65537), NOT), (dict(max_chunk=0), NOT), (dict(max_chunk=2 ** 20 + 1), NOT),
    (dict(q_heads=2048), NOT), (dict(q_heads=34), NOT)])
def test_chunk_refusals_before_device(L, kw, status):
    h = ctypes.c_void_p()
    assert L.eg_chunk_plan_create(ctypes.addressof(_chunk_problem(**kw)), ctypes.byref(h)) == status and not h.value
    assert eg.last_error_detail()


def test_chunk_null_arguments(L):
    h = ctypes.c_void_p()
    assert L.eg_chunk_plan_create(None, ctypes.byref(h)) == BAD
    assert L.eg_chunk_plan_create(None, None) == BAD
    assert L.eg_chunk_plan_run(None, None, None, None) == BAD
    assert L.eg_chunk_plan_workspace_bytes(None, None) == BAD
    assert L.eg_chunk_plan_device_status(None) == BAD
    assert L.eg_chunk_plan_set_test_stall(None, 0, 0) == BAD
    assert L.eg_chunk_plan_destroy(None) == eg.EG_OK


def _lora(**kw):
    return _set(prompt.eg_lora_args(rows=4, sequences=2, adapters=3, inputs=64, outputs=128, rank=16, dtype=0, x=16, x_row=64, a=16, b=16, scales=16,
                                    seq_start=16, adapter=16, base=32, base_row=128, out=16, out_row=128, workspace=16, workspace_bytes=1 << 20), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(sequences=-1), BAD), (dict(adapters=-1), BAD), (dict(rows=(1 << 24) + 1), NOT), (dict(sequences=65537), NOT),
    (dict(inputs=0), NOT), (dict(inputs=68), NOT), (dict(outputs=4), NOT), (dict(inputs=(1 << 20) + 8), NOT), (dict(rank=0), NOT), (dict(rank=12), NOT),
    (dict(rank=136), NOT), (dict(dtype=2), NOT), (dict(dtype=9), BAD), (dict(adapters=1 << 30), NOT), (dict(x=None), BAD), (dict(x=24), BAD),
    (dict(x_row=0), BAD), (dict(x_row=65), BAD), (dict(a=None), BAD), (dict(b=8), BAD), (dict(scales=18), BAD), (dict(seq_start=None), BAD),
    (dict(adapter=None), BAD), (dict(adapter=17), BAD), (dict(base=40), BAD), (dict(base_row=4), BAD), (dict(out=None), BAD), (dict(out_row=120), BAD),
    (dict(base=16, base_row=256), BAD), (dict(workspace=None), BAD), (dict(workspace=24), BAD), (dict(workspace_bytes=100), BAD)])
def test_lora_refusals_before_device(L, kw, status):
    assert L.eg_lora(ctypes.addressof(_lora(**kw)), None) == status
    assert eg.last_error_detail()


def test_lora_without_work_and_hooks(L):
    assert L.eg_lora(None, None) == BAD
    assert L.eg_lora_workspace_bytes(None, None) == BAD
    assert L.eg_lora_workspace_bytes(ctypes.addressof(_lora()), None) == BAD
    n = ctypes.c_size_t()
    assert L.eg_lora_workspace_bytes(ctypes.addressof(_lora(rows=5)), ctypes.byref(n)) == eg.EG_OK and n.value == 5 * 2 * 16 * 2 + 32
    assert L.eg_lora(ctypes.addressof(_lora(rows=0, x=None, out=None)), None) == eg.EG_OK
    assert L.eg_lora(ctypes.addressof(_lora(sequences=0, seq_start=None)), None) == eg.EG_OK
    for bad in (-1, 2):
        assert L.eg_lora_set_test_stall(0, bad) == BAD
    assert L.eg_lora_set_test_stall(0, 0) == eg.EG_OK
