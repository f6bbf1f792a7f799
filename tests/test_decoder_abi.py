"""The C ABI of the decoder operators without a GPU: exports, struct layouts,
and refusals that come before any device work."""
import ctypes
import os
import re

import pytest

import epilogue_tcgen05_tmem_gb300 as eg
from epilogue_tcgen05_tmem_gb300 import _build, decoder

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "eg_decoder.h")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return eg.lib()


def _source():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_exports_every_declared_function(L):
    names = set(re.findall(r"EG_API\s+[\w\s\*]+?\b(eg_\w+)\s*\(", _source()))
    assert names == set(decoder.EXPORTED)
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
    assert [f for f, _ in getattr(decoder, name)._fields_] == fields


def _rope(**kw):
    a = decoder.eg_rope_args(tokens=4, q_heads=2, kv_heads=1, head_dim=64, rot_dim=64, dtype=0, pairs=0, eps=1e-6, page_size=16,
                             cos_sin=16, max_positions=8, q=16, k=16, v=16, q_out=16, k_out=16)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), eg.EG_ERR_INVALID_ARG), (dict(q_heads=-2), eg.EG_ERR_INVALID_ARG), (dict(dtype=3), eg.EG_ERR_INVALID_ARG),
    (dict(head_dim=63), eg.EG_ERR_UNSUPPORTED), (dict(head_dim=258), eg.EG_ERR_UNSUPPORTED), (dict(rot_dim=66), eg.EG_ERR_INVALID_ARG),
    (dict(rot_dim=3), eg.EG_ERR_INVALID_ARG), (dict(pairs=2), eg.EG_ERR_INVALID_ARG), (dict(cos_sin=None), eg.EG_ERR_INVALID_ARG),
    (dict(max_positions=0), eg.EG_ERR_INVALID_ARG), (dict(q=None), eg.EG_ERR_INVALID_ARG), (dict(k=17), eg.EG_ERR_INVALID_ARG),
    (dict(q_token=-1), eg.EG_ERR_INVALID_ARG), (dict(positions=4), eg.EG_ERR_INVALID_ARG),
    (dict(q_weight=16, eps=float("nan")), eg.EG_ERR_INVALID_ARG), (dict(tokens=1 << 25), eg.EG_ERR_UNSUPPORTED)])
def test_rope_refusals_before_device(L, kw, status):
    a = _rope(**kw)
    assert L.eg_qk_norm_rope(ctypes.addressof(a), None) == status
    assert eg.last_error_detail()
    g = decoder.eg_rope_grads(dq=16, dk=16)
    if "q" not in kw and "k" not in kw and "q_token" not in kw:  # inputs that an unweighted gradient does not read
        assert L.eg_qk_norm_rope_backward(ctypes.addressof(a), ctypes.addressof(g), None) == status


def test_append_refusals_before_device(L):
    c = decoder.eg_kv_cache(k=16, v=16, num_pages=1, page_stride=1024, token_stride=64, head_stride=64)
    a = _rope()
    for args, cache, slots in ((None, c, 16), (a, None, 16), (a, c, None), (a, c, 12), (_rope(page_size=0), c, 16), (_rope(v=None), c, 16),
                               (a, decoder.eg_kv_cache(num_pages=1), 16), (a, decoder.eg_kv_cache(k=16, v=16, num_pages=-1), 16)):
        s = L.eg_kv_append(ctypes.addressof(args) if args else None, ctypes.addressof(cache) if cache else None, slots, None)
        assert s == eg.EG_ERR_INVALID_ARG and eg.last_error_detail()


def test_null_arguments(L):
    assert L.eg_qk_norm_rope(None, None) == eg.EG_ERR_INVALID_ARG
    assert L.eg_qk_norm_rope_backward(None, None, None) == eg.EG_ERR_INVALID_ARG
    assert L.eg_qk_norm_rope_workspace_bytes(None, None) == eg.EG_ERR_INVALID_ARG
    assert L.eg_qk_norm_rope_workspace_bytes(ctypes.addressof(_rope()), None) == eg.EG_ERR_INVALID_ARG


def _score(**kw):
    a = decoder.eg_score_args(rows=2, vocab=64, dtype=0, top=2, logits=16, row_stride=64, tokens=16, logprob=16, lse=16, entropy=16,
                              top_ids=16, top_logprobs=16)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), eg.EG_ERR_INVALID_ARG), (dict(vocab=-1), eg.EG_ERR_INVALID_ARG), (dict(vocab=0), eg.EG_ERR_INVALID_ARG),
    (dict(dtype=7), eg.EG_ERR_INVALID_ARG), (dict(logits=None), eg.EG_ERR_INVALID_ARG), (dict(logits=15), eg.EG_ERR_INVALID_ARG),
    (dict(row_stride=63), eg.EG_ERR_INVALID_ARG), (dict(tokens=4), eg.EG_ERR_INVALID_ARG), (dict(rows=1 << 25), eg.EG_ERR_UNSUPPORTED)])
def test_score_refusals_before_device(L, kw, status):
    a = _score(**kw)
    g = decoder.eg_score_grads(lse=16, d_logits=16, d_row_stride=64)
    assert L.eg_token_logprobs(ctypes.addressof(a), None) == status
    assert L.eg_token_logprobs_backward(ctypes.addressof(a), ctypes.addressof(g), None) == status
    assert eg.last_error_detail()


def test_score_refusals_of_one_direction(L):
    for kw, status in ((dict(top=-1), eg.EG_ERR_UNSUPPORTED), (dict(top=33), eg.EG_ERR_UNSUPPORTED), (dict(top=30, vocab=8), eg.EG_ERR_INVALID_ARG),
                       (dict(lse=2), eg.EG_ERR_INVALID_ARG), (dict(top_ids=4), eg.EG_ERR_INVALID_ARG)):
        assert L.eg_token_logprobs(ctypes.addressof(_score(**kw)), None) == status
    for kw in (dict(lse=None), dict(d_entropy=16), dict(d_logits=None), dict(d_row_stride=63), dict(d_logprob=2)):
        g = decoder.eg_score_grads(lse=16, d_logits=16, d_row_stride=64)
        for n, v in kw.items():
            setattr(g, n, v)
        assert L.eg_token_logprobs_backward(ctypes.addressof(_score()), ctypes.addressof(g), None) == eg.EG_ERR_INVALID_ARG
    assert L.eg_token_logprobs(None, None) == eg.EG_ERR_INVALID_ARG
    assert L.eg_token_logprobs_backward(ctypes.addressof(_score()), None, None) == eg.EG_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(q_heads=0), eg.EG_ERR_INVALID_ARG), (dict(q_heads=5), eg.EG_ERR_INVALID_ARG), (dict(head_dim=0), eg.EG_ERR_UNSUPPORTED),
    (dict(head_dim=132), eg.EG_ERR_UNSUPPORTED), (dict(dtype=2), eg.EG_ERR_UNSUPPORTED), (dict(dtype=-1), eg.EG_ERR_INVALID_ARG),
    (dict(page_size=20), eg.EG_ERR_UNSUPPORTED), (dict(max_batch=0), eg.EG_ERR_UNSUPPORTED), (dict(max_tree=300), eg.EG_ERR_UNSUPPORTED)])
def test_tree_refusals_before_device(L, kw, status):
    p = decoder.eg_tree_problem(q_heads=4, kv_heads=2, head_dim=64, dtype=0, page_size=16, max_batch=1, max_tree=1)
    for n, v in kw.items():
        setattr(p, n, v)
    h = ctypes.c_void_p()
    assert L.eg_tree_plan_create(ctypes.addressof(p), ctypes.byref(h)) == status and not h.value
    assert eg.last_error_detail()


def test_tree_null_arguments(L):
    h = ctypes.c_void_p()
    assert L.eg_tree_plan_create(None, ctypes.byref(h)) == eg.EG_ERR_INVALID_ARG
    assert L.eg_tree_plan_create(None, None) == eg.EG_ERR_INVALID_ARG
    assert L.eg_tree_plan_run(None, None, None, None) == eg.EG_ERR_INVALID_ARG
    assert L.eg_tree_plan_workspace_bytes(None, None) == eg.EG_ERR_INVALID_ARG
    assert L.eg_tree_plan_device_status(None) == eg.EG_ERR_INVALID_ARG
    assert L.eg_tree_plan_set_test_stall(None, 0, 0) == eg.EG_ERR_INVALID_ARG
    assert L.eg_tree_plan_destroy(None) == eg.EG_OK


def test_score_hook_refusals(L):
    for bad in (-1, 2):
        assert L.eg_token_logprobs_set_test_stall(0, bad) == eg.EG_ERR_INVALID_ARG
    assert L.eg_token_logprobs_set_test_stall(0, 0) == eg.EG_OK
