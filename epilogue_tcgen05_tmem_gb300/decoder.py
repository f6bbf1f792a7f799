"""The operators between a decoder's linear layers: thin Python binding of
``include/eg_decoder.h``.

``qk_norm_rope`` / ``qk_norm_rope_backward`` norm queries and keys per head and
rotate them by their positions; ``kv_append`` does the same on the way into a
paged key/value cache.  All take torch CUDA tensors [tokens, heads, head_dim]
by their strides (the last dimension contiguous), so parts of one projection's
output are passed as they are.  ``TreeAttention`` is a plan for attention of
drafted token trees (or single tokens) over that cache.  ``token_logprobs`` and its gradient take logits
[rows, vocab].  Every call runs on the current stream unless ``stream`` gives
another.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

EL_DTYPES = {"bf16": 0, "f16": 1, "f32": 2}

EXPORTED = ("eg_qk_norm_rope", "eg_qk_norm_rope_backward", "eg_qk_norm_rope_workspace_bytes",
            "eg_kv_append", "eg_tree_plan_create", "eg_tree_plan_workspace_bytes",
            "eg_tree_plan_run", "eg_tree_plan_device_status", "eg_tree_plan_set_test_stall",
            "eg_tree_plan_destroy",
            "eg_token_logprobs", "eg_token_logprobs_backward")

_i64, _i32, _f32, _p = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p


class eg_rope_args(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("q_heads", _i32), ("kv_heads", _i32), ("head_dim", _i32),
                ("rot_dim", _i32), ("dtype", _i32), ("pairs", _i32), ("eps", _f32),
                ("page_size", _i32), ("cos_sin", _p), ("max_positions", _i64), ("positions", _p),
                ("q_weight", _p), ("k_weight", _p), ("q", _p), ("k", _p), ("v", _p),
                ("q_token", _i64), ("q_head", _i64), ("k_token", _i64), ("k_head", _i64),
                ("v_token", _i64), ("v_head", _i64), ("q_out", _p), ("k_out", _p),
                ("qo_token", _i64), ("qo_head", _i64), ("ko_token", _i64), ("ko_head", _i64)]


class eg_rope_grads(ctypes.Structure):
    _fields_ = [("dq", _p), ("dk", _p), ("dq_token", _i64), ("dq_head", _i64), ("dk_token", _i64),
                ("dk_head", _i64), ("dq_weight", _p), ("dk_weight", _p), ("workspace", _p),
                ("workspace_bytes", ctypes.c_size_t)]


class eg_kv_cache(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("num_pages", _i64), ("page_stride", _i64),
                ("token_stride", _i64), ("head_stride", _i64)]


class eg_tree_problem(ctypes.Structure):
    _fields_ = [("q_heads", _i32), ("kv_heads", _i32), ("head_dim", _i32), ("dtype", _i32),
                ("page_size", _i32), ("max_batch", _i32), ("max_tree", _i32)]


class eg_tree_args(ctypes.Structure):
    _fields_ = [("batch", _i32), ("tokens", _i32), ("q", _p), ("o", _p), ("q_token", _i64),
                ("q_head", _i64), ("o_token", _i64), ("o_head", _i64), ("block_table", _p),
                ("table_stride", _i64), ("context_lens", _p), ("q_start", _p), ("mask", _p),
                ("mask_stride", _i64), ("scale", _f32), ("lse", _p)]


class eg_score_args(ctypes.Structure):
    _fields_ = [("rows", _i64), ("vocab", _i64), ("dtype", _i32), ("top", _i32), ("logits", _p),
                ("row_stride", _i64), ("tokens", _p), ("logprob", _p), ("lse", _p),
                ("entropy", _p), ("top_ids", _p), ("top_logprobs", _p)]


class eg_score_grads(ctypes.Structure):
    _fields_ = [("lse", _p), ("entropy", _p), ("d_logprob", _p), ("d_entropy", _p),
                ("d_logits", _p), ("d_row_stride", _i64)]


def _packer(cls):
    """Fills a C struct in one step: the same layout as the ctypes class."""
    code = {_i64: "q", _i32: "i", _f32: "f", _p: "Q", ctypes.c_size_t: "Q"}
    s = struct.Struct("@" + "".join(code[t] for _, t in cls._fields_) + "0q")
    assert s.size == ctypes.sizeof(cls)
    return s.pack


_pack_rope, _pack_grads, _pack_cache = _packer(eg_rope_args), _packer(eg_rope_grads), _packer(eg_kv_cache)
_pack_tree = _packer(eg_tree_args)
_pack_score, _pack_score_grads = _packer(eg_score_args), _packer(eg_score_grads)


def declare(L: ctypes.CDLL) -> None:
    """Argument and result types of the entry points."""
    for name, args in (("eg_qk_norm_rope", [_p, _p]),
                       ("eg_qk_norm_rope_backward", [_p, _p, _p]),
                       ("eg_qk_norm_rope_workspace_bytes", [_p, ctypes.POINTER(ctypes.c_size_t)]),
                       ("eg_kv_append", [_p, _p, _p, _p]),
                       ("eg_tree_plan_create", [_p, ctypes.POINTER(_p)]),
                       ("eg_tree_plan_workspace_bytes", [_p, ctypes.POINTER(ctypes.c_size_t)]),
                       ("eg_tree_plan_run", [_p, _p, _p, _p]),
                       ("eg_tree_plan_device_status", [_p]),
                       ("eg_tree_plan_set_test_stall", [_p, ctypes.c_uint64, _i32]),
                       ("eg_tree_plan_destroy", [_p]),
                       ("eg_token_logprobs", [_p, _p]),
                       ("eg_token_logprobs_backward", [_p, _p, _p])):
        f = getattr(L, name)
        f.argtypes, f.restype = args, ctypes.c_int


def _eg():
    import epilogue_tcgen05_tmem_gb300 as eg
    return eg


_CODES = {}


def _code(t) -> int:
    if not _CODES:
        import torch
        _CODES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    try:
        return _CODES[t.dtype]
    except KeyError:
        raise ValueError(f"bf16, fp16 or float32 tensors are taken, not {t.dtype}") from None


def _stream_of(t, stream):
    """The stream to queue on; the tensor's device has to be the current one."""
    import torch
    if not t.is_cuda:
        raise ValueError("CUDA tensors are taken")
    at = t.device.index
    if at != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on cuda:{at}, which is not the current device")
    return torch._C._cuda_getCurrentRawStream(at) if stream is None else stream


def _new(shape, dtype, device, stream):
    """An uninitialised tensor, allocated for the stream that the call is queued on."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(name, t, like=None, heads=None):
    """(pointer, token stride, head stride) of a [tokens, heads, head_dim] tensor."""
    if t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] > 1):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with a contiguous last dimension")
    if like is not None and (t.dtype != like.dtype or t.shape[0] != like.shape[0] or t.shape[2] != like.shape[2]
                             or t.device != like.device or (heads is not None and t.shape[1] != heads)):
        raise ValueError(f"{name} {tuple(t.shape)} {t.dtype} does not match {tuple(like.shape)} {like.dtype}")
    return t.data_ptr(), t.stride(0), t.stride(1)


def _side(name, t, dtype, shape, device):
    """Pointer of a contiguous side input, 0 for None."""
    if t is None:
        return 0
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on {device}: got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _table(cos_sin, q):
    """(pointer, positions, rot_dim) of the table of cosines and sines."""
    import torch
    if cos_sin is None:
        return 0, 0, 0
    if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32 or not cos_sin.is_contiguous() or cos_sin.device != q.device:
        raise ValueError("cos_sin must be a contiguous float32 tensor [positions, rot_dim] on the tensors' device")
    return cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1]


def _rope_fields(q, k, cos_sin, positions, q_weight, k_weight, eps, pairs, page, v=(0, 0, 0), q_heads=None):
    import torch
    t, dim = k.shape[0], k.shape[2]
    hq = q.shape[1] if q is not None else 0
    table, count, rot = _table(cos_sin, k)
    qp, qt, qh = _rows("q", q, k) if q is not None else (0, 0, 0)
    kp, kt, kh = _rows("k", k)
    return (t, hq, k.shape[1], dim, rot, _code(k), int(bool(pairs)), eps, page, table, count,
            _side("positions", positions, torch.int64, (t,), k.device),
            _side("q_weight", q_weight, k.dtype, (dim,), k.device),
            _side("k_weight", k_weight, k.dtype, (dim,), k.device),
            qp, kp, v[0], qt, qh, kt, kh, v[1], v[2])


def qk_norm_rope(q, k, cos_sin, positions=None, q_weight=None, k_weight=None, eps=1e-6, pairs=False,
                 q_out=None, k_out=None, stream=None):
    """Queries [T, Hq, D] and keys [T, Hk, D], each normed per head where its
    weight [D] is given, then rotated by cos_sin [positions, rot_dim] float32
    (cosines, then sines); positions int64 [T] (None: 0, 1, 2, ...).  With
    ``pairs`` neighbouring values are a pair, else values rot_dim / 2 apart.
    Returns (q_out, k_out), new tensors unless given (they may be q and k)."""
    import torch
    eg = _eg()
    st = _stream_of(k, stream)
    fields = _rope_fields(q, k, cos_sin, positions, q_weight, k_weight, eps, pairs, 0)
    q_out = _new(q.shape, q.dtype, q.device, stream) if q_out is None else q_out
    k_out = _new(k.shape, k.dtype, k.device, stream) if k_out is None else k_out
    qo, qot, qoh = _rows("q_out", q_out, q, q.shape[1])
    ko, kot, koh = _rows("k_out", k_out, k, k.shape[1])
    eg._check(eg.lib().eg_qk_norm_rope(_pack_rope(*fields, qo, ko, qot, qoh, kot, koh), st))
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, cos_sin, positions=None, q_weight=None, k_weight=None,
                          eps=1e-6, pairs=False, dq=None, dk=None, stream=None):
    """Gradients of ``qk_norm_rope`` for the given gradients of its outputs:
    (dq, dk, dq_weight, dk_weight), the weights' in float32 (None without a
    weight).  dq / dk may be dq_out / dk_out."""
    import torch
    eg = _eg()
    st = _stream_of(k, stream)
    fields = _rope_fields(q, k, cos_sin, positions, q_weight, k_weight, eps, pairs, 0)
    qo, qot, qoh = _rows("dq_out", dq_out, q, q.shape[1])
    ko, kot, koh = _rows("dk_out", dk_out, k, k.shape[1])
    args = _pack_rope(*fields, qo, ko, qot, qoh, kot, koh)
    dq = _new(q.shape, q.dtype, q.device, stream) if dq is None else dq
    dk = _new(k.shape, k.dtype, k.device, stream) if dk is None else dk
    pq, qt, qh = _rows("dq", dq, q, q.shape[1])
    pk, kt, kh = _rows("dk", dk, k, k.shape[1])
    dqw = dkw = work = None
    need = ctypes.c_size_t(0)
    if q_weight is not None or k_weight is not None:
        eg._check(eg.lib().eg_qk_norm_rope_workspace_bytes(args, ctypes.byref(need)))
        work = _new(need.value, torch.uint8, k.device, stream)
        dqw = _new(q.shape[2], torch.float32, k.device, stream) if q_weight is not None else None
        dkw = _new(k.shape[2], torch.float32, k.device, stream) if k_weight is not None else None
    grads = _pack_grads(pq, pk, qt, qh, kt, kh, dqw.data_ptr() if dqw is not None else 0,
                        dkw.data_ptr() if dkw is not None else 0, work.data_ptr() if work is not None else 0, need.value)
    eg._check(eg.lib().eg_qk_norm_rope_backward(args, grads, st))
    return dq, dk, dqw, dkw


def _cache(k_cache, v_cache, like):
    """Packed eg_kv_cache of [pages, page_size, kv_heads, head_dim] tensors (views
    of heads-first storage too), after checking them against `like`'s last dimensions."""
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        if c.dim() != 4 or c.dtype != like.dtype or c.device != like.device or (c.stride(3) != 1 and c.shape[3] > 1):
            raise ValueError(f"{name} must be {like.dtype} [pages, page_size, kv_heads, head_dim] on {like.device} with a "
                             "contiguous last dimension")
    if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    s = k_cache.stride()
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), k_cache.shape[0], s[0], s[1], s[2])


def kv_append(k, v, k_cache, v_cache, slots, q=None, cos_sin=None, positions=None, q_weight=None,
              k_weight=None, eps=1e-6, pairs=False, q_out=None, stream=None):
    """Append keys (normed and rotated as by ``qk_norm_rope``) and values
    [T, Hk, D] to the paged cache [pages, page_size, Hk, D] at slots int64 [T]
    (page * page_size + place; a slot outside the cache appends nothing).  With
    q the queries are normed and rotated in the same launch; returns q_out."""
    import torch
    eg = _eg()
    st = _stream_of(k, stream)
    cache = _cache(k_cache, v_cache, k)
    if k_cache.shape[2] != k.shape[1] or k_cache.shape[3] != k.shape[2]:
        raise ValueError(f"the cache {tuple(k_cache.shape)} does not hold heads of k {tuple(k.shape)}")
    if slots is None:
        raise ValueError("slots is missing")
    fields = _rope_fields(q, k, cos_sin, positions, q_weight, k_weight, eps, pairs, k_cache.shape[1],
                          _rows("v", v, k, k.shape[1]))
    qo, qot, qoh = 0, 0, 0
    if q is not None:
        q_out = _new(q.shape, q.dtype, q.device, stream) if q_out is None else q_out
        qo, qot, qoh = _rows("q_out", q_out, q, q.shape[1])
    eg._check(eg.lib().eg_kv_append(_pack_rope(*fields, qo, 0, qot, qoh, 0, 0), cache,
                                    _side("slots", slots, torch.int64, (k.shape[0],), k.device), st))
    return q_out if q is not None else None


# ------------------------------------------------------- tree attention ---

class TreeAttention:
    """A plan for attention of drafted token trees over a paged cache:
    ``max_batch`` sequences of up to ``max_tree`` drafted tokens each (1: ordinary
    decoding).  It owns the workspace for sequences split over the GPU; its runs
    must not overlap on the GPU."""

    def __init__(self, q_heads, kv_heads, head_dim, dtype="bf16", page_size=16, max_batch=1, max_tree=1):
        eg = _eg()
        self.handle = None
        self.q_heads, self.kv_heads, self.head_dim, self.page_size = q_heads, kv_heads, head_dim, page_size
        self.max_batch, self.max_tree = max_batch, max_tree
        h = _p()
        problem = eg_tree_problem(q_heads, kv_heads, head_dim, EL_DTYPES[dtype], page_size, max_batch, max_tree)
        eg._check(eg.lib().eg_tree_plan_create(ctypes.addressof(problem), ctypes.byref(h)))
        self.handle, self._dtype = h.value, EL_DTYPES[dtype]

    @property
    def workspace_bytes(self) -> int:
        eg, n = _eg(), ctypes.c_size_t()
        eg._check(eg.lib().eg_tree_plan_workspace_bytes(self.handle, ctypes.byref(n)))
        return n.value

    def run(self, q, k_cache, v_cache, block_table, context_lens, q_start, mask=None, scale=None, out=None, lse=None, stream=None):
        """Packed queries q [tokens, q_heads, head_dim] of the sequences' trees
        (rows q_start[b] .. q_start[b + 1]) over the cache [pages, page_size,
        kv_heads, head_dim]; block_table int32 [batch, pages of a sequence],
        context_lens int32 [batch], q_start int32 [batch + 1]; mask int32 words
        [tokens, words] (None: each token sees the drafted ones up to itself).
        The drafted tokens' own keys and values are in the cache already, after
        the context.  ``scale``: of the scores, 1 / sqrt(head_dim) when None.
        Returns o like q; lse float32 [tokens, q_heads] is written where given."""
        import torch
        eg = _eg()
        st = _stream_of(q, stream)
        qp, qt, qh = _rows("q", q)
        tokens, heads, dim = q.shape
        if heads != self.q_heads or dim != self.head_dim or _code(q) != self._dtype:
            raise ValueError(f"q {tuple(q.shape)} {q.dtype} does not fit the plan")
        cache = _cache(k_cache, v_cache, q)
        if k_cache.shape[1:] != (self.page_size, self.kv_heads, dim):
            raise ValueError(f"the cache {tuple(k_cache.shape)} does not fit the plan")
        batch = context_lens.shape[0]
        if block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.shape[0] != batch or block_table.device != q.device \
                or (block_table.stride(1) != 1 and block_table.shape[1] > 1):
            raise ValueError("block_table must be int32 [batch, pages] with contiguous rows on the tensors' device")
        stride = block_table.shape[1]
        if batch > 1 and block_table.stride(0) != stride:
            raise ValueError("block_table must be contiguous")
        words = at_mask = 0
        if mask is not None:
            if mask.dim() != 2 or mask.dtype != torch.int32 or mask.shape[0] != tokens or not mask.is_contiguous() or mask.device != q.device:
                raise ValueError("mask must be contiguous int32 words [tokens, words] on the tensors' device")
            words, at_mask = mask.shape[1], mask.data_ptr() or 4  # no words: refused for their number, not taken for no mask
        out = _new(q.shape, q.dtype, q.device, stream) if out is None else out
        op, ot, oh = _rows("out", out, q, heads)
        args = _pack_tree(batch, tokens, qp, op, qt, qh, ot, oh, block_table.data_ptr(), stride,
                          _side("context_lens", context_lens, torch.int32, (batch,), q.device),
                          _side("q_start", q_start, torch.int32, (batch + 1,), q.device),
                          at_mask, words, dim ** -0.5 if scale is None else scale,
                          _side("lse", lse, torch.float32, (tokens, heads), q.device))
        eg._check(eg.lib().eg_tree_plan_run(self.handle, args, cache, st))
        return out

    def device_status(self) -> int:
        return _eg().lib().eg_tree_plan_device_status(self.handle)

    def set_test_stall(self, wait_limit_ns: int, stall_producer: int):
        eg = _eg()
        eg._check(eg.lib().eg_tree_plan_set_test_stall(self.handle, wait_limit_ns, int(stall_producer)))

    def close(self):
        if getattr(self, "handle", None):
            _eg().lib().eg_tree_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------- log probabilities ---

class TokenLogProbs(NamedTuple):
    """Per row: the given token's log probability, log sum exp of the logits,
    the entropy; and the top alternatives (ids, log probabilities)."""
    logprob: "torch.Tensor"       # noqa: F821  [rows] float32
    lse: "torch.Tensor"           # noqa: F821  [rows] float32
    entropy: "torch.Tensor"       # noqa: F821  [rows] float32
    top_ids: "torch.Tensor | None"       # noqa: F821  [rows, top] int64
    top_logprobs: "torch.Tensor | None"  # noqa: F821  [rows, top] float32


def _logits(name, x):
    if x.dim() != 2 or (x.stride(1) != 1 and x.shape[1] > 1):
        raise ValueError(f"{name} must be [rows, vocab] with a contiguous last dimension")
    return x.data_ptr(), (x.stride(0) if x.shape[0] > 1 else max(x.stride(0), x.shape[1]))


def token_logprobs(logits, tokens=None, top=0, stream=None) -> TokenLogProbs:
    """Log probabilities of tokens int64 [rows] (an id outside the vocabulary:
    none is given, 0) under logits [rows, vocab], with lse, entropy and the
    ``top`` (0..32) best alternatives, of equal logits the lowest id first."""
    import torch
    eg = _eg()
    st = _stream_of(logits, stream)
    x, stride = _logits("logits", logits)
    rows, vocab = logits.shape
    given = _side("tokens", tokens, torch.int64, (rows,), logits.device)
    logprob, lse, entropy = _new((3, rows), torch.float32, logits.device, stream).unbind(0)
    ids = best = None
    if top:
        ids = _new((rows, top), torch.int64, logits.device, stream)
        best = _new((rows, top), torch.float32, logits.device, stream)
    eg._check(eg.lib().eg_token_logprobs(
        _pack_score(rows, vocab, _code(logits), top, x, stride, given, logprob.data_ptr(), lse.data_ptr(), entropy.data_ptr(),
                    ids.data_ptr() if top else 0, best.data_ptr() if top else 0), st))
    return TokenLogProbs(logprob, lse, entropy, ids, best)


def token_logprobs_backward(logits, tokens, lse, entropy, d_logprob=None, d_entropy=None, out=None, stream=None):
    """The gradient to the logits, from what ``token_logprobs`` gave for them
    and the gradients of its log probabilities and entropies (float32 [rows],
    None: zero).  ``out`` may be the logits themselves."""
    import torch
    eg = _eg()
    st = _stream_of(logits, stream)
    x, stride = _logits("logits", logits)
    rows, vocab = logits.shape
    out = _new((rows, vocab), logits.dtype, logits.device, stream) if out is None else out
    d, d_stride = _logits("out", out)
    if out.shape != logits.shape or out.dtype != logits.dtype or out.device != logits.device:
        raise ValueError(f"out {tuple(out.shape)} {out.dtype} does not match {tuple(logits.shape)} {logits.dtype}")
    side = [_side(n, t, torch.float32, (rows,), logits.device)
            for n, t in (("lse", lse), ("entropy", entropy), ("d_logprob", d_logprob), ("d_entropy", d_entropy))]
    given = _side("tokens", tokens, torch.int64, (rows,), logits.device)
    eg._check(eg.lib().eg_token_logprobs_backward(
        _pack_score(rows, vocab, _code(logits), 0, x, stride, given, 0, 0, 0, 0, 0), _pack_score_grads(*side, d, d_stride), st))
    return out
