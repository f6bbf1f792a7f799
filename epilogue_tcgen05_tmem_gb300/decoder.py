"""The operators between a decoder's linear layers: thin Python binding of
``include/eg_decoder.h``.

``qk_norm_rope`` / ``qk_norm_rope_backward`` norm queries and keys per head and
rotate them by their positions; ``kv_append`` does the same on the way into a
paged key/value cache.  All take torch CUDA tensors [tokens, heads, head_dim]
by their strides (the last dimension contiguous), so parts of one projection's
output are passed as they are.  ``TreeAttention`` is a plan for attention of
drafted token trees (or single tokens) over that cache.  ``token_logprobs`` and its gradient take logits
[rows, vocab].  Every call runs on the current stream unless ``stream`` gives
another.  None records autograd, as the linear plans do not: gradients come
from the ``_backward`` calls.
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
            "eg_token_logprobs", "eg_token_logprobs_backward", "eg_token_logprobs_device_status",
            "eg_token_logprobs_set_test_stall")

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
                       ("eg_token_logprobs_device_status", []),
                       ("eg_token_logprobs_set_test_stall", [ctypes.c_uint64, _i32]),
                       ("eg_token_logprobs_backward", [_p, _p, _p])):
        f = getattr(L, name)
        f.argtypes, f.restype = args, ctypes.c_int


class _Bound:
    """torch and the library, bound at the first call: these calls are as short
    as the kernels they launch, so nothing is looked up twice."""
    ready = False

    @classmethod
    def load(cls):
        import torch

        import epilogue_tcgen05_tmem_gb300 as eg
        lib = eg.lib()
        cls.eg, cls.torch, cls.empty = eg, torch, torch.empty
        cls.raw_stream, cls.current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        cls.f32, cls.i32, cls.i64 = torch.float32, torch.int32, torch.int64
        cls.code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
        for name in EXPORTED + eg.prompt.EXPORTED:
            setattr(cls, name[3:], staticmethod(getattr(lib, name)))
        cls.ready = True


_b = _Bound


def _fail(status):
    raise _b.eg.EgError(status, _b.eg.last_error_detail())


def _code(t) -> int:
    try:
        return _b.code[t.dtype]
    except KeyError:
        raise ValueError(f"bf16, fp16 or float32 tensors are taken, not {t.dtype}") from None


def _stream_of(t, stream):
    """The stream to queue on; the tensor's device has to be the current one."""
    at = t.get_device()
    if at != _b.current():
        if at < 0:
            raise ValueError("CUDA tensors are taken")
        raise ValueError(f"the tensors are on cuda:{at}, which is not the current device")
    return _b.raw_stream(at) if stream is None else stream


def _new(shape, dtype, device, stream):
    """An uninitialised tensor, allocated for the stream that the call is queued on."""
    if stream is None:
        return _b.empty(shape, dtype=dtype, device=device)
    cuda = _b.torch.cuda
    with cuda.stream(cuda.ExternalStream(stream, device=device)):
        return _b.empty(shape, dtype=dtype, device=device)


def _rows(name, t, shape, dtype, device):
    """(pointer, token stride, head stride) of a [tokens, heads, head_dim] tensor."""
    s = t.stride()
    if t.shape != shape or t.dtype is not dtype or t.device != device or (s[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on {device} with a contiguous last dimension: got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr(), s[0], s[1]


def _side(name, t, dtype, shape, device):
    """Pointer of a contiguous side input, 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on {device}: got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _heads(name, t):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    return t.shape


def _rope_fields(q, k, cos_sin, positions, q_weight, k_weight, eps, pairs, page, v):
    """The fields of eg_rope_args up to the outputs."""
    tokens, heads, dim = shape = _heads("k", k)
    dtype, device = k.dtype, k.device
    kp, kt, kh = _rows("k", k, shape, dtype, device)
    qp = qt = qh = hq = vp = vt = vh = table = count = rot = at = qw = kw = 0
    if q is not None:
        hq = _heads("q", q)[1]
        qp, qt, qh = _rows("q", q, (tokens, hq, dim), dtype, device)
    if v is not None:
        vp, vt, vh = _rows("v", v, shape, dtype, device)
    if cos_sin is not None:
        if cos_sin.dim() != 2 or cos_sin.dtype is not _b.f32 or not cos_sin.is_contiguous() or cos_sin.device != device:
            raise ValueError("cos_sin must be a contiguous float32 tensor [positions, rot_dim] on the tensors' device")
        table = cos_sin.data_ptr()
        count, rot = cos_sin.shape
    if positions is not None:
        at = _side("positions", positions, _b.i64, (tokens,), device)
    if q_weight is not None:
        qw = _side("q_weight", q_weight, dtype, (dim,), device)
    if k_weight is not None:
        kw = _side("k_weight", k_weight, dtype, (dim,), device)
    return (tokens, hq, heads, dim, rot, _code(k), 1 if pairs else 0, eps, page, table, count,
            at, qw, kw, qp, kp, vp, qt, qh, kt, kh, vt, vh)


def _out(name, given, like, stream):
    """(tensor, pointer, token stride, head stride) of an output like `like`."""
    if given is not None:
        return (given, *_rows(name, given, like.shape, like.dtype, like.device))
    shape = like.shape
    new = _new(shape, like.dtype, like.device, stream)
    return new, new.data_ptr(), shape[1] * shape[2], shape[2]


def qk_norm_rope(q, k, cos_sin, positions=None, q_weight=None, k_weight=None, eps=1e-6, pairs=False,
                 q_out=None, k_out=None, stream=None):
    """Queries [T, Hq, D] and keys [T, Hk, D], each normed per head where its
    weight [D] is given, then rotated by cos_sin [positions, rot_dim] float32
    (cosines, then sines); positions int64 [T] (None: 0, 1, 2, ...).  With
    ``pairs`` neighbouring values are a pair, else values rot_dim / 2 apart.
    Returns (q_out, k_out), new tensors unless given (they may be q and k)."""
    if not _b.ready:
        _b.load()
    st = _stream_of(k, stream)
    fields = _rope_fields(q, k, cos_sin, positions, q_weight, k_weight, eps, pairs, 0, None)
    q_out, qo, qot, qoh = _out("q_out", q_out, q, stream)
    k_out, ko, kot, koh = _out("k_out", k_out, k, stream)
    status = _b.qk_norm_rope(_pack_rope(*fields, qo, ko, qot, qoh, kot, koh), st)
    if status:
        _fail(status)
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, cos_sin, positions=None, q_weight=None, k_weight=None,
                          eps=1e-6, pairs=False, dq=None, dk=None, stream=None):
    """Gradients of ``qk_norm_rope`` for the given gradients of its outputs:
    (dq, dk, dq_weight, dk_weight), the weights' in float32 (None without a
    weight).  dq / dk may be dq_out / dk_out."""
    if not _b.ready:
        _b.load()
    st = _stream_of(k, stream)
    fields = _rope_fields(q, k, cos_sin, positions, q_weight, k_weight, eps, pairs, 0, None)
    dtype, device, dim = k.dtype, k.device, k.shape[2]
    qo, qot, qoh = _rows("dq_out", dq_out, q.shape, dtype, device)
    ko, kot, koh = _rows("dk_out", dk_out, k.shape, dtype, device)
    args = _pack_rope(*fields, qo, ko, qot, qoh, kot, koh)
    dq, pq, qt, qh = _out("dq", dq, q, stream)
    dk, pk, kt, kh = _out("dk", dk, k, stream)
    dqw = dkw = work = None
    need = ctypes.c_size_t(0)
    if q_weight is not None or k_weight is not None:
        status = _b.qk_norm_rope_workspace_bytes(args, ctypes.byref(need))
        if status:
            _fail(status)
        work = _new(need.value // 4, _b.f32, device, stream)
        dqw = _new(dim, _b.f32, device, stream) if q_weight is not None else None
        dkw = _new(dim, _b.f32, device, stream) if k_weight is not None else None
    grads = _pack_grads(pq, pk, qt, qh, kt, kh, 0 if dqw is None else dqw.data_ptr(), 0 if dkw is None else dkw.data_ptr(),
                        0 if work is None else work.data_ptr(), need.value)
    status = _b.qk_norm_rope_backward(args, grads, st)
    if status:
        _fail(status)
    return dq, dk, dqw, dkw


def _cache(k_cache, v_cache, shape, dtype, device):
    """Packed eg_kv_cache of [pages, *shape] tensors (views of heads-first
    storage too)."""
    s = k_cache.stride()
    if k_cache.shape[1:] != shape or k_cache.dtype is not dtype or k_cache.device != device or (s[3] != 1 and shape[2] > 1):
        raise ValueError(f"k_cache must be {dtype} [pages, {', '.join(map(str, shape))}] on {device} with a contiguous last "
                         f"dimension: got {k_cache.dtype} {tuple(k_cache.shape)} on {k_cache.device}")
    if v_cache.shape != k_cache.shape or v_cache.stride() != s or v_cache.dtype is not dtype or v_cache.device != device:
        raise ValueError("k_cache and v_cache must have the same type, shape and strides")
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), k_cache.shape[0], s[0], s[1], s[2])


def kv_append(k, v, k_cache, v_cache, slots, q=None, cos_sin=None, positions=None, q_weight=None,
              k_weight=None, eps=1e-6, pairs=False, q_out=None, stream=None):
    """Append keys (normed and rotated as by ``qk_norm_rope``) and values
    [T, Hk, D] to the paged cache [pages, page_size, Hk, D] at slots int64 [T]
    (page * page_size + place; a slot outside the cache appends nothing).  With
    q the queries are normed and rotated in the same launch; returns q_out."""
    if not _b.ready:
        _b.load()
    st = _stream_of(k, stream)
    if slots is None or k_cache.dim() != 4:
        raise ValueError("slots is missing" if slots is None else "the cache must be [pages, page_size, kv_heads, head_dim]")
    page = k_cache.shape[1]
    fields = _rope_fields(q, k, cos_sin, positions, q_weight, k_weight, eps, pairs, page, v)
    dtype, device = k.dtype, k.device
    cache = _cache(k_cache, v_cache, (page, fields[2], fields[3]), dtype, device)
    qo = qot = qoh = 0
    if q is not None:
        q_out, qo, qot, qoh = _out("q_out", q_out, q, stream)
    else:
        q_out = None
    status = _b.kv_append(_pack_rope(*fields, qo, 0, qot, qoh, 0, 0), cache, _side("slots", slots, _b.i64, (fields[0],), device), st)
    if status:
        _fail(status)
    return q_out


# ------------------------------------------------------- tree attention ---

class TreeAttention:
    """A plan for attention of drafted token trees over a paged cache:
    ``max_batch`` sequences of up to ``max_tree`` drafted tokens each (1: ordinary
    decoding).  It owns the workspace for sequences split over the GPU; its runs
    must not overlap on the GPU."""

    def __init__(self, q_heads, kv_heads, head_dim, dtype="bf16", page_size=16, max_batch=1, max_tree=1):
        if not _b.ready:
            _b.load()
        self.handle = None
        self.q_heads, self.kv_heads, self.head_dim, self.page_size = q_heads, kv_heads, head_dim, page_size
        self.max_batch, self.max_tree = max_batch, max_tree
        h = _p()
        problem = eg_tree_problem(q_heads, kv_heads, head_dim, EL_DTYPES[dtype], page_size, max_batch, max_tree)
        status = _b.tree_plan_create(ctypes.addressof(problem), ctypes.byref(h))
        if status:
            _fail(status)
        self.handle = h.value
        self._dtype = {"bf16": _b.torch.bfloat16, "f16": _b.torch.float16}[dtype]
        self._place = (page_size, kv_heads, head_dim)

    @property
    def workspace_bytes(self) -> int:
        n = ctypes.c_size_t()
        status = _b.tree_plan_workspace_bytes(self.handle, ctypes.byref(n))
        if status:
            _fail(status)
        return n.value

    def run(self, q, k_cache, v_cache, block_table, context_lens, q_start, mask=None, scale=None, out=None, lse=None, stream=None):
        """Packed queries q [tokens, q_heads, head_dim] of the sequences' trees
        (rows q_start[b] .. q_start[b + 1]) over the cache [pages, page_size,
        kv_heads, head_dim]; block_table int32 [batch, pages of a sequence],
        context_lens int32 [batch], q_start int32 [batch + 1]; mask int32 words
        [tokens, words] (None: each token sees the drafted ones up to itself).
        The drafted tokens' own keys and values are in the cache already, after
        the context.  ``scale``: of the scores, 1 / sqrt(head_dim) when None.
        Returns o like q; lse float32 [tokens, q_heads] is written where given.
        Rows that are no sequence's (from q_start[batch] on, a sequence's past
        max_tree) are left as they were in ``out`` and lse, undefined in a new o."""
        st = _stream_of(q, stream)
        tokens = _heads("q", q)[0]
        shape, dtype, device = (tokens, self.q_heads, self.head_dim), self._dtype, q.device
        qp, qt, qh = _rows("q", q, shape, dtype, device)
        if k_cache.dim() != 4:
            raise ValueError("the cache must be [pages, page_size, kv_heads, head_dim]")
        cache = _cache(k_cache, v_cache, self._place, dtype, device)
        batch, width = block_table.shape
        table = _side("block_table", block_table, _b.i32, (batch, width), device)
        words = at_mask = 0
        if mask is not None:
            words = mask.shape[1]
            # a mask without words is refused for their number, not taken for none
            at_mask = _side("mask", mask, _b.i32, (tokens, words), device) or 4
        out, op, ot, oh = _out("out", out, q, stream)
        args = _pack_tree(batch, tokens, qp, op, qt, qh, ot, oh, table, width,
                          _side("context_lens", context_lens, _b.i32, (batch,), device),
                          _side("q_start", q_start, _b.i32, (batch + 1,), device), at_mask, words,
                          self.head_dim ** -0.5 if scale is None else scale,
                          0 if lse is None else _side("lse", lse, _b.f32, (tokens, self.q_heads), device))
        status = _b.tree_plan_run(self.handle, args, cache, st)
        if status:
            _fail(status)
        return out

    def device_status(self) -> int:
        return _b.tree_plan_device_status(self.handle)

    def set_test_stall(self, wait_limit_ns: int, stall_producer: int):
        status = _b.tree_plan_set_test_stall(self.handle, wait_limit_ns, int(stall_producer))
        if status:
            _fail(status)

    def close(self):
        if getattr(self, "handle", None):
            _b.tree_plan_destroy(self.handle)
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
    """(pointer, row stride) of [rows, vocab] logits."""
    if x.dim() != 2:
        raise ValueError(f"{name} must be [rows, vocab]")
    stride, one = x.stride()
    rows, vocab = x.shape
    if one != 1 and vocab > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return x.data_ptr(), stride if rows > 1 else max(stride, vocab)


def token_logprobs(logits, tokens=None, top=0, stream=None) -> TokenLogProbs:
    """Log probabilities of tokens int64 [rows] (an id outside the vocabulary:
    none is given, 0) under logits [rows, vocab], with lse, entropy and the
    ``top`` (0..32) best alternatives, of equal logits the lowest id first."""
    if not _b.ready:
        _b.load()
    st = _stream_of(logits, stream)
    x, stride = _logits("logits", logits)
    rows, vocab = logits.shape
    device, f32 = logits.device, _b.f32
    given = 0 if tokens is None else _side("tokens", tokens, _b.i64, (rows,), device)
    logprob, lse, entropy = _new(rows, f32, device, stream), _new(rows, f32, device, stream), _new(rows, f32, device, stream)
    ids = best = None
    at_ids = at_best = 0
    if top:
        ids, best = _new((rows, top), _b.i64, device, stream), _new((rows, top), f32, device, stream)
        at_ids, at_best = ids.data_ptr(), best.data_ptr()
    status = _b.token_logprobs(_pack_score(rows, vocab, _code(logits), top, x, stride, given, logprob.data_ptr(), lse.data_ptr(),
                                           entropy.data_ptr(), at_ids, at_best), st)
    if status:
        _fail(status)
    return TokenLogProbs(logprob, lse, entropy, ids, best)


def token_logprobs_device_status() -> int:
    """Synchronises the current device: EG_ERR_DEVICE_TIMEOUT, once, when a wait of ``token_logprobs`` on it ran past its limit
    (EG_WAIT_CAP_MS) since the last call; the rows concerned are NaN."""
    if not _b.ready:
        _b.load()
    return _b.token_logprobs_device_status()


def token_logprobs_set_test_stall(wait_limit_ns: int, stall_loader: int):
    """Testing hook for failure detection (see include/eg_decoder.h)."""
    if not _b.ready:
        _b.load()
    status = _b.token_logprobs_set_test_stall(wait_limit_ns, int(stall_loader))
    if status:
        _fail(status)


def token_logprobs_backward(logits, tokens, lse, entropy, d_logprob=None, d_entropy=None, out=None, stream=None):
    """The gradient to the logits, from what ``token_logprobs`` gave for them
    and the gradients of its log probabilities and entropies (float32 [rows],
    None: zero).  ``out`` may be the logits themselves."""
    if not _b.ready:
        _b.load()
    st = _stream_of(logits, stream)
    x, stride = _logits("logits", logits)
    rows, vocab = logits.shape
    device, f32 = logits.device, _b.f32
    if out is None:
        out = _new((rows, vocab), logits.dtype, device, stream)
    d, d_stride = _logits("out", out)
    if out.shape != logits.shape or out.dtype is not logits.dtype or out.device != device:
        raise ValueError(f"out {tuple(out.shape)} {out.dtype} does not match {tuple(logits.shape)} {logits.dtype}")
    side = [_side(n, t, f32, (rows,), device)
            for n, t in (("lse", lse), ("entropy", entropy), ("d_logprob", d_logprob), ("d_entropy", d_entropy))]
    given = _side("tokens", tokens, _b.i64, (rows,), device)
    status = _b.token_logprobs_backward(_pack_score(rows, vocab, _code(logits), 0, x, stride, given, 0, 0, 0, 0, 0),
                                        _pack_score_grads(*side, d, d_stride), st)
    if status:
        _fail(status)
    return out
