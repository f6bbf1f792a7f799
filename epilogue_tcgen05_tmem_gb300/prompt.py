"""The operators that take in a prompt: thin Python binding of
``include/eg_prompt.h``.

``add_rms_norm`` adds to the residual stream and norms it, with an output in 16
bits or as the codes and scales that an 8-bit linear plan takes;
``add_rms_norm_backward`` is its gradient.  ``ChunkAttention`` is a plan for
attention of chunks of new tokens over a paged cache, all of it or a sliding
window and the first places.  ``lora`` adds the low-rank adapters of many
requests to a shared projection's output.  All take torch CUDA tensors by their
row strides (the last dimension contiguous).  Every call runs on the current
stream unless ``stream`` gives another.  None records autograd, as the linear
plans do not.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

from .decoder import EL_DTYPES, _b, _cache, _code, _fail, _heads, _new, _out, _packer, _rows, _side, _stream_of

EXPORTED = ("eg_add_rms_norm", "eg_add_rms_norm_backward", "eg_add_rms_norm_workspace_bytes",
            "eg_chunk_plan_create", "eg_chunk_plan_workspace_bytes", "eg_chunk_plan_run", "eg_chunk_plan_device_status",
            "eg_chunk_plan_set_test_stall", "eg_chunk_plan_destroy",
            "eg_lora", "eg_lora_workspace_bytes", "eg_lora_device_status", "eg_lora_set_test_stall")

_i64, _i32, _f32, _p, _size = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class eg_norm_args(ctypes.Structure):
    _fields_ = [("rows", _i64), ("width", _i64), ("dtype", _i32), ("quant", _i32), ("eps", _f32), ("x", _p), ("residual", _p),
                ("weight", _p), ("x_row", _i64), ("residual_row", _i64), ("sum", _p), ("out", _p), ("sum_row", _i64),
                ("out_row", _i64), ("codes", _p), ("codes_row", _i64), ("scales", _p)]


class eg_norm_grads(ctypes.Structure):
    _fields_ = [("rows", _i64), ("width", _i64), ("dtype", _i32), ("eps", _f32), ("d_out", _p), ("sum", _p), ("weight", _p),
                ("d_sum", _p), ("d_out_row", _i64), ("sum_row", _i64), ("d_sum_row", _i64), ("dx", _p), ("dx_row", _i64),
                ("d_weight", _p), ("workspace", _p), ("workspace_bytes", _size)]


class eg_chunk_problem(ctypes.Structure):
    _fields_ = [("q_heads", _i32), ("kv_heads", _i32), ("head_dim", _i32), ("dtype", _i32), ("page_size", _i32), ("max_batch", _i32),
                ("max_chunk", _i32)]


class eg_chunk_args(ctypes.Structure):
    _fields_ = [("batch", _i32), ("tokens", _i32), ("q", _p), ("o", _p), ("q_token", _i64), ("q_head", _i64), ("o_token", _i64),
                ("o_head", _i64), ("block_table", _p), ("table_stride", _i64), ("context_lens", _p), ("q_start", _p), ("window", _i32),
                ("sinks", _i32), ("scale", _f32), ("lse", _p)]


class eg_lora_args(ctypes.Structure):
    _fields_ = [("rows", _i32), ("sequences", _i32), ("adapters", _i32), ("inputs", _i32), ("outputs", _i32), ("rank", _i32), ("dtype", _i32),
                ("x", _p), ("x_row", _i64), ("a", _p), ("b", _p), ("scales", _p), ("seq_start", _p), ("adapter", _p), ("base", _p),
                ("base_row", _i64), ("out", _p), ("out_row", _i64), ("workspace", _p), ("workspace_bytes", _size)]


_pack_norm, _pack_norm_grads = _packer(eg_norm_args), _packer(eg_norm_grads)
_pack_chunk, _pack_lora = _packer(eg_chunk_args), _packer(eg_lora_args)
_packers = {"add_rms_norm_workspace_bytes": _pack_norm_grads, "lora_workspace_bytes": _pack_lora}


def declare(L: ctypes.CDLL) -> None:
    """Argument and result types of the entry points."""
    for name, args in (("eg_add_rms_norm", [_p, _p]),
                       ("eg_add_rms_norm_backward", [_p, _p]),
                       ("eg_add_rms_norm_workspace_bytes", [_p, ctypes.POINTER(_size)]),
                       ("eg_chunk_plan_create", [_p, ctypes.POINTER(_p)]),
                       ("eg_chunk_plan_workspace_bytes", [_p, ctypes.POINTER(_size)]),
                       ("eg_chunk_plan_run", [_p, _p, _p, _p]),
                       ("eg_chunk_plan_device_status", [_p]),
                       ("eg_chunk_plan_set_test_stall", [_p, ctypes.c_uint64, _i32]),
                       ("eg_chunk_plan_destroy", [_p]),
                       ("eg_lora", [_p, _p]),
                       ("eg_lora_workspace_bytes", [_p, ctypes.POINTER(_size)]),
                       ("eg_lora_device_status", []),
                       ("eg_lora_set_test_stall", [ctypes.c_uint64, _i32])):
        f = getattr(L, name)
        f.argtypes, f.restype = args, ctypes.c_int


def _matrix(name, t, shape, dtype, device):
    """(pointer, row stride) of a [rows, width] tensor."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or ((s := t.stride())[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on {device} with a contiguous last dimension: got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr(), s[0]


@functools.lru_cache(maxsize=256)
def _bytes(call, device, *fields):
    """What a workspace call says of these sizes on the current device (of that
    number); it says the same every time."""
    need = _size(0)
    status = getattr(_b, call)(_packers[call](*fields), ctypes.byref(need))
    if status:
        _fail(status)
    return need.value


def _result(name, given, shape, dtype, device, stream):
    """(tensor, pointer, row stride) of an output."""
    if given is not None:
        return (given, *_matrix(name, given, shape, dtype, device))
    new = _new(shape, dtype, device, stream)
    return new, new.data_ptr(), shape[1]


# ------------------------------------------------------- norm of the sum ---

QUANT = {None: 0, "e4m3": 1, "int8": 2, "e4m3_block": 3}


class NormResult(NamedTuple):
    """out [rows, width] (None where not wanted), the new residual stream, and
    the codes [rows, width] (uint8 E4M3 codes or int8) with their scales."""
    out: "torch.Tensor | None"      # noqa: F821
    sum: "torch.Tensor"             # noqa: F821
    codes: "torch.Tensor | None"    # noqa: F821
    scales: "torch.Tensor | None"   # noqa: F821  float32 [rows] or [rows, width / 128]


def add_rms_norm(x, weight, residual=None, eps=1e-6, quant=None, keep_out=False, out=None, sum_out=None, stream=None) -> NormResult:
    """x [rows, width] plus ``residual``, and the sum's root-mean-square norm
    times weight [width].  ``quant``: "e4m3", "int8" (a scale for each row) or
    "e4m3_block" (one for each 128 columns) gives the norm as codes and scales
    that a linear plan takes for A and s_a; the norm in x's type comes without
    ``quant``, and with ``keep_out`` or ``out`` beside the codes.  ``sum_out``
    may be x or residual; without a residual the sum is x itself."""
    if not _b.ready:
        _b.load()
    st = _stream_of(x, stream)
    if x.dim() != 2:
        raise ValueError("x must be [rows, width]")
    rows, width = shape = x.shape
    dtype, device = x.dtype, x.device
    code = _code(x)
    try:
        mode = QUANT[quant]
    except KeyError:
        raise ValueError(f"quant must be one of {tuple(QUANT)}: got {quant!r}") from None
    px, x_row = _matrix("x", x, shape, dtype, device)
    w = _side("weight", weight, dtype, (width,), device)
    pr = r_row = ps = s_row = po = o_row = pc = c_row = pz = 0
    total = x
    if residual is not None:
        pr, r_row = _matrix("residual", residual, shape, dtype, device)
        total, ps, s_row = _result("sum_out", sum_out, shape, dtype, device, stream)
    elif sum_out is not None:
        raise ValueError("sum_out without a residual: the sum is x")
    if mode == 0 or keep_out or out is not None:
        out, po, o_row = _result("out", out, shape, dtype, device, stream)
    codes = scales = None
    if mode:
        codes = _new(shape, _b.torch.int8 if mode == 2 else _b.torch.uint8, device, stream)
        scales = _new((rows, width // 128) if mode == 3 else rows, _b.f32, device, stream)
        pc, c_row, pz = codes.data_ptr(), width, scales.data_ptr()
    status = _b.add_rms_norm(_pack_norm(rows, width, code, mode, eps, px, pr, w, x_row, r_row, ps, po, s_row, o_row, pc, c_row, pz), st)
    if status:
        _fail(status)
    return NormResult(out, total, codes, scales)


def add_rms_norm_backward(d_out, sum, weight, eps=1e-6, d_sum=None, dx=None, stream=None):
    """Gradients of ``add_rms_norm`` from that of its norm and, where given, of
    its sum: (dx, d_weight).  dx [rows, width] is the gradient of x and of the
    residual alike (it may be d_out or d_sum), d_weight float32 [width]."""
    if not _b.ready:
        _b.load()
    st = _stream_of(sum, stream)
    if sum.dim() != 2:
        raise ValueError("sum must be [rows, width]")
    rows, width = shape = sum.shape
    dtype, device = sum.dtype, sum.device
    code = _code(sum)
    pz, z_row = _matrix("sum", sum, shape, dtype, device)
    pd, d_row = _matrix("d_out", d_out, shape, dtype, device)
    w = _side("weight", weight, dtype, (width,), device)
    pa = a_row = 0
    if d_sum is not None:
        pa, a_row = _matrix("d_sum", d_sum, shape, dtype, device)
    dx, px, x_row = _result("dx", dx, shape, dtype, device, stream)
    need = _bytes("add_rms_norm_workspace_bytes", _b.current(), rows, width, code, eps, *(0,) * 12)
    work = _new(need // 4, _b.f32, device, stream)
    dw = _new(width, _b.f32, device, stream)
    status = _b.add_rms_norm_backward(_pack_norm_grads(rows, width, code, eps, pd, pz, w, pa, d_row, z_row, a_row, px, x_row, dw.data_ptr(),
                                                       work.data_ptr(), need), st)
    if status:
        _fail(status)
    return dx, dw


# ------------------------------------------------------ chunk attention ---

class ChunkAttention:
    """A plan for causal attention of chunks of new tokens over a paged cache:
    ``max_batch`` sequences of up to ``max_chunk`` new tokens each (1: ordinary
    decoding).  It owns the workspace for sequences split over the GPU; its runs
    must not overlap on the GPU."""

    def __init__(self, q_heads, kv_heads, head_dim, dtype="bf16", page_size=16, max_batch=1, max_chunk=1):
        if not _b.ready:
            _b.load()
        self.handle = None
        self.q_heads, self.kv_heads, self.head_dim, self.page_size = q_heads, kv_heads, head_dim, page_size
        self.max_batch, self.max_chunk = max_batch, max_chunk
        h = _p()
        problem = eg_chunk_problem(q_heads, kv_heads, head_dim, EL_DTYPES[dtype], page_size, max_batch, max_chunk)
        status = _b.chunk_plan_create(ctypes.addressof(problem), ctypes.byref(h))
        if status:
            _fail(status)
        self.handle = h.value
        self._dtype = {"bf16": _b.torch.bfloat16, "f16": _b.torch.float16}[dtype]
        self._place = (page_size, kv_heads, head_dim)

    @property
    def workspace_bytes(self) -> int:
        n = _size()
        status = _b.chunk_plan_workspace_bytes(self.handle, ctypes.byref(n))
        if status:
            _fail(status)
        return n.value

    def run(self, q, k_cache, v_cache, block_table, context_lens, q_start, window=0, sinks=0, scale=None, out=None, lse=None, stream=None):
        """Packed queries q [tokens, q_heads, head_dim] of the sequences' new
        tokens (rows q_start[b] .. q_start[b + 1]) over the cache [pages,
        page_size, kv_heads, head_dim]; block_table int32 [batch, pages of a
        sequence], context_lens int32 [batch] (places before the chunk), q_start
        int32 [batch + 1].  The new tokens' own keys and values are in the cache
        already, after the context.  A token sees the places up to its own: with
        ``window`` only the last ``window`` of them and the first ``sinks``.
        ``scale``: of the scores, 1 / sqrt(head_dim) when None.  Returns o like
        q; lse float32 [tokens, q_heads] is written where given.  Rows that are
        no sequence's (from q_start[batch] on, a sequence's past max_chunk) are
        left as they were in ``out`` and lse, undefined in a new o."""
        st = _stream_of(q, stream)
        tokens = _heads("q", q)[0]
        shape, dtype, device = (tokens, self.q_heads, self.head_dim), self._dtype, q.device
        qp, qt, qh = _rows("q", q, shape, dtype, device)
        if k_cache.dim() != 4:
            raise ValueError("the cache must be [pages, page_size, kv_heads, head_dim]")
        cache = _cache(k_cache, v_cache, self._place, dtype, device)
        batch, width = block_table.shape
        table = _side("block_table", block_table, _b.i32, (batch, width), device)
        out, op, ot, oh = _out("out", out, q, stream)
        args = _pack_chunk(batch, tokens, qp, op, qt, qh, ot, oh, table, width,
                           _side("context_lens", context_lens, _b.i32, (batch,), device),
                           _side("q_start", q_start, _b.i32, (batch + 1,), device), window, sinks,
                           self.head_dim ** -0.5 if scale is None else scale,
                           0 if lse is None else _side("lse", lse, _b.f32, (tokens, self.q_heads), device))
        status = _b.chunk_plan_run(self.handle, args, cache, st)
        if status:
            _fail(status)
        return out

    def device_status(self) -> int:
        return _b.chunk_plan_device_status(self.handle)

    def set_test_stall(self, wait_limit_ns: int, stall_producer: int):
        status = _b.chunk_plan_set_test_stall(self.handle, wait_limit_ns, int(stall_producer))
        if status:
            _fail(status)

    def close(self):
        if getattr(self, "handle", None):
            _b.chunk_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --------------------------------------------------- low-rank adapters ----

def lora(x, a, b, seq_start, adapter, scales=None, base=None, out=None, stream=None):
    """Low-rank adapters of many requests beside a shared projection: for the
    rows seq_start[i] .. seq_start[i + 1] of x [rows, inputs], with the adapter
    n = adapter[i] (int32; none where it is outside the bank),

        out = base + scales[n] * (x @ a[n].T) @ b[n].T

    a [adapters, rank, inputs] and b [adapters, outputs, rank] are the bank
    (adapters of a lower rank padded with zeros), scales float32 [adapters]
    (None: 1), base [rows, outputs] the projection's output (None: 0; give it as
    ``out`` too to add in place).  Without a base the result is what a linear
    plan takes as its residual before the activation.  Rows that no sequence has
    are left as they were in ``out``, undefined in a new one."""
    if not _b.ready:
        _b.load()
    st = _stream_of(x, stream)
    if x.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x must be [rows, inputs], a [adapters, rank, inputs] and b [adapters, outputs, rank]")
    rows, inputs = x.shape
    adapters, rank = a.shape[:2]
    outputs = b.shape[1]
    dtype, device = x.dtype, x.device
    px, x_row = _matrix("x", x, x.shape, dtype, device)
    pa, pb = _side("a", a, dtype, (adapters, rank, inputs), device), _side("b", b, dtype, (adapters, outputs, rank), device)
    sequences = adapter.shape[0]
    start = _side("seq_start", seq_start, _b.i32, (sequences + 1,), device)
    which = _side("adapter", adapter, _b.i32, (sequences,), device)
    ps = _side("scales", scales, _b.f32, (adapters,), device)
    pbase = base_row = 0
    if base is not None:
        pbase, base_row = _matrix("base", base, (rows, outputs), dtype, device)
    out, po, out_row = _result("out", out, (rows, outputs), dtype, device, stream)
    code = _code(x)
    need = _bytes("lora_workspace_bytes", _b.current(), rows, sequences, adapters, inputs, outputs, rank, code, *(0,) * 13)
    work = _new(need, _b.torch.uint8, device, stream)
    status = _b.lora(_pack_lora(rows, sequences, adapters, inputs, outputs, rank, code, px, x_row, pa, pb, ps, start, which, pbase, base_row, po, out_row,
                                work.data_ptr(), need), st)
    if status:
        _fail(status)
    return out


def lora_device_status() -> int:
    """Synchronises the current device: EG_ERR_DEVICE_TIMEOUT, once, when a wait of ``lora`` on it ran past its limit (EG_WAIT_CAP_MS) since
    the last call; what the calls since then wrote is not to be used."""
    if not _b.ready:
        _b.load()
    return _b.lora_device_status()


def lora_set_test_stall(wait_limit_ns: int, stall_loader: int):
    """Testing hook for failure detection (see include/eg_prompt.h)."""
    if not _b.ready:
        _b.load()
    status = _b.lora_set_test_stall(wait_limit_ns, int(stall_loader))
    if status:
        _fail(status)
