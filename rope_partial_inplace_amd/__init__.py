"""Python binding of librope_amd.so, the MI355X (gfx950) RoPE apply library.

Argument marshalling only: tensors are described (pointer, dtype, shape, strides) and handed
to the C ABI declared in ``include/rope.h`` together with the current HIP stream; every step
of both operations runs in the library's HIP kernels.  PyTorch provides device memory and
streams.  There is no fallback: if the library is not built this import fails.

  rope_partial_inplace(x, cos, sin, rotary_mode=1, partial_slice=None, stream=None)
  rope_partial_inplace_backward(g, cos, sin, rotary_mode=1, partial_slice=None, stream=None)
  InplacePartialRotaryMul.apply(x, cos, sin, partial_slice, rotary_mode)
                                                  (autograd; x must not be a leaf)
  inplace_partial_rotary_mul(x, r1, r2, *, rotary_mode="interleave", partial_slice=None)
  inplace_partial_rotary_mul_backward(grad, r1, r2, *, rotary_mode="interleave",
                                      partial_slice=None)
                                                  (the pages' Python interface: same calls,
                                                  autograd when x requires grad)
  rope_with_cos_sin_cache(positions, query_in, key_in, cos_sin_cache, mrope_section,
                          head_size, is_neox_style, query_out=None, key_out=None, stream=None)
  rope_with_cos_sin_cache_v2(..., is_neox_style, cache_mode, query_out=None, ...)
  rope_append_paged_cache(positions, slots, key, key_cache, cos_sin_cache, value=None,
                          value_cache=None, query=None, query_out=None, query_rot_start=0,
                          key_rot_start=0, is_neox_style=True, stream=None)
  rope_latent_attention_paged(query, latent_cache, page_table, seq_lens, latent_dim, scale,
                              query_offsets=None, out=None, lse=None, stream=None)
  rope_latent_attention(query, key, key_rope, value, scale, causal=True, num_sequences=None,
                        query_offsets=None, key_offsets=None, out=None, lse=None, stream=None)
  rope_latent_attention_backward(grad, query, key, key_rope, value, out, lse, scale, causal=True,
                                 num_sequences=None, query_offsets=None, key_offsets=None,
                                 stream=None)
  latent_attention(query, key, key_rope, value, scale, ...)      (the same, with autograd)
  rope_append_paged_cache_q8(positions, key, value, key_cache, value_cache, key_scales,
                             value_scales, page_table, seq_lens, cos_sin_cache,
                             query_offsets=None, query=None, query_out=None, query_rot_start=0,
                             key_rot_start=0, is_neox_style=True, stream=None)
  rope_attention_paged_q8(query, key_cache, value_cache, key_scales, value_scales, page_table,
                          seq_lens, scale, query_offsets=None, out=None, lse=None, stream=None)
  rope_copy_pages(sources, targets, caches, stream=None)
  rope_fork_pages(page_table, seq_lens, parents, ref_counts, page_size, caches=(), grow=None,
                  page_table_out=None, seq_lens_out=None, ref_counts_out=None, shortage=None,
                  stream=None)
  rope_compact_pages(page_table, ref_counts, caches=(), page_table_out=None,
                     ref_counts_out=None, page_map=None, live=None, stream=None)
  PageCaches(caches, whole=())        (the caches of all layers, described once for those three)

Pages defining the operations:
  [IPRM] "CANN ops-transformer 的 aclnnInplacePartialRotaryMul 算子：Inplace 部分旋转位置编码接口详解与实现剖析"
  [RSCC] "CANN ops-transformer 旋转位置编码算子 RopeWithSinCosCache 深度解析：cache 化 RoPE 的计算原理与 aclnn 两段式调用实战"
"""
from __future__ import annotations

import ctypes
import os
import struct

from .build import LIB_PATH

ROPE_OK = 0
ROPE_ERR_PARAM_NULLPTR = 161001
ROPE_ERR_PARAM_INVALID = 161002
ROPE_ERR_RUNTIME = 361001

ROPE_F32, ROPE_F16, ROPE_BF16, ROPE_I64, ROPE_I8, ROPE_E4M3 = 0, 1, 2, 3, 4, 5


class RopeTensor(ctypes.Structure):
    """Mirror of ``rope_tensor`` in include/rope.h."""

    _fields_ = [
        ("data", ctypes.c_void_p),
        ("dtype", ctypes.c_int),
        ("ndim", ctypes.c_int32),
        ("shape", ctypes.c_int64 * 4),
        ("stride", ctypes.c_int64 * 4),
    ]


class RopeError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"rope error {code}: {message}")
        self.code = code


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python __graft_entry__.py` at the repository root")
    import torch  # noqa: F401  its HIP runtime first: the library then uses it, not a second one
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    lib.rope_partial_inplace.argtypes = [P(RopeTensor), P(RopeTensor), P(RopeTensor),
                                         ctypes.c_int64, P(ctypes.c_int64), ctypes.c_int64,
                                         ctypes.c_void_p]
    lib.rope_partial_inplace.restype = ctypes.c_int
    lib.rope_partial_inplace_backward.argtypes = lib.rope_partial_inplace.argtypes
    lib.rope_partial_inplace_backward.restype = ctypes.c_int
    lib.rope_with_cos_sin_cache.argtypes = [P(RopeTensor), P(RopeTensor), P(RopeTensor),
                                            P(RopeTensor), P(ctypes.c_int64), ctypes.c_int64,
                                            ctypes.c_int64, ctypes.c_int, P(RopeTensor),
                                            P(RopeTensor), ctypes.c_void_p]
    lib.rope_with_cos_sin_cache.restype = ctypes.c_int
    lib.rope_with_cos_sin_cache_v2.argtypes = [P(RopeTensor), P(RopeTensor), P(RopeTensor),
                                               P(RopeTensor), P(ctypes.c_int64), ctypes.c_int64,
                                               ctypes.c_int64, ctypes.c_int, ctypes.c_int64,
                                               P(RopeTensor), P(RopeTensor), ctypes.c_void_p]
    lib.rope_with_cos_sin_cache_v2.restype = ctypes.c_int
    T = ctypes.c_void_p  # a RopeTensor by reference, or its bytes
    lib.rope_append_paged_cache.argtypes = [T, T, T, T, T, T, ctypes.c_int64, ctypes.c_int64,
                                            ctypes.c_int, T, T, T, ctypes.c_void_p]
    lib.rope_append_paged_cache.restype = ctypes.c_int
    lib.rope_latent_attention_paged_workspace.argtypes = [ctypes.c_int64] * 4
    lib.rope_latent_attention_paged_workspace.restype = ctypes.c_int64
    lib.rope_latent_attention_paged.argtypes = [T, T, T, T, T, ctypes.c_int64, ctypes.c_double,
                                                T, T, ctypes.c_void_p, ctypes.c_int64,
                                                ctypes.c_void_p]
    lib.rope_latent_attention_paged.restype = ctypes.c_int
    where = [T, T, ctypes.c_int64, ctypes.c_double, ctypes.c_int]  # offsets, B, scale, causal
    lib.rope_latent_attention.argtypes = [T, T, T, T, *where, T, T, ctypes.c_void_p]
    lib.rope_latent_attention.restype = ctypes.c_int
    lib.rope_latent_attention_backward_workspace.argtypes = [ctypes.c_int64] * 3
    lib.rope_latent_attention_backward_workspace.restype = ctypes.c_int64
    lib.rope_latent_attention_backward.argtypes = [T] * 7 + where + [T] * 4 + [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]
    lib.rope_latent_attention_backward.restype = ctypes.c_int
    lib.rope_append_paged_cache_q8.argtypes = [T] * 8 + [ctypes.c_int64, ctypes.c_int64,
                                                         ctypes.c_int] + [T] * 5 + [ctypes.c_void_p]
    lib.rope_append_paged_cache_q8.restype = ctypes.c_int
    lib.rope_attention_paged_q8_workspace.argtypes = [ctypes.c_int64] * 5
    lib.rope_attention_paged_q8_workspace.restype = ctypes.c_int64
    lib.rope_attention_paged_q8.argtypes = [T] * 8 + [ctypes.c_double, T, T, ctypes.c_void_p,
                                                      ctypes.c_int64, ctypes.c_void_p]
    lib.rope_attention_paged_q8.restype = ctypes.c_int
    lists = [T, ctypes.c_int64]  # caches, their number
    memory = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]  # workspace, bytes, stream
    lib.rope_copy_pages.argtypes = [T, T, *lists, ctypes.c_void_p]
    lib.rope_copy_pages.restype = ctypes.c_int
    lib.rope_fork_pages_workspace.argtypes = [ctypes.c_int64] * 3
    lib.rope_fork_pages_workspace.restype = ctypes.c_int64
    lib.rope_fork_pages.argtypes = [T] * 5 + [ctypes.c_int64, *lists] + [T] * 4 + memory
    lib.rope_fork_pages.restype = ctypes.c_int
    lib.rope_compact_pages_workspace.argtypes = [ctypes.c_int64]
    lib.rope_compact_pages_workspace.restype = ctypes.c_int64
    lib.rope_compact_pages.argtypes = [T, T, *lists] + [T] * 4 + memory
    lib.rope_compact_pages.restype = ctypes.c_int
    lib.rope_last_error.argtypes = []
    lib.rope_last_error.restype = ctypes.c_char_p
    return lib


LIB = _load()


def last_error() -> str:
    return LIB.rope_last_error().decode()


def _dtype_code(t) -> int:
    import torch
    return {torch.float32: ROPE_F32, torch.float16: ROPE_F16, torch.bfloat16: ROPE_BF16,
            torch.int64: ROPE_I64, torch.int8: ROPE_I8,
            torch.float8_e4m3fn: ROPE_E4M3}.get(t.dtype, 99)


def describe(t) -> RopeTensor:
    """A ``rope_tensor`` describing a torch tensor (which must outlive the call)."""
    if t.dim() > 4:
        raise RopeError(ROPE_ERR_PARAM_INVALID, "tensors of more than 4 dims are not supported")
    return RopeTensor(t.data_ptr() if t.numel() > 0 else None, _dtype_code(t), t.dim(),
                      tuple(t.shape), t.stride())


def _int_array(values):
    if values is None:
        return None, 0
    vals = [int(v) for v in values]
    return (ctypes.c_int64 * max(len(vals), 1))(*vals), len(vals)


def _device_of(tensors):
    dev = None
    for t in tensors:
        if t is None or t.numel() == 0:
            continue
        if not t.is_cuda:
            raise RopeError(ROPE_ERR_PARAM_INVALID,
                            "tensors must live in GPU memory (torch device 'cuda')")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise RopeError(ROPE_ERR_PARAM_INVALID, "tensors are on different devices")
    return dev


def _stream_handle(stream, dev):
    import torch
    if stream is None:
        if dev is None:
            return None
        stream = torch.cuda.current_stream(dev)
    return getattr(stream, "cuda_stream", stream)


def _check(code: int):
    if code != ROPE_OK:
        raise RopeError(code, last_error())


def _on_device(dev, fn, args) -> int:
    """fn(*args) with the tensors' GPU as the current HIP device: the library launches on the
    current device, which must own the stream and the tensors."""
    import torch
    if dev is None or dev.index is None or dev.index == torch.cuda.current_device():
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def rope_partial_inplace(x, cos, sin, rotary_mode: int = 1, partial_slice=None, stream=None):
    """In-place partial RoPE on x[..., start:end) ([IPRM §计算原理与公式]): rotary_mode 1
    interleave, 0 half mode (x1, x2 the two halves of the slice)."""
    dev = _device_of([x, cos, sin])
    dx, dc, ds = describe(x), describe(cos), describe(sin)
    sl, sl_len = _int_array(partial_slice)
    _check(_on_device(dev, LIB.rope_partial_inplace,
                      (ctypes.byref(dx), ctypes.byref(dc), ctypes.byref(ds), int(rotary_mode),
                       sl, sl_len, _stream_handle(stream, dev))))


def rope_partial_inplace_backward(g, cos, sin, rotary_mode: int = 1, partial_slice=None,
                                  stream=None):
    """Gradient of rope_partial_inplace with respect to x, in place on the incoming gradient
    ``g`` ([IPRM §Python 接口与自动微分]; the transpose of the forward pair map)."""
    dev = _device_of([g, cos, sin])
    dg, dc, ds = describe(g), describe(cos), describe(sin)
    sl, sl_len = _int_array(partial_slice)
    _check(_on_device(dev, LIB.rope_partial_inplace_backward,
                      (ctypes.byref(dg), ctypes.byref(dc), ctypes.byref(ds), int(rotary_mode),
                       sl, sl_len, _stream_handle(stream, dev))))


def _autograd_function():
    import torch

    class InplacePartialRotaryMul(torch.autograd.Function):
        """Autograd wrapper ([IPRM §Python 接口与自动微分]): forward rotates x in place and marks
        it dirty; backward runs the backward kernel on a contiguous copy of the incoming
        gradient; cos and sin get no gradient."""

        @staticmethod
        def forward(ctx, x, cos, sin, partial_slice=None, rotary_mode=1):
            rope_partial_inplace(x, cos, sin, rotary_mode, partial_slice)
            ctx.mark_dirty(x)
            ctx.save_for_backward(cos, sin)
            ctx.partial_slice = partial_slice
            ctx.rotary_mode = rotary_mode
            return x

        @staticmethod
        def backward(ctx, grad):
            cos, sin = ctx.saved_tensors
            g = grad.contiguous().clone()
            rope_partial_inplace_backward(g, cos, sin, ctx.rotary_mode, ctx.partial_slice)
            return g, None, None, None, None

    return InplacePartialRotaryMul


def __getattr__(name):  # autograd functions are made on first use
    make = {"InplacePartialRotaryMul": _autograd_function,
            "LatentAttention": _latent_autograd_function}.get(name)
    if make is not None:
        fn = make()
        globals()[name] = fn
        return fn
    raise AttributeError(name)


_ROTARY_MODES = {"interleave": 1, "half": 0}


def _rotary_mode_code(rotary_mode) -> int:
    if isinstance(rotary_mode, str):
        if rotary_mode not in _ROTARY_MODES:
            raise RopeError(ROPE_ERR_PARAM_INVALID,
                            f"rotary_mode {rotary_mode!r}: 'interleave' or 'half' (or 1 / 0)")
        return _ROTARY_MODES[rotary_mode]
    return int(rotary_mode)


def inplace_partial_rotary_mul(x, r1, r2, *, rotary_mode="interleave", partial_slice=None):
    """The Python interface of [IPRM §Python 接口与自动微分]: rotates x in place (r1 = cos,
    r2 = sin) and returns None.  rotary_mode is "interleave" (1) or "half" (0, reading R21).
    When autograd records x (x requires grad and grad mode is on), the call goes through
    InplacePartialRotaryMul, so the gradient of x comes from the backward kernel and r1, r2 get
    none; x must then not be a leaf (rotate a copy such as ``y = x * 1.0``)."""
    import torch
    mode = _rotary_mode_code(rotary_mode)
    if x.requires_grad and torch.is_grad_enabled():
        __getattr__("InplacePartialRotaryMul").apply(x, r1, r2, partial_slice, mode)
    else:
        rope_partial_inplace(x, r1, r2, mode, partial_slice)


def inplace_partial_rotary_mul_backward(grad, r1, r2, *, rotary_mode="interleave",
                                        partial_slice=None):
    """The gradient op named by [IPRM §Python 接口与自动微分], in place on ``grad`` (the
    transpose of each slice pair's rotation; outside the slice the gradient passes through).
    Returns None."""
    rope_partial_inplace_backward(grad, r1, r2, _rotary_mode_code(rotary_mode), partial_slice)


def _cache_args(positions, query_in, key_in, cos_sin_cache, mrope_section, head_size,
                is_neox_style, cache_mode, query_out, key_out, stream):
    """(C function, its arguments, objects to keep alive) of one cos/sin-cache call: the V1
    entry point when cache_mode is None, else the V2 one."""
    tensors = (positions, query_in, key_in, cos_sin_cache, query_out, key_out)
    dev = _device_of(list(tensors))
    descs = [describe(t) for t in tensors]
    ms, ms_len = _int_array(mrope_section)
    head = (ctypes.byref(descs[0]), ctypes.byref(descs[1]), ctypes.byref(descs[2]),
            ctypes.byref(descs[3]), ms, ms_len, int(head_size), int(bool(is_neox_style)))
    tail = (ctypes.byref(descs[4]), ctypes.byref(descs[5]), _stream_handle(stream, dev))
    if cache_mode is None:
        return LIB.rope_with_cos_sin_cache, head + tail, (tensors, descs, ms), dev
    return (LIB.rope_with_cos_sin_cache_v2, head + (int(cache_mode),) + tail,
            (tensors, descs, ms), dev)


def _with_cos_sin_cache(positions, query_in, key_in, cos_sin_cache, mrope_section, head_size,
                        is_neox_style, cache_mode, query_out, key_out, stream):
    import torch
    if head_size is None:
        head_size = cos_sin_cache.shape[-1]
    if query_out is None:
        query_out = torch.empty(query_in.shape, dtype=query_in.dtype, device=query_in.device)
    if key_out is None:
        key_out = torch.empty(key_in.shape, dtype=key_in.dtype, device=key_in.device)
    fn, args, _keep, dev = _cache_args(positions, query_in, key_in, cos_sin_cache,
                                       mrope_section, head_size, is_neox_style, cache_mode,
                                       query_out, key_out, stream)
    _check(_on_device(dev, fn, args))
    return query_out, key_out


def rope_with_cos_sin_cache(positions, query_in, key_in, cos_sin_cache, mrope_section=None,
                            head_size: int | None = None, is_neox_style: bool = True,
                            query_out=None, key_out=None, stream=None):
    """RoPE with a cos/sin cache ([RSCC §设计动机]); returns (query_out, key_out).

    Outputs are allocated (contiguous) when not given; ``head_size`` defaults to the cache's
    rotaryDim."""
    return _with_cos_sin_cache(positions, query_in, key_in, cos_sin_cache, mrope_section,
                               head_size, is_neox_style, None, query_out, key_out, stream)


def rope_with_cos_sin_cache_v2(positions, query_in, key_in, cos_sin_cache, mrope_section=None,
                               head_size: int | None = None, is_neox_style: bool = True,
                               cache_mode: int = 0, query_out=None, key_out=None, stream=None):
    """The V2 form with ``cache_mode`` ([RSCC §V2 接口：cacheMode 扩展]): 0 sectioned,
    1 interleaved mrope stitching.  Other arguments as rope_with_cos_sin_cache."""
    return _with_cos_sin_cache(positions, query_in, key_in, cos_sin_cache, mrope_section,
                               head_size, is_neox_style, int(cache_mode), query_out, key_out,
                               stream)


# ---- paged cache and latent attention ---------------------------------------------------------
# A decoding step's calls take the GPU a few microseconds, so their marshalling is kept short:
# descriptions are packed as bytes, and the device and stream read as numbers.

_PACK = {n: struct.Struct(f"Pii{n}q{8 * (4 - n)}x{n}q{8 * (4 - n)}x").pack for n in range(1, 5)}
_DTYPE_CODES = {}


def _pack(t):
    """The bytes of a ``rope_tensor`` describing a torch tensor (None stays None)."""
    if t is None:
        return None
    shape = t.shape
    n = len(shape)
    pack = _PACK.get(n)
    if pack is None:
        raise RopeError(ROPE_ERR_PARAM_INVALID, "tensors must have 1 to 4 dims")
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        code = _DTYPE_CODES[t.dtype] = _dtype_code(t)
    return pack(t.data_ptr(), code, n, *shape, *t.stride())


def _device_index(tensors) -> int:
    """GPU of the tensors (-1: none of them has elements)."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        d = t.get_device()
        if d != dev:
            if t.numel() == 0:
                continue
            if d < 0:
                raise RopeError(ROPE_ERR_PARAM_INVALID,
                                "tensors must live in GPU memory (torch device 'cuda')")
            if dev is not None:
                raise RopeError(ROPE_ERR_PARAM_INVALID, "tensors are on different devices")
            dev = d
    return -1 if dev is None else dev


def _raw_stream(stream, dev: int):
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else None
    return getattr(stream, "cuda_stream", stream)


def _run_on(dev: int, fn, *args):
    """One C call with GPU `dev` as the current HIP device."""
    import torch
    if dev < 0 or dev == torch._C._cuda_getDevice():
        code = fn(*args)
    else:
        with torch.cuda.device(dev):
            code = fn(*args)
    if code != ROPE_OK:
        raise RopeError(code, last_error())


def _new(stream, dev: int, *specs):
    """New tensors of (shape, dtype, a tensor on their device), None for a spec of None.  Torch
    allocates them for the stream that the call runs on: outputs and workspaces belong to it."""
    import torch
    if stream is None or dev < 0:
        return [s and s[2].new_empty(s[0], dtype=s[1]) for s in specs]
    if not isinstance(stream, torch.cuda.Stream):
        handle = getattr(stream, "cuda_stream", stream)
        stream = (torch.cuda.ExternalStream(handle, device=dev) if handle
                  else torch.cuda.default_stream(dev))
    with torch.cuda.stream(stream):
        return [s and s[2].new_empty(s[0], dtype=s[1]) for s in specs]


def rope_append_paged_cache(positions, slots, key, key_cache, cos_sin_cache, value=None,
                            value_cache=None, query=None, query_out=None,
                            query_rot_start: int = 0, key_rot_start: int = 0,
                            is_neox_style: bool = True, stream=None):
    """Rotate a batch's keys (and queries) by position and append keys and values to a paged
    cache: key [T, Nk, D] and value [T, Nk, Dv] go to row slots[t] % pageSize of page
    slots[t] // pageSize of key_cache [pages, pageSize, Nk, D] and value_cache
    [pages, pageSize, Nk, Dv]; a slot out of range is skipped.  Elements
    [rot_start, rot_start + rotaryDim) of every head are rotated, rotaryDim the width of
    cos_sin_cache [maxSeqLen, rotaryDim].  Returns query_out [T, Nq, Dq] (allocated when not
    given; it may be query itself), or None without a query."""
    dev = _device_index((positions, slots, query, key, value, cos_sin_cache, query_out, key_cache,
                         value_cache))
    if query is not None and query_out is None:
        query_out, = _new(stream, dev, (query.shape, query.dtype, query))
    _run_on(dev, LIB.rope_append_paged_cache, _pack(positions), _pack(slots), _pack(query),
            _pack(key), _pack(value), _pack(cos_sin_cache), query_rot_start, key_rot_start,
            bool(is_neox_style), _pack(query_out), _pack(key_cache), _pack(value_cache),
            _raw_stream(stream, dev))
    return query_out


def rope_latent_attention_paged(query, latent_cache, page_table, seq_lens, latent_dim: int,
                                scale: float, query_offsets=None, out=None, lse=None,
                                stream=None):
    """Latent attention over a paged cache, absorbed form: query [T, heads, latent_dim + 64]
    against latent_cache [pages, pageSize, latent_dim + 64] (or [pages, pageSize, 1, ...], as the
    append fills it), whose rows are keys and, in their first latent_dim elements, values of every
    head.  page_table [B, maxPages], seq_lens [B] (the queries' own tokens included) and
    query_offsets [B + 1] are int64; without offsets every sequence has T / B queries.  Query i of
    n sees the cached rows below seq_len - n + 1 + i.  Returns (out [T, heads, latent_dim],
    lse [T, heads] float32); rows outside all sequences are not written, so pass out and lse where
    they are to be defined."""
    import torch
    dev = _device_index((query, latent_cache, page_table, seq_lens, query_offsets, out, lse))
    if latent_cache.dim() == 4 and latent_cache.shape[2] == 1:
        latent_cache = latent_cache.squeeze(2)
    if query.dim() != 3 or seq_lens.dim() != 1:
        raise RopeError(ROPE_ERR_PARAM_INVALID, "query must be 3-D and seq_lens 1-D")
    T, heads, _ = query.shape
    need = LIB.rope_latent_attention_paged_workspace(T, heads, latent_dim, seq_lens.shape[0])
    new_out, new_lse, workspace = _new(
        stream, dev,
        ((T, heads, max(0, latent_dim)), query.dtype, query) if out is None else None,
        ((T, heads), torch.float32, query) if lse is None else None, (need, torch.uint8, query))
    out, lse = out if new_out is None else new_out, lse if new_lse is None else new_lse
    _run_on(dev, LIB.rope_latent_attention_paged, _pack(query), _pack(latent_cache),
            _pack(page_table), _pack(seq_lens), _pack(query_offsets), latent_dim, scale,
            _pack(out), _pack(lse), workspace.data_ptr(), need, _raw_stream(stream, dev))
    return out, lse


def _sequences(num_sequences, query_offsets):
    """num_sequences of the C call: 1 by default, 0 where the offsets give it."""
    if num_sequences is None:
        return 1 if query_offsets is None else 0
    return int(num_sequences)


def rope_latent_attention(query, key, key_rope, value, scale: float, causal: bool = True,
                          num_sequences: int | None = None, query_offsets=None, key_offsets=None,
                          out=None, lse=None, stream=None):
    """Latent attention, expanded form: query [Tq, heads, dim + 64] against key [Tk, heads, dim]
    and, in the last 64 elements, key_rope [Tk, 64], which all heads share; value [Tk, heads, dim].
    Sequences are packed one behind the other: int64 query_offsets and key_offsets [B + 1], or
    num_sequences (1 by default) of equal length.  Causal: of n queries and m keys query i sees the
    first m - n + 1 + i keys.  Returns (out [Tq, heads, dim], lse [Tq, heads] float32); rows outside
    all sequences are not written, so pass out and lse where they are to be defined.  Not recorded
    by autograd: that is latent_attention."""
    import torch
    dev = _device_index((query, key, key_rope, value, query_offsets, key_offsets, out, lse))
    if query.dim() != 3 or value.dim() != 3:
        raise RopeError(ROPE_ERR_PARAM_INVALID, "query and value must be 3-D")
    T, heads, _ = query.shape
    new_out, new_lse = _new(
        stream, dev,
        ((T, heads, value.shape[2]), query.dtype, query) if out is None else None,
        ((T, heads), torch.float32, query) if lse is None else None)
    out, lse = out if new_out is None else new_out, lse if new_lse is None else new_lse
    _run_on(dev, LIB.rope_latent_attention, _pack(query), _pack(key), _pack(key_rope),
            _pack(value), _pack(query_offsets), _pack(key_offsets),
            _sequences(num_sequences, query_offsets), scale, bool(causal), _pack(out), _pack(lse),
            _raw_stream(stream, dev))
    return out, lse


def rope_latent_attention_backward(grad, query, key, key_rope, value, out, lse, scale: float,
                                   causal: bool = True, num_sequences: int | None = None,
                                   query_offsets=None, key_offsets=None, stream=None):
    """Gradients of rope_latent_attention's out with respect to (query, key, key_rope, value), for
    the gradient ``grad`` of out; out and lse are the forward call's.  Rows outside all sequences get
    zeros."""
    import torch
    dev = _device_index((grad, query, key, key_rope, value, out, lse, query_offsets, key_offsets))
    if query.dim() != 3:
        raise RopeError(ROPE_ERR_PARAM_INVALID, "query must be 3-D")
    need = LIB.rope_latent_attention_backward_workspace(query.shape[0], key.shape[0],
                                                        query.shape[1])
    *grads, workspace = _new(stream, dev,
                             *((t.shape, t.dtype, t) for t in (query, key, key_rope, value)),
                             (need, torch.uint8, query))
    _run_on(dev, LIB.rope_latent_attention_backward, _pack(grad), _pack(query), _pack(key),
            _pack(key_rope), _pack(value), _pack(out), _pack(lse), _pack(query_offsets),
            _pack(key_offsets), _sequences(num_sequences, query_offsets), scale, bool(causal),
            *map(_pack, grads), workspace.data_ptr(), need, _raw_stream(stream, dev))
    return tuple(grads)


def _latent_autograd_function():
    import torch

    class LatentAttention(torch.autograd.Function):
        """Autograd wrapper of the expanded form; rows outside all sequences are zero in the
        output and in the gradients."""

        @staticmethod
        def forward(ctx, query, key, key_rope, value, scale, causal=True, num_sequences=None,
                    query_offsets=None, key_offsets=None):
            out = lse = None
            if query_offsets is not None:
                out = torch.zeros((*query.shape[:2], value.shape[2]), dtype=query.dtype,
                                  device=query.device)
            out, lse = rope_latent_attention(query, key, key_rope, value, scale, causal,
                                             num_sequences, query_offsets, key_offsets, out=out)
            ctx.save_for_backward(query, key, key_rope, value, out, lse, query_offsets,
                                  key_offsets)
            ctx.where = (scale, causal, num_sequences)
            return out

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, grad):
            *saved, q_off, k_off = ctx.saved_tensors
            if not grad.is_contiguous() or grad.data_ptr() % 16:  # expanded, transposed, a slice
                grad = grad.clone(memory_format=torch.contiguous_format)
            grads = rope_latent_attention_backward(grad, *saved, *ctx.where, q_off, k_off)
            return (*grads, None, None, None, None, None)

    return LatentAttention


def latent_attention(query, key, key_rope, value, scale: float, causal: bool = True,
                     num_sequences: int | None = None, query_offsets=None, key_offsets=None):
    """rope_latent_attention with autograd: returns out [Tq, heads, dim]; query, key, key_rope and
    value get gradients from the backward kernels.  Forward and backward may be captured into a graph,
    both in one capture and after a warm-up on a side stream; as for every torch function, no eager
    graph of the same leaves may be alive then."""
    fn = globals().get("LatentAttention") or __getattr__("LatentAttention")
    return fn.apply(query, key, key_rope, value, scale, causal, num_sequences, query_offsets,
                    key_offsets)


# ---- paged cache in 8 bits ----------------------------------------------------------------------

def rope_append_paged_cache_q8(positions, key, value, key_cache, value_cache, key_scales,
                               value_scales, page_table, seq_lens, cos_sin_cache,
                               query_offsets=None, query=None, query_out=None,
                               query_rot_start: int = 0, key_rot_start: int = 0,
                               is_neox_style: bool = True, stream=None):
    """Rotate a batch's keys (and queries) by position and append keys and values to a paged cache of
    8-bit codes: key [T, Nk, D] and value [T, Nk, Dv] go to the last places of their sequences in
    key_cache [pages, pageSize, Nk, D] and value_cache [pages, pageSize, Nk, Dv] (int8 or
    float8_e4m3fn), with float32 scales [pages, blocks, Nk] for each block of pageSize / blocks tokens
    and head.  page_table [B, maxPages], seq_lens [B] (the new tokens included) and query_offsets
    [B + 1] (the packed batch's) are int64; without offsets every sequence has T / B new tokens.
    Where a block's scale has to grow, the codes of the sequence's earlier tokens in it are rounded
    anew.  Rotation as in rope_append_paged_cache.  Returns query_out [T, Nq, Dq] (allocated when not
    given; it may be query itself), or None without a query."""
    dev = _device_index((positions, query, key, value, cos_sin_cache, page_table, seq_lens,
                         query_offsets, query_out, key_cache, value_cache, key_scales,
                         value_scales))
    if query is not None and query_out is None:
        query_out, = _new(stream, dev, (query.shape, query.dtype, query))
    _run_on(dev, LIB.rope_append_paged_cache_q8, _pack(positions), _pack(query), _pack(key),
            _pack(value), _pack(cos_sin_cache), _pack(page_table), _pack(seq_lens),
            _pack(query_offsets), query_rot_start, key_rot_start, bool(is_neox_style),
            _pack(query_out), _pack(key_cache), _pack(value_cache), _pack(key_scales),
            _pack(value_scales), _raw_stream(stream, dev))
    return query_out


def rope_attention_paged_q8(query, key_cache, value_cache, key_scales, value_scales, page_table,
                            seq_lens, scale: float, query_offsets=None, out=None, lse=None,
                            stream=None):
    """Grouped-query attention over a paged cache of 8-bit codes: query [T, heads, D] (float16 or
    bfloat16, D 64, 128 or 256) against key_cache and value_cache [pages, pageSize, Nk, D] (int8 or
    float8_e4m3fn) with float32 scales [pages, blocks, Nk]; query head h reads key head
    h // (heads // Nk).  page_table [B, maxPages], seq_lens [B] (the queries' own tokens included) and
    query_offsets [B + 1] are int64; without offsets every sequence has T / B queries.  Query i of n
    sees the cached tokens below seq_len - n + 1 + i.  Returns (out [T, heads, D], lse [T, heads]
    float32); rows outside all sequences are not written, so pass out and lse where they are to be
    defined.  Tiles are sized by the mean number of queries: sequences that decode and long pieces of
    prompts are faster in two calls than in one.  Not recorded by autograd."""
    import torch
    dev = _device_index((query, key_cache, value_cache, key_scales, value_scales, page_table,
                         seq_lens, query_offsets, out, lse))
    if query.dim() != 3 or key_cache.dim() != 4 or seq_lens.dim() != 1:
        raise RopeError(ROPE_ERR_PARAM_INVALID,
                        "query must be 3-D, key_cache 4-D and seq_lens 1-D")
    T, heads, width = query.shape
    need = LIB.rope_attention_paged_q8_workspace(T, heads, key_cache.shape[2], width,
                                                 seq_lens.shape[0])
    new_out, new_lse, workspace = _new(
        stream, dev, ((T, heads, width), query.dtype, query) if out is None else None,
        ((T, heads), torch.float32, query) if lse is None else None, (need, torch.uint8, query))
    out, lse = out if new_out is None else new_out, lse if new_lse is None else new_lse
    _run_on(dev, LIB.rope_attention_paged_q8, _pack(query), _pack(key_cache), _pack(value_cache),
            _pack(key_scales), _pack(value_scales), _pack(page_table), _pack(seq_lens),
            _pack(query_offsets), scale, _pack(out), _pack(lse), workspace.data_ptr(), need,
            _raw_stream(stream, dev))
    return out, lse


# ---- pages of a cache ------------------------------------------------------------------------------

def _as_pages(t):
    """A cache as [pages, elements of a page], whose pages are dense blocks in any order of dimensions."""
    if t.dim() < 2 or t.numel() == 0:
        return t
    reach = 1
    for stride, size in sorted((t.stride(d), t.shape[d]) for d in range(1, t.dim()) if t.shape[d] > 1):
        if stride != reach:
            raise RopeError(ROPE_ERR_PARAM_INVALID, "a page of a cache must be one dense block")
        reach *= size
    return t.as_strided((t.shape[0], reach), (t.stride(0), 1))


class PageCaches:
    """The caches of all layers, described once: a program that copies, forks or compacts pages at
    every step makes one of its list (keys, values and scales, [pages, ...] each) and passes it in the
    list's place.  The tensors must keep their storage while the object is used.

    A fork copies only the tokens of a page that is not full where a cache is [pages, page_size, ...] (3
    or 4 dims) or a float32 [pages, n, m], n a divisor of page_size (scales of n blocks); dimension 1 is then
    taken for tokens.  Caches in ``whole`` are copied by whole pages whatever their shape: those where it is
    something else, such as as many heads as a page has tokens, or scales of heads."""

    def __init__(self, caches, whole=()):
        self.tensors = [*caches, *map(_as_pages, whole)]
        self.device = _device_index(self.tensors)
        self.packed = b"".join(map(_pack, self.tensors)) or None


def _page_caches(caches, dev: int):
    """(PageCaches, device): the list described, on the device of the other tensors."""
    if not isinstance(caches, PageCaches):
        caches = PageCaches(caches)
    if dev >= 0 and caches.device >= 0 and dev != caches.device:
        raise RopeError(ROPE_ERR_PARAM_INVALID, "tensors are on different devices")
    return caches, max(dev, caches.device)


def rope_copy_pages(sources, targets, caches, stream=None):
    """Copy pages: page targets[i] of every cache becomes a copy of page sources[i] (int64 [N]); a pair
    with a number out of range is skipped.  Targets have to be distinct, and none the source of another
    pair.  caches: tensors [pages, ...] whose pages are dense blocks, or a PageCaches of them."""
    caches, dev = _page_caches(caches, _device_index((sources, targets)))
    _run_on(dev, LIB.rope_copy_pages, _pack(sources), _pack(targets), caches.packed,
            len(caches.tensors), _raw_stream(stream, dev))


def rope_fork_pages(page_table, seq_lens, parents, ref_counts, page_size: int, caches=(),
                    grow=None, page_table_out=None, seq_lens_out=None, ref_counts_out=None,
                    shortage=None, stream=None):
    """The next step's sequences continue this step's: new row i has all seq_lens[parents[i]] tokens of
    sequence parents[i] (an empty row without pages where that is out of range; a new sequence continues
    one of length 0) and room for grow[i] more.  Full pages
    are shared, a last page that is not full is copied in all caches for every row but the first that
    continues its sequence (for that one, too, if something else holds the page), and new pages are the
    lowest with ref_counts 0.  Caches [pages, page_size, ...] of 3 or 4 dims and float32 scales [pages, n, m],
    n a divisor of page_size, are taken to hold tokens, or blocks of them, in dimension 1, and only the
    sequence's are copied; all others go by whole pages, and so do those that PageCaches is given as
    ``whole``.  Sequences without a row end.  All index tensors are int64: page_table
    [B, maxPages], seq_lens [B], parents and grow [R], ref_counts [pages] (holds on each page).  Returns
    (page_table_out [R, maxPages], seq_lens_out [R], ref_counts_out [pages], shortage [1]), allocated
    where not given; ref_counts_out may be ref_counts itself, page_table_out may be wider.  shortage is
    the number of pages that were wanted and not free; -1 stands for them in page_table_out."""
    import torch
    caches, dev = _page_caches(caches, _device_index((page_table, seq_lens, parents, ref_counts, grow,
                                                      page_table_out, seq_lens_out, ref_counts_out,
                                                      shortage)))
    if page_table.dim() != 2 or parents.dim() != 1 or ref_counts.dim() != 1:
        raise RopeError(ROPE_ERR_PARAM_INVALID,
                        "page_table must be 2-D, parents and ref_counts 1-D")
    rows, pages, like, i64 = parents.shape[0], ref_counts.shape[0], page_table, torch.int64
    need = LIB.rope_fork_pages_workspace(page_table.shape[0], rows, pages)
    given = (page_table_out, seq_lens_out, ref_counts_out, shortage)
    shapes = ((rows, page_table.shape[1]), (rows,), (pages,), (1,))
    *new, workspace = _new(stream, dev, *((s, i64, like) if g is None else None
                                          for g, s in zip(given, shapes)),
                           (need, torch.uint8, like))
    outs = tuple(g if n is None else n for g, n in zip(given, new))
    _run_on(dev, LIB.rope_fork_pages, _pack(page_table), _pack(seq_lens), _pack(parents),
            _pack(grow), _pack(ref_counts), page_size, caches.packed, len(caches.tensors),
            *map(_pack, outs), workspace.data_ptr(), need, _raw_stream(stream, dev))
    return outs


def rope_compact_pages(page_table, ref_counts, caches=(), page_table_out=None, ref_counts_out=None,
                       page_map=None, live=None, stream=None):
    """The pages in use (ref_counts above 0) move, in all caches, to the lowest numbers: the k-th one
    from number `live` on to the k-th free page below.  Returns (page_table_out, ref_counts_out,
    page_map, live): the table and the holds under the new numbers, page_map [pages] with the new
    number of every page in use and -1 for the others, live [1] the number of pages in use; all int64,
    allocated where not given.  page_table_out may be page_table and ref_counts_out ref_counts."""
    import torch
    caches, dev = _page_caches(caches, _device_index((page_table, ref_counts, page_table_out,
                                                      ref_counts_out, page_map, live)))
    if ref_counts.dim() != 1:
        raise RopeError(ROPE_ERR_PARAM_INVALID, "ref_counts must be 1-D")
    pages, like, i64 = ref_counts.shape[0], ref_counts, torch.int64
    need = LIB.rope_compact_pages_workspace(pages)
    given = (page_table_out, ref_counts_out, page_map, live)
    shapes = (page_table.shape, (pages,), (pages,), (1,))
    *new, workspace = _new(stream, dev, *((s, i64, like) if g is None else None
                                          for g, s in zip(given, shapes)),
                           (need, torch.uint8, like))
    outs = tuple(g if n is None else n for g, n in zip(given, new))
    _run_on(dev, LIB.rope_compact_pages, _pack(page_table), _pack(ref_counts), caches.packed,
            len(caches.tensors), *map(_pack, outs), workspace.data_ptr(), need,
            _raw_stream(stream, dev))
    return outs


class PreparedCall:
    """A call whose arguments are marshalled once (for tight launch loops): invoking it
    issues exactly one C-ABI call with the prebuilt descriptors.  The tensors must stay
    alive and keep their storage while the object is used."""

    def __init__(self, fn, args, keep, dev=None):
        self._fn, self._args, self._keep, self._dev = fn, args, keep, dev

    def __call__(self) -> None:
        _check(_on_device(self._dev, self._fn, self._args))


def prepare_partial_inplace(x, cos, sin, rotary_mode: int = 1, partial_slice=None,
                            stream=None, backward: bool = False) -> PreparedCall:
    dev = _device_of([x, cos, sin])
    dx, dc, ds = describe(x), describe(cos), describe(sin)
    sl, sl_len = _int_array(partial_slice)
    args = (ctypes.byref(dx), ctypes.byref(dc), ctypes.byref(ds), int(rotary_mode), sl, sl_len,
            _stream_handle(stream, dev))
    fn = LIB.rope_partial_inplace_backward if backward else LIB.rope_partial_inplace
    return PreparedCall(fn, args, (x, cos, sin, dx, dc, ds, sl), dev)


def prepare_with_cos_sin_cache(positions, query_in, key_in, cos_sin_cache, mrope_section,
                               head_size, is_neox_style, query_out, key_out, stream=None,
                               cache_mode: int | None = None) -> PreparedCall:
    """cache_mode None: the V1 entry point; else the V2 one with that cacheMode."""
    fn, args, keep, dev = _cache_args(positions, query_in, key_in, cos_sin_cache, mrope_section,
                                      head_size, is_neox_style, cache_mode, query_out, key_out,
                                      stream)
    return PreparedCall(fn, args, keep, dev)
