"""Sequence operators over voxel tokens: rotary positions, the root-mean-square
norm, and linear attention with a decay for each head.

A model that reads a batch's voxels as sequences holds one row per active voxel
in the batch's voxel order, grid after grid; ``offsets`` (int64 ``[B + 1]`` on
the GPU) says where each grid's rows start.  Nothing is padded.  The calls
marshal pointers, sizes and strides to ``libtb.so`` (C ABI in ``include/tb.h``)
on torch's current stream; they never wait for the GPU.

Training: ``rotary``, ``rms_norm`` and ``linear_attention`` take part in
autograd; their ``*_backward`` calls are public too.  Generation:
``linear_attention_step`` updates the states in place, one token per stream.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct
from typing import Optional, Sequence, Tuple

__all__ = ["rotary_frequencies", "rotary", "rotary_backward", "rms_norm", "rms_norm_fp8", "rms_norm_backward",
           "linear_attention", "linear_attention_backward", "linear_attention_step", "linear_attention_status"]

# the argument structs of include/tb.h, field by field
_ROTARY = struct.Struct("@6P10q11if")
_NORM = struct.Struct("@6P5q3if")
_NORM_BACKWARD = struct.Struct("@7P6q2if4x")
_LINEAR = struct.Struct("@9P10q5if")
_LINEAR_BACKWARD = struct.Struct("@9P10q5if6P8q")
_STEP = struct.Struct("@7P10q4if4x")

_torch = None
_types = None
_calls = None
_get_device = None
_get_stream = None


def _start():
    global _torch, _types, _calls, _get_device, _get_stream
    import torch

    from . import TBError, lib  # noqa: F401
    L = lib()
    calls = {}
    for name in ("tb_rotary", "tb_rms_norm", "tb_rms_norm_backward", "tb_linear_attention",
                 "tb_linear_attention_backward", "tb_linear_attention_step"):
        fn = getattr(L, name)
        fn.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
        fn.restype = ctypes.c_int
        calls[name] = fn
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    L.tb_rms_norm_backward_workspace.argtypes = [i64, i32]
    L.tb_rms_norm_backward_workspace.restype = i64
    calls["norm_workspace"] = L.tb_rms_norm_backward_workspace
    L.tb_linear_attention_workspace.argtypes = [i64, i32, i32, i32, i32, i32, i32]
    L.tb_linear_attention_workspace.restype = i64
    calls["linear_workspace"] = L.tb_linear_attention_workspace
    _types = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    _get_device = torch._C._cuda_getDevice
    _get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda d: torch.cuda.current_stream(d).cuda_stream)
    _torch = torch
    _calls = calls


def _bad(message: str):
    from . import TBError
    raise TBError(1, message)


def _call(name: str, args: bytes, device: int):
    status = _calls[name](args, _get_stream(device))
    if status:
        from . import TBError, lib
        raise TBError(status, lib().tb_last_error().decode())


def _device(what: str, x) -> int:
    if not x.is_cuda:
        _bad("%s: tensors must be on the GPU" % what)
    d = x.get_device()
    if d != _get_device():
        _bad("%s: tensors live on device %d, current device is %d" % (what, d, _get_device()))
    return d


def _same(what: str, name: str, x, shape, dtype, device: int):
    if tuple(x.shape) != tuple(shape) or x.dtype != dtype or x.get_device() != device:
        _bad("%s: %s must be %s %s on device %d, got %s %s on device %d"
             % (what, name, dtype, tuple(shape), device, x.dtype, tuple(x.shape), x.get_device()))


def _rows(what: str, name: str, x):
    """A [rows, heads, dim] tensor with unit stride inside its heads."""
    if x.dim() != 3:
        _bad("%s: %s must have 3 dimensions (rows, heads, elements), got %d" % (what, name, x.dim()))
    if x.stride(2) != 1 and x.shape[2] > 1:
        x = x.contiguous()
    return x


def _type(what: str, x) -> int:
    t = _types.get(x.dtype)
    if t is None:
        _bad("%s: expected dtype float32/float16/bfloat16, got %s" % (what, x.dtype))
    return t


def _streamed(fn):
    """Runs the call on `stream` where one is given: its outputs are allocated
    there, and its inputs are kept from reuse until that stream is done."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if _torch is None:
            _start()
        if stream is None:
            return fn(*args, **kw)
        raw = getattr(stream, "cuda_stream", stream) or 0
        on = stream if isinstance(stream, _torch.cuda.Stream) else _torch.cuda.ExternalStream(int(raw))
        for x in list(args) + list(kw.values()):
            if isinstance(x, _torch.Tensor) and x.is_cuda:
                x.record_stream(on)
        with _torch.cuda.stream(on):
            return fn(*args, **kw)
    return call


def _tracked(*xs) -> bool:
    return _torch.is_grad_enabled() and any(x is not None and x.requires_grad for x in xs)


# ------------------------------------------------------------------------------------------------------------ rotary

def _even(pairs: int, axes: int) -> Tuple[int, ...]:
    return tuple(pairs // axes + (a < pairs % axes) for a in range(axes))


def rotary_frequencies(dim: int, base: float = 10000.0, axes: int = 1, sections: Optional[Sequence[int]] = None,
                       scaling: Optional[str] = None, factor: float = 1.0, original: int = 8192,
                       fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """Turns per unit of position for the ``dim / 2`` pairs of a rotated head:
    an int64 tensor of 64-bit fixed-point fractions of a turn, as ``rotary``
    takes it.  Pair i of the n pairs of an axis has the frequency
    ``base ** (-i / n)`` radians per unit.  ``sections``: pairs per position
    axis (default: as even as they come).

    ``scaling`` stretches positions for contexts ``factor`` times the
    ``original`` length: "linear" divides every frequency by the factor; "base"
    raises the base so that the slowest frequency is divided by it and the
    fastest kept; "parts" keeps frequencies that turn at least ``fast`` times
    in the original context, divides those that turn at most ``slow`` times,
    and blends between."""
    import torch
    if dim < 2 or dim % 2:
        _bad("rotary_frequencies: %d is not an even number of elements" % dim)
    sections = _even(dim // 2, axes) if sections is None else tuple(int(n) for n in sections)
    if sum(sections) != dim // 2 or not 1 <= len(sections) <= 3 or min(sections) < 0:
        _bad("rotary_frequencies: sections %s of %d pairs" % (sections, dim // 2))
    if scaling not in (None, "linear", "base", "parts") or not factor > 0 or not base > 0:
        _bad("rotary_frequencies: scaling %r by %r" % (scaling, factor))
    if scaling == "parts" and not (fast > slow > 0 and original > 0):
        _bad("rotary_frequencies: parts between %r and %r turns of %r positions" % (slow, fast, original))
    table = []
    for n in sections:
        b = base * factor ** (n / (n - 1)) if scaling == "base" and n > 1 else base
        for i in range(n):
            f = b ** (-i / n)
            if scaling == "linear":
                f /= factor
            elif scaling == "parts":
                turns = original * f / (2 * math.pi)
                keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
                f = f * keep + f / factor * (1.0 - keep)
            x = int(f / (2 * math.pi) * 2.0 ** 64) % 2 ** 64
            table.append(x - 2 ** 64 if x >= 2 ** 63 else x)
    return torch.tensor(table, dtype=torch.int64, device=device)


def _rotary(q, k, positions, turns, layout, sections, amplitude, inplace, inverse, what):
    device = _device(what, q)
    kind = _type(what, q)
    q = q if inplace else _rows(what, "q", q)
    tokens, qh, dim = q.shape
    kh = 0
    if k is not None:
        k = k if inplace else _rows(what, "k", k)
        kh = k.shape[1] if k.dim() == 3 else -1
        _same(what, "k", k, (tokens, kh, dim), q.dtype, device)
    pairs = turns.shape[0]
    _same(what, "frequencies", turns, (pairs,), _torch.int64, device)
    if positions.dtype != _torch.int32 and positions.dtype != _torch.int64:
        _bad("%s: positions must be int32 or int64, got %s" % (what, positions.dtype))
    axes = 1 if positions.dim() == 1 else positions.shape[1] if positions.dim() == 2 else 0
    if positions.shape[0] != tokens or positions.get_device() != device or not 1 <= axes <= 3:
        _bad("%s: positions must be [%d] or [%d, 1 to 3] on device %d, got %s"
             % (what, tokens, tokens, device, tuple(positions.shape)))
    if axes > 1 and positions.stride(1) != 1:
        positions = positions.contiguous()
    if turns.stride(0) != 1:
        turns = turns.contiguous()
    if sections is None:
        sections = _even(pairs, axes)
    if len(sections) != axes or sum(sections) != pairs:
        _bad("%s: sections %s of %d pairs on %d axes" % (what, tuple(sections), pairs, axes))
    lay = 0 if layout == "half" else 1 if layout == "interleaved" else _bad("%s: unknown layout %r" % (what, layout))
    if inplace:
        for name, x in (("q", q), ("k", k)):
            if x is not None and (x.dim() != 3 or x.stride(2) != 1 or
                                  any(s == 0 and n > 1 for s, n in zip(x.stride(), x.shape))):
                _bad("%s: %s cannot be turned in place (unit stride inside a head, no repeated rows)" % (what, name))
        qo, ko = q, k
    else:
        qo = _torch.empty((tokens, qh, dim), dtype=q.dtype, device=q.device)
        ko = None if k is None else _torch.empty((tokens, kh, dim), dtype=q.dtype, device=q.device)
    qs, qos = q.stride(), qo.stride()
    if k is None:
        ks = kos = (0, 0)
        kp = kop = 0
    else:
        ks, kos, kp, kop = k.stride(), ko.stride(), k.data_ptr(), ko.data_ptr()
    _call("tb_rotary", _ROTARY.pack(q.data_ptr(), kp, qo.data_ptr(), kop, positions.data_ptr(), turns.data_ptr(),
                                    tokens, qs[0], qs[1], ks[0], ks[1], qos[0], qos[1], kos[0], kos[1],
                                    positions.stride(0), qh, kh, dim, pairs, axes, sections[0],
                                    sections[1] if axes > 1 else 0, lay, kind, positions.dtype == _torch.int64,
                                    inverse, amplitude), device)
    return qo, ko


@functools.lru_cache(None)
def _functions():
    """The autograd functions, made once torch is loaded."""
    import torch

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, positions, turns, layout, sections, amplitude):
            ctx.save_for_backward(positions, turns)
            ctx.how = layout, sections, amplitude
            return _rotary(q, k, positions, turns, layout, sections, amplitude, False, False, "rotary")

        @staticmethod
        def backward(ctx, dq, dk):
            dq, dk = _rotary(dq, dk, *ctx.saved_tensors, *ctx.how, False, True, "rotary_backward")
            return dq, dk, None, None, None, None, None

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, residual, eps):
            y, h, _ = _norm(x, weight, residual, eps, False, "rms_norm")
            ctx.save_for_backward(h, weight)
            ctx.eps, ctx.added = eps, residual is not None
            return (y, h) if residual is not None else y

        @staticmethod
        def backward(ctx, dy, dh=None):
            h, weight = ctx.saved_tensors
            dx, dw = _norm_backward(dy, h, weight, dh, ctx.eps)
            return dx, dw, dx if ctx.added else None, None

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, decay, offsets, state, scale, return_state):
            ctx.save_for_backward(q, k, v, decay, offsets, state)
            ctx.scale, ctx.returned = scale, return_state
            o, last = _linear(q, k, v, decay, offsets, state, scale, return_state)
            return (o, last) if return_state else o

        @staticmethod
        def backward(ctx, do, dstate=None):
            q, k, v, decay, offsets, state = ctx.saved_tensors
            dq, dk, dv, first = _linear_backward(do, q, k, v, decay, offsets, state, ctx.scale, dstate,
                                                 state is not None and ctx.needs_input_grad[5])
            return dq, dk, dv, None, None, first, None, None

    return Rotary, Norm, Linear


@_streamed
def rotary(q, k, positions, frequencies, layout: str = "half", sections: Optional[Sequence[int]] = None,
           amplitude: float = 1.0, inplace: bool = False):
    """Turns queries ``q [T, H, D]`` and keys ``k [T, Hk, D]`` (or None) by
    their tokens' positions; returns both.  ``positions``: int32 or int64 [T],
    or [T, axes] with 2 or 3 axes (a voxel's coordinates), whose ``sections``
    say how many pairs each axis turns (default: as even as they come).
    ``frequencies``: ``rotary_frequencies(R, ...)`` for the first R elements of
    each head; the others pass through.  ``layout``: "half" pairs element i
    with i + R/2, "interleaved" 2 i with 2 i + 1.  ``amplitude`` scales the
    turned elements (long contexts).  ``inplace``: q and k are overwritten."""
    if _tracked(q, k):
        if inplace:
            _bad("rotary: in place is for tensors without gradients")
        if k is None:
            return _functions()[0].apply(q, q[:, :0], positions, frequencies, layout, sections, amplitude)[0], None
        return _functions()[0].apply(q, k, positions, frequencies, layout, sections, amplitude)
    return _rotary(q, k, positions, frequencies, layout, sections, amplitude, inplace, False, "rotary")


@_streamed
def rotary_backward(dq, dk, positions, frequencies, layout: str = "half", sections: Optional[Sequence[int]] = None,
                    amplitude: float = 1.0, inplace: bool = False):
    """Gradients of ``rotary``'s q and k from those of its outputs: the turn by
    the opposite angles."""
    return _rotary(dq, dk, positions, frequencies, layout, sections, amplitude, inplace, True, "rotary_backward")


# -------------------------------------------------------------------------------------------------------------- norm

def _flat(what, name, x):
    """[rows, width] with unit stride inside a row."""
    if x.dim() != 2:
        if x.dim() < 1:
            _bad("%s: %s has no rows" % (what, name))
        x = x.reshape(-1, x.shape[-1]) if x.numel() else x.new_empty((math.prod(x.shape[:-1]), x.shape[-1]))
    return x if x.stride(1) == 1 or x.shape[1] == 1 else x.contiguous()


def _norm(x, weight, residual, eps, fp8, what):
    device = _device(what, x)
    kind = _type(what, x)
    shape = x.shape
    x2 = _flat(what, "x", x)
    rows, width = x2.shape
    _same(what, "weight", weight, (width,), x.dtype, device)
    if weight.stride(0) != 1 and width > 1:
        weight = weight.contiguous()
    h = h2 = r2 = None
    if residual is not None:
        _same(what, "residual", residual, shape, x.dtype, device)
        r2 = _flat(what, "residual", residual)
        h2 = _torch.empty((rows, width), dtype=x.dtype, device=x.device)
        h = h2 if len(shape) == 2 else h2.view(shape)
    y2 = _torch.empty((rows, width), dtype=_torch.float8_e4m3fn if fp8 else x.dtype, device=x.device)
    scale = _torch.empty(shape[:-1], dtype=_torch.float32, device=x.device) if fp8 else None
    _call("tb_rms_norm", _NORM.pack(x2.data_ptr(), 0 if r2 is None else r2.data_ptr(), weight.data_ptr(),
                                    y2.data_ptr(), 0 if h2 is None else h2.data_ptr(),
                                    scale.data_ptr() if fp8 else 0, rows, x2.stride(0),
                                    0 if r2 is None else r2.stride(0), width, width, width, kind, fp8, eps), device)
    return y2 if len(shape) == 2 else y2.view(shape), x if h is None else h, scale


@_streamed
def rms_norm(x, weight, residual=None, eps: float = 1e-6):
    """``h = x + residual`` and ``y = h / sqrt(mean(h ** 2) + eps) * weight``
    over the last dimension; returns (y, h).  Without a residual h is x.  The
    sum is held in 32 bits: y is computed from it before h is rounded."""
    if _tracked(x, weight, residual):
        out = _functions()[1].apply(x, weight, residual, eps)
        return out if residual is not None else (out, x)
    y, h, _ = _norm(x, weight, residual, eps, False, "rms_norm")
    return y, h


@_streamed
def rms_norm_fp8(x, weight, residual=None, eps: float = 1e-6):
    """``rms_norm`` with y in 8 bits for the product that follows: returns
    (q, scale, h) with q float8_e4m3fn and a 32-bit scale for each row,
    ``y = q * scale``, ``scale = max |y| / 448`` (0 for a row of zeros)."""
    if _tracked(x, weight, residual):
        _bad("rms_norm_fp8: the 8-bit output has no gradient")
    q, h, scale = _norm(x, weight, residual, eps, True, "rms_norm_fp8")
    return q, scale, h


def _norm_backward(dy, h, weight, dh, eps):
    what = "rms_norm_backward"
    device = _device(what, h)
    kind = _type(what, h)
    shape = h.shape
    h2 = _flat(what, "h", h)
    rows, width = h2.shape
    _same(what, "dy", dy, shape, h.dtype, device)
    _same(what, "weight", weight, (width,), h.dtype, device)
    if weight.stride(0) != 1 and width > 1:
        weight = weight.contiguous()
    dy2, dh2 = _flat(what, "dy", dy), None
    if dh is not None:
        _same(what, "dh", dh, shape, h.dtype, device)
        dh2 = _flat(what, "dh", dh)
    dx = _torch.empty((rows, width), dtype=h.dtype, device=h.device)
    dw = _torch.empty((width,), dtype=h.dtype, device=h.device)
    size = _calls["norm_workspace"](rows, width)
    work = _torch.empty((size,), dtype=_torch.uint8, device=h.device)
    _call("tb_rms_norm_backward",
          _NORM_BACKWARD.pack(dy2.data_ptr(), h2.data_ptr(), weight.data_ptr(), 0 if dh2 is None else dh2.data_ptr(),
                              dx.data_ptr(), dw.data_ptr(), work.data_ptr(), rows, dy2.stride(0), h2.stride(0),
                              0 if dh2 is None else dh2.stride(0), width, size, width, kind, eps), device)
    return dx if len(shape) == 2 else dx.view(shape), dw


@_streamed
def rms_norm_backward(dy, h, weight, dh=None, eps: float = 1e-6):
    """Gradients (dx, dweight) of ``rms_norm`` from dy and, where the residual
    stream goes on, from h's own gradient ``dh``; h as the forward call
    returned it.  dx is the gradient of both x and the residual."""
    return _norm_backward(dy, h, weight, dh, eps)


# -------------------------------------------------------------------------------------------------- linear attention

def _linear_inputs(what, q, k, v, decay, offsets, state):
    device = _device(what, q)
    kind = _type(what, q)
    q, k, v = _rows(what, "q", q), _rows(what, "k", k), _rows(what, "v", v)
    tokens, heads, key = q.shape
    value = v.shape[2]
    _same(what, "k", k, (tokens, heads, key), q.dtype, device)
    _same(what, "v", v, (tokens, heads, value), q.dtype, device)
    _same(what, "decay", decay, (heads,), _torch.float32, device)
    if decay.stride(0) != 1:
        decay = decay.contiguous()
    grids = 1
    if offsets is not None:
        grids = offsets.shape[0] - 1 if offsets.dim() == 1 else -1
        if grids < 0 or offsets.dtype != _torch.int64 or offsets.get_device() != device:
            _bad("%s: offsets must be int64 [grids + 1] on device %d" % (what, device))
        if offsets.stride(0) != 1:
            offsets = offsets.contiguous()
    if state is not None:
        _same(what, "state", state, (grids, heads, key, value), _torch.float32, device)
        state = state.contiguous()
    return device, kind, q, k, v, decay, offsets, state, (tokens, grids, heads, key, value)


def _linear(q, k, v, decay, offsets, state, scale, return_state):
    what = "linear_attention"
    device, kind, q, k, v, decay, offsets, state, sizes = _linear_inputs(what, q, k, v, decay, offsets, state)
    tokens, grids, heads, key, value = sizes
    if decay.requires_grad and _torch.is_grad_enabled():
        _bad("linear_attention: the decay is a constant and has no gradient")
    out = _torch.empty((tokens, heads, value), dtype=q.dtype, device=q.device)
    last = _torch.empty((grids, heads, key, value), dtype=_torch.float32, device=q.device) if return_state else None
    size = _calls["linear_workspace"](*sizes, kind, 0)
    work = _torch.empty((size,), dtype=_torch.uint8, device=q.device) if size else None
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    _call("tb_linear_attention",
          _LINEAR.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), decay.data_ptr(),
                       0 if offsets is None else offsets.data_ptr(), 0 if state is None else state.data_ptr(),
                       0 if last is None else last.data_ptr(), work.data_ptr() if size else 0, tokens,
                       qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], heads * value, value, size, grids, heads, key, value,
                       kind, scale), device)
    return out, last


def _linear_backward(do, q, k, v, decay, offsets, state, scale, dstate, want):
    what = "linear_attention_backward"
    device, kind, q, k, v, decay, offsets, state, sizes = _linear_inputs(what, q, k, v, decay, offsets, state)
    tokens, grids, heads, key, value = sizes
    do = _rows(what, "do", do)
    _same(what, "do", do, (tokens, heads, value), q.dtype, device)
    if dstate is not None:
        _same(what, "dstate", dstate, (grids, heads, key, value), _torch.float32, device)
        dstate = dstate.contiguous()
    new = lambda n: _torch.empty((tokens, heads, n), dtype=q.dtype, device=q.device)  # noqa: E731
    dq, dk, dv = new(key), new(key), new(value)
    first = _torch.empty((grids, heads, key, value), dtype=_torch.float32, device=q.device) if want else None
    size = _calls["linear_workspace"](*sizes, kind, 1)
    work = _torch.empty((size,), dtype=_torch.uint8, device=q.device) if size else None
    qs, ks, vs, gs = q.stride(), k.stride(), v.stride(), do.stride()
    _call("tb_linear_attention_backward",
          _LINEAR_BACKWARD.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), 0, decay.data_ptr(),
                                0 if offsets is None else offsets.data_ptr(),
                                0 if state is None else state.data_ptr(), 0, work.data_ptr() if size else 0, tokens,
                                qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], 0, 0, size, grids, heads, key, value, kind,
                                scale, do.data_ptr(), 0 if dstate is None else dstate.data_ptr(), dq.data_ptr(),
                                dk.data_ptr(), dv.data_ptr(), 0 if first is None else first.data_ptr(), gs[0], gs[1],
                                heads * key, key, heads * key, key, heads * value, value), device)
    return dq, dk, dv, first


@_streamed
def linear_attention(q, k, v, decay, offsets=None, state=None, scale: Optional[float] = None,
                     return_state: bool = False):
    """Linear attention with a decay for each head over the rows of each grid:
    ``S_t = decay * S_(t-1) + k_t v_t^T``, ``o_t = scale * q_t S_t``.  q, k
    ``[T, H, K]``, v ``[T, H, V]`` of one type (K, V <= 128), decay float32
    ``[H]`` in [0, 1], offsets int64 ``[B + 1]`` (None: one grid).  ``state``:
    float32 ``[B, H, K, V]`` states to start from (None: zero).  ``scale``:
    default ``K ** -0.5``.  Returns (o, last states or None)."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    if _tracked(q, k, v, decay, state):
        if decay.requires_grad:
            _bad("linear_attention: the decay is a constant and has no gradient")
        out = _functions()[2].apply(q, k, v, decay, offsets, state, scale, return_state)
        return out if return_state else (out, None)
    return _linear(q, k, v, decay, offsets, state, scale, return_state)


@_streamed
def linear_attention_backward(do, q, k, v, decay, offsets=None, state=None, scale: Optional[float] = None,
                              dstate=None):
    """Gradients (dq, dk, dv, dstate0) of ``linear_attention`` from ``do`` and,
    where the last states were used, from their gradient ``dstate``.  dstate0
    is the gradient of ``state`` (None without one)."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    return _linear_backward(do, q, k, v, decay, offsets, state, scale, dstate, state is not None)


def linear_attention_status(stream=None):
    """Waits for the stream; raises TBError(TB_ERR_DEVICE_TIMEOUT) where a
    bounded wait inside a linear-attention kernel gave up since the last call."""
    from . import TBError, _stream, lib
    status = lib().tb_linear_attention_status(ctypes.c_void_p(_stream(stream)))
    if status:
        raise TBError(status, lib().tb_last_error().decode())


@_streamed
def linear_attention_step(q, k, v, decay, state, slots=None, scale: Optional[float] = None):
    """One token for each of N streams: q, k ``[N, H, K]``, v ``[N, H, V]``
    (K, V <= 256).  ``state``: float32 ``[S, H, K, V]``, updated in place;
    stream n uses the state of slot n, or of ``slots[n]`` (int32 [N]; a slot
    outside the states, such as -1, is left out and gives zeros; no two streams
    may share one).  Returns o ``[N, H, V]``."""
    what = "linear_attention_step"
    device = _device(what, q)
    kind = _type(what, q)
    q, k, v = _rows(what, "q", q), _rows(what, "k", k), _rows(what, "v", v)
    streams, heads, key = q.shape
    value = v.shape[2]
    _same(what, "k", k, (streams, heads, key), q.dtype, device)
    _same(what, "v", v, (streams, heads, value), q.dtype, device)
    _same(what, "decay", decay, (heads,), _torch.float32, device)
    if decay.stride(0) != 1:
        decay = decay.contiguous()
    count = state.shape[0] if state.dim() == 4 else -1
    _same(what, "state", state, (count, heads, key, value), _torch.float32, device)
    if not state.is_contiguous():
        _bad("linear_attention_step: the states must be contiguous")
    if slots is not None:
        _same(what, "slots", slots, (streams,), _torch.int32, device)
        if slots.stride(0) != 1:
            slots = slots.contiguous()
    if _tracked(q, k, v, decay, state):
        _bad("linear_attention_step: a step in place has no gradient (linear_attention has)")
    out = _torch.empty((streams, heads, value), dtype=q.dtype, device=q.device)
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    _call("tb_linear_attention_step",
          _STEP.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), decay.data_ptr(), state.data_ptr(),
                     0 if slots is None else slots.data_ptr(), streams, count, qs[0], qs[1], ks[0], ks[1], vs[0],
                     vs[1], heads * value, value, heads, key, value, kind,
                     key ** -0.5 if scale is None else scale), device)
    return out
