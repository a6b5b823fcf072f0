"""Sequence operators over voxel tokens: rotary positions, the root-mean-square
and the layer norm, linear attention with a decay for each head, and the
selective scan of a state-space model with its short causal convolution.

A model that reads a batch's voxels as sequences holds one row per active voxel
in the batch's voxel order, grid after grid; ``offsets`` (int64 ``[B + 1]`` on
the GPU) says where each grid's rows start.  Nothing is padded.  The calls
marshal pointers, sizes and strides to ``libtb.so`` (C ABI in ``include/tb.h``)
on torch's current stream; they never wait for the GPU.

Training: ``rotary``, ``rms_norm``, ``layer_norm``, ``linear_attention``,
``causal_conv`` and ``selective_scan`` take part in autograd (first
derivatives; second ones and forward mode are refused); their ``*_backward``
calls are public too.  Generation: ``linear_attention_step``,
``causal_conv_step`` and ``selective_scan_step`` update the states in place, one
token per stream.  Writes in place raise torch's version counters.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional, Sequence, Tuple

__all__ = ["rotary_frequencies", "rotary", "rotary_backward", "rms_norm", "rms_norm_fp8", "rms_norm_backward",
           "layer_norm", "layer_norm_backward",
           "linear_attention", "linear_attention_backward", "linear_attention_step", "linear_attention_status",
           "causal_conv", "causal_conv_backward", "causal_conv_step",
           "selective_scan", "selective_scan_backward", "selective_scan_step"]


class _Native:
    """The compiled entry points (``_seq.so``), loaded at the first call."""

    def __getattr__(self, name):
        from . import LIB_PATH, TBError, lib
        lib()
        if not os.path.exists(os.path.join(os.path.dirname(LIB_PATH), "_seq.so")):
            raise TBError(-1, "_seq.so is not built (run __graft_entry__.build() or "
                              "python -m sparse_voxel_grid_leaf_gb300._build)")
        import torch  # noqa: F401  (its libraries are the module's)

        from . import _seq
        _seq.set_error(TBError)
        global _native
        _native = _seq
        return getattr(_seq, name)


_native = _Native()


def _bad(message: str):
    from . import TBError
    raise TBError(1, message)


def _on_stream(fn, stream, *args, **kw):
    """The call on `stream`: its outputs are allocated there, and its inputs
    are kept from reuse until that stream is done."""
    import torch
    raw = getattr(stream, "cuda_stream", stream) or 0
    on = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(raw))
    for x in list(args) + list(kw.values()):
        if isinstance(x, torch.Tensor) and x.is_cuda:
            x.record_stream(on)
    with torch.cuda.stream(on):
        return fn(*args, **kw)


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


@functools.lru_cache(None)
def _functions():
    """The autograd functions, made once torch is loaded.  Their backward calls
    record nothing, so gradients of their gradients are refused."""
    import torch
    from torch.autograd.function import once_differentiable

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, positions, frequencies, *how):
            ctx.save_for_backward(positions, frequencies)
            ctx.how = how
            return _native.rotary(q, k, positions, frequencies, *how, False, False)

        @staticmethod
        @once_differentiable
        def backward(ctx, dq, dk):
            dq, dk = _native.rotary(dq, dk, *ctx.saved_tensors, *ctx.how, False, True)
            return dq, dk, None, None, None, None, None

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, residual, eps):
            y, h, _ = _native.norm(x, weight, residual, eps, False)
            ctx.save_for_backward(h, weight)
            ctx.eps, ctx.added = eps, residual is not None
            return (y, h) if residual is not None else y

        @staticmethod
        @once_differentiable
        def backward(ctx, dy, dh=None):
            h, weight = ctx.saved_tensors
            dx, dw = _native.norm_backward(dy, h, weight, dh, ctx.eps)
            return dx, dw, dx if ctx.added else None, None

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, decay, offsets, state, scale, return_state):
            ctx.save_for_backward(q, k, v, decay, offsets, state)
            ctx.scale = scale
            o, last = _native.linear(q, k, v, decay, offsets, state, scale, return_state)
            return (o, last) if return_state else o

        @staticmethod
        @once_differentiable
        def backward(ctx, do, dstate=None):
            dq, dk, dv, first = _native.linear_backward(*ctx.saved_tensors, ctx.scale, do, dstate,
                                                        ctx.needs_input_grad[5])
            return dq, dk, dv, None, None, first, None, None

    class LayerNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, residual, eps):
            y, h = _native.layer_norm(x, weight, bias, residual, eps)
            ctx.save_for_backward(h, weight)
            ctx.eps, ctx.biased, ctx.added = eps, bias is not None, residual is not None
            return (y, h) if residual is not None else y

        @staticmethod
        @once_differentiable
        def backward(ctx, dy, dh=None):
            h, weight = ctx.saved_tensors
            dx, dw, db = _native.layer_norm_backward(dy, h, weight, dh, ctx.eps)
            return dx, dw, db if ctx.biased else None, dx if ctx.added else None, None

    class Conv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, offsets, state, activation, return_state):
            ctx.save_for_backward(x, weight, bias, offsets, state)
            ctx.activation = activation
            y, last = _native.conv(x, weight, bias, offsets, state, activation, return_state)
            return (y, last) if return_state else y

        @staticmethod
        @once_differentiable
        def backward(ctx, dy, dstate=None):
            dx, dw, db, first = _native.conv_backward(dy, *ctx.saved_tensors, ctx.activation, dstate)
            return dx, dw, db, None, first, None, None

    class Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, dt, a, b, c, d, z, dt_bias, softplus, offsets, state, return_state):
            ctx.save_for_backward(x, dt, a, b, c, d, z, dt_bias, offsets, state)
            ctx.softplus = softplus
            y, last = _native.scan(x, dt, a, b, c, d, z, dt_bias, softplus, offsets, state, return_state)
            return (y, last) if return_state else y

        @staticmethod
        @once_differentiable
        def backward(ctx, dy, dstate=None):
            *rows, offsets, state = ctx.saved_tensors
            *grads, first = _native.scan_backward(*rows, ctx.softplus, offsets, state, dy, dstate)
            return (*grads, None, None, first, None)

    return Rotary, Norm, Linear, LayerNorm, Conv, Scan


def rotary(q, k, positions, frequencies, layout: str = "half", sections: Optional[Sequence[int]] = None,
           amplitude: float = 1.0, inplace: bool = False, stream=None):
    """Turns queries ``q [T, H, D]`` and keys ``k [T, Hk, D]`` (or None) by
    their tokens' positions; returns both.  ``positions``: int32 or int64 [T],
    or [T, axes] with 2 or 3 axes (a voxel's coordinates), whose ``sections``
    say how many pairs each axis turns (default: as even as they come).
    ``frequencies``: ``rotary_frequencies(R, ...)`` for the first R elements of
    each head; the others pass through.  ``layout``: "half" pairs element i
    with i + R/2, "interleaved" 2 i with 2 i + 1.  ``amplitude`` scales the
    turned elements (long contexts).  ``inplace``: q and k are overwritten."""
    if stream is not None:
        return _on_stream(rotary, stream, q, k, positions, frequencies, layout, sections, amplitude, inplace)
    out = _native.rotary(q, k, positions, frequencies, layout, sections, amplitude, inplace, False)
    if out is not None:
        return out
    if k is None:
        return _functions()[0].apply(q, q[:, :0], positions, frequencies, layout, sections, amplitude)[0], None
    return _functions()[0].apply(q, k, positions, frequencies, layout, sections, amplitude)


def rotary_backward(dq, dk, positions, frequencies, layout: str = "half", sections: Optional[Sequence[int]] = None,
                    amplitude: float = 1.0, inplace: bool = False, stream=None):
    """Gradients of ``rotary``'s q and k from those of its outputs: the turn by
    the opposite angles."""
    if stream is not None:
        return _on_stream(rotary_backward, stream, dq, dk, positions, frequencies, layout, sections, amplitude, inplace)
    out = _native.rotary(dq, dk, positions, frequencies, layout, sections, amplitude, inplace, True)
    return _bad("rotary_backward: gradients of gradients are not made") if out is None else out


# -------------------------------------------------------------------------------------------------------------- norm

def rms_norm(x, weight, residual=None, eps: float = 1e-6, stream=None):
    """``h = x + residual`` and ``y = h / sqrt(mean(h ** 2) + eps) * weight``
    over the last dimension; returns (y, h).  Without a residual h is x.  The
    sum is held in 32 bits: y is computed from it before h is rounded."""
    if stream is not None:
        return _on_stream(rms_norm, stream, x, weight, residual, eps)
    out = _native.norm(x, weight, residual, eps, False)
    if out is not None:
        return out[0], out[1]
    out = _functions()[1].apply(x, weight, residual, eps)
    return out if residual is not None else (out, x)


def rms_norm_fp8(x, weight, residual=None, eps: float = 1e-6, stream=None):
    """``rms_norm`` with y in 8 bits for the product that follows: returns
    (q, scale, h) with q float8_e4m3fn and a 32-bit scale for each row,
    ``y = q * scale``, ``scale = max |y| / 448`` (0 for a row of zeros)."""
    if stream is not None:
        return _on_stream(rms_norm_fp8, stream, x, weight, residual, eps)
    q, h, scale = _native.norm(x, weight, residual, eps, True)
    return q, scale, h


def rms_norm_backward(dy, h, weight, dh=None, eps: float = 1e-6, stream=None):
    """Gradients (dx, dweight) of ``rms_norm`` from dy and, where the residual
    stream goes on, from h's own gradient ``dh``; h as the forward call
    returned it.  dx is the gradient of both x and the residual."""
    if stream is not None:
        return _on_stream(rms_norm_backward, stream, dy, h, weight, dh, eps)
    return _native.norm_backward(dy, h, weight, dh, eps)


def layer_norm(x, weight, bias=None, residual=None, eps: float = 1e-5, stream=None):
    """``h = x + residual`` and ``y = (h - mean(h)) / sqrt(var(h) + eps) *
    weight + bias`` over the last dimension, var the mean of (h - mean(h)) ** 2;
    returns (y, h).  Without a residual h is x.  The sum is held in 32 bits: y
    is computed from it before h is rounded."""
    if stream is not None:
        return _on_stream(layer_norm, stream, x, weight, bias, residual, eps)
    out = _native.layer_norm(x, weight, bias, residual, eps)
    if out is not None:
        return out
    out = _functions()[3].apply(x, weight, bias, residual, eps)
    return out if residual is not None else (out, x)


def layer_norm_backward(dy, h, weight, dh=None, eps: float = 1e-5, stream=None):
    """Gradients (dx, dweight, dbias) of ``layer_norm`` from dy and, where the
    residual stream goes on, from h's own gradient ``dh``; h as the forward call
    returned it.  dx is the gradient of both x and the residual."""
    if stream is not None:
        return _on_stream(layer_norm_backward, stream, dy, h, weight, dh, eps)
    return _native.layer_norm_backward(dy, h, weight, dh, eps)


# -------------------------------------------------------------------------------------------------- linear attention

def linear_attention(q, k, v, decay, offsets=None, state=None, scale: Optional[float] = None,
                     return_state: bool = False, stream=None):
    """Linear attention with a decay for each head over the rows of each grid:
    ``S_t = decay * S_(t-1) + k_t v_t^T``, ``o_t = scale * q_t S_t``.  q, k
    ``[T, H, K]``, v ``[T, H, V]`` of one type (K, V <= 128), decay float32
    ``[H]`` in [0, 1], offsets int64 ``[B + 1]``, not decreasing (None: one
    grid).  Rows before the first offset or past the last belong to no grid:
    their outputs and gradients are zeros.  ``state``: float32 ``[B, H, K, V]``
    states to start from (None: zero).  ``scale``: default ``K ** -0.5``.
    Returns (o, last states or None)."""
    if stream is not None:
        return _on_stream(linear_attention, stream, q, k, v, decay, offsets, state, scale, return_state)
    out = _native.linear(q, k, v, decay, offsets, state, scale, return_state)
    if out is not None:
        return out
    out = _functions()[2].apply(q, k, v, decay, offsets, state, scale, return_state)
    return out if return_state else (out, None)


def linear_attention_backward(do, q, k, v, decay, offsets=None, state=None, scale: Optional[float] = None,
                              dstate=None, stream=None):
    """Gradients (dq, dk, dv, dstate0) of ``linear_attention`` from ``do`` and,
    where the last states were used, from their gradient ``dstate``.  dstate0
    is the gradient of ``state`` (None without one)."""
    if stream is not None:
        return _on_stream(linear_attention_backward, stream, do, q, k, v, decay, offsets, state, scale, dstate)
    return _native.linear_backward(q, k, v, decay, offsets, state, scale, do, dstate, state is not None)


def linear_attention_step(q, k, v, decay, state, slots=None, scale: Optional[float] = None, stream=None):
    """One token for each of N streams: q, k ``[N, H, K]``, v ``[N, H, V]``
    (K, V <= 256).  ``state``: float32 ``[S, H, K, V]``, updated in place;
    stream n uses the state of slot n, or of ``slots[n]`` (int32 [N]; a slot
    outside the states, such as -1, is left out and gives zeros; no two streams
    may share one).  Returns o ``[N, H, V]``."""
    if stream is not None:
        return _on_stream(linear_attention_step, stream, q, k, v, decay, state, slots, scale)
    return _native.step(q, k, v, decay, state, slots, scale)


def linear_attention_status(stream=None):
    """Waits for the stream; raises TBError(TB_ERR_DEVICE_TIMEOUT) where a
    bounded wait inside a linear-attention kernel, on any stream, gave up since
    the last call for this stream (or, at its first, since the library was loaded)."""
    from . import TBError, _stream, lib
    status = lib().tb_linear_attention_status(ctypes.c_void_p(_stream(stream)))
    if status:
        raise TBError(status, lib().tb_last_error().decode())


# ------------------------------------------------------------------------------------------------------- state space

def causal_conv(x, weight, bias=None, offsets=None, state=None, activation: Optional[str] = "silu",
                return_state: bool = False, stream=None):
    """Short causal convolution of every channel over the rows of each grid:
    ``y_t = act(bias + sum_j weight[:, j] * x_(t - W + 1 + j))`` with x ``[T,
    C]``, weight ``[C, W]``, 2 to 4 taps, and bias ``[C]`` of one type, offsets
    int64 ``[B + 1]``, not decreasing (None: one grid).  ``activation``: "silu"
    or None.  ``state``: ``[B, W - 1, C]`` of the same type, the rows before each
    grid's first, oldest first (None: zeros).  Rows before the first offset or
    past the last belong to no grid: their outputs and gradients are zeros.
    Returns (y, last states or None); the last states are the last W - 1 rows of
    state and grid together."""
    if stream is not None:
        return _on_stream(causal_conv, stream, x, weight, bias, offsets, state, activation, return_state)
    out = _native.conv(x, weight, bias, offsets, state, activation, return_state)
    if out is not None:
        return out
    out = _functions()[4].apply(x, weight, bias, offsets, state, activation, return_state)
    return out if return_state else (out, None)


def causal_conv_backward(dy, x, weight, bias=None, offsets=None, state=None, activation: Optional[str] = "silu",
                         dstate=None, stream=None):
    """Gradients (dx, dweight, dbias, dstate0) of ``causal_conv`` from dy and,
    where the last states were used, from their gradient ``dstate``.  dbias and
    dstate0 are None where bias and state are."""
    if stream is not None:
        return _on_stream(causal_conv_backward, stream, dy, x, weight, bias, offsets, state, activation, dstate)
    return _native.conv_backward(dy, x, weight, bias, offsets, state, activation, dstate)


def causal_conv_step(x, weight, state, bias=None, slots=None, activation: Optional[str] = "silu", stream=None):
    """One row for each of N streams: x ``[N, C]``.  ``state``: ``[S, W - 1, C]``
    of x's type, updated in place (the oldest row leaves, x enters); stream n
    uses the state of slot n, or of ``slots[n]`` (int32 [N]; a slot outside the
    states, such as -1, is left out and gives zeros; no two streams may share
    one).  Returns y ``[N, C]``."""
    if stream is not None:
        return _on_stream(causal_conv_step, stream, x, weight, state, bias, slots, activation)
    return _native.conv_step(x, weight, state, bias, slots, activation)


def selective_scan(x, dt, a, b, c, d=None, z=None, dt_bias=None, softplus: bool = True, offsets=None, state=None,
                   return_state: bool = False, stream=None):
    """The scan of a selective state-space model over the rows of each grid:
    ``delta_t = softplus(dt_t + dt_bias)``, ``h_t = exp(delta_t * a) * h_(t-1) +
    delta_t * x_t * b_t``, ``y_t = (c_t . h_t + d * x_t) * silu(z_t)``.  x, dt, z
    ``[T, C]`` and b, c ``[T, G, N]`` (or ``[T, N]``) of one type, C / G
    consecutive channels to a group; a ``[C, N]``, d and dt_bias ``[C]`` float32;
    N <= 256.  z None: no gate.  ``softplus`` False: delta is dt + dt_bias
    itself.  offsets int64 ``[B + 1]``, not decreasing (None: one grid).  Rows
    before the first offset or past the last belong to no grid: their outputs and
    gradients are zeros.  ``state``: float32 ``[B, C, N]`` states to start from
    (None: zero).  Returns (y, last states or None)."""
    if stream is not None:
        return _on_stream(selective_scan, stream, x, dt, a, b, c, d, z, dt_bias, softplus, offsets, state, return_state)
    out = _native.scan(x, dt, a, b, c, d, z, dt_bias, softplus, offsets, state, return_state)
    if out is not None:
        return out
    out = _functions()[5].apply(x, dt, a, b, c, d, z, dt_bias, softplus, offsets, state, return_state)
    return out if return_state else (out, None)


def selective_scan_backward(dy, x, dt, a, b, c, d=None, z=None, dt_bias=None, softplus: bool = True, offsets=None,
                            state=None, dstate=None, stream=None):
    """Gradients (dx, ddt, da, db, dc, dd, dz, ddt_bias, dstate0) of
    ``selective_scan`` from dy and, where the last states were used, from their
    gradient ``dstate``; None for inputs that are None."""
    if stream is not None:
        return _on_stream(selective_scan_backward, stream, dy, x, dt, a, b, c, d, z, dt_bias, softplus, offsets, state,
                          dstate)
    return _native.scan_backward(x, dt, a, b, c, d, z, dt_bias, softplus, offsets, state, dy, dstate)


def selective_scan_step(x, dt, a, b, c, state, d=None, z=None, dt_bias=None, softplus: bool = True, slots=None,
                        stream=None):
    """One token for each of N streams: rows as ``selective_scan`` takes them.
    ``state``: float32 ``[S, C, N]``, updated in place; stream n uses the state
    of slot n, or of ``slots[n]`` (int32 [N]; a slot outside the states, such as
    -1, is left out and gives zeros; no two streams may share one).  Returns y
    ``[N, C]``."""
    if stream is not None:
        return _on_stream(selective_scan_step, stream, x, dt, a, b, c, state, d, z, dt_bias, softplus, slots)
    return _native.scan_step(x, dt, a, b, c, d, z, dt_bias, softplus, slots, state)
