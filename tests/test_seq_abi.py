"""Sequence operators without a GPU: the refusals that come before any device
work, through the C calls and through Python, and the frequencies."""
import ctypes
import struct

import pytest

# the argument structs of include/tb.h, field by field
ROTARY, NORM, NORM_BACKWARD = struct.Struct("@6P10q11if"), struct.Struct("@6P5q3if"), struct.Struct("@7P6q2if4x")
LINEAR, STEP = struct.Struct("@9P10q5if"), struct.Struct("@7P10q4if4x")


@pytest.fixture(scope="module")
def lib():
    from sparse_voxel_grid_leaf_gb300 import _build
    L = ctypes.CDLL(_build.build())
    L.tb_last_error.restype = ctypes.c_char_p
    return L


def test_refusals_before_any_device_work(lib):
    def refused(name, args, word):
        st = getattr(lib, name)(args, None)
        assert st in (1, 7), (name, st)
        assert word in lib.tb_last_error(), lib.tb_last_error()

    for name in ("tb_rotary", "tb_rms_norm", "tb_rms_norm_backward", "tb_linear_attention",
                 "tb_linear_attention_backward", "tb_linear_attention_step"):
        refused(name, None, b"args is NULL")
    p = 64  # a pointer that no refused call follows

    def rotary(tokens=4, dim=64, pairs=32, axes=1, sections=(0, 0), layout=0, kind=2, at=p, heads=2):
        return ROTARY.pack(at, at, at, at, at, at, tokens, *[64] * 8, 1, heads, 1, dim, pairs, axes, *sections,
                                layout, kind, 0, 0, 1.0)
    refused("tb_rotary", rotary(kind=3), b"type")
    refused("tb_rotary", rotary(tokens=-1), b"negative")
    refused("tb_rotary", rotary(pairs=33), b"pairs")
    refused("tb_rotary", rotary(dim=258), b"pairs")
    refused("tb_rotary", rotary(axes=4), b"axes")
    refused("tb_rotary", rotary(axes=2, sections=(20, 11)), b"sections")
    refused("tb_rotary", rotary(layout=2), b"layout")
    refused("tb_rotary", rotary(at=0), b"pointer")
    assert lib.tb_rotary(rotary(tokens=0, at=0), None) == 0

    def norm(x=p, scale=0, rows=4, width=64, kind=2, fp8=0):
        return NORM.pack(x, 0, p, p, 0, scale, rows, 64, 0, 64, 0, width, kind, fp8, 1e-6)
    refused("tb_rms_norm", norm(x=0), b"pointer")
    refused("tb_rms_norm", norm(fp8=1), b"pointer")
    refused("tb_rms_norm", norm(width=0), b"size")
    refused("tb_rms_norm", norm(width=16385), b"16384")
    refused("tb_rms_norm", norm(kind=-1), b"type")
    assert lib.tb_rms_norm(norm(rows=0), None) == 0
    refused("tb_rms_norm_backward", NORM_BACKWARD.pack(p, p, p, 0, p, 0, p, 4, 64, 64, 0, 64, 0, 64, 2, 1e-6),
            b"pointer")

    def linear(q=p, tokens=4, grids=1, heads=2, key=64, value=64, kind=2, offsets=0, decay=p):
        return LINEAR.pack(q, p, p, p, decay, offsets, 0, 0, 0, tokens, *[64] * 8, 0, grids, heads, key, value,
                                kind, 1.0)
    refused("tb_linear_attention", linear(q=0), b"pointer")
    refused("tb_linear_attention", linear(decay=0), b"pointer")
    refused("tb_linear_attention", linear(key=129), b"128")
    refused("tb_linear_attention", linear(value=0), b"size")
    refused("tb_linear_attention", linear(kind=4), b"type")
    refused("tb_linear_attention", linear(grids=2), b"without offsets")
    refused("tb_linear_attention", linear(grids=0, offsets=p), b"without grids")
    refused("tb_linear_attention", linear(tokens=1 << 31), b"2^31")
    refused("tb_linear_attention_backward", linear() + bytes(112), b"pointer")

    def step(streams=4, slots=0, key=64, count=4, state=p):
        return STEP.pack(p, p, p, p, p, state, slots, streams, count, *[64] * 8, 2, key, 64, 2, 1.0)
    refused("tb_linear_attention_step", step(key=257), b"256")
    refused("tb_linear_attention_step", step(count=3), b"4 streams, 3 states")
    refused("tb_linear_attention_step", step(state=0), b"pointer")
    refused("tb_linear_attention_step", step(state=p + 4), b"pointer")
    assert lib.tb_linear_attention_step(step(streams=0), None) == 0


def test_host_tensors_are_refused(lib):
    torch = pytest.importorskip("torch")
    import sparse_voxel_grid_leaf_gb300 as tb
    x = torch.zeros(2, 1, 64)
    with pytest.raises(tb.TBError):
        tb.linear_attention(x, x, x, torch.ones(1))
    with pytest.raises(tb.TBError):
        tb.rms_norm(x, torch.ones(64))
    with pytest.raises(tb.TBError):
        tb.rotary(x, None, torch.zeros(2, dtype=torch.int32), tb.rotary_frequencies(64, device="cpu"))


def test_frequencies_are_fixed_point_turns():
    torch = pytest.importorskip("torch")
    import math

    import sparse_voxel_grid_leaf_gb300 as tb
    f = tb.rotary_frequencies(12, base=100.0, axes=3, device="cpu")
    assert f.dtype == torch.int64 and f.shape == (6,)
    want = [100.0 ** (-i / 2) / (2 * math.pi) for _ in range(3) for i in range(2)]
    assert all(abs(a / 2.0 ** 64 - b) < 1e-16 for a, b in zip(f.tolist(), want))
    for bad in (dict(dim=3), dict(dim=0), dict(dim=8, sections=(1, 2)), dict(dim=8, scaling="x"),
                dict(dim=8, scaling="parts", factor=2.0, fast=1.0, slow=2.0), dict(dim=8, factor=0.0)):
        with pytest.raises(tb.TBError):
            tb.rotary_frequencies(**bad, device="cpu")
