"""State-space operators and layer norm without a GPU: the refusals that come
before any device work, through the C calls and through Python."""
import ctypes
import struct

import pytest

# the argument structs of include/tb.h, field by field
NORM, NORM_BACKWARD = struct.Struct("@6P5q3if"), struct.Struct("@7P6q2if4x")
CONV, CONV_STEP = struct.Struct("@7P3q5i4x"), struct.Struct("@6P4q4i")
SCAN, SCAN_STEP = struct.Struct("@13P10q6i"), struct.Struct("@11P10q5i4x")


@pytest.fixture(scope="module")
def lib():
    from sparse_voxel_grid_leaf_gb300 import _build
    L = ctypes.CDLL(_build.build())
    L.tb_last_error.restype = ctypes.c_char_p
    for name in ("tb_selective_scan_workspace", "tb_causal_conv_backward_workspace", "tb_layer_norm_backward_workspace"):
        getattr(L, name).restype = ctypes.c_int64
    return L


P = 4096  # a pointer that no refused call follows


def refused(lib, name, args, word, *more):
    st = getattr(lib, name)(args, *more, None)
    assert st in (1, 7), (name, st)
    assert word in lib.tb_last_error(), lib.tb_last_error()


def test_norm(lib):
    def norm(x=P, rows=4, width=64, kind=2, fp8=0, scale=0):
        return NORM.pack(x, 0, P, P, 0, scale, rows, 64, 0, 64, 0, width, kind, fp8, 1e-5)
    refused(lib, "tb_layer_norm", None, b"args is NULL", None)
    refused(lib, "tb_layer_norm", norm(x=0), b"tb_layer_norm: bad pointer", None)
    refused(lib, "tb_layer_norm", norm(fp8=1, scale=P), b"pointer", None)  # it has no 8-bit output
    refused(lib, "tb_layer_norm", norm(width=16385), b"16384", None)
    refused(lib, "tb_layer_norm", norm(kind=3), b"type", None)
    assert lib.tb_layer_norm(norm(rows=0), None, None) == 0
    refused(lib, "tb_layer_norm_backward", NORM_BACKWARD.pack(P, P, P, 0, P, 0, P, 4, 64, 64, 0, 64, 0, 64, 2, 1e-5), b"pointer",
            ctypes.c_void_p(P))
    assert lib.tb_layer_norm_backward_workspace(ctypes.c_int64(100), 64) >= 100 * 64 * 4 * 2


def test_conv(lib):
    def conv(x=P, w=P, y=P, offsets=0, tokens=4, grids=1, channels=8, taps=4, kind=2):
        return CONV.pack(x, w, 0, y, offsets, 0, 0, tokens, 8, 8, grids, channels, taps, kind, 1)
    for name in ("tb_causal_conv", "tb_causal_conv_backward", "tb_causal_conv_step"):
        refused(lib, name, None, b"args is NULL")
    for name, rest in (("tb_causal_conv", b""), ("tb_causal_conv_backward", bytes(80))):
        refused(lib, name, conv(x=0) + rest, b"pointer")
        refused(lib, name, conv(w=0) + rest, b"pointer")
        refused(lib, name, conv(taps=1) + rest, b"taps")
        refused(lib, name, conv(taps=5) + rest, b"taps")
        refused(lib, name, conv(channels=0) + rest, b"size")
        refused(lib, name, conv(tokens=-1) + rest, b"size")
        refused(lib, name, conv(grids=-1) + rest, b"size")
        refused(lib, name, conv(kind=4) + rest, b"type")
        refused(lib, name, conv(grids=2) + rest, b"without offsets")
        refused(lib, name, conv(grids=0, offsets=P) + rest, b"without grids")
        refused(lib, name, conv(tokens=1 << 31) + rest, b"2^31")
    refused(lib, "tb_causal_conv", conv(y=0), b"pointer")
    refused(lib, "tb_causal_conv_backward", conv() + bytes(80), b"pointer")

    def step(x=P, state=P, slots=0, streams=4, count=4, taps=4):
        return CONV_STEP.pack(x, P, 0, P, state, slots, streams, count, 8, 8, 8, taps, 2, 1)
    refused(lib, "tb_causal_conv_step", step(count=3), b"4 streams, 3 states")
    refused(lib, "tb_causal_conv_step", step(state=0), b"pointer")
    refused(lib, "tb_causal_conv_step", step(x=0), b"pointer")
    refused(lib, "tb_causal_conv_step", step(taps=9), b"taps")
    assert lib.tb_causal_conv_step(step(streams=0), None) == 0


def test_scan(lib):
    def scan(x=P, a=P, y=P, offsets=0, tokens=4, grids=1, channels=8, states=16, groups=1, kind=2):
        return SCAN.pack(x, P, P, P, 0, y, a, 0, 0, offsets, 0, 0, 0, tokens, *[8] * 8, 0, grids, channels, states, groups, kind, 1)
    assert struct.calcsize("@13P10q6i") == SCAN.size
    for name in ("tb_selective_scan", "tb_selective_scan_backward", "tb_selective_scan_step"):
        refused(lib, name, None, b"args is NULL")
    for name, rest in (("tb_selective_scan", b""), ("tb_selective_scan_backward", bytes(120))):
        refused(lib, name, scan(x=0) + rest, b"pointer")
        refused(lib, name, scan(a=0) + rest, b"pointer")
        refused(lib, name, scan(states=257) + rest, b"256")
        refused(lib, name, scan(states=0) + rest, b"size")
        refused(lib, name, scan(groups=3) + rest, b"groups")
        refused(lib, name, scan(kind=-1) + rest, b"type")
        refused(lib, name, scan(grids=2) + rest, b"without offsets")
        refused(lib, name, scan(grids=0, offsets=P) + rest, b"without grids")
        refused(lib, name, scan(tokens=1 << 31) + rest, b"2^31")
    refused(lib, "tb_selective_scan", scan(y=0), b"pointer")
    refused(lib, "tb_selective_scan_backward", scan() + bytes(120), b"pointer")

    def step(x=P, state=P, slots=0, streams=4, count=4, states=16, groups=1):
        return SCAN_STEP.pack(x, P, P, P, 0, P, P, 0, 0, state, slots, streams, count, *[8] * 8, 8, states, groups, 2, 1)
    refused(lib, "tb_selective_scan_step", step(count=3), b"4 streams, 3 states")
    refused(lib, "tb_selective_scan_step", step(state=0), b"pointer")
    refused(lib, "tb_selective_scan_step", step(state=P + 4), b"pointer")
    refused(lib, "tb_selective_scan_step", step(states=300), b"256")
    refused(lib, "tb_selective_scan_step", step(groups=5), b"groups")
    assert lib.tb_selective_scan_step(step(streams=0), None) == 0
    assert lib.tb_selective_scan_workspace(ctypes.c_int64(-1), 1, 8, 16, 1, 1) == 0
    assert lib.tb_selective_scan_workspace(ctypes.c_int64(100), 1, 8, 16, 1, 1) > 0


def test_host_tensors_are_refused(lib):
    torch = pytest.importorskip("torch")
    import sparse_voxel_grid_leaf_gb300 as tb
    x, a, bc = torch.zeros(2, 8), torch.zeros(8, 4), torch.zeros(2, 4)
    for call in (lambda: tb.causal_conv(x, torch.zeros(8, 4)), lambda: tb.selective_scan(x, x, a, bc, bc),
                 lambda: tb.layer_norm(x, torch.ones(8)), lambda: tb.selective_scan_step(x, x, a, bc, bc, torch.zeros(2, 8, 4)),
                 lambda: tb.causal_conv_step(x, torch.zeros(8, 4), torch.zeros(2, 3, 8))):
        with pytest.raises(tb.TBError):
            call()


def test_the_gradients_workspace_grows_with_rows_and_slots(lib):
    """Its arrays one by one, in bytes: what every row takes, and what every segment does, of which a grid has one for
    each 16 to 64 rows and one more.  A grid's rows are not rounded up to a segment's."""
    def made(tokens, grids, channels, states, groups):
        return lib.tb_selective_scan_workspace(ctypes.c_int64(tokens), grids, channels, states, groups, 1)

    def most(tokens, grids, channels, states, groups, sms=256):
        per = channels // groups
        wide = (per + 63) // 64 * 64 * groups
        pad = 8 if states <= 8 else (states + 15) // 16 * 16
        slots, quads = tokens // 16 + grids, (per + 127) // 128
        runs = min(slots, 12 * sms // (groups * quads) + 1)
        row = wide * (pad + 1) / 2 + 8 * pad * groups * quads + (12 * channels if states > 16 else 0)
        return tokens * row + slots * 4 * wide * (2 * pad + 1) + runs * 4 * wide * (pad + 2) + 10 * 256

    for case in [(20000, 20000, 1024, 16, 1), (60000, 40000, 1024, 16, 1), (32768, 4096, 2048, 16, 1), (16384, 2048, 2048, 64, 1),
                 (124807, 16, 1024, 16, 1), (1333, 5, 202, 12, 2), (0, 7, 64, 16, 1), (7, 1, 1, 1, 1), (100, 300, 96, 4, 2),
                 (5000, 1, 300, 256, 3)]:
        assert 0 < made(*case) <= most(*case), case
    assert made(20000, 20000, 1024, 16, 1) < 3e9
    # one more empty grid takes a segment's states at its ends, and their decay
    assert made(20000, 20001, 1024, 16, 1) - made(20000, 20000, 1024, 16, 1) <= 4 * 1024 * 33 + 4 * 1024 * 18 + 2560


def test_sizes_that_are_refused_ask_for_no_workspace(lib):
    """2^25 groups of one channel are 2^31 channels in whole tiles: the call refuses them, and the workspace's size is
    not what 32 bits make of theirs."""
    n = 1 << 25
    for backward in (0, 1):
        assert lib.tb_selective_scan_workspace(ctypes.c_int64(1), 1, n, 1, n, backward) == 0
        assert lib.tb_selective_scan_workspace(ctypes.c_int64(1 << 31), 1, 8, 16, 1, backward) == 0
    assert lib.tb_selective_scan_workspace(ctypes.c_int64(1), 1, n - 1, 1, n - 1, 1) > 0
    args = SCAN.pack(P, P, P, P, 0, P, P, 0, 0, 0, 0, 0, 0, 1, *[n] * 8, 0, 1, n, 1, n, 2, 1)
    refused(lib, "tb_selective_scan", args, b"2^31 channels")
    # the gradient's rows, its own gradients and strides behind the struct of the scan
    refused(lib, "tb_selective_scan_backward", args + bytes(120), b"2^31 channels")
