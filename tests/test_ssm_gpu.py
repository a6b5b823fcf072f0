"""The state-space operators and the layer norm on the GPU against their plain
64-bit forms.  Every element's bound is the reference's for 32-bit arithmetic
and half a step of the type that it is rounded to, derived beside the reference."""
import pytest

from tests import _ssm_reference as R
from tests._seq_reference import TINY, UNIT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_voxel_grid_leaf_gb300 as tb  # noqa: E402

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def near(got, want, dtype, what=""):
    value, bound = want
    assert got.shape == value.shape and got.dtype == dtype, (what, got.shape, value.shape)
    bound = bound + UNIT[dtype] * (value.abs() + bound) + TINY[dtype]
    off = (got.double() - value).abs()
    assert torch.isfinite(got).all(), what
    worst = (off / bound).max().item() if off.numel() else 0.0
    assert (off <= bound).all(), "%s: %.3g times the bound" % (what, worst)


def offsets_of(lengths, lead=0):
    ends = [lead]
    for n in lengths:
        ends.append(ends[-1] + n)
    return torch.tensor(ends, device="cuda")


# ------------------------------------------------------------------------------------------------------ convolution

CONV = [([1], 1, 4), ([5], 8, 2), ([0, 3, 1, 2, 0, 40, 0], 33, 4), ([300], 64, 4), ([700, 2, 0, 133], 128, 3),
        ([64] * 9, 24, 2), ([1500], 8, 4), ([900, 37], 260, 4), ([3] * 40, 1040, 4)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("lengths,channels,taps", CONV, ids=str)
@pytest.mark.parametrize("silu,bias,state", [(True, True, True), (False, False, False), (True, False, True), (True, True, False)])
def test_causal_conv(dtype, lengths, channels, taps, silu, bias, state):
    g = gen(channels + taps + len(lengths))
    n = sum(lengths)
    wide = normal(g, n, 2 * channels + 8, dtype=dtype)
    x = wide[:, 8:8 + channels]
    kept = wide.clone()
    w = normal(g, channels, taps, dtype=dtype)
    b = normal(g, channels, dtype=dtype) if bias else None
    s = normal(g, len(lengths), taps - 1, channels, dtype=dtype) if state else None
    dy = normal(g, n, channels, dtype=dtype)
    dlast = normal(g, len(lengths), taps - 1, channels, dtype=dtype)
    how = dict(offsets=offsets_of(lengths), state=s, activation="silu" if silu else None)
    want = R.conv(x, w, b, lengths, s, silu, dy, dlast)
    y, last = tb.causal_conv(x, w, b, return_state=True, **how)
    near(y, want[0], dtype, "y")
    assert torch.equal(last.double(), want[1][0])
    assert torch.equal(tb.causal_conv(x, w, b, **how)[0], y)
    dx, dw, db, first = tb.causal_conv_backward(dy, x, w, b, dstate=dlast, **how)
    near(dx, want[2], dtype, "dx")
    near(dw, want[3], dtype, "dw")
    if bias:
        near(db, want[4], dtype, "db")
    else:
        assert db is None
    if state:
        near(first, want[5], dtype, "dstate0")
    else:
        assert first is None
    assert torch.equal(wide, kept)
    want = R.conv(x, w, b, lengths, s, silu, dy)
    dx, dw, db, first = tb.causal_conv_backward(dy, x, w, b, **how)
    near(dx, want[2], dtype, "dx without dstate")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("streams,channels,taps", [(1, 1, 2), (3, 8, 4), (32, 96, 3), (70, 33, 4), (5, 1024, 4)])
@pytest.mark.parametrize("slots", [False, True])
def test_causal_conv_step(dtype, streams, channels, taps, slots):
    g = gen(streams + channels)
    w, b = normal(g, channels, taps, dtype=dtype), normal(g, channels, dtype=dtype)
    x = normal(g, streams, channels + 8, dtype=dtype)[:, 8:]
    state = normal(g, streams + 3, taps - 1, channels, dtype=dtype)
    at = torch.randperm(streams + 3, generator=g, device="cuda")[:streams].int()
    if slots and streams > 2:
        at[1], at[2] = -1, streams + 3
    where = at if slots else torch.arange(streams, device="cuda", dtype=torch.int32)
    kept = state.clone()
    for silu in (True, False):
        state.copy_(kept)
        y = tb.causal_conv_step(x, w, state, b, slots=at if slots else None, activation="silu" if silu else None)
        new = kept.clone()
        for i, s in enumerate(where.tolist()):
            if not 0 <= s < streams + 3:
                assert (y[i] == 0).all()
                continue
            want = R.conv(x[i:i + 1], w, b, [1], kept[s:s + 1], silu)
            near(y[i:i + 1], want[0], dtype)
            new[s] = torch.cat([kept[s, 1:], x[i:i + 1]])
        assert torch.equal(state, new)


# ---------------------------------------------------------------------------------------------------- selective scan

def scan_inputs(seed, lengths, channels, states, groups, dtype, gate=True, skip=True, bias=True, state=True, pad=0):
    g = gen(seed)
    n = sum(lengths)
    rows = normal(g, n, 4 * channels + pad, dtype=dtype)
    x, dt, z, dy = (rows[:, i * channels + pad:(i + 1) * channels + pad] for i in range(4))
    dt = dt * 0.5 if not pad else dt
    bc = normal(g, n, 2 * groups * states + pad, dtype=dtype)[:, pad:]
    b, c = (r.unflatten(1, (groups, states)) for r in bc.split(groups * states, 1))
    a = -(torch.arange(1, states + 1, device="cuda") * torch.exp(0.3 * normal(g, channels, states))).float()
    step = torch.exp(torch.rand(channels, generator=g, device="cuda") * 4 - 6)
    dt_bias = (step + torch.log(-torch.expm1(-step))) if bias else None
    d = normal(g, channels) if skip else None
    s = normal(g, len(lengths), channels, states) if state else None
    dlast = normal(g, len(lengths), channels, states)
    return dict(x=x, dt=dt, a=a, b=b, c=c, d=d, z=z if gate else None, dt_bias=dt_bias), s, dy, dlast


NAMES = ["dx", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias", "dstate0"]
SCAN = [([1], 1, 1, 1), ([7], 3, 4, 1), ([0, 5, 1, 0, 30, 8, 9, 0], 34, 16, 2), ([150], 64, 16, 1), ([120, 3, 64], 100, 12, 1),
        ([257], 96, 24, 3), ([33, 65], 40, 64, 1), ([90], 16, 130, 2), ([600], 8, 16, 1), ([40] * 12, 129, 5, 1),
        ([31], 8, 256, 1)]


def compare_scan(lengths, channels, states, groups, dtype, softplus=True, **how):
    rows, s, dy, dlast = scan_inputs(sum(lengths) + channels + states, lengths, channels, states, groups, dtype, **how)
    args = [rows[k] for k in ("x", "dt", "a", "b", "c")]
    if not softplus:
        rows["dt_bias"] = None
        rows["dt"] = args[1] = args[1].float().abs().mul(0.1).to(dtype)
    more = {k: rows[k] for k in ("d", "z", "dt_bias")}
    more.update(softplus=softplus, offsets=offsets_of(lengths), state=s)
    want = R.scan(*args, rows["d"], rows["z"], rows["dt_bias"], softplus, lengths, s, dy, dlast)
    y, last = tb.selective_scan(*args, return_state=True, **more)
    near(y, want[0], dtype, "y")
    near(last, want[1], torch.float32, "last")
    assert torch.equal(tb.selective_scan(*args, **more)[0], y)
    got = tb.selective_scan_backward(dy, *args, dstate=dlast, **more)
    given = dict(dd=rows["d"], dz=rows["z"], ddt_bias=rows["dt_bias"], dstate0=s)
    for name, v, w in zip(NAMES, got, want[2:]):
        if name in given and given[name] is None:
            assert v is None, name
        else:
            near(v, w, torch.float32 if name in ("da", "dd", "ddt_bias", "dstate0") else dtype, name)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("lengths,channels,states,groups", SCAN, ids=str)
def test_selective_scan(dtype, lengths, channels, states, groups):
    compare_scan(lengths, channels, states, groups, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("gate,skip,bias,state,softplus", [
    (False, True, True, False, True), (True, False, False, True, True), (False, False, False, False, False),
    (True, True, False, True, False)])
def test_selective_scan_without_some_inputs(dtype, gate, skip, bias, state, softplus):
    compare_scan([70, 0, 33], 40, 16, 1, dtype, softplus, gate=gate, skip=skip, bias=bias, state=state)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("states", [6, 16, 40])
def test_selective_scan_of_odd_rows(dtype, states):
    """Rows that no 16-byte copy can read, next to one another in one buffer."""
    compare_scan([120, 41], 51, states, 1, dtype, pad=3)
    compare_scan([200], 64, states, 2, dtype, pad=1)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("states", [4, 16, 20])
def test_selective_scan_whole_and_in_segments(dtype, states):
    """Many short grids (walked whole) and one long one (split) against the same rows in 64 bits."""
    compare_scan([11] * 30, 70, states, 1, dtype)
    compare_scan([1100], 16, states, 1, dtype)


def test_wide_scans():
    """Several blocks of channels and states a slot, and more than a block's quads of the gradient."""
    compare_scan([45, 20], 600, 16, 2, torch.bfloat16)
    compare_scan([30, 35], 300, 33, 1, torch.float32)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("streams,channels,states,groups", [
    (1, 1, 1, 1), (2, 64, 16, 1), (5, 96, 12, 3), (40, 33, 7, 1), (3, 40, 64, 2), (300, 128, 16, 1), (2, 8, 256, 1)])
@pytest.mark.parametrize("slots", [False, True])
def test_selective_scan_step(dtype, streams, channels, states, groups, slots):
    for pad in (0, 3):
        rows, s, _, _ = scan_inputs(streams + channels, [1] * streams, channels, states, groups, dtype, pad=pad)
        state = torch.cat([s, s[:1] * 0 + 7])
        at = torch.randperm(streams + 1, generator=gen(1), device="cuda")[:streams].int()
        if slots and streams > 2:
            at[1], at[2] = -1, streams + 1
        where = at if slots else torch.arange(streams, device="cuda", dtype=torch.int32)
        kept = state.clone()
        live = (where >= 0) & (where <= streams)
        first = kept[where.clamp(0, streams).long()]
        args = [rows[k] for k in ("x", "dt", "a", "b", "c")]
        more = {k: rows[k] for k in ("d", "z", "dt_bias")}
        y = tb.selective_scan_step(*args, state, slots=at if slots else None, **more)
        want = R.scan(*args, rows["d"], rows["z"], rows["dt_bias"], True, [1] * streams, first)
        near(y[live], tuple(w[live] for w in want[0]), dtype, "y")
        assert (y[~live] == 0).all()
        at_live = where[live].long()
        near(state[at_live], tuple(w[live] for w in want[1]), torch.float32, "state")
        rest = torch.ones(streams + 1, dtype=torch.bool, device="cuda")
        rest[at_live] = False
        assert torch.equal(state[rest], kept[rest])


# -------------------------------------------------------------------------------------------------------- layer norm

@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 8), (700, 64), (5, 77), (900, 77), (3, 1001), (800, 1001), (650, 1024),
                                        (4, 2048), (700, 1536), (3, 5001), (40, 4096), (3, 16384), (620, 4096), (2, 16383)])
@pytest.mark.parametrize("residual,bias", [(True, True), (False, False)])
def test_layer_norm(dtype, rows, width, residual, bias):
    g = gen(rows + width)
    for mean, strided in ((0.0, False), (8.0, True)):  # rows with a mean far from zero, of a wider buffer
        x = normal(g, rows, width + (8 if strided else 0), dtype=dtype)
        x = (x + mean).to(dtype)[:, -width:]
        r = normal(g, rows, width, dtype=dtype, scale=2.0) if residual else None
        w = (1 + 0.2 * normal(g, width)).to(dtype)
        b = normal(g, width, dtype=dtype) if bias else None
        y, h = tb.layer_norm(x, w, b, r, eps=1e-5)
        want, sums = R.layer_norm(x, w, b, r, 1e-5)
        near(y, want, dtype, "y")
        if residual:
            near(h, sums, dtype, "h")
        else:
            assert h is x
        dy = normal(g, rows, width, dtype=dtype)
        got = tb.layer_norm_backward(dy, h, w, dh=r, eps=1e-5)
        for name, v, ref in zip(("dx", "dw", "db"), got, R.layer_norm_backward(dy, h, w, r, 1e-5)):
            near(v, ref, dtype, name)


def test_layer_norm_of_constant_rows_and_no_rows():
    w, b = torch.full((64,), 2.0, device="cuda"), torch.full((64,), 0.5, device="cuda")
    y, _ = tb.layer_norm(torch.full((3, 64), 1e4, device="cuda"), w, b)
    assert torch.equal(y, torch.full_like(y, 0.5))
    y, h = tb.layer_norm(torch.zeros(0, 64, device="cuda"), w, b)
    assert y.shape == (0, 64)
    dx, dw, db = tb.layer_norm_backward(y, h, w)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    x = torch.randn(2, 3, 64, device="cuda")
    y, _ = tb.layer_norm(x, w, b)
    assert torch.equal(y.flatten(0, 1), tb.layer_norm(x.flatten(0, 1), w, b)[0])


# ---------------------------------------------------------------------------------------------------- rows and edges

@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_rows_of_no_grid(dtype):
    """Rows before the first offset and past the last, of any values: zeros out, and nothing of them elsewhere."""
    lengths, lead, tail = [70, 0, 25], 9, 14
    n = sum(lengths)
    rows, s, dy, dlast = scan_inputs(3, lengths, 40, 16, 1, dtype)
    g = gen(5)
    w, b = normal(g, 40, 4, dtype=dtype), normal(g, 40, dtype=dtype)
    cs, cl = normal(g, 3, 3, 40, dtype=dtype), normal(g, 3, 3, 40, dtype=dtype)

    def padded(t):
        return torch.cat([t.new_full((lead,) + t.shape[1:], float("nan")), t, t.new_full((tail,) + t.shape[1:], float("inf"))])

    def every(r, dy, offsets):
        args = [r[k] for k in ("x", "dt", "a", "b", "c")]
        more = dict({k: r[k] for k in ("d", "z", "dt_bias")}, offsets=offsets, state=s)
        conv = dict(offsets=offsets, state=cs)
        return [*tb.selective_scan(*args, return_state=True, **more), *tb.selective_scan_backward(dy, *args, dstate=dlast, **more),
                *tb.causal_conv(r["x"], w, b, return_state=True, **conv),
                *tb.causal_conv_backward(dy, r["x"], w, b, dstate=cl, **conv)]

    want = every(rows, dy, offsets_of(lengths))
    wide = {k: padded(v) if v is not None and v.shape[0] == n else v for k, v in rows.items()}
    got = every(wide, padded(dy), offsets_of(lengths, lead))
    for x, y in zip(want, got):
        if x.shape[0] == n:
            assert (y[:lead] == 0).all() and (y[lead + n:] == 0).all()
            y = y[lead:lead + n]
        # sums over rows may run over other parts of them
        assert torch.equal(x, y) or torch.allclose(x.float(), y.float(), rtol=2 * UNIT[x.dtype] + 200 * R.U, atol=1e-4)


def test_not_a_number_stays_in_its_grid_and_channel():
    rows, s, _, _ = scan_inputs(8, [60, 50, 70], 70, 16, 1, torch.float32)
    args = [rows[k] for k in ("x", "dt", "a", "b", "c")]
    more = dict({k: rows[k] for k in ("d", "z", "dt_bias")}, offsets=offsets_of([60, 50, 70]), state=s)
    want, _ = tb.selective_scan(*args, **more)
    w = torch.randn(70, 4, device="cuda")
    conv, _ = tb.causal_conv(args[0], w, offsets=more["offsets"])
    args[0] = args[0].clone()
    args[0][109, 5] = float("nan")  # a grid's last row
    got, _ = tb.selective_scan(*args, **more)
    assert torch.isnan(got[109, 5])
    got[109, 5] = want[109, 5]
    assert torch.equal(got, want)
    got, _ = tb.causal_conv(args[0], w, offsets=more["offsets"])
    assert torch.isnan(got[109, 5])
    got[109, 5] = conv[109, 5]
    assert torch.equal(got, conv)


@pytest.mark.parametrize("states", [5, 16, 40])
def test_steps_of_zero_keep_the_states(states):
    """exp(0) is 1 to the bit, for every row, tile and segment of a walk, and backward."""
    lengths = [1500, 3, 77]
    rows, s, dy, dlast = scan_inputs(14, lengths, 40, states, 1, torch.float32)
    args = [rows["x"], torch.zeros_like(rows["x"]), rows["a"], rows["b"], rows["c"]]
    more = dict(softplus=False, offsets=offsets_of(lengths), state=s)
    _, last = tb.selective_scan(*args, return_state=True, **more)
    assert torch.equal(last, s)
    first = tb.selective_scan_backward(torch.zeros_like(dy), *args, dstate=dlast, **more)[8]
    assert torch.equal(first, dlast)
    state = s.clone()
    tb.selective_scan_step(*(v[:3] for v in args[:2]), args[2], *(v[:3] for v in args[3:]), state, softplus=False)
    assert torch.equal(state, s)


@pytest.mark.parametrize("states", [5, 16, 40])
@pytest.mark.parametrize("lengths", [[13, 8, 0, 3], [333], [11] * 30], ids=str)
def test_rates_of_minus_infinity(states, lengths):
    """States without memory, next to others: of the reference their rates are finite, and exp(delta a) the same 0."""
    rows, s, dy, dlast = scan_inputs(41, lengths, 40, states, 1, torch.float32)
    none = torch.rand(40, states, generator=gen(3), device="cuda") < 0.5
    none[0], none[1] = True, False
    args = [rows[k] for k in ("x", "dt", "a", "b", "c")]
    more = {k: rows[k] for k in ("d", "z", "dt_bias")}
    args[2] = args[2].masked_fill(none, -1e30)
    want = R.scan(*args, more["d"], more["z"], more["dt_bias"], True, lengths, s, dy, dlast)
    args[2] = args[2].masked_fill(none, -float("inf"))
    y, last = tb.selective_scan(*args, offsets=offsets_of(lengths), state=s, return_state=True, **more)
    near(y, want[0], torch.float32, "y")
    near(last, want[1], torch.float32, "last")
    got = tb.selective_scan_backward(dy, *args, offsets=offsets_of(lengths), state=s, dstate=dlast, **more)
    for name, v, w in zip(NAMES, got, want[2:]):
        near(v, w, torch.float32, name)
    if len(lengths) == 30:
        state = s.clone()
        first = torch.arange(0, 330, 11, device="cuda")
        part = [v[first] if v.shape[0] == 330 else v for v in args]
        y = tb.selective_scan_step(*part, state, d=more["d"], z=more["z"][first], dt_bias=more["dt_bias"])
        near(y, tuple(v[first] for v in want[0]), torch.float32, "step")
        assert torch.isfinite(state).all()


@pytest.mark.parametrize("states", [4, 16, 20])
@pytest.mark.parametrize("rate", [3.0, 12.0])
def test_states_that_grow(states, rate):
    """Rates above zero.  Over a segment, and over a tile at 12 a row, the decay as a whole is beyond 32 bits, where
    the walk is not: states that are zero until the last rows, with a gradient that is until the first ones, and small
    ones that grow for a while."""
    n, c = 230, 40
    g = gen(int(rate) + states)
    a = 1.0 + 0.05 * torch.rand(c, states, generator=g, device="cuda")
    b, k = normal(g, n, 1, states), normal(g, n, 1, states)
    few = int(70 / rate)  # exp(74) at most from a state or gradient to the end
    x, dy = normal(g, n, c), normal(g, n, c)
    x[:n - few] = 0
    dy[few:] = 0
    compare_growth(x, torch.full((n, c), rate, device="cuda"), a, b, k, torch.zeros(1, c, states, device="cuda"), dy,
                   torch.zeros(1, c, states, device="cuda"))
    dt = torch.zeros(n, c, device="cuda")
    dt[:int(120 / rate)] = rate  # exp(126) from first to last, of values that are 1e-36 as they come
    compare_growth(*(normal(g, n, c, scale=1e-36), dt, a, b, k), *(normal(g, *v, scale=1e-36) for v in ((1, c, states), (n, c), (1, c, states))))


def compare_growth(x, dt, a, b, c, state, dy, dlast):
    lengths = [x.shape[0]]
    want = R.scan(x, dt, a, b, c, None, None, None, False, lengths, state, dy, dlast)
    y, last = tb.selective_scan(x, dt, a, b, c, softplus=False, state=state, return_state=True)
    got = tb.selective_scan_backward(dy, x, dt, a, b, c, softplus=False, state=state, dstate=dlast)
    # Products of values of 1e-36 are below 2^-126, where a product is off by up to 2^-150 (TINY) whatever its size, and
    # sums add nothing to that.  db and dc add a product for each channel; g . b, h . c and a . q one for each state, which
    # ddt and dx multiply by a (below 2) or delta, off by TINY once more; da adds q delta, q off by TINY, for each row.
    # (A walk of db row by row in 32 bits is off by 4 TINY where it is 1e-43, of 40 channels.)
    (rows, channels), states = x.shape, a.shape[1]
    floor = (channels + 3 * states + rows) * (1 + dt.max().double()) * TINY[torch.float32]
    given = [(name, v) for name, v in zip(NAMES, got) if v is not None]
    for (name, v), (w, bound) in zip([("y", y), ("last", last)] + given, [w for w, k in zip(want, ["y", "last"] + NAMES)
                                                                          if k not in ("dd", "dz", "ddt_bias")]):
        near(v, (w, bound + floor), torch.float32, name)


def test_many_grids():
    """More grids than blocks of any kernel, a row or none in each, against the same rows as one token of each stream."""
    n, dtype = 20000, torch.float32
    lengths = [i % 2 for i in range(2 * n)]
    rows, s, dy, dlast = scan_inputs(15, lengths, 8, 16, 1, dtype)
    args = [rows[k] for k in ("x", "dt", "a", "b", "c")]
    more = {k: rows[k] for k in ("d", "z", "dt_bias")}
    y, last = tb.selective_scan(*args, offsets=offsets_of(lengths), state=s, return_state=True, **more)
    # the same formula in two orders: sums of 16 products, whose magnitudes stay below 50, and some ten roundings
    state = s[1::2].clone()
    want = tb.selective_scan_step(*args, state, **more)
    assert torch.allclose(y, want, rtol=100 * R.U, atol=100 * R.U * 50) and torch.equal(last[::2], s[::2])
    assert torch.allclose(last[1::2], state, rtol=100 * R.U, atol=1e-6)
    got = tb.selective_scan_backward(dy, *args, offsets=offsets_of(lengths), state=s, dstate=dlast, **more)
    assert torch.equal(got[8][::2], dlast[::2]) and all(torch.isfinite(v).all() for v in got)
    w, cs = normal(gen(1), 8, 4), normal(gen(2), 2 * n, 3, 8)
    y, last = tb.causal_conv(args[0], w, offsets=offsets_of(lengths), state=cs, return_state=True)
    one = cs[1::2].clone()
    want = tb.causal_conv_step(args[0], w, one)
    assert torch.allclose(y, want, rtol=1e-5, atol=1e-6) and torch.equal(last[1::2], one) and torch.equal(last[::2], cs[::2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_grids_of_every_length(dtype):
    """Lengths of 0 to 40 in no order, so that segments start anywhere in eight rows and end anywhere in them."""
    lengths = [(i * 17) % 41 for i in range(41)]
    compare_scan(lengths, 72, 16, 1, dtype)
    compare_scan(lengths, 40, 20, 2, dtype)
    compare_scan([200] + lengths[:20] + [1] * 30, 16, 4, 1, dtype)


def test_many_grids_of_many_channels():
    """The gradient's workspace is its rows' and its slots'; each grid by itself gives the same."""
    n, c = 20000, 1024
    lengths = [1] * n
    rows, _, dy, _ = scan_inputs(16, lengths, c, 16, 1, torch.bfloat16, state=False)
    args = [rows[k] for k in ("x", "dt", "a", "b", "c")]
    more = {k: rows[k] for k in ("d", "z", "dt_bias")}
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    got = tb.selective_scan_backward(dy, *args, offsets=offsets_of(lengths), **more)
    torch.cuda.synchronize()
    # 2 states of 16 a channel and grid, and the rest of the workspace and the outputs, each a small part of that
    assert torch.cuda.max_memory_allocated() - before < 1.35 * 2 * 4 * n * c * 16
    some = torch.arange(0, n, 997, device="cuda")
    part = [v[some] if v.shape[0] == n else v for v in args]
    want = R.scan(*part, more["d"], more["z"][some], more["dt_bias"], True, [1] * len(some), None, dy[some])[2:]
    for name, v, w in zip(NAMES, got, want):
        if name in ("dx", "ddt", "db", "dc", "dz"):
            near(v[some], w, torch.bfloat16, name)


@pytest.mark.parametrize("lead,tail", [(0, 0), (130, 0), (130, 95), (700, 1300)])
def test_segments_between_rows_of_no_grid(lead, tail):
    """Segments by the first rows of their grids: rows before and past them, more grids than a warp has lanes, empty ones
    at both ends."""
    for lengths in ([0, 0, 700, 0, 25, 1, 0], [90 + i % 7 for i in range(70)], [0] * 40 + [900] + [0] * 40):
        n = sum(lengths)
        rows, s, dy, dlast = scan_inputs(51, lengths, 16, 16, 1, torch.float32)
        names = ("x", "dt", "a", "b", "c")
        want = R.scan(*(rows[k] for k in names), rows["d"], rows["z"], rows["dt_bias"], True, lengths, s, dy, dlast)

        def padded(t):
            if t is None or t.shape[0] != n:
                return t
            return torch.cat([t.new_full((lead,) + t.shape[1:], float("nan")), t, t.new_full((tail,) + t.shape[1:], float("inf"))])

        args = [padded(rows[k]) if k != "a" else rows[k] for k in names]
        more = dict(d=rows["d"], z=padded(rows["z"]), dt_bias=rows["dt_bias"], offsets=offsets_of(lengths, lead), state=s)
        y, last = tb.selective_scan(*args, return_state=True, **more)
        near(last, want[1], torch.float32, "last")
        got = tb.selective_scan_backward(padded(dy), *args, dstate=dlast, **more)
        for name, v, w in zip(["y"] + NAMES, (y,) + tuple(got), want[:1] + want[2:]):
            if name in ("y", "dx", "ddt", "dz", "db", "dc"):
                assert (v[:lead] == 0).all() and (v[lead + n:] == 0).all(), name
                v = v[lead:lead + n]
            near(v, w, torch.float32, name)


def test_time_of_many_grids_grows_with_their_number():
    """The gradient of ten times the grids takes ten times as long, and some; by the square it would take a hundred."""
    def time(n):
        rows, _, dy, _ = scan_inputs(17, [1] * n, 64, 16, 1, torch.bfloat16, state=False)
        args, offsets = [rows[k] for k in ("x", "dt", "a", "b", "c")], offsets_of([1] * n)
        took = []
        for _ in range(4):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            tb.selective_scan_backward(dy, *args, offsets=offsets)
            end.record()
            torch.cuda.synchronize()
            took.append(start.elapsed_time(end))
        return min(took[1:])

    assert time(200000) < 25 * time(20000)


def test_no_rows_and_no_grids():
    rows, s, dy, dlast = scan_inputs(2, [0, 0], 40, 16, 1, torch.float32)
    args = [rows[k] for k in ("x", "dt", "a", "b", "c")]
    more = dict({k: rows[k] for k in ("d", "z", "dt_bias")}, offsets=offsets_of([0, 0]), state=s)
    y, last = tb.selective_scan(*args, return_state=True, **more)
    assert y.shape == (0, 40) and torch.equal(last, s)
    got = tb.selective_scan_backward(dy, *args, dstate=dlast, **more)
    assert torch.equal(got[8], dlast) and all((got[i] == 0).all() for i in (2, 5, 7))
    w, cs = torch.randn(40, 4, device="cuda"), torch.randn(2, 3, 40, device="cuda")
    y, last = tb.causal_conv(args[0], w, offsets=more["offsets"], state=cs, return_state=True)
    assert torch.equal(last, cs)
    dx, dw, _, first = tb.causal_conv_backward(y, args[0], w, offsets=more["offsets"], state=cs, dstate=cs)
    assert torch.equal(first, cs) and (dw == 0).all()
    none = dict(more, offsets=torch.zeros(1, dtype=torch.int64, device="cuda"), state=None)
    y, last = tb.selective_scan(*args, return_state=True, **none)
    assert last.shape == (0, 40, 16)
    assert (tb.selective_scan_backward(dy, *args, **none)[2] == 0).all()
    y, last = tb.causal_conv(args[0], w, offsets=none["offsets"], return_state=True)
    assert last.shape == (0, 3, 40)
    state = torch.randn(3, 40, 16, device="cuda")
    assert tb.selective_scan_step(*args, state).shape == (0, 40)
    assert tb.causal_conv_step(args[0], w, torch.randn(2, 3, 40, device="cuda")).shape == (0, 40)


def test_offsets_outside_the_rows_are_clamped():
    rows, _, _, _ = scan_inputs(4, [64], 40, 16, 1, torch.bfloat16)
    args = [rows[k] for k in ("x", "dt", "a", "b", "c")]
    w = normal(gen(1), 40, 4, dtype=torch.bfloat16)
    far = torch.tensor([-5, 64, 1 << 40], device="cuda")
    assert torch.equal(tb.selective_scan(*args, offsets=far)[0], tb.selective_scan(*args)[0])
    assert torch.equal(tb.causal_conv(args[0], w, offsets=far)[0], tb.causal_conv(args[0], w)[0])
    # offsets that decrease name rows twice: outputs of no meaning, but none outside
    back = torch.tensor([0, 64, 3, 50, 20, 64], device="cuda")
    tb.selective_scan(*args, offsets=back, return_state=True)
    tb.selective_scan_backward(args[0], *args, offsets=back)
    tb.causal_conv(args[0], w, offsets=back, return_state=True)
    tb.causal_conv_backward(args[0], args[0], w, offsets=back)
    torch.cuda.synchronize()


def test_rows_past_32_bits():
    """Rows of one buffer of more than 2^31 elements give what the same rows give by themselves."""
    rows, stride, c = 36000, 60008, 64
    wide = torch.empty(rows, stride, device="cuda", dtype=torch.bfloat16)
    assert wide.numel() > 2 ** 31
    g = gen(8)
    parts = []
    for i in range(5):
        part = normal(g, rows, c, dtype=torch.bfloat16)
        view = wide[:, stride - c * (i + 1):stride - c * i]
        view.copy_(part)
        parts.append((part, view))
    a, w = -torch.rand(c, 16, generator=g, device="cuda"), normal(g, c, 4, dtype=torch.bfloat16)
    ends, one = torch.tensor([0, 20000, 20000, rows], device="cuda"), torch.ones(c, device="cuda", dtype=torch.bfloat16)

    def every(x, dt, z, bc, dy):
        b, k = bc[:, :16], bc[:, 16:32]
        return [tb.selective_scan(x, dt, a, b, k, z=z, offsets=ends)[0],
                *(v for v in tb.selective_scan_backward(dy, x, dt, a, b, k, z=z, offsets=ends) if v is not None),
                tb.causal_conv(x, w, offsets=ends)[0], *tb.causal_conv_backward(dy, x, w, offsets=ends)[:2],
                tb.layer_norm(x, one)[0], *tb.layer_norm_backward(dy, x, one)]

    for x, y in zip(every(*(p for p, _ in parts)), every(*(v for _, v in parts))):
        assert torch.equal(x, y)


# ------------------------------------------------------------------------------------- together, streams, refusals

def block(x, p, offsets, how):
    """A state-space block: norm, projection, convolution, scan, projection."""
    y, h = how["norm"](x, p["norm"], p["norm_bias"])
    xz = y @ p["enter"]
    u, z = xz.chunk(2, 1)
    u = how["conv"](u, p["taps"], p["taps_bias"], offsets)
    rest = u @ p["rows"]
    dt, b, c = rest.split([u.shape[1], 8, 8], 1)
    o = how["scan"](u, dt, -torch.exp(p["rate"]), b, c, p["skip"], z, p["step"], offsets)
    return x + o @ p["leave"]


def plain(lengths):
    """The block's operators in elementary torch, differentiable."""
    def conv(u, w, b, offsets):
        out, begin = [], 0
        for n in lengths:
            row = torch.nn.functional.pad(u[begin:begin + n], (0, 0, w.shape[1] - 1, 0))
            out.append(sum(row[j:j + n] * w[:, j] for j in range(w.shape[1])) + b)
            begin += n
        return torch.nn.functional.silu(torch.cat(out))

    def scan(u, dt, a, b, c, d, z, bias, offsets):
        delta, out, begin = torch.nn.functional.softplus(dt + bias), [], 0
        for n in lengths:
            h = torch.zeros_like(a)
            for t in range(begin, begin + n):
                h = torch.exp(delta[t][:, None] * a) * h + (delta[t] * u[t])[:, None] * b[t]
                out.append(h @ c[t] + d * u[t])
            begin += n
        return torch.stack(out) * torch.nn.functional.silu(z)

    return dict(norm=lambda x, w, b: (torch.nn.functional.layer_norm(x, x.shape[1:], w, b, 1e-5), x), conv=conv, scan=scan)


def ours():
    return dict(norm=lambda x, w, b: tb.layer_norm(x, w, b), conv=lambda u, w, b, o: tb.causal_conv(u, w, b, o)[0],
                scan=lambda u, dt, a, b, c, d, z, bias, o: tb.selective_scan(u, dt, a, b, c, d, z, bias, offsets=o)[0])


def block_parameters(width, inner, seed):
    g = gen(seed)
    p = dict(norm=1 + 0.1 * normal(g, width), norm_bias=0.1 * normal(g, width), enter=normal(g, width, 2 * inner, scale=width ** -0.5),
             taps=normal(g, inner, 4, scale=0.5), taps_bias=0.1 * normal(g, inner), rows=normal(g, inner, inner + 16, scale=inner ** -0.5),
             rate=0.5 * normal(g, inner, 8), skip=normal(g, inner), step=normal(g, inner) - 3,
             leave=normal(g, inner, width, scale=inner ** -0.5))
    return {k: v.requires_grad_() for k, v in p.items()}


def test_a_block_and_its_gradients():
    """The operators in a block, in 32 bits, against the same block in 64 bits by torch's own gradients.  Between the two
    lie some 40 operations, matrix products of up to 48 terms among them, and 24 rows of recurrence: 2000 U of the
    largest value cover their roundings."""
    lengths = [24, 1, 0, 15]
    offsets = offsets_of(lengths)
    p = block_parameters(24, 48, 3)
    x = normal(gen(4), sum(lengths), 24).requires_grad_()
    q = {k: v.detach().double().requires_grad_() for k, v in p.items()}
    x64 = x.detach().double().requires_grad_()
    seed = normal(gen(6), sum(lengths), 24)
    got, want = block(x, p, offsets, ours()), block(x64, q, offsets, plain(lengths))
    assert (got.double() - want).abs().max() <= 2000 * R.U * want.abs().max()
    got.backward(seed)
    want.backward(seed.double())
    for name, u, v in [("x", x, x64)] + [(k, p[k], q[k]) for k in p]:
        assert (u.grad.double() - v.grad).abs().max() <= 2000 * R.U * v.grad.abs().max(), name


def test_gradients_against_differences():
    """Along random directions: the difference of the 64-bit reference's outputs, by which the calls' gradients are
    measured too, so that neither leans on a formula for gradients."""
    lengths = [9, 4]
    rows, s, dy, dlast = scan_inputs(12, lengths, 6, 4, 1, torch.float32)
    args = [rows[k] for k in ("x", "dt", "a", "b", "c", "d", "z", "dt_bias")]

    def loss(args, s):
        y, last = (v for v, _ in R.scan(*args[:5], args[5], args[6], args[7], True, lengths, s)[:2])
        return (y * dy.double()).sum() + (last * dlast.double()).sum()

    grads = tb.selective_scan_backward(dy, *args, offsets=offsets_of(lengths), state=s, dstate=dlast)
    inputs, step = args + [s], 2.0 ** -20
    for i, g in enumerate(grads):
        way = torch.randn_like(inputs[i]).double()
        ends = []
        for sign in (1, -1):
            moved = [v.double() for v in inputs]
            moved[i] = moved[i] + sign * step * way
            ends.append(loss(moved[:8], moved[8]))
        slope, got = (ends[0] - ends[1]) / (2 * step), (g.double() * way).sum()
        assert abs(slope - got) <= 1e-5 * (g.double() * way).abs().sum(), NAMES[i]
    x, w, b = normal(gen(1), 13, 6), normal(gen(2), 6, 4), normal(gen(3), 6)
    cs, cl = normal(gen(4), 2, 3, 6), normal(gen(5), 2, 3, 6)
    grads = tb.causal_conv_backward(dy, x, w, b, offsets=offsets_of(lengths), state=cs, dstate=cl)

    def conv_loss(x, w, b, cs):
        y, last = (v for v, _ in R.conv(x, w, b, lengths, cs, True)[:2])
        return (y * dy.double()).sum() + (last * cl.double()).sum()

    for i, g in enumerate(grads):
        way, ends = torch.randn_like([x, w, b, cs][i]).double(), []
        for sign in (1, -1):
            moved = [v.double() for v in (x, w, b, cs)]
            moved[i] = moved[i] + sign * step * way
            ends.append(conv_loss(*moved))
        assert abs((ends[0] - ends[1]) / (2 * step) - (g.double() * way).sum()) <= 1e-5 * (g.double() * way).abs().sum()
    grads = tb.layer_norm_backward(dy, x, w[:, 0].contiguous())
    for i, g in enumerate(grads):
        way, ends = torch.randn_like([x, b, b][i]).double(), []
        for sign in (1, -1):
            moved = [x.double(), w[:, 0].double(), 0 * b.double()]
            moved[i] = moved[i] + sign * step * way
            ends.append((R.layer_norm(moved[0], moved[1], moved[2], None, 1e-5)[0][0] * dy.double()).sum())
        assert abs((ends[0] - ends[1]) / (2 * step) - (g.double() * way).sum()) <= 1e-5 * (g.double() * way).abs().sum()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_prompt_and_steps_go_on_as_the_whole(dtype):
    """The last states of a prompt, and then one token a stream, give what the whole rows give."""
    lengths, more = [50, 20, 0], 5
    total = [n + more for n in lengths]
    rows, _, _, _ = scan_inputs(7, total, 40, 16, 1, dtype, state=False)
    w, b = normal(gen(1), 40, 4, dtype=dtype), normal(gen(2), 40, dtype=dtype)
    u, _ = tb.causal_conv(rows["x"], w, b, offsets_of(total))
    args = {k: rows[k] for k in ("dt", "b", "c", "z")}
    rest = {k: rows[k] for k in ("d", "dt_bias")}
    whole = R.scan(u, args["dt"], rows["a"], args["b"], args["c"], rest["d"], args["z"], rest["dt_bias"], True, total, None)
    begin = [0, total[0], total[0] + total[1]]
    head = torch.cat([torch.arange(n, device="cuda") + o for n, o in zip(lengths, begin)])
    uh, conv_state = tb.causal_conv(rows["x"][head], w, b, offsets_of(lengths), return_state=True)
    assert torch.equal(uh, u[head])
    _, state = tb.selective_scan(uh, args["dt"][head], rows["a"], args["b"][head], args["c"][head], z=args["z"][head],
                                 offsets=offsets_of(lengths), return_state=True, **rest)
    for t in range(more):
        at = torch.tensor([o + n + t for n, o in zip(lengths, begin)], device="cuda")
        x = tb.causal_conv_step(rows["x"][at], w, conv_state, b)
        assert torch.equal(x, u[at])
        y = tb.selective_scan_step(x, args["dt"][at], rows["a"], args["b"][at], args["c"][at], state, z=args["z"][at], **rest)
        near(y, tuple(v[at] for v in whole[0]), dtype)
    near(state, whole[1], torch.float32)


def test_streams_and_graphs():
    lengths = [900, 40, 0, 333]
    rows, s, dy, dlast = scan_inputs(31, lengths, 96, 16, 1, torch.bfloat16)
    args = [rows[k] for k in ("x", "dt", "a", "b", "c")]
    more = dict({k: rows[k] for k in ("d", "z", "dt_bias")}, offsets=offsets_of(lengths), state=s)
    w, one = normal(gen(1), 96, 4, dtype=torch.bfloat16), torch.ones(96, dtype=torch.bfloat16, device="cuda")
    token = [v[:4] for v in args[:2]] + [args[2]] + [v[:4] for v in args[3:]]

    def every(stream=None):
        u, cl = tb.causal_conv(args[0], w, offsets=more["offsets"], return_state=True, stream=stream)
        y, last = tb.selective_scan(u, *args[1:], return_state=True, stream=stream, **more)
        grads = tb.selective_scan_backward(dy, u, *args[1:], dstate=dlast, stream=stream, **more)
        conv = tb.causal_conv_backward(grads[0], args[0], w, offsets=more["offsets"], stream=stream)
        n, _ = tb.layer_norm(y, one, stream=stream)
        norm = tb.layer_norm_backward(dy, y, one, stream=stream)
        step = tb.selective_scan_step(*token, last, stream=stream)
        conv_step = tb.causal_conv_step(token[0], w, cl, stream=stream)
        return [v for v in (u, cl, y, last, *grads, *conv, n, *norm, step, conv_step) if v is not None]

    want = every()
    torch.cuda.synchronize()
    again = every()  # sums in a fixed order: the same bits
    assert all(torch.equal(x, y) for x, y in zip(want, again))
    side = torch.cuda.Stream()
    got = every(side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(every())
    for graph, out in zip(graphs, outs):
        for x in out:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, out))


def test_two_streams_at_once():
    """Calls of two streams at the same time keep their workspaces apart."""
    rows, s, dy, _ = scan_inputs(33, [3000], 64, 16, 1, torch.float32)
    args = [rows[k] for k in ("x", "dt", "a", "b", "c")]
    want = [v for v in tb.selective_scan_backward(dy, *args) if v is not None]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for stream in streams:
            got.append(tb.selective_scan_backward(dy, *args, stream=stream))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(x, y) for x, y in zip(want, [v for v in g if v is not None]))


def test_refusals():
    x = torch.randn(8, 12, device="cuda")
    w, a, bc = torch.randn(12, 4, device="cuda"), -torch.rand(12, 16, device="cuda"), torch.randn(8, 16, device="cuda")
    one, ends = torch.ones(12, device="cuda"), torch.tensor([0, 8], device="cuda")
    conv, h = torch.randn(1, 3, 12, device="cuda"), torch.randn(1, 12, 16, device="cuda")
    bad = [
        lambda: tb.causal_conv(x.double(), w.double()),
        lambda: tb.causal_conv(x, w.bfloat16()),
        lambda: tb.causal_conv(x, w[:11]),
        lambda: tb.causal_conv(x, w[:, :1]),
        lambda: tb.causal_conv(x, torch.randn(12, 5, device="cuda")),
        lambda: tb.causal_conv(x[0], w),
        lambda: tb.causal_conv(x, w, one[:3]),
        lambda: tb.causal_conv(x, w, offsets=ends.int()),
        lambda: tb.causal_conv(x, w, offsets=ends, state=conv.half()),
        lambda: tb.causal_conv(x, w, offsets=ends, state=conv[:, :2]),
        lambda: tb.causal_conv(x, w, activation="relu"),
        lambda: tb.causal_conv(x.cpu(), w.cpu()),
        lambda: tb.causal_conv_backward(x[:7], x, w),
        lambda: tb.causal_conv_backward(x, x, w, dstate=conv[:, :1]),
        lambda: tb.causal_conv_step(x, w, conv),  # one state for eight streams
        lambda: tb.causal_conv_step(x, w, conv.expand(8, 3, 12)),
        lambda: tb.causal_conv_step(x, w, conv, slots=torch.zeros(8, device="cuda", dtype=torch.int64)),
        lambda: tb.selective_scan(x, x.half(), a, bc, bc),
        lambda: tb.selective_scan(x, x[:7], a, bc, bc),
        lambda: tb.selective_scan(x, x, a.bfloat16(), bc, bc),
        lambda: tb.selective_scan(x, x, a[:11], bc, bc),
        lambda: tb.selective_scan(x, x, a, bc[:, :8], bc),
        lambda: tb.selective_scan(x, x, a, bc[:, None].expand(8, 5, 16), bc[:, None].expand(8, 5, 16)),  # 12 channels
        lambda: tb.selective_scan(x, x, a, bc[:, None].expand(8, 2, 16), bc),
        lambda: tb.selective_scan(x, x, a, bc, bc, d=one[:3]),
        lambda: tb.selective_scan(x, x, a, bc, bc, dt_bias=one.half()),
        lambda: tb.selective_scan(x, x, a, bc, bc, z=x[:, :11]),
        lambda: tb.selective_scan(x, x, a, bc, bc, offsets=ends, state=h[:, :, :8]),
        lambda: tb.selective_scan(x, x, a, bc, bc, offsets=ends.cpu()),
        lambda: tb.selective_scan(x, x, -torch.rand(12, 257, device="cuda"), torch.randn(8, 257, device="cuda"),
                                  torch.randn(8, 257, device="cuda")),
        lambda: tb.selective_scan_backward(x[:7], x, x, a, bc, bc),
        lambda: tb.selective_scan_step(x, x, a, bc, bc, h),
        lambda: tb.selective_scan_step(x, x, a, bc, bc, h.expand(8, 12, 16)),
        lambda: tb.selective_scan_step(x, x, a, bc, bc, h.half()),
        lambda: tb.layer_norm(x, one[:3]),
        lambda: tb.layer_norm(x, one, one.half()),
        lambda: tb.layer_norm(x, one, one, x[:7]),
        lambda: tb.layer_norm(x.int(), one),
        lambda: tb.layer_norm(torch.zeros(2, 16385, device="cuda"), torch.zeros(16385, device="cuda")),
        lambda: tb.layer_norm_backward(x[:7], x, one),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(tb.TBError):
            call()
            print("refusal %d did not come" % i)
    torch.cuda.synchronize()


def differentiable():
    """Each differentiable call as a function of one tensor [24, 12]."""
    g = gen(9)
    w, a, bc, one = normal(g, 12, 4), -torch.rand(12, 16, device="cuda"), normal(g, 24, 16), torch.ones(12, device="cuda")
    return {"conv": lambda x: tb.causal_conv(x, w)[0], "scan": lambda x: tb.selective_scan(x, x, a, bc, bc)[0],
            "layer_norm": lambda x: tb.layer_norm(x, one, one)[0], "layer_norm_residual": lambda x: tb.layer_norm(x, one, one, x)[0]}


@pytest.mark.parametrize("name", ["conv", "scan", "layer_norm", "layer_norm_residual"])
def test_what_autograd_is_told(name):
    """First derivatives with create_graph as without; second ones and forward mode refused."""
    import torch.autograd.forward_ad as fwAD
    call = differentiable()[name]
    x = normal(gen(2), 24, 12).requires_grad_()
    want, = torch.autograd.grad(call(x).square().sum(), x)
    got, = torch.autograd.grad(call(x).square().sum(), x, create_graph=True)
    assert torch.equal(got, want)
    with pytest.raises(RuntimeError):
        (got.square().sum() + x.sum()).backward()
    with fwAD.dual_level():
        with pytest.raises((RuntimeError, NotImplementedError)):
            call(fwAD.make_dual(x.detach(), x.detach()))


def test_steps_are_writes_and_backward_calls_record_nothing():
    x, w, a, bc = (normal(gen(i), *s) for i, s in enumerate([(4, 12), (12, 4), (12, 16), (4, 16)]))
    a = -a.abs()
    conv, h = normal(gen(5), 4, 3, 12), normal(gen(6), 4, 12, 16)
    t = x.clone().requires_grad_()
    for state, step in ((conv, lambda: tb.causal_conv_step(x, w, conv)), (h, lambda: tb.selective_scan_step(x, x, a, bc, bc, h))):
        k = torch.randn_like(state).requires_grad_()
        y = (k * state).sum()
        before = state._version
        step()
        assert state._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    one = torch.ones(12, device="cuda")
    for call in (lambda: tb.causal_conv_step(t, w, conv), lambda: tb.selective_scan_step(t, x, a, bc, bc, h),
                 lambda: tb.causal_conv_backward(t, x, w), lambda: tb.causal_conv_backward(x, t, w),
                 lambda: tb.selective_scan_backward(t, x, x, a, bc, bc), lambda: tb.selective_scan_backward(x, x, t, a, bc, bc),
                 lambda: tb.layer_norm_backward(t, x, one), lambda: tb.layer_norm_backward(x, x, one, t)):
        with pytest.raises(tb.TBError):
            call()
        with torch.no_grad():
            call()


def test_a_training_step_in_a_graph():
    """Forward and backward by autograd, captured and replayed."""
    lengths = [130, 0, 60]
    p = block_parameters(24, 48, 5)
    x = normal(gen(4), sum(lengths), 24)
    offsets = offsets_of(lengths)

    def step():
        grads = torch.autograd.grad(block(x, p, offsets, ours()).square().sum(), list(p.values()))
        return grads

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [g.clone() for g in step()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for g in out:
        g.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for g, v in zip(out, want):  # the products of the library may run in another order under capture
        assert torch.allclose(g, v, rtol=1e-4, atol=1e-4 * v.abs().max().item())
