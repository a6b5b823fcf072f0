"""The sequence operators on the GPU against their plain 64-bit forms.

Tolerances, element by element.  A value rounded to a type of unit roundoff u
is off by u |value|; a sum of n terms held in 32 bits by at most (n + a few)
2^-24 of the sum of its terms' magnitudes; an operand that a kernel rounds to
16 bits before a product adds its unit roundoff times that same sum, once for
each such operand (linear attention in bfloat16 rounds at most three: the
weights of a chunk, the state, the decayed values)."""
import math

import pytest

from tests import _seq_reference as R

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


def near(got, want, size, dtype, terms=8, roundings=0, what=""):
    """|got - want| <= u |want| + (terms 2^-24 + roundings u16) size + the type's smallest step."""
    assert got.shape == want.shape and got.dtype == dtype, what
    bound = R.UNIT[dtype] * want.abs() + (terms * 2.0 ** -24 + roundings * 2.0 ** -8) * size + R.TINY[dtype]
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    worst = (off / bound.clamp(min=1e-300)).max().item() if off.numel() else 0.0
    assert (off <= bound).all(), "%s: %.3g times the bound" % (what, worst)


# ------------------------------------------------------------------------------------------------------------ rotary

@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,kv,dim,rotated,axes", [
    (1, 1, 1, 2, 2, 1), (3, 2, 1, 64, 64, 1), (257, 5, 3, 64, 64, 3), (1000, 8, 2, 128, 64, 1), (33, 3, 3, 96, 48, 2),
    (41, 2, 2, 35, 10, 1), (17, 70, 1, 256, 256, 3), (5000, 4, 4, 80, 80, 3), (19, 3, 2, 256, 6, 3)])
def test_rotary(dtype, layout, tokens, heads, kv, dim, rotated, axes):
    g = gen(tokens + dim)
    qkv = normal(g, tokens, heads + 2 * kv, dim, dtype=dtype)
    q, k = qkv[:, :heads], qkv[:, heads:heads + kv]
    kept = qkv.clone()
    shape = (tokens,) if axes == 1 else (tokens, axes)
    pos = torch.randint(-(1 << 20), 1 << 20, shape, generator=g, device="cuda", dtype=torch.int32)
    f = tb.rotary_frequencies(rotated, axes=axes, scaling="parts", factor=4.0)
    sections = [rotated // 2 // axes + (a < rotated // 2 % axes) for a in range(axes)]
    for call, inverse in ((tb.rotary, False), (tb.rotary_backward, True)):
        outs = call(q, k, pos, f, layout=layout, amplitude=1.25)
        for x, y in zip((q, k), outs):
            want, size = R.rotary(x, pos, f, layout, sections, 1.25, inverse)
            near(y, want, size, dtype, what="inverse" if inverse else "turn")
            assert torch.equal(y[..., rotated:], x[..., rotated:])
    assert torch.equal(qkv, kept)
    y = tb.rotary(q, k, pos, f, layout=layout, amplitude=1.25)
    tb.rotary(q, k, pos, f, layout=layout, amplitude=1.25, inplace=True)
    assert torch.equal(qkv[:, :heads], y[0]) and torch.equal(qkv[:, heads:heads + kv], y[1])
    assert torch.equal(qkv[:, heads + kv:], kept[:, heads + kv:])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,kv,dim,rotated,axes", [
    (257, 4, 1, 48, 24, 3), (3000, 2, 2, 80, 40, 3), (19, 3, 1, 12, 8, 1), (700, 1, 1, 20, 20, 1), (65, 5, 3, 44, 36, 2)])
def test_rotary_of_rows_at_any_four_elements(dtype, layout, tokens, heads, kv, dim, rotated, axes):
    test_rotary(dtype, layout, tokens, heads, kv, dim, rotated, axes)


def test_rotary_positions():
    """64-bit positions beyond 2^31, one huge section, positions as columns of a wider tensor, no keys."""
    g = gen(4)
    q = normal(g, 50, 2, 64)
    wide = torch.randint(-(1 << 45), 1 << 45, (50, 7), generator=g, device="cuda")
    pos = wide[:, 2:5]
    f = tb.rotary_frequencies(64, sections=(1, 30, 1))
    y, none = tb.rotary(q, None, pos, f, sections=(1, 30, 1))
    assert none is None
    want, size = R.rotary(q, pos, f, "half", (1, 30, 1), 1.0)
    near(y, want, size, torch.float32)
    # a position of zero turns nothing; a shared row of queries is read, not written
    f = tb.rotary_frequencies(64)
    y, _ = tb.rotary(q[:1].expand(50, 2, 64), None, torch.zeros(50, dtype=torch.int32, device="cuda"), f)
    assert torch.equal(y, q[:1].expand(50, 2, 64))
    y, z = tb.rotary(q[:0], q[:0, :1], wide[:0, 0], f)
    assert y.shape == (0, 2, 64) and z.shape == (0, 1, 64)


def test_rotary_frequencies():
    f = tb.rotary_frequencies(64, base=500.0, device="cpu").double() / 2.0 ** 64 * 2 * math.pi
    want = torch.tensor([500.0 ** (-i / 32) for i in range(32)], dtype=torch.float64)
    assert ((f - want).abs() <= 1e-15 * want).all()
    lin = tb.rotary_frequencies(64, base=500.0, scaling="linear", factor=8.0, device="cpu").double()
    assert torch.allclose(lin * 8, f * 2.0 ** 64 / (2 * math.pi), rtol=1e-14)
    up = tb.rotary_frequencies(64, base=500.0, scaling="base", factor=8.0, device="cpu").double() / 2.0 ** 64 * 2 * math.pi
    assert abs(up[0] / f[0] - 1) < 1e-12 and abs(up[-1] * 8 / f[-1] - 1) < 1e-12
    parts = tb.rotary_frequencies(64, scaling="parts", factor=8.0, original=4096, device="cpu").double()
    plain = tb.rotary_frequencies(64, device="cpu").double()
    assert parts[0] == plain[0] and abs(parts[-1] * 8 / plain[-1] - 1) < 1e-12
    assert ((parts <= plain) & (parts >= plain / 8 * (1 - 1e-12))).all()


# -------------------------------------------------------------------------------------------------------------- norm

@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,width", [(1, 1), (5, 7), (3, 64), (1000, 64), (700, 1000), (33, 1001), (2000, 1536),
                                        (16, 2048), (1, 16384), (9, 16384), (5, 9999)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(dtype, rows, width, residual):
    g = gen(rows * 7 + width)
    x = normal(g, rows, width + 24, dtype=dtype, scale=2.0)[:, 8:8 + width]  # rows with a stride
    r = normal(g, rows, width, dtype=dtype, scale=3.0) if residual else None
    w = normal(g, width, dtype=dtype)
    y, h = tb.rms_norm(x, w, r, eps=1e-5)
    want, sum_ = R.norm(x, w, r, 1e-5)
    near(y, want, want.abs(), dtype, terms=width + 16, what="y")
    if residual:
        near(h, sum_, sum_.abs(), dtype, terms=2, what="h")
    else:
        assert h is x
    q, scale, h8 = tb.rms_norm_fp8(x, w, r, eps=1e-5)
    assert q.dtype == torch.float8_e4m3fn and q.shape == x.shape and scale.shape == (rows,)
    assert (h8 is x) if r is None else torch.equal(h8, h)
    top = want.abs().amax(-1) / 448
    assert ((scale.double() - top).abs() <= (width + 20) * 2.0 ** -24 * top).all()
    # half a step of three fraction bits, or of the smallest step 2^-9, of a number up to 448
    back, real = q.double(), want / top[:, None].clamp(min=1e-300)
    assert ((back - real).abs() <= 2.0 ** -4 * real.abs().clamp(min=2.0 ** -6) * (1 + 1e-3) + (width + 40) * 2.0 ** -23).all()


def test_norm_rows_that_are_special():
    g = gen(1)
    x = normal(g, 6, 128, dtype=torch.bfloat16)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    y, _ = tb.rms_norm(x, w)
    q, scale, _ = tb.rms_norm_fp8(x, w)
    assert (y[1] == 0).all() and (q[1].float() == 0).all() and scale[1] == 0
    assert torch.isnan(y[2]).all() and torch.isnan(q[2].float()).all()
    assert torch.isnan(y[3, 7]) and (y[3, :7] == 0).all()
    for i in (0, 4, 5):
        want, _ = R.norm(x[i:i + 1], w, None, 1e-6)
        near(y[i:i + 1], want, want.abs(), torch.bfloat16, terms=150)
    y, h = tb.rms_norm(x[:0], w, x[:0])
    assert y.shape == (0, 128) and h.shape == (0, 128)
    y, _ = tb.rms_norm(x[4:].reshape(1, 2, 128), w)
    assert y.shape == (1, 2, 128)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,width", [(0, 64), (1, 1), (1, 64), (5, 7), (700, 1000), (33, 1001), (3000, 1536),
                                        (40, 16384), (4000, 128), (5, 9999)])
@pytest.mark.parametrize("passing", [False, True])
def test_norm_backward(dtype, rows, width, passing):
    g = gen(rows * 3 + width)
    h = normal(g, rows, width, dtype=dtype, scale=2.0)
    dy = normal(g, rows, width + 8, dtype=dtype)[:, :width]
    dh = normal(g, rows, width, dtype=dtype) if passing else None
    w = normal(g, width, dtype=dtype)
    dx, dw = tb.rms_norm_backward(dy, h, w, dh, eps=1e-5)
    want, wantw, size, sizew = R.norm_backward(dy, h, w, dh, 1e-5)
    near(dx, want, size, dtype, terms=3 * width + 30, what="dx")
    near(dw, wantw, sizew, dtype, terms=rows + width + 30, what="dweight")
    again = tb.rms_norm_backward(dy, h, w, dh, eps=1e-5)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,width", [(700, 1001), (613, 5819), (40, 8191), (3, 16381), (1300, 40), (5000, 8), (700, 3)])
def test_norm_of_rows_that_start_anywhere(dtype, rows, width):
    """Dense rows of odd widths, from narrower than a warp to as wide as they may be."""
    g = gen(rows + width)
    x, r, dy = (normal(g, rows, width, dtype=dtype, scale=s) for s in (2.0, 3.0, 1.0))
    w = normal(g, width, dtype=dtype)
    for res in (None, r):
        y, h = tb.rms_norm(x, w, res, eps=1e-5)
        want, sum_ = R.norm(x, w, res, 1e-5)
        near(y, want, want.abs(), dtype, terms=width + 16, what="y")
        if res is not None:
            near(h, sum_, sum_.abs(), dtype, terms=2, what="h")
        q, scale, _ = tb.rms_norm_fp8(x, w, res, eps=1e-5)
        top = want.abs().amax(-1) / 448
        assert ((scale.double() - top).abs() <= (width + 20) * 2.0 ** -24 * top).all()
        back, real = q.double(), want / top[:, None].clamp(min=1e-300)
        assert ((back - real).abs() <= 2.0 ** -4 * real.abs().clamp(min=2.0 ** -6) * (1 + 1e-3) + (width + 40) * 2.0 ** -23).all()
        dx, dw = tb.rms_norm_backward(dy, x, w, res, eps=1e-5)
        want, wantw, size, sizew = R.norm_backward(dy, x, w, res, 1e-5)
        near(dx, want, size, dtype, terms=3 * width + 30, what="dx")
        near(dw, wantw, sizew, dtype, terms=rows + width + 30, what="dweight")
        again = tb.rms_norm_backward(dy, x, w, res, eps=1e-5)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_norm_gradient_against_differences():
    g = gen(3)
    x, r, w = (normal(g, 40, 96, scale=2.0), normal(g, 40, 96), normal(g, 96))
    dy, dh = normal(g, 40, 96), normal(g, 40, 96)
    inputs = [t.clone().requires_grad_() for t in (x, w, r)]
    y, h = tb.rms_norm(*inputs)
    ((y * dy).sum() + (h * dh).sum()).backward()
    for i, t in enumerate((x, w, r)):
        step = normal(g, *t.shape)
        sides = []
        for e in (1e-4, -1e-4):
            a = [x.double(), w.double(), r.double()]
            a[i] = a[i] + e * step.double()
            y, h = R.norm(a[0], a[1], a[2], 1e-6)
            sides.append((y * dy.double()).sum() + (h * dh.double()).sum())
        want = (sides[0] - sides[1]) / 2e-4
        got = (inputs[i].grad.double() * step.double()).sum()
        size = (inputs[i].grad.double() * step.double()).abs().sum()
        assert abs(got - want) <= 1e-5 * size  # 400 roundings of 2^-24, and the difference's own 1e-8


# -------------------------------------------------------------------------------------------------- linear attention

def attention_inputs(seed, lengths, heads, key, value, dtype, state=True, decay=None, pad=0):
    g = gen(seed)
    n = sum(lengths)
    qkv = normal(g, n, heads * (2 * key + value) + pad, dtype=dtype)[:, :heads * (2 * key + value)]
    q, k, v = (x.unflatten(1, (heads, -1)) for x in qkv.split([heads * key, heads * key, heads * value], 1))
    ends = torch.tensor([0] + list(lengths), device="cuda").cumsum(0)
    if decay is None:
        decay = [1 - 2.0 ** -(1 + 9 * h / max(1, heads - 1)) for h in range(heads)]
    s = normal(g, len(lengths), heads, key, value) if state else None
    ds = normal(g, len(lengths), heads, key, value) if state else None
    do = normal(g, n, heads, value, dtype=dtype)
    return q, k, v, torch.tensor(decay, dtype=torch.float32, device="cuda"), ends, s, do, ds


def check_attention(lengths, heads, key, value, dtype, state, decay=None, seed=0, pad=0, scale=0.37):
    q, k, v, decay, ends, s, do, ds = attention_inputs(seed, lengths, heads, key, value, dtype, state, decay, pad)
    o, last = tb.linear_attention(q, k, v, decay, ends, state=s, scale=scale, return_state=True)
    grads = tb.linear_attention_backward(do, q, k, v, decay, ends, state=s, scale=scale, dstate=ds)
    want = R.attention(q, k, v, decay, lengths, s, scale, do, ds)
    size = R.attention_sizes(q, k, v, decay, lengths, s, scale, do, ds)
    # products, sums over the head and over the rows, and the powers of the decay
    terms = 2 * (max(key, value) + max(lengths, default=0) + 64)
    rounds = 3 if dtype == torch.bfloat16 else 0
    names = ["o", "last", "dq", "dk", "dv", "dstate"]
    got = [o, last, *grads]
    for name, x, y, z in zip(names, got, want, size):
        if x is None:
            assert name == "dstate" and s is None
            continue
        kind = torch.float32 if name in ("last", "dstate") else dtype
        near(x, y, z, kind, terms=terms, roundings=0 if kind == torch.float32 else rounds, what=name)
        if x.numel() >= 4096 and kind == torch.bfloat16:
            # four independent roundings of root mean square at most u / sqrt(3) each
            rel = ((x.double() - y).norm() / y.norm()).item()
            assert rel <= 2 * 2.0 ** -8 / math.sqrt(3), "%s: %.3g" % (name, rel)
    return got


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("key,value", [(64, 64), (128, 128), (40, 72), (128, 64), (1, 3), (33, 17), (96, 128), (8, 8)])
@pytest.mark.parametrize("state", [False, True])
def test_attention_head_sizes(dtype, key, value, state):
    check_attention([70, 0, 1, 129, 64], 2, key, value, dtype, state, seed=key + value)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("lengths", [[1], [2], [63], [64], [65], [127], [128], [0], [0, 0, 5], [3, 0], [200, 1, 1, 64, 0],
                                     [1] * 70, [1000, 37]], ids=str)
def test_attention_lengths(dtype, lengths):
    check_attention(lengths, 3, 64, 64, dtype, True, seed=len(lengths))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("key,value", [(64, 64), (128, 128)])
def test_attention_decays(dtype, key, value):
    """No decay, no memory, a decay that underflows within a few rows, and ordinary ones."""
    check_attention([300, 77], 6, key, value, dtype, True, decay=[1.0, 0.0, 1e-30, 0.5, 0.97, 0.9999], seed=9)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("lengths", [[5000], [0, 4001, 3, 1200]], ids=str)
def test_attention_split_along_the_rows(dtype, lengths):
    """Few heads and long grids: the walk is cut into segments."""
    check_attention(lengths, 1, 64, 64, dtype, True, seed=2, decay=[0.9995])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_attention_strides(dtype):
    """Rows of a packed projection whose stride is no multiple of 16 bytes."""
    check_attention([90, 40], 2, 64, 64, dtype, False, pad=3)


def test_attention_defaults():
    q, k, v, decay, _, _, do, _ = attention_inputs(5, [150], 2, 64, 64, torch.bfloat16, False)
    o, none = tb.linear_attention(q, k, v, decay)
    assert none is None
    ends = torch.tensor([0, 150], device="cuda")
    same, _ = tb.linear_attention(q, k, v, decay, ends, scale=64 ** -0.5)
    assert torch.equal(o, same)
    a = tb.linear_attention_backward(do, q, k, v, decay)
    b = tb.linear_attention_backward(do, q, k, v, decay, ends, scale=64 ** -0.5)
    assert a[3] is None and all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
    empty = torch.empty(0, 2, 64, device="cuda")
    o, last = tb.linear_attention(empty, empty, empty, decay, torch.zeros(1, dtype=torch.int64, device="cuda"),
                                  return_state=True)
    assert o.shape == (0, 2, 64) and last.shape == (0, 2, 64, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_attention_keeps_what_is_not_finite_where_it_belongs(dtype):
    """A NaN or infinity reaches its own grid's outputs from its row on, and no others."""
    lengths = [100, 77, 50]
    q, k, v, decay, ends, s, do, _ = attention_inputs(8, lengths, 2, 64, 64, dtype)
    clean, _ = tb.linear_attention(q, k, v, decay, ends, state=s, return_state=True)
    for x, bad in ((k, float("nan")), (v, float("inf")), (q, float("nan"))):
        y = x.clone()
        y[100 + 30, 1, 3] = bad
        args = [y if t is x else t for t in (q, k, v)]
        o, last = tb.linear_attention(*args, decay, ends, state=s, return_state=True)
        others = torch.ones(227, 2, dtype=torch.bool, device="cuda")
        others[130:177, 1] = False
        assert torch.equal(o[others], clean[others])
        assert not torch.isfinite(o[130, 1]).all()
        if x is q:
            assert torch.isfinite(last).all() and torch.isfinite(o[131:]).all()
        else:
            assert not torch.isfinite(last[1, 1]).all()
            assert torch.isfinite(last[[0, 2]]).all() and torch.isfinite(last[1, 0]).all()


def test_attention_gradient_against_differences():
    lengths = [50, 0, 21]
    q, k, v, decay, ends, s, do, ds = attention_inputs(11, lengths, 2, 24, 40, torch.float32)
    inputs = [x.contiguous().clone().requires_grad_() for x in (q, k, v, s)]
    o, last = tb.linear_attention(inputs[0], inputs[1], inputs[2], decay, ends, state=inputs[3], scale=0.2, return_state=True)
    ((o * do).sum() + (last * ds).sum()).backward()
    g = gen(12)
    for i in range(4):
        step = normal(g, *inputs[i].shape).double()
        sides = []
        for e in (1e-4, -1e-4):
            a = [x.detach().double() for x in inputs]
            a[i] = a[i] + e * step
            o, last = R.attention(a[0], a[1], a[2], decay, lengths, a[3], 0.2)
            sides.append((o * do.double()).sum() + (last * ds.double()).sum())
        want = (sides[0] - sides[1]) / 2e-4
        got = (inputs[i].grad.double() * step).sum()
        size = (inputs[i].grad.double() * step).abs().sum()
        assert abs(got - want) <= 2e-5 * size  # 300 roundings of 2^-24, and the difference's own


def test_autograd_of_a_block():
    """The three operators in one graph; the gradients of shared heads sum."""
    g = gen(13)
    x = normal(g, 120, 64, dtype=torch.bfloat16).requires_grad_()
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    pos = torch.arange(120, dtype=torch.int32, device="cuda")
    f = tb.rotary_frequencies(32)
    decay = torch.tensor([0.9, 0.99], device="cuda")
    y, h = tb.rms_norm(x, w, x.detach() * 0.5)
    q, k = tb.rotary(y.view(120, 2, 32), y.view(120, 2, 32)[:, :1], pos, f)
    o, _ = tb.linear_attention(q, k.expand(120, 2, 32), y.view(120, 2, 32), decay)
    (o.float().sum() + h.float().sum()).backward()
    assert x.grad.shape == x.shape and torch.isfinite(x.grad).all() and x.grad.abs().sum() > 0
    assert torch.isfinite(w.grad).all() and w.grad.abs().sum() > 0
    q, none = tb.rotary(x.view(120, 2, 32), None, pos, f)
    assert none is None and q.requires_grad


# -------------------------------------------------------------------------------------------------------------- step

@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("streams,heads,key,value", [(1, 1, 1, 1), (2, 8, 64, 64), (3, 2, 128, 128), (5, 3, 40, 72),
                                                     (2, 2, 33, 17), (1, 2, 256, 256), (4, 1, 200, 250)])
def test_step(dtype, streams, heads, key, value):
    g = gen(key + value)
    q, k, v = (normal(g, streams, heads, n + 5, dtype=dtype)[..., :n] for n in (key, key, value))
    state = normal(g, streams, heads, key, value)
    decay = torch.linspace(0, 1, heads, device="cuda")
    before = state.clone()
    o = tb.linear_attention_step(q, k, v, decay, state, scale=0.5)
    n = [1] * streams
    want = R.attention(q, k, v, decay, n, before, 0.5)
    size = R.attention_sizes(q, k, v, decay, n, before, 0.5)
    near(o, want[0], size[0], dtype, terms=key + 16, what="o")
    near(state, want[1], size[1], torch.float32, terms=4, what="state")


def test_step_slots():
    g = gen(6)
    q, k, v = (normal(g, 4, 2, 64, dtype=torch.bfloat16) for _ in range(3))
    states = normal(g, 6, 2, 64, 64)
    before = states.clone()
    decay = torch.tensor([0.5, 0.9], device="cuda")
    slots = torch.tensor([5, -1, 6, 0], dtype=torch.int32, device="cuda")
    o = tb.linear_attention_step(q, k, v, decay, states, slots=slots)
    want = R.attention(q[[0, 3]], k[[0, 3]], v[[0, 3]], decay, [1, 1], before[[5, 0]], 64 ** -0.5)
    size = R.attention_sizes(q[[0, 3]], k[[0, 3]], v[[0, 3]], decay, [1, 1], before[[5, 0]], 64 ** -0.5)
    near(o[[0, 3]], want[0], size[0], torch.bfloat16, terms=80)
    near(states[[5, 0]], want[1], size[1], torch.float32, terms=4)
    assert (o[1:3] == 0).all() and torch.equal(states[1:5], before[1:5])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_steps_follow_the_prompt(dtype):
    """A prompt in one call and its last rows token by token give the same."""
    q, k, v, decay, ends, s, _, _ = attention_inputs(21, [40, 40], 2, 64, 64, dtype)
    o, last = tb.linear_attention(q, k, v, decay, ends, state=s, return_state=True)
    cut = torch.tensor([0, 30, 60], device="cuda")
    rows = torch.cat([torch.arange(30), torch.arange(40, 70)]).cuda()
    part, state = tb.linear_attention(q[rows], k[rows], v[rows], decay, cut, state=s, return_state=True)
    size = R.attention_sizes(q, k, v, decay, [40, 40], s, 0.125)
    rounds = 6 if dtype == torch.bfloat16 else 0  # two results, three roundings each
    near(part, o[rows].double(), size[0][rows], dtype, terms=500, roundings=rounds)
    for t in range(30, 40):
        at = torch.tensor([t, 40 + t], device="cuda")
        got = tb.linear_attention_step(q[at], k[at], v[at], decay, state)
        near(got, o[at].double(), size[0][at] + o[at].double().abs(), dtype, terms=500,
             roundings=rounds + 1 if rounds else 2.0 ** -2 if dtype == torch.float16 else 0)
    near(state, last.double(), size[1], torch.float32, terms=500)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_rows_past_32_bits(dtype):
    """Rows of one buffer of more than 2^31 elements give what the same rows give by themselves."""
    g = gen(8)
    rows, stride = 36000, 60008
    wide = torch.empty(rows, stride, device="cuda", dtype=dtype)
    assert wide.numel() > 2 ** 31
    parts = []
    for i in range(4):  # q, k, v and an output gradient of two heads, near the ends of the rows
        part = normal(g, rows, 2, 64, dtype=dtype)
        view = wide[:, stride - 128 * (i + 1):stride - 128 * i].unflatten(1, (2, 64))
        view.copy_(part)
        parts.append((part, view))
    decay = torch.tensor([0.9, 0.99], device="cuda")
    ends = torch.tensor([0, 20000, 20000, rows], device="cuda")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    f, w = tb.rotary_frequencies(64), normal(g, 64, dtype=dtype)

    def every(q, k, v, do):
        return [*tb.rotary(q, k, pos, f), tb.rms_norm(q[:, 1], w)[0], *tb.rms_norm_backward(do[:, 1], q[:, 1], w),
                tb.linear_attention(q, k, v, decay, ends)[0],
                *(x for x in tb.linear_attention_backward(do, q, k, v, decay, ends) if x is not None)]

    for x, y in zip(every(*(p for p, _ in parts)), every(*(v for _, v in parts))):
        assert torch.equal(x, y)


# ------------------------------------------------------------------------------------------- streams, graphs, refusals

def test_streams_and_graphs():
    q, k, v, decay, ends, s, do, _ = attention_inputs(31, [3000, 500], 2, 64, 64, torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(3500, dtype=torch.int32, device="cuda")
    f = tb.rotary_frequencies(64)

    def block(stream=None):
        a, b = tb.rotary(q, k, pos, f, stream=stream)
        o, last = tb.linear_attention(a, b, v, decay, ends, state=s, return_state=True, stream=stream)
        grads = tb.linear_attention_backward(do, a, b, v, decay, ends, state=s, stream=stream)
        y, _ = tb.rms_norm(o, w, stream=stream)
        dy, dw = tb.rms_norm_backward(do, o, w, stream=stream)
        return [o, last, y, dy, dw, *grads]

    want = block()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = block(side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block()
    for x in outs:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, outs))


def test_refusals():
    x = torch.randn(8, 2, 64, device="cuda")
    f = tb.rotary_frequencies(64)
    pos = torch.arange(8, dtype=torch.int32, device="cuda")
    decay = torch.ones(2, device="cuda")
    w = torch.ones(64, device="cuda")
    ends = torch.tensor([0, 8], device="cuda")
    state = torch.zeros(1, 2, 64, 64, device="cuda")
    bad = [
        lambda: tb.rotary(x.double(), None, pos, f),
        lambda: tb.rotary(x, x.bfloat16(), pos, f),
        lambda: tb.rotary(x, x[:7], pos, f),
        lambda: tb.rotary(x, None, pos[:7], f),
        lambda: tb.rotary(x, None, pos.float(), f),
        lambda: tb.rotary(x, None, pos, f.int()),
        lambda: tb.rotary(x, None, pos, tb.rotary_frequencies(66)),
        lambda: tb.rotary(x, None, pos, f, layout="quarter"),
        lambda: tb.rotary(x, None, pos[:, None].expand(8, 3), f, sections=(30, 1, 2)),
        lambda: tb.rotary(x[:1].expand(8, 2, 64), None, pos, f, inplace=True),
        lambda: tb.rotary(torch.randn(8, 2, 300, device="cuda"), None, pos, f),
        lambda: tb.rotary(x.requires_grad_(), None, pos, f, inplace=True),
        lambda: tb.rotary_frequencies(63),
        lambda: tb.rotary_frequencies(64, scaling="twice"),
        lambda: tb.rms_norm(x, w.bfloat16()),
        lambda: tb.rms_norm(x, w[:63]),
        lambda: tb.rms_norm(x, w, x[:7]),
        lambda: tb.rms_norm(torch.zeros(2, 16385, device="cuda"), torch.zeros(16385, device="cuda")),
        lambda: tb.rms_norm(x.int(), w),
        lambda: tb.rms_norm_fp8(x, w),  # x asks for a gradient by now
        lambda: tb.rms_norm_backward(x[:7], x, w),
        lambda: tb.linear_attention(x, x, x, decay.double()),
        lambda: tb.linear_attention(x, x, x, decay[:1]),
        lambda: tb.linear_attention(x, x[:, :, :32], x, decay),
        lambda: tb.linear_attention(x, x, x, decay, ends.int()),
        lambda: tb.linear_attention(x, x, x, decay, ends.cpu()),
        lambda: tb.linear_attention(x, x, x, decay, ends, state=state[:, :1]),
        lambda: tb.linear_attention(x, x, x, decay, ends, state=state.bfloat16()),
        lambda: tb.linear_attention(x, x, x, decay.clone().requires_grad_()),
        lambda: tb.linear_attention(*(torch.zeros(4, 1, 129, device="cuda") for _ in range(3)), decay[:1]),
        lambda: tb.linear_attention_step(x, x, x, decay, state),  # one state for eight streams
        lambda: tb.linear_attention_step(x.detach(), x.detach(), x.detach(), decay, state),
        lambda: tb.linear_attention_step(x.detach(), x.detach(), x.detach(), decay, state.expand(8, 2, 64, 64)),
        lambda: tb.linear_attention_step(x.detach(), x.detach(), x.detach(), decay, state, slots=pos.long()),
        lambda: tb.linear_attention(x.cpu(), x.cpu(), x.cpu(), decay.cpu()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(tb.TBError):
            call()
            print("refusal %d did not come" % i)
    assert torch.cuda.current_stream().query() or True
    torch.cuda.synchronize()


def test_offsets_outside_the_rows_are_clamped():
    """Offsets that reach past the rows (or before them) read and write none outside."""
    q, k, v, decay, _, _, _, _ = attention_inputs(41, [64], 1, 64, 64, torch.bfloat16)
    o, _ = tb.linear_attention(q, k, v, decay, torch.tensor([-5, 64, 1 << 40], device="cuda"))
    want, _ = tb.linear_attention(q, k, v, decay)
    assert torch.equal(o, want)


def test_the_example_learns_and_walks():
    """examples/voxel_sequence.py: the operators together, in training and voxel by voxel."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "voxel_sequence.py")
    spec = importlib.util.spec_from_file_location("voxel_sequence", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, off_by = example.run(steps=30, say=None)
    assert all(math.isfinite(x) for x in losses) and losses[-1] < 0.9 * losses[0]
    # two paths through two blocks in bfloat16: outputs of size one, a few units of 2^-8 each
    assert off_by <= 16 * 2.0 ** -8


def test_example_coordinates_are_the_batch_order():
    import importlib.util
    import os

    import numpy as np
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "voxel_sequence.py")
    spec = importlib.util.spec_from_file_location("voxel_sequence", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    ijk = np.array([[9, 0, 0], [0, 0, 1], [0, 0, 0], [-1, 2, 3], [5, 5, 5]], np.int32)
    b = tb.from_ijk(torch.from_numpy(ijk).cuda(), torch.tensor([0, 3, 3, 5]).cuda())
    at, offsets = example.voxel_coordinates(b)
    assert offsets.tolist() == [0, 3, 3, 5]
    assert at.tolist() == [[0, 0, 0], [0, 0, 1], [9, 0, 0], [-1, 2, 3], [5, 5, 5]]
