"""The sequence operators on the GPU where their inputs are at an edge."""
import ctypes
import threading

import pytest

from tests import _seq_reference as R
from tests.test_seq_abi import NORM

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_voxel_grid_leaf_gb300 as tb  # noqa: E402
from tests.test_seq_gpu import attention_inputs, gen, near, normal  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


# -------------------------------------------------------------------------------------------------- very small values

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("rows,width", [(5, 128), (700, 128), (3, 77), (700, 777), (4, 5001)], ids=str)
@pytest.mark.parametrize("residual", [False, True])
def test_fp8_norm_of_very_small_rows(dtype, rows, width, residual):
    """Rows whose largest h w is far below the reciprocal of the largest number: zeros stay zero and the others keep
    their places between 0 and 448.  The magnitudes stay normal numbers, so the bounds are those of any row."""
    g = gen(rows + width)
    x = torch.rand(rows, width, generator=g, device="cuda") * 0.9 + 0.1
    x = x * torch.where(torch.rand(rows, width, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    small = torch.tensor([2.0 ** -122, 2.0 ** -119, 2.0 ** -121, 2.0 ** -110, 1.0], device="cuda")
    x = (x * small[torch.arange(rows, device="cuda") % 5][:, None]).to(dtype)
    x[:, ::3] = 0
    w = (torch.rand(width, generator=g, device="cuda") * 7 + 1).to(dtype)
    r = torch.zeros_like(x) if residual else None
    q, scale, _ = tb.rms_norm_fp8(x, w, r, eps=1e-6)
    want, _ = R.norm(x, w, r, 1e-6)
    top = want.abs().amax(-1) / 448
    assert ((scale.double() - top).abs() <= (width + 20) * 2.0 ** -24 * top + 2.0 ** -149).all()
    back, real = q.double(), want / top[:, None]
    assert (back[:, ::3] == 0).all()
    assert ((back - real).abs() <= 2.0 ** -4 * real.abs().clamp(min=2.0 ** -6) * (1 + 1e-3) + (width + 40) * 2.0 ** -23).all()


@pytest.mark.parametrize("width", [128, 77])
def test_fp8_norm_of_one_tiny_element(width):
    """A row of zeros with one element: 448 there, of its sign, and zeros; also where the element is subnormal and
    where weights of zeros are large."""
    x = torch.zeros(4, width, device="cuda")
    x[0, 3], x[1, 3], x[2, 5], x[3, 6] = 1e-37, -1e-37, 1e-42, -2.0 ** -149
    w = torch.ones(width, device="cuda")
    w[10] = 1e38
    q, scale, _ = tb.rms_norm_fp8(x, w)
    want = torch.zeros(4, width, device="cuda")
    want[0, 3], want[1, 3], want[2, 5], want[3, 6] = 448, -448, 448, -448
    assert torch.equal(q.float(), want)
    assert torch.isfinite(scale).all() and (scale >= 0).all()
    assert ((scale[:2].double() - 1e-37 * 1e3 / 448).abs() <= 1e-6 * 1e-34 / 448).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("rows,width", [(5, 128), (700, 128), (3, 77), (700, 777)], ids=str)
@pytest.mark.parametrize("eps", [0.0, 1e-30])
def test_norm_gradient_of_small_rows(dtype, rows, width, eps):
    """1 / the root mean square of a row may be far above the cube root of the largest number."""
    g = gen(width)
    h, dy = normal(g, rows, width, dtype=dtype, scale=1e-14), normal(g, rows, width, dtype=dtype)
    w = normal(g, width, dtype=dtype)
    dx, dw = tb.rms_norm_backward(dy, h, w, eps=eps)
    want, wantw, size, sizew = R.norm_backward(dy, h, w, None, eps)
    near(dx, want, size, dtype, terms=3 * width + 30, what="dx")
    near(dw, wantw, sizew, dtype, terms=rows + width + 30, what="dweight")


# ------------------------------------------------------------------------------------------- rows that no grid covers

def poisoned(*shapes_and_types):
    """Leaves NaN in memory that the allocator hands out next."""
    for shape, dtype in shapes_and_types * 2:
        torch.full(shape, float("nan"), dtype=dtype, device="cuda")


UNCOVERED = [([3, 50], 64), ([0, 20, 41], 64), ([10, 10, 64], 64), ([5, 5, 5], 33), ([70, 90], 64), ([-9, 30], 64),
             ([2, 9, 17, 20], 30), ([700, 4000], 6000), ([1, 3000], 3001)]


@pytest.mark.parametrize("dtype,key,value,pad", [
    (torch.bfloat16, 64, 64, 0), (torch.bfloat16, 128, 128, 0), (torch.bfloat16, 64, 64, 3), (torch.float16, 128, 64, 0),
    (torch.float32, 40, 72, 0), (torch.float32, 33, 17, 1)], ids=str)
@pytest.mark.parametrize("offsets,tokens", UNCOVERED, ids=str)
def test_rows_of_no_grid_are_zeros(dtype, key, value, pad, offsets, tokens):
    """Outputs and gradients of rows before the first offset and past the last one are zeros; those of the grids are
    the recurrence's.  Three heads: an ordinary one, one without memory, a pair's lone second half."""
    heads, scale = 3, 0.4
    q, k, v, decay, _, _, do, _ = attention_inputs(tokens, [tokens], heads, key, value, dtype, False,
                                                   [0.97, 0.0, 0.9], pad)
    off = torch.tensor(offsets, device="cuda")
    shapes = [((tokens, heads, n), dtype) for n in (key, key, value)]
    poisoned(*shapes)
    o, _ = tb.linear_attention(q, k, v, decay, off, scale=scale)
    poisoned(*shapes)
    dq, dk, dv, _ = tb.linear_attention_backward(do, q, k, v, decay, off, scale=scale)
    ends = [min(max(x, 0), tokens) for x in offsets]
    inside = slice(ends[0], ends[-1])
    lengths = [b - a for a, b in zip(ends, ends[1:])]
    args = (q[inside], k[inside], v[inside], decay, lengths, None, scale, do[inside])
    want, size = R.attention(*args), R.attention_sizes(*args)
    terms = 2 * (max(key, value) + max(lengths) + 64)
    for name, x, i in (("o", o, 0), ("dq", dq, 2), ("dk", dk, 3), ("dv", dv, 4)):
        outside = torch.cat([x[:ends[0]], x[ends[-1]:]])
        assert (outside == 0).all(), name
        near(x[inside], want[i], size[i], dtype, terms=terms, roundings=3 if dtype == torch.bfloat16 else 0, what=name)


def test_padding_rows_do_not_reach_a_weight():
    """A buffer of a fixed capacity: what lies past the last grid is no part of the projection's gradient."""
    g = gen(3)
    x, w = normal(g, 4096, 32), normal(g, 32, 192).requires_grad_()
    decay = torch.tensor([0.9], device="cuda")
    grads = []
    for n in (4096, 1000):
        rows = x[:n]
        poisoned(*[((n, 1, 64), torch.float32)] * 4)
        q, k, v = (rows @ w).unflatten(1, (3, 1, 64)).unbind(1)
        o, _ = tb.linear_attention(q, k, v, decay, torch.tensor([0, 400, 1000], device="cuda"))
        grad, = torch.autograd.grad((o * 0.01).square().sum(), w)
        grads.append(grad)
    assert torch.isfinite(grads[0]).all()
    size = grads[1].abs().max()
    # 1000 roundings of 2^-24, of terms whose magnitudes add up to some sqrt(1000) times their sum
    assert ((grads[0] - grads[1]).abs() <= 2e-3 * size).all()


# --------------------------------------------------------------------------------------------------------- infinities

@pytest.mark.parametrize("dtype,key,value", [(torch.bfloat16, 64, 64), (torch.bfloat16, 128, 128),
                                             (torch.float16, 64, 64), (torch.float32, 96, 64)], ids=str)
@pytest.mark.parametrize("scale", [0.5, -0.5, 0.0])
def test_sign_of_infinity(dtype, key, value, scale):
    """One infinite element among positive ones: what it reaches has the scale's sign (NaN for a scale of zero)."""
    g = gen(key)
    q, k, v, do = (torch.rand(64, 2, n, generator=g, device="cuda").add(0.5).to(dtype) for n in (key, key, value, value))
    decay, ends = torch.tensor([0.9, 0.99], device="cuda"), torch.tensor([0, 64], device="cuda")
    first = torch.zeros(1, 2, key, value, device="cuda")

    def reached(x):
        assert (torch.isnan(x) if scale == 0 else x == (float("inf") if scale > 0 else -float("inf"))).all()

    bad = v.clone()
    bad[20, 1, 3] = float("inf")
    o, last = tb.linear_attention(q, k, bad, decay, ends, scale=scale, return_state=True)
    reached(o[20:, 1, 3])
    assert torch.isfinite(o[:20]).all() and torch.isfinite(o[:, 0]).all() and torch.isfinite(o[:, 1, :3]).all()
    assert (last[0, 1, :, 3] == float("inf")).all() and torch.isfinite(last[0, 0]).all()
    bad = do.clone()
    bad[20, 1, 3] = float("inf")
    dq, dk, dv, dfirst = tb.linear_attention_backward(bad, q, k, v, decay, ends, state=first, scale=scale)
    reached(dv[:21, 1, 3])
    assert torch.isfinite(dv[21:]).all() and torch.isfinite(dv[:, 0]).all()
    reached(dfirst[0, 1, :, 3])
    bad = q.clone()
    bad[20, 1, 3] = float("inf")
    dq, dk, dv, _ = tb.linear_attention_backward(do, bad, k, v, decay, ends, state=first, scale=scale)
    reached(dk[:21, 1, 3])
    assert torch.isfinite(dk[21:]).all() and torch.isfinite(dk[:, 0]).all()


# ------------------------------------------------------------------------------------------------------------- states

def test_step_of_states_at_any_element():
    """Contiguous states that start off a 16-byte boundary, as a slice of a pool does for odd sizes."""
    g = gen(5)
    pool = normal(g, 4, 3, 5, 7)
    q, k, v = (normal(g, 3, 3, n) for n in (5, 5, 7))
    decay = torch.tensor([0.5, 0.9, 1.0], device="cuda")
    before, state = pool.clone(), pool[1:]
    assert state.data_ptr() % 16
    o = tb.linear_attention_step(q, k, v, decay, state, scale=0.5)
    want = R.attention(q, k, v, decay, [1, 1, 1], before[1:], 0.5)
    size = R.attention_sizes(q, k, v, decay, [1, 1, 1], before[1:], 0.5)
    near(o, want[0], size[0], torch.float32, terms=24)
    near(state, want[1], size[1], torch.float32, terms=4)
    assert torch.equal(pool[0], before[0])


# -------------------------------------------------------------------------------------------------- several host threads

def test_two_threads_of_different_widths():
    """Widths whose kernels take different amounts of shared memory, from two host threads at once."""
    lib = tb.lib()
    failed, start = [], threading.Barrier(2)

    def go(width):
        stream = torch.cuda.Stream()
        x, w = torch.randn(700, width, device="cuda").bfloat16(), torch.ones(width, device="cuda").bfloat16()
        y = torch.empty_like(x)
        args = NORM.pack(x.data_ptr(), 0, w.data_ptr(), y.data_ptr(), 0, 0, 700, width, 0, width, 0, width, 2, 0, 1e-6)
        torch.cuda.synchronize()
        start.wait()
        for _ in range(20000):
            st = lib.tb_rms_norm(args, ctypes.c_void_p(stream.cuda_stream))
            if st:
                failed.append((width, st, lib.tb_last_error()))
                break
        stream.synchronize()

    threads = [threading.Thread(target=go, args=(width,)) for width in (8191, 4001)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
