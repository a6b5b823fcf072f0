"""Linear attention where the call is split along the rows, or its grids are
taken in the order of their lengths: each kernel, head size, type and kind of
decay against the recurrence in 64 bits."""
import pytest

from tests import _seq_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import ctypes  # noqa: E402

import sparse_voxel_grid_leaf_gb300 as tb  # noqa: E402
from tests.test_seq_gpu import TYPES, attention_inputs, near  # noqa: E402

CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def is_split(tokens, grids, heads, key, value, dtype, backward):
    """Whether the library cuts such a call into segments: only then it asks for a workspace."""
    f = tb.lib().tb_linear_attention_workspace
    f.restype = ctypes.c_int64
    return f(ctypes.c_int64(tokens), grids, heads, key, value, CODE[dtype], backward) > 0


def compare(lengths, heads, key, value, dtype, state, decay, split, pad=0, scale=0.3):
    """Outputs with and without the states that come out, and all gradients."""
    for backward in (0, 1):
        assert is_split(sum(lengths), len(lengths), heads, key, value, dtype, backward) == split[backward]
    q, k, v, d, ends, s, do, ds = attention_inputs(sum(lengths) + key, lengths, heads, key, value, dtype, state, decay, pad)
    want = R.attention(q, k, v, d, lengths, s, scale, do, ds)
    size = R.attention_sizes(q, k, v, d, lengths, s, scale, do, ds)
    o, last = tb.linear_attention(q, k, v, d, ends, state=s, scale=scale, return_state=True)
    alone, _ = tb.linear_attention(q, k, v, d, ends, state=s, scale=scale)
    dq, dk, dv, first = tb.linear_attention_backward(do, q, k, v, d, ends, state=s, scale=scale, dstate=ds)
    # products, sums over the head and over the rows, and the powers of the decay; in bfloat16 three operands of 16 bits
    terms = 2 * (max(key, value) + max(lengths) + 64)
    rounds = 3 if dtype == torch.bfloat16 else 0
    for name, x, i in (("o", o, 0), ("o alone", alone, 0), ("last", last, 1), ("dq", dq, 2), ("dk", dk, 3), ("dv", dv, 4),
                       ("first", first, 5)):
        if x is None:
            assert name == "first" and s is None
        elif i in (1, 5):
            near(x, want[i], size[i], torch.float32, terms=terms, what=name)
        else:
            near(x, want[i], size[i], dtype, terms=terms, roundings=rounds, what=name)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("key,value", [(64, 64), (128, 128), (128, 40), (40, 72), (33, 17)])
@pytest.mark.parametrize("state", [False, True])
def test_one_grid_in_segments(dtype, key, value, state):
    """Heads of every size, three of them (a pair and a lone one), with no memory, a steep decay and a long one."""
    compare([1901], 3, key, value, dtype, state, [0.0, 0.5, 0.9995], (True, True))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("key,value", [(64, 64), (128, 128), (33, 17)])
def test_unequal_grids_in_segments(dtype, key, value):
    """Empty grids, one shorter than a segment, one of whole segments, and rows of an odd stride."""
    compare([1900, 1, 0, 1536], 2, key, value, dtype, True, [0.3, 0.998], (True, True))
    compare([1900, 1, 0, 1536], 2, key, value, dtype, False, [0.6, 1.0], (True, True), pad=3)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("key,value", [(64, 64), (128, 128)])
def test_steep_decays_in_segments(dtype, key, value):
    """Heads that go by the recurrence, alone and next to one that goes by chunks."""
    compare([1100], 4, key, value, dtype, True, [0.1, 0.33, 0.35, 1e-30], (True, True))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("key,value", [(64, 64), (96, 128)])
def test_grids_in_the_order_of_their_lengths(dtype, key, value):
    """More walks than multiprocessors over unequal grids, two of them empty, some of the same length."""
    lengths = [(37 * i * i + 11 * i) % 97 for i in range(41)] + [0, 0, 130, 130, 64]
    compare(lengths, 8, key, value, dtype, True, None, (False, False))
