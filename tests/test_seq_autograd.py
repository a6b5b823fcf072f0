"""What torch's autograd is told of the sequence operators."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import torch.autograd.forward_ad as fwAD  # noqa: E402

import sparse_voxel_grid_leaf_gb300 as tb  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def rows(n=24, heads=2, dim=64):
    return torch.randn(n, heads, dim, device="cuda")


def calls():
    """Each differentiable call as a function of one tensor [24, 2, 64]."""
    pos = torch.arange(24, dtype=torch.int32, device="cuda")
    f, w = tb.rotary_frequencies(64), torch.ones(64, device="cuda")
    decay, k, v = torch.tensor([0.9, 0.99], device="cuda"), rows(), rows()
    return {"rotary": lambda x: tb.rotary(x, k, pos, f)[0],
            "rotary_alone": lambda x: tb.rotary(x, None, pos, f)[0],
            "norm": lambda x: tb.rms_norm(x, w)[0],
            "norm_residual": lambda x: tb.rms_norm(x, w, k)[0],
            "linear": lambda x: tb.linear_attention(x, k, v, decay)[0]}


NAMES = ["rotary", "rotary_alone", "norm", "norm_residual", "linear"]


@pytest.mark.parametrize("name", NAMES)
def test_second_derivatives_are_refused(name):
    """A penalty on a gradient next to another term: an error, not the other term's gradient alone."""
    call = calls()[name]
    x = rows().requires_grad_()
    grad, = torch.autograd.grad(call(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (grad.square().sum() + x.sum()).backward()


@pytest.mark.parametrize("name", NAMES)
def test_first_derivatives_with_create_graph(name):
    call = calls()[name]
    x = rows().requires_grad_()
    want, = torch.autograd.grad(call(x).square().sum(), x)
    got, = torch.autograd.grad(call(x).square().sum(), x, create_graph=True)
    assert torch.equal(got, want)


def test_backward_calls_refuse_tracked_tensors():
    x, w, decay = rows(), torch.ones(64, device="cuda"), torch.tensor([0.9, 0.99], device="cuda")
    pos, f, t = torch.arange(24, dtype=torch.int32, device="cuda"), tb.rotary_frequencies(64), rows().requires_grad_()
    state = torch.zeros(1, 2, 64, 64, device="cuda")
    bad = [lambda: tb.rotary_backward(t, x, pos, f),
           lambda: tb.rms_norm_backward(t, x, w),
           lambda: tb.rms_norm_backward(x, t, w),
           lambda: tb.rms_norm_backward(x, x, w, t),
           lambda: tb.rms_norm_backward(x, x, w.clone().requires_grad_()),
           lambda: tb.linear_attention_backward(t, x, x, x, decay),
           lambda: tb.linear_attention_backward(x, t, x, x, decay),
           lambda: tb.linear_attention_backward(x, x, x, t, decay),
           lambda: tb.linear_attention_backward(x, x, x, x, decay, state=state, dstate=state.clone().requires_grad_())]
    for call in bad:
        with pytest.raises(tb.TBError):
            call()
        with torch.no_grad():
            call()


def test_a_step_is_a_write_of_its_states():
    """States that a backward pass still needs: an error where the step has overwritten them."""
    x, decay = rows(1), torch.tensor([0.9, 0.99], device="cuda")
    state = torch.randn(1, 2, 64, 64, device="cuda")
    q = rows().requires_grad_()
    o, _ = tb.linear_attention(q, rows(), rows(), decay, torch.tensor([0, 24], device="cuda"), state=state)
    before = state._version
    tb.linear_attention_step(x, x, x, decay, state)
    assert state._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()


def test_a_turn_in_place_is_a_write():
    pos, f = torch.arange(24, dtype=torch.int32, device="cuda"), tb.rotary_frequencies(64)
    qk = rows(24, 4)
    q, k = qk[:, :2], qk[:, 2:]
    w = torch.randn(24, 2, 64, device="cuda", requires_grad=True)
    for call, inputs in ((tb.rotary, (q, k)), (tb.rotary_backward, (q, k)), (tb.rotary, (q, None)), (tb.rotary, (k, None))):
        y = w * qk[:, :2] + w * qk[:, 2:]  # saves both
        before = qk._version
        call(*inputs, pos, f, inplace=True)
        assert qk._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
    before = qk._version
    tb.rotary(q, k, pos, f)
    assert qk._version == before


def test_writes_under_inference_mode():
    """As torch's own writes in place: anything in it, none to its tensors outside."""
    pos, f = torch.arange(24, dtype=torch.int32, device="cuda"), tb.rotary_frequencies(64)
    decay, x, outside = torch.tensor([0.9, 0.99], device="cuda"), rows(), torch.zeros(24, 2, 64, 64, device="cuda")
    with torch.inference_mode():
        inside, q = torch.zeros(24, 2, 64, 64, device="cuda"), rows()
        for state in (inside, outside):
            tb.linear_attention_step(x, x, x, decay, state)
        tb.rotary(q, None, pos, f, inplace=True)
    assert torch.equal(inside, outside)
    with pytest.raises(RuntimeError, match="inference tensor"):
        tb.linear_attention_step(x, x, x, decay, inside)
    assert torch.equal(inside, outside)


@pytest.mark.parametrize("name", NAMES)
def test_forward_mode_is_refused(name):
    call = calls()[name]
    with fwAD.dual_level():
        x = fwAD.make_dual(rows(), rows())
        with pytest.raises((RuntimeError, NotImplementedError)):
            call(x)


def test_forward_mode_is_refused_in_place_and_backward():
    x, w, decay = rows(), torch.ones(64, device="cuda"), torch.tensor([0.9, 0.99], device="cuda")
    pos, f = torch.arange(24, dtype=torch.int32, device="cuda"), tb.rotary_frequencies(64)
    state = torch.zeros(24, 2, 64, 64, device="cuda")
    with fwAD.dual_level():
        t = fwAD.make_dual(rows(), rows())
        for call in (lambda: tb.rotary(t, None, pos, f, inplace=True), lambda: tb.rotary_backward(t, None, pos, f),
                     lambda: tb.rms_norm_fp8(t, w), lambda: tb.rms_norm_backward(t, x, w),
                     lambda: tb.linear_attention_backward(t, x, x, x, decay),
                     lambda: tb.linear_attention_step(t, x, x, decay, state)):
            with pytest.raises(tb.TBError):
                call()
