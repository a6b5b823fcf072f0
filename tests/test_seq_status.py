"""The report of a linear-attention kernel whose bounded wait gave up, by waits
of a few polls that nothing ends: no GPU fault, the context stays usable."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_voxel_grid_leaf_gb300 as tb  # noqa: E402
from tests.test_seq_gpu import check_attention  # noqa: E402

TIMEOUT = 6


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def give_up(kernel, stream):
    assert tb.lib().tb_linear_attention_selftest_wait(kernel, 1 << 10, stream.cuda_stream) == 0


def reported(stream):
    try:
        tb.linear_attention_status(stream)
    except tb.TBError as e:
        assert e.status == TIMEOUT
        return True
    return False


@pytest.mark.parametrize("kernel", [0, 1])
def test_a_wait_that_gives_up_is_reported_once(kernel):
    stream = torch.cuda.current_stream()
    reported(stream)
    assert not reported(stream)
    give_up(kernel, stream)
    give_up(kernel, stream)
    assert reported(stream)
    assert not reported(stream)
    for dtype in (torch.bfloat16, torch.float32):
        check_attention([70, 0, 129], 2, 64, 64, dtype, True, seed=1)
    assert not reported(stream)


def test_refused_selftests():
    lib, stream = tb.lib(), torch.cuda.current_stream().cuda_stream
    for kernel, polls in ((-1, 8), (2, 8), (0, 0), (1, (1 << 22) + 1)):
        assert lib.tb_linear_attention_selftest_wait(kernel, polls, stream) == 1


@pytest.mark.parametrize("kernel", [0, 1])
def test_every_stream_has_its_report(kernel):
    """What gave up on one stream is not used up by a status call of another one."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        reported(s)
    assert not reported(a) and not reported(b)
    give_up(kernel, b)
    b.synchronize()
    assert reported(a)  # its own outputs may be as good as they were: the report does not say which call it was
    assert reported(b)
    assert not reported(a) and not reported(b)
    give_up(kernel, a)
    a.synchronize()
    assert reported(a) and not reported(a) and reported(b)
