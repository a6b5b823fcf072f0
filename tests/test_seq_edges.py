"""The sequence operators on the GPU where their inputs are at an edge."""
import pytest

from tests import _seq_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_voxel_grid_leaf_gb300 as tb  # noqa: E402
from tests.test_seq_gpu import gen  # noqa: E402


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
