"""Finite rows whose sums leave 32 bits: every result of such a row is NaN, and those of the rows beside it are their own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_layer_norm import check_forward, det, make  # noqa: E402,F401


@pytest.mark.parametrize("cols", [8, 41, 300, 4096, 9000])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_sums_past_the_range(det, kind, cols):  # noqa: F811
    x, _, w, b = make(7, cols, kind, cols)
    x[1] = 2e38 * torch.where(torch.arange(cols) % 2 == 0, 1.0, 0.9)        # its sum
    x[3] = 3e25 * x[3].sign() + (x[3] == 0)                                 # its squares alone
    x[5, 0] = 1e20
    r = det.det_layer_norm(x.cuda(), w.cuda(), b.cuda())
    assert r.out[[1, 3, 5]].isnan().all() and r.mean[[3, 5]].isfinite().all()
    keep = [0, 2, 4, 6]
    check_forward(type(r)(*(t[keep] for t in r)), x[keep], w, b, 1e-5)
