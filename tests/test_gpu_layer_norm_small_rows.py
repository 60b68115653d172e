"""Gradients of the layer norm for rows of deviations so small that the square of their reciprocal passes 32 bits: the
definition, rstd (gw - mean(gw) - xh mean(gw xh)), stays finite.  Tolerances as in test_gpu_layer_norm."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_layer_norm import check_backward, det, make  # noqa: E402,F401


@pytest.mark.parametrize("cols", [8, 41, 264, 1021, 4096, 5000, 8200, 16383])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_small_deviations_without_an_eps(det, cols, kind):  # noqa: F811
    x, g, w, _ = make(20, cols, torch.float32, cols, offset=0.0)
    # the squares of the smallest are subnormal, so rstd is compared with nothing: the gradient takes it as given
    # (gradients along the rows, so that mean(gw xh) is not small)
    g = torch.sign(x) + 0.25 * g
    x, g = (x * torch.logspace(-20, -15, 20)[:, None]).to(kind), g.to(kind)
    r = det.det_layer_norm(x.cuda(), w.cuda(), eps=0.0)
    assert r.rstd.isfinite().all() and float(r.rstd.max()) > 2e19
    grads = det.det_layer_norm_backward(g.cuda(), x.cuda(), r.mean, r.rstd, w.cuda())
    assert grads.x.isfinite().all()
    check_backward(grads, g, x, r.mean.cpu(), r.rstd.cpu(), w, torch.float32)
