"""The gradients of the language-model operators have no derivative: asking for one is an error, not a gradient without it."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build
    _build.build()
    from deterministic_floating_point_gb300 import autograd, det
    return det, autograd


def test_log_probabilities(mods):
    _, autograd = mods
    x = torch.randn(4, 50, device="cuda", requires_grad=True)
    t = torch.arange(4, dtype=torch.int32, device="cuda")
    lp, ent = autograd.token_logprobs(x, t)
    (g,) = torch.autograd.grad(lp.sum() + ent.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):          # a penalty on the gradient beside another loss
        ((g * g).sum() + (x * x).sum()).backward()
    # the first derivative under create_graph is the one without it
    (h,) = torch.autograd.grad(sum(r.sum() for r in autograd.token_logprobs(x, t)), x)
    assert torch.equal(g, h)


def test_relative_bias(mods):
    det, autograd = mods
    bounds = det.det_relative_bounds(8, 20)
    table = torch.randn(8, 2, device="cuda", requires_grad=True)
    w = torch.randn(2, 12, 30, device="cuda", requires_grad=True)
    out = autograd.relative_bias(table, bounds, 12, 30)
    (g,) = torch.autograd.grad((out * w).sum(), table, create_graph=True)
    with pytest.raises(RuntimeError):
        ((g * g).sum() + (table * table).sum()).backward()
