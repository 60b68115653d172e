"""Shapes and strides of the logits that det_token_logprobs takes."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def det():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    return d


@pytest.mark.parametrize("lead", [(2, 3), (5,), (), (2, 1, 4), (0, 3)])
def test_an_empty_vocabulary(det, lead):
    """Rows without a logit: log probability 0 (no token is in the vocabulary), lse -inf, entropy 0, whatever the shape."""
    used = torch.full((1000,), 7.0, device="cuda")            # the results' memory is not 0 by chance
    del used
    x = torch.zeros(*lead, 0, device="cuda")
    t = torch.zeros(lead, dtype=torch.int32, device="cuda")
    filler = [torch.full((max(t.numel(), 1),), 7.0, device="cuda") for _ in range(16)]
    del filler
    r = det.det_token_logprobs(x, t)
    assert r.logprob.shape == lead and r.lse.shape == lead
    assert torch.all(r.logprob == 0) and torch.all(r.lse == -math.inf) and torch.all(r.entropy == 0)
    g = det.det_token_logprobs_backward(x, t, r.lse, r.entropy, grad_logprob=torch.ones_like(r.lse))
    assert g.shape == x.shape
