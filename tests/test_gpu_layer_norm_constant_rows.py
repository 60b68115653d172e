"""Rows whose mean is exact: constant ones whose sums are exact in 32 bits, at widths where n (1 / n) is not 1 in 32 bits.  What
the mean leaves is 0, so the result is the bias."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_layer_norm import det  # noqa: E402,F401

ALL = [n for n in range(1, 16385) if np.float32(n) * (np.float32(1) / np.float32(n)) != 1]
WIDTHS = [n for k, n in enumerate(ALL) if n < 130 or k % 97 == 0] + [16383]


def test_the_widths():
    assert 41 in WIDTHS and len(ALL) > 2000


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, torch.float16])
def test_constant_rows(det, kind):  # noqa: F811
    for cols in WIDTHS:
        # whole numbers whose sums stay below 2^24, so that every order of adding them is exact
        values = torch.tensor([1000.0, -3.0, 0.0, 1.0, -640.0, 7.0])
        values = values[values.abs() * cols < 2**24]
        x = values[:, None].expand(-1, cols).to(kind).contiguous()
        w = torch.full((cols,), 3.0)
        b = torch.linspace(-1, 1, cols)
        r = det.det_layer_norm(x.cuda(), w.cuda(), b.cuda())
        assert torch.equal(r.mean.cpu(), values), cols
        assert torch.equal(r.out.cpu(), b.to(kind).expand(values.numel(), cols)), cols
        assert float((r.rstd.cpu() - 1e-5 ** -0.5).abs().max()) <= 4 * 2.0 ** -24 * 1e-5 ** -0.5
