"""det_paged_attention where one token takes nearly all the weight and its value is 0: the output is the other tokens',
whose weights are small.

Tolerance, relative to the output (all its terms have one sign): the scores are exact (one product that is not 0, a
scale of 2^-3), their differences d <= 18 are rounded once and multiplied by log2(e): 3 u d, u = 2^-24; the exponential 2^-22;
weights in two parts of the type: 2^-17 for bf16, for f16 2^-22 or 2^-40 of the largest weight (2^-14 of e^-18);
the sums 64 u; one rounding to the type, and f16's subnormal step.  The bound is twice that."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def det():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    return d


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim,heads", [(64, 1), (64, 9), (64, 17), (128, 1), (128, 9), (256, 1), (256, 9)])
@pytest.mark.parametrize("length", [2, 16, 600])
def test_small_weights(det, dtype, dim, heads, length):
    g = torch.Generator().manual_seed(length)
    pages = -(-length // 16)
    above = [4.0, 8.0, 10.0, 12.0, 14.0, 16.0, 17.0]          # of the first token over the others, a sequence each
    q = torch.zeros(len(above), heads, dim)
    q[..., 0] = 8.0
    k = torch.zeros(len(above) * pages, 16, 1, dim)
    v = (500 + 500 * torch.rand(k.shape, generator=g)).to(DTYPES[dtype])
    v[::pages, 0] = 0
    for b, s in enumerate(above):
        k[b * pages, 0, 0, 0] = s
    table = torch.arange(len(above) * pages, dtype=torch.int32).view(len(above), pages)
    lengths = torch.full((len(above),), length, dtype=torch.int32)
    r = det.det_paged_attention(q.to(DTYPES[dtype]).cuda(), k.to(DTYPES[dtype]).cuda(), v.cuda(), table.cuda(),
                                lengths.cuda(), scale=0.125)
    u, half = (2.0 ** -8, 2.0 ** -17) if dtype == "bf16" else (2.0 ** -11, 2.0 ** -14)
    for b, s in enumerate(above):
        vv = v[b * pages:(b + 1) * pages, :, 0].double().reshape(-1, dim)[1:length]
        want = vv.sum(0) * math.exp(-s) / (1 + (length - 1) * math.exp(-s))
        tol = 2 * (3 * 2.0 ** -24 * 18 + 2.0 ** -22 + half + 64 * 2.0 ** -24) + u
        err = (r.out[b].double().cpu() - want).abs()
        assert torch.all(err <= tol * want + 2.0 ** -24), (s, (err / want).max())
