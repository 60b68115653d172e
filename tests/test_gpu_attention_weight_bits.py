"""The weights of the softmax have 32-bit accuracy in the second product, whatever the cache's type: seen where large terms
of the output cancel, so that its own rounding to 16 bits is small.

A token with the value 0 has the largest score; two others nearly as large ones and values whose terms cancel to the
values' last bit, and a fourth one takes that away as far as its own last bit goes.  Tolerance relative to sum w |v|
(the output's terms; errors of the weights' sum scale an output that is near 0): scores exact, their differences of at most 1/2
times log2(e) 1.5 u, the exponential 4 u, the parts of the weights 1 u, additions 8 u, u = 2^-24; twice that, and the rounding of
the output."""
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
@pytest.mark.parametrize("dim,heads", [(64, 1), (64, 16), (64, 17), (128, 8), (128, 16), (256, 8), (256, 16)])
def test_cancelling_outputs(det, dtype, dim, heads):
    g = torch.Generator().manual_seed(dim + heads)
    dt, batch = DTYPES[dtype], 64
    score = torch.zeros(batch, 4)
    score[:, 1:] = -0.5 * torch.rand(batch, 3, generator=g)
    score = score.to(dt).double()
    w = torch.softmax(score, 1)[:, :, None]
    v = torch.zeros(batch, 4, dim, dtype=torch.float64)
    v[:, 1] = (0.5 + 0.5 * torch.rand(batch, dim, generator=g)).to(dt).double()
    for j in (2, 3):
        v[:, j] = (-(w * v).sum(1) / w[:, j]).to(dt).double()
    q = torch.zeros(batch, heads, dim, dtype=dt)
    q[..., 0] = 8
    k = torch.zeros(batch, 16, 1, dim, dtype=dt)
    k[:, :4, 0, 0] = score.to(dt)
    vc = torch.zeros(batch, 16, 1, dim, dtype=dt)
    vc[:, :4, 0] = v.to(dt)
    table = torch.arange(batch, dtype=torch.int32)[:, None].cuda()
    n = torch.full((batch,), 4, dtype=torch.int32).cuda()
    out = det.det_paged_attention(q.cuda(), k.cuda(), vc.cuda(), table, n, scale=0.125).out.double().cpu()
    want = (w * v).sum(1)[:, None]
    size = (w * v.abs()).sum(1)[:, None]
    u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    tol = 2 * 14.5 * 2.0 ** -24 * size + u * want.abs() + (2.0 ** -24 if dtype == "f16" else 0)
    err = (out - want).abs()
    assert torch.all(err <= tol), (err / size).max() * 2 ** 24
