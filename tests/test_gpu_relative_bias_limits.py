"""det_relative_bias at the most queries that its documentation allows (below 2^20)."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("q_len", [1_048_560, 1_048_561, (1 << 20) - 1])
@pytest.mark.parametrize("k_len", [8, 9])
def test_most_queries(det, dtype, q_len, k_len):
    bounds = det.det_relative_bounds(32, 128)
    table = torch.randn(32, 1, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    got = det.det_relative_bias(table, bounds, q_len, k_len)
    r = torch.arange(k_len, device="cuda")[None, :] - torch.arange(q_len, device="cuda")[:, None]
    bucket = torch.bucketize((-r).clamp(min=0), bounds.long(), right=True)
    assert torch.equal(got[0], table[:, 0][bucket])
