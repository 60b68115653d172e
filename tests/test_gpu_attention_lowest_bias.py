"""A learned bias of the type's lowest value, or of other values near the end of 32 bits' range: a finite score, not a mask
of -inf.  Where every token of a head has it the softmax is that of what is left after rounding to 32 bits."""
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


def cache(length, heads, dim, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    pages = -(-length // 16)
    k, v = (torch.randn(pages, 16, heads, dim, generator=g).to(dtype).cuda() for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32).view(1, -1).cuda()
    return k, v, table, torch.tensor([length], dtype=torch.int32).cuda(), torch.randn(1, heads, dim, generator=g).to(dtype).cuda()


def expected(q, k, v, length, bias, scale):
    """In 32-bit scores, sums in 64 bits."""
    kk, vv = (t.flatten(0, 1)[:length].double() for t in (k, v))
    x = (torch.einsum("hd,nhd->hn", q[0].double(), kk) * scale).float() + bias
    p = torch.softmax(x.double(), 1)
    size = (torch.einsum("hd,nhd->hn", q[0].double().abs(), kk.abs()) * scale).amax(1)
    return torch.einsum("hn,nhd->hd", p, vv), torch.logsumexp(x.double(), 1), size


@pytest.mark.parametrize("table_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("length", [9, 300, 3000, 20_000])
def test_every_token_at_the_lowest_value(det, table_dtype, length):
    """Both parts of the bias (near distances looked up, far ones held), one chunk and many.  The values' mean is held to
    2^-8 of the largest value (one rounding to bf16 of at most 2^-9, sums and weights far below it), lse to the scores' 32-bit
    sums (D + 8 roundings at the size of sum |q k|, twice) and its own rounding."""
    k, v, pages, n, q = cache(length, 4, 64, torch.bfloat16)
    low = torch.finfo(table_dtype).min
    bounds = torch.tensor([1, 40], dtype=torch.int32, device="cuda")
    bias = torch.full((3, 4), low, dtype=table_dtype, device="cuda")
    bias[:, 3] = 0                                            # a head without it
    q[:, 2] = 0                                               # and one without scores
    r = det.det_paged_attention(q, k, v, pages, n, bias_table=bias, bias_bounds=bounds)
    out, lse, size = expected(q, k, v, length, bias[0].float()[:, None].expand(-1, length), 0.125)
    if table_dtype is torch.float16:
        # scores next to -65504 keep steps of 2^-8 in 32 bits: what is left of them depends on the order of two
        # roundings, so the head with scores has only to be finite
        assert torch.isfinite(r.out).all() and torch.isfinite(r.lse).all()
        heads = [2, 3]
    else:
        heads = [0, 1, 2, 3]
    vmax = v.double().abs().amax()
    assert torch.all((r.out[0].double() - out).abs()[heads] <= 2.0 ** -8 * vmax)
    assert torch.all((r.lse[0].double() - lse).abs() <= 2.0 ** -18 + 2.0 ** -22 * 72 * size + 2.0 ** -22 * lse.abs())


def test_values_near_the_end_of_the_range(det):
    """-2.6e38 is far above -3e38, and both are above the lowest value: the nearer tokens take all the weight."""
    length = 700
    k, v, pages, n, q = cache(length, 2, 128, torch.bfloat16, 1)
    bounds = torch.tensor([8, 600], dtype=torch.int32, device="cuda")
    bias = torch.tensor([[-2.6e38, -3e38], [-3e38, -2.6e38], [torch.finfo(torch.float32).min] * 2], device="cuda")
    r = det.det_paged_attention(q, k, v, pages, n, bias_table=bias, bias_bounds=bounds)
    vv = v.flatten(0, 1)[:length].double()
    want = torch.stack((vv[length - 8:, 0].mean(0), vv[length - 600:length - 8, 1].mean(0)))
    assert torch.all((r.out[0].double() - want).abs() <= 2.0 ** -8 * vv.abs().amax())
    assert torch.all((r.lse[0] / -2.6e38 - 1).abs() < 2.0 ** -22)
    # large scores of the other sign, and a bias of -inf beside the lowest value
    bias = torch.tensor([[3e38, -math.inf], [2.9e38, torch.finfo(torch.float32).min], [-math.inf, -math.inf]], device="cuda")
    r = det.det_paged_attention(q, k, v, pages, n, bias_table=bias, bias_bounds=bounds)
    want = torch.stack((vv[length - 8:, 0].mean(0), vv[length - 600:length - 8, 1].mean(0)))
    assert torch.all((r.out[0].double() - want).abs() <= 2.0 ** -8 * vv.abs().amax())
