"""det_token_logprobs of logits far from 0, with bounds that do not grow with the logits: log p and the entropy
depend on the differences of logits alone, which are exact at the sizes here.

Tolerances as in the tests of finite masks: twice 9 x 2^-22 (the exponential, and 8 raises of a sum to a larger
maximum) + (58 + chunks) additions + 3 u log V for log S, and 2^-22 |log p| for the two roundings after it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_logprobs import reference  # noqa: E402


@pytest.fixture(scope="module")
def det():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    return d


def check(r, x, tokens):
    lp, ent, _ = reference(x, tokens)
    u, lv, chunks = 2.0 ** -24, np.log(x.shape[1]), x.shape[1] / 8192 + 1
    part = 9 * 2.0 ** -22 + (58 + chunks) * u
    err = np.abs(r.logprob.double().cpu().numpy() - lp)
    assert np.all(err <= 2 * (part + 3 * u * lv) + 2.0 ** -22 * np.abs(lp)), err.max()
    err = np.abs(r.entropy.double().cpu().numpy() - ent)
    assert np.all(err <= 2 * (part * (1 + 2 * lv) + 3 * u * (lv * lv + 2 * lv + 2))), err.max()


SHIFTS = [0.0, 1e3, -1e3, 1e4, -1e4, -3e4, 1e5, -1e6, 1e7, -1e9]


@pytest.mark.parametrize("vocab", [1000, 40_003, 131_072])
def test_equal_logits(det, vocab):
    """Rows of one value: every log probability is -log V; all sums have the same maximum when they are joined."""
    tokens = np.full(len(SHIFTS), vocab - 1, np.int32)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.tensor(SHIFTS, device="cuda")[:, None].to(dtype).expand(-1, vocab).contiguous()
        check(det.det_token_logprobs(x, torch.from_numpy(tokens).cuda()), x, tokens)
    y = torch.tensor([-3e4, 6e4, -6.1e4], device="cuda", dtype=torch.float16)[:, None].expand(-1, vocab).contiguous()
    check(det.det_token_logprobs(y, torch.from_numpy(tokens[:3]).cuda()), y, tokens[:3])


@pytest.mark.parametrize("vocab", [1000, 40_003, 131_072])
def test_shifted_logits(det, vocab):
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy((rng.standard_normal((len(SHIFTS), vocab)) * 3 + np.asarray(SHIFTS)[:, None]).astype(np.float32)).cuda()
    tokens = rng.integers(0, vocab, len(SHIFTS)).astype(np.int32)
    t = torch.from_numpy(tokens).cuda()
    r = det.det_token_logprobs(x, t)
    check(r, x, tokens)
    # few rows are split over CTAs, many are not: the same bits
    many = det.det_token_logprobs(x.repeat(40, 1), t.repeat(40))
    assert torch.equal(many.logprob.view(40, -1), r.logprob.expand(40, -1))
    assert torch.equal(many.entropy.view(40, -1), r.entropy.expand(40, -1))


@pytest.mark.parametrize("vocab", [1000, 40_003])
@pytest.mark.parametrize("spread", [0, 3, 40])
def test_around_two_to_the_24(det, vocab, spread):
    """Where 32-bit logits become 2 apart, and rows whose logits lie on both sides of it."""
    rng = np.random.default_rng(spread)
    at = np.asarray([1.6e7, -1.6e7, 2.0 ** 24, -2.0 ** 24, 2.0 ** 24 + 2, -2.0 ** 24 - 2, 2.0 ** 24 - 1, 1 - 2.0 ** 24, 5e7, -5e7])
    x = torch.from_numpy((rng.integers(-spread, spread + 1, (len(at), vocab)) + at[:, None]).astype(np.float32)).cuda()
    tokens = rng.integers(0, vocab, len(at)).astype(np.int32)
    r = det.det_token_logprobs(x, torch.from_numpy(tokens).cuda())
    check(r, x, tokens)
    y = x.clone()                                   # a mask's size in most of a row
    y[:, vocab // 4:] = torch.from_numpy(-np.abs(at).astype(np.float32)).cuda()[:, None]
    y[:, 5] = 1.0
    check(det.det_token_logprobs(y, torch.from_numpy(tokens).cuda()), y, tokens)
