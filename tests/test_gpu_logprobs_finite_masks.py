"""det_token_logprobs on rows masked by finite constants, against the definition in 64 bits.

Tolerance of log p = (x - m) - log S.  u = 2^-24, V the vocabulary.  x - m is rounded once at its own size, the result
once.  A term of S is off by 2^-22 (exponential) and 3 u |d| (d = x - m, whose mean under p is at most log V), and by 2^-22
more for each time its sum is brought to a larger maximum: a mask's sum is raised to the first logit above it, and
of the sums that count a few times more, 8 here; the additions are 58 and one for each chunk.  A logit that is held to more
than its type's bits is not needed: x and m are the type's.  Every bound is twice that sum.  None of it grows with |m|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_logprobs import DTYPES, grad_reference, reference, top_reference  # noqa: E402

MASKS = [-1e4, -1e5, -1e6, -1e9, -1e10, -1e12, -1e18, -1e20, -1e30]


@pytest.fixture(scope="module")
def det():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    return d


def parts(vocab):
    u, lv = 2.0 ** -24, np.log(vocab)
    chunks = vocab / 8192 + 1
    return 9 * 2.0 ** -22 + (58 + chunks) * u, u, lv


def off(got, want, tol, what):
    got = got.double().cpu().numpy()
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - want) <= tol))
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def check(det, x, tokens, k):
    vocab = x.shape[1]
    r = det.det_token_logprobs(x, torch.from_numpy(tokens).cuda(), top_k=k)
    lp, ent, lse = reference(x, tokens)
    part, u, lv = parts(vocab)
    tol = 2 * (part + 3 * u * lv)
    off(r.lse, lse, tol + 2.0 ** -23 * np.abs(lse), "lse")
    off(r.logprob, lp, tol + 2.0 ** -22 * np.abs(lp), "logprob")
    off(r.entropy, ent, 2 * (part * (1 + 2 * lv) + 3 * u * (lv * lv + 2 * lv + 2)), "entropy")
    want = top_reference(x, k)
    assert np.array_equal(r.top_index.cpu().numpy(), want)
    want_lp = np.stack([reference(x, want[:, j])[0] for j in range(k)], 1)
    off(r.top_logprob, want_lp, tol + 2.0 ** -22 * np.abs(want_lp), "top_logprob")
    return r


def masked_rows(rng, vocab, dtype):
    """For each mask a row with no token left, with one, a tenth and half of them."""
    x = torch.from_numpy((rng.standard_normal((4 * len(MASKS), vocab)) * 3).astype(np.float32))
    tokens = np.zeros(len(x), np.int32)
    for i, mask in enumerate(MASKS):
        for j, share in enumerate((0.0, None, 0.1, 0.5)):
            keep = np.zeros(vocab, bool)
            if share is None:
                keep[rng.integers(vocab)] = True
            else:
                keep = rng.random(vocab) < share
            row = 4 * i + j
            x[row, torch.from_numpy(~keep)] = mask
            # a token that is left, or in every other row a masked one
            left, gone = np.flatnonzero(keep), np.flatnonzero(~keep)
            tokens[row] = gone[len(gone) // 2] if i % 2 or len(left) == 0 else left[-1]
    return x.to(DTYPES[dtype]).cuda(), tokens


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [1000, 40_003, 131_072])
def test_finite_masks(det, dtype, vocab):
    rng = np.random.default_rng(vocab)
    x, tokens = masked_rows(rng, vocab, dtype)
    r = check(det, x, tokens, 5)
    for few in ([0, 1], [16, 17, 18, 19], [34, 35]):     # few rows are split over CTAs
        one = det.det_token_logprobs(x[few].contiguous(), torch.from_numpy(tokens[few]).cuda(), top_k=5)
        assert all(torch.equal(a[few], b) for a, b in zip(r, one))
    # and many, and rows at odd elements
    many = x.repeat(9, 1)
    assert torch.equal(det.det_token_logprobs(many).lse.view(9, -1), r.lse.expand(9, -1))
    wide = torch.zeros(x.shape[0], vocab + 1, dtype=x.dtype, device="cuda")
    wide[:, 1:] = x
    assert torch.equal(det.det_token_logprobs(wide[:, 1:]).entropy, r.entropy)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_several_masks_in_a_row(det, dtype):
    """Masks that are added up, or that differ from word to word."""
    rng = np.random.default_rng(1)
    vocab = 20_003
    x = torch.from_numpy((rng.standard_normal((6, vocab)) * 3).astype(np.float32))
    x[0] = torch.from_numpy(rng.choice(np.asarray(MASKS, np.float32), vocab))
    x[1] = x[0]
    x[1, 19_999] = 1.0
    x[2, : vocab // 2] -= 1e9
    x[3] = -1e10
    x[3, ::2] = -2e10
    x[4] = -1e12
    x[4, 4096:] = -1e30
    x[5] = -1e18
    x[5, -1] = -1e10
    check(det, x.to(DTYPES[dtype]).cuda(), np.array([5, 19_999, 20_000, 6, 7, vocab - 1], np.int32), 20)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_logits(det, dtype):
    """Large positive maxima, and rows of them alone."""
    rng = np.random.default_rng(2)
    x = torch.from_numpy((rng.standard_normal((6, 20_003)) * 3).astype(np.float32))
    for i, v in enumerate((1e6, 1e9, 1e10, 1e18, 1e30, 3e38)):
        x[i, 100:100 + 50 * (i + 1)] = v
    check(det, x.to(DTYPES[dtype]).cuda(), np.full(6, 100, np.int32), 5)
    y = x.clone()
    y[:] = torch.tensor([1e6, 1e9, 1e10, 1e18, 1e30, 3e38])[:, None]
    check(det, y.to(DTYPES[dtype]).cuda(), np.full(6, 100, np.int32), 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient(det, dtype):
    """A probability is off by the error of log p, its gradient by that at the size of its terms, and one rounding."""
    rng = np.random.default_rng(3)
    vocab = 10_003
    x, tokens = masked_rows(rng, vocab, dtype)
    t = torch.from_numpy(tokens).cuda()
    r = det.det_token_logprobs(x, t)
    gl, gh = (rng.standard_normal(len(tokens)).astype(np.float32) for _ in range(2))
    got = det.det_token_logprobs_backward(x, t, r.lse, r.entropy, grad_logprob=torch.from_numpy(gl).cuda(),
                                          grad_entropy=torch.from_numpy(gh).cuda())
    want = grad_reference(x, tokens, gl, gh)
    part, u, lv = parts(vocab)
    _, ent, lse = reference(x, tokens)
    xs = x.double().cpu().numpy()
    m = xs.max(1)[:, None]
    logp = (xs - m) - np.log(np.exp(xs - m).sum(1))[:, None]
    far = np.clip(-logp, 0, 800)
    # log p: as above, and lse rounded at its size where it is used (below 1024)
    err = 2 * (part + 3 * u * lv) + 2.0 ** -22 * (far + np.minimum(np.abs(lse), 1024)[:, None] + 1)
    mag = np.exp(-far) * (np.abs(gl)[:, None] + np.abs(gh)[:, None] * (far + ent[:, None] + 2))
    round_ = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]
    tol = 2 * (mag * err * (1 + lv) + round_ * np.abs(want)) + 2.0 ** -22 * np.abs(gl).max() * 2.0 ** -2 + 2.0 ** -126
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
