"""det_token_logprobs and its gradient against 64-bit statements of the
definitions.

Tolerances.  u = 2^-24, d = x - m, V the vocabulary.  The exponent d log2(e) is off by at most 3 u |d|
(the subtraction, the product and the constant) and the exponential by 2^-22, so a term of S is off by 2^-22 +
3 u |d| of itself; the sum adds u for each addition in a row (16 in a thread's chunk, a join for each chunk, 5 + 16 joins
of 2 roundings: 58 + chunks).  Weighted by the probabilities p the mean of |d| is at most log V (entropy = log S +
mean |d| <= log V), and that of d^2 at most (log V)^2 + 2 log V + 2.  So
  lse:      2^-22 + (58 + chunks) u + 3 u log V, and one rounding at its own size
  entropy:  the terms are weighted by |d| as well: (2^-22 + (58 + chunks) u)(1 + 2 log V) + 3 u E d^2
Every bound below is twice that."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def det():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    return d


def reference(x, tokens):
    """logprob, entropy, lse in 64 bits from the definition; x is [rows, vocab]."""
    x = x.double().cpu().numpy()
    n, vocab = x.shape
    lp, ent, lse = np.zeros(n), np.zeros(n), np.full(n, -np.inf)
    for r in range(n):
        row = x[r]
        if np.isnan(row).any() or np.isposinf(row).any():
            lse[r] = ent[r] = np.nan
            lp[r] = np.nan if 0 <= tokens[r] < vocab else 0.0
            continue
        live = row > -np.inf
        m, logs = 0.0, 0.0
        if live.any():
            # log p = (x - m) - log S: at the types' lowest values x - lse would lose log S even in 64 bits
            m = row.max()
            logs = np.log(np.exp(row[live] - m).sum())
            lse[r] = m + logs
            ll = (row[live] - m) - logs
            ent[r] = -(np.exp(ll) * ll).sum()
        if 0 <= tokens[r] < vocab:
            lp[r] = (row[tokens[r]] - m) - logs if row[tokens[r]] > -np.inf else -np.inf
    return lp, ent, lse


def top_reference(x, k):
    x = x.double().cpu().numpy()
    key = np.where(np.isnan(x), np.inf, x)
    # NaN above +inf
    return np.stack([np.lexsort((np.arange(x.shape[1]), -key[r], ~np.isnan(x[r])))[:k] for r in range(x.shape[0])])


def close(got, want, tol):
    got = got.double().cpu().numpy()
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        assert np.all(same | (np.abs(got - want) <= tol)), np.nanmax(np.abs(got - want)[~same])


def check(det, x, tokens, k):
    vocab = x.shape[1]
    r = det.det_token_logprobs(x, torch.from_numpy(tokens).cuda(), top_k=k)
    lp, ent, lse = reference(x, tokens)
    chunks = vocab / (512 * 16) + 1
    u, lv = 2.0 ** -24, np.log(vocab)
    part = 2.0 ** -22 + (58 + chunks) * u
    tol = 2 * (part + 3 * u * lv)
    size = np.nan_to_num(np.abs(lse), posinf=0, neginf=0, nan=0)
    close(r.lse, lse, tol + 2.0 ** -22 * size)
    close(r.logprob, lp, tol + 2.0 ** -22 * (size + np.nan_to_num(np.abs(lp), posinf=0, neginf=0, nan=0)))
    close(r.entropy, ent, 2 * (part * (1 + 2 * lv) + 3 * u * (lv * lv + 2 * lv + 2)))
    if k:
        want = top_reference(x, k)
        assert np.array_equal(r.top_index.cpu().numpy(), want)
        # the reference's own log probabilities of those tokens
        want_lp = np.stack([reference(x, want[:, j])[0] for j in range(k)], 1)
        close(r.top_logprob, want_lp, (tol + 2.0 ** -22 * size)[:, None] + 2.0 ** -22 * np.nan_to_num(np.abs(want_lp), posinf=0, neginf=0))
    return r


def logits(rng, rows, vocab, dtype, scale=3.0):
    return torch.from_numpy((rng.standard_normal((rows, vocab)) * scale).astype(np.float32)).to(DTYPES[dtype]).cuda()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 32, 33, 511, 1023, 1024, 1025, 8191, 8193, 16384, 16385, 32767, 50001, 131072])
def test_against_64_bits(det, dtype, vocab):
    rng = np.random.default_rng(vocab)
    rows = 5
    x = logits(rng, rows, vocab, dtype)
    tokens = rng.integers(-2, vocab + 2, rows).astype(np.int32)
    tokens[0] = vocab - 1
    for k in sorted({0, 1, min(5, vocab), min(32, vocab)}):
        check(det, x, tokens, k)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_masks_and_special_rows(det, dtype):
    rng = np.random.default_rng(3)
    vocab = 20_003
    low = torch.finfo(DTYPES[dtype]).min
    x = logits(rng, 12, vocab, dtype)
    x[0] = -np.inf                                   # empty
    x[1] = -np.inf
    x[1, 17] = -3.0                                  # one token left
    x[2] = low                                       # uniform at the type's lowest value
    x[3] = low
    x[3, vocab - 1] = 2.0
    x[4, ::2] = -np.inf
    x[5, 1:] = -np.inf
    x[6, 40] = float("nan")
    x[7, 41] = float("inf")
    x[8] = 0.0                                       # all equal: the alternatives are the lowest indices
    x[9, :] = -0.0
    x[9, 1::2] = 0.0                                 # -0 and +0 are equal
    x[10] = low
    x[10, 100:200] = -np.inf
    x[11] = torch.linspace(0, 30, vocab)             # rising: the best lie together at the end
    tokens = np.array([3, 17, 5, vocab - 1, 0, 1, 2, 3, vocab, -1, 150, vocab - 1], np.int32)
    for k in (0, 3, 32):
        check(det, x, tokens, k)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("vocab", [67, 4099, 131072])
def test_fewer_tokens_left_than_alternatives(det, dtype, vocab):
    """The mask's value (or a value that many share, anywhere in the row) fills the alternatives by index."""
    rng = np.random.default_rng(vocab)
    low = torch.finfo(DTYPES[dtype]).min
    x = logits(rng, 12, vocab, dtype)
    for row, (mask, left) in enumerate([(-np.inf, 2), (-np.inf, 19), (-np.inf, 31), (low, 3), (low, 20), (-3e4, 7)]):
        keep = rng.permutation(vocab)[:left]
        kept = x[row, keep].clone()
        x[row] = mask
        x[row, keep] = kept
    x[6, : vocab // 2] = -20.0                       # a shared value in the row's second half, few above it
    x[6, vocab // 2:] = 4.0
    x[6, rng.permutation(vocab)[:9]] = 9.0
    x[7] = -20.0
    x[7, vocab - 40:] = 4.0                          # and at its end only
    x[7, 3] = 5.0
    x[8] = -np.inf
    x[8, vocab - 33:] = low
    x[9] = float("nan")
    x[10] = 1.0
    x[10, ::3] = float("nan")
    x[11] = -np.inf
    x[11, vocab - 1] = float("inf")
    tokens = rng.integers(0, vocab, 12).astype(np.int32)
    for k in (1, 20, 32):
        check(det, x, tokens, k)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_alternatives_past_the_lists(det, dtype):
    """More equal elements than a row's end lists: many threads' (some warps have none of them), or many of few threads."""
    vocab = 40_003
    per_word = 1 if dtype == "f32" else 2
    thread = torch.arange(vocab, device="cuda") // per_word % 256
    chunk = torch.arange(vocab, device="cuda") // per_word // 8192
    x = torch.full((6, vocab), -1.0, device="cuda")
    x[0] = torch.where(thread < 32, -20.0, 4.0)
    x[0, 777] = 9.0
    x[1] = torch.where(thread % 64 < 32, -20.0, 4.0)
    x[1, 39_999] = 9.0
    x[2] = torch.where((thread < 100) & (chunk == 0), 5.0, -1.0)
    x[3] = torch.where((thread < 100) & (chunk == 1), 5.0, -1.0)
    x[4] = torch.where((thread < 20) & (chunk == 0), 5.0, -1.0)
    x[4, 6:40_000:3001] = 6.0
    x[5] = torch.where(thread == 255, 3.0, -1.0)
    x = x.to(DTYPES[dtype])
    for k in (1, 7, 20, 32):
        check(det, x, np.full(6, 777, np.int32), k)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_alternatives_with_many_ties(det, dtype):
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.integers(0, 4, (6, 40_001)).astype(np.float32)).to(DTYPES[dtype]).cuda()
    x[1, 1000:] = -np.inf
    x[2, 5:] = -np.inf
    check(det, x, np.zeros(6, np.int32), 32)
    # the 32 best all belong to one thread's elements, or to one warp's
    y = torch.zeros(3, 40_000, dtype=DTYPES[dtype], device="cuda")
    y[0, 6:40_000:1024] = 5.0
    y[1, 64:128] = 7.0
    y[2, :] = torch.arange(40_000, device="cuda").remainder(512).to(y.dtype)
    check(det, y, np.zeros(3, np.int32), 32)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_a_row_does_not_depend_on_its_batch_or_alignment(det, dtype):
    rng = np.random.default_rng(7)
    rows, vocab = 300, 10_007
    x = logits(rng, rows, vocab, dtype)
    tokens = torch.from_numpy(rng.integers(0, vocab, rows).astype(np.int32)).cuda()
    a = det.det_token_logprobs(x, tokens, top_k=7)
    for again in range(3):
        b = det.det_token_logprobs(x, tokens, top_k=7)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    wide = torch.full((rows, vocab + 13), 9.0, dtype=x.dtype, device="cuda")
    for shift in range(9):
        wide[:, shift:shift + vocab] = x
        b = det.det_token_logprobs(wide[:, shift:shift + vocab], tokens, top_k=7)
        assert all(torch.equal(p, q) for p, q in zip(a, b)), shift
    for r in (0, 1, 123, 299):
        b = det.det_token_logprobs(x[r:r + 1], tokens[r:r + 1], top_k=7)
        assert all(torch.equal(p[r:r + 1], q) for p, q in zip(a, b))
    # three dimensions, and another stream with its own outputs
    b = det.det_token_logprobs(x.view(3, 100, vocab), tokens.view(3, 100), top_k=7)
    assert all(torch.equal(p.view(q.shape), q) for p, q in zip(a, b))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = det.det_token_logprobs(x, tokens, top_k=7, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("vocab", [16_385, 40_001, 65_536, 100_003])
def test_few_rows_and_many_rows_give_the_same_bits(det, dtype, vocab):
    """Few rows are split over several CTAs each, many are not."""
    rng = np.random.default_rng(vocab)
    rows = 170
    x = logits(rng, rows, vocab, dtype)
    x[3] = -np.inf
    x[4, : vocab // 2] = -np.inf
    x[5] = torch.finfo(x.dtype).min
    x[6, 5] = float("nan")
    x[7] = 1.5                                             # ties over all parts
    tokens = torch.from_numpy(rng.integers(0, vocab, rows).astype(np.int32)).cuda()
    many = det.det_token_logprobs(x, tokens, top_k=9)
    for rs in ([0], [3, 4, 5, 6, 7], list(range(60, 100))):
        few = det.det_token_logprobs(x[rs].contiguous(), tokens[rs].contiguous(), top_k=9)
        for a, b in zip(many, few):
            assert torch.equal(torch.nan_to_num(a[rs].float(), nan=12345.0), torch.nan_to_num(b.float(), nan=12345.0))
    check(det, x[:9].contiguous(), tokens[:9].cpu().numpy(), 9)


def test_empty_shapes_and_no_tokens(det):
    for shape in ((0, 100), (3, 0), (0, 0), (2, 0, 50)):
        x = torch.zeros(shape, device="cuda")
        t = torch.zeros(shape[:-1], dtype=torch.int32, device="cuda")
        r = det.det_token_logprobs(x, t)
        assert r.logprob.shape == x.shape[:-1]
        assert torch.all(r.logprob == 0) and torch.all(r.lse == -np.inf) and torch.all(r.entropy == 0)
        g = det.det_token_logprobs_backward(x, t, r.lse, r.entropy, grad_logprob=torch.ones_like(r.lse))
        assert g.shape == x.shape
    x = torch.randn(4, 77, device="cuda")
    r = det.det_token_logprobs(x, top_k=2)
    assert r.logprob is None and torch.equal(r.top_index[:, 0], x.argmax(1).int())


def grad_reference(x, tokens, gl, gh):
    x = x.double().cpu().numpy()
    rows, vocab = x.shape
    _, ent, lse = reference(torch.from_numpy(x), tokens)
    out = np.zeros_like(x)
    for r in range(rows):
        if lse[r] == -np.inf:
            continue
        live = x[r] > -np.inf
        m = x[r].max()
        lp = (x[r][live] - m) - np.log(np.exp(x[r][live] - m).sum())
        p = np.exp(lp)
        g = gl[r] if 0 <= tokens[r] < vocab else 0.0
        out[r, live] = -p * (g + gh[r] * (lp + ent[r]))
        if 0 <= tokens[r] < vocab:
            out[r, tokens[r]] += g
    return out


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("vocab", [1, 2, 7, 64, 1000, 4095, 4099, 33_333])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_gradient_against_64_bits(det, dtype, vocab, shift):
    rng = np.random.default_rng(vocab + shift)
    rows = 7
    x = logits(rng, rows, vocab + shift, dtype)[:, shift:]
    if vocab > 2:
        x[1] = -np.inf
        x[2, 1:] = -np.inf
        x[3] = torch.finfo(x.dtype).min
    tokens = rng.integers(-1, vocab + 1, rows).astype(np.int32)
    tokens[1:4] = 0
    tt = torch.from_numpy(tokens).cuda()
    r = det.det_token_logprobs(x, tt)
    gl = rng.standard_normal(rows).astype(np.float32)
    gh = rng.standard_normal(rows).astype(np.float32)
    u = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    tiny = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -24}[dtype]     # f16's subnormal step
    for a, b in ((gl, gh), (gl, None), (None, gh), (None, None)):
        out = torch.full((rows, vocab + 5), 7.0, dtype=x.dtype, device="cuda")
        got = det.det_token_logprobs_backward(
            x, tt, r.lse, r.entropy, grad_logprob=None if a is None else torch.from_numpy(a).cuda(),
            grad_entropy=None if b is None else torch.from_numpy(b).cuda(), out=out[:, 2:2 + vocab])
        want = grad_reference(x, tokens, a if a is not None else 0 * gl, b if b is not None else 0 * gh)
        # p is off by the error of lse and of its exponent (|lp| + |lse| + 16 times 2^-22, relatively; |lse| counts up to
        # 1024, beyond which the sum is taken again), and the bracket by the same at the size of its terms; then
        # one rounding to the type
        _, ent, lse = reference(x, tokens)
        size = np.minimum(np.nan_to_num(np.abs(lse), neginf=0), 1024)[:, None]
        xs = x.double().cpu().numpy()
        m = np.where(np.isneginf(lse), 0, xs.max(1))
        with np.errstate(divide="ignore"):
            logp = (xs - m[:, None]) - np.where(np.isneginf(lse), 0, np.log(np.exp(xs - m[:, None]).sum(1)))[:, None]
        far = np.clip(-logp, 0, 800)
        mag = np.exp(-far) * ((np.abs(gl)[:, None] if a is not None else 0) +
                              (np.abs(gh)[:, None] * (far + ent[:, None] + 1) if b is not None else 0))
        tol = 2 * (mag * (far + size + 16) * 2.0 ** -22 + u * np.abs(want) + tiny) + 2.0 ** -126
        err = np.abs(got.double().cpu().numpy() - want)
        assert np.all(err <= tol + 2 * 2.0 ** -24 * np.abs(gl).max()), (err - tol).max()
        assert torch.all(out[:, :2] == 7) and torch.all(out[:, 2 + vocab:] == 7)      # nothing beside the rows


def test_gradient_against_differences(det):
    from deterministic_floating_point_gb300 import autograd
    rng = np.random.default_rng(11)
    x = logits(rng, 3, 41, "f32", 1.5)
    tokens = torch.tensor([4, -1, 40], dtype=torch.int32, device="cuda")
    wl = torch.tensor([0.7, -1.1, 0.4], device="cuda")
    wh = torch.tensor([0.2, 0.5, -0.9], device="cuda")
    xr = x.clone().requires_grad_(True)
    lp, ent = autograd.token_logprobs(xr, tokens)
    ((lp * wl).sum() + (ent * wh).sum()).backward()

    def loss(z):
        a, b, _ = reference(z, tokens.cpu().numpy())
        return (a * wl.double().cpu().numpy()).sum() + (b * wh.double().cpu().numpy()).sum()

    base = x.double().cpu()
    h = 1e-5
    for r in range(3):
        for v in range(41):
            d = torch.zeros_like(base)
            d[r, v] = h
            want = (loss(base + d) - loss(base - d)) / (2 * h)     # off by h^2 third derivatives: below 1e-9
            assert abs(float(xr.grad[r, v]) - want) < 5e-6


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_autograd_forms(det, dtype):
    from deterministic_floating_point_gb300 import autograd
    rng = np.random.default_rng(12)
    x = logits(rng, 24, 501, dtype)
    tokens = torch.from_numpy(rng.integers(-1, 501, 24).astype(np.int32)).cuda()
    grads = []
    for shape in ((24, 501), (2, 3, 4, 501)):
        xr = x.view(shape).clone().requires_grad_(True)
        lp, ent = autograd.token_logprobs(xr, tokens.view(shape[:-1]))
        (lp.sum() - 0.1 * ent.sum()).backward()              # expanded gradients
        grads.append(xr.grad.view(24, 501))
    assert torch.equal(*grads)
    xr = x.clone().requires_grad_(True)
    autograd.token_logprobs(xr, tokens)[0].sum().backward()  # the entropy unused
    r = det.det_token_logprobs(x, tokens)
    want = det.det_token_logprobs_backward(x, tokens, r.lse, grad_logprob=torch.ones(24, device="cuda"))
    assert torch.equal(xr.grad, want)


def test_graph_capture(det):
    x = torch.randn(9, 5003, device="cuda", dtype=torch.bfloat16)
    t = torch.arange(9, dtype=torch.int32, device="cuda")
    det.det_token_logprobs(x, t, top_k=4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = det.det_token_logprobs(x, t, top_k=4)
    for seed in range(3):
        x.copy_(torch.randn(9, 5003, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
        g.replay()
        assert all(torch.equal(p, q) for p, q in zip(r, det.det_token_logprobs(x, t, top_k=4)))


def test_large_offsets(det):
    """Rows beyond 2^31 elements into the logits."""
    rows, vocab = 40_000, 60_001
    x = torch.zeros(rows, vocab, dtype=torch.float16, device="cuda")
    x[rows - 1] = torch.randn(vocab, device="cuda").half()
    t = torch.full((rows,), 7, dtype=torch.int32, device="cuda")
    r = det.det_token_logprobs(x, t, top_k=3)
    one = det.det_token_logprobs(x[-1:].clone(), t[-1:], top_k=3)
    assert all(torch.equal(p[-1:], q) for p, q in zip(r, one))
    g = det.det_token_logprobs_backward(x, t, r.lse, r.entropy, grad_logprob=torch.ones_like(r.lse))
    h = det.det_token_logprobs_backward(x[-1:].clone(), t[-1:], one.lse, one.entropy, grad_logprob=torch.ones_like(one.lse))
    assert torch.equal(g[-1:], h)
