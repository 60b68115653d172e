"""det_embedding and its gradient.  The forward is one product and one rounding, the gradient the sums of
det_scatter_add_rows in 32 bits, one product and one rounding: both are compared bit for bit with a statement on the
CPU, the sums with the oracle's."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def det():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    oracle.build()
    return d


def bits(t):
    return t.detach().cpu().contiguous().view(torch.uint8)


def same(a, b):
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(bits(a), bits(b))


def forward_of(table, tokens, scale, dtype):
    t = tokens.long()
    known = (t >= 0) & (t < table.shape[0])
    rows = torch.zeros(*t.shape, table.shape[1])
    if table.shape[0]:
        rows = table.float()[t.clamp(0, table.shape[0] - 1)] * torch.tensor(scale, dtype=torch.float32)
    return torch.where(known[..., None], rows, torch.zeros(())).to(dtype)


def gradient_of(grad, tokens, vocab, scale, dtype, old=None):
    g = grad.float().reshape(-1, grad.shape[-1]).numpy()
    total, _ = oracle.det_scatter_add_rows(np.zeros((vocab, g.shape[1]), np.float32), tokens.reshape(-1).numpy(), g)
    total = torch.from_numpy(total) * torch.tensor(scale, dtype=torch.float32)
    if old is None:
        return total.to(dtype)
    met = torch.zeros(vocab, dtype=torch.bool)
    t = tokens.reshape(-1).long()
    met[t[(t >= 0) & (t < vocab)]] = True
    return torch.where(met[:, None], (old.float() + total).to(dtype), old)


SIZES = [(0, 5, 8), (1, 1, 1), (1, 5, 7), (3, 40, 8), (33, 5, 64), (64, 1000, 250), (130, 7, 256), (257, 1025, 257),
         (1000, 300, 1001), (70, 70000, 24), (5, 3, 9000)]


@pytest.mark.parametrize("n,vocab,dim", SIZES)
@pytest.mark.parametrize("kind", list(DTYPES))
def test_forward(det, n, vocab, dim, kind):
    g = torch.Generator().manual_seed(n + dim)
    table = torch.randn(vocab, dim, generator=g).to(DTYPES[kind])
    tokens = torch.randint(-2, vocab + 2, (n,), generator=g, dtype=torch.int32)
    for scale in (1.0, dim ** 0.5):
        for dtype in DTYPES.values():
            got = det.det_embedding(table.cuda(), tokens.cuda(), scale=scale, dtype=dtype)
            assert same(got, forward_of(table, tokens, scale, dtype))


def test_forward_of_strided_tables_shapes_and_addresses(det):
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(50, 300, generator=g).bfloat16()
    tokens = torch.randint(0, 50, (3, 5), generator=g, dtype=torch.int32)
    for cut in (slice(0, 256), slice(8, 264), slice(1, 250), slice(3, 4)):
        got = det.det_embedding(wide.cuda()[:, cut], tokens.cuda(), scale=3.0)
        assert same(got, forward_of(wide[:, cut], tokens, 3.0, torch.bfloat16))
    room = torch.empty(15 * 64 + 8, dtype=torch.float16, device="cuda")
    for off in (0, 1, 8):
        out = room[off:off + 15 * 64].view(3, 5, 64)
        got = det.det_embedding(wide.cuda()[:, :64], tokens.cuda(), out=out)
        assert got.data_ptr() == out.data_ptr() and same(got, forward_of(wide[:, :64], tokens, 1.0, torch.float16))
    # no vocabulary, infinities and NaN
    assert det.det_embedding(torch.empty(0, 8, device="cuda"), tokens.cuda()).eq(0).all()
    table = torch.tensor([[float("inf"), float("nan"), -0.0, 1e38]])
    got = det.det_embedding(table.cuda(), torch.zeros(1, dtype=torch.int32).cuda(), scale=10.0).cpu()[0]
    assert got[0] == float("inf") and got[1].isnan() and got[2] == 0 and got[3] == float("inf")


@pytest.mark.parametrize("n,vocab,dim", SIZES)
@pytest.mark.parametrize("kind", list(DTYPES))
def test_gradient(det, n, vocab, dim, kind):
    g = torch.Generator().manual_seed(n + dim)
    grad = torch.randn(n, dim, generator=g).to(DTYPES[kind])
    tokens = torch.randint(-2, vocab + 2, (n,), generator=g, dtype=torch.int32)
    for scale in (1.0, dim ** 0.5):
        for dtype in DTYPES.values():
            got = det.det_embedding_backward(grad.cuda(), tokens.cuda(), vocab, scale=scale, dtype=dtype)
            assert same(got, gradient_of(grad, tokens, vocab, scale, dtype))


# runs of every length around a block of 32 ranks, around whole blocks, and of most places
@pytest.mark.parametrize("dim", [3, 64, 328])
@pytest.mark.parametrize("lengths", [[31], [32], [33], [64, 65], [1, 31, 32, 33, 34, 1, 1, 95, 96, 97], [5000, 3, 1],
                                     [255, 256, 257, 258], [8191], [2] * 40 + [1023, 1025], [16 * 1024 + 1, 700]])
def test_gradient_of_long_runs(det, lengths, dim):
    g = torch.Generator().manual_seed(sum(lengths))
    tokens = torch.repeat_interleave(torch.arange(len(lengths)) * 3 + 1, torch.tensor(lengths)).int()
    tokens = tokens[torch.randperm(tokens.numel(), generator=g)].contiguous()
    vocab = 3 * len(lengths) + 2
    for kind, dtype in (("f32", torch.float32), ("bf16", torch.bfloat16), ("bf16", torch.float32)):
        grad = torch.randn(tokens.numel(), dim, generator=g).to(DTYPES[kind])
        got = det.det_embedding_backward(grad.cuda(), tokens.cuda(), vocab, scale=0.75, dtype=dtype)
        assert same(got, gradient_of(grad, tokens, vocab, 0.75, dtype))
        old = torch.randn(vocab, dim, generator=g).to(dtype)
        table = old.cuda()
        det.det_embedding_backward(grad.cuda(), tokens.cuda(), vocab, scale=0.75, grad_table=table, accumulate=True)
        assert same(table, gradient_of(grad, tokens, vocab, 0.75, dtype, old))


@pytest.mark.parametrize("window", [100, 700, 5000, 40000])
def test_gradient_does_not_depend_on_the_launch(det, window):
    """The number of tokens and columns decides how many positions a warp takes."""
    g = torch.Generator().manual_seed(window)
    tokens = (torch.rand(window, generator=g) ** 4 * 2000).int()
    grad = torch.randn(window, 520, generator=g).bfloat16()
    want = det.det_embedding_backward(grad.cuda(), tokens.cuda(), 2000, dtype=torch.float32)
    for c in range(0, 520, 104):
        got = det.det_embedding_backward(grad[:, c:c + 104].cuda(), tokens.cuda(), 2000, dtype=torch.float32)
        assert torch.equal(got, want[:, c:c + 104])
    # the same rows among others
    more = torch.cat([tokens, torch.randint(2000, 3000, (window,), generator=g).int()])
    order = torch.argsort(torch.rand(2 * window, generator=g))
    order = torch.cat([order[order < window].sort().values, order[order >= window]])     # the old ones keep theirs
    mixed = torch.zeros(2 * window, dtype=torch.long)
    places = torch.randperm(2 * window, generator=g)
    mixed[places[:window].sort().values] = order[:window]
    mixed[places[window:].sort().values] = order[window:]
    both = torch.cat([grad, torch.randn(window, 520, generator=g).bfloat16()])
    got = det.det_embedding_backward(both[mixed].cuda(), more[mixed].contiguous().cuda(), 3000, dtype=torch.float32)
    assert torch.equal(got[:2000], want)
    assert same(want[:, :3], gradient_of(grad[:, :3], tokens, 2000, 1.0, torch.float32))


def test_gradient_of_strided_rows_and_skipped_ones(det):
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(200, 80, generator=g).half()
    tokens = torch.randint(0, 9, (200,), generator=g, dtype=torch.int32)
    tokens[::3] = -1
    wide[::3] = float("nan")                                       # a skipped row is not read
    for cut in (slice(0, 64), slice(8, 72), slice(1, 60)):
        got = det.det_embedding_backward(wide.cuda()[:, cut], tokens.cuda(), 9, dtype=torch.float32)
        clean = torch.where((tokens < 0)[:, None], torch.zeros(()).half(), wide)[:, cut]
        assert same(got, gradient_of(clean, tokens, 9, 1.0, torch.float32))
    grad = wide[:, :64].view(20, 10, 64).cuda()
    got = det.det_embedding_backward(grad, tokens.view(20, 10).cuda(), 9, dtype=torch.float32)
    assert same(got, det.det_embedding_backward(grad.view(200, 64), tokens.cuda(), 9, dtype=torch.float32))


def test_autograd(det):
    from deterministic_floating_point_gb300 import autograd
    g = torch.Generator().manual_seed(6)
    table = torch.randn(40, 48, generator=g)
    tokens = torch.randint(-1, 40, (6, 30), generator=g, dtype=torch.int32)
    weights = torch.randn(6, 30, 48, generator=g).bfloat16()
    leaf = table.cuda().requires_grad_(True)
    out = autograd.embedding(leaf, tokens.cuda(), scale=2.0, dtype=torch.bfloat16)
    (out * weights.cuda()).sum().backward()
    assert leaf.grad.dtype == torch.float32
    assert same(leaf.grad, gradient_of(weights, tokens, 40, 2.0, torch.float32))
    # an expanded gradient, and differences of the formula (linear, so exact but for roundings of 64 bits)
    leaf.grad = None
    autograd.embedding(leaf, tokens.cuda()).sum().backward()
    count = torch.bincount(tokens[tokens >= 0].long(), minlength=40)
    assert torch.equal(leaf.grad.cpu(), count[:, None].expand(40, 48).float())
    d = torch.randn(40, 48, generator=g).double()
    t = tokens.long().clamp(min=0)
    f = lambda w: (torch.where((tokens >= 0)[..., None], 2.0 * w[t], torch.zeros(()).double()) * weights.double()).sum()
    slope = (f(table.double() + d) - f(table.double() - d)) / 2
    grad = gradient_of(weights, tokens, 40, 2.0, torch.float32).double()
    assert abs(float((grad * d).sum() - slope)) <= 2.0 ** -20 * float((grad.abs() * d.abs()).sum() + 1)
