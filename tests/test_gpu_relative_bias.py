"""det_relative_bias and its gradient against plain statements: the forward is a
table lookup and has to be equal, the gradient is a sum in 64 bits.

Tolerance of the gradient: u = 2^-24 relative to the sum of |g| in a bucket for each addition in a row; the sums are trees of
short runs, at most 256 additions on any path of the sizes here, and the result is rounded once to the table's type."""
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


def buckets_of(bounds, q_len, k_len, off, both):
    r = np.arange(k_len)[None, :] - np.arange(q_len)[:, None] - off
    n = np.abs(r) if both else np.maximum(-r, 0)
    k = np.searchsorted(np.asarray(bounds), n, side="right")
    return np.where((r > 0) & both, k + len(bounds) + 1, k)


BOUNDS = {
    "log32": lambda det: det.det_relative_bounds(32, 128, device="cpu").tolist(),
    "one": lambda det: [],
    "clip": lambda det: list(range(1, 40)),
    "repeated": lambda det: [0, 0, 3, 3, 3, 10, 500],          # empty buckets, and one that nothing reaches
    "many": lambda det: list(range(1, 2048)),
}

SHAPES = [(1, 1, 0), (1, 1, 5), (1, 300, 299), (7, 5, 0), (5, 7, 2), (64, 64, 0), (65, 129, 64), (130, 67, 0),
          (33, 520, 487), (8, 8, -20), (257, 263, 1000)]


@pytest.mark.parametrize("name", list(BOUNDS))
@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_forward_is_the_table_entry(det, name, both, dtype):
    bounds = BOUNDS[name](det)
    rows = (len(bounds) + 1) * (2 if both else 1)
    rng = np.random.default_rng(rows)
    for heads, (q_len, k_len, off) in zip((1, 3, 2, 5, 1, 8, 2, 3, 4, 1, 2), SHAPES):
        table = torch.from_numpy(rng.standard_normal((rows, heads)).astype(np.float32)).to(DTYPES[dtype]).cuda()
        bt = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        k = torch.from_numpy(buckets_of(bounds, q_len, k_len, off, both)).cuda()
        want = table.t()[:, k]
        got = det.det_relative_bias(table, bt, q_len, k_len, q_offset=off, bidirectional=both)
        assert got.dtype == table.dtype and torch.equal(got, want), (heads, q_len, k_len, off)
        for other in DTYPES.values():
            if table.dtype == torch.float32:
                got = det.det_relative_bias(table, bt, q_len, k_len, q_offset=off, bidirectional=both, dtype=other)
                assert torch.equal(got, want.to(other))
    # results at every alignment of the first element
    table = table[:, :1].contiguous()
    for shift in range(9):
        room = torch.full((9 + 37 * 53 + 9,), 3.0, dtype=table.dtype, device="cuda")
        out = room[shift:shift + 37 * 53].view(1, 37, 53)
        det.det_relative_bias(table, bt, 37, 53, bidirectional=both, out=out)
        k = torch.from_numpy(buckets_of(bounds, 37, 53, 0, both)).cuda()
        assert torch.equal(out, table.t()[:, k])
        assert torch.all(room[:shift] == 3) and torch.all(room[shift + 37 * 53:] == 3)


def grad_reference(g, bounds, off, both):
    g = g.double().cpu().numpy()
    if g.ndim == 4:
        a, g = np.abs(g).sum(0), g.sum(0)
    else:
        a = np.abs(g)
    heads, q_len, k_len = g.shape
    k = buckets_of(bounds, q_len, k_len, off, both).reshape(-1)
    rows = (len(bounds) + 1) * (2 if both else 1)
    out, size = np.zeros((rows, heads)), np.zeros((rows, heads))
    for h in range(heads):
        out[:, h] = np.bincount(k, weights=g[h].reshape(-1), minlength=rows)
        size[:, h] = np.bincount(k, weights=a[h].reshape(-1), minlength=rows)
    return out, size


@pytest.mark.parametrize("name", list(BOUNDS))
@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_gradient_against_64_bits(det, name, both, dtype):
    bounds = BOUNDS[name](det)
    bt = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(len(bounds))
    for batch, heads, (q_len, k_len, off) in zip((1, 2, 3, 1, 2, 4, 2, 1, 3, 2, 2), (1, 3, 2, 5, 1, 8, 2, 3, 4, 1, 2), SHAPES):
        g = torch.from_numpy(rng.standard_normal((batch, heads, q_len, k_len)).astype(np.float32)).to(DTYPES[dtype]).cuda()
        want, size = grad_reference(g, bounds, off, both)
        got = det.det_relative_bias_backward(g, bt, q_offset=off, bidirectional=both)
        assert got.dtype == torch.float32
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= 256 * 2.0 ** -24 * size), (q_len, k_len)
        assert torch.equal(got, det.det_relative_bias_backward(g, bt, q_offset=off, bidirectional=both))
        again = det.det_relative_bias_backward(g, bt, q_offset=off, bidirectional=both, dtype=torch.bfloat16)
        assert torch.equal(again, got.bfloat16())
        one, _ = grad_reference(g[0], bounds, off, both)
        got1 = det.det_relative_bias_backward(g[0], bt, q_offset=off, bidirectional=both)
        assert np.all(np.abs(got1.double().cpu().numpy() - one) <= 256 * 2.0 ** -24 * size)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_gradient_bits_do_not_depend_on_layout(det, dtype):
    """Strides, alignment and the place of a head in the call change nothing."""
    rng = np.random.default_rng(2)
    bounds = det.det_relative_bounds(32, 128)
    for q_len, k_len in ((100, 203), (72, 136), (3, 1000)):
        g = torch.from_numpy(rng.standard_normal((2, 3, q_len, k_len)).astype(np.float32)).to(DTYPES[dtype]).cuda()
        want = det.det_relative_bias_backward(g, bounds, bidirectional=False, q_offset=50)
        for shift in range(9):
            room = torch.full((2, 3, q_len, k_len + 11), 5.0, dtype=g.dtype, device="cuda")
            room[..., shift:shift + k_len] = g
            assert torch.equal(det.det_relative_bias_backward(room[..., shift:shift + k_len], bounds, q_offset=50), want)
        perm = g.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
        assert torch.equal(det.det_relative_bias_backward(perm, bounds, q_offset=50), want)
        flip = g[:, [2, 0, 1]].contiguous()
        assert torch.equal(det.det_relative_bias_backward(flip, bounds, q_offset=50), want[:, [2, 0, 1]])
        # a broadcast gradient: batch and query strides of 0
        row = g[:1, :, :1].expand(2, 3, q_len, k_len)
        assert torch.equal(det.det_relative_bias_backward(row, bounds), det.det_relative_bias_backward(row.contiguous(), bounds))


def test_gradient_of_nothing_and_special_values(det):
    bounds = det.det_relative_bounds(8, 20)
    for shape in ((0, 2, 4, 5), (2, 2, 0, 5), (2, 2, 4, 0)):
        got = det.det_relative_bias_backward(torch.zeros(shape, device="cuda"), bounds)
        assert got.shape == (8, 2) and torch.all(got == 0)
    assert det.det_relative_bias_backward(torch.zeros((2, 0, 4, 5), device="cuda"), bounds).shape == (8, 0)
    assert det.det_relative_bias(torch.zeros(8, 2, device="cuda"), bounds, 0, 5).shape == (2, 0, 5)
    g = torch.zeros(1, 2, 40, 40, device="cuda")
    g[0, 0, 30, 30] = float("nan")          # distance 0
    g[0, 1, 30, 10] = float("inf")          # distance 20
    got = det.det_relative_bias_backward(g, bounds)
    assert torch.isnan(got[0, 0]) and torch.all(got[1:, 0] == 0)
    assert got[7, 1] == float("inf") and torch.all(got[:7, 1] == 0)
    # memory beside the pairs is not read
    room = torch.full((1, 1, 50, 64), float("nan"), device="cuda")
    room[..., :50] = 1.0
    assert torch.equal(det.det_relative_bias_backward(room[..., :50], bounds)[:, 0].cpu(),
                       torch.from_numpy(grad_reference(torch.ones(1, 50, 50), bounds.tolist(), 0, False)[0][:, 0]).float())


def test_exact_integer_sums_over_long_ranges(det):
    """Whole numbers: every order gives the same sum, so the result has to be equal."""
    rng = np.random.default_rng(8)
    bounds = det.det_relative_bounds(32, 128)
    for batch, heads, q_len, k_len, dt in ((3, 2, 1500, 2100, torch.float32), (2, 2, 2048, 2048, torch.bfloat16),
                                           (1, 1, 1, 30_001, torch.float32), (1, 1, 9000, 16, torch.float16)):
        g = torch.from_numpy(rng.integers(-1, 2, (batch, heads, q_len, k_len)).astype(np.float32)).to(dt).cuda()
        for both in (False, True):
            b = bounds[:15].contiguous() if both else bounds
            want, _ = grad_reference(g, b.tolist(), 3, both)
            assert np.array_equal(det.det_relative_bias_backward(g, b, q_offset=3, bidirectional=both).double().cpu().numpy(), want)


def test_autograd_and_differences(det):
    from deterministic_floating_point_gb300 import autograd
    rng = np.random.default_rng(9)
    bounds = det.det_relative_bounds(16, 40, bidirectional=True)
    for dt in DTYPES.values():
        table = torch.from_numpy(rng.standard_normal((16, 3))).to(dt).cuda().requires_grad_(True)
        w = torch.from_numpy(rng.standard_normal((4, 3, 30, 45))).float().cuda()
        bias = autograd.relative_bias(table, bounds, 30, 45, bidirectional=True, batch=4)
        assert bias.shape == (4, 3, 30, 45) and bias.stride(0) == 0
        (bias.float() * w).sum().backward()
        k = torch.from_numpy(buckets_of(bounds.tolist(), 30, 45, 0, True)).cuda()
        ref = table.detach().double().requires_grad_(True)
        (ref.t()[:, k][None] * w.double()).sum().backward()
        # bias.float()'s gradient is rounded to the type pair by pair, then the sum once
        u = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dt]
        size = torch.zeros(16, 3, dtype=torch.float64, device="cuda").index_add_(
            0, k.reshape(-1), w.double().abs().sum(0).reshape(3, -1).t())
        assert torch.all((table.grad.double() - ref.grad).abs() <= 2 * u * size)
        single = autograd.relative_bias(table, bounds, 30, 45, bidirectional=True)
        table.grad = None
        single.sum().backward()                # a gradient of stride 0
        assert torch.equal(table.grad.float(), torch.bincount(k.reshape(-1), minlength=16).float()[:, None].expand(16, 3).to(dt).float())
    # against differences: the loss is linear in the table, so any step gives the derivative
    table = torch.zeros(16, 1, device="cuda")
    w = torch.from_numpy(rng.integers(-2, 3, (1, 20, 20)).astype(np.float32)).cuda()
    grad = det.det_relative_bias_backward(w, bounds, bidirectional=True)
    for row in range(16):
        t = table.clone()
        t[row] = 1.0
        assert float((det.det_relative_bias(t, bounds, 20, 20, bidirectional=True) * w).sum()) == float(grad[row])


def test_other_stream_and_graph(det):
    g = torch.randn(2, 2, 300, 300, device="cuda")
    bounds = det.det_relative_bounds(32, 128)
    want = det.det_relative_bias_backward(g, bounds)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = det.det_relative_bias_backward(g, bounds, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = det.det_relative_bias_backward(g, bounds)
    g.mul_(2.0)
    graph.replay()
    assert torch.equal(out, 2 * want)
    # leftover contents of the workspace do not matter
    n = det.lib().det_relative_bias_backward_workspace_bytes(2, 2, 300, 300, 31, 0)
    ws = det.workspace(n, "cuda")
    ws.fill_(255)
    assert torch.equal(det.det_relative_bias_backward(g, bounds, workspace=ws), 2 * want)
