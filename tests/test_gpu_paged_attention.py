"""det_paged_attention against the definition in 64 bits.

Tolerance of the output: the weights are held to 2^-16 of themselves or better (two 16-bit parts), scores are 32-bit sums of
exact products (D + 2 roundings at the size of sum |q k|, u = 2^-24) and the output is rounded once to its type:
|error| <= 2 (2^-15 + 2 u log2(e) (D + 8) max sum |scale q k|) max |v| + u_type |out|.  Of lse: the same without the weights' part."""
import math

import numpy as np
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


def make(seed, lengths, heads, kv_heads, dim, page, dtype, spare=2):
    g = torch.Generator().manual_seed(seed)
    batch = len(lengths)
    used = [-(-max(n, 0) // page) for n in lengths]
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=g)
    table = torch.full((batch, max(1, max(used))), -1, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u].int()
        at += u
    k = torch.randn(pages, page, kv_heads, dim, generator=g).to(DTYPES[dtype])
    v = torch.randn(pages, page, kv_heads, dim, generator=g).to(DTYPES[dtype])
    for b, n in enumerate(lengths):
        if n > 0 and n % page:
            k[int(table[b, used[b] - 1]), n % page:] = float("nan")     # never written: must not be read
            v[int(table[b, used[b] - 1]), n % page:] = float("nan")
    q = torch.randn(batch, heads, dim, generator=g).to(DTYPES[dtype])
    return [t.cuda() for t in (q, k, v, table, torch.tensor(lengths, dtype=torch.int32))]


def reference(q, k, v, table, lengths, scale=None, bias=None, bounds=None, keep=None):
    q, k, v, table = q.double().cpu(), k.double().cpu(), v.double().cpu(), table.cpu().long()
    batch, heads, dim = q.shape
    page, kv_heads = k.shape[1:3]
    scale = dim ** -0.5 if scale is None else scale
    out = torch.zeros_like(q)
    lse = torch.full((batch, heads), -math.inf, dtype=torch.float64)
    size = torch.zeros(batch, heads, dtype=torch.float64)      # largest sum |scale q k|
    for b in range(batch):
        n = min(max(int(lengths[b]), 0), table.shape[1] * page)
        at = torch.arange(n)
        p = table[b][at // page] if n else at
        ok = (p >= 0) & (p < k.shape[0])
        at, p = at[ok], p[ok]
        if len(at) == 0:
            continue
        kk, vv = k[p, at % page], v[p, at % page]              # tokens, kv_heads, dim
        kk = kk.repeat_interleave(heads // kv_heads, 1)
        vv = vv.repeat_interleave(heads // kv_heads, 1)
        x = torch.einsum("hd,nhd->hn", q[b], kk) * scale
        size[b] = (torch.einsum("hd,nhd->hn", q[b].abs(), kk.abs()) * abs(scale)).amax(1)
        if bias is not None:
            bucket = torch.from_numpy(np.searchsorted(np.asarray(bounds), (n - 1 - at).numpy(), side="right"))
            x = x + bias.double().cpu()[bucket].t()
        live = x.amax(1) > -math.inf
        lse[b] = torch.logsumexp(x, 1)
        w = torch.exp(x - torch.where(live, lse[b], torch.zeros_like(lse[b]))[:, None])
        out[b] = torch.einsum("hn,nhd->hd", w, vv)
    return out, lse, size


def check(det, args, **kw):
    q, k, v, table, lengths = args
    r = det.det_paged_attention(q, k, v, table, lengths, **kw)
    ref = {"scale": kw.get("scale"), "bias": kw.get("bias_table"),
           "bounds": kw["bias_bounds"].tolist() if "bias_bounds" in kw else None}
    out, lse, size = reference(q, k, v, table, lengths.tolist(), **ref)
    dim = q.shape[-1]
    if kw.get("bias_table") is not None:
        b = kw["bias_table"].double().cpu()
        size = size + torch.where(torch.isfinite(b), b.abs(), torch.zeros_like(b)).amax()
    vmax = torch.nan_to_num(v.double().cpu()).abs().amax()
    score = 2 * 2.0 ** -24 * 1.4427 * (dim + 8) * size
    u = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -11
    tol = 2 * (2.0 ** -15 + score)[..., None] * vmax + u * out.abs() + (2.0 ** -24 if u < 2.0 ** -8 else 0)
    err = (r.out.double().cpu() - out).abs()
    assert torch.all(err <= tol), (err - tol).max()
    got = r.lse.double().cpu()
    none = lse == -math.inf
    assert torch.equal(got == -math.inf, none)
    assert torch.all((got - lse).abs()[~none] <= (2 * (2.0 ** -20 + score) + 2.0 ** -22 * lse.abs())[~none])
    return r


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (8, 2), (7, 1), (16, 2), (18, 2), (40, 1), (33, 1)])
def test_heads_and_short_lengths(det, dtype, dim, heads, kv_heads):
    lengths = [1, 0, 2, 15, 16, 17, 63, 64, 65, 100, 255, 256, 257, 300, 513]
    check(det, make(heads, lengths, heads, kv_heads, dim, 16, dtype))


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 100, 1000])
@pytest.mark.parametrize("dim", [64, 128])
def test_page_sizes(det, page, dim):
    check(det, make(page, [700, 1, 0, 33, 1025], 8, 2, dim, page, "bf16"))


@pytest.mark.parametrize("lengths", [[8191, 8192, 8193], [16_383, 32_768, 32_769], [70_001], [0, 0, 0], [131_072, 1]])
def test_long_lengths(det, lengths):
    check(det, make(len(lengths), lengths, 4, 1, 64, 64, "bf16"))
    check(det, make(len(lengths), lengths, 8, 8, 128, 16, "f16")) if max(lengths) < 40_000 else None


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 48, 20])
def test_numbers_of_chunks(det, dim, page):
    """Sequences of one to 33 chunks of every size in one call, whatever the longest one is."""
    lengths = [512, 513, 768, 1024, 1025, 4096, 4097, 8192, 8193, 16_384, 16_385, 1, 0]
    q, k, v, table, n = make(dim, lengths, 18, 2, dim, page, "bf16")
    check(det, (q, k, v, table, n))
    for longest in (1000, 8192):
        r = det.det_paged_attention(q, k, v, table, n, max_len=longest)
        cut = det.det_paged_attention(q, k, v, table, n.clamp(max=longest))
        assert torch.equal(r.out, cut.out) and torch.equal(r.lse, cut.lse)
    # queries at odd elements
    odd = torch.zeros(len(lengths), 18, dim + 1, dtype=q.dtype, device="cuda")
    odd[..., 1:] = q
    r, want = det.det_paged_attention(odd[..., 1:], k, v, table, n), det.det_paged_attention(q, k, v, table, n)
    assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (8, 2), (12, 1)])
def test_learned_bias(det, dtype, heads, kv_heads):
    rng = np.random.default_rng(heads)
    args = make(5, [1, 700, 128, 129, 0, 3000], heads, kv_heads, 64, 16, dtype)
    for table_dtype in (torch.float32, torch.bfloat16, torch.float16):
        bounds = det.det_relative_bounds(32, 128)
        table = torch.from_numpy(rng.standard_normal((32, heads)) * 3).to(table_dtype).cuda()
        check(det, args, bias_table=table, bias_bounds=bounds)
    table = torch.randn(1, heads, device="cuda")
    check(det, args, bias_table=table, bias_bounds=torch.zeros(0, dtype=torch.int32, device="cuda"))
    # a bias of -inf masks distances; here everything but the nearest 8 tokens, or everything
    bounds = torch.tensor([8], dtype=torch.int32, device="cuda")
    table = torch.zeros(2, heads, device="cuda")
    table[1] = -math.inf
    check(det, args, bias_table=table, bias_bounds=bounds)
    table[0, 0] = -math.inf
    r = check(det, args, bias_table=table, bias_bounds=bounds)
    assert torch.all(r.out[:, 0] == 0) and torch.all(r.lse[:, 0] == -math.inf)


def test_bias_matches_the_bias_operator(det):
    """The bias of the last query of det_relative_bias is the one the attention adds."""
    bounds = det.det_relative_bounds(32, 128, bidirectional=True)
    table = torch.randn(32, 4, device="cuda")
    n = 500
    q, k, v, pages, lengths = make(1, [n], 4, 4, 64, 16, "f16")
    row = det.det_relative_bias(table, bounds, 1, n, q_offset=n - 1, bidirectional=True)[:, 0]
    got = check(det, (torch.zeros_like(q), k, v, pages, lengths), bias_table=table[:16].contiguous(), bias_bounds=bounds)
    assert torch.allclose(got.lse[0], torch.logsumexp(row.double(), 1).float(), rtol=0, atol=1e-5)
    both = det.det_paged_attention(q, k, v, pages, lengths, bias_table=table, bias_bounds=bounds)
    half = det.det_paged_attention(q, k, v, pages, lengths, bias_table=table[:16].contiguous(), bias_bounds=bounds)
    assert torch.equal(both.out, half.out)


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (4, 4, 64), (16, 1, 256)])
def test_a_sequence_does_not_depend_on_its_batch(det, heads, kv_heads, dim):
    lengths = [5000, 0, 300, 9000, 256, 12]
    q, k, v, table, n = make(3, lengths, heads, kv_heads, dim, 16, "bf16")
    a = det.det_paged_attention(q, k, v, table, n)
    for _ in range(3):
        b = det.det_paged_attention(q, k, v, table, n)
        assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
    for i in range(len(lengths)):
        b = det.det_paged_attention(q[i:i + 1], k, v, table[i:i + 1], n[i:i + 1], max_len=lengths[i])
        assert torch.equal(a.out[i:i + 1], b.out) and torch.equal(a.lse[i:i + 1], b.lse)
    # another order of the pages in memory
    perm = torch.randperm(k.shape[0], device="cuda")
    inv = torch.argsort(perm).int()
    moved = torch.where(table >= 0, inv[table.clamp(min=0).long()], table)
    b = det.det_paged_attention(q, k[perm], v[perm], moved, n)
    assert torch.equal(a.out, b.out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = det.det_paged_attention(q, k, v, table, n, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a.out, b.out)


def test_strides(det):
    lengths = [100, 777, 3]
    q, k, v, table, n = make(4, lengths, 8, 2, 64, 16, "f16")
    want = det.det_paged_attention(q, k, v, table, n)
    # heads before tokens, keys and values interleaved, wider rows, a wider table, shifted queries
    kh = k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    both = torch.stack((k, v), 3)
    wide = torch.full((*k.shape[:3], 96), float("nan"), dtype=k.dtype, device="cuda")
    wide[..., 16:80] = v
    wq = torch.zeros(3, 9, 71, dtype=q.dtype, device="cuda")
    wq[:, :8, 3:67] = q
    wt = torch.full((3, table.shape[1] + 5), 12345678, dtype=torch.int32, device="cuda")
    wt[:, :table.shape[1]] = table
    for kk, vv, qq, tt in ((kh, v, q, table), (both[:, :, :, 0], both[:, :, :, 1], q, table),
                           (k, wide[..., 16:80], wq[:, :8, 3:67], wt[:, :table.shape[1]]), (k, v, q, wt)):
        got = det.det_paged_attention(qq, kk, vv, tt, n)
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)


def test_skipped_pages_and_cut_lengths(det):
    q, k, v, table, n = make(6, [640, 640, 640, 640], 4, 2, 64, 16, "bf16")
    table[0, 3] = -1
    table[0, 39] = k.shape[0]
    table[1, :] = 2_000_000_000
    table[2, 1:] = -5
    n[3] = 100_000                       # beyond the table: cut to it
    r = check(det, (q, k, v, table, n))
    assert torch.all(r.out[1] == 0) and torch.all(r.lse[1] == -math.inf)
    n2 = torch.tensor([-7, 640, 640, 10], dtype=torch.int32, device="cuda")
    r = check(det, (q, k, v, table, n2))
    assert torch.all(r.out[0] == 0)
    # max_len cuts, and a cut sequence is the shorter sequence
    n3 = torch.tensor([640, 640, 640, 640], dtype=torch.int32, device="cuda")
    a = det.det_paged_attention(q, k, v, table, n3, max_len=100)
    b = det.det_paged_attention(q, k, v, table, torch.full_like(n3, 100))
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_no_sequences_no_pages(det):
    q, k, v, table, n = make(6, [10, 20], 4, 2, 64, 16, "bf16")
    assert det.det_paged_attention(q[:0], k, v, table[:0], n[:0]).out.shape == (0, 4, 64)
    r = det.det_paged_attention(q, k, v, table[:, :0], n)
    assert torch.all(r.out == 0) and torch.all(r.lse == -math.inf)
    r = det.det_paged_attention(q, k[:0], v[:0], table, n)
    assert torch.all(r.out == 0) and torch.all(r.lse == -math.inf)
    r = det.det_paged_attention(q, k, v, table, n, max_len=0)
    assert torch.all(r.out == 0)


def test_special_values(det):
    q, k, v, table, n = make(8, [300, 300, 300], 4, 4, 64, 16, "bf16")
    page = int(table[0, 2])
    k[page, 5, 1] = float("nan")           # head 1 of sequence 0
    v[int(table[1, 2]), 5, 2, 7] = float("inf")
    v[int(table[1, 3]), 5, 2, 8] = float("nan")
    r = det.det_paged_attention(q, k, v, table, n)
    assert torch.all(torch.isnan(r.out[0, 1])) and torch.isnan(r.lse[0, 1])
    assert not torch.isnan(r.out[0, [0, 2, 3]]).any()
    assert torch.isnan(r.out[1, 2, 8]) and not torch.isfinite(r.out[1, 2, 7])
    assert torch.isfinite(r.out[1, [0, 1, 3]]).all() and torch.isfinite(r.out[2]).all()
    # large scores: one token takes all the weight
    q2, k2, v2, t2, n2 = make(9, [500], 2, 2, 64, 16, "bf16")
    k2.mul_(60)
    check(det, (q2 * 10, k2, v2, t2, n2))
    check(det, make(9, [500], 2, 2, 64, 16, "bf16"), scale=-0.3)
    check(det, make(9, [500], 2, 2, 64, 16, "bf16"), scale=0.0)


def test_offsets_beyond_32_bits(det):
    """A cache of more than 2^31 elements whose used pages lie at its end."""
    pages, page = 40_000, 128
    k = torch.empty(pages, page, 4, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 1 << 31
    k[-8:] = torch.randn(8, page, 4, 128, device="cuda").bfloat16()
    v[-8:] = torch.randn(8, page, 4, 128, device="cuda").bfloat16()
    q = torch.randn(1, 8, 128, device="cuda").bfloat16()
    n = torch.tensor([1000], dtype=torch.int32, device="cuda")
    table = torch.arange(pages - 8, pages, dtype=torch.int32, device="cuda").flip(0)[None]
    got = det.det_paged_attention(q, k, v, table, n)
    small = det.det_paged_attention(q, k[-8:], v[-8:], table - (pages - 8), n)
    assert torch.equal(got.out, small.out) and torch.equal(got.lse, small.lse)
    check(det, (q, k[-8:], v[-8:], table - (pages - 8), n))


def test_graph_and_leftover_workspace(det):
    q, k, v, table, n = make(10, [5000, 100], 8, 2, 64, 16, "bf16")
    want = det.det_paged_attention(q, k, v, table, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = det.det_paged_attention(q, k, v, table, n)
    for lengths in ([5000, 100], [17, 4000], [0, 1]):
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        table[:] = table[0].clone() if max(lengths) > 100 else table
        graph.replay()
        now = det.det_paged_attention(q, k, v, table, n)
        assert torch.equal(r.out, now.out) and torch.equal(r.lse, now.lse)
    q, k, v, table, n = make(10, [5000, 100], 8, 2, 64, 16, "bf16")
    need = det.lib().det_paged_attention_workspace_bytes(2, 8, 64, table.shape[1] * 16)
    ws = det.workspace(need, "cuda")
    ws.fill_(255)
    got = det.det_paged_attention(q, k, v, table, n, workspace=ws)
    assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)
