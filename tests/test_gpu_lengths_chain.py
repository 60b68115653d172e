"""det_paged_attention in a decoding loop: lengths and pages change between calls on the device, without a synchronization."""
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


@pytest.mark.parametrize("lengths", [[500, 1010, 1, 8190, 511, 1023], [16_380, 3, 16_384, 2000, 40, 9000]])
def test_lengths_that_grow_between_calls(det, lengths):
    """Steps over the edges where a sequence gets a second chunk, or chunks of another size."""
    g = torch.Generator().manual_seed(1)
    batch, page, per = len(lengths), 16, 1100
    k, v = (torch.randn(batch * per, page, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    q0 = torch.randn(batch, 16, 64, generator=g).bfloat16().cuda()
    table0 = torch.randperm(batch * per, generator=g).int().view(batch, per).cuda()
    n0 = torch.tensor(lengths, dtype=torch.int32).cuda()

    def chain(wait):
        q, n, table, got = q0.clone(), n0.clone(), table0.clone(), []
        for step in range(24):
            r = det.det_paged_attention(q, k, v, table, n)
            if wait:
                torch.cuda.synchronize()
            n += 1 if step % 5 else 97          # what the next call reads
            n.copy_(n.roll(1))
            table.copy_(table.roll(1, 0))
            q.copy_(r.out)
            q += q0
            got += [r.out, r.lse]
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return got
    want = chain(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))


def test_lengths_written_by_the_library_between_calls(det):
    """The lengths come from a kernel of the library that is itself launched early (the alternatives' indices)."""
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(300, 16, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.randperm(300, generator=g).int().view(3, 100).cuda()
    q0 = torch.randn(3, 4, 64, generator=g).bfloat16().cuda()
    scores = torch.randn(3, 1600, generator=g).cuda()

    def chain(wait):
        q, got = q0, []
        for step in range(12):
            n = det.det_token_logprobs(scores.roll(step * 37, 1), top_k=1).top_index.view(3)
            if wait:
                torch.cuda.synchronize()
            r = det.det_paged_attention(q, k, v, table, n)
            if wait:
                torch.cuda.synchronize()
            q = r.out
            got += [n, r.out, r.lse]
        torch.cuda.synchronize()
        return got
    want = chain(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))
