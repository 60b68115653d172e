"""Sums of -0.0 in the embedding's gradient: a row counts as +0.0 before anything is added to it, as in
det_scatter_add_rows, so without accumulate no sum is -0.0.  Compared bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
from test_gpu_embedding import det, same  # noqa: E402,F401

RUNS = [1, 2, 7, 8, 9, 32, 33, 64, 300]          # a run of each token: within a block, whole ones, joined ones


def make(dim, dtype, extra, seed):
    """Every token's columns: all -0.0, all +0.0, one value among -0.0, values that cancel, as far as the run allows."""
    g = torch.Generator().manual_seed(seed)
    tokens = torch.cat([torch.repeat_interleave(torch.arange(len(RUNS)), torch.tensor(RUNS)) * 2 + 1,
                        torch.full((extra,), 2 * len(RUNS) + 1)]).int()
    order = torch.randperm(tokens.numel(), generator=g)
    grad = torch.full((tokens.numel(), dim), -0.0)
    grad[:, 1::5] = 0.0
    grad[:, 2::5] = torch.randn(grad[:, 2::5].shape, generator=g)
    first = torch.cat([torch.ones(1, dtype=torch.bool), tokens[1:] != tokens[:-1]])
    grad[first, 3::5] = 1.5
    grad[torch.cat([torch.zeros(1, dtype=torch.bool), first[:-1]]) & ~first, 3::5] = -1.5      # 1.5 - 1.5 is +0.0
    return tokens[order].contiguous(), grad[order].to(dtype).contiguous(), 2 * len(RUNS) + 3


@pytest.mark.parametrize("extra", [0, 40_000])   # past the small sort
@pytest.mark.parametrize("dim", [5, 64, 250])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, torch.float16])
def test_sums_of_negative_zeros(det, kind, dim, extra):  # noqa: F811
    tokens, grad, vocab = make(dim, kind, extra, dim)
    total, _ = oracle.det_scatter_add_rows(np.zeros((vocab, dim), np.float32), tokens.numpy(), grad.float().numpy())
    total = torch.from_numpy(total)
    tc, gc = tokens.cuda(), grad.cuda()
    for scale in (1.0, -1.0, -0.75):
        want = total * torch.tensor(scale) + 0.0
        for dtype in (torch.float32, torch.bfloat16):
            got = det.det_embedding_backward(gc, tc, vocab, scale=scale, dtype=dtype)
            assert same(got, want.to(dtype)), (scale, dtype)
            table = torch.zeros(vocab, dim, dtype=dtype, device="cuda")
            det.det_embedding_backward(gc, tc, vocab, scale=scale, grad_table=table, accumulate=True)
            assert same(table, got)
    # on a table of -0.0, as det_scatter_add_rows on it
    old = np.full((vocab, dim), -0.0, np.float32)
    want, _ = oracle.det_scatter_add_rows(old.copy(), tokens.numpy(), grad.float().numpy())
    table = torch.from_numpy(old).cuda()
    det.det_embedding_backward(gc, tc, vocab, grad_table=table, accumulate=True)
    assert same(table, torch.from_numpy(want))


def test_a_masked_token_met_once(det):  # noqa: F811
    grad = -(torch.zeros(3, 8, device="cuda"))
    got = det.det_embedding_backward(grad, torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda"), 6)
    assert not torch.signbit(got).any()
