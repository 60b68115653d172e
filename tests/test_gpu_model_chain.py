"""The language-model operators after one another on one stream: their kernels are launched before the kernel ahead has
ended, and must have waited for its results.  Each chain is run with a synchronization after every call and without."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def det():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    return d


def both_ways(chain):
    def run(wait):
        step = torch.cuda.synchronize if wait else (lambda: None)
        result = chain(step)
        torch.cuda.synchronize()
        return result
    want = run(True)
    for _ in range(3):
        got = run(False)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_attention_of_its_own_output(det):
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(600, 16, 4, 64, generator=g).bfloat16().cuda() for _ in range(2))
    q0 = torch.randn(6, 16, 64, generator=g).bfloat16().cuda()
    table = torch.randperm(600, generator=g).int().view(6, 100).cuda()
    lengths = torch.tensor([1600, 1, 500, 700, 1200, 90], dtype=torch.int32).cuda()

    def chain(step):
        q, lses, kk = q0, [], k.clone()
        for i in range(12):
            r = det.det_paged_attention(q, kk, v, table, lengths)
            step()
            q = (r.out if i % 2 else r.out * 3)
            kk[i, 3, :, :] = q[0, :4]       # the next call reads what this one gave
            lses.append(r.lse)
            step()
        return [q, *lses]
    both_ways(chain)


def test_bias_of_its_own_gradient(det):
    bounds = det.det_relative_bounds(32, 128)
    table0 = torch.randn(32, 8, generator=torch.Generator().manual_seed(2)).cuda()

    def chain(step):
        table, all_tables = table0, []
        for i in range(8):
            bias = det.det_relative_bias(table, bounds, 700 + i, 901)
            step()
            table = det.det_relative_bias_backward(bias, bounds)
            step()
            table = table / table.abs().amax()
            one = det.det_relative_bias(table, bounds, 1, 901, q_offset=900)
            step()
            all_tables += [table, one]
        return all_tables
    both_ways(chain)


@pytest.mark.parametrize("rows", [2, 400])
def test_log_probabilities_of_their_own_gradient(det, rows):
    x0 = torch.randn(rows, 40_001, generator=torch.Generator().manual_seed(3)).cuda()
    ones = torch.ones(rows, device="cuda")

    def chain(step):
        x, results = x0, []
        tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        for _ in range(6):
            r = det.det_token_logprobs(x, tokens, top_k=4)
            step()
            tokens = r.top_index[:, 1].contiguous()
            g = det.det_token_logprobs_backward(x, tokens, r.lse, r.entropy, grad_logprob=ones, grad_entropy=r.entropy)
            step()
            again = det.det_token_logprobs(g, tokens, top_k=4)   # reads the gradient at once
            step()
            x = x + g
            results += [r.logprob, r.entropy, again.lse, again.top_index]
        return results
    both_ways(chain)


def test_operators_after_each_other(det):
    """Logits' gradient, attention, bias and a sort of the library read what the operator before has written."""
    g = torch.Generator().manual_seed(4)
    bounds = det.det_relative_bounds(32, 128)
    k, v = (torch.randn(64, 16, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.arange(64).int().view(2, 32).cuda()
    lengths = torch.tensor([512, 300], dtype=torch.int32).cuda()
    q0 = torch.randn(2, 4, 64, generator=g).bfloat16().cuda()

    def chain(step):
        q, results = q0, []
        for _ in range(6):
            out, lse = det.det_paged_attention(q, k, v, table, lengths)
            step()
            r = det.det_token_logprobs(out.view(8, 64), top_k=8)
            step()
            bins = r.top_index.view(-1)
            total = torch.zeros(64, device="cuda")
            det.det_scatter_add(total, bins, r.top_logprob.view(-1))
            step()
            bias = det.det_relative_bias(total.view(32, 2).contiguous(), bounds, 64, 64)
            step()
            q = (bias.view(-1)[:512].view(2, 4, 64) + out.float()).bfloat16()
            step()
            results += [out, lse, total, bias]
        return results
    both_ways(chain)
