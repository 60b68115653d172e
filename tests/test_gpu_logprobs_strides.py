"""Logits and tokens of the strides that programs have: a padded vocabulary, and the shift of tokens by one."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def mods():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build
    _build.build()
    from deterministic_floating_point_gb300 import autograd, det
    return det, autograd


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lead", [(3, 17), (1, 17), (17, 1), (2, 3, 4), (1, 1)])
def test_a_padded_vocabulary(mods, dtype, lead):
    det, _ = mods
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(*lead, 1024, generator=g).to(DTYPES[dtype]).cuda()
    tokens = torch.randint(0, 1003, lead, generator=g).int().cuda()
    x = wide[..., :1003]
    got, want = (det.det_token_logprobs(t, tokens, top_k=3) for t in (x, x.contiguous()))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    gl = torch.randn(lead, generator=g).cuda()
    a, b = (det.det_token_logprobs_backward(t, tokens, want.lse, grad_logprob=gl) for t in (x, x.contiguous()))
    assert torch.equal(a, b)


def test_rows_at_different_strides_are_refused(mods):
    det, _ = mods
    x = torch.randn(3, 5, 40, device="cuda")
    t = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        det.det_token_logprobs(x[:, :-1], t)
    with pytest.raises(ValueError):
        det.det_token_logprobs(x.transpose(0, 1), t.t().contiguous())


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_the_shift(mods, dtype):
    """autograd of logits[:, :-1] against tokens[:, 1:]: the results and the gradient of whole logits with a token of -1 at the end."""
    det, autograd = mods
    g = torch.Generator().manual_seed(2)
    x0 = torch.randn(3, 9, 501, generator=g).to(DTYPES[dtype]).cuda()
    tokens = torch.randint(0, 501, (3, 9), generator=g).int().cuda()
    w = torch.randn(3, 8, generator=g).cuda()
    x = x0.clone().requires_grad_(True)
    lp, ent = autograd.token_logprobs(x[:, :-1], tokens[:, 1:])
    ((lp + 0.3 * ent) * w).sum().backward()
    y = x0.clone().requires_grad_(True)
    ends = torch.cat([tokens[:, 1:], torch.full_like(tokens[:, :1], -1)], 1)
    lp2, ent2 = autograd.token_logprobs(y, ends)
    ((lp2 + 0.3 * ent2)[:, :-1] * w).sum().backward()
    assert torch.equal(lp, lp2[:, :-1]) and torch.equal(ent, ent2[:, :-1]) and torch.equal(x.grad, y.grad)
    # columns that are not neighbours, and transposed rows
    z = x0.clone().requires_grad_(True)
    autograd.token_logprobs(z[..., ::2], tokens // 2)[0].sum().backward()
    assert torch.all(z.grad[..., 1::2] == 0) and torch.any(z.grad != 0)
    a = autograd.token_logprobs(x0.transpose(0, 1), tokens.t())
    b = autograd.token_logprobs(x0, tokens)
    assert torch.equal(a[0].t(), b[0]) and torch.equal(a[1].t(), b[1])
