"""The embedding, the layer norm, the linear recurrence and their gradients as they are used together: after one another,
in captured graphs, on several streams, and at the ends of their ranges.  What is compared are bits: the values of each
are held against 64 bits by its own tests."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402


@pytest.fixture(scope="module")
def det():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    oracle.build()
    return d


def equal(a, b):
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)


class Model:
    """A small language model's inputs: tokens to embeddings, norm, recurrence, logits, log probabilities."""

    def __init__(self, batch, time, width, vocab, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.table = (torch.randn(vocab, width, generator=g) * 0.5).to(dtype).cuda()
        self.weight = (torch.rand(width, generator=g) + 0.5).cuda()
        self.bias = (torch.randn(width, generator=g) * 0.1).cuda()
        self.gate = (torch.randn(batch, time, width, generator=g) + 1).to(dtype).cuda()
        self.initial = torch.randn(batch, width, generator=g).cuda()
        self.tokens = torch.randint(-1, vocab, (batch, time), generator=g, dtype=torch.int32).cuda()
        self.next = torch.randint(0, vocab, (batch * time,), generator=g, dtype=torch.int32).cuda()
        self.lengths = torch.randint(0, time + 1, (batch,), generator=g, dtype=torch.int32).cuda()
        self.grad = torch.randn(batch, time, width, generator=g).to(dtype).cuda()
        self.ones = torch.ones(batch * time).cuda()

    def forward(self, det, step=lambda: None):
        e = det.det_embedding(self.table, self.tokens, scale=3.0)
        step()
        n = det.det_layer_norm(e, self.weight, self.bias)
        step()
        r = det.det_linear_recurrence(n.out, self.gate, self.initial, lengths=self.lengths, keep_states=True)
        step()
        return e, n, r

    def backward(self, det, e, n, r, grad, step=lambda: None, embed_ws=None, norm_ws=None):
        gr = det.det_linear_recurrence_backward(grad, n.out, self.gate, r.states, lengths=self.lengths)
        step()
        gn = det.det_layer_norm_backward(gr.x, e, n.mean, n.rstd, self.weight, workspace=norm_ws)
        step()
        ge = det.det_embedding_backward(gn.x, self.tokens, self.table.shape[0], scale=3.0, workspace=embed_ws)
        step()
        return [gr.x, gr.gate, gr.initial, gn.x, gn.weight, gn.bias, ge]

    def all(self, det, step=lambda: None, **ws):
        e, n, r = self.forward(det, step)
        # logits without a product: the states themselves, one column a token of a small vocabulary
        rows = r.out.view(-1, r.out.shape[-1])
        next = self.next % rows.shape[1]
        p = det.det_token_logprobs(rows, next)
        step()
        gp = det.det_token_logprobs_backward(rows, next, p.lse, p.entropy, grad_logprob=self.ones)
        step()
        return [e, n.out, n.mean, n.rstd, r.out, r.final, r.states, p.logprob, gp,
                *self.backward(det, e, n, r, gp.view(r.out.shape), step, **ws)]

    def workspaces(self, det):
        rows, width = self.tokens.numel(), self.table.shape[1]
        lib = det.lib()
        return dict(embed_ws=det.workspace(lib.det_embedding_backward_workspace_bytes(rows, self.table.shape[0], width), "cuda"),
                    norm_ws=det.workspace(lib.det_layer_norm_backward_workspace_bytes(rows, width), "cuda"))


CASES = [(3, 1, 64, 50, torch.float32), (2, 7, 250, 50, torch.bfloat16), (2, 700, 264, 300, torch.bfloat16),
         (1, 2000, 65, 70_000, torch.float16), (9, 2100, 128, 500, torch.float32)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_training_step_with_and_without_waiting(det, case):
    model = Model(*case)
    want = model.all(det, torch.cuda.synchronize)
    for _ in range(4):
        got = model.all(det)
        torch.cuda.synchronize()
        assert all(equal(a, b) for a, b in zip(got, want))
    # on the way to the parameters nothing is lost: autograd's gradients are these
    from deterministic_floating_point_gb300 import autograd
    leaves = [t.clone().requires_grad_(True) for t in (model.table, model.weight, model.bias, model.gate, model.initial)]
    table, weight, bias, gate, initial = leaves
    h = autograd.layer_norm(autograd.embedding(table, model.tokens, scale=3.0), weight, bias)
    h, _ = autograd.linear_recurrence(h, gate, initial, lengths=model.lengths)
    rows = h.view(-1, h.shape[-1])
    logprob, _ = autograd.token_logprobs(rows, model.next % rows.shape[1])
    logprob.sum().backward()
    by_hand = dict(zip(("x", "gate", "initial", "nx", "weight", "bias", "table"), want[9:]))
    for name, leaf in zip(("table", "weight", "bias", "gate", "initial"), leaves):
        assert equal(leaf.grad, by_hand[name]), name


@pytest.mark.parametrize("case", CASES, ids=str)
def test_graphs_that_share_workspaces(det, case):
    """A step captured twice over the same workspaces, replayed in turn on changed inputs."""
    models = [Model(*case, seed=s) for s in (1, 2)]
    ws = models[0].workspaces(det)
    for w in ws.values():
        w.fill_(0x5a)
    for m in models:
        m.all(det)                                       # before a capture: attributes of kernels are set
    torch.cuda.synchronize()
    graphs, results = [], []
    for m in models:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(m.all(det, **ws))
        graphs.append(graph)
    for seed in (1, 3, 4):
        for m, seed_of in zip(models, (seed, seed + 10)):
            new = Model(*case, seed=seed_of)
            for name, t in vars(new).items():
                getattr(m, name).copy_(t)
        for graph in graphs:
            graph.replay()
        got = [[t.clone() for t in r] for r in results]
        for m, r in zip(models, got):
            assert all(equal(a, b) for a, b in zip(r, m.all(det)))


def test_streams_at_once(det):
    """The same step on three streams at a time, each with its own tensors, while the others run."""
    cases = [CASES[2], CASES[4], CASES[3]]
    models = [Model(*c, seed=i) for i, c in enumerate(cases)]
    want = [m.all(det) for m in models]
    streams = [torch.cuda.Stream() for _ in models]
    torch.cuda.synchronize()
    got = [[] for _ in models]
    for _ in range(6):
        for m, s, g in zip(models, streams, got):
            with torch.cuda.stream(s):
                g.append(m.all(det))
    torch.cuda.synchronize()
    for runs, w in zip(got, want):
        for r in runs:
            assert all(equal(a, b) for a, b in zip(r, w))


def test_a_given_stream_orders_the_calls(det):
    """stream= alone decides the order: inputs that come late on that stream, results that are read on it."""
    m = Model(*CASES[2])
    e, n, r = m.forward(det)
    want = m.backward(det, e, n, r, m.grad)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    tokens, late = torch.full_like(m.tokens, -1), torch.zeros_like(m.grad)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        a = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            a = a @ a * 1e-3
        tokens.copy_(m.tokens)
        late.copy_(m.grad)
    e1 = det.det_embedding(m.table, tokens, scale=3.0, stream=side)
    n1 = det.det_layer_norm(e1, m.weight, m.bias, stream=side)
    r1 = det.det_linear_recurrence(n1.out, m.gate, m.initial, lengths=m.lengths, keep_states=True, stream=side)
    gr = det.det_linear_recurrence_backward(late, n1.out, m.gate, r1.states, lengths=m.lengths, stream=side)
    gn = det.det_layer_norm_backward(gr.x, e1, n1.mean, n1.rstd, m.weight, stream=side)
    ge = det.det_embedding_backward(gn.x, tokens, m.table.shape[0], scale=3.0, stream=side)
    side.synchronize()
    for a, b in zip([e1, n1.out, r1.out, r1.final, gr.x, gr.gate, gr.initial, gn.x, gn.weight, gn.bias, ge],
                    [e, n.out, r.out, r.final, *want]):
        assert equal(a, b)


def test_serving_steps_are_the_prompt_s(det):
    """Tokens one a call, states in place, captured once: the bits of each step are those of its rows in the prompt up to
    the recurrence; that one's, 32-bit over 8 steps, are too."""
    m = Model(4, 8, 96, 40, torch.float32)
    e, n, r = m.forward(det)
    whole = det.det_linear_recurrence(n.out, m.gate, m.initial)
    token, gate, state = m.tokens[:, :1].clone(), m.gate[:, :1].clone(), m.initial.clone()

    def one():
        x = det.det_layer_norm(det.det_embedding(m.table, token, scale=3.0), m.weight, m.bias).out
        return det.det_linear_recurrence(x, gate, state, final=state).out
    one()
    state.copy_(m.initial)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = one()
    for t in range(8):
        token.copy_(m.tokens[:, t:t + 1])
        gate.copy_(m.gate[:, t:t + 1])
        graph.replay()
        assert equal(out[:, 0], whole.out[:, t])
    assert equal(state, whole.final)


def test_no_second_derivatives(det):
    from deterministic_floating_point_gb300 import autograd
    m = Model(*CASES[1])
    table, x, gate = (t.float().requires_grad_(True) for t in (m.table, m.grad, m.gate))
    for out, leaf in ((autograd.embedding(table, m.tokens), table), (autograd.layer_norm(x, m.weight, m.bias), x),
                      (autograd.linear_recurrence(x, gate)[0], gate)):
        (g,) = torch.autograd.grad((out * out).sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError):
            g.square().sum().backward()


def test_gradient_of_the_norm_in_place(det):
    """grad_x over grad, as the C interface has it."""
    for rows, cols, dtype in ((40, 264, torch.bfloat16), (41, 63, torch.bfloat16), (300, 1000, torch.float32)):
        g = torch.Generator().manual_seed(cols)
        x, grad = (torch.randn(rows, cols, generator=g).to(dtype).cuda() for _ in range(2))
        w = torch.randn(cols, generator=g).cuda()
        r = det.det_layer_norm(x, w)
        want = det.det_layer_norm_backward(grad, x, r.mean, r.rstd, w)
        ws = det.workspace(det.lib().det_layer_norm_backward_workspace_bytes(rows, cols), "cuda")
        gw, gb = torch.empty_like(w), torch.empty_like(w)
        code = {torch.float32: 0, torch.bfloat16: 2}[dtype]
        rc = det.lib().det_layer_norm_backward(grad.data_ptr(), cols, x.data_ptr(), cols, code, rows, cols,
                                               r.mean.data_ptr(), r.rstd.data_ptr(), w.data_ptr(), 0, grad.data_ptr(),
                                               gw.data_ptr(), gb.data_ptr(), ws.data_ptr(), ws.numel(),
                                               torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        assert equal(grad, want.x) and equal(gw, want.weight) and equal(gb, want.bias)


def test_empty_sizes(det):
    none = torch.zeros(0, 8, device="cuda")
    tokens = torch.tensor([0, 1, -5], dtype=torch.int32, device="cuda")
    assert (det.det_embedding(none, tokens) == 0).all()
    assert det.det_embedding_backward(torch.ones(3, 8, device="cuda"), tokens, 0).shape == (0, 8)
    assert det.det_embedding(torch.zeros(4, 0, device="cuda"), tokens).shape == (3, 0)
    assert det.det_embedding_backward(torch.ones(3, 0, device="cuda"), tokens, 4).shape == (4, 0)
    old = torch.ones(4, 8, device="cuda")
    det.det_embedding_backward(torch.ones(0, 8, device="cuda"), tokens[:0], 4, grad_table=old, accumulate=True)
    assert (old == 1).all()


@pytest.mark.parametrize("n,vocab", [(70_000, 3), (16_384, 300_000), (16_385, 40), (200_000, 300_000),
                                     (32_768, 3), (32_768, 200_000), (32_769, 3), (20_001, 262_144),
                                     (5_000, 524_288), (5_000, 524_289)])
def test_embedding_gradients_of_either_sort(det, n, vocab):
    """Runs of one token as long as the call, tables past the small sort's, tokens outside at both ends, values that are not
    finite: a column of NaN is the token's own."""
    g = torch.Generator().manual_seed(n)
    tokens = torch.randint(0, vocab, (n,), generator=g, dtype=torch.int32)
    tokens[n // 4: n // 2] = vocab - 1
    tokens[::97] = -1
    tokens[1::97] = 2**31 - 1
    tokens[2::97] = -2**31
    tokens[3::97] = vocab
    grad = torch.randn(n, 12, generator=g)
    bad = int(tokens[5])
    grad[5, 7] = float("nan")
    grad[n // 3, 3] = float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        d = grad.to(dtype)
        total, _ = oracle.det_scatter_add_rows(np.zeros((vocab, 12), np.float32), tokens.numpy(), d.float().numpy())
        want = torch.from_numpy(total)
        for odd in (0, 1):
            wide = torch.zeros(n * 12 + 8, dtype=dtype, device="cuda")
            wide[odd:odd + n * 12].copy_(d.view(-1))
            got = det.det_embedding_backward(wide[odd:odd + n * 12].view(n, 12), tokens.cuda(), vocab, dtype=torch.float32).cpu()
            assert torch.equal(got.isnan(), want.isnan()) and bool(got[bad, 7].isnan())
            assert torch.equal(got.nan_to_num(), want.nan_to_num())


# ---------------------------------------------------------------------------
# The ends of the ranges


def test_embedding_of_the_widest_rows(det):
    dim = 2**21
    g = torch.Generator().manual_seed(1)
    table = torch.randn(3, dim, generator=g).bfloat16().cuda()
    tokens = torch.tensor([2, 0, -1, 2], dtype=torch.int32, device="cuda")
    out = det.det_embedding(table, tokens)
    assert equal(out[0], table[2]) and equal(out[1], table[0]) and not out[2].any() and equal(out[3], table[2])
    grad = torch.randn(4, dim, device="cuda").bfloat16()
    got = det.det_embedding_backward(grad, tokens, 3, dtype=torch.float32)
    assert equal(got[2], grad[0].float() + grad[3].float()) and equal(got[0], grad[1].float()) and not got[1].any()


def test_embedding_past_32_bit_offsets(det):
    vocab, dim = 530_000, 4_100                          # 2.17e9 elements
    table = torch.empty(vocab, dim, dtype=torch.bfloat16, device="cuda").normal_()
    tokens = torch.tensor([0, vocab - 1, vocab - 1, vocab - 7, 5, vocab], dtype=torch.int32, device="cuda")
    out = det.det_embedding(table, tokens)
    assert equal(out[:5], table[tokens[:5].long()]) and not out[5].any()
    del out
    grad = torch.randn(6, dim, device="cuda").bfloat16()
    got = det.det_embedding_backward(grad, tokens, vocab)
    assert equal(got[vocab - 1], (grad[1].float() + grad[2].float()).bfloat16())
    for row, i in ((0, 0), (vocab - 7, 3), (5, 4)):
        assert equal(got[row], grad[i])
    got[tokens[:5].long()] = 0
    assert not got.any()
    del got
    # as many places
    n = vocab
    many = torch.randint(0, 1000, (n,), dtype=torch.int32, device="cuda")
    many[-1] = 999
    out = det.det_embedding(table[:1000], many)
    assert out.numel() > 2**31 and equal(out[-3000:], table[many[-3000:].long()]) and equal(out[:3000], table[many[:3000].long()])
    del out
    got = det.det_embedding_backward(table, many, 1000, dtype=torch.float32)
    for c in (slice(0, 3), slice(dim - 3, dim)):
        total, _ = oracle.det_scatter_add_rows(np.zeros((1000, 3), np.float32), many.cpu().numpy(),
                                               table[:, c].float().cpu().numpy())
        assert equal(got[:, c].cpu(), torch.from_numpy(total))


def test_norm_past_32_bit_offsets(det):
    rows, cols = 140_000, 16_000                         # 2.24e9 elements
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.rand(cols, device="cuda") + 0.5
    r = det.det_layer_norm(x, w)
    tail = slice(rows - 300, rows)
    part = det.det_layer_norm(x[tail], w)
    assert equal(r.out[tail], part.out) and equal(r.mean[tail], part.mean) and equal(r.rstd[tail], part.rstd)
    grad = r.out
    grad.random_(-2, 3)                                  # whole numbers: their sums are exact
    b = det.det_layer_norm_backward(grad, x, r.mean, r.rstd, w)
    p = det.det_layer_norm_backward(grad[tail], x[tail], part.mean, part.rstd, w)
    assert equal(b.x[tail], p.x)
    assert equal(b.bias, sum(g.float().sum(0) for g in grad.split(20_000)))


def test_recurrence_past_32_bit_offsets(det):
    """A decay of 0 cuts a sequence: what follows it has the bits of a run that starts there, and what comes before it the
    gradients of one that ends there."""
    time, channels = 1_048_700, 2_112                    # 2.21e9 elements
    first, cut = 1024, 1_040_000
    assert first % 128 == 0 and cut % 128 == 0 and cut * channels > 2**31
    x = torch.empty(1, time, channels, dtype=torch.bfloat16, device="cuda").normal_()
    gate = torch.empty_like(x).uniform_(0.2, 0.98)
    gate[:, first] = 0
    gate[:, cut] = 0
    grad = torch.empty_like(x).normal_()
    r = det.det_linear_recurrence(x, gate, form="decay", keep_states=True)
    b = det.det_linear_recurrence_backward(grad, x, gate, r.states, form="decay")
    end = det.det_linear_recurrence(x[:, cut:], gate[:, cut:], form="decay", keep_states=True)
    assert equal(r.out[:, cut:], end.out) and equal(r.final, end.final)
    e = det.det_linear_recurrence_backward(grad[:, cut:], x[:, cut:], gate[:, cut:], end.states, form="decay")
    assert equal(b.x[:, cut:], e.x) and equal(b.gate[:, cut + 1:], e.gate[:, 1:])
    head = det.det_linear_recurrence(x[:, :first], gate[:, :first], form="decay", keep_states=True)
    assert equal(r.out[:, :first], head.out)
    h = det.det_linear_recurrence_backward(grad[:, :first], x[:, :first], gate[:, :first], head.states, form="decay")
    assert equal(b.x[:, :first], h.x) and equal(b.gate[:, :first], h.gate) and equal(b.initial, h.initial)


def test_recurrence_of_far_strides(det):
    buf = torch.empty(2**31 + 2**29, dtype=torch.bfloat16, device="cuda")
    for shape, strides in (((2, 300, 70), (2**31 + 8, 72, 1)), ((2, 300, 70), (2**31 + 7, 71, 1)),
                           ((1, 19, 70), (0, 2**27 + 8, 1)), ((1, 19, 70), (0, 2**27 + 5, 1)), ((1, 7, 70), (0, 2**28 + 10, 1))):
        x = buf.as_strided(shape, strides)
        x.copy_(torch.randn(shape, device="cuda"))
        gate = torch.randn(shape, device="cuda").bfloat16()
        near = x.contiguous()
        for a, b in ((x, gate), (gate, x)):
            far = det.det_linear_recurrence(a, b, keep_states=True)
            want = det.det_linear_recurrence(a.contiguous(), b.contiguous(), keep_states=True)
            assert equal(far.out, want.out) and equal(far.final, want.final) and equal(far.states, want.states)
            got = det.det_linear_recurrence_backward(x, a, b, far.states)
            want = det.det_linear_recurrence_backward(near, a.contiguous(), b.contiguous(), want.states)
            assert all(equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("time", [2, 9])
def test_recurrence_of_the_largest_batch(det, time):
    g = torch.Generator().manual_seed(time)
    x, gate = (torch.randn(65_535, time, 3, generator=g).cuda() for _ in range(2))
    r = det.det_linear_recurrence(x, gate, keep_states=True)
    b = det.det_linear_recurrence_backward(x, x, gate, r.states)
    some = slice(65_000, 65_535)
    part = det.det_linear_recurrence(x[some], gate[some], keep_states=True)
    assert equal(r.out[some], part.out) and equal(r.final[some], part.final)
    p = det.det_linear_recurrence_backward(x[some], x[some], gate[some], part.states)
    assert all(equal(a[some], c) for a, c in zip(b, p))
