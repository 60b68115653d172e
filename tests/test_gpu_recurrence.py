"""det_linear_recurrence and its gradients against a 64-bit run through the steps on the CPU.

Tolerances, u = 2^-24.  A state is a sum of terms, each a product of an input and the decays after it.  However the
steps are grouped, a term that is k steps old has passed at most 2 k + 40 roundings (a product and a sum a step, and
those of joining pieces), and each decay and 1 - decay is off by at most GATE u (32-bit gates of the sigmoid form: exp,
a sum, a division and a difference, 6 units at most; the hardware's exp of 16-bit gates: 4 + |z| more; decays as given are
exact).  So with S[t] = |a| S[t-1] + |u[t]| and W[t] = |a| (W[t-1] + S[t-1]), the sum of the terms' sizes times their age,
the state is off by at most ((2 + GATE) W + (40 + GATE) S) u.  Backwards the same holds for l, and a gradient is a
product of such values.  Results in T are rounded by half a step.

Below 2^-126 a rounding is off by up to half of 2^-149 instead, and decays are at most 1 here: the 2 k + 40 roundings of
a path add up to at most (2 time + 40) 2^-150, whatever the terms' sizes; a gradient multiplies that by a state and an input."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def det():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    return d


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, tol, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape
    off = (got - want).abs()
    assert bool((off <= tol).all()), (what, float((off - tol).max()), float(off.max()))


def rounded(tol, want, dtype):
    return tol * 1.01 + half_step(dtype) * want.abs() * 1.01 + torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def make(batch, time, channels, dtype, form, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(batch, time, channels, generator=g).to(dtype)
    if form == "sigmoid":
        gate = (torch.randn(batch, time, channels, generator=g) * 2 + 2).to(dtype)
    else:
        gate = (1 - torch.rand(batch, time, channels, generator=g) ** 2 * 0.6).to(dtype)
        gate = gate * torch.where(torch.rand(batch, time, channels, generator=g) < 0.05, -1.0, 1.0).to(dtype)
    initial = torch.randn(batch, channels, generator=g)
    grad = torch.randn(batch, time, channels, generator=g).to(dtype)
    grad_final = torch.randn(batch, channels, generator=g)
    return x, gate, initial, grad, grad_final


class Exact:
    """Everything in 64 bits, and the bounds."""

    def __init__(self, x, gate, initial, form, lengths=None, grad=None, grad_final=None):
        batch, time, channels = x.shape
        dtype = x.dtype
        n = torch.full((batch,), time) if lengths is None else lengths.long().clamp(0, time)
        valid = (torch.arange(time)[None, :] < n[:, None])[:, :, None]
        xd, z = (torch.where(valid, t.double(), torch.zeros(()).double()) for t in (x, gate))
        if form == "sigmoid":
            a, rest = torch.sigmoid(z), torch.sigmoid(-z)
            k = 6 + (0 if dtype == torch.float32 else 4 + float(z.abs().max()) if z.numel() else 0)
        else:
            a, rest, k = z, torch.ones_like(z), 0
        a = torch.where(valid, a, torch.ones(()).double())
        u = torch.where(valid, rest * xd, torch.zeros(()).double())
        h = torch.zeros(batch, channels).double() if initial is None else initial.double()
        S, W = h.abs(), torch.zeros_like(h)
        floor = (2 * time + 40) * 2.0 ** -150
        hs, before, e_before, es = [], [], [], []
        for t in range(time):
            before.append(h), e_before.append(((2 + k) * W + (40 + k) * S) * U + floor)
            W = a[:, t].abs() * (W + S)
            h, S = a[:, t] * h + u[:, t], a[:, t].abs() * S + u[:, t].abs()
            hs.append(h), es.append(((2 + k) * W + (40 + k) * S) * U + floor)
        self.final, self.e_final = h, ((2 + k) * W + (40 + k) * S) * U + floor
        if time:
            self.out = torch.where(valid, torch.stack(hs, 1), torch.zeros(()).double())
            self.e_out = torch.where(valid, torch.stack(es, 1), torch.zeros(()).double())
            self.before = torch.stack(before, 1)
        else:
            self.out = self.e_out = torch.zeros(batch, 0, channels).double()
        if grad is None and grad_final is None:
            return
        g = torch.zeros_like(xd) if grad is None else torch.where(valid, grad.double(), torch.zeros(()).double())
        m = torch.zeros(batch, channels).double() if grad_final is None else grad_final.double()
        S, W = m.abs(), torch.zeros_like(m)
        gx, gg, ex, eg = [], [], [], []
        for t in reversed(range(time)):
            l, Sl = m + g[:, t], S + g[:, t].abs()
            el = ((2 + k) * W + (40 + k) * Sl) * U + floor
            d = before[t] - xd[:, t] if form == "sigmoid" else before[t]
            big = before[t].abs() + (xd[:, t].abs() if form == "sigmoid" else 0)
            both = (a[:, t] * rest[:, t]).abs() if form == "sigmoid" else torch.ones_like(l)
            gx.append(l * rest[:, t]), ex.append((el + (k + 2) * U * Sl) * rest[:, t].abs())
            gg.append(l * d * (a[:, t] * rest[:, t] if form == "sigmoid" else 1))
            eg.append((el * big + Sl * e_before[t] + (2 * k + 8) * U * Sl * big) * both)
            W = a[:, t].abs() * (W + Sl)
            m, S = a[:, t] * l, a[:, t].abs() * Sl
        self.g_initial, self.e_initial = m, ((2 + k) * W + (40 + k) * S) * U + floor

        def stack(v):
            return torch.where(valid, torch.stack(v[::-1], 1), torch.zeros(()).double()) if time else torch.zeros_like(xd)
        self.gx, self.gg, self.ex, self.eg = stack(gx), stack(gg), stack(ex), stack(eg)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def run_both(det, x, gate, initial, grad, grad_final, form, lengths=None):
    xc, gc, ic, dc, fc, lc = cuda(x, gate, initial, grad, grad_final, lengths)
    e = Exact(x, gate, initial, form, lengths, grad, grad_final)
    r = det.det_linear_recurrence(xc, gc, ic, form=form, lengths=lc, keep_states=True)
    close(r.out, e.out, rounded(e.e_out, e.out, x.dtype), "out")
    close(r.final, e.final, e.e_final * 1.01, "final")
    if x.numel():
        close(r.states, e.before[:, ::128], e.e_out.abs().amax() * 1.01 + e.e_final.amax(), "states")
    b = det.det_linear_recurrence_backward(dc, xc, gc, r.states, grad_final=fc, form=form, lengths=lc)
    close(b.x, e.gx, rounded(e.ex, e.gx, x.dtype), "grad x")
    close(b.gate, e.gg, rounded(e.eg, e.gg, x.dtype), "grad gate")
    close(b.initial, e.g_initial, e.e_initial * 1.01, "grad initial")
    return r, b


TIMES = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 127, 128, 129, 256, 300, 513, 1023, 1024, 1025, 2500]


@pytest.mark.parametrize("time", TIMES)
@pytest.mark.parametrize("form", ["decay", "sigmoid"])
@pytest.mark.parametrize("kind", list(DTYPES))
def test_lengths_types_and_forms(det, time, form, kind):
    batch, channels = (3, 70) if time < 1000 else (2, 65)
    run_both(det, *make(batch, time, channels, DTYPES[kind], form, time), form)


@pytest.mark.parametrize("channels", [1, 2, 31, 63, 64, 66, 129, 600])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_channels(det, channels, kind):
    for time in (5, 40, 200):
        run_both(det, *make(2, time, channels, DTYPES[kind], "sigmoid", channels), "sigmoid")


def test_no_steps_no_batch_no_channels(det):
    for shape in ((2, 0, 8), (0, 5, 8), (2, 5, 0)):
        x, gate, initial, grad, grad_final = make(*shape, torch.bfloat16, "decay", 1)
        r, b = run_both(det, x, gate, initial, grad, grad_final, "decay")
        if shape[1] == 0:
            assert torch.equal(r.final.cpu(), initial) and torch.equal(b.initial.cpu(), grad_final)


@pytest.mark.parametrize("time", [9, 128, 700, 2300])
@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_ragged_lengths(det, time, kind):
    """Steps past a sequence's end are not read and give zeros."""
    lengths = torch.tensor([time, 0, 1, time - 1, time // 2, 2 * time, -3], dtype=torch.int32)
    for form in ("decay", "sigmoid"):
        x, gate, initial, grad, grad_final = make(7, time, 33, DTYPES[kind], form, time)
        for b, n in enumerate(lengths.clamp(0, time).tolist()):
            for t in (x, gate, grad):
                t[b, n:] = float("nan")
        r, g = run_both(det, x, gate, initial, grad, grad_final, form, lengths)
        # the same sequences alone and cut at their ends: the same bits
        for b, n in enumerate(lengths.clamp(0, time).tolist()):
            xc, gc, ic = cuda(x[b:b + 1, :n].contiguous(), gate[b:b + 1, :n].contiguous(), initial[b:b + 1])
            one = det.det_linear_recurrence(xc, gc, ic, form=form)
            assert torch.equal(one.out[0], r.out[b, :n]) and torch.equal(one.final[0], r.final[b])
            if kind == "f32" and n:
                assert torch.equal(r.final[b], r.out[b, n - 1])


def test_missing_operands(det):
    x, gate, initial, grad, grad_final = make(2, 300, 40, torch.bfloat16, "sigmoid", 2)
    run_both(det, x, gate, None, grad, grad_final, "sigmoid")
    run_both(det, x, gate, initial, None, grad_final, "sigmoid")
    run_both(det, x, gate, initial, grad, None, "sigmoid")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_strides_and_alignment_do_not_change_bits(det, kind):
    dtype = DTYPES[kind]
    x, gate, initial, grad, grad_final = (t.cuda() for t in make(3, 270, 50, dtype, "sigmoid", 7))
    r = det.det_linear_recurrence(x, gate, initial, keep_states=True)
    b = det.det_linear_recurrence_backward(grad, x, gate, r.states, grad_final=grad_final)
    for off, pad in ((0, 6), (1, 4), (2, 8), (3, 0)):
        wide = torch.full((3, 3, 270, 50 + off + pad), float("nan"), dtype=dtype, device="cuda")
        for i, t in enumerate((x, gate, grad)):
            wide[i, :, :, off:off + 50] = t
        xs, gs, ds = (wide[i, :, :, off:off + 50] for i in range(3))
        r2 = det.det_linear_recurrence(xs, gs, initial, keep_states=True)
        b2 = det.det_linear_recurrence_backward(ds, xs, gs, r2.states, grad_final=grad_final)
        assert all(torch.equal(p, q) for p, q in zip((*r, *b), (*r2, *b2)))
    # time before batch
    xt, gt = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (x, gate))
    assert torch.equal(det.det_linear_recurrence(xt, gt, initial).out, r.out)


def test_bits_do_not_depend_on_what_follows_or_lies_beside(det):
    x, gate, initial, _, _ = (t.cuda() for t in make(2, 3000, 130, torch.bfloat16, "sigmoid", 8))
    whole = det.det_linear_recurrence(x, gate, initial)
    for n in (1, 16, 17, 128, 129, 1000, 1024, 1025, 2048, 2900):
        cut = det.det_linear_recurrence(x[:, :n].contiguous(), gate[:, :n].contiguous(), initial)
        assert torch.equal(cut.out, whole.out[:, :n]), n
    part = det.det_linear_recurrence(x[1:, :, 64:], gate[1:, :, 64:], initial[1:, 64:].contiguous())
    assert torch.equal(part.out, whole.out[1:, :, 64:])


def test_step_by_step_in_place(det):
    """Serving: one step a call, the states updated in place; in 32 bits step by step is what 8 steps at once do."""
    x, gate, initial, _, _ = (t.cuda() for t in make(5, 8, 300, torch.float32, "sigmoid", 9))
    whole = det.det_linear_recurrence(x, gate, initial)
    state = initial.clone()
    for t in range(8):
        r = det.det_linear_recurrence(x[:, t:t + 1], gate[:, t:t + 1], state, final=state)
        assert r.final.data_ptr() == state.data_ptr() and torch.equal(r.out[:, 0], whole.out[:, t])
    assert torch.equal(state, whole.final)
    # whole prompts in place too
    x, gate, initial, _, _ = (t.cuda() for t in make(3, 2000, 200, torch.bfloat16, "sigmoid", 10))
    whole = det.det_linear_recurrence(x, gate, initial)
    for _ in range(5):
        state = initial.clone()
        assert torch.equal(det.det_linear_recurrence(x, gate, state, final=state).out, whole.out)
        assert torch.equal(state, whole.final)


def test_gates_at_their_ends(det):
    """Closed and open gates, decays of 0 and 1, and products of decays that leave the range of 32 bits."""
    x = torch.randn(1, 600, 4, generator=torch.Generator().manual_seed(3))
    gate = torch.zeros(1, 600, 4)
    gate[:, :, 0], gate[:, :, 1], gate[:, :, 2] = float("inf"), -float("inf"), 90.0
    r = det.det_linear_recurrence(x.cuda(), gate.cuda(), torch.full((1, 4), 5.0).cuda())
    assert (r.out[:, :, 0] == 5).all() and torch.equal(r.out[:, :, 1].cpu(), x[:, :, 1]) and (r.out[:, :, 2] == 5).all()
    ones, zeros = torch.ones(1, 600, 4), torch.zeros(1, 600, 4)
    r = det.det_linear_recurrence(ones.cuda(), ones.cuda(), form="decay")
    assert torch.equal(r.out.cpu(), torch.arange(1, 601).float()[None, :, None].expand(1, 600, 4))
    assert torch.equal(det.det_linear_recurrence(x.cuda(), zeros.cuda(), form="decay").out.cpu(), x)
    # growth by 4 a step from a state of 0 that stays 0
    assert (det.det_linear_recurrence(zeros.cuda(), (4 * ones).cuda(), form="decay").out == 0).all()
    # a reset between documents, and a NaN before it that reaches no other channel
    gate = torch.full((1, 600, 4), 0.9)
    gate[:, 300] = 0
    y = x.clone()
    y[0, 100, 1] = float("nan")
    r = det.det_linear_recurrence(y.cuda(), gate.cuda(), form="decay")
    after = det.det_linear_recurrence(x[:, 300:].cuda(), gate[:, 300:].cuda(), form="decay")
    e = Exact(x[:, 300:], gate[:, 300:], None, "decay")
    for c in (0, 2, 3):
        close(r.out[:, 300:, c], e.out[:, :, c], rounded(e.e_out, e.out, torch.float32)[:, :, c])
    assert r.out[0, :100].isfinite().all() and r.out[0, 100:, 1].isnan().all() and r.out[0, :, 0].isfinite().all()
    assert after.out.isfinite().all()


def test_autograd_against_differentiation_and_differences(det):
    from deterministic_floating_point_gb300 import autograd

    def plain(x, gate, h, form):
        outs = []
        for t in range(x.shape[1]):
            a = torch.sigmoid(gate[:, t]) if form == "sigmoid" else gate[:, t]
            h = a * h + ((1 - a) if form == "sigmoid" else 1) * x[:, t]
            outs.append(h)
        return torch.stack(outs, 1), h
    for form in ("decay", "sigmoid"):
        x, gate, initial, grad, grad_final = make(2, 150, 20, torch.float32, form, 11)
        leaves = [t.cuda().requires_grad_(True) for t in (x, gate, initial)]
        out, final = autograd.linear_recurrence(*leaves, form=form)
        ((out * grad.cuda()).sum() + (final * grad_final.cuda()).sum()).backward()
        ref = [t.double().requires_grad_(True) for t in (x, gate, initial)]
        out, final = plain(*ref, form)
        ((out * grad.double()).sum() + (final * grad_final.double()).sum()).backward()
        e = Exact(x, gate, initial, form, None, grad, grad_final)
        tols = (rounded(e.ex, e.gx, torch.float32), rounded(e.eg, e.gg, torch.float32), e.e_initial * 1.01)
        for got, want, tol in zip(leaves, ref, tols):
            close(got.grad, want.grad, tol + 1e-14)
        gen, step = torch.Generator().manual_seed(12), 1e-5
        for i, t in enumerate((x, gate, initial)):
            d = torch.randn(t.shape, generator=gen).double()
            value = []
            for sign in (1, -1):
                args = [a.double() for a in (x, gate, initial)]
                args[i] = args[i] + sign * step * d
                out, final = plain(*args, form)
                value.append((out * grad.double()).sum() + (final * grad_final.double()).sum())
            slope = (value[0] - value[1]) / (2 * step)
            got = (leaves[i].grad.double().cpu() * d).sum()
            # 32-bit gradients; the differences' second-order error (step^2 times third derivatives) and roundings
            assert abs(float(got - slope)) <= float((tols[i] * d.abs()).sum()) + 1e-5 * (1 + abs(float(slope)))
    # only one of the outputs is used, and an expanded gradient
    out, final = autograd.linear_recurrence(*leaves, form="sigmoid")
    (g1,) = torch.autograd.grad(final.sum(), leaves[2], retain_graph=True)
    (g2,) = torch.autograd.grad(out.sum(), leaves[0])
    assert g1.isfinite().all() and g2.isfinite().all()
