"""Gates of the sigmoid form at their ends, in every type and in the kernels for few and for many steps: the decays that
gates give, one by one, and closed, open and NaN gates with their gradients.

Bounds, u = 2^-24, of a and 1 - a.  32 bits: expf 2 u, a sum u, __fdividef 4 u, a difference u: 8 u.  16 bits: the exponent is off by
the constant's rounding, 0.22 u, and the product's, u, times |z|; ex2 4 u, a sum u, the reciprocal 2 u, a product u: (8 + 1.22 |z|) u.
There a is less by the a of -87, below 2^-125, so that a closed gate closes for good; and what is below 2^-126 is 0."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_recurrence import DTYPES, Exact, close, det, make, rounded  # noqa: E402,F401

U = 2.0 ** -24


def every(dtype):
    """Every value of 16 bits; of 32, every exponent and what lies around the ends."""
    if dtype != torch.float32:
        return torch.arange(-32768, 32768).to(torch.int16).view(dtype)
    g = torch.Generator().manual_seed(1)
    v = torch.cat([torch.randn(20000, generator=g) * 30, torch.linspace(-110, 110, 40001),
                   torch.logspace(-45, 38, 2000), torch.tensor([float("inf"), float("nan"), 0.0])])
    v = torch.cat([v, -v])
    return torch.cat([v, torch.zeros(-v.numel() % 256)])


@pytest.mark.parametrize("time", [1, 9, 300])
@pytest.mark.parametrize("kind", list(DTYPES))
def test_the_decay_of_every_gate(det, kind, time):  # noqa: F811
    """The first step's gate is the value, the others are open and add nothing: the final state is a, or 1 - a."""
    dtype = DTYPES[kind]
    z = every(dtype).view(-1, 256)
    batch = z.shape[0]
    gate = torch.full((batch, time, 256), float("inf"), dtype=dtype)
    gate[:, 0] = z
    x = torch.zeros(batch, time, 256, dtype=dtype)
    a = det.det_linear_recurrence(x.cuda(), gate.cuda(), torch.ones(batch, 256).cuda()).final.cpu().double()
    x[:, 0] = 1
    rest = det.det_linear_recurrence(x.cuda(), gate.cuda()).final.cpu().double()
    zd = z.double()
    assert torch.equal(a.isnan(), zd.isnan()) and torch.equal(rest.isnan(), zd.isnan())
    if dtype == torch.float32:
        units, less = torch.full_like(zd, 8.0), 0.0
    else:
        units, less = 8 + 1.22 * zd.abs().clamp(max=128), 2.0 ** -125
    for got, want, off in ((a, torch.sigmoid(zd), less), (rest, torch.sigmoid(-zd), 0.0)):
        ok = (got - want).abs() <= want * units * U + off + 2.0 ** -126
        assert bool((ok | zd.isnan()).all()), zd[~(ok | zd.isnan())][:5]
        assert not (got[~zd.isnan()] < 0).any()
    if dtype != torch.float32:
        assert (a[zd <= -87] == 0).all() and not (a > 1).any()
    assert (a[zd >= 25] == 1).all() and (rest[zd == float("inf")] == 0).all() and (a[zd == -float("inf")] == 0).all()


@pytest.mark.parametrize("time", [1, 5, 8, 9, 300, 2100])
@pytest.mark.parametrize("kind", list(DTYPES))
def test_large_gates(det, kind, time):  # noqa: F811
    """Gates up to 70 in size against 64 bits (beyond, a is a sum of what 2^-125 takes off), inputs that are zero among them."""
    x, gate, initial, grad, grad_final = make(2, time, 130, DTYPES[kind], "sigmoid", time)
    gate = (gate.float() * 14).clamp(-70, 70).to(DTYPES[kind])
    x[..., ::3] = 0
    initial *= 1e4
    e = Exact(x, gate, initial, "sigmoid", None, grad, grad_final)
    r = det.det_linear_recurrence(x.cuda(), gate.cuda(), initial.cuda(), keep_states=True)
    # The class counts 10 + |z| units for 16-bit gates, 80 in all; 8 + 1.22 * 70 and one for what is taken off a (2^-125 of
    # 2^-101 at least) are 95.  Its roundings below 2^-126 are of states; those of products of decays, 2^-150 each, are
    # multiplied by a state, here of up to 1e5, and again by a state or an input in the gate's gradient.
    tiny = (2 * time + 40) * 2.0 ** -150 * 1e5
    close(r.out, e.out, rounded(e.e_out * 1.3 + tiny, e.out, x.dtype), "out")
    close(r.final, e.final, e.e_final * 1.3 + tiny, "final")
    b = det.det_linear_recurrence_backward(grad.cuda(), x.cuda(), gate.cuda(), r.states, grad_final=grad_final.cuda())
    close(b.x, e.gx, rounded(e.ex * 1.3 + tiny, e.gx, x.dtype), "x")
    close(b.gate, e.gg, rounded(e.eg * 1.3 + 1e5 * tiny, e.gg, x.dtype), "gate")
    close(b.initial, e.g_initial, e.e_initial * 1.3 + tiny, "initial")


def ends(dtype):
    low, high = float(torch.finfo(dtype).min), float(torch.finfo(dtype).max)
    closed = [-float("inf"), low, -200.0] + ([-87.0, -88.0] if dtype != torch.float32 else [])
    return closed, [float("inf"), high, 200.0, 88.0 if dtype != torch.float32 else 105.0]


@pytest.mark.parametrize("time", [5, 8, 9, 300, 2100])
@pytest.mark.parametrize("kind", list(DTYPES))
def test_closed_and_open_gates(det, kind, time):  # noqa: F811
    dtype = DTYPES[kind]
    closed, opened = ends(dtype)
    gen = torch.Generator().manual_seed(time)
    channels = 2 * (len(closed) + len(opened)) + 3
    x = torch.randn(2, time, channels, generator=gen).to(dtype)
    gate = torch.randn(2, time, channels, generator=gen).to(dtype)
    at = time // 2
    for c, z in enumerate(closed):
        gate[:, at, 2 * c] = z
    for c, z in enumerate(opened):
        gate[:, :, 2 * (len(closed) + c)] = z
    grad = torch.randn(2, time, channels, generator=gen).to(dtype)
    grad_final = torch.randn(2, channels, generator=gen)
    initial = torch.full((2, channels), 1e30)
    r = det.det_linear_recurrence(x.cuda(), gate.cuda(), initial.cuda(), keep_states=True)
    b = det.det_linear_recurrence_backward(grad.cuda(), x.cuda(), gate.cuda(), r.states, grad_final=grad_final.cuda())
    zero = det.det_linear_recurrence(x.cuda(), gate.cuda(), torch.zeros(2, channels).cuda())
    for c in range(len(closed)):
        c = 2 * c
        # a closed gate removes the state, however large: the output is the input, and what follows does not know of it
        assert torch.equal(r.out[:, at, c].cpu(), x[:, at, c])
        assert torch.equal(r.out[:, at:, c], zero.out[:, at:, c]) and torch.equal(r.final[:, c], zero.final[:, c])
        assert (b.gate[:, at, c] == 0).all()
        # and nothing comes back through it: steps before it have the gradients of their own grad alone
        short = det.det_linear_recurrence_backward(grad[:, :at].contiguous().cuda(), x[:, :at].contiguous().cuda(),
                                                   gate[:, :at].contiguous().cuda(),
                                                   r.states[:, :-(-at // 128)].contiguous())
        assert torch.equal(b.x[:, :at, c], short.x[..., c]) and torch.equal(b.initial[:, c], short.initial[:, c])
    for c in range(len(opened)):
        c = 2 * (len(closed) + c)
        # an open one keeps it, bit for bit, and adds nothing to it
        assert torch.equal(r.final[:, c].cpu(), initial[:, c])
        assert torch.equal(r.out[:, :, c].cpu(), initial[:, :1].expand(2, time).to(dtype))
        total = grad[:, :, c].double().sum(1) + grad_final[:, c].double()
        size = grad[:, :, c].double().abs().sum(1) + grad_final[:, c].double().abs()
        close(b.initial[:, c], total, (2 * time + 40) * U * size)
        # a (1 - a) is below 2^-126
        assert (b.x[:, :, c].abs() <= 2.0 ** -120).all() and (b.gate[:, :, c].abs() <= 1e30 * 2.0 ** -110).all()


@pytest.mark.parametrize("time", [5, 9, 300, 2100])
@pytest.mark.parametrize("kind", list(DTYPES))
@pytest.mark.parametrize("form", ["sigmoid", "decay"])
def test_a_nan_gate_stays_in_its_channel(det, form, kind, time):  # noqa: F811
    x, gate, initial, grad, grad_final = make(2, time, 70, DTYPES[kind], form, time)
    at = time // 2

    def both(gate):
        r = det.det_linear_recurrence(x.cuda(), gate.cuda(), initial.cuda(), form=form, keep_states=True)
        b = det.det_linear_recurrence_backward(grad.cuda(), x.cuda(), gate.cuda(), r.states, grad_final=grad_final.cuda(),
                                               form=form)
        return r.out, r.final, b.x, b.gate, b.initial
    want = both(gate)
    bad = gate.clone()
    for c in (0, 33, 68):                        # each beside others in a word
        bad[1, at, c] = float("nan")
    got = both(bad)
    others = [c for c in range(70) if c not in (0, 33, 68)]
    for p, q in zip(got, want):
        assert torch.equal(p[..., others], q[..., others]) and torch.equal(p[0], q[0])
    for c in (0, 33, 68):
        out, final, gx, gg, gi = (p[1, ..., c] for p in got)
        assert torch.equal(out[:at], want[0][1, :at, c]) and out[at:].isnan().all() and final.isnan()
        assert torch.equal(gx[at + 1:], want[2][1, at + 1:, c]) and gx[:at].isnan().all() and gi.isnan()
        assert gg[:at].isnan().all() and gg[at + 1:].isnan().all()      # through l before it, through h after it
        # at the step itself a given decay's gradient is l h, which does not know of it
        if form == "decay":
            assert torch.equal(gg[at], want[3][1, at, c]) and torch.equal(gx[at], want[2][1, at, c])
        else:
            assert gg[at].isnan() and gx[at].isnan()
