"""The bits of a channel's gradients in the linear recurrence, and of a row's in the layer norm, do not depend on where the
operands lie, on the channels beside it, on whether its tile is whole, or on how the sequence's end is told."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_recurrence import DTYPES, det, make  # noqa: E402,F401


def shifted(t, off):
    """t at an odd place, in rows of an odd stride."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + 9), float("nan"), dtype=t.dtype, device="cuda")
    wide[..., off:off + t.shape[-1]] = t
    return wide[..., off:off + t.shape[-1]]


@pytest.mark.parametrize("time", [1, 5, 8, 9, 16, 33, 128, 300, 1000, 2100])
@pytest.mark.parametrize("form", ["decay", "sigmoid"])
@pytest.mark.parametrize("kind", list(DTYPES))
def test_recurrence(det, kind, form, time):  # noqa: F811
    inputs = [t.cuda() for t in make(2, time, 200, DTYPES[kind], form, time)]

    def all_of(x, gate, initial, grad, grad_final, lengths=None):
        r = det.det_linear_recurrence(x, gate, initial, form=form, lengths=lengths, keep_states=True)
        b = det.det_linear_recurrence_backward(grad, x, gate, r.states, grad_final=grad_final, form=form, lengths=lengths)
        return [r.out, r.final, r.states, b.x, b.gate, b.initial]
    want = all_of(*inputs)
    x, gate, initial, grad, grad_final = inputs
    for off in (1, 2, 3, 8):
        got = all_of(shifted(x, off), shifted(gate, off), initial, shifted(grad, off), grad_final)
        assert [torch.equal(p, q) for p, q in zip(got, want)] == [True] * 6, off
    for n in (1, 31, 50, 64, 129, 130, 199):
        got = all_of(*(t[..., :n].contiguous() for t in inputs))
        assert [torch.equal(p, q[..., :n]) for p, q in zip(got, want)] == [True] * 6, n
    for more in (1, 8, 1000):
        def longer(t):
            return torch.cat([t, torch.full((2, more, 200), float("nan"), dtype=t.dtype, device="cuda")], 1)
        lengths = torch.full((2,), time, dtype=torch.int32, device="cuda")
        got = all_of(longer(x), longer(gate), initial, longer(grad), grad_final, lengths)
        got = [p[:, :q.shape[1]] if p.dim() == 3 else p for p, q in zip(got, want)]
        assert [torch.equal(p, q) for p, q in zip(got, want)] == [True] * 6, more


@pytest.mark.parametrize("cols", [7, 64, 100, 256, 264, 768, 2048, 4100, 5000, 8192, 8200, 12000, 16383, 16384])
@pytest.mark.parametrize("kind", list(DTYPES))
def test_norm(det, kind, cols):  # noqa: F811
    gen = torch.Generator().manual_seed(cols)
    x, g = (torch.randn(30, cols, generator=gen).to(DTYPES[kind]).cuda() for _ in range(2))
    w, b = (torch.rand(cols, generator=gen) + 0.5).cuda(), torch.randn(cols, generator=gen).cuda()
    r = det.det_layer_norm(x, w, b)
    want = [*r, *det.det_layer_norm_backward(g, x, r.mean, r.rstd, w)]
    for off in (1, 2, 3, 8):
        r = det.det_layer_norm(shifted(x, off), w, b)
        got = [*r, *det.det_layer_norm_backward(shifted(g, off), shifted(x, off), r.mean, r.rstd, w)]
        assert [torch.equal(p, q) for p, q in zip(got, want)] == [True] * 6, off
