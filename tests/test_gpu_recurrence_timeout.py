"""The recurrence's bounded waits, made to run out on purpose: a test hook withholds the message of one round from the first of
the CTAs that share a sequence.  The launch ends by itself, what was known before that round has its bits, everything from there
on is NaN, and the next call is right again.  Nothing here faults or hangs the GPU: every wait is bounded in time, and the
withheld message is simply never sent."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_recurrence import DTYPES, det, make  # noqa: E402,F401

LIMIT_NS = 5_000_000    # 5 ms


def of_bits(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("withheld", [0, 1, 2, 5])
@pytest.mark.parametrize("form", ["decay", "sigmoid"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_a_wait_that_runs_out(det, kind, form, withheld):  # noqa: F811
    time, channels = 128 * 8 * 8 + 77, 40        # eight rounds and a part, with as many CTAs as a sequence may have
    x, gate, initial, grad, grad_final = (t.cuda() for t in make(1, time, channels, DTYPES[kind], form, withheld))
    want = det.det_linear_recurrence(x, gate, initial, form=form, keep_states=True)
    back = det.det_linear_recurrence_backward(grad, x, gate, want.states, grad_final=grad_final, form=form)
    assert det.lib().det_test_recurrence_withhold(withheld, LIMIT_NS) == 0
    try:
        got = det.det_linear_recurrence(x, gate, initial, form=form, keep_states=True)
        lost = det.det_linear_recurrence_backward(grad, x, gate, want.states, grad_final=grad_final, form=form)
        torch.cuda.synchronize()
    finally:
        assert det.lib().det_test_recurrence_withhold(-1, 0) == 0
    # the first step that is NaN is a round's, of 128 steps for each CTA
    known = int((~got.out.isnan().any(-1)).sum())
    ranks = known // (128 * withheld) if withheld else 8
    assert known == withheld * ranks * 128 and (withheld == 0 or ranks in (1, 2, 4, 8))
    assert torch.equal(got.out[:, :known], want.out[:, :known]) and got.out[:, known:].isnan().all()
    assert got.final.isnan().all()
    assert torch.equal(got.states[:, :known // 128], want.states[:, :known // 128])
    assert got.states[:, known // 128:].isnan().all()
    # and the gradient's from the end
    known = int((~lost.x.isnan().any(-1)).sum())
    assert torch.equal(lost.x[:, time - known:], back.x[:, time - known:]) and lost.x[:, :time - known].isnan().all()
    assert torch.equal(lost.gate[:, time - known:], back.gate[:, time - known:])
    assert lost.gate[:, :time - known].isnan().all() and lost.initial.isnan().all()
    # the context is as it was
    assert of_bits(det.det_linear_recurrence(x, gate, initial, form=form, keep_states=True), want)
    assert of_bits(det.det_linear_recurrence_backward(grad, x, gate, want.states, grad_final=grad_final, form=form), back)


def test_a_round_past_the_end_changes_nothing(det):  # noqa: F811
    x, gate, initial, _, _ = (t.cuda() for t in make(2, 300, 40, torch.bfloat16, "sigmoid", 1))
    want = det.det_linear_recurrence(x, gate, initial)
    assert det.lib().det_test_recurrence_withhold(1000, LIMIT_NS) == 0
    try:
        got = det.det_linear_recurrence(x, gate, initial)
        torch.cuda.synchronize()
    finally:
        det.lib().det_test_recurrence_withhold(-1, 0)
    assert torch.equal(got.out, want.out) and torch.equal(got.final, want.final)
