"""The language-model operators make the tensors' device the current one for the library's call (no GPU: the library, the
tensors' device and the current device are stand-ins)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from deterministic_floating_point_gb300 import det  # noqa: E402


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on the second GPU."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))


def on_device(t):
    return torch.Tensor._make_subclass(OnDevice, t)


@pytest.fixture
def calls(monkeypatch):
    state = {"current": 0, "calls": []}

    class Library:
        def __getattr__(self, name):
            if name.endswith("_workspace_bytes"):
                return lambda *a: 256
            if name == "det_status_string":
                return lambda code: b"refused"
            return lambda *a: state["calls"].append((name, state["current"], a[-1])) or state.get("rc", 0)

    @contextlib.contextmanager
    def device(d):
        before, state["current"] = state["current"], d.index
        try:
            yield
        finally:
            state["current"] = before
    monkeypatch.setattr(det, "lib", lambda: Library())
    monkeypatch.setattr(det, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(det, "_empty", lambda shape, dtype, device, stream: on_device(torch.empty(shape, dtype=dtype)))
    monkeypatch.setattr(det, "_current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "device", device)
    return state


def run_all():
    x, t = on_device(torch.zeros(2, 8)), on_device(torch.zeros(2, dtype=torch.int32))
    row, bounds = on_device(torch.zeros(2)), on_device(torch.zeros(3, dtype=torch.int32))
    det.det_token_logprobs(x, t, top_k=2)
    det.det_token_logprobs_backward(x, t, row, row, grad_logprob=row)
    det.det_relative_bias(on_device(torch.zeros(4, 2)), bounds, 3, 3)
    det.det_relative_bias_backward(on_device(torch.zeros(2, 3, 3)), bounds)
    cache = on_device(torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16))
    det.det_paged_attention(on_device(torch.zeros(2, 4, 64, dtype=torch.bfloat16)), cache, cache,
                            on_device(torch.zeros(2, 1, dtype=torch.int32)), t)


NAMES = ["det_token_logprobs", "det_token_logprobs_backward", "det_relative_bias", "det_relative_bias_backward",
         "det_paged_attention"]


@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_the_tensors_device(calls, current):
    calls["current"] = current
    run_all()
    # the current device in the call, and the stream of the tensors' device
    assert calls["calls"] == [(name, 1, 1001) for name in NAMES]
    assert calls["current"] == current


def test_the_device_is_put_back_after_an_error(calls):
    calls["rc"] = 3
    with pytest.raises(det.DetError):
        run_all()
    assert calls["current"] == 0 and len(calls["calls"]) == 1


def test_a_stream_given_as_a_handle_is_one_of_the_tensors_device(monkeypatch):
    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: made.append((handle, device)))
    det._stream_object(5, torch.device("cuda", 1))
    assert made == [(5, torch.device("cuda", 1))]
