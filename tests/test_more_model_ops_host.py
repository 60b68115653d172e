"""Embedding, layer norm and recurrence on the host: refusals (no GPU)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def det():
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    d.lib()
    return d


FAKE = ctypes.c_void_p(1 << 20)            # never dereferenced: the checks fail first
ODD = ctypes.c_void_p((1 << 20) + 1)


def caller(fn, ok):
    def call(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return fn(*a)
    return call


def test_embedding_refusals(det):
    call = caller(det.lib().det_embedding, [FAKE, 0, 100, 64, 64, FAKE, 10, 1.0, FAKE, 2, None])
    assert call(_1=1) == 2 and call(_9=7) == 2                                     # types
    assert call(_0=None) == 1 and call(_5=None) == 1 and call(_8=None) == 1
    assert call(_2=-1) == 1 and call(_3=-1) == 1 and call(_4=-1) == 1 and call(_6=-1) == 1
    assert call(_0=ODD) == 1 and call(_5=ODD) == 1 and call(_8=ODD) == 1
    assert call(_2=1 << 31) == 3 and call(_3=(1 << 21) + 1) == 3 and call(_6=1 << 31) == 3
    assert call(_6=0) == 0 and call(_3=0) == 0                                     # nothing to do
    size = det.lib().det_embedding_backward_workspace_bytes
    assert size(-1, 5, 5) == 0 and size(5, -1, 5) == 0 and size(5, 5, -1) == 0 and size(0, 0, 0) > 0
    need = size(10, 100, 64)
    call = caller(det.lib().det_embedding_backward, [FAKE, 2, 10, 64, 64, FAKE, 1.0, FAKE, 0, 100, 0, FAKE, need, None])
    assert call(_1=1) == 2 and call(_8=9) == 2
    assert call(_0=None) == 1 and call(_5=None) == 1 and call(_7=None) == 1
    assert call(_2=-1) == 1 and call(_3=-1) == 1 and call(_4=-1) == 1 and call(_9=-1) == 1
    assert call(_0=ODD) == 1 and call(_7=ODD) == 1
    assert call(_2=1 << 31) == 3 and call(_9=1 << 31) == 3
    assert call(_11=None) == 4 and call(_12=need - 1) == 4 and call(_11=ctypes.c_void_p((1 << 20) + 128)) == 4
    assert call(_9=0) == 0 and call(_3=0) == 0


def test_layer_norm_refusals(det):
    call = caller(det.lib().det_layer_norm, [FAKE, 2, 10, 64, 64, FAKE, FAKE, 0, 1e-5, FAKE, FAKE, FAKE, None])
    assert call(_1=1) == 2 and call(_7=1) == 2
    assert call(_0=None) == 1 and call(_9=None) == 1
    assert call(_2=-1) == 1 and call(_3=-1) == 1 and call(_3=0) == 1 and call(_4=-1) == 1
    assert call(_8=-1e-5) == 1 and call(_8=float("nan")) == 1
    for at in ("_0", "_5", "_6", "_9", "_10", "_11"):
        assert call(**{at: ODD}) == 1
    assert call(_2=1 << 31) == 3 and call(_3=16385) == 3
    assert call(_2=0) == 0
    size = det.lib().det_layer_norm_backward_workspace_bytes
    need = size(10, 64)
    call = caller(det.lib().det_layer_norm_backward,
                  [FAKE, 64, FAKE, 64, 2, 10, 64, FAKE, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, need, None])
    assert call(_4=1) == 2 and call(_10=1) == 2
    for at in ("_0", "_2", "_7", "_8"):
        assert call(**{at: None}) == 1
    assert call(_1=-1) == 1 and call(_3=-1) == 1 and call(_5=-1) == 1 and call(_6=0) == 1
    assert call(_5=1 << 31) == 3 and call(_6=16385) == 3
    assert call(_14=None) == 4 and call(_15=need - 1) == 4
    assert call(_5=0, _12=None, _13=None) == 0 and call(_11=None, _12=None, _13=None) == 0


def test_recurrence_refusals(det):
    call = caller(det.lib().det_linear_recurrence,
                  [FAKE, 640, 64, FAKE, 640, 64, 2, 1, 3, 10, 64, FAKE, FAKE, FAKE, FAKE, FAKE, None])
    assert call(_6=1) == 2
    assert call(_7=2) == 1 and call(_7=-1) == 1                                    # form
    assert call(_0=None) == 1 and call(_3=None) == 1 and call(_13=None) == 1
    for at in ("_1", "_2", "_4", "_5", "_8", "_9", "_10"):
        assert call(**{at: -1}) == 1
    for at in ("_0", "_3", "_11", "_12", "_13", "_14", "_15"):
        assert call(**{at: ODD}) == 1
    assert call(_8=65536) == 3 and call(_9=1 << 31) == 3 and call(_10=1 << 31) == 3
    assert call(_8=0) == 0 and call(_10=0) == 0
    call = caller(det.lib().det_linear_recurrence_backward,
                  [FAKE, 640, 64, FAKE, 640, 64, FAKE, 640, 64, 2, 1, 3, 10, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None])
    assert call(_9=1) == 2 and call(_10=2) == 1
    for at in ("_3", "_6", "_14", "_17", "_18"):
        assert call(**{at: None}) == 1
    for at in ("_1", "_2", "_4", "_5", "_7", "_8", "_11", "_12", "_13"):
        assert call(**{at: -1}) == 1
    for at in ("_0", "_3", "_6", "_14", "_15", "_16", "_17", "_18", "_19"):
        assert call(**{at: ODD}) == 1
    assert call(_11=65536) == 3
    assert call(_11=0) == 0 and call(_13=0) == 0


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on the second GPU."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))


def on_device(t):
    return torch.Tensor._make_subclass(OnDevice, t)


@pytest.fixture
def calls(det, monkeypatch):
    """The binding against a library that notes its calls, on tensors that only say where they lie."""
    made = []

    class Library:
        def __getattr__(self, name):
            if name.endswith("_workspace_bytes"):
                return lambda *a: 256
            if name == "det_status_string":
                return lambda code: b"refused"
            return lambda *a: made.append((name, a)) or 0

    monkeypatch.setattr(det, "lib", lambda: Library())
    monkeypatch.setattr(det, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(det, "_empty", lambda shape, dtype, device, stream: on_device(torch.empty(shape, dtype=dtype)))
    monkeypatch.setattr(det, "_current_device", lambda: 1)
    return made


def test_binding_refuses_shapes_types_and_devices(det, calls):
    table, tokens = on_device(torch.zeros(9, 4)), on_device(torch.zeros(3, dtype=torch.int32))
    x, gate = on_device(torch.zeros(2, 5, 4)), on_device(torch.zeros(2, 5, 4))
    row, w = on_device(torch.zeros(2, 5)), on_device(torch.zeros(4))
    states = on_device(torch.zeros(2, 1, 4))
    bad = [
        lambda: det.det_embedding(torch.zeros(9, 4), tokens),
        lambda: det.det_embedding(table, torch.zeros(3, dtype=torch.int32)),
        lambda: det.det_embedding(table, on_device(torch.zeros(3, dtype=torch.int64))),
        lambda: det.det_embedding(on_device(torch.zeros(9)), tokens),
        lambda: det.det_embedding(on_device(torch.zeros(4, 9).t()), tokens),
        lambda: det.det_embedding(on_device(torch.zeros(9, 4, dtype=torch.float64)), tokens),
        lambda: det.det_embedding(table, tokens, out=on_device(torch.zeros(3, 5))),
        lambda: det.det_embedding(table, tokens, dtype=torch.float16, out=on_device(torch.zeros(3, 4))),
        lambda: det.det_embedding_backward(on_device(torch.zeros(4, 4)), tokens, 9),
        lambda: det.det_embedding_backward(on_device(torch.zeros(3, 4)), tokens, 9, accumulate=True),
        lambda: det.det_embedding_backward(on_device(torch.zeros(3, 4)), tokens, 9, grad_table=on_device(torch.zeros(8, 4))),
        lambda: det.det_embedding_backward(on_device(torch.zeros(3, 4)), tokens, 9,
                                           workspace=on_device(torch.zeros(8, dtype=torch.uint8))),
        lambda: det.det_layer_norm(x, on_device(torch.zeros(5))),
        lambda: det.det_layer_norm(x, w, on_device(torch.zeros(4, dtype=torch.bfloat16))),
        lambda: det.det_layer_norm(x, w, torch.zeros(4)),
        lambda: det.det_layer_norm(on_device(torch.zeros(())), w),
        lambda: det.det_layer_norm(on_device(torch.zeros(2, 5, 8)[:, :3, :4].transpose(0, 1)), w),
        lambda: det.det_layer_norm(x, w, out=on_device(torch.zeros(2, 5, 4, dtype=torch.float16))),
        lambda: det.det_layer_norm_backward(on_device(torch.zeros(2, 5, 4, dtype=torch.float16)), x, row, row, w),
        lambda: det.det_layer_norm_backward(x, x, on_device(torch.zeros(10)), row, w),
        lambda: det.det_layer_norm_backward(x, x, row, row, w, dtype=torch.float16),
        lambda: det.det_layer_norm_backward(x, x, row, row, dtype=torch.float64),
        lambda: det.det_linear_recurrence(x, on_device(torch.zeros(2, 5, 3))),
        lambda: det.det_linear_recurrence(x, on_device(torch.zeros(2, 5, 4, dtype=torch.float16))),
        lambda: det.det_linear_recurrence(x, gate, form="other"),
        lambda: det.det_linear_recurrence(x, gate, on_device(torch.zeros(2, 4, dtype=torch.float16))),
        lambda: det.det_linear_recurrence(x, gate, on_device(torch.zeros(4))),
        lambda: det.det_linear_recurrence(x, gate, lengths=on_device(torch.zeros(3, dtype=torch.int32))),
        lambda: det.det_linear_recurrence(on_device(torch.zeros(2, 4, 5).transpose(1, 2)), gate),
        lambda: det.det_linear_recurrence(on_device(torch.zeros(5, 4)), on_device(torch.zeros(5, 4))),
        lambda: det.det_linear_recurrence_backward(x, x, gate, on_device(torch.zeros(2, 2, 4))),
        lambda: det.det_linear_recurrence_backward(x, x, gate, states, grad_final=on_device(torch.zeros(2, 5))),
        lambda: det.det_linear_recurrence_backward(on_device(torch.zeros(2, 5, 5)), x, gate, states),
    ]
    for k, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, det.DetError)):
            f()
        assert not calls, k


def test_calls_run_on_the_tensors_device_and_stream(det, calls, monkeypatch):
    import contextlib
    state = {"current": 0}

    @contextlib.contextmanager
    def device(d):
        before, state["current"] = state["current"], d.index
        try:
            yield
        finally:
            state["current"] = before
    seen = []

    class Library:
        def __getattr__(self, name):
            if name.endswith("_workspace_bytes"):
                return lambda *a: 256
            return lambda *a: seen.append((name, state["current"], a[-1])) or 0
    monkeypatch.setattr(det, "lib", lambda: Library())
    monkeypatch.setattr(det, "_current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "device", device)
    x, row, w = on_device(torch.zeros(2, 5, 4)), on_device(torch.zeros(2, 5)), on_device(torch.zeros(4))
    tokens = on_device(torch.zeros(2, 5, dtype=torch.int32))
    det.det_embedding(on_device(torch.zeros(9, 4)), tokens)
    det.det_embedding_backward(x, tokens, 9)
    det.det_layer_norm(x, w)
    det.det_layer_norm_backward(x, x, row, row, w)
    det.det_linear_recurrence(x, x)
    det.det_linear_recurrence_backward(x, x, x, on_device(torch.zeros(2, 1, 4)))
    assert seen == [(n, 1, 1001) for n in ("det_embedding", "det_embedding_backward", "det_layer_norm",
                                           "det_layer_norm_backward", "det_linear_recurrence",
                                           "det_linear_recurrence_backward")]
    assert state["current"] == 0
