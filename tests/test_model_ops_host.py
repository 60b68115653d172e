"""Language-model operators on the host: refusals and the bucket bounds (no GPU)."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def det():
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    d.lib()
    return d


FAKE = ctypes.c_void_p(1 << 20)            # never dereferenced: the checks fail first


def test_logprobs_refusals(det):
    f = det.lib().det_token_logprobs
    ok = [FAKE, 4, 100, 100, FAKE, 0, FAKE, FAKE, FAKE, 3, FAKE, FAKE, None]

    def call(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return f(*a)
    assert call(_5=1) == 2 and call(_5=9) == 2                     # dtype (f64 among them)
    assert call(_0=None) == 1 and call(_4=None) == 1               # null logits; logprob without tokens
    assert call(_1=-1) == 1 and call(_2=-1) == 1 and call(_3=-1) == 1
    assert call(_9=-1) == 1 and call(_9=33) == 1                   # alternatives
    assert call(_2=2) == 1                                         # more alternatives than tokens
    assert call(_1=1 << 31) == 3 and call(_2=1 << 31) == 3
    assert call(_0=ctypes.c_void_p((1 << 20) + 2)) == 1            # f32 at an odd address
    assert call(_1=0) == 0                                         # nothing to do
    g = det.lib().det_token_logprobs_backward
    ok = [FAKE, 4, 100, 100, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, 100, None]

    def back(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return g(*a)
    assert back(_5=7) == 2 and back(_6=None) == 1 and back(_10=None) == 1
    assert back(_4=None) == 1 and back(_7=None) == 1
    assert back(_11=99) == 1                                       # rows of the result overlap
    assert back(_1=0) == 0 and back(_2=0) == 0


def test_relative_bias_refusals(det):
    f = det.lib().det_relative_bias
    assert f(FAKE, 0, 4, FAKE, 31, 0, 8, 8, 0, FAKE, 1, None) == 2
    assert f(FAKE, 5, 4, FAKE, 31, 0, 8, 8, 0, FAKE, 0, None) == 2
    assert f(None, 0, 4, FAKE, 31, 0, 8, 8, 0, FAKE, 0, None) == 1
    assert f(FAKE, 0, 4, None, 31, 0, 8, 8, 0, FAKE, 0, None) == 1
    assert f(FAKE, 0, 4, FAKE, 31, 0, -8, 8, 0, FAKE, 0, None) == 1
    assert f(FAKE, 0, 4, FAKE, 2048, 0, 8, 8, 0, FAKE, 0, None) == 3
    assert f(FAKE, 0, 65536, FAKE, 31, 0, 8, 8, 0, FAKE, 0, None) == 3
    assert f(FAKE, 0, 4, FAKE, 31, 0, 1 << 30, 1 << 30, 0, FAKE, 0, None) == 3
    assert f(FAKE, 0, 4, FAKE, 31, 0, 8, 8, 1 << 31, FAKE, 0, None) == 3
    assert f(FAKE, 0, 4, FAKE, 31, 0, 8, 8, -(1 << 40), FAKE, 0, None) == 3
    assert f(FAKE, 0, 4, FAKE, 31, 0, 0, 8, 0, FAKE, 0, None) == 0
    g = det.lib().det_relative_bias_backward
    ok = [FAKE, 0, 2, 4, 8, 8, 256, 64, 8, FAKE, 31, 0, 0, FAKE, 0, FAKE, 1 << 30, None]
    assert g(*ok[:1], 1, *ok[2:]) == 2
    assert g(None, *ok[1:]) == 1
    assert g(*ok[:2], -1, *ok[3:]) == 1
    assert g(*ok[:15], FAKE, 16, None) == 4
    assert g(*ok[:15], ctypes.c_void_p((1 << 20) + 8), 1 << 30, None) == 4
    assert det.lib().det_relative_bias_backward_workspace_bytes(-1, 4, 8, 8, 31, 0) == 0


def test_attention_refusals(det):
    f = det.lib().det_paged_attention
    #      q     sb    sh  k     page   token head v     page   token head pages page table ts mp  len   B  H  KV D  dt  scale bias bd bounds nb max  out   lse   ws    bytes    stream
    ok = [FAKE, 512, 64, FAKE, 2048, 128, 64, FAKE, 2048, 128, 64, 10, 16, FAKE, 8, 8, FAKE, 2, 8, 2, 64, 2, 0.1, None, 0, None, 0, 128, FAKE, FAKE, FAKE, 1 << 30, None]

    def call(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return f(*a)
    assert call(_21=0) == 2 and call(_21=1) == 2                    # 32-bit caches
    assert call(_23=FAKE, _24=1) == 2                               # the bias' type
    assert call(_20=96) == 1 and call(_18=7) == 1 and call(_19=0) == 1 and call(_12=0) == 1
    assert call(_0=None) == 1 and call(_3=None) == 1 and call(_13=None) == 1 and call(_16=None) == 1 and call(_28=None) == 1
    assert call(_5=127) == 1 and call(_8=2047) == 1                 # strides that are no multiples of 8
    assert call(_7=ctypes.c_void_p((1 << 20) + 8)) == 1             # alignment
    assert call(_23=FAKE, _26=4) == 1                               # bounds missing
    assert call(_17=70000) == 3 and call(_27=(1 << 31) - 1) == 3
    assert call(_30=None) == 4 and call(_31=16) == 4
    assert call(_17=0) == 0
    need = det.lib().det_paged_attention_workspace_bytes
    assert need(2, 8, 64, 100) >= 256 and need(2, 8, 64, 100_000) > need(2, 8, 64, 1000) and need(-1, 8, 64, 10) == 0


def test_host_tensors_and_wrong_types_are_refused(det):
    x, t = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: det.det_token_logprobs(x, t),
                 lambda: det.det_token_logprobs_backward(x, t, x[:, 0]),
                 lambda: det.det_relative_bias(torch.zeros(4, 2), torch.zeros(3, dtype=torch.int32), 3, 3),
                 lambda: det.det_relative_bias_backward(torch.zeros(2, 3, 3), torch.zeros(3, dtype=torch.int32)),
                 lambda: det.det_paged_attention(torch.zeros(2, 4, 64, dtype=torch.bfloat16), cache, cache, t[:, None], t)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("buckets,reach,both", [(32, 128, False), (32, 128, True), (64, 1024, False), (8, 17, False), (2, 5, False)])
def test_bounds_are_the_logarithm_s(det, buckets, reach, both):
    """Against the formula in floating point, away from the distances where the logarithm is a whole number."""
    bounds = det.det_relative_bounds(buckets, reach, bidirectional=both, device="cpu").tolist()
    n = buckets // 2 if both else buckets
    exact = max(n // 2, 1)
    assert len(bounds) == n - 1 and bounds == sorted(bounds)
    for d in range(0, 3 * reach):
        got = sum(b <= d for b in bounds)
        if d < exact:
            assert got == d
        else:
            x = math.log(d / exact) / math.log(reach / exact) * (n - exact)
            if abs(x - round(x)) > 1e-9 or x > n - exact:
                assert got == min(exact + int(x), n - 1)
            else:
                assert got == min(exact + round(x), n - 1)


def test_bounds_refusals(det):
    for a, kw in (((1, 10), {}), ((7, 100), {"bidirectional": True}), ((32, 16), {}), ((32, 8), {"bidirectional": True})):
        with pytest.raises(ValueError):
            det.det_relative_bounds(*a, device="cpu", **kw)


def test_workspace_query_of_the_gradient(det):
    q = det.lib().det_relative_bias_backward_workspace_bytes
    assert q(1, 1, 1, 1, 0, 0) > 0 and q(2, 16, 2048, 2048, 31, 1) >= q(1, 16, 2048, 2048, 31, 1)
