"""det_layer_norm refuses an infinite eps (no GPU: the check comes first)."""
import ctypes

import pytest


def test_an_infinite_eps_is_refused():
    pytest.importorskip("torch")
    from deterministic_floating_point_gb300 import _build, det
    _build.build()
    fake = ctypes.c_void_p(1 << 20)            # never dereferenced
    for eps in (float("inf"), float("-inf"), float("nan"), -1e-30):
        assert det.lib().det_layer_norm(fake, 0, 10, 64, 64, None, None, 0, eps, fake, None, None, None) == 1
