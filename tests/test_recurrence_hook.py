"""The recurrence's test hook checks its arguments (no GPU)."""


def test_recurrence_withhold_hook_checks_its_limit():
    from deterministic_floating_point_gb300 import _build, det
    _build.build()
    lib = det.lib()
    assert lib.det_test_recurrence_withhold(5, 0) == 1                 # no limit
    assert lib.det_test_recurrence_withhold(5, 3 * 10**9) == 1         # above the 2 s default
    assert lib.det_test_recurrence_withhold(1 << 31, 10**6) == 1       # more rounds than there are
    assert lib.det_test_recurrence_withhold(-1, 0) == 0                # clearing always works
