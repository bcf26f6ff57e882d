"""CPU tests of the test hooks' argument checks: refused before anything is launched."""
import ctypes

from test_delta_fp8_abi import _P, BIG, INVALID, SHAPE, _args, lib  # noqa: F401 (fixture)


def test_delta_hook_refusals(lib):  # noqa: F811
    f = lib.hyena_debug_delta_rule
    a = ctypes.byref(_args())
    assert f(None, 9 * BIG, 1 << 36, 1000, 0, None) == INVALID
    assert f(a, 9 * BIG, 1 << 36, 0, 0, None) == INVALID                  # no budget
    assert f(a, None, 0, 1000, 0, None) == 5                              # no workspace
    assert f(ctypes.byref(_args(L=16)), 9 * BIG, 1 << 36, 1000, 0, None) == SHAPE      # token by token: no waits
    assert f(ctypes.byref(_args(q=None)), 9 * BIG, 1 << 36, 1000, 0, None) == INVALID


def test_proj_hook_refusals(lib):  # noqa: F811
    f = lib.hyena_debug_proj_fp8
    assert f(*_P, 0, 0, None) == INVALID                                  # no budget
    assert f(*_P, 1000, 3, None) == INVALID and f(*_P, 1000, -1, None) == INVALID
    assert f(*_P[:6], 2, 8, *_P[8:], 1000, 0, None) == SHAPE              # 16 rows: no waits
    assert f(None, *_P[1:], 1000, 1, None) == INVALID
    assert f(*_P[:8], 72, *_P[9:], 1000, 1, None) == SHAPE
