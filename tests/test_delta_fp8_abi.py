"""CPU tests of the delta rule's and the e4m3 operators' argument checks: bad
arguments are refused before anything is launched (no GPU needed; the
pointers are never dereferenced)."""
import ctypes

import pytest

from fft_long_convolution_02_b200 import binding as hb

OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
BIG = 1 << 40          # far apart, so nothing overlaps by accident


@pytest.fixture(scope="module")
def lib():
    from fft_long_convolution_02_b200 import build
    build.build()
    return hb.load()


def _args(**kw):
    """B = 2, L = 64, 2 key heads of 32, 4 value heads of 16, bf16, [B, C, L] contiguous."""
    B, L, Hk, Hv, dk, dv = 2, 64, 2, 4, 32, 16
    i3 = ctypes.c_int64 * 3
    ck, cv = i3(Hk * dk * L, L, 1), i3(Hv * dv * L, L, 1)
    gs = (Hv * L, L, 1)
    a = hb.DeltaRule(B, L, Hk, Hv, dk, dv, hb.HYENA_BF16, 0, 0.0, BIG, 2 * BIG, 3 * BIG, 4 * BIG, 5 * BIG, 6 * BIG,
                     ck, ck, cv, cv, i3(*gs), i3(*gs))
    for n, v in kw.items():
        setattr(a, n, i3(*v) if isinstance(v, tuple) else v)
    return a


def test_packed_struct_is_the_declared_one():
    """The binding packs the struct from numbers: byte for byte what its fields give."""
    i3 = ctypes.c_int64 * 3
    st = [(1, 2, 3), (4, 5, 6), (7, 8, 9), (10, 11, 12), (13, 14, 15), (16, 17, 18)]
    a = hb.DeltaRule(21, 22, 23, 24, 25, 26, 1, 1, 0.5, 31, 32, 33, 34, 35, 36, *(i3(*x) for x in st), 41, 42, 43)
    packed = hb._DELTA.pack(21, 22, 23, 24, 25, 26, 1, 1, 0.5, 31, 32, 33, 34, 35, 36, *sum(st, ()), 41, 42, 43)
    assert packed == bytes(a)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
    (dict(B=0), INVALID), (dict(L=0), INVALID), (dict(dk=0), INVALID), (dict(Hv=0), INVALID), (dict(Hk=0), INVALID),
    (dict(B=65536), SHAPE), (dict(L=(1 << 30) + 1), SHAPE), (dict(Hv=3), SHAPE), (dict(dk=129), SHAPE),
    (dict(dv=257), SHAPE), (dict(Hk=8), SHAPE), (dict(Hv=8192), SHAPE),
    (dict(B=65535, L=1 << 30), SHAPE),
    (dict(dtype=2), INVALID), (dict(flags=2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(q=BIG + 1), ALIGN), (dict(o=4 * BIG + 1), ALIGN), (dict(g=5 * BIG + 2), ALIGN), (dict(beta=6 * BIG + 2), ALIGN),
    (dict(lengths=7 * BIG + 2), ALIGN), (dict(state_in=7 * BIG + 8), ALIGN), (dict(state_out=7 * BIG + 4), ALIGN),
    (dict(k_stride=(-1, 64, 1)), INVALID), (dict(v_stride=(1 << 41, 64, 1)), INVALID),
    (dict(o_stride=(0, 64, 1)), INVALID), (dict(o_stride=(4096, 32, 1)), INVALID), (dict(o_stride=(4096, 64, 0)), INVALID),
    (dict(o=BIG), INVALID), (dict(o=2 * BIG + 64), INVALID), (dict(o=5 * BIG), INVALID),
    (dict(state_in=4 * BIG), INVALID), (dict(state_out=3 * BIG), INVALID), (dict(state_out=4 * BIG + 16), INVALID),
    (dict(state_in=7 * BIG, state_out=7 * BIG + 16), INVALID), (dict(lengths=4 * BIG), INVALID),
])
def test_delta_rule_refusals(lib, change, want):
    a = _args(**change)
    assert lib.hyena_delta_rule(ctypes.byref(a), 9 * BIG, 1 << 36, None) == want
    assert lib.hyena_last_error_detail()


def test_delta_rule_workspace_refusals(lib):
    """Chunked sequences want their workspace: its size, alignment and a place of its own."""
    need = lib.hyena_delta_rule_workspace_bytes(2, 64, 2, 4, 32, 16, hb.HYENA_BF16)
    assert need > 0
    assert lib.hyena_delta_rule_workspace_bytes(2, 16, 2, 4, 32, 16, hb.HYENA_BF16) == 0
    assert lib.hyena_delta_rule_workspace_bytes(2, 64, 2, 4, 32, 16, hb.HYENA_F32) == 0
    a = ctypes.byref(_args())
    assert lib.hyena_delta_rule(a, None, 0, None) == 5
    assert lib.hyena_delta_rule(a, 9 * BIG, need - 1, None) == 5
    assert lib.hyena_delta_rule(a, 9 * BIG + 8, need, None) == ALIGN
    for at in (BIG, 2 * BIG, 3 * BIG, 4 * BIG, 5 * BIG, 6 * BIG):
        assert lib.hyena_delta_rule(a, at, need, None) == INVALID


def test_delta_rule_null_struct(lib):
    assert lib.hyena_delta_rule(None, None, 0, None) == INVALID
    assert lib.hyena_delta_rule_step(None, BIG, 4, None, None) == INVALID


@pytest.mark.parametrize("change,states,n,slots,want", [
    (dict(L=2), 8 * BIG, 2, None, INVALID), (dict(state_in=7 * BIG), 8 * BIG, 2, None, INVALID),
    (dict(state_out=7 * BIG), 8 * BIG, 2, None, INVALID), (dict(lengths=7 * BIG), 8 * BIG, 2, None, INVALID),
    ({}, None, 2, None, INVALID), ({}, 8 * BIG + 4, 2, None, ALIGN), ({}, 8 * BIG, 2, 9 * BIG + 1, ALIGN),
    ({}, 8 * BIG, 1, None, INVALID), ({}, 8 * BIG, 0, 9 * BIG, INVALID),
    ({}, BIG, 2, None, INVALID), ({}, 4 * BIG, 2, None, INVALID), ({}, 5 * BIG, 2, None, INVALID),
    ({}, 8 * BIG, 2, 8 * BIG, INVALID), ({}, 8 * BIG, 2, 4 * BIG, INVALID), (dict(dk=200), 8 * BIG, 2, None, SHAPE),
])
def test_delta_step_refusals(lib, change, states, n, slots, want):
    a = _args(**{"L": 1, **change})
    assert lib.hyena_delta_rule_step(ctypes.byref(a), states, n, slots, None) == want


def test_delta_workspace_of_bad_arguments(lib):
    f = lib.hyena_delta_rule_workspace_bytes
    assert f(65535, 1 << 30, 1, 4096, 64, 64, 1) == 0     # would not fit 64 bits of bytes
    assert f(0, 64, 1, 1, 64, 64, 1) == 0 and f(1, 64, 2, 3, 64, 64, 1) == 0 and f(1, 64, 1, 1, 64, 64, 5) == 0


@pytest.mark.parametrize("args,want", [
    ((None, BIG, 2 * BIG, 1, 8, 128, 1, 0), INVALID), ((BIG, None, 2 * BIG, 1, 8, 128, 1, 0), INVALID),
    ((BIG, 2 * BIG, None, 1, 8, 128, 1, 0), INVALID), ((BIG, 2 * BIG, 3 * BIG, 0, 8, 128, 1, 0), INVALID),
    ((BIG, 2 * BIG, 3 * BIG, 1, 0, 128, 1, 0), INVALID), ((BIG, 2 * BIG, 3 * BIG, 1, 8, 0, 1, 0), INVALID),
    ((BIG, 2 * BIG, 3 * BIG, 1, 8, 120, 1, 0), SHAPE), ((BIG, 2 * BIG, 3 * BIG, 65536, 8, 128, 1, 0), SHAPE),
    ((BIG, 2 * BIG, 3 * BIG, 1, 1 << 31, 128, 1, 0), SHAPE), ((BIG, 2 * BIG, 3 * BIG, 1, 8, (1 << 20) + 16, 1, 0), SHAPE),
    ((BIG, 2 * BIG, 3 * BIG, 1, 8, 128, 7, 0), INVALID),
    ((BIG + 8, 2 * BIG, 3 * BIG, 1, 8, 128, 1, 0), ALIGN), ((BIG, 2 * BIG + 8, 3 * BIG, 1, 8, 128, 1, 0), ALIGN),
    ((BIG, 2 * BIG, 3 * BIG + 2, 1, 8, 128, 1, 0), ALIGN),
    ((BIG, BIG + 16, 3 * BIG, 1, 8, 128, 1, 1), INVALID), ((BIG, 2 * BIG, 2 * BIG + 16, 1, 8, 128, 1, 0), INVALID),
])
def test_quantize_refusals(lib, args, want):
    assert lib.hyena_quantize_fp8(*args, None) == want


@pytest.mark.parametrize("args,want", [
    ((None, BIG, 2 * BIG, 8, 128, 1), INVALID), ((BIG, 2 * BIG, 3 * BIG, 0, 128, 1), INVALID),
    ((BIG, 2 * BIG, 3 * BIG, 8, 100, 1), SHAPE), ((BIG, 2 * BIG, 3 * BIG, (1 << 20) + 1, 128, 1), SHAPE),
    ((BIG, 2 * BIG + 4, 3 * BIG, 8, 128, 1), ALIGN), ((BIG, BIG, 3 * BIG, 8, 128, 1), INVALID),
])
def test_quantize_weight_refusals(lib, args, want):
    assert lib.hyena_quantize_fp8_weight(*args, None) == want


_P = (BIG, 2 * BIG, 3 * BIG, 4 * BIG, 5 * BIG, 6 * BIG, 2, 64, 128, 48, 0)


@pytest.mark.parametrize("at,value,want", [
    (0, None, INVALID), (1, None, INVALID), (2, None, INVALID), (3, None, INVALID), (5, None, INVALID),
    (6, 0, INVALID), (7, 0, INVALID), (8, 0, INVALID), (9, 0, INVALID),
    (8, 72, SHAPE), (8, (1 << 20) + 16, SHAPE), (9, (1 << 20) + 1, SHAPE), (6, 65536, SHAPE), (7, 1 << 30, SHAPE),
    (0, BIG + 8, ALIGN), (2, 3 * BIG + 8, ALIGN), (5, 6 * BIG + 2, ALIGN), (1, 2 * BIG + 2, ALIGN),
    (3, 4 * BIG + 1, ALIGN), (4, 5 * BIG + 2, ALIGN),
    (5, BIG + 16, INVALID), (5, 2 * BIG, INVALID), (5, 3 * BIG, INVALID), (5, 4 * BIG, INVALID), (5, 5 * BIG, INVALID),
])
def test_proj_refusals(lib, at, value, want):
    a = list(_P)
    a[at] = value
    assert lib.hyena_proj_fp8(*a, None) == want
