"""GPU: the delta rule where magnitudes differ by many orders inside a chunk of
tokens: gates of either sign, keys and values far larger than their
neighbours, states that a gate empties.

Outputs are compared token by token (and, where some channels are scaled,
group of channels by group), so that a large token does not hide a small one.
Tolerance of a token's output: it is rounded once to bf16 (2^-8 of it at most).
It is the sum of what the state before the chunk gives, whose elements are
rounded to 11 bits (2^-11 of a term), and of P_ij U_j over the chunk's tokens up
to it, both factors rounded (2^-10 of a term); the terms may cancel to any
extent (a state that one token dominates is of rank one, and a single product
q.k decides all channels), so these count by the sum of their magnitudes, which
terms() forms in float64.  The roundings of fp32 count STATE() of these and of
the magnitudes of q.S (q.k, too, may be small against its own terms).
The state is held to STATE() of its norm: growing it by a gate scales its error
with it."""
import numpy as np
import pytest

from oracle import delta_rule as dr
from test_gpu_delta_rule import STATE, Case, _cuda, _np, _rel  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu

# narrow scans (few heads), 64 and 128 channels a CTA
SHAPES = [(1, 150, 1, 2, 64, 64), (1, 130, 2, 2, 128, 128), (40, 66, 2, 4, 64, 64), (19, 130, 2, 4, 128, 128)]


def terms(c):
    """[B, Hv, dv, L], twice.  An output's terms summed by magnitude, with chunks of 64 tokens:
    scale (sum_r |q_r| e^{G_i} |S_r| of the state before the chunk + sum_{j <= i} e^{G_i - G_j} |q_i.k_j| |u_j|);
    and with these scale sum_r |q_r| |S_r| of the state that the token reads."""
    n = lambda t, H: _np(t).reshape(c.B, H, -1, c.L).repeat(c.Hv // H, 1).transpose(3, 0, 1, 2)      # [L, B, Hv, d]
    q, k, v = n(c.q, c.Hk), n(c.k, c.Hk), n(c.v, c.Hv)
    if c.l2norm:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + dr.NORM_EPS) for x in (q, k))
    a, beta = np.exp(_np(c.g)).transpose(2, 0, 1), _np(c.beta).transpose(2, 0, 1)
    S = np.zeros((c.B, c.Hv, c.dk, c.dv)) if c.s0 is None else _np(c.s0)
    out, read = np.empty((c.L, c.B, c.Hv, c.dv)), np.empty((c.L, c.B, c.Hv, c.dv))
    for t in range(c.L):
        if t % 64 == 0:
            S0, ks, us, decay = np.abs(S), [], [], np.zeros((0, c.B, c.Hv))
        S = S * a[t][..., None, None]
        S0, decay = S0 * a[t][..., None, None], np.concatenate([decay * a[t], np.ones((1, c.B, c.Hv))])
        u = beta[t][..., None] * (v[t] - np.einsum("bhkv,bhk->bhv", S, k[t]))
        S = S + k[t][..., None] * u[..., None, :]
        ks.append(k[t])
        us.append(np.abs(u))
        p = np.abs(np.einsum("jbhk,bhk->jbh", np.array(ks), q[t])) * decay
        out[t] = np.einsum("bhkv,bhk->bhv", S0, np.abs(q[t])) + np.einsum("jbh,jbhv->bhv", p, np.array(us))
        read[t] = out[t] + np.einsum("bhkv,bhk->bhv", np.abs(S), np.abs(q[t]))
    return tuple(x.transpose(1, 2, 3, 0) * c.dk ** -0.5 for x in (out, read))


def check_tokens(c, o, s1, groups=(slice(None),)):
    """Every token of every row, for each group of a head's channels; then the state."""
    ro, rs = c.oracle()
    assert np.isfinite(rs).all()
    shape = (c.B, c.Hv, c.dv, c.L)
    got, ref = _np(o).reshape(shape), ro.reshape(shape)
    once, parts = (2.0 ** -8, 2.0 ** -10) if c.dtype == "bf16" else (0.0, 0.0)
    for ch in groups:
        num, den, mag, read = (np.linalg.norm(x[:, :, ch], axis=(1, 2)) for x in (got - ref, ref, *terms(c)))
        over = num / np.maximum(once * den + parts * mag + STATE(c.dk, c.L) * read, 1e-300)
        worst = np.unravel_index(np.argmax(over), num.shape)
        assert over[worst] <= 1, (worst, num[worst], den[worst], mag[worst], read[worst])
        assert _rel(_np(s1)[..., ch], rs[..., ch]) <= STATE(c.dk, c.L)


def _gates(c, kind):
    import torch
    t = torch.arange(c.L, device="cuda")
    if kind == "normal":
        g = torch.Generator().manual_seed(11)
        return torch.randn(c.B, c.Hv, c.L, generator=g).cuda()
    a, b = {"+0.4": (0.4, 0.4), "+1 -1": (1.0, -1.0), "+0.7 -0.7": (0.7, -0.7), "+1 -2": (1.0, -2.0), "-1 +1": (-1.0, 1.0)}[kind]
    return torch.where(t % 2 == 0, a, b).expand(c.B, c.Hv, c.L).contiguous()


@pytest.mark.parametrize("kind", ["+1 -1", "+0.7 -0.7", "+1 -2", "-1 +1", "normal", "+0.4"])
@pytest.mark.parametrize("layout", ["first", "last"])
@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv", SHAPES)
def test_gates_of_either_sign(B, L, Hk, Hv, dk, dv, layout, kind):
    """Gates whose positive ones alone would sum to e^30 and more while their running sum stays small; ones that walk
    up and down by e^20 in a chunk; ones that grow the state by e^25 in each."""
    c = Case(B, L, Hk, Hv, dk, dv, layout=layout)
    c.g = _gates(c, kind)
    check_tokens(c, *c.run())


def test_gates_of_either_sign_of_shared_key_heads():
    """Chunks enough for the value heads of a key head to be taken together."""
    c = Case(200, 130, 1, 4, 16, 16)
    c.g = _gates(c, "+1 -1")
    c.g[:, 1::2] *= -1
    check_tokens(c, *c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["first", "last"])
def test_a_late_large_key(dtype, layout):
    """Keys of 1e-5 and at the end of a chunk one of 1e6: what comes before it keeps its outputs, and what comes after
    sums both.  Without a state before, so that the chunk's own keys make them."""
    c = Case(1, 64 + 61, 1, 1, 64, 64, dtype, layout, l2norm=False, state=False, decay=0.0)
    c.k.mul_(1e-5)
    c.k[:, :, 62] *= 1e11
    c.beta[:, :, 62] = 1e-13
    check_tokens(c, *c.run())


def _far(c, kind):
    """One channel of every head, or all of them, far from the other tokens; returns the channels."""
    one = 5 if c.dv <= 64 else 70
    v = c.v.view(c.B, c.Hv, c.dv, c.L) if c.v.is_contiguous() else c.v.unflatten(1, (c.Hv, c.dv))
    if kind == "late value":                              # the tokens before it in its chunk
        v[:, :, one, 50] = 1e12
    elif kind == "last value":                            # a chunk of two tokens, the second large
        v[:, :, one, 65] = 1e12
    elif kind == "value, then a reset":
        v[:, :, one, 40] = 1e9
        c.g[:, :, 41] = float("-inf")
    elif kind == "value, then a strong decay":
        v[:, :, one, 40] = 1e9
        c.g[:, :, 42] = -25.0
    elif kind == "value, then a decay to the last token":
        v[:, :, one, 30] = 3e8
        c.g[:, :, 63] = -18.0
    elif kind == "masked value":                          # write strength 0: it does not exist
        v[:, :, one, 20] = 1e30
        c.beta[:, :, 20] = 0.0
    elif kind == "weak value":                            # write strength 1e-10
        v[:, :, one, 20] = 1e10
        c.beta[:, :, 20] = 1e-10
    elif kind == "state, then a reset":
        c.s0[..., one] *= 1e9
        c.g[:, :, 20] = float("-inf")
    elif kind == "state, then a strong decay":
        c.s0[..., one] *= 1e9
        c.g[:, :, 20] = -22.0
    elif kind == "state of all channels, then a reset":
        c.s0 *= 1e12
        c.g[:, :, 66 if c.L > 100 else 33] = float("-inf")
        return None
    return one


KINDS = ["late value", "last value", "value, then a reset", "value, then a strong decay",
         "value, then a decay to the last token", "masked value", "weak value", "state, then a reset",
         "state, then a strong decay", "state of all channels, then a reset"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["first", "last"])
@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv", [(1, 150, 1, 2, 64, 64), (1, 66, 1, 1, 40, 24), (1, 130, 2, 2, 128, 128),
                                             (40, 66, 2, 4, 64, 64), (19, 130, 2, 4, 128, 128)])
def test_magnitudes_far_apart_in_a_chunk(B, L, Hk, Hv, dk, dv, layout, kind):
    c = Case(B, L, Hk, Hv, dk, dv, layout=layout, decay=0.05)
    one = _far(c, kind)
    rest = [d for d in range(dv) if d != one]
    check_tokens(c, *c.run(), groups=(rest,) if one is None else ([one], rest))


@pytest.mark.parametrize("kind", KINDS)
def test_magnitudes_far_apart_fp32_storage(kind):
    c = Case(1, 80, 1, 2, 64, 64, "f32", decay=0.05)
    one = _far(c, kind)
    rest = [d for d in range(64) if d != one]
    check_tokens(c, *c.run(), groups=(rest,) if one is None else ([one], rest))


@pytest.mark.parametrize("layout", ["first", "last"])
def test_magnitudes_far_apart_without_norms_or_gates(layout):
    """The same through unnormalised keys, no decay, full write strength, a ragged batch."""
    import torch
    c = Case(3, 100, 1, 2, 64, 64, layout=layout, l2norm=False, decay=0.0, lengths=[100, 70, 3])
    c.v.unflatten(1, (2, 64))[:, :, 7, 60] = 1e12
    ref, (mag, read) = c.oracle(), (x.reshape(3, 128, 100) for x in terms(c))
    o, s1 = c.run(c.out(fill=3.0))
    got, live = _np(o), np.isfinite(ref[0])
    assert (got[~live] == 3.0).all() and (live[1, :, :70].all() and not live[1, :, 70:].any())
    err = np.abs(got - ref[0])[live]
    assert (err <= (2.0 ** -8 * np.abs(ref[0]) + 2.0 ** -10 * mag + STATE(64, 100) * read)[live]).all()
    n = _np(s1)
    for ch in ([7], [d for d in range(64) if d != 7]):
        assert _rel(n[..., ch], ref[1][..., ch]) <= STATE(64, 100)
    assert torch.isfinite(s1).all()


@pytest.mark.parametrize("layout", ["first", "last"])
@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv", [(1, 150, 1, 2, 64, 64), (40, 66, 2, 4, 64, 64), (19, 100, 2, 4, 128, 120)])
def test_far_apart_without_gate_tensors_and_with_a_scale(B, L, Hk, Hv, dk, dv, layout):
    """No gates (as zeros and ones), a scale of one's own, the state in place, no final state wanted: the same outputs."""
    import torch
    c = Case(B, L, Hk, Hv, dk, dv, layout=layout, gates=False)
    c.v.unflatten(1, (Hv, dv))[:, :, 3, 40] = 1e12
    o, s1 = c.run(scale=0.25)
    half, _ = c.run(scale=0.125)
    assert torch.equal(o, half * 2)
    s = c.s0.clone()
    o2, _ = c.run(scale=0.25, state_in=s, state_out=s)
    assert torch.equal(o2, o) and torch.equal(s, s1)
    o3, _ = c.run(scale=0.25, state_out=None)
    assert torch.equal(o3, o)
    c.g, c.beta = torch.zeros(B, Hv, L, device="cuda"), torch.ones(B, Hv, L, device="cuda")
    o4, s4 = c.run(scale=0.25)
    assert torch.equal(o4, o) and torch.equal(s4, s1)
    ro, rs = c.oracle(scale=0.25)
    rest = [d for d in range(dv) if d != 3]
    for ch in ([3], rest):
        assert _rel(_np(s1)[..., ch], rs[..., ch]) <= STATE(dk, L)
    early = _np(o).reshape(B, Hv, dv, L)[:, :, 3, :40]             # before the large value, whose channel they share
    ref = ro.reshape(B, Hv, dv, L)[:, :, 3, :40]
    mag, read = (x[:, :, 3, :40] * 0.25 * dk ** 0.5 for x in terms(c))
    assert (np.abs(early - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag + STATE(dk, L) * read).all()


@pytest.mark.parametrize("kind", ["values half zero", "every third token masked", "left 40 masked", "zero keys", "one token repeated",
                                  "zeros, then small, then large", "masked, then small, then large", "all masked"])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv", [(1, 150, 1, 2, 64, 64), (40, 66, 2, 4, 64, 64), (19, 100, 2, 4, 128, 128)])
def test_tokens_that_write_nothing(B, L, Hk, Hv, dk, dv, state, kind):
    """Exact zeros among the writes, alone and before a small write that a large one follows."""
    c = Case(B, L, Hk, Hv, dk, dv, layout="last", state=state, decay=0.05)
    v = c.v.unflatten(1, (Hv, dv))
    groups = (slice(None),)
    if kind == "values half zero":
        c.v.relu_()
    elif kind == "every third token masked":
        c.beta[:, :, ::3] = 0
    elif kind == "left 40 masked":
        c.beta[:, :, :40] = 0
    elif kind == "zero keys":
        c.k[:, :, ::5] = 0
    elif kind == "one token repeated":
        c.k[:], c.v[:] = c.k[:, :, :1].clone(), c.v[:, :, :1].clone()
        c.beta.fill_(1.0)
    elif kind == "all masked":
        c.beta.fill_(0.0)
        if not state:                                     # nothing at all: zeros out
            o, s1 = c.run()
            assert (o == 0).all() and (s1 == 0).all()
            return
    else:
        if kind.startswith("zeros"):
            v[:, :, 9, :11] = 0
        else:
            c.beta[:, :, :11] = 0
        v[:, :, 9, 12] = 1e14
        groups = ([9], [d for d in range(dv) if d != 9])
    check_tokens(c, *c.run(), groups=groups)


@pytest.mark.parametrize("layout", ["first", "last"])
@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv", [(1, 17, 1, 2, 100, 64), (1, 81, 1, 2, 64, 64), (40, 66, 2, 4, 64, 64), (19, 100, 2, 4, 128, 128)])
def test_large_value_masked_at_a_reset_on_the_last_token(B, L, Hk, Hv, dk, dv, layout):
    """Nothing of the chunk remains behind it, and its largest residual writes nothing: the outputs before it still count."""
    c = Case(B, L, Hk, Hv, dk, dv, layout=layout, decay=0.05)
    c.v.unflatten(1, (Hv, dv))[:, :, :, L - 1] = 1e25
    c.beta[:, :, L - 1] = 0.0
    c.g[:, :, L - 1] = float("-inf")
    ro, _ = c.oracle()
    o, s1 = c.run()
    assert (s1 == 0).all()
    mag, read = (x.reshape(B, Hv * dv, L)[:, :, :-1] for x in terms(c))
    err, ref = np.abs(_np(o) - ro)[:, :, :-1], np.abs(ro)[:, :, :-1]
    assert (err <= 2.0 ** -8 * ref + 2.0 ** -10 * mag + STATE(dk, L) * read).all()


@pytest.mark.parametrize("layout", ["first", "last"])
@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv", [(1, 150, 1, 2, 64, 64), (40, 66, 2, 4, 64, 64), (19, 100, 2, 4, 128, 128)])
def test_masked_run_under_a_strong_decay(B, L, Hk, Hv, dk, dv, layout):
    """Tokens that write nothing read what fades, by e^-10 a token, in their own size."""
    c = Case(B, L, Hk, Hv, dk, dv, layout=layout, decay=0.05)
    c.beta[:, :, 20:26] = 0.0
    c.g[:, :, 20:26] = -10.0
    check_tokens(c, *c.run())
