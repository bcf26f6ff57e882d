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
terms() forms in float64.  So do the roundings of the state, STATE() of it.
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
    """[B, Hv, dv, L]: an output's terms summed by magnitude, with chunks of 64 tokens:
    scale (sum_r |q_r| e^{G_i} |S_r| of the state before the chunk + sum_{j <= i} e^{G_i - G_j} |q_i.k_j| |u_j|)."""
    n = lambda t, H: _np(t).reshape(c.B, H, -1, c.L).repeat(c.Hv // H, 1).transpose(3, 0, 1, 2)      # [L, B, Hv, d]
    q, k, v = n(c.q, c.Hk), n(c.k, c.Hk), n(c.v, c.Hv)
    if c.l2norm:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + dr.NORM_EPS) for x in (q, k))
    a, beta = np.exp(_np(c.g)).transpose(2, 0, 1), _np(c.beta).transpose(2, 0, 1)
    S = np.zeros((c.B, c.Hv, c.dk, c.dv)) if c.s0 is None else _np(c.s0)
    out = np.empty((c.L, c.B, c.Hv, c.dv))
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
    return out.transpose(1, 2, 3, 0) * c.dk ** -0.5


def check_tokens(c, o, s1, groups=(slice(None),), tokens=slice(None)):
    """Every token of every row, for each group of a head's channels; then the state."""
    ro, rs = c.oracle()
    assert np.isfinite(rs).all()
    shape = (c.B, c.Hv, c.dv, c.L)
    got, ref, mag = _np(o).reshape(shape), ro.reshape(shape), terms(c)
    once, parts = (2.0 ** -8, 2.0 ** -10) if c.dtype == "bf16" else (0.0, 0.0)
    for ch in groups:
        num, den, size = (np.linalg.norm(x[:, :, ch, tokens], axis=(1, 2)) for x in (got - ref, ref, mag))
        over = num / np.maximum(once * den + (parts + STATE(c.dk, c.L)) * size, 1e-300)
        worst = np.unravel_index(np.argmax(over), num.shape)
        assert over[worst] <= 1, (worst, num[worst], den[worst], size[worst])
        assert _rel(_np(s1)[..., ch], rs[..., ch]) <= STATE(c.dk, c.L)


def _gates(c, kind):
    import torch
    t = torch.arange(c.L, device="cuda")
    a, b = {"+1 -1": (1.0, -1.0), "+0.7 -0.7": (0.7, -0.7), "+1 -2": (1.0, -2.0), "-1 +1": (-1.0, 1.0)}[kind]
    return torch.where(t % 2 == 0, a, b).expand(c.B, c.Hv, c.L).contiguous()


@pytest.mark.parametrize("kind", ["+1 -1", "+0.7 -0.7", "+1 -2", "-1 +1"])
@pytest.mark.parametrize("layout", ["first", "last"])
@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv", SHAPES)
def test_gates_of_either_sign(B, L, Hk, Hv, dk, dv, layout, kind):
    """Gates whose positive ones alone would sum to e^30 and more while their running sum stays small."""
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
    """Keys of 1e-5 and at the end of a chunk one of 1e6: what comes before it keeps its outputs.  Without a state
    before, so that the chunk's own keys make them."""
    c = Case(1, 64 + 61, 1, 1, 64, 64, dtype, layout, l2norm=False, state=False, decay=0.0)
    c.k.mul_(1e-5)
    c.k[:, :, 62] *= 1e11
    c.beta[:, :, 62] = 1e-13
    check_tokens(c, *c.run(), tokens=slice(62))
