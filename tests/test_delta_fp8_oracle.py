"""CPU: the float64 oracles of the delta rule and of the e4m3 operators,
pinned to hand-derived values and to identities of their definitions."""
import numpy as np
import pytest

from oracle import delta_rule as dr
from oracle import fp8


def test_delta_rule_two_tokens_by_hand():
    # one head, dk = 2, dv = 1, scale 1: S starts (1, 2)
    q = np.array([[[1.0, 0.0], [0.0, 2.0]]])           # q_0 = (1, 0), q_1 = (0, 2)
    k = np.array([[[1.0, 0.0], [0.0, 1.0]]])           # k_0 = (1, 0), k_1 = (0, 1)
    v = np.array([[[5.0, 7.0]]])
    g = np.log(np.array([[[0.5, 1.0]]]))
    beta = np.array([[[0.5, 1.0]]])
    S0 = np.array([[[[1.0], [2.0]]]])
    o, S = dr.delta_rule(q, k, v, g, beta, 1, 1, S0, scale=1.0)
    # token 0: S = (.5, 1); u = .5 (5 - .5) = 2.25; S = (2.75, 1); o = 2.75
    # token 1: u = 7 - 1 = 6; S = (2.75, 7); o = 14
    np.testing.assert_allclose(o[0, 0], [2.75, 14.0])
    np.testing.assert_allclose(S[0, 0, :, 0], [2.75, 7.0])


def test_delta_rule_writes_what_it_reads_back():
    """beta = 1, no decay, unit keys: reading with the last key gives the last value."""
    rng = np.random.default_rng(1)
    q = rng.standard_normal((1, 8, 5))
    v = rng.standard_normal((1, 3, 5))
    o, _ = dr.delta_rule(q, q, v, None, None, 1, 1, scale=1.0, l2norm=True)
    n = np.sqrt((q * q).sum(1))                          # the eps under the root: 1e-6 of |x|^2
    np.testing.assert_allclose(o[0], v[0], rtol=1e-4 / n.min() ** 2, atol=1e-4)


def test_delta_rule_chunk_identity():
    """The chunked form (a triangular solve) equals the recurrence, and a split
    sequence with the carried state equals the whole."""
    rng = np.random.default_rng(2)
    n, dk, dv = 12, 4, 3
    q, k, v = rng.standard_normal((dk, n)), rng.standard_normal((dk, n)) * 0.5, rng.standard_normal((dv, n))
    g, beta, S0 = -rng.random(n), rng.random(n), rng.standard_normal((dk, dv))
    o, S = dr.delta_rule(q[None], k[None], v[None], g[None, None], beta[None, None], 1, 1, S0[None, None], scale=1.0)
    G = np.cumsum(g)
    D = np.tril(np.exp(G[:, None] - G[None, :]))
    A = np.tril(beta[:, None] * D * (k.T @ k), -1)
    U = np.linalg.solve(np.eye(n) + A, beta[:, None] * (v.T - np.exp(G)[:, None] * (k.T @ S0)))
    np.testing.assert_allclose(o[0].T, np.exp(G)[:, None] * (q.T @ S0) + (D * (q.T @ k)) @ U, rtol=1e-10)
    np.testing.assert_allclose(S[0, 0], np.exp(G[-1]) * S0 + k @ (np.exp(G[-1] - G)[:, None] * U), rtol=1e-10)
    m = 5
    o1, S1 = dr.delta_rule(q[None, :, :m], k[None, :, :m], v[None, :, :m], g[None, None, :m], beta[None, None, :m], 1, 1,
                           S0[None, None], scale=1.0)
    o2, S2 = dr.delta_rule(q[None, :, m:], k[None, :, m:], v[None, :, m:], g[None, None, m:], beta[None, None, m:], 1, 1,
                           S1, scale=1.0)
    np.testing.assert_allclose(np.concatenate([o1, o2], -1), o, rtol=1e-12)
    np.testing.assert_allclose(S2, S, rtol=1e-12)


def test_e4m3_grid():
    """Every e4m3 number is its own nearest; midpoints go to the even one."""
    bits = np.arange(127)
    vals = np.where(bits < 8, bits * 2.0 ** -9, (1 + (bits % 8) / 8) * np.exp2(bits // 8 - 7.0))
    assert vals[-1] == 448.0
    np.testing.assert_array_equal(fp8.e4m3(vals), vals)
    np.testing.assert_array_equal(fp8.e4m3(-vals), -vals)
    mid = (vals[:-1] + vals[1:]) / 2
    np.testing.assert_array_equal(fp8.e4m3(mid), np.where(bits[:-1] % 2 == 0, vals[:-1], vals[1:]))
    assert fp8.e4m3(1e9) == 448.0 and np.isnan(fp8.e4m3(np.nan))


@pytest.mark.parametrize("K", [16, 128, 144, 304])
def test_quantize_and_proj_oracle(K):
    rng = np.random.default_rng(K)
    x, w = rng.standard_normal((2, 5, K)), rng.standard_normal((130, K))
    q, s = fp8.quantize_rows(x)
    # a block's largest value stands for itself to an fp32 rounding; every value to half an e4m3 step
    back = fp8.dequantize_rows(q, s)
    amax = np.abs(x[..., :128]).max(-1)
    np.testing.assert_allclose(np.abs(back[..., :128]).max(-1), amax, rtol=2.0 ** -22)
    assert (np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s.max() * 2.0 ** -10) * (1 + 1e-6)).all()
    wq, ws = fp8.quantize_weight(w)
    out = fp8.proj(q, s, wq, ws)
    want = np.zeros((2, 5, 130))
    for n in range(130):
        for k in range(K):
            want[:, :, n] += q[:, :, k] * s[:, k // 128] * wq[n, k] * ws[n // 128, k // 128]
    np.testing.assert_allclose(out, want, rtol=1e-10, atol=1e-12)
