"""The gated delta rule in float64, token by token, from its definition:

    S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;  o = scale S^T q

Plain numpy; shares no code with the CUDA path."""
import numpy as np

NORM_EPS = 1e-6


def _heads(x, H, B, L):
    """[B, H d, L] -> [L, B, H, d]."""
    return np.ascontiguousarray(np.asarray(x, np.float64).reshape(B, H, -1, L).transpose(3, 0, 1, 2))


def delta_rule(q, k, v, g, beta, Hk, Hv, state=None, lengths=None, scale=None, l2norm=False):
    """q, k [B, Hk dk, L], v [B, Hv dv, L], g, beta [B, Hv, L] or None, state
    [B, Hv, dk, dv] or None, lengths [B] or None.  Returns (o [B, Hv dv, L] with
    NaN behind a row's length, the state after each row's last token)."""
    B, _, L = q.shape
    dk, dv = q.shape[1] // Hk, v.shape[1] // Hv
    q, k, v = _heads(q, Hk, B, L), _heads(k, Hk, B, L), _heads(v, Hv, B, L)
    scale = dk ** -0.5 if scale is None else scale
    S = np.zeros((B, Hv, dk, dv)) if state is None else np.array(state, np.float64)
    o = np.full((B, Hv * dv, L), np.nan)
    head = np.arange(Hv) // (Hv // Hk)
    for b in range(B):
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        for t in range(n):
            kt, qt = k[t, b], q[t, b]
            if l2norm:
                kt = kt / np.sqrt((kt * kt).sum(-1, keepdims=True) + NORM_EPS)
                qt = qt / np.sqrt((qt * qt).sum(-1, keepdims=True) + NORM_EPS)
            kt, qt = kt[head], qt[head]
            a = np.ones(Hv) if g is None else np.exp(np.asarray(g[b, :, t], np.float64))
            w = np.ones(Hv) if beta is None else np.asarray(beta[b, :, t], np.float64)
            S[b] = a[:, None, None] * S[b]
            u = w[:, None] * (v[t, b] - np.einsum("hkv,hk->hv", S[b], kt))
            S[b] += kt[:, :, None] * u[:, None, :]
            o[b, :, t] = scale * np.einsum("hkv,hk->hv", S[b], qt).reshape(-1)
    return o, S
