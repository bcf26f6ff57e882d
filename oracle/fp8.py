"""e4m3 with a scale for each block of 128, and products of such operands, in
float64.  Plain numpy; shares no code with the CUDA path."""
import numpy as np

E4M3_MAX = 448.0
TINY = np.float32(2.0 ** -126)


def e4m3(y):
    """Nearest e4m3 value, ties to even, saturating; NaN stays."""
    y = np.asarray(y, np.float64)
    _, e = np.frexp(np.where(np.isfinite(y), y, 0.0))
    ulp = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.round(y / ulp) * ulp, -E4M3_MAX, E4M3_MAX)


def _scale(amax):
    """amax / 448 as an fp32 number, at least 2^-126 (a NaN stays)."""
    s = (np.asarray(amax, np.float64) / E4M3_MAX).astype(np.float32)
    return np.where(s < TINY, TINY, s)


def quantize_rows(x):
    """x [B, L, K] -> values [B, L, K], scales [B, ceil(K/128), L] (fp32).  The
    quotient is an fp32 number: float64 division, rounded once more, gives it."""
    x = np.asarray(x, np.float64)
    B, L, K = x.shape
    n = -(-K // 128)
    q, s = np.empty_like(x), np.empty((B, n, L), np.float32)
    for j in range(n):
        b = x[:, :, 128 * j:128 * j + 128]
        s[:, j] = _scale(np.abs(b).max(-1))
        with np.errstate(invalid="ignore"):
            q[:, :, 128 * j:128 * j + 128] = e4m3((b / s[:, j][..., None].astype(np.float64)).astype(np.float32))
    return q, s


def quantize_weight(w):
    """w [N, K] -> values [N, K], scales [ceil(N/128), ceil(K/128)] (fp32)."""
    w = np.asarray(w, np.float64)
    N, K = w.shape
    q, s = np.empty_like(w), np.empty((-(-N // 128), -(-K // 128)), np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = np.s_[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            s[i, j] = _scale(np.abs(w[at]).max())
            q[at] = e4m3((w[at] / np.float64(s[i, j])).astype(np.float32))
    return q, s


def dequantize_rows(q, s):
    K = q.shape[2]
    return np.asarray(q, np.float64) * np.asarray(s, np.float64).transpose(0, 2, 1)[:, :, np.arange(K) // 128]


def dequantize_weight(q, s):
    N, K = q.shape
    return np.asarray(q, np.float64) * np.asarray(s, np.float64)[np.arange(N) // 128][:, np.arange(K) // 128]


def proj(xq, xs, wq, ws, bias=None):
    """[B, L, N] in float64."""
    out = dequantize_rows(xq, xs) @ dequantize_weight(wq, ws).T
    return out if bias is None else out + np.asarray(bias, np.float64)
