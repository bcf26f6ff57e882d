"""GPU: quantisation to e4m3 with a scale for each block of 128, the projection
of such operands, and the layer that runs them around the delta rule.

Quantisation is compared value for value: scale and quotient are fp32 numbers
by definition.  The projection's products of e4m3 numbers are exact in fp32;
its sums round by at most K 2^-24 of the sum of magnitudes (tested per
element against that sum), then once to bf16 (half a step, 2^-8)."""
import numpy as np
import pytest

from fft_long_convolution_02_b200 import binding as hb
from oracle import delta_rule as dr
from oracle import fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fft_long_convolution_02_b200 import build
    build.build()


def _np(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def _f8(t):
    import torch
    return _np(t.to(torch.float32))


def _quantize(x, first):
    import torch
    B, L, K = (x.shape[0], x.shape[2], x.shape[1]) if first else x.shape
    xq = torch.zeros(B, L, K, dtype=torch.float8_e4m3fn, device="cuda")
    xs = torch.full((B, -(-K // 128), L), float("nan"), device="cuda")
    hb.hyena_quantize_fp8(x, xq, xs, channels_first=first)
    torch.cuda.synchronize()
    return xq, xs


def _wide(shape, seed):
    """Values over many orders, zeros among them, some on e4m3 midpoints of their block."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(3.0 * torch.randn(*shape, generator=g))
    return torch.where(torch.rand(*shape, generator=g) < 0.1, torch.zeros(()), x)


@pytest.mark.parametrize("B,L,K", [(1, 1, 16), (2, 7, 128), (1, 64, 144), (3, 65, 272), (1, 130, 768), (2, 200, 2000)])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize(B, L, K, first, dtype):
    import torch
    x = _wide((B, L, K), L + K).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    x[0, 0, :16] = 0
    xq, xs = _quantize(x.transpose(1, 2).contiguous() if first else x, first)
    q, s = fp8.quantize_rows(_np(x))
    np.testing.assert_array_equal(xs.cpu().numpy(), s)
    np.testing.assert_array_equal(_f8(xq), q)


@pytest.mark.parametrize("mag", [1e-44, 1e-38, 1e-30, 2.0 ** -61, 1e-18, 1e18, 3e38])
@pytest.mark.parametrize("first", [False, True])
def test_quantize_magnitudes(mag, first):
    """Blocks near both ends of fp32, either side of where the quotient is divided plainly."""
    import torch
    g = torch.Generator().manual_seed(5)
    x = ((torch.rand(1, 70, 160, generator=g) * 2 - 1).double() * mag).float().cuda()
    xq, xs = _quantize(x.transpose(1, 2).contiguous() if first else x, first)
    q, s = fp8.quantize_rows(_np(x))
    np.testing.assert_array_equal(xs.cpu().numpy(), s)
    np.testing.assert_array_equal(_f8(xq), q)


@pytest.mark.parametrize("first", [False, True])
def test_quantize_zero_and_not_finite(first):
    import torch
    x = torch.ones(1, 8, 256, device="cuda")
    x[0, 0] = 0
    x[0, 1, 5] = float("nan")
    x[0, 2, 6] = float("inf")
    x[0, 3, 130] = float("-inf")
    xq, xs = _quantize(x.transpose(1, 2).contiguous() if first else x, first)
    v = fp8.dequantize_rows(_f8(xq), xs.cpu().numpy())
    assert (v[0, 0] == 0).all() and np.isnan(v[0, 1, :128]).all() and np.isnan(v[0, 2, :128]).all()
    assert np.isnan(v[0, 3, 128:]).all()
    np.testing.assert_allclose(v[0, 1:3, 128:], 1.0, rtol=2.0 ** -22)
    np.testing.assert_allclose(v[0, 3:, :128], 1.0, rtol=2.0 ** -22)


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (130, 144), (300, 784)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_weight(N, K, dtype):
    import torch
    w = _wide((N, K), N + K).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    wq = torch.zeros(N, K, dtype=torch.float8_e4m3fn, device="cuda")
    ws = torch.full((-(-N // 128), -(-K // 128)), float("nan"), device="cuda")
    hb.hyena_quantize_fp8_weight(w, wq, ws)
    torch.cuda.synchronize()
    q, s = fp8.quantize_weight(_np(w))
    np.testing.assert_array_equal(ws.cpu().numpy(), s)
    np.testing.assert_array_equal(_f8(wq), q)


def _operands(B, L, K, N, seed, spread=2.0):
    """Random e4m3 numbers and scales over several powers of two."""
    import torch
    g = torch.Generator().manual_seed(seed)
    xq = (torch.randn(B, L, K, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
    wq = (torch.randn(N, K, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
    xs = torch.exp(spread * torch.randn(B, -(-K // 128), L, generator=g)).mul_(1e-2).cuda()
    ws = torch.exp(spread * torch.randn(-(-N // 128), -(-K // 128), generator=g)).mul_(1e-3).cuda()
    return xq, xs, wq, ws, torch.randn(N, generator=g).cuda()


def _check_proj(out, first, xq, xs, wq, ws, bias):
    got = _np(out).transpose(0, 2, 1) if first else _np(out)
    x, w = fp8.dequantize_rows(_f8(xq), _np(xs)), fp8.dequantize_weight(_f8(wq), _np(ws))
    b = 0.0 if bias is None else _np(bias)
    ref, mag = x @ w.T + b, np.abs(x) @ np.abs(w).T + np.abs(b)
    K = x.shape[2]
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + mag * (K + 8) * 2.0 ** -24 * (1 + 2.0 ** -8)).all()
    assert np.linalg.norm(got - ref) <= (2.0 ** -8 + 1e-5) * np.linalg.norm(ref)


PROJ = [
    # B, L, K, N: a few tokens, small products, ragged tiles, several waves
    (1, 1, 16, 1), (1, 1, 2048, 2304), (1, 4, 128, 16), (2, 4, 784, 100), (1, 9, 272, 33), (4, 5, 512, 130), (1, 32, 768, 300),
    (1, 33, 768, 300), (3, 11, 144, 257), (1, 128, 128, 64), (2, 100, 784, 1000), (1, 130, 48, 129), (3, 333, 784, 1000),
    (1, 777, 1040, 520), (2, 1024, 768, 2304), (1, 6000, 256, 1100), (4, 1500, 400, 1032),
]


@pytest.mark.parametrize("B,L,K,N", PROJ)
@pytest.mark.parametrize("first", [False, True])
def test_proj(B, L, K, N, first):
    import torch
    ops = _operands(B, L, K, N, B + L + K + N)
    bias = ops[4] if (L + N) % 2 else None
    out = torch.full((B, N, L) if first else (B, L, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    hb.hyena_proj_fp8(*ops[:4], bias, out, channels_first=first)
    torch.cuda.synchronize()
    hb.hyena_kernel_status()
    _check_proj(out, first, *ops[:4], bias)


@pytest.mark.parametrize("L", [8, 200])
def test_proj_cancelling_sums(L):
    """Two halves of K that cancel but for a small rest: the sums really are fp32."""
    import torch
    K, N = 1024, 256
    xq, xs, wq, ws, _ = _operands(1, L, K // 2, N, 3, spread=0.0)
    r = torch.randn(N, K // 2, generator=torch.Generator().manual_seed(9)).cuda()
    x2 = torch.cat([xq.float(), xq.float()], 2).to(torch.float8_e4m3fn)
    w2 = torch.cat([wq.float(), -wq.float()], 1)
    w2[:, :128] = torch.where(r[:, :128] > 1.5, 2.0 ** -9 * torch.ones(()).cuda(), w2[:, :128])
    w2 = w2.to(torch.float8_e4m3fn)
    xs2, ws2 = torch.cat([xs, xs], 1), torch.cat([ws, ws], 1)
    out = torch.empty(1, L, N, dtype=torch.bfloat16, device="cuda")
    hb.hyena_proj_fp8(x2, xs2, w2, ws2, None, out)
    torch.cuda.synchronize()
    got = _np(out)
    x, w = fp8.dequantize_rows(_f8(x2), _np(xs2)), fp8.dequantize_weight(_f8(w2), _np(ws2))
    ref, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + mag * (K + 8) * 2.0 ** -24 * (1 + 2.0 ** -8)).all()


def test_proj_keeps_its_surroundings_and_repeats():
    """Outputs inside a larger buffer, captured and replayed: the same bits, nothing beside them."""
    import torch
    B, L, K, N = 1, 331, 400, 130
    xq, xs, wq, ws, bias = _operands(B, L, K, N, 77)
    buf = torch.full((B * N * L + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = buf[32:-32].view(B, N, L)
    hb.hyena_proj_fp8(xq, xs, wq, ws, bias, out, channels_first=True)
    torch.cuda.synchronize()
    first = out.clone()
    _check_proj(out, True, xq, xs, wq, ws, bias)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        hb.hyena_proj_fp8(xq, xs, wq, ws, bias, out, channels_first=True)
    out.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and (buf[:32] == 9.0).all() and (buf[-32:] == 9.0).all()


def test_proj_at_the_benchmarked_size_sampled():
    """B = 4, L = 8192, D = 768, the three channel blocks of an order-2 projection: 64 positions and 64 outputs."""
    import torch
    B, L, K, N = 4, 8192, 768, 2304
    xq, xs, wq, ws, bias = _operands(B, L, K, N, 1)
    out = torch.empty(B, N, L, dtype=torch.bfloat16, device="cuda")
    hb.hyena_proj_fp8(xq, xs, wq, ws, bias, out, channels_first=True)
    torch.cuda.synchronize()
    hb.hyena_kernel_status()
    rng = np.random.default_rng(2)
    at = np.sort(rng.choice(L, 64, replace=False))
    _check_proj(out[:, :, at], True, xq[:, at], xs[:, :, at], wq, ws, bias)


def test_binding_refuses_wrong_tensors():
    import torch
    xq, xs, wq, ws, bias = _operands(1, 8, 256, 32, 1)
    out = torch.empty(1, 8, 32, dtype=torch.bfloat16, device="cuda")
    good = [xq, xs, wq, ws, bias, out]
    for i, t in ((0, xq.float()), (1, xs[:, :1]), (2, wq[:, :128]), (3, ws.double()), (4, bias[:31]), (5, out.float()),
                 (0, xq.cpu()), (5, out.transpose(1, 2))):
        a = list(good)
        a[i] = t
        with pytest.raises(ValueError):
            hb.hyena_proj_fp8(*a)
    with pytest.raises(ValueError):
        hb.hyena_quantize_fp8(torch.zeros(1, 8, 256, device="cuda"), xq, xs[:, :, :4])
    with pytest.raises(TypeError):
        hb.hyena_quantize_fp8(torch.zeros(1, 8, 256, device="cuda", dtype=torch.float16), xq, xs)


def _layer(seed, D, Hk, Hv, dk, dv):
    import torch
    g = torch.Generator().manual_seed(seed)
    C = 2 * Hk * dk + Hv * dv
    w = {}
    for name, n, k in (("in", C, D), ("out", D, Hv * dv)):
        W = (torch.randn(n, k, generator=g) * k ** -0.5).to(torch.bfloat16).cuda()
        wq = torch.empty(n, k, dtype=torch.float8_e4m3fn, device="cuda")
        ws = torch.empty(-(-n // 128), -(-k // 128), device="cuda")
        hb.hyena_quantize_fp8_weight(W, wq, ws)
        w[name] = (wq, ws, torch.randn(n, generator=g).mul_(0.1).cuda())
    w["taps"] = (torch.randn(C, 3, generator=g) * 0.5).cuda()
    return w, C


@pytest.mark.parametrize("B,L,D,Hk,Hv,dk,dv", [(2, 256, 192, 1, 2, 64, 64), (1, 1024, 256, 2, 2, 128, 128)])
def test_layer_of_the_operators(orc, B, L, D, Hk, Hv, dk, dv):
    """x -> e4m3 -> input projection -> short conv -> delta rule -> e4m3 ->
    output projection, each stage against the oracle on what the stage before
    gave, the whole without a copy or a synchronisation between."""
    import torch
    w, C = _layer(3, D, Hk, Hv, dk, dv)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(B, L, D, generator=g).to(torch.bfloat16).cuda()
    decay = (-0.2 * torch.rand(B, Hv, L, generator=g)).cuda()
    beta = torch.sigmoid(torch.randn(B, Hv, L, generator=g)).cuda()
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")
    f8 = torch.float8_e4m3fn
    xq, xs, u, uc = e(B, L, D, dt=f8), e(B, -(-D // 128), L, dt=torch.float32), e(B, C, L), e(B, C, L)
    y, out, s1 = e(B, Hv * dv, L), e(B, L, D), e(B, Hv, dk, dv, dt=torch.float32)
    yq, ys = e(B, L, Hv * dv, dt=f8), e(B, -(-Hv * dv // 128), L, dt=torch.float32)
    n = hb.hyena_delta_rule_workspace_bytes(B, L, Hk, Hv, dk, dv, torch.bfloat16)
    ws = e(n, dt=torch.uint8) if n else None
    hb.hyena_quantize_fp8(x, xq, xs)
    hb.hyena_proj_fp8(xq, xs, *w["in"], u, channels_first=True)
    hb.hyena_shortconv(u, uc, w["taps"])
    q, k, v = uc[:, :Hk * dk], uc[:, Hk * dk:2 * Hk * dk], uc[:, 2 * Hk * dk:]
    hb.hyena_delta_rule(q, k, v, decay, beta, y, Hk, Hv, None, s1, l2norm=True, workspace=ws)
    hb.hyena_quantize_fp8(y, yq, ys, channels_first=True)
    hb.hyena_proj_fp8(yq, ys, *w["out"], out)
    torch.cuda.synchronize()
    hb.hyena_kernel_status()
    np.testing.assert_array_equal(_f8(xq), fp8.quantize_rows(_np(x))[0])
    _check_proj(u, True, xq, xs, *w["in"])
    ro, rs = dr.delta_rule(_np(q), _np(k), _np(v), _np(decay), _np(beta), Hk, Hv, l2norm=True)
    assert np.linalg.norm(_np(y) - ro) <= (2.0 ** -8 + 3 * 2.0 ** -11 + 1e-4) * np.linalg.norm(ro)
    assert np.linalg.norm(_np(s1) - rs) <= 2 * np.sqrt(dk * (L + 16.0)) * 2.0 ** -24 * np.linalg.norm(rs)
    np.testing.assert_array_equal(_f8(yq), fp8.quantize_rows(_np(y).transpose(0, 2, 1))[0])
    _check_proj(out, False, yq, ys, *w["out"])

    # the next token of every sequence through the few-token and single-token forms
    x1 = torch.randn(1, B, D, generator=g).to(torch.bfloat16).cuda()
    x1q, x1s, u1 = e(1, B, D, dt=f8), e(1, -(-D // 128), B, dt=torch.float32), e(1, B, C)
    y1, y1q, y1s, out1 = e(1, B, Hv * dv), e(1, B, Hv * dv, dt=f8), e(1, -(-Hv * dv // 128), B, dt=torch.float32), e(1, B, D)
    s = s1.clone()
    hb.hyena_quantize_fp8(x1, x1q, x1s)
    hb.hyena_proj_fp8(x1q, x1s, *w["in"], u1)
    q1, k1, v1 = u1[0, :, :Hk * dk], u1[0, :, Hk * dk:2 * Hk * dk], u1[0, :, 2 * Hk * dk:]
    hb.hyena_delta_rule_step(q1, k1, v1, decay[:, :, 0], beta[:, :, 0], y1[0], s, Hk, Hv, l2norm=True)
    hb.hyena_quantize_fp8(y1, y1q, y1s)
    hb.hyena_proj_fp8(y1q, y1s, *w["out"], out1)
    torch.cuda.synchronize()
    hb.hyena_kernel_status()
    _check_proj(u1, False, x1q, x1s, *w["in"])
    ro, rs = dr.delta_rule(_np(q1)[:, :, None], _np(k1)[:, :, None], _np(v1)[:, :, None], _np(decay[:, :, :1]),
                           _np(beta[:, :, :1]), Hk, Hv, _np(s1), l2norm=True)
    assert np.linalg.norm(_np(y1[0]) - ro[:, :, 0]) <= (2.0 ** -8 + 1e-5) * np.linalg.norm(ro)
    assert np.linalg.norm(_np(s) - rs) <= 1e-6 * np.linalg.norm(rs)
    _check_proj(out1, False, y1q, y1s, *w["out"])
