"""GPU: the 8-bit projection's stores at the edges of its tiles: columns cut inside
a box, a half of the columns wholly behind N, the second CTA of a pair wholly
behind M, a row tile that ends in another batch row; every output compared, and
the memory on both sides of the output unchanged.  Tolerances as in the
projection's other tests."""
import pytest

from fft_long_convolution_02_b200 import binding as hb
from test_gpu_fp8 import _check_proj, _cuda, _operands  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu

EDGES = [
    # B, L, K, N
    (1, 128 * 47, 400, 1100),      # pairs of CTAs: an odd number of row tiles, 1100 = 4 x 256 + 76
    (3, 128 * 15, 272, 1033),      # 45 row tiles over three batch rows, an odd N
    (1, 128 * 75, 128, 384),       # the last tile's second half of columns behind N
    (2, 128 * 40, 48, 520),        # pairs, 8 columns in the last tile
    (4, 128 * 6, 400, 600),        # 128-wide tiles
    (1, 128, 144, 33),             # 64-wide tiles: one and a half columns' boxes
    (1, 256, 784, 65),
    (5, 24, 272, 100),             # rows of a tile from several batch rows
    (1, 128 * 47 + 8, 272, 1096),  # rows that end inside a tile: stored one by one where channels come first
]


@pytest.mark.parametrize("B,L,K,N", EDGES)
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_proj_edges(B, L, K, N, first, bias):
    import torch
    xq, xs, wq, ws, b = _operands(B, L, K, N, 3 * L + N)
    buf = torch.full((B * N * L + 4096,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = buf[2048:-2048].view((B, N, L) if first else (B, L, N))
    hb.hyena_proj_fp8(xq, xs, wq, ws, b if bias else None, out, channels_first=first)
    torch.cuda.synchronize()
    hb.hyena_kernel_status()
    assert (buf[:2048] == 9.0).all() and (buf[-2048:] == 9.0).all()
    _check_proj(out, first, xq, xs, wq, ws, b if bias else None)
