"""GPU: the bounded waits of the 8-bit projection.  With no products issued every
role's wait runs out (2 ms); with a warp's staged part kept back, the warp that
stores the half gives up.  The timeout has to reach the status word, every
output has to be NaN and nothing beside them written, and the next call as
ever.  Nothing faults, traps or hangs."""
import pytest

from fft_long_convolution_02_b200 import binding as hb
from test_gpu_fp8 import _check_proj, _cuda, _operands  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu

# 64- and 128-wide tiles, pairs of CTAs (an odd number of row tiles, columns behind N), several tiles a CTA
SHAPES = [(1, 384, 272, 72), (2, 2560, 128, 520), (1, 128 * 47, 400, 1096), (3, 128 * 40, 144, 2304)]


def _run(B, L, K, N, first, hold, seed):
    import torch
    ops = _operands(B, L, K, N, seed)
    buf = torch.full((B * N * L + 128,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = buf[64:-64].view((B, N, L) if first else (B, L, N))
    hb.hyena_kernel_status()                                      # start from a clear record
    hb.hyena_debug_proj_fp8(*ops, out, 2_000_000, hold, channels_first=first)
    torch.cuda.synchronize()
    assert (buf[:64] == 9.0).all() and (buf[-64:] == 9.0).all()
    return ops, out


@pytest.mark.parametrize("B,L,K,N", SHAPES)
@pytest.mark.parametrize("first,hold", [(False, 1), (True, 1), (True, 2)])
def test_wait_timeout_is_reported(B, L, K, N, first, hold):
    import torch
    ops, out = _run(B, L, K, N, first, hold, 5)
    with pytest.raises(hb.HyenaError) as e:
        hb.hyena_kernel_status()
    assert e.value.status == 8                                    # HYENA_ERR_TIMEOUT
    hb.hyena_kernel_status()                                      # reading cleared it
    assert torch.isnan(out.float()).all()
    hb.hyena_proj_fp8(*ops, out, channels_first=first)
    torch.cuda.synchronize()
    hb.hyena_kernel_status()
    _check_proj(out, first, *ops)


@pytest.mark.parametrize("first,hold", [(False, 0), (True, 0), (False, 2)])
def test_hook_that_withholds_nothing_is_the_call(first, hold):
    """A staged part is only handed over in the channels-first store."""
    import torch
    ops, out = _run(2, 2560, 128, 520, first, hold, 6)
    hb.hyena_kernel_status()
    want = torch.empty_like(out)
    hb.hyena_proj_fp8(*ops, want, channels_first=first)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
