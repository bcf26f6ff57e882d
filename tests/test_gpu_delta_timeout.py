"""GPU: the bounded waits of the delta rule's scans.  The test hook never frees
one chunk's stage, so the loading warps' wait for it and the scanning warps'
wait for the chunk that would follow run out (2 ms).  The timeout has to reach
the status word, the outputs from that chunk on and the state have to be NaN,
those before it right, and the next call as ever.  Nothing faults, traps or
hangs."""
import pytest

from fft_long_convolution_02_b200 import binding as hb
from test_gpu_delta_rule import Case, _cuda  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu

# narrow scans, 64 and 128 channels a CTA (of which the last has fewer)
SHAPES = [(1, 400, 1, 2, 64, 64), (1, 390, 1, 1, 128, 40), (40, 270, 2, 4, 64, 64), (19, 270, 2, 4, 128, 120)]


@pytest.mark.parametrize("hold", [0, 1])
@pytest.mark.parametrize("layout", ["first", "last"])
@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv", SHAPES)
def test_scan_wait_timeout_is_reported(B, L, Hk, Hv, dk, dv, layout, hold):
    import torch
    c = Case(B, L, Hk, Hv, dk, dv, layout=layout)
    hb.hyena_kernel_status()                                      # start from a clear record
    want, state = c.run()
    o, s1, ws = c.out(fill=0.0), torch.zeros_like(c.s0), c.workspace()
    hb.hyena_debug_delta_rule(c.q, c.k, c.v, c.g, c.beta, o, Hk, Hv, c.s0, s1, ws, 2_000_000, hold, l2norm=True)
    torch.cuda.synchronize()
    with pytest.raises(hb.HyenaError) as e:
        hb.hyena_kernel_status()
    assert e.value.status == 8                                    # HYENA_ERR_TIMEOUT
    hb.hyena_kernel_status()                                      # reading cleared it
    at = 64 * (hold + 2)
    assert torch.equal(o[:, :, :at], want[:, :, :at])
    assert torch.isnan(o[:, :, at:].float()).all() and torch.isnan(s1).all()
    o2, s2 = c.run()
    assert torch.equal(o2, want) and torch.equal(s2, state)


def test_outputs_without_a_state_are_marked_too():
    """No state_out, an output inside a wider buffer: NaN in the call's own places only."""
    import torch
    c = Case(1, 200, 1, 1, 64, 48)
    wide = torch.full((1, 50, 220), 7.0, dtype=torch.bfloat16, device="cuda")
    o = wide[:, 1:49, 10:210]
    hb.hyena_debug_delta_rule(c.q, c.k, c.v, c.g, c.beta, o, 1, 1, c.s0, None, c.workspace(), 2_000_000, 0, l2norm=True)
    torch.cuda.synchronize()
    with pytest.raises(hb.HyenaError):
        hb.hyena_kernel_status()
    assert torch.isnan(o[:, :, 128:].float()).all() and torch.isfinite(o[:, :, :128].float()).all()
    wide[:, 1:49, 10:210] = 7.0
    assert (wide == 7.0).all()


def test_hook_without_a_held_stage_is_the_call():
    import torch
    c = Case(2, 300, 1, 2, 64, 64)
    want, state = c.run()
    o, s1 = c.out(), torch.empty_like(state)
    hb.hyena_debug_delta_rule(c.q, c.k, c.v, c.g, c.beta, o, 1, 2, c.s0, s1, c.workspace(), 2_000_000_000, l2norm=True)
    torch.cuda.synchronize()
    hb.hyena_kernel_status()
    assert torch.equal(o, want) and torch.equal(s1, state)
