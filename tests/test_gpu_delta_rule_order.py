"""GPU: the delta rule behind kernels that make its operands on the same stream.
The scan is launched early (programmatic stream serialisation); everything that
it reads, the lengths among it, has to be what the kernels before it left."""
import pytest

from fft_long_convolution_02_b200 import binding as hb
from test_gpu_delta_rule import Case, _cuda  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["first", "last"])
@pytest.mark.parametrize("captured", [False, True])
def test_lengths_gates_and_state_made_just_before(layout, captured):
    """Lengths, gates, values and the state are written by kernels right before the call, another time with other values;
    a replayed graph does the same."""
    import torch
    B, L = 4, 300
    want, cases = [], [Case(B, L, 1, 2, 64, 64, layout=layout, seed=s, lengths=n) for s, n in ((1, [300, 7, 0, 129]), (2, [1, 300, 64, 0]))]
    for c in cases:
        want.append(c.run(c.out(fill=0.0)))
    live = Case(B, L, 1, 2, 64, 64, layout=layout, lengths=[0] * B)
    o, s1, ws = live.out(fill=0.0), torch.empty_like(live.s0), live.workspace()

    def step():
        hb.hyena_delta_rule(live.q, live.k, live.v, live.g, live.beta, o, 1, 2, live.s0, s1, live.lengths, l2norm=True,
                            workspace=ws)

    source = [torch.empty_like(getattr(live, n)) for n in ("q", "k", "v", "g", "beta", "s0", "lengths")]

    def take():
        o.zero_()
        for n, t in zip(("q", "k", "v", "g", "beta", "s0", "lengths"), source):
            getattr(live, n).copy_(t)
        step()

    if captured:
        take()
        torch.cuda.synchronize()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            take()
    for i in (0, 1, 0):
        for n, t in zip(("q", "k", "v", "g", "beta", "s0", "lengths"), source):
            t.copy_(getattr(cases[i], n))
        graph.replay() if captured else take()
        torch.cuda.synchronize()
        hb.hyena_kernel_status()
        assert torch.equal(o, want[i][0]) and torch.equal(s1, want[i][1])
