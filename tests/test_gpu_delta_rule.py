"""GPU: the gated delta rule (whole sequences and the single-token step)
against the float64 oracle.

Tolerances, on 2-norms.  The state is fp32 throughout: a token's contraction
over dk products of fp32 numbers rounds by about sqrt(dk) 2^-24 of its result,
and the roundings of L tokens are independent and do not grow (decay <= 1,
beta |k|^2 <= 2), so the state is within STATE(dk, L) = 2 sqrt(dk (L + 16)) 2^-24
of the oracle's.  Products of the state formed from two 11-bit parts round by
2^-22 an element at most, less than a contraction's own rounding for dk >= 16.
An output is rounded once to its type (half a step: 2^-8 for bf16); where its
operands go through the tensor cores as fp16 (state, writes, scores), each of
the three adds at most 2^-11."""
import numpy as np
import pytest

from fft_long_convolution_02_b200 import binding as hb
from oracle import delta_rule as dr

pytestmark = pytest.mark.gpu


def STATE(dk, L):
    return 2.0 * np.sqrt(max(dk, 16) * (L + 16.0)) * 2.0 ** -24


def OUT(dtype, dk, L):
    return STATE(dk, L) + (2.0 ** -8 + 3 * 2.0 ** -11 if dtype == "bf16" else 0.0)


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


def _rel(a, b):
    return np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-300)


class Case:
    def __init__(self, B, L, Hk, Hv, dk, dv, dtype="bf16", layout="first", l2norm=True, state=True, lengths=None,
                 decay=0.1, seed=0, gates=True, pad=0):
        import torch
        self.__dict__.update(B=B, L=L, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype, l2norm=l2norm)
        g = torch.Generator().manual_seed(seed + 1000 * L + dk + 7 * dv)
        C = 2 * Hk * dk + Hv * dv
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        u = torch.randn(B, C, L, generator=g)
        if not l2norm:
            u[:, :2 * Hk * dk] *= dk ** -0.5
        if layout == "first":
            u = torch.cat([u, torch.zeros(B, C, pad)], 2).to(dt).cuda()[:, :, :L]
        else:
            u = torch.cat([u.transpose(1, 2), torch.zeros(B, L, pad)], 2).to(dt).cuda()[:, :, :C].transpose(1, 2)
        self.q, self.k, self.v = u[:, :Hk * dk], u[:, Hk * dk:2 * Hk * dk], u[:, 2 * Hk * dk:]
        self.g = (-decay * torch.rand(B, Hv, L, generator=g) * 4).cuda() if gates else None
        self.beta = torch.sigmoid(torch.randn(B, Hv, L, generator=g)).cuda() if gates else None
        self.s0 = torch.randn(B, Hv, dk, dv, generator=g).mul_(0.5).cuda() if state else None
        self.lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
        self.layout = layout

    def out(self, fill=float("nan")):
        import torch
        shape = (self.B, self.Hv * self.dv, self.L)
        if self.layout == "first":
            return torch.full(shape, fill, dtype=self.q.dtype, device="cuda")
        return torch.full((shape[0], shape[2], shape[1]), fill, dtype=self.q.dtype, device="cuda").transpose(1, 2)

    def workspace(self):
        import torch
        n = hb.hyena_delta_rule_workspace_bytes(self.B, self.L, self.Hk, self.Hv, self.dk, self.dv, self.q.dtype)
        return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None

    def run(self, o=None, stream=None, **kw):
        import torch
        o = self.out() if o is None else o
        s1 = torch.full((self.B, self.Hv, self.dk, self.dv), float("nan"), device="cuda")
        a = dict(state_in=self.s0, state_out=s1, lengths=self.lengths, l2norm=self.l2norm, workspace=self.workspace())
        a.update(kw)
        hb.hyena_delta_rule(self.q, self.k, self.v, self.g, self.beta, o, self.Hk, self.Hv, stream=stream, **a)
        torch.cuda.synchronize()
        hb.hyena_kernel_status()
        return o, a["state_out"]

    def oracle(self, **kw):
        n = lambda t: None if t is None else _np(t)
        return dr.delta_rule(_np(self.q), _np(self.k), _np(self.v), n(self.g), n(self.beta), self.Hk, self.Hv,
                             n(self.s0), None if self.lengths is None else self.lengths.cpu().numpy(),
                             l2norm=self.l2norm, **kw)

    def check(self, o, s1, ref=None):
        ro, rs = ref or self.oracle()
        got, live = _np(o), np.isfinite(ro)
        if live.any():
            assert _rel(got[live], ro[live]) <= OUT(self.dtype, self.dk, self.L)
            for b in range(self.B):                       # row by row too: a bad row does not hide
                m = live[b]
                if m.any():
                    assert _rel(got[b][m], ro[b][m]) <= 2 * OUT(self.dtype, self.dk, self.L)
        if s1 is not None:
            assert _rel(_np(s1), rs) <= STATE(self.dk, self.L)
        return got, live


SHAPES = [
    # B, L, Hk, Hv, dk, dv
    (1, 1, 1, 1, 16, 16), (2, 2, 1, 2, 64, 64), (1, 17, 2, 2, 64, 64), (2, 63, 1, 1, 128, 128), (1, 64, 2, 4, 128, 128),
    (2, 65, 1, 1, 128, 64), (1, 128, 3, 3, 64, 96), (1, 200, 1, 3, 100, 40), (2, 129, 2, 2, 40, 24), (1, 300, 1, 1, 128, 160),
    (1, 96, 1, 2, 1, 1), (1, 70, 1, 1, 7, 256), (1, 512, 2, 2, 128, 128),
    # heads enough for the wider scans: one, then two warps a scheduler
    (20, 130, 2, 4, 64, 64), (10, 200, 2, 4, 128, 128), (10, 70, 4, 4, 100, 120),
    (40, 70, 2, 4, 64, 64), (19, 130, 2, 4, 128, 128), (40, 65, 4, 4, 100, 120),
]


@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv", SHAPES)
@pytest.mark.parametrize("layout", ["first", "last"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences(B, L, Hk, Hv, dk, dv, layout, dtype):
    c = Case(B, L, Hk, Hv, dk, dv, dtype, layout, l2norm=(L % 2 == 0))
    c.check(*c.run())


@pytest.mark.parametrize("layout", ["first", "last"])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_strided_views(layout, pad):
    """Rows of the projected stream that do not start on 16 bytes, and padded ones that do."""
    c = Case(2, 136, 1, 2, 64, 64, layout=layout, pad=pad)
    c.check(*c.run())


def test_sliced_time_and_offset_output():
    """Every other position of a stream, and an output inside a wider buffer that keeps its surroundings."""
    import torch
    c = Case(1, 160, 1, 1, 64, 64)
    q, k, v = c.q, c.k, c.v
    c.q, c.k, c.v = q[:, :, ::2], k[:, :, ::2], v[:, :, ::2]
    c.g, c.beta, c.L = c.g[:, :, ::2], c.beta[:, :, ::2], 80
    wide = torch.full((1, 66, 90), 7.0, dtype=torch.bfloat16, device="cuda")
    o = wide[:, 1:65, 5:85]
    c.check(*c.run(o))
    wide[:, 1:65, 5:85] = 7.0
    assert (wide == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["first", "last"])
def test_lengths(dtype, layout):
    """A padded batch: NaN and infinities behind a row's end change nothing, and
    its outputs there stay what they were; lengths outside [0, L] are clamped."""
    import torch
    L = 200
    lengths = [0, 1, 63, 64, 65, 200, 199, 500, -3]
    c = Case(len(lengths), L, 1, 2, 64, 64, dtype, layout, lengths=lengths, l2norm=False)
    ref = c.oracle()
    for b, n in enumerate(lengths):
        n = min(max(n, 0), L)
        for t, bad in ((c.q, float("nan")), (c.k, float("inf")), (c.v, float("nan")), (c.g, float("nan")),
                       (c.beta, float("-inf"))):
            t[b, :, n:] = bad
    o, s1 = c.run(c.out(fill=3.0))
    got, live = c.check(o, s1, ref)
    assert (got[~live] == 3.0).all()
    assert torch.equal(s1[0], c.s0[0]) and torch.equal(s1[8], c.s0[8])      # length 0: the state before


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [40, 150])
def test_without_state_gates_or_final_state(dtype, L):
    c = Case(2, L, 1, 1, 64, 64, dtype, state=False, gates=False)
    c.check(*c.run())
    o, _ = c.run(state_out=None)
    c.check(o, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_state_in_place(dtype):
    c = Case(2, 130, 1, 2, 64, 64, dtype)
    ref = c.oracle()
    s = c.s0.clone()
    o, _ = c.run(state_in=s, state_out=s)
    c.check(o, s, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", [0.0, 5.0, 60.0])
def test_decays(dtype, decay):
    """No decay, decays that empty the state within a few tokens, and ones that underflow."""
    c = Case(1, 192, 1, 2, 64, 64, dtype, decay=decay)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_growing_gates(dtype):
    """Gates of either sign: a chunk's products may grow the state too (up to e^3 here)."""
    c = Case(1, 130, 1, 2, 64, 64, dtype)
    c.g[:] = (c.g + 0.2) * 0.25
    c.g[:, :, 20:40] = 0.15
    c.check(*c.run())


@pytest.mark.parametrize("Hk,Hv", [(2, 4), (1, 3), (1, 4), (1, 8), (2, 10)])
@pytest.mark.parametrize("layout", ["first", "last"])
def test_shared_key_heads_of_many_chunks(Hk, Hv, layout):
    """Chunks enough for the value heads of a key head to be taken together, by twos, threes and fours."""
    B, L = 12, 64 * 16 * 5 + 9
    c = Case(B, L, Hk, Hv, 16, 16, layout=layout, lengths=[L, 100] + [int(L * b / B) for b in range(2, B)])
    import torch
    o, s1 = c.run()
    d = Case(B, L, Hv, Hv, 16, 16, layout=layout)          # the same with the key heads written out
    r = Hv // Hk
    rep = lambda x: x.reshape(B, Hk, 16, L).repeat_interleave(r, 1).reshape(B, Hv * 16, L)
    d.q, d.k, d.v, d.g, d.beta, d.s0, d.lengths = rep(c.q), rep(c.k), c.v, c.g, c.beta, c.s0, c.lengths
    o2, s2 = d.run()
    for b in range(B):
        n = int(c.lengths[b])
        assert torch.equal(o[b, :, :n], o2[b, :, :n])
    assert torch.equal(s1, s2)
    few = [1]                                              # and against the oracle where that is quick
    ro, rs = dr.delta_rule(*(_np(t[few]) for t in (c.q, c.k, c.v, c.g, c.beta)), Hk, Hv, _np(c.s0[few]), [100], l2norm=True)
    assert _rel(_np(o[1, :, :100]), ro[0, :, :100]) <= OUT("bf16", 16, 100)
    assert _rel(_np(s1[few]), rs) <= STATE(16, 100)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_reset_by_minus_infinity(dtype):
    """g = -inf empties the state: what came before is forgotten exactly, inside a chunk and on its border."""
    import torch
    c = Case(1, 200, 1, 1, 64, 64, dtype)
    for t in (0, 5, 64, 100, 101, 199):
        c.g[:, :, t] = float("-inf")
    o, s1 = c.run()
    c.check(o, s1)
    c.v[:, :, :100] += 1.0                                # the far past
    o2, s2 = c.run()
    assert torch.equal(o[:, :, 101:199], o2[:, :, 101:199]) and torch.equal(s1, s2)


def test_strong_reset_then_weak_decay():
    """Decays that differ by orders inside a chunk: their partial sums must not
    lose the weak ones behind the strong."""
    c = Case(1, 192, 1, 1, 64, 64, decay=1e-3)
    c.g[:, :, 3::50] = -3000.0
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_keys(dtype):
    """One key for all tokens with full write strength: the triangular system is
    as far from the identity as it gets (all its entries are 1)."""
    import torch
    c = Case(1, 160, 1, 1, 64, 64, dtype, gates=False)
    c.k[:] = c.k[:, :, :1].clone()
    c.beta = torch.ones(1, 1, 160, device="cuda")
    c.check(*c.run())


@pytest.mark.parametrize("mag", [1e-12, 1e4, 1e15])
def test_magnitudes(mag):
    """Values far from 1: the rule is linear in v and S, so nothing depends on their size."""
    c = Case(1, 130, 1, 1, 64, 64, state=True)
    c.v *= mag
    c.s0 *= mag
    c.check(*c.run())


def test_small_and_large_columns_together():
    """Value channels of very unequal size keep their own relative error."""
    c = Case(1, 130, 1, 1, 64, 64, state=False)
    c.v[:, ::2] *= 1e6
    o, s1 = c.run()
    ro, rs = c.oracle()
    for part in (np.s_[:, 0::2], np.s_[:, 1::2]):
        assert _rel(_np(o)[part], ro[part]) <= OUT("bf16", 64, 130)
    for part in (np.s_[..., 0::2], np.s_[..., 1::2]):
        assert _rel(_np(s1)[part], rs[part]) <= STATE(64, 130)


def test_unnormalised_keys_of_unequal_size():
    """Keys from 1e-3 to 1e3 with write strengths that keep beta |k|^2 <= 1."""
    import torch
    c = Case(1, 130, 1, 1, 64, 64, l2norm=False)
    s = torch.logspace(-3, 3, 130, device="cuda")[torch.randperm(130, device="cuda", generator=torch.Generator("cuda").manual_seed(3))]
    c.k.copy_((c.k.float() * s).to(c.k.dtype))
    n2 = (c.k.float() ** 2).sum(1, keepdim=True)
    c.beta = (c.beta / n2.clamp(min=1.0)).contiguous()
    c.check(*c.run())


def test_scale():
    c = Case(1, 70, 1, 1, 64, 64, "f32")
    o, s1 = c.run(scale=0.25)
    c.check(o, s1, c.oracle(scale=0.25))


def test_zero_vectors_with_norms():
    """Zero queries and keys under the norm stay zero."""
    c = Case(1, 70, 1, 1, 64, 64)
    c.q[:, :, 10:20] = 0
    c.k[:, :, 15:30] = 0
    c.check(*c.run())


@pytest.mark.parametrize("dtype,layout,L", [("bf16", "first", 1000), ("bf16", "last", 2048), ("f32", "first", 1000)])
def test_split_sequence_carries_the_state(dtype, layout, L):
    """A sequence in three calls (uneven pieces) and its last token by the step,
    against the whole in one call: the state within twice its own error."""
    import torch
    c = Case(2, L, 2, 4, 64, 64, dtype, layout, decay=0.01)
    o, s1 = c.run()
    cuts = [0, 100, 613, L - 1]
    s = c.s0.clone()
    parts = []
    for a, b in zip(cuts, cuts[1:]):
        op = torch.empty_like(o[:, :, a:b])
        n = hb.hyena_delta_rule_workspace_bytes(2, b - a, 2, 4, 64, 64, c.q.dtype)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        hb.hyena_delta_rule(c.q[:, :, a:b], c.k[:, :, a:b], c.v[:, :, a:b], c.g[:, :, a:b], c.beta[:, :, a:b], op, 2, 4,
                            s, s, l2norm=True, workspace=ws)
        parts.append(op)
    last = torch.empty(2, 4 * 64, dtype=o.dtype, device="cuda")
    hb.hyena_delta_rule_step(c.q[:, :, -1], c.k[:, :, -1], c.v[:, :, -1], c.g[:, :, -1], c.beta[:, :, -1], last, s, 2, 4,
                             l2norm=True)
    torch.cuda.synchronize()
    hb.hyena_kernel_status()
    whole = torch.cat(parts + [last[:, :, None]], 2)
    assert _rel(_np(whole), _np(o)) <= 2 * OUT(dtype, 64, L)
    assert _rel(_np(s), _np(s1)) <= 2 * STATE(64, L)


def test_same_results_twice_and_on_another_stream():
    """No order of atomics in the results; another stream with its own workspace at the same time."""
    import torch
    c = Case(2, 700, 2, 2, 128, 128, state=False)
    o, s1 = c.run()
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for st in streams:
        oo, ss, ws = c.out(), torch.empty_like(s1), c.workspace()
        torch.cuda.synchronize()
        hb.hyena_delta_rule(c.q, c.k, c.v, c.g, c.beta, oo, 2, 2, None, ss, l2norm=True, workspace=ws, stream=st)
        outs.append((oo, ss, ws))
    torch.cuda.synchronize()
    for oo, ss, _ in outs:
        assert torch.equal(oo, o) and torch.equal(ss, s1)


def test_captured_and_replayed():
    import torch
    c = Case(2, 300, 1, 2, 64, 64)
    o, s1 = c.run()
    oo, ss, ws = c.out(), torch.empty_like(s1), c.workspace()
    pool, po = c.s0.clone(), torch.empty(2, 128, dtype=o.dtype, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        hb.hyena_delta_rule(c.q, c.k, c.v, c.g, c.beta, oo, 1, 2, c.s0, ss, l2norm=True, workspace=ws)
        hb.hyena_delta_rule_step(c.q[:, :, 0], c.k[:, :, 0], c.v[:, :, 0], c.g[:, :, 0], c.beta[:, :, 0], po, pool, 1, 2,
                                 l2norm=True)
    for _ in range(2):
        oo.fill_(0)
        ss.fill_(0)
        pool.copy_(c.s0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(oo, o) and torch.equal(ss, s1)
        assert _rel(_np(po), _np(o[:, :, 0])) <= 2 * OUT("bf16", 64, 1)


def test_long_sequence_sampled():
    """L = 4097 in two heads, every output against the oracle."""
    c = Case(1, 4097, 1, 2, 64, 32, decay=0.02)
    c.check(*c.run())


@pytest.mark.parametrize("dtype,L", [("bf16", 80), ("bf16", 9), ("f32", 20)])
def test_broadcast_operands(dtype, L):
    """Keys shared by the batch, one query for all positions and one gate for all heads, as views of stride 0."""
    c = Case(3, L, 2, 2, 64, 64, dtype)
    c.k = c.k[:1].expand(3, -1, -1)
    c.q = c.q[:, :, :1].expand(-1, -1, L)
    c.g, c.beta = c.g[:, :1].expand(-1, 2, -1), c.beta[:1].expand(3, -1, -1)
    c.check(*c.run())


@pytest.mark.parametrize("L", [70, 5])
def test_offsets_beyond_32_bits(L):
    """Batch rows more than 2^31 elements apart, of the stream and of the output."""
    import torch
    c = Case(2, L, 1, 1, 64, 64)
    far = (1 << 31) + 64
    buf = torch.empty(far + 4 * 64 * L, dtype=torch.bfloat16, device="cuda")
    views = [torch.as_strided(buf, (2, 64, L), (far, L, 1), 64 * L * i) for i in range(4)]
    for v, t in zip(views, (c.q, c.k, c.v)):
        v.copy_(t)
    o = torch.full((far + 64 * L,), 0, dtype=torch.bfloat16, device="cuda")
    c.q, c.k, c.v = views[:3]
    o2 = torch.as_strided(o, (2, 64, L), (far, L, 1))
    c.check(*c.run(o2))
    assert int(torch.count_nonzero(o[64 * L:far])) == 0


def test_step_slot_beyond_32_bits():
    """A pool of more than 2^31 floats: the last state is the one that changes."""
    import torch
    n = (1 << 31) // (64 * 64) + 3
    c = Case(1, 1, 1, 1, 64, 64, "bf16", "last")
    ro, rs = c.oracle()
    pool = torch.empty(n, 1, 64, 64, device="cuda")
    pool[-1] = c.s0[0]
    pool[2] = 4.0                                         # where the index would land, cut to 32 bits
    o = torch.empty(1, 64, dtype=torch.bfloat16, device="cuda")
    hb.hyena_delta_rule_step(c.q[:, :, 0], c.k[:, :, 0], c.v[:, :, 0], c.g[:, :, 0], c.beta[:, :, 0], o, pool, 1, 1,
                             torch.tensor([n - 1], dtype=torch.int32, device="cuda"), l2norm=True)
    torch.cuda.synchronize()
    hb.hyena_kernel_status()
    assert _rel(_np(o), ro[:, :, 0]) <= OUT("bf16", 64, 1)
    assert _rel(_np(pool[-1]), rs[0]) <= STATE(64, 1) and (pool[2] == 4.0).all()


# ------------------------------------------------------------------------ step
@pytest.mark.parametrize("B,Hk,Hv,dk,dv", [(1, 1, 1, 128, 128), (3, 2, 4, 64, 96), (2, 1, 3, 100, 40), (5, 1, 1, 7, 33),
                                           (2, 2, 2, 1, 1), (1, 1, 1, 128, 256), (70, 1, 2, 64, 64), (160, 2, 2, 128, 100)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("l2norm", [True, False])
def test_step(B, Hk, Hv, dk, dv, dtype, l2norm):
    import torch
    c = Case(B, 3, Hk, Hv, dk, dv, dtype, "last", l2norm=l2norm)
    ro, rs = c.oracle()
    s = c.s0.clone()
    for t in range(3):
        o = torch.full((B, Hv * dv), float("nan"), dtype=c.q.dtype, device="cuda")
        hb.hyena_delta_rule_step(c.q[:, :, t], c.k[:, :, t], c.v[:, :, t], c.g[:, :, t], c.beta[:, :, t], o, s, Hk, Hv,
                                 l2norm=l2norm)
        torch.cuda.synchronize()
        assert _rel(_np(o), ro[:, :, t]) <= OUT(dtype, dk, 3)
    hb.hyena_kernel_status()
    assert _rel(_np(s), rs) <= STATE(dk, 3)


def test_step_slots():
    """States in a pool: only the named ones change, padding rows are left alone."""
    import torch
    B = 6
    c = Case(B, 1, 1, 2, 64, 64, "bf16", "last")
    ro, rs = c.oracle()
    slots = [9, 0, -1, 4, 7, -1]
    pool = torch.randn(11, 2, 64, 64, device="cuda")
    for b, s in enumerate(slots):
        if s >= 0:
            pool[s] = c.s0[b]
    before = pool.clone()
    o = torch.full((B, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    hb.hyena_delta_rule_step(c.q[:, :, 0], c.k[:, :, 0], c.v[:, :, 0], c.g[:, :, 0], c.beta[:, :, 0], o, pool, 1, 2,
                             torch.tensor(slots, dtype=torch.int32, device="cuda"), l2norm=True)
    torch.cuda.synchronize()
    hb.hyena_kernel_status()
    for b, s in enumerate(slots):
        if s < 0:
            assert (o[b] == 5.0).all()
        else:
            assert _rel(_np(o[b]), ro[b, :, 0]) <= OUT("bf16", 64, 1)
            assert _rel(_np(pool[s]), rs[b]) <= STATE(64, 1)
    rest = [i for i in range(11) if i not in slots]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("slots", [[0, 3, 3, 1], [0, 1, 2, 5]])
def test_step_bad_slots_are_reported(slots):
    """A slot named twice, or out of range: that row gets NaN, no state is
    written for it, and the status call says so; the others are as ever."""
    import torch
    c = Case(4, 1, 1, 1, 64, 64, "bf16", "last")
    ro, rs = c.oracle()
    pool = torch.zeros(5, 1, 64, 64, device="cuda")
    good = [b for b, s in enumerate(slots) if s < 5 and s not in slots[:b]]
    for b in good:
        pool[slots[b]] = c.s0[b]
    before = pool.clone()
    o = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    hb.hyena_delta_rule_step(c.q[:, :, 0], c.k[:, :, 0], c.v[:, :, 0], c.g[:, :, 0], c.beta[:, :, 0], o, pool, 1, 1,
                             torch.tensor(slots, dtype=torch.int32, device="cuda"), l2norm=True)
    with pytest.raises(hb.HyenaError) as e:
        hb.hyena_kernel_status()
    assert e.value.status == 1
    hb.hyena_kernel_status()                              # read and cleared
    for b, s in enumerate(slots):
        if b in good:
            assert _rel(_np(o[b]), ro[b, :, 0]) <= OUT("bf16", 64, 1)
            assert _rel(_np(pool[s]), rs[b]) <= STATE(64, 1)
        else:
            assert torch.isnan(o[b]).all()
    rest = [i for i in range(5) if i not in [slots[b] for b in good]]
    assert torch.equal(pool[rest], before[rest])


def test_binding_refuses_wrong_tensors():
    import torch
    c = Case(2, 32, 1, 2, 64, 64)
    o = c.out()
    bad = [dict(q=c.q.cpu()), dict(k=c.k[:, :32]), dict(v=c.v.float()), dict(g=c.g.double()), dict(beta=c.beta[:, :1]),
           dict(o=o[:, :, :16])]
    for b in bad:
        a = dict(q=c.q, k=c.k, v=c.v, g=c.g, beta=c.beta, o=o)
        a.update(b)
        with pytest.raises((ValueError, TypeError)):
            hb.hyena_delta_rule(*a.values(), 1, 2, workspace=c.workspace())
    for kw in (dict(state_in=c.s0[:1]), dict(state_out=c.s0.half()), dict(state_in=c.s0.transpose(2, 3)),
               dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            hb.hyena_delta_rule(c.q, c.k, c.v, c.g, c.beta, o, 1, 2, workspace=c.workspace(), **kw)
    with pytest.raises(ValueError):
        hb.hyena_delta_rule(c.q, c.k, c.v, c.g, c.beta, o, 3, 2, workspace=c.workspace())
