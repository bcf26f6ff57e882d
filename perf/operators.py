"""The sequence-mixer and 8-bit projection operators: cases, plain forms, exact values.

Four operators of a layer that mixes tokens by the gated delta rule instead
of a long convolution, and whose projections are 8-bit products:

  delta   hyena_delta_rule       whole sequences, from and to a state
  step    hyena_delta_rule_step  one token a sequence, states updated in place
  quant   hyena_quantize_fp8 (activations, either layout) and
          hyena_quantize_fp8_weight (128 x 128 blocks)
  proj    hyena_proj_fp8         out = x W^T + bias on e4m3 operands with a
          scale for each block of 128

`own` selects the framework's kernels; without it `run` computes the same in
elementary torch operations in fp32 (positions' decays in fp64).
"""
import math

import torch

own = False

EPS = 1e-6        # under the root of the query and key norms
E4M3_MAX = 448.0
CHUNK = 64        # the plain form's chunk


# ----------------------------------------------------------------- cases
def listed():
    return [
        # a prompt's tail of a few tokens for one sequence: latency
        dict(name="delta tail 1x17", op="delta", B=1, L=17, Hk=4, Hv=4, dk=64, dv=64, dtype="bf16", first=True,
             l2norm=True, state=True, ragged=False),
        # the benchmarked width and length (D = 768, L = 8192, B = 4) as six heads of 128, in the layout of the
        # input projection
        dict(name="delta d768 l8k", op="delta", B=4, L=8192, Hk=6, Hv=6, dk=128, dv=128, dtype="bf16", first=True,
             l2norm=True, state=False, ragged=False),
        # a large prefill: many heads, queries and keys shared by two value heads, channels contiguous
        dict(name="delta prefill 16x4096", op="delta", B=16, L=4096, Hk=8, Hv=16, dk=128, dv=128, dtype="bf16",
             first=False, l2norm=True, state=True, ragged=False),
        # a padded batch of unequal prompts at uneven sizes
        dict(name="delta ragged 5x1000", op="delta", B=5, L=1000, Hk=3, Hv=6, dk=64, dv=96, dtype="bf16", first=False,
             l2norm=False, state=True, ragged=True),
        # generation: one sequence, and a large batch whose states lie in a pool
        dict(name="step 1", op="step", B=1, Hk=6, Hv=6, dk=128, dv=128, dtype="bf16", l2norm=True, pool=0),
        dict(name="step 256 of a pool", op="step", B=256, Hk=8, Hv=16, dk=128, dv=128, dtype="bf16", l2norm=True,
             pool=300),
        # activations on their way to the input projection, and the mixer's output on its way to the output projection
        dict(name="quant x d768 l8k", op="quant", what="last", B=4, L=8192, K=768, dtype="bf16"),
        dict(name="quant y uneven", op="quant", what="first", B=3, L=1000, K=2000, dtype="bf16"),
        # the input projection at the benchmarked size, a wide one, an uneven one, and one of a few tokens
        dict(name="proj in d768 l8k", op="proj", B=4, L=8192, K=768, N=2304, first=True, bias=True),
        dict(name="proj wide", op="proj", B=4, L=8192, K=2048, N=4096, first=False, bias=False),
        dict(name="proj uneven", op="proj", B=3, L=333, K=784, N=1000, first=True, bias=True),
        dict(name="proj 4 tokens", op="proj", B=1, L=4, K=2048, N=6144, first=False, bias=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "step", "quant", "proj", "proj"])
    if op == "delta":
        while True:
            c = dict(op=op, B=_log(rng, 1, 32), L=_log(rng, 1, 8192), Hk=rng.choice([1, 2, 3, 4, 6, 8, 16]), Hv=0,
                     dk=rng.choice([16, 40, 64, 64, 100, 128, 128, 128]), dv=rng.choice([24, 64, 96, 128, 128, 128, 160]),
                     dtype=rng.choice(["bf16"] * 5 + ["f32"]), first=rng.random() < 0.5, l2norm=rng.random() < 0.7,
                     state=rng.random() < 0.6, ragged=rng.random() < 0.4)
            c["Hv"] = c["Hk"] * rng.choice([1, 1, 2, 4])
            n = c["B"] * c["L"] * c["Hv"]
            # the largest listed case bounds the size; fp32 storage is for short sequences
            if n * c["dk"] * c["dv"] <= 16 * 4096 * 16 * 128 * 128 and not (c["dtype"] == "f32" and c["L"] > 2048):
                return c
    if op == "step":
        B = _log(rng, 1, 256)
        Hk = rng.choice([1, 2, 4, 6, 8])
        return dict(op=op, B=B, Hk=Hk, Hv=Hk * rng.choice([1, 2]), dk=rng.choice([16, 64, 100, 128, 128]),
                    dv=rng.choice([24, 64, 96, 128, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    l2norm=rng.random() < 0.7, pool=rng.choice([0, B + 3, 300]))
    if op == "quant":
        what = rng.choice(["last", "first", "weight"])
        L = _log(rng, 1, 8192)
        return dict(op=op, what=what, B=1 if what == "weight" else _log(rng, 1, 4), L=L, K=16 * _log(rng, 1, 128),
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    B, L = _log(rng, 1, 4), _log(rng, 1, 8192)
    return dict(op=op, B=B, L=L, K=16 * _log(rng, 1, 128), N=_log(rng, 16, 4096), first=rng.random() < 0.5,
                bias=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _storage(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gates(g, case, *shape_front):
    """Log decays and write strengths as a layer makes them: a rate a head in [1, 16] times a softplus, and a sigmoid.
    The head is the last axis here."""
    Hv = case["Hv"]
    rate = 1.0 + 15.0 * _rand(g, Hv)
    step = 0.001 * (100.0 ** _rand(g, Hv))                      # softplus(bias) between 0.001 and 0.1
    bias = torch.log(torch.expm1(step))
    decay = -rate * torch.nn.functional.softplus(_randn(g, *shape_front, Hv) + bias)
    return decay, torch.sigmoid(_randn(g, *shape_front, Hv))


def _scale(amax):
    # a true division: dividing by a number multiplies by its reciprocal on the device
    return (amax / torch.full_like(amax, E4M3_MAX)).clamp(min=torch.finfo(torch.float32).tiny)


def _to_fp8_rows(x):
    """[B, L, K] fp32 to e4m3 with a scale a row and block of 128: values [B, L, K], scales [B, K / 128, L]."""
    B, L, K = x.shape
    n = -(-K // 128)
    p = torch.nn.functional.pad(x, (0, n * 128 - K)).view(B, L, n, 128)
    s = _scale(p.abs().amax(-1))
    q = (p / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(B, L, n * 128)[..., :K].contiguous(), s.transpose(1, 2).contiguous()


def _to_fp8_weight(w):
    """[N, K] fp32 to e4m3 with a scale a block of 128 x 128."""
    N, K = w.shape
    a, b = -(-N // 128), -(-K // 128)
    p = torch.nn.functional.pad(w, (0, b * 128 - K, 0, a * 128 - N)).view(a, 128, b, 128)
    s = _scale(p.abs().amax((1, 3)))
    q = (p / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(a * 128, b * 128)[:N, :K].contiguous(), s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "delta":
        B, L, Hk, Hv, dk, dv = (case[k] for k in ("B", "L", "Hk", "Hv", "dk", "dv"))
        dt = _storage(case)
        C = 2 * Hk * dk + Hv * dv
        # the projected stream holds q, k and v as blocks of channels; [B, C, L] views of it whichever way it lies
        scale = 1.0 if case["l2norm"] else dk ** -0.5          # keys of about unit length reach the rule
        u = (_randn(g, B, C, L) if case["first"] else _randn(g, B, L, C)).mul_(scale).to(dt)
        u = u if case["first"] else u.transpose(1, 2)
        st["q"], st["k"], st["v"] = u[:, : Hk * dk], u[:, Hk * dk: 2 * Hk * dk], u[:, 2 * Hk * dk:]
        decay, beta = _gates(g, case, B, L)
        if case["first"]:
            st["g"], st["beta"] = decay.transpose(1, 2).contiguous(), beta.transpose(1, 2).contiguous()
        else:
            st["g"], st["beta"] = decay.transpose(1, 2), beta.transpose(1, 2)
        st["state_in"] = _randn(g, B, Hv, dk, dv) * 0.3 if case["state"] else None
        st["lengths"] = None
        if case["ragged"]:
            n = (_rand(g, B) * (L + 1)).to(torch.int32).clamp(max=L)
            n[0] = L
            st["lengths"] = n
        o = torch.zeros((B, Hv * dv, L) if case["first"] else (B, L, Hv * dv), dtype=dt, device="cuda")
        st["o"] = o if case["first"] else o.transpose(1, 2)
        st["state_out"] = torch.empty(B, Hv, dk, dv, device="cuda")
    elif op == "step":
        B, Hk, Hv, dk, dv = (case[k] for k in ("B", "Hk", "Hv", "dk", "dv"))
        dt = _storage(case)
        C = 2 * Hk * dk + Hv * dv
        scale = 1.0 if case["l2norm"] else dk ** -0.5
        u = _randn(g, B, C).mul_(scale).to(dt)
        st["q"], st["k"], st["v"] = u[:, : Hk * dk], u[:, Hk * dk: 2 * Hk * dk], u[:, 2 * Hk * dk:]
        st["g"], st["beta"] = _gates(g, case, B)
        n = max(case["pool"], B)
        st["pool"] = _randn(g, n, Hv, dk, dv) * 0.3
        st["slots"] = torch.randperm(n, generator=g, device="cuda")[:B].to(torch.int32) if case["pool"] else None
        st["o"] = torch.zeros(B, Hv * dv, dtype=dt, device="cuda")
    elif op == "quant":
        B, L, K = case["B"], case["L"], case["K"]
        n = -(-K // 128)
        dt = _storage(case)
        if case["what"] == "weight":
            st["x"] = (_randn(g, L, K) * K ** -0.5).to(dt)
            st["xq"] = torch.empty(L, K, dtype=torch.float8_e4m3fn, device="cuda")
            st["xs"] = torch.empty(-(-L // 128), n, device="cuda")
        else:
            # channels of very unequal size, as activations have them
            size = torch.exp(1.5 * _randn(g, K))
            x = _randn(g, B, L, K) * size
            st["x"] = (x if case["what"] == "last" else x.transpose(1, 2).contiguous()).to(dt)
            st["xq"] = torch.empty(B, L, K, dtype=torch.float8_e4m3fn, device="cuda")
            st["xs"] = torch.empty(B, n, L, device="cuda")
    else:
        B, L, K, N = (case[k] for k in ("B", "L", "K", "N"))
        st["xq"], st["xs"] = _to_fp8_rows(_randn(g, B, L, K))
        st["Wq"], st["Ws"] = _to_fp8_weight(_randn(g, N, K) * K ** -0.5)
        st["bias"] = 0.1 * _randn(g, N) if case["bias"] else None
        st["out"] = torch.empty((B, N, L) if case["first"] else (B, L, N), dtype=torch.bfloat16, device="cuda")
    return st


# ----------------------------------------------------------- plain forms
def _heads(x, H):
    """[B, H d, L] to [B, H, L, d] in fp32."""
    B, C, L = x.shape
    return x.float().reshape(B, H, C // H, L).transpose(2, 3)


def _unit(x):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)


def _delta_inputs(s):
    """q, k, v [B, Hv, L, d], decay and strength [B, Hv, L] in fp32, with the positions behind a sequence's end inert."""
    c = s["case"]
    r = c["Hv"] // c["Hk"]
    q, k, v = _heads(s["q"], c["Hk"]), _heads(s["k"], c["Hk"]), _heads(s["v"], c["Hv"])
    if c["l2norm"]:
        q, k = _unit(q), _unit(k)
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    g, beta, live = s["g"], s["beta"], None
    if s["lengths"] is not None:
        live = torch.arange(c["L"], device="cuda")[None, :] < s["lengths"][:, None]
        m = live[:, None, :]
        q, k, v = (torch.where(m[..., None], x, 0.0) for x in (q, k, v))
        g, beta = torch.where(m, g, 0.0), torch.where(m, beta, 0.0)
    return q, k, v, g, beta, live


def _plain_delta(s):
    """The chunked form: inside a chunk the writes solve a triangular system, between chunks the state is carried."""
    c = s["case"]
    B, L, Hv, dk, dv = (c[x] for x in ("B", "L", "Hv", "dk", "dv"))
    q, k, v, g, beta, live = _delta_inputs(s)
    n = -(-L // CHUNK)
    pad = n * CHUNK - L
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).reshape(B * Hv, n, CHUNK, -1) for x in (q, k, v))
    g, beta = (torch.nn.functional.pad(x, (0, pad)).reshape(B * Hv, n, CHUNK) for x in (g, beta))
    G = torch.cumsum(g.double(), -1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    decay = torch.where(low, G[..., :, None] - G[..., None, :], -math.inf).float().exp()        # e^{G_i - G_j}, j <= i
    into, last = G.float().exp(), G[..., -1:]
    out = (last - G).float().exp()
    A = beta[..., None] * decay * torch.matmul(k, k.transpose(-1, -2))
    T = torch.eye(CHUNK, device="cuda").expand(B * Hv, n, CHUNK, CHUNK).clone()                  # (1 + strict lower A)^-1
    for i in range(1, CHUNK):
        T[..., i, :i] = -torch.matmul(A[..., i: i + 1, :i], T[..., :i, :i]).squeeze(-2)
    T = T * beta[..., None, :]
    P = decay * torch.matmul(q, k.transpose(-1, -2))
    S = (s["state_in"].reshape(B * Hv, dk, dv).clone() if s["state_in"] is not None
         else torch.zeros(B * Hv, dk, dv, device="cuda"))
    y = torch.empty_like(v)
    for j in range(n):
        kj, e = k[:, j], into[:, j, :, None]
        U = torch.matmul(T[:, j], v[:, j] - e * torch.matmul(kj, S))
        y[:, j] = e * torch.matmul(q[:, j], S) + torch.matmul(P[:, j], U)
        S = last[:, j, :, None].float().exp() * S + torch.matmul((out[:, j, :, None] * kj).transpose(-1, -2), U)
    y = (y.reshape(B, Hv, n * CHUNK, dv)[:, :, :L] * dk ** -0.5).transpose(2, 3).reshape(B, Hv * dv, L).to(s["o"].dtype)
    s["o"].copy_(y if live is None else torch.where(live[:, None, :], y, s["o"]))
    s["state_out"].copy_(S.view(B, Hv, dk, dv))
    return {"o": s["o"], "state": s["state_out"]}


def _plain_step(s):
    c = s["case"]
    B, Hk, Hv, dk, dv = (c[x] for x in ("B", "Hk", "Hv", "dk", "dv"))
    q, k, v = (s[x].float().reshape(B, h, -1) for x, h in (("q", Hk), ("k", Hk), ("v", Hv)))
    if c["l2norm"]:
        q, k = _unit(q), _unit(k)
    q, k = (x.repeat_interleave(Hv // Hk, 1) for x in (q, k))
    at = s["slots"].long() if s["slots"] is not None else slice(None)
    S = s["pool"][at] * s["g"].exp()[..., None, None]
    u = s["beta"][..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["pool"][at] = S
    s["o"].copy_(((S * q[..., None]).sum(-2) * dk ** -0.5).reshape(B, Hv * dv))
    return {"o": s["o"], "state": s["pool"]}


def _plain_quant(s):
    if s["case"]["what"] == "weight":
        q, sc = _to_fp8_weight(s["x"].float())
    else:
        x = s["x"].float()
        q, sc = _to_fp8_rows(x if s["case"]["what"] == "last" else x.transpose(1, 2).contiguous())
    return {"q": q, "scale": sc}


def _plain_proj(s):
    K, N = s["case"]["K"], s["case"]["N"]
    x = s["xq"].float() * s["xs"].transpose(1, 2).repeat_interleave(128, 2)[..., :K]
    w = s["Wq"].float() * s["Ws"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    out = torch.matmul(x, w.t())
    if s["bias"] is not None:
        out = out + s["bias"]
    return {"out": (out.transpose(1, 2) if s["case"]["first"] else out).to(torch.bfloat16).contiguous()}


# ------------------------------------------------------------------- run
def _own(s):
    from fft_long_convolution_02_b200 import binding as hb
    c = s["case"]
    if c["op"] == "delta":
        if "ws" not in s:
            n = hb.hyena_delta_rule_workspace_bytes(c["B"], c["L"], c["Hk"], c["Hv"], c["dk"], c["dv"], s["q"].dtype)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        hb.hyena_delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], c["Hk"], c["Hv"], s["state_in"],
                            s["state_out"], s["lengths"], l2norm=c["l2norm"], workspace=s["ws"])
        return {"o": s["o"], "state": s["state_out"]}
    if c["op"] == "step":
        hb.hyena_delta_rule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], s["pool"], c["Hk"], c["Hv"],
                                 s["slots"], l2norm=c["l2norm"])
        return {"o": s["o"], "state": s["pool"]}
    if c["op"] == "quant":
        if c["what"] == "weight":
            hb.hyena_quantize_fp8_weight(s["x"], s["xq"], s["xs"])
        else:
            hb.hyena_quantize_fp8(s["x"], s["xq"], s["xs"], channels_first=c["what"] == "first")
        return {"q": s["xq"], "scale": s["xs"]}
    hb.hyena_proj_fp8(s["xq"], s["xs"], s["Wq"], s["Ws"], s["bias"], s["out"], channels_first=c["first"])
    return {"out": s["out"]}


def run(state):
    if own:
        return _own(state)
    return {"delta": _plain_delta, "step": _plain_step, "quant": _plain_quant, "proj": _plain_proj}[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "delta":
        B, L, Hk, Hv, dk, dv = (case[k] for k in ("B", "L", "Hk", "Hv", "dk", "dv"))
        es = 2 if case["dtype"] == "bf16" else 4
        state = 4 * B * Hv * dk * dv
        return {"bytes": B * L * (es * (2 * Hk * dk + 2 * Hv * dv) + 8 * Hv) + state * (2 if case["state"] else 1),
                "flops": 6 * B * L * Hv * dk * dv}
    if op == "step":
        B, Hk, Hv, dk, dv = (case[k] for k in ("B", "Hk", "Hv", "dk", "dv"))
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": B * (es * (2 * Hk * dk + 2 * Hv * dv) + 8 * Hv + 8 * Hv * dk * dv),
                "flops": 7 * B * Hv * dk * dv}
    if op == "quant":
        B, L, K = case["B"], case["L"], case["K"]
        es = 2 if case["dtype"] == "bf16" else 4
        rows = -(-L // 128) if case["what"] == "weight" else B * L
        return {"bytes": B * L * K * (es + 1) + 4 * rows * -(-K // 128), "flops": 2 * B * L * K}
    B, L, K, N = (case[k] for k in ("B", "L", "K", "N"))
    n = -(-K // 128)
    return {"bytes": B * L * (K + 4 * n) + N * K + 4 * n * -(-N // 128) + (4 * N if case["bias"] else 0) + 2 * B * L * N,
            "flops": 2 * B * L * K * N}


# ----------------------------------------------------------------- exact
def _e4m3(y):
    """Nearest e4m3 value (ties to even, saturating) of fp64 numbers."""
    _, e = torch.frexp(y)
    ulp = torch.exp2((e.double() - 1).clamp(min=-6.0) - 3)
    return (torch.round(y / ulp) * ulp).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_unit(x):
    return x * (x.square().sum(-1, keepdim=True) + EPS).rsqrt()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "delta":
        # token by token, from the definition
        B, L, Hk, Hv, dk, dv = (case[k] for k in ("B", "L", "Hk", "Hv", "dk", "dv"))
        q, k, v = (s[x].double().view(B, h, -1, L).permute(3, 0, 1, 2) if case["first"] else
                   s[x].transpose(1, 2).double().view(B, L, h, -1).permute(1, 0, 2, 3)
                   for x, h in (("q", Hk), ("k", Hk), ("v", Hv)))
        if case["l2norm"]:
            q, k = _exact_unit(q), _exact_unit(k)
        head = torch.arange(Hv, device="cuda") // (Hv // Hk)
        S = torch.zeros(B, Hv, dk, dv, dtype=torch.float64, device="cuda")
        if case["state"]:
            S += s["state_in"]
        a, b = s["g"].double().exp().permute(2, 0, 1), s["beta"].double().permute(2, 0, 1)
        o = s["o"].double()
        for t in range(L):
            kt, qt = k[t][:, head], q[t][:, head]
            new = S * a[t][..., None, None]
            u = b[t][..., None] * (v[t] - torch.einsum("bhk,bhkv->bhv", kt, new))
            new = new + kt[..., None] * u[..., None, :]
            y = torch.einsum("bhk,bhkv->bhv", qt, new).reshape(B, Hv * dv) / math.sqrt(dk)
            if s["lengths"] is None:
                S, o[:, :, t] = new, y
            else:
                go = t < s["lengths"]
                S = torch.where(go[:, None, None, None], new, S)
                o[:, :, t] = torch.where(go[:, None], y, o[:, :, t])
        return {"o": o, "state": S}
    if op == "step":
        B, Hk, Hv, dk, dv = (case[k] for k in ("B", "Hk", "Hv", "dk", "dv"))
        head = torch.arange(Hv, device="cuda") // (Hv // Hk)
        q, k, v = (s[x].double().view(B, h, -1) for x, h in (("q", Hk), ("k", Hk), ("v", Hv)))
        if case["l2norm"]:
            q, k = _exact_unit(q), _exact_unit(k)
        q, k = q[:, head], k[:, head]
        pool = s["pool"].double()
        at = torch.arange(B, device="cuda") if s["slots"] is None else s["slots"].long()
        S = pool[at] * s["g"].double().exp()[..., None, None]
        u = s["beta"].double()[..., None] * (v - torch.einsum("bhk,bhkv->bhv", k, S))
        S = S + k[..., None] * u[..., None, :]
        pool[at] = S
        return {"o": torch.einsum("bhk,bhkv->bhv", q, S).reshape(B, Hv * dv) / math.sqrt(dk), "state": pool}
    if op == "quant":
        # scale and quotient are fp32 numbers by the operator's definition; a quotient in fp64 rounds to the same fp32
        tiny = torch.finfo(torch.float32).tiny
        x = s["x"].double()
        if case["what"] == "first":
            x = x.transpose(1, 2)
        if case["what"] == "weight":
            q, sc = torch.empty_like(x), torch.empty(-(-case["L"] // 128), -(-case["K"] // 128), device="cuda")
            for i in range(sc.shape[0]):
                for j in range(sc.shape[1]):
                    b = x[128 * i: 128 * i + 128, 128 * j: 128 * j + 128]
                    sc[i, j] = (b.abs().max() / E4M3_MAX).float().clamp(min=tiny)
                    q[128 * i: 128 * i + 128, 128 * j: 128 * j + 128] = _e4m3((b / sc[i, j].double()).float().double())
            return {"q": q, "scale": sc.double()}
        q, cols = torch.empty_like(x).contiguous(), []
        for j in range(-(-case["K"] // 128)):
            b = x[..., 128 * j: 128 * j + 128]
            sc = (b.abs().amax(-1) / E4M3_MAX).float().clamp(min=tiny).double()
            q[..., 128 * j: 128 * j + 128] = _e4m3((b / sc[..., None]).float().double())
            cols.append(sc)
        return {"q": q, "scale": torch.stack(cols, 1)}
    B, L, K, N = (case[k] for k in ("B", "L", "K", "N"))
    kb, nb = torch.arange(K, device="cuda") // 128, torch.arange(N, device="cuda") // 128
    w = s["Wq"].double() * s["Ws"].double()[nb][:, kb]
    out = torch.empty(B, L, N, dtype=torch.float64, device="cuda")
    for b in range(B):
        out[b] = (s["xq"][b].double() * s["xs"][b].double()[kb].t()) @ w.t()
    if s["bias"] is not None:
        out += s["bias"].double()
    return {"out": out.transpose(1, 2).contiguous() if case["first"] else out}
