"""Measured cases of the operators of a gated delta-rule block: rotary
positions, layer norm (forward, backward) and the gated delta rule
(chunkwise forward, backward, one decode step).

``run`` computes an operator in its plain form (elementary torch operations
in 32 bits, 64 where a comment says so) or, with ``own`` set, by this
library's entry points.  ``exact`` gives the same outputs in 64 bits from the
operators' definitions.

The gated delta rule, per value head, with S [dk, dv]:
    S' = exp(g_t) S_{t-1},  u_t = beta_t (v_t - S'^T k_t),
    S_t = S' + k_t u_t^T,   o_t = S_t^T q_t.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # Serving, one token for each of 64 sequences: half layout, half of
        # the head turned, frequencies stretched for a long context.
        {"name": "rotary 64x1 16/16x256", "op": "rotary", "B": 64, "N": 1, "H": 16, "Hk": 16, "d": 256, "rd": 128,
         "layout": "half", "scaling": "yarn", "dtype": "bf16"},
        # Prefill of one 8k sequence, all of the head, consecutive pairs.
        {"name": "rotary 1x8192 16/16x256", "op": "rotary", "B": 1, "N": 8192, "H": 16, "Hk": 16, "d": 256, "rd": 256,
         "layout": "interleaved", "scaling": "linear", "dtype": "bf16"},
        # The norm before a block at a decode batch of 64 tokens.
        {"name": "ln forward 64x2048", "op": "ln_forward", "rows": 64, "d": 2048, "dtype": "bf16"},
        # The norm of a training batch of 2 x 4096 tokens.
        {"name": "ln forward 8192x2048", "op": "ln_forward", "rows": 8192, "d": 2048, "dtype": "bf16"},
        # An odd width and row count, in 32 bits (no vector divides a row).
        {"name": "ln backward 4099x1001 f32", "op": "ln_backward", "rows": 4099, "d": 1001, "dtype": "f32"},
        # The norm's backward pass of a training batch of 2 x 4096 tokens.
        {"name": "ln backward 8192x2048", "op": "ln_backward", "rows": 8192, "d": 2048, "dtype": "bf16"},
        # Prefill of a padded batch of four prompts of different lengths that
        # continue given states, two value heads to a key head.
        {"name": "delta forward 4x2047 8/16x128x128", "op": "delta_forward", "B": 4, "N": 2047, "Hk": 8, "H": 16,
         "dk": 128, "dv": 128, "ragged": True, "state": True, "dtype": "bf16"},
        # Prefill of one 8k sequence with 16 heads of 256 and 512.
        {"name": "delta forward 1x8192 16x256x512", "op": "delta_forward", "B": 1, "N": 8192, "Hk": 16, "H": 16,
         "dk": 256, "dv": 512, "ragged": False, "state": False, "dtype": "bf16"},
        # One token of a single sequence: the latency of a step.
        {"name": "delta decode 1 8/16x128x128", "op": "delta_decode", "B": 1, "Hk": 8, "H": 16, "dk": 128, "dv": 128,
         "dtype": "bf16"},
        # One token of 64 sequences with 1 GB of states.
        {"name": "delta decode 64 16x256x512", "op": "delta_decode", "B": 64, "Hk": 16, "H": 16, "dk": 256, "dv": 512,
         "dtype": "bf16"},
        # The backward pass of short odd sequences with heads of 64.
        {"name": "delta backward 2x1000 8x64x64", "op": "delta_backward", "B": 2, "N": 1000, "Hk": 8, "H": 8, "dk": 64,
         "dv": 64, "ragged": False, "state": True, "dtype": "bf16"},
        # The backward pass of one 4k sequence with 16 heads of 128.
        {"name": "delta backward 1x4096 16x128x128", "op": "delta_backward", "B": 1, "N": 4096, "Hk": 16, "H": 16,
         "dk": 128, "dv": 128, "ragged": False, "state": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "ln_forward", "ln_backward", "delta_forward", "delta_decode", "delta_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rotary":
        Hk = rng.choice([1, 2, 4, 8, 16])
        d = rng.choice([64, 96, 128, 256])
        B = _log(rng, 1, 64)
        return {"op": op, "B": B, "N": _log(rng, 1, 8192 // B), "Hk": Hk, "H": Hk * rng.choice([1, 2, 4]) if Hk < 8 else 16,
                "d": d, "rd": rng.choice([d, d // 2, d // 4]), "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "yarn"]), "dtype": dtype}
    if op in ("ln_forward", "ln_backward"):
        return {"op": op, "rows": _log(rng, 1, 8192), "d": _log(rng, 17, 2048), "dtype": dtype}
    if op == "delta_decode":
        Hk = rng.choice([1, 2, 4, 8])
        return {"op": op, "B": _log(rng, 1, 64), "Hk": Hk, "H": Hk * rng.choice([1, 2]), "dk": rng.choice([16, 64, 100, 128, 256]),
                "dv": 4 * _log(rng, 4, 128), "dtype": dtype}
    Hk = rng.choice([2, 4, 8])
    c = {"op": op, "B": _log(rng, 1, 4), "Hk": Hk, "H": Hk * rng.choice([1, 2])}
    if op == "delta_forward" and dtype == "f32":  # token by token on the CUDA cores: short sequences
        return dict(c, N=_log(rng, 1, 500), dk=rng.choice([16, 64, 128]), dv=4 * _log(rng, 4, 32),
                    ragged=rng.choice([True, False]), state=rng.choice([True, False]), dtype=dtype)
    top = 2048 if op == "delta_backward" else 4096
    return dict(c, N=_log(rng, 1, top), dk=rng.choice([64, 128, 256]) if op == "delta_forward" else rng.choice([64, 128]),
                dv=rng.choice([64, 128, 192, 256]) if op == "delta_forward" else rng.choice([64, 128]),
                ragged=rng.choice([True, False]), state=rng.choice([True, False]), dtype="bf16")


def lengths_of(c):
    """Tokens of each sequence of a padded batch: N, then fewer and fewer."""
    return [c["N"] - (3 * b * c["N"]) // (4 * c["B"]) if c["ragged"] else c["N"] for b in range(c["B"])]


# ------------------------------------------------------------------ inputs

def frequencies(rd, scaling, base=10000.0, factor=8.0, original=4096):
    """(angle per position of each pair, factor on cos and sin)."""
    p = torch.arange(rd // 2, dtype=torch.float64)
    f = base ** (-2 * p / rd)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":  # pairs that turn often keep their angle, those that turn less than once get it divided
        def dim(turns):
            return rd * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rd - 1)
        ramp = ((p - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    c, dt = case, DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    st = {"case": dict(c)}
    if c["op"] == "rotary":
        st["q"], st["k"] = normal(c["B"], c["N"], c["H"], c["d"]).to(dt), normal(c["B"], c["N"], c["Hk"], c["d"]).to(dt)
        first = torch.randint(0, 32768, (c["B"], 1), generator=gen, device=dev)
        st["positions"] = first + torch.arange(c["N"], device=dev)  # each sequence at its own place
        st["freqs"], st["scale"] = frequencies(c["rd"], c["scaling"])
        return st
    if c["op"] in ("ln_forward", "ln_backward"):
        st["x"] = (normal(c["rows"], c["d"]) * 2 + 0.5).to(dt)
        st["gain"], st["bias"] = (1 + 0.1 * normal(c["d"])).to(dt), (0.1 * normal(c["d"])).to(dt)
        if c["op"] == "ln_backward":
            st["dout"] = normal(c["rows"], c["d"]).to(dt)
            x = st["x"].double()
            st["mean"] = x.mean(-1).float()
            st["rstd"] = (x.var(-1, unbiased=False) + 1e-5).rsqrt().float()
        return st
    lead = (c["B"],) if c["op"] == "delta_decode" else (c["B"], c["N"])

    def unit(*shape):
        x = normal(*shape)
        return x / x.norm(dim=-1, keepdim=True)

    st["q"], st["k"] = (unit(*lead, c["Hk"], c["dk"]) * c["dk"] ** -0.5).to(dt), unit(*lead, c["Hk"], c["dk"]).to(dt)
    st["v"] = normal(*lead, c["H"], c["dv"]).to(dt)
    # decays: some heads forget in a few tokens, others keep for hundreds
    rate = torch.exp(torch.linspace(math.log(0.003), math.log(0.5), c["H"], device=dev))
    st["g"] = -rate * torch.nn.functional.softplus(normal(*lead, c["H"]))
    st["beta"] = torch.sigmoid(normal(*lead, c["H"]))
    if c["op"] == "delta_decode":
        st["state"] = 0.3 * normal(c["B"], c["H"], c["dk"], c["dv"])
        return st
    st["initial_state"] = 0.3 * normal(c["B"], c["H"], c["dk"], c["dv"]) if c["state"] else None
    st["lengths"] = torch.tensor(lengths_of(c), dtype=torch.int32, device=dev) if c["ragged"] else None
    if c["op"] == "delta_forward":
        # rows behind a sequence's end are not written: the program's buffer holds zeros there
        st["out"] = torch.zeros(c["B"], c["N"], c["H"], c["dv"], dtype=dt, device=dev)
    else:
        st["dout"] = normal(c["B"], c["N"], c["H"], c["dv"]).to(dt)
        st["dfinal"] = 0.3 * normal(c["B"], c["H"], c["dk"], c["dv"]) if c["state"] else None
    return st


# --------------------------------------------------------------- plain forms

def _rotary(x, cos, sin, rd, layout):
    y = x.float().clone()
    a, b = (y[..., 0:rd:2], y[..., 1:rd:2]) if layout == "interleaved" else (y[..., : rd // 2], y[..., rd // 2: rd])
    u, w = a * cos - b * sin, a * sin + b * cos
    a.copy_(u)
    b.copy_(w)
    return y.to(x.dtype)


def _rotary_plain(st):
    c = st["case"]
    # a far position times a frequency: 64 bits, 32 after the cosine
    ang = st["positions"].double()[..., None, None] * st["freqs"].to(st["q"].device)
    cos, sin = (ang.cos() * st["scale"]).float(), (ang.sin() * st["scale"]).float()
    return [_rotary(st[n], cos, sin, c["rd"], c["layout"]) for n in ("q", "k")]


def _ln_forward_plain(st, eps=1e-5):
    x = st["x"].float()
    mean = x.mean(-1)
    xc = x - mean[:, None]
    rstd = ((xc * xc).mean(-1) + eps).rsqrt()
    y = xc * rstd[:, None] * st["gain"].float() + st["bias"].float()
    return [y.to(st["x"].dtype), mean, rstd]


def _ln_backward_plain(st):
    x, dy = st["x"].float(), st["dout"].float()
    xh = (x - st["mean"][:, None]) * st["rstd"][:, None]
    dn = dy * st["gain"].float()
    dx = st["rstd"][:, None] * (dn - dn.mean(-1, keepdim=True) - xh * (dn * xh).mean(-1, keepdim=True))
    return [dx.to(st["x"].dtype), (dy * xh).sum(0), dy.sum(0)]


def _whole_sequence(st, wide):
    """The operands of the rule over the whole sequence at once, [B, H, N, .]:
    with G the running sum of g, D_ij = exp(G_i - G_j) for i >= j and
    A = strictly lower part of beta_i D_ij (k_i . k_j),
        (I + A) U = beta (V - exp(G) K S0),  O = (Q K^T o D) U + exp(G) Q S0,
        S_N = exp(G_N) S0 + (exp(G_N - G) K)^T U.
    G is summed and subtracted in 64 bits: it grows along the sequence."""
    c = st["case"]
    rep = c["H"] // c["Hk"]
    q, k = (st[n].to(wide).repeat_interleave(rep, 2).transpose(1, 2) for n in ("q", "k"))
    v = st["v"].to(wide).transpose(1, 2)
    g, beta = st["g"].double().transpose(1, 2), st["beta"].to(wide).transpose(1, 2)
    if st["lengths"] is not None:  # tokens behind the end change nothing
        live = (torch.arange(c["N"], device=q.device) < st["lengths"][:, None])[:, None]
        g, beta = g * live, beta * live
        q, k, v = (x * live[..., None] for x in (q, k, v))
    G = g.cumsum(-1)
    i = torch.arange(c["N"], device=q.device)
    D = (G[..., :, None] - G[..., None, :]).masked_fill_(i[:, None] < i, -math.inf).exp_().to(wide)
    to_end, since = (G[..., -1:] - G).exp().to(wide)[..., None], G.exp().to(wide)[..., None]
    A = (k @ k.transpose(-1, -2)).mul_(D).mul_(beta[..., None]).tril_(-1)
    s0 = st["initial_state"]
    s0 = torch.zeros(c["B"], c["H"], c["dk"], c["dv"], dtype=wide, device=q.device) if s0 is None else s0.to(wide)
    read = k @ s0
    U = torch.linalg.solve_triangular(A, beta[..., None] * (v - since * read), upper=False, unitriangular=True)
    return q, k, v, beta, D, to_end, since, A, s0, read, U


def _delta_forward_plain(st):
    q, k, v, beta, D, to_end, since, A, s0, read, U = _whole_sequence(st, torch.float32)
    out = (q @ k.transpose(-1, -2)).mul_(D) @ U + since * (q @ s0)
    state = since[..., -1:, :] * s0 + (to_end * k).transpose(-1, -2) @ U
    return [out.transpose(1, 2).to(st["v"].dtype).contiguous(), state]


def _delta_backward_plain(st):
    """The derivatives of the whole-sequence form.  In 64 bits: the gradient
    of a gate is a difference of sums over the sequence.  A decay exponent
    G_i multiplies what row i reads (q_i, and k_i in A and in K S0) and
    divides what it writes (k_i in the scores, in A and in S_N)."""
    c = st["case"]
    q, k, v, beta, D, to_end, since, A, s0, read, U = _whole_sequence(st, torch.float64)
    do = st["dout"].double().transpose(1, 2)
    if st["lengths"] is not None:
        live = (torch.arange(c["N"], device=q.device) < st["lengths"][:, None])[:, None]
        do = torch.where(live[..., None], do, 0.0)
    dS = torch.zeros_like(s0) if st["dfinal"] is None else st["dfinal"].double()
    P = (q @ k.transpose(-1, -2)) * D
    dU = P.transpose(-1, -2) @ do + to_end * (k @ dS)
    dY = torch.linalg.solve_triangular(A.transpose(-1, -2), dU, upper=True, unitriangular=True)
    err = (v - since * read) - ((k @ k.transpose(-1, -2)) * D).tril(-1) @ U  # u = beta err
    dbeta = (dY * err).sum(-1)
    dR = beta[..., None] * dY
    dP = (do @ U.transpose(-1, -2)) * D
    dA = -(dR @ U.transpose(-1, -2)).mul_(D).tril_(-1)
    dq = since * (do @ s0.transpose(-1, -2)) + dP @ k
    reads = dA @ k - since * (dR @ s0.transpose(-1, -2))
    writes = dP.transpose(-1, -2) @ q + dA.transpose(-1, -2) @ k + to_end * (U @ dS.transpose(-1, -2))
    last = since[..., -1:, :] * s0 + (to_end * k).transpose(-1, -2) @ U
    dG = (q * dq).sum(-1) + (k * reads).sum(-1) - (k * writes).sum(-1)
    dG[..., -1] += (dS * last).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1)
    ds0 = since[..., -1:, :] * dS + (since * q).transpose(-1, -2) @ do - (since * k).transpose(-1, -2) @ dR
    if st["lengths"] is not None:
        dg, dbeta = dg * live, dbeta * live
    dk, dt = reads + writes, st["q"].dtype

    def shared(x):  # the gradient of a key head is the sum over its value heads
        return x.reshape(c["B"], c["Hk"], -1, c["N"], c["dk"]).sum(2).transpose(1, 2).to(dt).contiguous()

    grads = [shared(dq), shared(dk), dR.transpose(1, 2).to(dt).contiguous(), dg.transpose(1, 2).float().contiguous(),
             dbeta.transpose(1, 2).float().contiguous()]
    return grads + ([ds0.float()] if st["initial_state"] is not None else [])


def _delta_decode_plain(st):
    c = st["case"]
    rep = c["H"] // c["Hk"]
    q, k = (st[n].float().repeat_interleave(rep, 1)[..., None] for n in ("q", "k"))
    S = st["state"] * st["g"].exp()[..., None, None]
    u = st["beta"][..., None] * (st["v"].float() - (k * S).sum(-2))
    S += k * u[..., None, :]
    st["state"].copy_(S)
    return [(q * S).sum(-2).to(st["v"].dtype), st["state"]]


# --------------------------------------------------------------- one pass

def _run_own(st):
    import linear_recurrent_sequence_chunkwise_b200 as R
    c = st["case"]
    if c["op"] == "rotary":
        return list(R.ret_rotary(st["q"], st["k"], freqs=st["freqs"], positions=st["positions"], layout=c["layout"],
                                 scale=st["scale"]))
    if c["op"] == "ln_forward":
        return list(R.ret_layernorm_forward(st["x"], st["gain"], st["bias"], eps=1e-5, want_stats=True))
    if c["op"] == "ln_backward":
        return list(R.ret_layernorm_backward(st["dout"], st["x"], st["mean"], st["rstd"], st["gain"]))
    if c["op"] == "delta_forward":
        return list(R.ret_delta_forward_chunkwise(st["q"], st["k"], st["v"], st["g"], st["beta"], out=st["out"],
                                                  initial_state=st["initial_state"], lengths=st["lengths"],
                                                  want_final_state=True))
    if c["op"] == "delta_decode":
        return [R.ret_delta_decode_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"],
                                        out_dtype=st["v"].dtype), st["state"]]
    return [t for t in R.ret_delta_backward_chunkwise(st["q"], st["k"], st["v"], st["g"], st["beta"], st["dout"],
                                                      initial_state=st["initial_state"], dfinal_state=st["dfinal"],
                                                      lengths=st["lengths"], grad_dtype=st["q"].dtype) if t is not None]


PLAIN = {"rotary": _rotary_plain, "ln_forward": _ln_forward_plain, "ln_backward": _ln_backward_plain,
         "delta_forward": _delta_forward_plain, "delta_backward": _delta_backward_plain, "delta_decode": _delta_decode_plain}


def run(st):
    return _run_own(st) if own else PLAIN[st["case"]["op"]](st)


def work(case):
    """Each input read once, each output written once; the delta rule's
    operations are those of its token-by-token form."""
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "rotary":
        n = c["B"] * c["N"] * (c["H"] + c["Hk"])
        return {"bytes": 2 * n * c["d"] * e + c["B"] * c["N"] * 8, "flops": 3 * n * c["rd"]}
    if c["op"] == "ln_forward":
        return {"bytes": (2 * c["rows"] + 2) * c["d"] * e + 8 * c["rows"], "flops": 8 * c["rows"] * c["d"]}
    if c["op"] == "ln_backward":
        return {"bytes": (3 * c["rows"] + 1) * c["d"] * e + 8 * c["rows"] + 8 * c["d"], "flops": 12 * c["rows"] * c["d"]}
    state = c["B"] * c["H"] * c["dk"] * c["dv"]
    tokens = c["B"] if c["op"] == "delta_decode" else sum(lengths_of(c))
    qk, vo, gates = tokens * c["Hk"] * c["dk"] * e, tokens * c["H"] * c["dv"] * e, tokens * c["H"] * 4
    token_work = tokens * c["H"] * c["dk"] * c["dv"]
    if c["op"] == "delta_decode":
        return {"bytes": 2 * qk + 2 * vo + 2 * gates + 8 * state, "flops": 7 * token_work}
    if c["op"] == "delta_forward":
        return {"bytes": 2 * qk + 2 * vo + 2 * gates + 4 * state * (2 if c["state"] else 1), "flops": 7 * token_work}
    # the states again, then the gradients
    return {"bytes": 4 * qk + 3 * vo + 4 * gates + (12 * state if c["state"] else 0), "flops": 19 * token_work}


# ---------------------------------------------------------------- 64 bits

def _exact_rotary(st):
    c, outs = st["case"], []
    turn = torch.polar(torch.tensor(st["scale"], dtype=torch.float64, device=st["q"].device),
                       st["positions"].double()[:, :, None, None] * st["freqs"].to(st["q"].device))
    for x in (st["q"].double(), st["k"].double()):
        rd = c["rd"]
        pairs = x[..., :rd].unflatten(-1, (rd // 2, 2) if c["layout"] == "interleaved" else (2, rd // 2))
        if c["layout"] == "half":
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        if c["layout"] == "half":
            z = z.transpose(-1, -2)
        outs.append(torch.cat([z.flatten(-2), x[..., rd:]], -1))
    return outs


def _exact_ln(st, eps=1e-5):
    x = st["x"].double()
    if st["case"]["op"] == "ln_forward":
        n = x.shape[-1]
        mean = x.sum(-1) / n
        var = ((x - mean[:, None]) ** 2).sum(-1) / n
        rstd = 1 / (var + eps).sqrt()
        return [st["gain"].double() * ((x - mean[:, None]) * rstd[:, None]) + st["bias"].double(), mean, rstd]
    dy, r = st["dout"].double(), st["rstd"].double()[:, None]
    h = (x - st["mean"].double()[:, None]) * r
    t, n = dy * st["gain"].double(), x.shape[-1]
    dx = r * (t - (t.sum(-1, keepdim=True) + h * (t * h).sum(-1, keepdim=True)) / n)
    return [dx, torch.einsum("rd,rd->d", dy, h), torch.einsum("rd->d", dy)]


def _exact_delta(st):
    """Token by token; the backward pass walks the same steps in reverse."""
    c = st["case"]
    one = c["op"] == "delta_decode"
    N, B, H, Hk, dk, dv = (1 if one else c["N"]), c["B"], c["H"], c["Hk"], c["dk"], c["dv"]
    rep = H // Hk
    q, k, v, a, beta = (st[n].double() for n in ("q", "k", "v", "g", "beta"))
    if one:
        q, k, v, a, beta = (x[:, None] for x in (q, k, v, a, beta))
    q, k = (x.repeat_interleave(rep, 2) for x in (q, k))
    a = a.exp()
    live = torch.ones(B, N, 1, dtype=torch.float64, device=q.device)
    if not one and st["lengths"] is not None:
        live = (torch.arange(N, device=q.device) < st["lengths"][:, None]).double()[..., None]
        a, beta = 1 + (a - 1) * live, beta * live
    S = st["state"] if one else st["initial_state"]
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=q.device) if S is None else S.double().clone()
    back = c["op"] == "delta_backward"
    kept = torch.empty(N, *S.shape, dtype=torch.float64, device=q.device) if back else None
    u = torch.empty(B, N, H, dv, dtype=torch.float64, device=q.device)
    out = torch.empty_like(u)
    for t in range(N):
        if back:
            kept[t] = S
        S = S * a[:, t, :, None, None]
        kt = k[:, t]
        u[:, t] = beta[:, t, :, None] * (v[:, t] - (kt[..., None, :] @ S)[..., 0, :])
        S = torch.baddbmm(S.reshape(-1, dk, dv), kt.reshape(-1, dk, 1), u[:, t].reshape(-1, 1, dv)).view_as(S)
        if not back:
            out[:, t] = (q[:, t, :, None, :] @ S)[..., 0, :]
    if one:
        return [out[:, 0], S]
    if not back:
        return [out * live[..., None], S]
    do = torch.where(live[..., None] > 0, st["dout"].double(), 0.0)
    dS = torch.zeros_like(S) if st["dfinal"] is None else st["dfinal"].double().clone()
    dq, dkk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(u)
    dg, dbeta = torch.empty_like(a), torch.empty_like(a)
    for t in range(N - 1, -1, -1):
        qt, kt, ut, dot = q[:, t, :, :, None], k[:, t, :, :, None], u[:, t, :, None, :], do[:, t, :, None, :]
        before = kept[t]
        decayed = before * a[:, t, :, None, None]
        dq[:, t] = ((decayed + kt * ut) @ dot.transpose(-1, -2))[..., 0]
        dS = dS + qt * dot
        du = (kt.transpose(-1, -2) @ dS)
        miss = v[:, t, :, None, :] - kt.transpose(-1, -2) @ decayed
        dbeta[:, t] = (du * miss).sum((-1, -2))
        dvv[:, t] = beta[:, t, :, None] * du[..., 0, :]
        dp = -dvv[:, t][..., None, :]
        dkk[:, t] = (dS @ ut.transpose(-1, -2) + decayed @ dp.transpose(-1, -2))[..., 0]
        dS = dS + kt * dp
        dg[:, t] = (dS * decayed).sum((-1, -2))
        dS = dS * a[:, t, :, None, None]
    dq, dkk = (x.unflatten(2, (Hk, rep)).sum(3) * live[..., None] for x in (dq, dkk))
    return [dq, dkk, dvv, dg * live, dbeta * live] + ([dS] if st["initial_state"] is not None else [])


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(st)
    return _exact_ln(st) if case["op"].startswith("ln") else _exact_delta(st)
