"""The sequence operators next to the depthwise convolution, as measured cases.

A linear-attention token mixer reads its queries, keys and values through a
short causal depthwise convolution, keeps what it has read in one matrix per
head with the gated delta rule, and leaves through a gated normalization; the
block around it adds the result to the residual stream and normalizes that for
the next block.  Each case here is one pass through one of those operators:

  conv_fwd / conv_step / conv_bwd      causal depthwise 1-D convolution over
                                       packed sequences, one token per cached
                                       sequence, and the gradients
  delta_fwd / delta_step / delta_bwd   gated delta rule, chunked over packed
                                       sequences, recurrent over a state cache,
                                       and the gradients
  norm_fwd / norm_bwd                  norm after a block, its gate, residual
                                       scale and residual, and the norm before
                                       the next block

``run`` computes the plain form with elementary torch operations in fp32 where
``own`` is false and calls the library where it is true; ``exact`` computes
the definition in fp64, token by token for the delta rule.
"""
import math
import random

import torch

own = False

DEV = "cuda"
CHUNK = 64            # tokens a chunk of the plain delta rule
NORM_EPS = 1e-6       # of the key and query lengths
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one user's next token: the convolution of the mixer's 16 query, 16
        # key and 32 value heads of 128 channels; nothing but latency
        dict(name="conv_step_one", op="conv_step", dtype="bf16", rows=1, C=8192, K=4, act="silu"),
        # prefill and training of packed prompts
        dict(name="conv_fwd_packed", op="conv_fwd", dtype="bf16", tokens=16384, seqs=7, C=8192, K=4,
             act="silu", state=True),
        # training in fp32 with an odd channel count (no 16-byte rows) and a
        # filter of three taps
        dict(name="conv_bwd_odd", op="conv_bwd", dtype="f32", tokens=8191, seqs=3, C=2049, K=3,
             act="silu", state=True),
        # training of packed documents, the mixer's channels
        dict(name="conv_bwd_packed", op="conv_bwd", dtype="bf16", tokens=8192, seqs=4, C=8192, K=4,
             act="silu", state=False),
        # one user's next token
        dict(name="delta_step_one", op="delta_step", dtype="bf16", rows=1, Hk=16, Hv=32, Dk=128,
             Dv=128),
        # a full serving batch, one token per sequence
        dict(name="delta_step_batch", op="delta_step", dtype="bf16", rows=96, Hk=16, Hv=32, Dk=128,
             Dv=128),
        # prefill of packed prompts, continued from a cache
        dict(name="delta_fwd_packed", op="delta_fwd", dtype="bf16", tokens=8192, seqs=5, Hk=16, Hv=32,
             Dk=128, Dv=128, state=True),
        # one long document: only heads and value columns are parallel
        dict(name="delta_fwd_long", op="delta_fwd", dtype="f16", tokens=5003, seqs=1, Hk=6, Hv=6,
             Dk=96, Dv=104, state=False),
        # a training step
        dict(name="delta_bwd_packed", op="delta_bwd", dtype="bf16", tokens=4096, seqs=4, Hk=8, Hv=16,
             Dk=128, Dv=128, state=True),
        # the mixer's gated norm: every head of every token is a row
        dict(name="norm_fwd_heads", op="norm_fwd", dtype="bf16", rows=262144, D=128, after="rms",
             act="silu", per=1, residual=False, scale=False, before="none"),
        # between two blocks of a transformer of 4096 channels
        dict(name="norm_fwd_block", op="norm_fwd", dtype="bf16", rows=8192, D=4096, after="rms",
             act="none", per=0, residual=True, scale=True, before="rms"),
        # training of a channel-last image block of 96 channels at 56x56:
        # LayerNorm, one sigmoid gate per image, layer scale, residual
        dict(name="norm_bwd_image", op="norm_bwd", dtype="f16", rows=64 * 56 * 56, D=96, after="layer",
             act="sigmoid", per=56 * 56, residual=True, scale=True, before="layer"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_step", "conv_bwd", "delta_fwd", "delta_step", "delta_bwd",
                     "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("conv"):
        c = dict(op=op, dtype=dtype, C=_spread(rng, 16, 8192), K=rng.randint(2, 6),
                 act=rng.choice(["silu", "none"]))
        if op == "conv_step":
            return dict(c, rows=_spread(rng, 1, 256))
        return dict(c, tokens=_spread(rng, 1, 8192), seqs=rng.randint(1, 9),
                    state=rng.random() < 0.5)
    if op.startswith("delta"):
        hk = rng.choice([1, 2, 3, 4, 8])
        c = dict(op=op, dtype=dtype, Hk=hk, Hv=hk * rng.choice([1, 2, 3]),
                 Dk=rng.choice([64, 128, _spread(rng, 16, 192)]),
                 Dv=rng.choice([64, 128, _spread(rng, 16, 192)]))
        if op == "delta_step":
            return dict(c, rows=_spread(rng, 1, 128))
        return dict(c, tokens=_spread(rng, 1, 4096 if op == "delta_fwd" else 2048),
                    seqs=rng.randint(1, 6), state=rng.random() < 0.5)
    d = _spread(rng, 32, 8192)
    rows = _spread(rng, 1, min(65536, 2 ** 25 // d))
    act = rng.choice(["none", "silu", "sigmoid"])
    return dict(op=op, dtype=dtype, rows=rows, D=d, after=rng.choice(["rms", "layer", "none"]),
                act=act, per=rng.choice([0, 1, max(1, rows // 5)]) if act == "none"
                else rng.choice([1, max(1, rows // 5)]),
                residual=rng.random() < 0.7, scale=rng.random() < 0.5,
                before=rng.choice(["rms", "layer"]))


def _lengths(tokens, seqs):
    """Ragged lengths that add up to ``tokens``: uneven shares, the same for
    every seed."""
    seqs = max(1, min(seqs, tokens))
    rng = random.Random(1000003 * seqs + tokens)
    share = [rng.uniform(0.5, 1.5) for _ in range(seqs)]
    cut = [0]
    for i in range(seqs):
        cut.append(tokens if i + 1 == seqs else int(tokens * sum(share[:i + 1]) / sum(share)))
    return [b - a for a, b in zip(cut, cut[1:])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device=DEV) * std + mean).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=gen, device=DEV) * (hi - lo) + lo

    op, s = case["op"], {"case": case, "op": case["op"]}
    if op.endswith("_step"):
        rows = case["rows"]
        slots = rows + 3  # the cache has room for more sequences than run now
        s["slots"] = torch.randperm(slots, generator=gen, device=DEV)[:rows].to(torch.int32)
    elif "tokens" in case:
        s["lens"] = _lengths(case["tokens"], case["seqs"])
        off = [0]
        for n in s["lens"]:
            off.append(off[-1] + n)
        s["offsets"] = torch.tensor(off, dtype=torch.int32, device=DEV)
        B, T = len(s["lens"]), case["tokens"]

    if op.startswith("conv"):
        C, K = case["C"], case["K"]
        s["w"] = normal(K, C, std=1.0 / math.sqrt(K))
        s["bias"] = normal(C, std=0.1, dtype=torch.float32)
        if op == "conv_step":
            s["x"] = normal(rows, C)
            s["state"] = normal(slots, K - 1, C)
        else:
            s["x"] = normal(T, C)
            s["state_in"] = normal(B, K - 1, C) if case["state"] else None
            if op == "conv_bwd":
                s["dy"] = normal(T, C)
    elif op.startswith("delta"):
        Hk, Hv, Dk, Dv = (case[n] for n in ("Hk", "Hv", "Dk", "Dv"))
        n = rows if op == "delta_step" else T
        # the convolution's output, queries, keys and values side by side
        mixed = torch.nn.functional.silu(normal(n, 2 * Hk * Dk + Hv * Dv, dtype=torch.float32)).to(dt)
        q, k, v = mixed.split([Hk * Dk, Hk * Dk, Hv * Dv], dim=1)
        s["q"], s["k"], s["v"] = q.unflatten(1, (Hk, Dk)), k.unflatten(1, (Hk, Dk)), v.unflatten(1, (Hv, Dv))
        rate = uniform(Hv, lo=0.0, hi=4.0)  # heads that forget slowly and heads that forget fast
        s["g"] = -rate * torch.nn.functional.softplus(normal(n, Hv, std=1.0, mean=-2.0, dtype=torch.float32))
        s["beta"] = torch.sigmoid(normal(n, Hv, dtype=torch.float32))
        if op == "delta_step":
            s["state"] = normal(slots, Hv, Dk, Dv, std=0.3, dtype=torch.float32)
        else:
            s["state_in"] = normal(B, Hv, Dk, Dv, std=0.3, dtype=torch.float32) if case["state"] else None
            if op == "delta_bwd":
                s["do"] = normal(T, Hv, Dv)
                s["dstate_out"] = normal(B, Hv, Dk, Dv, std=0.1, dtype=torch.float32) if case["state"] else None
    else:
        R, D, per = case["rows"], case["D"], case["per"]
        s["o"] = normal(R, D, mean=0.1)
        s["residual"] = normal(R, D) if case["residual"] else None
        s["gate"] = normal(-(-R // per), D) if per else None
        s["scale"] = uniform(D, lo=0.1, hi=0.5) if case["scale"] else None
        for side in ("after", "before"):
            kind = case[side]
            s["w_" + side] = uniform(D, lo=0.5, hi=1.5) if kind != "none" else None
            s["b_" + side] = normal(D, std=0.1, dtype=torch.float32) if kind == "layer" else None
        if op == "norm_bwd":
            s["dh"], s["dy"] = normal(R, D), normal(R, D)
    if own:
        import depthwise_convolution_amd as dw
        if op.startswith("conv"):
            s["plan"] = dw.CausalDepthwiseConv1d(case["C"], case["K"], case["dtype"], act=case["act"])
        elif op.startswith("delta"):
            s["plan"] = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, case["dtype"], normalize=True, eps=NORM_EPS)
        else:
            s["plan"] = dw.BlockNorm(case["D"], case["dtype"], after=case["after"], before=case["before"],
                                     gate_act=case["act"])
    return s


def work(case):
    e, op = BYTES[case["dtype"]], case["op"]
    if op.startswith("conv"):
        C, K = case["C"], case["K"]
        if op == "conv_step":
            n = case["rows"] * C
            return {"bytes": e * (2 * n + 2 * n * (K - 1) + K * C) + 4 * C, "flops": 2 * K * n}
        n, st = case["tokens"] * C, (K - 1) * C * min(case["seqs"], case["tokens"])
        if op == "conv_fwd":
            return {"bytes": e * (2 * n + K * C + st * (2 if case["state"] else 1)) + 4 * C,
                    "flops": 2 * K * n}
        return {"bytes": e * (3 * n + K * C + (2 * st if case["state"] else 0)) + 4 * C * (K + 2),
                "flops": 6 * K * n}
    if op.startswith("delta"):
        Hk, Hv, Dk, Dv = (case[n] for n in ("Hk", "Hv", "Dk", "Dv"))
        n = case["rows"] if op == "delta_step" else case["tokens"]
        mat = Hv * Dk * Dv
        io = e * n * (2 * Hk * Dk + 2 * Hv * Dv) + 8 * n * Hv
        if op == "delta_step":
            return {"bytes": io + 8 * n * mat, "flops": 6 * n * mat}
        seqs = min(case["seqs"], n)
        if op == "delta_fwd":
            return {"bytes": io + 4 * seqs * mat * (2 if case["state"] else 1), "flops": 6 * n * mat}
        return {"bytes": 2 * io + (12 * seqs * mat if case["state"] else 0), "flops": 18 * n * mat}
    R, D, per = case["rows"], case["D"], case["per"]
    n, gate = R * D, (-(-R // per) * D if per else 0)
    params = D * ((1 if case["scale"] else 0) + sum({"none": 0, "rms": 1, "layer": 2}[case[s]]
                                                    for s in ("after", "before")))
    res = 1 if case["residual"] else 0
    if op == "norm_fwd":
        return {"bytes": e * (n * (2 + res + (case["before"] != "none")) + gate) + 4 * params, "flops": 16 * n}
    return {"bytes": e * (n * (4 + 2 * res) + 2 * gate) + 8 * params, "flops": 40 * n}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    op, plan, case = s["op"], s["plan"], s["case"]
    if op == "conv_fwd":
        state = torch.empty((len(s["lens"]), case["K"] - 1, case["C"]), device=DEV, dtype=s["x"].dtype)
        y = plan(s["x"], s["w"], s["bias"], offsets=s["offsets"], state_in=s["state_in"], state_out=state)
        return {"y": y, "state": state}
    if op == "conv_step":
        y = plan.step(s["x"], s["w"], s["bias"], state=s["state"], slots=s["slots"])
        return {"y": y, "state": s["state"]}
    if op == "conv_bwd":
        dx, dw, dbias, dstate = plan.backward(s["x"], s["w"], s["dy"], s["bias"], offsets=s["offsets"],
                                              state_in=s["state_in"])
        return {"dx": dx, "dw": dw, "dbias": dbias, "dstate": dstate}
    if op == "delta_fwd":
        state = torch.empty((len(s["lens"]), case["Hv"], case["Dk"], case["Dv"]), device=DEV)
        o = plan(s["q"], s["k"], s["v"], s["g"], s["beta"], offsets=s["offsets"], state_in=s["state_in"],
                 state_out=state)
        return {"o": o, "state": state}
    if op == "delta_step":
        o = plan.step(s["q"], s["k"], s["v"], s["g"], s["beta"], state=s["state"], slots=s["slots"])
        return {"o": o, "state": s["state"]}
    if op == "delta_bwd":
        dq, dk, dv, dg, dbeta, dstate = plan.backward(
            s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], offsets=s["offsets"],
            state_in=s["state_in"], dstate_out=s["dstate_out"])
        return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta, "dstate": dstate}
    names = ("residual", "gate", "scale", "w_after", "b_after", "w_before", "b_before")
    args = {n: s[n] for n in names}
    per = max(1, case["per"])
    if op == "norm_fwd":
        h, y = plan(s["o"], rows_per_gate=per, **args)
        return {"h": h, "y": y}
    grads = plan.backward(s["o"], s["dh"], s["dy"], rows_per_gate=per, **args)
    return dict(zip(("do",) + names, grads))


def _run_plain(s):
    op, case = s["op"], s["case"]
    dt = DTYPES[case["dtype"]]
    if op == "conv_fwd":
        y, state = _conv_plain(s["x"].float(), s["w"].float(), s["bias"], s["offsets"],
                               None if s["state_in"] is None else s["state_in"].float(), case["act"])
        return {"y": y.to(dt), "state": state.to(dt)}
    if op == "conv_step":
        at = s["slots"].long()
        window = torch.cat([s["state"][at], s["x"][:, None]], dim=1)
        z = (window.float() * s["w"].float()).sum(1) + s["bias"]
        s["state"][at] = window[:, 1:]
        return {"y": (z * torch.sigmoid(z) if case["act"] == "silu" else z).to(dt), "state": s["state"]}
    if op == "conv_bwd":
        leaves = [s["x"].float(), s["w"].float(), s["bias"].clone()]
        if s["state_in"] is not None:
            leaves.append(s["state_in"].float())
        leaves = [t.detach().requires_grad_() for t in leaves]
        y, _ = _conv_plain(leaves[0], leaves[1], leaves[2], s["offsets"],
                           leaves[3] if len(leaves) == 4 else None, case["act"])
        grads = torch.autograd.grad(y, leaves, s["dy"].float())
        return {"dx": grads[0].to(dt), "dw": grads[1], "dbias": grads[2],
                "dstate": grads[3].to(dt) if len(leaves) == 4 else None}
    if op == "delta_fwd":
        o, state = _delta_plain(s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["beta"], s["offsets"],
                                max(s["lens"]), s["state_in"])
        return {"o": o.to(dt), "state": state}
    if op == "delta_step":
        at = s["slots"].long()
        q, k = _unit(s["q"].float()) / math.sqrt(case["Dk"]), _unit(s["k"].float())
        group = case["Hv"] // case["Hk"]
        q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
        S = s["state"][at] * torch.exp(s["g"])[..., None, None]
        u = s["beta"][..., None] * (s["v"].float() - (S * k[..., None]).sum(-2))
        S = S + k[..., None] * u[..., None, :]
        s["state"][at] = S
        return {"o": (S * q[..., None]).sum(-2).to(dt), "state": s["state"]}
    if op == "delta_bwd":
        leaves = [s["q"].float(), s["k"].float(), s["v"].float(), s["g"].clone(), s["beta"].clone()]
        if s["state_in"] is not None:
            leaves.append(s["state_in"].clone())
        leaves = [t.detach().requires_grad_() for t in leaves]
        o, state = _delta_plain(*leaves[:5], s["offsets"], max(s["lens"]), leaves[5] if len(leaves) == 6 else None)
        outs, gives = [o], [s["do"].float()]
        if s["dstate_out"] is not None:
            outs, gives = outs + [state], gives + [s["dstate_out"]]
        grads = torch.autograd.grad(outs, leaves, gives)
        return {"dq": grads[0].to(dt), "dk": grads[1].to(dt), "dv": grads[2].to(dt), "dg": grads[3],
                "dbeta": grads[4], "dstate": grads[5] if len(leaves) == 6 else None}
    names = ("residual", "gate", "scale", "w_after", "b_after", "w_before", "b_before")
    if op == "norm_fwd":
        h, y = _norm_plain(case, s["o"].float(), *(None if s[n] is None else s[n].float() for n in names))
        return {"h": h.to(dt), "y": None if y is None else y.to(dt)}
    leaves = {n: s[n].float().clone().requires_grad_() for n in ("o",) + names if s[n] is not None}
    h, y = _norm_plain(case, *(leaves.get(n) for n in ("o",) + names))
    outs, gives = ([h], [s["dh"].float()]) if y is None else ([h, y], [s["dh"].float(), s["dy"].float()])
    grads = dict(zip(leaves, torch.autograd.grad(outs, list(leaves.values()), gives)))
    return {"do" if n == "o" else n: (grads[n].to(s[n].dtype) if n in grads else None) for n in ("o",) + names}


def _conv_plain(x, w, bias, offsets, state, act):
    K, T = w.shape[0], x.shape[0]
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(offsets[1:].contiguous(), t, right=True)
    pos = t - offsets[seq]
    z = bias.expand(T, -1)
    for k in range(K):
        back = K - 1 - k
        xk = torch.where((pos >= back)[:, None], x[(t - back).clamp_min(0)], 0.0)
        if state is not None and back:
            early = (pos < back).nonzero()[:, 0]
            xk = xk.index_put((early,), state[seq[early], pos[early] + k])
        z = z + w[k] * xk
    r = torch.arange(K - 1, device=DEV)
    at = (offsets[1:] - offsets[:-1])[:, None] + r  # rows of [state; x]
    last = x[(offsets[:-1, None] + at - (K - 1)).clamp(0, T - 1)]
    old = torch.zeros_like(last) if state is None else state[torch.arange(len(offsets) - 1, device=DEV)[:, None],
                                                              at.clamp_max(K - 2)]
    return (z * torch.sigmoid(z) if act == "silu" else z), torch.where((at >= K - 1)[..., None], last, old)


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + NORM_EPS)


def _delta_plain(q, k, v, g, beta, offsets, longest, state):
    """The gated delta rule, CHUNK tokens at a time, on the sequences padded to one length."""
    B, Hk, Hv, Dk, Dv = len(offsets) - 1, k.shape[1], v.shape[1], k.shape[2], v.shape[2]
    n = -(-longest // CHUNK)
    pos = torch.arange(n * CHUNK, device=DEV)
    live = pos < (offsets[1:] - offsets[:-1])[:, None]
    at = (offsets[:-1, None] + pos).clamp_max(q.shape[0] - 1)

    def pad(x):  # [T, H, ...] -> [B, H, n, CHUNK, ...], zeros behind each sequence
        x = torch.where(live.view(B, -1, *[1] * (x.dim() - 1)), x[at], 0.0)
        x = x if x.shape[2] == Hv else x.repeat_interleave(Hv // Hk, 2)
        return x.transpose(1, 2).unflatten(2, (n, CHUNK))

    q, k, v, g, beta = pad(_unit(q) / math.sqrt(Dk)), pad(_unit(k)), pad(v), pad(g), pad(beta)
    b = g.double().cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, device=DEV, dtype=torch.bool).tril()
    decay = torch.exp((b[..., :, None] - b[..., None, :]).masked_fill(~lower, -math.inf)).float()
    A = (beta[..., None] * decay * (k @ k.transpose(-1, -2).contiguous())).tril(-1)
    inv = torch.eye(CHUNK, device=DEV).expand_as(A)
    i, size = torch.arange(CHUNK, device=DEV), 1
    while size < CHUNK:  # the inverse of 1 + A by blocks of twice the size
        block = (i[:, None] // size == i // size + 1) & (i[:, None] // size % 2 == 1)
        inv = inv - inv @ (A * block) @ inv
        size *= 2
    P = decay * (q @ k.transpose(-1, -2).contiguous())
    left, right = torch.exp(b).float()[..., None], torch.exp(b[..., -1:] - b).float()[..., None]
    S = torch.zeros(B, Hv, Dk, Dv, device=DEV) if state is None else state
    out = []
    for c in range(n):
        kc, rc = k[:, :, c], left[:, :, c]
        u = inv[:, :, c] @ (beta[:, :, c, :, None] * (v[:, :, c] - rc * (kc @ S)))
        out.append(rc * (q[:, :, c] @ S) + P[:, :, c] @ u)
        S = rc[:, :, -1:] * S + kc.transpose(-1, -2).contiguous() @ (right[:, :, c] * u)
    o = torch.stack(out, 2).flatten(2, 3).transpose(1, 2)
    return o[live], S


def _normed(x, kind, w, b):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * w
    return x if b is None else x + b


def _norm_plain(case, o, residual, gate, scale, w_after, b_after, w_before, b_before):
    t = _normed(o, case["after"], w_after, b_after)
    if gate is not None:
        act = {"none": lambda x: x, "silu": lambda x: x * torch.sigmoid(x), "sigmoid": torch.sigmoid}[case["act"]]
        row = torch.arange(o.shape[0], device=DEV) // case["per"]
        t = t * act(gate if case["per"] == 1 else gate[row])
    t = t if scale is None else t * scale
    h = t if residual is None else residual + t
    return h, None if case["before"] == "none" else _normed(h, case["before"], w_before, b_before)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"].startswith("conv"):
            return _conv_exact(s)
        if case["op"].startswith("delta"):
            return _delta_exact(s)
        return _norm_exact(s)


def _silu_and_slope(z):
    p = 1 / (1 + torch.exp(-z))
    return z * p, p * (1 + z * (1 - p))


def _conv_exact(s):
    case, K = s["case"], s["case"]["K"]
    x, w, bias = s["x"].double(), s["w"].double(), s["bias"].double()
    if s["op"] == "conv_step":
        state = s["state"].double()
        y = torch.empty_like(x)
        for i, slot in enumerate(s["slots"].tolist()):
            rows = torch.cat([state[slot], x[i:i + 1]])
            z = bias + (rows * w).sum(0)
            y[i] = _silu_and_slope(z)[0] if case["act"] == "silu" else z
            state[slot] = rows[1:]
        return {"y": y, "state": state}
    C, start, ys, states = case["C"], 0, [], []
    dxs, dw, dbias, dstates = [], torch.zeros_like(w), torch.zeros_like(bias), []
    for i, n in enumerate(s["lens"]):
        old = torch.zeros(K - 1, C, device=DEV, dtype=torch.float64) if s["state_in"] is None else s["state_in"][i].double()
        ext = torch.cat([old, x[start:start + n]])
        z = bias + sum(w[k] * ext[k:k + n] for k in range(K))
        y, slope = _silu_and_slope(z) if case["act"] == "silu" else (z, torch.ones_like(z))
        ys.append(y)
        states.append(ext[n:])
        if s["op"] == "conv_bwd":
            dz = s["dy"][start:start + n].double() * slope
            dext = torch.zeros_like(ext)
            for k in range(K):
                dext[k:k + n] += w[k] * dz
                dw[k] += (dz * ext[k:k + n]).sum(0)
            dbias += dz.sum(0)
            dxs.append(dext[K - 1:])
            dstates.append(dext[:K - 1])
        start += n
    if s["op"] == "conv_fwd":
        return {"y": torch.cat(ys), "state": torch.stack(states)}
    return {"dx": torch.cat(dxs), "dw": dw, "dbias": dbias,
            "dstate": None if s["state_in"] is None else torch.stack(dstates)}


def _delta_exact(s):
    """Token by token, each sequence a row of a batch; the gradients by the
    recurrence run backwards over the kept states."""
    case = s["case"]
    Hk, Hv, Dk, Dv = (case[n] for n in ("Hk", "Hv", "Dk", "Dv"))
    G = Hv // Hk
    step = s["op"] == "delta_step"
    lens = [1] * case["rows"] if step else s["lens"]
    B, L = len(lens), max(lens)
    back = s["op"] == "delta_bwd"
    if back and 8 * L * B * Hv * Dk * Dv > 48 * 2 ** 30:
        return None
    starts = [sum(lens[:i]) for i in range(B)]

    def pad(x):  # [T, ...] -> [L, B, ...]
        out = torch.zeros((L, B) + tuple(x.shape[1:]), device=DEV, dtype=torch.float64)
        for i in range(B):
            out[:lens[i], i] = x[starts[i]:starts[i] + lens[i]]
        return out

    def unpad(x):
        return torch.cat([x[:lens[i], i] for i in range(B)])

    q0, k0, v, g, beta = (pad(s[n]) for n in ("q", "k", "v", "g", "beta"))
    rq = ((q0 ** 2).sum(-1, keepdim=True) + NORM_EPS) ** -0.5
    rk = ((k0 ** 2).sum(-1, keepdim=True) + NORM_EPS) ** -0.5
    grow = lambda x: x.repeat_interleave(G, 2)  # noqa: E731
    q, k = grow(q0 * rq) * Dk ** -0.5, grow(k0 * rk)
    if step:
        whole = s["state"].double()
        S = whole[s["slots"].long()]
    elif s["state_in"] is None:
        S = torch.zeros(B, Hv, Dk, Dv, device=DEV, dtype=torch.float64)
    else:
        S = s["state_in"].double()
    o, kept = torch.empty_like(v), [S]
    fade = torch.exp(g)
    for t in range(L):
        S = S * fade[t][..., None, None]
        u = beta[t][..., None] * (v[t] - torch.einsum("bhkv,bhk->bhv", S, k[t]))
        S = S + torch.einsum("bhk,bhv->bhkv", k[t], u)
        o[t] = torch.einsum("bhkv,bhk->bhv", S, q[t])
        if back:
            kept.append(S)
    if step:
        whole[s["slots"].long()] = S
        return {"o": unpad(o), "state": whole}
    if not back:
        return {"o": unpad(o), "state": S}
    do = pad(s["do"])
    dS = torch.zeros_like(S) if s["dstate_out"] is None else s["dstate_out"].double()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(g), torch.empty_like(beta)
    for t in reversed(range(L)):
        faded = kept[t] * fade[t][..., None, None]
        miss = v[t] - torch.einsum("bhkv,bhk->bhv", faded, k[t])
        dq[t] = torch.einsum("bhkv,bhv->bhk", kept.pop(), do[t])
        dS = dS + torch.einsum("bhk,bhv->bhkv", q[t], do[t])
        du = torch.einsum("bhkv,bhk->bhv", dS, k[t])
        dm = beta[t][..., None] * du
        dv[t], dbeta[t] = dm, (du * miss).sum(-1)
        dk[t] = torch.einsum("bhkv,bhv->bhk", dS, beta[t][..., None] * miss) - torch.einsum("bhkv,bhv->bhk", faded, dm)
        dS = dS - torch.einsum("bhk,bhv->bhkv", k[t], dm)
        dg[t] = (dS * faded).sum((-1, -2))
        dS = dS * fade[t][..., None, None]

    def through(d, x, r, scale):  # heads that share a key, and the unit length
        d = d.unflatten(2, (Hk, G)).sum(3) * scale
        unit = x * r
        return r * (d - unit * (unit * d).sum(-1, keepdim=True))

    return {"dq": unpad(through(dq, q0, rq, Dk ** -0.5)), "dk": unpad(through(dk, k0, rk, 1.0)), "dv": unpad(dv),
            "dg": unpad(dg), "dbeta": unpad(dbeta), "dstate": None if s["state_in"] is None else dS}


def _norm_exact(s):
    case, D, per = s["case"], s["case"]["D"], s["case"]["per"]
    get = lambda n: None if s[n] is None else s[n].double()  # noqa: E731
    o, res, gate, scale = get("o"), get("residual"), get("gate"), get("scale")

    def norm(x, kind, w, b):
        if kind == "none":
            return x, None, None
        c = x - x.mean(-1, keepdim=True) if kind == "layer" else x
        r = (c.square().sum(-1, keepdim=True) / D + NORM_EPS) ** -0.5
        return c * r * w + (0 if b is None else b), c * r, r

    def norm_back(dy, kind, w, unit, r):  # dx, dw, db
        if kind == "none":
            return dy, None, None
        d = dy * w
        dx = d - unit * (unit * d).mean(-1, keepdim=True)
        if kind == "layer":
            dx = dx - d.mean(-1, keepdim=True)
        return r * dx, (dy * unit).sum(0), dy.sum(0)

    n, unit_a, r_a = norm(o, case["after"], get("w_after"), get("b_after"))
    if gate is None:
        a = slope = torch.ones((), device=DEV, dtype=torch.float64)
    elif case["act"] == "none":
        a, slope = gate, torch.ones_like(gate)
    elif case["act"] == "silu":
        a, slope = _silu_and_slope(gate)
    else:
        a = 1 / (1 + torch.exp(-gate))
        slope = a * (1 - a)
    spread = lambda x: x if per <= 1 else x.repeat_interleave(per, 0)[:case["rows"]]  # noqa: E731
    c = 1.0 if scale is None else scale
    t = n * spread(a)
    h = t * c + (0 if res is None else res)
    y, unit_b, r_b = norm(h, case["before"], get("w_before"), get("b_before"))
    if s["op"] == "norm_fwd":
        return {"h": h, "y": None if case["before"] == "none" else y}
    dh = s["dh"].double()
    dw_b = db_b = None
    if case["before"] != "none":
        back, dw_b, db_b = norm_back(s["dy"].double(), case["before"], get("w_before"), unit_b, r_b)
        dh = dh + back
    dscale = None if scale is None else (dh * t).sum(0)
    dt = dh * c
    dgate = None
    if gate is not None:
        dgate = dt * n * spread(slope)
        if per > 1:
            short = gate.shape[0] * per - case["rows"]
            dgate = torch.nn.functional.pad(dgate, (0, 0, 0, short)).unflatten(0, (-1, per)).sum(1)
    do, dw_a, db_a = norm_back(dt * spread(a), case["after"], get("w_after"), unit_a, r_a)
    return {"do": do, "residual": None if res is None else dh, "gate": dgate, "scale": dscale, "w_after": dw_a,
            "b_after": db_a if s["b_after"] is not None else None, "w_before": dw_b,
            "b_before": db_b if s["b_before"] is not None else None}
