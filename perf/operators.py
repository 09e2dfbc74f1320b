"""Cases, plain forms and exact values of the gated delta rule and the state cache.

The gated delta rule is the linear recurrence next to the SSD scan whose update
erases before it writes.  Per sequence and head h (group h // (nheads / ngroups)),
with the state S of shape (headdim, dstate):

    S_t = exp(g_t) S_{t-1} + beta_t (v_t - exp(g_t) S_{t-1} k_t) k_t^T
    o_t = scale S_t q_t

Three operators are timed: its chunked form over whole sequences (forward, and
forward with the gradients), its recurrent form over the few tokens of a decode
step, on states held in a slotted cache, and the 8-bit cache that parks states
(quantised as they are written, and read back).

``own`` chooses between the plain form (elementary torch operations) and the
framework's calls; ``exact`` evaluates the definition in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64  # tokens per chunk of the plain form


# ------------------------------------------------------------------ cases ----
def listed():
    delta = dict(batch=1, heads=64, groups=8, headdim=64, dstate=128, io="bf16", lens="", init=False)
    step = dict(kind="step", heads=64, groups=8, headdim=64, dstate=128, io="bf16", tokens=1, slots=0, pad=0)
    return [
        # one short prompt: launches and the chain of chunks count, not bandwidth
        dict(delta, name="prefill_short", kind="fwd", seqlen=100, heads=32, groups=4),
        # continued prompts of a serving batch, packed, one empty and one of one token
        dict(delta, name="prefill_packed", kind="fwd", seqlen=8191, init=True, lens="1203,0,517,1,4096,63,2000,311"),
        # one long document
        dict(delta, name="prefill_long", kind="fwd", seqlen=131072, heads=32, groups=4, init=True),
        # fp32 activations, an odd length, heads with their own keys
        dict(delta, name="prefill_f32", kind="fwd", batch=2, seqlen=1001, heads=16, groups=16, headdim=128, dstate=64,
             io="f32", init=True),
        # a layer's training step at the size that the framework's benchmark uses
        dict(delta, name="train_layer", kind="train", batch=2, seqlen=8192),
        # a packed training batch with square heads and carried states
        dict(delta, name="train_packed", kind="train", seqlen=4099, heads=16, groups=4, headdim=128, init=True,
             lens="1000,1,1777,0,1321"),
        # a small fp32 problem, as a gradient check runs
        dict(delta, name="train_f32_small", kind="train", seqlen=256, heads=4, groups=1, headdim=16, dstate=16,
             io="f32", init=True),
        # one user's next token
        dict(step, name="step_one", batch=1),
        # a full decode batch with states anywhere in the cache, some rows of it padding
        dict(step, name="step_batch", batch=256, slots=320, pad=6),
        # drafted tokens of several users run through the recurrence at once
        dict(step, name="step_draft", batch=24, tokens=5, heads=32, groups=16, headdim=128, slots=32),
        # one layer's states of a few users parked in 8 bits and taken up again
        dict(name="park_int8", kind="cache", batch=4, heads=64, headdim=64, dstate=128, slots=16, format="int8"),
        # many users' states with square heads, as 8-bit floating point
        dict(name="park_e4m3", kind="cache", batch=96, heads=32, headdim=128, dstate=128, slots=128, format="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("fwd", "fwd", "train", "train", "step", "cache"))
    groups = rng.choice((1, 2, 4, 8, 16))
    heads = groups * rng.choice((1, 2, 4, 8) if groups <= 8 else (1, 2, 4))
    headdim, dstate = rng.choice((16, 32, 64, 128)), rng.choice((16, 32, 64, 128))
    if kind == "cache":
        batch = _log(rng, 1, 128)
        return dict(kind=kind, batch=batch, heads=heads, headdim=headdim, dstate=dstate,
                    slots=batch + rng.randrange(0, 40), format=rng.choice(("int8", "e4m3")))
    io = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if kind == "step":
        batch = _log(rng, 1, 200)
        return dict(kind=kind, batch=batch, heads=heads, groups=groups, headdim=headdim, dstate=dstate, io=io,
                    tokens=rng.choice((1, 1, 1, 2, 3, 4, 6, 8)), slots=batch + rng.randrange(1, 40),
                    pad=rng.randrange(0, 1 + batch // 8))
    case = dict(kind=kind, batch=1, seqlen=_log(rng, 1, 12000), heads=heads, groups=groups, headdim=headdim,
                dstate=dstate, io=io, lens="", init=rng.random() < 0.5)
    if rng.random() < 0.5:
        cuts = sorted(rng.randrange(0, case["seqlen"] + 1) for _ in range(rng.randrange(1, 9)))
        ends = cuts + [case["seqlen"]]
        case["lens"] = ",".join(str(b - a) for a, b in zip([0] + cuts, ends))
    elif case["seqlen"] < 4000:
        case["batch"] = rng.randrange(1, 5)
    return case


def work(case):
    c = case
    state = c["heads"] * c["headdim"] * c["dstate"]
    if c["kind"] == "cache":  # fp32 in, codes out, codes in, fp32 out; two scales of a row; an absolute value and a product
        n = c["batch"] * state
        return {"bytes": n * 10 + 4 * 4 * n // c["dstate"], "flops": 4 * n}
    io = 2 if c["io"] == "bf16" else 4
    qk, vo, gates = 2 * c["groups"] * c["dstate"] * io, 2 * c["heads"] * c["headdim"] * io, 8 * c["heads"]
    if c["kind"] == "step":  # live rows alone move anything
        live = c["batch"] - c["pad"]
        n = live * c["tokens"]
        return {"bytes": n * (qk + vo + gates) + live * state * 8, "flops": 6 * n * state}
    n = c["batch"] * c["seqlen"]
    nst = len(c["lens"].split(",")) if c["lens"] else c["batch"]
    states = nst * state * 4 * (2 if c["init"] else 1)
    if c["kind"] == "fwd":
        return {"bytes": n * (qk + vo + gates) + states, "flops": 6 * n * state}
    # gradients: q, k, v, dout in and dq, dk, dv out once more, the gates' gradients, both states' gradients
    return {"bytes": n * (3 * qk + 5 * vo // 2 + 2 * gates) + 2 * states, "flops": 18 * n * state}


# ----------------------------------------------------------------- inputs ----
def _dtype(case):
    return torch.float32 if case["io"] == "f32" else torch.bfloat16


def _tokens(c, L, gen):
    """q, k (unit rows, from an activation that leaves them correlated), v, and the gates:
    steps softplus(N(0,1) + U[-4,-2]) times -A with A log-uniform on [1, 16], beta a sigmoid."""
    dev, b, io = "cuda", c["batch"], _dtype(c)
    rand = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    silu = lambda x: x * torch.sigmoid(x)  # noqa: E731
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    q = unit(silu(rand(b, L, c["groups"], c["dstate"]))).to(io)
    k = unit(silu(rand(b, L, c["groups"], c["dstate"]))).to(io)
    v = silu(rand(b, L, c["heads"], c["headdim"])).to(io)
    bias = torch.rand(c["heads"], generator=gen, device=dev) * 2 - 4
    a = torch.exp(torch.rand(c["heads"], generator=gen, device=dev) * math.log(16.0))
    g = -a * torch.log1p(torch.exp(rand(b, L, c["heads"]) + bias))
    beta = torch.sigmoid(1.5 * rand(b, L, c["heads"]))
    return dict(q=q, k=k, v=v, g=g, beta=beta)


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    if c["kind"] == "cache":
        shape = (c["batch"], c["heads"], c["headdim"], c["dstate"])
        states = rand(*shape) * torch.exp(rand(*shape[:3], 1))
        states[0, 0, 0] = 0.0  # a row that nothing was written to
        slots = torch.randperm(c["slots"], generator=gen, device=dev)[: c["batch"]].to(torch.int32)
        code = torch.int8 if c["format"] == "int8" else torch.float8_e4m3fn
        codes = torch.zeros(c["slots"], *shape[1:], device=dev, dtype=torch.int8).view(code)
        return dict(case=c, states=states, slots=slots, codes=codes,
                    scales=torch.zeros(c["slots"], *shape[1:3], device=dev))
    if c["kind"] == "step":
        s = dict(_tokens(c, c["tokens"], gen), case=c)
        n = c["slots"] or c["batch"]
        s["states"] = 0.3 * rand(n, c["heads"], c["headdim"], c["dstate"])
        s["slots"], s["out"] = None, torch.zeros_like(s["v"])
        if c["slots"]:
            at = torch.randperm(n, generator=gen, device=dev)[: c["batch"]].to(torch.int32)
            at[c["batch"] - c["pad"]:] = -1  # padding rows of a batch of fixed size
            s["slots"] = at
        return s
    s = dict(_tokens(c, c["seqlen"], gen), case=c, cu=None)
    nst = c["batch"]
    if c["lens"]:
        lens = [int(n) for n in c["lens"].split(",")]
        nst = len(lens)
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(nst + 1)], dtype=torch.int32, device=dev)
    shape = (nst, c["heads"], c["headdim"], c["dstate"])
    s["init"] = 0.3 * rand(*shape) if c["init"] else None
    if c["kind"] == "train":
        s["dout"] = rand(*s["v"].shape).to(_dtype(c))
        s["d_final"] = 0.3 * rand(*shape) if c["init"] else None
    return s


# ------------------------------------------------------------------- runs ----
def run(state):
    s, c = state, state["case"]
    if c["kind"] == "cache":
        return _run_cache(s)
    scale = c["dstate"] ** -0.5
    if c["kind"] == "step":
        return _run_step(s, scale)
    if own:
        from mamba_ssd_chunked_03_amd import ssd
        args = (s["q"], s["k"], s["v"], s["g"], s["beta"])
        if c["kind"] == "fwd":
            out, final = ssd.delta_fwd(*args, scale=scale, init=s["init"], cu_seqlens=s["cu"])
            return {"out": out, "final": final}
        ws = torch.empty(ssd.delta_workspace_bytes(s["q"], s["v"], s["cu"], backward=True), dtype=torch.uint8,
                         device=s["q"].device)
        out, final = ssd.delta_fwd(*args, scale=scale, init=s["init"], cu_seqlens=s["cu"], workspace=ws,
                                   save_for_backward=True)
        grads = ssd.delta_bwd(*args, s["dout"], scale=scale, init=s["init"], d_final=s["d_final"],
                              cu_seqlens=s["cu"], workspace=ws, from_saved=True)
        return {"out": out, "final": final, **grads}
    names = ["q", "k", "v", "g", "beta"] + (["init"] if s["init"] is not None else [])
    lens = [int(n) for n in c["lens"].split(",")] if c["lens"] else None
    if c["kind"] == "fwd":
        out, final = _plain(*[s[n].float() for n in names[:5]], s["init"], lens, scale)
        return {"out": out.to(s["v"].dtype), "final": final}
    leaves = [s[n].float().requires_grad_() for n in names]
    out, final = _plain(*leaves[:5], leaves[5] if len(leaves) > 5 else None, lens, scale)
    loss = (out * s["dout"].float()).sum()
    if s["d_final"] is not None:
        loss = loss + (final * s["d_final"]).sum()
    grads = dict(zip(names, torch.autograd.grad(loss, leaves)))
    got = {"out": out.detach().to(s["v"].dtype), "final": final.detach(), "dg": grads["g"], "dbeta": grads["beta"],
           "d_init": grads.get("init")}
    for n in ("q", "k", "v"):
        got["d" + n] = grads[n].to(s[n].dtype)
    return got


def _unit_inverse(a):
    """(I + a)^-1 of strictly lower triangular a (..., C, C): blocks of 1, 2, 4, ... rows joined in pairs."""
    n = a.shape[-1]
    t = torch.ones_like(a[..., :1, :1]).expand(*a.shape[:-2], n, 1).unsqueeze(-1)  # (..., blocks, b, b)
    b = 1
    while b < n:
        pairs = a.unflatten(-1, (-1, 2 * b)).unflatten(-3, (-1, 2 * b)).diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        t1, t2 = t[..., 0::2, :, :], t[..., 1::2, :, :]
        low = -(t2 @ pairs[..., b:, :b] @ t1)
        t = torch.cat([torch.cat([t1, torch.zeros_like(low)], -1), torch.cat([low, t2], -1)], -2)
        b *= 2
    return t[..., 0, :, :]


def _plain(q, k, v, g, beta, init, lens, scale):
    """The chunked form in 32 bits.  Within a chunk, with G the running sum of g and
    D_ij = exp(G_i - G_j) for j <= i:
        M = tril(k k^T * D, -1),  u = (I + beta M)^-1 beta (v - exp(G) k S^T)
        o = scale (exp(G) q S^T + (q k^T * D) u),  S' = exp(G_C) S + (exp(G_C - G) u)^T k."""
    B, L, H, P = v.shape
    per = H // k.shape[2]
    # sequences as rows, padded to whole chunks with tokens that change nothing (zeros)
    if lens:
        Lp = max(1, -(-max(lens) // CHUNK)) * CHUNK
        at = torch.full((len(lens), Lp), L, dtype=torch.long)
        for i, n in enumerate(lens):
            at[i, :n] = torch.arange(n) + sum(lens[:i])
        at = at.to(v.device)
        rows = lambda x: torch.cat([x[0], torch.zeros_like(x[0, :1])])[at]  # noqa: E731
    else:
        Lp = max(1, -(-L // CHUNK)) * CHUNK
        rows = lambda x: torch.cat([x, x.new_zeros(B, Lp - L, *x.shape[2:])], 1)  # noqa: E731
    n = Lp // CHUNK
    cut = lambda x: rows(x).unflatten(1, (n, CHUNK)).movedim(3, 1)  # noqa: E731  (rows, heads, chunks, C, ...)
    heads = lambda x: x.repeat_interleave(per, 1)  # noqa: E731
    q, k, v, g, beta = cut(q), cut(k), cut(v), cut(g), cut(beta).unsqueeze(-1)
    G = g.double().cumsum(-1)  # differences of long sums
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
    D = torch.where(low, G.unsqueeze(-1) - G.unsqueeze(-2), -math.inf).exp().float()
    eG, eC = G.exp().float().unsqueeze(-1), (G[..., -1:] - G).exp().float().unsqueeze(-1)
    M = heads(k @ k.mT) * D.tril(-1)
    W = heads(q @ k.mT) * D
    q, k = heads(q), heads(k)
    T = _unit_inverse(beta * M)
    u0, kb = T @ (beta * v), T @ (beta * eG * k)
    qe, ke, last = scale * eG * q, (eC * k), eG[..., -1:, :]
    S = v.new_zeros(v.shape[0], H, P, k.shape[-1]) if init is None else init
    out = []
    for c in range(n):
        u = u0[:, :, c] - kb[:, :, c] @ S.mT
        out.append(qe[:, :, c] @ S.mT + scale * (W[:, :, c] @ u))
        S = last[:, :, c] * S + u.mT @ ke[:, :, c]
    o = torch.stack(out, 2).movedim(1, 3).flatten(1, 2)  # (rows, Lp, heads, headdim)
    if not lens:
        return o[:, :L], S
    return torch.cat([o[i, :n] for i, n in enumerate(lens)]).unsqueeze(0), S


def _run_step(s, scale):
    if own:
        from mamba_ssd_chunked_03_amd import ssd
        out = ssd.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], slots=s["slots"], scale=scale,
                             out=s["out"])
        return {"out": out, "states": s["states"]}
    per = s["v"].shape[2] // s["k"].shape[2]
    live = s["case"]["batch"] - s["case"]["pad"]
    at = slice(None) if s["slots"] is None else s["slots"][:live].long()
    q, k, v, g, beta = (s[n][:live].float() for n in ("q", "k", "v", "g", "beta"))
    q, k = q.repeat_interleave(per, 2), k.repeat_interleave(per, 2)
    S, out = s["states"][at], []
    for t in range(v.shape[1]):
        S = S * g[:, t].exp()[..., None, None]
        u = beta[:, t].unsqueeze(-1) * (v[:, t] - (S * k[:, t].unsqueeze(-2)).sum(-1))
        S = S + u.unsqueeze(-1) * k[:, t].unsqueeze(-2)
        out.append(scale * (S * q[:, t].unsqueeze(-2)).sum(-1))
    s["states"][at] = S
    s["out"][:live] = torch.stack(out, 1).to(s["out"].dtype)
    return {"out": s["out"], "states": s["states"]}


def _run_cache(s):
    """Per state row (the dstate values of one headdim index): int8 codes rint(x / scale) with
    scale = max|x| / 127, or e4m3 codes of x / scale with the smallest power of two that
    keeps max|x| / scale at most 448."""
    if own:
        from mamba_ssd_chunked_03_amd import ssd
        ssd.state_cache_write(s["states"], s["codes"], s["scales"], slots=s["slots"])
        back = ssd.state_cache_read(s["codes"], s["scales"], slots=s["slots"])
        return {"states": back, "scales": s["scales"]}
    x, at = s["states"], s["slots"].long()
    top = x.abs().amax(-1)
    if s["codes"].dtype == torch.int8:
        scale = (top.double() / 127).float()  # (64 bits: codes next to a border)
        codes = (x.double() / torch.where(scale > 0, scale, 1.0).double().unsqueeze(-1)).round().clamp(-127, 127)
    else:
        m, e = torch.frexp(top)
        scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), e - torch.where(m <= 0.875, 9, 8)), 0.0)
        codes = x / torch.where(scale > 0, scale, 1.0).unsqueeze(-1)
    s["codes"][at] = codes.to(s["codes"].dtype)
    s["scales"][at] = scale
    return {"states": s["codes"][at].float() * s["scales"][at].unsqueeze(-1), "scales": s["scales"]}


# ------------------------------------------------------------------ exact ----
def _exact_cache(s):
    x, at = s["states"].double(), s["slots"].long()
    top = x.abs().max(-1).values
    if s["codes"].dtype == torch.int8:
        scale = (top / 127).float().double()  # held in 32 bits by definition
        ratio = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
        back = torch.round(ratio) * scale[..., None]
    else:
        power = torch.ceil(torch.log2(top / 448))
        power = torch.where(448 * torch.exp2(power - 1) >= top, power - 1, power)  # log2's own rounding
        scale = torch.where(top > 0, torch.exp2(power), torch.zeros_like(top))
        y = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
        # e4m3: steps of 2^(exponent - 3), exponents from -6 (below it the steps of -6)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        back = torch.round(y / step) * step * scale[..., None]
    scales = s["scales"].double()
    scales[at] = scale
    return {"states": back, "scales": scales}


def _token_loop(q, k, v, g, beta, S, scale, keep=0):
    """The recurrence token by token over (rows, L, heads, ...) in 64 bits; every `keep`-th state."""
    out, kept = torch.empty_like(v), []
    decay = g.exp()
    for t in range(v.shape[1]):
        if keep and t % keep == 0:
            kept.append(S)
        S = S * decay[:, t, :, None, None]
        u = (v[:, t] - (S @ k[:, t, :, :, None])[..., 0]) * beta[:, t, :, None]
        S = S.addcmul_(u[..., None], k[:, t, :, None, :])
        out[:, t] = (S @ q[:, t, :, :, None])[..., 0] * scale
    return out, S, kept


def _adjoint(q, k, v, g, beta, do, dS, scale, kept, keep):
    """The recurrence's adjoint, states replayed from every `keep`-th one."""
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    L = v.shape[1]
    decay = g.exp()
    for first in range((L - 1) // keep * keep, -1, -keep):
        S, before = kept[first // keep], []
        for t in range(first, min(L, first + keep)):
            D = S * decay[:, t, :, None, None]
            r = v[:, t] - (D @ k[:, t, :, :, None])[..., 0]  # what the erased state leaves to write
            S = D + (beta[:, t, :, None] * r)[..., None] * k[:, t, :, None, :]
            before.append((D, r, S))
        for t in range(min(L, first + keep) - 1, first - 1, -1):
            D, r, S = before.pop()
            dq[:, t] = scale * (do[:, t, :, None, :] @ S)[..., 0, :]
            dS = dS + scale * do[:, t, :, :, None] * q[:, t, :, None, :]
            du = (dS @ k[:, t, :, :, None])[..., 0]
            db[:, t] = (du * r).sum(-1)
            dr = beta[:, t, :, None] * du
            dv[:, t] = dr
            dk[:, t] = ((beta[:, t, :, None] * r)[..., None, :] @ dS)[..., 0, :] - (dr[..., None, :] @ D)[..., 0, :]
            dS = dS - dr[..., None] * k[:, t, :, None, :]
            dg[:, t] = (dS * D).sum((-1, -2))
            dS = dS * decay[:, t, :, None, None]
    return dq, dk, dv, dg, db, dS


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["kind"] == "cache":
        return _exact_cache(s)
    scale, per = 1.0 / math.sqrt(c["dstate"]), c["heads"] // c["groups"]
    wide = {n: s[n].double() for n in ("q", "k", "v", "g", "beta")}
    for n in ("q", "k"):
        wide[n] = wide[n].repeat_interleave(per, 2)
    if c["kind"] == "step":
        states, out = s["states"].double(), s["out"].double()
        live = c["batch"] - c["pad"]
        at = torch.arange(live, device=out.device) if s["slots"] is None else s["slots"][:live].long()
        out[:live], states[at], _ = _token_loop(*[wide[n][:live] for n in ("q", "k", "v", "g", "beta")], states[at],
                                                scale)
        return {"out": out, "states": states}
    if c["lens"]:  # one row a sequence, padded with zeros: they leave the state as it is
        lens = [int(n) for n in c["lens"].split(",")]
        parts = lambda x: torch.nn.utils.rnn.pad_sequence(list(x[0].split(lens)), batch_first=True)  # noqa: E731
        joined = lambda x: torch.cat([x[i, :n] for i, n in enumerate(lens)])[None]  # noqa: E731
    else:
        parts = joined = lambda x: x  # noqa: E731
    args = [parts(wide[n]) for n in ("q", "k", "v", "g", "beta")]
    shape = (args[2].shape[0], c["heads"], c["headdim"], c["dstate"])
    S = s["init"].double() if c["init"] else torch.zeros(shape, dtype=torch.float64, device="cuda")
    if c["kind"] == "fwd":
        out, S, _ = _token_loop(*args, S, scale)
        return {"out": joined(out), "final": S}
    keep = 64
    out, S, kept = _token_loop(*args, S, scale, keep)
    dS = s["d_final"].double() if s["d_final"] is not None else torch.zeros_like(S)
    dq, dk, dv, dg, db, dS = _adjoint(*args, parts(s["dout"].double()), dS, scale, kept, keep)
    group = lambda x: joined(x).unflatten(2, (c["groups"], per)).sum(3)  # noqa: E731
    return {"out": joined(out), "final": S, "dq": group(dq), "dk": group(dk), "dv": joined(dv), "dg": joined(dg),
            "dbeta": joined(db), "d_init": dS if c["init"] else None}
