"""Seeded problems of the gated delta rule for its tests."""
import math

import numpy as np
import torch


def make(batch, seqlen, heads, groups, headdim, dstate, io="bf16", init=True, lengths=None, seed=0, keys="unit",
         gates="usual", d_final=True):
    """keys: "unit" unit rows; "equal": every key of a group the same (beta 1 where gates is
    "ones"), the hardest triangle.  gates: "usual" (-softplus steps, sigmoid beta), "ones" (g 0,
    beta 1), "zero_beta" (a third of the betas 0), "resets" (some gates -inf), "strong" (g down
    to -40)."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    dt = torch.float32 if io == "f32" else torch.bfloat16
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = unit(rand(batch, seqlen, groups, dstate)), unit(rand(batch, seqlen, groups, dstate))
    if keys == "equal":
        k = k[:, :1].expand_as(k).contiguous() if seqlen else k
    v, dout = rand(batch, seqlen, heads, headdim), rand(batch, seqlen, heads, headdim)
    a = torch.exp(torch.rand(heads, generator=gen) * math.log(16.0))
    g = -a * torch.nn.functional.softplus(rand(batch, seqlen, heads) - 3)
    beta = torch.sigmoid(1.5 * rand(batch, seqlen, heads))
    u = torch.rand(batch, seqlen, heads, generator=gen)
    if gates == "ones":
        g, beta = torch.zeros_like(g), torch.ones_like(beta)
    elif gates == "zero_beta":
        beta = torch.where(u < 0.34, torch.zeros_like(beta), beta)
    elif gates == "resets":
        g = torch.where(u < 0.05, torch.full_like(g, -math.inf), g)
    elif gates == "strong":
        g = torch.where(u < 0.3, -40 * u / 0.3, g)
    nst = batch if lengths is None else len(lengths)
    states = lambda: 0.3 * rand(nst, heads, headdim, dstate)  # noqa: E731
    cu = None
    if lengths is not None:
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32))
    return dict(q=q.to(dt), k=k.to(dt), v=v.to(dt), g=g, beta=beta, dout=dout.to(dt), cu=cu, scale=dstate ** -0.5,
                init=states() if init else None, d_final=states() if d_final else None)


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def oracle_fwd(d):
    from oracle import delta
    return delta.fwd(f64(d["q"]), f64(d["k"]), f64(d["v"]), f64(d["g"]), f64(d["beta"]), d["scale"], f64(d["init"]),
                     None if d["cu"] is None else d["cu"].tolist())


def oracle_bwd(d):
    from oracle import delta
    return delta.bwd(f64(d["q"]), f64(d["k"]), f64(d["v"]), f64(d["g"]), f64(d["beta"]), d["scale"], f64(d["dout"]),
                     f64(d["init"]), f64(d["d_final"]), None if d["cu"] is None else d["cu"].tolist())


def cuda(d):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in d.items()}
