"""Token-by-token fp64 gated delta rule and its adjoint (test infrastructure only).

Per sequence and head h, group h // (nheads // ngroups), state S (P x N):

    D_t = exp(g_t) S_{t-1}
    r_t = v_t - D_t k_t
    S_t = D_t + beta_t r_t k_t^T
    o_t = scale S_t q_t,             S_{-1} = init (zeros when absent)

Layouts: q, k (batch, seqlen, ngroups, N); v (batch, seqlen, nheads, P); g, beta (batch,
seqlen, nheads); states (nseq, nheads, P, N).  ``cu_seqlens``: packed sequences of the
single batch row.  The backward is the loop's adjoint written out by hand, with every
state kept (the problems are small).  ``quantise`` is the state cache's rounding.
"""
import numpy as np


def _spans(batch, seqlen, cu):
    if cu is None:
        return [(b, 0, seqlen) for b in range(batch)]
    return [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def fwd(q, k, v, g, beta, scale, init=None, cu_seqlens=None, keep=False):
    """(o, final); with keep also {(sequence, t): (D, r, S)}."""
    q, k, v, g, beta = (np.asarray(x, dtype=np.float64) for x in (q, k, v, g, beta))
    batch, seqlen, H, P = v.shape
    G, N = k.shape[2:]
    head = np.arange(H) // (H // G)
    spans = _spans(batch, seqlen, cu_seqlens)
    o = np.zeros_like(v)
    final = np.zeros((len(spans), H, P, N))
    kept = {}
    for s, (b, t0, t1) in enumerate(spans):
        S = np.zeros((H, P, N)) if init is None else np.array(init[s], dtype=np.float64)
        for t in range(t0, t1):
            D = S * np.exp(g[b, t])[:, None, None]
            r = v[b, t] - np.einsum("hpn,hn->hp", D, k[b, t][head])
            S = D + (beta[b, t][:, None] * r)[:, :, None] * k[b, t][head][:, None, :]
            o[b, t] = scale * np.einsum("hpn,hn->hp", S, q[b, t][head])
            if keep:
                kept[s, t] = (D, r, S)
        final[s] = S
    return (o, final, kept) if keep else (o, final)


def bwd(q, k, v, g, beta, scale, dout, init=None, d_final=None, cu_seqlens=None):
    """Gradients of <dout, o> + <d_final, final>: dict dq, dk, dv, dg, dbeta, d_init."""
    q, k, v, g, beta, dout = (np.asarray(x, dtype=np.float64) for x in (q, k, v, g, beta, dout))
    batch, seqlen, H, P = v.shape
    G, N = k.shape[2:]
    per = H // G
    head = np.arange(H) // per
    spans = _spans(batch, seqlen, cu_seqlens)
    _, _, kept = fwd(q, k, v, g, beta, scale, init, cu_seqlens, keep=True)
    out = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dg": np.zeros_like(g),
           "dbeta": np.zeros_like(beta), "d_init": np.zeros((len(spans), H, P, N))}
    groups = lambda x: x.reshape(G, per, N).sum(1)  # noqa: E731
    for s, (b, t0, t1) in enumerate(spans):
        dS = np.zeros((H, P, N)) if d_final is None else np.array(d_final[s], dtype=np.float64)
        for t in range(t1 - 1, t0 - 1, -1):
            D, r, S = kept[s, t]
            kt, qt, bt = k[b, t][head], q[b, t][head], beta[b, t][:, None]
            out["dq"][b, t] = groups(scale * np.einsum("hp,hpn->hn", dout[b, t], S))
            dS = dS + scale * dout[b, t][:, :, None] * qt[:, None, :]
            du = np.einsum("hpn,hn->hp", dS, kt)
            out["dbeta"][b, t] = (du * r).sum(-1)
            dr = bt * du
            out["dv"][b, t] = dr
            out["dk"][b, t] = groups(np.einsum("hp,hpn->hn", bt * r, dS) - np.einsum("hp,hpn->hn", dr, D))
            dD = dS - dr[:, :, None] * kt[:, None, :]
            out["dg"][b, t] = (dD * D).sum((-1, -2))
            dS = dD * np.exp(g[b, t])[:, None, None]
        out["d_init"][s] = dS
    return out


def quantise(x, fmt):
    """(values read back, scales) of the state cache for rows x (..., N) of finite fp32 values."""
    x = np.asarray(x, dtype=np.float64)
    top = np.abs(x).max(-1, keepdims=True)
    if fmt == "int8":
        scale = (top / 127).astype(np.float32).astype(np.float64)
        safe = np.where(scale > 0, scale, 1.0)
        codes = np.where(scale > 0, np.clip(np.rint(x / safe), -127, 127), 0.0)
        return codes * scale, scale[..., 0]
    # smallest power of two with top <= 448 scale
    _, e = np.frexp(top / 448.0)  # top / 448 = m 2^e, m in [1/2, 1)
    scale = np.ldexp(1.0, e - (np.ldexp(0.5, e) * 448.0 >= top))
    scale = np.where(top > 0, np.maximum(scale, 2.0 ** -126), 0.0)
    y = x / np.where(scale > 0, scale, 1.0)
    _, ey = np.frexp(np.where(y == 0, 1.0, y))
    step = np.ldexp(1.0, np.maximum(ey - 1, -6) - 3)  # 3 bits below the leading one; subnormals below 2^-6
    return np.rint(y / step) * step * scale, scale[..., 0]
