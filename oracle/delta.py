"""fp64 oracle of the gated delta rule, rotary positions and layer norm
(numpy): the definitions step by step, sharing nothing with the CUDA library.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------- the gated delta rule

def delta_forward(q, k, v, g, beta, lengths=None, initial_state=None):
    """q, k [B, N, Hk, dk], v [B, N, H, dv], g and beta [B, N, H]: token by token
        S' = exp(g) S,  u = beta (v - S'^T k),  S = S' + k u^T,  o = S^T q.
    Returns (out, final state); rows behind a sequence's end are zero."""
    B, N, Hk, dk = q.shape
    H, dv = v.shape[2:]
    rep = H // Hk
    out = np.zeros((B, N, H, dv))
    S = np.zeros((B, H, dk, dv)) if initial_state is None else np.array(initial_state, np.float64)
    for b in range(B):
        for t in range(N if lengths is None else int(np.clip(lengths[b], 0, N))):
            kt, qt = np.repeat(k[b, t], rep, axis=0), np.repeat(q[b, t], rep, axis=0)
            Sd = np.exp(g[b, t])[:, None, None] * S[b]
            u = beta[b, t][:, None] * (v[b, t] - np.einsum("hkv,hk->hv", Sd, kt))
            S[b] = Sd + kt[:, :, None] * u[:, None, :]
            out[b, t] = np.einsum("hkv,hk->hv", S[b], qt)
    return out, S


def delta_backward(q, k, v, g, beta, dout, lengths=None, initial_state=None, dfinal_state=None):
    """Gradients of sum(out * dout) + sum(final_state * dfinal_state) by the chain
    rule through every token, last to first: dict with dq, dk, dv, dg, dbeta,
    dinitial_state.  Padded rows get zeros."""
    B, N, Hk, dk_ = q.shape
    H, dv_ = v.shape[2:]
    rep = H // Hk
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, dbeta = np.zeros_like(g), np.zeros_like(beta)
    dS0 = np.zeros((B, H, dk_, dv_))
    for b in range(B):
        n = N if lengths is None else int(np.clip(lengths[b], 0, N))
        S = np.zeros((H, dk_, dv_)) if initial_state is None else np.array(initial_state[b], np.float64)
        steps = []
        for t in range(n):
            kt = np.repeat(k[b, t], rep, axis=0)
            a = np.exp(g[b, t])[:, None, None]
            Sd = a * S
            err = v[b, t] - np.einsum("hkv,hk->hv", Sd, kt)
            u = beta[b, t][:, None] * err
            S = Sd + kt[:, :, None] * u[:, None, :]
            steps.append((Sd, err, u, S, a))
        dS = np.zeros((H, dk_, dv_)) if dfinal_state is None else np.array(dfinal_state[b], np.float64)
        for t in reversed(range(n)):
            Sd, err, u, S, a = steps[t]
            kt, qt = np.repeat(k[b, t], rep, axis=0), np.repeat(q[b, t], rep, axis=0)
            do = dout[b, t]
            dqh = np.einsum("hkv,hv->hk", S, do)
            dS = dS + qt[:, :, None] * do[:, None, :]
            du = np.einsum("hkv,hk->hv", dS, kt)
            dkh = np.einsum("hkv,hv->hk", dS, u)
            dbeta[b, t] = (du * err).sum(-1)
            derr = beta[b, t][:, None] * du
            dv[b, t] = derr
            dkh -= np.einsum("hkv,hv->hk", Sd, derr)
            dSd = dS - kt[:, :, None] * derr[:, None, :]
            dg[b, t] = (dSd * Sd).sum((-1, -2))
            dS = a * dSd
            dq[b, t] = dqh.reshape(Hk, rep, dk_).sum(1)
            dk[b, t] = dkh.reshape(Hk, rep, dk_).sum(1)
        dS0[b] = dS
    return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta, "dinitial_state": dS0}


# ------------------------------------------------------------ rotary positions

def rotary(x, positions, freqs, layout="interleaved", scale=1.0, inverse=False):
    """x [B, N, heads, d] with pair p at position n turned by n freqs[p] (the
    negative angle with ``inverse``) and multiplied by scale; positions [B, N]."""
    r = 2 * len(freqs)
    out = np.array(x, np.float64)
    ang = np.asarray(positions, np.float64)[:, :, None, None] * np.asarray(freqs, np.float64)
    c, s = scale * np.cos(ang), scale * np.sin(ang) * (-1 if inverse else 1)
    ia, ib = (np.arange(0, r, 2), np.arange(1, r, 2)) if layout == "interleaved" else \
        (np.arange(r // 2), np.arange(r // 2, r))
    a, b = np.array(x[..., ia], np.float64), np.array(x[..., ib], np.float64)
    out[..., ia] = a * c - b * s
    out[..., ib] = a * s + b * c
    return out


# ------------------------------------------------------------------ layer norm

def layernorm(x, gain=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last dimension, biased variance."""
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if gain is not None:
        y = y * gain
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layernorm_backward(dy, x, mean, rstd, gain=None):
    """(dx, dgain, dbias) for given mean and rstd of the rows."""
    h = (x - mean[..., None]) * rstd[..., None]
    t = dy if gain is None else dy * gain
    dx = rstd[..., None] * (t - t.mean(-1, keepdims=True) - h * (t * h).mean(-1, keepdims=True))
    lead = tuple(range(x.ndim - 1))
    return dx, (dy * h).sum(lead), dy.sum(lead)
