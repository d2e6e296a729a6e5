"""The gated delta rule and beam search in plain numpy, fp64, token by token.

Per sequence and value head, with S [N, N] (row = value channel, column = key channel), k and q of
the head's key head (brought to unit length when ``qk_norm``), q times ``scale``:

    e_t = v_t - exp(g_t) S_{t-1} k_t;  S_t = exp(g_t) S_{t-1} + beta_t e_t k_t^T;  y_t = S_t q_t
"""
from __future__ import annotations

import numpy as np

from .reference import _f64


def _unit(x, eps):
    return x / np.sqrt(np.sum(x * x, axis=-1, keepdims=True) + eps)


def _heads(x, H):
    return np.repeat(x, H // x.shape[-2], axis=-2)


def delta_recurrence(q, k, v, g, beta, S0=None, *, scale=None, qk_norm=False, norm_eps=1e-6):
    """q, k [B, T, Hk, N], v [B, T, H, N], g, beta [B, T, H]; returns (y, S_T)."""
    q, k, v, g, beta = (_f64(x) for x in (q, k, v, g, beta))
    B, T, H, N = v.shape
    if qk_norm:
        q, k = _unit(q, norm_eps), _unit(k, norm_eps)
    q = _heads(q, H) * (N ** -0.5 if scale is None else scale)
    k = _heads(k, H)
    S = np.zeros((B, H, N, N)) if S0 is None else _f64(S0).copy()
    y = np.empty((B, T, H, N))
    for t in range(T):
        S = np.exp(g[:, t])[:, :, None, None] * S
        e = v[:, t] - np.einsum("bhij,bhj->bhi", S, k[:, t])
        S = S + (beta[:, t][..., None] * e)[..., :, None] * k[:, t][..., None, :]
        y[:, t] = np.einsum("bhij,bhj->bhi", S, q[:, t])
    return y, S


def delta_backward(q, k, v, g, beta, S0, dy, dS_T, *, scale=None, qk_norm=False, norm_eps=1e-6):
    """Gradients of <dy, y> + <dS_T, S_T>: the chain rule through delta_recurrence, one token at a
    time in reverse, every state kept. Returns dict of dq, dk, dv, dg, dbeta, dS0."""
    q0, k0, v, g, beta, dy = (_f64(x) for x in (q, k, v, g, beta, dy))
    B, T, H, N = v.shape
    Hk = k0.shape[-2]
    sc = N ** -0.5 if scale is None else scale
    q, k = (_heads(_unit(x, norm_eps) if qk_norm else x, H) for x in (q0, k0))
    q = q * sc
    S = np.zeros((B, H, N, N)) if S0 is None else _f64(S0).copy()
    kept, errs, decayed = [], [], []
    for t in range(T):
        kept.append(S)
        P = np.exp(g[:, t])[:, :, None, None] * S
        e = v[:, t] - np.einsum("bhij,bhj->bhi", P, k[:, t])
        S = P + (beta[:, t][..., None] * e)[..., :, None] * k[:, t][..., None, :]
        errs.append(e)
        decayed.append(P)
    dS = np.zeros((B, H, N, N)) if dS_T is None else _f64(dS_T).copy()
    out = {n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))}
    for t in range(T - 1, -1, -1):
        b, e, P, kt = beta[:, t][..., None], errs[t], decayed[t], k[:, t]
        St = P + (b * e)[..., :, None] * kt[..., None, :]
        dS = dS + dy[:, t][..., :, None] * q[:, t][..., None, :]
        out["dq"][:, t] = np.einsum("bhij,bhi->bhj", St, dy[:, t])
        du = np.einsum("bhij,bhj->bhi", dS, kt)                 # of u = beta e
        out["dbeta"][:, t] = np.sum(du * e, axis=-1)
        de = b * du
        out["dv"][:, t] = de
        dP = dS - de[..., :, None] * kt[..., None, :]
        out["dk"][:, t] = np.einsum("bhij,bhi->bhj", dS, b * e) - np.einsum("bhij,bhi->bhj", P, de)
        out["dg"][:, t] = np.sum(dP * P, axis=(-1, -2))
        dS = np.exp(g[:, t])[:, :, None, None] * dP
    out["dq"] = out["dq"] * sc
    for n, x in (("dq", q0), ("dk", k0)):
        d = out[n].reshape(B, T, Hk, H // Hk, N).sum(axis=3)
        if qk_norm:
            r = 1.0 / np.sqrt(np.sum(x * x, axis=-1, keepdims=True) + norm_eps)
            d = r * (d - x * r * np.sum(x * r * d, axis=-1, keepdims=True))
        out[n] = d
    out["dS0"] = dS
    return out


def beam_select(logits, scores, M, finished=None, eos=0):
    """Every continuation scored, sorted from the best down (equal scores: lowest beam, then lowest
    token); fewer than M: score -inf, parent and token -1."""
    x, s = _f64(logits), _f64(scores)
    B, K, V = x.shape
    out_s = np.full((B, M), -np.inf)
    parents, tokens = np.full((B, M), -1, np.int32), np.full((B, M), -1, np.int32)
    for b in range(B):
        cand = []
        for j in range(K):
            if finished is not None and finished[b, j]:
                cand.append((s[b, j], j, eos))
                continue
            row = np.where(np.isnan(x[b, j]), -np.inf, x[b, j])
            top = row.max()
            if not np.isfinite(top):
                continue
            norm = top + np.log(np.sum(np.exp(row - top)))
            val = s[b, j] + (row - norm)
            order = np.argsort(-val, kind="stable")[:M]
            cand += [(val[t], j, int(t)) for t in order]
        cand = [c for c in cand if c[0] > -np.inf]
        cand.sort(key=lambda c: (-c[0], c[1], c[2]))
        for i, (val, j, t) in enumerate(cand[:M]):
            out_s[b, i], parents[b, i], tokens[b, i] = val, j, t
    return out_s, parents, tokens
