"""The selective state space scan, its short convolution and the draft
verification in fp64 numpy, token by token.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).  Plain definitions of
include/kda_ssm.h and include/kda_spec.h, one sequence or one request at a
time, no chunks and no fusion.

Shapes of one sequence: x [T, H, P], dt [T, H] (raw), B, C [T, G, N], A, D,
dt_bias [H], S [H, N, P]; convolution x [T, c], w [c, W], cache [W - 1, c].
"""
from __future__ import annotations

import numpy as np


def softplus(x):
    x = np.asarray(x, np.float64)
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-np.asarray(x, np.float64)))


def conv(x, w, bias=None, cache=None, activation=True):
    """Returns (y [T, c], cache afterwards)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    W = w.shape[1]
    old = np.zeros((W - 1, x.shape[1])) if cache is None else np.asarray(cache, np.float64)
    line = np.concatenate([old, x])
    T = x.shape[0]
    z = np.zeros_like(x) if bias is None else np.tile(np.asarray(bias, np.float64), (T, 1))
    for t in range(T):
        for j in range(W):
            z[t] += w[:, j] * line[t + j]
    return (z * sigmoid(z) if activation else z), line[T:].copy()


def conv_backward(x, w, bias, cache, gy, activation=True):
    """Returns (gx, gw, gbias, gcache)."""
    x, w, gy = (np.asarray(a, np.float64) for a in (x, w, gy))
    W, T = w.shape[1], x.shape[0]
    old = np.zeros((W - 1, x.shape[1])) if cache is None else np.asarray(cache, np.float64)
    line = np.concatenate([old, x])
    gline, gw, gb = np.zeros_like(line), np.zeros_like(w), np.zeros(x.shape[1])
    for t in range(T):
        z = np.zeros(x.shape[1]) if bias is None else np.array(bias, np.float64)
        for j in range(W):
            z += w[:, j] * line[t + j]
        s = sigmoid(z)
        gz = gy[t] * (s + z * s * (1 - s)) if activation else gy[t]
        for j in range(W):
            gline[t + j] += w[:, j] * gz
            gw[:, j] += gz * line[t + j]
        gb += gz
    return gline[W - 1:], gw, gb, gline[:W - 1]


def _heads(t, H):
    """[G, N] of one token as [H, N]."""
    return np.repeat(np.asarray(t, np.float64), H // t.shape[0], axis=0)


def _dt(dt, dt_bias, soft):
    raw = np.asarray(dt, np.float64)
    if dt_bias is not None:
        raw = raw + np.asarray(dt_bias, np.float64)
    return raw, (softplus(raw) if soft else raw)


def scan(x, dt, A, B, C, D=None, S0=None, dt_bias=None, soft=True):
    """Returns (y [T, H, P], S_T)."""
    x, A = np.asarray(x, np.float64), np.asarray(A, np.float64)
    T, H, P = x.shape
    N = B.shape[2]
    S = np.zeros((H, N, P)) if S0 is None else np.array(S0, np.float64)
    _, d = _dt(dt, dt_bias, soft)
    y = np.zeros_like(x)
    for t in range(T):
        S = np.exp(d[t] * A)[:, None, None] * S + (d[t][:, None] * _heads(B[t], H))[:, :, None] * x[t][:, None, :]
        y[t] = np.einsum("hnp,hn->hp", S, _heads(C[t], H))
        if D is not None:
            y[t] += np.asarray(D, np.float64)[:, None] * x[t]
    return y, S


def scan_backward(x, dt, A, B, C, D, S0, gy, gS=None, dt_bias=None, soft=True):
    """Returns a dict of the gradients x, dt (raw), A, B, C, D, bias, S0."""
    x, A, gy = (np.asarray(a, np.float64) for a in (x, A, gy))
    T, H, P = x.shape
    G, N = B.shape[1:]
    raw, d = _dt(dt, dt_bias, soft)
    S = np.zeros((H, N, P)) if S0 is None else np.array(S0, np.float64)
    before = []
    for t in range(T):
        before.append(S)
        S = np.exp(d[t] * A)[:, None, None] * S + (d[t][:, None] * _heads(B[t], H))[:, :, None] * x[t][:, None, :]
    R = np.zeros((H, N, P)) if gS is None else np.array(gS, np.float64)
    g = {"x": np.zeros_like(x), "B": np.zeros((T, G, N)), "C": np.zeros((T, G, N)), "dt": np.zeros((T, H)),
         "A": np.zeros(H), "D": np.zeros(H)}
    after = S
    for t in range(T - 1, -1, -1):
        Bh, Ch, e = _heads(B[t], H), _heads(C[t], H), np.exp(d[t] * A)
        g["C"][t] = np.einsum("hnp,hp->hn", after, gy[t]).reshape(G, H // G, N).sum(1)
        R = R + Ch[:, :, None] * gy[t][:, None, :]
        into = np.einsum("hnp,hp->hn", R, x[t])
        g["B"][t] = (d[t][:, None] * into).reshape(G, H // G, N).sum(1)
        g["x"][t] = d[t][:, None] * np.einsum("hnp,hn->hp", R, Bh)
        if D is not None:
            g["x"][t] += np.asarray(D, np.float64)[:, None] * gy[t]
        g["D"] += np.einsum("hp,hp->h", gy[t], x[t])
        ga = e * np.einsum("hnp,hnp->h", R, before[t])
        g["A"] += d[t] * ga
        g["dt"][t] = np.einsum("hn,hn->h", into, Bh) + A * ga
        R = e[:, None, None] * R
        after = before[t]
    if soft:
        g["dt"] *= sigmoid(raw)
    g["bias"] = g["dt"].sum(0)
    g["S0"] = R
    return g


def verify(p, drafts, u, u_next, q=None, n_draft=None):
    """One request: p [K + 1, V], drafts [K], u [K], q [K, V] or None.
    Returns (n_accepted, tokens [K + 1])."""
    p = np.where(np.asarray(p, np.float64) > 0, np.asarray(p, np.float64), 0.0)
    K, V = len(drafts), p.shape[1]
    if q is not None:
        q = np.where(np.asarray(q, np.float64) > 0, np.asarray(q, np.float64), 0.0)
    kb = K if n_draft is None else min(max(int(n_draft), 0), K)
    n = 0
    while n < kb:
        d = int(drafts[n])
        if not 0 <= d < V:
            break
        qd = 1.0 if q is None else q[n, d]
        if not float(u[n]) * qd < p[n, d]:
            break
        n += 1
    r = p[n].copy()
    if n < kb:
        if q is not None:
            r = np.maximum(r - q[n], 0.0)
        elif 0 <= int(drafts[n]) < V:
            r[int(drafts[n])] = 0.0
    if not r.sum() > 0:
        r = p[n]
    token = 0
    if r.sum() > 0:
        run = np.cumsum(r)
        past = np.nonzero(run > float(u_next) * run[-1])[0]
        token = int(past[0]) if len(past) else int(np.nonzero(r > 0)[0][-1])
    return n, np.array([int(d) for d in drafts[:n]] + [token] + [-1] * (K - n))
