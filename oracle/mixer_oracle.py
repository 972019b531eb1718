"""fp64 CPU oracle of the token-mixer operators: the short causal convolution, the head norm
with position rotation and the selective state space scan, each with its backward. Plain
loops over tokens, numpy float64, nothing shared with the CUDA library."""
from __future__ import annotations

import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _sigmoid(a):
    e = np.exp(-np.abs(a))
    return np.where(a >= 0, 1.0, e) / (1.0 + e)


def _lens(lens, B, N):
    return [N] * B if lens is None else [int(min(max(n, 0), N)) for n in lens]


# ----------------------------------------------------------------------------- convolution
def short_conv(x, w, bias=None, act=True, state=None, lens=None):
    """y[t] = act(bias + sum_j w[j] x[t-j]); returns (y, state after the last token)."""
    x, w, bias, state = map(_f, (x, w, bias, state))
    B, N, D = x.shape
    K = w.shape[0]
    y = np.zeros((B, N, D))
    new = np.zeros((B, K - 1, D))
    for b, n in enumerate(_lens(lens, B, N)):
        hist = np.concatenate([np.zeros((K - 1, D)) if state is None else state[b], x[b, :n]])
        for t in range(n):
            pre = sum(w[j] * hist[K - 1 + t - j] for j in range(K)) + (0.0 if bias is None else bias)
            y[b, t] = pre * _sigmoid(pre) if act else pre
        new[b] = hist[n:]
    return y, new


def short_conv_backward(x, w, dy, bias=None, act=True, state=None, lens=None, dstate=None):
    """Gradients of sum(dy * y) + sum(dstate * new state): dx, dw, dbias, dstate_in."""
    x, w, dy, bias, state, dstate = map(_f, (x, w, dy, bias, state, dstate))
    B, N, D = x.shape
    K = w.shape[0]
    dx, dw, db, ds = np.zeros((B, N, D)), np.zeros((K, D)), np.zeros(D), np.zeros((B, K - 1, D))
    for b, n in enumerate(_lens(lens, B, N)):
        hist = np.concatenate([np.zeros((K - 1, D)) if state is None else state[b], x[b, :n]])
        dh = np.zeros_like(hist)
        if dstate is not None:
            dh[n:] += dstate[b]
        for t in range(n):
            g = dy[b, t]
            if act:
                pre = sum(w[j] * hist[K - 1 + t - j] for j in range(K)) + (0.0 if bias is None else bias)
                s = _sigmoid(pre)
                g = g * s * (1.0 + pre * (1.0 - s))
            db += g
            for j in range(K):
                dw[j] += g * hist[K - 1 + t - j]
                dh[K - 1 + t - j] += w[j] * g
        ds[b], dx[b, :n] = dh[:K - 1], dh[K - 1:]
    return dx, dw, db, ds


# ----------------------------------------------------------------------------- heads
def _pairs(h, rot, pairs):
    p = np.arange(rot // 2)
    return (2 * p, 2 * p + 1) if pairs == "interleaved" else (p, p + rot // 2)


def _rotate(x, pos, inv_freq, pairs, sign=1.0):
    """x [B,N,H,h], pos [B,N]."""
    if inv_freq is None:
        return x
    ang = pos.astype(np.float64)[:, :, None, None] * _f(inv_freq)
    c, s = np.cos(ang), sign * np.sin(ang)
    i, j = _pairs(x.shape[-1], 2 * len(inv_freq), pairs)
    y = x.copy()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def _inv_norm(x, norm, eps):
    if norm is None:
        return np.ones(x.shape[:-1] + (1,))
    sq = (x * x).sum(-1, keepdims=True)
    return 1.0 / np.sqrt((sq / x.shape[-1] if norm == "rms" else sq) + eps)


def head_norm_rope(x, w=None, norm="l2", eps=1e-6, inv_freq=None, positions=None, pairs="halves"):
    """[B,N,H,h] -> [B,H,N,h]."""
    x = _f(x)
    y = x * _inv_norm(x, norm, eps) * (1.0 if w is None else _f(w))
    return _rotate(y, np.asarray(positions), inv_freq, pairs).transpose(0, 2, 1, 3)


def head_norm_rope_backward(x, dout, w=None, norm="l2", eps=1e-6, inv_freq=None, positions=None,
                            pairs="halves"):
    """Gradients of x [B,N,H,h] and w for dout [B,H,N,h]."""
    x = _f(x)
    g = _rotate(_f(dout).transpose(0, 2, 1, 3), np.asarray(positions), inv_freq, pairs, -1.0)
    r = _inv_norm(x, norm, eps)
    dw = (g * x * r).sum((0, 1, 2))
    g = g * (1.0 if w is None else _f(w))
    dx = g * r
    if norm is not None:
        dot = (g * x).sum(-1, keepdims=True)
        dx = dx - x * r ** 3 * (dot / x.shape[-1] if norm == "rms" else dot)
    return dx, dw


# ----------------------------------------------------------------------------- selective scan
def _delta(dt, dt_bias, softplus):
    raw = dt if dt_bias is None else dt + dt_bias
    return (np.maximum(raw, 0) + np.log1p(np.exp(-np.abs(raw))) if softplus else raw), raw


def selective_scan(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True, state=None,
                   lens=None):
    """Returns (y [B,N,D], states [B,N+1,D,S]: states[t] is the one before token t)."""
    u, dt, A, Bm, Cm, D, z, dt_bias, state = map(_f, (u, dt, A, Bm, Cm, D, z, dt_bias, state))
    B, N, d = u.shape
    S, rep = A.shape[1], d // Bm.shape[2]
    delta, _ = _delta(dt, dt_bias, softplus)
    y, hs = np.zeros((B, N, d)), np.zeros((B, N + 1, d, S))
    for b, n in enumerate(_lens(lens, B, N)):
        if state is not None:
            hs[b, 0] = state[b]
        for t in range(N):
            if t >= n:
                hs[b, t + 1] = hs[b, t]
                continue
            Bt, Ct = np.repeat(Bm[b, t], rep, 0), np.repeat(Cm[b, t], rep, 0)
            hs[b, t + 1] = np.exp(delta[b, t][:, None] * A) * hs[b, t] + (delta[b, t] * u[b, t])[:, None] * Bt
            y[b, t] = (Ct * hs[b, t + 1]).sum(-1) + (0.0 if D is None else D * u[b, t])
            if z is not None:
                y[b, t] *= z[b, t] * _sigmoid(z[b, t])
    return y, hs


def selective_scan_backward(u, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, softplus=True,
                            state=None, lens=None, dstate=None):
    """Gradients of sum(dy * y) + sum(dstate * last state), as a dict."""
    _, hs = selective_scan(u, dt, A, Bm, Cm, D, z, dt_bias, softplus, state, lens)
    u, dt, A, Bm, Cm, dy, D, z, dt_bias, dstate = map(_f, (u, dt, A, Bm, Cm, dy, D, z, dt_bias, dstate))
    B, N, d = u.shape
    S, G = A.shape[1], Bm.shape[2]
    rep = d // G
    delta, raw = _delta(dt, dt_bias, softplus)
    o = {"du": np.zeros_like(u), "ddt": np.zeros_like(u), "dA": np.zeros_like(A),
         "dB": np.zeros_like(Bm), "dC": np.zeros_like(Cm), "dD": np.zeros(d),
         "dz": np.zeros_like(u), "ddt_bias": np.zeros(d), "dstate": np.zeros((B, d, S))}
    for b, n in enumerate(_lens(lens, B, N)):
        dh = np.zeros((d, S)) if dstate is None else dstate[b].copy()
        for t in range(n - 1, -1, -1):
            Bt, Ct = np.repeat(Bm[b, t], rep, 0), np.repeat(Cm[b, t], rep, 0)
            g = dy[b, t]
            if z is not None:
                s = _sigmoid(z[b, t])
                pre = (Ct * hs[b, t + 1]).sum(-1) + (0.0 if D is None else D * u[b, t])
                o["dz"][b, t] = g * pre * s * (1.0 + z[b, t] * (1.0 - s))
                g = g * z[b, t] * s
            o["dD"] += g * u[b, t]
            o["dC"][b, t] = (g[:, None] * hs[b, t + 1]).reshape(G, rep, S).sum(1)
            dh = dh + g[:, None] * Ct
            a = np.exp(delta[b, t][:, None] * A)
            p = dh * a * hs[b, t]
            x = (dh * Bt).sum(-1)
            o["dA"] += delta[b, t][:, None] * p
            o["dB"][b, t] = (dh * (delta[b, t] * u[b, t])[:, None]).reshape(G, rep, S).sum(1)
            o["du"][b, t] = delta[b, t] * x + (0.0 if D is None else D * g)
            dd = (A * p).sum(-1) + u[b, t] * x
            if softplus:
                dd = dd * _sigmoid(raw[b, t])
            o["ddt"][b, t] = dd
            o["ddt_bias"] += dd
            dh = a * dh
        o["dstate"][b] = dh
    return o
