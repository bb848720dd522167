"""Float64 oracle of the selective state space scan, its single-token step and the
norms around a block: plain numpy from the formulas, token by token.  Test
infrastructure only; shares no code with the library.

``scan`` also returns, per output element, how large the rounding errors of an fp32
evaluation can get, in units of its rounding 2^-24: every token multiplies the state by
a decay (relative error at most 3 + 2 |delta a| units: the step size, the product and
the exponential) and adds a product, each rounded; a term's earlier errors shrink with
the term.
"""
from __future__ import annotations

import numpy as np
import torch


def f64(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.detach().to("cpu", torch.float64).numpy()
    return np.asarray(t, dtype=np.float64)


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def scan(x, b, c, dt, a, d=None, dt_bias=None, h0=None, cu_seqlens=None, soft=False):
    """x [B,T,HV,dv], b, c [B,T,HK,dk], dt [B,T,HV] -> y, hT, y_abs, y_units, h_units:
    the results, sum |terms| of every output, and the error bounds described above."""
    x, b, c, dt, a = f64(x), f64(b), f64(c), f64(dt), f64(a)
    B, T, HV, dv = x.shape
    HK, dk = b.shape[2:]
    d = np.zeros(HV) if d is None else f64(d)
    delta = dt + (0 if dt_bias is None else f64(dt_bias))
    delta = softplus(delta) if soft else delta
    if cu_seqlens is None:
        spans = [(n, 0, T) for n in range(B)]
    else:
        cu = [int(v) for v in cu_seqlens]
        spans = [(0, cu[n], cu[n + 1]) for n in range(len(cu) - 1)]
    N = len(spans)
    y, y_abs, y_units = np.zeros(x.shape), np.zeros(x.shape), np.zeros(x.shape)
    hT, h_units = np.zeros((N, HV, dv, dk)), np.zeros((N, HV, dv, dk))
    group = np.arange(HV) // (HV // HK)
    for n, (row, t0, t1) in enumerate(spans):
        S = np.zeros((HV, dv, dk)) if h0 is None else f64(h0)[n].copy()
        A = np.abs(S)
        E = np.zeros(S.shape)
        for t in range(t0, t1):
            g = delta[row, t] * a
            al = np.exp(g)[:, None, None]
            bt, ct = b[row, t][group], c[row, t][group]
            u = delta[row, t][:, None] * x[row, t]
            add = u[:, :, None] * bt[:, None, :]
            S = al * S + add
            with np.errstate(invalid="ignore"):
                per = np.where(np.isfinite(g), np.minimum(3 + 2 * np.abs(g), 1e300), 0)[:, None, None]
            E = al * E + (per + 1) * al * A + 4 * np.abs(add)
            A = al * A + np.abs(add)
            dx = d[:, None] * x[row, t]
            y[row, t] = np.einsum("hvk,hk->hv", S, ct) + dx
            y_abs[row, t] = np.einsum("hvk,hk->hv", A, np.abs(ct)) + np.abs(dx)
            y_units[row, t] = np.einsum("hvk,hk->hv", E, np.abs(ct)) + (dk + 2) * y_abs[row, t]
        hT[n], h_units[n] = S, E
    return y, hT, y_abs, y_units, h_units


def chunk_terms(x, b, c, dt, a, dt_bias=None, h0=None, cu_seqlens=None, soft=False, chunk=128):
    """How y comes about when a sequence is run in chunks: per output sum |terms| of its own
    chunk, sum |terms| from before it, and the sum of the squares of what an evaluation with
    rounded scores, weighted values and states rounds -- each score times its value, each
    weighted value's and each state element's part of the output."""
    x, b, c, dt, a = f64(x), f64(b), f64(c), f64(dt), f64(a)
    B, T, HV, dv = x.shape
    HK, dk = b.shape[2:]
    delta = dt + (0 if dt_bias is None else f64(dt_bias))
    delta = softplus(delta) if soft else delta
    if cu_seqlens is None:
        spans = [(n, n, 0, T) for n in range(B)]
    else:
        cu = [int(v) for v in cu_seqlens]
        spans = [(n, 0, cu[n], cu[n + 1]) for n in range(len(cu) - 1)]
    near, far, squares = np.zeros(x.shape), np.zeros(x.shape), np.zeros(x.shape)
    for n, row, t0, t1 in spans:
        for h in range(HV):
            g = h // (HV // HK)
            S = np.zeros((dv, dk)) if h0 is None else f64(h0)[n, h].copy()
            A, V = np.abs(S), np.zeros((dv, dk, dk))     # sum |terms|; sum of w^2 x^2 b b^T
            for s in range(t0, t1, chunk):
                at = slice(s, min(s + chunk, t1))
                X, Bm, Cm, dl = x[row, at, h], b[row, at, g], c[row, at, g], delta[row, at, h]
                run = np.cumsum(dl * a[h])
                low = np.tri(len(run), dtype=bool)
                score = np.exp(np.where(low, run[:, None] - run[None], -np.inf)) * dl * (Cm @ Bm.T)
                into = np.exp(run)[:, None]
                terms = np.exp(np.where(low, run[:, None] - run[None], -np.inf)) * dl * (np.abs(Cm) @ np.abs(Bm).T)
                near[row, at, h] = terms @ np.abs(X)
                far[row, at, h] = into * (np.abs(Cm) @ A.T)
                squares[row, at, h] = (score ** 2) @ (X ** 2) + into ** 2 * (
                    (Cm ** 2) @ (S ** 2).T + np.einsum("tk,vkl,tl->tv", Cm, V, Cm, optimize=True))
                w = dl * np.exp(run[-1] - run)
                keep = np.exp(run[-1])
                S = keep * S + (w[:, None] * X).T @ Bm
                A = keep * A + (w[:, None] * np.abs(X)).T @ np.abs(Bm)
                V = keep ** 2 * V + np.einsum("tv,tk,tl->vkl", (w[:, None] * X) ** 2, Bm, Bm, optimize=True)
    return near, far, squares


def conv_token(row, weight, bias, state, silu):
    """One token of the short convolution: row [N,C], state [N,W-1,C] -> out, new state."""
    row, weight, state = f64(row), f64(weight), f64(state)
    taps = np.concatenate([state, row[:, None]], axis=1)
    out = np.einsum("nwc,cw->nc", taps, weight) + (0 if bias is None else f64(bias))
    return (out * sigmoid(out) if silu else out), taps[:, 1:]


def step(xbc, dt, a, state, d=None, dt_bias=None, soft=False):
    """One token after its convolution: xbc [N,C], state [N,HV,dv,dk] -> y, state, y_abs,
    y_units, h_units."""
    state = f64(state)
    N, HV, dv, dk = state.shape
    xbc = f64(xbc)
    HK = (xbc.shape[1] - HV * dv) // (2 * dk)
    x = xbc[:, :HV * dv].reshape(N, 1, HV, dv)
    b = xbc[:, HV * dv:HV * dv + HK * dk].reshape(N, 1, HK, dk)
    c = xbc[:, HV * dv + HK * dk:].reshape(N, 1, HK, dk)
    y, hT, ya, yu, hu = scan(x, b, c, f64(dt)[:, None], a, d, dt_bias, state, None, soft)
    return y[:, 0], hT, ya[:, 0], yu[:, 0], hu


def gate(z, act):
    return sigmoid(z) * (z if act == "silu" else 1)


def rms(u, eps):
    return u / np.sqrt(np.mean(u * u, axis=-1, keepdims=True) + eps)


def gated_norm(o, z, weight, eps, act, gate_first, unit_offset):
    o = f64(o)
    f = 1.0 if z is None else gate(f64(z), act)
    w = 1.0 if weight is None else f64(weight) + (1 if unit_offset else 0)
    return rms(o * f, eps) * w if gate_first else rms(o, eps) * w * f


def residual_norm(x, residual, weight, post_weight, z, scale, eps, act, unit_offset):
    off = 1 if unit_offset else 0
    t = f64(x)
    if post_weight is not None:
        t = rms(t, eps) * (f64(post_weight) + off)
    if z is not None:
        t = t * gate(f64(z), act)
    h = scale * t + (0 if residual is None else f64(residual))
    return rms(h, eps) * (1.0 if weight is None else f64(weight) + off), h, scale * t
