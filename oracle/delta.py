"""TEST INFRASTRUCTURE ONLY: the gated delta rule and the norm of queries and keys with its
rotation, fp64, CPU, one token at a time.

The reference names gated delta networks among the layers of hybrid models (clova.ai page,
"Why optimize Mamba-2?") without writing them out; the reading is the published gated delta
rule (include/ssd.h), its gradients by reverse differentiation of the same steps.  Plain numpy.
Pinned in tests/test_oracle_delta.py against autograd, central finite differences, the SSD
recurrence, a least-squares property and torch's rms_norm.
"""
from __future__ import annotations

import numpy as np

from .layer import padding_rows
from .recurrence import seq_ranges, to_f64


def delta_fwd(q, k, v, g, beta, scale, init=None, cu_seqlens=None, every=64):
    """q, k (b, T, G, N), v (b, T, H, P), g, beta (b, T, H), init (nseq, H, P, N).  Returns (out,
    final, w, starts): out and the rows w like v, NaN for tokens outside every sequence; starts:
    the state before every `every`-th token of each sequence, a list per sequence."""
    q, k, v, g, beta, init = (to_f64(x) for x in (q, k, v, g, beta, init))
    b, T, G, N = q.shape
    H, P = v.shape[2:]
    rep = H // G
    fl = lambda x: x.reshape((b * T,) + x.shape[2:])  # noqa: E731
    q, k, v, g, beta = (fl(x) for x in (q, k, v, g, beta))
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    begin, lens = seq_ranges(b, T, cu_seqlens)
    out, w = np.full((b * T, H, P), np.nan), np.full((b * T, H, P), np.nan)
    final, starts = np.zeros((len(begin), H, P, N)), []
    for s, (at, n) in enumerate(zip(begin, lens)):
        S = np.zeros((H, P, N)) if init is None else init[s].copy()
        starts.append([])
        for t in range(n):
            if t % every == 0:
                starts[-1].append(S.copy())
            i = at + t
            S = S * np.exp(g[i])[:, None, None]
            w[i] = beta[i][:, None] * (v[i] - np.einsum("hpn,hn->hp", S, k[i]))
            S = S + w[i][:, :, None] * k[i][:, None, :]
            out[i] = scale * np.einsum("hpn,hn->hp", S, q[i])
        final[s] = S
    shape = (b, T, H, P)
    return out.reshape(shape), final, w.reshape(shape), starts


def delta_bwd(q, k, v, g, beta, dout, scale, init=None, cu_seqlens=None, dfinal=None):
    """Gradients of sum(out * dout) + sum(final * dfinal): a dict with q, k, v, g, beta and
    init; rows of tokens outside every sequence are zeros."""
    q, k, v, g, beta, dout, init, dfinal = (to_f64(x) for x in (q, k, v, g, beta, dout, init, dfinal))
    b, T, G, N = q.shape
    H, P = v.shape[2:]
    rep = H // G
    shapes = dict(q=q.shape, k=k.shape, v=v.shape, g=g.shape, beta=beta.shape)
    fl = lambda x: x.reshape((b * T,) + x.shape[2:])  # noqa: E731
    q, k, v, g, beta, dout = (fl(x) for x in (q, k, v, g, beta, dout))
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    begin, lens = seq_ranges(b, T, cu_seqlens)
    d = dict(q=np.zeros_like(q), k=np.zeros_like(k), v=np.zeros_like(v), g=np.zeros_like(g),
             beta=np.zeros_like(beta), init=np.zeros((len(begin), H, P, N)))
    mul = lambda S, x: np.einsum("hpn,hn->hp", S, x)  # noqa: E731
    tmul = lambda S, x: np.einsum("hpn,hp->hn", S, x)  # noqa: E731
    outer = lambda x, y: x[:, :, None] * y[:, None, :]  # noqa: E731
    for s, (at, n) in enumerate(zip(begin, lens)):
        S = [np.zeros((H, P, N)) if init is None else init[s]]
        for i in range(at, at + n):
            A = S[-1] * np.exp(g[i])[:, None, None]
            S.append(A + outer(beta[i][:, None] * (v[i] - mul(A, k[i])), k[i]))
        dS = np.zeros((H, P, N)) if dfinal is None else dfinal[s].copy()
        for t in reversed(range(n)):
            i = at + t
            a = np.exp(g[i])
            A = S[t] * a[:, None, None]
            miss = v[i] - mul(A, k[i])
            d["q"][i] = scale * tmul(S[t + 1], dout[i])
            dS = dS + scale * outer(dout[i], q[i])
            dw = mul(dS, k[i])
            d["k"][i] = tmul(dS, beta[i][:, None] * miss) - tmul(A, beta[i][:, None] * dw)
            d["beta"][i] = np.sum(dw * miss, 1)
            d["v"][i] = beta[i][:, None] * dw
            dA = dS - outer(beta[i][:, None] * dw, k[i])
            d["g"][i] = np.sum(dA * A, (1, 2))
            dS = dA * a[:, None, None]
        d["init"][s] = dS
    for x in ("q", "k"):
        d[x] = d[x].reshape(b * T, G, rep, N).sum(2)
    for x, sh in shapes.items():
        d[x] = d[x].reshape(sh)
    return d


def delta_step(q, k, v, g, beta, states, scale, slots=None):
    """q, k (batch, G, N), v (batch, H, P), g, beta (batch, H), states (nslots, H, P, N).
    Returns (out, new states); out is NaN in padding's rows."""
    q, k, v, g, beta, states = (to_f64(x) for x in (q, k, v, g, beta, states))
    states = states.copy()
    out = np.full(v.shape, np.nan)
    pad = padding_rows(slots, v.shape[0], states.shape[0])
    for b in range(v.shape[0]):
        if pad[b]:
            continue
        s = b if slots is None else int(slots[b])
        o, f, _, _ = delta_fwd(q[None, b:b + 1], k[None, b:b + 1], v[None, b:b + 1], g[None, b:b + 1],
                               beta[None, b:b + 1], scale, states[s][None])
        out[b], states[s] = o[0, 0], f[0]
    return out, states


def turns(positions, inv_freq):
    """cos and sin of position times frequency, (..., 1, R)."""
    a = to_f64(positions)[..., None, None] * to_f64(inv_freq)
    return np.cos(a), np.sin(a)


def rotate(x, cos, sin, interleaved):
    R = cos.shape[-1]
    y = x.copy()
    a, b = (np.s_[..., 0:2 * R:2], np.s_[..., 1:2 * R:2]) if interleaved else \
        (np.s_[..., :R], np.s_[..., R:2 * R])
    y[a] = x[a] * cos - x[b] * sin
    y[b] = x[b] * cos + x[a] * sin
    return y


def _scale_of(x, norm, eps):
    m = np.mean(x * x, -1, keepdims=True) if norm == "rms" else np.sum(x * x, -1, keepdims=True)
    return 1.0 / np.sqrt(m + eps)


def head_norm_fwd(x, weight=None, norm="rms", eps=1e-6, positions=None, inv_freq=None,
                  interleaved=False):
    """x (..., heads, D): q or k."""
    x, weight = to_f64(x), to_f64(weight)
    y = x * _scale_of(x, norm, eps)
    if weight is not None:
        y = y * weight
    return y if positions is None else rotate(y, *turns(positions, inv_freq), interleaved)


def head_norm_bwd(x, dout, weight=None, norm="rms", eps=1e-6, positions=None, inv_freq=None,
                  interleaved=False):
    """Gradients of sum(out * dout): (dx, dweight or None)."""
    x, weight, d = to_f64(x), to_f64(weight), to_f64(dout)
    if positions is not None:
        cos, sin = turns(positions, inv_freq)
        d = rotate(d, cos, -sin, interleaved)
    r = _scale_of(x, norm, eps)
    n = x * r
    dw = None if weight is None else np.sum(d * n, tuple(range(d.ndim - 1)))
    dn = d if weight is None else d * weight
    dot = np.mean(dn * n, -1, keepdims=True) if norm == "rms" else np.sum(dn * n, -1, keepdims=True)
    return r * (dn - n * dot), dw
