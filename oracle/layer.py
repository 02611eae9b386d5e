"""TEST INFRASTRUCTURE ONLY: the operators around the SSD in a Mamba-2 layer,
fp64, CPU: the short causal convolution, the single-token state update and the
norms around a block.

The pages list the layer's kernels (clova.ai page, table "Share of compute time
by kernel") without writing these steps out; the readings are the Mamba-2
layer's depthwise causal convolution with SiLU, one step of the recurrence
(include/ssd.h), and RMS norms after and before a block with a gate, a
residual scale and the residual sum between them.  Plain numpy, one token at a
time.  Pinned in tests/test_oracle_layer.py against torch's conv1d, silu and
rms_norm, autograd, central finite differences, and the C recurrence.
"""
from __future__ import annotations

import math

import numpy as np

from .recurrence import seq_ranges, to_f64


def _sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def conv_fwd(x, w, bias=None, init=None, cu_seqlens=None, silu=True):
    """x (b, T, C), w (C, K), init (nseq, K-1, C).  Returns (out, final, pre);
    out and pre are NaN for tokens outside every sequence."""
    x, w, bias, init = to_f64(x), to_f64(w), to_f64(bias), to_f64(init)
    b, T, C = x.shape
    K = w.shape[1]
    starts, lens = seq_ranges(b, T, cu_seqlens)
    flat = x.reshape(b * T, C)
    pre = np.full((b * T, C), np.nan)
    final = np.zeros((len(starts), K - 1, C))
    for s, (st, n) in enumerate(zip(starts, lens)):
        rows = [init[s, k] if init is not None else np.zeros(C) for k in range(K - 1)]
        for t in range(n):
            rows.append(flat[st + t])
            v = np.zeros(C) if bias is None else bias.copy()
            for k in range(K):
                v = v + w[:, k] * rows[t + k]
            pre[st + t] = v
        final[s] = np.stack(rows[len(rows) - (K - 1):])
    out = pre * _sigmoid(pre) if silu else pre.copy()
    return out.reshape(b, T, C), final, pre.reshape(b, T, C)


def conv_bwd(x, w, dout, bias=None, init=None, cu_seqlens=None, silu=True, dfinal=None):
    """Gradients of sum(out * dout) + sum(final * dfinal): a dict with x, weight,
    bias, init and dpre (the gradient at pre).  x's rows outside every sequence
    are NaN."""
    _, _, pre = conv_fwd(x, w, bias, init, cu_seqlens, silu)
    x, w, dout, init, dfinal = (to_f64(v) for v in (x, w, dout, init, dfinal))
    b, T, C = x.shape
    K = w.shape[1]
    starts, lens = seq_ranges(b, T, cu_seqlens)
    flat, d, pre = x.reshape(b * T, C), dout.reshape(b * T, C), pre.reshape(b * T, C)
    sg = _sigmoid(pre)
    dpre = d * (sg * (1.0 + pre * (1.0 - sg))) if silu else d.copy()
    dx = np.full((b * T, C), np.nan)
    dinit = np.zeros((len(starts), K - 1, C))
    dw, db = np.zeros((C, K)), np.zeros(C)
    for s, (st, n) in enumerate(zip(starts, lens)):
        rows = np.zeros((n + K - 1, C))               # initial state, then the tokens
        if init is not None:
            rows[:K - 1] = init[s]
        rows[K - 1:] = flat[st:st + n]
        drows = np.zeros_like(rows)
        for t in range(n):
            db += dpre[st + t]
            for k in range(K):
                drows[t + k] += w[:, k] * dpre[st + t]
                dw[:, k] += rows[t + k] * dpre[st + t]
        if dfinal is not None:
            drows[n:] += dfinal[s]
        dinit[s] = drows[:K - 1]
        dx[st:st + n] = drows[K - 1:]
    return {"x": dx.reshape(b, T, C), "weight": dw, "bias": db, "initial_states": dinit,
            "dpre": dpre.reshape(b, T, C)}


def padding_rows(slots, batch, nslots):
    """Rows that take no step: no slot of the cache, or an earlier row's slot."""
    if slots is None:
        return [False] * batch
    seen, pad = set(), []
    for v in slots:
        v = int(v)
        pad.append(not 0 <= v < nslots or v in seen)
        seen.add(v)
    return pad


def conv_step(x, states, w, bias=None, slots=None, silu=True):
    """x (batch, C), states (nslots, K-1, C).  Returns (out, new states); out is
    NaN in padding's rows."""
    x, states, w, bias = to_f64(x), to_f64(states).copy(), to_f64(w), to_f64(bias)
    out = np.full(x.shape, np.nan)
    pad = padding_rows(slots, x.shape[0], states.shape[0])
    for b in range(x.shape[0]):
        if pad[b]:
            continue
        s = b if slots is None else int(slots[b])
        o, f, _ = conv_fwd(x[b][None, None], w, bias, states[s][None], None, silu)
        out[b], states[s] = o[0, 0], f[0]
    return out, states


def ssd_step(x, dt, A, B, C, states, D=None, dt_bias=None, slots=None, dt_min=0.0,
             dt_max=math.inf):
    """x (batch, H, P), dt (batch, H), B, C (batch, G, N), states (nslots, H, P,
    N).  Returns (out, new states); out is NaN in padding's rows."""
    x, dt, A, B, C, D, dt_bias = (to_f64(v) for v in (x, dt, A, B, C, D, dt_bias))
    states = to_f64(states).copy()
    batch, H, P = x.shape
    G = B.shape[1]
    out = np.full(x.shape, np.nan)
    pad = padding_rows(slots, batch, states.shape[0])
    for b in range(batch):
        if pad[b]:
            continue
        s = b if slots is None else int(slots[b])
        for h in range(H):
            g = h // (H // G)
            u = dt[b, h] + (dt_bias[h] if dt_bias is not None else 0.0)
            delta = min(max(np.logaddexp(0.0, u), dt_min), dt_max)
            hs = math.exp(delta * A[h]) * states[s, h] + delta * np.outer(x[b, h], B[b, g])
            states[s, h] = hs
            out[b, h] = hs @ C[b, g] + (D[h] * x[b, h] if D is not None else 0.0)
    return out, states


def gate_act(kind, z):
    """The gate's factor and its derivative."""
    if kind == "linear":
        return z, np.ones_like(z)
    s = _sigmoid(z)
    if kind == "sigmoid":
        return s, s * (1.0 - s)
    return z * s, s * (1.0 + z * (1.0 - s))


def block_norm_fwd(x, residual, pre_w, gate=None, kind="sigmoid", post_w=None, scale=None,
                   alpha=1.0, eps=1e-5):
    """Rows (T, C).  Returns (out, h)."""
    x, residual, pre_w, gate, post_w, scale = (to_f64(v) for v in (x, residual, pre_w, gate, post_w,
                                                                   scale))
    p = x
    if post_w is not None:
        p = x / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps) * post_w
    if gate is not None:
        p = p * gate_act(kind, gate)[0]
    h = alpha * p if scale is None else alpha * scale * p
    if residual is not None:
        h = h + residual
    return h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * pre_w, h


def block_norm_bwd(x, residual, pre_w, dout, dh_out=None, gate=None, kind="sigmoid", post_w=None,
                   scale=None, alpha=1.0, eps=1e-5):
    """Gradients of sum(out * dout) + sum(h * dh_out): a dict."""
    _, h = block_norm_fwd(x, residual, pre_w, gate, kind, post_w, scale, alpha, eps)
    x, pre_w, dout, dh_out, gate, post_w, scale = (
        to_f64(v) for v in (x, pre_w, dout, dh_out, gate, post_w, scale))
    g = {}
    r2 = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    n, dn = h * r2, dout * pre_w
    dh = r2 * (dn - n * np.mean(dn * n, axis=1, keepdims=True))
    if dh_out is not None:
        dh = dh + dh_out
    g["pre_weight"], g["residual"] = np.sum(dout * n, axis=0), dh
    act, dact = gate_act(kind, gate) if gate is not None else (np.ones_like(x), np.zeros_like(x))
    m, p = x, x
    if post_w is not None:
        r1 = 1.0 / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)
        m = x * r1
        p = m * post_w
    if scale is not None:
        g["scale"] = np.sum(dh * alpha * p * act, axis=0)
    du = dh * alpha * (scale if scale is not None else 1.0)
    if gate is not None:
        g["gate"] = du * p * dact
    dp = du * act
    if post_w is not None:
        g["post_weight"] = np.sum(dp * m, axis=0)
        dm = dp * post_w
        dp = r1 * (dm - m * np.mean(dm * m, axis=1, keepdims=True))
    g["x"] = dp
    return g
