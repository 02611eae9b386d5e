"""The gated delta rule and its gradients in 64 bits, one token at a time, on whatever device the
inputs are on: oracle/delta.py's recurrence for sizes that are slow there.  tests/test_delta_device.py
holds it to the oracle."""
import torch

from tests.delta_cases import TOL_GATE, TOL_STATE, inside, within
from tests.helpers import assert_close


def _ranges(b, T, cu):
    if cu is None:
        return [(s * T, T) for s in range(b)]
    return [(int(a), int(z) - int(a)) for a, z in zip(cu[:-1], cu[1:])]


def rule(x, scale, cu=None, dout=None, dfinal=None):
    """x: q, k (b, T, G, N), v (b, T, H, P), g, beta (b, T, H), initial_states or None.  Returns out,
    final and, with dout, the gradients as a dict; rows of tokens outside every sequence are zeros.
    Equal rows run side by side."""
    d = {n: (None if t is None else t.double()) for n, t in x.items()}
    b, T, H, P = d["v"].shape
    N, rep = d["q"].shape[-1], H // d["q"].shape[2]
    q, k = (d[n].repeat_interleave(rep, 2).flatten(0, 1) for n in "qk")
    v, g, beta = (d[n].flatten(0, 1) for n in ("v", "g", "beta"))
    do = None if dout is None else dout.double().flatten(0, 1)
    spans = _ranges(b, T, cu)
    groups = [list(range(b))] if cu is None else [[s] for s in range(len(spans))]
    zeros = lambda: torch.zeros((len(spans), H, P, N), dtype=torch.float64, device=v.device)  # noqa: E731
    init = zeros() if d["initial_states"] is None else d["initial_states"]
    out, final = torch.zeros_like(v), zeros()
    grads = None if do is None else dict(q=torch.zeros_like(q), k=torch.zeros_like(k), v=torch.zeros_like(v),
                                         g=torch.zeros_like(g), beta=torch.zeros_like(beta), init=zeros())
    mul = lambda S, y: (S * y[..., None, :]).sum(-1)  # noqa: E731
    tmul = lambda S, y: (S * y[..., :, None]).sum(-2)  # noqa: E731
    outer = lambda y, z: y[..., :, None] * z[..., None, :]  # noqa: E731
    for seqs in groups:
        at = torch.tensor([spans[s][0] for s in seqs], device=v.device)
        n = spans[seqs[0]][1]
        S, states = init[seqs], []
        for t in range(n):
            i = at + t
            states.append(S)
            A = S * torch.exp(g[i])[..., None, None]
            S = A + outer(beta[i][..., None] * (v[i] - mul(A, k[i])), k[i])
            out[i] = scale * mul(S, q[i])
        final[seqs] = S
        if do is None:
            continue
        states.append(S)
        dS = zeros()[seqs] if dfinal is None else dfinal.double()[seqs]
        for t in reversed(range(n)):
            i = at + t
            a, be = torch.exp(g[i])[..., None, None], beta[i][..., None]
            A = states[t] * a
            miss = v[i] - mul(A, k[i])
            grads["q"][i] = scale * tmul(states[t + 1], do[i])
            dS = dS + scale * outer(do[i], q[i])
            dw = mul(dS, k[i])
            grads["k"][i] = tmul(dS, be * miss) - tmul(A, be * dw)
            grads["beta"][i] = (dw * miss).sum(-1)
            grads["v"][i] = be * dw
            dS = dS - outer(be * dw, k[i])
            grads["g"][i] = (dS * A).sum((-1, -2))
            dS = dS * a
        grads["init"][seqs] = dS
    if grads is not None:
        for name in "qk":
            grads[name] = grads[name].unflatten(1, (-1, rep)).sum(2)
        grads = {n: (t if n == "init" else t.unflatten(0, (b, T))) for n, t in grads.items()}
    return out.unflatten(0, (b, T)), final, grads


def check(x, scale, cu=None, dout=None, dfinal=None, forward=None, backward=None):
    """delta_fwd's and delta_bwd's results on `x` (on the GPU) against the rule."""
    out, final, ref = rule(x, scale, cu, dout if backward is not None else None, dfinal)
    dt = "f32" if x["q"].dtype == torch.float32 else "bf16"
    m = inside(x, cu).to(out.device)
    if forward is not None:
        assert_close(forward[0][m], out[m].cpu().numpy(), dt, "out")
        within(forward[1], final.cpu().numpy(), TOL_STATE[dt], "states")
    if backward is None:
        return
    for n in ("q", "k", "v", "g", "beta"):
        r = ref[n].cpu().numpy()
        if dt == "f32":
            within(backward[n], r, 1e-4, n)
        elif n in ("g", "beta") and x["g"].dtype == torch.float32:
            within(backward[n], r, TOL_GATE[dt], n)
        else:
            assert_close(backward[n], r, "bf16", n)
    if x["initial_states"] is not None:
        within(backward["initial_states"], ref["init"].cpu().numpy(), TOL_GATE[dt], "initial_states")
