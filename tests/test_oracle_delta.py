"""Pins of the gated delta rule's and the query/key norm's fp64 oracle (CPU)."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import delta
from oracle.recurrence import ssd_recurrence


def draw(b=1, T=9, H=4, G=2, P=3, N=5, seed=0, unit=True):
    r = np.random.default_rng(seed)
    q, k = r.standard_normal((b, T, G, N)), r.standard_normal((b, T, G, N))
    if unit:
        q, k = (x / np.linalg.norm(x, axis=-1, keepdims=True) for x in (q, k))
    return dict(q=q, k=k, v=r.standard_normal((b, T, H, P)), g=-r.random((b, T, H)),
                beta=r.random((b, T, H)), scale=0.4)


def torch_fwd(q, k, v, g, beta, scale, init):
    """The recurrence as products with (1 - beta k k^T), for autograd."""
    b, T, G, N = q.shape
    H = v.shape[2]
    S, outs = init, []
    for t in range(T):
        kt = k[:, t].repeat_interleave(H // G, 1)
        S = torch.exp(g[:, t])[..., None, None] * (
            S - beta[:, t, :, None, None] * (S @ kt[..., None]) * kt[..., None, :])
        S = S + (beta[:, t, :, None] * v[:, t])[..., None] * kt[..., None, :]
        outs.append(scale * (S @ q[:, t].repeat_interleave(H // G, 1)[..., None])[..., 0])
    return torch.stack(outs, 1), S


@pytest.mark.parametrize("G", [1, 2, 4])
def test_against_autograd_of_another_form(G):
    x = draw(b=2, G=G)
    r = np.random.default_rng(1)
    init, do, df = r.standard_normal((2, 4, 3, 5)), r.standard_normal((2, 9, 4, 3)), r.standard_normal((2, 4, 3, 5))
    t = {n: torch.tensor(v, requires_grad=True) for n, v in x.items() if n != "scale"}
    ti = torch.tensor(init, requires_grad=True)
    out, S = torch_fwd(**t, scale=x["scale"], init=ti)
    o, f, w, _ = delta.delta_fwd(**x, init=init)
    np.testing.assert_allclose(o, out.detach().numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(f, S.detach().numpy(), rtol=1e-12, atol=1e-13)
    ((out * torch.tensor(do)).sum() + (S * torch.tensor(df)).sum()).backward()
    d = delta.delta_bwd(**{n: x[n] for n in ("q", "k", "v", "g", "beta", "scale")}, dout=do, init=init, dfinal=df)
    for n in ("q", "k", "v", "g", "beta"):
        np.testing.assert_allclose(d[n], t[n].grad.numpy(), rtol=1e-11, atol=1e-12, err_msg=n)
    np.testing.assert_allclose(d["init"], ti.grad.numpy(), rtol=1e-11, atol=1e-12)


def test_gradients_by_central_differences():
    x = draw(T=5)
    r = np.random.default_rng(2)
    init, do, df = r.standard_normal((1, 4, 3, 5)), r.standard_normal((1, 5, 4, 3)), r.standard_normal((1, 4, 3, 5))

    def loss(y, i):
        o, f, _, _ = delta.delta_fwd(**y, init=i)
        return np.sum(o * do) + np.sum(f * df)

    d = delta.delta_bwd(**x, dout=do, init=init, dfinal=df)
    for n in ("q", "k", "v", "g", "beta", "init"):
        u = r.standard_normal((init if n == "init" else x[n]).shape)
        h = 1e-5
        if n == "init":
            num = (loss(x, init + h * u) - loss(x, init - h * u)) / (2 * h)
        else:
            num = (loss({**x, n: x[n] + h * u}, init) - loss({**x, n: x[n] - h * u}, init)) / (2 * h)
        assert abs(num - np.sum(d[n] * u)) <= 1e-7 * max(1.0, abs(num)), n


def test_without_what_it_forgets_it_is_the_ssd():
    """Keys that never overlap: each token writes where nothing was, S k is zero, and the rule is
    the SSD with x = beta v, B = k, C = q and exp(g) as decay."""
    T, H, G, P, N = 6, 4, 2, 3, 6
    x = draw(T=T, H=H, G=G, P=P, N=N)
    x["k"] = np.broadcast_to(np.eye(N)[None, :, None, :], (1, T, G, N)).copy()
    o, f, w, _ = delta.delta_fwd(**x)
    np.testing.assert_allclose(w, x["beta"][..., None] * x["v"])
    # the SSD with delta = 1 (dt is raw: log(e - 1)) and one A per head, so one g per head
    x["g"][:] = x["g"][:, :1]
    o, f, w, _ = delta.delta_fwd(**x)
    dt = np.full((1, T, H), np.log(np.expm1(1.0)))
    y, fs = ssd_recurrence(torch.tensor(w), torch.tensor(dt), None, torch.tensor(x["g"][0, 0]),
                           torch.tensor(x["k"]), torch.tensor(x["q"]), None)
    np.testing.assert_allclose(o, x["scale"] * y, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(f, fs, rtol=1e-10, atol=1e-12)


def test_step_of_one_stores_what_it_is_told():
    """beta 1, no decay: after a token, its (unit) key reads back its value, and orthogonal
    directions are as before."""
    x = draw(T=1)
    x["beta"][:], x["g"][:] = 1.0, 0.0
    init = np.random.default_rng(3).standard_normal((1, 4, 3, 5))
    _, f, _, _ = delta.delta_fwd(**x, init=init)
    k = np.repeat(x["k"][0, 0], 2, 0)
    np.testing.assert_allclose(np.einsum("hpn,hn->hp", f[0], k), x["v"][0, 0], atol=1e-12)
    u = np.random.default_rng(4).standard_normal((4, 5))
    u -= np.sum(u * k, 1, keepdims=True) * k
    np.testing.assert_allclose(np.einsum("hpn,hn->hp", f[0], u), np.einsum("hpn,hn->hp", init[0], u), atol=1e-12)


def test_packed_sequences_do_not_meet():
    x = draw(T=11)
    cu = [1, 1, 4, 9]
    init = np.random.default_rng(5).standard_normal((3, 4, 3, 5))
    do = np.random.default_rng(6).standard_normal((1, 11, 4, 3))
    o, f, w, st = delta.delta_fwd(**x, init=init, cu_seqlens=cu, every=2)
    d = delta.delta_bwd(**x, dout=do, init=init, cu_seqlens=cu)
    assert np.isnan(o[:, [0, 9, 10]]).all() and not np.isnan(o[:, 1:9]).any()
    np.testing.assert_array_equal(f[0], init[0])
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        part = {n: v[:, a:b] if n != "scale" else v for n, v in x.items()}
        po, pf, _, _ = delta.delta_fwd(**part, init=init[s:s + 1])
        np.testing.assert_array_equal(o[:, a:b], po)
        np.testing.assert_array_equal(f[s], pf[0])
        assert len(st[s]) == (b - a + 1) // 2
        pd = delta.delta_bwd(**part, dout=do[:, a:b], init=init[s:s + 1])
        for n in ("q", "k", "v", "g", "beta"):
            np.testing.assert_array_equal(d[n][:, a:b], pd[n])
            assert not d[n][:, [0, 9, 10]].any()


def test_step_is_the_rule_on_slots():
    r = np.random.default_rng(7)
    x = draw(b=1, T=4)
    row = {n: v[0] if n != "scale" else v for n, v in x.items()}
    st = r.standard_normal((3, 4, 3, 5))
    out, new = delta.delta_step(**row, states=st, slots=[2, -1, 2, 0])
    o, f, _, _ = delta.delta_fwd(*(x[n][:, :1] for n in ("q", "k", "v", "g", "beta")), x["scale"], st[2:3])
    np.testing.assert_array_equal(out[0], o[0, 0])
    np.testing.assert_array_equal(new[2], f[0])
    assert np.isnan(out[1]).all() and np.isnan(out[2]).all()
    np.testing.assert_array_equal(new[1], st[1])


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("R,interleaved", [(0, False), (3, False), (3, True), (4, False)])
def test_head_norm(norm, weight, R, interleaved):
    r = np.random.default_rng(8)
    D = 8
    x, d = r.standard_normal((5, 2, D)), r.standard_normal((5, 2, D))
    w = 1 + 0.3 * r.standard_normal(D) if weight else None
    rot = dict(positions=r.integers(-5, 1000, 5), inv_freq=r.random(R), interleaved=interleaved) if R else {}
    y = delta.head_norm_fwd(x, w, norm, 1e-3, **rot)
    tx = torch.tensor(x, requires_grad=True)
    tw = torch.tensor(w, requires_grad=True) if weight else None
    if norm == "rms":
        ty = F.rms_norm(tx, (D,), tw, 1e-3)
    else:
        ty = tx / torch.sqrt((tx * tx).sum(-1, keepdim=True) + 1e-3) * (tw if weight else 1.0)
    if R:
        # as a product with a rotation matrix per position
        m = torch.eye(D, dtype=torch.float64).repeat(5, 1, 1)
        a = torch.tensor(rot["positions"])[:, None] * torch.tensor(rot["inv_freq"])
        i = torch.arange(R)
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + R)
        m[:, p, p], m[:, q, q], m[:, p, q], m[:, q, p] = torch.cos(a), torch.cos(a), -torch.sin(a), torch.sin(a)
        ty = torch.einsum("tde,the->thd", m, ty)
    np.testing.assert_allclose(y, ty.detach().numpy(), rtol=1e-11, atol=1e-12)
    (ty * torch.tensor(d)).sum().backward()
    dx, dw = delta.head_norm_bwd(x, d, w, norm, 1e-3, **rot)
    np.testing.assert_allclose(dx, tx.grad.numpy(), rtol=1e-10, atol=1e-11)
    if weight:
        np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-10, atol=1e-11)
    else:
        assert dw is None
