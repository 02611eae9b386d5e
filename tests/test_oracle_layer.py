"""The fp64 oracle of the operators around the SSD, pinned to things other than
itself (CPU): torch's conv1d, silu and rms_norm, autograd, central finite
differences, hand-derived values and the C recurrence."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import layer
from oracle.recurrence import ssd_recurrence

T64 = torch.float64


def rnd(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=T64)


def test_conv_by_hand():
    # one channel, taps 1, 10, 100 (the last on the token itself), no activation
    x = torch.tensor([[[1.0], [2.0], [3.0]]], dtype=T64)
    w = torch.tensor([[1.0, 10.0, 100.0]], dtype=T64)
    out, final, _ = layer.conv_fwd(x, w, torch.tensor([0.5], dtype=T64),
                                   torch.tensor([[[7.0], [8.0]]], dtype=T64), silu=False)
    assert out[0, :, 0].tolist() == [187.5, 218.5, 321.5]
    assert final[0, :, 0].tolist() == [2.0, 3.0]
    # a sequence shorter than the state keeps rows of it
    _, final, _ = layer.conv_fwd(x[:, :1], w, None, torch.tensor([[[7.0], [8.0]]], dtype=T64))
    assert final[0, :, 0].tolist() == [8.0, 1.0]


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_equals_torch_conv1d_and_autograd(K, silu):
    b, T, C = 2, 9, 5
    x, w, bias = rnd(b, T, C, seed=1), rnd(C, K, seed=2), rnd(C, seed=3)
    init, dout, dfin = rnd(b, K - 1, C, seed=4), rnd(b, T, C, seed=5), rnd(b, K - 1, C, seed=6)
    leaves = [v.clone().requires_grad_(True) for v in (x, w, bias, init)]
    full = torch.cat([leaves[3], leaves[0]], 1)
    y = F.conv1d(full.transpose(1, 2), leaves[1][:, None], leaves[2], groups=C).transpose(1, 2)
    y = F.silu(y) if silu else y
    fin = full[:, T:]
    ((y * dout).sum() + (fin * dfin).sum()).backward()
    out, final, _ = layer.conv_fwd(x, w, bias, init, silu=silu)
    np.testing.assert_allclose(out, y.detach().numpy(), rtol=0, atol=1e-13)
    np.testing.assert_array_equal(final, fin.detach().numpy())
    g = layer.conv_bwd(x, w, dout, bias, init, silu=silu, dfinal=dfin)
    for k, leaf in zip(("x", "weight", "bias", "initial_states"), leaves):
        np.testing.assert_allclose(g[k], leaf.grad.numpy(), rtol=0, atol=1e-12)


def test_conv_packed_equals_separate_runs():
    lens, C, K = (3, 0, 1, 6), 4, 4
    cu = torch.tensor([0, 3, 3, 4, 10], dtype=torch.int32)
    x, w, init, dout = rnd(1, 10, C, seed=1), rnd(C, K, seed=2), rnd(4, 3, C, seed=3), rnd(1, 10, C, seed=4)
    dfin = rnd(4, 3, C, seed=5)
    out, final, _ = layer.conv_fwd(x, w, None, init, cu)
    g = layer.conv_bwd(x, w, dout, None, init, cu, dfinal=dfin)
    dw = 0.0
    for s, n in enumerate(lens):
        sl = slice(int(cu[s]), int(cu[s]) + n)
        o, f, _ = layer.conv_fwd(x[:, sl], w, None, init[s:s + 1])
        h = layer.conv_bwd(x[:, sl], w, dout[:, sl], None, init[s:s + 1], dfinal=dfin[s:s + 1])
        np.testing.assert_array_equal(out[:, sl], o)
        np.testing.assert_array_equal(final[s], f[0])
        np.testing.assert_array_equal(g["x"][:, sl], h["x"])
        np.testing.assert_array_equal(g["initial_states"][s], h["initial_states"][0])
        dw = dw + h["weight"]
    np.testing.assert_allclose(g["weight"], dw, rtol=0, atol=1e-13)


def test_conv_steps_equal_one_prompt():
    C, K, T = 3, 4, 7
    x, w, bias = rnd(2, T, C, seed=1), rnd(C, K, seed=2), rnd(C, seed=3)
    out, final, _ = layer.conv_fwd(x, w, bias)
    states = np.zeros((5, K - 1, C))
    for t in range(T):
        y, states = layer.conv_step(x[:, t], states, w, bias, slots=[3, 1])
        np.testing.assert_allclose(y, out[:, t], rtol=0, atol=1e-15)
    np.testing.assert_array_equal(states[[3, 1]], final)
    assert not states[[0, 2, 4]].any()


def test_padding_rows():
    assert layer.padding_rows([2, -1, 2, 5, 0, 4], 6, 5) == [False, True, True, True, False, False]


def test_steps_equal_the_recurrence():
    H, P, N, G, T = 4, 3, 5, 2, 6
    x, dt = rnd(1, T, H, P, seed=1), rnd(1, T, H, seed=2) - 1
    A, B, C = -torch.exp(rnd(H, seed=3)), rnd(1, T, G, N, seed=4), rnd(1, T, G, N, seed=5)
    D, bias, init = rnd(H, seed=6), rnd(H, seed=7), rnd(1, H, P, N, seed=8)
    y, fin = ssd_recurrence(x, dt, bias, A, B, C, D, init=init, dt_min=0.2, dt_max=0.9)
    st = init.numpy()
    for t in range(T):
        o, st = layer.ssd_step(x[:, t], dt[:, t], A, B[:, t], C[:, t], st, D, bias, dt_min=0.2,
                               dt_max=0.9)
        np.testing.assert_allclose(o[0], y[0, t], rtol=0, atol=1e-12)
    np.testing.assert_allclose(st, fin, rtol=0, atol=1e-12)


@pytest.mark.parametrize("kind", [None, "linear", "sigmoid", "silu"])
@pytest.mark.parametrize("post", [True, False])
def test_block_norm_equals_torch_and_autograd(kind, post):
    T, C, alpha, eps = 4, 7, 0.3, 1e-3
    x, res, pre, sc = rnd(T, C, seed=1), rnd(T, C, seed=2), rnd(C, seed=3), rnd(C, seed=4)
    gate = rnd(T, C, seed=5) if kind else None
    pw = rnd(C, seed=6) if post else None
    dout, dh = rnd(T, C, seed=7), rnd(T, C, seed=8)
    leaves = {k: v.clone().requires_grad_(True) for k, v in
              dict(x=x, residual=res, pre_weight=pre, scale=sc, gate=gate, post_weight=pw).items()
              if v is not None}
    p = F.rms_norm(leaves["x"], (C,), leaves["post_weight"], eps) if post else leaves["x"]
    if kind:
        z = leaves["gate"]
        p = p * {"linear": lambda v: v, "sigmoid": torch.sigmoid, "silu": F.silu}[kind](z)
    h = leaves["residual"] + alpha * leaves["scale"] * p
    out = F.rms_norm(h, (C,), leaves["pre_weight"], eps)
    ((out * dout).sum() + (h * dh).sum()).backward()
    kw = dict(gate=gate, kind=kind, post_w=pw, scale=sc, alpha=alpha, eps=eps)
    o, hh = layer.block_norm_fwd(x, res, pre, **kw)
    np.testing.assert_allclose(o, out.detach().numpy(), rtol=0, atol=1e-13)
    np.testing.assert_allclose(hh, h.detach().numpy(), rtol=0, atol=1e-13)
    g = layer.block_norm_bwd(x, res, pre, dout, dh, **kw)
    assert set(g) == set(leaves)
    for k, leaf in leaves.items():
        np.testing.assert_allclose(g[k], leaf.grad.numpy(), rtol=0, atol=1e-12)


def test_gradients_by_finite_differences():
    T, C, K, e = 5, 3, 3, 1e-6
    x, w, bias, dout = rnd(1, T, C, seed=1), rnd(C, K, seed=2), rnd(C, seed=3), rnd(1, T, C, seed=4)
    g = layer.conv_bwd(x, w, dout, bias)

    def loss(x, w, bias):
        return float((layer.conv_fwd(x, w, bias)[0] * dout.numpy()).sum())
    args = dict(x=x, w=w, bias=bias)
    for k, name in (("x", "x"), ("w", "weight"), ("bias", "bias")):
        for i in range(args[k].numel()):
            d = torch.zeros_like(args[k])
            d.view(-1)[i] = e
            diff = (loss(**{**args, k: args[k] + d}) - loss(**{**args, k: args[k] - d})) / (2 * e)
            assert abs(diff - g[name].reshape(-1)[i]) < 1e-7

    res, pre, pw, gate = rnd(T, C, seed=5), rnd(C, seed=6), rnd(C, seed=7), rnd(T, C, seed=8)
    kw = dict(kind="silu", alpha=0.7)
    gb = layer.block_norm_bwd(x[0], res, pre, dout[0], gate=gate, post_w=pw, **kw)

    def nloss(**a):
        return float((layer.block_norm_fwd(a["x"], a["residual"], a["pre"], gate=a["gate"],
                                           post_w=a["pw"], **kw)[0] * dout[0].numpy()).sum())
    args = dict(x=x[0], residual=res, pre=pre, pw=pw, gate=gate)
    for k, name in (("x", "x"), ("residual", "residual"), ("pre", "pre_weight"),
                    ("pw", "post_weight"), ("gate", "gate")):
        for i in range(args[k].numel()):
            d = torch.zeros_like(args[k])
            d.view(-1)[i] = e
            diff = (nloss(**{**args, k: args[k] + d}) - nloss(**{**args, k: args[k] - d})) / (2 * e)
            assert abs(diff - gb[name].reshape(-1)[i]) < 1e-7


def test_planted_mistakes_are_caught():
    """Each of these readings differs from the oracle's on ordinary inputs."""
    x, w, init = rnd(1, 6, 3, seed=1), rnd(3, 4, seed=2), rnd(1, 3, 3, seed=3)
    out, final, _ = layer.conv_fwd(x, w, None, init)
    for o, f, _ in (layer.conv_fwd(x, w.flip(1), None, init),            # taps reversed
                    layer.conv_fwd(x, w, None, init.flip(1)),            # state newest first
                    layer.conv_fwd(x, w, None, None)):                   # state dropped
        assert np.abs(o - out).max() > 1e-2
    h, res = rnd(4, 5, seed=4), rnd(4, 5, seed=5)
    o, _ = layer.block_norm_fwd(h, res, torch.ones(5, dtype=T64), alpha=0.5)
    o2, _ = layer.block_norm_fwd(h, res, torch.ones(5, dtype=T64))       # scale dropped
    assert np.abs(o - o2).max() > 1e-2
