"""Calls of the operators around the SSD that are easy to make by mistake, or that leave
something out (GPU): refused, or answered as documented."""
import ctypes

import pytest
import torch

from state_space_model_ssd_amd import binding

pytestmark = pytest.mark.gpu


def conv_args(T=40, C=24, K=4, b=1, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return r(b, T, C).to(dtype), r(C, K)


def test_conv_backward_without_output_gradients_is_refused():
    x, w = conv_args()
    with pytest.raises(ValueError, match="douts"):
        binding.conv_bwd(x, w, None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,splits,cu", [
    (200, (24, 8, 8), [10, 90, 90, 170]),
    (200, (33, 2, 5), [0, 120]),                    # behind the last sequence only
    (9000, (1500, 20, 17), [4000, 4100, 8999]),     # long runs, rows that are not whole vectors
    (70, (1, 0, 0), [70, 70, 70]),                  # no token lies in a sequence
    (70, (40, 0, 0), [3, 3, 69]),
])
def test_conv_rows_outside_every_sequence_are_zeros_where_the_call_makes_them(T, splits, cu, dtype):
    x, w = conv_args(T, sum(splits), dtype=dtype)
    douts = [o.contiguous() for o in x.split(splits, -1)]
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kw = dict(splits=splits, cu_seqlens=cu)
    lo, hi = int(cu[0]), int(cu[-1])
    outs = [torch.full_like(o, 7.0) for o in douts]
    dx = torch.full_like(x, 7.0)
    *want, _ = binding.conv_fwd(x, w, outs=outs, **kw)
    gwant = binding.conv_bwd(x, w, douts, dx=dx, **kw)
    # memory that the next call's tensors are likely to be made from
    stale = [torch.full_like(t, float("nan")) for t in (*douts, x, x, x) for _ in range(2)]
    del stale
    *got, _ = binding.conv_fwd(x, w, **kw)
    stale = [torch.full_like(x, float("nan")) for _ in range(4)]
    del stale
    g = binding.conv_bwd(x, w, douts, **kw)
    torch.cuda.synchronize()
    for a, b in zip((*got, g["x"]), (*want, gwant["x"])):
        assert torch.equal(a[:, lo:hi], b[:, lo:hi])
        assert not a[:, :lo].any() and not a[:, hi:].any()
        assert (b[:, :lo] == 7).all() and (b[:, hi:] == 7).all()
    assert torch.equal(g["weight"], gwant["weight"])


def test_conv_malformed_packing_with_rows_to_clear_stays_in_bounds():
    """Entries are clamped to the tensor before a row is counted, so every row cleared is
    one of the tensor's; guard rows around it keep what they held."""
    wide = torch.full((1, 154, 16), 3.0, device="cuda")
    w = torch.randn((16, 4), device="cuda")
    x = wide[:, 2:152]
    p = binding.ConvProblemC(1, 150, 1, 16, 0, 0, 4, 0, 0, binding.SSD_F32, 1, 1)
    out = torch.full((154, 16), 5.0, device="cuda")
    for bad in ([100, 50], [-5, 10 ** 9], [150, 0], [2 ** 31 - 1, -2 ** 31], [-9, -3]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        code = binding.load_library().ssd_conv_fwd(
            ctypes.byref(p), x.data_ptr(), w.data_ptr(), None, None, cu.data_ptr(),
            out[2:].data_ptr(), None, None, None, torch.cuda.current_stream().cuda_stream)
        assert code == binding.SSD_OK
        torch.cuda.synchronize()
        assert (out[:2] == 5).all() and (out[152:] == 5).all()


def test_shared_memory_is_refused():
    """Calls that would read what they write: in place where nothing says so."""
    x, w = conv_args(b=2)
    st = torch.zeros((2, 3, 24), device="cuda")
    steps = x[:, 0].contiguous()
    h, n = x.clone(), torch.ones(24, device="cuda")
    heads = steps.view(2, 3, 8)
    states = torch.zeros((2, 3, 8, 8), device="cuda")
    v = torch.ones(3, device="cuda")
    for call in (lambda: binding.conv_fwd(x, w, initial_states=st, final_states=st),
                 lambda: binding.conv_fwd(x, w, outs=[x, None, None]),
                 lambda: binding.conv_bwd(x, w, [h, None, None], dx=h),
                 lambda: binding.conv_bwd(x, w, [h, None, None], dx=x),
                 lambda: binding.conv_step(steps, st, w, outs=[steps, None, None]),
                 lambda: binding.ssd_step(heads, steps[:, :3], v, heads[:, :1], heads[:, 1:2], states,
                                          out=heads),
                 lambda: binding.block_norm_fwd(x, h, n, out=h),
                 lambda: binding.block_norm_fwd(x, h, n, residual_out=x),
                 lambda: binding.block_norm_fwd(x, x, n, out=x, residual_out=x)):
        with pytest.raises(binding.SsdError) as e:
            call()
        assert e.value.code == binding.SSD_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert not st.any() and not states.any()


def test_columns_of_one_tensor_are_taken():
    """x and its gradient as columns of one wider tensor; a stream that is also the
    block's output, normed in place."""
    x, w = conv_args(T=130, b=2)
    dout = torch.randn_like(x)
    want = binding.conv_bwd(x, w, [dout, None, None])
    wide = torch.full((2, 130, 60), 3.0, device="cuda")
    wide[..., 2:26] = x
    g = binding.conv_bwd(wide[..., 2:26], w, [dout, None, None], dx=wide[..., 30:54])
    n = torch.rand(24, device="cuda")
    o1, h1 = binding.block_norm_fwd(x, x, n)
    y = x.clone()
    o2, h2 = binding.block_norm_fwd(y, y, n, out=y)
    torch.cuda.synchronize()
    assert torch.equal(wide[..., 30:54], want["x"]) and torch.equal(g["weight"], want["weight"])
    assert torch.equal(wide[..., 2:26], x)
    assert all((wide[..., s] == 3).all() for s in (slice(0, 2), slice(26, 30), slice(54, 60)))
    assert torch.equal(o1, y) and torch.equal(h1, h2)


@pytest.mark.parametrize("N", [3, 16, 130])
@pytest.mark.parametrize("where", ["dt", "dt_bias", "A"])
def test_step_keeps_a_nan_it_is_given(where, N):
    """A step size (or decay) of NaN makes its head's state and output NaN, as the formula
    does, and no other's; it is not clamped to a number."""
    g = torch.Generator(device="cuda").manual_seed(N)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    b, H, P = 3, 4, 5
    x, dt, B, C, A, bias, st = r(b, H, P), r(b, H), r(b, 2, N), r(b, 2, N), -r(H).abs(), r(H), r(b, H, P, N)
    clean = st.clone()
    want = binding.ssd_step(x, dt, A, B, C, clean, dt_bias=bias, dt_min=0.01, dt_max=1.0)
    bad = torch.zeros((b, H), dtype=torch.bool, device="cuda")
    if where == "dt":
        dt[1, 2] = float("nan")
        bad[1, 2] = True
    else:
        (bias if where == "dt_bias" else A)[2] = float("nan")
        bad[:, 2] = True
    out = binding.ssd_step(x, dt, A, B, C, st, dt_bias=bias, dt_min=0.01, dt_max=1.0)
    torch.cuda.synchronize()
    assert torch.isnan(out[bad]).all() and torch.isnan(st[bad]).all()
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(st[~bad], clean[~bad])
