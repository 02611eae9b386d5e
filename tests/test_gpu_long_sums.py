"""Weight gradients summed over very many tokens (GPU).  A channel's terms are all the
same number, different from channel to channel, so that the roundings of a long chain
of additions all go the same way, and the exact sums are known.

Every addition is off by at most U = 2^-24 of its result, and no partial sum exceeds the
total, so a sum is off by at most U of the total for each addition that a term passes.
"""
import pytest
import torch

from state_space_model_ssd_amd import binding
from tests.layer_bounds import U

pytestmark = pytest.mark.gpu


def constants(C):
    """C numbers of three decimal digits, as fp32 holds them."""
    return torch.tensor([0.1 + 0.013 * (i % 90) for i in range(C)], dtype=torch.float32)


def held(got, want, n, what):
    err = ((got.double().cpu() - want).abs() / want.abs()).max().item()
    print(f"  {what}: {err / U:.1f} U of {n} U", flush=True)
    assert err <= n * U, (what, err / U)


@pytest.mark.parametrize("T,C,K,dtype,nseq,segment,segments", [
    (2 ** 23, 12, 2, "f32", None, 18 * 15, 31),    # short runs of 15 tokens: 547 a wave, 18 a segment
    (2 ** 21, 40, 4, "bf16", None, 5 * 61, 7),     # long runs of 61 tokens: 34 a wave, 5 a segment
    (2 ** 20, 6, 3, "f32", 5000, 19 * 14, 5),      # packed: sequences of 209 and 210 tokens
])
def test_conv_weight_gradients_over_many_tokens(T, C, K, dtype, nseq, segment, segments):
    """Without activation, with x = 1 (and states of 1) every tap's gradient and the bias'
    are the sum of dout: T equal terms, each product with 1 exact.  A term passes one
    addition per token of its segment, one per segment, 4 for the waves, then 8 + 3 + 4
    in the column sums."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    c = constants(C).to(dt)
    x = torch.ones((1, T, C), dtype=dt, device="cuda")
    dout = c.cuda().expand(1, T, C).contiguous()
    w, bias = torch.zeros((C, K), device="cuda"), torch.zeros(C, device="cuda")
    cu = None
    if nseq is not None:
        cu = torch.linspace(0, T, nseq + 1, dtype=torch.float64).round().to(torch.int32).cuda()
    init = torch.ones((nseq or 1, K - 1, C), dtype=dt, device="cuda")
    g = binding.conv_bwd(x, w, [dout, None, None], bias, initial_states=init, cu_seqlens=cu,
                         activation=None)
    torch.cuda.synchronize()
    want, n = c.double() * T, segment + segments + 4 + 15
    held(g["bias"], want, n, "dbias")
    held(g["weight"], want[:, None].expand(C, K), n, "dweight")


@pytest.mark.parametrize("T,C,dtype,residual,segment,segments", [
    (2 ** 23, 4, "f32", "f32", 64, 33),            # one wave a row: 2048 rows and more each
    (2 ** 20 + 3, 260, "bf16", "f32", 64, 9),      # two waves a row, 513 rows each
    (2 ** 20 + 3, 261, "bf16", "bf16", 64, 9),     # the same, rows not whole vectors
    (2 ** 17, 5000, "bf16", "bf16", 64, 9),        # eight waves a row, four vectors a lane
])
def test_block_norm_weight_gradients_over_many_rows(T, C, dtype, residual, segment, segments):
    """x = 1, no residual, weights and scale of 1: both norms' factors are 1 within 4 U (the
    mean's product, half of it through the root, the root's 2), the same in every row.
    dout is c and -c at neighbouring channels, so every sum over a row is 0 exactly: dn =
    dout and dh = dout + dresidual_out = 2 dout.  Then dpre_weight = T dout, dscale = 2 T
    dout and dpost_weight = 2 T dout, every term off by at most 4 + 4 U for the factors and
    8 U for its own operations, the same way in every row.

    A term passes one addition per row of its segment, one per segment, 4 for rows that
    share a workgroup, and 16 + 3 + 16 in the column sums of up to 2048 partial rows.  A
    device with fewer than 256 compute units walks further: twice the segments."""
    dt, rdt = (torch.float32 if d == "f32" else torch.bfloat16 for d in (dtype, residual))
    c = torch.zeros(C)
    c[0::2][:C // 2] = constants(C // 2)
    c[1::2][:C // 2] = -constants(C // 2)
    c = c.to(dt)
    x = torch.ones((T, C), dtype=dt, device="cuda")
    dout = c.cuda().expand(T, C).contiguous()
    w = torch.ones(C, device="cuda")
    dres = dout if rdt == dt else dout.to(rdt)
    g = binding.block_norm_bwd(x, None, w, dout, dres, post_weight=w, scale=w, eps=0.0,
                               residual_dtype=rdt)
    torch.cuda.synchronize()
    keep = c != 0
    n = segment + 2 * segments + 4 + 16 + 3 + 16 + 16
    for k, f in (("pre_weight", 1), ("scale", 2), ("post_weight", 2)):
        held(g[k].cpu()[keep], f * c[keep].double() * T, n, "d" + k)
