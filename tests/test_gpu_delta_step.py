"""The gated delta rule for one token per sequence on the GPU, against the 64-bit update.

Bounds, with U = 2^-24: a S within 5 U (exp 4 U), its products with k and q and their sums
(at most 4 in a lane and 6 exchanges) 20 U of the sum of absolute values; w beta times that
and 2 U of its two terms; the state |k| err(w) + 8 U of its terms; the output likewise, and
its rounding."""
import numpy as np
import pytest
import torch

from oracle import delta
from state_space_model_ssd_amd import binding
from tests.delta_cases import DT, dev, draw, unit
from tests.helpers import f64, rel_l2
from tests.layer_bounds import RND, TINY, U, check

pytestmark = pytest.mark.gpu


def inputs(b=3, H=4, G=2, P=16, N=32, dtype="bf16", gate="f32", slots=None, seed=0):
    r = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    t, gt = DT[dtype], DT[gate]
    return dict(q=unit(rn(b, G, N)).to(t), k=unit(rn(b, G, N)).to(t), v=rn(b, H, P).to(t),
                g=(-rn(b, H).abs()).to(gt), beta=torch.rand((b, H), generator=r).to(gt),
                states=rn(slots or b, H, P, N))


def compare(x, got, after, scale, slots=None):
    ro, rs = delta.delta_step(**{n: f64(v) for n, v in x.items()}, scale=scale, slots=slots)
    q, k, v, g, beta, S = (f64(x[n]) for n in ("q", "k", "v", "g", "beta", "states"))
    rep = v.shape[1] // q.shape[1]
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    ts = np.zeros_like(rs)
    to = np.zeros_like(ro)
    for b in np.flatnonzero(~np.isnan(ro[:, 0, 0])):
        s = b if slots is None else int(slots[b])
        A = np.abs(S[s]) * np.exp(g[b])[:, None, None]
        ka, qa = np.abs(k[b])[:, None, :], np.abs(q[b])[:, None, :]
        sk = (A * ka).sum(-1)
        w = beta[b][:, None] * (np.abs(v[b]) + sk)
        ew = beta[b][:, None] * 20 * U * sk + 4 * U * w
        ts[s] = ka * ew[..., None] + 8 * U * (A + w[..., None] * ka) + TINY
        kq = (ka * qa).sum(-1)
        to[b] = abs(scale) * (20 * U * (A * qa).sum(-1) + ew * kq + 24 * U * w * kq) + RND[
            "bf16" if x["q"].dtype == torch.bfloat16 else "f32"] * np.abs(ro[b]) + TINY
    check(got, ro, to, "out")
    check(after, rs, ts, "states")


SHAPES = [(1, 1, 1, 1, 1), (2, 4, 2, 16, 32), (3, 6, 3, 17, 5), (2, 8, 1, 64, 128), (5, 2, 2, 33, 100),
          (1, 3, 3, 128, 256), (4, 5, 5, 7, 2), (130, 16, 4, 64, 64), (2, 4, 4, 257, 30)]


@pytest.mark.parametrize("dtype,gate", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_step(shape, dtype, gate):
    x = inputs(*shape, dtype, gate)
    d = dev(x)
    got = binding.delta_step(**d, scale=0.3)
    compare(x, got, d["states"], 0.3)


def test_scale_is_by_default_that_of_the_prompt():
    d = dev(inputs())
    s = d["states"].clone()
    a = binding.delta_step(**d)
    b = binding.delta_step(**dict(d, states=s), scale=32 ** -0.5)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slots_padding_and_repeats(dtype):
    """Slots in any order; rows outside the cache and rows whose slot an earlier row has are
    padding: their outputs and every other slot stay."""
    x = inputs(b=7, dtype=dtype, slots=6)
    slots = torch.tensor([4, -1, 0, 4, 6, 2, 2 ** 31 - 1], dtype=torch.int32)
    d = dev(x)
    out = torch.full_like(d["v"], 9.0)
    binding.delta_step(**d, scale=0.3, slots=slots.cuda(), out=out)
    compare(x, out, d["states"], 0.3, slots.numpy())
    assert bool((out[[1, 3, 4, 6]] == 9).all())
    for s in (1, 3, 5):
        assert torch.equal(d["states"][s].cpu(), x["states"][s])
    d = dev(x)
    assert not binding.delta_step(**d, scale=0.3, slots=slots.cuda())[[1, 3, 4, 6]].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_columns_of_one_row(dtype):
    """q, k and v (and the gates) as columns of the projection's rows, of odd widths."""
    x = inputs(b=4, H=4, G=2, P=17, N=31, dtype=dtype)
    q, k, v = (x[n].flatten(1) for n in "qkv")
    row = torch.cat((q, k, v, torch.zeros(4, 3, dtype=q.dtype)), 1).cuda()
    nq, nv = q.shape[1], v.shape[1]
    gates = torch.cat((x["g"], x["beta"]), 1).cuda()
    d = dev(x)
    keep = row.clone()
    got = binding.delta_step(row[:, :nq].unflatten(1, (2, 31)), row[:, nq:2 * nq].unflatten(1, (2, 31)),
                             row[:, 2 * nq:2 * nq + nv].unflatten(1, (4, 17)), gates[:, :4], gates[:, 4:],
                             d["states"], scale=0.3)
    compare(x, got, d["states"], 0.3)
    assert torch.equal(row, keep)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_at_their_ends(dtype):
    x = inputs(b=4, dtype=dtype)
    x["g"][0], x["g"][1], x["beta"][2], x["beta"][3] = -float("inf"), 0, 0, 1
    d = dev(x)
    got = binding.delta_step(**d, scale=0.3)
    compare(x, got, d["states"], 0.3)


def test_nan_stays_in_its_head():
    x = dev(inputs(b=3, H=4, G=4, P=32, N=64))
    clean = {n: v.clone() for n, v in x.items()}
    want = binding.delta_step(**clean)
    x["k"][1, 2, 5] = float("nan")
    got = binding.delta_step(**x)
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[1, 2] = False
    assert got[1, 2].isnan().all() and torch.equal(got[keep], want[keep])
    ks = torch.ones_like(x["states"], dtype=torch.bool)
    ks[1, 2] = False
    assert torch.equal(x["states"][ks], clean["states"][ks])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_go_on_from_a_prompt(dtype):
    """A prompt, then 70 single tokens on its states: the prompt of all of them."""
    x = draw(2, 170, 4, 2, 32, 64, dtype)
    whole = binding.delta_fwd(**dev(x))
    first = dev({n: (v if n == "initial_states" else v[:, :100].contiguous()) for n, v in x.items()})
    _, states, _ = binding.delta_fwd(**first)
    d, outs = dev(x), []
    for t in range(100, 170):
        outs.append(binding.delta_step(*(d[n][:, t] for n in ("q", "k", "v", "g", "beta")), states))
    outs = torch.stack(outs, 1)
    # both are within their bound of the recurrence: twice the prompt's
    assert rel_l2(outs, whole[0][:, 100:]) <= (2e-5 if dtype == "f32" else 2e-2)
    assert rel_l2(states, whole[1]) <= (2e-5 if dtype == "f32" else 2 ** -13)


def test_far_slots():
    """A slot behind 2^31 values of the cache."""
    H, P, N = 4, 64, 128
    n = 2 ** 31 // (H * P * N) + 3
    if torch.cuda.mem_get_info()[0] < 3 * n * H * P * N * 4 // 2:
        pytest.skip("too little memory")
    x = inputs(b=2, H=H, P=P, N=N)
    cache = torch.zeros((n, H, P, N), device="cuda")
    cache[n - 1] = x["states"][0].cuda()
    cache[0] = x["states"][1].cuda()
    small = dev(x)
    want = binding.delta_step(**small)
    d = dev(x)
    got = binding.delta_step(**dict(d, states=cache), slots=torch.tensor([n - 1, 0], dtype=torch.int32).cuda())
    assert torch.equal(got, want) and torch.equal(cache[n - 1], small["states"][0])
    assert torch.equal(cache[0], small["states"][1]) and not cache[1].any() and not cache[n - 2].any()


def test_in_a_graph():
    """Captured once, replayed on a batch whose slots change, eager calls between."""
    x = dev(inputs(b=4, H=4, P=32, N=64, slots=9))
    slots = torch.tensor([0, 1, 2, 3], dtype=torch.int32).cuda()
    start, out = x["states"].clone(), torch.zeros_like(x["v"])
    binding.delta_step(**x, slots=slots, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.delta_step(**x, slots=slots, out=out)
    x["states"].copy_(start)
    states = start.clone()
    for i, s in enumerate(([0, 1, 2, 3], [8, 3, -1, 0], [5, 5, 1, 0], [3, 2, 1, 0])):
        slots.copy_(torch.tensor(s))
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.full_like(out, 7)
        binding.delta_step(**dict(x, states=states), slots=slots, out=want)
        assert torch.equal(out, want) and torch.equal(x["states"], states), i


def test_no_rows_and_refusals():
    d = dev(inputs(b=0, slots=2))
    assert binding.delta_step(**d).shape == (0, 4, 16)
    x = dev(inputs())
    for kw in (dict(k=x["k"].float()), dict(v=x["v"][:2]), dict(g=x["g"].double()), dict(beta=x["beta"][:, :2]),
               dict(states=x["states"].bfloat16()), dict(states=x["states"][:2]),
               dict(states=x["states"].transpose(2, 3)), dict(q=x["q"].cpu()),
               dict(q=x["q"].transpose(1, 2).contiguous().transpose(1, 2)),
               dict(slots=torch.zeros(3, dtype=torch.int64, device="cuda")),
               dict(slots=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(out=x["v"]),
               dict(out=x["v"].float()), dict(scale=float("inf"))):
        with pytest.raises((ValueError, binding.SsdError)):
            binding.delta_step(**dict(x, **kw))
