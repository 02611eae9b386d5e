"""Packed batches of the gated delta rule on the GPU: more sequences than the plan adds up at a
time, and lengths that make no sense, backward too."""
import numpy as np
import pytest
import torch

from state_space_model_ssd_amd import binding
from tests.delta_cases import check_bwd, check_fwd, dev, draw, draw_grads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [256, 257, 600])
def test_several_hundred_sequences(n):
    """256 at a time; the rest takes up where these left off."""
    lens = [(13 * i) % 9 + (130 if i % 255 == 0 else 0) for i in range(n)]
    cu = torch.tensor(list(np.cumsum([2] + lens)), dtype=torch.int32)
    x = draw(1, int(cu[-1]) + 3, 2, 1, 16, 32, nseq=n, seed=15)
    check_fwd(binding.delta_fwd(**dev(x), cu_seqlens=cu.cuda()), x, 32 ** -0.5, cu)
    dout, dfin = draw_grads(x)
    got = binding.delta_bwd(**dev(x), cu_seqlens=cu.cuda(), dout=dout.cuda(), dfinal_states=dfin.cuda())
    check_bwd(got, x, dout, dfin, 32 ** -0.5, cu)


GUARD = 64          # rows before and behind


class Guarded:
    """A tensor between rows that nothing may write."""

    def __init__(self, like):
        self.n = like.shape[0]
        self.all = torch.full((self.n + 2 * GUARD,) + like.shape[1:], 5.0, dtype=like.dtype, device="cuda")
        self.own = self.all[GUARD:GUARD + self.n]

    def kept(self):
        return bool((self.all[:GUARD] == 5).all()) and bool((self.all[GUARD + self.n:] == 5).all())


SHORT = (64, [[0, -5, 64], [0, 100, 50], [0, 50, 10 ** 6], [-3, 20, 64], [2 ** 31 - 1, 0, 1]])
LONG = (6000, [[0, 6000, 100], [0, -5, 10 ** 9], [4000, 0, 6000], [0, 6000, -1]])
FORTH = [0, 300] * 150 + [0]                     # 300 sequences of all tokens or none
CASES = [(T, cu) for T, cus in (SHORT, LONG) for cu in cus] + [(300, FORTH), (300, [-7] + FORTH[1:] + [2 ** 31 - 1])]


@pytest.mark.parametrize("clear", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_bad_lengths_stay_in_bounds(case, dtype, clear):
    """Forward and backward, whatever they write lying between guard rows."""
    T, lens = CASES[case]
    n = len(lens) - 1
    print(f"  {T} tokens, {n} sequences, {lens[:6]}", flush=True)
    x = draw(1, T, 2, 1, 16, 32, dtype, nseq=n)
    d, cu = dev(x), torch.tensor(lens, dtype=torch.int32).cuda()
    dout, dfin = (t.cuda() for t in draw_grads(x))
    flat = {k: (v if k == "initial_states" else v[0]) for k, v in d.items()}
    prob = binding.DeltaProblemC(1, T, 2, 16, 32, 1, n, binding._DT[d["q"].dtype], binding.SSD_F32, 0.3, clear)
    lib, stream = binding.load_library(), torch.cuda.current_stream().cuda_stream
    ins = [d[k].data_ptr() for k in ("q", "k", "v", "g", "beta", "initial_states")] + [cu.data_ptr()]
    grads = [Guarded(flat[k]) for k in ("q", "k", "v", "g", "beta", "initial_states")]
    out, fin = Guarded(flat["v"]), Guarded(flat["initial_states"])
    for fn, size, mine in ((lib.ssd_delta_fwd, lib.ssd_delta_fwd_workspace_size, [out, fin]),
                           (lib.ssd_delta_bwd, lib.ssd_delta_bwd_workspace_size, grads)):
        need = size(prob)
        ws = Guarded(torch.empty((need + 255) // 256, 256, dtype=torch.uint8))
        more = [] if mine is not grads else [dout.data_ptr(), dfin.data_ptr()]
        assert fn(prob, *ins, *more, *[m.own.data_ptr() for m in mine], ws.own.data_ptr(), need, stream) == 0
        torch.cuda.synchronize()
        assert all(m.kept() for m in [*mine, ws])
