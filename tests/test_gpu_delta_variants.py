"""The gated delta rule at sizes that take each variant of its launches (GPU): a wave that walks
over a group's heads, two and four waves of states, states kept rounded or as pairs, long sequences
cut with either.  Against the recurrence in 64 bits, one token at a time."""
import pytest
import torch

from state_space_model_ssd_amd import binding
from tests.delta_cases import dev, draw, draw_grads
from tests.delta_device import check

pytestmark = pytest.mark.gpu
CUS = 256                       # what the library's rules compare with below


@pytest.fixture(autouse=True)
def device():
    if torch.cuda.get_device_properties(0).multi_processor_count != CUS:
        pytest.skip("other variants on a device of another size")


def run(b, T, H, G, P, N, dtype, gate, cu=None, keep=False, seed=21, decay=0.02, bwd=True):
    x = draw(b, T, H, G, P, N, dtype, gate, nseq=None if cu is None else len(cu) - 1, seed=seed, decay=decay)
    if keep:
        x["g"].zero_()
    dout, dfin = (t.cuda() for t in draw_grads(x))
    x, c = dev(x), None if cu is None else torch.tensor(cu, dtype=torch.int32)
    kw = {} if cu is None else dict(cu_seqlens=c.cuda())
    fwd = binding.delta_fwd(**x, **kw)
    grads = binding.delta_bwd(**x, **kw, dout=dout, dfinal_states=dfin) if bwd else None
    check(x, N ** -0.5, c, dout, dfin, fwd, grads)


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("N", [32, 64, 128])
def test_heads_of_a_group_in_turn(N, dtype, gate):
    """Chunks times groups beyond four waves a CU; three heads to a group."""
    b, T, H, G = 3, 703, 96, 32
    assert b * ((T + 63) // 64) * G > 4 * CUS
    run(b, T, H, G, 16, N, dtype, gate)


@pytest.mark.parametrize("dtype,gate", TYPES)
def test_heads_of_a_group_in_turn_packed(dtype, gate):
    cu = [0, 1, 65, 65, 700, 1400, 2100]
    assert 35 * 32 > 4 * CUS
    run(1, 2105, 64, 32, 32, 64, dtype, gate, cu)


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("P,N", [(64, 64), (64, 128), (80, 64), (128, 128), (48, 32)])
def test_four_waves_of_states(P, N, dtype, gate):
    """Sequences times heads times blocks of 64 rows beyond half of the CUs, with bf16 gates many
    enough that states are kept rounded."""
    b, T, H = 3, 470, 48
    assert 2 * b * H * ((P + 63) // 64) > CUS and b * T * H > 65536
    run(b, T, H, 16, P, N, dtype, gate)


@pytest.mark.parametrize("N", [32, 64, 128])
def test_two_waves_of_states_rounded(N):
    b, T, H, P = 1, 2112, 32, 64
    assert 2 * b * H * ((P + 63) // 64) <= CUS and b * T * H > 65536
    run(b, T, H, 16, P, N, "bf16", "bf16")


@pytest.mark.parametrize("P,N,gate", [(16, 32, "bf16"), (32, 64, "bf16"), (16, 128, "bf16"), (48, 64, "bf16"),
                                      (48, 64, "f32")])
def test_cut_with_states_rounded(P, N, gate):
    """16 heads of 128 chunks: segments of 16, whose chains fill the device several times; P 48 takes
    four waves of states for them."""
    assert 8192 * 16 > 65536
    run(1, 8192, 16, 8, P, N, "bf16", gate, decay=0.003)


@pytest.mark.parametrize("cu", [[0, 8192], [3, 5000, 5000, 5001, 8150]])
def test_packed_cut_with_states_rounded(cu):
    run(1, 8192, 16, 8, 32, 64, "bf16", "bf16", cu, decay=0.003)


@pytest.mark.parametrize("dtype,gate,H", [("bf16", "bf16", 16), ("bf16", "f32", 2), ("f32", "f32", 2)])
def test_cut_without_decay(dtype, gate, H):
    """g = 0, backward too: nothing a segment hands on is forgotten but where a key comes again."""
    run(1, 4224, H, H, 16, 64, dtype, gate, keep=True)
