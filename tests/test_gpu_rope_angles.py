"""attn_sink_qkv_rope at angles far below a turn, and its check of positions."""
import pytest
import torch

from attention_learnable_head_gb300 import binding
from test_gpu_step import BF, DEV, _clean

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
def test_small_angles_keep_their_bits(interleaved):
    """x = (1, 0) in every pair gives (cos, sin).  inv_freq / 2 pi is a whole number of
    2^-64 turns, off by half of one and by 2^-52 of itself, times the position; the rest
    are roundings: to fp32 and of the sine, below 2^-21 together, and half a bf16 step,
    2^-8."""
    pos = torch.tensor([1, -1, 2, 3, 7, 100, 4096])
    freq = torch.tensor([3e-9, -3e-9, 1e-7, 1e-8, 2.5e-10, 1e-12, 1e-5, 2.0 ** -20] +
                        [10.0 ** (-4 - 0.3 * i) for i in range(24)])
    x = torch.zeros(len(pos), 3, 64)
    a = torch.arange(32) * 2 if interleaved else torch.arange(32)
    b = a + 1 if interleaved else a + 32
    x[:, :, a] = 1.0
    q, k, _ = binding.qkv_rope(x.to(BF).to(DEV), pos.int().to(DEV), freq.to(DEV), heads_q=1,
                               heads_kv=1, interleaved=interleaved)
    angle = pos.double()[:, None] * freq.double()
    for y in (q[:, 0].cpu().double(), k[:, 0].cpu().double()):
        far = pos.double().abs()[:, None] * 2.0 ** -62
        for d, ref in ((a, angle.cos()), (b, angle.sin())):
            err = (y[:, d] - ref).abs()
            assert (err <= (2.0 ** -8 + 2.0 ** -20) * ref.abs() + far).all(), (err / ref.abs()).max()
    _clean()


def test_positions_without_a_dimension_are_refused():
    x = torch.zeros(1, 3, 64, dtype=BF, device=DEV)
    one = torch.zeros((), dtype=torch.int32, device=DEV)
    for run in (lambda: binding.qkv_rope(x, one, torch.ones(32, device=DEV), heads_q=1, heads_kv=1),
                lambda: binding.qkv_rope_backward(x, one, torch.ones(32, device=DEV), x[:, :1],
                                                  x[:, 1:2], x[:, 2:], heads_q=1, heads_kv=1)):
        with pytest.raises(ValueError, match="positions"):
            run()
    _clean()
