"""kda_attn_rope: numbers come out as numbers, and channels behind the pairs bit for bit."""

import pytest
import torch

from _util import kda
from test_rope_gpu import D, near, rope64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pairs", [1, 11, 32, 63])
def test_channels_behind_the_pairs_keep_their_bits(pairs, interleaved, dtype):
    """Any bits: NaN of every kind, infinities, -0."""
    K = kda()
    gen = torch.Generator().manual_seed(pairs)
    bits = torch.randint(-1 << 15, 1 << 15, (512, 3, D), generator=gen, dtype=torch.int16).cuda()
    bits[:, :, -1] |= 0x7c01 if dtype == torch.float16 else 0x7f81         # not numbers
    x = bits.view(dtype)
    assert bool(torch.isnan(x[..., -1]).all())
    pos = torch.arange(512, dtype=torch.int32).cuda()
    y = torch.zeros_like(x)
    K.kda_attn_rope(x, None, pos, torch.rand(pairs, generator=gen).cuda(), y,
                    interleaved=interleaved)
    assert torch.equal(y.view(torch.int16)[..., 2 * pairs:], bits[..., 2 * pairs:])
    K.kda_attn_rope(x, None, pos, torch.rand(pairs).cuda(), interleaved=interleaved)
    assert torch.equal(x.view(torch.int16)[..., 2 * pairs:], y.view(torch.int16)[..., 2 * pairs:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved,pairs", [(False, 64), (True, 64), (False, 61), (True, 7)])
def test_far_positions_give_numbers(interleaved, pairs, dtype):
    K = kda()
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 16777217, -123456789],
                       dtype=torch.int32).cuda()
    x = torch.randn((7, 2, D), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    inv = torch.tensor([1.0, 4.0, -0.7, 1e-4, 0.0, -4.0, -1e-20] + [0.3] * 57).cuda()[:pairs]
    y = torch.empty_like(x)
    K.kda_attn_rope(x, None, pos, inv, y, interleaved=interleaved)
    assert bool(torch.isfinite(y).all())
    near(y, x, rope64(x, pos[:, None], inv, [0] * pairs, interleaved, 1.0), pairs, interleaved, 1.0)


@pytest.mark.parametrize("interleaved,pairs", [(False, 64), (True, 64), (False, 21)])
def test_more_than_2_to_the_31_values_are_numbers(interleaved, pairs):
    K, rows, heads = kda(), 66000, 256
    x = torch.randn((rows, heads, D), generator=torch.Generator(device="cuda").manual_seed(3),
                    device="cuda", dtype=torch.bfloat16)
    assert x.numel() > 1 << 31
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    inv = 10000.0 ** (-torch.arange(pairs, device="cuda") / pairs)
    kept = {r: x[r:r + 3].clone() for r in (0, 33001, rows - 3)}
    K.kda_attn_rope(x, None, pos, inv, interleaved=interleaved)
    K.kda_sync_status()
    assert all(bool(torch.isfinite(part).all()) for part in x.split(8000))
    for r, was in kept.items():
        ref = rope64(was, pos[r:r + 3, None], inv, [0] * pairs, interleaved, 1.0)
        near(x[r:r + 3], was, ref, pairs, interleaved, 1.0)
