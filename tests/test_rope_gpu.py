"""kda_attn_rope against rotations in 64 bits."""

import pytest
import torch

from _util import kda

pytestmark = pytest.mark.gpu
D = 128


def rope64(x, pos, inv_freq, axis, interleaved, factor):
    y, pairs = x.double().clone(), inv_freq.numel()
    p = torch.arange(pairs, device=x.device)
    a = pos.double()[:, axis] * inv_freq.double()
    c, s = (a.cos() * factor)[:, None], (a.sin() * factor)[:, None]
    i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)
    u, w = x.double()[..., i], x.double()[..., j]
    y[..., i], y[..., j] = u * c - w * s, w * c + u * s
    return y


def near(y, x, ref, pairs, interleaved, factor):
    """Half a step of the result; cosine, sine (2^-22 of a turn and their own roundings) and
    two FP32 operations: under 2^-18 of the pair's size."""
    p = torch.arange(pairs, device=x.device)
    i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)
    size = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    size[..., i] = size[..., j] = x.double()[..., i].abs() + x.double()[..., j].abs()
    half = torch.finfo(x.dtype).eps / 2
    bound = half * ref.abs() + 2.0 ** -18 * abs(factor) * size + torch.finfo(x.dtype).tiny
    over = ((y.double() - ref).abs() - bound)
    over = over.nan_to_num(0.0)
    assert float(over.max()) <= 0, (float(over.max()), int((over > 0).sum()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,kv,pairs,axes", [
    (1, 1, 1, 64, 1), (5, 8, 2, 32, 3), (64, 32, 8, 64, 1), (300, 5, 1, 11, 2), (2000, 3, 3, 48, 4),
    (1217, 4, 0, 1, 1), (9, 7, 1, 63, 1)])
def test_rope(rows, heads, kv, pairs, axes, interleaved, dtype):
    K = kda()
    g = torch.Generator().manual_seed(rows)
    x = torch.randn((rows, heads + kv + 1, D), generator=g).to(dtype).cuda()
    q, k = x[:, :heads], x[:, heads:heads + kv] if kv else None
    pos = torch.randint(0, 1 << 21, (rows, axes), generator=g, dtype=torch.int32).cuda()
    inv = torch.pow(10000.0, -torch.arange(pairs).double() / pairs).float().cuda()
    axis = [(3 * p) % axes for p in range(pairs)]
    want = [None if y is None else rope64(y, pos, inv, axis, interleaved, 1.25) for y in (q, k)]
    qo = torch.empty((rows, heads, D), dtype=dtype, device="cuda")
    ko = torch.empty((rows, kv, D), dtype=dtype, device="cuda") if kv else None
    K.kda_attn_rope(q, k, pos, inv, qo, ko, pair_axis=axis, interleaved=interleaved, factor=1.25)
    near(qo, q, want[0], pairs, interleaved, 1.25)
    assert torch.equal(qo[..., 2 * pairs:], q[..., 2 * pairs:])
    if kv:
        near(ko, k, want[1], pairs, interleaved, 1.25)
    # in place, in a wider row: the same bits, and the rest of the row as it was
    last = x[:, -1].clone()
    K.kda_attn_rope(q, k, pos, inv, pair_axis=axis, interleaved=interleaved, factor=1.25)
    assert torch.equal(q, qo) and (not kv or torch.equal(k, ko)) and torch.equal(x[:, -1], last)


def test_far_and_negative_positions():
    K = kda()
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 16777217, -123456789],
                       dtype=torch.int32).cuda()
    x = torch.randn((7, 2, D), generator=torch.Generator().manual_seed(1)).half().cuda()
    inv = torch.tensor([1.0, 4.0, -0.7, 1e-4, 0.0] + [0.3] * 59).cuda()
    y = torch.empty_like(x)
    K.kda_attn_rope(x, None, pos, inv, y)
    near(y, x, rope64(x, pos[:, None], inv, [0] * 64, False, 1.0), 64, False, 1.0)
    assert torch.equal(y[0], x[0])


def test_values_that_are_not_finite_stay_in_their_pair():
    K = kda()
    x = torch.randn((3, 2, D)).to(torch.bfloat16).cuda()
    x[1, 1, 100] = float("nan")
    x[1, 1, 3] = float("inf")
    inv, pos = torch.rand(32).cuda(), torch.arange(3, dtype=torch.int32).cuda()
    for interleaved, pairs in ((False, 32), (True, 32), (False, 11)):
        y = torch.empty_like(x)
        K.kda_attn_rope(x, None, pos, inv[:pairs], y, interleaved=interleaved)
        off = (~torch.isfinite(y)).nonzero().tolist()
        pair = {3, 2} if interleaved else {3, 3 + pairs}
        assert {tuple(o[:2]) for o in off} == {(1, 1)} and {o[2] for o in off} == pair | {100}


def test_four_dimensions_and_no_rows():
    K = kda()
    x = torch.randn((2, 3, 4, D)).to(torch.bfloat16).cuda()
    inv = torch.rand(64).cuda()
    pos = torch.arange(6, dtype=torch.int32).cuda()
    y, z = torch.empty_like(x), torch.empty_like(x.flatten(0, 1))
    K.kda_attn_rope(x, None, pos.view(2, 3), inv, y)
    K.kda_attn_rope(x.flatten(0, 1), None, pos, inv, z)
    assert torch.equal(y.flatten(0, 1), z)
    K.kda_attn_rope(x[:0].flatten(0, 1), None, pos[:0], inv)
    with pytest.raises(ValueError):
        K.kda_attn_rope(x.flatten(0, 1), None, pos.view(3, 2), inv)
    with pytest.raises(ValueError):
        K.kda_attn_rope(z[:3], None, pos.view(3, 2), inv)              # two axes, no pair_axis
    with pytest.raises(ValueError):
        K.kda_attn_rope(z[:3], None, pos.view(3, 2), inv, pair_axis=[2] * 64)
    with pytest.raises(TypeError):
        K.kda_attn_rope(z, None, pos.long(), inv)
