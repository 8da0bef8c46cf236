"""The 4-bit cache's rows at the ends of BF16's range."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from _attn import D, Host, bf16_below
from _util import kda
from test_attn_kv4_gpu import dev

pytestmark = pytest.mark.gpu


def exact(row):
    """One row of 128 numbers by the documented formula in rational numbers (64 bits lose the
    least of them beside the largest): codes, s, m."""
    codes, s, m = [], [], []
    for x in np.asarray(row).reshape(2, 64):
        least = float(bf16_below(x.min()))
        room = (Fraction(float(x.max())) - Fraction(least)) / 15
        step = -float(bf16_below(-float(room)))
        if Fraction(step) < room:   # a quotient just above a BF16 number: the next one
            step = -float(bf16_below(np.nextafter(-step, -np.inf)))
        assert Fraction(step) >= room
        for y in x:
            codes.append(round((Fraction(float(y)) - Fraction(least)) / Fraction(step)))
        s.append(step)
        m.append(least)
    return codes, s, m


def test_append_of_the_largest_numbers():
    """Groups whose values lie further apart than FP32's largest number: steps and codes are those
    of the documented formula all the same."""
    K = kda()
    rng = np.random.default_rng(50)
    top = float(torch.finfo(torch.bfloat16).max)
    rows = []
    for low, high in ((-top, top), (-top, 0.5 * top), (-0.4 * top, 0.7 * top), (-top, -0.2 * top),
                      (-1e37, top), (-0.03 * top, 0.02 * top), (0.0, top), (-top, 0.0)):
        x = np.linspace(low, high, 64)
        mixed = rng.uniform(0, 1, 64) * (high - low) + low if high - low < top else np.where(
            rng.integers(0, 2, 64) > 0, high, low) * rng.uniform(0, 1, 64)
        mixed[:4] = (low, high, 0.5 * (low + high), 2.0 ** -130 if low <= 0 else low)
        rows.append(np.concatenate([x, mixed]))
    x = torch.tensor(np.stack(rows)).clamp(-top, top)[:, None].to(torch.bfloat16)
    assert bool(torch.isfinite(x).all())
    n, page = x.shape[0], 16
    table = np.zeros((1, 1), dtype=np.int32)
    cache = np.zeros((1, 1, page * 144), dtype=np.uint8)
    got = dev(cache)
    K.kda_attn_kv4_append(x.cuda(), x.flip(0).cuda(), got, dev(table),
                          torch.tensor([n], dtype=torch.int32).cuda())
    host = Host(cache)
    for i, row in enumerate(x.double().numpy()[:, 0]):
        for which, tok in (("k", i), ("v", n - 1 - i)):
            host.write(which, 0, tok, 0, *exact(row))
    assert np.array_equal(got.cpu().numpy(), cache)
    a, b = torch.empty_like(x).cuda(), torch.empty_like(x).cuda()
    K.kda_attn_kv4_read(a, b, got, dev(table), torch.tensor([n], dtype=torch.int32).cuda())
    assert not bool(torch.isnan(a).any()) and not bool(torch.isnan(b).any())
