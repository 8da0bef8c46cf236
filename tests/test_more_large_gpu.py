"""Linear attention, rotary rows and page copies over arrays whose offsets pass 32 bits, in
elements and in bytes: the last rows, states and pages, against their 64-bit forms."""

import pytest
import torch

from _lin import D, close
from _util import kda
from test_rope_gpu import near, rope64

pytestmark = pytest.mark.gpu


def draw(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def test_prompt_of_more_than_2_to_the_31_values():
    K, g, heads = kda(), gen(1), 128
    lens = [140000, 300, 1]
    rows = sum(lens)
    assert rows * heads * D > 1 << 31
    q, k, v = (draw(g, rows, heads, D) for _ in range(3))
    q /= 11.3
    k /= 11.3
    decay = -torch.rand((rows, heads), generator=g, device="cuda")
    S = torch.randn((3, heads, D, D), generator=g, device="cuda")
    o, out = torch.full_like(v, 7.0), torch.empty_like(S)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    K.kda_lin_prefill(q, k, v, decay, o, S, out, cu_seqlens=cu)
    K.kda_sync_status()
    for n in (1, 2):
        a, b = int(cu[n]), int(cu[n + 1])
        for h in (0, heads - 1):
            d = {x: y[a:b, h:h + 1] for x, y in (("q", q), ("k", k), ("v", v), ("g", decay))}
            d["state"] = S[n:n + 1, h:h + 1]
            close(o[a:b, h:h + 1], out[n:n + 1, h:h + 1], d, torch.bfloat16)


def test_decode_of_more_than_2_to_the_31_states_values():
    K, g, n, heads = kda(), gen(2), 2100, 64
    S = torch.randn((n, heads, D, D), generator=g, device="cuda")
    assert S.numel() > 1 << 31
    q, k, v = (draw(g, n, 1, heads, D) for _ in range(3))
    decay = -torch.rand((n, 1, heads), generator=g, device="cuda")
    o, last, first = torch.empty_like(v), S[-1:].clone(), S[:1].clone()
    K.kda_lin_decode(q, k, v, decay, o, S, S)
    K.kda_sync_status()
    for i, was in ((n - 1, last), (0, first)):
        d = dict(q=q[i], k=k[i], v=v[i], g=decay[i], state=was)
        close(o[i], S[i:i + 1], d, torch.bfloat16)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_rows_of_more_than_2_to_the_31_values(interleaved):
    K, g, rows, heads = kda(), gen(3), 66000, 256
    x = draw(g, rows, heads, D)
    assert x.numel() > 1 << 31
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    inv = 10000.0 ** (-torch.arange(64, device="cuda") / 64)
    kept = {r: x[r:r + 3].clone() for r in (0, rows - 3)}
    K.kda_attn_rope(x, None, pos, inv, interleaved=interleaved)
    K.kda_sync_status()
    for r, was in kept.items():
        ref = rope64(was, pos[r:r + 3, None], inv, [0] * 64, interleaved, 1.0)
        near(x[r:r + 3], was, ref, 64, interleaved, 1.0)


def test_pages_behind_4_gigabytes():
    K, pages = kda(), 60000
    cache = K.kv4_cache(pages, 8, 64)
    assert cache.numel() > 1 << 32
    cache[:2].random_(generator=gen(4))
    cache[-2:].random_(generator=gen(5))
    first, last = cache[:2].clone(), cache[-2:].clone()
    src = torch.tensor([0, pages - 1, 1], dtype=torch.int32).cuda()
    dst = torch.tensor([pages - 3, 5, 59001], dtype=torch.int32).cuda()
    K.kda_attn_kv4_copy([cache], src, dst, torch.tensor([3], dtype=torch.int32).cuda())
    K.kda_sync_status()
    assert torch.equal(cache[pages - 3], first[0]) and torch.equal(cache[5], last[1])
    assert torch.equal(cache[59001], first[1])
    assert torch.equal(cache[:2], first) and torch.equal(cache[-2:], last)
