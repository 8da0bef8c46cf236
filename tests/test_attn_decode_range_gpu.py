"""kda_attn_kv4_decode where the cache's values differ much in size between sequences and within
one, and with the weights' rounding that its header states."""

import numpy as np
import pytest
import torch

from _attn import D, Host, attend64, bf16_bits, close, random_cache
from _util import kda
from test_attn_kv4_gpu import dev, pages_for

pytestmark = pytest.mark.gpu


def v_parameters(data, page):
    """uint16 [pages, kv, tokens, 2, (step, minimum)], a view."""
    v = data[:, :, page * 136:].view(np.uint16)
    return v.reshape(v.shape[:2] + (page, 2, 2))


def decode(q, data, table, lens, window=0):
    K = kda()
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    K.kda_attn_kv4_decode(q, dev(data), dev(table), torch.tensor(lens, dtype=torch.int32).cuda(),
                          o, lse=lse, window=window)
    K.kda_sync_status()
    return o, lse


def check(q, o, lse, host, table, lens, kv, which, window=0):
    """Of the sequences `which`: weights times steps enter the product in FP16."""
    for n in which:
        k, v, size = (torch.from_numpy(np.stack([host.rows(w, table[n], lens[n], h, big)
                                                 for h in range(kv)], 1))
                      for w, big in (("k", False), ("v", False), ("v", True)))
        ref = attend64(q[n].double().cpu(), k, v, window, moved=size)
        close(o[n].cpu(), lse[n].cpu(), ref, q.dtype, weights=torch.float16)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5])
@pytest.mark.parametrize("rows,heads", [(1, 4), (4, 2), (4, 8), (8, 1), (8, 16)])
@pytest.mark.parametrize("lens", [[1, 400], [5, 0, 3, 2, 130]])
def test_the_largest_windows_and_short_sequences(lens, rows, heads, window):
    """A length below the rows less such a window passes 32 bits."""
    rng = np.random.default_rng(43)
    table, total = pages_for(rng, lens, 32)
    data = random_cache(rng, total, 1, 32)
    q = torch.randn((len(lens), rows, heads, D), generator=torch.Generator().manual_seed(44)).to(
        torch.float16).cuda()
    o, lse = decode(q, data, table, lens, window)
    check(q, o, lse, Host(data), table, lens, 1, range(len(lens)), window)


def small_steps(n_seqs, length, page, others, seed):
    """A cache whose odd sequences have 32 rows of V without a step and then steps of about 1e-6,
    and whose even ones have steps of about `others`."""
    rng = np.random.default_rng(seed)
    lens = [length] * n_seqs
    table, total = pages_for(rng, lens, page)
    data = random_cache(rng, total, 1, page)
    par = v_parameters(data, page)
    step, least = rng.uniform(0.5, 1.0, (n_seqs, length, 2)), rng.normal(0, 4, (n_seqs, length, 2))
    pos = np.arange(length)
    for n in range(n_seqs):
        unit = np.where(pos < 32, 0.0, 1e-6) if n % 2 else np.full(length, others)
        bits = np.stack([bf16_bits(step[n] * unit[:, None]),
                         bf16_bits(least[n] * (1e-6 if n % 2 else others))], -1)
        par[table[n, pos // page], 0, pos % page] = bits
    return data, table, lens


@pytest.mark.parametrize("heads,rows", [(1, 1), (4, 2), (8, 2), (4, 8)])
@pytest.mark.parametrize("n_seqs", [2, 701])
def test_small_steps_behind_rows_without_a_step(n_seqs, heads, rows):
    """Small values keep their precision, whatever the CTA worked on before."""
    q = torch.randn((n_seqs, rows, heads, D), generator=torch.Generator().manual_seed(41)).to(
        torch.bfloat16).cuda()
    got = []
    for others in (0.3, 3e4, 3e-9):
        data, table, lens = small_steps(n_seqs, 150, 16, others, 42)
        o, lse = decode(q, data, table, lens)
        check(q, o, lse, Host(data), table, lens, 1, range(1, n_seqs, 1 if n_seqs < 9 else 50))
        got.append((o[1::2], lse[1::2]))
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("name", ["append", "read", "decode"])
def test_no_sequences_are_refused(name):
    K = kda()
    cache = K.kv4_cache(2, 1, 16)
    table, lens = (torch.zeros(shape, dtype=torch.int32, device="cuda") for shape in ((0, 2), (0,)))
    x = torch.zeros((0, 1, D), dtype=torch.float16, device="cuda")
    with pytest.raises(K.KdaError, match="n_seqs"):
        if name == "decode":
            K.kda_attn_kv4_decode(x, cache, table, lens, x.clone())
        else:
            getattr(K, "kda_attn_kv4_" + name)(x, x, cache, table, lens)
    if name != "decode":
        y = torch.zeros((3, 1, D), dtype=torch.float16, device="cuda")
        with pytest.raises(ValueError, match="divide"):
            getattr(K, "kda_attn_kv4_" + name)(y, y, cache, table, lens)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page,lens,rows,heads,kv,window", [
    (64, [1, 64, 65, 200], 1, 8, 2, 0), (32, [300, 15, 16, 17, 257], 8, 4, 2, 0),
    (16, [400, 70, 3], 3, 4, 2, 64), (64, [150, 90], 8, 16, 1, 0), (256, [700, 2, 513], 5, 12, 2, 100),
    (128, [5000, 1], 4, 4, 1, 0), (64, [4097, 63], 1, 4, 2, 0)])
def test_weights_keep_eleven_bits(page, lens, rows, heads, kv, window, dtype):
    """Weights times steps are rounded to FP16, not to fewer bits."""
    rng = np.random.default_rng(45)
    table, total = pages_for(rng, lens, page)
    data = random_cache(rng, total, kv, page)
    q = torch.randn((len(lens), rows, heads, D), generator=torch.Generator().manual_seed(46)).to(
        dtype).cuda()
    o, lse = decode(q, data, table, lens, window)
    check(q, o, lse, Host(data), table, lens, kv, range(len(lens)), window)


@pytest.mark.parametrize("rows,heads", [(1, 4), (4, 8)])
@pytest.mark.parametrize("q_exp,v_exp", [(95, 0), (-60, 0), (0, 96), (0, -60), (95, 96)])
def test_queries_and_values_far_from_one(q_exp, v_exp, rows, heads):
    """The ends of what the header states."""
    rng = np.random.default_rng(47)
    lens = [700, 90]
    table, total = pages_for(rng, lens, 64)
    data = random_cache(rng, total, 1, 64)
    par = v_parameters(data, 64)
    # exponents up: a BF16 number's are bits 7..14 (values here reach 4)
    par[:] += np.uint16((v_exp - (2 if v_exp > 0 else 0)) % 512 << 7)
    q = torch.randn((2, rows, heads, D), generator=torch.Generator().manual_seed(48)).clamp(-2, 2)
    q = (q * 2.0 ** q_exp).to(torch.bfloat16).cuda()
    K = kda()
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    scale = 0.09 * 2.0 ** -q_exp
    K.kda_attn_kv4_decode(q, dev(data), dev(table), torch.tensor(lens, dtype=torch.int32).cuda(),
                          o, lse=lse, scale=scale)
    K.kda_sync_status()
    host = Host(data)
    for n, length in enumerate(lens):
        k, v, size = (torch.from_numpy(host.rows(w, table[n], length, 0, big))[:, None]
                      for w, big in (("k", False), ("v", False), ("v", True)))
        assert 0 < float(v.abs().max()) <= 2.0 ** max(v_exp, 2)
        ref = attend64(q[n].double().cpu(), k, v, scale=scale, moved=size)
        close(o[n].cpu(), lse[n].cpu(), ref, q.dtype, weights=torch.float16)
