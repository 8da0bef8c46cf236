"""The 4-bit paged cache: what append writes, read returns and decode attends over, against the
documented layout and a plain 64-bit form."""

import itertools

import numpy as np
import pytest
import torch

from _attn import D, TYPES, Host, attend64, close, quantise, random_cache
from _util import kda

pytestmark = pytest.mark.gpu


def pages_for(rng, lens, page, spare=2):
    """A page table of pages in no order, and the number of pages of the cache."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    order = rng.permutation(total)
    table = np.zeros((len(lens), max(1, max(need) + 1)), dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, total


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def offsets(rows):
    return torch.tensor([0] + list(itertools.accumulate(rows)), dtype=torch.int32).cuda()


# ---------------------------------------------------------------- append

def host_append(cache, table, lens, new, k, v):
    h = Host(cache)
    at = 0
    for n, (length, r) in enumerate(zip(lens, new)):
        for i in range(r):
            pos = length - r + i
            for which, x in (("k", k), ("v", v)):
                c, s, m = quantise(x[at + i:at + i + 1])
                for hd in range(x.shape[1]):
                    h.write(which, table[n, pos // h.page], pos % h.page, hd, c[0, hd], s[0, hd],
                            m[0, hd])
        at += r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page,kv,ctx,new", [
    (16, 1, [0], [1]), (16, 2, [3, 15, 16, 0], [2, 1, 33, 16]), (64, 3, [60, 0], [70, 5]),
    (32, 2, [7, 0, 100], [9, 0, 1]), (128, 1, [120], [20]), (256, 1, [0, 250], [3, 30])])
def test_append_writes_the_documented_bytes(page, kv, ctx, new, dtype):
    K = kda()
    rng = np.random.default_rng(page + kv)
    lens = [a + b for a, b in zip(ctx, new)]
    table, total = pages_for(rng, lens, page)
    cache = rng.integers(0, 256, (total, kv, page * 144), dtype=np.uint8)
    g = torch.Generator().manual_seed(page)
    k, v = ((torch.randn((sum(new), kv, D), generator=g) * 2 + 0.3).to(dtype) for _ in range(2))
    got = dev(cache)
    K.kda_attn_kv4_append(k.cuda(), v.cuda(), got, dev(table),
                          torch.tensor(lens, dtype=torch.int32).cuda(), cu_seqlens=offsets(new))
    K.kda_sync_status()
    host_append(cache, table, lens, new, k.double().numpy(), v.double().numpy())
    assert np.array_equal(got.cpu().numpy(), cache)   # bytes of other tokens among them


def test_append_uniform_strided_rows_and_other_stream():
    K = kda()
    rng = np.random.default_rng(5)
    lens, new, kv, page = [40, 17, 64], [4, 4, 4], 2, 32
    table, total = pages_for(rng, lens, page)
    cache = np.zeros((total, kv, page * 144), dtype=np.uint8)
    g = torch.Generator().manual_seed(6)
    both = torch.randn((12, 2 * kv * D + 16), generator=g).to(torch.bfloat16).cuda()
    k = both[:, :kv * D].unflatten(1, (kv, D))
    v = both[:, kv * D:2 * kv * D].unflatten(1, (kv, D))
    got = dev(cache)
    t, ln = dev(table), torch.tensor(lens, dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        K.kda_attn_kv4_append(k, v, got, t, ln)
    side.synchronize()
    host_append(cache, table, lens, new, k.cpu().double().numpy(), v.cpu().double().numpy())
    assert np.array_equal(got.cpu().numpy(), cache)


def test_append_at_the_borders_between_codes():
    """Values on, next to and between the borders; groups of one value; steps that are BF16
    numbers exactly and steps that are not."""
    K = kda()
    rows = []
    for lo, step in ((0.0, 1.0), (-3.75, 0.5), (-1.5, 0.25), (2.0, 0.0), (-0.0, 0.0), (5.0, 0.375),
                     (-100.0, 2.0), (0.0, 2.0 ** -20)):
        x = lo + step * (np.arange(64) % 31) / 2.0          # codes and halves
        rows.append(np.concatenate([x, x[::-1] * 1.0078125]))
    # a tiny value beside the border at zero: -1.5 s, s = 1
    x = np.linspace(-1.5, 13.5, 64)
    x[10:14] = (2.0 ** -30, -2.0 ** -30, 0.0, 2.0 ** -14)
    rows.append(np.concatenate([x, -x]))
    rng = np.random.default_rng(0)
    for _ in range(200):
        rows.append(rng.normal(0, 2.0 ** rng.integers(-12, 12), D) + rng.normal(0, 4))
    for dtype in TYPES:
        x = torch.tensor(np.stack(rows))[:, None].clamp(-60000, 60000).to(dtype)
        n = x.shape[0]
        page = 64
        table = np.arange(-(-n // page) + 1, dtype=np.int32)[None]
        cache = np.zeros((table.size, 1, page * 144), dtype=np.uint8)
        got = dev(cache)
        K.kda_attn_kv4_append(x.cuda(), x.flip(0).cuda(), got, dev(table),
                              torch.tensor([n], dtype=torch.int32).cuda())
        host_append(cache, table, [n], [n], x.double().numpy(), x.flip(0).double().numpy())
        assert np.array_equal(got.cpu().numpy(), cache)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_value_spoils_its_group_only(bad):
    K = kda()
    g = torch.Generator().manual_seed(7)
    k = torch.randn((5, 1, D), generator=g).to(torch.bfloat16)
    v = k.flip(0).contiguous()
    k[2, 0, 70] = bad
    cache, table = K.kv4_cache(1, 1, 16), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    ln = torch.tensor([5], dtype=torch.int32).cuda()
    K.kda_attn_kv4_append(k.cuda(), v.cuda(), cache, table, ln)
    a, b = torch.empty((5, 1, D), dtype=torch.bfloat16, device="cuda"), torch.empty(
        (5, 1, D), dtype=torch.bfloat16, device="cuda")
    K.kda_attn_kv4_read(a, b, cache, table, ln)
    assert bool(torch.isnan(a[2, 0, 64:]).all())
    a[2, 0, 64:] = 0
    assert bool(torch.isfinite(a.float()).all()) and bool(torch.isfinite(b.float()).all())


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page,kv,ctx,new", [
    (16, 1, [0], [1]), (32, 2, [3, 0, 40], [30, 17, 0]), (64, 1, [100, 0], [29, 64]),
    (256, 2, [0], [300])])
def test_read_returns_the_cached_values(page, kv, ctx, new, dtype):
    K = kda()
    rng = np.random.default_rng(page)
    lens = [a + b for a, b in zip(ctx, new)]
    table, total = pages_for(rng, lens, page)
    data = random_cache(rng, total, kv, page)
    T = sum(new)
    wide = [torch.full((T, kv * D + 8), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    k, v = (w[:, :kv * D].unflatten(1, (kv, D)) for w in wide)
    K.kda_attn_kv4_read(k, v, dev(data), dev(table), torch.tensor(lens, dtype=torch.int32).cuda(),
                        cu_seqlens=offsets(new))
    K.kda_sync_status()
    host = Host(data)
    for which, got, w in (("k", k, wide[0]), ("v", v, wide[1])):
        at = 0
        for n, r in enumerate(new):
            for h in range(kv):
                ref = host.rows(which, table[n], lens[n], h)[lens[n] - r:]
                # m + s c rounds once to FP32 and once to the type
                tol = np.abs(ref) * (torch.finfo(dtype).eps / 2 + 2.0 ** -23) + 2.0 ** -24
                assert (np.abs(got[at:at + r, h].double().cpu().numpy() - ref) <= tol).all()
            at += r
        assert bool((w[:, kv * D:] == 7).all())


# ---------------------------------------------------------------- decode

def decode_case(page, lens, rows, heads, kv, dtype, window=0, seed=0, spoil=True, ws=None):
    K = kda()
    rng = np.random.default_rng(seed)
    table, total = pages_for(rng, lens, page)
    data = random_cache(rng, total, kv, page)
    if spoil:  # whatever lies behind a sequence's end: parameters that are NaN
        for n, length in enumerate(lens):
            if length % page:
                blk = data[table[n, length // page]]
                for at in (page * 64, page * 136):
                    blk[:, at + length % page * 8:at + page * 8] = 0xFF
    g = torch.Generator().manual_seed(seed)
    N = len(lens)
    q = torch.randn((N, rows, heads, D), generator=g).to(dtype).cuda()
    o = torch.full_like(q, 7.0)
    lse = torch.full((N, rows, heads), 7.0, device="cuda")
    K.kda_attn_kv4_decode(q, dev(data), dev(table), torch.tensor(lens, dtype=torch.int32).cuda(),
                          o, lse=lse, window=window, workspace=ws)
    K.kda_sync_status()
    host = Host(data)
    for n, length in enumerate(lens):
        k, v = (torch.from_numpy(np.stack([host.rows(w, table[n], length, h) for h in range(kv)],
                                          1)) for w in "kv")
        size = torch.from_numpy(np.stack([host.rows("v", table[n], length, h, True)
                                          for h in range(kv)], 1))
        ref = attend64(q[n].double().cpu(), k, v, window, moved=size)
        # weights times steps enter the product in BF16
        close(o[n].cpu(), lse[n].cpu(), ref, dtype, weights=torch.bfloat16)
    return o, lse


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 2), (5, 1), (16, 1), (7, 7)])
@pytest.mark.parametrize("rows,lens", [(1, [1, 64, 65, 200]), (4, [4, 130, 33])])
def test_decode_heads(rows, lens, heads, kv, dtype):
    decode_case(64, lens, rows, heads, kv, dtype, seed=heads)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("rows", [1, 2, 8])
def test_decode_pages_and_rows(page, rows):
    decode_case(page, [300, 15, 16, 17, 257], rows, 4, 2, torch.bfloat16, seed=page + rows)


@pytest.mark.parametrize("lens", [[0], [0, 1, 2, 3], [5, 0, 8]])
def test_decode_rows_that_see_nothing(lens):
    o, lse = decode_case(16, lens, 4, 4, 1, torch.bfloat16, seed=3)
    for n, length in enumerate(lens):
        empty = max(0, 4 - length)
        assert bool((o[n, :empty] == 0).all()) and bool((lse[n, :empty] == -float("inf")).all())


@pytest.mark.parametrize("window", [1, 5, 64, 100, 2 ** 31 - 1])
def test_decode_window(window):
    decode_case(32, [400, 70, 3], 3, 4, 2, torch.float16, window=window, seed=window % 97)


def test_decode_many_query_heads():
    decode_case(64, [150, 90], 8, 16, 1, torch.bfloat16, seed=8)     # 128 query rows a KV head
    decode_case(64, [150], 5, 12, 2, torch.bfloat16, seed=9)


def test_decode_long_and_ragged():
    decode_case(64, [4097, 1, 2500, 63], 1, 4, 2, torch.bfloat16, seed=10)
    decode_case(128, [9001], 2, 4, 1, torch.float16, seed=11)


def test_decode_many_sequences():
    rng = np.random.default_rng(12)
    decode_case(16, [int(x) for x in rng.integers(0, 40, 1100)], 1, 2, 1, torch.bfloat16, seed=12)


def test_decode_scale_and_large_queries():
    """Scores far from zero, and query values across FP16's and BF16's range."""
    K = kda()
    rng = np.random.default_rng(13)
    table, total = pages_for(rng, [333], 64)
    data = random_cache(rng, total, 1, 64)
    host = Host(data)
    k, v = (torch.from_numpy(host.rows(w, table[0], 333, 0))[:, None] for w in "kv")
    size = torch.from_numpy(host.rows("v", table[0], 333, 0, True))[:, None]
    for unit in (2.0 ** -30, 2.0 ** 40):
        q = (torch.randn((1, 1, 2, D), generator=torch.Generator().manual_seed(1)) * unit
             ).to(torch.bfloat16)
        o, lse = torch.empty_like(q).cuda(), torch.empty((1, 1, 2), device="cuda")
        K.kda_attn_kv4_decode(q.cuda(), dev(data), dev(table),
                              torch.tensor([333], dtype=torch.int32).cuda(), o, lse=lse,
                              scale=0.1 / unit)
        ref = attend64(q[0].double(), k, v, scale=0.1 / unit, moved=size)
        close(o[0].cpu(), lse[0].cpu(), ref, torch.bfloat16, weights=torch.bfloat16)


def test_decode_same_bits_again_graph_and_dirty_workspace():
    K = kda()
    rng = np.random.default_rng(14)
    lens = [3000, 20, 777]
    table, total = pages_for(rng, [3200, 900, 900], 64)
    cache, t = dev(random_cache(rng, total, 2, 64)), dev(table)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    q = torch.randn((3, 2, 8, D), generator=torch.Generator().manual_seed(2)).to(
        torch.bfloat16).cuda()
    ws = K.kda_attn_kv4_workspace(3, 2, 8, 2)
    o, lse = torch.empty_like(q), torch.empty((3, 2, 8), device="cuda")
    K.kda_attn_kv4_decode(q, cache, t, ln, o, lse=lse, workspace=ws)
    first = o.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kda_attn_kv4_decode(q, cache, t, ln, o, lse=lse, workspace=ws)
    for fill in (0, 0xFF, 0x5A):
        ws.fill_(fill)
        o.fill_(7.0)
        graph.replay()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    # the same graph for other lengths
    ln.copy_(torch.tensor([100, 850, 1], dtype=torch.int32))
    graph.replay()
    want = torch.empty_like(o)
    K.kda_attn_kv4_decode(q, cache, t, ln, want)
    assert torch.equal(o, want)
    K.kda_sync_status()


def test_decode_equals_prefill_over_read_rows():
    """The cache's values through read and kda_attn_prefill: the same attention."""
    K = kda()
    rng = np.random.default_rng(15)
    lens, rows = [200, 77], 3
    table, total = pages_for(rng, lens, 32)
    cache, t = dev(random_cache(rng, total, 2, 32)), dev(table)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    q = torch.randn((2, rows, 4, D), generator=torch.Generator().manual_seed(3)).half().cuda()
    o, lse = torch.empty_like(q), torch.empty((2, rows, 4), device="cuda")
    K.kda_attn_kv4_decode(q, cache, t, ln, o, lse=lse)
    k, v = (torch.empty((sum(lens), 2, D), dtype=torch.float16, device="cuda") for _ in range(2))
    K.kda_attn_kv4_read(k, v, cache, t, ln, cu_seqlens=offsets(lens))
    o2, lse2 = torch.empty_like(q), torch.empty((2, rows, 4), device="cuda")
    K.kda_attn_prefill(q.view(-1, 4, D), k, v, o2.view(-1, 4, D), lse=lse2.view(-1, 4),
                       cu_seqlens=offsets([rows] * 2), cu_seqlens_k=offsets(lens))
    # k and v rounded to FP16 move a score by 2^-11 |q||k| / sqrt(128), a few 2^-9 at most
    assert float((o - o2).abs().max()) < 0.05 and float((lse - lse2).abs().max()) < 0.02


def test_cache_past_32_bits():
    """Pages whose byte offsets pass 2^32."""
    K = kda()
    kv, page = 8, 256
    pages = (1 << 32) // (kv * page * 144) + 40
    cache = torch.empty((pages, kv, page * 144), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[pages - 1, 0, pages - 7]], dtype=torch.int32).cuda()
    n = 600
    ln = torch.tensor([n], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn((n, kv, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    K.kda_attn_kv4_append(k, v, cache, table, ln)
    a, b = torch.empty_like(k), torch.empty_like(v)
    K.kda_attn_kv4_read(a, b, cache, table, ln)
    q = torch.randn((1, 1, 16, D), generator=g).to(torch.bfloat16).cuda()
    o, lse = torch.empty_like(q), torch.empty((1, 1, 16), device="cuda")
    K.kda_attn_kv4_decode(q, cache, table, ln, o, lse=lse)
    K.kda_sync_status()
    for x, y in ((k, a), (v, b)):
        c, s, m = quantise(x.double().cpu().numpy())
        ref = (m[..., None] + s[..., None] * c.reshape(c.shape[:2] + (2, 64))).reshape(c.shape)
        got = y.double().cpu().numpy()
        assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 * 1.001).all()
    ref = attend64(q[0].double(), a.double(), b.double())
    # a and b are the cache's values rounded to BF16
    assert float((o[0].double() - ref[0]).abs().max()) < 0.05


@pytest.mark.parametrize("kind", ["page_high", "page_negative", "len_high", "len_negative",
                                  "len_below_rows"])
def test_bad_pages_and_lengths_are_reported(kind):
    """Nothing outside the cache is touched: the kernels check every page number and length before
    they use it."""
    K = kda()
    page, kv = 16, 2
    whole = torch.full((10, kv, page * 144), 0x3C, dtype=torch.uint8, device="cuda")
    cache = whole[3:7]
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    ln = torch.tensor([20, 30], dtype=torch.int32)
    if kind == "page_high":
        table[1, 1] = 4
    if kind == "page_negative":
        table[1, 0] = -1
    if kind == "len_high":
        ln[1] = 33
    if kind == "len_negative":
        ln[1] = -1
    if kind == "len_below_rows":
        ln[1] = 3
    table, ln = table.cuda(), ln.cuda()
    x = torch.randn((40, kv, D), generator=torch.Generator().manual_seed(5)).to(
        torch.bfloat16).cuda()
    K.kda_attn_kv4_append(x, x, cache, table, ln)
    with pytest.raises(K.KdaError, match="cache"):
        K.kda_sync_status()
    assert bool((whole[:3] == 0x3C).all()) and bool((whole[7:] == 0x3C).all())
    a, b = torch.empty_like(x), torch.empty_like(x)
    K.kda_attn_kv4_read(a, b, cache, table, ln)
    with pytest.raises(K.KdaError, match="cache"):
        K.kda_sync_status()
    q = torch.randn((2, 1, 4, D), generator=torch.Generator().manual_seed(6)).to(
        torch.bfloat16).cuda()
    o = torch.full_like(q, 7.0)
    K.kda_attn_kv4_decode(q, cache, table, ln, o)
    if kind != "len_below_rows":   # one query row: 3 positions are enough
        with pytest.raises(K.KdaError, match="cache"):
            K.kda_sync_status()
    K.kda_sync_status()


def test_binding_refusals():
    K = kda()
    cache = K.kv4_cache(4, 2, 32)
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    ln = torch.ones(2, dtype=torch.int32, device="cuda")
    x = torch.zeros((2, 2, D), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 4, D), dtype=torch.bfloat16, device="cuda")
    for call, error in (
            (lambda: K.kda_attn_kv4_append(x.float(), x, cache, table, ln), TypeError),
            (lambda: K.kda_attn_kv4_append(x, x.half(), cache, table, ln), TypeError),
            (lambda: K.kda_attn_kv4_append(x[:, :1], x[:, :1], cache, table, ln), ValueError),
            (lambda: K.kda_attn_kv4_append(x, x, cache[..., :-1], table, ln), ValueError),
            (lambda: K.kda_attn_kv4_append(x, x, cache, table.long(), ln), TypeError),
            (lambda: K.kda_attn_kv4_append(x, x, cache, table[:1], ln), ValueError),
            (lambda: K.kda_attn_kv4_append(x, x, cache, table, ln, ln), ValueError),
            (lambda: K.kda_attn_kv4_decode(q, cache, table, ln, x), ValueError),
            (lambda: K.kda_attn_kv4_decode(q[:1], cache, table, ln, q[:1]), ValueError),
            (lambda: K.kda_attn_kv4_decode(q, cache.cpu(), table, ln, q.clone()), TypeError),
            (lambda: K.kv4_cache(4, 2, 33), ValueError)):
        with pytest.raises(error):
            call()
    assert K.kda_attn_kv4_decode(q, cache, table, ln, q.clone()) is None
    K.kda_sync_status()
