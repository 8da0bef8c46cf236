"""kda_attn_prefill over batches with more items than multiprocessors, against a plain 64-bit form
of whole sequences: ragged lengths, large scores, masks."""

import itertools
import math

import pytest
import torch

from _attn import D, TYPES, close
from _util import kda

pytestmark = pytest.mark.gpu

# 32 heads over 8, 64 tokens to an item: 12 sequences that make some 500 items, most of them with a
# last tile that is not full and starts behind position 127.
RAGGED = [500, 333, 1, 270, 0, 777, 150, 461, 190, 64, 299, 135]


def offsets(lens):
    return torch.tensor([0] + list(itertools.accumulate(lens)), dtype=torch.int32).cuda()


def draw(seed, lq, lk, heads, kv, dtype, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((sum(lq), heads, D), generator=g) * spread
    k = torch.randn((sum(lk), kv, D), generator=g)
    v = torch.randn((sum(lk), kv, D), generator=g) + 0.5
    return [x.to(dtype).cuda() for x in (q, k, v)]


def whole64(q, k, v, window=0, scale=1 / math.sqrt(D)):
    """All rows of one sequence at a time: o, lse, sum of weights times |v| (attend64's values)."""
    R, H = q.shape[:2]
    L, Hk = k.shape[:2]
    pos = torch.arange(R, device=q.device)[:, None] + (L - R)
    key = torch.arange(L, device=q.device)[None]
    sees = (key <= pos) & ((key > pos - window) if window else (key >= 0))
    some = sees.any(1)
    o = torch.zeros((R, H, D), dtype=torch.float64, device=q.device)
    lse = torch.full((R, H), -math.inf, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(o)
    for h in range(H if bool(some.any()) else 0):
        hk = h // (H // Hk)
        s = (q[some, h].double() @ k[:, hk].double().T * scale).masked_fill(~sees[some], -math.inf)
        lse[some, h] = torch.logsumexp(s, 1)
        w = torch.exp(s - lse[some, h][:, None])
        o[some, h] = w @ v[:, hk].double()
        mag[some, h] = w @ v[:, hk].double().abs()
    return o, lse, mag


def check(q, k, v, o, lse, lq, lk, window=0):
    a = b = 0
    for m, n in zip(lq, lk):
        rows, keys = slice(a, a + m), slice(b, b + n)
        if m:
            close(o[rows], lse[rows], whole64(q[rows], k[keys], v[keys], window), q.dtype)
        a, b = a + m, b + n


def call(q, k, v, lq, lk, window=0, ws=None):
    K = kda()
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    K.kda_attn_prefill(q, k, v, o, lse=lse, cu_seqlens=offsets(lq), cu_seqlens_k=offsets(lk),
                       window=window, workspace=ws)
    K.kda_sync_status()
    return o, lse


@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("dtype", TYPES)
def test_large_scores_of_other_sequences_rows(dtype, window):
    """A last tile that is not full is loaded with the next sequence's queries behind its own,
    which score far above 10 against this sequence's keys.  They change nothing: rows follow the
    formula, and repeats give the same bits."""
    q, k, v = draw(31, RAGGED, RAGGED, 32, 8, dtype, spread=6.0)
    o, lse = call(q, k, v, RAGGED, RAGGED, window)
    check(q, k, v, o, lse, RAGGED, RAGGED, window)
    for _ in range(8):
        o2, lse2 = call(q, k, v, RAGGED, RAGGED, window)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cu", [[0, 5000, 4000, 10000], [0, 10000] * 4 + [0, 10000],
                                [0, 7000, 20000, 10000], [0, -50, 6000, 10000]])
def test_offsets_that_fall_with_many_items(cu):
    """The plan's list would not hold the items of sequences that overlap: none is taken, the
    status says so, and nothing outside o is written."""
    K = kda()
    T = cu[-1]
    q, k, v = draw(32, [T], [T], 32, 8, torch.bfloat16)
    guard = torch.full((T + 600, 32, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 600, 32), 7.0, device="cuda")
    ws = K.kda_attn_prefill_workspace(T, len(cu) - 1, 32, 8)
    ws.fill_(0x5A)
    K.kda_attn_prefill(q, k, v, guard[300:300 + T], lse=lse[300:300 + T], workspace=ws,
                       cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    with pytest.raises(K.KdaError, match="cu_seqlens"):
        K.kda_sync_status()
    assert bool((guard == 7).all()) and bool((lse == 7).all())


def test_offsets_short_of_the_total_with_many_items():
    """Offsets that rise but do not start at 0 and end at the total: reported, and the rows that
    they name are done."""
    K = kda()
    lens = [300, 0, 900]
    q, k, v = draw(33, [40] + lens + [60], [40] + lens + [60], 32, 8, torch.float16)
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    K.kda_attn_prefill(q, k, v, o, lse=lse, cu_seqlens=offsets(lens) + 40)
    with pytest.raises(K.KdaError, match="cu_seqlens"):
        K.kda_sync_status()
    check(*(x[40:1240] for x in (q, k, v, o, lse)), lens, lens)
    for x in (o, lse):
        assert bool((x[:40] == 7).all()) and bool((x[1240:] == 7).all())


def steep(T, peaks, rows, dtype, heads=2, kv=2):
    """Scores 0 but for `peaks`, key: score; the last `rows` of T rows are queries."""
    q = torch.ones((rows, heads, D), dtype=dtype, device="cuda")
    k = torch.zeros((T, kv, D), dtype=dtype, device="cuda")
    for at, score in peaks.items():
        k[at] = score / math.sqrt(D)
    v = torch.randn((T, kv, D), generator=torch.Generator().manual_seed(34)).clamp(-1.2, 1.2)
    return q, k, v.to(dtype).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", [60, 70, 86, 87.7, 88.4, 95])
@pytest.mark.parametrize("T,peaks,rows,window", [
    (700, [40], 600, 0), (700, [200], 700, 0), (700, [200], 500, 333),  # items whole
    (3001, [200], 4, 0), (3001, [500], 4, 2800),                        # shares of an item's keys
    (3001, [500, 512], 4, 0)])                                          # in two shares
def test_one_key_far_above_the_first(T, peaks, rows, window, score, dtype):
    """Weights are taken relative to scores seen first: of a key 2^86 to 2^138 above them, and of
    keys far below it, nothing is lost.  (Values are small enough that their sums stay finite.)"""
    q, k, v = steep(T, {at: score + 2 * i for i, at in enumerate(peaks)}, rows, dtype)
    o, lse = call(q, k, v, [rows], [T], window)
    check(q, k, v, o, lse, [rows], [T], window)


@pytest.mark.parametrize("score", [86, 87.7, 88.4])
def test_one_key_far_above_the_first_in_a_batch(score):
    lens = [700, 64, 900, 333]
    parts = [steep(n, {min(200, n // 2): score}, n, torch.bfloat16, 32, 8) for n in lens]
    q, k, v = (torch.cat(x) for x in zip(*parts))
    o, lse = call(q, k, v, lens, lens)
    check(q, k, v, o, lse, lens, lens)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3])
@pytest.mark.parametrize("lq,lk,heads,kv", [
    ([5, 70, 4], [2, 0, 4], 8, 2), ([700, 400, 900], [3, 399, 130], 16, 8), ([9], [4], 4, 1)])
def test_the_largest_windows_and_rows_before_the_first_key(lq, lk, heads, kv, window, dtype):
    """Positions below zero less such a window pass 32 bits."""
    q, k, v = draw(35, lq, lk, heads, kv, dtype)
    o, lse = call(q, k, v, lq, lk, window)
    check(q, k, v, o, lse, lq, lk, window)


def test_windows_past_the_c_type():
    """Any window of more positions than there are is none; below zero all are refused."""
    K = kda()
    q, k, v = draw(36, [200], [200], 4, 2, torch.bfloat16)
    o, want = torch.empty_like(q), torch.empty_like(q)
    K.kda_attn_prefill(q, k, v, want)
    cache, table = K.kv4_cache(4, 2, 64), torch.arange(4, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([200], dtype=torch.int32).cuda()
    K.kda_attn_kv4_append(k, v, cache, table, lens)
    one, one_want = torch.empty_like(q[:1]), torch.empty_like(q[:1])
    K.kda_attn_kv4_decode(q[-1:].clone(), cache, table, lens, one_want)
    for window in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 + 1):
        K.kda_attn_prefill(q, k, v, o, window=window)
        K.kda_attn_kv4_decode(q[-1:].clone(), cache, table, lens, one, window=window)
        assert torch.equal(o, want) and torch.equal(one, one_want)
    for window in (-1, -2 ** 31, -2 ** 32, -2 ** 32 + 5):
        with pytest.raises(K.KdaError):
            K.kda_attn_prefill(q, k, v, o, window=window)
        with pytest.raises(K.KdaError):
            K.kda_attn_kv4_decode(q[-1:].clone(), cache, table, lens, one, window=window)
    K.kda_sync_status()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lq,lk,heads,kv,window", [
    (RAGGED, RAGGED, 32, 8, 0),
    (RAGGED, [n + 7 * i for i, n in enumerate(RAGGED)], 20, 4, 250),     # behind contexts
    (RAGGED, [max(0, n - 40 * (i % 5)) for i, n in enumerate(RAGGED)], 16, 16, 0),  # empty rows
    ([n % 61 + 1 for n in range(40)], [n % 61 + 1 for n in range(40)], 8, 8, 0),    # short ones
    ([1] * 200, [9 * n + 1 for n in range(200)], 6, 2, 0),               # single rows
    ([1, 3000, 2], [1, 4096, 700], 32, 8, 1000),
    ([2200], [2300], 24, 24, 0)])                                        # one, no list
def test_batches_with_more_items_than_multiprocessors(lq, lk, heads, kv, window, dtype):
    """Items by a list and tickets, over several rounds; the same bits again."""
    q, k, v = draw(37, lq, lk, heads, kv, dtype)
    o, lse = call(q, k, v, lq, lk, window)
    check(q, k, v, o, lse, lq, lk, window)
    ws = kda().kda_attn_prefill_workspace(sum(lq), len(lq), heads, kv)
    for fill in (0, 0xFF, 0x5A):
        ws.fill_(fill)
        o2, lse2 = call(q, k, v, lq, lk, window, ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_batch_in_a_graph_with_other_offsets(dtype):
    """The plan is made anew at each replay, from the offsets that are there then."""
    K = kda()
    T, n = sum(RAGGED), len(RAGGED)
    cu = offsets(RAGGED)
    q, k, v = draw(38, [T], [T], 32, 8, dtype)
    ws = K.kda_attn_prefill_workspace(T, n, 32, 8)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    K.kda_attn_prefill(q, k, v, o, lse=lse, cu_seqlens=cu, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kda_attn_prefill(q, k, v, o, lse=lse, cu_seqlens=cu, workspace=ws)
    for lens in (RAGGED[::-1], [T] + [0] * (n - 1), [T // n] * (n - 1) + [T - T // n * (n - 1)]):
        cu.copy_(offsets(lens))
        ws.fill_(0xAB)
        o.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        K.kda_sync_status()
        check(q, k, v, o, lse, lens, lens)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("lens,heads,kv,window", [
    ([90, 150, 40], 4, 1, 0),                                  # an item to a multiprocessor
    (RAGGED, 32, 8, 0), (RAGGED, 32, 8, 100)])                 # many more items
def test_rows_that_do_not_see_a_bad_value_follow_the_formula(lens, heads, kv, window, what, bad,
                                                             dtype):
    """Bad values in several sequences, of one head: rows of other heads, rows before them, rows
    whose window has left them behind and other sequences' rows follow the formula."""
    q, k, v = draw(39, lens, lens, heads, kv, dtype)
    sees = torch.zeros(sum(lens), dtype=torch.bool)
    at = 0
    for n in lens:
        if n > 80:
            x = k if what == "k" else v
            x[at + 2 * n // 3, kv - 1, 5] = bad
            last = min(at + n, at + 2 * n // 3 + window) if window else at + n
            sees[at + 2 * n // 3:last] = True
        at += n
    o, lse = call(q, k, v, lens, lens, window)
    group = heads // kv
    hit = torch.zeros(q.shape[:2], dtype=torch.bool)
    hit[sees, heads - group:] = True
    hit = hit.cuda()
    if what == "v":
        got = o[hit][:, 5]
        assert bool((torch.isnan(got) if bad != bad else got == bad).all())
    elif bad != bad:
        assert bool(torch.isnan(o[hit]).all())
    k, v = (torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0) for x in (k, v))
    a = 0
    for n in lens:
        rows = slice(a, a + n)
        if n:
            ref = whole64(q[rows], k[rows], v[rows], window)
            clean = ~hit[rows]
            close(o[rows][clean], lse[rows][clean], [x[clean] for x in ref], dtype)
        a += n


@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("lens", [[333], RAGGED])
def test_sharp_softmax_fp16(lens, window):
    """Scores of +-100 and more: the maximum of a row moves in many blocks, weights underflow."""
    q, k, v = draw(40, lens, lens, 32, 8, torch.float16, spread=30.0)
    o, lse = call(q, k, v, lens, lens, window)
    check(q, k, v, o, lse, lens, lens, window)


@pytest.mark.parametrize("lens,heads,kv", [([600], 1, 1), ([600, 333, 900], 16, 16)])
def test_growing_scores_fp16(lens, heads, kv):
    """Every key beats all before it: the shift moves in every block."""
    q = torch.ones((sum(lens), heads, D), dtype=torch.float16, device="cuda")
    k = torch.cat([torch.arange(n, device="cuda") for n in lens])[:, None, None] / 16.0
    k = (k * torch.ones((1, kv, D), device="cuda")).half()
    v = torch.randn((sum(lens), kv, D), generator=torch.Generator().manual_seed(41)).half().cuda()
    o, lse = call(q, k, v, lens, lens)
    a = 0
    for n in lens:
        rows = slice(a, a + n)
        ro, rl, mag = whole64(q[rows], k[rows], v[rows])
        # scores reach 6400 (log2: 9200): FP32 holds them, and their products with scale and
        # log2 e, to 2^-10 together, which a weight's relative size moves by
        half = torch.finfo(torch.float16).eps / 2
        err = (o[rows].double() - ro).abs()
        assert bool((err <= half * ro.abs() + (half + 2.0 ** -9) * mag).all())
        assert float((lse[rows].double() - rl).abs().max()) <= 2.0 ** -9
        a += n
