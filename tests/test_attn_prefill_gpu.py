"""kda_attn_prefill against a plain 64-bit form: lengths, heads, masks, views, streams."""

import itertools

import pytest
import torch

from _attn import D, TYPES, attend64, close
from _util import kda

pytestmark = pytest.mark.gpu


def offsets(lens):
    return torch.tensor([0] + list(itertools.accumulate(lens)), dtype=torch.int32).cuda()


def draw(seed, lq, lk, heads, kv, dtype, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((sum(lq), heads, D), generator=g) * spread
    k = torch.randn((sum(lk), kv, D), generator=g)
    v = torch.randn((sum(lk), kv, D), generator=g) + 0.5
    return [x.to(dtype).cuda() for x in (q, k, v)]


def check(q, k, v, o, lse, lq, lk, window, dtype, rows=None):
    """Compares every sequence; `rows`: only so many of each one's last rows."""
    a = b = 0
    for m, n in zip(lq, lk):
        r = m if rows is None else min(rows, m)
        sl = slice(a + m - r, a + m)
        ref = attend64(q[sl].double(), k[b:b + n].double(), v[b:b + n].double(), window)
        close(o[sl], lse[sl], ref, dtype)
        a, b = a + m, b + n


def run(lq, lk, heads, kv, dtype, window=0, seed=0, spread=1.0, rows=None):
    K = kda()
    q, k, v = draw(seed, lq, lk, heads, kv, dtype, spread)
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    K.kda_attn_prefill(q, k, v, o, lse=lse, cu_seqlens=offsets(lq), cu_seqlens_k=offsets(lk),
                       window=window)
    K.kda_sync_status()
    check(q, k, v, o, lse, lq, lk, window, dtype, rows)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 2), (5, 1), (14, 2), (16, 1)])
@pytest.mark.parametrize("lq,lk", [([1], [1]), ([2, 1, 17], [2, 1, 17]), ([130], [130])])
def test_small_prompts(lq, lk, heads, kv, dtype):
    run(lq, lk, heads, kv, dtype)


@pytest.mark.parametrize("heads,kv,lens", [
    (2, 1, [255, 1, 256, 257]), (3, 1, [400]), (8, 8, [129, 64]), (128, 1, [9]), (100, 1, [37])])
def test_tile_edges_and_head_groups(heads, kv, lens):
    run(lens, lens, heads, kv, torch.bfloat16, seed=3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lq,lk", [
    ([1, 3], [500, 129]),          # a chunk behind its context
    ([5, 70, 4], [2, 0, 4]),       # fewer keys than queries: rows that see nothing
    ([0, 6, 0, 0, 9, 0], [0, 6, 0, 3, 9, 0])])   # empty sequences
def test_context_empty_rows_and_empty_sequences(lq, lk, dtype):
    run(lq, lk, 8, 2, dtype, seed=4)


@pytest.mark.parametrize("window", [1, 2, 63, 128, 200, 1 << 30, 2 ** 31 - 1])
def test_window(window):
    run([300, 5, 41], [300, 260, 41], 4, 2, torch.bfloat16, window=window, seed=5)


def test_long_prompt_last_rows():
    run([5000], [5000], 4, 1, torch.bfloat16, seed=6, rows=6)
    run([700], [9001], 2, 2, torch.float16, seed=7, rows=5)


def test_sharp_softmax():
    """Scores of +-100 and more: the running maximum moves a lot and weights underflow."""
    run([333], [333], 4, 2, torch.bfloat16, seed=8, spread=30.0)


def test_growing_scores():
    """Every key beats all before it, so the maximum moves at every step."""
    K = kda()
    T = 600
    q = torch.ones((T, 1, D), dtype=torch.bfloat16, device="cuda")
    k = (torch.arange(T, device="cuda")[:, None, None] / 16.0 * torch.ones((1, 1, D), device="cuda")
         ).to(torch.bfloat16)
    v = torch.randn((T, 1, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    o, lse = torch.empty_like(q), torch.empty((T, 1), device="cuda")
    K.kda_attn_prefill(q, k, v, o, lse=lse)
    ref = attend64(q.double(), k.double(), v.double())
    # scores reach 4200: FP32 holds them to 2^-12
    half = torch.finfo(torch.bfloat16).eps / 2
    err = (o.double() - ref[0]).abs()
    assert bool((err <= half * ref[0].abs() + (half + 2.0 ** -9) * ref[2]).all())
    assert float((lse.double() - ref[1]).abs().max()) <= 4200 * 2.0 ** -22


def test_uniform_form_and_no_lse():
    K = kda()
    q, k, v = draw(9, [3 * 70], [3 * 90], 4, 2, torch.bfloat16)
    o = torch.empty_like(q)
    K.kda_attn_prefill(q.view(3, 70, 4, D), k.view(3, 90, 2, D), v.view(3, 90, 2, D),
                       o.view(3, 70, 4, D))
    for n in range(3):
        ref = attend64(q[n * 70:n * 70 + 70].double(), k[n * 90:n * 90 + 90].double(),
                       v[n * 90:n * 90 + 90].double())
        close(o[n * 70:n * 70 + 70], None, ref, torch.bfloat16)


def test_strided_views_and_untouched_neighbours():
    """q, k, v as slices of one projection, o into a wider buffer."""
    K = kda()
    T, H, Hk = 150, 6, 2
    g = torch.Generator().manual_seed(10)
    buf = torch.randn((T, (H + 2 * Hk) * D + 64), generator=g).to(torch.bfloat16).cuda()
    q = buf[:, :H * D].unflatten(1, (H, D))
    k = buf[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
    v = buf[:, (H + Hk) * D:(H + 2 * Hk) * D].unflatten(1, (Hk, D))
    wide = torch.full((T, H * D + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = wide[:, 8:8 + H * D].unflatten(1, (H, D)), torch.empty((T, H), device="cuda")
    K.kda_attn_prefill(q, k, v, o, lse=lse)
    check(q, k, v, o, lse, [T], [T], 0, torch.bfloat16)
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + H * D:] == 7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("heads", [4, 1])
def test_masked_places_have_no_influence(bad, what, heads):
    """A bad value at one key: rows that do not see it keep their bits, in its own sequence and in
    the others; rows that see it follow the formula."""
    K = kda()
    lens, at = [90, 150, 40], 90 + 77
    q, k, v = draw(11, lens, lens, heads, 1, torch.bfloat16)
    cu = offsets(lens)
    o1, l1, o2, l2 = (torch.empty(s, dtype=t, device="cuda") for s, t in
                      ((q.shape, q.dtype), (q.shape[:2], torch.float32)) * 2)
    K.kda_attn_prefill(q, k, v, o1, lse=l1, cu_seqlens=cu)
    x = k if what == "k" else v
    x[at, 0, 5] = bad
    K.kda_attn_prefill(q, k, v, o2, lse=l2, cu_seqlens=cu)
    sees = torch.zeros(sum(lens), dtype=torch.bool)
    sees[at:90 + 150] = True
    sees = sees.cuda()
    # the bits may differ by the path that met the value, never by more than the roundings
    check(q[~sees], k, v, o2[~sees], l2[~sees], [], [], 0, torch.bfloat16)
    same = (o1[~sees].double() - o2[~sees].double()).abs()
    assert bool((same <= 2.0 ** -7 * o1[~sees].double().abs() + 2.0 ** -7).all())
    assert bool(torch.isfinite(o2[~sees].float()).all()) and bool(torch.isfinite(l2[~sees]).all())
    got = o2[sees].float()
    if what == "v":
        assert bool((torch.isnan(got[..., 5]) if bad != bad else got[..., 5] == bad).all())
        other = torch.cat([got[..., :5], got[..., 6:]], -1)
        assert bool(torch.isfinite(other).all())
    elif bad != bad:
        assert bool(torch.isnan(got).all())


def test_window_hides_old_bad_values():
    K = kda()
    T, w = 400, 64
    q, k, v = draw(12, [T], [T], 4, 2, torch.bfloat16)
    v[100] = float("nan")
    k[101] = float("inf")
    o, lse = torch.empty_like(q), torch.empty((T, 4), device="cuda")
    K.kda_attn_prefill(q, k, v, o, lse=lse, window=w)
    clean = torch.ones(T, dtype=torch.bool)
    clean[100:101 + w] = False
    clean = clean.cuda()
    assert bool(torch.isfinite(o[clean].float()).all()) and bool(torch.isfinite(lse[clean]).all())
    tail = slice(101 + w, T)
    ref = attend64(q[tail].double(), k[102:].double(), v[102:].double(), w)
    close(o[tail], lse[tail], ref, torch.bfloat16)


def test_other_stream_and_graph_replay():
    K = kda()
    lens = [200, 31]
    q, k, v = draw(13, lens, lens, 8, 2, torch.bfloat16)
    cu = offsets(lens)
    ws = K.kda_attn_prefill_workspace(231, 2, 8, 2)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        K.kda_attn_prefill(q, k, v, o, lse=lse, cu_seqlens=cu, workspace=ws)
    side.synchronize()
    check(q, k, v, o, lse, lens, lens, 0, torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kda_attn_prefill(q, k, v, o, lse=lse, cu_seqlens=cu, workspace=ws)
    # other lengths through the same graph: offsets are read on the device
    lens = [30, 201]
    cu.copy_(offsets(lens))
    ws.fill_(0xAB)
    for seed in (14, 15):
        for x, y in zip((q, k, v), draw(seed, lens, lens, 8, 2, torch.bfloat16)):
            x.copy_(y)
        o.fill_(7.0)
        graph.replay()
        K.kda_sync_status()
        check(q, k, v, o, lse, lens, lens, 0, torch.bfloat16)


def test_repeats_give_the_same_bits():
    K = kda()
    lens = [700, 3, 1200]
    q, k, v = draw(16, lens, lens, 8, 2, torch.float16)
    outs = []
    for _ in range(3):
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        K.kda_attn_prefill(q, k, v, o, lse=lse, cu_seqlens=offsets(lens))
        outs.append((o, lse))
    assert all(torch.equal(a, b) for r in outs[1:] for a, b in zip(r, outs[0]))


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [0, 50, 60, 99], [1, 50, 60, 100],
                                [0, 50, 200, 100], [0, -5, 60, 100]])
def test_malformed_offsets_are_reported(cu):
    K = kda()
    q, k, v = draw(17, [100], [100], 4, 2, torch.bfloat16)
    guard = torch.full((140, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    K.kda_attn_prefill(q, k, v, guard[20:120], cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    with pytest.raises(K.KdaError, match="cu_seqlens"):
        K.kda_sync_status()
    assert bool((guard[:20] == 7).all()) and bool((guard[120:] == 7).all())
    K.kda_attn_prefill(q, k, v, guard[20:120])
    K.kda_sync_status()


def test_rows_past_32_bits():
    """Key rows whose element offsets pass 2^31 (and byte offsets 2^32)."""
    K = kda()
    T, wide = 70000, 32768
    big = torch.zeros((T, wide), dtype=torch.bfloat16, device="cuda")
    q, k, v = draw(18, [3], [T], 2, 1, torch.bfloat16)
    kk, vv = big[:, :D].unflatten(1, (1, D)), big[:, D:2 * D].unflatten(1, (1, D))
    kk.copy_(k)
    vv.copy_(v)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    K.kda_attn_prefill(q, kk, vv, o, lse=lse)
    check(q, k, v, o, lse, [3], [T], 0, torch.bfloat16)


def test_binding_refusals():
    K = kda()
    q, k, v = draw(19, [10], [10], 4, 2, torch.bfloat16)
    o = torch.empty_like(q)
    with pytest.raises(TypeError):
        K.kda_attn_prefill(q.float(), k, v, o)
    with pytest.raises(TypeError):
        K.kda_attn_prefill(q, k.half(), v, o)
    with pytest.raises(TypeError):
        K.kda_attn_prefill(q.cpu(), k, v, o)
    with pytest.raises(ValueError):
        K.kda_attn_prefill(q, k, v[:5], o)
    with pytest.raises(ValueError):
        K.kda_attn_prefill(q, k, v, o[:, :2])
    with pytest.raises(ValueError):
        K.kda_attn_prefill(q, k.transpose(0, 1), v.transpose(0, 1), o)
    with pytest.raises(K.KdaError):
        K.kda_attn_prefill(q, k, v, o, window=-1)
    with pytest.raises(K.KdaError):
        K.kda_attn_prefill(q, k, v, o, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lq,lk,heads,kv,window", [
    ([1], [4000], 8, 2, 0), ([16, 0, 3], [6000, 900, 2], 5, 1, 0), ([40, 7], [3000, 5000], 4, 4, 700),
    ([300], [2100], 16, 1, 0)])
def test_few_queries_behind_many_keys(lq, lk, heads, kv, window, dtype):
    """So few items that CTAs share an item's keys and a second kernel joins them."""
    run(lq, lk, heads, kv, dtype, window=window, seed=20)


def test_shared_items_and_hidden_bad_values():
    K = kda()
    q, k, v = draw(21, [6], [5000], 4, 2, torch.bfloat16)
    v[4997, 0, 3] = float("nan")      # seen by the last three rows
    v[100] = float("inf")             # by none, with the window
    k[101] = float("nan")
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    K.kda_attn_prefill(q, k, v, o, lse=lse, window=4000)
    k[101], v[100] = 0, 0
    ref = attend64(q.double(), k.double(), torch.nan_to_num(v).double(), 4000)
    seen = torch.zeros_like(o, dtype=torch.bool)
    seen[3:, :2, 3] = True
    assert bool(torch.isnan(o[seen]).all())
    o[seen] = ref[0][seen].to(o.dtype)
    close(o, lse, ref, torch.bfloat16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lq,lk,heads,kv,window", [
    (2048, 8300, 32, 8, 0), (2500, 10300, 16, 16, 0), (2040, 12500, 20, 4, 9000)])
def test_chunk_whose_last_items_share_their_keys(lq, lk, heads, kv, window, dtype):
    """More items than fill whole rounds: the keys of the last ones are cut.  A NaN among the
    values is seen by the rows from 40 on only."""
    K = kda()
    q, k, v = draw(22, [lq], [lk], heads, kv, dtype)
    v[lk - lq + 40, 0, 5] = float("nan")
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    K.kda_attn_prefill(q, k, v, o, lse=lse, window=window)
    K.kda_sync_status()
    group = heads // kv
    assert bool(torch.isfinite(o[:40]).all())
    assert bool(torch.isnan(o[40:, :group, 5]).all())
    o[40:, :group, 5] = 0
    assert bool(torch.isfinite(o).all())
    plain = torch.nan_to_num(v).double()
    for i in (0, 1, 39, 40, 63, 64, lq // 2, lq - 70, lq - 1):
        n = lk - lq + i + 1
        ref = attend64(q[i:i + 1].double(), k[:n].double(), plain[:n], window)
        if i >= 40:
            ref[0][:, :group, 5] = 0
        close(o[i:i + 1], lse[i:i + 1], ref, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lq,lk,heads,kv,window", [
    (2000, 2000, 32, 8, 0), (1100, 1500, 24, 24, 0), (1290, 1290, 32, 32, 300)])
def test_one_sequence_of_a_few_rounds(lq, lk, heads, kv, window, dtype):
    """More items than multiprocessors, of one sequence: no list of them is written."""
    K = kda()
    q, k, v = draw(23, [lq], [lk], heads, kv, dtype)
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    K.kda_attn_prefill(q, k, v, o, lse=lse, window=window)
    K.kda_sync_status()
    assert bool(torch.isfinite(o).all()) and not bool((lse == 7.0).any())
    for i in list(range(0, lq, 97)) + [lq - 1]:
        n = lk - lq + i + 1
        ref = attend64(q[i:i + 1].double(), k[:n].double(), v[:n].double(), window)
        close(o[i:i + 1], lse[i:i + 1], ref, dtype)
