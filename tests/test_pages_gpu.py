"""The pages of the 4-bit cache: resize, fork, compact and copy against the same on the host."""

import pytest
import torch

import _pages
from _util import kda

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


SIZES = [(1, 1, 1, 16, 1.0), (1, 3, 5, 16, 0.5), (4, 6, 40, 16, 0.6), (33, 7, 200, 32, 0.8),
         (300, 20, 5000, 64, 0.9), (5, 900, 30001, 128, 0.2), (1500, 3, 4097, 256, 0.7)]


def finish(K, enough):
    if enough:
        K.kda_sync_status()
        return
    with pytest.raises(K.KdaError) as e:
        K.kda_sync_status()
    assert e.value.status == 5 and "no free pages" in str(e.value)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("seed", range(3))
def test_resize(size, seed):
    K = kda()
    n, width, pages, page, fill = size
    table, lens, refs, r = _pages.some_state(seed, *size)
    lens = [min(width * page, max(0, x + r.choice([0, 1, -page, 3 * page, -x]))) for x in lens]
    t, f = ints(table), ints(refs)
    K.kda_attn_kv4_resize(t, ints(lens), f, page=page)
    enough = _pages.resize(table, lens, refs, page)
    assert t.tolist() == table and f.tolist() == refs
    finish(K, enough)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(size, seed, in_place):
    K = kda()
    n, width, pages, page, fill = size
    table, lens, refs, r = _pages.some_state(seed, *size)
    parent = [r.choice([-1, i, r.randrange(n), r.randrange(min(n, 3))]) for i in range(n)]
    t, l, f = ints(table), ints(lens), ints(refs)
    outs = dict(page_table_out=torch.empty_like(t), lens_out=torch.empty_like(l),
                refs_out=torch.empty_like(f))
    src, dst, count = K.kda_attn_kv4_fork(t, l, f, ints(parent), page=page,
                                          **({} if in_place else outs))
    if in_place:
        outs = dict(page_table_out=t, lens_out=l, refs_out=f)
    else:
        assert t.tolist() == table and l.tolist() == lens and f.tolist() == refs
    table, lens, pairs, enough = _pages.fork(table, lens, refs, parent, page)
    assert outs["page_table_out"].tolist() == table and outs["lens_out"].tolist() == lens
    assert outs["refs_out"].tolist() == refs
    k = len(pairs)
    assert count.tolist() == [k]
    assert list(zip(src.tolist(), dst.tolist())) == pairs + [(-1, -1)] * (n - k)
    finish(K, enough)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(size, seed, in_place):
    K = kda()
    table, lens, refs, r = _pages.some_state(seed, *size)
    t, f = ints(table), ints(refs)
    outs = {} if in_place else dict(page_table_out=torch.empty_like(t),
                                    refs_out=torch.empty_like(f))
    src, dst, count = K.kda_attn_kv4_compact(t, f, **outs)
    table, pairs = _pages.compact(table, refs)
    assert outs.get("page_table_out", t).tolist() == table
    assert outs.get("refs_out", f).tolist() == refs
    k = len(pairs)
    assert count.tolist() == [k]
    assert list(zip(src.tolist(), dst.tolist())) == pairs + [(-1, -1)] * (src.numel() - k)
    K.kda_sync_status()


@pytest.mark.parametrize("n_pages,kv,page,caches,pairs", [(5, 1, 16, 1, 2), (40, 3, 64, 3, 17),
                                                          (300, 8, 128, 2, 140), (9, 5, 256, 128, 4)])
def test_copy(n_pages, kv, page, caches, pairs):
    K = kda()
    all_ = [torch.randint(0, 256, (n_pages, kv, page * 144), dtype=torch.uint8, device="cuda")
            for _ in range(caches)]
    want = [c.clone() for c in all_]
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1))
    src, dst = order[:pairs].int().cuda(), order[pairs:2 * pairs].int().cuda()
    for c in want:
        c[dst[:pairs - 1].long()] = c[src[:pairs - 1].long()]
    K.kda_attn_kv4_copy(all_, src, dst, ints([pairs - 1]))
    K.kda_sync_status()
    assert all(torch.equal(x, y) for x, y in zip(all_, want))
    K.kda_attn_kv4_copy(all_[0], src, dst, ints([0]))
    K.kda_attn_kv4_copy(all_[0], src[:0], dst[:0], ints([0]))
    K.kda_sync_status()
    # numbers that are no pages are left out, and more than the list holds
    src[0] = -1
    if pairs > 1:
        src[1] = n_pages
    K.kda_attn_kv4_copy(all_[0], src, dst, ints([1 << 30]))
    want[0][dst[2:].long()] = want[0][src[2:].long()]
    with pytest.raises(K.KdaError):
        K.kda_sync_status()
    assert torch.equal(all_[0], want[0])


def test_entries_lens_and_parents_out_of_range():
    K = kda()
    t, f = ints([[7, 99, -1], [2, -5, -1]]), ints([0, 0, 1, 0, 0, 0, 0, 1, 0, 0])
    K.kda_attn_kv4_resize(t, ints([400, -3]), f, page=16)
    assert t.tolist() == [[7, 0, 1], [-1, -1, -1]]
    assert f.tolist() == [1, 1, 0, 0, 0, 0, 0, 1, 0, 0]
    with pytest.raises(K.KdaError):
        K.kda_sync_status()
    t, f, l = ints([[7, 99, -1], [2, -1, -1]]), ints([0, 0, 1, 0, 0, 0, 0, 1, 0, 0]), ints([20, 9])
    K.kda_attn_kv4_fork(t, l, f, ints([5, -7]), page=16)
    assert t.tolist() == [[-1] * 3] * 2 and f.sum().item() == 0 and l.tolist() == [0, 0]
    with pytest.raises(K.KdaError):
        K.kda_sync_status()
    # pages that the table names and the counts call free
    t, f = ints([[7, 0, -1]]), ints([0, 0, 1, 0, 0, 0, 0, 0, 0, 1])
    src, dst, count = K.kda_attn_kv4_compact(t, f)
    assert t.tolist() == [[-1, -1, -1]] and f.tolist() == [1, 1] + [0] * 8
    assert count.item() == 2 and src.tolist()[:2] == [2, 9] and dst.tolist()[:2] == [0, 1]
    with pytest.raises(K.KdaError):
        K.kda_sync_status()


def test_a_beam_search_over_the_cache():
    """Rows grow, fork and end, the pages are compacted: what the decode sees of each row stays
    what was appended to it."""
    K = kda()
    kv, page, rows, pages = 2, 16, 6, 64
    cache = K.kv4_cache(pages, kv, page)
    table, refs = torch.full((rows, 8), -1, dtype=torch.int32).cuda(), ints([0] * pages)
    lens = ints([0] * rows)
    history = [[] for _ in range(rows)]
    gen, r = torch.Generator().manual_seed(5), __import__("random").Random(5)
    ws = K.kda_attn_kv4_pages_workspace(pages, rows, 8)

    def grow(count):
        nonlocal lens
        lens = lens + count
        K.kda_attn_kv4_resize(table, lens, refs, page=page, workspace=ws)
        x = torch.randn((rows * count, kv, 128), generator=gen).to(torch.bfloat16).cuda()
        K.kda_attn_kv4_append(x, -x, cache, table, lens)
        for n in range(rows):
            history[n] = history[n] + list(x[n * count:(n + 1) * count])

    def look():
        cu = torch.tensor([0] + [len(h) for h in history]).cumsum(0).to(torch.int32).cuda()
        k = torch.empty((int(cu[-1]), kv, 128), dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        K.kda_attn_kv4_read(k, v, cache, table, lens, cu_seqlens=cu)
        K.kda_sync_status()
        want = torch.stack([x for h in history for x in h])
        # half of a step of (max - min) / 15, which is below 0.45, and the BF16 roundings
        assert float((k - want).abs().max()) < 0.25 and float((v + want).abs().max()) < 0.25
        assert refs.tolist() == torch.bincount(table[table >= 0].long(), minlength=pages).tolist()

    grow(37)
    for step in range(12):
        parent = [r.randrange(rows) for _ in range(rows)]
        src, dst, count = K.kda_attn_kv4_fork(table, lens, refs, ints(parent), page=page,
                                              workspace=ws)
        K.kda_attn_kv4_copy(cache, src, dst, count)
        history = [list(history[p]) for p in parent]
        grow(1 + step % 3)
        if step % 4 == 3:
            src, dst, count = K.kda_attn_kv4_compact(table, refs, workspace=ws)
            K.kda_attn_kv4_copy(cache, src, dst, count)
            assert int(table.max()) + 1 == int((refs > 0).sum())
        look()
    # rejected rows are taken back; ended rows give everything back
    lens = (lens - 20).clamp_min(0)
    K.kda_attn_kv4_resize(table, lens, refs, page=page, workspace=ws)
    history = [h[:int(n)] for h, n in zip(history, lens)]
    look()
    lens.zero_()
    K.kda_attn_kv4_resize(table, lens, refs, page=page, workspace=ws)
    assert int(refs.abs().sum()) == 0 and int(table.max()) == -1


def test_captured_calls():
    K = kda()
    table, lens, refs, r = _pages.some_state(1, 33, 7, 300, 32, 0.6)
    parent = [r.randrange(33) for _ in range(33)]
    t, l, f, p = ints(table), ints(lens), ints(refs), ints(parent)
    ws = K.kda_attn_kv4_pages_workspace(300, 33, 7)
    src, dst, count = (torch.zeros(x, dtype=torch.int32, device="cuda") for x in (33, 33, 1))
    cache = torch.randint(0, 256, (300, 2, 32 * 144), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kda_attn_kv4_fork(t, l, f, p, src=src, dst=dst, count=count, page=32, workspace=ws)
        K.kda_attn_kv4_copy(cache, src, dst, count)
        K.kda_attn_kv4_resize(t, l, f, page=32, workspace=ws)
    want = cache.clone()
    for _ in range(3):
        graph.replay()
        table, lens, pairs, enough = _pages.fork(table, lens, refs, parent, 32)
        assert enough
        _pages.resize(table, lens, refs, 32)
        for s, d in pairs:
            want[d] = want[s]
        torch.cuda.synchronize()
        assert t.tolist() == table and l.tolist() == lens and f.tolist() == refs
        assert torch.equal(cache, want)
    K.kda_sync_status()
