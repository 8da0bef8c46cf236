"""The serving example's operators in one run: linear layers, rotary rows, attention over pages that
are given, shared, copied, gathered and freed, each step against its 64-bit form."""

import pytest
import torch

import _pages
from _attn import attend64, close as attend_close
from _lin import D, close as lin_close
from _util import kda
from test_hybrid_example_gpu import example, stored
from test_pages_gpu import ints
from test_rope_gpu import near, rope64

pytestmark = pytest.mark.gpu


class Recorder:
    """The package, with the calls named kept: inputs before and outputs after."""

    def __init__(self, package, names):
        self.package, self.names, self.calls = package, names, []

    def __getattr__(self, name):
        call = getattr(self.package, name)
        if name not in self.names:
            return call

        def recorded(*args, **kw):
            def copies():
                return [a.clone() if isinstance(a, torch.Tensor)
                        else [x.clone() for x in a] if isinstance(a, list) else a for a in args]
            before = copies()
            call(*args, **kw)
            self.calls.append((name, before, copies(), kw))
        return recorded


def check_rope(before, after):
    q, k, pos, inv = before
    axis = [0] * inv.numel()
    for x, y in ((q, after[0]), (k, after[1])):
        near(y, x, rope64(x, pos[:, None], inv, axis, False, 1.0), inv.numel(), False, 1.0)


def check_lin(name, before, after, kw):
    q, k, v, g, _, state = before[:6]
    o, S = after[4:6]
    if name == "kda_lin_prefill":
        cu = kw["cu_seqlens"].tolist()
        for n in range(len(cu) - 1):
            lin_close(o, S, dict(q=q, k=k, v=v, g=g, state=state), o.dtype, (cu[n], cu[n + 1]), n)
        return
    for n in range(q.shape[0]):
        d = dict(q=q[n], k=k[n], v=v[n], g=g, state=state[n:n + 1])
        lin_close(o[n], S[n:n + 1], d, o.dtype)
        last = after[7][-1][n]
        assert torch.equal(last, S[n])


def test_a_run(monkeypatch):
    """Four sequences: two prompt chunks, rows of which some stay, samples of one prompt, pages
    gathered, rows again, a sequence that ends."""
    mod, trace = example(), []
    record = Recorder(kda(), ("kda_lin_prefill", "kda_lin_decode", "kda_attn_rope"))
    monkeypatch.setattr(mod, "K", record)
    m = mod.Model(dim=256, heads=4, kv_heads=2, n_seqs=4, krows=4, longest=192, page=32,
                  trace=trace)
    gen = torch.Generator().manual_seed(1)

    def draw(rows):
        return torch.randn((rows, 256), generator=gen).to(torch.bfloat16).cuda()

    keys = [[] for _ in range(4)]              # each sequence's rows of (k, v), as they were given

    def take(new):
        """Looks at the last attention step and adds its rows."""
        q, k, v, o, lens = trace[-1]
        first, at = not any(keys), 0
        prompt = len(set(new)) > 1 or new[0] > 4
        for n, r in enumerate(new):
            part = slice(at, at + r)
            at += r
            keys[n] += list(zip(k[part].cpu(), v[part].cpu()))
            assert int(lens[n]) == len(keys[n])
            kc, vc = (torch.stack([x[i] for x in keys[n]]) for i in (0, 1))
            if first:
                kk, vv, moved = kc.double(), vc.double(), None
            else:
                kk, (vv, moved) = stored(kc)[0], stored(vc)
            if prompt and not first:           # read rounds the cache's values
                kk, vv = (x.to(torch.bfloat16).double() for x in (kk, vv))
                moved = None
            ref = attend64(q[part].cpu().double(), kk, vv, moved=moved)
            attend_close(o[part].cpu(), None, ref, torch.bfloat16)

    def pages():
        """Counts, and pages for exactly the positions there are."""
        refs = [0] * m.attn.refs.numel()
        for n, row in enumerate(m.attn.table.tolist()):
            held = -(-len(keys[n]) // 32)
            assert all(v >= 0 for v in row[:held]) and all(v == -1 for v in row[held:])
            for v in row[:held]:
                refs[v] += 1
        assert m.attn.refs.tolist() == refs
        return refs

    for new in ([70, 1, 33, 20], [5, 40, 64, 30]):
        m.chunk(draw(sum(new)), new)
        take(new)
        pages()
    m.rows(draw(16))
    take([4] * 4)
    kept = [2, 4, 1, 3]
    m.keep(kept, 4)
    for n, x in enumerate(kept):
        del keys[n][len(keys[n]) - 4 + x:]
    pages()
    parent = [0, 2, 2, 2]
    states = m.lin.state.clone()
    m.fork(parent)
    keys = [list(keys[p]) for p in parent]
    assert torch.equal(m.lin.state, states[parent])
    before = pages()
    assert max(before) > 1                     # pages are shared
    m.compact()
    after = pages()
    used = sum(x > 0 for x in before)
    assert sorted(after) == sorted(before) and all(x > 0 for x in after[:used])
    m.rows(draw(16))
    take([4] * 4)
    m.keep([4, 3, 2, 1], 4)
    for n, x in enumerate([4, 3, 2, 1]):
        del keys[n][len(keys[n]) - 4 + x:]
    m.fork([-1, 1, 2, 3])
    keys[0] = []
    assert not bool(m.lin.state[0].any()) and m.lens.tolist() == m.positions
    pages()
    m.rows(draw(16))
    take([4] * 4)
    pages()
    kda().kda_sync_status()
    names = [c[0] for c in record.calls]
    assert names.count("kda_lin_prefill") == 2 and names.count("kda_lin_decode") == 3
    for name, before, after, kw in record.calls:
        if name == "kda_attn_rope":
            check_rope(before, after)
        else:
            check_lin(name, before, after, kw)


def test_many_rows_fork():
    """More rows than shared memory holds of them."""
    K = kda()
    size = (13001, 2, 20000, 16, 0.8)
    table, lens, refs, r = _pages.some_state(5, *size)
    parent = [r.choice([-1, i, r.randrange(13001), r.randrange(3)]) for i in range(13001)]
    t, l, f = ints(table), ints(lens), ints(refs)
    src, dst, count = K.kda_attn_kv4_fork(t, l, f, ints(parent), page=16)
    table, lens, pairs, enough = _pages.fork(table, lens, refs, parent, 16)
    assert t.tolist() == table and l.tolist() == lens and f.tolist() == refs
    k = len(pairs)
    assert count.tolist() == [k] and list(zip(src.tolist(), dst.tolist()))[:k] == pairs
    if enough:
        K.kda_sync_status()
    else:
        with pytest.raises(K.KdaError):
            K.kda_sync_status()


def test_two_captured_calls_of_linear_attention_on_one_workspace():
    """Two graphs, one workspace, replayed in turn: each with the bits of its eager call."""
    K = kda()
    gen = torch.Generator().manual_seed(2)
    runs = []
    ws = K.kda_lin_prefill_workspace(1400, 3, 4)
    for lens in ([700, 300, 400], [1, 1300, 99]):
        rows = sum(lens)
        q, k = (torch.nn.functional.normalize(torch.randn((rows, 4, D), generator=gen), dim=-1)
                .to(torch.bfloat16).cuda() for _ in range(2))
        v = torch.randn((rows, 4, D), generator=gen).to(torch.bfloat16).cuda()
        g = -torch.rand((rows, 4), generator=gen).cuda()
        S = torch.randn((3, 4, D, D), generator=gen).cuda()
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
        want, Sw = torch.empty_like(v), torch.empty_like(S)
        K.kda_lin_prefill(q, k, v, g, want, S, Sw, cu_seqlens=cu)
        o, So = torch.empty_like(v), torch.empty_like(S)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            K.kda_lin_prefill(q, k, v, g, o, S, So, cu_seqlens=cu, workspace=ws)
        runs.append((graph, o, So, want, Sw, (q, k, v, g, S, cu)))
    for _ in range(3):
        for graph, *_ in runs:
            graph.replay()
    K.kda_sync_status()
    for _, o, So, want, Sw, _ in runs:
        assert torch.equal(o, want) and torch.equal(So, Sw)


def test_arguments_are_refused():
    K = kda()
    q = torch.zeros((4, 2, D), dtype=torch.bfloat16).cuda()
    v, g = torch.zeros((4, 4, D), dtype=torch.bfloat16).cuda(), torch.zeros((4, 4)).cuda()
    o, S = torch.empty_like(v), torch.zeros((1, 4, D, D)).cuda()
    cu = torch.tensor([0, 4], dtype=torch.int32).cuda()
    for wrong in (dict(v=v[:3]), dict(k=q[:, :1]), dict(out=o[:, :3]), dict(g=g[:, :2]),
                  dict(state_in=S[:, :2]), dict(state_out=S.expand(2, -1, -1, -1)),
                  dict(t=3, cu_seqlens=cu), dict(workspace=torch.empty(64, device="cpu"))):
        args = dict(q=q, k=q, v=v, g=g, out=o, state_in=S, state_out=S)
        args.update(wrong)
        with pytest.raises(ValueError):
            K.kda_lin_prefill(**args)
    for wrong in (dict(q=q.float()), dict(g=g.half()), dict(v=v.half()), dict(q=q.cpu()),
                  dict(state_in=S.half())):
        args = dict(q=q, k=q, v=v, g=g, out=o, state_in=S, state_out=S)
        args.update(wrong)
        with pytest.raises((TypeError, ValueError)):
            K.kda_lin_prefill(**args)
        with pytest.raises((TypeError, ValueError)):
            K.kda_lin_decode(**args)
    with pytest.raises(K.KdaError):            # a workspace that is too small
        K.kda_lin_prefill(q, q, v, g, o, S, S,
                          workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(K.KdaError):            # nine tokens
        x = torch.zeros((1, 9, 4, D), dtype=torch.bfloat16).cuda()
        K.kda_lin_decode(x, x, x, torch.zeros(4).cuda(), torch.empty_like(x), S, S)
    table, lens, refs = ints([[0, -1]]), ints([3]), ints([1, 0, 0])
    for call in (lambda: K.kda_attn_kv4_resize(table[0], lens, refs),
                 lambda: K.kda_attn_kv4_resize(table, ints([1, 2]), refs),
                 lambda: K.kda_attn_kv4_fork(table, lens, refs, ints([0, 0])),
                 lambda: K.kda_attn_kv4_fork(table, lens, refs, lens, src=ints([0, 0])),
                 lambda: K.kda_attn_kv4_compact(table, refs, dst=ints([0, 0])),
                 lambda: K.kda_attn_kv4_copy([], lens, lens, lens),
                 lambda: K.kda_attn_kv4_copy(torch.empty((3, 2, 145), dtype=torch.uint8).cuda(),
                                             lens, lens, lens)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises((TypeError, ValueError)):
        K.kda_attn_kv4_resize(table.long(), lens, refs)
    with pytest.raises((TypeError, ValueError)):
        K.kda_attn_kv4_resize(table.cpu(), lens, refs)
    with pytest.raises(K.KdaError):            # a page length that there is none of
        K.kda_attn_kv4_resize(table, lens, refs, page=48)
    K.kda_sync_status()


def test_the_example_runs(capsys):
    example().main()
    assert "a step" in capsys.readouterr().out
