"""kda_lin_prefill where heads of sequences are cut between multiprocessors: few long ones, many
ragged ones, each way the pieces are joined, states in place, no offsets."""

import pytest
import torch

from _lin import D, close, inputs
from _util import kda

pytestmark = pytest.mark.gpu


def cu_of(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()


# sequences' lengths, heads: pieces of their own (the state folded from a few, from 22 by a
# kernel of its own), equal pieces (folded; from more than ten), handed over between two,
# pieces as long as the longest
CASES = [([2000], 3), ([17000], 1), ([3000], 40), ([20000], 8), ([900] * 2, 110),
         ([100 + 170 * i for i in range(12)], 30), ([5, 1, 0, 64, 3000] + [200] * 30, 9),
         ([130] * 300, 2), ([2000, 900, 1500, 1900], 34), ([900, 100, 0, 1100, 700], 11)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,heads", CASES)
def test_cut_chains(lens, heads, dtype):
    K = kda()
    d = inputs(len(lens) + heads, sum(lens), heads, heads, dtype, rate=0.3, n_seqs=len(lens))
    o, S = torch.empty_like(d["v"]), torch.empty_like(d["state"])
    call = (d["q"], d["k"], d["v"], d["g"])
    K.kda_lin_prefill(*call, o, d["state"], S, cu_seqlens=cu_of(lens))
    K.kda_sync_status()
    longest = max(range(len(lens)), key=lambda n: lens[n])
    for n in {0, longest, len(lens) - 1}:
        a = sum(lens[:n])
        for h in {0, heads // 2, heads - 1}:
            one = {x: d[x][:, h:h + 1] for x in ("q", "k", "v", "g")}
            one["state"] = d["state"][:, h:h + 1]
            close(o[:, h:h + 1], S[:, h:h + 1], one, dtype, rows=(a, a + lens[n]), n=n)
    # the states in place: the same bits, whoever writes first; and again
    for _ in range(2):
        S2, o2 = d["state"].clone(), torch.empty_like(o)
        K.kda_lin_prefill(*call, o2, S2, S2, cu_seqlens=cu_of(lens))
        K.kda_sync_status()
        assert torch.equal(o, o2) and torch.equal(S, S2)
    # no states: as states of zero
    zero, S3, o3 = torch.zeros_like(S), torch.empty_like(S), torch.empty_like(o)
    K.kda_lin_prefill(*call, o2, zero, S2, cu_seqlens=cu_of(lens))
    K.kda_lin_prefill(*call, o3, None, S3, cu_seqlens=cu_of(lens))
    K.kda_sync_status()
    assert torch.equal(o2, o3) and torch.equal(S2, S3)


@pytest.mark.parametrize("n,T,heads", [(1, 5000, 7), (3, 1000, 100), (5, 2000, 64), (40, 9, 16),
                                       (4, 2000, 32), (2, 900, 12), (1, 1300, 30)])
def test_without_offsets(n, T, heads):
    """Sequences of one length, with offsets and without: the same bits."""
    K = kda()
    d = inputs(n, n * T, heads, heads, torch.bfloat16, n_seqs=n)
    o, S = torch.empty_like(d["v"]), torch.empty_like(d["state"])
    K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], o, d["state"], S, cu_seqlens=cu_of([T] * n))
    q, k, v, g = (d[x].unflatten(0, (n, T)) for x in ("q", "k", "v", "g"))
    o2, S2 = torch.empty_like(v), d["state"].clone()
    K.kda_lin_prefill(q, k, v, g, o2, S2, S2)
    K.kda_sync_status()
    assert torch.equal(o2.flatten(0, 1), o) and torch.equal(S, S2)


def test_captured_hand_over():
    """Calls whose multiprocessors hand states on, in a graph, one behind the other on one
    workspace."""
    K = kda()
    lens, heads = [700 + 90 * i for i in range(10)], 40
    d = inputs(3, sum(lens), heads, 8, torch.bfloat16, n_seqs=10)
    cu, ws = cu_of(lens), K.kda_lin_prefill_workspace(sum(lens), 10, heads)
    want, S1 = torch.empty_like(d["v"]), d["state"].clone()
    for _ in range(2):
        K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], want, S1, S1, cu_seqlens=cu)
    o, S2 = torch.empty_like(want), d["state"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], o, S2, S2, cu_seqlens=cu,
                              workspace=ws)
    ws.fill_(0x77)
    graph.replay()
    K.kda_sync_status()
    assert torch.equal(o, want) and torch.equal(S1, S2)
    S2.copy_(d["state"])
    graph.replay()
    K.kda_sync_status()
    assert torch.equal(o, want) and torch.equal(S1, S2)


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace, one kind cut and summed up, one
    handed over: the bits of calls one at a time."""
    K = kda()
    runs = []
    for seed, (lens, heads) in enumerate([([700 + 90 * i for i in range(10)], 40), ([6000], 20)]):
        d = inputs(seed, sum(lens), heads, heads, torch.bfloat16, n_seqs=len(lens))
        cu, ws = cu_of(lens), K.kda_lin_prefill_workspace(sum(lens), len(lens), heads)
        call = (d["q"], d["k"], d["v"], d["g"])
        want, S = torch.empty_like(d["v"]), torch.empty_like(d["state"])
        K.kda_lin_prefill(*call, want, d["state"], S, cu_seqlens=cu)
        outs = [(torch.empty_like(want), torch.empty_like(S)) for _ in range(6)]
        runs.append((torch.cuda.Stream(), call, d["state"], cu, ws, want, S, outs))
    torch.cuda.synchronize()
    for i in range(6):
        for stream, call, state, cu, ws, _, _, outs in runs:
            with torch.cuda.stream(stream):
                K.kda_lin_prefill(*call, outs[i][0], state, outs[i][1], cu_seqlens=cu,
                                  workspace=ws)
    torch.cuda.synchronize()
    K.kda_sync_status()
    for *_, want, S, outs in runs:
        for o, So in outs:
            assert torch.equal(o, want) and torch.equal(So, S)


@pytest.mark.parametrize("n,heads", [(33, 3), (1025, 2), (5000, 1)])
def test_many_sequences(n, heads):
    """Ragged ones, a third of them empty, a long one among them."""
    K = kda()
    gen = torch.Generator().manual_seed(n)
    lens = (torch.randint(0, 60, (n,), generator=gen) * (torch.rand(n, generator=gen) > 0.3)).tolist()
    lens[n // 2] = 2500
    d = inputs(n, sum(lens), heads, heads, torch.bfloat16, rate=0.3, n_seqs=n)
    o, S = torch.empty_like(d["v"]), torch.empty_like(d["state"])
    call = (d["q"], d["k"], d["v"], d["g"])
    K.kda_lin_prefill(*call, o, d["state"], S, cu_seqlens=cu_of(lens))
    K.kda_sync_status()
    starts = [0]
    for x in lens:
        starts.append(starts[-1] + x)
    look = set(range(0, n, max(1, n // 40))) | {n // 2 - 1, n // 2, n // 2 + 1, n - 1}
    for i in look:
        one = {x: d[x][:, :1] for x in ("q", "k", "v", "g")}
        one["state"] = d["state"][:, :1]
        close(o[:, :1], S[:, :1], one, torch.bfloat16, rows=(starts[i], starts[i + 1]), n=i)
    empty = torch.tensor([x == 0 for x in lens]).cuda()
    assert torch.equal(S[empty], d["state"][empty])
    # each sequence is as it is alone, whichever CTA has it: in place too
    S2, o2 = d["state"].clone(), torch.empty_like(o)
    K.kda_lin_prefill(*call, o2, S2, S2, cu_seqlens=cu_of(lens))
    K.kda_sync_status()
    assert torch.equal(o, o2) and torch.equal(S, S2)
