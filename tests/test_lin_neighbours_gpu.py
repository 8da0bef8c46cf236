"""kda_lin_prefill: what lies behind a sequence's last token, or in another sequence, reaches
nothing of its own."""

import pytest
import torch

from _lin import D, inputs
from _util import kda

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def cu_of(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()


def prefill(K, d, cu=None, t=None):
    o, S = torch.full_like(d["v"], 7.0), torch.full_like(d["state"], 7.0)
    K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], o, state_in=d["state"], state_out=S, t=t,
                      cu_seqlens=cu)
    return o, S


def same_bits(a, b):
    kind = torch.int16 if a.dtype != torch.float32 else torch.int32
    return torch.equal(a.view(kind), b.view(kind))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t", [100, 700])
@pytest.mark.parametrize("heads,qk", [(16, 1), (6, 6)])
def test_rows_behind_the_last_token_in_a_large_batch(heads, qk, t, dtype):
    """Value heads that share q and k, whose V therefore arrives last: NaN behind t, and zeros, give
    the same bits."""
    K, n, pad = kda(), 40, 28
    d = inputs(t, n * (t + pad), heads, qk, dtype, n_seqs=n)
    d = {x: y if x == "state" else y.unflatten(0, (n, t + pad)) for x, y in d.items()}
    runs = []
    for _ in range(4):
        for fill in (0.0, float("nan")):
            for x in ("q", "k", "v", "g"):
                d[x][:, t:] = fill
            runs.append(prefill(K, d, t=t))
    K.kda_sync_status()
    o, S = runs[0]
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(S).all())
    for o2, S2 in runs[1:]:
        assert same_bits(o, o2) and same_bits(S, S2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("other", [2.0 ** 13, float("inf"), float("nan")])
@pytest.mark.parametrize("most", [90, 900])
def test_sequences_beside_larger_values(most, other, dtype):
    """Every other sequence's values are 2^13 times as large, or not finite: the others have the
    bits that they have beside zeros."""
    K, n, heads = kda(), 120, 16
    gen = torch.Generator().manual_seed(most)
    lens = torch.randint(1, most, (n,), generator=gen).tolist()
    d = inputs(most, sum(lens), heads, 1, dtype, n_seqs=n)
    cu = cu_of(lens)
    rows = torch.cat([torch.full((x,), i % 2 == 1) for i, x in enumerate(lens)]).cuda()
    want = None
    for fill in (0.0, other, other, other):
        v = d["v"].clone()
        # (FP16's largest is 65504: 7 times 2^13 stays below)
        v[rows] = v[rows].clamp(-7, 7) * fill if fill != 0 else 0
        o, S = prefill(K, dict(d, v=v), cu)
        K.kda_sync_status()
        o, S = o[~rows], S[0::2]
        if want is None:
            want = o, S
            assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(S).all())
        assert same_bits(o, want[0]) and same_bits(S, want[1])


@pytest.mark.parametrize("lens,heads", [([100] * 60, 12), ([1, 128, 60] * 60, 5), ([520] * 40, 9),
                                        ([1900], 3)])
def test_values_that_are_not_finite_in_many_chunks(lens, heads):
    """Chunks with such values behind each other, every other one, and in sequences that one
    multiprocessor works on in turn: the columns that they are in are NaN from there on, and
    everything else has the bits that it has with zeros in their place."""
    K, dtype = kda(), torch.bfloat16
    d = inputs(heads, sum(lens), heads, heads, dtype, n_seqs=len(lens))
    gen = torch.Generator().manual_seed(heads)
    chunks = [(a, min(128, x - a), s) for s, x in zip(cu_of(lens).tolist(), lens)
              for a in range(0, x, 128)]
    v = d["v"].clone()
    first = torch.full((len(lens), heads, D), 1 << 30)         # the first such row of a column
    starts = cu_of(lens).tolist()
    for i, (a, count, s) in enumerate(chunks):
        for h in range(heads):
            # heads of which no chunk, each, every other one, or some hold one
            if not (h % 4 == 1 or h % 4 == 2 and i % 2 or
                    h % 4 == 3 and torch.rand((), generator=gen) < 0.5):
                continue
            r = s + a + int(torch.randint(0, count, (), generator=gen))
            col = int(torch.randint(0, D, (), generator=gen))
            v[r, h, col] = (float("nan"), float("inf"), -float("inf"))[(i + h) % 3]
            n = starts.index(s)
            first[n, h, col] = min(int(first[n, h, col]), r)
    cu = cu_of(lens)
    want, S_want = prefill(K, dict(d, v=torch.where(torch.isfinite(v), v, 0)), cu)
    K.kda_sync_status()
    row = torch.arange(sum(lens))
    n_of = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
    bad = (row[:, None, None] >= first[n_of]).cuda()
    bad_S = (first < 1 << 30).cuda()[:, :, None, :].expand(-1, -1, D, -1)
    for _ in range(5):
        o, S = prefill(K, dict(d, v=v), cu)
        K.kda_sync_status()
        assert not bool(torch.isfinite(o[bad]).any()) and same_bits(o[~bad], want[~bad])
        assert not bool(torch.isfinite(S[bad_S]).any()) and same_bits(S[~bad_S], S_want[~bad_S])
