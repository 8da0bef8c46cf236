"""Linear attention with a decay for each head: kda_lin_prefill and kda_lin_decode against the
recurrence in 64 bits."""

import pytest
import torch

from _lin import D, SCALE, close, inputs, walk64
from _util import kda

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def cu_of(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()


def prefill(K, d, lens, **kw):
    o = torch.full_like(d["v"], float("nan"))
    S = torch.full((len(lens), d["v"].shape[1], D, D), float("nan"), device="cuda")
    K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], o, state_in=d["state"], state_out=S,
                      cu_seqlens=cu_of(lens), **kw)
    K.kda_sync_status()
    return o, S


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 7, 8, 9, 31, 32, 33, 127, 128, 129, 255, 256, 257, 640, 1000])
def test_one_sequence(T, dtype):
    K = kda()
    d = inputs(T, T, 2, 2, dtype)
    close(*prefill(K, d, [T]), d, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", [[1, 300, 0, 129, 5], [0, 0, 64], [200] * 9, [1] * 40, [1500, 3]])
@pytest.mark.parametrize("heads,qk", [(3, 3), (10, 2)])
def test_packed(lens, heads, qk, dtype):
    K = kda()
    d = inputs(7, sum(lens), heads, qk, dtype, n_seqs=len(lens))
    o, S = prefill(K, d, lens)
    at = 0
    for n, x in enumerate(lens):
        close(o, S, d, dtype, rows=(at, at + x), n=n)
        at += x


@pytest.mark.parametrize("T,heads,n", [(4096, 2, 1), (3000, 40, 1), (2500, 16, 3), (900, 200, 1),
                                       (700, 30, 12), (16384, 1, 1)])
def test_chains_shared_by_multiprocessors(T, heads, n):
    """Long sequences of few heads, and more chains than multiprocessors: some heads are checked."""
    K = kda()
    lens = [T - 37 * i for i in range(n)]
    d = inputs(T, sum(lens), heads, heads, torch.bfloat16, rate=0.3, n_seqs=n)
    o, S = prefill(K, d, lens)
    for i in {0, n - 1}:
        a = sum(lens[:i])
        for h in {0, heads // 2, heads - 1}:
            one = {x: d[x][:, h:h + 1] for x in ("q", "k", "v", "g")}
            one["state"] = d["state"][:, h:h + 1]
            close(o[:, h:h + 1], S[:, h:h + 1], one, torch.bfloat16, rows=(a, a + lens[i]), n=i)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,t_pad", [(5, 9), (150, 150), (130, 200)])
def test_padded_rows(t, t_pad, dtype):
    """Rows behind t hold NaN, are not read and not written."""
    K = kda()
    d = inputs(3, 2 * t_pad, 4, 4, dtype, n_seqs=2)
    v4 = {x: d[x].unflatten(0, (2, t_pad)) for x in ("q", "k", "v", "g")}
    for x in v4.values():
        x[:, t:] = float("nan")
    o = torch.full_like(v4["v"], 7.0)
    S = torch.empty_like(d["state"])
    K.kda_lin_prefill(v4["q"], v4["k"], v4["v"], v4["g"], o, state_in=d["state"], state_out=S, t=t)
    K.kda_sync_status()
    assert bool((o[:, t:] == 7.0).all())
    for n in range(2):
        one = {x: v4[x][n, :t] for x in v4}
        one["state"] = d["state"][n:n + 1]
        close(o[n, :t], S[n:n + 1], one, dtype)


def test_strided_rows_decay_for_each_head_state_in_place_no_state():
    K = kda()
    dtype, T, heads, qk = torch.bfloat16, 300, 6, 3
    d = inputs(11, T, heads, qk, dtype)
    wide = torch.randn((T, 2 * qk + 2 * heads + 1, D)).to(dtype).cuda()
    wide[:, :qk], wide[:, qk:2 * qk], wide[:, 2 * qk:2 * qk + heads] = d["q"], d["k"], d["v"]
    gates = torch.full((T, heads + 3), float("nan"), device="cuda")
    gates[:, :heads] = d["g"]
    out = wide[:, 2 * qk + heads:2 * qk + 2 * heads]
    S = d["state"].clone()
    K.kda_lin_prefill(wide[:, :qk], wide[:, qk:2 * qk], wide[:, 2 * qk:2 * qk + heads],
                      gates[:, :heads], out, state_in=S, state_out=S)
    close(out, S, d, dtype)
    d["g"], d["state"] = d["g"][5].clone(), None
    o = torch.empty_like(d["v"])
    K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], o, scale=2.5)
    close(o, None, d, dtype, scale=2.5)
    K.kda_sync_status()


@pytest.mark.parametrize("T", [4, 300])
def test_strong_and_infinite_decays(T):
    """Decays that leave nothing, -inf among them, between tokens that forget little."""
    K = kda()
    d = inputs(5, T, 3, 3, torch.bfloat16, rate=0.05)
    d["g"][::3, 0] = -float("inf")
    d["g"][1::7, 1] = -60.0
    d["g"][:, 2] = -3e38
    o, S = prefill(K, d, [T])
    d["g"] = d["g"].double().clamp_min(-1e4)
    close(o, S, d, torch.bfloat16)


@pytest.mark.parametrize("T", [6, 400])
@pytest.mark.parametrize("which", ["q", "k", "v", "g"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_tokens_before_one_that_is_not_finite(T, which, value):
    K = kda()
    at = T * 3 // 4
    d = inputs(9, T, 2, 2, torch.bfloat16)
    if which == "g":
        if value != value:
            d["g"][at, 1] = value
        else:
            return
    else:
        d[which][at, 1, 17] = value
    o, S = prefill(K, d, [T])
    clean = {x: y.clone() for x, y in d.items()}
    clean["q"][at:], clean["k"][at:], clean["v"][at:], clean["g"][at:] = 0, 0, 0, 0
    close(o, None, clean, torch.bfloat16, rows=(0, at))
    if which == "q":
        assert not bool(torch.isfinite(o[at, 1]).any())
        assert bool(torch.isfinite(o[at + 1:]).all()) and bool(torch.isfinite(S).all())
    elif which == "v":
        assert not bool(torch.isfinite(o[at:, 1, 17]).any())
        assert not bool(torch.isfinite(S[0, 1, :, 17]).any())
        assert bool(torch.isfinite(o[:, 1, :17]).all()) and bool(torch.isfinite(o[:, 1, 18:]).all())
    else:
        assert not bool(torch.isfinite(o[at, 1]).any())
    assert bool(torch.isfinite(o[:, 0]).all()) and bool(torch.isfinite(S[0, 0]).all())


@pytest.mark.parametrize("size", [2.0 ** -12, 1.0, 2.0 ** 10])
def test_fp16_values_small_and_large(size):
    """States and values near the ends of FP16's range keep their precision."""
    K = kda()
    d = inputs(13, 500, 2, 2, torch.float16, rate=0.01)
    d["v"] = (d["v"].float() * size).half()
    d["state"] = d["state"] * size * 16
    o, S = prefill(K, d, [500])
    ro, rs, _ = walk64(d["q"], d["k"], d["v"], d["g"], d["state"][0])
    assert float((S[0].double() - rs).norm() / rs.norm()) < 2.0 ** -17
    assert float((o.double() - ro).norm() / ro.norm()) < 2.0 ** -9


def test_results_repeat_and_offsets_are_checked():
    K = kda()
    lens = [700, 90, 1300]
    d = inputs(21, sum(lens), 8, 8, torch.bfloat16, n_seqs=3)
    o, S = prefill(K, d, lens)
    o2, S2 = prefill(K, d, lens)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    for bad in ([0, 700, 600, 2090], [0, 700, 790, 2091], [1, 700, 790, 2090]):
        o2, S2 = torch.full_like(o, 5.0), torch.full_like(S, 5.0)
        K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], o2, state_in=d["state"], state_out=S2,
                          cu_seqlens=torch.tensor(bad, dtype=torch.int32).cuda())
        with pytest.raises(K.KdaError) as e:
            K.kda_sync_status()
        assert e.value.status == 5 and "linear attention 0x1" in str(e.value)
    assert torch.equal(o2[700:790], o[700:790])      # the second sequence's offsets are sound
    assert torch.equal(S2[1], S[1])


def test_another_stream_and_a_captured_call():
    K = kda()
    d = inputs(31, 2000, 4, 4, torch.bfloat16)
    o, S = prefill(K, d, [2000])
    cu, ws = cu_of([2000]), K.kda_lin_prefill_workspace(2000, 1, 4)
    o2, S2 = torch.zeros_like(o), torch.zeros_like(S)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], o2, d["state"], S2, cu_seqlens=cu,
                          workspace=ws)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], o2, d["state"], S2, cu_seqlens=cu,
                          workspace=ws)
        K.kda_lin_decode(d["q"][:1], d["k"][:1], d["v"][:1], d["g"][:1], o2[:1], S2, S2)
    d["v"].copy_(d["v"].flip(0))
    ws.fill_(0xa5)
    want_o, want_S = prefill(K, d, [2000])
    K.kda_lin_decode(d["q"][:1], d["k"][:1], d["v"][:1], d["g"][:1], want_o[:1], want_S, want_S)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, want_o) and torch.equal(S2, want_S)


# ---------------------------------------------------------------- decode

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,krows,heads,qk", [(1, 1, 1, 1), (3, 4, 6, 2), (2, 8, 5, 5), (64, 1, 4, 4),
                                              (1, 3, 170, 34)])
def test_decode(n, krows, heads, qk, dtype):
    K = kda()
    d = inputs(n + krows, n * krows, heads, qk, dtype, n_seqs=n)
    split = {x: d[x].unflatten(0, (n, krows)) for x in ("q", "k", "v", "g")}
    o, S = torch.empty_like(split["v"]), torch.empty_like(d["state"])
    snaps = [torch.empty_like(S) for _ in range(krows)]
    K.kda_lin_decode(split["q"], split["k"], split["v"], split["g"], o, d["state"], S, snaps)
    K.kda_sync_status()
    assert torch.equal(snaps[-1], S)
    flat = o.flatten(0, 1)
    for i in range(n):
        close(flat, S, d, dtype, rows=(i * krows, (i + 1) * krows), n=i)
    # k calls of one row: the same bits; the state in place; fewer snapshots
    S1 = d["state"].clone()
    for t in range(krows):
        o1 = torch.empty((n, heads, D), dtype=dtype, device="cuda")
        K.kda_lin_decode(split["q"][:, t], split["k"][:, t], split["v"][:, t], split["g"][:, t], o1,
                         S1, S1)
        assert torch.equal(o1, o[:, t]) and torch.equal(S1, snaps[t])
    S2 = d["state"].clone()
    few = [torch.empty_like(S)] if krows > 1 else []
    K.kda_lin_decode(split["q"], split["k"], split["v"], split["g"], o, S2, S2, few, scale=SCALE)
    assert torch.equal(S2, S) and all(torch.equal(x, y) for x, y in zip(few, snaps))


def test_decode_goes_on_from_a_prompt():
    """A prompt of 300 tokens, then rows of 4 and 1: as one prompt of 305."""
    K = kda()
    d = inputs(41, 305, 4, 2, torch.bfloat16)
    S = d["state"].clone()
    o = torch.empty_like(d["v"])
    K.kda_lin_prefill(d["q"][:300], d["k"][:300], d["v"][:300], d["g"][:300], o[:300], S, S)
    for a, b in ((300, 304), (304, 305)):
        q, k, v, g, out = (x[a:b].unsqueeze(0) for x in (d["q"], d["k"], d["v"], d["g"], o))
        K.kda_lin_decode(q, k, v, g, out, S, S)
    close(o, S, d, torch.bfloat16)
