"""Linear attention on addresses and strides that are multiples of 16 bytes and of no more."""

import pytest
import torch

from _lin import D, inputs
from _util import kda

pytestmark = pytest.mark.gpu


def moved(x):
    """x's values 16 bytes behind a larger power of two."""
    by = 16 // x.element_size()
    y = torch.empty(x.numel() + by, dtype=x.dtype, device="cuda")[by:].view(x.shape)
    assert y.data_ptr() % 32 == 16
    return y.copy_(x)


def apart(x):
    """Rows of heads with 16 bytes between them, 16 bytes behind a larger power of two."""
    rows, heads = x.shape[:2]
    y = torch.full((rows * (heads * D + 8) + 8,), float("nan"), dtype=x.dtype, device="cuda")
    y = y[8:].view(rows, heads * D + 8)[:, :heads * D].unflatten(1, (heads, D))
    return y.copy_(x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,heads,qk", [([5], 2, 2), ([50, 3], 4, 2), ([2000], 3, 3),
                                           ([19000], 1, 1), ([700 + 90 * i for i in range(6)], 30, 6),
                                           ([33, 100, 0, 500], 3, 1)])
def test_prompts(lens, heads, qk, dtype):
    K = kda()
    d = inputs(len(lens), sum(lens), heads, qk, dtype, n_seqs=len(lens))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    want, S = torch.empty_like(d["v"]), d["state"].clone()
    K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], want, S, S, cu_seqlens=cu)
    o, S2 = apart(torch.zeros_like(want)), moved(d["state"])
    ws = moved(K.kda_lin_prefill_workspace(sum(lens), len(lens), heads))
    K.kda_lin_prefill(apart(d["q"]), apart(d["k"]), apart(d["v"]), d["g"], o, S2, S2,
                      cu_seqlens=cu, workspace=ws)
    K.kda_sync_status()
    assert torch.equal(o, want) and torch.equal(S2, S)


@pytest.mark.parametrize("n,krows,heads", [(2, 3, 4), (9, 1, 20)])
def test_rows(n, krows, heads):
    K, dtype = kda(), torch.bfloat16
    d = inputs(n, n * krows, heads, heads, dtype, n_seqs=n)
    split = [d[x].unflatten(0, (n, krows)) for x in ("q", "k", "v", "g")]
    want, S = torch.empty_like(split[2]), torch.empty_like(d["state"])
    snaps = [torch.empty_like(S) for _ in range(krows)]
    K.kda_lin_decode(*split, want, d["state"], S, snaps)
    rows = [apart(d[x]).unflatten(0, (n, krows)) for x in ("q", "k", "v")]
    o = apart(torch.zeros_like(d["v"])).unflatten(0, (n, krows))
    S2, snaps2 = moved(d["state"]), [moved(torch.zeros_like(S)) for _ in range(krows)]
    K.kda_lin_decode(*rows, split[3], o, S2, S2, snaps2)
    K.kda_sync_status()
    assert torch.equal(o, want) and torch.equal(S2, S)
    assert all(torch.equal(a, b) for a, b in zip(snaps, snaps2))
