"""kda_lin_prefill with tokens that are not finite, in heads that one multiprocessor has, that are
cut and summed up, and that are handed over."""

import pytest
import torch

from _lin import D, close, inputs
from _util import kda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("which,value", [(w, x) for w in "qkv" for x in (float("nan"), float("inf"))]
                         + [("g", float("nan"))])
@pytest.mark.parametrize("lens,heads", [([400], 2), ([2600], 2), ([17000], 1), ([1000] * 5, 40),
                                        ([300, 1, 1500, 40], 16)])
def test_a_token_that_is_not_finite(lens, heads, which, value, dtype):
    K = kda()
    d = inputs(len(lens), sum(lens), heads, heads, dtype, rate=0.3, n_seqs=len(lens))
    n, h = max(range(len(lens)), key=lambda i: lens[i]), heads - 1
    start = sum(lens[:n])
    stop, at = start + lens[n], start + lens[n] * 2 // 5
    if which == "g":
        d["g"][at, h] = value
    else:
        d[which][at, h, 17] = value
    o, S = torch.full_like(d["v"], 7.0), torch.empty_like(d["state"])
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], o, d["state"], S, cu_seqlens=cu)
    K.kda_sync_status()

    def one(h, lo=0, hi=D):
        """A head; v's columns [lo, hi) of it, the others zeros."""
        x = {y: d[y][:, h:h + 1].clone() for y in ("q", "k", "v", "g")}
        x["state"] = d["state"][:, h:h + 1].clone()
        x["v"][..., :lo], x["v"][..., hi:] = 0, 0
        x["state"][..., :lo], x["state"][..., hi:] = 0, 0
        return x

    short = lens[n] <= 3000                    # (the walks in 64 bits take their time)
    # the tokens before it
    assert bool(torch.isfinite(o[start:at, h]).all())
    if short:
        close(o[:, h:h + 1], None, one(h), dtype, rows=(start, at), n=n)
    here, rest = o[at, h], o[at + 1:stop, h]
    if which == "q":
        assert not bool(torch.isfinite(here).any()) and bool(torch.isfinite(rest).all())
        x = one(h)
        x["q"][at] = 0
        y = o[:, h:h + 1].clone()
        y[at] = 0
        if short:
            close(y, S[:, h:h + 1], x, dtype, rows=(start, stop), n=n)
    elif which == "v":
        col = torch.arange(D, device="cuda") == 17
        assert not bool(torch.isfinite(o[at:stop, h, 17]).any())
        assert not bool(torch.isfinite(S[n, h, :, 17]).any())
        for lo, hi in ((0, 17), (18, D)) if short else ():     # the other columns
            y, z = o[:, h:h + 1].clone(), S[:, h:h + 1].clone()
            y[..., :lo], y[..., hi:], z[..., :lo], z[..., hi:] = 0, 0, 0, 0
            close(y, z, one(h, lo, hi), dtype, rows=(start, stop), n=n)
        assert bool(torch.isfinite(o[at:stop, h][:, ~col]).all())
    else:
        assert not bool(torch.isfinite(here).any()) and not bool(torch.isfinite(rest).any())
        if which == "k":                       # (what that channel of k is added to)
            assert not bool(torch.isfinite(S[n, h, 17]).any())
            assert bool(torch.isfinite(S[n, h, :17]).all() and torch.isfinite(S[n, h, 18:]).all())
        else:
            assert not bool(torch.isfinite(S[n, h]).any())
    # every other head, and the same head of other sequences
    others = torch.ones((sum(lens), heads), dtype=torch.bool)
    others[start:stop, h] = False
    assert bool(torch.isfinite(o[others.cuda()]).all())
    for i, j in {(n, 0), (0, h), (len(lens) - 1, 0)} - {(n, h)}:
        a = sum(lens[:i])
        if lens[i] <= 3000:
            close(o[:, j:j + 1], S[:, j:j + 1], one(j), dtype, rows=(a, a + lens[i]), n=i)
