"""kda_lin_prefill: the weights' range, and decays beside ones that leave nothing."""

import pytest
import torch

from _lin import D, close, inputs
from _util import kda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2.0 ** -10, 2.0 ** -5, 2.0 ** 12])
@pytest.mark.parametrize("T", [100, 700])
def test_products_of_any_size(T, size):
    """q . k from 2^-24 to above FP16's largest number: v and the scale make up for it."""
    K = kda()
    d = inputs(T, T, 3, 3, torch.float16, rate=0.1)
    d["q"], d["k"] = (d[x].float().mul(size).half() for x in ("q", "k"))
    d["v"] = (d["v"].float() * min(1 / size, 1024.0)).half()
    scale = 16 / size if size < 1 else 16 / size ** 2
    d["state"] = d["state"] * (1.0 if size < 1 else size)
    o, S = torch.full_like(d["v"], float("nan")), torch.empty_like(d["state"])
    K.kda_lin_prefill(d["q"], d["k"], d["v"], d["g"], o, d["state"], S, scale=scale)
    K.kda_sync_status()
    assert bool(torch.isfinite(o).all())
    close(o, S, d, torch.float16, scale=scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("least", [-20.0, -110.0, -float("inf")])
def test_weights_behind_tokens_that_leave_nothing(least, dtype):
    """28 tokens of each 32 leave next to nothing; of the other four, token t weighs the one before
    it by exp(g_t), a number of the type, and itself by 1: both come out exactly, as decays are
    good to 2^-20 and half a step is 2^-12 (BF16: 2^-9)."""
    K, T, heads = kda(), 128, 64
    gen = torch.Generator().manual_seed(3)
    q = torch.zeros((T, heads, D), dtype=dtype, device="cuda")
    q[..., 0] = 1
    v = torch.eye(D, dtype=dtype, device="cuda")[:, None].expand(T, heads, D).contiguous()
    w = (0.5 + 0.5 * torch.rand((T, heads), generator=gen)).to(dtype)
    g = torch.log(w.double()).float()
    strong = torch.arange(T) % 32 < 28
    g[strong] = least if least == -float("inf") else \
        least * (1 - 0.2 * torch.rand((int(strong.sum()), heads), generator=gen))
    o = torch.empty_like(v)
    K.kda_lin_prefill(q, q, v, g.cuda(), o, scale=1.0)
    K.kda_sync_status()
    for t in range(T):
        assert bool((o[t, :, t] == 1).all())
        if t % 32 > 28:
            assert torch.equal(o[t, :, t - 1].cpu(), w[t]), t
