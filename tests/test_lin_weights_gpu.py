"""kda_lin_prefill: the weights' range."""

import pytest
import torch

from _lin import close, inputs
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
