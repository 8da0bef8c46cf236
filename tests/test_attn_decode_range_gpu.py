"""kda_attn_kv4_decode where the cache's values differ much in size between sequences and within
one, and with the weights' rounding that its header states."""

import numpy as np
import pytest
import torch

from _attn import D, Host, attend64, close, random_cache
from _util import kda
from test_attn_kv4_gpu import dev, pages_for

pytestmark = pytest.mark.gpu


def decode(q, data, table, lens, window=0):
    K = kda()
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    K.kda_attn_kv4_decode(q, dev(data), dev(table), torch.tensor(lens, dtype=torch.int32).cuda(),
                          o, lse=lse, window=window)
    K.kda_sync_status()
    return o, lse


def check(q, o, lse, host, table, lens, kv, which, window=0):
    """Of the sequences `which`: weights times steps enter the product in FP16."""
    for n in which:
        k, v, size = (torch.from_numpy(np.stack([host.rows(w, table[n], lens[n], h, big)
                                                 for h in range(kv)], 1))
                      for w, big in (("k", False), ("v", False), ("v", True)))
        ref = attend64(q[n].double().cpu(), k, v, window, moved=size)
        close(o[n].cpu(), lse[n].cpu(), ref, q.dtype, weights=torch.float16)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5])
@pytest.mark.parametrize("rows,heads", [(1, 4), (4, 2), (4, 8), (8, 1), (8, 16)])
@pytest.mark.parametrize("lens", [[1, 400], [5, 0, 3, 2, 130]])
def test_the_largest_windows_and_short_sequences(lens, rows, heads, window):
    """A length below the rows less such a window passes 32 bits."""
    rng = np.random.default_rng(43)
    table, total = pages_for(rng, lens, 32)
    data = random_cache(rng, total, 1, 32)
    q = torch.randn((len(lens), rows, heads, D), generator=torch.Generator().manual_seed(44)).to(
        torch.float16).cuda()
    o, lse = decode(q, data, table, lens, window)
    check(q, o, lse, Host(data), table, lens, 1, range(len(lens)), window)
