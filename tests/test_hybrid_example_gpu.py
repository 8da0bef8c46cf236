"""The example that serves a KDA and a full-attention layer together: its attention steps against
the plain 64-bit form, and rejected rows that leave no trace."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from _attn import attend64, close, quantise

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "hybrid_serving", os.path.join(ROOT, "examples", "hybrid_serving.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def stored(x):
    """What the cache holds of x [rows, heads, 128], and max(|value|, |s (code - 8)|)."""
    c, s, m = quantise(x.double().cpu().numpy())
    s, m = s.repeat(64, -1), m.repeat(64, -1)
    y = m + s * c
    return torch.from_numpy(y), torch.from_numpy(np.maximum(abs(y), abs(s * (c - 8.0))))


CHUNKS = ([70, 1, 33], [5, 40, 64])


def serve(trace=None, rejected=0):
    """Two prompt chunks, four rows of which two stay, four rows that all stay.  `rejected` seeds
    the two rows that do not stay."""
    model = example().Model(dim=256, heads=4, kv_heads=2, n_seqs=3, krows=4, longest=192, page=32,
                            trace=trace)
    g = torch.Generator().manual_seed(1)

    def draw(rows, gen=g):
        return torch.randn((rows, 256), generator=gen).to(torch.bfloat16).cuda()

    outs = [model.chunk(draw(sum(new)), new) for new in CHUNKS]
    x = draw(12)
    x.view(3, 4, 256)[:, 2:] = draw(6, torch.Generator().manual_seed(9 + rejected)).view(3, 2, 256)
    outs.append(model.rows(x).view(3, 4, 256)[:, :2].clone())
    model.keep([2, 2, 2], 4)
    outs.append(model.rows(draw(12)))
    model.keep([4, 4, 4], 4)
    from _util import kda
    kda().kda_sync_status()
    assert model.lens.tolist() == model.positions == [75 + 6, 41 + 6, 97 + 6]
    return outs


def test_attention_steps_against_the_plain_form():
    trace = []
    outs = serve(trace)
    assert all(bool(torch.isfinite(y).all()) for y in outs)
    history = [([], []) for _ in range(3)]
    for step, (q, k, v, o, lens) in enumerate(trace):
        new = CHUNKS[step] if step < 2 else [4] * 3
        at = 0
        for n, r in enumerate(new):
            part = slice(at, at + r)
            at += r
            for rows, x in zip(history[n], (k, v)):
                rows.append(x[part].cpu())
            kc, vc = (torch.cat(rows) for rows in history[n])
            assert int(lens[n]) == len(kc)
            if step == 0:      # nothing behind it: the rows as they are
                keys, values, moved = kc.double(), vc.double(), None
            else:
                keys, (values, moved) = stored(kc)[0], stored(vc)
            if step == 1:      # read rounds the cache's values
                keys, values = (x.to(torch.bfloat16).double() for x in (keys, values))
                moved = None
            ref = attend64(q[part].cpu().double(), keys, values, moved=moved)
            close(o[part].cpu(), None, ref, torch.bfloat16)
            if step == 2:      # two of the four rows stay
                for rows in history[n]:
                    rows[-1] = rows[-1][:2]


def test_rejected_rows_leave_no_trace():
    for a, b in zip(serve(rejected=0), serve(rejected=1)):
        assert torch.equal(a, b)
