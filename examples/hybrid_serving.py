"""A KDA layer, a layer of linear attention with a decay for each head and a full-attention layer
served together, as hybrid decoders stack them.

The linear layers keep a state of fixed size per sequence, the full-attention layer a 4-bit paged
cache of its keys and values, whose pages kda_attn_kv4_resize gives and frees on the device.  Three
steps, each over a batch of sequences:

* a first prompt chunk: kda_attn_prefill over the rows at hand, kda_attn_kv4_append to keep them;
* a later chunk: append first, kda_attn_kv4_read for the context, kda_attn_prefill with more keys
  than queries;
* rows to be verified (one row: plain decoding): append, kda_attn_kv4_decode.  Rows that the
  verification rejects are taken back: the linear layers return to the snapshot after the last
  row kept, the full-attention layer counts fewer positions.

Between them sequences may go on from others (samples of one prompt, beams): kda_attn_kv4_fork
shares what pages they can, kda_attn_kv4_copy fills the rest.  kda_attn_kv4_compact gathers the
pages in use at the cache's beginning.

Weights and inputs are random; projections are plain matrix products.

    python examples/hybrid_serving.py
"""

import itertools
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_prepare_gb300 as K  # noqa: E402

D = 128
BF16 = torch.bfloat16


def _weight(gen, *shape):
    w = torch.randn(shape, generator=gen) / math.sqrt(shape[0])
    return w.to(BF16).cuda()


def offsets(rows):
    return torch.tensor([0] + list(itertools.accumulate(rows)), dtype=torch.int32).cuda()


class KdaLayer:
    def __init__(self, gen, dim, heads, n_seqs, krows):
        self.heads, hd = heads, heads * D
        self.w_in = _weight(gen, dim, 3 * hd)
        # forget gate | output gate | beta; rows 8 columns a piece, as kda_gate takes them
        self.w_gate = _weight(gen, dim, 2 * hd + -(-heads // 8) * 8)
        self.w_conv = (torch.randn((3 * hd, 4), generator=gen) / 2).to(BF16).cuda()
        self.w_norm = torch.ones(D, dtype=BF16).cuda()
        self.w_out = _weight(gen, hd, dim)
        self.dt_bias, self.a_log = torch.zeros(hd).cuda(), torch.zeros(heads).cuda()
        self.state = torch.zeros((n_seqs, heads, D, D)).cuda()
        self.conv = torch.zeros((n_seqs, 3 * hd, 4)).cuda()
        self.state_after = torch.zeros((krows,) + self.state.shape).cuda()
        self.conv_after = torch.zeros((krows,) + self.conv.shape).cuda()

    def _mixed(self, x, dtype):
        hd, rows = self.heads * D, x.shape[0]
        gates = x @ self.w_gate
        g = torch.empty((rows, self.heads, D), dtype=dtype, device="cuda")
        beta = torch.empty((rows, self.heads), dtype=dtype, device="cuda")
        K.kda_gate(gates[:, :hd], self.dt_bias, self.a_log, gates[:, 2 * hd:], g, beta, -5.0)
        return x @ self.w_in, g, beta, gates[:, hd:2 * hd].contiguous()

    def _out(self, core, gate):
        out = torch.empty_like(gate)
        K.kda_o_norm_gated(core.view(core.shape[0], -1), gate, self.w_norm, out)
        return out @ self.w_out

    def chunk(self, x, cu):
        mixed, g, beta, gate = self._mixed(x, BF16)
        rows, hd = x.shape[0], self.heads * D
        qkv = torch.empty_like(mixed)
        K.kda_conv_silu_l2(self.conv, mixed, self.w_conv, qkv, cu_seqlens=cu)
        q, k, v = (y.unflatten(1, (self.heads, D)) for y in qkv.split(hd, 1))
        core = torch.empty((rows, self.heads, D), device="cuda")
        K.kda_prefill(self.state, q, k, v, g, beta, core, rows, 64, cu_seqlens=cu)
        return self._out(core, gate)

    def rows(self, x, n_seqs, krows):
        mixed, g, beta, gate = self._mixed(x, torch.float32)
        shape = (n_seqs, krows, self.heads, D)
        qkv = torch.empty_like(mixed)
        K.kda_conv_silu_l2_k(self.conv, mixed.view(n_seqs, krows, -1), self.w_conv,
                             qkv.view(n_seqs, krows, -1), list(self.conv_after[:krows]))
        q, k, v = (y.float().reshape(shape) for y in qkv.split(self.heads * D, 1))
        core = torch.empty(shape, device="cuda")
        K.kda_decode_k(self.state, q, k, v, g.view(shape), beta.view(shape[:3]), core,
                       list(self.state_after[:krows]))
        return self._out(core.view(n_seqs * krows, -1), gate)

    def keep(self, kept):
        n = torch.arange(kept.numel(), device="cuda")
        self.state.copy_(self.state_after[kept - 1, n])
        self.conv.copy_(self.conv_after[kept - 1, n])


class LinearLayer:
    """Heads that forget at fixed rates, from a token in two to one in 256."""

    def __init__(self, gen, dim, heads, n_seqs, krows):
        self.heads = heads
        self.w_in = _weight(gen, dim, 3 * heads * D)
        self.w_out = _weight(gen, heads * D, dim)
        self.g = -torch.exp2(torch.linspace(-1, -8, heads)).cuda()
        self.state = torch.zeros((n_seqs, heads, D, D)).cuda()
        self.state_after = torch.zeros((krows,) + self.state.shape).cuda()

    def _qkv(self, x, *lead):
        q, k, v = (x @ self.w_in).view(*lead, 3, self.heads, D).unbind(-3)
        q, k = (torch.nn.functional.normalize(y.float(), dim=-1).to(BF16) for y in (q, k))
        return q, k, v, torch.empty_like(q)

    def _out(self, o, rows):
        o = torch.nn.functional.rms_norm(o, (D,))
        return o.view(rows, -1) @ self.w_out

    def chunk(self, x, cu):
        q, k, v, o = self._qkv(x, x.shape[0])
        K.kda_lin_prefill(q, k, v, self.g, o, self.state, self.state, cu_seqlens=cu)
        return self._out(o, x.shape[0])

    def rows(self, x, n_seqs, krows):
        q, k, v, o = self._qkv(x, n_seqs, krows)
        K.kda_lin_decode(q, k, v, self.g, o, self.state, self.state,
                         list(self.state_after[:krows]))
        return self._out(o, x.shape[0])

    def keep(self, kept):
        self.state.copy_(self.state_after[kept - 1, torch.arange(kept.numel(), device="cuda")])


class AttentionLayer:
    """`trace`, a list, receives what the attention calls saw and gave, step by step."""

    def __init__(self, gen, dim, heads, kv_heads, n_seqs, krows, longest, page=64, trace=None):
        self.heads, self.kv = heads, kv_heads
        self.w_in = _weight(gen, dim, (heads + 2 * kv_heads) * D)
        self.w_out = _weight(gen, heads * D, dim)
        width = -(-longest // page)
        self.page, pages = page, n_seqs * width
        self.cache = K.kv4_cache(pages, kv_heads, page)
        self.table = torch.full((n_seqs, width), -1, dtype=torch.int32).cuda()
        self.refs = torch.zeros(pages, dtype=torch.int32).cuda()
        self.workspace = K.kda_attn_kv4_workspace(n_seqs, krows, heads, kv_heads)
        self.pages_workspace = K.kda_attn_kv4_pages_workspace(pages, n_seqs, width)
        self.inv_freq = (10000.0 ** (-torch.arange(D // 2) / (D // 2))).cuda()
        self.trace = trace

    def resize(self, lens):
        K.kda_attn_kv4_resize(self.table, lens, self.refs, self.page, self.pages_workspace)

    def fork(self, lens, parent):
        moves = K.kda_attn_kv4_fork(self.table, lens, self.refs, parent, page=self.page,
                                    workspace=self.pages_workspace)
        K.kda_attn_kv4_copy([self.cache], *moves)

    def compact(self):
        moves = K.kda_attn_kv4_compact(self.table, self.refs, workspace=self.pages_workspace)
        K.kda_attn_kv4_copy([self.cache], *moves)

    def _qkv(self, x, positions):
        heads = (x @ self.w_in).unflatten(1, (-1, D))
        q, k, v = heads.split((self.heads, self.kv, self.kv), 1)
        K.kda_attn_rope(q, k, positions, self.inv_freq)
        return q, k, v

    def _out(self, q, k, v, o, lens):
        if self.trace is not None:
            self.trace.append(tuple(y.clone() for y in (q, k, v, o.view(q.shape), lens)))
        return o.view(o.shape[0], -1) @ self.w_out

    def chunk(self, x, cu, lens, positions, context=None):
        """`lens` counts the chunk's rows, whose positions are `positions`; `context`, each
        sequence's positions with them as a list, unless the chunk is every sequence's first."""
        q, k, v = self._qkv(x, positions)
        self.resize(lens)
        o = torch.empty((x.shape[0], self.heads, D), dtype=BF16, device="cuda")
        K.kda_attn_kv4_append(k, v, self.cache, self.table, lens, cu_seqlens=cu)
        if context is None:
            K.kda_attn_prefill(q, k, v, o, cu_seqlens=cu)
        else:
            cu_k = offsets(context)
            kc, vc = (torch.empty((sum(context), self.kv, D), dtype=BF16, device="cuda")
                      for _ in range(2))
            K.kda_attn_kv4_read(kc, vc, self.cache, self.table, lens, cu_seqlens=cu_k)
            K.kda_attn_prefill(q, kc, vc, o, cu_seqlens=cu, cu_seqlens_k=cu_k)
        return self._out(q, k, v, o, lens)

    def rows(self, x, n_seqs, krows, lens):
        rows = torch.arange(-krows, 0, dtype=torch.int32, device="cuda")
        q, k, v = self._qkv(x, (lens[:, None] + rows).view(-1))
        self.resize(lens)
        q4 = q.contiguous().view(n_seqs, krows, self.heads, D)
        o = torch.empty_like(q4)
        K.kda_attn_kv4_append(k, v, self.cache, self.table, lens)
        K.kda_attn_kv4_decode(q4, self.cache, self.table, lens, o, workspace=self.workspace)
        return self._out(q, k, v, o.view(n_seqs * krows, self.heads, D), lens)


class Model:
    def __init__(self, dim=1024, heads=8, kv_heads=2, n_seqs=4, krows=4, longest=8192, page=64,
                 seed=0, trace=None):
        gen = torch.Generator().manual_seed(seed)
        self.n, self.krows = n_seqs, krows
        self.kda = KdaLayer(gen, dim, heads, n_seqs, krows)
        self.lin = LinearLayer(gen, dim, heads, n_seqs, krows)
        self.attn = AttentionLayer(gen, dim, heads, kv_heads, n_seqs, krows, longest, page, trace)
        self.lens = torch.zeros(n_seqs, dtype=torch.int32).cuda()
        self.positions = [0] * n_seqs      # lens, as the host knows it

    def _norm(self, x):
        return torch.nn.functional.rms_norm(x, x.shape[-1:])

    def chunk(self, x, new):
        """x [sum of new, dim], new: rows of each sequence."""
        first = not any(self.positions)
        at = torch.cat([torch.arange(a, a + b) for a, b in zip(self.positions, new)])
        self.positions = [a + b for a, b in zip(self.positions, new)]
        cu = offsets(new)
        self.lens += cu.diff()
        x = x + self.kda.chunk(self._norm(x), cu)
        x = x + self.lin.chunk(self._norm(x), cu)
        return x + self.attn.chunk(self._norm(x), cu, self.lens, at.to(torch.int32).cuda(),
                                   None if first else self.positions)

    def rows(self, x):
        """x [n_seqs * krows, dim]: krows rows of each sequence (no host work that a graph could
        not replay)."""
        krows = x.shape[0] // self.n
        self.lens += krows
        x = x + self.kda.rows(self._norm(x), self.n, krows)
        x = x + self.lin.rows(self._norm(x), self.n, krows)
        return x + self.attn.rows(self._norm(x), self.n, krows, self.lens)

    def keep(self, kept, krows):
        """The first kept[n] >= 1 of the krows rows of sequence n stay."""
        self.positions = [a + b for a, b in zip(self.positions, kept)]
        kept = torch.tensor(kept).cuda()
        self.kda.keep(kept)
        self.lin.keep(kept)
        self.lens += (kept - krows).to(torch.int32)
        self.attn.resize(self.lens)

    def fork(self, parent):
        """Sequence n goes on from sequence parent[n], or (-1) is over."""
        self.positions = [self.positions[p] if p >= 0 else 0 for p in parent]
        parent = torch.tensor(parent, dtype=torch.int32).cuda()
        self.attn.fork(self.lens, parent)      # (and the lengths)
        live = parent >= 0
        for state in (self.kda.state, self.kda.conv, self.lin.state):
            new = state[parent.clamp(min=0)]
            state.copy_(torch.where(live.view(-1, *[1] * (new.dim() - 1)), new, 0))

    def compact(self):
        self.attn.compact()


def main():
    torch.manual_seed(0)
    model = Model(dim=4096, heads=32, kv_heads=8, n_seqs=16, krows=4, longest=8192)
    for new in ([2000 + 100 * n for n in range(16)], [1000] * 16):
        x = torch.randn((sum(new), 4096), dtype=BF16, device="cuda")
        model.chunk(x, new)
    x = torch.randn((64, 4096), dtype=BF16, device="cuda")
    model.rows(x)
    model.keep([1 + n % 4 for n in range(16)], 4)
    K.kda_sync_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = model.rows(x)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    graph.replay()
    model.keep([4] * 16, 4)
    start.record()
    for _ in range(20):
        graph.replay()
        model.keep([1 + n % 4 for n in range(16)], 4)
    stop.record()
    K.kda_sync_status()
    assert torch.isfinite(y).all() and model.lens.tolist() == model.positions
    print("16 sequences of %d to %d positions, 4 rows each: %.3f ms a step" % (
        min(model.positions), max(model.positions), start.elapsed_time(stop) / 20))
    model.fork([n // 4 for n in range(16)])    # four samples of each of the first four
    model.compact()
    graph.replay()
    model.keep([4] * 16, 4)
    K.kda_sync_status()
    assert torch.isfinite(y).all() and model.lens.tolist() == model.positions
    used = int((model.attn.refs > 0).sum())
    print("16 sequences over 4 prompts: %d pages of %d in use" % (used, model.attn.refs.numel()))


if __name__ == "__main__":
    main()
