"""The binding's calls in C take what their forms in Python take, to the same effect, and refuse the
rest with the same kind of error."""

import numpy
import pytest
import torch

import _pages
from _util import kda

pytestmark = pytest.mark.gpu
D = 128


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def rows(*shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(len(shape))).to(dtype).cuda()


def wide(x):
    """The same values, heads 16 bytes past a power of two apart from row to row."""
    heads = x.shape[-2]
    y = torch.zeros(x.shape[:-2] + ((heads + 1) * D,), dtype=x.dtype, device="cuda")
    y = y[..., :heads * D].unflatten(-1, (heads, D))
    return y.copy_(x)


def lin(K):
    d = dict(q=rows(6, 2, D), k=rows(6, 2, D), v=rows(6, 4, D), g=-torch.rand((6, 4)).cuda(),
             out=rows(6, 4, D), state_in=torch.randn((1, 4, D, D)).cuda(),
             state_out=torch.zeros((1, 4, D, D)).cuda(), t=None, cu_seqlens=None, scale=0.5,
             workspace=K.kda_lin_prefill_workspace(64, 8, 4))
    d["q"] /= 16
    four = {x: d[x].unflatten(0, (2, 3)) for x in ("q", "k", "v", "g", "out")}
    two = {x: torch.randn((2, 4, D, D)).cuda() for x in ("state_in", "state_out")}
    return d, four, two


def cases(K):
    """(call, arguments, ways to change them)"""
    d, four, two = lin(K)
    cu = ints([0, 2, 6])
    any_rows = [lambda x: x[:5], lambda x: x[:, :1], lambda x: x.half(), lambda x: x.cpu(), wide,
                lambda x: x[:0], lambda x: x[..., :64], lambda x: x.transpose(-1, -2),
                lambda x: x.unsqueeze(0), lambda x: x.flatten(), lambda x: x[:1].expand(6, -1, -1),
                lambda x: None, lambda x: 3, lambda x: x[::2]]
    any_array = [lambda x: x.long(), lambda x: x.float(), lambda x: x.cpu(), lambda x: x[:-1],
                 lambda x: x[:0], lambda x: x.unsqueeze(0), lambda x: None, lambda x: [1, 2],
                 lambda x: torch.stack([x, x], -1)[..., 0]]
    any_state = [lambda x: x[:, :2], lambda x: x.half(), lambda x: x.cpu(), lambda x: None,
                 lambda x: x.transpose(-1, -2), lambda x: x.expand(2, -1, -1, -1), lambda x: x[0]]
    any_space = [lambda x: None, lambda x: x[:64], lambda x: x.cpu(), lambda x: x.view(torch.float32),
                 lambda x: x[::2], lambda x: x.view(2, -1), lambda x: x[:0], lambda x: 7]
    any_number = [lambda x: 2, lambda x: numpy.float32(0.25), lambda x: torch.tensor(0.25),
                  lambda x: "0.5", lambda x: None, lambda x: float("nan"), lambda x: True,
                  lambda x: torch.tensor([0.25, 1.0])]
    any_gate = any_rows[:4] + [lambda x: x.float(), lambda x: -torch.rand(4).cuda(),
                               lambda x: -torch.rand(5).cuda(), lambda x: None,
                               lambda x: torch.stack([x, x], 1)[:, 0],
                               lambda x: torch.stack([x, x], 2)[..., 0], lambda x: x[:1].expand(6, 4)]
    lengths = [(lambda y: lambda x: y)(y) for y in (0, 3, 6, 7, -1, 2.0, numpy.int64(4), True, "3")]
    offsets = [(lambda y: lambda x: y)(y) for y in (cu, cu[1:2], cu.long(), cu.cpu(), [0, 6], cu[:0])]
    change = dict(q=any_rows, k=any_rows, v=any_rows, out=any_rows, g=any_gate, state_in=any_state,
                  state_out=any_state, scale=any_number)
    yield "kda_lin_prefill", d, dict(change, t=lengths, cu_seqlens=offsets, workspace=any_space)
    yield ("kda_lin_prefill", dict(d, cu_seqlens=cu, **two),
           dict(change, t=lengths, cu_seqlens=offsets, workspace=any_space))
    yield ("kda_lin_prefill", dict(d, **four, **two),
           dict(change, t=lengths, cu_seqlens=offsets, workspace=any_space))
    base = {x: d[x] for x in ("scale",)}
    snaps = [torch.zeros((2, 4, D, D)).cuda() for _ in range(4)]
    lists = [lambda x: (), lambda x: x[:1], lambda x: tuple(x), lambda x: x + x[:1],
             lambda x: x[:2] + [None], lambda x: x * 4, lambda x: None, lambda x: [y.half() for y in x],
             lambda x: [y[:1] for y in x], lambda x: torch.stack(x)]
    yield ("kda_lin_decode", dict(base, **four, **two, snapshots=snaps[:3]),
           dict(change, snapshots=lists))
    yield ("kda_lin_decode", dict(base, q=d["q"][:2], k=d["k"][:2], v=d["v"][:2], g=d["g"][:2],
                                  out=d["out"][:2], **two, snapshots=snaps[:1]),
           dict(change, snapshots=lists))
    q, k = rows(6, 4, D), rows(6, 2, D)
    freq, pos = torch.rand(32).cuda(), torch.arange(12, dtype=torch.int32).cuda()
    axes = [(lambda y: lambda x: y)(y) for y in
            ([0, 1] * 16, [0] * 31, [2] * 32, [-1] * 32, bytes([1] * 32), torch.ones(32).int(),
             numpy.zeros(32, dtype=numpy.int64), [0.0] * 32, None, "x" * 32, [300] * 32)]
    flags = [(lambda y: lambda x: y)(y) for y in (True, 1, 0, None, "yes", 2)]
    change = dict(q=any_rows, k=any_rows, q_out=any_rows, k_out=any_rows, inv_freq=any_array,
                  positions=any_array + [lambda x: pos, lambda x: pos.view(6, 2), lambda x: pos.view(2, 6)],
                  pair_axis=axes, interleaved=flags, factor=any_number)
    yield ("kda_attn_rope", dict(q=q, k=k, positions=pos[:6], inv_freq=freq, q_out=rows(6, 4, D),
                                 k_out=rows(6, 2, D), pair_axis=None, interleaved=False, factor=1.0),
           change)
    yield ("kda_attn_rope", dict(q=q.unflatten(0, (2, 3)), k=None, positions=pos.view(2, 3, 2),
                                 inv_freq=freq, q_out=None, k_out=None, pair_axis=[0, 1] * 16,
                                 interleaved=True, factor=1.0),
           dict(q=any_rows, k=[lambda x: k.unflatten(0, (2, 3)), lambda x: k], q_out=[lambda x: q],
                k_out=[lambda x: k], positions=any_array, pair_axis=axes, interleaved=flags))
    table, lens, refs, _ = _pages.some_state(3, 5, 4, 40, 16, 0.5)
    table, lens, refs, parent = ints(table), ints(lens), ints(refs), ints([1, 1, -1, 0, 4])
    ws = K.kda_attn_kv4_pages_workspace(40, 5, 4)
    pages = [(lambda y: lambda x: y)(y) for y in (32, 48, 0, -16, 16.0, "16", None, numpy.int32(64),
                                                 1 << 20, True)]
    tables = any_array + [lambda x: x[0], lambda x: x[:, :2], lambda x: x.t().contiguous()]
    yield ("kda_attn_kv4_resize", dict(page_table=table, lens=lens, refs=refs, page=16, workspace=ws),
           dict(page_table=tables, lens=any_array, refs=any_array, page=pages, workspace=any_space))
    five, one = ints([0] * 5), ints([0])
    yield ("kda_attn_kv4_fork",
           dict(page_table=table, lens=lens, refs=refs, parent=parent, page_table_out=table.clone(),
                lens_out=lens.clone(), refs_out=refs.clone(), src=five, dst=five.clone(), count=one,
                page=16, workspace=ws),
           dict(page_table=tables, lens=any_array, refs=any_array, parent=any_array,
                page_table_out=tables, lens_out=any_array, refs_out=any_array, src=any_array,
                dst=any_array, count=any_array, page=pages, workspace=any_space))
    half = ints([0] * 20)
    yield ("kda_attn_kv4_compact",
           dict(page_table=table, refs=refs, page_table_out=table.clone(), refs_out=refs.clone(),
                src=half, dst=half.clone(), count=one, workspace=ws),
           dict(page_table=tables, refs=any_array, page_table_out=tables, refs_out=any_array,
                src=any_array, dst=any_array, count=any_array, workspace=any_space))
    caches = [torch.randint(0, 256, (9, 2, 16 * 144), dtype=torch.uint8, device="cuda")
              for _ in range(3)]
    yield ("kda_attn_kv4_copy", dict(caches=caches, src=ints([0, 1, 2]), dst=ints([5, 6, 7]),
                                     count=ints([2])),
           dict(caches=[lambda x: x[0], lambda x: tuple(x), lambda x: [], lambda x: x * 50,
                        lambda x: [x[0], x[1][:5]], lambda x: [y.float() for y in x],
                        lambda x: [y.cpu() for y in x], lambda x: [y[:, :, :2000] for y in x],
                        lambda x: [y[0] for y in x], lambda x: [y[::2] for y in x], lambda x: None,
                        lambda x: [None], lambda x: torch.stack(x)],
                src=any_array, dst=any_array, count=any_array))


def flat(x):
    if isinstance(x, torch.Tensor):
        return [x]
    return [z for y in x for z in flat(y)] if isinstance(x, (list, tuple)) else []


def outcome(K, name, args):
    """What a call does: its error's kind, or every tensor's bytes behind it."""
    copies = {}

    def fresh(x):
        if isinstance(x, torch.Tensor):
            if id(x) not in copies:
                y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=x.device)
                # (a broadcast tensor is one row written once)
                copies[id(x)] = y.copy_(x) if 0 not in x.stride() or not x.numel() else x
            return copies[id(x)]
        return type(x)(fresh(y) for y in x) if type(x) in (list, tuple) else x

    args = {x: fresh(y) for x, y in args.items()}
    try:
        got = getattr(K, name)(**args)
    except Exception as e:
        kind = type(e).__name__
        return "KdaError %d" % e.status if kind == "KdaError" else kind
    try:
        K.kda_sync_status()
        status = "clean"
    except K.KdaError as e:
        status = str(e)
    seen = [x for y in args if y != "workspace" for x in flat(args[y])] + flat(got or ())
    return status, [x.clone(memory_format=torch.contiguous_format).view(-1).view(torch.uint8).tolist()
                    if x.numel() < 5000 else x.cpu().reshape(-1).view(torch.uint8).numpy().tobytes()
                    for x in seen if x.numel()]


def test_both_forms_take_the_same(monkeypatch):
    K, taken, wrong = kda(), {}, []
    real = K._fast
    assert type(real).__name__ == "module"
    for name, args, change in cases(K):
        tries = [("as it is", args)]
        for x, ways in change.items():
            for i, way in enumerate(ways):
                try:
                    tries.append(("%s %d" % (x, i), dict(args, **{x: way(args[x])})))
                except (AttributeError, IndexError, RuntimeError, TypeError, ValueError):
                    pass                       # (no such change of this argument)
        for what, given in tries:
            both = []
            for fast in (real, K._Slow()):
                monkeypatch.setattr(K, "_fast", fast)
                both.append(outcome(K, name, given))
            if both[0] != both[1]:
                wrong.append((name, what, [x if isinstance(x, str) else x[0] for x in both]))
            taken.setdefault(name, []).append(isinstance(both[0], tuple))
    assert not wrong, "\n".join(map(str, wrong))
    for name, ok in taken.items():             # both kinds were among them
        assert ok[0] and 0 < sum(ok) < len(ok), (name, sum(ok), len(ok))
