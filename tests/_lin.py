"""Linear attention with a decay for each head, token by token in 64 bits, and the
tolerances that follow from the roundings the calls are allowed (no code shared
with the library)."""

import math

import torch

D = 128
SCALE = 1 / math.sqrt(D)


def inputs(seed, rows, heads, qk, dtype, rate=1.0, n_seqs=1, state=True, dev="cuda"):
    """q, k of unit length, v of unit spread, g [rows, heads] from heads that forget at
    `rate` a token to ones that hardly do."""
    g = torch.Generator().manual_seed(seed)

    def unit(h):
        x = torch.randn((rows, h, D), generator=g)
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype).to(dev)

    d = dict(q=unit(qk), k=unit(qk), v=torch.randn((rows, heads, D), generator=g).to(dtype).to(dev))
    rates = rate * torch.exp2(-8 * torch.rand(heads, generator=g))
    d["g"] = (-rates * torch.rand((rows, heads), generator=g) * 2).to(dev)
    d["state"] = None
    if state:
        d["state"] = (torch.randn((n_seqs, heads, D, D), generator=g) * 0.3).to(dev)
    return d


def walk64(q, k, v, g, state, scale=SCALE, keep=()):
    """One sequence: q, k [T, qk, D], v [T, H, D], g [T, H] or [H]; state [H, D, D] or None.
    Returns o, S, the states after the rows in `keep`."""
    T, H = v.shape[:2]
    share = H // q.shape[1]
    S = torch.zeros((H, D, D), dtype=torch.float64, device=v.device) if state is None \
        else state.double().clone()
    o = torch.zeros((T, H, D), dtype=torch.float64, device=v.device)
    q, k, v = q.double().repeat_interleave(share, 1), k.double().repeat_interleave(share, 1), \
        v.double()
    decay = torch.exp(g.double().expand(T, H))
    kept = []
    for t in range(T):
        S = S * decay[t, :, None, None] + k[t, :, :, None] * v[t, :, None, :]
        o[t] = torch.einsum("hi,hij->hj", q[t], S) * scale
        if t in keep:
            kept.append(S.clone())
    return o, S, kept


def bounds(q, k, v, g, state, dtype, scale=SCALE):
    """Largest errors of o and of the state, |o| aside.  With o_abs, S_abs the recurrence
    of absolute values, and o_half, S_half that of half the decay:

    o: each product of a weight and a value rounds the weight, or the state's entry, to 16
    bits once, half a step of o_abs; sums of up to T + 128 FP32 terms: under 2^-12 of it.
    S: v times its decay is kept as two 16-bit numbers, half a step squared of it (BF16:
    2^-18; FP16 less), and sums as above, (T + 64) 2^-24.
    Both: a decay over x = |sum of g| is off by 2^-21 x of itself (FP32 sums of up to
    128 numbers), and x e^-x is below e^(-x/2): 2^-21 of o_half, S_half."""
    a = [x.double().abs() for x in (q, k, v)]
    s = None if state is None else state.double().abs()
    o_abs, S_abs, _ = walk64(*a, g, s, abs(scale))
    o_half, S_half, _ = walk64(*a, g.double().clamp_min(-1e4) / 2, s, abs(scale))
    half = torch.finfo(dtype).eps / 2
    T = v.shape[0]
    return ((half + 2.0 ** -12) * o_abs + 2.0 ** -21 * o_half,
            (2.0 ** -17 + (T + 64) * 2.0 ** -24) * S_abs + 2.0 ** -21 * S_half)


def close(o, S, d, dtype, rows=None, n=0, scale=SCALE):
    """o's rows [a, b) and state n against the 64-bit walk of those rows."""
    a, b = rows if rows else (0, d["v"].shape[0])
    g = d["g"] if d["g"].dim() == 1 else d["g"][a:b]
    s0 = None if d["state"] is None else d["state"][n]
    args = (d["q"][a:b], d["k"][a:b], d["v"][a:b], g, s0)
    ro, rs, _ = walk64(*args, scale=scale)
    bo, bs = bounds(*args, dtype, scale=scale)
    half = torch.finfo(dtype).eps / 2
    if b > a:
        over = (o[a:b].double() - ro).abs() - (half * ro.abs() + bo + torch.finfo(dtype).tiny)
        assert float(over.max()) <= 0, ("o", float(over.max()), int((over > 0).sum()))
    if S is not None:
        over = (S[n].double() - rs).abs() - (bs + 2.0 ** -126)
        assert float(over.max()) <= 0, ("state", float(over.max()), int((over > 0).sum()))
