"""Plain 64-bit forms of the full-attention calls, and the tolerances that follow from the
roundings they are allowed (no code shared with the library)."""

import math

import numpy as np
import torch

D = 128
TYPES = [torch.bfloat16, torch.float16]


def attend64(q, k, v, window=0, scale=1 / math.sqrt(D), moved=None):
    """One sequence: q [R, H, D], k, v [L, Hk, D] (64 bits).  Returns o [R, H, D], lse [R, H] and
    sum_j p_j |v_j|, the size that roundings of the weights act on (`moved`: other values in the
    place of |v|)."""
    moved = v.abs() if moved is None else moved
    R, H = q.shape[:2]
    L, Hk = k.shape[:2]
    o = torch.zeros((R, H, D), dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(o)
    lse = torch.full((R, H), -math.inf, dtype=torch.float64, device=q.device)
    for h in range(H):
        hk = h // (H // Hk)
        for i in range(R):
            p = L - R + i
            lo = max(0, p - window + 1) if window else 0
            if p < lo:
                continue
            s = (k[lo:p + 1, hk] @ q[i, h]) * scale
            lse[i, h] = torch.logsumexp(s, 0)
            w = torch.exp(s - lse[i, h])
            o[i, h] = w @ v[lo:p + 1, hk]
            mag[i, h] = w @ moved[lo:p + 1, hk]
    return o, lse, mag


def close(o, lse, ref, dtype, weights=None):
    """|o - ref| <= the output's rounding, plus the weights' (`weights`: their type), plus FP32
    scores: 128 products of size ~|q||k| with 2^-24 each move a score, and so a weight's relative
    size, by less than 2^-12 here."""
    r, rl, mag = ref
    half = torch.finfo(dtype).eps / 2
    wide = torch.finfo(weights or dtype).eps / 2
    err = (o.double() - r).abs()
    bound = half * r.abs() + (wide + 2.0 ** -12) * mag + torch.finfo(dtype).tiny
    assert bool((err <= bound).all()), (
        "o: worst excess %g" % float((err - bound).max()), int((err > bound).sum()))
    if lse is not None:
        empty = torch.isinf(rl)
        assert bool((lse[empty] == -math.inf).all())
        d = (lse.double() - rl)[~empty].abs()
        assert d.numel() == 0 or float(d.max()) <= 2.0 ** -12, "lse: %g" % float(d.max())


# ---------------------------------------------------------------- the 4-bit cache

def bf16_below(x):
    """The largest BF16 <= x, x a float64 array of normal numbers or zero."""
    m, e = np.frexp(x)
    return np.ldexp(np.floor(m * 256.0), e - 8)


def quantise(x):
    """x [rows, heads, 128] (float64, exact inputs) -> codes [rows, heads, 128], s, m [.., 2]."""
    g = x.reshape(x.shape[:-1] + (2, 64))
    m = bf16_below(g.min(-1))
    s = -bf16_below(-((g.max(-1) - m) / 15.0))
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint((g - m[..., None]) / s[..., None])
    c = np.where(s[..., None] > 0, np.clip(c, 0, 15), 0).astype(np.uint8)
    return c.reshape(x.shape), s, m


def place(which, tok, ch):
    """(byte of the 16-token group, shift) of a code, as the header gives it."""
    a, b, j, x = ch // 64, ch // 16 % 4, ch // 8 % 2, ch % 8
    if which == "k":
        i, g, t, e = tok // 8, tok % 8, x // 2, x % 2
    else:
        i, g, t, e = tok // 8, x, tok % 8 // 2, tok % 2
    return 512 * a + 16 * (4 * g + t) + 4 * b + 2 * e + i, 4 * j


def bf16_bits(x):
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


class Host:
    """A paged cache on the host, written and read a value at a time."""

    def __init__(self, data):
        self.data = data                       # uint8 [pages, kv, page * 144]
        self.page = data.shape[2] // 144

    def _base(self, which):
        return 0 if which == "k" else self.page * 72

    def write(self, which, page, tok, h, codes, s, m):
        blk = self.data[page, h]
        base = self._base(which)
        for ch in range(D):
            at, sh = place(which, tok % 16, ch)
            at += base + tok // 16 * 1024
            blk[at] = (int(blk[at]) & ~(15 << sh) & 255) | int(codes[ch]) << sh
        for a in range(2):
            for n, val in enumerate((s[a], m[a])):
                bits = int(bf16_bits(val))
                at = base + self.page * 64 + tok * 8 + 4 * a + 2 * n
                blk[at], blk[at + 1] = bits & 255, bits >> 8

    def rows(self, which, table, length, h, size=False):
        """Values [length, 128] of one sequence and head, float64; with `size`, max(|value|,
        |s (code - 8)|): what roundings of a weight times a step act on."""
        pos = np.arange(length)
        blk = self.data[table[pos // self.page], h]
        base, tok = self._base(which), pos % self.page
        ch = np.arange(D)
        a, b, j, x = ch // 64, ch // 16 % 4, ch // 8 % 2, ch % 8
        t = tok[:, None] % 16
        if which == "k":
            inner = 16 * (4 * (t % 8) + x // 2) + 2 * (x % 2) + t // 8
        else:
            inner = 16 * (4 * x + t % 8 // 2) + 2 * (t % 2) + t // 8
        at = base + tok[:, None] // 16 * 1024 + 512 * a + 4 * b + inner
        code = np.take_along_axis(blk, at, 1) >> (4 * j) & 15
        par = np.take_along_axis(blk, base + self.page * 64 + tok[:, None] * 8 + np.arange(8), 1)
        par = np.ascontiguousarray(par).view(np.uint16).astype(np.uint32) << 16
        par = np.ascontiguousarray(par).view(np.float32).astype(np.float64)
        step = par[:, 0::2].repeat(64, 1)
        value = par[:, 1::2].repeat(64, 1) + step * code
        return np.maximum(np.abs(value), np.abs(step * (code - 8.0))) if size else value


def random_cache(rng, pages, kv, page):
    """Codes at random, steps and minima as rows of unit spread leave them."""
    data = rng.integers(0, 256, (pages, kv, page * 144), dtype=np.uint8)
    for at in (page * 64, page * 136):
        s = rng.uniform(0.2, 0.4, (pages, kv, page * 2))
        m = -7.5 * s + rng.normal(0, 0.3, s.shape)
        par = np.stack([bf16_bits(s), bf16_bits(m)], -1)
        data[:, :, at:at + page * 8] = par.reshape(pages, kv, -1).view(np.uint8)
    return data
