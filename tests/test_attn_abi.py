"""The full-attention calls refuse bad arguments before anything reaches the device."""

import ctypes

import numpy as np
import pytest

V, I, F, U64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint64, ctypes.c_size_t
I64 = ctypes.c_int64
BUF = ctypes.create_string_buffer(64)
P = ctypes.cast(ctypes.addressof(BUF) + (16 - ctypes.addressof(BUF) % 16) % 16, V)
ODD = V(P.value + 8)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    L = ctypes.CDLL(__graft_entry__._library_builder().build())
    L.kda_last_error.restype = ctypes.c_char_p
    return L


def caller(fn, names, ok):
    def call(**kw):
        assert set(kw) <= set(names)
        return fn(*[kw.get(n, v) for n, v in zip(names, ok)])
    return call


def test_prefill_refusals(lib):
    f = lib.kda_attn_prefill
    f.argtypes = [V] * 5 + [I, I, V, V] + [I] * 5 + [I64] * 4 + [I, F, V, SZ, U64]
    names = "q k v o lse tq tk cq ck n h hk hd dt qs ks vs os w sc ws wsb st".split()
    call = caller(f, names, (P, P, P, P, None, 10, 10, None, None, 1, 4, 2, 128, 1, 512, 256, 256,
                             512, 0, 0.1, P, BIG, 0))
    assert call(hd=64) == 2 and call(dt=0) == 2 and call(dt=3) == 1
    assert call(h=5) == 1 and call(h=0) == 1 and call(hk=0) == 1 and call(hk=-2) == 1
    assert call(h=258, hk=2, qs=258 * 128, os=258 * 128) == 2   # more than 128 heads per KV head
    assert call(n=0) == 1 and call(tq=-1) == 1 and call(tk=-1) == 1
    assert call(w=-1) == 1
    assert call(sc=0.0) == 1 and call(sc=-1.0) == 1 and call(sc=float("nan")) == 1
    assert call(sc=float("inf")) == 1
    assert call(cq=P) == 1 and call(ck=P) == 1                  # they come together
    for p in "qkvo":
        assert call(**{p: None}) == 1 and b"null" in lib.kda_last_error()
        assert call(**{p: ODD}) == 1 and b"aligned" in lib.kda_last_error()
    assert call(qs=508) == 1 and call(qs=516) == 1 and call(ks=248) == 1 and call(os=384) == 1
    assert call(tq=1 << 30, n=4) == 1                           # rows past 2^31
    assert call(wsb=0) == 3 and call(ws=None) == 3 and call(ws=ODD) == 1
    assert call(tq=0, q=None, k=None, v=None, o=None, ws=None) == 0  # no rows: nothing to do
    assert b"kda_attn_prefill" in lib.kda_last_error()


def test_rows_refusals(lib):
    names = "k v ks vs t cu n hk hd dt c np pg tb mp ln st".split()
    for name in ("kda_attn_kv4_append", "kda_attn_kv4_read"):
        f = getattr(lib, name)
        f.argtypes = [V, V, I64, I64, I, V, I, I, I, I, V, I64, I, V, I, V, U64]
        call = caller(f, names, (P, P, 256, 256, 4, None, 2, 2, 128, 1, P, 9, 64, P, 3, P, 0))
        assert call(hd=64) == 2 and call(dt=0) == 2 and call(dt=9) == 1
        assert call(pg=8) == 2 and call(pg=48) == 2 and call(pg=512) == 2
        assert call(n=0) == 1 and call(hk=0) == 1 and call(np=0) == 1 and call(mp=0) == 1
        assert call(mp=1 << 26) == 1                            # positions past 2^31
        assert call(t=-1) == 1
        for p in ("k", "v", "c", "tb", "ln"):
            assert call(**{p: None}) == 1 and b"null" in lib.kda_last_error()
        for p in ("k", "v", "c"):
            assert call(**{p: ODD}) == 1 and b"aligned" in lib.kda_last_error()
        assert call(tb=V(P.value + 2)) == 1 and call(ln=V(P.value + 2)) == 1
        assert call(ks=248) == 1 and call(vs=260) == 1
        assert call(t=0, k=None, v=None) == 0
        assert name.encode() in lib.kda_last_error()


def test_decode_refusals(lib):
    f = lib.kda_attn_kv4_decode
    f.argtypes = [V, V, I64, I, V, I, V, V, V] + [I] * 7 + [F, V, SZ, U64]
    names = "q c np pg tb mp ln o lse n k h hk hd dt w sc ws wsb st".split()
    call = caller(f, names, (P, P, 9, 64, P, 3, P, P, None, 2, 1, 4, 2, 128, 1, 0, 0.1, P, BIG, 0))
    assert call(hd=64) == 2 and call(dt=0) == 2 and call(dt=7) == 1 and call(pg=65) == 2
    assert call(k=0) == 1 and call(k=9) == 1
    assert call(h=3) == 1 and call(h=0) == 1 and call(hk=0) == 1 and call(n=0) == 1
    assert call(w=-1) == 1 and call(sc=0.0) == 1 and call(sc=float("inf")) == 1
    for p in ("q", "o", "c", "tb", "ln"):
        assert call(**{p: None}) == 1
    for p in ("q", "o", "c"):
        assert call(**{p: ODD}) == 1
    assert call(wsb=0) == 3 and call(ws=None) == 3 and call(ws=ODD) == 1
    assert b"kda_attn_kv4_decode" in lib.kda_last_error()


def test_workspace_sizes(lib):
    f = lib.kda_attn_prefill_workspace_size
    f.restype, f.argtypes = SZ, [I64, I, I, I]
    assert f(100, 1, 4, 2) > 0 and f(100000, 16, 32, 8) >= f(100, 16, 32, 8)
    assert f(-1, 1, 4, 2) == 0 and f(10, 0, 4, 2) == 0 and f(10, 1, 3, 2) == 0
    g = lib.kda_attn_kv4_workspace_size
    g.restype, g.argtypes = SZ, [I] * 4
    assert g(1, 1, 4, 2) > 0 and g(64, 8, 32, 8) >= g(64, 1, 32, 8)
    assert g(0, 1, 4, 2) == 0 and g(1, 9, 4, 2) == 0 and g(1, 1, 3, 2) == 0


def test_injected_launch_failure(lib, monkeypatch):
    monkeypatch.setenv("KDA_FAULT_INJECT", "launch")
    f = lib.kda_attn_kv4_append
    f.argtypes = [V, V, I64, I64, I, V, I, I, I, I, V, I64, I, V, I, V, U64]
    assert f(P, P, 256, 256, 4, None, 2, 2, 128, 1, P, 9, 64, P, 3, P, 0) == 4
    assert b"injected" in lib.kda_last_error()


def test_host_cache_layout_is_a_bijection():
    """The documented layout gives every code of a group its own four bits, and every byte one
    token."""
    from _attn import place
    for which in "kv":
        seen, owner = set(), {}
        for tok in range(16):
            for ch in range(128):
                at = place(which, tok, ch)
                assert 0 <= at[0] < 1024 and at not in seen
                seen.add(at)
                assert owner.setdefault(at[0], tok) == tok
        assert len(seen) == 2048


def test_quantise_error_is_half_a_step():
    from _attn import quantise
    import torch
    x = torch.randn((50, 2, 128), generator=torch.Generator().manual_seed(0)) * 3 + 1
    x = x.to(torch.bfloat16).double().numpy()
    c, s, m = quantise(x)
    back = m[..., None] + s[..., None] * c.reshape(50, 2, 2, 64)
    err = np.abs(back - x.reshape(back.shape))
    assert (err <= s[..., None] / 2 + 1e-12).all() and c.max() == 15 and c.min() == 0
