"""Linear attention, rotary positions and the page calls refuse bad arguments before anything
reaches the device."""

import ctypes
import random

import pytest

V, I, F, U64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint64, ctypes.c_size_t
I64 = ctypes.c_int64
BUF = ctypes.create_string_buffer(64)
P = ctypes.cast(ctypes.addressof(BUF) + (16 - ctypes.addressof(BUF) % 16) % 16, V)
P2 = V(P.value + 16)
ODD = V(P.value + 8)
ODDER = V(P.value + 2)
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


def rows_refusals(lib, call):
    assert call(hd=64) == 2 and call(dt=0) == 2 and call(dt=3) == 1
    assert call(n=0) == 1 and call(h=0) == 1 and call(hq=0) == 1 and call(h=5) == 1
    assert call(sc=float("nan")) == 1 and call(sc=float("inf")) == 1
    for p in ("q", "k", "v", "o", "g"):
        assert call(**{p: None}) == 1 and b"null" in lib.kda_last_error()
    for p in ("q", "k", "v", "o", "si", "so"):
        assert call(**{p: ODD}) == 1 and b"aligned" in lib.kda_last_error()
    assert call(g=ODDER) == 1
    assert call(qs=248) == 1 and call(ks=260) == 1 and call(vs=504) == 1 and call(os=508) == 1
    assert call(gs=3) == 1 and call(gs=-4) == 1


def test_lin_prefill_refusals(lib):
    f = lib.kda_lin_prefill
    f.argtypes = [V] * 7 + [I, I, V] + [I] * 5 + [I64] * 5 + [F, V, SZ, U64]
    names = "si so q k v g o t tp cu n h hq hd dt qs ks vs gs os sc ws wsb st".split()
    call = caller(f, names, (P, P, P, P, P, P, P, 20, 20, None, 1, 4, 2, 128, 1, 256, 256, 512, 4,
                             512, 0.1, P, BIG, 0))
    rows_refusals(lib, call)
    assert call(t=-1) == 1 and call(t=21) == 1 and call(cu=P, tp=30) == 1 and call(cu=ODDER) == 1
    assert call(t=1 << 30, tp=1 << 30, n=4) == 1                # rows past 2^31
    assert call(wsb=0) == 3 and call(ws=None) == 3 and call(ws=ODD) == 1
    assert b"kda_lin_prefill" in lib.kda_last_error()


def test_lin_decode_refusals(lib):
    f = lib.kda_lin_decode
    f.argtypes = [V] * 7 + [I] * 6 + [I64] * 5 + [F, V, I, U64]
    names = "si so q k v g o n kr h hq hd dt qs ks vs gs os sc sn ns st".split()
    snaps = (V * 2)(P2, P2)
    call = caller(f, names, (P, P, P, P, P, P, P, 1, 2, 4, 2, 128, 1, 256, 256, 512, 4, 512, 0.1,
                             None, 0, 0))
    rows_refusals(lib, call)
    assert call(kr=0) == 1 and call(kr=9) == 1
    assert call(ns=1) == 1 and call(sn=snaps, ns=3) == 1 and call(sn=snaps, ns=-1) == 1
    assert call(sn=(V * 2)(P2, None), ns=2) == 1 and call(sn=(V * 2)(P2, ODD), ns=2) == 1
    assert call(sn=(V * 2)(P2, P), ns=2) == 1 and b"alias" in lib.kda_last_error()
    assert b"kda_lin_decode" in lib.kda_last_error()


def test_rope_refusals(lib):
    f = lib.kda_attn_rope
    f.argtypes = [V] * 4 + [I64] + [I] * 4 + [I64] * 4 + [V, I, V, I, V, I, F, U64]
    names = "q k qo ko r h hk hd dt qs ks qos kos pos ax fr np pa il fa st".split()
    axis = (ctypes.c_uint8 * 64)(*([0, 1] * 32))
    call = caller(f, names, (P, P, P2, P2, 5, 4, 2, 128, 1, 512, 256, 512, 256, P, 2, P, 64, axis, 0,
                             1.0, 0))
    assert call(hd=64) == 2 and call(dt=0) == 2 and call(dt=5) == 1
    assert call(r=-1) == 1 and call(r=1 << 31) == 1 and call(h=0) == 1 and call(hk=-1) == 1
    assert call(ax=0) == 1 and call(ax=5) == 1 and call(ax=1) == 1 and call(np=0) == 1
    assert call(np=65) == 1 and call(fa=float("inf")) == 1 and call(fa=float("nan")) == 1
    for p in ("q", "k", "qo", "ko", "pos", "fr"):
        assert call(**{p: None}) == 1
    for p in ("q", "k", "qo", "ko"):
        assert call(**{p: ODD}) == 1
    assert call(pos=ODDER) == 1 and call(fr=ODDER) == 1
    assert call(qs=504) == 1 and call(ks=260) == 1 and call(qos=510) == 1 and call(kos=128) == 1
    assert call(qo=P, qos=1024) == 1 and b"row stride" in lib.kda_last_error()
    assert call(r=0, q=None, k=None, pos=None) == 0
    assert b"kda_attn_rope" in lib.kda_last_error()


def test_pages_refusals(lib):
    f = lib.kda_attn_kv4_resize
    f.argtypes = [V] * 3 + [I, I, I64, I, V, SZ, U64]
    resize = caller(f, "tb ln rf n mp np pg ws wsb st".split(), (P, P, P, 3, 4, 9, 64, P, BIG, 0))
    f = lib.kda_attn_kv4_fork
    f.argtypes = [V] * 10 + [I, I, I64, I, V, SZ, U64]
    fork = caller(f, "tb ln rf pa to lo ro sr ds ct n mp np pg ws wsb st".split(),
                  (P,) * 10 + (3, 4, 9, 64, P, BIG, 0))
    f = lib.kda_attn_kv4_compact
    f.argtypes = [V] * 7 + [I, I, I64, V, SZ, U64]
    compact = caller(f, "tb rf to ro sr ds ct n mp np ws wsb st".split(),
                     (P,) * 7 + (3, 4, 9, P, BIG, 0))
    for call, arrays in ((resize, "tb ln rf"), (fork, "tb ln rf pa to lo ro sr ds ct"),
                         (compact, "tb rf to ro sr ds ct")):
        for p in arrays.split():
            assert call(**{p: None}) == 1 and b"null" in lib.kda_last_error()
            assert call(**{p: ODDER}) == 1 and b"aligned" in lib.kda_last_error()
        assert call(n=0) == 1 and call(mp=0) == 1 and call(np=0) == 1 and call(np=1 << 31) == 1
        assert call(n=1 << 16, mp=1 << 15) == 1                 # a table past 2^31 entries
        assert call(ws=None) == 3 and call(wsb=16) == 3 and call(ws=ODD) == 1
    for call in (resize, fork):
        assert call(pg=8) == 2 and call(pg=48) == 2 and call(mp=1 << 26) == 1


def test_copy_refusals(lib):
    f = lib.kda_attn_kv4_copy
    f.argtypes = [V, I, I64, I, I, V, V, V, I, U64]
    caches = (V * 129)(*[P.value] * 129)
    call = caller(f, "c n np pg hk sr ds ct mx st".split(), (caches, 2, 9, 64, 2, P, P, P, 4, 0))
    assert call(n=0) == 1 and call(n=129) == 1 and call(c=None) == 1 and call(mx=-1) == 1
    assert call(np=0) == 1 and call(hk=0) == 1 and call(pg=8) == 2
    assert call(c=(V * 2)(P, None)) == 1 and call(c=(V * 2)(P, ODD)) == 1
    for p in ("sr", "ds", "ct"):
        assert call(**{p: None}) == 1 and call(**{p: ODDER}) == 1
    assert call(mx=0) == 0


def test_workspace_sizes(lib):
    f = lib.kda_lin_prefill_workspace_size
    f.restype, f.argtypes = SZ, [I64, I, I]
    assert f(100, 1, 4) > 0 and f(0, 1, 1) > 0 and f(100000, 16, 32) >= f(100, 16, 32)
    assert f(-1, 1, 4) == 0 and f(10, 0, 4) == 0 and f(10, 1, 0) == 0 and f(1 << 31, 1, 1) == 0
    g = lib.kda_attn_kv4_pages_workspace_size
    g.restype, g.argtypes = SZ, [I64, I, I]
    assert g(1, 1, 1) > 0 and g(1000, 10, 10) > g(100, 10, 10)
    assert g(0, 1, 1) == 0 and g(1, 0, 1) == 0 and g(1, 1, 0) == 0 and g(1 << 31, 1, 1) == 0
    assert g(10, 1 << 16, 1 << 15) == 0


def test_injected_launch_failure(lib, monkeypatch):
    monkeypatch.setenv("KDA_FAULT_INJECT", "launch")
    f = lib.kda_lin_decode
    f.argtypes = [V] * 7 + [I] * 6 + [I64] * 5 + [F, V, I, U64]
    assert f(P, P, P, P, P, P, P, 1, 2, 4, 2, 128, 1, 256, 256, 512, 4, 512, 0.1, None, 0, 0) == 4
    assert b"injected" in lib.kda_last_error()


def test_host_pages_keep_their_counts():
    """The page calls' plain forms: every page is named as often as it is counted, forks keep
    contents apart, and compacting leaves no holes."""
    import _pages
    for seed in range(20):
        table, lens, refs, r = _pages.some_state(seed, 12, 6, 60, 16, 0.7)
        kept = list(refs)
        for row in table:
            for v in row:
                if v >= 0:
                    kept[v] -= 1
        parent = [r.choice([-1, n, r.randrange(12)]) for n in range(12)]
        table, lens, pairs, _ = _pages.fork(table, lens, refs, parent, 16)
        assert len({d for _, d in pairs}) == len(pairs)
        assert not {s for s, _ in pairs} & {d for _, d in pairs}
        lens = [max(0, n - random.Random(seed).randint(0, 20)) for n in lens]
        _pages.resize(table, lens, refs, 16)
        named = [0] * 60
        for row in table:
            for v in row:
                if v >= 0:
                    named[v] += 1
        assert [a + b for a, b in zip(named, kept)] == refs and min(refs) >= 0
        table, _ = _pages.compact(table, refs)
        used = sum(x > 0 for x in refs)
        assert all(x > 0 for x in refs[:used]) and max(v for row in table for v in row) < used
