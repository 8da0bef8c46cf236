"""What a hybrid decoder's serving step needs next to the KDA core and the full-attention calls,
case by case: linear attention with a decay for each head (prompts, and rows of a decode step),
rotary positions with several axes, and the pages of the 4-bit cache when sequences are forked,
grow, end, or are moved together.

``run`` computes a case in plain torch operations, or with the library's calls where ``own``
is true.  ``exact`` computes it in 64 bits, written apart.

Linear attention.  Per head a state S [128 key channels, 128 value channels]:
    S_t = exp(g_t) S_{t-1} + k_t v_t^T,      o_t = scale * q_t^T S_t
with one g per token and head, or one per head.  Value heads share the q and k heads in groups.

Rotary positions.  Pair p of a head turns by positions[row, axis of p] * inv_freq[p].

Pages.  page_table [sequences, width] names the pages of each sequence (-1: none), refs counts
how often each page is named.  Forking: sequence n goes on from sequence parent[n] (-1: it ends),
sharing its pages but for a last one that is partly filled, which the first child keeps and each
other one gets a copy of.  Resizing: each sequence holds the pages that its length takes.
Compacting: the pages in use become the lowest-numbered ones.  New pages are the
lowest-numbered free ones.
"""

import math
import random

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
CHUNK = 128          # of the plain form of linear attention
TOKEN_BYTES = 144    # of one token and KV head in the 4-bit cache
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The smallest prompt: 64 tokens on 2 heads, where latency is all.
        dict(name="lin_prompt_T64_H2", op="prompt", n=1, lo=64, hi=64, heads=2, qk=2, gate="token",
             state="none", dtype="bf16", lengths=0),
        # The prefill workload: one prompt of 8192 tokens on 32 heads, behind a carried state.
        dict(name="lin_prompt_T8192_H32", op="prompt", n=1, lo=8192, hi=8192, heads=32, qk=32,
             gate="token", state="carried", dtype="bf16", lengths=1),
        # The front end's packed batch: 16 prompts of 512 to 8192 tokens.
        dict(name="lin_prompt_16seq_512to8192", op="prompt", n=16, lo=512, hi=8192, heads=32,
             qk=32, gate="token", state="none", dtype="bf16", lengths=2),
        # Ragged prompts down to one token behind carried states; five value heads to a key head,
        # a fixed decay for each head.
        dict(name="lin_prompt_7seq_H20", op="prompt", n=7, lo=1, hi=4001, heads=20, qk=4,
             gate="head", state="carried", dtype="fp16", lengths=3),
        # The decode workload: 64 sequences, one token each.
        dict(name="lin_decode_N64", op="decode", n=64, rows=1, snaps=0, heads=32, qk=32,
             gate="token", dtype="bf16"),
        # Speculative verification of a few users: 4 rows, the state kept after each.
        dict(name="lin_decode_N3_k4", op="decode", n=3, rows=4, snaps=4, heads=16, qk=8,
             gate="token", dtype="fp16"),
        # Positions of one decode step of 64 sequences far into their documents.
        dict(name="rope_N64", op="rope", rows=64, heads=32, kv=8, axes=1, turned=128,
             interleaved=False, reach=1000000, dtype="bf16"),
        # The front end's batch with video in it: time, height and width, half of each head turned.
        dict(name="rope_69000_video", op="rope", rows=69001, heads=32, kv=8, axes=3, turned=64,
             interleaved=True, reach=20000, dtype="bf16"),
        # A beam search of 4 beams over a short prompt: latency.
        dict(name="fork_4rows", op="fork", groups=1, beams=4, lo=300, hi=300, kv=4, page=16,
             caches=1, lengths=4),
        # 64 prompts of 2000 to 8192 tokens with 8 beams each, the caches of 4 layers.
        dict(name="fork_512rows", op="fork", groups=64, beams=8, lo=2000, hi=8192, kv=8, page=64,
             caches=4, lengths=5),
        # A small pool, two fifths in use.
        dict(name="compact_250pages", op="compact", pages=250, used=0.4, n=9, kv=2, page=32,
             caches=1, lengths=6),
        # A pool of 1.2 GB a layer, a third in use after most sequences ended, two layers.
        dict(name="compact_16000pages", op="compact", pages=16001, used=0.33, n=64, kv=8, page=64,
             caches=2, lengths=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), work(c)["bytes"])
    while True:
        c = dict(op=rng.choice(["prompt", "prompt", "prompt", "decode", "decode", "rope", "fork",
                                "compact"]))
        if c["op"] in ("prompt", "decode"):
            c["qk"] = rng.choice([1, 2, 3, 4, 8, 16, 32])
            c["heads"] = c["qk"] * rng.choice([1, 1, 1, 2, 3, 4, 5])
            c["gate"] = rng.choice(["token", "token", "head"])
        if c["op"] in ("prompt", "decode", "rope"):
            c["dtype"] = rng.choice(["bf16", "fp16"])
        if c["op"] == "prompt":
            c["n"], c["hi"] = _log(rng, 1, 64), _log(rng, 1, 16384)
            c["lo"] = max(1, int(c["hi"] * rng.choice([0.02, 0.3, 1.0])))
            c["state"] = rng.choice(["none", "carried"])
        elif c["op"] == "decode":
            c["n"], c["rows"] = _log(rng, 1, 256), rng.choice([1, 1, 2, 3, 4, 5, 8])
            c["snaps"] = rng.choice([0, c["rows"]])
        elif c["op"] == "rope":
            c["kv"] = rng.choice([1, 2, 3, 4, 8])
            c["rows"], c["heads"] = _log(rng, 1, 100000), c["kv"] * rng.choice([1, 4, 5, 8])
            c["axes"], c["turned"] = rng.choice([1, 1, 2, 3]), rng.choice([128, 128, 96, 64, 22])
            c["interleaved"], c["reach"] = rng.random() < 0.5, _log(rng, 1, 2000000)
        else:
            c["kv"], c["page"] = rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128])
            c["caches"] = rng.choice([1, 2, 5])
        if c["op"] == "fork":
            c["groups"], c["beams"] = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 8, 16])
            c["hi"] = _log(rng, 1, 8192)
            c["lo"] = max(1, int(c["hi"] * rng.choice([0.1, 1.0])))
        if c["op"] == "compact":
            c["pages"], c["used"] = _log(rng, 20, 50000), rng.choice([0.05, 0.3, 0.6, 0.95])
            c["n"] = _log(rng, 1, 200)
        if c["op"] in ("prompt", "fork", "compact"):
            c["lengths"] = rng.randrange(1, 1 << 30)
        if work(c)["bytes"] <= most[c["op"]]:
            return c


def _between(lengths, salt, n, lo, hi):
    r = random.Random(1000003 * lengths + salt)
    return [r.randint(lo, hi) for _ in range(n)]


def _prompt_lens(c):
    return _between(c["lengths"], 1, c["n"], c["lo"], c["hi"])


def _beam_lens(c):
    """Of each group: the prompt's tokens, and those of each beam behind it."""
    prompt = _between(c["lengths"], 1, c["groups"], c["lo"], c["hi"])
    return prompt, _between(c["lengths"], 2, c["groups"], 1, 200)


def _beam_parents(c):
    """The beam that each beam goes on from; one in twenty ends."""
    r = random.Random(1000003 * c["lengths"] + 3)
    b = c["beams"]
    return [-1 if r.random() < 0.05 else n // b * b + r.randrange(b)
            for n in range(c["groups"] * b)]


def _copied(c):
    """Pages that a fork copies: a partly filled one for each child but the first."""
    prompt, more = _beam_lens(c)
    seen, count = set(), 0
    for p in _beam_parents(c):
        if p >= 0 and p in seen:
            g = p // c["beams"]
            count += (prompt[g] + more[g]) % c["page"] != 0
        seen.add(p)
    return count


def _pool(c):
    """Pages of a fork's pool, and the table's width."""
    page = c["page"]
    prompt, more = _beam_lens(c)
    need = sum(p // page + c["beams"] * (-(-(p + m) // page) - p // page)
               for p, m in zip(prompt, more))
    rows = c["groups"] * c["beams"]
    return need + need // 4 + 2 * rows + 1, -(-(c["hi"] + 200) // page) + 2


def _moved(c):
    """Pages that compacting moves: those in use past the number of pages in use."""
    r = random.Random(1000003 * c["lengths"] + 4)
    used = sorted(r.sample(range(c["pages"]), max(1, int(c["pages"] * c["used"]))))
    return used, sum(p >= len(used) for p in used)


def work(c):
    if c["op"] in ("prompt", "decode"):
        rows = sum(_prompt_lens(c)) if c["op"] == "prompt" else c["n"] * c["rows"]
        states = 2 if c["op"] == "decode" or c["state"] == "carried" else 1
        if c["op"] == "decode":
            states += c["snaps"]
        gates = rows * c["heads"] * 4 if c["gate"] == "token" else c["heads"] * 4
        return {"bytes": rows * 2 * D * 2 * (c["qk"] + c["heads"]) + gates
                + states * c["n"] * c["heads"] * D * D * 4,
                "flops": 4 * D * D * rows * c["heads"]}
    if c["op"] == "rope":
        each = c["rows"] * (c["heads"] + c["kv"]) * D
        return {"bytes": 4 * each + 4 * c["rows"] * c["axes"], "flops": 3 * each}
    if c["op"] == "fork":
        pages, width = _pool(c)
        moved, ints = _copied(c), 2 * c["groups"] * c["beams"] * width + 2 * pages
    else:
        moved, ints = _moved(c)[1], 4 * c["pages"]
    block = c["kv"] * c["page"] * TOKEN_BYTES
    return {"bytes": 2 * moved * c["caches"] * block + 4 * ints, "flops": 0}


# ------------------------------------------------------------------ inputs

def _cu(rows, device):
    return torch.tensor([0] + rows, dtype=torch.int64).cumsum(0).to(torch.int32).to(device)


def _lin_inputs(st, c, g, rows, dev):
    """q and k of unit length as the front end leaves them, v of unit spread; heads that forget
    within a few tokens and heads that hardly forget."""
    dt = TYPES[c["dtype"]]

    def unit(heads):
        x = torch.randn((rows, heads, D), generator=g, device=dev)
        return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dt)

    # k and v lie side by side, as one projection gives them
    kv = torch.cat([unit(c["qk"]), torch.randn((rows, c["heads"], D), generator=g,
                                               device=dev).to(dt)], 1)
    st["q"] = unit(c["qk"])
    st["k"], st["v"] = kv[:, :c["qk"]], kv[:, c["qk"]:]
    rate = torch.exp2(-9 * torch.rand(c["heads"], generator=g, device=dev))
    st["g"] = -rate
    if c["gate"] == "token":
        x = torch.randn((rows, c["heads"]), generator=g, device=dev)
        st["g"] = -rate * torch.log1p(torch.exp(x))
    st["o"] = torch.empty((rows, c["heads"], D), dtype=dt, device=dev)
    shape = (c["n"], c["heads"], D, D)
    st["state"] = None
    if c.get("state") != "none":
        st["state"] = torch.randn(shape, generator=g, device=dev) * 0.3
    st["state_out"] = torch.empty(shape, device=dev)


def _cache(c, g, pages, dev):
    """The caches of some layers, parameters and codes as an append leaves them."""
    kv, page = c["kv"], c["page"]
    caches = []
    for _ in range(c["caches"]):
        cache = torch.randint(0, 256, (pages, kv, page * TOKEN_BYTES), generator=g, device=dev,
                              dtype=torch.uint8)
        for at in (page * 64, page * 136):
            par = cache[:, :, at:at + page * 8].unflatten(2, (page * 2, 4))
            par.copy_(torch.randn((pages, kv, page * 2, 2), generator=g, device=dev)
                      .to(torch.bfloat16).view(torch.uint8))
        caches.append(cache)
    return caches


def _beams(c, order):
    """The page table of a beam search: prompt pages that a group shares, then pages of each
    beam; and how often each page is named."""
    page, (pages, width) = c["page"], _pool(c)
    table = torch.full((c["groups"] * c["beams"], width), -1, dtype=torch.int32)
    lens, at, n = [], 0, 0
    for p, m in zip(*_beam_lens(c)):
        shared, all_ = p // page, -(-(p + m) // page)
        prompt = order[at:at + shared]
        at += shared
        for _ in range(c["beams"]):
            table[n, :shared] = prompt
            table[n, shared:all_] = order[at:at + all_ - shared]
            at, n = at + all_ - shared, n + 1
            lens.append(p + m)
    refs = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
    return table, refs, torch.tensor(lens, dtype=torch.int32)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 29)
    st = dict(c)
    if c["op"] == "prompt":
        lens = _prompt_lens(c)
        _lin_inputs(st, c, g, sum(lens), dev)
        st["lens"], st["cu"] = lens, _cu(lens, dev)
    elif c["op"] == "decode":
        _lin_inputs(st, c, g, c["n"] * c["rows"], dev)
        for name in ("q", "k", "v", "o"):
            st[name] = st[name].unflatten(0, (c["n"], c["rows"]))
        if c["gate"] == "token":
            st["g"] = st["g"].unflatten(0, (c["n"], c["rows"]))
        st["after"] = [torch.empty_like(st["state"]) for _ in range(c["snaps"])]
    elif c["op"] == "rope":
        dt, shape = TYPES[c["dtype"]], (c["rows"], c["heads"] + c["kv"], D)
        # one projection's output, v's heads left out
        x = torch.randn(shape, generator=g, device=dev).to(dt)
        st["q"], st["k"] = x[:, :c["heads"]], x[:, c["heads"]:]
        st["q_out"], st["k_out"] = (torch.empty_like(y, memory_format=torch.contiguous_format)
                                    for y in (st["q"], st["k"]))
        st["pos"] = torch.randint(0, c["reach"], (c["rows"], c["axes"]), generator=g, device=dev,
                                  dtype=torch.int32)
        pairs = c["turned"] // 2
        p = torch.arange(pairs, device=dev, dtype=torch.float64)
        st["inv_freq"] = torch.pow(10000.0, -p / pairs).float()
        st["pair_axis"] = [i * c["axes"] // pairs for i in range(pairs)]
    elif c["op"] == "fork":
        pages, width = _pool(c)
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
        table, refs, lens = _beams(c, order)
        st["table"], st["refs"], st["lens_t"] = table.to(dev), refs.to(dev), lens.to(dev)
        st["parent"] = torch.tensor(_beam_parents(c), dtype=torch.int32, device=dev)
        st["caches"] = _cache(c, g, pages, dev)
        for name in ("table", "refs", "lens_t"):
            st[name + "_out"] = torch.empty_like(st[name])
        st["src"], st["dst"] = (torch.empty_like(st["lens_t"]) for _ in range(2))
        st["count"] = torch.empty(1, dtype=torch.int32, device=dev)
    else:
        used, _ = _moved(c)
        order = torch.tensor(used, dtype=torch.int32, device=dev)
        order = order[torch.randperm(len(used), generator=g, device=dev)]
        width = -(-len(used) // c["n"]) + 1
        st["table"] = torch.full((c["n"], width), -1, dtype=torch.int32, device=dev)
        at = torch.arange(len(used), device=dev)
        st["table"][at % c["n"], at // c["n"]] = order
        # sequences name the first page of the first one too: a prefix that they share
        st["table"][:, 0] = torch.where(st["table"][:, 0] >= 0, st["table"][0, 0], -1)
        st["refs"] = torch.zeros(c["pages"], dtype=torch.int32, device=dev)
        named = st["table"][st["table"] >= 0].long()
        st["refs"].index_add_(0, named, torch.ones_like(named, dtype=torch.int32))
        # and pages that no sequence names are kept for later ones
        st["refs"][order.long()] = st["refs"][order.long()].clamp_min(1)
        st["caches"] = _cache(c, g, c["pages"], dev)
        for name in ("table", "refs"):
            st[name + "_out"] = torch.empty_like(st[name])
        st["src"], st["dst"] = (torch.empty(c["pages"] // 2, dtype=torch.int32, device=dev)
                                for _ in range(2))
        st["count"] = torch.empty(1, dtype=torch.int32, device=dev)
    return st


# ------------------------------------------------------------------ the library's calls

def _own(s):
    import gated_delta_rule_prepare_gb300 as K
    if s["op"] == "prompt":
        if "ws" not in s:
            s["ws"] = K.kda_lin_prefill_workspace(s["q"].shape[0], s["n"], s["heads"])
        K.kda_lin_prefill(s["q"], s["k"], s["v"], s["g"], s["o"], state_in=s["state"],
                          state_out=s["state_out"], cu_seqlens=s["cu"], workspace=s["ws"])
        return {"o": s["o"], "state": s["state_out"]}
    if s["op"] == "decode":
        K.kda_lin_decode(s["q"], s["k"], s["v"], s["g"], s["o"], s["state"], s["state_out"],
                         snapshots=s["after"])
        return {"o": s["o"], "state": s["state_out"], "after": s["after"]}
    if s["op"] == "rope":
        K.kda_attn_rope(s["q"], s["k"], s["pos"], s["inv_freq"], s["q_out"], s["k_out"],
                        pair_axis=s["pair_axis"], interleaved=s["interleaved"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if "ws" not in s:
        s["ws"] = K.kda_attn_kv4_pages_workspace(s["refs"].numel(), s["table"].shape[0],
                                                 s["table"].shape[1])
    lists = dict(src=s["src"], dst=s["dst"], count=s["count"], workspace=s["ws"])
    if s["op"] == "fork":
        K.kda_attn_kv4_fork(s["table"], s["lens_t"], s["refs"], s["parent"], s["table_out"],
                            s["lens_t_out"], s["refs_out"], page=s["page"], **lists)
        K.kda_attn_kv4_copy(s["caches"], s["src"], s["dst"], s["count"])
        lens = s["lens_t_out"] + 1
        K.kda_attn_kv4_resize(s["table_out"], lens, s["refs_out"], page=s["page"],
                              workspace=s["ws"])
    else:
        K.kda_attn_kv4_compact(s["table"], s["refs"], s["table_out"], s["refs_out"], **lists)
        K.kda_attn_kv4_copy(s["caches"], s["src"], s["dst"], s["count"])
    return _pages_out(s)


def _pages_out(s):
    out = {"table": s["table_out"], "refs": s["refs_out"], "src": s["src"], "dst": s["dst"],
           "count": s["count"], "caches": s["caches"]}
    if s["op"] == "fork":
        out["lens"] = s["lens_t_out"]
    return out


# ------------------------------------------------------------------ plain torch operations

def _chunks(s):
    """Rows of each chunk [K, C], which of them are there, each chunk's sequence, and the first
    chunk of each sequence [n + 1]."""
    lens = (s["cu"][1:] - s["cu"][:-1]).long()
    count = (lens + CHUNK - 1) // CHUNK
    first = torch.cat([count.new_zeros(1), count.cumsum(0)])
    total = sum(-(-x // CHUNK) for x in s["lens"])
    seq = torch.repeat_interleave(torch.arange(s["n"], device=lens.device), count,
                                  output_size=total)
    at = (torch.arange(total, device=lens.device) - first[seq])[:, None] * CHUNK
    at = at + torch.arange(CHUNK, device=lens.device)
    ok = at < lens[seq][:, None]
    return s["cu"][seq].long()[:, None] + torch.where(ok, at, 0), ok, seq, first


def _plain_prompt(s):
    rows, ok, seq, first = _chunks(s)
    G, C = s["heads"] // s["qk"], CHUNK

    def chunked(x, share):            # [rows, h, 128] to [heads, K, C, 128], absent rows zero
        y = torch.where(ok[:, :, None, None], x[rows].float(), 0.0).permute(2, 0, 1, 3)
        return y.repeat_interleave(share, 0)

    q, k, v = chunked(s["q"], G), chunked(s["k"], G), chunked(s["v"], 1)
    g = s["g"].double().expand(s["q"].shape[0], s["heads"])
    g = torch.where(ok[:, :, None], g[rows], 0.0).permute(2, 0, 1)       # [heads, K, C]
    cum = g.cumsum(2)
    total = cum[:, :, -1]
    # within chunks
    causal = torch.ones((C, C), dtype=torch.bool, device=q.device).tril()
    w = torch.where(causal, cum[:, :, :, None] - cum[:, :, None], -math.inf).exp().float()
    o = torch.matmul(torch.matmul(q, k.transpose(2, 3)).mul_(w), v)
    del w
    # what each chunk adds to the state, and the states in front of the chunks
    k = k * (total[:, :, None] - cum).exp().float()[..., None]
    add = torch.matmul(k.transpose(2, 3), v).flatten(2)                  # [heads, K, 128 * 128]
    run = torch.cat([total.new_zeros((s["heads"], 1)), total.cumsum(1)], 1)
    same = seq[:, None] == seq
    before = same.tril(-1)
    w = torch.where(before, run[:, :-1, None] - run[:, None, 1:], -math.inf).exp().float()
    start = torch.matmul(w, add)
    n = torch.arange(s["n"], device=q.device)
    w = torch.where(n[:, None] == seq, run[:, first[1:], None] - run[:, None, 1:], -math.inf)
    last = torch.matmul(w.exp().float(), add)                            # [heads, n, 128 * 128]
    if s["state"] is not None:
        s0 = s["state"].transpose(0, 1).flatten(2)
        start += (run[:, :-1] - run[:, first[:-1]][:, seq]).exp().float()[..., None] * s0[:, seq]
        last += (run[:, first[1:]] - run[:, first[:-1]]).exp().float()[..., None] * s0
    o += torch.matmul(q, start.unflatten(2, (D, D))) * cum.exp().float()[..., None]
    s["o"][rows[ok]] = (o * SCALE).permute(1, 2, 0, 3)[ok].to(s["o"].dtype)
    s["state_out"].copy_(last.unflatten(2, (D, D)).transpose(0, 1))
    return {"o": s["o"], "state": s["state_out"]}


def _plain_decode(s):
    G = s["heads"] // s["qk"]
    S = s["state"].clone()
    g = s["g"].expand(s["n"], s["rows"], s["heads"])
    for t in range(s["rows"]):
        q, k = (s[x][:, t].float().repeat_interleave(G, 1) for x in ("q", "k"))
        S = S * g[:, t].exp()[..., None, None] + k[..., :, None] * s["v"][:, t].float()[..., None, :]
        s["o"][:, t] = ((q * SCALE)[..., :, None] * S).sum(2).to(s["o"].dtype)
        if t < s["snaps"]:
            s["after"][t].copy_(S)
    s["state_out"].copy_(S)
    return {"o": s["o"], "state": s["state_out"], "after": s["after"]}


def _plain_rope(s):
    axis = torch.tensor(s["pair_axis"], device=s["pos"].device)
    # angles of far positions have few bits left in 32
    angle = s["pos"][:, axis].double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = s["turned"]
    for name in ("q", "k"):
        x, y = s[name].float(), s[name + "_out"]
        if s["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
        else:
            a, b = x[..., :r // 2], x[..., r // 2:r]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
        y.copy_(torch.cat([turned, x[..., r:]], 2))
    return {"q": s["q_out"], "k": s["k_out"]}


def _named(refs, entries, by):
    """refs with `by` for each entry that names a page."""
    there = entries >= 0
    return refs.index_add_(0, entries.clamp_min(0).flatten().long(),
                           (there.to(torch.int32) * by).flatten())


def _free_pages(refs, wanted):
    """The lowest-numbered free pages for the places where `wanted`, in their order; -1 where
    there are no more."""
    order = torch.sort((refs > 0).to(torch.int8), stable=True)[1].to(torch.int32)
    rank = wanted.flatten().long().cumsum(0).view(wanted.shape) - 1
    got = order[rank.clamp(0, refs.numel() - 1)]
    return torch.where(wanted & (rank < (refs <= 0).sum()), got, -1)


def _listed_pairs(s, keep, src, dst):
    """The pairs where `keep`, in order, into the lists; -1 behind them."""
    n = s["src"].numel()
    order = torch.sort((~keep).to(torch.int8), stable=True)[1][:n]
    s["count"].copy_(keep.sum().to(torch.int32))
    for name, x in (("src", src), ("dst", dst)):
        s[name].fill_(-1)
        s[name][:order.numel()] = torch.where(keep[order], x[order], -1)


def _plain_copy(s):
    n = int(s["count"])
    src, dst = s["src"][:n].long(), s["dst"][:n].long()
    for cache in s["caches"]:
        cache[dst] = cache[src]


def _plain_fork(s):
    page, table, rows = s["page"], s["table"], s["table"].shape[0]
    entry = torch.arange(table.shape[1], device=table.device)
    n = torch.arange(rows, device=table.device, dtype=torch.int32)
    live = s["parent"] >= 0
    p = s["parent"].clamp_min(0).long()
    lens = torch.where(live, s["lens_t"][p], 0)
    held = (lens + page - 1) // page
    new = torch.where(entry < held[:, None], table[p], -1)
    first = torch.full_like(n, rows)
    first.scatter_reduce_(0, p, torch.where(live, n, rows), "amin")
    copied = live & (lens % page != 0) & (first[p] != n)
    at_copy = copied[:, None] & (entry == held[:, None] - 1)
    refs = _named(s["refs"].clone(), table, -1)
    refs = _named(refs, torch.where(at_copy, -1, new), 1)
    got = _free_pages(refs, copied)
    src = torch.where(at_copy, new, 0).sum(1).to(torch.int32)
    new = torch.where(at_copy, got[:, None], new)
    s["table_out"].copy_(new)
    s["refs_out"].copy_(_named(refs, got, 1))
    s["lens_t_out"].copy_(torch.where(copied & (got < 0), lens // page * page, lens))
    _listed_pairs(s, got >= 0, src, got)
    _plain_copy(s)
    # and the pages for one more token of each
    table, refs = s["table_out"], s["refs_out"]
    held = (s["lens_t_out"] + page) // page
    over = torch.where(entry >= held[:, None], table, -1)
    _named(refs, over, -1)
    table[entry >= held[:, None]] = -1
    got = _free_pages(refs, (entry < held[:, None]) & (table < 0))
    table.copy_(torch.where(got >= 0, got, table))
    _named(refs, got, 1)
    return _pages_out(s)


def _plain_compact(s):
    refs = s["refs"]
    at = torch.arange(refs.numel(), device=refs.device, dtype=torch.int32)
    used = refs > 0
    count = used.sum()
    to_move, hole = used & (at >= count), ~used & (at < count)
    movers, holes = at[to_move], at[hole]      # equally many
    place = at.clone()
    place[movers.long()] = holes
    table = s["table"]
    s["table_out"].copy_(torch.where(table >= 0, place[table.clamp_min(0).long()], table))
    s["refs_out"].copy_(torch.where(to_move, 0, refs))
    s["refs_out"][holes.long()] = refs[movers.long()]
    _listed_pairs(s, torch.ones_like(movers, dtype=torch.bool), movers, holes)
    _plain_copy(s)
    return _pages_out(s)


_PLAIN = {"prompt": _plain_prompt, "decode": _plain_decode, "rope": _plain_rope,
          "fork": _plain_fork, "compact": _plain_compact}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ 64 bits

def _walk64(S, q, k, v, g):
    """One token of some chains by the recurrence: S [m, heads, 128, 128] in place."""
    share = S.shape[1] // q.shape[1]
    S.mul_(torch.exp(g)[..., None, None])
    S.add_(torch.einsum("nhi,nhj->nhij", k.repeat_interleave(share, 1), v))
    return torch.einsum("nhi,nhij->nhj", q.repeat_interleave(share, 1), S) / math.sqrt(D)


def _lin64(s, lens):
    """All chains, token by token; the longest sequences first, so that those that go on are the
    first ones."""
    order = sorted(range(len(lens)), key=lambda n: -lens[n])
    start = [0]
    for x in lens:
        start.append(start[-1] + x)
    q, k, v, o = (s[x].reshape(-1, s[x].shape[-2], D) for x in ("q", "k", "v", "o"))
    o = torch.zeros(o.shape, dtype=torch.float64, device=o.device)
    g = s["g"].reshape(-1, s["heads"]).expand(o.shape[0], -1)
    S = torch.zeros(s["state_out"].shape, dtype=torch.float64, device=o.device)
    if s["state"] is not None:
        S = s["state"].double()[order]
    after, left = [], len(order)
    base = torch.tensor([start[n] for n in order], device=o.device)
    for t in range(max(lens)):
        while lens[order[left - 1]] <= t:
            left -= 1
        r = base[:left] + t
        o[r] = _walk64(S[:left], q[r].double(), k[r].double(), v[r].double(), g[r].double())
        if t < s.get("snaps", 0):
            after.append(S.clone())
    back = torch.empty_like(S)
    back[order] = S
    return o, back, after


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None                   # whole numbers and bytes
    s = prepare(case, seed)
    if case["op"] == "prompt":
        o, S, _ = _lin64(s, s["lens"])
        return {"o": o, "state": S}
    if case["op"] == "decode":
        o, S, after = _lin64(s, [case["rows"]] * case["n"])
        return {"o": o.view(s["o"].shape), "state": S, "after": after}
    out, r = {}, case["turned"]
    for name in ("q", "k"):
        y = s[name].double()
        for p in range(r // 2):
            a, b = (2 * p, 2 * p + 1) if case["interleaved"] else (p, p + r // 2)
            by = s["pos"][:, s["pair_axis"][p]].double() * s["inv_freq"][p].double()
            turn = torch.polar(torch.ones_like(by), by)[:, None]
            z = torch.complex(y[:, :, a], y[:, :, b]) * turn
            y[:, :, a], y[:, :, b] = z.real, z.imag
        out[name] = y
    return out
