"""Operators of a 4-bit paged K/V cache and of its pages: the cases they are measured on, and their plain forms.

  write    new key/value rows into the 4-bit cache (a prompt's rows, or one token a sequence), with the metadata of
           the pages they touch, and the rows read back as the values the codes stand for
  decode   attention of one query token a sequence over the 4-bit cache: softmax (alpha = 1) or alpha-entmax, over
           every page or over each head's kept pages
  fork     one beam step of the page table: rows follow their parents, partial last pages are copied, dropped rows
           are freed, and every live row grows by one token
  compact  live blocks move to the low end of the pool and the page table follows
  copy     a list of blocks from one pool to another (a sequence swapped out or in)

Quantisation, per (token, kv head, 64 coordinates): lo = min, s = bf16((max - lo) / 15),
code = clamp(rint(fl(fl(x - lo) * fl(1 / s))), 0, 15), value = fl(s * code + lo), every fl() a rounding to fp32.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 64        # coordinates that share a scale and an offset
TILE = 32         # pages of one metadata tile


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the first answer of a short chat: launch latency is all there is
        dict(name="softmax_short", op="decode", B=1, Hq=8, Hkv=2, d=64, P=16, L=701, alpha=1.0, k=0),
        # a serving batch at mixed lengths
        dict(name="softmax_batch_32k", op="decode", B=8, Hq=32, Hkv=8, d=128, P=32, L=32768, alpha=1.0, k=0),
        # every head its own keys (no grouping), short head dimension
        dict(name="softmax_mha_64k", op="decode", B=2, Hq=32, Hkv=32, d=64, P=32, L=65536, alpha=1.0, k=0),
        # full-cache entmax over long contexts
        dict(name="entmax_128k", op="decode", B=4, Hq=32, Hkv=8, d=128, P=32, L=131072, alpha=1.5, k=0),
        # one very long context of which 2 % of the pages are kept
        dict(name="entmax_1m_kept", op="decode", B=1, Hq=32, Hkv=8, d=128, P=64, L=1048576, alpha=1.5, k=330),
        # a batch of ungrouped heads over a small page budget
        dict(name="entmax_mha_kept", op="decode", B=16, Hq=32, Hkv=32, d=64, P=32, L=65536, alpha=2.0, k=32),
        # one decode step's tokens of a serving batch
        dict(name="append_32", op="write", B=32, Hq=32, Hkv=8, d=128, P=64, L=4095, new=1),
        # a batch of prompts of mixed lengths, rows inside a fused projection's output
        dict(name="prompts", op="write", B=12, Hq=32, Hkv=8, d=128, P=64, L=4096, new=4096),
        # a beam search step over one layer
        dict(name="beams_small", op="fork", B=8, Hkv=8, d=128, P=16, L=1000, bufs=2, metas=1),
        # a beam search step over the pages of sixteen layers
        dict(name="beams_layers", op="fork", B=32, Hkv=2, d=128, P=64, L=4096, bufs=32, metas=16),
        # a half-empty pool of one gigabyte packed
        dict(name="compact_pool", op="compact", B=24, Hkv=8, d=128, P=64, L=8192, bufs=2),
        # a sequence of sixteen layers swapped into another pool
        dict(name="swap_out", op="copy", Hkv=8, d=128, P=32, bufs=32, blocks=128, n=61),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "write", "fork", "compact", "copy"])
    d, P = rng.choice([64, 128]), rng.choice([16, 32, 64])
    if op == "decode":
        Hkv = rng.choice([1, 2, 4, 8, 16])
        G = rng.choice([1, 2, 4, 8])
        kept = rng.random() < 0.4
        L = _log(rng, 1, 500000 if kept else 131072)
        most = (1 << 28) // (Hkv * d * L) // (1 if kept else 2)
        B = max(1, min(_log(rng, 1, 32), most))
        alpha = rng.choice([1.25, 1.5, 2.0]) if kept or rng.random() < 0.5 else 1.0
        if kept and rng.random() < 0.2:
            alpha = 1.0
        k = min(_log(rng, 1, 400), -(-L // P), max(1, (1 << 27) // (B * Hkv * G * P * d))) if kept else 0
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, P=P, L=L, alpha=alpha, k=k)
    if op == "write":
        Hkv = rng.choice([1, 2, 4, 8])
        L = _log(rng, 1, 8192)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, L)
        B = min(_log(rng, 1, 64), max(1, 65536 // L))
        return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv, d=d, P=P, L=L, new=new)
    if op == "fork":
        return dict(op=op, B=_log(rng, 2, 48), Hkv=rng.choice([1, 2]), d=d, P=P, L=_log(rng, 2, 3000),
                    bufs=2 * rng.randint(1, 8), metas=rng.randint(0, 6))
    if op == "compact":
        return dict(op=op, B=_log(rng, 1, 32), Hkv=rng.choice([1, 2, 4]), d=d, P=P, L=_log(rng, 40, 6000), bufs=2)
    blocks = _log(rng, 2, 300)
    return dict(op=op, Hkv=rng.choice([1, 2, 4]), d=d, P=P, bufs=rng.randint(1, 24), blocks=blocks,
                n=rng.randint(1, blocks))


# ------------------------------------------------------------------ inputs

def _cdiv(a, b):
    return -(-a // b)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _lens(case):
    """Lengths of the batch: the longest is L, the others spread below it (the same for every seed, as are all shapes)."""
    L = case["L"]
    rng = random.Random(case["B"] * 1000003 + L)
    return [L] + [rng.randint(max(1, L // 2), L) for _ in range(case["B"] - 1)]


def _rows(g, lens, Hkv, d, P):
    """Key and value rows of every token, packed sequence after sequence: bf16 [sum lens, Hkv, d].  Keys have a scale
    of their own for each channel and an offset for each page, values are plain."""
    n = sum(lens)
    chan = torch.exp(0.5 * torch.randn(Hkv, d, generator=g, device="cuda"))
    k = torch.randn(n, Hkv, d, generator=g, device="cuda") * chan
    pages = torch.cat([torch.arange(l, device="cuda") // P for l in lens])
    off = 0.3 * torch.randn(max(lens) // P + 1, Hkv, 1, generator=g, device="cuda")
    k = (k + off[pages]).bfloat16()
    v = torch.randn(n, Hkv, d, generator=g, device="cuda").bfloat16()
    return k, v


def _starts(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def _cache_inputs(case, seed):
    """What both forms and the 64-bit answer start from."""
    g = _gen(seed)
    B, Hkv, d, P = case["B"], case["Hkv"], case["d"], case["P"]
    lens = _lens(case)
    Np = _cdiv(max(lens), P)
    nb = B * Np + 3
    table = torch.randperm(nb, generator=g, device="cuda")[:B * Np].view(B, Np).int()
    k, v = _rows(g, lens, Hkv, d, P)
    return g, lens, Np, nb, table, k, v


def _decode_inputs(case, seed):
    g, lens, Np, nb, table, k, v = _cache_inputs(case, seed)
    B, Hq, Hkv, d, P = case["B"], case["Hq"], case["Hkv"], case["d"], case["P"]
    q = torch.randn(B, Hq, d, generator=g, device="cuda").bfloat16()
    sel = cnt = None
    if case["k"]:
        # each head keeps the pages whose mean key it agrees with most
        page = torch.cat([b * Np + torch.arange(l, device="cuda") // P for b, l in enumerate(lens)])
        mean = torch.zeros(B * Np, Hkv, d, device="cuda").index_add_(0, page, k.float()).view(B, Np, Hkv, d)
        s = torch.einsum("bhgd,bnhd->bhgn", q.float().view(B, Hkv, Hq // Hkv, d), mean).reshape(B, Hq, Np)
        have = torch.tensor([_cdiv(l, P) for l in lens], device="cuda")
        s = s.masked_fill(torch.arange(Np, device="cuda") >= have[:, None, None], -math.inf)
        best = s.topk(case["k"], -1).indices
        cnt = have.clamp(max=case["k"])[:, None].expand(B, Hq).int().contiguous()
        dead = torch.arange(case["k"], device="cuda") >= cnt[..., None]
        best = best.masked_fill(dead, Np).sort(-1).values
        sel = torch.full((B, Hq, Np), -7, dtype=torch.int32, device="cuda")
        sel[..., :case["k"]] = best.masked_fill(dead, -7).int()
    return lens, Np, nb, table, k, v, q, sel, cnt


def _write_inputs(case, seed):
    g, lens, Np, nb, table, k, v = _cache_inputs(case, seed)
    rng = random.Random(case["L"] * 1000003 + case["new"])
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    new = [min(l, case["new"]) if case["new"] in (1, case["L"]) else rng.randint(0, min(l, case["new"])) for l in lens]
    new[0] = max(1, new[0])
    n = sum(new)
    fused = torch.randn(n, Hq + 2 * Hkv, d, generator=g, device="cuda").bfloat16()
    return lens, new, Np, nb, table, k, v, fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]


def _pool_inputs(case, seed):
    """A page table of B rows over a pool with free blocks; some rows share the full pages of a common prefix."""
    rng = np.random.RandomState(seed % (1 << 31))
    B, P, L = case["B"], case["P"], case["L"]
    Np = _cdiv(L + 1, P) + 1
    lens = rng.randint(max(1, L // 3), L + 1, B)
    lens[0] = L
    spare = B * Np if case["op"] == "compact" else B + 2
    nb = B * Np + spare
    perm = rng.permutation(nb)
    table = np.full((B, Np), -1, np.int64)
    used = 0
    for b in range(B):
        n = _cdiv(int(lens[b]), P)
        common = min(int(lens[b - 1]) // P, int(lens[b]) // P) // 2 if b % 2 else 0
        if common:
            table[b, :common] = table[b - 1, :common]
        table[b, common:n] = perm[used:used + n - common]
        used += n - common
    parent = np.where(rng.rand(B) < 0.5, np.arange(B), rng.randint(0, B, B))
    parent[rng.rand(B) < 0.1] = -1
    if B > 1:
        parent[:2] = 0
    as_int = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    return nb, Np, as_int(table), as_int(lens), as_int(parent)


def _blocks(g, bufs, blocks, values):
    """What the pages hold, as the 16-bit words that are moved."""
    return torch.randint(-32768, 32768, (bufs, blocks, values), generator=g, device="cuda", dtype=torch.int16)


def _meta_bytes(case, Np):
    return case["B"] * case["Hkv"] * _cdiv(Np, TILE) * TILE * 12 * case["d"]


# ------------------------------------------------------------------ plain forms: the 4-bit cache

def _quantise(x):
    """bf16 [..., d] -> codes uint8 [..., d/2] (even coordinate in the low half) and bf16 [..., d/GROUP, 2] (s, lo)."""
    x = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1), x.amax(-1)
    s = ((hi - lo) / 15).bfloat16().float()
    s = torch.where(s < 2.0 ** -126, 0, s)
    inv = torch.where(s > 0, 1 / s, 0)
    c = ((x - lo[..., None]) * inv[..., None]).round().clamp(0, 15).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack([s, lo], -1).bfloat16()


def _values(c, p):
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    p = p.float()
    return (p[..., 0:1] * c + p[..., 1:2]).flatten(-2)


def _tail_places(lens, new, table, P):
    """Block and slot of the last new[b] tokens of every sequence, packed."""
    b = torch.cat([torch.full((m,), i, device="cuda") for i, m in enumerate(new)])
    pos = torch.cat([torch.arange(l - m, l, device="cuda") for l, m in zip(lens, new)])
    return table.long()[b, pos // P], pos % P


def _plain_cache(case, lens, nb, table, k, v):
    Hkv, d, P = case["Hkv"], case["d"], case["P"]
    blk, slot = _tail_places(lens, lens, table, P)
    cache = []
    for x in (k, v):
        c = torch.full((nb, Hkv, P, d // 2), 255, dtype=torch.uint8, device="cuda")
        p = torch.full((nb, Hkv, P, d // GROUP, 2), math.nan, dtype=torch.bfloat16, device="cuda")
        c[blk, :, slot], p[blk, :, slot] = _quantise(x)
        cache.append((c, p))
    return cache


def _plain_softmax(s):
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    t = e.sum(-1, keepdim=True)
    return e / t, (m + torch.log(t))[..., 0]


def _plain_entmax(z, r):
    """The weights [z - tau]_+^r with sum 1, tau by bisection in 64 bits."""
    z = z.double()
    top = z.amax(-1, keepdim=True)
    lo, hi = top - 1, top
    for _ in range(48):
        mid = (lo + hi) / 2
        over = (z - mid).clamp_min(0).pow(r).sum(-1, keepdim=True) >= 1
        lo, hi = torch.where(over, mid, lo), torch.where(over, hi, mid)
    return (z - lo).clamp_min(0).pow(r).float(), lo[..., 0].float()


def _plain_decode(st):
    case = st["case"]
    B, Hq, Hkv, d, P, alpha = (case[x] for x in ("B", "Hq", "Hkv", "d", "P", "alpha"))
    (kc, kp), (vc, vp) = st["cache"]
    table, lens, q = st["table"].long(), st["lens"], st["q"].float()
    slot = torch.arange(P, device="cuda")
    if st["sel"] is None:
        # keys and values of every page, shared by the heads of a group
        q = q.view(B, Hkv, -1, d)
        K, V = (_values(c[table], p[table]).transpose(1, 2).reshape(B, Hkv, -1, d) for c, p in ((kc, kp), (vc, vp)))
        ok = (torch.arange(K.shape[2], device="cuda") < lens[:, None])[:, None]
    else:
        q = q.view(B, Hq, 1, d)
        k = case["k"]
        live = torch.arange(k, device="cuda") < st["cnt"][..., None]
        sel = torch.where(live, st["sel"][..., :k].long(), 0)
        blk = table[:, None].expand(B, Hq, -1).gather(-1, sel)
        head = (torch.arange(Hq, device="cuda") // (Hq // Hkv))[None, :, None].expand_as(blk)
        K, V = (_values(c[blk, head], p[blk, head]).reshape(B, Hq, -1, d) for c, p in ((kc, kp), (vc, vp)))
        pos = sel[..., None] * P + torch.arange(P, device="cuda")
        ok = (live[..., None] & (pos < lens[:, None, None, None])).reshape(B, Hq, -1)
    s = torch.matmul(q, K.transpose(-1, -2)) / math.sqrt(d)
    s = torch.where(ok[:, :, None], s, -math.inf)
    p, t = _plain_softmax(s) if alpha == 1 else _plain_entmax((alpha - 1) * s, 1 / (alpha - 1))
    o = torch.matmul(p, torch.where(ok[..., None], V, 0))
    return {"out": o.reshape(B, Hq, d), "tau": t.reshape(B, Hq)}


def _bf16_down(x):
    i = x.view(torch.int32)
    return torch.where(x < 0, (i + 0xffff) & -0x10000, i & -0x10000).view(torch.float32).bfloat16()


def _record_places(b, page, Hkv, d, tiles):
    """Element offsets of coordinate j of a page's record: in the bound region (bf16, kmin; kmax 512 behind it) and in
    the moment region (fp32, mean; var 512 behind it).  b, page [n] -> [n, Hkv, d]."""
    h, j = torch.arange(Hkv, device="cuda")[:, None], torch.arange(d, device="cuda")
    T = ((b[:, None, None] * Hkv + h) * tiles + page[:, None, None] // TILE) * 64 * d
    s, c, e = page[:, None, None] % TILE, j // 16, j % 16
    return (T + c * 1024 + s * 16 + 8 * ((e // 8) ^ ((s >> 2) & 1)) + e % 8,
            T + c * 1024 + s * 16 + 4 * ((e // 4) ^ ((s >> 1) & 3)) + e % 4)


def _plain_write(st):
    case = st["case"]
    B, Hkv, d, P = case["B"], case["Hkv"], case["d"], case["P"]
    (kc, kp), (vc, vp) = st["cache"]
    blk, slot = _tail_places(st["host_lens"], st["new"], st["table"], P)
    kc[blk, :, slot], kp[blk, :, slot] = _quantise(st["k_new"])
    vc[blk, :, slot], vp[blk, :, slot] = _quantise(st["v_new"])
    # the metadata of every page that got a row, from the values of all its tokens
    b = torch.cat([torch.full((_cdiv(l, P) - (l - m) // P if m else 0,), i, device="cuda")
                   for i, (l, m) in enumerate(zip(st["host_lens"], st["new"]))])
    page = torch.cat([torch.arange((l - m) // P, _cdiv(l, P) if m else (l - m) // P, device="cuda")
                      for l, m in zip(st["host_lens"], st["new"])])
    at = st["table"].long()[b, page]
    x = _values(kc[at], kp[at])                                               # [n, Hkv, P, d]
    n = (st["lens"].long()[b] - page * P).clamp(max=P)[:, None, None]
    ok = (torch.arange(P, device="cuda") < n)[..., None]
    low = torch.where(ok, x, math.inf).amin(2)
    high = torch.where(ok, x, -math.inf).amax(2)
    x = torch.where(ok, x, 0).double()
    mean = x.sum(2) / n
    var = (x.square().sum(2) / n - mean.square()).clamp_min(0)
    at_bound, at_moment = _record_places(b, page, Hkv, d, st["tiles"])
    st["bound"][at_bound] = _bf16_down(low)
    st["bound"][at_bound + 512] = -_bf16_down(-high)
    st["moment"][at_moment] = mean.float()
    st["moment"][at_moment + 512] = var.float()
    return {"k": _values(kc[blk, :, slot], kp[blk, :, slot]).bfloat16(),
            "v": _values(vc[blk, :, slot], vp[blk, :, slot]).bfloat16(), "bound": st["bound"], "moment": st["moment"]}


# ------------------------------------------------------------------ plain forms: pages

def _live(table, lens, nb, P):
    """Which blocks a row of the table holds, and the pages each row has."""
    n = (lens + P - 1) // P
    inside = torch.arange(table.shape[1], device="cuda") < n[:, None]
    live = torch.zeros(nb + 1, dtype=torch.int32, device="cuda")
    live.index_fill_(0, torch.where(inside, table, nb).long().flatten(), 1)
    return live[:nb], n


def _plain_fork(st):
    P, nb, bufs = st["case"]["P"], st["nb"], st["bufs"]
    table, lens, parent = st["table"], st["lens"], st["parent"].long()
    B, Np = table.shape
    live, _ = _live(table, lens, nb, P)
    fresh = torch.argsort(live, stable=True)                                  # free blocks first, ascending
    p = parent.clamp_min(0)
    L = torch.where(parent >= 0, lens[p], 0)
    n = (L + P - 1) // P
    row = torch.where(torch.arange(Np, device="cuda") < n[:, None], table[p], -1)
    # a partial last page stays with the parent's own row, else with the first row that continues it
    me = torch.arange(B, device="cuda")
    earlier = ((parent[:, None] == parent) & (me < me[:, None])).any(1)
    copies = (parent >= 0) & (L % P != 0) & (parent != me) & (earlier | (parent[p] == p))
    last = (n - 1).clamp_min(0).long()[:, None]
    src = row.gather(1, last)[:, 0].long()
    dst = fresh[(copies.long().cumsum(0) - 1).clamp_min(0)]
    at = copies.nonzero()[:, 0]
    row.scatter_(1, last, torch.where(copies, dst, src).int()[:, None])
    bufs[:, dst[at]] = bufs[:, src[at]]
    if st["meta_in"] is not None:
        here = (torch.arange(st["tiles"], device="cuda") < ((n + TILE - 1) // TILE)[:, None])
        b, t = here.nonzero(as_tuple=True)
        for i, o in ((st["meta_in"][0], st["meta_out"][0]), (st["meta_in"][1], st["meta_out"][1])):
            o[:, b, :, t] = i[:, p[b], :, t]
    # every live row grows by one token
    live, n = _live(row, L, nb, P)
    fresh = torch.argsort(live, stable=True)
    need = (st["add"] > 0) & (L % P == 0) & (parent >= 0)
    at = need.nonzero()[:, 0]
    row[at, n[at].long()] = fresh[:at.shape[0]].int()
    return {"table": row, "lens": L + torch.where(parent >= 0, st["add"], 0), "bufs": bufs,
            "meta": None if st["meta_in"] is None else st["meta_out"][2]}


def _plain_compact(st):
    P, nb, bufs, table = st["case"]["P"], st["nb"], st["bufs"], st["table"]
    live, n = _live(table, st["lens"], nb, P)
    ids = torch.arange(nb, device="cuda")
    n_live = live.sum()
    move = ids[(live > 0) & (ids >= n_live)]
    into = ids[(live == 0) & (ids < n_live)]
    remap = torch.where(live > 0, ids, -1)
    remap[move] = into
    bufs[:, into] = bufs[:, move]
    inside = torch.arange(table.shape[1], device="cuda") < n[:, None]
    out = torch.where(inside, remap[table.long().clamp_min(0)], -1).int()
    return {"table": out, "remap": remap.int(), "n_live": n_live.int().view(1), "bufs": bufs}


def _plain_copy(st):
    st["other"][:, st["dst"].long()] = st["bufs"][:, st["src"].long()]
    return {"bufs": st["other"]}


# ------------------------------------------------------------------ prepare, run

def _regions(meta, case, Np):
    """A metadata buffer's bound region (bf16) and moment region (fp32)."""
    cut = case["B"] * case["Hkv"] * _cdiv(Np, TILE) * 128 * case["d"]
    return meta[:cut].view(torch.bfloat16), meta[cut:].view(torch.float32)


def _by_row(metas, case, Np):
    """Metadata buffers [n, bytes] as [n, B, Hkv, tiles, bytes] of both regions, and whole."""
    cut = case["B"] * case["Hkv"] * _cdiv(Np, TILE) * 128 * case["d"]
    form = (metas.shape[0], case["B"], case["Hkv"], _cdiv(Np, TILE), -1)
    return metas[:, :cut].view(form), metas[:, cut:].view(form), metas


def _own_cache(case, lens, Np, nb, table, k, v):
    from sparse_entmax_kv_b200 import kv4, native
    shape = native.Shape(case["B"], case["Hq"], case["Hkv"], case["d"], case["P"], Np, nb)
    k4, v4 = kv4.alloc_cache(shape, "cuda")
    k4.fill_(255)
    v4.fill_(255)
    at = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kv4.entmaxkv_kv4_write(shape, k, v, _starts(lens), table, at, k4, v4)
    return shape, k4, v4


def prepare(case, seed):
    op = case["op"]
    st = {"case": case}
    if op == "decode":
        lens, Np, nb, table, k, v, q, sel, cnt = _decode_inputs(case, seed)
        st |= dict(table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), q=q, sel=sel, cnt=cnt)
        if own:
            from sparse_entmax_kv_b200 import kv4
            st["shape"], st["k4"], st["v4"] = _own_cache(case, lens, Np, nb, table, k, v)
            st["out"] = torch.empty(case["B"], case["Hq"], case["d"], device="cuda")
            st["tau"] = torch.empty(case["B"], case["Hq"], device="cuda")
            st["ws"] = kv4.alloc_workspace(st["shape"], "cuda")
        else:
            st["cache"] = _plain_cache(case, lens, nb, table, k, v)
    elif op == "write":
        lens, new, Np, nb, table, k, v, k_new, v_new = _write_inputs(case, seed)
        st |= dict(table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), k_new=k_new, v_new=v_new,
                   host_lens=lens, new=new, tiles=_cdiv(Np, TILE), starts=_starts(new))
        st["meta"] = torch.zeros(_meta_bytes(case, Np), dtype=torch.uint8, device="cuda")
        st["bound"], st["moment"] = _regions(st["meta"], case, Np)
        if own:
            st["shape"], st["k4"], st["v4"] = _own_cache(case, lens, Np, nb, table, k, v)
            st["k_back"], st["v_back"] = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (k_new, v_new))
        else:
            st["cache"] = _plain_cache(case, lens, nb, table, k, v)
    elif op in ("fork", "compact"):
        g = _gen(seed)
        st["nb"], Np, st["table"], st["lens"], st["parent"] = _pool_inputs(case, seed)
        values = case["Hkv"] * case["P"] * case["d"]
        st["bufs"] = _blocks(g, case["bufs"], st["nb"], values)
        st["tiles"], st["meta_in"], st["meta_out"] = _cdiv(Np, TILE), None, None
        st["add"] = (st["parent"] >= 0).int()
        if case.get("metas"):
            size = (case["metas"], _meta_bytes(case, Np))
            a = torch.randint(0, 256, size, generator=g, device="cuda", dtype=torch.uint8)
            st["meta_in"], st["meta_out"] = _by_row(a, case, Np), _by_row(torch.zeros_like(a), case, Np)
        if own:
            from sparse_entmax_kv_b200 import native, pages
            st["shape"] = native.Shape(case["B"], case["Hkv"], case["Hkv"], case["d"], case["P"], Np, st["nb"])
            st["ws"] = pages.alloc_workspace(st["shape"], "cuda")
            st["table_out"], st["lens_out"] = torch.empty_like(st["table"]), torch.empty_like(st["lens"])
            st["remap"] = torch.empty(st["nb"], dtype=torch.int32, device="cuda")
            st["n_live"] = torch.empty(1, dtype=torch.int32, device="cuda")
            st["pools"] = pages.Buffers(st["bufs"].unbind(0))
            if st["meta_in"] is not None:
                st["metas"] = (pages.Buffers(st["meta_in"][2].unbind(0)), pages.Buffers(st["meta_out"][2].unbind(0)))
    else:
        g = _gen(seed)
        values, nb, n = case["Hkv"] * case["P"] * case["d"], case["blocks"], case["n"]
        st["bufs"] = _blocks(g, case["bufs"], nb, values)
        st["other"] = torch.zeros_like(st["bufs"])
        st["src"], st["dst"] = (torch.randperm(nb, generator=g, device="cuda")[:n].int() for _ in range(2))
        if own:
            from sparse_entmax_kv_b200 import pages
            st["from"], st["into"] = pages.Buffers(st["bufs"].unbind(0)), pages.Buffers(st["other"].unbind(0))
    return st


def _own_run(st):
    from sparse_entmax_kv_b200 import kv4, pages
    case = st["case"]
    if case["op"] == "decode":
        kv4.entmaxkv_kv4_decode(st["shape"], st["q"], st["k4"], st["v4"], st["table"], st["lens"], case["alpha"],
                                st["out"], st["tau"], st["sel"], st["cnt"], workspace=st["ws"])
        return {"out": st["out"], "tau": st["tau"]}
    if case["op"] == "write":
        at = (st["starts"], st["table"], st["lens"])
        kv4.entmaxkv_kv4_write(st["shape"], st["k_new"], st["v_new"], *at, st["k4"], st["v4"], st["meta"])
        kv4.entmaxkv_kv4_read(st["shape"], st["k4"], st["v4"], *at, st["k_back"], st["v_back"])
        return {"k": st["k_back"], "v": st["v_back"], "bound": st["bound"], "moment": st["moment"]}
    if case["op"] == "fork":
        metas = st.get("metas", (None, None))
        pages.entmaxkv_pages_fork(st["shape"], st["parent"], st["table"], st["lens"], st["table_out"], st["lens_out"],
                                  st["pools"], metas[0], metas[1], workspace=st["ws"])
        pages.entmaxkv_pages_grow(st["shape"], st["add"], st["table_out"], st["lens_out"], workspace=st["ws"])
        return {"table": st["table_out"], "lens": st["lens_out"], "bufs": st["bufs"],
                "meta": None if st["meta_in"] is None else st["meta_out"][2]}
    if case["op"] == "compact":
        pages.entmaxkv_pages_compact(st["shape"], st["table"], st["lens"], st["table_out"], st["pools"], st["remap"],
                                     st["n_live"], workspace=st["ws"])
        return {"table": st["table_out"], "remap": st["remap"], "n_live": st["n_live"], "bufs": st["bufs"]}
    pages.entmaxkv_pages_copy(st["from"], st["into"], st["src"], st["dst"])
    return {"bufs": st["other"]}


_plain = {"decode": _plain_decode, "write": _plain_write, "fork": _plain_fork, "compact": _plain_compact,
          "copy": _plain_copy}


def run(state):
    return _own_run(state) if own else _plain[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, d, P = case["op"], case["d"], case["P"]
    if op == "decode":
        # the mean length of _lens is 3/4 L for all but the first row; kept pages are counted once for each head that
        # has keys of its own.  Entmax weights are zero off the support, so only the keys have to be read whole.
        B, Hq, Hkv, L = case["B"], case["Hq"], case["Hkv"], case["L"]
        tokens = L + (B - 1) * 0.75 * L
        if case["k"]:
            tokens = min(tokens, B * case["k"] * P)
        row = Hkv * (d / 2 + d / GROUP * 4)
        io = B * Hq * d * 6 + B * Hq * 4 + (B * Hq * case["k"] * 4 if case["k"] else 0)
        return {"bytes": tokens * row * (2 if case["alpha"] == 1 else 1) + io,
                "flops": tokens * Hq * d * (4 if case["alpha"] == 1 else 2)}
    if op == "write":
        # rows in, codes out, codes in, rows out, and a record of 12 d bytes a page
        B, Hkv, L = case["B"], case["Hkv"], case["L"]
        mean = L + (B - 1) * 0.75 * L
        rows = B if case["new"] == 1 else mean if case["new"] == L else max(1, 0.5 * B * case["new"])
        pages = max(B, rows / P)
        return {"bytes": rows * Hkv * 2 * (2 * d * 2 + 2 * (d / 2 + d / GROUP * 4)) + pages * Hkv * 12 * d, "flops": 0}
    block = case["Hkv"] * P * d * 2
    if op == "copy":
        return {"bytes": 2 * case["n"] * case["bufs"] * block, "flops": 0}
    B, Np = case["B"], _cdiv(case["L"] + 1, P) + 1
    held = B * Np * 0.5
    if op == "compact":
        # of the held blocks (a third to a half of the pool) about two thirds sit above the boundary
        return {"bytes": 2 * 0.6 * held * case["bufs"] * block + 2 * held * 4, "flops": 0}
    # about a third of the rows copy a partial page; metadata rows follow their parents
    rows = 0.9 * B * _cdiv(_cdiv(int(0.67 * case["L"]), P), TILE)
    meta = rows * case["Hkv"] * TILE * 12 * d * case["metas"]
    return {"bytes": 2 * (0.3 * B * case["bufs"] * block + meta + held * 4), "flops": 0}


# ------------------------------------------------------------------ the definition, in 64 bits

def _f32(x):
    return x.float().double()


def _exact_values(x):
    """The values that bf16 rows [..., d] are held as, in 64 bits, with the definition's fp32 roundings made one by one."""
    shape = x.shape
    x = x.double().reshape(-1, GROUP)
    lo = x.min(1, keepdim=True).values
    s = _f32(_f32(x.max(1, keepdim=True).values - lo) / 15).float().bfloat16().double()
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    inv = torch.where(s > 0, _f32(1 / s), torch.zeros_like(s))
    code = torch.clip(torch.round(_f32(_f32(x - lo) * inv)), 0, 15)
    return _f32(s * code + lo).reshape(shape)


def _exact_head(q, K, V, alpha):
    """One head: q [d], K and V [n, d]."""
    s = K @ q / math.sqrt(q.shape[0])
    if alpha == 1:
        t = torch.logsumexp(s, 0)
        return torch.exp(s - t) @ V, t
    z, r = (alpha - 1) * s, 1 / (alpha - 1)
    near = (z > z.max() - 1).nonzero()[:, 0]  # no weight exceeds 1
    z = z[near]
    lo, hi = z.max() - 1, z.max()
    for _ in range(60):
        mid = 0.5 * (lo + hi)
        full = (z - mid).clamp(min=0).pow(r).sum() >= 1
        lo, hi = torch.where(full, mid, lo), torch.where(full, hi, mid)
    return (z - lo).clamp(min=0).pow(r) @ V[near], lo


def _exact_decode(case, seed):
    lens, Np, nb, table, k, v, q, sel, cnt = _decode_inputs(case, seed)
    B, Hq, Hkv, d, P = case["B"], case["Hq"], case["Hkv"], case["d"], case["P"]
    if B * Hq > 1100:
        return None
    at = np.concatenate([[0], np.cumsum(lens)])
    out = torch.empty(B, Hq, d, dtype=torch.float64, device="cuda")
    tau = torch.empty(B, Hq, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(Hkv):
            rows = slice(int(at[b]), int(at[b + 1]))
            kx, vx = k[rows, h], v[rows, h]
            whole = None if sel is not None else (_exact_values(kx), _exact_values(vx))
            for x in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                if sel is None:
                    K, V = whole
                else:
                    tok = (sel[b, x, :int(cnt[b, x])].long()[:, None] * P + torch.arange(P, device="cuda")).flatten()
                    tok = tok[tok < lens[b]]
                    K, V = _exact_values(kx[tok]), _exact_values(vx[tok])
                out[b, x], tau[b, x] = _exact_head(q[b, x].double(), K, V, case["alpha"])
    return {"out": out, "tau": tau}


def _exact_write(case, seed):
    lens, new, Np, nb, table, k, v, k_new, v_new = _write_inputs(case, seed)
    B, Hkv, d, P = case["B"], case["Hkv"], case["d"], case["P"]
    bound = torch.zeros(B * Hkv * _cdiv(Np, TILE) * 64 * d, dtype=torch.float64, device="cuda")
    moment = torch.zeros_like(bound)
    at, new_at = np.concatenate([[0], np.cumsum(lens)]), np.concatenate([[0], np.cumsum(new)])
    for b in range(B):
        if not new[b]:
            continue
        first = (lens[b] - new[b]) // P
        old = k[int(at[b]) + first * P:int(at[b + 1]) - new[b]]
        x = _exact_values(torch.cat([old, k_new[int(new_at[b]):int(new_at[b + 1])]]))
        n = _cdiv(lens[b], P) - first
        page = torch.arange(first, first + n, device="cuda")
        of = torch.arange(x.shape[0], device="cuda") // P
        count = torch.bincount(of, minlength=n).double()[:, None, None]
        of = of[:, None, None].expand_as(x)
        zero = torch.zeros(n, Hkv, d, dtype=torch.float64, device="cuda")
        mean = zero.scatter_add(0, of, x) / count
        var = zero.scatter_add(0, of, (x - mean.gather(0, of)).square()) / count
        kb, mo = _record_places(torch.full((n,), b, device="cuda"), page, Hkv, d, _cdiv(Np, TILE))
        bound[kb] = zero.scatter_reduce(0, of, x, "amin", include_self=False)
        bound[kb + 512] = zero.scatter_reduce(0, of, x, "amax", include_self=False)
        moment[mo], moment[mo + 512] = mean, var
    return {"k": _exact_values(k_new), "v": _exact_values(v_new), "bound": bound, "moment": moment}


def exact(case, seed):
    if case["op"] == "decode":
        return _exact_decode(case, seed)
    if case["op"] == "write":
        return _exact_write(case, seed)
    return None  # whole numbers: tables, and the words of blocks that are moved
