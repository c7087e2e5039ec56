"""Plain references of the 4-bit cache and of the page operations (numpy, 64 bits, from the headers' definitions)."""
import numpy as np

GROUP = 64


def f32(x):
    return np.asarray(x, np.float32).astype(np.float64)


def bf16(x):
    """Round to the nearest bf16, ties to even (finite inputs), as float64."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = ((u + ((u >> 16) & 1) + 0x7FFF) >> 16) << 16
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def quantise(x):
    """x [..., d] (bf16 values) -> codes [..., d] int, s and lo [..., d / GROUP]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        rng = f32(hi - lo)
        bad = ~np.isfinite(g).all(-1) | ~np.isfinite(rng)
        s = np.where(bad, 0, bf16(f32(np.where(bad, 0, rng) * f32(1 / 15))))
        s = np.where(s < 2.0 ** -126, 0, s)
        inv = np.where(s > 0, f32(1 / np.where(s > 0, s, 1)), 0)
        c = np.clip(np.rint(f32(f32(g - np.where(bad, 0, lo)[..., None]) * inv[..., None])), 0, 15)
    c = np.where(bad[..., None], 0, c).astype(np.int64)
    return c.reshape(x.shape), np.where(bad, np.nan, s), np.where(bad, np.nan, lo)


def values(c, s, lo):
    g = c.reshape(c.shape[:-1] + (c.shape[-1] // GROUP, GROUP))
    return f32(s[..., None] * g + lo[..., None]).reshape(c.shape)


def _bits16(x):
    """bf16 bit patterns of bf16 values (every NaN as 0x7fc0)."""
    u = (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint32)
    return np.where(np.isnan(x), 0x7FC0, u)


def pack_tile(c, s, lo, values_layout):
    """One 16-token tile [16, d] as its 9 d bytes, from the documented layout."""
    d = c.shape[-1]
    words = np.zeros(2 * d, np.uint64)
    for t in range(16):
        for j in range(d):
            g, r = j // 64, j % 64
            if values_layout:
                x = 2 * ((t >> 1) & 3) if d == 128 else 4 * ((t >> 2) & 1)
                w = (t >> 1) * (d // 4) + ((r // 8) ^ x) * (d // 32) + 2 * g + (r // 4) % 2
                bit = 16 * (t & 1) + 4 * (r % 4)
            else:
                w = t * (d // 8) + (r // 16) * (d // 32) + 2 * g + (r // 8) % 2
                n = r % 8
                bit = 16 * (n & 1) + 4 * (n >> 1)
            words[w] |= np.uint64(int(c[t, j]) << bit)
    params = _bits16(s) | (_bits16(lo) << 16)
    return np.concatenate([words.astype("<u4").view(np.uint8), params.reshape(-1).astype("<u4").view(np.uint8)])


def code_mask(d, tokens, values_layout):
    """Bytes-as-bits mask of what the given tokens of a tile own (1 bits)."""
    c = np.zeros((16, d), np.int64)
    c[tokens] = 15
    z = np.zeros((16, d // 64))
    m = pack_tile(c, z, z, values_layout)
    par = m[8 * d:].view("<u4").reshape(16, -1)
    par[tokens] = 0xFFFFFFFF
    return m


def attention(q, K, V, alpha):
    """One head in 64 bits: (out, tau or log-sum-exp, weights)."""
    d = q.shape[0]
    if K.shape[0] == 0:
        return np.zeros(d), np.nan, np.zeros(0)
    s = K @ q / np.sqrt(d)
    if alpha == 1:
        m = s.max()
        e = np.exp(s - m)
        return (e / e.sum()) @ V, m + np.log(e.sum()), e / e.sum()
    z, r = (alpha - 1) * s, 1 / (alpha - 1)
    lo, hi = z.max() - 1, z.max()
    for _ in range(80):
        mid = (lo + hi) / 2
        if (np.maximum(z - mid, 0) ** r).sum() >= 1:
            lo = mid
        else:
            hi = mid
    p = np.maximum(z - lo, 0) ** r
    return p @ V, lo, p


def attention_bounds(q, s, V, p, alpha, support_gap=0.0):
    """How far an fp32 evaluation of one head may be off: (out, tau).

    A score is s sum q (16 + c) + (lo - 16 s) sum q, summed in fp32: every one of the d products is at most
    31 s |q_j|, every addition rounds (or truncates) by at most 2^-23 of the partial sum, and the errors of d
    additions in random directions grow like sqrt(d); four of those is the bound taken for a score.  Softmax weights
    move by at most twice that, relatively; entmax weights p = (z - tau)^r by r p^(1 - 1/r) times twice the error of
    z.  The exponential and the division add 2^-22 of the weight, the sum over n values sqrt(n) 2^-24 of its terms.
    """
    d = q.shape[0]
    scale = (alpha - 1 if alpha > 1 else 1) / np.sqrt(d)
    smax = np.repeat(s.max(0), GROUP) if s.size else np.zeros(d)
    dz = 4 * np.sqrt(d) * 2.0 ** -23 * scale * np.sum(31 * smax * np.abs(q)) + 2.0 ** -22
    vmax = np.abs(V).max() + 15 * s.max() if V.size else 0.0
    r = 1 / (alpha - 1) if alpha > 1 else 1.0
    pw = p[p > 0]
    moved = 2 * r * dz * np.sum(pw ** (1 - 1 / r) if alpha > 1 else pw)
    # tokens just under tau may enter the support with weight (2 dz)^r
    moved += len(p) * (2 * dz) ** r if alpha > 1 else 0
    return vmax * (moved + 2.0 ** -21 + np.sqrt(len(p)) * 2.0 ** -24), 2 * dz + 2.0 ** -20


def record(x, P_tokens):
    """kmin, kmax (bf16 rounded outwards), mean, var of the first P_tokens rows of x [P, d] (fp32 values)."""
    x = x[:P_tokens]

    def down(v):
        u = np.ascontiguousarray(v, np.float32).view(np.uint32).astype(np.uint64)
        u = np.where(v < 0, u + 0xFFFF, u)
        return ((u >> 16) << 16).astype(np.uint32).view(np.float32)
    n, parts = x.shape[0], 1024 // x.shape[1]
    s1 = s2 = 0.0
    for p in range(parts):  # every parts-th token, then the partial sums in order
        a, b = np.zeros(x.shape[1]), np.zeros(x.shape[1])
        for t in range(p, n, parts):
            a = a + x[t]
            b = b + x[t] * x[t]
        s1, s2 = (a, b) if p == 0 else (s1 + a, s2 + b)
    mean = s1 / n
    var = np.maximum(s2 / n - mean * mean, 0)
    return down(x.min(0)), -down(-x.max(0)), mean.astype(np.float32), var.astype(np.float32)


def meta_arrays(meta, B, Hkv, max_pages, d):
    """A metadata buffer as kmin, kmax, mean, var [B, Hkv, tiles * 32, d] (float32)."""
    tiles = -(-max_pages // 32)
    nt = B * Hkv * tiles
    bound = meta[:nt * 128 * d].view(np.uint16).reshape(nt, d // 16, 2, 32, 2, 8)
    moment = meta[nt * 128 * d:].view(np.float32).reshape(nt, d // 16, 2, 32, 4, 4)
    out = []
    for a, pieces in ((bound, 2), (moment, 4)):
        for which in range(2):
            y = np.empty((nt, 32, d), a.dtype)
            for sl in range(32):
                for ch in range(d // 16):
                    for h in range(pieces):
                        x = ((sl >> 2) & 1) if pieces == 2 else ((sl >> 1) & 3)
                        w = 16 // pieces
                        y[:, sl, ch * 16 + h * w:ch * 16 + (h + 1) * w] = a[:, ch, which, sl, h ^ x]
            if pieces == 2:
                y = (y.astype(np.uint32) << 16).view(np.float32)
            out.append(y.reshape(B, Hkv, tiles * 32, d))
    return out


# ------------------------------------------------------------------ pages

def used_blocks(table, lens, P, nb, hold=None):
    refs = np.zeros(nb, np.int64) if hold is None else np.maximum(np.asarray(hold, np.int64), 0)
    for b, L in enumerate(lens):
        for p in range(-(-max(int(L), 0) // P)):
            if 0 <= table[b][p] < nb:
                refs[table[b][p]] += 1
    return refs


def fork(parent, table, lens, P, nb, hold=None):
    """New table, lengths, the (src, dst) pages to copy, and whether blocks ran out."""
    B, mp = table.shape
    free = [i for i, r in enumerate(used_blocks(table, lens, P, nb, hold)) if r == 0]
    out, L_out, pairs, short = np.full((B, mp), -1, np.int32), np.zeros(B, np.int32), [], False
    for b in range(B):
        p = parent[b]
        if p < 0:
            continue
        L = int(lens[p])
        n = -(-L // P)
        out[b, :n] = table[p, :n]
        keeper = p if parent[p] == p else min(x for x in range(B) if parent[x] == p)
        if L % P and b != keeper:
            if free:
                pairs.append((int(table[p, n - 1]), free[0]))
                out[b, n - 1] = free.pop(0)
            else:
                short = True
                out[b, n - 1] = -1
                L -= L % P
        L_out[b] = L
    return out, L_out, pairs, short


def grow(add, table, lens, P, nb, hold=None):
    B, mp = table.shape
    table, lens = table.copy(), lens.copy()
    free = [i for i, r in enumerate(used_blocks(table, lens, P, nb, hold)) if r == 0]
    total, short = 0, False
    for b in range(B):
        if add[b] <= 0 or lens[b] + add[b] > mp * P:
            continue
        n0, n1 = -(-int(lens[b]) // P), -(-int(lens[b] + add[b]) // P)
        total += n1 - n0
        if total > len(free) and n1 > n0:
            short = True
            continue
        table[b, n0:n1] = free[total - (n1 - n0):total]
        lens[b] += add[b]
    return table, lens, short


def compact(table, lens, P, nb, hold=None):
    refs = used_blocks(table, lens, P, nb, hold)
    live = int((refs > 0).sum())
    holes = [i for i in range(live) if refs[i] == 0]
    movers = [i for i in range(live, nb) if refs[i] > 0]
    remap = np.where(refs > 0, np.arange(nb), -1)
    for s, t in zip(movers, holes):
        remap[s] = t
    out = np.full_like(table, -1)
    for b, L in enumerate(lens):
        n = -(-max(int(L), 0) // P)
        out[b, :n] = remap[table[b, :n]]
    return out, remap, live, list(zip(movers, holes))
