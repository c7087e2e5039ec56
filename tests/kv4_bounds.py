"""The 4-bit cache and its attention in 64 bits from the definition, with bounds of an fp32 evaluation that follow its
arithmetic token by token (numpy)."""
import numpy as np

from kv4_ref import GROUP, bf16, f32


def quantise(x):
    """x [..., d] (finite bf16 values) -> codes [..., d], s and lo [..., d / GROUP]; s = bf16(fl(fl(max - lo) / 15))."""
    x = np.asarray(x, np.float64)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    lo = g.min(-1)
    s = bf16(f32(f32(g.max(-1) - lo) / 15))  # 64 bits and then 32: no quotient of 24 bits by 15 lies that near a tie
    s = np.where(s < 2.0 ** -126, 0, s)
    inv = np.where(s > 0, f32(1 / np.where(s > 0, s, 1)), 0)
    c = np.clip(np.rint(f32(f32(g - lo[..., None]) * inv[..., None])), 0, 15)
    return c.reshape(x.shape).astype(np.int64), s, lo


def values(c, s, lo):
    g = c.reshape(c.shape[:-1] + (c.shape[-1] // GROUP, GROUP))
    return f32(s[..., None] * g + lo[..., None]).reshape(c.shape)


def _spread(x):
    """A number of each group, for each of its coordinates."""
    return np.repeat(x, GROUP, -1)


def _scores(q, keys, scale):
    """Scaled scores of one head, and how far an fp32 evaluation of each may be off.

    With k = s (c - 8) + o, o = lo + 8 s, a score is sum over the groups of s A + o Q, A = sum q (c - 8), Q = sum q.
    A comes from four tensor-core products of 16 terms; each keeps at least 24 bits below the largest of its 17
    addends, so A is off by at most 4 * 17 * 2^-23 < 2^-16 of sum |q (c - 8)| (this covers the query's coordinates
    below 2^-27 of the largest, too).  Q takes 20 additions, o one rounding: 2^-19 of |o| sum |q|.  The value itself
    is rounded to fp32 in the definition: 2^-24 of sum |q k|.  Scale and sum: 2^-20 of the score.
    """
    c, s, lo = keys
    o = lo + 8 * s
    K = values(c, s, lo)
    z = scale * (K @ q)
    aq = np.abs(q)
    off = scale * (2.0 ** -16 * (_spread(s) * np.abs(c - 8)) @ aq + 2.0 ** -19 * _spread(np.abs(o)) @ aq
                   + 2.0 ** -24 * np.abs(K) @ aq)
    return z, off + 2.0 ** -20 * np.abs(z) + 2.0 ** -126


def _rise(x, e, r):
    """The most that [x]_+^r moves when x moves by e."""
    f = lambda y: np.maximum(y, 0) ** r  # noqa: E731
    return np.maximum(f(x + e) - f(x), f(x) - f(x - e))


def attention(q, keys, vals, alpha):
    """One head: q [d], keys and vals (codes, s, lo) of its tokens -> out, tau (or log-sum-exp), and the bounds of both.

    Weights move with the scores.  Softmax: each by a factor of at most exp(2 max dz).  Entmax: tau moves by at most
    the largest dz, so x = z - tau by twice that; weights of moved scores still sum to 1, so what each adds is its
    move times |v - o|.  The solver's tau, and z and tau as fp32 counted from the largest z, put each x off by
    another 2^-23 + 3 * 2^-25 < 2^-22, after which the sum may not be 1: those moves count times |v|.  (Above alpha =
    2 a token next to tau gets what the others leave, and the sum is 1.)  Powers, sums and the division add 2^-18 of
    the terms' size: of p s c and p lo (entmax) or p s (c - 8) and p (lo + 8 s) (softmax), which may cancel in a value
    near zero, so 16 s + |lo| is taken for either.  Only tokens that can have weight count, so the bound is far
    below the output itself.
    """
    d = q.shape[0]
    scale = (alpha - 1 if alpha > 1 else 1.0) / np.sqrt(d)
    z, dz = _scores(q, keys, scale)
    c, s, lo = vals
    V = values(c, s, lo)
    size = _spread(16 * s + np.abs(lo))
    top = z.max()
    if alpha == 1:
        p = np.exp(z - top)
        tau = top + np.log(p.sum())
        p /= p.sum()
        moved, loose = p * np.expm1(np.minimum(2 * dz[p > 2.0 ** -60].max(), 1.0)), 0 * p
    else:
        r, x = 1 / (alpha - 1), z - top
        a, b = -1.0, 0.0
        for _ in range(100):
            mid = (a + b) / 2
            a, b = (mid, b) if (np.maximum(x - mid, 0) ** r).sum() >= 1 else (a, mid)
        p = np.maximum(x - a, 0) ** r
        edge = (x > a) & (x <= b)  # more bits than there are tell x from tau: what the others leave
        if r < 1 and edge.any():
            p = np.where(x > b, np.maximum(x - b, 0) ** r, 0)
            p[edge] = (1 - p.sum()) / edge.sum()
        tau = top + a
        near = x - a > -2.0 ** -8
        e = 2 * dz[near].max()
        moved = _rise(x - a, e, r)
        loose = _rise(x - a, e + 2.0 ** -22, r) - moved if r >= 1 else 0 * p
    o = p @ V
    do = moved @ np.abs(V - o) + loose @ np.abs(V) + 2.0 ** -18 * (p @ size) + 2.0 ** -126
    return o, tau, do, dz[p > 2.0 ** -60].max() + 2.0 ** -21 + 2.0 ** -22 * abs(tau)
