"""The 4-bit cache where ranges end: values without a step, scores and values of any size, steps on a rounding's
border, and outputs held to bounds that no wrong output meets."""
import numpy as np
import pytest
import torch

import kv4_bounds as exact
from sparse_entmax_kv_b200 import kv4, native as nv
from test_kv4 import Case, f64_of

gpu = pytest.mark.gpu


def head_of(c, b, h, alpha, tok=None):
    """What exact.attention gives for head h of sequence b of a Case."""
    rows, kvh = c.rows_of(b), h // (c.Hq // c.Hkv)
    tok = slice(None) if tok is None else tok
    k, v = (exact.quantise(f64_of(x[rows][:, kvh])[tok]) for x in (c.k, c.v))
    return exact.attention(f64_of(c.q[b, h]), k, v, alpha)


def check(c, alpha, out, tau, sharp=True):
    """Every head within its bounds; sharp: bounds that an output of zeros, or of another head, does not meet."""
    out, tau = f64_of(out), f64_of(tau)
    for b in range(c.B):
        for h in range(c.Hq):
            o, t, do, dt = head_of(c, b, h, alpha)
            assert (np.abs(out[b, h] - o) <= do).all(), (b, h, np.abs(out[b, h] - o).max(), do.max())
            assert abs(tau[b, h] - t) <= dt, (b, h, tau[b, h], t, dt)
            if sharp:
                assert (np.abs(o) > 4 * do).any() and (np.abs(np.roll(o, 1) - o) > 4 * do).any(), (b, h)


def prescribe(scores, zero=None, big=None):
    """rows for Case: key t gives a query of ones the score sqrt(d) scores[t] (constant keys: s = 0, lo the value);
    values of tokens in `zero` are zero, those of tokens in `big` larger by a factor."""
    def rows(k, v):
        k[:] = scores[:, None, None]
        if zero is not None:
            v[zero] = 0.0
        if big is not None:
            v[big[0]] *= big[1]
    return rows


# ------------------------------------------------------------------ softmax weights of value rows without a step

@gpu
@pytest.mark.parametrize("G,d,P", [(1, 64, 16), (4, 64, 16), (2, 128, 32), (8, 128, 64)])
@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("rise", [15.0, 18.0, 19.0, 24.0, 60.0])
def test_rising_scores_of_zero_values(G, d, P, long, rise):
    """Rows of zeros (padding, sinks) carry weight but no p s: their weights have to stay in range by themselves.
    Tiles of score 0, of `rise` and of rise + 2 (natural units), the first two with values of zero, in every order;
    the list is one CTA's, or cut over the GPU."""
    L = 5000 if long else 900
    at = np.random.RandomState(int(rise) + G).randint(0, 3, -(-L // 16)).repeat(16)[:L]
    scores = torch.tensor([0.0, rise, rise + 2])[at] / np.sqrt(d)
    c = Case(1, G, 1, d, P, [L], seed=G, rows=prescribe(scores, zero=torch.from_numpy(at < 2)))
    c.q[:] = 1.0
    c.write(meta=False)
    check(c, 1.0, *c.decode(1.0))


@gpu
@pytest.mark.parametrize("step", [20.0, 27.0])
def test_runs_of_zero_values(step):
    """Runs of 64 zero tiles, the scores of each run `step` (powers of two) above the last, then values of their own."""
    L = 16 * 64 * 6
    run = np.arange(L) // 1024
    scores = torch.from_numpy(run * (step * np.log(2) / 8)).float()
    c = Case(1, 2, 1, 64, 16, [L], rows=prescribe(scores, zero=torch.from_numpy(run < 5)))
    c.q[:] = 1.0
    c.write(meta=False)
    check(c, 1.0, *c.decode(1.0))


@gpu
@pytest.mark.parametrize("value", [0.0, 1.0])
@pytest.mark.parametrize("L", [900, 40000])
def test_values_without_a_step(value, L):
    """All values zero, or all one: the output is that value, and the log-sum-exp is finite and right."""
    def rows(k, v):
        v[:] = value
    c = Case(1, 4, 1, 64, 16, [L], seed=1, rows=rows)
    c.write(meta=False)
    out, tau = c.decode(1.0)
    check(c, 1.0, out, tau, sharp=False)
    assert (out - value).abs().max() <= 2.0 ** -18


# ------------------------------------------------------------------ references of one head far apart

@gpu
@pytest.mark.parametrize("L", [900, 5000])
@pytest.mark.parametrize("power", [40, 60, 90])
def test_zero_values_beside_large_ones(L, power):
    """Equal scores, half of the tokens with values of zero, half with values near 2^power (in turn by 16, and by 512):
    the references of the two differ by more than an exponent of fp32 holds."""
    for width in (16, 512):
        half = torch.arange(L) // width % 2 == 0
        c = Case(1, 4, 1, 64, 16, [L], seed=power, rows=prescribe(torch.zeros(L), half, (~half, 2.0 ** power)))
        c.write(meta=False)
        check(c, 1.0, *c.decode(1.0))


# ------------------------------------------------------------------ scores of any size

@gpu
@pytest.mark.parametrize("L", [1, 900, 5000])
@pytest.mark.parametrize("score", [-2.0 ** 120, -2.0 ** 101, 2.0 ** 120])
def test_softmax_of_scores_far_from_zero(L, score):
    """Tokens of equal scores share the weight evenly, however low (or high) the score is."""
    c = Case(1, 2, 1, 64, 16, [L], seed=2, rows=prescribe(torch.full((L,), 2.0 ** 50)))
    c.q[:] = score / 2.0 ** 53
    c.write(meta=False)
    out, tau = c.decode(1.0)
    # equal keys have the same score to the bit, so the weights are 1 / L: sums of L terms and the products' 2^-18
    V = exact.values(*exact.quantise(f64_of(c.v[:, 0])))
    assert np.abs(f64_of(out[0]) - V.mean(0)).max() <= 2.0 ** -18 * np.abs(V).max()
    assert np.abs(f64_of(tau[0]) / score - 1).max() <= 2.0 ** -20


# ------------------------------------------------------------------ the step

def bordering_groups(n, seed=0):
    """[n, 64] bf16 rows whose range is a whole multiple of 15 away from a border of the step's rounding to bf16:
    (max - lo) / 15 is halfway between two bf16 values, and a product with a rounded 1/15 need not be."""
    g = torch.Generator().manual_seed(seed)
    x = torch.empty(n, 64)
    got = 0
    while got < n:
        # 15 (2 m + 1) in units of a half step, and a minimum fine enough to reach it
        m = int(torch.randint(128, 256, (1,), generator=g))
        e = int(torch.randint(-12, 4, (1,), generator=g))
        rng = 15 * (2 * m + 1) * 2.0 ** (e - 1)
        hi = float(torch.tensor(rng).bfloat16())
        lo = hi - rng
        if lo == 0 or float(torch.tensor(lo).bfloat16()) != lo:
            continue
        row = lo + (hi - lo) * torch.rand(64, generator=g)
        row[3], row[40] = lo, hi
        x[got] = row.bfloat16().float().clamp(lo, hi)
        got += 1
    return x


def test_bordering_groups_are_on_the_border():
    x = bordering_groups(200).double().numpy()
    r = (x.max(-1) - x.min(-1)) / 15
    assert (exact.f32(r) == r).all()
    up = exact.bf16(r * (1 + 2.0 ** -20))
    assert (up != exact.bf16(r * (1 - 2.0 ** -20))).all()
    by_product = exact.bf16(exact.f32(r * 15 * exact.f32(1 / 15)))
    assert (by_product != exact.bf16(r)).any()  # the two readings of the step differ on them


@gpu
@pytest.mark.parametrize("d,P", [(64, 16), (128, 64)])
def test_step_on_a_border(d, P):
    """Steps that lie halfway between two bf16 values round to even, as the division by 15 says."""
    n = 300
    x = bordering_groups(2 * n * d // 64).view(2, n, 1, d)
    c = Case(1, 1, 1, d, P, [n], rows=lambda k, v: (k.copy_(x[0]), v.copy_(x[1])))
    c.write()
    back = [torch.empty(n, 1, d, device="cuda") for _ in range(2)]
    kv4.entmaxkv_kv4_read(c.shape, c.k4, c.v4, c.start, c.table, c.seq, *back)
    for rows, got in ((c.k, back[0]), (c.v, back[1])):
        assert torch.equal(got.cpu().double(), torch.from_numpy(exact.values(*exact.quantise(f64_of(rows)))))


@gpu
@pytest.mark.parametrize("off,scale", [(3.0, 1.0), (0.0, 1.0), (100.0, 0.1), (-20.0, 5.0)])
def test_rows_with_an_offset_or_an_outlier(off, scale):
    """Rows read back as the definition has them: offset data, and small rows with one large value a group."""
    def rows(k, v):
        k[:] = k * scale + off
        v *= 0.05
        v.view(n, 2, 2, 64)[..., 7] = 6.875
    n = 3000
    c = Case(1, 2, 2, 128, 32, [n], seed=3, rows=rows)
    c.write()
    back = [torch.empty(n, 2, 128, device="cuda") for _ in range(2)]
    kv4.entmaxkv_kv4_read(c.shape, c.k4, c.v4, c.start, c.table, c.seq, *back)
    for x, got in ((c.k, back[0]), (c.v, back[1])):
        assert torch.equal(got.cpu().double(), torch.from_numpy(exact.values(*exact.quantise(f64_of(x)))))


# ------------------------------------------------------------------ the same bits from every call

def rising(L, kept, seed, shares=64):
    """Scores of which `kept` lie within 1 of the largest (as entmax counts them, alpha 1.5: z = score / 2), in random
    places, and the rest a little below, so that what a share lists depends on what it has heard of the others."""
    rng = np.random.RandomState(seed)
    z = -1.0 - rng.rand(L) * 3.0
    z[rng.permutation(L)[:kept]] = -rng.rand(kept) * 0.9
    return torch.from_numpy(z).float()


@gpu
@pytest.mark.parametrize("L,kept", [(60000, 3500), (60000, 4000), (200000, 3000), (60000, 4300)])
@pytest.mark.parametrize("d", [64, 128])
def test_listed_candidates_do_not_show(L, kept, d):
    """The candidates kept are about as many as fit on chip; how many more were listed on the way depends on timing,
    the result may not.  Other work runs beside the calls."""
    c = Case(1, 4, 2, d, 32, [L], rows=lambda k, v: k.copy_(2 * rising(L, kept, 5)[:, None, None] / np.sqrt(d)))
    c.q[:] = 1.0
    c.q[0, 1], c.q[0, 3] = 1.5, 0.5
    c.write(meta=False)
    want = c.decode(1.5)
    check(c, 1.5, *want, sharp=False)
    other = torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda")
    for i in range(60):
        if i % 3 == 0:
            with torch.cuda.stream(other):
                x @ x
        got = c.decode(1.5)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_supports_beyond_the_chip_do_not_depend_on_the_lists(d):
    """More tokens with weight than fit on chip, and as many listed that have none."""
    L = 100000
    rng = np.random.RandomState(1)
    z = -0.9 - rng.rand(L)
    z[rng.permutation(L)[:20000]] = 0.0
    z[:] += 0.001 * rng.rand(L)
    c = Case(1, 2, 1, d, 32, [L], rows=lambda k, v: k.copy_(torch.from_numpy(4 * z).float()[:, None, None] / np.sqrt(d)))
    c.q[:] = 1.0
    c.write(meta=False)
    want = c.decode(1.25)
    other = torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda")
    for i in range(60):
        if i % 3 == 0:
            with torch.cuda.stream(other):
                x @ x
        got = c.decode(1.25)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i


@gpu
@pytest.mark.parametrize("at", [777, 50000])
@pytest.mark.parametrize("kept,extra,alpha", [(3500, 1500, 1.5), (3500, 3000, 1.5), (20000, 80000, 1.25)])
@pytest.mark.parametrize("d", [64, 128])
def test_one_score_above_the_rest_is_heard_of_late(d, kept, extra, alpha, at):
    """One token 0.5 above the others: until a share hears of it, it lists `extra` tokens that carry no weight beside
    it, in numbers that change from call to call, around what fits on chip (4096) and far beyond it."""
    L = 100000
    rng = np.random.RandomState(1)
    z, p = -2.0 - rng.rand(L), rng.permutation(L)
    z[p[:kept]] = -(0.49 if kept < 4096 else 0.001) * rng.rand(kept)
    z[p[kept:kept + extra]] = -0.55 - 0.4 * rng.rand(extra)
    z[at] = 0.5
    c = Case(1, 2, 1, d, 32, [L], rows=prescribe(torch.from_numpy(z / (alpha - 1)).float() / np.sqrt(d)))
    c.q[:] = 1.0
    c.write(meta=False)
    want = c.decode(alpha)
    check(c, alpha, *want, sharp=False)
    other = torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda")
    for i in range(60):
        if i % 3 == 0:
            with torch.cuda.stream(other):
                x @ x
        got = c.decode(alpha)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i


@gpu
@pytest.mark.parametrize("alpha", [1.25, 1.5, 2.0, 3.0])
@pytest.mark.parametrize("score", [2.0 ** 23, 2.0 ** 25, -2.0 ** 26, 1e8, -1e8, 1e12, -2.0 ** 120])
def test_entmax_of_scores_far_from_zero(alpha, score):
    """The largest token carries weight however large its score is: one alone, or several alike."""
    for L, top in ((1, [0]), (700, [345]), (700, [3, 44, 699]), (30000, [12345, 23000])):
        a = torch.full((L,), 1.0 if score < 0 else 0.5)
        a[top] = 0.75 if score < 0 else 1.0
        c = Case(1, 2, 1, 64, 16, [L], seed=len(top), rows=prescribe(a * 2.0 ** 30))
        c.q[:] = score / 8 / 2.0 ** 30
        c.write(meta=False)
        out, tau = c.decode(alpha)
        V = exact.values(*exact.quantise(f64_of(c.v[:, 0])))[top]
        # z is the same to the bit for equal keys, so the weights are equal: (1 / n)
        assert np.abs(f64_of(out[0]) - V.mean(0)).max() <= 2.0 ** -19 * np.abs(V).max(), (L, top)
        z = (alpha - 1) * float(c.q[0, 0, 0]) * 8 * float(a[top[0]]) * 2.0 ** 30
        assert np.abs(f64_of(tau[0]) - (z - len(top) ** (1 - alpha))).max() <= 2.0 ** -21 * abs(z), (L, top)


@gpu
@pytest.mark.parametrize("alpha", [1.25, 1.5, 2.0])
@pytest.mark.parametrize("offset", [0.0, 20.0, -180.0])
def test_entmax_weights_do_not_feel_a_common_offset(alpha, offset):
    """A common offset of the scores leaves the weights: tau is solved below the largest z, so what is lost is each
    score's own rounding.  The first 64 coordinates hold the offset, the others what tells the tokens apart."""
    def rows(k, v):
        k[..., :64] = offset
        k[..., 64:] = (torch.randint(0, 24, (k.shape[0],), generator=torch.Generator().manual_seed(6)) / 64)[:, None, None]
    c = Case(1, 2, 1, 128, 16, [600], seed=6, rows=rows)
    c.q[:] = 1.0
    c.write(meta=False)
    check(c, alpha, *c.decode(alpha))


# ------------------------------------------------------------------ eight heads a group

@gpu
@pytest.mark.parametrize("d,P", [(64, 32), (128, 16)])
def test_eight_heads_are_as_exact_as_four(d, P):
    """Long softmax of eight heads that share their keys: no further from 64 bits than the same heads in groups of
    four over the same cache (their weights take other columns of the products, and the same two parts)."""
    c = Case(1, 8, 1, d, P, [60000], seed=11)
    c.write(meta=False)
    out = f64_of(c.decode(1.0)[0])
    want = np.stack([head_of(c, 0, h, 1.0)[0] for h in range(8)])
    off = np.linalg.norm(out[0] - want) / np.linalg.norm(want)
    four = nv.Shape(1, 4, 1, d, P, c.mp, c.shape.num_blocks)
    parts, q = [], c.q
    for h in (0, 4):
        c.q = q[:, h:h + 4].contiguous()
        got = torch.empty(1, 4, d, device="cuda")
        parts.append(f64_of(c.decode(1.0, shape=four, out=got, tau=torch.empty(1, 4, device="cuda"))[0])[0])
    ref_off = np.linalg.norm(np.concatenate(parts) - want) / np.linalg.norm(want)
    assert off <= 2 * ref_off + 2.0 ** -24, (off, ref_off)


# ------------------------------------------------------------------ alpha > 2: tokens next to the threshold

@gpu
@pytest.mark.parametrize("alpha", [3.0, 5.0, 10.0, 100.0, 1000.0])
@pytest.mark.parametrize("gap", [0.01, 0.35, 0.9])
@pytest.mark.parametrize("n", [1, 3, 5000])
def test_weight_next_to_the_threshold(alpha, gap, n):
    """One token above n equal ones (and others without weight): theirs is p with n p + (gap + p^(alpha-1))^r = 1, where
    gap + p^(alpha-1) is the first one's distance from tau, which in fp32 is no longer told from gap."""
    L, d = n + 40, 64
    # z = (alpha - 1) 8 k: the first token's, the n equal ones', and what lies 3 below
    k = np.full(L, -3.0)
    k[17], k[30:30 + n] = 0.0, -gap
    c = Case(1, 1, 1, d, 16, [L], seed=n, rows=prescribe(torch.from_numpy(k).float()))
    c.q[:] = 1 / (8 * (alpha - 1))
    c.write(meta=False)
    out, tau = c.decode(alpha)
    z = (alpha - 1) * f64_of(c.k[:, 0, 0]) * float(c.q[0, 0, 0]) * 8
    r, gap = 1 / (alpha - 1), z[17] - z[30]
    a, b = 0.0, 1.0 / n
    for _ in range(200):
        p = (a + b) / 2
        a, b = (p, b) if n * p + (gap + p ** (alpha - 1)) ** r < 1 else (a, p)
    codes, s, lo = exact.quantise(f64_of(c.v[:, 0]))
    V = exact.values(codes, s, lo)
    want = (1 - n * p) * V[17] + p * V[30:30 + n].sum(0)
    # dz < 2^-20 (scores below 4): the first weight moves by r gap^(r - 1) 2 dz < 2^-12 at gap = 0.01 and by less
    # above, and the others' sum by as much the other way; powers and sums add 2^-18 of their terms.  A term is the
    # sum of p s c and p lo, each rounded by itself, so its size is p (15 s + |lo|), not p |v|
    first, others = V[17], V[30:30 + n].mean(0)
    size = np.repeat(15 * s + np.abs(lo), 64, -1)
    tol = r * gap ** (r - 1) * 2.0 ** -19 * np.abs(first - others)
    tol = tol + 2.0 ** -18 * ((1 - n * p) * size[17] + p * size[30:30 + n].sum(0))
    assert (np.abs(f64_of(out[0, 0]) - want) <= tol).all()
    assert abs(float(tau[0, 0]) - (z[30] - p ** (alpha - 1))) <= 2.0 ** -18


# ------------------------------------------------------------------ outputs held to sharp bounds

@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.25, 1.5, 1.7, 2.0, 3.0, 10.0, 1000.0])
@pytest.mark.parametrize("G,Hkv,d,P", [(1, 3, 64, 16), (2, 1, 128, 32), (4, 2, 128, 16), (8, 1, 64, 64)])
def test_outputs_to_sharp_bounds(alpha, G, Hkv, d, P):
    """Every head within bounds that an output of zeros, or with its coordinates moved on by one, breaks."""
    c = Case(3, G * Hkv, Hkv, d, P, [1, P - 1, 700], seed=int(alpha * 10) + G)
    c.write(meta=False)
    check(c, alpha, *c.decode(alpha))
    assert nv.get_status() == 0


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.25, 1.5, 2.0, 3.0, 30.0])
@pytest.mark.parametrize("G,d,P", [(1, 64, 32), (4, 128, 16)])
def test_kept_pages_to_sharp_bounds(alpha, G, d, P):
    c = Case(1, 2 * G, 2, d, P, [900], seed=8)
    c.write()
    n = -(-900 // P)
    rng = np.random.RandomState(2)
    sel = np.full((1, c.Hq, c.mp), -9, np.int32)
    picks = [np.sort(rng.choice(n, 9, False)) for _ in range(c.Hq)]
    for h, p in enumerate(picks):
        sel[0, h, :9] = p
    out, tau = c.decode(alpha, torch.from_numpy(sel).cuda(), torch.full((1, c.Hq), 9, dtype=torch.int32, device="cuda"))
    out, tau = f64_of(out), f64_of(tau)
    for h, p in enumerate(picks):
        tok = (p[:, None] * P + np.arange(P)).reshape(-1)
        o, t, do, dt = head_of(c, 0, h, alpha, tok[tok < 900])
        assert (np.abs(out[0, h] - o) <= do).all(), (h, np.abs(out[0, h] - o).max(), do.max())
        assert abs(tau[0, h] - t) <= dt and (np.abs(o) > 4 * do).any()


@pytest.mark.parametrize("alpha", [1.0, 1.5, 2.0, 3.0, 10.0, 1000.0])
def test_the_bounds_are_sharp(alpha):
    """Without a GPU: an fp32 evaluation meets the bounds; zeros, another order of the coordinates, the uniform mean
    and the output of softmax (for entmax) or of entmax (for softmax) do not."""
    rng = np.random.RandomState(int(alpha))
    q, K, V = rng.randn(128), rng.randn(700, 128), rng.randn(700, 128)
    q, K, V = (exact.bf16(x) for x in (q, K, V))
    k, v = exact.quantise(K), exact.quantise(V)
    o, t, do, dt = exact.attention(q, k, v, alpha)
    Kf, Vf, qf = (np.asarray(x, np.float32) for x in (exact.values(*k), exact.values(*v), q))
    z = Kf @ qf * np.float32((alpha - 1 if alpha > 1 else 1) / np.sqrt(128))
    if alpha == 1:
        w = np.exp(z - z.max())
        w /= w.sum()
    else:
        w = np.maximum(z - np.float32(t), 0) ** np.float32(1 / (alpha - 1))
    near = w @ Vf
    assert (np.abs(near - o) <= do).all()
    other = exact.attention(q, k, v, 1.0 if alpha > 1 else 1.5)[0]
    for wrong in (0 * o, np.roll(o, 1), exact.values(*v).mean(0), other):
        assert (np.abs(wrong - o) > do).any()
    assert (np.abs(o) > 4 * do).any() and dt < 1e-3 * max(1, alpha - 1)
