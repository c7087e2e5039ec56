"""The 4-bit cache: rows in, rows out, metadata, and the attention over it, against plain 64-bit references; the
host-side refusals run without a GPU."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import kv4_ref as ref
from sparse_entmax_kv_b200 import kv4, native as nv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, FAKE_ODD = C.c_void_p(0x10000), C.c_void_p(0x10008)


def shp(**kw):
    d = dict(B=2, Hq=8, Hkv=2, d=128, page_size=32, max_pages=64, num_blocks=128, kv_begin=0, kv_count=0)
    d.update(kw)
    return nv.Shape(*[d[f] for f, _ in nv.Shape._fields_])


# ------------------------------------------------------------------ host side

def test_header_and_binding_agree():
    txt = open(os.path.join(ROOT, "include", "entmaxkv_kv4.h")).read()
    names = set(re.findall(r"ENTMAXKV_API\s+[\w\s\*]+?\b(entmaxkv_\w+)\s*\(", txt))
    assert names == set(kv4.EXPORTED)
    for n in names:
        assert hasattr(kv4.lib(), n)


def test_sizes():
    assert kv4.bytes_of(shp()) == 128 * 2 * 32 * 128 * 9 // 16
    assert kv4.bytes_of(shp(d=64, page_size=16)) == 128 * 2 * 16 * 64 * 9 // 16
    assert kv4.bytes_of(shp(d=96)) == 0
    assert kv4.workspace_size(shp()) >= 2 * 8 * 64 * 32 * 8  # z and row of every token and head
    assert kv4.workspace_size(shp(B=0)) == (1 << 64) - 1
    with pytest.raises(nv.EntmaxKVError, match="ERR_SHAPE"):
        kv4.alloc_cache(shp(d=96), "cpu")
    with pytest.raises(nv.EntmaxKVError, match="ERR_SHAPE"):
        kv4.alloc_workspace(shp(B=0), "cpu")


def test_argument_codes():
    L = kv4.lib()
    s = C.byref(shp())

    def rows(fn, sh=s, k=FAKE, v=FAKE, stride=256, start=FAKE, n=5, pt=FAKE, sl=FAKE, a=FAKE, b=FAKE, kind=0, meta=None):
        if fn == "write":
            return L.entmaxkv_kv4_write(sh, k, v, stride, start, n, pt, sl, a, b, meta, None)
        return L.entmaxkv_kv4_read(sh, a, b, stride, start, n, pt, sl, kind, k, v, None)
    for fn in ("write", "read"):
        assert rows(fn, sh=None) == -1
        for kw in (dict(k=None), dict(v=None), dict(pt=None), dict(sl=None), dict(a=None), dict(b=None)):
            assert rows(fn, **kw) == -1
        for kw in (dict(k=FAKE_ODD), dict(v=FAKE_ODD), dict(a=FAKE_ODD), dict(b=FAKE_ODD)):
            assert rows(fn, **kw) == -8
        assert rows(fn, stride=255) == -2      # shorter than a row
        assert rows(fn, stride=260) == -2      # not a multiple of 8
        assert rows(fn, n=-1) == -2
        assert rows(fn, start=None, n=3) == -2  # one row a sequence
        assert rows(fn, sh=C.byref(shp(d=96))) == -2
        assert rows(fn, sh=C.byref(shp(kv_begin=2))) == -2
    assert rows("write", meta=FAKE_ODD) == -8
    assert rows("read", kind=2) == -4

    need = kv4.workspace_size(shp())

    def dec(sh=s, q=FAKE, k=FAKE, v=FAKE, pt=FAKE, sl=FAKE, sel=None, cnt=None, a=1.5, out=FAKE, ws=FAKE, n=need):
        return L.entmaxkv_kv4_decode(sh, q, k, v, pt, sl, sel, cnt, a, out, None, ws, n, None)
    assert dec(sh=None) == -1
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(pt=None), dict(sl=None), dict(out=None),
               dict(sel=FAKE), dict(cnt=FAKE)):
        assert dec(**kw) == -1
    for kw in (dict(q=FAKE_ODD), dict(k=FAKE_ODD), dict(v=FAKE_ODD), dict(ws=C.c_void_p(0x10010))):
        assert dec(**kw) == -8
    for a in (0.5, float("nan"), float("inf")):
        assert dec(a=a) == -3
    assert dec(n=need - 1) == -5 and dec(ws=None) == -5
    assert dec(sh=C.byref(shp(Hq=6, Hkv=4))) == -2
    assert dec(sh=C.byref(shp(max_pages=200000)), sel=FAKE, cnt=FAKE, n=1 << 50) == -2


def test_binding_refuses_what_does_not_fit():
    sh = shp(num_blocks=4, max_pages=2)
    rows = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        kv4.entmaxkv_kv4_write(sh, rows, rows, None, i32(2, 2), i32(2), i32(1), i32(1))
    with pytest.raises(TypeError):
        kv4.entmaxkv_kv4_write(sh, rows.float(), rows, None, i32(2, 2), i32(2), i32(1), i32(1))
    with pytest.raises(ValueError, match="expected"):
        kv4.sized(i32(3), (2,), "x")


# ------------------------------------------------------------------ GPU

gpu = pytest.mark.gpu


def bits_of(t):
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def f64_of(t):
    return t.detach().cpu().double().numpy()


class Case:
    """A cache with random rows in random blocks, every byte that no token owns set to 255."""

    def __init__(self, B, Hq, Hkv, d, P, lens, seed=0, scale=1.0, rows=None):
        g = torch.Generator().manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.d, self.P, self.lens = B, Hq, Hkv, d, P, list(lens)
        self.mp = max(1, -(-max(lens) // P)) + 1
        nb = B * self.mp + 2
        self.shape = nv.Shape(B, Hq, Hkv, d, P, self.mp, nb)
        self.table = torch.randperm(nb, generator=g)[:B * self.mp].view(B, self.mp).int().cuda()
        self.seq = torch.tensor(lens, dtype=torch.int32).cuda()
        n = sum(lens)
        k = torch.randn(n, Hkv, d, generator=g) * torch.exp(0.5 * torch.randn(Hkv, d, generator=g)) * scale
        v = torch.randn(n, Hkv, d, generator=g)
        if rows is not None:
            rows(k, v)
        self.k, self.v = k.bfloat16().cuda(), v.bfloat16().cuda()
        self.q = torch.randn(B, Hq, d, generator=g).bfloat16().cuda()
        self.start = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()
        self.k4, self.v4 = kv4.alloc_cache(self.shape, "cuda")
        self.k4.fill_(255)
        self.v4.fill_(255)
        self.meta = torch.zeros(nv.meta_bytes(self.shape), dtype=torch.uint8, device="cuda")
        self.ws = kv4.alloc_workspace(self.shape, "cuda")

    def write(self, meta=True):
        kv4.entmaxkv_kv4_write(self.shape, self.k, self.v, self.start, self.table, self.seq, self.k4, self.v4,
                               self.meta if meta else None)

    def decode(self, alpha, sel=None, cnt=None, shape=None, ws=None, out=None, tau=None):
        out = torch.full((self.B, self.Hq, self.d), 7.0, device="cuda") if out is None else out
        tau = torch.full((self.B, self.Hq), 7.0, device="cuda") if tau is None else tau
        kv4.entmaxkv_kv4_decode(shape or self.shape, self.q, self.k4, self.v4, self.table, self.seq, alpha, out, tau,
                                sel, cnt, workspace=self.ws if ws is None else ws)
        return out, tau

    def rows_of(self, b):
        a = int(self.start[b])
        return slice(a, a + self.lens[b])

    def check_decode(self, alpha, out, tau, sel=None, cnt=None, heads=None):
        out, tau, q = f64_of(out), f64_of(tau), f64_of(self.q)
        sel_h = None if sel is None else sel.cpu().numpy()
        cnt_h = None if cnt is None else cnt.cpu().numpy()
        G = self.Hq // self.Hkv
        for b in range(self.B):
            rows = self.rows_of(b)
            Kc = ref.quantise(f64_of(self.k[rows]))
            Vc = ref.quantise(f64_of(self.v[rows]))
            K, V = ref.values(*Kc), ref.values(*Vc)
            for h in range(self.Hq) if heads is None else heads:
                tok = np.arange(self.lens[b])
                if sel is not None:
                    keep = sel_h[b, h, :cnt_h[b, h]]
                    tok = tok[np.isin(tok // self.P, keep)]
                o, t, p = ref.attention(q[b, h], K[tok, h // G], V[tok, h // G], alpha)
                if len(tok) == 0:
                    assert (out[b, h] == 0).all() and np.isnan(tau[b, h])
                    continue
                s = Kc[1][tok, h // G]
                do, dt = ref.attention_bounds(q[b, h], s, V[tok, h // G], p, alpha)
                assert np.abs(out[b, h] - o).max() <= do, (b, h, np.abs(out[b, h] - o).max(), do)
                assert abs(tau[b, h] - t) <= dt, (b, h, tau[b, h], t, dt)


def special_rows(k, v):
    n = k.shape[0]
    k[0] = 3.0                                   # a constant group: s = 0
    if n > 1:
        v[1] = 0.0
        k[1, :, :5] = 1e-40                      # subnormal spread: s below 2^-126
        k[1, :, 5:] = 0.0
    if n > 2:
        k[2] *= 1e30
        v[2] *= 1e30
    if n > 3:
        k[3, :, 1::2] = -k[3, :, 1::2].abs() * 1e-30


@gpu
@pytest.mark.parametrize("d,P", [(64, 16), (64, 64), (128, 16), (128, 32), (128, 64)])
def test_write_gives_the_documented_bytes(d, P):
    c = Case(5, 4, 2, d, P, [0, 1, P - 1, P + 1, 3 * P + 7], rows=special_rows)
    c.write()
    table = c.table.cpu().numpy()
    tile_bytes, per = 9 * d, P // 16
    got = [x.cpu().numpy().reshape(-1, 2, per, tile_bytes) for x in (c.k4, c.v4)]
    want = [np.full_like(x, 255) for x in got]
    for b in range(c.B):
        rows = c.rows_of(b)
        for which, x in enumerate((c.k, c.v)):
            codes, s, lo = ref.quantise(f64_of(x[rows]))
            for t0 in range(0, c.lens[b], 16):
                m = min(16, c.lens[b] - t0)
                for h in range(2):
                    cc, ss, ll = np.zeros((16, d), np.int64), np.zeros((16, d // 64)), np.zeros((16, d // 64))
                    cc[:m], ss[:m], ll[:m] = codes[t0:t0 + m, h], s[t0:t0 + m, h], lo[t0:t0 + m, h]
                    tile = want[which][table[b, t0 // P], h, (t0 % P) // 16]
                    mask = ref.code_mask(d, np.arange(m), which == 1)
                    tile[:] = (ref.pack_tile(cc, ss, ll, which == 1) & mask) | (tile & ~mask)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)
    # the metadata of every page, to the bit
    arrays = ref.meta_arrays(c.meta.cpu().numpy(), c.B, 2, c.mp, d)
    for b in range(c.B):
        K = ref.values(*ref.quantise(f64_of(c.k[c.rows_of(b)])))
        for p in range(-(-c.lens[b] // P)):
            for h in range(2):
                x = K[p * P:(p + 1) * P, h]
                for got_a, want_a in zip(arrays, ref.record(x, x.shape[0])):
                    np.testing.assert_array_equal(got_a[b, h, p], want_a)
        for p in range(-(-c.lens[b] // P), arrays[0].shape[2]):
            assert not arrays[2][b, :, p].any()
    assert nv.get_status() == 0


@gpu
@pytest.mark.parametrize("d,P", [(64, 16), (128, 32)])
def test_tokens_one_by_one_give_the_prompt_bytes(d, P):
    """Appending (no row_start) and chunks of prompts leave the same cache and metadata as one write."""
    lens = [P + 3, 2 * P, 5]
    a, b = Case(3, 2, 1, d, P, lens), Case(3, 2, 1, d, P, lens)
    a.write()
    cut = [7, P + 1, 5]
    first = torch.tensor([0] + list(np.cumsum(cut)), dtype=torch.int32).cuda()
    k0 = torch.cat([b.k[b.rows_of(i)][:cut[i]] for i in range(3)])
    v0 = torch.cat([b.v[b.rows_of(i)][:cut[i]] for i in range(3)])
    kv4.entmaxkv_kv4_write(b.shape, k0, v0, first, b.table, torch.tensor(cut, dtype=torch.int32).cuda(), b.k4, b.v4,
                           b.meta)
    at = list(cut)
    while at != lens:
        # sequences that are done have length 0 for the step: skipped
        step = [x + 1 if x < l else 0 for x, l in zip(at, lens)]
        rows = [int(b.start[i]) + max(0, min(at[i], lens[i] - 1)) for i in range(3)]
        kv4.entmaxkv_kv4_write(b.shape, b.k[rows], b.v[rows], None, b.table,
                               torch.tensor(step, dtype=torch.int32).cuda(), b.k4, b.v4, b.meta)
        at = [max(x, s) for x, s in zip(at, step)]
    assert torch.equal(a.k4, b.k4) and torch.equal(a.v4, b.v4) and torch.equal(a.meta, b.meta)
    assert nv.get_status() == 0


@gpu
@pytest.mark.parametrize("d,P,dtype", [(64, 16, torch.float32), (128, 64, torch.bfloat16), (128, 16, torch.float32)])
def test_read_back_and_strided_rows(d, P, dtype):
    """Rows inside a fused projection go in and come out by stride; only the tail asked for is written."""
    lens, Hkv = [4, P, 2 * P + 9], 3
    c = Case(3, 3, Hkv, d, P, lens)
    fused = torch.zeros(sum(lens), 2 * Hkv + 2, d, dtype=torch.bfloat16, device="cuda")
    fused[:, 1:1 + Hkv], fused[:, 1 + Hkv:1 + 2 * Hkv] = c.k, c.v
    kv4.entmaxkv_kv4_write(c.shape, fused[:, 1:1 + Hkv], fused[:, 1 + Hkv:1 + 2 * Hkv], c.start, c.table, c.seq,
                           c.k4, c.v4)
    tail = [0, P, P + 2]
    start = torch.tensor([0] + list(np.cumsum(tail)), dtype=torch.int32).cuda()
    out = torch.full((sum(tail), 2 * Hkv + 1, d), 5.0, dtype=dtype, device="cuda")
    kv4.entmaxkv_kv4_read(c.shape, c.k4, c.v4, start, c.table, c.seq, out[:, :Hkv], out[:, Hkv:2 * Hkv])
    assert (out[:, 2 * Hkv] == 5).all()
    for x, o in ((c.k, out[:, :Hkv]), (c.v, out[:, Hkv:2 * Hkv])):
        want = np.concatenate([ref.values(*ref.quantise(f64_of(x[c.rows_of(b)][c.lens[b] - tail[b]:])))
                               for b in range(3) if tail[b]])
        want = torch.from_numpy(want).float().to(dtype)
        assert torch.equal(o.cpu(), want)
    # one row a sequence: the last token
    last = [torch.empty(3, Hkv, d, dtype=dtype, device="cuda") for _ in range(2)]
    kv4.entmaxkv_kv4_read(c.shape, c.k4, c.v4, None, c.table, c.seq, *last)
    want = torch.from_numpy(ref.values(*ref.quantise(f64_of(c.k[[x - 1 for x in np.cumsum(lens)]])))).float().to(dtype)
    assert torch.equal(last[0].cpu(), want)


@gpu
def test_rows_that_do_not_fit_are_skipped_and_reported():
    c = Case(4, 2, 1, 64, 16, [20, 20, 20, 20])
    c.write()
    before = c.k4.clone()
    rows = torch.randn(8, 1, 64, device="cuda").bfloat16()
    nv.get_status(clear=True)

    def write(start, lens, table=None):
        kv4.entmaxkv_kv4_write(c.shape, rows, rows, torch.tensor(start, dtype=torch.int32).cuda(),
                               c.table if table is None else table, torch.tensor(lens, dtype=torch.int32).cuda(),
                               c.k4, c.v4, c.meta)
        return nv.get_status(clear=True)
    assert write([0, 0, 0, 0, 9], [20] * 4) == nv.STATUS_BAD_LENGTH        # rows past the end
    assert write([0, 3, 1, 1, 1], [1, 20, 20, 20]) == nv.STATUS_BAD_LENGTH  # 3 rows for a length of 1; a row of -2
    assert write([0, 1, 1, 1, 1], [c.mp * 16 + 1, 20, 20, 20]) == nv.STATUS_BAD_LENGTH
    assert torch.equal(before, c.k4)
    bad = c.table.clone()
    bad[0, 1] = c.shape.num_blocks
    assert write([0, 1, 1, 1, 1], [20] * 4, bad) == nv.STATUS_BAD_PAGE
    bad[0, 1] = -1
    assert write([0, 1, 1, 1, 1], [20] * 4, bad) == nv.STATUS_BAD_PAGE
    assert torch.equal(before, c.k4)
    assert write([0, 0, 0, 0, 0], [20] * 4) == 0                           # nothing to write
    empty = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    kv4.entmaxkv_kv4_write(c.shape, empty, empty, torch.zeros(5, dtype=torch.int32).cuda(), c.table, c.seq, c.k4, c.v4)
    assert torch.equal(before, c.k4)


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.25, 1.5, 1.7, 2.0])
@pytest.mark.parametrize("G,Hkv,d,P", [(1, 3, 64, 16), (2, 1, 128, 32), (4, 2, 128, 16), (8, 1, 64, 64), (1, 2, 128, 64)])
def test_decode_every_page(alpha, G, Hkv, d, P):
    c = Case(6, G * Hkv, Hkv, d, P, [1, 0, P, P - 1, 5 * P + 3, 1111], seed=int(alpha * 100) + G)
    c.write(meta=False)
    out, tau = c.decode(alpha)
    c.check_decode(alpha, out, tau)
    assert nv.get_status() == 0


@gpu
@pytest.mark.parametrize("B", [1, 5, 30, 80])
@pytest.mark.parametrize("G,Hkv,d,P", [(1, 2, 64, 16), (2, 2, 128, 32), (4, 2, 64, 64), (8, 2, 128, 16)])
def test_short_sequences(B, G, Hkv, d, P):
    """Softmax of sequences that one CTA takes whole, up to the lengths and numbers of groups where it stops."""
    rng = np.random.RandomState(B)
    lens = rng.randint(0, 400, B)
    lens[0] = 930 if B == 1 else 0
    lens[-1] = 1  # the table: 58 pages of 16 and one more
    if B == 80:
        lens[5] = 2900
    c = Case(B, G * Hkv, Hkv, d, P, [int(x) for x in lens] if B > 1 else [930], seed=B)
    c.q[-1, 0, 3] = float("inf")
    c.write(meta=False)
    nv.get_status(clear=True)
    out, tau = c.decode(1.0)
    assert nv.get_status(clear=True) == nv.STATUS_NONFINITE
    assert out[-1, 0].isnan().all() and bool(tau[-1, 0].isnan())
    c.q[-1, 0, 3] = 0.0
    out, tau = c.decode(1.0)
    c.check_decode(1.0, out, tau)


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.5, 2.0])
@pytest.mark.parametrize("G,Hkv,d,P", [(1, 2, 64, 16), (4, 2, 128, 32), (8, 1, 128, 64)])
def test_decode_kept_pages(alpha, G, Hkv, d, P):
    """Each head its own pages: none, the partial last one, all of them, a few."""
    c = Case(3, G * Hkv, Hkv, d, P, [700, 0, 5], seed=3)
    c.write()
    rng = np.random.RandomState(1)
    sel = np.full((3, c.Hq, c.mp), -9, np.int32)
    cnt = np.zeros((3, c.Hq), np.int32)
    for b in (0, 2):
        n = -(-c.lens[b] // P)
        for h in range(c.Hq):
            pick = [[], [n - 1], list(range(n)), sorted(rng.choice(n, max(1, n // 3), False))][(h + b) % 4]
            cnt[b, h] = len(pick)
            sel[b, h, :len(pick)] = pick
    sel, cnt = torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda()
    out, tau = c.decode(alpha, sel, cnt)
    c.check_decode(alpha, out, tau, sel, cnt)
    assert nv.get_status() == 0


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.5])
@pytest.mark.parametrize("ks,vs,qs", [(1e-20, 1.0, 1e20), (1e20, 1.0, 1e-20), (1.0, 1e30, 1.0), (1.0, 1e-25, 1.0),
                                      (1e-30, 1e-30, 1.0), (4.0, 1.0, 8.0)])
def test_scales(alpha, ks, vs, qs):
    """Keys, values and queries of any magnitude; the last case has scores far apart (one token takes nearly all)."""
    def rows(k, v):
        v *= vs
    c = Case(2, 4, 2, 128, 32, [700, 33], seed=9, scale=ks, rows=rows)
    c.q = (c.q.float() * qs).bfloat16()
    c.write(meta=False)
    out, tau = c.decode(alpha)
    c.check_decode(alpha, out, tau)
    assert nv.get_status() == 0


@gpu
@pytest.mark.parametrize("alpha", [1.05, 1.1, 3.0, 10.0])
def test_unusual_alphas(alpha):
    c = Case(2, 2, 1, 64, 16, [2000, 50], seed=4)
    c.write(meta=False)
    out, tau = c.decode(alpha)
    c.check_decode(alpha, out, tau)


@gpu
@pytest.mark.parametrize("alpha", [1.001, 1.01, 30.0, 1000.0])
def test_alphas_far_from_the_usual_ones(alpha):
    c = Case(2, 4, 2, 64, 16, [900, 1], seed=14)
    c.write(meta=False)
    out, tau = c.decode(alpha)
    c.check_decode(alpha, out, tau)
    assert nv.get_status() == 0


@gpu
def test_values_that_grow_along_the_sequence():
    """The reference of the softmax has to follow p s wherever it rises: steps 2^60 apart, scores 40 apart."""
    def rows(k, v):
        n = k.shape[0]
        v *= 2.0 ** torch.linspace(-30, 30, n)[:, None, None]
        k *= torch.linspace(0, 6, n)[:, None, None]
    c = Case(1, 4, 1, 64, 16, [900], seed=6, rows=rows)
    c.write(meta=False)
    c.check_decode(1.0, *c.decode(1.0))


@gpu
def test_constant_values():
    """Groups without a step (s = 0): only the offsets count, however large they are and wherever they appear."""
    def rows(k, v):
        v[:] = torch.arange(v.shape[0])[:, None, None] % 7 - 3.0
        v[200] = 1e30
        v[300] = -1e35
    c = Case(1, 4, 1, 64, 16, [500], seed=7, rows=rows)
    c.write(meta=False)
    c.check_decode(1.0, *c.decode(1.0))
    c.check_decode(1.5, *c.decode(1.5))


@gpu
@pytest.mark.parametrize("alpha,scale", [(1.25, 1.0), (1.25, 0.2), (1.5, 0.1)])
def test_more_candidates_than_fit_on_chip(alpha, scale):
    """Thousands of tokens above max z - 1: the histogram's cut, and supports beyond it."""
    c = Case(2, 2, 1, 64, 32, [40000, 12345], seed=8, scale=scale)
    c.write(meta=False)
    out, tau = c.decode(alpha)
    c.check_decode(alpha, out, tau)
    again = c.decode(alpha)
    assert torch.equal(out, again[0]) and torch.equal(tau, again[1])


@gpu
@pytest.mark.parametrize("alpha", [1.5, 2.0])
def test_large_supports(alpha):
    """All scores nearly equal: every token carries weight, far more than the threshold kernel holds on chip."""
    c = Case(2, 4, 2, 64, 32, [9000, 4096], scale=0.01)
    c.write(meta=False)
    out, tau = c.decode(alpha)
    c.check_decode(alpha, out, tau)


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.5])
def test_scores_and_selection_run_on_the_4bit_metadata(alpha):
    """The bound of the 4-bit keys' metadata bounds every score, and a selection by it that keeps every page gives the
    full result (lists of selections are cut among the warps in another way, so the sums are not the same to the bit)."""
    c = Case(2, 8, 2, 128, 32, [333, 64])
    c.write()
    bbox = torch.full((2, 8, c.mp), -1e30, device="cuda")
    nv.entmaxkv_score_pages(c.shape, c.q, c.meta, c.seq, bbox)
    sel = torch.empty((2, 8, c.mp), dtype=torch.int32, device="cuda")
    cnt = torch.empty((2, 8), dtype=torch.int32, device="cuda")
    nv.entmaxkv_select(c.shape, c.seq, bbox, None, None, nv.TOPK, c.mp, alpha, 0.0, sel, cnt)
    assert cnt.cpu().tolist() == [[11] * 8, [2] * 8]
    c.check_decode(alpha, *c.decode(alpha))
    c.check_decode(alpha, *c.decode(alpha, sel, cnt), sel, cnt)
    q, bound = f64_of(c.q), f64_of(bbox)
    for b in range(2):
        K = ref.values(*ref.quantise(f64_of(c.k[c.rows_of(b)])))
        for h in range(8):
            s = K[:, h // 4] @ q[b, h] / np.sqrt(128)
            for p in range(-(-c.lens[b] // 32)):
                top = s[p * 32:(p + 1) * 32].max()
                assert top <= bound[b, h, p] + abs(bound[b, h, p]) * 2.0 ** -23  # the bound is rounded once to fp32


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.5])
def test_values_that_are_not_finite(alpha):
    def rows(k, v):
        k[5, 0, 3] = float("nan")     # sequence 0, kv head 0
        v[20 + 4, 1, 70] = float("inf")  # sequence 1, kv head 1, second group
    c = Case(2, 4, 2, 128, 16, [20, 20], rows=rows)
    c.q[1, 0, 9] = float("nan")
    c.write(meta=False)
    nv.get_status(clear=True)
    out, tau = c.decode(alpha)
    assert nv.get_status(clear=True) == nv.STATUS_NONFINITE
    o = out.isnan().cpu()
    assert o[0, :2].all() and tau[0, :2].isnan().all()       # a NaN key reaches both heads of its group
    assert not o[0, 2:].any()
    assert o[1, 0].all() and bool(tau[1, 0].isnan())         # a query that is not finite
    assert not o[1, 1].any()
    if alpha == 1.0:                                         # every value row carries weight
        assert o[1, 2:, 64:].all() and not o[1, 2:, :64].any()
    back = torch.empty(40, 2, 128, device="cuda")
    kv4.entmaxkv_kv4_read(c.shape, c.k4, c.v4, c.start, c.table, c.seq, back, torch.empty_like(back))
    assert back[5, 0, :64].isnan().all() and not back[5, 0, 64:].isnan().any()


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.5])
def test_values_that_are_not_finite_in_pages_of_other_heads(alpha):
    """A page that only some heads of the group keep may hold anything for the others."""
    def rows(k, v):
        k[20, 0, 3] = float("inf")
        v[21] = float("nan")
    c = Case(1, 2, 1, 128, 16, [60], rows=rows)
    c.write(meta=False)
    sel = torch.zeros(1, 2, c.mp, dtype=torch.int32, device="cuda")
    sel[0, 0, :2] = torch.tensor([0, 3])
    sel[0, 1, :3] = torch.tensor([0, 1, 3])
    cnt = torch.tensor([[2, 3]], dtype=torch.int32, device="cuda")
    out, tau = c.decode(alpha, sel, cnt)
    assert out[0, 1].isnan().all() and bool(tau[0, 1].isnan())
    c.check_decode(alpha, out, tau, sel, cnt, heads=[0])
    assert nv.get_status(clear=True) == 0


@gpu
def test_bad_pages_and_lengths_in_decode():
    c = Case(2, 4, 2, 64, 16, [40, 40])
    c.write(meta=False)
    nv.get_status(clear=True)
    c.table[0, 1] = c.shape.num_blocks + 5
    out, tau = c.decode(1.5)
    assert nv.get_status(clear=True) == nv.STATUS_BAD_PAGE
    sel = torch.tensor([0, 2], dtype=torch.int32).cuda().expand(2, 4, 2)
    full = torch.zeros(2, 4, c.mp, dtype=torch.int32, device="cuda")
    full[..., :2] = sel
    cnt = torch.full((2, 4), 2, dtype=torch.int32, device="cuda")
    want, wtau = c.decode(1.5, full, cnt)
    assert torch.equal(out[0], want[0]) and torch.equal(tau[0], wtau[0])  # the bad page is skipped
    assert nv.get_status(clear=True) == 0
    c.seq[1] = c.mp * 16 + 100
    c.decode(1.0)
    assert nv.get_status(clear=True) & nv.STATUS_BAD_LENGTH


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.5])
@pytest.mark.parametrize("G", [1, 2])
def test_bad_selections(G, alpha):
    """Entries outside the sequence are left out, entries given twice count once, counts beyond the pages are cut."""
    c = Case(1, 2 * G, 2, 64, 16, [100])           # 7 pages
    c.write(meta=False)

    def run(entries, n):
        sel = torch.full((1, 2 * G, c.mp), 5, dtype=torch.int32, device="cuda")
        sel[0, :, :len(entries)] = torch.tensor(entries, dtype=torch.int32)
        cnt = torch.full((1, 2 * G), n, dtype=torch.int32, device="cuda")
        out, tau = c.decode(alpha, sel, cnt)
        return out, tau, nv.get_status(clear=True)
    nv.get_status(clear=True)
    want = run([0, 2, 5], 3)
    assert want[2] == 0
    twice = run([0, 0, 2, 5, 5], 5)
    assert twice[2] in (0, nv.STATUS_BAD_SELECTION)
    beyond = run([-1, 0, 2, 5, 7], 5)
    assert beyond[2] == nv.STATUS_BAD_SELECTION
    for got in (twice, beyond):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    none = run([0], -3)
    assert none[2] == nv.STATUS_BAD_SELECTION and (none[0] == 0).all() and none[1].isnan().all()
    assert run(list(range(7)), 8)[2] & nv.STATUS_BAD_SELECTION


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.5])
def test_head_ranges_share_a_workspace_and_streams(alpha):
    """Calls on disjoint kv-head ranges on two streams at once, one workspace: the bits of one call."""
    c = Case(3, 12, 6, 64, 16, [900, 77, 2000])
    c.write(meta=False)
    want, wtau = c.decode(alpha)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out, tau = torch.zeros_like(want), torch.zeros_like(wtau)
    for _ in range(3):
        for st, (k0, n) in zip(streams, ((0, 2), (2, 4))):
            with torch.cuda.stream(st):
                c.decode(alpha, shape=c.shape.kv_range(k0, n), out=out, tau=tau)
    torch.cuda.synchronize()
    # the split of the page list follows the number of groups in the call, so the sums may be cut elsewhere
    c.check_decode(alpha, out, tau)
    part, ptau = torch.full_like(out, 9.0), torch.full_like(tau, 9.0)
    c.decode(alpha, shape=c.shape.kv_range(2, 4), out=part, tau=ptau)
    assert (part[:, :4] == 9).all() and torch.equal(part[:, 4:], out[:, 4:])
    # writes of disjoint ranges too
    k4, v4 = c.k4.clone(), c.v4.clone()
    c.k4.fill_(255)
    c.v4.fill_(255)
    for k0, n in ((0, 2), (2, 4)):
        kv4.entmaxkv_kv4_write(c.shape.kv_range(k0, n), c.k, c.v, c.start, c.table, c.seq, c.k4, c.v4)
    assert torch.equal(k4, c.k4) and torch.equal(v4, c.v4)


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.5])
def test_captured_step_replays(alpha):
    """Write and decode in one graph, replayed with other rows and longer sequences; two graphs share a workspace."""
    c = Case(2, 8, 2, 128, 32, [500, 90])
    c.write()
    k_new, v_new = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(
        2, 2, 128, dtype=torch.bfloat16, device="cuda")
    out, tau = torch.empty(2, 8, 128, device="cuda"), torch.empty(2, 8, device="cuda")

    def step():
        kv4.entmaxkv_kv4_write(c.shape, k_new, v_new, None, c.table, c.seq, c.k4, c.v4, c.meta)
        c.decode(alpha, out=out, tau=tau)
    c.seq += 1
    step()  # warm-up on the first new token
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    gen = torch.Generator().manual_seed(4)
    ks, vs = [], []
    for i in range(4):
        if i:
            c.seq += 1
        k_new.copy_(torch.randn(2, 2, 128, generator=gen))
        v_new.copy_(torch.randn(2, 2, 128, generator=gen))
        ks.append(k_new.clone())
        vs.append(v_new.clone())
        graphs[i % 2].replay()
    rows = lambda x, new, b: torch.cat([x[c.rows_of(b)]] + [y[b:b + 1] for y in new])  # noqa: E731
    k, v = (torch.cat([rows(x, new, b) for b in range(2)]) for x, new in ((c.k, ks), (c.v, vs)))
    c.k, c.v, c.lens = k, v, [504, 94]
    c.start = torch.tensor([0, 504, 598], dtype=torch.int32).cuda()
    c.check_decode(alpha, out, tau)
    again = [torch.empty_like(out), torch.empty_like(tau)]
    c.decode(alpha, out=again[0], tau=again[1])
    assert torch.equal(again[0], out) and torch.equal(again[1], tau)


@gpu
def test_pinned_rows_and_output():
    c = Case(2, 8, 2, 64, 16, [33, 16])
    c.write()
    want, _ = c.decode(1.5)
    k = torch.randn(2, 2, 64).bfloat16().pin_memory()
    v = torch.randn(2, 2, 64).bfloat16().pin_memory()
    kv4.entmaxkv_kv4_write(c.shape, k, v, None, c.table, c.seq, c.k4, c.v4)
    back = [torch.empty(2, 2, 64, device="cuda") for _ in range(2)]
    kv4.entmaxkv_kv4_read(c.shape, c.k4, c.v4, None, c.table, c.seq, *back)
    assert torch.equal(back[1].cpu(), torch.from_numpy(ref.values(*ref.quantise(v.double().numpy()))).float())
    host = torch.empty(2, 8, 64).pin_memory()
    out, _ = c.decode(1.5)
    c.decode(1.5, out=host)
    torch.cuda.synchronize()
    assert torch.equal(host, out.cpu())


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.5])
def test_blocks_beyond_four_gigabytes(alpha):
    """Blocks at the far end of caches of 4.8 GB each."""
    nb = 130000
    shape = nv.Shape(1, 16, 8, 128, 64, 3, nb)
    assert kv4.bytes_of(shape) > 1 << 32
    k4, v4 = kv4.alloc_cache(shape, "cuda")
    c = Case(1, 16, 8, 128, 64, [150], seed=2)
    c.shape, c.k4, c.v4, c.mp = shape, k4, v4, 3
    c.table = torch.tensor([[nb - 1, 116600, nb - 2]], dtype=torch.int32, device="cuda")
    c.ws = kv4.alloc_workspace(shape, "cuda")
    c.write(meta=False)
    c.check_decode(alpha, *c.decode(alpha))
    back = [torch.empty(150, 8, 128, device="cuda") for _ in range(2)]
    kv4.entmaxkv_kv4_read(shape, k4, v4, c.start, c.table, c.seq, *back)
    for x, b in ((c.k, back[0]), (c.v, back[1])):
        assert torch.equal(b.cpu(), torch.from_numpy(ref.values(*ref.quantise(f64_of(x)))).float())
    assert nv.get_status() == 0


@gpu
@pytest.mark.parametrize("alpha", [1.0, 1.5])
def test_a_stream_that_is_given(alpha):
    """Calls go to the stream they are given, not to the current one."""
    c = Case(2, 8, 2, 64, 16, [500, 90])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    big = torch.empty(1 << 26, device="cuda")
    with torch.cuda.stream(side):
        big.fill_(1.0)  # keeps the side stream busy while the current one runs ahead
    kv4.entmaxkv_kv4_write(c.shape, c.k, c.v, c.start, c.table, c.seq, c.k4, c.v4, c.meta, stream=side)
    out, tau = torch.empty(2, 8, 64, device="cuda"), torch.empty(2, 8, device="cuda")
    kv4.entmaxkv_kv4_decode(c.shape, c.q, c.k4, c.v4, c.table, c.seq, alpha, out, tau, workspace=c.ws, stream=side)
    side.synchronize()
    c.check_decode(alpha, out, tau)


@gpu
def test_binding_refusals_on_the_gpu():
    c = Case(2, 4, 2, 64, 16, [10, 20])
    with pytest.raises(ValueError, match="packed"):
        kv4.entmaxkv_kv4_write(c.shape, c.k.transpose(0, 1).contiguous().transpose(0, 1), c.v, c.start, c.table, c.seq,
                               c.k4, c.v4)
    with pytest.raises(ValueError, match="one row a sequence"):
        kv4.entmaxkv_kv4_write(c.shape, c.k, c.v, None, c.table, c.seq, c.k4, c.v4)
    with pytest.raises(ValueError, match="k4"):
        kv4.entmaxkv_kv4_write(c.shape, c.k, c.v, c.start, c.table, c.seq, c.k4[16:], c.v4)
    with pytest.raises(ValueError, match="seq_lens"):
        kv4.entmaxkv_kv4_decode(c.shape, c.q, c.k4, c.v4, c.table, c.seq[:1], 1.5, torch.empty(2, 4, 64, device="cuda"),
                                workspace=c.ws)
    with pytest.raises(nv.EntmaxKVError, match="ERR_ALPHA"):
        c.decode(0.9)
    with pytest.raises(nv.EntmaxKVError, match="ERR_WORKSPACE"):
        c.decode(1.5, ws=c.ws[:256])
    assert nv.get_status() == 0
