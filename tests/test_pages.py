"""Counting, forking, growing, compacting and copying pages, against plain simulations; the refusals run without a
GPU.  At the end a run of everything together: prompts, decode steps, forks, compaction, over a 4-bit cache."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import kv4_ref as ref
from sparse_entmax_kv_b200 import kv4, native as nv, pages

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, FAKE2, FAKE_ODD = C.c_void_p(0x10000), C.c_void_p(0x20000), C.c_void_p(0x10008)


def shp(**kw):
    d = dict(B=2, Hq=8, Hkv=2, d=128, page_size=32, max_pages=64, num_blocks=128, kv_begin=0, kv_count=0)
    d.update(kw)
    return nv.Shape(*[d[f] for f, _ in nv.Shape._fields_])


def cbufs(*ptrs, size=1024):
    base = (C.c_void_p * max(1, len(ptrs)))(*ptrs)
    b = pages._CBuffers(len(ptrs), size, base)
    b.keep = base
    return b


# ------------------------------------------------------------------ host side

def test_header_and_binding_agree():
    txt = open(os.path.join(ROOT, "include", "entmaxkv_pages.h")).read()
    names = set(re.findall(r"ENTMAXKV_API\s+[\w\s\*]+?\b(entmaxkv_\w+)\s*\(", txt))
    assert names == set(pages.EXPORTED)
    for n in names:
        assert hasattr(pages.lib(), n)
    bits = dict(re.findall(r"ENTMAXKV_STATUS_(\w+)\s*=\s*(\d+)", txt))
    assert bits == {"NO_BLOCK": str(pages.STATUS_NO_BLOCK), "BAD_ROW": str(pages.STATUS_BAD_ROW)}
    assert f"ENTMAXKV_MAX_BUFFERS {pages.MAX_BUFFERS}" in txt


def test_argument_codes():
    L = pages.lib()
    s = C.byref(shp())
    n = pages.workspace_size(shp())
    assert n >= 128 * 4 and pages.workspace_size(shp(d=96)) == (1 << 64) - 1
    assert pages.workspace_size(shp(kv_count=1)) == (1 << 64) - 1     # pages hold every head
    ok = cbufs(0x30000)

    def refs(sh=s, pt=FAKE, sl=FAKE, r=FAKE, f=None, ws=FAKE, m=n):
        return L.entmaxkv_pages_refs(sh, pt, sl, None, r, f, ws, m, None)

    def fork(sh=s, par=FAKE, ti=FAKE, li=FAKE, to=FAKE2, lo=FAKE2, b=ok, mi=None, mo=None, ws=FAKE, m=n):
        r = lambda x: None if x is None else C.byref(x)  # noqa: E731
        return L.entmaxkv_pages_fork(sh, par, ti, li, None, to, lo, r(b), r(mi), r(mo), ws, m, None)

    def grow(sh=s, add=FAKE, pt=FAKE, sl=FAKE, ws=FAKE, m=n):
        return L.entmaxkv_pages_grow(sh, add, None, pt, sl, ws, m, None)

    def compact(sh=s, ti=FAKE, li=FAKE, to=FAKE, b=ok, rm=FAKE, nl=FAKE, ws=FAKE, m=n):
        return L.entmaxkv_pages_compact(sh, ti, li, None, to, None if b is None else C.byref(b), rm, nl, ws, m, None)
    for fn in (refs, fork, grow, compact):
        assert fn(sh=None) == -1
        assert fn(sh=C.byref(shp(d=96))) == -2
        assert fn(sh=C.byref(shp(kv_begin=1))) == -2
        assert fn(ws=None) == -5 and fn(m=n - 1) == -5
        assert fn(ws=C.c_void_p(0x10010)) == -8
    assert refs(pt=None) == -1 and refs(sl=None) == -1 and refs(r=None) == -1
    for kw in (dict(par=None), dict(ti=None), dict(li=None), dict(to=None), dict(lo=None), dict(b=None),
               dict(mi=cbufs(0x40000))):
        assert fork(**kw) == -1
    assert fork(b=cbufs(0x30008)) == -8
    assert fork(b=cbufs(0x30000, size=1000)) == -2
    assert fork(b=cbufs(0x30000, size=0)) == -2
    assert fork(b=cbufs(0)) == -1
    too_many = cbufs(0x30000)
    too_many.count = 257
    assert fork(b=too_many) == -2
    assert fork(to=FAKE) == -2 and fork(lo=FAKE) == -2                # in place: both or neither
    assert fork(mi=cbufs(0x40000), mo=cbufs(0x40000)) == -2           # metadata too
    assert fork(mi=cbufs(0x40000), mo=cbufs(0x50000, 0x60000)) == -2
    for kw in (dict(add=None), dict(pt=None), dict(sl=None)):
        assert grow(**kw) == -1
    for kw in (dict(ti=None), dict(li=None), dict(to=None), dict(b=None), dict(rm=None), dict(nl=None)):
        assert compact(**kw) == -1
    two = cbufs(0x30000, 0x40000)

    def copy(a=ok, na=4, b=ok, nb=4, si=FAKE, di=FAKE, k=2):
        return L.entmaxkv_pages_copy(C.byref(a), na, C.byref(b), nb, si, di, k, None)
    assert copy(b=two) == -2 and copy(b=cbufs(0x30000, size=2048)) == -2
    assert copy(na=0) == -2 and copy(nb=0) == -2 and copy(k=-1) == -2
    assert copy(si=None) == -1 and copy(di=None) == -1
    assert copy(a=cbufs(0x30008)) == -8
    assert copy(k=0) == 0


def test_buffers_check_what_they_are_given():
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA or pinned"):
        pages.Buffers([x])
    with pytest.raises(ValueError, match="at most"):
        pages.Buffers([x] * 257)
    for empty in (torch.zeros(0, 16), torch.zeros(4, 0), torch.tensor(1.0)):
        with pytest.raises(ValueError, match="at least one block"):
            pages.Buffers([empty])
    for n in (0, -4):
        with pytest.raises(ValueError, match="at least one block"):
            pages.Buffers([x], num_blocks=n)
    assert pages.Buffers([]).c.count == 0


# ------------------------------------------------------------------ GPU

gpu = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Pool:
    def __init__(self, B, P, mp, nb, lens, seed=0, share=True, bufs=3, words=24):
        rng = np.random.RandomState(seed)
        self.B, self.P, self.mp, self.nb, self.lens = B, P, mp, nb, np.asarray(lens, np.int32)
        self.shape = nv.Shape(B, 1, 1, 64, P, mp, nb)
        self.table = rng.randint(-5, nb + 5, (B, mp)).astype(np.int32)  # past the pages: anything
        perm, used = rng.permutation(nb), 0
        for b in range(B):
            n = -(-int(lens[b]) // P)
            common = min(int(lens[b - 1]) // P, int(lens[b]) // P) // 2 if share and b % 2 else 0
            self.table[b, :common] = self.table[b - 1, :common]
            self.table[b, common:n] = perm[used:used + n - common]
            used += n - common
        self.data = torch.randint(-2 ** 31, 2 ** 31 - 1, (bufs, nb, words), dtype=torch.int32, device="cuda")
        self.buffers = pages.Buffers(self.data.unbind(0))
        self.ws = torch.full((pages.workspace_size(self.shape),), 171, dtype=torch.uint8, device="cuda")

    def host_data(self):
        return self.data.cpu().numpy().copy()


@gpu
@pytest.mark.parametrize("hold", [False, True])
def test_refs(hold):
    p = Pool(5, 16, 9, 100, [0, 1, 16, 130, 144], seed=1)
    h = np.random.RandomState(2).randint(-1, 3, 100) if hold else None
    refs, free = torch.full((100,), 9, dtype=torch.int32, device="cuda"), i32([7])
    pages.entmaxkv_pages_refs(p.shape, i32(p.table), i32(p.lens), refs, free, None if h is None else i32(h),
                              workspace=p.ws)
    want = ref.used_blocks(p.table, p.lens, 16, 100, h)
    np.testing.assert_array_equal(refs.cpu().numpy(), want)
    assert int(free) == int((want == 0).sum())
    free.fill_(0)
    pages.entmaxkv_pages_refs(p.shape, i32(p.table), i32(p.lens), None, free, None if h is None else i32(h),
                              workspace=p.ws)
    assert int(free) == int((want == 0).sum()) and nv.get_status() == 0


FORKS = [
    (1, [33], [0]),
    (4, [5, 16, 31, 0], [0, 0, 0, 0]),          # one parent for all: the parent keeps its page
    (4, [5, 16, 31, 0], [2, 2, 3, 2]),          # the parent itself goes: the first child keeps
    (4, [5, 16, 31, 47], [1, 0, 3, 2]),         # a permutation
    (6, [1, 15, 17, 100, 64, 2], [-1, 3, 3, -1, 5, 5]),
    (40, list(np.random.RandomState(5).randint(0, 120, 40)), list(np.random.RandomState(6).randint(-1, 40, 40))),
]


@gpu
@pytest.mark.parametrize("B,lens,parent", FORKS)
@pytest.mark.parametrize("hold", [False, True])
def test_fork(B, lens, parent, hold):
    p = Pool(B, 16, 10, 12 * B + 8, lens, seed=B)
    h = (np.arange(p.nb) % 7 == 0).astype(np.int32) if hold else None
    want_t, want_l, pairs, short = ref.fork(parent, p.table, p.lens, 16, p.nb, h)
    want = p.host_data()
    for s, d in pairs:
        want[:, d] = want[:, s]
    t_out, l_out = torch.full((B, 10), 77, dtype=torch.int32, device="cuda"), i32([77] * B)
    table, lens_d = i32(p.table), i32(p.lens)
    pages.entmaxkv_pages_fork(p.shape, i32(parent), table, lens_d, t_out, l_out, p.buffers,
                              hold=None if h is None else i32(h), workspace=p.ws)
    assert not short and nv.get_status() == 0
    np.testing.assert_array_equal(t_out.cpu().numpy(), want_t)
    np.testing.assert_array_equal(l_out.cpu().numpy(), want_l)
    np.testing.assert_array_equal(p.host_data(), want)
    np.testing.assert_array_equal(table.cpu().numpy(), p.table)  # the old table is only read


@gpu
@pytest.mark.parametrize("bufs,metas", [(17, 1), (2, 17)])
def test_many_buffers(bufs, metas):
    """Beyond the numbers of buffers that the small launches have room for: fork, and compaction."""
    p = Pool(3, 16, 4, 30, [20, 35, 1], seed=3, bufs=bufs)
    parent = [1, 1, 0]
    want_t, want_l, pairs, _ = ref.fork(parent, p.table, p.lens, 16, 30)
    want = p.host_data()
    for s, d in pairs:
        want[:, d] = want[:, s]
    n = nv.meta_bytes(p.shape)
    a = torch.randint(0, 256, (metas, n), dtype=torch.uint8, device="cuda")
    o = torch.zeros_like(a)
    t_out, l_out = i32(np.zeros((3, 4))), i32([0] * 3)
    pages.entmaxkv_pages_fork(p.shape, i32(parent), i32(p.table), i32(p.lens), t_out, l_out, p.buffers,
                              pages.Buffers(a.unbind(0)), pages.Buffers(o.unbind(0)), workspace=p.ws)
    np.testing.assert_array_equal(t_out.cpu().numpy(), want_t)
    np.testing.assert_array_equal(p.host_data(), want)
    cut = 3 * 128 * 64
    for base, size in ((0, 128 * 64), (cut, 256 * 64)):
        for b, q in enumerate(parent):
            assert torch.equal(o[:, base + b * size:base + (b + 1) * size], a[:, base + q * size:base + (q + 1) * size])
    want_t, remap, live, pairs = ref.compact(want_t, want_l, 16, 30)
    for s, d in pairs:
        want[:, d] = want[:, s]
    r_out, n_live = i32([0] * 30), i32([0])
    pages.entmaxkv_pages_compact(p.shape, t_out, l_out, t_out, p.buffers, r_out, n_live, workspace=p.ws)
    assert int(n_live) == live and nv.get_status() == 0
    np.testing.assert_array_equal(p.host_data(), want)


@gpu
def test_fork_without_enough_blocks():
    p = Pool(4, 16, 3, 6, [20, 0, 0, 0], share=False)
    parent = [0, 0, 0, 0]
    hold = np.zeros(6, np.int32)
    hold[[i for i in range(6) if i not in p.table[0, :2]][:3]] = 1  # one block is left
    want_t, want_l, pairs, short = ref.fork(parent, p.table, p.lens, 16, 6, hold)
    assert short and len(pairs) == 1 and list(want_l) == [20, 20, 16, 16]
    t_out, l_out = i32(np.zeros((4, 3))), i32([0] * 4)
    pages.entmaxkv_pages_fork(p.shape, i32(parent), i32(p.table), i32(p.lens), t_out, l_out, p.buffers,
                              hold=i32(hold), workspace=p.ws)
    assert nv.get_status() == pages.STATUS_NO_BLOCK
    np.testing.assert_array_equal(t_out.cpu().numpy(), want_t)
    np.testing.assert_array_equal(l_out.cpu().numpy(), want_l)


@gpu
def test_fork_in_place():
    p = Pool(6, 16, 5, 60, [33, 0, 70, 0, 16, 5])
    parent = [0, 0, 2, 2, -1, 5]                # two forks into empty rows, one row freed
    want_t, want_l, pairs, _ = ref.fork(parent, p.table, p.lens, 16, 60)
    want = p.host_data()
    for s, d in pairs:
        want[:, d] = want[:, s]
    n = nv.meta_bytes(p.shape)
    meta = torch.randint(0, 256, (2, n), dtype=torch.uint8, device="cuda")
    want_meta = meta.cpu().numpy().copy()
    tiles, cut = 1, 6 * 128 * 64
    for b, q in ((1, 0), (3, 2)):
        for base, size in ((0, 128 * 64), (cut, 256 * 64)):
            want_meta[:, base + b * size * tiles:base + (b + 1) * size * tiles] = \
                want_meta[:, base + q * size * tiles:base + (q + 1) * size * tiles]
    table, lens = i32(p.table), i32(p.lens)
    metas = pages.Buffers(meta.unbind(0))
    pages.entmaxkv_pages_fork(p.shape, i32(parent), table, lens, table, lens, p.buffers, metas, metas, workspace=p.ws)
    assert nv.get_status() == 0
    got = table.cpu().numpy()
    for b in (0, 2, 5):                          # rows that stay are not touched, behind their pages neither
        np.testing.assert_array_equal(got[b], p.table[b])
    for b in (1, 3, 4):
        np.testing.assert_array_equal(got[b], want_t[b])
    np.testing.assert_array_equal(lens.cpu().numpy(), want_l)
    np.testing.assert_array_equal(p.host_data(), want)
    np.testing.assert_array_equal(meta.cpu().numpy(), want_meta)


@gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_fork_refuses_bad_parents(in_place):
    p = Pool(5, 16, 5, 60, [33, 20, 40, 10, 5])
    parent = [0, 9, -2, 4, 0]                    # 9 and -2 do not exist; in place row 4 is overwritten: not a parent
    table, lens = i32(p.table), i32(p.lens)
    t_out, l_out = (table, lens) if in_place else (i32(np.zeros((5, 5))), i32([9] * 5))
    pages.entmaxkv_pages_fork(p.shape, i32(parent), table, lens, t_out, l_out, p.buffers, workspace=p.ws)
    assert nv.get_status() == pages.STATUS_BAD_ROW
    effective = [0, 1, 2, 3, 0] if in_place else [0, -1, -1, 4, 0]
    want_t, want_l, _, _ = ref.fork(effective, p.table, p.lens, 16, 60)
    for b in range(5):
        n = -(-int(want_l[b]) // 16)
        np.testing.assert_array_equal(t_out.cpu().numpy()[b, :n], want_t[b, :n])
    np.testing.assert_array_equal(l_out.cpu().numpy(), want_l)


@gpu
@pytest.mark.parametrize("Hkv,d,mp", [(1, 64, 5), (3, 128, 70)])
def test_fork_moves_metadata(Hkv, d, mp):
    """Records of a row's pages follow it; records behind the row's last tile stay."""
    B, P = 4, 16
    lens = np.array([1, mp * P, 33 * P if mp > 33 else P, 0], np.int32)
    shape = nv.Shape(B, Hkv, Hkv, d, P, mp, B * mp)
    table = np.arange(B * mp, dtype=np.int32).reshape(B, mp)
    parent = [1, 2, 0, 1]
    a = torch.randint(0, 256, (2, nv.meta_bytes(shape)), dtype=torch.uint8, device="cuda")
    o = torch.full_like(a, 3)
    tiles = -(-mp // 32)
    want = o.cpu().numpy().copy()
    src, nt = a.cpu().numpy(), B * Hkv * tiles
    for b, q in enumerate(parent):
        used = -(-(-(-int(lens[q]) // P)) // 32)
        for base, size in ((0, 128 * d), (nt * 128 * d, 256 * d)):
            for h in range(Hkv):
                x, y = ((r * Hkv + h) * tiles * size + base for r in (b, q))
                want[:, x:x + used * size] = src[:, y:y + used * size]
    ws = pages.alloc_workspace(shape, "cuda")
    pages.entmaxkv_pages_fork(shape, i32(parent), i32(table), i32(lens), i32(table * 0), i32(lens), pages.Buffers([]),
                              pages.Buffers(a.unbind(0)), pages.Buffers(o.unbind(0)), workspace=ws)
    np.testing.assert_array_equal(o.cpu().numpy(), want)


@gpu
@pytest.mark.parametrize("hold", [False, True])
@pytest.mark.parametrize("B", [1, 7, 1500])
def test_grow(B, hold):
    rng = np.random.RandomState(B)
    lens = rng.randint(0, 60, B)
    add = rng.randint(-1, 70, B)
    add[rng.rand(B) < 0.4] = 1
    mp, P = 8, 16
    p = Pool(B, P, mp, 9 * B + 3, lens, seed=B)
    h = (np.arange(p.nb) % 5 == 0).astype(np.int32) if hold else None
    want_t, want_l, short = ref.grow(add, p.table, p.lens, P, p.nb, h)
    table, lens_d = i32(p.table), i32(p.lens)
    pages.entmaxkv_pages_grow(p.shape, i32(add), table, lens_d, None if h is None else i32(h), workspace=p.ws)
    too_long = ((p.lens + add > mp * P) & (add > 0)).any()
    assert nv.get_status() == (nv.STATUS_BAD_LENGTH if too_long else 0) | (pages.STATUS_NO_BLOCK if short else 0)
    np.testing.assert_array_equal(table.cpu().numpy(), want_t)
    np.testing.assert_array_equal(lens_d.cpu().numpy(), want_l)


@gpu
@pytest.mark.parametrize("B,mp,nb", [(3, 5, 7168 * 32), (3, 5, 7168 * 32 + 1), (4, 16384, 70000), (4, 16385, 70000),
                                     (1024, 3, 5000), (1025, 3, 5000)])
def test_where_the_plan_moves_off_the_chip(B, mp, nb):
    """Pools and tables around the sizes up to which one CTA marks the blocks and keeps the rows by itself."""
    P = 16
    rng = np.random.RandomState(nb)
    lens = rng.randint(0, min(mp, 40) * P, B)
    p = Pool(B, P, mp, nb, lens, seed=1, words=4, bufs=1)
    parent = rng.randint(-1, B, B)
    want_t, want_l, pairs, short = ref.fork(parent, p.table, p.lens, P, nb)
    want = p.host_data()
    for s, d in pairs:
        want[:, d] = want[:, s]
    t_out, l_out = torch.full((B, mp), 77, dtype=torch.int32, device="cuda"), i32([77] * B)
    pages.entmaxkv_pages_fork(p.shape, i32(parent), i32(p.table), i32(p.lens), t_out, l_out, p.buffers, workspace=p.ws)
    assert not short and nv.get_status() == 0
    np.testing.assert_array_equal(t_out.cpu().numpy(), want_t)
    np.testing.assert_array_equal(l_out.cpu().numpy(), want_l)
    add = rng.randint(0, 3, B)
    want_t, want_l, short = ref.grow(add, want_t, want_l, P, nb)
    pages.entmaxkv_pages_grow(p.shape, i32(add), t_out, l_out, workspace=p.ws)
    np.testing.assert_array_equal(t_out.cpu().numpy(), want_t)
    np.testing.assert_array_equal(l_out.cpu().numpy(), want_l)
    want_t, remap, live, pairs = ref.compact(want_t, want_l, P, nb)
    for s, d in pairs:
        want[:, d] = want[:, s]
    r_out, n_live = i32([-7] * nb), i32([-7])
    pages.entmaxkv_pages_compact(p.shape, t_out, l_out, t_out, p.buffers, r_out, n_live, workspace=p.ws)
    assert int(n_live) == live and nv.get_status(clear=True) in (0, nv.STATUS_BAD_LENGTH)
    np.testing.assert_array_equal(r_out.cpu().numpy(), remap)
    np.testing.assert_array_equal(t_out.cpu().numpy(), want_t)
    np.testing.assert_array_equal(p.host_data(), want)


@gpu
def test_grow_by_prompts():
    """Thousands of pages for one row beside rows that need one or none."""
    B, mp, P, nb = 40, 9000, 16, 30000
    lens = np.zeros(B, np.int64)
    lens[5], lens[6] = 31, 32
    add = np.ones(B, np.int64)
    add[3], add[7], add[11] = 8999 * 16 + 3, 700 * 16, 0
    p = Pool(B, P, mp, nb, lens, seed=2, share=False, words=4, bufs=1)
    want_t, want_l, short = ref.grow(add, p.table, p.lens, P, nb)
    assert not short
    table, lens_d = i32(p.table), i32(p.lens)
    pages.entmaxkv_pages_grow(p.shape, i32(add), table, lens_d, workspace=p.ws)
    assert nv.get_status() == 0
    np.testing.assert_array_equal(table.cpu().numpy(), want_t)
    np.testing.assert_array_equal(lens_d.cpu().numpy(), want_l)


@gpu
def test_grow_without_enough_blocks():
    """Needs are counted in order, those that fail too; a row that needs no block grows all the same."""
    p = Pool(5, 16, 6, 10, [16, 16, 10, 0, 16], share=False)
    add = [33, 80, 3, 16, 16]                    # needs 3, 5, 0, 1, 1 of 6 free blocks
    want_t, want_l, short = ref.grow(add, p.table, p.lens, 16, 10)
    assert short and list(want_l) == [49, 16, 13, 0, 16]
    table, lens = i32(p.table), i32(p.lens)
    pages.entmaxkv_pages_grow(p.shape, i32(add), table, lens, workspace=p.ws)
    assert nv.get_status() == pages.STATUS_NO_BLOCK
    np.testing.assert_array_equal(table.cpu().numpy(), want_t)
    np.testing.assert_array_equal(lens.cpu().numpy(), want_l)


@gpu
@pytest.mark.parametrize("B,nb,words,in_place", [(1, 4, 4, False), (3, 33, 28, True), (8, 1000, 4096, False),
                                                 (9, 5000, 4, True), (60, 40000, 4, False)])
def test_compact(B, nb, words, in_place):
    rng = np.random.RandomState(nb)
    mp = max(1, min(nb // B // 2, 300))
    lens = rng.randint(0, mp * 16 + 1, B)
    p = Pool(B, 16, mp, nb, lens, seed=nb, words=words, bufs=2)
    hold = (rng.rand(nb) < 0.05).astype(np.int32) if nb > 100 else None
    want_t, remap, live, pairs = ref.compact(p.table, p.lens, 16, nb, hold)
    want = p.host_data()
    for s, d in pairs:
        want[:, d] = want[:, s]
    table = i32(p.table)
    t_out = table if in_place else i32(np.zeros((B, mp)))
    r_out, n_live = i32([-7] * nb), i32([-7])
    pages.entmaxkv_pages_compact(p.shape, table, i32(p.lens), t_out, p.buffers, r_out, n_live,
                                 None if hold is None else i32(hold), workspace=p.ws)
    assert nv.get_status() == 0
    assert int(n_live) == live
    np.testing.assert_array_equal(r_out.cpu().numpy(), remap)
    np.testing.assert_array_equal(t_out.cpu().numpy(), want_t)
    np.testing.assert_array_equal(p.host_data(), want)


@gpu
@pytest.mark.parametrize("nb,words,n,bufs", [(5, 4, 1, 1), (40, 4096 + 4, 17, 3), (9, 33000, 9, 5), (700, 12, 700, 2), (6, 8, 4, 17)])
def test_copy(nb, words, n, bufs):
    g = torch.Generator().manual_seed(nb)
    a = torch.randint(-9, 9, (bufs, nb, words), dtype=torch.int32).cuda()
    b = torch.zeros(bufs, nb + 3, words, dtype=torch.int32, device="cuda")
    src, dst = torch.randint(0, nb, (n,), generator=g), torch.randperm(nb + 3, generator=g)[:n]
    want = b.clone()
    want[:, dst.cuda()] = a[:, src.cuda()]
    pages.entmaxkv_pages_copy(pages.Buffers(a.unbind(0)), pages.Buffers(b.unbind(0)), src.int().cuda(), dst.int().cuda())
    assert torch.equal(b, want)


@gpu
def test_copy_beyond_four_gigabytes():
    """Blocks at the far end of a 5 GB buffer, and blocks that end inside a chunk."""
    words, nb = 32768 + 4, 38000
    a = torch.empty(nb, words, dtype=torch.int32, device="cuda")
    a[nb - 1].copy_(torch.arange(words, dtype=torch.int32))
    a[nb - 2].fill_(7)
    b = torch.zeros(2, words, dtype=torch.int32, device="cuda")
    pages.entmaxkv_pages_copy(pages.Buffers([a]), pages.Buffers([b]), i32([nb - 1, nb - 2]), i32([1, 0]))
    assert torch.equal(b[1].cpu(), torch.arange(words, dtype=torch.int32)) and (b[0] == 7).all()
    pages.entmaxkv_pages_copy(pages.Buffers([b]), pages.Buffers([a]), i32([1]), i32([nb - 3]))
    assert torch.equal(a[nb - 3], b[1])


@gpu
def test_copy_to_pinned_memory_and_bad_ids():
    a = torch.randint(-9, 9, (2, 8, 64), dtype=torch.int32).cuda()
    host = torch.zeros(2, 4, 64, dtype=torch.int32).pin_memory()
    nv.get_status(clear=True)
    pages.entmaxkv_pages_copy(pages.Buffers(a.unbind(0)), pages.Buffers(host.unbind(0)), i32([7, 3, 8, 2, -1]),
                              i32([0, 3, 1, 4, 2]))
    torch.cuda.synchronize()
    assert nv.get_status(clear=True) == nv.STATUS_BAD_PAGE
    assert torch.equal(host[:, 0], a[:, 7].cpu()) and torch.equal(host[:, 3], a[:, 3].cpu())
    assert not host[:, 1:3].any()
    back = torch.zeros_like(a)
    pages.entmaxkv_pages_copy(pages.Buffers(host.unbind(0)), pages.Buffers(back.unbind(0)), i32([0, 3]), i32([5, 6]))
    assert torch.equal(back[:, 5], a[:, 7]) and torch.equal(back[:, 6], a[:, 3])


@gpu
def test_bad_entries_and_lengths_are_reported():
    p = Pool(2, 16, 4, 20, [40, 30], share=False)
    p.table[0, 1], p.table[1, 0] = 20, -1
    nv.get_status(clear=True)
    refs = i32([0] * 20)
    pages.entmaxkv_pages_refs(p.shape, i32(p.table), i32(p.lens), refs, workspace=p.ws)
    assert nv.get_status(clear=True) == nv.STATUS_BAD_PAGE
    np.testing.assert_array_equal(refs.cpu().numpy(), ref.used_blocks(p.table, p.lens, 16, 20))
    t_out, r_out, n_live = i32(np.zeros((2, 4))), i32([0] * 20), i32([0])
    pages.entmaxkv_pages_compact(p.shape, i32(p.table), i32(p.lens), t_out, p.buffers, r_out, n_live, workspace=p.ws)
    assert nv.get_status(clear=True) == nv.STATUS_BAD_PAGE
    assert int(n_live) == 3 and t_out.cpu()[0, 1] == -1 and t_out.cpu()[1, 0] == -1
    pages.entmaxkv_pages_refs(p.shape, i32(np.zeros((2, 4))), i32([65, 3]), refs, workspace=p.ws)
    assert nv.get_status(clear=True) == nv.STATUS_BAD_LENGTH
    assert refs[0] == 5


@gpu
def test_binding_refusals_on_the_gpu():
    p = Pool(2, 16, 4, 20, [40, 30])
    t, l = i32(p.table), i32(p.lens)
    with pytest.raises(ValueError, match="blocks"):
        pages.entmaxkv_pages_fork(p.shape, i32([0, 1]), t, l, t, l, pages.Buffers([p.data[0, :10].contiguous()]),
                                  workspace=p.ws)
    with pytest.raises(ValueError, match="metadata"):
        m = pages.Buffers([torch.zeros(64, dtype=torch.uint8, device="cuda")])
        pages.entmaxkv_pages_fork(p.shape, i32([0, 1]), t, l, t, l, p.buffers, m, m, workspace=p.ws)
    with pytest.raises(ValueError, match="parent"):
        pages.entmaxkv_pages_fork(p.shape, i32([0]), t, l, t, l, p.buffers, workspace=p.ws)
    with pytest.raises(TypeError, match="Buffers"):
        pages.entmaxkv_pages_fork(p.shape, i32([0, 1]), t, l, t, l, [p.data[0]], workspace=p.ws)
    with pytest.raises(ValueError, match="one shape"):
        pages.Buffers([p.data[0], p.data[1, :5]])
    with pytest.raises(TypeError, match="int32"):
        pages.entmaxkv_pages_grow(p.shape, i32([0, 1]).long(), t, l, workspace=p.ws)
    assert nv.get_status() == 0


@gpu
@pytest.mark.parametrize("alpha,captured", [(1.0, False), (1.5, False), (1.5, True)])
def test_beams_over_a_4bit_cache(alpha, captured):
    """Prompts, then steps of fork, grow, write and decode over two layers, a compaction in between; every step's
    attention against a plain cache that is copied row by row.  Captured: the step is one graph."""
    B, Hq, Hkv, d, P, mp, steps = 4, 4, 2, 64, 16, 6, 8
    nb = B * mp
    shape = nv.Shape(B, Hq, Hkv, d, P, mp, nb)
    g = torch.Generator().manual_seed(11)
    prompt = [20, 0, 37, 0]
    caches = [kv4.alloc_cache(shape, "cuda") for _ in range(2)]
    pool = pages.Buffers([x for c in caches for x in c], num_blocks=nb)
    metas = [[torch.zeros(nv.meta_bytes(shape), dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2)]
    meta_bufs = [pages.Buffers(m) for m in metas]
    ws, pws = kv4.alloc_workspace(shape, "cuda"), pages.alloc_workspace(shape, "cuda")
    tables = [i32(np.full((B, mp), -1)) for _ in range(2)]
    lens = [i32([0] * B) for _ in range(2)]
    pages.entmaxkv_pages_grow(shape, i32(prompt), tables[0], lens[0], workspace=pws)
    rows = torch.randn(2, 2, sum(prompt), Hkv, d, generator=g).bfloat16()
    start = i32([0, 20, 20, 57, 57])
    for layer in range(2):
        kv4.entmaxkv_kv4_write(shape, rows[layer, 0].cuda(), rows[layer, 1].cuda(), start, tables[0], lens[0],
                               *caches[layer], metas[0][layer])
    plain = [[rows[:, :, s:s + n] for s, n in zip((0, 20, 20, 57), prompt)]][0]   # [layer, k/v, token, ...] a row
    parent, add = i32([0] * B), i32([0] * B)
    new = torch.zeros(2, 2, B, Hkv, d, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, B, Hq, d, dtype=torch.bfloat16, device="cuda")
    out, tau = torch.zeros(2, B, Hq, d, device="cuda"), torch.zeros(2, B, Hq, device="cuda")

    def step(i):
        a, b = i % 2, (i + 1) % 2
        pages.entmaxkv_pages_fork(shape, parent, tables[a], lens[a], tables[b], lens[b], pool, meta_bufs[a],
                                  meta_bufs[b], workspace=pws)
        pages.entmaxkv_pages_grow(shape, add, tables[b], lens[b], workspace=pws)
        for layer in range(2):
            kv4.entmaxkv_kv4_write(shape, new[layer, 0], new[layer, 1], None, tables[b], lens[b], *caches[layer],
                                   metas[b][layer])
            kv4.entmaxkv_kv4_decode(shape, q[layer], *caches[layer], tables[b], lens[b], alpha, out[layer], tau[layer],
                                    workspace=ws)
    graphs = []
    if captured:
        for i in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[i]):
                step(i)
    nv.get_status(clear=True)
    rng = np.random.RandomState(3)
    for i in range(steps):
        alive = [b for b in range(B) if plain[b].shape[2] > 0]
        par = [int(rng.choice(alive)) for _ in range(B)] if i else [0, 0, 2, 2]
        if i == 4:
            par[1] = -1
        parent.copy_(i32(par))
        add.copy_(i32([int(p >= 0) for p in par]))
        fresh = torch.randn(2, 2, B, Hkv, d, generator=g).bfloat16()
        new.copy_(fresh)
        q.copy_(torch.randn(2, B, Hq, d, generator=g))
        graphs[i % 2].replay() if captured else step(i)
        empty = rows[:, :, :0]
        plain = [torch.cat([plain[p], fresh[:, :, b:b + 1]], 2) if p >= 0 else empty for b, p in enumerate(par)]
        assert nv.get_status(clear=True) == 0
        now = (i + 1) % 2
        assert lens[now].cpu().tolist() == [x.shape[2] for x in plain]
        for layer in range(2):
            for b in range(B):
                Kc, Vc = (ref.quantise(plain[b][layer, w].double().numpy()) for w in range(2))
                K, V = ref.values(*Kc), ref.values(*Vc)
                for h in range(Hq):
                    o, t, p = ref.attention(q[layer, b, h].cpu().double().numpy(), K[:, h // 2], V[:, h // 2], alpha)
                    got = out[layer, b, h].cpu().double().numpy()
                    if not len(p):
                        assert (got == 0).all()
                        continue
                    do, dt = ref.attention_bounds(q[layer, b, h].cpu().double().numpy(), Kc[1][:, h // 2],
                                                  V[:, h // 2], p, alpha)
                    assert np.abs(got - o).max() <= do and abs(float(tau[layer, b, h]) - t) <= dt
        if i == 5:  # pack the pool; the rows follow
            remap, n_live = i32([0] * nb), i32([0])
            pages.entmaxkv_pages_compact(shape, tables[now], lens[now], tables[now], pool, remap, n_live, workspace=pws)
            n = int(n_live)
            held = {int(x) for r, L in zip(tables[now].cpu(), lens[now].cpu()) for x in r[:-(-int(L) // P)]}
            assert held == set(range(n))
    # the metadata that came along is what a fresh build of the rows gives
    now = steps % 2
    for layer in range(2):
        again = torch.zeros_like(metas[now][layer])
        ln = lens[now].cpu().tolist()
        st = i32([0] + list(np.cumsum(ln)))
        k = torch.cat([x[layer, 0] for x in plain]).cuda()
        v = torch.cat([x[layer, 1] for x in plain]).cuda()
        k4, v4 = (torch.zeros_like(x) for x in caches[layer])
        own = i32(np.arange(B * mp).reshape(B, mp))
        kv4.entmaxkv_kv4_write(shape, k, v, st, own, lens[now], k4, v4, again)
        for x, y in zip(ref.meta_arrays(again.cpu().numpy(), B, Hkv, mp, d),
                        ref.meta_arrays(metas[now][layer].cpu().numpy(), B, Hkv, mp, d)):
            for b in range(B):
                np.testing.assert_array_equal(x[b, :, :-(-ln[b] // P)], y[b, :, :-(-ln[b] // P)])
