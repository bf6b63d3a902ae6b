"""The paged 4-bit cache on the GPU against the plain 64-bit model of page_util: rows in and out bit for bit, the
page operators' whole state and every byte of the pool, attention within bounds derived in page_util.tolerances."""
import numpy as np
import pytest
import torch

import page_util as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def up(x, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    return t if dt is None else t.to(dt)


class Both:
    """A reference pool and the same pool on the GPU."""

    def __init__(self, npages, D, page, L, B, Hkv, maxp, k_scale=1.0, v_scale=1.0, seed=0):
        from decoding_kv_cache_gb300 import kvc
        self.kvc = kvc
        rng = np.random.default_rng(seed)
        self.p = R.RefPool(npages, D, page, k_scale, v_scale, rng)
        self.t = R.RefPages(L, B, Hkv, maxp)
        self.pool = kvc.Pool.empty(npages, D, page, k_scale, v_scale, device=DEV)
        self.pool.data.copy_(up(self.p.data.reshape(npages, -1)))
        self.pages = kvc.Pages.empty(L, B, Hkv, maxp, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def check(self, what=""):
        torch.cuda.synchronize()
        eq = lambda a, b, n: np.testing.assert_array_equal(a.cpu().numpy(), b, err_msg=f"{what}: {n}")
        eq(self.pages.len, self.t.len, "len")
        eq(self.pages.table, self.t.table, "table")
        eq(self.pool.refs, self.p.refs, "refs")
        assert int(self.pool.nfree.item()) == self.p.nfree, f"{what}: nfree"
        eq(self.pool.free_list[:self.p.nfree], self.p.free[:self.p.nfree], "free_list")
        eq(self.pool.data, self.p.data.reshape(self.p.npages, -1), "data")
        assert int(self.status.item()) == self.p.status, f"{what}: status"

    def extend(self, add):
        a = up(np.asarray(add, np.int32))
        start = torch.full(self.t.shape, -9, dtype=torch.int32, device=DEV)
        self.kvc.kvc_page_extend(self.pool, self.pages, add=a, start=start, status=self.status)
        want = R.extend(self.p, self.t, add)
        np.testing.assert_array_equal(start.cpu().numpy(), want)
        return start

    def free(self, drop):
        self.kvc.kvc_page_free(self.pool, self.pages, drop=up(np.asarray(drop, np.int32)), status=self.status)
        R.free(self.p, self.t, drop)

    def fork(self, parent):
        L, _, Hkv = self.t.shape
        out = self.kvc.Pages(torch.full((L, len(parent), Hkv, self.t.maxp), 77, dtype=torch.int32, device=DEV),
                             torch.full((L, len(parent), Hkv), 77, dtype=torch.int32, device=DEV))
        self.kvc.kvc_page_fork(self.pool, self.pages, up(np.asarray(parent, np.int32)), out, status=self.status)
        self.t = R.fork(self.p, self.t, parent)
        self.pages = out

    def compact(self, lists, stride, per_seq=False):
        """lists {stream: list}; a bad one is given as (list, kept_len)"""
        shape = (self.t.shape[1],) if per_seq else self.t.shape
        idx = np.full(shape + (stride,), 1 << 29, np.int32)
        ln = np.zeros(shape, np.int32)
        ref = {}
        for s in self.t.streams():
            x = lists[s]
            bad = isinstance(x, tuple)
            at = s[1:2] if per_seq else s
            arr, n = (x if bad else (x, len(x)))
            idx[at][:len(arr)] = arr
            ln[at] = n
            ref[s] = None if bad else list(arr)
        self.kvc.kvc_page_compact(self.pool, self.pages, up(idx), up(ln), status=self.status)
        R.compact(self.p, self.t, ref)

    def store(self, k, v, start, n=None, dt="bf16"):
        """k, v: torch CPU tensors [B, T, Hkv, D]"""
        self.kvc.kvc_page_store(self.pool, self.pages, k, v, start, n=n, status=self.status)


def rand_rows(shape, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(torch.randn(shape[-1], generator=g))
    return x.to(DT[dt])


# ---- rows in and out ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt,D,page,T,scales", [
    ("bf16", 128, 64, 1, (1.0, 1.0)), ("bf16", 128, 16, 37, (0.5, 2.0)), ("bf16", 64, 32, 130, (1.0, 0.25)),
    ("f32", 128, 256, 300, (1.0, 1.0)), ("f32", 64, 16, 16, (0.125, 1.0)), ("bf16", 128, 128, 1000, (1.0, 1.0)),
    ("bf16", 128, 64, 8000, (1.0, 2.0)), ("f32", 64, 64, 13100, (1.0, 1.0)),
    ("bf16", 64, 64, 13100, (0.7, 1.0)),                                      # a tensor scale that is no power of two
])
def test_store_and_read_match_bit_for_bit(dt, D, page, T, scales):
    B, Hkv = 3, 2
    x = Both(3 * 2 * ((T + 50) // page + 2), D, page, 1, B, Hkv, (T + 50) // page + 1, *scales)
    x.extend([5, 0, 33])
    start = x.extend([T] * B)
    # the model's K and V: slices of one fused projection (strided), the ragged third sequence short by one
    kv = rand_rows((B, T, 2 * Hkv + 1, D), dt, T).to(DEV)
    k, v = kv[:, :, :Hkv], kv[:, :, Hkv:2 * Hkv]
    n = [T, max(T - 1, 0), T]
    x.store(k, v, start, n=up(np.array(n, np.int32)))
    R.store(x.p, x.t, k.double().cpu().numpy(), v.double().cpu().numpy(), start.cpu().numpy(), n)
    x.check("store")
    for count, first in ((T, None), (T + 60, 3)):
        ko = torch.full((1, B, Hkv, T + 61, D), -77.0, dtype=DT[dt], device=DEV)
        vo = ko.clone()
        x.kvc.kvc_page_read(x.pool, x.pages, ko, vo, first=start if first is None else None,
                            first_all=0 if first is None else first, count=count, status=x.status)
        only = torch.full_like(ko, -77.0)
        x.kvc.kvc_page_read(x.pool, x.pages, v=only, first=start if first is None else None,
                            first_all=0 if first is None else first, count=count)
        assert torch.equal(only, vo)
        for s in x.t.streams():
            f = int(start[s]) if first is None else first
            for j, o in enumerate((ko, vo)):
                want = torch.full((T + 61, D), -77.0, dtype=torch.float64)
                rows = R.rows(x.p, x.t, s, j)[f:f + count]
                # the code times its fp32 step in fp32, then the type's rounding (no rounding at all where the
                # tensor scale is a power of two: at most six bits)
                want[:len(rows)] = torch.from_numpy(rows).float().to(DT[dt]).double()
                assert torch.equal(o[s].double().cpu(), want), (s, j)
    x.check("read")


def test_store_special_values_and_refusals():
    D, page = 64, 16
    x = Both(20, D, page, 1, 2, 1, 4, 1.0, 1.0)
    start = x.extend([6, 6])
    k = torch.zeros((2, 6, 1, D))
    k[0, 0, 0, :8] = torch.tensor([6.0, -6.0, 0.25, 0.75, 1.25, -1.75, 2.5, 5.0])
    k[0, 1, 0, 3], k[0, 1, 0, 4], k[0, 1, 0, 20] = float("inf"), -float("inf"), 1e30
    k[0, 2, 0, 5], k[0, 2, 0, 6] = float("nan"), 2.0
    k[0, 3, 0, :] = float("nan")
    k[0, 4] = 1e-7
    k[0, 5, 0, :] = -0.0
    k[1] = torch.randn(6, 1, D, generator=torch.Generator().manual_seed(1)) * 2.0 ** -7
    v = -k.flip(3)
    x.store(k.to(DEV), v.to(DEV), start)
    R.store(x.p, x.t, k.double().numpy(), v.double().numpy(), start.cpu().numpy())
    x.check("special values")
    # skipped: start -1, rows past the length, a missing page, a shared page
    a = torch.ones((2, 1, 1, D), device=DEV)
    x.store(a, a, up(np.array([[[-1], [-1]]], np.int32)))
    x.check("no start")
    x.store(a, a, up(np.array([[[6], [-1]]], np.int32)))
    x.p.status |= R.BAD_INDEX
    x.check("past the length")
    x.fork([0, 0])
    x.status.zero_()
    x.p.status = 0
    x.store(a, a, up(np.array([[[0], [-1]]], np.int32)))
    x.p.status |= R.BAD_PAGE
    x.check("shared")
    x.pages.table[0, 1, 0, 0] = 1 << 30
    x.status.zero_()
    x.store(a, a, up(np.array([[[-1], [0]]], np.int32)))
    assert int(x.status.item()) == R.BAD_PAGE


@pytest.mark.parametrize("scales", [(1.0, 1.0), (2.0 ** -9, 2.0 ** 9), (2.0 ** 66, 2.0 ** -66), (0.7, 3.0)])
def test_store_every_bf16_value(scales):
    """All 65536 patterns, NaNs of either sign, infinities, zeros, subnormals and the largest among them, in groups of
    neighbours and in groups that mix magnitudes, with tensor scales of the short way and of the general one."""
    D, page, T = 64, 256, 1024
    x = Both(9, D, page, 1, 2, 1, 4, *scales)
    start = x.extend([T, T])
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    near = every.view(1, T, 1, D)
    far = every.view(D, T).T.reshape(1, T, 1, D)  # a row's patterns lie 1024 apart
    # rows with one value of all binades around each NaN, infinity and zero
    g = torch.Generator().manual_seed(8)
    rows = (torch.randn((1, T, 1, D), generator=g) * torch.exp2(torch.randint(-20, 20, (1, T, 1, 1), generator=g))).bfloat16()
    odd = torch.tensor([float("nan"), -float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 2.0 ** -133, -2.0 ** -126]).bfloat16()
    at = torch.randint(0, D, (T,), generator=g)
    rows[0, torch.arange(T), 0, at] = odd[torch.arange(T) % 8]
    k, v = torch.cat((near, rows)), torch.cat((far, rows.flip(3)))
    x.store(k.to(DEV), v.to(DEV), start)
    R.store(x.p, x.t, k.double().numpy(), v.double().numpy(), start.cpu().numpy())
    x.check("every value")


def test_store_rows_past_32_bits():
    """2^31 rows of K and V in one call (all of them the same row in memory, most without a page): the last ones
    land where they belong."""
    from decoding_kv_cache_gb300 import kvc
    D, page, T = 64, 256, 1 << 29
    maxp = T // page
    pool, pages = kvc.Pool.empty(8, D, page, device=DEV), kvc.Pages.empty(1, 1, 2, maxp, device=DEV)
    pages.len.fill_(T)
    pool.refs.fill_(1)
    pages.table[0, 0, 0, 0], pages.table[0, 0, 0, -1] = 3, 1
    pages.table[0, 0, 1, 5], pages.table[0, 0, 1, -1] = 6, 4
    k, v = rand_rows((1, 1, 2, D), "bf16", 5).to(DEV), rand_rows((1, 1, 2, D), "bf16", 6).to(DEV)
    start = torch.zeros((1, 1, 2), dtype=torch.int32, device=DEV)
    kvc.kvc_page_store(pool, pages, k.expand(1, T, 2, D), v.expand(1, T, 2, D), start)
    small = Both(2, D, page, 1, 1, 2, 1)
    s2 = small.extend([page])
    kvc.kvc_page_store(small.pool, small.pages, k.expand(1, page, 2, D), v.expand(1, page, 2, D), s2)
    for h, ids in ((0, (3, 1)), (1, (6, 4))):
        for p in ids:
            assert torch.equal(pool.data[p], small.pool.data[int(small.pages.table[0, 0, h, 0])])
    assert not pool.data[[0, 2, 5, 7]].any()


# ---- the page operators --------------------------------------------------------------------------
def random_lists(rng, t, shrink):
    lists = {}
    for s in t.streams():
        n = int(t.len[s])
        m = int(rng.integers(0, n + 1)) if shrink else n
        keep = np.sort(rng.choice(n, m, replace=False)) if n else np.zeros(0, np.int64)
        p = int(rng.integers(0, m + 1))  # a leading run that stays
        if rng.random() < 0.5:
            keep[:p] = np.arange(p)
            keep = np.unique(keep)
        lists[s] = keep
    return lists


@pytest.mark.parametrize("seed,D,page,L,B,Hkv,maxp,npages", [
    (0, 64, 16, 1, 2, 1, 8, 40), (1, 128, 64, 2, 3, 2, 5, 90), (2, 64, 32, 3, 5, 7, 6, 700),
    (3, 128, 16, 1, 9, 33, 4, 1500), (4, 64, 16, 2, 40, 4, 9, 2600), (5, 128, 256, 1, 4, 2, 2, 30),
    (6, 64, 16, 1, 1030, 1, 3, 2500),  # more sequences than the one-launch forms take
])
def test_random_sequences_of_page_operators(seed, D, page, L, B, Hkv, maxp, npages):
    """Extensions, forks, frees, evictions and stores in random order, the pool often nearly exhausted: tables,
    lengths, counts, the free list and every byte of the pool equal the model's after each."""
    rng = np.random.default_rng(seed)
    x = Both(npages, D, page, L, B, Hkv, maxp, seed=seed)
    x.check("init")
    for step in range(25):
        B = x.t.shape[1]
        op = rng.choice(["extend", "extend", "free", "fork", "compact", "compact"])
        what = f"step {step} {op}"
        if op == "extend":
            add = rng.integers(0, 2 * page, B) * (rng.random(B) < 0.7)
            if rng.random() < 0.2:
                add[rng.integers(0, B)] = rng.choice([-1, maxp * page + 1])
            x.extend([int(a) for a in add])
        elif op == "free":
            drop = rng.integers(0, 3 * page, B) * (rng.random(B) < 0.5)
            if rng.random() < 0.2:
                drop[rng.integers(0, B)] = rng.choice([-5, (1 << 31) - 1])
            x.free([int(d) for d in drop])
        elif op == "fork":
            parent = rng.integers(0, B, int(rng.integers(1, 2 * seed + 3)) if rng.random() < 0.4 else B)
            if rng.random() < 0.3:
                parent[0] = rng.choice([-1, B, -7])
            x.fork([int(p) for p in parent])
        else:
            lists = random_lists(rng, x.t, True)
            if rng.random() < 0.3:  # malformed lists: those streams stay
                for s in x.t.streams():
                    n = int(x.t.len[s])
                    if rng.random() < 0.2 and n >= 3:
                        lists[s] = [([0, 2, 1], 3), ([0, 0, 1], 3), ([0, 1, n], 3), ([0, 1], -1),
                                    (list(range(n)) + [n], n + 1), ([-1, 1, 2], 3)][int(rng.integers(0, 6))]
            x.compact(lists, maxp * page + 1)
        x.check(what)


@pytest.mark.parametrize("npages,L,B,Hkv,maxp,keep", [
    (20000, 2, 24, 8, 48, 700),    # several CTAs give pages back, each behind the marks of those before it
    (300000, 2, 4, 4, 500, 200),   # one launch whose CTAs take their words in two rounds
])
def test_pages_of_large_pools_given_back(npages, L, B, Hkv, maxp, keep):
    """Pages in use and given back lie all over the pool: counts, tables and the free list equal the model's."""
    from decoding_kv_cache_gb300 import kvc
    rng = np.random.default_rng(npages)
    x = Both.__new__(Both)
    x.kvc, x.p, x.t = kvc, R.RefPool(npages, 64, 16), R.RefPages(L, B, Hkv, maxp)
    x.p.data[:] = np.frombuffer(rng.bytes(x.p.data.size), np.uint8).reshape(x.p.data.shape)
    x.p.free = rng.permutation(npages).astype(np.int32)
    x.pool, x.pages = kvc.Pool.empty(npages, 64, 16, device=DEV), kvc.Pages.empty(L, B, Hkv, maxp, device=DEV)
    x.pool.data.copy_(up(x.p.data.reshape(npages, -1)))
    x.pool.free_list.copy_(up(x.p.free))
    x.status = torch.zeros(1, dtype=torch.int32, device=DEV)
    x.extend(rng.integers(1, 16 * maxp + 1, B).tolist())
    x.free(rng.integers(0, 8 * maxp, B).tolist())
    x.check("free")
    x.fork(rng.integers(0, B, B).tolist())
    x.check("fork")
    x.extend([int(min(a, 16 * maxp - n)) for a, n in zip(rng.integers(0, 50, B), x.t.len.max((0, 2)))])
    lists = {}
    for s in x.t.streams():
        n = int(x.t.len[s])
        lists[s] = np.sort(rng.choice(n, int(rng.integers(0, min(n, keep) + 1)), replace=False))
    x.compact(lists, keep)
    x.check("compact")
    x.free([1 << 30] * B)
    assert x.p.nfree == npages
    x.check("all given back")


def test_lists_per_sequence_and_exhausted_pool():
    x = Both(13, 128, 16, 1, 3, 2, 4, seed=3)
    x.extend([30, 30, 30])
    x.check("extend")  # 12 of 13 pages
    x.extend([10, 0, 0])  # two pages wanted, one free: nothing changes
    assert int(x.status.item()) == R.NO_PAGES
    x.check("exhausted")
    x.fork([0, 0, 1])
    x.status.zero_()
    x.p.status = 0
    lists = {s: [[0, 3, 4, 29], list(range(30)), [29]][s[1]] for s in x.t.streams()}
    x.compact(lists, 30, per_seq=True)
    x.check("per sequence")
    x.free([5, 5, 5])
    x.fork([2, 1, 1])
    x.extend([1, 12, 1])
    x.check("after")


def test_bad_pages_are_reported_not_followed():
    x = Both(10, 64, 16, 1, 2, 1, 4)
    x.extend([20, 20])
    for bad in (-1, 10, 1 << 30, -(1 << 31)):
        table = x.pages.table.clone()
        x.pages.table[0, 0, 0, 1] = bad
        before = x.pool.refs.clone()
        for op in ("extend", "compact", "free", "fork"):
            x.status.zero_()
            if op == "extend":
                x.kvc.kvc_page_extend(x.pool, x.pages, add=up(np.array([1, 0], np.int32)), status=x.status)
            elif op == "compact":
                ki = up(np.tile(np.arange(4, 24, dtype=np.int32), (1, 2, 1, 1)))
                kl = up(np.array([[[5], [0]]], np.int32)) * 0 + 5
                ki[..., :5] = torch.arange(3, 8, device=DEV)
                x.pages.len.copy_(up(np.array([[[20], [0]]], np.int32)))
                kl[0, 1] = 0
                x.kvc.kvc_page_compact(x.pool, x.pages, ki, kl, status=x.status)
                assert int(x.pages.len[0, 0, 0]) == 20
                assert torch.equal(x.pool.refs, before)
                x.pages.len.fill_(20)
            elif op == "free":
                x.kvc.kvc_page_free(x.pool, x.pages, drop=up(np.array([10, 0], np.int32)), status=x.status)
            else:
                out = x.kvc.Pages.empty(1, 2, 1, 4, device=DEV)
                x.pages.len.fill_(20)
                x.kvc.kvc_page_fork(x.pool, x.pages, up(np.array([0, 0], np.int32)), out, status=x.status)
            assert int(x.status.item()) & R.BAD_PAGE, (bad, op)
        x.pages.table.copy_(table)
        x.pages.len.fill_(20)
        x.pool.refs.copy_(before)
        x.pool.nfree.fill_(x.p.nfree)
        x.pool.free_list.copy_(up(x.p.free))


@pytest.mark.parametrize("Hkv,maxp", [(1, 4), (40, 300)])  # one launch each, and the wide forms
def test_what_free_and_fork_make_of_a_bad_page(Hkv, maxp):
    x = Both(1000, 64, 16, 1, 2, Hkv, maxp)
    x.extend([60, 20])
    good = int(x.t.table[0, 0, 0, 2])
    x.pages.table[0, 0, 0, 2] = 1000
    x.fork([0, 0])  # sequence 1's pages go, sequence 0's are shared but for the bad one, which both children hold
    assert int(x.status.item()) == R.BAD_PAGE
    assert x.pages.table[0, :, 0, 2].tolist() == [1000, 1000] and int(x.pool.refs[good]) == 1
    x.status.zero_()
    x.kvc.kvc_page_free(x.pool, x.pages, drop=up(np.array([40, 0], np.int32)), status=x.status)
    assert int(x.status.item()) == R.BAD_PAGE
    assert x.pages.len[0, :, 0].tolist() == [20, 60] and x.pages.table[0, 0, 0, :5].tolist()[2:4] == [-1, -1]
    assert (x.pages.table[0, 0, :, 2:4] == -1).all() and int(x.pages.table[0, 1, 0, 2]) == 1000
    assert int(x.pool.nfree) == 1000 - 4 * Hkv  # the four pages of each of sequence 0's streams, the bad entry's lost one too


@pytest.mark.parametrize("bad", [-1, 400, 1 << 30])
@pytest.mark.parametrize("Hkv,at", [(1, 0), (1, 1), (40, 0), (40, 1)])  # one finishing launch, and two
def test_compaction_with_a_damaged_free_list(Hkv, at, bad):
    """A free list that holds no page's number where a shared page has to be replaced: that stream stays as it
    was, shared pages are not written, the others take theirs."""
    x = Both(400, 64, 16, 1, 2, Hkv, 4, seed=at)
    x.extend([40, 0])
    x.fork([0, 0])
    x.check("fork")
    top = x.p.nfree - 1
    x.pool.free_list[top - at] = bad
    lists = {s: list(range(1, 40, 2)) for s in x.t.streams()}
    lists[(0, 0, 0)] = None  # two shared pages of each stream are replaced: the first stream's two are off the list
    idx = up(np.tile(np.arange(1, 40, 2, dtype=np.int32), (1, 2, Hkv, 1)))
    x.kvc.kvc_page_compact(x.pool, x.pages, idx, up(np.full((1, 2, Hkv), 20, np.int32)), status=x.status)
    x.p.nfree -= 2
    R.compact(x.p, x.t, lists)
    x.p.status = R.BAD_PAGE
    x.check("compaction")


@pytest.mark.parametrize("bad", [-1, 13000, 1 << 30])
@pytest.mark.parametrize("Hkv", [1, 140])  # the one-launch form, and the wide one
@pytest.mark.parametrize("at,copies", [(0, False), (39, False), (0, True), (33, True)])
def test_extension_with_a_damaged_free_list(Hkv, at, copies, bad):
    """A number out of range where a stream would take its page (the copy of a shared one, a fresh one): it
    stays as it was, the others take theirs."""
    x = Both(13000, 64, 16, 1, 2, Hkv, 42, seed=at)
    if copies:
        x.extend([20, 0])
        x.fork([0, 0])
    add = [630, 0 if copies else 630]  # 40 pages a stream; the first sequence's last page is copied where it is shared
    x.pool.free_list[x.p.nfree - 1 - at] = bad
    start = torch.full(x.t.shape, -9, dtype=torch.int32, device=DEV)
    x.kvc.kvc_page_extend(x.pool, x.pages, add=up(np.array(add, np.int32)), start=start, status=x.status)
    # the model: the first stream's pages are off the list, its own state is as before
    n0, row0, data0, s0 = int(x.t.len[0, 0, 0]), x.t.table[0, 0, 0].copy(), x.p.data.copy(), (0, 0, 0)
    want = R.extend(x.p, x.t, add)
    taken = np.setdiff1d(x.t.table[s0], row0)
    assert x.p.status == 0 and len(taken) == 40
    if copies:
        x.p.refs[row0[1]] += 1
    x.p.refs[taken], x.p.data[taken] = 0, data0[taken]
    x.t.len[s0], x.t.table[s0], want[s0] = n0, row0, -1
    x.p.status = R.BAD_PAGE
    np.testing.assert_array_equal(start.cpu().numpy(), want)
    x.check("extension")


@pytest.mark.parametrize("at,lost", [(31, 0), (32, 0), (128, 0), (299, 0), (300, 1), (430, 1)])
def test_long_extension_with_a_damaged_free_list(at, lost):
    """300 pages a stream: which of its reads of the free list meets the bad number makes no difference."""
    x = Both(700, 64, 16, 1, 2, 1, 300)
    x.pool.free_list[x.p.nfree - 1 - at] = 700
    start = torch.full(x.t.shape, -9, dtype=torch.int32, device=DEV)
    x.kvc.kvc_page_extend(x.pool, x.pages, add_all=4800, start=start, status=x.status)
    want = R.extend(x.p, x.t, [4800, 4800])
    x.p.refs[x.t.table[0, lost, 0]] = 0
    x.t.len[0, lost, 0], x.t.table[0, lost, 0], want[0, lost, 0] = 0, -1, -1
    x.p.status = R.BAD_PAGE
    np.testing.assert_array_equal(start.cpu().numpy(), want)
    x.check("extension")


# ---- attention -----------------------------------------------------------------------------------
def make_attend(dt, D, B, Hkv, G, T, page, lens, seed=0, k_scale=1.0, v_scale=1.0):
    lens = np.asarray(lens, np.int32).reshape(1, B, Hkv)
    maxp = max(1, R.npg(int(lens.max()), page))
    used = [R.npg(int(n), page) for n in lens.reshape(-1)]
    x = Both(sum(used) + 5, D, page, 1, B, Hkv, maxp, k_scale, v_scale, seed)
    rng = np.random.default_rng(seed + 1)
    order = rng.permutation(x.p.npages)
    at = 0
    for s, u in zip(x.t.streams(), used):
        x.t.table[s][:u] = order[at:at + u]
        at += u
        n = int(lens[s])
        x.t.len[s] = n
        if not n:
            continue
        rows = rng.standard_normal((2, n, D)) * np.exp(0.5 * rng.standard_normal((2, 1, D)))
        for j in range(2):
            c, sb = R.quantise(rows[j], x.p.ts[j])
            for i in range(n):
                p = x.t.table[s][i // page]
                x.p.piece(p, i, 2 * j)[:] = c[i]
                x.p.piece(p, i, 2 * j + 1)[:] = sb[i]
        for i in range(n, u * page):  # behind the length: NaN scales
            for j in range(2):
                x.p.piece(x.t.table[s][i // page], i, 2 * j + 1)[:] = 0x7f
    x.pool.data.copy_(up(x.p.data.reshape(x.p.npages, -1)))
    x.pages.table.copy_(up(x.t.table))
    x.pages.len.copy_(up(x.t.len))
    g = torch.Generator().manual_seed(seed + 2)
    q = torch.randn((B, T, Hkv * G, D), generator=g).to(DT[dt])
    return x, q


def check_attend(x, q, dt, scale=None, n_q=None, run=None):
    B, T, Hq, D = q.shape
    sc = D ** -0.5 if scale is None else scale
    out = torch.full((B, T, Hq, D), -55.0, dtype=DT[dt], device=DEV)
    lse = torch.full((B, T, Hq), -55.0, device=DEV)
    nq = None if n_q is None else up(np.asarray(n_q, np.int32))
    if run:
        run(out, lse)
    else:
        x.kvc.kvc_page_attend(x.pool, x.pages, q.to(DEV), out, lse=lse, n_q=nq, scale=scale, status=x.status)
    torch.cuda.synchronize()
    ref = R.attend(x.p, x.t, q.double().cpu().numpy(), sc, n_q)
    o, l = ref["out"], ref["lse"]
    tol, ltol = R.tolerances(dt, int(x.t.len.max()), D, ref)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        k = T if n_q is None else min(max(int(n_q[b]), 0), T)
        assert (got[b, k:] == -55.0).all() and (gl[b, k:] == -55.0).all(), "rows behind the last query"
        err = np.abs(got[b, :k] - o[b, :k])
        assert (err <= tol[b, :k]).all(), (b, float((err / tol[b, :k]).max()))
        empty = np.isneginf(l[b, :k])
        assert (np.isneginf(gl[b, :k]) == empty).all() and (got[b, :k][empty] == 0).all()
        le = np.abs(gl[b, :k][~empty] - l[b, :k][~empty])
        assert (le <= ltol[b, :k][~empty]).all(), float((le / ltol[b, :k][~empty]).max())
    assert int(x.status.item()) == 0
    return out, lse


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("B,Hkv,G,T,page,lens", [
    (1, 1, 1, 1, 16, [1]),
    (2, 2, 1, 1, 16, [0, 1, 15, 16]),
    (3, 2, 4, 1, 64, [17, 63, 64, 65, 0, 200]),
    (2, 1, 8, 1, 256, [255, 300]),
    (1, 3, 7, 1, 32, [31, 500, 2]),
    (2, 2, 5, 3, 64, [2, 0, 130, 3]),       # fewer tokens than queries: the first see none
    (1, 2, 3, 17, 16, [17, 160]),
    (2, 1, 4, 40, 128, [100, 333]),
    (1, 1, 16, 5, 64, [77]),
    (1, 2, 1, 130, 64, [140, 100]),
])
def test_attend(dt, D, B, Hkv, G, T, page, lens):
    x, q = make_attend(dt, D, B, Hkv, G, T, page, lens, seed=B * 7 + T)
    check_attend(x, q, dt)


@pytest.mark.parametrize("dt,D,B,Hkv,G,T,n", [("bf16", 128, 1, 1, 4, 1, 6000), ("f32", 64, 2, 2, 2, 1, 3001),
                                              ("bf16", 64, 1, 2, 8, 20, 2500), ("f32", 128, 1, 1, 3, 2, 4097),
                                              # several units a CTA, streams cut between CTAs, two row blocks
                                              ("bf16", 128, 4, 8, 4, 16, 3000), ("bf16", 64, 4, 8, 5, 40, 2200)])
def test_attend_long(dt, D, B, Hkv, G, T, n):
    rng = np.random.default_rng(n)
    x, q = make_attend(dt, D, B, Hkv, G, T, 64, rng.integers(n // 8, n + 1, B * Hkv), seed=n)
    check_attend(x, q, dt)


@pytest.mark.parametrize("dt,D,G,T,n", [("bf16", 128, 4, 33, 120000), ("bf16", 64, 8, 20, 150000), ("bf16", 128, 5, 1, 60000),
                                         ("f32", 64, 2, 3, 40000)])
def test_attend_many_units_a_cta(dt, D, G, T, n):
    """Long streams: dozens of work units for every CTA, the model's product formed on the GPU in 64 bits."""
    from decoding_kv_cache_gb300 import kvc
    B, Hkv, page = 2, 1, 256
    maxp = R.npg(n, page)
    pool, pages = kvc.Pool.empty(2 * maxp + 3, D, page, device=DEV), kvc.Pages.empty(1, B, Hkv, maxp, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    start = torch.zeros((1, B, Hkv), dtype=torch.int32, device=DEV)
    lens = torch.tensor([n, n - 777], dtype=torch.int32, device=DEV)
    kvc.kvc_page_extend(pool, pages, add=lens, start=start, status=status)
    g = torch.Generator(device=DEV).manual_seed(n)
    k, v = (torch.randn((B, n, Hkv, D), generator=g, device=DEV).to(DT[dt]) for _ in range(2))
    kvc.kvc_page_store(pool, pages, k, v, start, n=lens, status=status)
    q = (2 * torch.randn((B, T, Hkv * G, D), generator=g, device=DEV)).to(DT[dt])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kvc.kvc_page_attend(pool, pages, q, out, lse=lse, status=status)
    K = torch.zeros((1, B, Hkv, n, D), device=DEV)
    V = torch.zeros_like(K)
    kvc.kvc_page_read(pool, pages, K, V, status=status)
    assert int(status.item()) == 0
    for b in range(B):
        m = int(lens[b])
        kk, vv = K[0, b, 0, :m].double(), V[0, b, 0, :m].double()
        for i in (0, T // 2, T - 1):
            seen = m - T + i + 1
            qq = q[b, i].double()
            s = qq @ kk[:seen].T / D ** 0.5
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[:, None])
            ref = dict(out=p @ vv[:seen], lse=z, mass=p @ vv[:seen].abs(), vmax=vv[:seen].abs().amax(0) + 0 * qq,
                       logit=(qq.abs() @ kk[:seen].abs().T / D ** 0.5).amax(-1))
            ref = {name: x.cpu().numpy() for name, x in ref.items()}
            tol, ltol = R.tolerances(dt, seen, D, ref)
            assert (np.abs(out[b, i].double().cpu().numpy() - ref["out"]) <= tol).all()
            assert (np.abs(lse[b, i].double().cpu().numpy() - ref["lse"]) <= ltol).all()


@pytest.mark.parametrize("dt,D,G,T", [("bf16", 128, 4, 1), ("bf16", 64, 2, 10), ("f32", 64, 4, 3), ("bf16", 128, 4, 40)])
@pytest.mark.parametrize("seed", [0, 1])
def test_attend_many_short_streams(dt, D, G, T, seed):
    """Streams of no, one and few units between long ones: shares that hold only a stream's beginning."""
    rng = np.random.default_rng(seed)
    B, Hkv = 12, 5
    lens = rng.choice([0, 1, 2, 63, 64, 65, 127, 128, 129, 200, 600], B * Hkv).tolist()
    lens[int(rng.integers(B * Hkv))] = 1500
    x, q = make_attend(dt, D, B, Hkv, G, T, 64, lens, seed=seed)
    check_attend(x, q, dt)


@pytest.mark.parametrize("dt,T", [("bf16", 6), ("bf16", 30), ("f32", 6)])
def test_attend_strided_ragged_scaled(dt, T):
    x, q0 = make_attend(dt, 128, 4, 2, 3, T, 32, [90, 80, 3, 4, 50, 60, 0, 0], seed=5, k_scale=0.3, v_scale=7.0)
    fused = torch.zeros((4, T, 11, 128), dtype=DT[dt], device=DEV)  # the query part of a fused projection's row
    fused[:, :, 2:8] = q0.to(DEV)
    q = fused[:, :, 2:8]
    for n_q in ([6, 4, 0, 6], [1, T, 99, -3]):
        run = lambda out, lse: x.kvc.kvc_page_attend(x.pool, x.pages, q, out, lse=lse, scale=0.37, status=x.status,
                                                     n_q=up(np.array(n_q, np.int32)))
        check_attend(x, q0, dt, scale=0.37, n_q=n_q, run=run)
    qt = q0.to(DEV).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)  # [B, Hq, T, D] in memory
    run = lambda out, lse: x.kvc.kvc_page_attend(x.pool, x.pages, qt, out, lse=lse, status=x.status)
    check_attend(x, q0, dt, run=run)


@pytest.mark.parametrize("dt,D,G,T,page,lens", [
    ("bf16", 128, 4, 4, 64, [700, 3, 0, 1, 2000, 64]),   # split streams
    ("f32", 64, 3, 5, 16, [900, 4, 5, 0, 33, 16]),
    ("bf16", 64, 2, 8, 32, [200, 7, 0, 8, 9, 100]),      # whole streams
    ("bf16", 128, 4, 300, 64, [700, 299, 300, 1, 0, 301]),  # ten row blocks
])
def test_attend_fewer_queries_than_rows(dt, D, G, T, page, lens):
    """n_q on each kernel: sequences with none, one, some and all of their queries, some of them before any token."""
    x, q = make_attend(dt, D, 3, 2, G, T, page, lens, seed=T)
    for n_q in ([0, 1, T], [T - 1, 2, 0], [T + 5, -1, T // 2]):
        run = lambda out, lse: x.kvc.kvc_page_attend(x.pool, x.pages, q.to(DEV), out, lse=lse, status=x.status,
                                                     n_q=up(np.array(n_q, np.int32)))
        check_attend(x, q, dt, n_q=n_q, run=run)


@pytest.mark.parametrize("dt,T", [("bf16", 2), ("bf16", 20), ("f32", 2)])
def test_attend_extreme_logits(dt, T):
    """Large and negative scales, one dominant key, zero queries: the running maximum has to follow."""
    x, q = make_attend(dt, 64, 2, 2, 2, T, 16, [300, 40, 16, 129], seed=11)
    for scale in (0.0, -0.5, 4.0, 30.0, 1e-6):
        check_attend(x, q, dt, scale=scale)
    q[0] = 0
    q[1] *= 1000.0
    check_attend(x, q, dt, scale=0.125)
    q[1] *= 2.0 ** -40
    check_attend(x, q, dt, scale=0.125)


@pytest.mark.parametrize("T,cap", [(1, 4), (1, 40), (20, 4)])
def test_attend_bad_pages_take_no_part(T, cap):
    """On each of the kernels (short tables, long tables, many rows)."""
    x, q = make_attend("bf16", 128, 2, 1, 2, T, 16, [64, 40], seed=2)
    table = torch.full((1, 2, 1, cap), -1, dtype=torch.int32, device=DEV)
    table[..., :4] = x.pages.table
    table[0, 0, 0, 1] = 12345678
    table[0, 1, 0, 1] = -1
    pages = x.kvc.Pages(table, x.pages.len)
    out, lse = torch.zeros((2, T, 2, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((2, T, 2), device=DEV)
    x.kvc.kvc_page_attend(x.pool, pages, q.to(DEV), out, lse=lse, status=x.status)
    assert int(x.status.item()) == R.BAD_PAGE
    for b, n in ((0, 64), (1, 40)):
        K, V = R.rows(x.p, x.t, (0, b, 0), 0), R.rows(x.p, x.t, (0, b, 0), 1)
        for i in range(T):
            seen = np.setdiff1d(np.arange(n - T + i + 1), np.arange(16, 32))
            ref = R.attend_rows(q[b, i].double().numpy(), K[seen], V[seen], 128 ** -0.5)
            tol, ltol = R.tolerances("bf16", 64, 128, ref)
            assert (np.abs(out[b, i].double().cpu().numpy() - ref["out"]) <= tol).all()
            assert (np.abs(lse[b, i].double().cpu().numpy() - ref["lse"]) <= ltol).all()
    x.pages.len[0, 1, 0] = 1 << 20  # a length beyond the table: an empty stream
    x.status.zero_()
    x.kvc.kvc_page_attend(x.pool, pages, q.to(DEV), out, lse=lse, status=x.status)
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all() and int(x.status.item()) == R.BAD_PAGE


def test_offsets_past_32_bits():
    """A pool of 5 GB whose streams lie in its last pages: store, read, attention and compaction there."""
    from decoding_kv_cache_gb300 import kvc
    D, page = 128, 256
    npages = (5 << 30) // kvc.kvc_page_bytes(D, page)
    pool = kvc.Pool.empty(npages, D, page, device=DEV)
    pool.free_list.copy_(torch.arange(npages, dtype=torch.int32, device=DEV))  # the last pages first
    pages = kvc.Pages.empty(1, 1, 2, 4, device=DEV)
    start = torch.zeros((1, 1, 2), dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    n = 700
    kvc.kvc_page_extend(pool, pages, add_all=n, start=start, status=status)
    assert int(pages.table[0, 0, 0, 0]) == npages - 1
    k, v = rand_rows((1, n, 2, D), "bf16", 1).to(DEV), rand_rows((1, n, 2, D), "bf16", 2).to(DEV)
    kvc.kvc_page_store(pool, pages, k, v, start, status=status)
    small = Both(10, D, page, 1, 1, 2, 4)
    s2 = small.extend([n])
    small.store(k, v, s2)
    idx = torch.arange(0, n, 2, dtype=torch.int32, device=DEV).expand(1, 1, 2, -1).contiguous()
    kl = torch.full((1, 1, 2), n // 2, dtype=torch.int32, device=DEV)
    q = rand_rows((1, 1, 8, D), "bf16", 3).to(DEV)
    outs = []
    for p, t in ((pool, pages), (small.pool, small.pages)):
        kvc.kvc_page_compact(p, t, idx, kl, status=status)
        out, ko = torch.empty_like(q), torch.empty((1, 1, 2, n // 2, D), dtype=torch.bfloat16, device=DEV)
        kvc.kvc_page_attend(p, t, q, out, status=status)
        kvc.kvc_page_read(p, t, ko, status=status)
        outs.append((out, ko))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert int(status.item()) == 0


# ---- a run of them together ------------------------------------------------------------------------
def test_decode_with_evictions_forks_and_rollback():
    """Prompt, decode steps with attention, an eviction ranked by kvc_score on the read-back keys (per-head
    budgets), a fork, drafts and their rollback: the cache and every attention follow the model."""
    from decoding_kv_cache_gb300 import kvc
    L, B, Hkv, G, D, page, T0 = 2, 2, 2, 2, 64, 16, 61
    Hq = Hkv * G
    x = Both(200, D, page, L, B, Hkv, 8, seed=9)
    seed = [100]

    def rows(T, heads, B=B):
        seed[0] += 1
        return rand_rows((B, T, heads, D), "bf16", seed[0])

    def add(T):
        start = x.extend([T] * x.t.shape[1])
        for l in range(L):
            k, v = rows(T, Hkv, x.t.shape[1]), rows(T, Hkv, x.t.shape[1])
            lay, one = x.pages.layer(l), R.RefPages(1, x.t.shape[1], Hkv, x.t.maxp)
            one.table, one.len = x.t.table[l:l + 1], x.t.len[l:l + 1]
            kvc.kvc_page_store(x.pool, lay, k.to(DEV), v.to(DEV), start[l:l + 1], status=x.status)
            R.store(x.p, one, k.double().numpy(), v.double().numpy(), start[l:l + 1].cpu().numpy())
            q = rows(T, Hq, x.t.shape[1])
            run = lambda out, lse: kvc.kvc_page_attend(x.pool, lay, q.to(DEV), out, lse=lse, status=x.status)
            both = Both.__new__(Both)
            both.__dict__.update(x.__dict__)
            both.t = one
            check_attend(both, q, "bf16", run=run)

    add(T0)
    for _ in range(3):
        add(1)
    N = T0 + 3
    K = torch.zeros((L, B, Hkv, N, D), dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    kvc.kvc_page_read(x.pool, x.pages, K, V, status=x.status)
    for s in x.t.streams():
        assert torch.equal(K[s].double().cpu(), torch.from_numpy(R.rows(x.p, x.t, s, 0)))
    cache = kvc.Cache(K, V, Hq)
    g = torch.Generator().manual_seed(4)
    qr = torch.randn((L, B, Hq, 16, D), generator=g).to(torch.bfloat16).to(DEV)
    qb = torch.randn((L, B, Hq, 32, D), generator=g).to(torch.bfloat16).to(DEV)
    cnt = torch.full((L, B, Hq), 20, dtype=torch.int32, device=DEV)
    scores = torch.empty((L, B, Hkv, N), device=DEV)
    kvc.kvc_score(cache, qr, qb, cnt, 16, N - 1, 1e4, scores)
    kept = torch.empty((L, B, Hkv, N), dtype=torch.int32, device=DEV)
    klen = torch.empty((L, B, Hkv), dtype=torch.int32, device=DEV)
    budget = torch.tensor([[[40, 25], [33, 64]], [[20, 48], [22, 39]]], dtype=torch.int32, device=DEV)
    kvc.kvc_select(scores, 4, 8, kept, klen, budget=budget, status=x.status)
    kvc.kvc_page_compact(x.pool, x.pages, kept, klen, status=x.status)
    R.compact(x.p, x.t, {s: kept[s][:int(klen[s])].cpu().tolist() for s in x.t.streams()})
    x.check("eviction")
    assert (x.t.len == budget.cpu().numpy()).all()
    # the dense cache's compaction keeps the same rows
    kvc.kvc_compact(cache, kept, klen, status=x.status)
    K2 = torch.zeros_like(K)
    kvc.kvc_page_read(x.pool, x.pages, K2)
    for s in x.t.streams():
        assert torch.equal(K2[s][:int(klen[s])], K[s][:int(klen[s])])
    add(2)
    x.fork([1, 1, 0])
    x.check("fork")
    add(4)
    x.free([3, 0, 4])
    x.check("rollback")
    add(1)
    x.compact({s: list(range(1, int(x.t.len[s]), 3)) for s in x.t.streams()}, 128)
    x.check("second eviction")
    add(1)
    x.check("end")


def test_captured_and_replayed_with_new_lengths():
    """A decode step (room, rows, attention) captured once and replayed while the lengths grow: each replay equals
    an eager run of the model's state."""
    from decoding_kv_cache_gb300 import kvc
    x, q = make_attend("bf16", 128, 2, 2, 4, 1, 16, [30, 16, 5, 100], seed=21)
    # room in the table for growth
    pool = kvc.Pool.empty(64, 128, 16, device=DEV)
    pages = kvc.Pages.empty(1, 2, 2, 12, device=DEV)
    start = torch.zeros((1, 2, 2), dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(kvc.kvc_page_workspace_size(pool, pages), dtype=torch.uint8, device=DEV)
    aws = torch.empty(kvc.kvc_page_attend_workspace_size(pool, pages, 8, 1), dtype=torch.uint8, device=DEV)
    kvc.kvc_page_extend(pool, pages, add=up(np.array([33, 15], np.int32)), start=start)
    k0 = rand_rows((2, 33, 2, 128), "bf16", 1).to(DEV)
    kvc.kvc_page_store(pool, pages, k0, k0, start, n=up(np.array([33, 15], np.int32)))
    k, v = rand_rows((2, 1, 2, 128), "bf16", 2).to(DEV), rand_rows((2, 1, 2, 128), "bf16", 3).to(DEV)
    qd, out, lse = q.to(DEV), torch.zeros((2, 1, 8, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 1, 8), device=DEV)

    def step(stream=None):
        kvc.kvc_page_extend(pool, pages, add_all=1, start=start, status=status, workspace=ws)
        kvc.kvc_page_store(pool, pages, k, v, start, status=status)
        kvc.kvc_page_attend(pool, pages, qd, out, lse=lse, status=status, workspace=aws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(20):
        k.copy_(rand_rows((2, 1, 2, 128), "bf16", 100 + i))
        qd.copy_(rand_rows((2, 1, 8, 128), "bf16", 200 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert int(pages.len[0, 0, 0]) == 33 + 2 + i and int(status.item()) == 0
        o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
        kvc.kvc_page_attend(pool, pages, qd, o2, lse=l2, status=status)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        K = torch.zeros((1, 2, 2, 80, 128), device=DEV)
        V = torch.zeros_like(K)
        kvc.kvc_page_read(pool, pages, K, V)
        n = int(pages.len[0, 1, 1])
        ref = R.attend_rows(qd[1, 0, 4:].double().cpu().numpy(), K[0, 1, 1, :n].double().cpu().numpy(),
                            V[0, 1, 1, :n].double().cpu().numpy(), 128 ** -0.5)
        tol, ltol = R.tolerances("bf16", n, 128, ref)
        assert (np.abs(out[1, 0, 4:].double().cpu().numpy() - ref["out"]) <= tol).all()
        assert (np.abs(lse[1, 0, 4:].double().cpu().numpy() - ref["lse"]) <= ltol).all()


@pytest.mark.parametrize("L,B,Hkv,maxp,npages", [(1, 3, 2, 8, 120), (2, 24, 8, 48, 9000)])  # one launch each, and the wide forms
def test_page_operators_captured_and_replayed(L, B, Hkv, maxp, npages):
    """Room, eviction, fork and rollback captured once; each replay with new numbers equals the model's, eager calls
    between the replays use the same workspace."""
    from decoding_kv_cache_gb300 import kvc
    rng = np.random.default_rng(B)
    x = Both(npages, 64, 16, L, B, Hkv, maxp, seed=B)
    S, other = x.t.shape, kvc.Pages.empty(L, B, Hkv, maxp, device=DEV)
    ws = torch.empty(kvc.kvc_page_workspace_size(x.pool, x.pages), dtype=torch.uint8, device=DEV)
    add, drop, parent = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
    kept, klen = torch.zeros(S + (64,), dtype=torch.int32, device=DEV), torch.zeros(S, dtype=torch.int32, device=DEV)
    a, b = x.pages, other

    def step():
        kvc.kvc_page_extend(x.pool, a, add=add, status=x.status, workspace=ws)
        kvc.kvc_page_compact(x.pool, a, kept, klen, status=x.status, workspace=ws)
        kvc.kvc_page_fork(x.pool, a, parent, b, status=x.status, workspace=ws)
        kvc.kvc_page_free(x.pool, b, drop=drop, status=x.status, workspace=ws)
        kvc.kvc_page_fork(x.pool, b, parent, a, status=x.status, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # nothing to do yet: no tokens, empty lists
    torch.cuda.current_stream().wait_stream(side)
    R.fork(x.p, x.t, [0] * B)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.check("captured")
    for i in range(6):
        ad, dr = rng.integers(0, 40, B), rng.integers(0, 30, B)
        pa = rng.integers(0, B, B)
        lists, idx, ln = {}, np.zeros(S + (64,), np.int32), np.zeros(S, np.int32)
        for s in x.t.streams():
            n = int(x.t.len[s]) + int(ad[s[1]])
            m = int(rng.integers(min(n, 20), min(n, 50) + 1))
            lists[s] = np.sort(rng.choice(n, m, replace=False))
            idx[s][:m], ln[s] = lists[s], m
        for t, v in ((add, ad), (drop, dr), (parent, pa), (kept, idx), (klen, ln)):
            t.copy_(up(np.ascontiguousarray(v, np.int32)))
        graph.replay()
        R.extend(x.p, x.t, ad.tolist())
        R.compact(x.p, x.t, lists)
        x.t = R.fork(x.p, x.t, pa.tolist())
        R.free(x.p, x.t, dr.tolist())
        x.t = R.fork(x.p, x.t, pa.tolist())
        x.check(f"replay {i}")
        kvc.kvc_page_free(x.pool, a, drop_all=1, status=x.status, workspace=ws)
        R.free(x.p, x.t, [1] * B)
        x.check(f"between {i}")


def test_streams_with_their_own_workspaces():
    from decoding_kv_cache_gb300 import kvc
    a, qa = make_attend("bf16", 128, 4, 4, 4, 1, 64, [900] * 16, seed=31)
    b, qb = make_attend("bf16", 128, 2, 2, 8, 3, 16, [333, 500, 7, 64], seed=32)
    c, qc = make_attend("bf16", 128, 2, 2, 2, 40, 64, [900, 1200, 70, 400], seed=33)
    ref = [torch.empty_like(q, device=DEV) for q in (qa, qb, qc)]
    got = [torch.empty_like(q, device=DEV) for q in (qa, qb, qc)]
    qs = [qa.to(DEV), qb.to(DEV), qc.to(DEV)]
    for x, q, o in zip((a, b, c), qs, ref):
        kvc.kvc_page_attend(x.pool, x.pages, q, o)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in qs]
    ws = [torch.empty(kvc.kvc_page_attend_workspace_size(x.pool, x.pages, q.shape[2], q.shape[1]), dtype=torch.uint8,
                      device=DEV) for x, q in zip((a, b, c), qs)]
    for _ in range(20):
        for x, q, o, s, w in zip((a, b, c), qs, got, st, ws):
            kvc.kvc_page_attend(x.pool, x.pages, q, o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(r, o) for r, o in zip(ref, got))


@pytest.mark.parametrize("handle", [False, True])
def test_a_calls_own_workspace_outlives_it_on_another_stream(handle):
    from decoding_kv_cache_gb300 import kvc
    x, q = make_attend("bf16", 128, 2, 2, 4, 1, 64, [900, 30, 700, 0], seed=34)
    qd = q.to(DEV)
    ref, got = torch.empty_like(qd), torch.empty_like(qd)
    kvc.kvc_page_attend(x.pool, x.pages, qd, ref)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)  # some 25 ms
    stream = s.cuda_stream if handle else s
    n = 3 << 20
    p, size, ws = kvc._page_ws(lambda: n, x.pool, None, stream)
    assert size == n
    del ws
    assert torch.empty(n, dtype=torch.uint8, device=DEV).data_ptr() != p
    kvc.kvc_page_attend(x.pool, x.pages, qd, got, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(ref, got)


def test_binding_refuses_wrong_tensors():
    from decoding_kv_cache_gb300 import kvc
    pool, pages = kvc.Pool.empty(8, 64, 16, device=DEV), kvc.Pages.empty(2, 2, 2, 4, device=DEV)
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(kvc.KvcError) as e:
        kvc.kvc_page_attend(pool, pages, q, torch.empty_like(q))  # two layers at once
    assert e.value.code == -1
    lay = pages.layer(1)
    for bad in (q[..., :32], q.transpose(2, 3), q.cpu()):
        with pytest.raises(ValueError):
            kvc.kvc_page_attend(pool, lay, bad, torch.empty_like(q))
    with pytest.raises(ValueError):
        kvc.kvc_page_attend(pool, lay, q, torch.empty_like(q).float())
    with pytest.raises(ValueError):
        kvc.kvc_page_extend(pool, pages, add=torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        kvc.kvc_page_extend(pool, pages, add=torch.zeros(2, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        kvc.kvc_page_store(pool, lay, q[:, :, :2], q[:, :, :2].float(), torch.zeros((1, 2, 2), dtype=torch.int32, device=DEV))
    with pytest.raises(kvc.KvcError):
        kvc.Pool.empty(8, 96, 16, device=DEV)
    with pytest.raises(kvc.KvcError) as e:
        kvc.kvc_page_fork(pool, pages, torch.zeros(2, dtype=torch.int32, device=DEV), pages)
    assert e.value.code == -1
