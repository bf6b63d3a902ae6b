"""The plain model of the paged cache against hand-worked values, and the entry points' refusals (no GPU)."""
import ctypes as C

import numpy as np
import pytest

import page_util as R


def test_quantise_handworked():
    x = np.zeros((1, 64))
    x[0, :8] = [6.0, -6.0, 0.25, 0.75, 1.25, -1.75, 2.5, 5.0]     # scale 1: ties go to the even code
    x[0, 16:20] = [448.0 * 6, -1e9, 1e9, 3.0]                     # saturates at 448 * 6
    x[0, 32] = 1e-5                                               # the smallest scale, 2^-9
    codes, sb = R.quantise(x, 1.0)
    assert [R.E4M3[b] for b in sb[0]] == [1.0, 448.0, 2.0 ** -9, 2.0 ** -9]
    assert list(codes[0, :4]) == [0xF7, 0x20, 0xC2, 0x64]  # 7 15 | 0 2 | 2 12 | 4 6
    v = R.values(codes, sb, 1.0)
    assert list(v[0, :8]) == [6.0, -6.0, 0.0, 1.0, 1.0, -2.0, 2.0, 4.0]
    assert list(v[0, 16:20]) == [2688.0, -2688.0, 2688.0, 0.0]
    assert v[0, 32] == 0.0 and v[0, 48] == 0.0


def test_quantise_is_nearest():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * np.exp(rng.standard_normal((200, 1)) * 2)
    codes, sb = R.quantise(x, 0.5)
    v = R.values(codes, sb, 0.5)
    step = np.repeat(R.E4M3[sb] * 0.5, 16, -1)
    # the widest code interval is 2 steps (half of it 1); a scale is within 2^-4 of amax / (6 ts), which leaves at
    # most 0.4 steps cut off, or for the subnormal ones (steps of 2^-9) within 2^-10: 6 ts 2^-10 cut off
    assert (np.abs(v - x) <= step + 6 * 0.5 * 2.0 ** -10).all()


def e2m1_of(y):
    """The magnitude code of |y| (fp32 or exact), ties to the even code, saturating."""
    a = np.abs(y)
    return sum(((a > b) if k % 2 == 0 else (a >= b)).astype(np.int64)
               for k, b in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))


def test_rounded_reciprocals_decide_as_exact_quotients_do():
    """The store's short way for bf16 rows and tensor scales that are powers of two (page_store.cu), in fp32 as the
    kernel computes it, over every bf16 significand: every scale, with its reciprocal an ulp off either way, and every
    code under every scale, likewise. A power of two as tensor scale shifts exponents only: 1 stands for all."""
    f, one = np.float32, np.float32(1)
    bits = lambda x: np.asarray(x, f).view(np.uint32)
    ulps = lambda x: [np.asarray(bits(x).astype(np.int64) + d, np.int64).astype(np.uint32).view(f) for d in (-1, 0, 1)]
    sig = np.arange(128, 256, dtype=np.float64)
    # scales: quotients from a quarter of the smallest scale to four times the largest
    amax = (sig[:, None] * np.exp2(np.arange(-18, 12))[None]).ravel()
    want = R.quantise(np.repeat(amax[:, None], 64, 1), 1.0)[1][:, 0]
    assert amax.min() / 6 < 2.0 ** -11 and amax.max() / 6 > 4 * 448 and want.min() == 1 and want.max() == 126
    for inv6 in ulps(one / f(6)):
        q = np.clip(amax.astype(f) * inv6, f(2.0 ** -9), f(448))
        q = ((bits(q) + np.uint32(0x400)) & np.uint32(0xfffff800)).view(f).astype(np.float64)
        pos = R.E4M3[:127]
        hi = np.clip(np.searchsorted(pos, q), 1, 126)
        dl, dh = q - pos[hi - 1], pos[hi] - q
        np.testing.assert_array_equal(np.where((dl < dh) | ((dl == dh) & (hi % 2 == 1)), hi - 1, hi), want)
    # codes
    for sb in range(1, 127):
        step = R.E4M3[sb]
        e = np.arange(-5, 6) + np.floor(np.log2(step)) - 7
        x = (sig[:, None] * np.exp2(e)[None]).ravel()
        assert x.min() / step < 0.125 and x.max() / step > 16
        borders = np.array((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)) * step  # exact: at most seven bits
        want = sum(((x > b) if k % 2 == 0 else (x >= b)).astype(np.int64) for k, b in enumerate(borders))
        for r in ulps(one / f(step)):
            for sign in (1, -1):
                # the product has at most 32 bits and its sum with 1536 at most 53: one rounding, as fma's
                y = (sign * x * np.float64(r) + 1536).astype(f) - f(1536)
                np.testing.assert_array_equal(e2m1_of(y), want, err_msg=str((sb, r, sign)))


def test_reference_extend_copies_on_write():
    p = R.RefPool(8, 64, 16)
    t = R.RefPages(1, 2, 1, 4)
    assert (R.extend(p, t, [20, 0]) == [[[0], [0]]]).all()
    assert list(t.table[0, 0, 0]) == [0, 1, -1, -1] and p.nfree == 6
    t = R.fork(p, t, [0, 0])
    assert list(p.refs[:2]) == [2, 2]
    R.extend(p, t, [1, 1])  # both write the shared last page: the lower sequence keeps it
    assert list(t.table[0, 0, 0]) == [0, 1, -1, -1] and list(t.table[0, 1, 0]) == [0, 2, -1, -1]
    assert list(p.refs[:3]) == [2, 1, 1] and p.nfree == 5
    R.free(p, t, [21, 0])
    assert p.nfree == 6 and list(p.free[:6]) == [7, 6, 5, 4, 3, 1] and list(p.refs[:3]) == [1, 0, 1]


@pytest.fixture(scope="module")
def lib():
    from decoding_kv_cache_gb300 import build, kvc
    build.build()
    return kvc.lib()


def _pool(kvc, **kw):
    return kvc.kvc_pool(**{**dict(D=128, page=64, npages=100, pad_=0, k_scale=1.0, v_scale=1.0, data=0x10000,
                                  refs=0x20000, free_list=0x30000, nfree=0x40000), **kw})


def _pages(kvc, **kw):
    return kvc.kvc_pages(**{**dict(L=1, B=2, Hkv=2, maxp=8, table=0x100000, len=0x200000), **kw})


def test_page_bytes(lib):
    assert lib.kvc_page_bytes(128, 64) == 4 * 2304 and lib.kvc_page_bytes(64, 16) == 1152
    for D, page in ((96, 64), (128, 8), (128, 48), (128, 512), (128, 0), (128, -16)):
        assert lib.kvc_page_bytes(D, page) == 0


@pytest.mark.parametrize("pool,pages,code", [
    (dict(D=96), {}, -3), (dict(page=48), {}, -1), (dict(npages=0), {}, -1), (dict(npages=1 << 29), {}, -9),
    (dict(pad_=1), {}, -1), (dict(k_scale=0.0), {}, -1), (dict(v_scale=float("nan")), {}, -1),
    (dict(k_scale=float("inf")), {}, -1), (dict(data=None), {}, -1), (dict(data=0x10008), {}, -8),
    (dict(refs=None), {}, -1), (dict(nfree=0x40002), {}, -8),
    ({}, dict(L=0), -1), ({}, dict(B=1 << 20, Hkv=2), -9), ({}, dict(maxp=0), -1), ({}, dict(maxp=1 << 25), -9),
    ({}, dict(table=None), -1), ({}, dict(len=0x200002), -8),
])
def test_every_entry_refuses_bad_pools_and_pages(lib, pool, pages, code):
    from decoding_kv_cache_gb300 import kvc
    p, t, o = _pool(kvc, **pool), _pages(kvc, **pages), _pages(kvc, table=0x900000, len=0xa00000)
    ws, nb, st = 0x1000000, 1 << 40, (C.c_int64 * 3)(512, 256, 128)
    assert lib.kvc_page_workspace_size(C.byref(p), C.byref(t)) == 0
    assert lib.kvc_page_init(C.byref(p), C.byref(t), None) == code
    assert lib.kvc_page_extend(C.byref(p), C.byref(t), None, 1, None, None, ws, nb, None) == code
    assert lib.kvc_page_free(C.byref(p), C.byref(t), None, 1, None, ws, nb, None) == code
    assert lib.kvc_page_fork(C.byref(p), C.byref(t), 0x1000, C.byref(o), None, ws, nb, None) == code
    assert lib.kvc_page_compact(C.byref(p), C.byref(t), 0x1000, 0x1000, 8, 0, None, ws, nb, None) == code
    assert lib.kvc_page_store(C.byref(p), C.byref(t), 0, 1, 0x1000, st, 0x1000, st, None, 0x1000, None, None) == code
    assert lib.kvc_page_read(C.byref(p), C.byref(t), 0, None, 0, 8, 0x1000, None, 8, None, None) == code
    assert lib.kvc_page_attend(C.byref(p), C.byref(t), 0, 4, 1, 0x1000, st, None, 0.1, 0x1000, None, None, ws, nb,
                               None) == code
    assert lib.kvc_page_attend_workspace_size(C.byref(p), C.byref(t), 4, 1) == 0


def test_page_operators_refuse_bad_arguments(lib):
    from decoding_kv_cache_gb300 import kvc
    p, t = _pool(kvc), _pages(kvc)
    ws, nb = 0x1000000, 1 << 40
    P, T = C.byref(p), C.byref(t)
    need = lib.kvc_page_workspace_size(P, T)
    assert need > 0
    for w, b in ((None, nb), (ws, need - 1), (ws + 16, nb)):
        assert lib.kvc_page_extend(P, T, None, 1, None, None, w, b, None) == -7
        assert lib.kvc_page_free(P, T, None, 1, None, w, b, None) == -7
        assert lib.kvc_page_compact(P, T, 0x1000, 0x1000, 8, 0, None, w, b, None) == -7
    assert lib.kvc_page_extend(P, T, None, -1, None, None, ws, nb, None) == -1
    assert lib.kvc_page_free(P, T, None, -1, None, ws, nb, None) == -1
    o = lambda **kw: C.byref(_pages(kvc, **{**dict(table=0x900000, len=0xa00000), **kw}))
    fork = lambda out, parent=0x1000: lib.kvc_page_fork(P, T, parent, out, None, ws, nb, None)
    assert fork(o(), None) == -1 and fork(o(L=2)) == -1 and fork(o(Hkv=4)) == -1 and fork(o(maxp=9)) == -1
    assert fork(T) == -1 and fork(o(table=0x100000 + 64)) == -1 and fork(o(len=0x200004)) == -1  # overlapping
    assert fork(o(B=1 << 21)) == -9
    assert lib.kvc_page_compact(P, T, None, 0x1000, 8, 0, None, ws, nb, None) == -1
    assert lib.kvc_page_compact(P, T, 0x1000, None, 8, 0, None, ws, nb, None) == -1
    assert lib.kvc_page_compact(P, T, 0x1000, 0x1000, 0, 0, None, ws, nb, None) == -1
    assert lib.kvc_page_compact(P, T, 0x1000, 0x1000, 8, 2, None, ws, nb, None) == -1


def test_rows_refused(lib):
    from decoding_kv_cache_gb300 import kvc
    p, t = _pool(kvc), _pages(kvc)
    S = lambda a=512, b=256, c=128: (C.c_int64 * 3)(a, b, c)

    def store(**kw):
        d = {**dict(t=t, dt=0, T=1, k=0x1000, ks=S(), v=0x2000, vs=S(), start=0x3000), **kw}
        return lib.kvc_page_store(C.byref(p), C.byref(d["t"]), d["dt"], d["T"], d["k"], d["ks"], d["v"], d["vs"], None,
                                  d["start"], None, None)
    assert store(dt=2) == -2 and store(T=0) == -1 and store(k=None) == -1 and store(v=None) == -1
    assert store(start=None) == -1 and store(k=0x1008) == -8 and store(ks=S(512, 256, 100)) == -8
    assert store(vs=S(-512)) == -1 and store(ks=None) == -1 and store(t=_pages(kvc, L=2)) == -1

    def read(**kw):
        d = {**dict(dt=0, first=0, count=8, k=0x1000, v=0x2000, ncap=8), **kw}
        return lib.kvc_page_read(C.byref(p), C.byref(t), d["dt"], None, d["first"], d["count"], d["k"], d["v"],
                                 d["ncap"], None, None)
    assert read(dt=-1) == -2 and read(k=None, v=None) == -1 and read(count=0) == -1 and read(ncap=7) == -1
    assert read(first=-1) == -1 and read(v=0x2004) == -8

    def attend(**kw):
        d = {**dict(t=t, dt=0, Hq=4, T=1, q=0x1000, qs=S(), scale=0.1, out=0x2000, lse=None, ws=0x1000000, nb=1 << 40), **kw}
        return lib.kvc_page_attend(C.byref(p), C.byref(d["t"]), d["dt"], d["Hq"], d["T"], d["q"], d["qs"], None,
                                   d["scale"], d["out"], d["lse"], None, d["ws"], d["nb"], None)
    assert attend(dt=3) == -2 and attend(Hq=0) == -1 and attend(Hq=5) == -5 and attend(T=0) == -1
    assert attend(q=None) == -1 and attend(q=0x1004) == -8 and attend(qs=S(512, 256, 4)) == -8
    assert attend(scale=float("nan")) == -1 and attend(out=None) == -1 and attend(out=0x2008) == -8
    assert attend(lse=0x3001) == -8 and attend(ws=None) == -7 and attend(nb=8) == -7 and attend(ws=0x1000010) == -7
    assert attend(t=_pages(kvc, L=3)) == -1 and attend(T=1 << 30) == -9
    p.k_scale = 1e20
    assert attend(scale=1e30) == -1  # their product is no finite number


def test_page_totals_stay_in_32_bits(lib):
    """2^20 streams of 2^11 entries: a call could ask for 2^31 pages, one more than its 32-bit sums hold."""
    from decoding_kv_cache_gb300 import kvc
    p, o = _pool(kvc, page=16), _pages(kvc, L=16, B=256, Hkv=256, maxp=1 << 11, table=0x900000000, len=0xf00000000)
    ws, nb = 0x1000000, 1 << 50
    t = _pages(kvc, L=16, B=256, Hkv=256, maxp=(1 << 11) - 1)
    assert lib.kvc_page_workspace_size(C.byref(p), C.byref(t)) > 0
    assert lib.kvc_page_workspace_size(C.byref(p), C.byref(o)) == 0
    assert lib.kvc_page_init(C.byref(p), C.byref(o), None) == -9
    assert lib.kvc_page_extend(C.byref(p), C.byref(o), None, 16, None, None, ws, nb, None) == -9
    assert lib.kvc_page_free(C.byref(p), C.byref(o), None, 16, None, ws, nb, None) == -9
    assert lib.kvc_page_fork(C.byref(p), C.byref(t), 0x1000, C.byref(o), None, ws, nb, None) == -9
    assert lib.kvc_page_compact(C.byref(p), C.byref(o), 0x1000, 0x1000, 8, 0, None, ws, nb, None) == -9


def test_fork_refuses_arrays_that_overlap_crosswise(lib):
    """The children's table in the parents' lengths, or their lengths in the parents' table."""
    from decoding_kv_cache_gb300 import kvc
    p, t = _pool(kvc), _pages(kvc)  # table: 2 * 2 * 8 words at 0x100000, len: 4 words at 0x200000
    for kw in (dict(table=0x200000 - 64, len=0xa00000), dict(table=0x900000, len=0x100000 + 124),
               dict(table=0x900000, len=0x900000 + 64)):
        o = _pages(kvc, **kw)
        assert lib.kvc_page_fork(C.byref(p), C.byref(t), 0x1000, C.byref(o), None, 0x1000000, 1 << 40, None) == -1
