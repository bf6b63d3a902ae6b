"""The plain model of the tree and window operators against hand-worked cases, and every refusal of their entry points on
the host (no GPU)."""
import ctypes as C

import numpy as np
import pytest

import page_util as R
import tree_util as Q


def words(*bits):
    return sum(1 << b for b in bits)


def test_tree_mask_handworked():
    #   0 - 1 - 3        2 (a second root) - 5
    #     \ 4
    parent = np.array([[-1, 0, -1, 1, 0, 2]], np.int32)
    mask, depth, status = Q.tree_mask(parent)
    assert list(mask[0, :, 0]) == [words(0), words(0, 1), words(2), words(0, 1, 3), words(0, 4), words(2, 5)]
    assert list(depth[0]) == [0, 1, 0, 2, 1, 1] and status == 0
    mask, depth, _ = Q.tree_mask(parent, window=2)
    assert list(mask[0, :, 0]) == [words(0), words(0, 1), words(2), words(1, 3), words(0, 4), words(2, 5)]
    mask, depth, _ = Q.tree_mask(parent, n_q=[4])
    assert list(mask[0, :, 0]) == [words(0), words(0, 1), words(2), words(0, 1, 3), 0, 0] and list(depth[0, 4:]) == [0, 0]
    for bad in ([[0]], [[-2]], [[-1, 1]], [[-1, 0, 3]]):
        mask, depth, status = Q.tree_mask(np.array(bad, np.int32))
        assert status == R.BAD_INDEX and not mask.any() and not depth.any()


def test_tree_verify_handworked():
    parent = np.array([[-1, 0, 0, 1, 2, 2]], np.int32)
    draft = np.array([[9, 5, 5, 6, 6, 7]], np.int32)
    #  the root's pick 5: the lower of drafts 1 and 2; behind it 6: draft 3
    path, n, nxt, _ = Q.tree_verify(parent, draft, np.array([[5, 6, 7, 8, 0, 0]], np.int32))
    assert list(path[0]) == [0, 1, 3, -1, -1, -1] and n[0] == 3 and nxt[0] == 8
    path, n, nxt, _ = Q.tree_verify(parent, draft, np.array([[4, 6, 7, 8, 0, 0]], np.int32))
    assert list(path[0]) == [0] + [-1] * 5 and n[0] == 1 and nxt[0] == 4
    path, n, nxt, _ = Q.tree_verify(parent, draft, np.array([[5, 6, 7, 8, 0, 0]], np.int32), n_q=[0])
    assert n[0] == 0 and nxt[0] == -1


def test_seen_tokens_handworked():
    see = lambda *a, **k: list(Q.seen_tokens(*a, **k))
    assert see(5, 1, 0) == [0, 1, 2, 3, 4]
    assert see(10, 2, 0, window=3, sinks=2) == [0, 1, 6, 7, 8] and see(10, 2, 1, window=3, sinks=2) == [0, 1, 7, 8, 9]
    assert see(10, 2, 1, window=1) == [9] and see(3, 5, 1) == [] and see(3, 5, 2) == [0]
    mask = np.array([words(0, 2)], np.uint32).view(np.int32)
    assert see(10, 4, 2, mask=mask) == [0, 1, 2, 3, 4, 5, 6, 8]
    assert see(10, 4, 2, window=3, sinks=1, mask=mask, depth=[0, 1, 1, 2]) == [0, 5, 6, 8]  # stands at 7
    assert see(10, 4, 2, window=3, sinks=1, mask=mask) == [0, 6, 8]                         # at 8


def test_slide_handworked():
    p, t = R.RefPool(12, 64, 16), R.RefPages(1, 3, 1, 8)
    R.extend(p, t, [100, 47, 16])  # 7, 3 and 1 pages
    gone = Q.slide(p, t, window=40, sinks=4)
    # 100 tokens: the next query sees from 61 on, so pages 1 and 2 (16..47) go; 47: from 8 on, nothing
    assert list(gone[0, :, 0]) == [32, 0, 0] and list(t.len[0, :, 0]) == [68, 47, 16]
    assert list(t.table[0, 0, 0]) == [0, 3, 4, 5, 6, -1, -1, -1] and p.nfree == 3 and list(p.free[:3]) == [11, 1, 2]


def test_a_slide_changes_no_windowed_attention():
    rng = np.random.default_rng(1)
    for _ in range(200):
        n, w, k, page = int(rng.integers(1, 200)), int(rng.integers(1, 80)), int(rng.integers(0, 40)), 16
        new = int(rng.integers(1, 5))
        p, t = R.RefPool(20, 64, page), R.RefPages(1, 1, 1, 16)
        R.extend(p, t, [n])
        token = {}  # (page, place) -> the token's number before the slide
        for j in range(n):
            token[t.table[0, 0, 0][j // page], j % page] = j
        Q.slide(p, t, w, k)
        m = int(t.len[0, 0, 0])
        for i in range(new):
            a = Q.seen_tokens(n + new, new, i, w, k)
            b = Q.seen_tokens(m + new, new, i, w, k)
            old = [token[t.table[0, 0, 0][j // page], j % page] if j < m else j - m + n for j in b]
            assert list(a) == old


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


@pytest.mark.parametrize("pool,pages,code", [
    (dict(D=96), {}, -3), (dict(page=48), {}, -1), (dict(npages=0), {}, -1), (dict(npages=1 << 29), {}, -9),
    (dict(k_scale=0.0), {}, -1), (dict(data=0x10008), {}, -8), (dict(refs=None), {}, -1),
    ({}, dict(L=0), -1), ({}, dict(B=1 << 20, Hkv=2), -9), ({}, dict(maxp=1 << 25), -9), ({}, dict(table=None), -1),
    ({}, dict(len=0x200002), -8),
])
def test_every_entry_refuses_bad_pools_and_pages(lib, pool, pages, code):
    from decoding_kv_cache_gb300 import kvc
    p, t = _pool(kvc, **pool), _pages(kvc, **pages)
    ws, nb, st = 0x1000000, 1 << 40, (C.c_int64 * 3)(512, 256, 128)
    P, T = C.byref(p), C.byref(t)
    assert lib.kvc_page_slide(P, T, 8, 0, None, None, ws, nb, None) == code
    assert lib.kvc_page_accept(P, T, 4, 0x1000, 0x1000, None, None, ws, nb, None) == code
    assert lib.kvc_page_attend_masked(P, T, 0, 4, 1, 0x1000, st, None, 8, 1, None, None, 0.1, 0x1000, None, None, ws, nb,
                                      None) == code
    assert lib.kvc_page_attend_masked_workspace_size(P, T, 4, 1, 8, 1) == 0


def test_attend_masked_refused(lib):
    from decoding_kv_cache_gb300 import kvc
    p, t = _pool(kvc), _pages(kvc)
    S = lambda a=512, b=256, c=128: (C.c_int64 * 3)(a, b, c)

    def attend(**kw):
        d = {**dict(t=t, dt=0, Hq=4, T=1, q=0x1000, qs=S(), window=8, sinks=1, mask=None, depth=None, scale=0.1, out=0x2000,
                    lse=None, ws=0x1000000, nb=1 << 40), **kw}
        return lib.kvc_page_attend_masked(C.byref(p), C.byref(d["t"]), d["dt"], d["Hq"], d["T"], d["q"], d["qs"], None,
                                          d["window"], d["sinks"], d["mask"], d["depth"], d["scale"], d["out"], d["lse"],
                                          None, d["ws"], d["nb"], None)
    assert attend(dt=3) == -2 and attend(Hq=0) == -1 and attend(Hq=5) == -5 and attend(T=0) == -1
    assert attend(q=None) == -1 and attend(q=0x1004) == -8 and attend(qs=S(512, 256, 4)) == -8 and attend(qs=None) == -1
    assert attend(scale=float("nan")) == -1 and attend(out=None) == -1 and attend(out=0x2008) == -8
    assert attend(lse=0x3001) == -8 and attend(ws=None) == -7 and attend(nb=8) == -7 and attend(ws=0x1000010) == -7
    assert attend(t=_pages(kvc, L=3)) == -1 and attend(T=1 << 30) == -9
    assert attend(window=-1) == -1 and attend(sinks=-1) == -1 and attend(depth=0x4000) == -1
    assert attend(mask=0x4002) == -8 and attend(mask=0x4000, depth=0x4001) == -8
    assert attend(mask=0x4000, T=kvc.KVC_TREE_MAX + 1) == -9
    size = lambda **kw: lib.kvc_page_attend_masked_workspace_size(C.byref(p), C.byref(t), *{
        **dict(Hq=4, T=1, window=8, sinks=1), **kw}.values())
    assert size() >= 256 and size(Hq=5) == 0 and size(T=0) == 0 and size(window=-1) == 0 and size(sinks=-1) == 0


def test_slide_and_accept_refused(lib):
    from decoding_kv_cache_gb300 import kvc
    p, t = _pool(kvc), _pages(kvc)
    P, T, ws, nb = C.byref(p), C.byref(t), 0x1000000, 1 << 40
    need = lib.kvc_page_workspace_size(P, T)
    slide = lambda window=8, sinks=0, gone=None, w=ws, b=nb: lib.kvc_page_slide(P, T, window, sinks, gone, None, w, b, None)
    assert slide(window=0) == -1 and slide(window=-5) == -1 and slide(sinks=-1) == -1 and slide(gone=0x1002) == -8
    acc = lambda n=4, path=0x1000, k=0x2000, nq=None, w=ws, b=nb: lib.kvc_page_accept(P, T, n, path, k, nq, None, w, b, None)
    assert acc(n=0) == -1 and acc(path=None) == -1 and acc(k=None) == -1 and acc(n=kvc.KVC_TREE_MAX + 1) == -9
    assert acc(path=0x1001) == -8 and acc(k=0x2002) == -8 and acc(nq=0x2001) == -8
    for w, b in ((None, nb), (ws, need - 1), (ws + 16, nb)):
        assert slide(w=w, b=b) == -7 and acc(w=w, b=b) == -7


def test_tree_operators_refused(lib):
    from decoding_kv_cache_gb300 import kvc
    mask = lambda B=2, T=4, parent=0x1000, nq=None, w=0, m=0x2000, d=None: lib.kvc_tree_mask(B, T, parent, nq, w, m, d, None, None)
    assert mask(B=0) == -1 and mask(T=0) == -1 and mask(parent=None) == -1 and mask(w=-1) == -1 and mask(m=None) == -1
    assert mask(T=kvc.KVC_TREE_MAX + 1) == -9 and mask(B=(1 << 20) + 1) == -9
    assert mask(parent=0x1002) == -8 and mask(m=0x2001) == -8 and mask(nq=0x3001) == -8 and mask(d=0x3002) == -8

    def verify(**kw):
        d = {**dict(B=2, T=4, parent=0x1000, draft=0x2000, target=0x3000, nq=None, path=0x4000, k=0x5000, nxt=None), **kw}
        return lib.kvc_tree_verify(*d.values(), None, None)
    assert verify(B=0) == -1 and verify(T=0) == -1 and verify(T=1025) == -9 and verify(B=1 << 21) == -9
    for name in ("parent", "draft", "target", "path", "k"):
        assert verify(**{name: None}) == -1 and verify(**{name: 0x9001}) == -8
    assert verify(nq=0x9002) == -8 and verify(nxt=0x9003) == -8
