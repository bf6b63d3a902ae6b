"""kvc_page_slide's wide form (more than 4096 streams, or a pool of more than 2^20 pages) against the plain model: tables, lengths,
counts, the free list and every byte."""
import numpy as np
import pytest
import torch

import page_util as R
import tree_util as Q
from test_gpu_page import DEV, Both, up

pytestmark = pytest.mark.gpu


def slide(x, window, sinks=0, bad=(), **kw):
    """One call; streams of `bad` have a length that is none."""
    gone = torch.full(x.t.shape, 77, dtype=torch.int32, device=DEV)
    x.kvc.kvc_page_slide(x.pool, x.pages, window, sinks, gone=gone, status=x.status, **kw)
    held = [(int(x.t.len[s]), x.t.table[s].copy()) for s in bad]
    for s in bad:
        x.t.len[s] = 0
    want = Q.slide(x.p, x.t, window, sinks)
    for s, (n, row) in zip(bad, held):  # left alone
        x.t.len[s], x.t.table[s], want[s] = n, row, -1
    if bad:
        x.p.status |= R.BAD_PAGE
    np.testing.assert_array_equal(gone.cpu().numpy(), want)


@pytest.mark.parametrize("L,B,Hkv,page,maxp", [(40, 14, 8, 16, 12), (1, 4099, 1, 32, 8), (13, 160, 2, 16, 10)])
def test_more_than_4096_streams(L, B, Hkv, page, maxp):
    """4480, 4099 (no multiple of anything) and 4160 streams of every length, pages shared by forks, lengths that are none."""
    rng = np.random.default_rng(L)
    x = Both(L * B * Hkv * maxp, 64, page, L, (B + 1) // 2, Hkv, maxp, seed=L)
    x.extend(rng.integers(0, maxp * page - 20, (B + 1) // 2).tolist())
    x.fork((np.arange(B) // 2).tolist())
    x.free(rng.integers(0, 2 * page, B).tolist())
    x.extend(rng.integers(0, 20, B).tolist())
    x.check("made")
    ws = torch.full((x.kvc.kvc_page_workspace_size(x.pool, x.pages),), 0xff, dtype=torch.uint8, device=DEV)
    for window, sinks in ((5 * page + 5, 4), (3 * page, page + 1), (page + 1, 0), (1 << 30, 0)):
        slide(x, window, sinks, workspace=ws)
        x.check((window, sinks))
    bad = [(0, 0, 0), (L - 1, B - 1, Hkv - 1), (L // 2, B // 2, Hkv // 2)]
    for s, n in zip(bad, (-1, maxp * page + 1, -(1 << 31))):
        x.t.len[s] = n
        x.pages.len[s] = n
    slide(x, 1, 0, bad=bad, workspace=ws)
    x.check("lengths that are none")
    slide(x, 1, 0, bad=bad)
    x.check("nothing left")


def test_pages_that_are_none_and_held_by_nobody():
    """4800 streams, among the entries given up numbers that are no page's and pages whose count is zero: reported, the streams'
    other pages go."""
    L, B, Hkv, page, maxp = 40, 15, 8, 16, 6
    x = Both(L * B * Hkv * maxp, 64, page, L, B, Hkv, maxp, seed=2)
    x.extend([5 * page + 3] * B)
    x.check("made")
    t = x.pages.table
    none, free = (3, 4, 5, 1), (39, 14, 7, 2)
    lost, held = int(t[none]), int(t[free])
    t[none] = 1 << 30
    x.pool.refs[held] = 0
    gone = torch.zeros(x.t.shape, dtype=torch.int32, device=DEV)
    x.kvc.kvc_page_slide(x.pool, x.pages, page, 2, gone=gone, status=x.status)
    assert int(x.status.item()) == R.BAD_PAGE
    assert (gone == 3 * page).all() and (x.pages.len == 2 * page + 3).all() and (x.pages.table[..., 3:] == -1).all()
    np.testing.assert_array_equal(x.pages.table[..., 0].cpu().numpy(), x.t.table[..., 0])
    np.testing.assert_array_equal(x.pages.table[..., 1:3].cpu().numpy(), x.t.table[..., 4:6])
    n = int(x.pool.nfree.item())
    assert n == x.p.nfree + 3 * L * B * Hkv - 2
    back = x.pool.free_list[x.p.nfree:n].cpu().numpy()
    assert (np.diff(back) > 0).all() and not {lost, held} & set(back.tolist())
    assert set(back.tolist()) == set(x.t.table[..., 1:4].reshape(-1).tolist()) - {lost, held}


def test_more_than_a_million_pages():
    kvc = __import__("decoding_kv_cache_gb300.kvc", fromlist=["kvc"])
    npages, page, L, B, Hkv, maxp = (1 << 20) + 77, 16, 3, 5, 7, 40
    pool, pages = kvc.Pool.empty(npages, 64, page, device=DEV), kvc.Pages.empty(L, B, Hkv, maxp, device=DEV)
    pool.free_list.copy_(torch.arange(npages, dtype=torch.int32, device=DEV))  # the last pages first
    p = R.RefPool(npages, 64, page)
    p.free = np.arange(npages, dtype=np.int32)
    t = R.RefPages(L, B, Hkv, maxp)
    rng, status = np.random.default_rng(3), torch.zeros(1, dtype=torch.int32, device=DEV)
    for window, sinks in ((100, 4), (33, 0), (1, 17)):
        add = rng.integers(0, 200, B)
        kvc.kvc_page_extend(pool, pages, add=up(add.astype(np.int32)), status=status)
        R.extend(p, t, add)
        gone = torch.zeros((L, B, Hkv), dtype=torch.int32, device=DEV)
        kvc.kvc_page_slide(pool, pages, window, sinks, gone=gone, status=status)
        np.testing.assert_array_equal(gone.cpu().numpy(), Q.slide(p, t, window, sinks))
        for a, b in ((pages.table, t.table), (pages.len, t.len), (pool.refs, p.refs)):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
        assert int(pool.nfree.item()) == p.nfree and int(status.item()) == 0
        np.testing.assert_array_equal(pool.free_list[:p.nfree].cpu().numpy(), p.free[:p.nfree])


def test_captured_and_replayed():
    """5120 streams: room, a slide and a rollback in a graph, with an eager slide on the same workspace between."""
    kvc = __import__("decoding_kv_cache_gb300.kvc", fromlist=["kvc"])
    L, B, Hkv, page, maxp = 40, 16, 8, 16, 8
    x = Both(L * B * Hkv * maxp, 64, page, L, B, Hkv, maxp, seed=4)
    ws = torch.empty(kvc.kvc_page_workspace_size(x.pool, x.pages), dtype=torch.uint8, device=DEV)
    add, drop = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)

    def step():
        kvc.kvc_page_extend(x.pool, x.pages, add=add, status=x.status, workspace=ws)
        kvc.kvc_page_slide(x.pool, x.pages, 40, 3, status=x.status, workspace=ws)
        kvc.kvc_page_free(x.pool, x.pages, drop=drop, status=x.status, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(5)
    for i in range(5):
        a, d = rng.integers(0, 60, B), rng.integers(0, 9, B)
        add.copy_(up(a.astype(np.int32)))
        drop.copy_(up(d.astype(np.int32)))
        graph.replay()
        R.extend(x.p, x.t, a)
        Q.slide(x.p, x.t, 40, 3)
        R.free(x.p, x.t, d)
        x.check(i)
        slide(x, 20, 0, workspace=ws)
        x.check((i, "eager"))
