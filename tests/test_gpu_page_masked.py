"""Windows and drafted trees over the paged 4-bit cache on the GPU, against the plain 64-bit model of tree_util: whole
numbers and every byte of the pool equal, attention within page_util.tolerances."""
import numpy as np
import pytest
import torch

import page_util as R
import tree_util as Q
from test_gpu_page import DEV, DT, Both, make_attend, rand_rows, up

pytestmark = pytest.mark.gpu


def kvc_():
    from decoding_kv_cache_gb300 import kvc
    return kvc


# ---- trees -----------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("B,T", [(1, 1), (3, 7), (2, 31), (2, 32), (2, 33), (5, 64), (3, 100), (2, 257), (1, 1024)])
def test_tree_mask(B, T):
    kvc, rng = kvc_(), np.random.default_rng(T)
    for n_q in (None, rng.integers(-1, T + 2, B)):
        for window in (0, 1, 3):
            parent = Q.random_trees(rng, B, T, n_q)
            want, wd, _ = Q.tree_mask(parent, n_q, window)
            mask = torch.full((B, T, (T + 31) // 32), 77, dtype=torch.int32, device=DEV)
            depth = torch.full((B, T), 77, dtype=torch.int32, device=DEV)
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            nq = None if n_q is None else up(n_q.astype(np.int32))
            kvc.kvc_tree_mask(up(parent), mask, depth, n_q=nq, window=window, status=status)
            np.testing.assert_array_equal(mask.cpu().numpy(), want)
            np.testing.assert_array_equal(depth.cpu().numpy(), wd)
            assert int(status.item()) == 0
            only = torch.full_like(mask, 77)
            kvc.kvc_tree_mask(up(parent), only, n_q=nq, window=window)
            assert torch.equal(only, mask)


def test_tree_chain_of_1024_and_malformed_parents():
    kvc, T = kvc_(), 1024
    parent = np.tile(np.arange(-1, T - 1, dtype=np.int32), (3, 1))
    parent[1, 700] = 700
    parent[2, 3] = -2
    mask, depth = torch.empty((3, T, 32), dtype=torch.int32, device=DEV), torch.empty((3, T), dtype=torch.int32, device=DEV)
    for n_q, bad in ((None, R.BAD_INDEX), ([T, 700, 3], 0)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        kvc.kvc_tree_mask(up(parent), mask, depth, n_q=None if n_q is None else up(np.array(n_q, np.int32)), status=status)
        want, wd, _ = Q.tree_mask(parent, n_q)
        np.testing.assert_array_equal(mask.cpu().numpy(), want)
        np.testing.assert_array_equal(depth.cpu().numpy(), wd)
        assert int(status.item()) == bad


@pytest.mark.parametrize("B,T", [(1, 1), (3, 7), (9, 32), (5, 33), (6, 100), (2, 1024)])
def test_tree_verify(B, T):
    kvc, rng = kvc_(), np.random.default_rng(T + B)
    for n_q in (None, rng.integers(-1, T + 2, B)):
        for tokens in (2, 5, 1 << 20):  # few tokens: siblings that are alike
            parent = Q.random_trees(rng, B, T, n_q)
            draft, target = rng.integers(-3, tokens, (2, B, T)).astype(np.int32)
            if tokens > 10:
                for b in range(B):
                    for i in range(1, Q.drafts(n_q, b, T)):
                        if parent[b, i] >= 0 and rng.random() < 0.8:
                            target[b, parent[b, i]] = draft[b, i]
            if B > 4:
                parent[4, 0] = 0  # malformed
            want = Q.tree_verify(parent, draft, target, n_q)
            path, n, nxt = (torch.full(s, 77, dtype=torch.int32, device=DEV) for s in ((B, T), (B,), (B,)))
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            kvc.kvc_tree_verify(up(parent), up(draft), up(target), path, n, next=nxt, status=status,
                                n_q=None if n_q is None else up(n_q.astype(np.int32)))
            for got, w in zip((path, n, nxt), want):
                np.testing.assert_array_equal(got.cpu().numpy(), w)
            assert int(status.item()) == want[3]


# ---- attention -------------------------------------------------------------------------------------------------
def check(x, q, dt, scale=None, n_q=None, window=0, sinks=0, mask=None, depth=None, bad=(), status=0, q_dev=None, **kw):
    """One call against the model. mask, depth: numpy. Returns out, lse."""
    B, T, Hq, D = q.shape
    sc = D ** -0.5 if scale is None else scale
    out = torch.full((B, T, Hq, D), -55.0, dtype=DT[dt], device=DEV)
    lse = torch.full((B, T, Hq), -55.0, device=DEV)
    dev = lambda v: None if v is None else up(np.asarray(v, np.int32))
    kvc_().kvc_page_attend_masked(x.pool, x.pages, q.to(DEV) if q_dev is None else q_dev, out, window=window, sinks=sinks,
                                  mask=dev(mask), depth=dev(depth), lse=lse, n_q=dev(n_q), scale=scale, status=x.status, **kw)
    torch.cuda.synchronize()
    ref = Q.attend(x.p, x.t, q.double().cpu().numpy(), sc, n_q, window, sinks, mask, depth, bad)
    tol, ltol = R.tolerances(dt, int(x.t.len.max()), D, ref)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        k = Q.drafts(n_q, b, T)
        assert (got[b, k:] == -55.0).all() and (gl[b, k:] == -55.0).all(), "rows behind the last query"
        err = np.abs(got[b, :k] - ref["out"][b, :k])
        assert (err <= tol[b, :k]).all(), (b, float((err / tol[b, :k]).max()))
        empty = np.isneginf(ref["lse"][b, :k])
        assert (np.isneginf(gl[b, :k]) == empty).all() and (got[b, :k][empty] == 0).all()
        le = np.abs(gl[b, :k][~empty] - ref["lse"][b, :k][~empty])
        assert (le <= ltol[b, :k][~empty]).all(), float((le / ltol[b, :k][~empty]).max())
    assert int(x.status.item()) == status
    return out, lse


SHAPES = [  # B, Hkv, G, T, page, lens
    (1, 1, 1, 1, 16, [1]),
    (2, 2, 1, 1, 16, [0, 1, 15, 16]),
    (3, 2, 4, 1, 64, [17, 63, 64, 65, 0, 200]),
    (2, 1, 8, 1, 256, [255, 300]),
    (1, 3, 7, 2, 32, [31, 500, 2]),
    (2, 2, 5, 3, 64, [2, 0, 130, 3]),       # fewer tokens than queries: the first see none
    (1, 2, 3, 17, 16, [17, 160]),
    (2, 1, 4, 40, 128, [100, 333]),
    (1, 1, 16, 5, 64, [77]),
    (1, 2, 1, 130, 64, [140, 100]),
    (1, 2, 7, 70, 64, [300, 69]),
]


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("B,Hkv,G,T,page,lens", SHAPES)
def test_window(dt, D, B, Hkv, G, T, page, lens):
    x, q = make_attend(dt, D, B, Hkv, G, T, page, lens, seed=B * 7 + T)
    n = max(lens)
    for window, sinks in {(1, 0), (2, 3), (16, 4), (17, 0), (65, 20), (max(1, n - 1), 1), (n + 5, 7), ((1 << 31) - 1, 0),
                          (max(1, n // 2), (1 << 31) - 1)}:
        check(x, q, dt, window=window, sinks=sinks)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("B,Hkv,G,T,page,lens", SHAPES)
def test_tree(dt, D, B, Hkv, G, T, page, lens):
    x, q = make_attend(dt, D, B, Hkv, G, T, page, lens, seed=B * 9 + T)
    rng = np.random.default_rng(T)
    parent = Q.random_trees(rng, B, T)
    mask, depth, _ = Q.tree_mask(parent)
    check(x, q, dt, mask=mask)
    for window, sinks in ((1, 0), (5, 2), (70, 9), (max(lens) + 3, 1)):
        check(x, q, dt, mask=Q.tree_mask(parent, window=window)[0], depth=depth, window=window, sinks=sinks)


@pytest.mark.parametrize("dt,D,G,T,page,lens", [
    ("bf16", 128, 4, 4, 64, [700, 3, 0, 1, 2000, 64]),
    ("f32", 64, 3, 5, 16, [900, 4, 5, 0, 33, 16]),
    ("bf16", 64, 2, 8, 32, [200, 7, 0, 8, 9, 100]),
    ("bf16", 128, 4, 90, 64, [700, 89, 90, 1, 0, 91]),
])
def test_any_mask_and_fewer_queries_than_rows(dt, D, G, T, page, lens):
    """Masks that are no tree's: random bits, bits past the last query, rows that see nothing of the drafts, or nothing at
    all; depths out of range; sequences with none, one, some and all of their queries."""
    x, q = make_attend(dt, D, 3, 2, G, T, page, lens, seed=T)
    rng = np.random.default_rng(T)
    W = (T + 31) // 32
    for n_q in (None, [0, 1, T], [T - 1, 2, 0], [T + 5, -1, T // 2]):
        mask = rng.integers(0, 1 << 32, (3, T, W), dtype=np.uint32)
        mask[:, T // 2] = 0
        mask[2] = 0
        depth = rng.integers(-3, T + 4, (3, T)).astype(np.int32)
        check(x, q, dt, n_q=n_q, mask=mask.view(np.int32), depth=depth, window=9, sinks=2)
        check(x, q, dt, n_q=n_q, mask=mask.view(np.int32), window=1)
        check(x, q, dt, n_q=n_q, mask=mask.view(np.int32))
        check(x, q, dt, n_q=n_q, window=7, sinks=1)


@pytest.mark.parametrize("dt,G,T,w", [("bf16", 4, 1, 100), ("bf16", 4, 1, 700), ("bf16", 4, 9, 200), ("bf16", 4, 50, 200), ("f32", 2, 2, 300)])
def test_no_lse_and_no_status(dt, G, T, w):
    x, q = make_attend(dt, 64, 2, 2, G, T, 16, [900, 30, 0, 700], seed=4)
    out, _ = check(x, q, dt, window=w, sinks=2)
    only = torch.full_like(out, -55.0)
    kvc_().kvc_page_attend_masked(x.pool, x.pages, q.to(DEV), only, window=w, sinks=2)
    assert torch.equal(out, only)


def test_no_window_and_no_mask_is_the_causal_attention():
    kvc = kvc_()
    for dt, G, T, lens in (("bf16", 4, 1, [900, 30, 0, 700]), ("bf16", 4, 30, [900, 30, 0, 700]), ("f32", 2, 3, [90, 2, 0, 1])):
        x, q = make_attend(dt, 128, 2, 2, G, T, 64, lens, seed=3)
        out, lse = check(x, q, dt, sinks=5)
        o2, l2 = torch.full_like(out, -55.0), torch.full_like(lse, -55.0)
        kvc.kvc_page_attend(x.pool, x.pages, q.to(DEV), o2, lse=l2)
        assert (o2.float() - out.float()).abs().max() <= 2.0 ** -6 * o2.float().abs().max()


@pytest.mark.parametrize("dt,T", [("bf16", 6), ("bf16", 30), ("f32", 6)])
def test_strided_scaled(dt, T):
    x, q0 = make_attend(dt, 128, 4, 2, 3, T, 32, [90, 80, 3, 4, 50, 60, 0, 0], seed=5, k_scale=0.3, v_scale=7.0)
    fused = torch.zeros((4, T, 11, 128), dtype=DT[dt], device=DEV)
    fused[:, :, 2:8] = q0.to(DEV)
    mask, depth, _ = Q.tree_mask(Q.random_trees(np.random.default_rng(2), 4, T))
    for qd in (fused[:, :, 2:8], q0.to(DEV).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)):
        check(x, q0, dt, scale=0.37, window=20, sinks=3, q_dev=qd)
        check(x, q0, dt, scale=-0.37, mask=mask, depth=depth, q_dev=qd, n_q=[1, T, 99, -3])


@pytest.mark.parametrize("dt,T", [("bf16", 2), ("bf16", 20), ("f32", 2)])
def test_extreme_logits(dt, T):
    x, q = make_attend(dt, 64, 2, 2, 2, T, 16, [300, 40, 16, 129], seed=11)
    mask, depth, _ = Q.tree_mask(Q.random_trees(np.random.default_rng(4), 2, T))
    args = (dict(window=33, sinks=4), dict(mask=mask), dict(mask=mask, depth=depth, window=50, sinks=3))
    for scale in (0.0, -0.5, 4.0, 30.0, 1e-6):
        for a in args:
            check(x, q, dt, scale=scale, **a)
    q[0] = 0
    q[1] *= 1000.0
    for a in args:
        check(x, q, dt, scale=0.125, **a)


@pytest.mark.parametrize("dt,T,cap", [("bf16", 1, 12), ("bf16", 1, 300), ("bf16", 20, 12), ("f32", 2, 12), ("bf16", 130, 12)])
def test_what_no_query_sees_does_not_count(dt, T, cap):
    """NaN scales and bad page numbers between the sinks and the window, behind the length, and in drafts that no row
    sees: nothing comes in, and what is not read is not reported. Bad pages that are seen are reported and take no
    part."""
    n, page, w, k = 120, 16, 20, 4
    x, q = make_attend(dt, 64, 2, 1, 2, T, page, [n + T, n], seed=2)
    table = torch.full((1, 2, 1, cap + (T > 100) * 16), -1, dtype=torch.int32, device=DEV)
    table[..., :x.pages.table.shape[-1]] = x.pages.table
    x.pages = x.kvc.Pages(table, x.pages.len)
    hidden = range(k, max(k, n - T + 1 - w))  # tokens that no query of either sequence sees (the second: base n - T)
    for j in hidden:
        for s in x.t.streams():
            for piece in (1, 3):
                x.p.piece(x.t.table[s][j // page], j, piece)[:] = 0x7f
    x.pool.data.copy_(up(x.p.data.reshape(x.p.npages, -1)))
    check(x, q, dt, window=w, sinks=k)
    if T == 1:  # whole pages that hold no seen token
        for e in range(1, (n - w) // page):
            x.pages.table[0, :, 0, e] = 1 << 29
        check(x, q, dt, window=w, sinks=k)
    x.pages.table[0, 0, 0, 0] = -1
    x.pages.table[0, 1, 0, (n - 1) // page] = 1 << 30
    bad = {(0, 0, 0), (1, 0, (n - 1) // page)}
    check(x, q, dt, window=w, sinks=k, bad=bad, status=R.BAD_PAGE)
    x.pages.len[0, 1, 0] = 1 << 20  # a length beyond the table: an empty stream
    x.t.len[0, 1, 0] = 0
    check(x, q, dt, window=w, sinks=k, bad=bad, status=R.BAD_PAGE)


def test_drafts_that_no_row_sees():
    """A draft with NaN scales that only one row's mask names: the other rows are not touched by it."""
    T, n = 24, 200
    x, q = make_attend("bf16", 128, 1, 1, 4, T, 64, [n], seed=8)
    for piece in (1, 3):
        x.p.piece(x.t.table[0, 0, 0][(n - T + 9) // 64], n - T + 9, piece)[:] = 0x7f
    x.pool.data.copy_(up(x.p.data.reshape(x.p.npages, -1)))
    parent = np.array([[-1] + [0] * (T - 1)], np.int32)
    mask, depth, _ = Q.tree_mask(parent)
    mask[0, 9] = mask[0, 8]  # nobody sees draft 9
    check(x, q, "bf16", mask=mask)
    x.p.piece(x.t.table[0, 0, 0][(n - T + 9) // 64], n - T + 9, 1)[:] = 0x38  # its keys are numbers, its values are not
    x.pool.data.copy_(up(x.p.data.reshape(x.p.npages, -1)))
    check(x, q, "bf16", mask=mask)


@pytest.mark.parametrize("dt,D,B,Hkv,G,T,n,w", [
    ("bf16", 128, 1, 2, 4, 1, 6000, 4000), ("f32", 64, 2, 2, 2, 1, 3001, 2500), ("bf16", 64, 1, 2, 8, 20, 2500, 1000),
    ("f32", 128, 1, 1, 3, 2, 4097, 4000), ("bf16", 128, 4, 8, 4, 16, 3000, 1500), ("bf16", 64, 2, 4, 5, 40, 2200, 700),
    ("bf16", 128, 1, 1, 4, 300, 1500, 400), ("bf16", 128, 1, 1, 7, 64, 2600, 0)])
def test_long(dt, D, B, Hkv, G, T, n, w):
    rng = np.random.default_rng(n)
    x, q = make_attend(dt, D, B, Hkv, G, T, 64, rng.integers(n // 8, n + 1, B * Hkv), seed=n)
    if w:
        check(x, q, dt, window=w, sinks=70)
    mask, depth, _ = Q.tree_mask(Q.random_trees(rng, B, T), window=w)
    check(x, q, dt, mask=mask, depth=depth, window=w, sinks=5)


@pytest.mark.parametrize("dt,D,G,T", [("bf16", 128, 4, 1), ("bf16", 64, 2, 10), ("f32", 64, 4, 3), ("bf16", 128, 4, 40)])
@pytest.mark.parametrize("seed", [0, 1])
def test_many_short_streams(dt, D, G, T, seed):
    rng = np.random.default_rng(seed)
    B, Hkv = 12, 5
    lens = rng.choice([0, 1, 2, 63, 64, 65, 127, 128, 129, 200, 600], B * Hkv).tolist()
    lens[int(rng.integers(B * Hkv))] = 1500
    x, q = make_attend(dt, D, B, Hkv, G, T, 64, lens, seed=seed)
    check(x, q, dt, window=100, sinks=4)
    mask, depth, _ = Q.tree_mask(Q.random_trees(rng, B, T))
    check(x, q, dt, mask=mask, depth=depth)


@pytest.mark.parametrize("dt,D,G,T,n,w", [("bf16", 128, 4, 33, 120000, 70000), ("bf16", 64, 8, 20, 150000, 0),
                                          ("bf16", 128, 5, 1, 60000, 50000), ("f32", 64, 2, 3, 40000, 30000),
                                          ("bf16", 128, 4, 500, 9000, 3000), ("bf16", 128, 4, 256, 40000, 0)])
def test_many_units_a_cta(dt, D, G, T, n, w):
    """Long streams: dozens of work units for every CTA, the model's product formed on the GPU in 64 bits."""
    kvc = kvc_()
    B, Hkv, page, k = 2, 1, 256, 300
    maxp = R.npg(n, page)
    pool, pages = kvc.Pool.empty(2 * maxp + 3, D, page, device=DEV), kvc.Pages.empty(1, B, Hkv, maxp, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    start = torch.zeros((1, B, Hkv), dtype=torch.int32, device=DEV)
    lens = torch.tensor([n, n - 777], dtype=torch.int32, device=DEV)
    kvc.kvc_page_extend(pool, pages, add=lens, start=start, status=status)
    g = torch.Generator(device=DEV).manual_seed(n)
    kk, vv = (torch.randn((B, n, Hkv, D), generator=g, device=DEV).to(DT[dt]) for _ in range(2))
    kvc.kvc_page_store(pool, pages, kk, vv, start, n=lens, status=status)
    q = (2 * torch.randn((B, T, Hkv * G, D), generator=g, device=DEV)).to(DT[dt])
    K = torch.zeros((1, B, Hkv, n, D), device=DEV)
    V = torch.zeros_like(K)
    kvc.kvc_page_read(pool, pages, K, V, status=status)
    parent = Q.random_trees(np.random.default_rng(n), B, T)
    tm, depth, _ = Q.tree_mask(parent, window=w)
    for mask in (None, tm) if w else (tm,):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
        kvc.kvc_page_attend_masked(pool, pages, q, out, window=w, sinks=k, lse=lse, status=status,
                                   mask=None if mask is None else up(mask), depth=None if mask is None else up(depth))
        assert int(status.item()) == 0
        for b in range(B):
            m = int(lens[b])
            for i in sorted({0, T // 2, T - 1}):
                seen = torch.from_numpy(Q.seen_tokens(m, T, i, w, k, None if mask is None else mask[b, i],
                                                      None if mask is None else depth[b])).to(DEV)
                ks, vs = K[0, b, 0, seen].double(), V[0, b, 0, seen].double()
                qq = q[b, i].double()
                s = qq @ ks.T / D ** 0.5
                z = torch.logsumexp(s, -1)
                p = torch.exp(s - z[:, None])
                ref = dict(out=p @ vs, lse=z, mass=p @ vs.abs(), vmax=vs.abs().amax(0) + 0 * qq,
                           logit=(qq.abs() @ ks.abs().T / D ** 0.5).amax(-1))
                ref = {name: v.cpu().numpy() for name, v in ref.items()}
                tol, ltol = R.tolerances(dt, len(seen), D, ref)
                assert (np.abs(out[b, i].double().cpu().numpy() - ref["out"]) <= tol).all()
                assert (np.abs(lse[b, i].double().cpu().numpy() - ref["lse"]) <= ltol).all()


# ---- pages that a window leaves behind, drafts that are kept -------------------------------------------------------
def slide(x, window, sinks=0):
    gone = torch.full(x.t.shape, 77, dtype=torch.int32, device=DEV)
    x.kvc.kvc_page_slide(x.pool, x.pages, window, sinks, gone=gone, status=x.status)
    np.testing.assert_array_equal(gone.cpu().numpy(), Q.slide(x.p, x.t, window, sinks))


def accept(x, path, n_path, n_q=None):
    dev = lambda v: None if v is None else up(np.asarray(v, np.int32))
    x.kvc.kvc_page_accept(x.pool, x.pages, dev(path), dev(n_path), n_q=dev(n_q), status=x.status)
    R.compact(x.p, x.t, Q.accept_lists(x.t, np.asarray(path), n_path, n_q))


@pytest.mark.parametrize("seed,D,page,L,B,Hkv,maxp,npages", [
    (0, 64, 16, 1, 1, 1, 8, 30), (1, 128, 16, 2, 3, 2, 10, 200), (2, 64, 32, 3, 2, 5, 40, 2000),
    (3, 128, 64, 4, 16, 8, 6, 4000),   # 512 streams: the wide forms
    (4, 64, 16, 1, 2, 2, 300, 1500), (5, 64, 16, 40, 4, 8, 40, 60000)])
def test_random_sequences_of_operators(seed, D, page, L, B, Hkv, maxp, npages):
    """Room, slides, accepted drafts, forks, evictions and rollback in any order: the whole state and every byte."""
    rng = np.random.default_rng(seed)
    x = Both(npages, D, page, L, B, Hkv, maxp, seed=seed)
    x.extend(rng.integers(0, maxp * page // 2, B).tolist())
    for step in range(30):
        op = rng.choice(["extend", "slide", "accept", "accept", "fork", "free", "compact"])
        Bn = x.t.shape[1]
        if op == "extend":
            x.extend(rng.integers(0, 2 * page, Bn).tolist())
        elif op == "slide":
            slide(x, int(rng.integers(1, maxp * page // 2 + 2)), int(rng.choice([0, 1, page, page + 1, 3 * page])))
        elif op == "accept":
            T = int(rng.choice([1, 5, 40]))
            n_q = rng.integers(-1, T + 2, Bn)
            path, n_path = np.full((Bn, T), -1, np.int32), np.zeros(Bn, np.int32)
            for b in range(Bn):
                n = Q.drafts(n_q, b, T)
                n_path[b] = rng.integers(0, n + 1)
                path[b, :n_path[b]] = np.sort(rng.choice(n, n_path[b], replace=False)) if n else []
            accept(x, path, n_path, n_q)
        elif op == "fork":
            x.fork(rng.integers(-1, Bn, B).tolist())
        elif op == "free":
            x.free(rng.integers(0, page, Bn).tolist())
        else:
            lists = {}
            for s in x.t.streams():
                n = int(x.t.len[s])
                lists[s] = np.sort(rng.choice(n, int(rng.integers(n // 2, n + 1)), replace=False))
            x.compact(lists, maxp * page)
        x.check(f"{step} {op}")


def test_slides_of_every_length():
    for page, window, sinks in ((16, 1, 0), (16, 16, 0), (16, 17, 1), (16, 40, 16), (16, 40, 17), (64, 100, 4), (16, 1 << 30, 0),
                                (16, (1 << 31) - 1, (1 << 31) - 1), (16, 1, 5000)):
        x = Both(600, 64, page, 1, 100, 1, 10 * 64 // page, seed=page)
        x.extend(list(range(100)))
        slide(x, window, sinks)
        x.check("slide")
        slide(x, window, sinks)
        x.check("nothing left")


def test_shared_pages_and_slides():
    """Pages between the sinks and the window that another sequence holds stay with it, whoever slides first."""
    x = Both(64, 64, 16, 2, 2, 2, 12, seed=3)
    x.extend([150, 40])
    x.fork([0, 0, 0, 1])
    x.free([0, 60, 0, 0])
    slide(x, 50, 4)
    x.check("shared")
    x.extend([1, 1, 40, 1])
    slide(x, 20, 0)
    x.check("again")


def test_accepted_drafts_on_shared_pages():
    """Drafts that two sequences share (a fork behind their storing): both take fresh pages, or the call does nothing
    when there are too few."""
    for spare in (12, 3):
        x = Both(10 + spare, 64, 16, 1, 1, 2, 6, seed=4)
        x.extend([70])
        x.fork([0, 0])
        path = np.array([[0, 2, 5, 29, -1] + [-1] * 25, [1, 2, 28] + [-1] * 27], np.int32)
        accept(x, path, [4, 3])
        x.check("shared drafts")


def test_bad_paths_and_pages():
    x = Both(60, 64, 16, 1, 6, 1, 6, seed=5)
    x.extend([40, 40, 40, 40, 3, 40])
    path = np.tile(np.arange(8, dtype=np.int32), (6, 1))
    path[0, 1] = 0          # not increasing
    path[1, 2] = 8          # past the drafts
    path[2, 0] = -1
    accept(x, path, [3, 3, 2, 9, 2, 3])  # the fourth too long, the fifth stream too short
    assert x.p.status == R.BAD_INDEX
    x.check("bad paths")
    accept(x, path[[5] * 6], [0, 1, 2, -1, 3, 3], [0, 1, 2, 3, 3, 2])
    x.check("bad numbers")
    x.status.zero_()
    # pages: one that a draft lies in, one between sinks and window, a length
    x.pages.table[0, 0, 0, 1] = 1 << 30
    x.pages.len[0, 1, 0] = 1 << 20
    x.pages.len[0, 2, 0] = -4
    before = x.pages.table[0, :3].clone(), x.pages.len[0, :3].clone()
    p = np.tile(np.array([1] + [-1] * 19, np.int32), (6, 1))
    x.kvc.kvc_page_accept(x.pool, x.pages, up(p), up(np.ones(6, np.int32)), status=x.status)
    assert int(x.status.item()) & R.BAD_PAGE
    assert torch.equal(before[0], x.pages.table[0, :3]) and torch.equal(before[1], x.pages.len[0, :3])
    x.status.zero_()
    gone = torch.zeros((1, 6, 1), dtype=torch.int32, device=DEV)
    n0 = int(x.pages.len[0, 0, 0])
    x.kvc.kvc_page_slide(x.pool, x.pages, 1, 0, gone=gone, status=x.status)
    assert int(x.status.item()) == R.BAD_PAGE
    assert gone[0, 0, 0] == n0 // 16 * 16 and int(x.pages.len[0, 0, 0]) == n0 % 16 and list(gone[0, 1:3, 0].tolist()) == [-1, -1]
    assert int(x.pages.table[0, 0, 0, 0]) == int(before[0][0, 0, n0 // 16]) and torch.equal(before[1][1:], x.pages.len[0, 1:3])


# ---- together --------------------------------------------------------------------------------------------------
def test_speculative_decoding_on_windowed_layers():
    """Prompt, then steps of a drafted tree: room, rows, mask, attention, the picks' path, accepted drafts and a slide; a
    fork in between. Cache and attention follow the model."""
    kvc = kvc_()
    L, B, Hkv, G, D, page, w, k = 2, 2, 2, 4, 64, 16, 45, 5
    x = Both(160, D, page, L, B, Hkv, 10, seed=9)
    rng, seed = np.random.default_rng(0), [100]

    def rows(T, heads):
        seed[0] += 1
        return rand_rows((x.t.shape[1], T, heads, D), "bf16", seed[0])

    def add(T, **seen):
        start = x.extend([T] * x.t.shape[1])
        for l in range(L):
            kk, vv = rows(T, Hkv), rows(T, Hkv)
            lay, one = x.pages.layer(l), R.RefPages(1, x.t.shape[1], Hkv, x.t.maxp)
            one.table, one.len = x.t.table[l:l + 1], x.t.len[l:l + 1]
            kvc.kvc_page_store(x.pool, lay, kk.to(DEV), vv.to(DEV), start[l:l + 1], status=x.status)
            R.store(x.p, one, kk.double().numpy(), vv.double().numpy(), start[l:l + 1].cpu().numpy())
            both = Both.__new__(Both)
            both.__dict__.update(x.__dict__)
            both.t, both.pages = one, lay
            check(both, rows(T, Hkv * G), "bf16", window=w, sinks=k, **seen)

    add(60)
    slide(x, w, k)
    x.check("prompt")
    for step in range(6):
        T, B = int(rng.integers(1, 40)), x.t.shape[1]
        parent = Q.random_trees(rng, B, T)
        draft, target = rng.integers(0, 3, (2, B, T)).astype(np.int32)
        mask, depth = torch.empty((B, T, (T + 31) // 32), dtype=torch.int32, device=DEV), torch.empty((B, T), dtype=torch.int32, device=DEV)
        kvc.kvc_tree_mask(up(parent), mask, depth, window=w, status=x.status)
        add(T, mask=mask.cpu().numpy(), depth=depth.cpu().numpy())
        path, n_path, nxt = (torch.empty(s, dtype=torch.int32, device=DEV) for s in ((B, T), (B,), (B,)))
        kvc.kvc_tree_verify(up(parent), up(draft), up(target), path, n_path, next=nxt, status=x.status)
        kvc.kvc_page_accept(x.pool, x.pages, path, n_path, status=x.status)
        wp, wn, wx, _ = Q.tree_verify(parent, draft, target)
        np.testing.assert_array_equal(nxt.cpu().numpy(), wx)
        R.compact(x.p, x.t, Q.accept_lists(x.t, wp, wn))
        x.check(f"accept {step}")
        slide(x, w, k)
        x.check(f"slide {step}")
        if step == 2:
            x.fork([1, 0, 1])
    add(1)
    x.check("end")


@pytest.mark.parametrize("L,B,Hkv,maxp,npages", [(1, 3, 2, 12, 120), (2, 24, 8, 48, 12000)])
def test_captured_and_replayed(L, B, Hkv, maxp, npages):
    """A speculative step captured once; each replay with new trees equals the model's, eager calls between the replays
    use the same workspaces."""
    kvc, rng = kvc_(), np.random.default_rng(B)
    x, T, G, D, w, k = Both(npages, 64, 16, L, B, Hkv, maxp, seed=B), 9, 2, 64, 70, 3
    ws = torch.empty(kvc.kvc_page_workspace_size(x.pool, x.pages), dtype=torch.uint8, device=DEV)
    lay = x.pages.layer(0)
    aws = torch.empty(kvc.kvc_page_attend_masked_workspace_size(x.pool, lay, Hkv * G, T, w, k), dtype=torch.uint8, device=DEV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    parent, draft, target, n_q = i32(B, T), i32(B, T), i32(B, T), i32(B)
    mask, depth, path, n_path, nxt, gone = i32(B, T, 1), i32(B, T), i32(B, T), i32(B), i32(B), i32(L, B, Hkv)
    q = rand_rows((B, T, Hkv * G, D), "bf16", 1)
    qd, out, lse = q.to(DEV), torch.zeros((B, T, Hkv * G, D), dtype=torch.bfloat16, device=DEV), torch.zeros((B, T, Hkv * G), device=DEV)

    def step():
        kvc.kvc_page_extend(x.pool, x.pages, add=n_q, status=x.status, workspace=ws)
        kvc.kvc_tree_mask(parent, mask, depth, n_q=n_q, window=w, status=x.status)
        kvc.kvc_page_attend_masked(x.pool, lay, qd, out, window=w, sinks=k, mask=mask, depth=depth, lse=lse, n_q=n_q,
                                   status=x.status, workspace=aws)
        kvc.kvc_tree_verify(parent, draft, target, path, n_path, next=nxt, n_q=n_q, status=x.status)
        kvc.kvc_page_accept(x.pool, x.pages, path, n_path, n_q=n_q, status=x.status, workspace=ws)
        kvc.kvc_page_slide(x.pool, x.pages, w, k, gone=gone, status=x.status, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # no drafts, no tokens
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.check("captured")
    x.extend(rng.integers(0, 100, B).tolist())
    for i in range(6):
        nq = rng.integers(0, T + 1, B)
        pa = Q.random_trees(rng, B, T, nq)
        dr, ta = rng.integers(0, 2, (2, B, T)).astype(np.int32)
        for t, v in ((parent, pa), (draft, dr), (target, ta), (n_q, nq)):
            t.copy_(up(np.ascontiguousarray(v, np.int32)))
        tab, ln = x.t.table.copy(), None
        graph.replay()
        R.extend(x.p, x.t, nq.tolist())
        m, d, _ = Q.tree_mask(pa, nq, w)
        np.testing.assert_array_equal(mask.cpu().numpy(), m)
        one = R.RefPages(1, B, Hkv, maxp)
        one.table, one.len = x.t.table[:1].copy(), x.t.len[:1].copy()
        ref = Q.attend(x.p, one, q.double().numpy(), D ** -0.5, nq, w, k, m, d)
        tol, ltol = R.tolerances("bf16", int(one.len.max()), D, ref)
        for b in range(B):
            assert (np.abs(out[b, :nq[b]].double().cpu().numpy() - ref["out"][b, :nq[b]]) <= tol[b, :nq[b]]).all()
        wp, wn, wx, _ = Q.tree_verify(pa, dr, ta, nq)
        np.testing.assert_array_equal(path.cpu().numpy(), wp)
        R.compact(x.p, x.t, Q.accept_lists(x.t, wp, wn, nq))
        np.testing.assert_array_equal(gone.cpu().numpy(), Q.slide(x.p, x.t, w, k))
        x.check(f"replay {i}")
        o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
        kvc.kvc_page_attend_masked(x.pool, lay, qd, o2, window=w, sinks=k, lse=l2, status=x.status, workspace=aws)
        kvc.kvc_page_slide(x.pool, x.pages, w // 2, k, status=x.status, workspace=ws)
        Q.slide(x.p, x.t, w // 2, k)
        x.check(f"between {i}")


def test_streams_with_their_own_workspaces():
    kvc = kvc_()
    made = [make_attend("bf16", 128, 4, 4, 4, 1, 64, [900] * 16, seed=31), make_attend("bf16", 128, 2, 2, 8, 3, 16, [333, 500, 7, 64], seed=32),
            make_attend("bf16", 128, 2, 2, 2, 40, 64, [900, 1200, 70, 400], seed=33),
            make_attend("bf16", 128, 1, 2, 4, 100, 64, [900, 1200], seed=34)]
    qs = [q.to(DEV) for _, q in made]
    ref, got = ([torch.empty_like(q) for q in qs] for _ in range(2))
    for (x, _), q, o in zip(made, qs, ref):
        kvc.kvc_page_attend_masked(x.pool, x.pages, q, o, window=300, sinks=4)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in qs]
    ws = [torch.empty(kvc.kvc_page_attend_masked_workspace_size(x.pool, x.pages, q.shape[2], q.shape[1], 300, 4),
                      dtype=torch.uint8, device=DEV) for (x, _), q in zip(made, qs)]
    for _ in range(20):
        for (x, _), q, o, s, w in zip(made, qs, got, st, ws):
            kvc.kvc_page_attend_masked(x.pool, x.pages, q, o, window=300, sinks=4, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(r, o) for r, o in zip(ref, got))


def test_binding_refuses_wrong_tensors():
    kvc = kvc_()
    pool, pages = kvc.Pool.empty(8, 64, 16, device=DEV), kvc.Pages.empty(2, 2, 2, 4, device=DEV)
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device=DEV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    with pytest.raises(kvc.KvcError) as e:
        kvc.kvc_page_attend_masked(pool, pages, q, torch.empty_like(q), window=3)  # two layers at once
    assert e.value.code == -1
    lay = pages.layer(1)
    for kw in (dict(mask=i32(2, 3)), dict(mask=i32(2, 3, 2)), dict(mask=i32(2, 3, 1).long()), dict(mask=i32(2, 3, 1).cpu()),
               dict(mask=i32(2, 3, 1), depth=i32(2, 4))):
        with pytest.raises(ValueError):
            kvc.kvc_page_attend_masked(pool, lay, q, torch.empty_like(q), **kw)
    for kw in (dict(window=-1), dict(window=3, sinks=-1), dict(depth=i32(2, 3))):
        with pytest.raises(kvc.KvcError):
            kvc.kvc_page_attend_masked(pool, lay, q, torch.empty_like(q), **kw)
    with pytest.raises(kvc.KvcError):
        kvc.kvc_page_slide(pool, pages, 0)
    with pytest.raises(ValueError):
        kvc.kvc_page_slide(pool, pages, 4, gone=i32(2, 2))
    with pytest.raises(ValueError):
        kvc.kvc_page_accept(pool, pages, i32(3, 3), i32(2))
    with pytest.raises(ValueError):
        kvc.kvc_page_accept(pool, pages, i32(2, 3), i32(3))
    for bad in (i32(2, 3).cpu(), i32(2, 3).long(), i32(6), i32(3, 2).T):
        with pytest.raises(ValueError):
            kvc.kvc_tree_mask(bad, i32(2, 3, 1))
    with pytest.raises(ValueError):
        kvc.kvc_tree_mask(i32(2, 3), i32(2, 3))
    with pytest.raises(ValueError):
        kvc.kvc_tree_verify(i32(2, 3), i32(2, 3), i32(2, 4), i32(2, 3), i32(2))


# ---- larger caches, made and checked on the GPU ---------------------------------------------------------------------
class Made:
    """A cache of given lengths stored on the GPU, with its rows read back and the model's sums in 64 bits."""

    def __init__(self, dt, D, B, Hkv, G, T, page, lens, seed, maxp=None):
        kvc = kvc_()
        self.kvc, self.dt, self.lens = kvc, dt, np.asarray(lens, np.int64).reshape(B, Hkv)
        n = int(self.lens.max())
        maxp = maxp or max(1, R.npg(n, page))
        self.pool, self.pages = kvc.Pool.empty(B * Hkv * R.npg(n, page) + 3, D, page, device=DEV), kvc.Pages.empty(1, B, Hkv, maxp, device=DEV)
        g = torch.Generator(device=DEV).manual_seed(seed)
        start = torch.zeros((1, B, Hkv), dtype=torch.int32, device=DEV)
        kvc.kvc_page_extend(self.pool, self.pages, add_all=n)
        kvc.kvc_page_store(self.pool, self.pages, *(torch.randn((B, n, Hkv, D), generator=g, device=DEV).to(DT[dt]) for _ in range(2)),
                           start)
        self.K, self.V = (torch.zeros((1, B, Hkv, n, D), device=DEV) for _ in range(2))
        kvc.kvc_page_read(self.pool, self.pages, self.K, self.V)
        self.pages.len.copy_(up(self.lens.astype(np.int32)[None]))  # the streams' ends differ; what lies behind is not theirs
        self.q = (2 * torch.randn((B, T, Hkv * G, D), generator=g, device=DEV)).to(DT[dt])

    def check(self, rows=None, n_q=None, window=0, sinks=0, mask=None, depth=None, ws=None):
        B, T, Hq, D = self.q.shape
        G = Hq // self.lens.shape[1]
        out, lse = torch.full_like(self.q, -55.0), torch.full(self.q.shape[:3], -55.0, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        dev = lambda v: None if v is None else up(np.asarray(v, np.int32))
        self.kvc.kvc_page_attend_masked(self.pool, self.pages, self.q, out, window=window, sinks=sinks, mask=dev(mask),
                                        depth=dev(depth), lse=lse, n_q=dev(n_q), status=status, workspace=ws)
        assert int(status.item()) == 0
        for b in range(B):
            nq = Q.drafts(n_q, b, T)
            assert (out[b, nq:] == -55.0).all() and (lse[b, nq:] == -55.0).all()
            for h in range(self.lens.shape[1]):
                m, hs = int(self.lens[b, h]), slice(h * G, (h + 1) * G)
                for i in (range(nq) if rows is None else sorted({0, nq // 2, nq - 1} & set(range(nq)))):
                    seen = torch.from_numpy(Q.seen_tokens(m, nq, i, window, sinks, None if mask is None else mask[b, i],
                                                          None if depth is None else depth[b])).to(DEV)
                    if len(seen) == 0:
                        assert (out[b, i, hs] == 0).all() and torch.isneginf(lse[b, i, hs]).all()
                        continue
                    ks, vs, qq = self.K[0, b, h, seen].double(), self.V[0, b, h, seen].double(), self.q[b, i, hs].double()
                    s = qq @ ks.T / D ** 0.5
                    z = torch.logsumexp(s, -1)
                    p = torch.exp(s - z[:, None])
                    ref = dict(out=p @ vs, lse=z, mass=p @ vs.abs(), vmax=vs.abs().amax(0) + 0 * qq,
                               logit=(qq.abs() @ ks.abs().T / D ** 0.5).amax(-1))
                    ref = {name: v.cpu().numpy() for name, v in ref.items()}
                    tol, ltol = R.tolerances(self.dt, len(seen), D, ref)
                    err = np.abs(out[b, i, hs].double().cpu().numpy() - ref["out"])
                    assert (err <= tol).all(), (b, h, i, float((err / tol).max()))
                    assert (np.abs(lse[b, i, hs].double().cpu().numpy() - ref["lse"]) <= ltol).all(), (b, h, i)
        return out, lse


@pytest.mark.parametrize("dt,D,B,Hkv,G,T,page,n,w", [
    ("bf16", 128, 1, 2, 4, 1, 64, 3000, 1200),   # eight CTAs a cluster
    ("bf16", 64, 2, 3, 3, 3, 16, 2500, 900),     # two row tiles
    ("f32", 128, 2, 2, 2, 2, 32, 2000, 700),
    ("f32", 64, 1, 4, 8, 2, 256, 1500, 1100),
    ("bf16", 128, 16, 8, 4, 1, 64, 1500, 1000),  # four
    ("bf16", 64, 32, 8, 2, 1, 64, 1000, 700),    # two
    ("f32", 64, 16, 8, 1, 1, 64, 1300, 800),
    ("bf16", 64, 10, 8, 2, 1, 32, 1000, 900),    # seven, five and three
    ("bf16", 128, 14, 8, 1, 1, 64, 800, 600),
    ("bf16", 64, 20, 8, 1, 1, 64, 800, 650),
    ("bf16", 128, 1, 3, 4, 1, 16, 300, 260)])    # few streams of few tokens
def test_a_cluster_of_ctas_a_stream(dt, D, B, Hkv, G, T, page, n, w):
    """Windows between what one CTA takes and what is split; streams shorter than the window, of one token and of none."""
    rng = np.random.default_rng(n)
    lens = rng.integers(1, n + 1, B * Hkv)
    lens[:2] = n, 0
    lens[-1] = rng.integers(1, 3)
    x = Made(dt, D, B, Hkv, G, T, page, lens, n)
    x.check(window=w, sinks=4)
    x.check(window=w, sinks=0, n_q=rng.integers(0, T + 1, B) if T > 1 else None)
    parent = Q.random_trees(rng, B, T)
    mask, depth, _ = Q.tree_mask(parent, window=w)
    x.check(window=w, sinks=70, mask=mask, depth=depth)


@pytest.mark.parametrize("D,G,T", [(128, 1, 17), (128, 4, 32), (64, 3, 43), (128, 8, 32), (64, 1, 257), (128, 5, 52),
                                   (128, 200, 1), (64, 300, 2), (128, 130, 3)])
def test_rows_around_a_block(D, G, T):
    """17, 128, 129, 256, 257 and 260 rows a KV head; streams of one unit, of a few, of less than the rows. Many query heads
    a KV head: a token's rows lie in several blocks."""
    rng = np.random.default_rng(T)
    x = Made("bf16", D, 2, 3, G, T, 64, [1000, 3, 129, 128, 700, T + 1], T)
    parent = Q.random_trees(rng, 2, T)
    mask, depth, _ = Q.tree_mask(parent)
    x.check(mask=mask)
    x.check(mask=mask, depth=depth, window=100, sinks=130, n_q=[T - 1, T // 2])
    x.check(window=60, sinks=3)
    x.check(window=513)


@pytest.mark.parametrize("D,T", [(128, 120), (64, 70), (128, 45)])
def test_uneven_query_rows_in_several_parts_a_cta(D, T):
    """Blocks of 256 and of 128 rows, more streams than CTAs have whole: rows of very different magnitudes, of none, strided,
    scaled by less than zero; and a row that is no number, which is no other row's matter."""
    rng = np.random.default_rng(T)
    B, Hkv, G = 12, 8, 2
    lens = rng.integers(T, 400, B * Hkv)
    lens[:3] = T, 1, 0
    x, q0 = make_attend("bf16", D, B, Hkv, G, T, 64, lens.tolist(), seed=T)
    up2 = 2.0 ** rng.integers(-30, 3, (B, T, G * Hkv, 1)) * 2.0 ** rng.integers(-12, 1, D)
    q0 = (q0.double() * torch.from_numpy(up2)).to(q0.dtype)  # powers of two: exact
    q0[:, 3] = 0
    q0[1, :, 1] = 0
    wide = torch.full((B, T, G * Hkv + 3, D), 7.0, dtype=torch.bfloat16, device=DEV)
    wide[:, :, 1:-2] = q0.to(DEV)
    qd = wide[:, :, 1:-2]
    mask, depth, _ = Q.tree_mask(Q.random_trees(rng, B, T))
    check(x, q0, "bf16", scale=0.5, mask=mask, depth=depth, q_dev=qd)
    out, lse = check(x, q0, "bf16", scale=-0.5, window=150, sinks=5, q_dev=qd)
    b, t, h = 5, T - 1, 6
    qd[b, t, h, 3] = float("nan")
    got, gl = torch.full_like(out, -55.0), torch.full_like(lse, -55.0)
    kvc_().kvc_page_attend_masked(x.pool, x.pages, qd, got, window=150, sinks=5, scale=-0.5, lse=gl, status=x.status)
    assert got[b, t, h].isnan().all() and gl[b, t, h].isnan()
    got[b, t, h], gl[b, t, h] = out[b, t, h], lse[b, t, h]
    assert torch.equal(got, out) and torch.equal(gl, lse) and int(x.status.item()) == 0


@pytest.mark.parametrize("dt,D,T,w", [("bf16", 128, 1, 100), ("bf16", 128, 1, 1500), ("bf16", 64, 3, 40000), ("f32", 128, 2, 20000),
                                      ("bf16", 128, 24, 30000), ("bf16", 64, 24, 30000), ("bf16", 128, 80, 30000)])
def test_a_wait_that_runs_out(dt, D, T, w):
    """As test_gpu_page_faults does it, on every kernel: the first CTA waits for an arrival that nothing makes. The call ends
    and says so, streams without a share of that CTA keep their results, the next call on the workspace is right."""
    import time
    kvc = kvc_()
    B, Hkv, G, n = 2, 3, 4, 40960
    x = Made(dt, D, B, Hkv, G, T, 64, [n] * (B * Hkv), T)
    ws = torch.empty(kvc.kvc_page_attend_masked_workspace_size(x.pool, x.pages, Hkv * G, T, w, 4), dtype=torch.uint8, device=DEV)
    res = []
    for mode, fill in ((0, False), (2, False), (2, True), (0, True)):
        if fill:
            ws.fill_(0xff)
        out, lse = torch.full_like(x.q, 9.0), torch.full(x.q.shape[:3], 9.0, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        kvc.kvc_debug_fault(mode)
        try:
            t0 = time.time()
            kvc.kvc_page_attend_masked(x.pool, x.pages, x.q, out, window=w, sinks=4, lse=lse, status=status, workspace=ws)
            torch.cuda.synchronize()
            took = time.time() - t0
        finally:
            kvc.kvc_debug_fault(0)
        assert int(status.item()) == (kvc.KVC_STATUS_TIMEOUT if mode else 0)
        assert took < 20.0
        res.append((out, lse))
    (o0, l0), *bad, (o3, l3) = res
    assert torch.equal(o0, o3) and torch.equal(l0, l3)
    for o, l in bad:
        assert torch.equal(o0[1:], o[1:]) and torch.equal(l0[1:], l[1:])
        assert torch.equal(o0[0, :, G:], o[0, :, G:]) and torch.equal(l0[0, :, G:], l[0, :, G:])  # the other heads
        assert not torch.equal(l0[0, :, :G], l[0, :, :G])
    assert torch.equal(bad[0][0], bad[1][0]) and torch.equal(bad[0][1], bad[1][1])  # nothing stale came in
    x.check(rows=3, window=w, sinks=4, ws=ws)


def test_offsets_past_32_bits():
    """A stream whose pages lie in a pool of 5 GB: attention under a window and a mask, a slide and accepted drafts there."""
    kvc = kvc_()
    D, page, n, T = 128, 256, 700, 40
    npages = (5 << 30) // kvc.kvc_page_bytes(D, page)
    pool = kvc.Pool.empty(npages, D, page, device=DEV)
    pool.free_list.copy_(torch.arange(npages, dtype=torch.int32, device=DEV))  # the last pages first
    pages = kvc.Pages.empty(1, 1, 2, 6, device=DEV)
    start = torch.zeros((1, 1, 2), dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kvc.kvc_page_extend(pool, pages, add_all=n, start=start, status=status)
    assert int(pages.table[0, 0, 0, 0]) == npages - 1
    k, v = rand_rows((1, n, 2, D), "bf16", 1).to(DEV), rand_rows((1, n, 2, D), "bf16", 2).to(DEV)
    kvc.kvc_page_store(pool, pages, k, v, start, status=status)
    small, same = kvc.Pool.empty(20, D, page, device=DEV), kvc.Pages.empty(1, 1, 2, 6, device=DEV)
    kvc.kvc_page_extend(small, same, add_all=n)
    kvc.kvc_page_store(small, same, k, v, start)
    mask, depth, _ = Q.tree_mask(Q.random_trees(np.random.default_rng(3), 1, T))
    path = np.full((1, T), -1, np.int32)
    path[0, :5] = 1, 3, 8, 9, 39
    for rows in (1, 4, T):
        q = rand_rows((1, rows, 8, D), "bf16", rows).to(DEV)
        for kw in (dict(window=300, sinks=4),) + ((dict(mask=up(mask), depth=up(depth)),) if rows == T else ()):
            a, b = torch.empty_like(q), torch.empty_like(q)
            kvc.kvc_page_attend_masked(pool, pages, q, a, status=status, **kw)
            kvc.kvc_page_attend_masked(small, same, q, b, **kw)
            assert torch.equal(a, b)
    for x, t in ((pool, pages), (small, same)):
        kvc.kvc_page_accept(x, t, up(path), up(np.array([5], np.int32)), status=status)
        kvc.kvc_page_slide(x, t, 200, 3, status=status)
    assert torch.equal(pages.len, same.len) and int(status.item()) == 0
    m = int(same.len[0, 0, 0])
    got = [torch.zeros((1, 1, 2, m, D), device=DEV) for _ in range(4)]
    kvc.kvc_page_read(pool, pages, *got[:2])
    kvc.kvc_page_read(small, same, *got[2:])
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])


def test_prompt_in_chunks_on_a_windowed_layer():
    """A prompt of 1500 tokens in chunks of 512, slid in between, against the dense rows: every query's window crosses the
    chunks."""
    kvc = kvc_()
    D, Hkv, G, N, w, k, page = 128, 2, 4, 1500, 400, 5, 64
    pool, pages = kvc.Pool.empty(40, D, page, device=DEV), kvc.Pages.empty(1, 1, Hkv, 20, device=DEV)
    kk, vv = rand_rows((1, N, Hkv, D), "bf16", 1).to(DEV), rand_rows((1, N, Hkv, D), "bf16", 2).to(DEV)
    q = rand_rows((1, N, Hkv * G, D), "bf16", 3).to(DEV)
    big, all_ = kvc.Pool.empty(60, D, page, device=DEV), kvc.Pages.empty(1, 1, Hkv, 30, device=DEV)
    start, zero = torch.zeros((1, 1, Hkv), dtype=torch.int32, device=DEV), torch.zeros((1, 1, Hkv), dtype=torch.int32, device=DEV)
    kvc.kvc_page_extend(big, all_, add_all=N)
    kvc.kvc_page_store(big, all_, kk, vv, zero)
    K, V = (torch.zeros((1, 1, Hkv, N, D), device=DEV) for _ in range(2))
    kvc.kvc_page_read(big, all_, K, V)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for a in range(0, N, 512):
        T = min(512, N - a)
        kvc.kvc_page_extend(pool, pages, add_all=T, start=start, status=status)
        kvc.kvc_page_store(pool, pages, kk[:, a:a + T], vv[:, a:a + T], start, status=status)
        out, lse = torch.empty((1, T, Hkv * G, D), dtype=torch.bfloat16, device=DEV), torch.empty((1, T, Hkv * G), device=DEV)
        kvc.kvc_page_attend_masked(pool, pages, q[:, a:a + T], out, window=w, sinks=k, lse=lse, status=status)
        kvc.kvc_page_slide(pool, pages, w, k, status=status)
        for i in range(0, T, 37):
            j = a + i
            seen = torch.tensor([t for t in range(j + 1) if t < k or t > j - w], device=DEV)
            for h in range(Hkv):
                ks, vs, qq = K[0, 0, h, seen].double(), V[0, 0, h, seen].double(), q[0, j, h * G:(h + 1) * G].double()
                s = qq @ ks.T / D ** 0.5
                z = torch.logsumexp(s, -1)
                p = torch.exp(s - z[:, None])
                ref = dict(out=p @ vs, lse=z, mass=p @ vs.abs(), vmax=vs.abs().amax(0) + 0 * qq,
                           logit=(qq.abs() @ ks.abs().T / D ** 0.5).amax(-1))
                ref = {name: v.cpu().numpy() for name, v in ref.items()}
                tol, ltol = R.tolerances("bf16", len(seen), D, ref)
                assert (np.abs(out[0, i, h * G:(h + 1) * G].double().cpu().numpy() - ref["out"]) <= tol).all()
                assert (np.abs(lse[0, i, h * G:(h + 1) * G].double().cpu().numpy() - ref["lse"]) <= ltol).all()
    assert int(status.item()) == 0 and int(pages.len[0, 0, 0]) < 600
