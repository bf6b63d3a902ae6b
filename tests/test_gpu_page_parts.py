"""Serving batches of short streams: many of them for every CTA of the tcgen05 kernels, whose roles are then parts apart.
Against the definition in 64 bits, formed for whole batches on the GPU, within page_util.tolerances."""
import numpy as np
import pytest
import torch

import page_util as R
import tree_util as Q
from test_gpu_page import DEV, up
from test_gpu_page_masked import Made, kvc_

pytestmark = pytest.mark.gpu


def seen_by_all(lens, nq, T, N, window, sinks, mask=None, depth=None):
    """[B, Hkv, T, N]: query i of sequence b sees token j of a stream; lens [B, Hkv], nq [B], mask and depth numpy."""
    lens, nq = torch.from_numpy(lens).to(DEV), torch.from_numpy(nq).to(DEV)
    B = lens.shape[0]
    j, i = torch.arange(N, device=DEV), torch.arange(T, device=DEV)
    base = (lens - nq[:, None])[..., None, None]
    d = i.expand(B, T) if depth is None else torch.minimum(up(depth).long().clamp(min=0), nq[:, None] - 1)
    pos = base + d[:, None, :, None]
    near = (j < sinks) | (j > pos - window) if window else torch.ones((1, 1, 1, N), dtype=torch.bool, device=DEV)
    u = (j - base).expand(B, lens.shape[1], 1, N)
    if mask is None:
        own = near & (u <= i[:, None])
    else:
        words = torch.from_numpy(np.ascontiguousarray(mask).view(np.uint32).astype(np.int64)).to(DEV)
        bits = (words[..., None] >> torch.arange(32, device=DEV) & 1).flatten(2)[:, :, :T] > 0  # [B, T, T]
        own = torch.gather(bits[:, None].expand(B, lens.shape[1], T, T), 3, u.clamp(0, T - 1).expand(-1, -1, T, -1))
    there = (j < lens[..., None, None]) & (i[:, None] < nq[:, None, None, None])
    return there & torch.where(u < 0, near, own)


def check(x, window=0, sinks=0, mask=None, depth=None, n_q=None, causal=False):
    """One call on a Made cache. Returns out, lse."""
    kvc = kvc_()
    q = x.q
    B, T, Hq, D = q.shape
    Hkv = x.lens.shape[1]
    out, lse = torch.full_like(q, -55.0), torch.full(q.shape[:3], -55.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dev = lambda v: None if v is None else up(np.asarray(v, np.int32))
    if causal:
        kvc.kvc_page_attend(x.pool, x.pages, q, out, lse=lse, n_q=dev(n_q), status=status)
    else:
        kvc.kvc_page_attend_masked(x.pool, x.pages, q, out, window=window, sinks=sinks, mask=dev(mask), depth=dev(depth), lse=lse,
                                   n_q=dev(n_q), status=status)
    assert int(status.item()) == 0
    nq = np.array([Q.drafts(n_q, b, T) for b in range(B)])
    N = x.K.shape[3]
    seen = seen_by_all(x.lens, nq, T, N, window, sinks, mask, depth)
    r = np.random.default_rng(T)
    for _ in range(20):  # the batch's rule against the model's, one query at a time
        b, h = int(r.integers(B)), int(r.integers(Hkv))
        if nq[b]:
            i = int(r.integers(nq[b]))
            one = Q.seen_tokens(int(x.lens[b, h]), int(nq[b]), i, window, sinks, None if mask is None else mask[b, i],
                                None if depth is None else depth[b])
            np.testing.assert_array_equal(torch.nonzero(seen[b, h, i]).view(-1).cpu().numpy(), one)
    behind = torch.arange(T, device=DEV) >= torch.from_numpy(nq).to(DEV)[:, None]
    assert (out[behind] == -55.0).all() and (lse[behind] == -55.0).all(), "rows behind the last query"
    for b0 in range(0, B, 16):
        s = slice(b0, min(B, b0 + 16))
        qq = q[s].double().unflatten(2, (Hkv, -1)).transpose(1, 2)  # [b, Hkv, T, G, D]
        k, v, see = x.K[0, s].double(), x.V[0, s].double(), seen[s][:, :, :, None]
        far = lambda z, other: torch.where(see, z, other)
        z = far(torch.einsum("bhtgd,bhnd->bhtgn", qq, k) / D ** 0.5, -torch.inf)
        lz = torch.logsumexp(z, -1)
        p = torch.exp(z - torch.where(torch.isinf(lz), 0.0, lz)[..., None])
        live = torch.arange(N, device=DEV) < torch.from_numpy(x.lens[s]).to(DEV)[..., None]
        ref = dict(out=torch.einsum("bhtgn,bhnd->bhtgd", p, v), lse=lz, mass=torch.einsum("bhtgn,bhnd->bhtgd", p, v.abs()),
                   vmax=(v.abs() * live[..., None]).amax(2)[:, :, None, None] + 0 * qq,
                   logit=far(torch.einsum("bhtgd,bhnd->bhtgn", qq.abs(), k.abs()) / D ** 0.5, 0.0).amax(-1))
        ref = {name: y.transpose(1, 2).flatten(2, 3).cpu().numpy() for name, y in ref.items()}  # [b, T, Hq, .]
        tol, ltol = R.tolerances(x.dt, int(x.lens.max()), D, ref)
        there = ~behind[s].cpu().numpy()[..., None]
        got, gl = out[s].double().cpu().numpy(), lse[s].double().cpu().numpy()
        err = np.where(there[..., None], np.abs(got - ref["out"]), 0.0)
        assert (err <= tol).all(), (b0, "out", float((err / tol).max()))
        empty = np.isneginf(ref["lse"]) & there
        assert (np.isneginf(gl) == empty).all() and (got[empty] == 0).all()
        le = np.abs(np.where(there & ~empty, gl, 0.0) - np.where(there & ~empty, ref["lse"], 0.0))
        assert (le <= ltol).all(), (b0, "lse", float((le / ltol).max()))
    return out, lse


def one_exponent(q):
    """The rows with their largest magnitude in [4, 8): they are all brought to fp16 by the same power of two."""
    q.clamp_(-3.75, 3.75)
    q[..., 5] = torch.where(q[..., 5] < 0, -4.0, 4.0)


@pytest.mark.parametrize("D,G,T,B,n", [(128, 4, 5, 75, 128), (64, 4, 32, 188, 128), (128, 1, 17, 188, 100), (64, 8, 3, 75, 60)])
def test_four_and_ten_streams_of_one_unit_a_cta(D, G, T, B, n):
    """600 and 1504 streams of at most 128 tokens, a work unit each: a CTA's roles are several streams apart."""
    rng = np.random.default_rng(B + T)
    lens = rng.integers(1, n + 1, B * 8)
    lens[::50] = n
    lens[7::40] = 0
    x = Made("bf16", D, B, 8, G, T, 16, lens, B + T)
    one_exponent(x.q)
    mask, depth, _ = Q.tree_mask(Q.random_trees(rng, B, T))
    a = check(x, mask=mask, depth=depth)
    for _ in range(3):  # the same again, bit for bit
        b = check(x, mask=mask, depth=depth)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(x, window=40, sinks=3)
    check(x, window=60, sinks=0, mask=mask, depth=depth)
    check(x, causal=True)


def uneven(q, rng):
    """Rows times powers of two that differ from sequence to sequence, token to token and head to head (exact): each has
    another factor."""
    B, T, Hq, _ = q.shape
    two = 2.0 ** rng.integers(-7, 2, (B, T, Hq, 1)) * 2.0 ** rng.integers(-4, 2, (B, 1, 1, 1))
    q.copy_((q.double() * torch.from_numpy(two).to(DEV)).to(q.dtype))


@pytest.mark.parametrize("D,G,T,B,n,w", [
    (128, 4, 5, 75, 128, 40), (128, 4, 5, 188, 128, 60), (64, 4, 32, 75, 128, 100), (64, 2, 60, 188, 128, 30), (128, 3, 6, 188, 128, 7),
    (128, 4, 65, 25, 128, 100), (64, 1, 257, 66, 128, 60), (128, 6, 64, 25, 128, 128),  # three blocks a stream
    (128, 4, 9, 100, 256, 50), (64, 4, 65, 30, 256, 200), (128, 8, 16, 130, 300, 150), (64, 5, 7, 90, 520, 260)])  # one unit to five
def test_uneven_rows_of_many_short_streams(D, G, T, B, n, w):
    """Streams of one unit and of a few, 600 to 1584 row blocks: four to ten a CTA. Every row has its own factor, sequences
    have all, some or none of their queries, streams hold more tokens than the window or fewer than the queries, or none."""
    rng = np.random.default_rng(B * T)
    lens = rng.integers(1, n + 1, B * 8)
    lens[::5] = n
    lens[3::40] = 0
    lens[5::30] = rng.integers(1, 5)
    x = Made("bf16", D, B, 8, G, T, 64, lens, B + T)
    uneven(x.q, rng)
    n_q = rng.integers(0, T + 1, B)
    n_q[::3] = T
    mask, depth, _ = Q.tree_mask(Q.random_trees(rng, B, T))
    check(x, mask=mask, depth=depth)
    check(x, mask=mask, depth=depth, n_q=n_q)
    check(x, window=w, sinks=5, n_q=n_q)
    check(x, window=w, sinks=0, mask=mask, depth=depth, n_q=n_q)
    check(x, causal=True, n_q=n_q)


@pytest.mark.parametrize("D,G,T,B,n,w", [(128, 4, 5, 100, 1500, 40), (64, 4, 32, 90, 1100, 30), (128, 4, 65, 30, 1200, 60), (128, 2, 100, 80, 900, 20)])
def test_windows_of_a_few_tokens_over_longer_streams(D, G, T, B, n, w):
    """A row block sees a unit or two of streams that are longer, blocks of 256 rows among them."""
    rng = np.random.default_rng(B + T)
    x = Made("bf16", D, B, 8, G, T, 64, rng.integers(1, n + 1, B * 8), B * T)
    uneven(x.q, rng)
    mask, depth, _ = Q.tree_mask(Q.random_trees(rng, B, T), window=w)
    check(x, window=w, sinks=3)
    check(x, window=w, sinks=0, mask=mask, depth=depth, n_q=rng.integers(0, T + 1, B))


def test_captured_and_replayed_with_new_lengths():
    """768 streams of other lengths and queries at each replay, an eager call on the same workspace between."""
    kvc, rng = kvc_(), np.random.default_rng(1)
    B, T, G, D, n = 96, 6, 4, 128, 256
    x = Made("bf16", D, B, 8, G, T, 64, [n] * (B * 8), 1)
    mask, depth, _ = Q.tree_mask(Q.random_trees(rng, B, T))
    first, q, m, d = x.q, x.q.clone(), up(mask), up(depth)
    out, lse, status = torch.zeros_like(q), torch.zeros(q.shape[:3], device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(kvc.kvc_page_attend_masked_workspace_size(x.pool, x.pages, 8 * G, T), dtype=torch.uint8, device=DEV)
    call = lambda: kvc.kvc_page_attend_masked(x.pool, x.pages, q, out, mask=m, depth=d, lse=lse, status=status, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(5):
        x.lens = rng.integers(0, n + 1, (B, 8))
        x.pages.len.copy_(up(x.lens.astype(np.int32)[None]))
        q.copy_(first)
        uneven(q, rng)
        x.q = q.clone()
        graph.replay()
        torch.cuda.synchronize()
        o, l = check(x, mask=mask, depth=depth)
        assert torch.equal(o, out) and torch.equal(l, lse) and int(status.item()) == 0
        kvc.kvc_page_attend_masked(x.pool, x.pages, q, torch.empty_like(q), window=50, sinks=2, status=status, workspace=ws)


@pytest.mark.parametrize("D,G,T,B,n", [(128, 4, 5, 75, 128), (64, 2, 60, 75, 250), (128, 4, 50, 75, 250)])
def test_a_wait_that_runs_out_among_many_streams(D, G, T, B, n):
    """The first CTA, with several streams of a unit or two, waits for an arrival that nothing makes: the call ends and says so, the
    other CTAs' streams keep their results, nothing of a workspace's former contents comes in, the next call is right."""
    kvc = kvc_()
    rng = np.random.default_rng(T)
    x = Made("bf16", D, B, 8, G, T, 64, rng.integers(n // 2, n + 1, B * 8), T)
    uneven(x.q, rng)
    ws = torch.empty(kvc.kvc_page_attend_masked_workspace_size(x.pool, x.pages, 8 * G, T, 40, 3), dtype=torch.uint8, device=DEV)
    res = []
    for mode, fill in ((0, 0x00), (2, 0x00), (2, 0xff), (0, 0xff)):
        ws.fill_(fill)
        out, lse = torch.full_like(x.q, 9.0), torch.full(x.q.shape[:3], 9.0, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        kvc.kvc_debug_fault(mode)
        try:
            kvc.kvc_page_attend_masked(x.pool, x.pages, x.q, out, window=40, sinks=3, lse=lse, status=status, workspace=ws)
            torch.cuda.synchronize()
        finally:
            kvc.kvc_debug_fault(0)
        assert int(status.item()) == (kvc.KVC_STATUS_TIMEOUT if mode else 0)
        res.append((out, lse))
    (o0, l0), *late, (o3, l3) = res
    assert torch.equal(o0, o3) and torch.equal(l0, l3)
    for o, l in late:
        assert torch.equal(o[2:], o0[2:]) and torch.equal(l[2:], l0[2:])  # a CTA has fewer than 16 streams
        assert not torch.equal(l[:2], l0[:2])
    assert torch.equal(late[0][0], late[1][0]) and torch.equal(late[0][1], late[1][1])
    check(x, window=40, sinks=3)


@pytest.mark.parametrize("dt,D,G,T,B,n,w", [("bf16", 128, 4, 1, 300, 200, 3500), ("bf16", 64, 2, 8, 250, 130, 3000), ("f32", 128, 4, 2, 160, 150, 2500),
                                            ("f32", 64, 4, 4, 120, 300, 4000), ("f32", 64, 2, 30, 40, 200, 2500)])
def test_few_rows_of_many_short_streams(dt, D, G, T, B, n, w):
    """Blocks of 8 and 16 rows, tables for many more tokens than the streams have: the streams' units are split over all CTAs,
    several whole streams each."""
    rng = np.random.default_rng(B + T)
    lens = rng.integers(1, n + 1, B * 8)
    lens[3::40] = 0
    x = Made(dt, D, B, 8, G, T, 64, lens, B, maxp=70)
    uneven(x.q, rng)
    n_q = rng.integers(0, T + 1, B)
    mask, depth, _ = Q.tree_mask(Q.random_trees(rng, B, T))
    check(x, mask=mask, depth=depth, n_q=n_q)
    check(x, window=w, sinks=2)
    check(x, window=w, sinks=0, mask=mask, depth=depth)
    check(x, causal=True, n_q=n_q)
