"""A bounded wait of the paged attention is made to run out, without a GPU fault: under kvc_debug_fault(2) one
barrier of the first CTA expects an arrival that nothing makes. The call must end within its bound and say so, streams
without a share of that CTA keep their results, the next call is right again on the same workspace."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def cache(dt, D, B, Hkv, G, T, n, page):
    from decoding_kv_cache_gb300 import kvc
    maxp = n // page
    pool, pages = kvc.Pool.empty(B * Hkv * maxp, D, page, device=DEV), kvc.Pages.empty(1, B, Hkv, maxp, device=DEV)
    start = torch.zeros((1, B, Hkv), dtype=torch.int32, device=DEV)
    kvc.kvc_page_extend(pool, pages, add_all=n, start=start)
    g = torch.Generator(device=DEV).manual_seed(n + T)
    k, v = (torch.randn((B, n, Hkv, D), generator=g, device=DEV).to(dt) for _ in range(2))
    kvc.kvc_page_store(pool, pages, k, v, start)
    return kvc, pool, pages, torch.randn((B, T, Hkv * G, D), generator=g, device=DEV).to(dt)


def run_out(dt, D, B, Hkv, G, T, n, page):
    """Results under the fault (out, lse), checked against those without it; the first CTA's units are all of
    sequence 0's first KV head."""
    kvc, pool, pages, q = cache(dt, D, B, Hkv, G, T, n, page)
    ws = torch.empty(kvc.kvc_page_attend_workspace_size(pool, pages, Hkv * G, T), dtype=torch.uint8, device=DEV)
    res = []
    # under the fault once on the workspace as the first call left it, once on one of NaNs and negative numbers
    for mode, fill in ((0, False), (2, False), (2, True), (0, True)):
        if fill:
            ws.fill_(0xff)
        out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:3], 9.0, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        kvc.kvc_debug_fault(mode)
        try:
            t0 = time.time()
            kvc.kvc_page_attend(pool, pages, q, out, lse=lse, status=status, workspace=ws)
            torch.cuda.synchronize()
            took = time.time() - t0
        finally:
            kvc.kvc_debug_fault(0)
        assert int(status.item()) == (kvc.KVC_STATUS_TIMEOUT if mode else 0)
        assert took < 20.0
        res.append((out, lse))
    (o0, l0), *bad, (o3, l3) = res
    assert torch.equal(o0, o3) and torch.equal(l0, l3)
    assert torch.isfinite(l0).all() and torch.isfinite(o0.float()).all()
    for o, l in bad:
        assert torch.equal(o0[1:], o[1:]) and torch.equal(l0[1:], l[1:])
        assert torch.equal(o0[0, :, G:], o[0, :, G:]) and torch.equal(l0[0, :, G:], l[0, :, G:])  # the other heads
        assert not (l0[0, :, :G] == l[0, :, :G]).any()  # the share of the CTA that gave up is missing
    assert torch.equal(bad[0][0], bad[1][0]) and torch.equal(bad[0][1], bad[1][1])  # nothing stale came in
    return bad[0]


@pytest.mark.parametrize("dt,D,T,n", [(torch.bfloat16, 128, 1, 256), (torch.bfloat16, 64, 4, 40960), (torch.float32, 128, 2, 20480)])
def test_a_copy_that_never_lands(dt, D, T, n):
    """Whole streams a CTA, and streams split over CTAs."""
    run_out(dt, D, 2, 3, 4, T, n, 64)


@pytest.mark.parametrize("D,T", [(128, 32), (64, 20)])
def test_many_rows_kernel_gives_up_in_a_long_stream(D, T):
    """The stream's first CTA gives up: the rows that need it hold nothing, not what an earlier call left."""
    out, lse = run_out(torch.bfloat16, D, 2, 3, 4, T, 32768, 64)
    assert (out[0, :, :4] == 0).all() and torch.isneginf(lse[0, :, :4]).all()


def test_many_rows_kernel_gives_up_between_short_streams():
    """Streams of one unit: the first CTA has finished one and gives up on its second."""
    B, Hkv, G, T = 40, 8, 4, 5
    kvc, pool, pages, q = cache(torch.bfloat16, 128, B, Hkv, G, T, 128, 64)
    ws = torch.empty(kvc.kvc_page_attend_workspace_size(pool, pages, Hkv * G, T), dtype=torch.uint8, device=DEV)
    good, glse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    kvc.kvc_page_attend(pool, pages, q, good, lse=glse, workspace=ws)
    out, lse = torch.full_like(q, 9.0), torch.full_like(glse, 9.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    kvc.kvc_debug_fault(2)
    try:
        kvc.kvc_page_attend(pool, pages, q, out, lse=lse, status=status, workspace=ws)
        torch.cuda.synchronize()
    finally:
        kvc.kvc_debug_fault(0)
    assert int(status.item()) == kvc.KVC_STATUS_TIMEOUT
    bad = slice(G, 2 * G)  # of sequence 0: its second KV head
    assert (out[0, :, bad] == 0).all() and torch.isneginf(lse[0, :, bad]).all()
    out[0, :, bad], lse[0, :, bad] = good[0, :, bad], glse[0, :, bad]
    assert torch.equal(out, good) and torch.equal(lse, glse)
