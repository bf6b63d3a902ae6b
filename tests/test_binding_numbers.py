"""Whole numbers that do not fit the C side's 32 bits are refused by the binding (no GPU): ctypes would keep their low bits,
and a window of 2^32 + 5 would give up all but 5 tokens."""
import ctypes as C
import types

import pytest
import torch


@pytest.fixture(scope="module")
def kvc():
    from decoding_kv_cache_gb300 import build, kvc
    build.build()
    kvc.lib()
    return kvc


def handles(kvc):
    dev = torch.device("cpu")
    c = kvc.kvc_pool(D=128, page=64, npages=100, pad_=0, k_scale=1.0, v_scale=1.0, data=0x10000, refs=0x20000, free_list=0x30000,
                     nfree=0x40000)
    t = kvc.kvc_pages(L=1, B=2, Hkv=2, maxp=8, table=0x100000, len=0x200000)
    pool = types.SimpleNamespace(c=c, ref=C.byref(c), device=dev, D=128, page=64, npages=100)
    return pool, types.SimpleNamespace(c=t, ref=C.byref(t), device=dev, shape=(1, 2, 2)), torch.empty(1 << 16, dtype=torch.uint8)


BIG = [1 << 31, (1 << 32) + 5, 1 << 32, -(1 << 31) - 1, (1 << 63) - 1]


@pytest.mark.parametrize("n", BIG)
def test_numbers_beyond_32_bits(kvc, n):
    pool, pages, ws = handles(kvc)
    q = torch.zeros((2, 1, 4, 128), dtype=torch.bfloat16)
    rows = torch.zeros((1, 2, 2, 3, 128))
    for call in (
            lambda: kvc.kvc_page_slide(pool, pages, n, workspace=ws), lambda: kvc.kvc_page_slide(pool, pages, 8, n, workspace=ws),
            lambda: kvc.kvc_page_attend_masked(pool, pages, q, q.clone(), window=n, workspace=ws),
            lambda: kvc.kvc_page_attend_masked(pool, pages, q, q.clone(), window=5, sinks=n, workspace=ws),
            lambda: kvc.kvc_page_attend_masked_workspace_size(pool, pages, 4, 1, n),
            lambda: kvc.kvc_page_attend_masked_workspace_size(pool, pages, 4, 1, 8, n),
            lambda: kvc.kvc_page_attend_masked_workspace_size(pool, pages, 4, n),
            lambda: kvc.kvc_page_attend_masked_workspace_size(pool, pages, n, 1),
            lambda: kvc.kvc_page_attend_workspace_size(pool, pages, n, 1),
            lambda: kvc.kvc_page_attend_workspace_size(pool, pages, 4, n),
            lambda: kvc.kvc_page_bytes(n, 64), lambda: kvc.kvc_page_bytes(128, n),
            lambda: kvc.kvc_page_extend(pool, pages, add_all=n, workspace=ws),
            lambda: kvc.kvc_page_free(pool, pages, drop_all=n, workspace=ws),
            lambda: kvc.kvc_page_read(pool, pages, rows, first_all=n),
            lambda: kvc.kvc_page_read(pool, pages, rows, count=n),
            lambda: kvc.kvc_epikv_workspace_size(n, 4), lambda: kvc.kvc_debug_fault(n)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_numbers_at_the_ends_are_checked_by_the_library(kvc):
    pool, pages, _ = handles(kvc)
    size = kvc.kvc_page_attend_masked_workspace_size
    assert size(pool, pages, 4, 1, (1 << 31) - 1, (1 << 31) - 1) == size(pool, pages, 4, 1) > 0
    assert size(pool, pages, 4, 1, -(1 << 31)) == 0
    with pytest.raises(kvc.KvcError):
        kvc.kvc_debug_fault(-(1 << 31))
