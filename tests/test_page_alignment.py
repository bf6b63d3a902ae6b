"""An int32 or float array that does not lie on 4 bytes is refused by every entry point of the paged cache on the host: on the
GPU its first access would fault."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def kvc():
    from decoding_kv_cache_gb300 import build, kvc
    build.build()
    return kvc


@pytest.mark.parametrize("off", [1, 2, 3])
def test_arrays_off_four_bytes(kvc, off):
    lib = kvc.lib()
    p = kvc.kvc_pool(D=128, page=64, npages=100, pad_=0, k_scale=1.0, v_scale=1.0, data=0x10000, refs=0x20000, free_list=0x30000, nfree=0x40000)
    t = kvc.kvc_pages(L=1, B=2, Hkv=2, maxp=8, table=0x100000, len=0x200000)
    o = kvc.kvc_pages(L=1, B=2, Hkv=2, maxp=8, table=0x300000, len=0x400000)
    P, T, O, st, ws, nb = C.byref(p), C.byref(t), C.byref(o), (C.c_int64 * 3)(512, 256, 128), 0x1000000, 1 << 40
    x, bad = 0x5000, 0x6000 + off
    calls = {  # the function, its arguments, and those that are such arrays
        "kvc_page_extend": ([P, T, x, 0, x, x, ws, nb, None], (2, 4, 5)),
        "kvc_page_free": ([P, T, x, 0, x, ws, nb, None], (2, 4)),
        "kvc_page_fork": ([P, T, x, O, x, ws, nb, None], (2, 4)),
        "kvc_page_compact": ([P, T, x, x, 8, 0, x, ws, nb, None], (2, 3, 6)),
        "kvc_page_store": ([P, T, 0, 1, x, st, x, st, x, x, x, None], (8, 9, 10)),
        "kvc_page_read": ([P, T, 0, x, 0, 4, x, x, 4, x, None], (3, 9)),
        "kvc_page_attend": ([P, T, 0, 4, 1, x, st, x, 0.1, x, x, x, ws, nb, None], (7, 10, 11)),
        "kvc_page_attend_masked": ([P, T, 0, 4, 1, x, st, x, 8, 1, x, x, 0.1, x, x, x, ws, nb, None], (7, 10, 11, 14, 15)),
        "kvc_page_slide": ([P, T, 8, 0, x, x, ws, nb, None], (4, 5)),
        "kvc_page_accept": ([P, T, 4, x, x, x, x, ws, nb, None], (3, 4, 5, 6)),
        "kvc_tree_mask": ([2, 4, x, x, 0, x, x, x, None], (2, 3, 5, 6, 7)),
        "kvc_tree_verify": ([2, 4, x, x, x, x, x, x, x, x, None], (2, 3, 4, 5, 6, 7, 8, 9)),
    }
    for name, (args, arrays) in calls.items():
        for i in arrays:
            a = list(args)
            a[i] = bad
            assert getattr(lib, name)(*a) == -8, (name, i)
