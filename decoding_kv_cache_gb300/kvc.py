"""Thin Python binding over libkvc's C ABI (``include/kvc.h``).

Argument marshalling only: tensors are passed as device pointers, sizes are read from
their shapes, and every launch happens inside libkvc on the current torch stream. There
is no fallback: if ``libkvc.so`` is missing the import of this module's functions fails.
Names and argument order follow the C entry points.
"""
from __future__ import annotations

import ctypes as C
import functools
import os
from typing import Optional, Sequence, Union

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkvc.so")

KVC_BF16, KVC_F32 = 0, 1
KVC_STATUS_BUDGET_RANGE, KVC_STATUS_COUNT_RANGE, KVC_STATUS_BAD_INDEX, KVC_STATUS_TIMEOUT = 0x1, 0x2, 0x4, 0x8
KVC_STATUS_NO_PAGES, KVC_STATUS_BAD_PAGE, KVC_STATUS_TABLE_FULL = 0x10, 0x20, 0x40
KVC_MAX_LAYERS = 128
KVC_TREE_MAX = 1024

EXPORTED = ("kvc_fps_update", "kvc_score_workspace_size", "kvc_score", "kvc_select", "kvc_compact",
            "kvc_evict_workspace_size", "kvc_evict", "kvc_evict_launch_count", "kvc_strerror", "kvc_abi_version",
            "kvc_score_static", "kvc_debug_fault", "kvc_head_budget", "kvc_append", "kvc_epikv_workspace_size",
            "kvc_epikv_score", "kvc_epikv_evict", "kvc_page_bytes", "kvc_page_workspace_size", "kvc_page_init",
            "kvc_page_extend", "kvc_page_store", "kvc_page_read", "kvc_page_fork", "kvc_page_free",
            "kvc_page_compact", "kvc_page_attend_workspace_size", "kvc_page_attend", "kvc_tree_mask", "kvc_tree_verify",
            "kvc_page_attend_masked_workspace_size", "kvc_page_attend_masked", "kvc_page_slide", "kvc_page_accept")
KVC_ABI_VERSION = 5
KVC_AGG_MAX, KVC_AGG_MEAN, KVC_AGG_SUM = 0, 1, 2
KVC_BUDGET_GIVEN, KVC_BUDGET_ENTROPY = 0, 1
ROW_AGG = {"max": KVC_AGG_MAX, "mean": KVC_AGG_MEAN}
GROUP_AGG = {"max": KVC_AGG_MAX, "sum": KVC_AGG_SUM}
HEAD_BUDGET = {"given": KVC_BUDGET_GIVEN, "entropy": KVC_BUDGET_ENTROPY}
# bf16 scoring kernel (a test and profiling aid; every kernel computes the same scores)
KERNEL = {"auto": 0, "resident": 1, "split": 2, "fused": 3, "wide": 4}
KVC_STATIC_SCRATCH_BYTES = 16 << 20


class KvcError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libkvc error {code}: {msg}")
        self.code = code


class kvc_cache(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("L", C.c_int32), ("B", C.c_int32), ("Hq", C.c_int32), ("Hkv", C.c_int32),
                ("D", C.c_int32), ("N", C.c_int32), ("pad_", C.c_int32), ("ncap", C.c_int64),
                ("K", C.POINTER(C.c_void_p)), ("V", C.POINTER(C.c_void_p))]


class kvc_opts(C.Structure):
    _fields_ = [("row_agg", C.c_int32), ("group_agg", C.c_int32), ("head_budget", C.c_int32),
                ("kernel", C.c_int32), ("entropy", C.c_void_p)]


class kvc_pool(C.Structure):
    _fields_ = [("D", C.c_int32), ("page", C.c_int32), ("npages", C.c_int32), ("pad_", C.c_int32),
                ("k_scale", C.c_float), ("v_scale", C.c_float), ("data", C.c_void_p), ("refs", C.c_void_p),
                ("free_list", C.c_void_p), ("nfree", C.c_void_p)]


class kvc_pages(C.Structure):
    _fields_ = [("L", C.c_int32), ("B", C.c_int32), ("Hkv", C.c_int32), ("maxp", C.c_int32), ("table", C.c_void_p),
                ("len", C.c_void_p)]


_lib = None


def lib():
    """Load libkvc.so (built by ``decoding_kv_cache_gb300.build``); raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m decoding_kv_cache_gb300.build` "
                          "(or __graft_entry__.build()) first")
    L = C.CDLL(LIB_PATH)
    vp, i32, i64, dbl, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_double, C.c_size_t
    pc = C.POINTER(kvc_cache)
    po = C.POINTER(kvc_opts)
    pl, pg, ps = C.POINTER(kvc_pool), C.POINTER(kvc_pages), C.POINTER(i64)
    sig = {
        "kvc_fps_update": (C.c_int, [i32, i32, i32, i32, i32, vp, i32, vp, vp, vp, vp]),
        "kvc_append": (C.c_int, [i32, i32, i32, i32, i32, vp, vp, i64, dbl, vp, i32, vp, vp, i32, vp, vp, vp]),
        "kvc_score_workspace_size": (sz, [pc, i32, i32]),
        "kvc_score": (C.c_int, [pc, vp, i32, vp, vp, i32, i32, i64, dbl, vp, vp, po, vp, sz, vp]),
        "kvc_select": (C.c_int, [vp, i32, i32, i32, i32, i32, i32, vp, i32, vp, vp, vp, vp]),
        "kvc_compact": (C.c_int, [pc, vp, vp, vp, vp]),
        "kvc_evict_workspace_size": (sz, [pc, i32, i32]),
        "kvc_evict": (C.c_int, [pc, vp, i32, vp, vp, i32, i32, i64, dbl, i32, i32, vp, i32, vp, vp, vp, vp, po, vp,
                                sz, vp]),
        "kvc_evict_launch_count": (C.c_int, [pc, i32, i32]),
        "kvc_score_static": (C.c_int, [pc, vp, i32, vp, vp, i32, i32, i64, dbl, vp, vp, po, vp]),
        "kvc_head_budget": (C.c_int, [vp, i32, i32, i32, i32, i32, i32, vp, i32, vp, vp, vp]),
        "kvc_epikv_workspace_size": (sz, [i32, i32]),
        "kvc_epikv_score": (C.c_int, [i32, i32, i32, i32, vp, vp, i32, C.c_float, vp, vp, vp, sz, vp]),
        "kvc_epikv_evict": (C.c_int, [pc, vp, vp, i32, i32, C.c_float, i32, i32, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
        "kvc_page_bytes": (sz, [i32, i32]),
        "kvc_page_workspace_size": (sz, [pl, pg]),
        "kvc_page_init": (C.c_int, [pl, pg, vp]),
        "kvc_page_extend": (C.c_int, [pl, pg, vp, i32, vp, vp, vp, sz, vp]),
        "kvc_page_store": (C.c_int, [pl, pg, i32, i32, vp, ps, vp, ps, vp, vp, vp, vp]),
        "kvc_page_read": (C.c_int, [pl, pg, i32, vp, i32, i32, vp, vp, i64, vp, vp]),
        "kvc_page_fork": (C.c_int, [pl, pg, vp, pg, vp, vp, sz, vp]),
        "kvc_page_free": (C.c_int, [pl, pg, vp, i32, vp, vp, sz, vp]),
        "kvc_page_compact": (C.c_int, [pl, pg, vp, vp, i32, i32, vp, vp, sz, vp]),
        "kvc_page_attend_workspace_size": (sz, [pl, pg, i32, i32]),
        "kvc_page_attend": (C.c_int, [pl, pg, i32, i32, i32, vp, ps, vp, C.c_float, vp, vp, vp, vp, sz, vp]),
        "kvc_tree_mask": (C.c_int, [i32, i32, vp, vp, i32, vp, vp, vp, vp]),
        "kvc_tree_verify": (C.c_int, [i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "kvc_page_attend_masked_workspace_size": (sz, [pl, pg, i32, i32, i32, i32]),
        "kvc_page_attend_masked": (C.c_int, [pl, pg, i32, i32, i32, vp, ps, vp, i32, i32, vp, vp, C.c_float, vp, vp, vp,
                                             vp, sz, vp]),
        "kvc_page_slide": (C.c_int, [pl, pg, i32, i32, vp, vp, vp, sz, vp]),
        "kvc_page_accept": (C.c_int, [pl, pg, i32, vp, vp, vp, vp, vp, sz, vp]),
        "kvc_strerror": (C.c_char_p, [C.c_int]),
        "kvc_abi_version": (C.c_int, []),
        "kvc_debug_fault": (C.c_int, [i32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def _check(rc: int):
    if rc != 0:
        raise KvcError(rc, lib().kvc_strerror(rc).decode())


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libkvc takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("libkvc takes contiguous tensors")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _i32(n, what: str) -> int:
    """A whole number for an int32 argument: of a larger one ctypes would keep the low bits."""
    if not -0x80000000 <= n <= 0x7fffffff:
        raise ValueError(f"{what} must fit 32 bits")
    return n


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KVC_BF16
    if t.dtype == torch.float32:
        return KVC_F32
    raise KvcError(-2, f"unsupported storage type {t.dtype}")


class Cache:
    """A ``kvc_cache`` over torch tensors: K/V either one [L,B,Hkv,ncap,D] tensor each or lists of
    per-layer [B,Hkv,ncap,D] tensors. ``N`` is the number of valid tokens per head (default ncap)."""

    def __init__(self, K: Union[torch.Tensor, Sequence[torch.Tensor]], V, Hq: int, N: Optional[int] = None):
        Ks = list(K.unbind(0)) if isinstance(K, torch.Tensor) else list(K)
        Vs = list(V.unbind(0)) if isinstance(V, torch.Tensor) else list(V)
        if len(Ks) != len(Vs) or not Ks:
            raise ValueError("K and V need the same, non-zero number of layers")
        B, Hkv, ncap, D = Ks[0].shape
        for t in Ks + Vs:
            if tuple(t.shape) != (B, Hkv, ncap, D) or t.dtype != Ks[0].dtype or not t.is_contiguous():
                raise ValueError("every layer of K and V must be a contiguous [B,Hkv,ncap,D] tensor of one dtype")
        self.layers_K, self.layers_V = Ks, Vs
        self._kp = (C.c_void_p * len(Ks))(*[t.data_ptr() for t in Ks])
        self._vp = (C.c_void_p * len(Vs))(*[t.data_ptr() for t in Vs])
        self.c = kvc_cache(dtype=_dtype_code(Ks[0]), L=len(Ks), B=B, Hq=_i32(Hq, "Hq"), Hkv=Hkv, D=D,
                           N=ncap if N is None else _i32(N, "N"), pad_=0, ncap=ncap,
                           K=C.cast(self._kp, C.POINTER(C.c_void_p)), V=C.cast(self._vp, C.POINTER(C.c_void_p)))

    @property
    def ref(self):
        return C.byref(self.c)

    @property
    def heads(self) -> int:
        return self.c.L * self.c.B * self.c.Hkv


def kvc_fps_update(qbuf: torch.Tensor, count: torch.Tensor, picks: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None):
    """Continual-FPS compression of every full [..., qmax, D] buffer in place (see kvc.h).
    ``count`` holds one int32 per buffer; ``picks`` (optional) is [..., qmax/2] int32."""
    qmax, D = qbuf.shape[-2], qbuf.shape[-1]
    nq = qbuf.numel() // (qmax * D)
    _check(lib().kvc_fps_update(_dtype_code(qbuf), 1, 1, nq, D, _p(qbuf), qmax, _p(count), _p(picks), _p(status),
                                _stream(stream)))


def kvc_append(q_pre: torch.Tensor, qbuf: torch.Tensor, count: torch.Tensor, q_recent: Optional[torch.Tensor],
               t: int, rope_theta: float = 1e4, q_post: Optional[torch.Tensor] = None,
               picks: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """One decode step's queries into the observation state (see kvc.h): ``q_pre`` [..., D] joins
    each head's [..., qmax, D] buffer (compressed when full), and ``q_post`` (or ``q_pre`` turned to
    ``t``) joins ring row ``t mod n_r`` of ``q_recent`` [..., n_r, D] (None or n_r = 0: no ring)."""
    qmax, D = qbuf.shape[-2], qbuf.shape[-1]
    nq = qbuf.numel() // (qmax * D)
    if q_pre.numel() != nq * D or (q_post is not None and q_post.numel() != nq * D):
        raise ValueError("q_pre / q_post need one [D] row per buffer")
    n_r = 0 if q_recent is None else q_recent.shape[-2]
    if q_recent is not None and q_recent.numel() != nq * n_r * D:
        raise ValueError("q_recent needs one [n_r, D] ring per buffer")
    _check(lib().kvc_append(_dtype_code(qbuf), 1, 1, nq, D, _p(q_pre), _p(q_post), int(t), float(rope_theta),
                            _p(qbuf), qmax, _p(count), _p(q_recent) if n_r else None, n_r, _p(picks), _p(status),
                            _stream(stream)))


def kvc_score_workspace_size(cache: Cache, n_r: int, n_b: int) -> int:
    return int(lib().kvc_score_workspace_size(cache.ref, _i32(n_r, "n_r"), _i32(n_b, "n_b")))


def kvc_evict_workspace_size(cache: Cache, n_r: int, n_b: int) -> int:
    return int(lib().kvc_evict_workspace_size(cache.ref, _i32(n_r, "n_r"), _i32(n_b, "n_b")))


def kvc_evict_launch_count(cache: Cache, n_r: int, n_b: int) -> int:
    return int(lib().kvc_evict_launch_count(cache.ref, _i32(n_r, "n_r"), _i32(n_b, "n_b")))


def kvc_debug_fault(mode: int) -> None:
    """Test-only fault switch (see include/kvc.h): 1 makes the scoring exchange wait run out, 2 a wait of
    the paged attention."""
    _check(lib().kvc_debug_fault(_i32(int(mode), "mode")))


def make_opts(row_agg: str = "max", group_agg: str = "max", head_budget: str = "given",
              entropy: Optional[torch.Tensor] = None, kernel: str = "auto"):
    """A ``kvc_opts`` (see kvc.h), or None for the defaults (max/max, budgets as given, no entropy,
    automatic kernel choice)."""
    if row_agg == "max" and group_agg == "max" and head_budget == "given" and entropy is None and kernel == "auto":
        return None
    return kvc_opts(row_agg=ROW_AGG[row_agg], group_agg=GROUP_AGG[group_agg], head_budget=HEAD_BUDGET[head_budget],
                    kernel=KERNEL[kernel], entropy=_p(entropy))


def _opts_ref(o):
    return None if o is None else C.byref(o)


def _workspace(nbytes: int, device, workspace):
    if workspace is not None:
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def kvc_score(cache: Cache, q_recent: torch.Tensor, qbuf: torch.Tensor, count: torch.Tensor, n_b: int, t: int,
              rope_theta: float, scores: torch.Tensor, beacon_picks: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream=None, row_agg: str = "max", group_agg: str = "max",
              entropy: Optional[torch.Tensor] = None, kernel: str = "auto"):
    """Scores of every cached key; ``row_agg``/``group_agg``/``entropy``/``kernel`` set kvc_opts."""
    n_r, qmax = q_recent.shape[-2], qbuf.shape[-2]
    ws = _workspace(kvc_score_workspace_size(cache, n_r, n_b), scores.device, workspace)
    o = make_opts(row_agg, group_agg, "given", entropy, kernel)
    _check(lib().kvc_score(cache.ref, _p(q_recent), n_r, _p(qbuf), _p(count), qmax, _i32(n_b, "n_b"), int(t),
                           float(rope_theta), _p(scores), _p(beacon_picks), _opts_ref(o), _p(ws),
                           ws.numel() * ws.element_size(),
                           _stream(stream)))


def kvc_score_static(cache: Cache, q_recent: torch.Tensor, qbuf: torch.Tensor, count: torch.Tensor, n_b: int,
                     t: int, rope_theta: float, scores: torch.Tensor, beacon_picks: Optional[torch.Tensor] = None,
                     stream=None, row_agg: str = "max", group_agg: str = "max",
                     entropy: Optional[torch.Tensor] = None, kernel: str = "auto"):
    """kvc_score with the library's fixed scratch region instead of a workspace (allocates nothing;
    see kvc.h for the size limit and the sharing rules)."""
    n_r, qmax = q_recent.shape[-2], qbuf.shape[-2]
    o = make_opts(row_agg, group_agg, "given", entropy, kernel)
    _check(lib().kvc_score_static(cache.ref, _p(q_recent), n_r, _p(qbuf), _p(count), qmax, _i32(n_b, "n_b"), int(t),
                                  float(rope_theta), _p(scores), _p(beacon_picks), _opts_ref(o), _stream(stream)))


def kvc_select(scores: torch.Tensor, prefix: int, recent: int, kept_idx: torch.Tensor, kept_len: torch.Tensor,
               budget: Optional[torch.Tensor] = None, budget_all: int = 0, status: Optional[torch.Tensor] = None,
               stream=None):
    L, B, Hkv, N = scores.shape
    _check(lib().kvc_select(_p(scores), L, B, Hkv, N, _i32(prefix, "prefix"), _i32(recent, "recent"), _p(budget),
                            _i32(int(budget_all), "budget_all"), _p(kept_idx), _p(kept_len), _p(status), _stream(stream)))


def kvc_compact(cache: Cache, kept_idx: torch.Tensor, kept_len: torch.Tensor, status: Optional[torch.Tensor] = None,
                stream=None):
    _check(lib().kvc_compact(cache.ref, _p(kept_idx), _p(kept_len), _p(status), _stream(stream)))


def kvc_evict(cache: Cache, q_recent: torch.Tensor, qbuf: torch.Tensor, count: torch.Tensor, n_b: int, t: int,
              rope_theta: float, prefix: int, recent: int, kept_len: torch.Tensor,
              budget: Optional[torch.Tensor] = None, budget_all: int = 0, kept_idx: Optional[torch.Tensor] = None,
              scores: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream=None, row_agg: str = "max", group_agg: str = "max",
              head_budget: str = "given", entropy: Optional[torch.Tensor] = None, kernel: str = "auto"):
    """The whole eviction step (beacons, scores, selection, in-place compaction) on one stream.
    ``row_agg``/``group_agg``/``head_budget``/``entropy``/``kernel`` set kvc_opts."""
    n_r, qmax = q_recent.shape[-2], qbuf.shape[-2]
    ws = _workspace(kvc_evict_workspace_size(cache, n_r, n_b), kept_len.device, workspace)
    o = make_opts(row_agg, group_agg, head_budget, entropy, kernel)
    _check(lib().kvc_evict(cache.ref, _p(q_recent), n_r, _p(qbuf), _p(count), qmax, _i32(n_b, "n_b"), int(t),
                           float(rope_theta), _i32(prefix, "prefix"), _i32(recent, "recent"), _p(budget),
                           _i32(int(budget_all), "budget_all"), _p(kept_idx), _p(kept_len), _p(scores),
                           _p(status), _opts_ref(o), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def kvc_head_budget(entropy: torch.Tensor, N: int, prefix: int, recent: int, budget_out: torch.Tensor,
                    budget: Optional[torch.Tensor] = None, budget_all: int = 0, status: Optional[torch.Tensor] = None,
                    stream=None):
    """Each (layer, sequence)'s budgets reallocated over its heads by entropy (see kvc.h)."""
    L, B, Hkv = entropy.shape
    _check(lib().kvc_head_budget(_p(entropy), L, B, Hkv, _i32(int(N), "N"), _i32(int(prefix), "prefix"),
                                 _i32(int(recent), "recent"), _p(budget),
                                 _i32(int(budget_all), "budget_all"), _p(budget_out), _p(status),
                                 _stream(stream)))


def kvc_epikv_workspace_size(B: int, N: int) -> int:
    return int(lib().kvc_epikv_workspace_size(_i32(B, "B"), _i32(N, "N")))


def kvc_epikv_score(hA: torch.Tensor, hB: torch.Tensor, window: int, eps: float, scores: torch.Tensor,
                    g: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """EPIKV scores [B, N] from two layers' hidden states [B, N, dm] (see kvc.h); ``g`` [2, B, N]
    optionally receives the two layers' signals."""
    B, N, dm = hA.shape
    if tuple(hB.shape) != (B, N, dm) or hB.dtype != hA.dtype:
        raise ValueError("hA and hB must be [B, N, dm] tensors of one dtype")
    ws = _workspace(kvc_epikv_workspace_size(B, N), hA.device, workspace)
    _check(lib().kvc_epikv_score(_dtype_code(hA), B, N, dm, _p(hA), _p(hB), _i32(int(window), "window"), float(eps), _p(g),
                                 _p(scores), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def kvc_epikv_evict(cache: Cache, hA: torch.Tensor, hB: torch.Tensor, window: int, eps: float, prefix: int,
                    recent: int, kept_len: torch.Tensor, budget: Optional[torch.Tensor] = None, budget_all: int = 0,
                    kept_idx: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Eviction by the EPIKV score: one kept list per sequence compacts all its layers and heads."""
    B, N, dm = hA.shape
    ws = _workspace(kvc_epikv_workspace_size(B, N), hA.device, workspace)
    _check(lib().kvc_epikv_evict(cache.ref, _p(hA), _p(hB), dm, _i32(int(window), "window"), float(eps),
                                 _i32(int(prefix), "prefix"), _i32(int(recent), "recent"), _p(budget),
                                 _i32(int(budget_all), "budget_all"), _p(kept_idx), _p(kept_len), _p(scores), _p(status),
                                 _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


# ---------------------------------------------------------------------------------------------
# the paged 4-bit cache
# ---------------------------------------------------------------------------------------------
def kvc_page_bytes(D: int, page: int) -> int:
    return int(lib().kvc_page_bytes(_i32(D, "D"), _i32(page, "page")))


def _ints(t: Optional[torch.Tensor], shape, dev, what: str, dtype=torch.int32):
    """The pointer of a contiguous tensor of the given shape and type on the pool's device, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}")
    return t.data_ptr()


class Pool:
    """A ``kvc_pool`` over torch tensors: ``data`` uint8 [npages, kvc_page_bytes(D, page)], ``refs`` and
    ``free_list`` int32 [npages], ``nfree`` int32 [1]. ``Pool.empty`` allocates and initialises them."""

    def __init__(self, data: torch.Tensor, refs: torch.Tensor, free_list: torch.Tensor, nfree: torch.Tensor, D: int,
                 page: int, k_scale: float = 1.0, v_scale: float = 1.0):
        nb = kvc_page_bytes(D, page)
        if not nb:
            raise KvcError(-3 if D not in (64, 128) else -1, "unsupported head dimension or page size")
        if not data.is_cuda:
            raise ValueError("libkvc takes CUDA tensors")
        n = data.shape[0]
        dev = data.device
        self.data, self.refs, self.free_list, self.nfree = data, refs, free_list, nfree
        self.device, self.D, self.page, self.npages = dev, D, page, n
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.c = kvc_pool(D=D, page=page, npages=n, pad_=0, k_scale=k_scale, v_scale=v_scale,
                          data=_ints(data, (n, nb), dev, "data", torch.uint8),
                          refs=_ints(refs, (n,), dev, "refs"), free_list=_ints(free_list, (n,), dev, "free_list"),
                          nfree=_ints(nfree, (1,), dev, "nfree"))
        self.ref = C.byref(self.c)

    @classmethod
    def empty(cls, npages: int, D: int, page: int = 64, k_scale: float = 1.0, v_scale: float = 1.0, device="cuda"):
        """A pool of ``npages`` free pages."""
        z = lambda shape, dt=torch.int32: torch.zeros(shape, dtype=dt, device=device)
        p = cls(z((npages, kvc_page_bytes(D, page)), torch.uint8), z(npages), z(npages), z(1), D, page, k_scale, v_scale)
        kvc_page_init(p)
        return p


class Pages:
    """A ``kvc_pages`` over torch tensors: ``table`` int32 [L, B, Hkv, maxp], ``len`` int32 [L, B, Hkv]."""

    def __init__(self, table: torch.Tensor, len: torch.Tensor):
        L, B, Hkv, maxp = table.shape
        dev = table.device
        self.table, self.len, self.device = table, len, dev
        self.c = kvc_pages(L=L, B=B, Hkv=Hkv, maxp=maxp, table=_ints(table, (L, B, Hkv, maxp), dev, "table"),
                           len=_ints(len, (L, B, Hkv), dev, "len"))
        self.shape = (L, B, Hkv)
        self.ref = C.byref(self.c)

    @classmethod
    def empty(cls, L: int, B: int, Hkv: int, maxp: int, device="cuda"):
        return cls(torch.full((L, B, Hkv, maxp), -1, dtype=torch.int32, device=device),
                   torch.zeros((L, B, Hkv), dtype=torch.int32, device=device))

    def layer(self, l: int) -> "Pages":
        return Pages(self.table[l:l + 1], self.len[l:l + 1])


def _page_call(name: str, pool: Pool, pages: Optional[Pages], stream, args):
    """One entry point on the pool's device: ``args`` follow the pool and the pages, the stream comes last."""
    dev = pool.device
    if pages is not None and pages.device != dev:
        raise ValueError("the pool and its pages are on different devices")
    stream = torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else _stream(stream)
    f = getattr(_lib or lib(), name)
    if dev.index == torch._C._cuda_getDevice():
        rc = f(pool.ref, None if pages is None else pages.ref, *args, stream)
    else:
        with torch.cuda.device(dev):
            rc = f(pool.ref, None if pages is None else pages.ref, *args, stream)
    if rc:
        _check(rc)


def _page_ws(nbytes, pool: Pool, workspace, stream):
    """(pointer, bytes, tensor) of the caller's workspace, or of one of nbytes() made for this call."""
    if workspace is None:
        workspace = torch.empty(max(nbytes(), 256), dtype=torch.uint8, device=pool.device)
        if stream is not None:  # it belongs to the current stream: not given out again before `stream` is done
            workspace.record_stream(stream if isinstance(stream, torch.cuda.Stream) else
                                    torch.cuda.ExternalStream(_stream(stream), device=pool.device))
    elif workspace.device != pool.device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the pool's device")
    return workspace.data_ptr(), workspace.nbytes, workspace


def _word(status, pool: Pool):
    return None if status is None else _ints(status, (1,), pool.device, "status")


def kvc_page_workspace_size(pool: Pool, pages: Pages) -> int:
    return int(lib().kvc_page_workspace_size(pool.ref, pages.ref))


def kvc_page_attend_workspace_size(pool: Pool, pages: Pages, Hq: int, T: int) -> int:
    return int(lib().kvc_page_attend_workspace_size(pool.ref, pages.ref, _i32(Hq, "Hq"), _i32(T, "T")))


def kvc_page_init(pool: Pool, pages: Optional[Pages] = None, stream=None):
    """Every page free and, with ``pages``, every stream empty."""
    _page_call("kvc_page_init", pool, pages, stream, ())


def kvc_page_extend(pool: Pool, pages: Pages, add: Optional[torch.Tensor] = None, add_all: int = 0,
                    start: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """Room for ``add`` [B] (or ``add_all``) more tokens in every stream; ``start`` [L, B, Hkv] receives the
    old lengths (see kvc.h)."""
    dev = pool.device
    wp, wb, ws = _page_ws(lambda: kvc_page_workspace_size(pool, pages), pool, workspace, stream)
    _page_call("kvc_page_extend", pool, pages, stream,
               (_ints(add, (pages.shape[1],), dev, "add"), _i32(int(add_all), "add_all"),
                _ints(start, pages.shape, dev, "start"), _word(status, pool), wp, wb))


def kvc_page_free(pool: Pool, pages: Pages, drop: Optional[torch.Tensor] = None, drop_all: int = 0,
                  status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """The last ``drop`` [B] (or ``drop_all``) tokens of every stream go, with the pages they leave empty."""
    wp, wb, ws = _page_ws(lambda: kvc_page_workspace_size(pool, pages), pool, workspace, stream)
    _page_call("kvc_page_free", pool, pages, stream,
               (_ints(drop, (pages.shape[1],), pool.device, "drop"), _i32(int(drop_all), "drop_all"), _word(status, pool),
                wp, wb))


def kvc_page_fork(pool: Pool, pages: Pages, parent: torch.Tensor, out: Pages, status: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """``out``'s sequence c becomes a copy of ``pages``' sequence ``parent[c]``; ``pages`` is given up."""
    if out.device != pool.device:
        raise ValueError("the pool and its pages are on different devices")
    wp, wb, ws = _page_ws(lambda: kvc_page_workspace_size(pool, pages), pool, workspace, stream)
    _page_call("kvc_page_fork", pool, pages, stream,
               (_ints(parent, (out.shape[1],), pool.device, "parent"), out.ref, _word(status, pool), wp, wb))


def kvc_page_compact(pool: Pool, pages: Pages, kept_idx: torch.Tensor, kept_len: torch.Tensor,
                     status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """The kept tokens to every stream's front: lists per stream ([L, B, Hkv, n] and [L, B, Hkv], as
    kvc_select's) or per sequence ([B, n] and [B], as kvc_epikv_evict's)."""
    per_seq = kept_idx.dim() == 2
    lead = (pages.shape[1],) if per_seq else pages.shape
    wp, wb, ws = _page_ws(lambda: kvc_page_workspace_size(pool, pages), pool, workspace, stream)
    _page_call("kvc_page_compact", pool, pages, stream,
               (_ints(kept_idx, lead + (kept_idx.shape[-1],), pool.device, "kept_idx"),
                _ints(kept_len, lead, pool.device, "kept_len"), kept_idx.shape[-1], int(per_seq), _word(status, pool),
                wp, wb))


_Strides = C.c_int64 * 3


@functools.lru_cache(maxsize=256)
def _strides(b: int, t: int, h: int):
    return _Strides(b, t, h)  # read by the call only


def _rows(x: torch.Tensor, shape, pool: Pool, what: str):
    """The pointer and strides of [B, T, heads, D] rows with contiguous channels."""
    s = x.stride()
    if x.device != pool.device or x.shape != shape or s[3] != 1:
        raise ValueError(f"{what} must be a {tuple(shape)} tensor on {pool.device} with contiguous channels")
    # a dimension of one row has no stride that counts
    return x.data_ptr(), _strides(s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0, s[2] if shape[2] > 1 else 0)


def kvc_page_store(pool: Pool, pages: Pages, k: torch.Tensor, v: torch.Tensor, start: torch.Tensor,
                   n: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """One layer's new rows ``k``, ``v`` [B, T, Hkv, D] (any batch, token and head strides that are multiples of
    16 bytes) into tokens ``start`` [1, B, Hkv] and on; ``n`` [B] rows of them (default all T)."""
    _, B, Hkv = pages.shape
    if k.dim() != 4 or v.dtype is not k.dtype:
        raise ValueError("k and v must be [B, T, Hkv, D] tensors of one dtype")
    shape = (B, k.shape[1], Hkv, pool.D)
    kp, ks = _rows(k, shape, pool, "k")
    vp, vs = _rows(v, shape, pool, "v")
    _page_call("kvc_page_store", pool, pages, stream,
               (_dtype_code(k), shape[1], kp, ks, vp, vs, _ints(n, (B,), pool.device, "n"),
                _ints(start, pages.shape, pool.device, "start"), _word(status, pool)))


def kvc_page_read(pool: Pool, pages: Pages, k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                  first: Optional[torch.Tensor] = None, first_all: int = 0, count: Optional[int] = None,
                  status: Optional[torch.Tensor] = None, stream=None):
    """Tokens ``first`` [L, B, Hkv] (or ``first_all``) and on of every stream into rows 0..count-1 (default
    all) of dense ``k``, ``v`` [L, B, Hkv, ncap, D]; rows past a stream's length are left as they were."""
    x = k if k is not None else v
    if x is None:
        raise ValueError("kvc_page_read needs k or v")
    shape = x.shape
    if len(shape) != 5 or shape[:3] != pages.shape or shape[4] != pool.D:
        raise ValueError("k and v must be [L, B, Hkv, ncap, D] tensors")
    ncap = shape[3]
    _page_call("kvc_page_read", pool, pages, stream,
               (_dtype_code(x), _ints(first, pages.shape, pool.device, "first"), _i32(int(first_all), "first_all"),
                ncap if count is None else _i32(int(count), "count"), _ints(k, shape, pool.device, "k", x.dtype),
                _ints(v, shape, pool.device, "v", x.dtype), ncap, _word(status, pool)))


def kvc_page_attend(pool: Pool, pages: Pages, q: torch.Tensor, out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                    n_q: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of ``q`` [B, T, Hq, D] (strided like kvc_page_store's rows), the newest T tokens' queries, over
    one layer of the cache; ``out`` [B, T, Hq, D], ``lse`` [B, T, Hq] fp32; ``scale`` defaults to 1/sqrt(D)."""
    B = pages.shape[1]
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be a [B, T, Hq, D] tensor")
    _, T, Hq, D = shape
    qp, qs = _rows(q, (B, T, Hq, pool.D), pool, "q")
    wp, wb, ws = _page_ws(lambda: kvc_page_attend_workspace_size(pool, pages, Hq, T), pool, workspace, stream)
    _page_call("kvc_page_attend", pool, pages, stream,
               (_dtype_code(q), Hq, T, qp, qs, _ints(n_q, (B,), pool.device, "n_q"),
                float(D ** -0.5 if scale is None else scale), _ints(out, shape, pool.device, "out", q.dtype),
                _ints(lse, (B, T, Hq), pool.device, "lse", torch.float32), _word(status, pool), wp, wb))


# ---------------------------------------------------------------------------------------------
# windows and drafted trees over the paged cache
# ---------------------------------------------------------------------------------------------
def _tree_call(name: str, parent: torch.Tensor, stream, args):
    """One tree entry point on the device of ``parent`` [B, T]; the stream comes last."""
    dev = parent.device
    stream = torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else _stream(stream)
    f = getattr(_lib or lib(), name)
    if dev.index == torch._C._cuda_getDevice():
        rc = f(*parent.shape, parent.data_ptr(), *args, stream)
    else:
        with torch.cuda.device(dev):
            rc = f(*parent.shape, parent.data_ptr(), *args, stream)
    if rc:
        _check(rc)


def _tree(parent: torch.Tensor):
    """(B, T, device) of a tree's parents."""
    if not parent.is_cuda:
        raise ValueError("libkvc takes CUDA tensors")
    if parent.dim() != 2 or parent.dtype is not torch.int32 or not parent.is_contiguous():
        raise ValueError("parent must be a contiguous int32 tensor [B, T]")
    return (*parent.shape, parent.device)


def kvc_tree_mask(parent: torch.Tensor, mask: torch.Tensor, depth: Optional[torch.Tensor] = None,
                  n_q: Optional[torch.Tensor] = None, window: int = 0, status: Optional[torch.Tensor] = None,
                  stream=None):
    """Which drafts each one sees: ``parent`` [B, T] to the bits ``mask`` [B, T, ceil(T/32)] (int32 words) of itself and
    its ancestors (the nearest ``window`` of them, 0: all) and its ``depth`` [B, T]; once a step, for all layers."""
    B, T, dev = _tree(parent)
    _tree_call("kvc_tree_mask", parent, stream,
               (_ints(n_q, (B,), dev, "n_q"), _i32(int(window), "window"), _ints(mask, (B, T, (T + 31) // 32), dev, "mask"),
                _ints(depth, (B, T), dev, "depth"), _ints(status, (1,), dev, "status")))


def kvc_tree_verify(parent: torch.Tensor, draft: torch.Tensor, target: torch.Tensor, path: torch.Tensor,
                    n_path: torch.Tensor, next: Optional[torch.Tensor] = None, n_q: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None):
    """The drafts that the model's picks confirm: token numbers ``draft`` [B, T] and, behind each draft, the model's
    ``target`` [B, T] to ``path`` [B, T] (ascending, -1 behind), ``n_path`` [B] and the pick behind it, ``next`` [B]."""
    B, T, dev = _tree(parent)
    _tree_call("kvc_tree_verify", parent, stream,
               (_ints(draft, (B, T), dev, "draft"), _ints(target, (B, T), dev, "target"), _ints(n_q, (B,), dev, "n_q"),
                _ints(path, (B, T), dev, "path"), _ints(n_path, (B,), dev, "n_path"), _ints(next, (B,), dev, "next"),
                _ints(status, (1,), dev, "status")))


def kvc_page_attend_masked_workspace_size(pool: Pool, pages: Pages, Hq: int, T: int, window: int = 0,
                                          sinks: int = 0) -> int:
    return int(lib().kvc_page_attend_masked_workspace_size(pool.ref, pages.ref, _i32(Hq, "Hq"), _i32(T, "T"),
                                                           _i32(window, "window"), _i32(sinks, "sinks")))


def kvc_page_attend_masked(pool: Pool, pages: Pages, q: torch.Tensor, out: torch.Tensor, window: int = 0, sinks: int = 0,
                           mask: Optional[torch.Tensor] = None, depth: Optional[torch.Tensor] = None,
                           lse: Optional[torch.Tensor] = None, n_q: Optional[torch.Tensor] = None,
                           scale: Optional[float] = None, status: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """kvc_page_attend where a query sees the first ``sinks`` tokens and those less than ``window`` positions back (0:
    all) and, with ``mask`` [B, T, ceil(T/32)] and ``depth`` [B, T] of kvc_tree_mask, of the queries' own tokens its
    ancestors."""
    B = pages.shape[1]
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be a [B, T, Hq, D] tensor")
    _, T, Hq, D = shape
    dev = pool.device
    qp, qs = _rows(q, (B, T, Hq, pool.D), pool, "q")
    wp, wb, ws = _page_ws(lambda: kvc_page_attend_masked_workspace_size(pool, pages, Hq, T, window, sinks), pool,
                          workspace, stream)
    _page_call("kvc_page_attend_masked", pool, pages, stream,
               (_dtype_code(q), Hq, T, qp, qs, _ints(n_q, (B,), dev, "n_q"), _i32(int(window), "window"),
                _i32(int(sinks), "sinks"), _ints(mask, (B, T, (T + 31) // 32), dev, "mask"), _ints(depth, (B, T), dev, "depth"),
                float(D ** -0.5 if scale is None else scale), _ints(out, shape, dev, "out", q.dtype),
                _ints(lse, (B, T, Hq), dev, "lse", torch.float32), _word(status, pool), wp, wb))


def kvc_page_slide(pool: Pool, pages: Pages, window: int, sinks: int = 0, gone: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Every stream's whole pages between the first ``sinks`` tokens and the last ``window`` are given up; ``gone``
    [L, B, Hkv] receives the tokens that went."""
    wp, wb, ws = _page_ws(lambda: kvc_page_workspace_size(pool, pages), pool, workspace, stream)
    _page_call("kvc_page_slide", pool, pages, stream,
               (_i32(int(window), "window"), _i32(int(sinks), "sinks"), _ints(gone, pages.shape, pool.device, "gone"),
                _word(status, pool), wp, wb))


def kvc_page_accept(pool: Pool, pages: Pages, path: torch.Tensor, n_path: torch.Tensor,
                    n_q: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """Of every stream's newest T (or ``n_q`` [B]) tokens those at ``path`` [B, T] stay, ``n_path`` [B] of them; the
    others go."""
    B, dev = pages.shape[1], pool.device
    if path.dim() != 2:
        raise ValueError("path must be a [B, T] tensor")
    wp, wb, ws = _page_ws(lambda: kvc_page_workspace_size(pool, pages), pool, workspace, stream)
    _page_call("kvc_page_accept", pool, pages, stream,
               (path.shape[1], _ints(path, (B, path.shape[1]), dev, "path"), _ints(n_path, (B,), dev, "n_path"),
                _ints(n_q, (B,), dev, "n_q"), _word(status, pool), wp, wb))
