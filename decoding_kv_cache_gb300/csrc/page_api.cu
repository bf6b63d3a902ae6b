// page_api.cu -- the extern "C" entry points of the paged 4-bit cache: argument checks, workspace
// layout, launches. As in api.cu, every check happens on the host before the first launch.
#include <math.h>

#include "page.cuh"

namespace kvc {
namespace {

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool at4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
template <typename... P>
bool all4(P... p) { return (at4(p) && ...); }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

int check_page(int D, int page, int* lp) {
  if (D != 64 && D != 128) return KVC_ERR_UNSUPPORTED_HEAD_DIM;
  for (int l = 4; l <= 8; ++l)
    if (page == 1 << l) {
      *lp = l;
      return KVC_OK;
    }
  return KVC_ERR_INVALID_ARG;
}

int check_pool(const kvc_pool* p, PoolGeom* g) {
  if (!p) return KVC_ERR_INVALID_ARG;
  int lp;
  const int rc = check_page(p->D, p->page, &lp);
  if (rc) return rc;
  if (p->npages < 1 || p->pad_ != 0 || !p->data || !p->refs || !p->free_list || !p->nfree) return KVC_ERR_INVALID_ARG;
  if (p->npages > (1 << 28)) return KVC_ERR_TOO_LARGE;
  for (float ts : {p->k_scale, p->v_scale})
    if (!(ts >= 1e-20f && ts <= 1e20f)) return KVC_ERR_INVALID_ARG;
  if (!at16(p->data) || !at4(p->refs) || !at4(p->free_list) || !at4(p->nfree)) return KVC_ERR_ALIGNMENT;
  *g = PoolGeom{p->D, lp, p->npages, {p->k_scale, p->v_scale}, static_cast<uint8_t*>(p->data), p->refs, p->free_list,
                p->nfree};
  return KVC_OK;
}

int check_pages(const kvc_pages* p, int lp, PageTab* t) {
  if (!p || p->L < 1 || p->B < 1 || p->Hkv < 1 || p->maxp < 1 || !p->table || !p->len) return KVC_ERR_INVALID_ARG;
  const long long most = 1LL << 20;
  if (p->L > most || p->B > most || p->Hkv > most || (long long)p->L * p->B > most ||
      (long long)p->L * p->B * p->Hkv > most)
    return KVC_ERR_TOO_LARGE;
  const long long S = (long long)p->L * p->B * p->Hkv;
  // page totals of a call are 32-bit sums: every entry filled at once has to fit
  if (((long long)p->maxp << lp) > (1LL << 30) || S * p->maxp >= (1LL << 31)) return KVC_ERR_TOO_LARGE;
  if (!at4(p->table) || !at4(p->len)) return KVC_ERR_ALIGNMENT;
  *t = PageTab{p->L, p->B, p->Hkv, (int)S, p->maxp, p->table, p->len};
  return KVC_OK;
}

size_t page_ws(const PoolGeom& g, const PageTab& t, PageWs* w, void* base) {
  char* b = static_cast<char*>(base);
  size_t off = 256;
  const size_t o_gone = off;  off += up256(((size_t)g.npages + 31) / 32 * 4);
  const size_t zero = off;
  const size_t o_need = off;  off += up256((size_t)t.S * 4);
  const size_t o_sums = off;  off += up256(((size_t)t.S + 255) / 256 * 4);
  const size_t o_plan = off;  off += up256((size_t)t.S * sizeof(int4));
  const size_t o_tab = off;   off += up256((size_t)t.S * t.maxp * 8);
  if (w) {
    w->head = reinterpret_cast<int32_t*>(b);
    w->gone = reinterpret_cast<uint32_t*>(b + o_gone);
    w->need = reinterpret_cast<int32_t*>(b + o_need);
    w->sums = reinterpret_cast<int32_t*>(b + o_sums);
    w->plan = reinterpret_cast<int4*>(b + o_plan);
    w->newtab = reinterpret_cast<int32_t*>(b + o_tab);
    w->zero_bytes = zero;
  }
  return off;
}

int check_ws(const PoolGeom& g, const PageTab& t, void* ws, size_t bytes, PageWs* w) {
  if (!ws || bytes < page_ws(g, t, nullptr, nullptr) || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return KVC_ERR_WORKSPACE;
  page_ws(g, t, w, ws);
  return KVC_OK;
}

// Strides (in elements) of [B][T][heads][D] rows that are read in 16-byte vectors.
int check_rows(const void* x, const int64_t* st, int es, RowStrides* out) {
  if (!x || !st) return KVC_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if (st[i] < 0 || st[i] > (1LL << 48)) return KVC_ERR_INVALID_ARG;
    if (st[i] * es % 16) return KVC_ERR_ALIGNMENT;
  }
  if (!at16(x)) return KVC_ERR_ALIGNMENT;
  *out = RowStrides{st[0], st[1], st[2]};
  return KVC_OK;
}

int elem_size(int dtype) { return dtype == KVC_BF16 ? 2 : dtype == KVC_F32 ? 4 : 0; }

// kvc_page_attend's and kvc_page_attend_masked's checks but for the workspace
int check_attend(const kvc_pool* pool, const kvc_pages* pages, int32_t dtype, int32_t Hq, int32_t T, const void* q,
                 const int64_t* q_strides, const int32_t* n_q, float scale, void* out, float* lse, int32_t* status,
                 AttendArgs* a) {
  int rc = check_pool(pool, &a->g);
  if (rc || (rc = check_pages(pages, a->g.lp, &a->t))) return rc;
  const int es = elem_size(dtype);
  if (!es) return KVC_ERR_UNSUPPORTED_DTYPE;
  if (a->t.L != 1 || Hq < 1 || T < 1 || !out || !isfinite(scale * a->g.ts[0])) return KVC_ERR_INVALID_ARG;
  if (Hq % a->t.Hkv) return KVC_ERR_NOT_DIVISIBLE;
  if ((long long)a->t.B * Hq > (1LL << 30) || (long long)a->t.B * Hq * T > (1LL << 30)) return KVC_ERR_TOO_LARGE;
  a->Hq = Hq;
  a->T = T;
  if (!attend_fits(*a)) return KVC_ERR_TOO_LARGE;
  if ((rc = check_rows(q, q_strides, es, &a->qs))) return rc;
  if (!at16(out) || !all4(lse, n_q, status)) return KVC_ERR_ALIGNMENT;
  a->q = q;
  a->out = out;
  a->lse = lse;
  a->n_q = n_q;
  a->scale = scale * a->g.ts[0];
  a->status = status;
  a->fault = debug_fault_mode() == 2;
  return KVC_OK;
}
bool ws_fits(const void* ws, size_t bytes, size_t need) {
  return ws && bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

SeenArgs seen_args(int32_t window, int32_t sinks, const uint32_t* mask, const int32_t* depth, int32_t T) {
  // no stream is longer than kSeenAll: beyond it both mean everything
  return SeenArgs{window > 0 && window < kSeenAll ? window : kSeenAll, sinks < kSeenAll ? sinks : kSeenAll, mask, depth,
                  (T + 31) / 32};
}

int check_tree(int32_t B, int32_t T, const int32_t* parent, const int32_t* status) {
  if (B < 1 || T < 1 || !parent) return KVC_ERR_INVALID_ARG;
  if (T > KVC_TREE_MAX || B > (1 << 20)) return KVC_ERR_TOO_LARGE;
  return all4(parent, status) ? KVC_OK : KVC_ERR_ALIGNMENT;
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" {

size_t kvc_page_bytes(int32_t D, int32_t page) {
  int lp;
  return check_page(D, page, &lp) ? 0 : (size_t)blk_bytes(D) << (lp - 4);
}

size_t kvc_page_workspace_size(const kvc_pool* pool, const kvc_pages* pages) {
  PoolGeom g;
  PageTab t;
  if (check_pool(pool, &g) || check_pages(pages, g.lp, &t)) return 0;
  return page_ws(g, t, nullptr, nullptr);
}

int kvc_page_init(const kvc_pool* pool, const kvc_pages* pages, void* stream) {
  PoolGeom g;
  PageTab t;
  int rc = check_pool(pool, &g);
  if (rc) return rc;
  if (pages && (rc = check_pages(pages, g.lp, &t))) return rc;
  return launch_page_init(g, pages ? &t : nullptr, static_cast<cudaStream_t>(stream));
}

int kvc_page_extend(const kvc_pool* pool, const kvc_pages* pages, const int32_t* add, int32_t add_all, int32_t* start,
                    int32_t* status, void* workspace, size_t ws_bytes, void* stream) {
  PoolGeom g;
  PageTab t;
  PageWs w;
  int rc = check_pool(pool, &g);
  if (rc || (rc = check_pages(pages, g.lp, &t))) return rc;
  if (!add && add_all < 0) return KVC_ERR_INVALID_ARG;
  if (!all4(add, start, status)) return KVC_ERR_ALIGNMENT;
  if ((rc = check_ws(g, t, workspace, ws_bytes, &w))) return rc;
  return launch_page_extend(g, t, add, add_all, start, status, w, static_cast<cudaStream_t>(stream));
}

int kvc_page_free(const kvc_pool* pool, const kvc_pages* pages, const int32_t* drop, int32_t drop_all, int32_t* status,
                  void* workspace, size_t ws_bytes, void* stream) {
  PoolGeom g;
  PageTab t;
  PageWs w;
  int rc = check_pool(pool, &g);
  if (rc || (rc = check_pages(pages, g.lp, &t))) return rc;
  if (!drop && drop_all < 0) return KVC_ERR_INVALID_ARG;
  if (!all4(drop, status)) return KVC_ERR_ALIGNMENT;
  if ((rc = check_ws(g, t, workspace, ws_bytes, &w))) return rc;
  return launch_page_free(g, t, drop, drop_all, status, w, static_cast<cudaStream_t>(stream));
}

int kvc_page_fork(const kvc_pool* pool, const kvc_pages* pages, const int32_t* parent, const kvc_pages* out,
                  int32_t* status, void* workspace, size_t ws_bytes, void* stream) {
  PoolGeom g;
  PageTab t, o;
  PageWs w;
  int rc = check_pool(pool, &g);
  if (rc || (rc = check_pages(pages, g.lp, &t)) || (rc = check_pages(out, g.lp, &o))) return rc;
  if (!parent || o.L != t.L || o.Hkv != t.Hkv || o.maxp != t.maxp) return KVC_ERR_INVALID_ARG;
  const size_t nt = (size_t)t.S * t.maxp * 4, no = (size_t)o.S * o.maxp * 4, lt = (size_t)t.S * 4, lo = (size_t)o.S * 4;
  if (overlap(t.table, nt, o.table, no) || overlap(t.len, lt, o.len, lo) || overlap(t.table, nt, o.len, lo) ||
      overlap(t.len, lt, o.table, no) || overlap(o.table, no, o.len, lo))
    return KVC_ERR_INVALID_ARG;
  if (!all4(parent, status)) return KVC_ERR_ALIGNMENT;
  if ((rc = check_ws(g, t, workspace, ws_bytes, &w))) return rc;
  return launch_page_fork(g, t, parent, o, status, w, static_cast<cudaStream_t>(stream));
}

int kvc_page_compact(const kvc_pool* pool, const kvc_pages* pages, const int32_t* kept_idx, const int32_t* kept_len,
                     int32_t kept_stride, int32_t list_per_seq, int32_t* status, void* workspace, size_t ws_bytes,
                     void* stream) {
  PoolGeom g;
  PageTab t;
  PageWs w;
  int rc = check_pool(pool, &g);
  if (rc || (rc = check_pages(pages, g.lp, &t))) return rc;
  if (!kept_idx || !kept_len || kept_stride < 1 || (list_per_seq != 0 && list_per_seq != 1)) return KVC_ERR_INVALID_ARG;
  if (!all4(kept_idx, kept_len, status)) return KVC_ERR_ALIGNMENT;
  if ((rc = check_ws(g, t, workspace, ws_bytes, &w))) return rc;
  return launch_page_compact(g, t, kept_idx, kept_len, kept_stride, list_per_seq, status, w,
                             static_cast<cudaStream_t>(stream));
}

int kvc_page_store(const kvc_pool* pool, const kvc_pages* pages, int32_t dtype, int32_t T, const void* k,
                   const int64_t* k_strides, const void* v, const int64_t* v_strides, const int32_t* n,
                   const int32_t* start, int32_t* status, void* stream) {
  StoreArgs a = {};
  int rc = check_pool(pool, &a.g);
  if (rc || (rc = check_pages(pages, a.g.lp, &a.t))) return rc;
  const int es = elem_size(dtype);
  if (!es) return KVC_ERR_UNSUPPORTED_DTYPE;
  if (a.t.L != 1 || T < 1 || !start) return KVC_ERR_INVALID_ARG;
  if ((rc = check_rows(k, k_strides, es, &a.xs[0])) || (rc = check_rows(v, v_strides, es, &a.xs[1]))) return rc;
  if (!all4(n, start, status)) return KVC_ERR_ALIGNMENT;
  a.x[0] = k;
  a.x[1] = v;
  a.T = T;
  a.by_T = FastDiv::make(T);
  for (int i = 0; i < 2; ++i) a.inv6[i] = 1.f / (6.f * a.g.ts[i]);
  a.by_hkv = FastDiv::make(a.t.Hkv);
  a.n = n;
  a.start = start;
  a.status = status;
  return launch_page_store(a, dtype, static_cast<cudaStream_t>(stream));
}

int kvc_page_read(const kvc_pool* pool, const kvc_pages* pages, int32_t dtype, const int32_t* first, int32_t first_all,
                  int32_t count, void* k, void* v, int64_t ncap, int32_t* status, void* stream) {
  ReadArgs a = {};
  int rc = check_pool(pool, &a.g);
  if (rc || (rc = check_pages(pages, a.g.lp, &a.t))) return rc;
  if (!elem_size(dtype)) return KVC_ERR_UNSUPPORTED_DTYPE;
  if ((!k && !v) || count < 1 || ncap < count || (!first && first_all < 0)) return KVC_ERR_INVALID_ARG;
  if (!at16(k) || !at16(v) || !all4(first, status)) return KVC_ERR_ALIGNMENT;
  a.out[0] = k;
  a.out[1] = v;
  a.first = first;
  a.first_all = first_all;
  a.count = count;
  a.by_count = FastDiv::make(count);
  a.ncap = ncap;
  a.status = status;
  return launch_page_read(a, dtype, static_cast<cudaStream_t>(stream));
}

size_t kvc_page_attend_workspace_size(const kvc_pool* pool, const kvc_pages* pages, int32_t Hq, int32_t T) {
  PoolGeom g;
  PageTab t;
  if (check_pool(pool, &g) || check_pages(pages, g.lp, &t) || Hq < 1 || Hq % t.Hkv || T < 1 ||
      (long long)t.B * Hq * T > (1LL << 30))
    return 0;
  return attend_ws_bytes(g, t, Hq, T);
}

int kvc_page_attend(const kvc_pool* pool, const kvc_pages* pages, int32_t dtype, int32_t Hq, int32_t T, const void* q,
                    const int64_t* q_strides, const int32_t* n_q, float scale, void* out, float* lse, int32_t* status,
                    void* workspace, size_t ws_bytes, void* stream) {
  AttendArgs a = {};
  const int rc = check_attend(pool, pages, dtype, Hq, T, q, q_strides, n_q, scale, out, lse, status, &a);
  if (rc) return rc;
  if (!ws_fits(workspace, ws_bytes, attend_ws_bytes(a.g, a.t, Hq, T))) return KVC_ERR_WORKSPACE;
  a.ws = workspace;
  return launch_page_attend(a, dtype, static_cast<cudaStream_t>(stream));
}

size_t kvc_page_attend_masked_workspace_size(const kvc_pool* pool, const kvc_pages* pages, int32_t Hq, int32_t T,
                                             int32_t window, int32_t sinks) {
  PoolGeom g;
  PageTab t;
  if (check_pool(pool, &g) || check_pages(pages, g.lp, &t) || Hq < 1 || Hq % t.Hkv || T < 1 || window < 0 || sinks < 0 ||
      (long long)t.B * Hq * T > (1LL << 30))
    return 0;
  return attend_masked_ws_bytes(g, t, Hq, T, seen_args(window, sinks, nullptr, nullptr, T));
}

int kvc_page_attend_masked(const kvc_pool* pool, const kvc_pages* pages, int32_t dtype, int32_t Hq, int32_t T,
                           const void* q, const int64_t* q_strides, const int32_t* n_q, int32_t window, int32_t sinks,
                           const uint32_t* mask, const int32_t* depth, float scale, void* out, float* lse,
                           int32_t* status, void* workspace, size_t ws_bytes, void* stream) {
  AttendArgs a = {};
  const int rc = check_attend(pool, pages, dtype, Hq, T, q, q_strides, n_q, scale, out, lse, status, &a);
  if (rc) return rc;
  if (window < 0 || sinks < 0 || (depth && !mask)) return KVC_ERR_INVALID_ARG;
  if (mask && T > KVC_TREE_MAX) return KVC_ERR_TOO_LARGE;
  if (!all4(mask, depth)) return KVC_ERR_ALIGNMENT;
  const SeenArgs m = seen_args(window, sinks, mask, depth, T);
  if (!ws_fits(workspace, ws_bytes, attend_masked_ws_bytes(a.g, a.t, Hq, T, m))) return KVC_ERR_WORKSPACE;
  a.ws = workspace;
  return launch_page_attend_masked(a, m, dtype, static_cast<cudaStream_t>(stream));
}

int kvc_page_slide(const kvc_pool* pool, const kvc_pages* pages, int32_t window, int32_t sinks, int32_t* gone,
                   int32_t* status, void* workspace, size_t ws_bytes, void* stream) {
  PoolGeom g;
  PageTab t;
  PageWs w;
  int rc = check_pool(pool, &g);
  if (rc || (rc = check_pages(pages, g.lp, &t))) return rc;
  if (window < 1 || sinks < 0) return KVC_ERR_INVALID_ARG;
  if (!all4(gone, status)) return KVC_ERR_ALIGNMENT;
  if ((rc = check_ws(g, t, workspace, ws_bytes, &w))) return rc;
  return launch_page_slide(g, t, window, sinks < kSeenAll ? sinks : kSeenAll, gone, status, w,
                           static_cast<cudaStream_t>(stream));
}

int kvc_page_accept(const kvc_pool* pool, const kvc_pages* pages, int32_t T, const int32_t* path, const int32_t* n_path,
                    const int32_t* n_q, int32_t* status, void* workspace, size_t ws_bytes, void* stream) {
  PoolGeom g;
  PageTab t;
  PageWs w;
  int rc = check_pool(pool, &g);
  if (rc || (rc = check_pages(pages, g.lp, &t))) return rc;
  if (T < 1 || !path || !n_path) return KVC_ERR_INVALID_ARG;
  if (T > KVC_TREE_MAX) return KVC_ERR_TOO_LARGE;
  if (!all4(path, n_path, n_q, status)) return KVC_ERR_ALIGNMENT;
  if ((rc = check_ws(g, t, workspace, ws_bytes, &w))) return rc;
  return launch_page_accept(g, t, T, path, n_path, n_q, status, w, static_cast<cudaStream_t>(stream));
}

int kvc_tree_mask(int32_t B, int32_t T, const int32_t* parent, const int32_t* n_q, int32_t window, uint32_t* mask,
                  int32_t* depth, int32_t* status, void* stream) {
  const int rc = check_tree(B, T, parent, status);
  if (rc) return rc;
  if (window < 0 || !mask) return KVC_ERR_INVALID_ARG;
  if (!all4(n_q, mask, depth)) return KVC_ERR_ALIGNMENT;
  return launch_tree_mask(B, T, parent, n_q, window, mask, depth, status, static_cast<cudaStream_t>(stream));
}

int kvc_tree_verify(int32_t B, int32_t T, const int32_t* parent, const int32_t* draft, const int32_t* target,
                    const int32_t* n_q, int32_t* path, int32_t* n_path, int32_t* next, int32_t* status, void* stream) {
  const int rc = check_tree(B, T, parent, status);
  if (rc) return rc;
  if (!draft || !target || !path || !n_path) return KVC_ERR_INVALID_ARG;
  if (!all4(draft, target, n_q, path, n_path, next)) return KVC_ERR_ALIGNMENT;
  return launch_tree_verify(B, T, parent, draft, target, n_q, path, n_path, next, status,
                            static_cast<cudaStream_t>(stream));
}

}  // extern "C"
