// page_compact.cu -- the kept rows of a paged 4-bit cache moved to each stream's front, in place.
//
// The counterpart of compact.cuh on pages: "prefix token 和最近一小段 token 始终保留", the rest of the
// budget by score (BeaconKV write-up, end of "打分时的 RoPE 对齐"); the kept list comes from kvc_select,
// one per head or one per sequence. The forward sweep is safe in place for the same reason as there:
// the list is strictly increasing with src[k] >= k, so a tile of destinations overwrites only rows whose
// kept copies belong to this tile or an earlier one. On pages two things are added. A destination page
// that another stream shares is not written: the stream takes a fresh page in its place, and the old
// page stays as the source. And the pages behind the kept rows are given back.
//
//   plan   a CTA per stream checks the list, finds the first row that moves and lists the destination
//          pages (marking those to be replaced); refs are read here only, before any stream's change
//   move   a CTA per stream numbers its fresh pages (in stream order), sweeps, then updates its row
//   push   the pages nobody holds any more join the free list (page_ops.cu)
#include "page.cuh"

namespace kvc {

int page_push(const PoolGeom& g, const PageWs& w, cudaStream_t s);

namespace {

constexpr int kPlanThreads = 128;
constexpr int kMoveThreads = 256;
constexpr int kTile = 64;  // tokens moved at a time

enum { kBad = 1, kMoves = 2 };  // plan.w

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PoolGeom g, PageTab t, const int32_t* kept_idx,
                                                           const int32_t* kept_len, int stride, int per_seq,
                                                           int32_t* status, PageWs w) {
  __shared__ int sm_bad, sm_k0, sm_need;
  griddep_wait();
  const int s = blockIdx.x, lst = per_seq ? s / t.Hkv % t.B : s;
  const int32_t* idx = kept_idx + (size_t)lst * stride;
  const int m = kept_len[lst], n = t.len[s];
  if (threadIdx.x == 0) {
    const bool badlen = n < 0 || n > ((long long)t.maxp << g.lp);
    if (badlen) status_or(status, KVC_STATUS_BAD_PAGE);
    sm_bad = badlen || m < 0 || m > n || m > stride;
    sm_k0 = m;
    sm_need = 0;
    if (s == 0) w.head[0] = *g.nfree;
  }
  __syncthreads();
  bool bad = sm_bad;
  int k0 = m;
  if (!bad) {
    for (int k = threadIdx.x; k < m; k += kPlanThreads) {
      const int v = idx[k], next = k + 1 < m ? idx[k + 1] : n;
      if (v < k || v >= next) bad = true;
      if (v != k && k < k0) k0 = k;
    }
  }
  if (bad) sm_bad = 1;
  atomicMin(&sm_k0, k0);
  __syncthreads();
  bad = sm_bad;
  k0 = sm_k0;
  int32_t* row = t.table + (size_t)s * t.maxp;
  int32_t* to = w.newtab + (size_t)s * t.maxp;
  if (!bad) {
    // every page the sweep reads must exist, and every page dropped
    const int e = pages_of(n, g.lp);
    for (int i = (k0 >> g.lp) + (int)threadIdx.x; i < e; i += kPlanThreads)
      if (!page_ok(g, row[i])) sm_bad = 1 | kBad << 1;
    if (k0 < m) {
      const int pe = pages_of(m, g.lp);
      int need = 0;
      for (int i = (k0 >> g.lp) + (int)threadIdx.x; i < pe; i += kPlanThreads) {
        const int p = row[i];
        const bool shared = page_ok(g, p) && g.refs[p] > 1;
        to[i] = shared ? -1 : p;
        need += shared;
      }
      if (need) atomicAdd(&sm_need, need);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    bad = sm_bad != 0;
    if (sm_bad) status_or(status, sm_bad > 1 ? KVC_STATUS_BAD_PAGE : KVC_STATUS_BAD_INDEX);
    const int need = bad ? 0 : sm_need;
    w.need[s] = need;
    if (need) atomicAdd(&w.head[1], need);
    // the first row written: with its page replaced, the page's unmoved rows go along
    int first = k0;
    if (!bad && k0 < m && to[k0 >> g.lp] < 0) first = k0 >> g.lp << g.lp;
    w.plan[s] = make_int4(first, m, n, bad ? kBad : k0 < m ? kMoves : 0);
  }
}

__device__ __forceinline__ void drop_one(const PoolGeom& g, const PageWs& w, int p) {
  const int old = atomicSub(&g.refs[p], 1);
  if (old == 1)
    atomicOr(&w.gone[p >> 5], 1u << (p & 31));
  else if (old < 1)
    atomicAdd(&g.refs[p], 1);
}

// One tile of kTile destinations: each thread carries U code vectors (16 bytes) and, the first ones,
// a token's scale vector of K or V (D/16 bytes).
template <int D>
struct Tile {
  static constexpr int kVec = D / 32;                          // code vectors of a token's row
  static constexpr int U = 2 * kTile * kVec / kMoveThreads;    // per thread
  static constexpr int kSc = 2 * kTile;                        // scale vectors of the tile
  uint4 c[U];
  uint64_t sc;
};

template <int D>
__device__ __forceinline__ uint8_t* row_of(const PoolGeom& g, int page_id, int tok, int piece) {
  const int in = tok & ((1 << g.lp) - 1);
  return block_of(g, page_id, in >> 4) + piece_off(D, piece) + (in & 15) * ((piece & 1) ? D / 16 : D / 2);
}

template <int D>
__device__ __forceinline__ void tile_load(const PoolGeom& g, const int32_t* row, const int32_t* idx, int t0, int m,
                                         Tile<D>& x) {
  using TT = Tile<D>;
#pragma unroll
  for (int u = 0; u < TT::U; ++u) {
    const int e = threadIdx.x + u * kMoveThreads;
    const int v = e % TT::kVec, k = t0 + e / TT::kVec % kTile, piece = e / (TT::kVec * kTile) * 2;
    if (k < m) {
      const int src = idx[k];
      x.c[u] = reinterpret_cast<const uint4*>(row_of<D>(g, row[src >> g.lp], src, piece))[v];
    }
  }
  if (threadIdx.x < TT::kSc) {
    const int k = t0 + threadIdx.x % kTile, piece = threadIdx.x / kTile * 2 + 1;
    if (k < m) {
      const int src = idx[k];
      const uint8_t* p = row_of<D>(g, row[src >> g.lp], src, piece);
      if constexpr (D == 128)
        x.sc = *reinterpret_cast<const uint64_t*>(p);
      else
        x.sc = *reinterpret_cast<const uint32_t*>(p);
    }
  }
}

template <int D>
__device__ __forceinline__ void tile_store(const PoolGeom& g, const int32_t* to, int t0, int m, const Tile<D>& x) {
  using TT = Tile<D>;
#pragma unroll
  for (int u = 0; u < TT::U; ++u) {
    const int e = threadIdx.x + u * kMoveThreads;
    const int v = e % TT::kVec, k = t0 + e / TT::kVec % kTile, piece = e / (TT::kVec * kTile) * 2;
    if (k < m) reinterpret_cast<uint4*>(row_of<D>(g, to[k >> g.lp], k, piece))[v] = x.c[u];
  }
  if (threadIdx.x < TT::kSc) {
    const int k = t0 + threadIdx.x % kTile, piece = threadIdx.x / kTile * 2 + 1;
    if (k < m) {
      uint8_t* p = row_of<D>(g, to[k >> g.lp], k, piece);
      if constexpr (D == 128)
        *reinterpret_cast<uint64_t*>(p) = x.sc;
      else
        *reinterpret_cast<uint32_t*>(p) = (uint32_t)x.sc;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(PoolGeom g, PageTab t, const int32_t* kept_idx, int stride,
                                                           int per_seq, int32_t* status, PageWs w) {
  __shared__ int sm[8], sm_base;
  griddep_wait();
  const int s = blockIdx.x;
  const int4 plan = w.plan[s];
  const int nfree = w.head[0], total = w.head[1];
  const bool none = total > 0 && (total > nfree || nfree > g.npages);
  if (s == 0 && threadIdx.x == 0) {
    if (none)
      status_or(status, KVC_STATUS_NO_PAGES);
    else
      *g.nfree = nfree - total;
    if (none) w.head[2] = 1;
  }
  if (none || (plan.w & kBad)) return;
  const int first = plan.x, m = plan.y, n = plan.z;
  int32_t* row = t.table + (size_t)s * t.maxp;
  int32_t* to = w.newtab + (size_t)s * t.maxp;
  const int need = w.need[s], p0 = first >> g.lp, pe = pages_of(m, g.lp);
  if (need) {  // number the fresh pages: the streams before this one, then this row in order
    int b = 0;
    for (int i = threadIdx.x; i < s; i += kMoveThreads) b += w.need[i];
    b = __reduce_add_sync(kFull, b);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = b;
    __syncthreads();
    if (threadIdx.x < 32) {
      int at = nfree - 1;
#pragma unroll
      for (int i = 0; i < 8; ++i) at -= sm[i];
      for (int i0 = p0; i0 < pe; i0 += 32) {
        const int i = i0 + (int)threadIdx.x;
        const bool want = i < pe && to[i] < 0;
        const unsigned mask = __ballot_sync(kFull, want);
        if (want) {
          const int p = g.free_list[at - __popc(mask & ((1u << threadIdx.x) - 1))];
          to[i] = page_ok(g, p) ? p : row[i];
          if (page_ok(g, p)) g.refs[p] = 1;
        }
        at -= __popc(mask);
      }
    }
    __syncthreads();
  }
  if (plan.w & kMoves) {
    const int32_t* idx = kept_idx + (size_t)(per_seq ? s / t.Hkv % t.B : s) * stride;
    Tile<D> cur, nxt;
    tile_load<D>(g, row, idx, first, m, cur);
    for (int t0 = first; t0 < m; t0 += kTile) {
      if (t0 + kTile < m) tile_load<D>(g, row, idx, t0 + kTile, m, nxt);
      __syncthreads();  // every thread's loads of this tile are done
      tile_store<D>(g, to, t0, m, cur);
      cur = nxt;
    }
  }
  __syncthreads();
  if (need) {
    for (int i = p0 + (int)threadIdx.x; i < pe; i += kMoveThreads) {
      const int old = row[i], p = to[i];
      if (p != old) {
        row[i] = p;
        drop_one(g, w, old);
      }
    }
  }
  for (int i = pe + (int)threadIdx.x; i < pages_of(n, g.lp); i += kMoveThreads) {
    drop_one(g, w, row[i]);
    row[i] = -1;
  }
  if (threadIdx.x == 0) t.len[s] = m;
}

}  // namespace

int launch_page_compact(const PoolGeom& g, const PageTab& t, const int32_t* kept_idx, const int32_t* kept_len,
                        int stride, int per_seq, int32_t* status, const PageWs& w, cudaStream_t s) {
  if (cudaMemsetAsync(w.head, 0, w.zero_bytes, s) != cudaSuccess) return KVC_ERR_LAUNCH;
  if (launch_pdl(plan_kernel, dim3(t.S), dim3(kPlanThreads), 0, s, false, g, t, kept_idx, kept_len, stride, per_seq,
                 status, w) != cudaSuccess)
    return KVC_ERR_LAUNCH;
  const cudaError_t e = g.D == 128 ? launch_pdl(move_kernel<128>, dim3(t.S), dim3(kMoveThreads), 0, s, false, g, t,
                                                kept_idx, stride, per_seq, status, w)
                                   : launch_pdl(move_kernel<64>, dim3(t.S), dim3(kMoveThreads), 0, s, false, g, t,
                                                kept_idx, stride, per_seq, status, w);
  if (e != cudaSuccess) return KVC_ERR_LAUNCH;
  return page_push(g, w, s);
}

}  // namespace kvc
