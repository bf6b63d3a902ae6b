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
//   plan   a CTA per stream clears its share of the bitmap, checks the list, finds the first row that moves and
//          lists the destination pages (marking those to be replaced); refs are read here only, before any
//          stream's change
//   move   a CTA per stream and per K or V numbers the fresh pages (in stream order) and sweeps
//   finish rows and lengths take their new values, pages are counted down, and those nobody holds any
//          more join the free list (page_ops.cu)
#include "page.cuh"

namespace kvc {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kMoveThreads = 128;
constexpr int kTile = 64;  // tokens moved at a time (36 layers x 8 heads: 36 us a cycle; 32 tokens 42, 128 tokens 41)

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PoolGeom g, PageTab t, const int32_t* kept_idx,
                                                           const int32_t* kept_len, int stride, int per_seq,
                                                           int32_t* status, PageWs w) {
  __shared__ int sm_bad, sm_k0, sm_need;
  griddep_launch();
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
    if (s == 0) {
      w.head[0] = *g.nfree;
      w.head[1] = 0;
    }
  }
  for (int i = s * kPlanThreads + (int)threadIdx.x; i < (g.npages + 31) / 32; i += t.S * kPlanThreads) w.gone[i] = 0u;
  __syncthreads();
  bool bad = sm_bad;
  int k0 = m;
  if (!bad) {
#pragma unroll 4
    for (int k = threadIdx.x; k < m; k += kPlanThreads) {  // four reads in flight
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
  int32_t* to_v = to + (size_t)t.S * t.maxp;  // the V rows' CTA numbers the same pages for itself
  if (!bad) {
    // every page the sweep reads must exist, and every page dropped
    const int e = pages_of(n, g.lp);
    for (int i = (k0 >> g.lp) + (int)threadIdx.x; i < e; i += kPlanThreads)
      if (!page_ok(g, row[i])) sm_bad = 1 | kCompactBad << 1;
    if (k0 < m) {
      const int pe = pages_of(m, g.lp);
      int need = 0;
      for (int i = (k0 >> g.lp) + (int)threadIdx.x; i < pe; i += kPlanThreads) {
        const int p = row[i];
        const bool shared = page_ok(g, p) && g.refs[p] > 1;
        to[i] = to_v[i] = shared ? -1 : p;
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
    // the first row written: with its page replaced, the page's unmoved rows go along
    int first = k0;
    if (!bad && k0 < m && to[k0 >> g.lp] < 0) first = k0 >> g.lp << g.lp;
    w.plan[s] = make_int4(first, m, n, bad ? kCompactBad : k0 < m ? kCompactMoves : 0);
  }
}

// A CTA moves the K or the V rows of a stream, kTile destinations at a time: a thread carries U code
// vectors (16 bytes) and, the first ones, a token's scales (D/16 bytes). Three reads hang on one another
// (list -> page number -> row), so each runs two tiles further ahead: while tile i is written, rows of tiles
// i+1 to i+3, page numbers of i+5 and list entries of i+7 are on their way. (With rows one tile ahead a tile
// takes a memory latency, whatever the rest: 24.5 us for 36 layers x 8 heads x 1792 kept of 2048.)
template <int D>
struct Move {
  static constexpr int kVec = D / 32;                    // code vectors of a token's row
  static constexpr int U = kTile * kVec / kMoveThreads;  // per thread
  static_assert(U >= 1 && kTile <= kMoveThreads, "a tile gives every thread a vector");
};

// Kept rows lie apart, and a plain load makes the L2 fetch 128 bytes for a row of 64: with this hint one row in
// four of 1 GB takes 48 us and not 80, a cycle of 28 x 8 x 4 heads that keep a quarter 102.2 and not 110.7 us, one
// that keeps 7 of 8 rows 35.9 and not 35.6. "memory": rows are read before others overwrite them.
__device__ __forceinline__ uint4 load_row(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// Five CTAs an SM, as the registers allow anyway: told so, the compiler orders the sweep's reads better (28 x 8 x 4
// heads that keep a quarter: 104.4 us a cycle without, 102.0 with).
template <int D>
__global__ void __launch_bounds__(kMoveThreads, 5) move_kernel(PoolGeom g, PageTab t, const int32_t* kept_idx, int stride,
                                                           int per_seq, int32_t* status, PageWs w) {
  __shared__ int sm[2 * kMoveThreads / 32];
  griddep_launch();
  griddep_wait();
  using M = Move<D>;
  constexpr int kWarpsM = kMoveThreads / 32;
  const int s = blockIdx.x >> 1, kv = blockIdx.x & 1;
  const int4 plan = w.plan[s];
  const int nfree = w.head[0];
  // pages the streams before this one take, and all (nearly always none): every CTA sums all streams' needs, two
  // or three reads a thread for some hundred streams; the sums of all CTAs grow with the square of the streams
  int before = 0, total = 0;
  for (int i = threadIdx.x; i < t.S; i += kMoveThreads) {
    const int v = w.need[i];
    total += v;
    if (i < s) before += v;
  }
  if (__syncthreads_or(total)) {
    before = __reduce_add_sync(kFull, before);
    total = __reduce_add_sync(kFull, total);
    if ((threadIdx.x & 31) == 0) {
      sm[threadIdx.x >> 5] = before;
      sm[kWarpsM + (threadIdx.x >> 5)] = total;
    }
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int i = 0; i < kWarpsM; ++i) {
      before += sm[i];
      total += sm[kWarpsM + i];
    }
  }
  const bool none = total > 0 && (total > nfree || nfree > g.npages);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (none) status_or(status, KVC_STATUS_NO_PAGES);
    w.head[1] = none ? -1 : total;  // for the kernels behind
  }
  if (none || (plan.w & kCompactBad)) return;
  const int first = plan.x, m = plan.y;
  const int32_t* row = t.table + (size_t)s * t.maxp;
  int32_t* to = w.newtab + ((size_t)kv * t.S + s) * t.maxp;
  const int need = w.need[s], pe = pages_of(m, g.lp);
  if (need) {  // the marked pages' numbers: what the streams before left, this row in order
    bool lost = false;
    if (threadIdx.x < 32) {
      int at = nfree - 1 - before;
      for (int i0 = first >> g.lp; i0 < pe; i0 += 32) {
        const int i = i0 + (int)threadIdx.x;
        const bool want = i < pe && to[i] < 0;
        const unsigned mask = __ballot_sync(kFull, want);
        if (want) {
          const int p = g.free_list[at - __popc(mask & ((1u << threadIdx.x) - 1))];
          if (page_ok(g, p))
            to[i] = p;
          else
            lost = true;  // the mark stays: the stream is left alone, here and by the finishing kernel
        }
        at -= __popc(mask);
      }
    }
    if (__syncthreads_or(lost)) {
      if (threadIdx.x == 0) status_or(status, KVC_STATUS_BAD_PAGE);
      return;
    }
  }
  if (!(plan.w & kCompactMoves)) return;

  const int32_t* idx = kept_idx + (size_t)(per_seq ? s / t.Hkv % t.B : s) * stride;
  const int lmask = (1 << g.lp) - 1;
  const int codes = kv ? piece_off(D, 2) : 0, scales = kv ? piece_off(D, 3) : piece_off(D, 1);
  const bool has_sc = threadIdx.x < kTile;
  // the tokens of a tile this thread serves: U for the codes, one for the scales
  const int v = threadIdx.x % M::kVec, k_of = threadIdx.x / M::kVec;
  constexpr int kStep = kMoveThreads / M::kVec;  // tokens between two of a thread's vectors
  struct Ahead {
    int tok[M::U + 1], page[M::U + 1];
  };
  auto read_list = [&](int t0, Ahead& x) {
#pragma unroll
    for (int u = 0; u < M::U; ++u) {
      const int k = t0 + k_of + u * kStep;
      x.tok[u] = k < m ? idx[k] : -1;
    }
    const int k = t0 + (int)threadIdx.x;
    x.tok[M::U] = has_sc && k < m ? idx[k] : -1;
  };
  auto read_pages = [&](Ahead& x) {
#pragma unroll
    for (int u = 0; u <= M::U; ++u) x.page[u] = x.tok[u] >= 0 ? row[x.tok[u] >> g.lp] : 0;
  };
  struct Rows {
    uint4 c[M::U];
    uint64_t sc;
  };
  auto read_rows = [&](const Ahead& x, Rows& r) {
#pragma unroll
    for (int u = 0; u < M::U; ++u)
      if (x.tok[u] >= 0) {
        const int in = x.tok[u] & lmask;
        r.c[u] = load_row(reinterpret_cast<const uint4*>(block_of(g, x.page[u], in >> 4) + codes + (in & 15) * (D / 2)) + v);
      }
    if (x.tok[M::U] >= 0) {
      const int in = x.tok[M::U] & lmask;
      const uint8_t* p = block_of(g, x.page[M::U], in >> 4) + scales + (in & 15) * (D / 16);
      if constexpr (D == 128)
        r.sc = *reinterpret_cast<const uint64_t*>(p);
      else
        r.sc = *reinterpret_cast<const uint32_t*>(p);
    }
  };
  auto write_rows = [&](int t0, const Rows& r) {
#pragma unroll
    for (int u = 0; u < M::U; ++u) {
      const int k = t0 + k_of + u * kStep;
      if (k < m) {
        const int in = k & lmask;
        reinterpret_cast<uint4*>(block_of(g, to[k >> g.lp], in >> 4) + codes + (in & 15) * (D / 2))[v] = r.c[u];
      }
    }
    const int k = t0 + (int)threadIdx.x;
    if (has_sc && k < m) {
      const int in = k & lmask;
      uint8_t* p = block_of(g, to[k >> g.lp], in >> 4) + scales + (in & 15) * (D / 16);
      if constexpr (D == 128)
        *reinterpret_cast<uint64_t*>(p) = r.sc;
      else
        *reinterpret_cast<uint32_t*>(p) = (uint32_t)r.sc;
    }
  };

  Ahead x[4];
  Rows r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) read_list(first + i * kTile, x[i]);
#pragma unroll
  for (int i = 0; i < 4; ++i) read_pages(x[i]);
#pragma unroll
  for (int i = 0; i < 3; ++i) read_rows(x[i], r[i]);
#pragma unroll
  for (int i = 0; i < 3; ++i) read_list(first + (4 + i) * kTile, x[i]);
  read_pages(x[0]);
  for (int t0 = first; t0 < m; t0 += 4 * kTile)
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // tile i = t0 / kTile + j
      const int ti = t0 + j * kTile;
      read_rows(x[(j + 3) & 3], r[(j + 3) & 3]);   // tile i + 3
      read_pages(x[(j + 1) & 3]);                  // i + 5
      read_list(ti + 7 * kTile, x[(j + 3) & 3]);   // i + 7
      __syncthreads();                             // every thread's rows of tile i are read
      write_rows(ti, r[j]);
    }
}

}  // namespace

int launch_page_compact(const PoolGeom& g, const PageTab& t, const int32_t* kept_idx, const int32_t* kept_len,
                        int stride, int per_seq, int32_t* status, const PageWs& w, cudaStream_t s) {
  if (launch_pdl(plan_kernel, dim3(t.S), dim3(kPlanThreads), 0, s, false, g, t, kept_idx, kept_len, stride, per_seq,
                 status, w) != cudaSuccess)
    return KVC_ERR_LAUNCH;
  if (launch_pdl(g.D == 128 ? move_kernel<128> : move_kernel<64>, dim3(2 * t.S), dim3(kMoveThreads), 0, s, false, g, t,
                 kept_idx, stride, per_seq, status, w) != cudaSuccess)
    return KVC_ERR_LAUNCH;
  return page_finish_compact(g, t, w, s);
}

}  // namespace kvc
