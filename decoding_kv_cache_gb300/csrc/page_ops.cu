// page_ops.cu -- pages of the 4-bit cache taken, shared, copied on write and given back.
//
// Every result is a function of the arguments alone: pages are taken from the free list's end in
// stream order, counted with integer atomics (whose order cannot show), and given back in the order
// of their numbers through a bitmap. A call that cannot get all its pages changes nothing.
#include <cooperative_groups.h>

#include "page.cuh"

namespace kvc {
namespace {

namespace cg = cooperative_groups;

constexpr int kCopyFlag = 1 << 30;
constexpr int kPlanThreads = 256;   // streams per planning CTA
constexpr int kAssignStreams = 8;   // streams per assigning CTA, a warp each
constexpr int kAssignThreads = 256;
constexpr int kPushThreads = 256;
constexpr int kPushWords = kPushThreads;  // bitmap words per giving-back CTA

__device__ __forceinline__ int warp_sum_i(int v) { return __reduce_add_sync(kFull, v); }

// block-wide sum for 256 threads; every thread gets it
__device__ __forceinline__ int block_sum(int v, int* sm) {
  v = warp_sum_i(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) t += sm[i];
  return t;
}

__global__ void init_kernel(PoolGeom g, PageTab t) {
  griddep_launch();
  griddep_wait();
  const long long n = (long long)g.npages, e = (long long)t.S * t.maxp;
  const long long step = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n || i < e; i += step) {
    if (i < n) {
      g.refs[i] = 0;
      g.free_list[i] = (int)(n - 1 - i);
    }
    if (i < e) t.table[i] = -1;
    if (i < t.S) t.len[i] = 0;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *g.nfree = g.npages;
}

// What stream s asks of an extension by `a` tokens: its length, the pages, whether its last page is
// partly filled; false (and a status bit) when the request cannot stand.
__device__ __forceinline__ bool extend_wants(const PoolGeom& g, const PageTab& t, int s, int a, int* n, int32_t* status) {
  *n = t.len[s];
  const long long cap = (long long)t.maxp << g.lp;
  if (*n < 0 || *n > cap) {
    status_or(status, KVC_STATUS_BAD_PAGE);
    return false;
  }
  if (a < 0) {
    status_or(status, KVC_STATUS_BAD_INDEX);
    return false;
  }
  if (*n + (long long)a > cap) {
    status_or(status, KVC_STATUS_TABLE_FULL);
    return false;
  }
  return true;
}

// Pages stream s takes (kCopyFlag when its last page is copied), -1 where the request cannot stand: the fresh
// ones behind its last page and, when that page is partly filled and shared, a copy of it. Of the streams
// that share a page and all write to it, the lowest sequence keeps it; the sharers of a page are sequences
// of the same layer and head (forks keep it so), found by comparing that page's number over the sequences,
// for shared last pages only.
__device__ __forceinline__ int extend_need(const PoolGeom& g, const PageTab& t, int s, const int32_t* add, int add_all,
                                           int32_t* status) {
  const int h = s % t.Hkv, b = s / t.Hkv % t.B, l = s / (t.Hkv * t.B);
  const int a = add ? add[b] : add_all;
  int n;
  if (!extend_wants(g, t, s, a, &n, status)) return -1;
  if (a == 0) return 0;
  const int need = pages_of(n + a, g.lp) - pages_of(n, g.lp);
  if (!(n & ((1 << g.lp) - 1))) return need;
  const int p = t.table[(size_t)s * t.maxp + (n >> g.lp)];
  if (!page_ok(g, p)) {
    status_or(status, KVC_STATUS_BAD_PAGE);
    return -1;
  }
  const int r = g.refs[p];
  if (r <= 1) return need;
  int writers = 0, lowest = b;
  for (int o = 0; o < t.B; ++o) {
    const int so = (l * t.B + o) * t.Hkv + h;
    const int ao = add ? add[o] : add_all, no = t.len[so];
    if (ao <= 0 || no <= 0 || no + (long long)ao > ((long long)t.maxp << g.lp) || !(no & ((1 << g.lp) - 1))) continue;
    if (t.table[(size_t)so * t.maxp + (no >> g.lp)] != p) continue;
    ++writers;
    if (o < lowest) lowest = o;
  }
  return lowest == b && writers >= r ? need : (need + 1) | kCopyFlag;
}

__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(PoolGeom g, PageTab t, const int32_t* add,
                                                                  int add_all, int32_t* status, PageWs w) {
  __shared__ int sm[8];
  griddep_launch();
  griddep_wait();
  const int s = blockIdx.x * kPlanThreads + threadIdx.x;
  int need = 0;
  if (s < t.S) {
    need = extend_need(g, t, s, add, add_all, status);
    w.need[s] = need;
  }
  const int sum = block_sum(need < 0 ? 0 : need & ~kCopyFlag, sm);
  if (threadIdx.x == 0) {
    w.sums[blockIdx.x] = sum;
    if (blockIdx.x == 0) w.head[0] = *g.nfree;
  }
}

__device__ __forceinline__ int need_of(const PageWs& w, int s) {
  const int v = w.need[s];
  return v < 0 ? 0 : v & ~kCopyFlag;
}

// Pages before stream s0 (a multiple of 32) and in all; every thread gets both.
__device__ __forceinline__ void need_before(const PageWs& w, int S, int s0, int* sm, int* before, int* total) {
  const int blk = s0 / kPlanThreads, nblk = (S + kPlanThreads - 1) / kPlanThreads;
  int b = 0, all = 0;
  for (int i = threadIdx.x; i < nblk; i += blockDim.x) {
    const int v = w.sums[i];
    all += v;
    if (i < blk) b += v;
  }
  const int s = blk * kPlanThreads + threadIdx.x;
  if (s < s0) b += need_of(w, s);
  *total = block_sum(all, sm);
  *before = block_sum(b, sm);
}

__device__ __forceinline__ void copy_page(const PoolGeom& g, int dst, int src, int lane) {
  const size_t bytes = (size_t)blk_bytes(g.D) << (g.lp - 4);
  uint4* d = reinterpret_cast<uint4*>(g.data + (size_t)dst * bytes);
  const uint4* x = reinterpret_cast<const uint4*>(g.data + (size_t)src * bytes);
  const int n = (int)(bytes / 16);
  constexpr int kDeep = 9;  // vectors a lane has in flight: two rounds for 64 tokens of D = 128
  for (int i = lane; i < n; i += kDeep * 32) {
    uint4 v[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (i + u * 32 < n) v[u] = x[i + u * 32];
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (i + u * 32 < n) d[i + u * 32] = v[u];
  }
}

// A warp hands stream s its pages (`before` pages go to the streams before it) and copies its page.
__device__ __forceinline__ void extend_stream(const PoolGeom& g, const PageTab& t, int s, int need, int before, bool none,
                                              int nfree, const int32_t* add, int add_all, int32_t* start,
                                              int32_t* status) {
  const int lane = threadIdx.x & 31;
  if (none || need < 0) {
    if (lane == 0 && start) start[s] = -1;
    return;
  }
  const int b = s / t.Hkv % t.B;
  const int a = add ? add[b] : add_all, n = t.len[s];
  const int k = need & ~kCopyFlag, copy = need & kCopyFlag ? 1 : 0;
  const int at = nfree - 1 - before;  // free-list slot of the stream's first page
  int32_t* row = t.table + (size_t)s * t.maxp;
  constexpr int kHeld = 4;
  int mine[kHeld];  // its first 128 pages, in one round of reads
  bool lost = false;
#pragma unroll
  for (int u = 0; u < kHeld; ++u) mine[u] = lane + 32 * u < k ? g.free_list[at - lane - 32 * u] : 0;
#pragma unroll
  for (int u = 0; u < kHeld; ++u) lost |= !page_ok(g, mine[u]);
  for (int j = lane + 32 * kHeld; j < k; j += 32) lost |= !page_ok(g, g.free_list[at - j]);
  if (__any_sync(kFull, lost)) {  // no page's number in the free list
    if (lane == 0) {
      status_or(status, KVC_STATUS_BAD_PAGE);
      if (start) start[s] = -1;
    }
    return;
  }
  const int first = pages_of(n, g.lp) - copy;
  auto take = [&](int j, int p) {
    if (j >= copy) row[first + j] = p;
    g.refs[p] = 1;
  };
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (lane + 32 * u < k) take(lane + 32 * u, mine[u]);
  for (int j = lane + 32 * kHeld; j < k; j += 32) take(j, g.free_list[at - j]);
  if (copy) {
    const int old = row[n >> g.lp], p = __shfl_sync(kFull, mine[0], 0);
    copy_page(g, p, old, lane);
    __syncwarp();
    if (lane == 0) {
      row[n >> g.lp] = p;
      atomicSub(&g.refs[old], 1);
    }
  }
  if (lane == 0) {
    t.len[s] = n + a;
    if (start) start[s] = n;
  }
}

// The pages handed out: a warp per stream.
__global__ void __launch_bounds__(kAssignThreads) extend_assign_kernel(PoolGeom g, PageTab t, const int32_t* add,
                                                                      int add_all, int32_t* start, int32_t* status,
                                                                      PageWs w) {
  __shared__ int sm[8];
  griddep_launch();
  griddep_wait();
  const int s0 = blockIdx.x * kAssignStreams, warp = threadIdx.x >> 5;
  int before, total;
  need_before(w, t.S, s0, sm, &before, &total);
  const int nfree = w.head[0];
  const bool none = total > nfree || nfree > g.npages;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (none)
      status_or(status, KVC_STATUS_NO_PAGES);
    else
      *g.nfree = nfree - total;
  }
  const int s = s0 + warp;
  if (s >= t.S) return;
  for (int i = s0; i < s; ++i) before += need_of(w, i);
  extend_stream(g, t, s, w.need[s], before, none, nfree, add, add_all, start, status);
}

// Counted down; a page whose last reference goes is marked.
__device__ __forceinline__ void drop_page(const PoolGeom& g, const PageWs& w, int p, int32_t* status) {
  if (!page_ok(g, p)) {
    status_or(status, KVC_STATUS_BAD_PAGE);
    return;
  }
  const int old = atomicSub(&g.refs[p], 1);
  if (old == 1)
    atomicOr(&w.gone[p >> 5], 1u << (p & 31));
  else if (old < 1) {
    atomicAdd(&g.refs[p], 1);
    status_or(status, KVC_STATUS_BAD_PAGE);
  }
}

// a warp per stream
__global__ void __launch_bounds__(256) free_kernel(PoolGeom g, PageTab t, const int32_t* drop, int drop_all,
                                                  int32_t* status, PageWs w) {
  griddep_launch();
  griddep_wait();
  const int s = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (s == 0 && lane == 0) w.head[0] = *g.nfree;
  if (s >= t.S) return;
  const int d = drop ? drop[s / t.Hkv % t.B] : drop_all, n = t.len[s];
  if (d < 0 || n < 0 || n > ((long long)t.maxp << g.lp)) {
    if (lane == 0) status_or(status, d < 0 ? KVC_STATUS_BAD_INDEX : KVC_STATUS_BAD_PAGE);
    return;
  }
  const int left = n > d ? n - d : 0;
  int32_t* row = t.table + (size_t)s * t.maxp;
  const int e = pages_of(n, g.lp);
  for (int i = pages_of(left, g.lp) + lane; i < e; i += 32) {
    drop_page(g, w, row[i], status);
    row[i] = -1;
  }
  __syncwarp();
  if (lane == 0) t.len[s] = left;
}

// Warps of the first t.S streams count their pages' new references (children - 1 each: old references
// plus every partial sum stay above zero unless all of a page's holders go, so the one that reaches
// zero is the last whatever the order); the others write the children's rows.
__global__ void __launch_bounds__(256) fork_kernel(PoolGeom g, PageTab t, const int32_t* parent, PageTab out,
                                                  int32_t* status, PageWs w) {
  griddep_launch();
  griddep_wait();
  const int i = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (i == 0 && lane == 0) w.head[0] = *g.nfree;
  const long long cap = (long long)t.maxp << g.lp;
  if (i < t.S) {
    const int b = i / t.Hkv % t.B, n = t.len[i];
    if (n < 0 || n > cap) {
      if (lane == 0) status_or(status, KVC_STATUS_BAD_PAGE);
      return;
    }
    int kids = 0;
    for (int o = lane; o < out.B; o += 32) kids += parent[o] == b;
    const int delta = warp_sum_i(kids) - 1;
    if (delta == 0) return;
    const int32_t* row = t.table + (size_t)i * t.maxp;
    const int e = pages_of(n, g.lp);
    for (int j = lane; j < e; j += 32) {
      const int p = row[j];
      if (delta < 0) {
        drop_page(g, w, p, status);
      } else if (page_ok(g, p)) {
        atomicAdd(&g.refs[p], delta);
      } else {
        status_or(status, KVC_STATUS_BAD_PAGE);
      }
    }
  } else if (i - t.S < out.S) {
    const int c = i - t.S;
    const int h = c % t.Hkv, l = c / (t.Hkv * out.B);
    const int b = parent[c / t.Hkv % out.B];
    int n = 0;
    const int32_t* row = nullptr;
    if (b >= 0 && b < t.B) {
      const int s = (l * t.B + b) * t.Hkv + h;
      n = t.len[s];
      if (n < 0 || n > cap) n = 0;
      row = t.table + (size_t)s * t.maxp;
    } else if (b != -1) {
      if (lane == 0) status_or(status, KVC_STATUS_BAD_INDEX);
    }
    const int e = pages_of(n, g.lp);
    int32_t* to = out.table + (size_t)c * t.maxp;
    for (int j = lane; j < t.maxp; j += 32) to[j] = j < e ? row[j] : -1;
    if (lane == 0) out.len[c] = n;
  }
}

// The marks of 32 words (one a lane), whose numbers start at word w0, to the free list from `at` on: a
// word at a time, its pages by the lanes whose bits are set, so that a run of pages is one store.
__device__ __forceinline__ void push_words(const PoolGeom& g, uint32_t m, int w0, int at) {
  const int lane = threadIdx.x & 31;
  int incl = __popc(m);
  const int mine = incl;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  at += incl - mine;
  for (unsigned any = __ballot_sync(kFull, m != 0); any; any &= any - 1) {
    const int j = __ffs(any) - 1;
    const uint32_t x = __shfl_sync(kFull, m, j);
    const int to = __shfl_sync(kFull, at, j) + __popc(x & ((1u << lane) - 1));
    if ((x >> lane & 1) && to >= 0 && to < g.npages) g.free_list[to] = (w0 + j) * 32 + lane;
  }
}

// The marked pages join the free list in the order of their numbers. Each CTA counts the marks before
// its words itself (the bitmap is small and in L2), so no CTA waits for another.
__global__ void __launch_bounds__(kPushThreads) push_kernel(PoolGeom g, PageWs w) {
  __shared__ int sm[8];
  griddep_launch();
  griddep_wait();
  const int words = (g.npages + 31) / 32, w0 = blockIdx.x * kPushWords;
  const int i = w0 + threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t m = i < words ? w.gone[i] : 0u;
  const int nfree = w.head[0] - max(w.head[1], 0);  // what the call took is off the list's end
  int c = 0;
  const uint4* g4 = reinterpret_cast<const uint4*>(w.gone);
#pragma unroll 4
  for (int k = threadIdx.x; k < w0 / 4; k += kPushThreads) {
    const uint4 v = g4[k];
    c += __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
  }
  const int base = block_sum(c, sm);
  const int in_warp = warp_sum_i(__popc(m));
  __syncthreads();
  if (lane == 0) sm[warp] = in_warp;
  __syncthreads();
  int at = nfree + base, all = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k < warp) at += sm[k];
    all += sm[k];
  }
  push_words(g, m, i - lane, at);
  if (w0 + kPushWords >= words && threadIdx.x == 0) *g.nfree = nfree + base + all;
}

// ---- frees and forks in one launch ----------------------------------------------------------------
// One cluster of eight CTAs does the counting, and its barrier stands where the wide form starts the
// next kernel (zeroed bitmap | counts | free list and lengths): three launches' overhead becomes one.
// Eight SMs suffice for the page entries of ordinary tables; the wide form takes over beyond
// kOneEntries entries, kOnePages pages or kOneSeqs sequences.
constexpr int kOneCtas = 8, kOneThreads = 1024;
constexpr long long kOneEntries = 1 << 14;
constexpr int kOnePages = 1 << 20, kOneSeqs = 1024;

// The marked pages join the free list: CTA r takes the r-th eighth of the bitmap's words.
__device__ __forceinline__ void cluster_push(cg::cluster_group& cl, const PoolGeom& g, const PageWs& w, int nfree) {
  __shared__ int sm[kOneThreads / 32], sm_total;
  const int rank = cl.block_rank(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int words = (g.npages + 31) / 32, per = (words + kOneCtas - 1) / kOneCtas;
  const int w0 = min(words, rank * per), w1 = min(words, w0 + per);
  int c = 0;
  for (int i = w0 + threadIdx.x; i < w1; i += kOneThreads) c += __popc(__ldcg(&w.gone[i]));
  c = warp_sum_i(c);
  if (lane == 0) sm[warp] = c;
  __syncthreads();
  if (warp == 0) {
    c = warp_sum_i(sm[lane]);
    if (lane == 0) sm_total = c;
  }
  cl.sync();
  int base = 0, all = 0;
  for (int r = 0; r < kOneCtas; ++r) {
    const int v = *cl.map_shared_rank(&sm_total, r);
    if (r < rank) base += v;
    all += v;
  }
  for (int i0 = w0; i0 < w1; i0 += kOneThreads) {
    const int i = i0 + threadIdx.x;
    const uint32_t m = i < w1 ? __ldcg(&w.gone[i]) : 0u;
    const int in_warp = warp_sum_i(__popc(m));
    __syncthreads();
    if (lane == 0) sm[warp] = in_warp;
    __syncthreads();
    const int v = sm[lane];
    push_words(g, m, i - lane, nfree + base + warp_sum_i(lane < warp ? v : 0));
    base += warp_sum_i(v);
  }
  if (rank == 0 && threadIdx.x == 0) *g.nfree = nfree + all;
  cl.sync();  // no CTA leaves while another reads its shared memory
}

__device__ __forceinline__ void cluster_zero(const PoolGeom& g, const PageWs& w, int at) {
  const int words = (g.npages + 31) / 32;
  for (int i = at; i < words; i += kOneCtas * kOneThreads) w.gone[i] = 0u;
}

__global__ void __cluster_dims__(kOneCtas, 1, 1) __launch_bounds__(kOneThreads)
    free_one_kernel(PoolGeom g, PageTab t, const int32_t* drop, int drop_all, int32_t* status, PageWs w) {
  griddep_launch();
  griddep_wait();
  cg::cluster_group cl = cg::this_cluster();
  const int at = cl.block_rank() * kOneThreads + threadIdx.x, step = kOneCtas * kOneThreads;
  const int nfree = *g.nfree;
  const long long cap = (long long)t.maxp << g.lp;
  cluster_zero(g, w, at);
  cl.sync();
  const int entries = t.S * t.maxp;
#pragma unroll 4
  for (int e = at; e < entries; e += step) {
    const int s = e / t.maxp, i = e - s * t.maxp;
    const int d = drop ? drop[s / t.Hkv % t.B] : drop_all, n = t.len[s], p = t.table[e];
    if (d < 0 || n < 0 || n > cap) {
      if (i == 0) status_or(status, d < 0 ? KVC_STATUS_BAD_INDEX : KVC_STATUS_BAD_PAGE);
      continue;
    }
    if (i >= pages_of(n > d ? n - d : 0, g.lp) && i < pages_of(n, g.lp)) {
      drop_page(g, w, p, status);
      t.table[e] = -1;
    }
  }
  cl.sync();
  for (int s = at; s < t.S; s += step) {
    const int d = drop ? drop[s / t.Hkv % t.B] : drop_all, n = t.len[s];
    if (d > 0 && n >= 0 && n <= cap) t.len[s] = n > d ? n - d : 0;
  }
  cluster_push(cl, g, w, nfree);
}

__global__ void __cluster_dims__(kOneCtas, 1, 1) __launch_bounds__(kOneThreads)
    fork_one_kernel(PoolGeom g, PageTab t, const int32_t* parent, PageTab out, int32_t* status, PageWs w) {
  __shared__ int kids[kOneSeqs];
  griddep_launch();
  griddep_wait();
  cg::cluster_group cl = cg::this_cluster();
  const int at = cl.block_rank() * kOneThreads + threadIdx.x, step = kOneCtas * kOneThreads;
  const int nfree = *g.nfree;
  const long long cap = (long long)t.maxp << g.lp;
  cluster_zero(g, w, at);
  for (int b = threadIdx.x; b < t.B; b += kOneThreads) kids[b] = 0;
  __syncthreads();
  for (int c = threadIdx.x; c < out.B; c += kOneThreads) {
    const int b = parent[c];
    if (b >= 0 && b < t.B)
      atomicAdd(&kids[b], 1);
    else if (b != -1)
      status_or(status, KVC_STATUS_BAD_INDEX);
  }
  cl.sync();
  const int entries = t.S * t.maxp;
#pragma unroll 4
  for (int e = at; e < entries; e += step) {
    const int s = e / t.maxp, i = e - s * t.maxp;
    const int n = t.len[s], p = t.table[e], delta = kids[s / t.Hkv % t.B] - 1;
    if (n < 0 || n > cap) {
      if (i == 0) status_or(status, KVC_STATUS_BAD_PAGE);
      continue;
    }
    if (i >= pages_of(n, g.lp) || delta == 0) continue;
    if (delta < 0)
      drop_page(g, w, p, status);
    else if (page_ok(g, p))
      atomicAdd(&g.refs[p], delta);
    else
      status_or(status, KVC_STATUS_BAD_PAGE);
  }
  const int oentries = out.S * t.maxp;
#pragma unroll 4
  for (int e = at; e < oentries; e += step) {
    const int c = e / t.maxp, i = e - c * t.maxp;
    const int b = parent[c / t.Hkv % out.B];
    int n = 0, p = -1;
    if (b >= 0 && b < t.B) {
      const int s = (c / (t.Hkv * out.B) * t.B + b) * t.Hkv + c % t.Hkv;
      n = t.len[s];
      if (n < 0 || n > cap) n = 0;
      p = t.table[(size_t)s * t.maxp + i];
    }
    out.table[e] = i < pages_of(n, g.lp) ? p : -1;
    if (i == 0) out.len[c] = n;
  }
  cl.sync();
  cluster_push(cl, g, w, nfree);
}

// Up to kOneStreams streams extended in one launch: every CTA of the cluster plans all of them (a thread each),
// the barrier stands between the reads and the changes, then a warp takes a stream.
constexpr int kOneStreams = 256;
__global__ void __cluster_dims__(kOneCtas, 1, 1) __launch_bounds__(kOneThreads)
    extend_one_kernel(PoolGeom g, PageTab t, const int32_t* add, int add_all, int32_t* start, int32_t* status) {
  __shared__ int sm_need[kOneStreams], sm_before[kOneStreams], sm_sum[kOneThreads / 32];
  griddep_launch();
  griddep_wait();
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nfree = *g.nfree;
  int need = 0;
  if ((int)threadIdx.x < t.S) need = extend_need(g, t, threadIdx.x, add, add_all, cl.block_rank() == 0 ? status : nullptr);
  const int mine = need < 0 ? 0 : need & ~kCopyFlag;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm_sum[warp] = incl;
  __syncthreads();
  int before = incl - mine, total = 0;
#pragma unroll
  for (int i = 0; i < kOneStreams / 32; ++i) {
    if (i < warp) before += sm_sum[i];
    total += sm_sum[i];
  }
  if (threadIdx.x < kOneStreams) {
    sm_need[threadIdx.x] = need;
    sm_before[threadIdx.x] = before;
  }
  cl.sync();
  const bool none = total > nfree || nfree > g.npages;
  if (cl.block_rank() == 0 && threadIdx.x == 0) {
    if (none)
      status_or(status, KVC_STATUS_NO_PAGES);
    else
      *g.nfree = nfree - total;
  }
  const int s = warp * kOneCtas + cl.block_rank();  // neighbours on different SMs
  if (s < t.S) extend_stream(g, t, s, sm_need[s], sm_before[s], none, nfree, add, add_all, start, status);
}

// ---- slides ---------------------------------------------------------------------------------------
// The entries that a slide takes out of a stream of n tokens: m from `first` on.
__device__ __forceinline__ int slide_count(const PoolGeom& g, int n, int window, int first) {
  return n < window ? 0 : max(0, ((n - window + 1) >> g.lp) - first);
}

// A warp slides stream s: the pages that go are counted down, the entries behind them move up, 256 read before
// they are written (their places lie before every later entry's).
__device__ __forceinline__ void slide_stream(const PoolGeom& g, const PageTab& t, const PageWs& w, int s, int n, int first,
                                             int m, int32_t* status) {
  const int lane = threadIdx.x & 31, e = pages_of(n, g.lp);
  int32_t* row = t.table + (size_t)s * t.maxp;
  for (int i = first + lane; i < first + m; i += 32) drop_page(g, w, row[i], status);
  __syncwarp();
  constexpr int kDeep = 8;
  for (int i0 = first; i0 < e; i0 += 32 * kDeep) {
    int p[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int i = i0 + 32 * u + lane + m;
      p[u] = i < e ? row[i] : -1;
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int i = i0 + 32 * u + lane;
      if (i < e) row[i] = p[u];
    }
    __syncwarp();
  }
  if (lane == 0) t.len[s] = n - (m << g.lp);
}

// Lane i of a warp looks at stream s0 + i * step; those that lose pages are slid one after another by the whole warp
// (in a decode step one in `page`).
__device__ __forceinline__ void slide_streams(const PoolGeom& g, const PageTab& t, const PageWs& w, int s0, int step,
                                              int window, int first, int32_t* gone, int32_t* status) {
  const int lane = threadIdx.x & 31;
  for (; s0 < t.S; s0 += 32 * step) {
    const long long s = s0 + (long long)lane * step;
    int n = 0, m = 0;
    if (s < t.S) {
      n = t.len[s];
      const bool bad = n < 0 || n > ((long long)t.maxp << g.lp);
      if (bad) status_or(status, KVC_STATUS_BAD_PAGE);
      m = bad ? 0 : slide_count(g, n, window, first);
      if (gone) gone[s] = bad ? -1 : m << g.lp;
    }
    for (unsigned any = __ballot_sync(kFull, m > 0); any; any &= any - 1) {
      const int j = __ffs(any) - 1;
      slide_stream(g, t, w, s0 + j * step, __shfl_sync(kFull, n, j), first, __shfl_sync(kFull, m, j), status);
    }
  }
}

// Streams a warp has in the wide form; up to kSlideOne streams a cluster has all. That is chosen by what a step's call costs the
// host: 36 x 8 x 8 streams called from Python 5.6 us and 8.5, with kvc_page_extend before 13 and 18. By the device's time alone
// (in a graph; the wide form in brackets) it holds up to some 768 streams, 5.4 us (6.8); 2304 take 5.9 (4.0), and where each gives
// up many pages at once, as behind a prompt, 768 streams 12.8 (14.2) with 16 pages, 18.8 (14.3) with 64, 2304 32 (16) with 64.
constexpr int kSlideStreams = 4, kSlideOne = 4096;
__global__ void __launch_bounds__(256) slide_kernel(PoolGeom g, PageTab t, int window, int first, int32_t* gone,
                                                   int32_t* status, PageWs w) {
  griddep_launch();
  griddep_wait();
  const int warps = gridDim.x * (blockDim.x >> 5), wi = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (wi == 0 && threadIdx.x == 0) w.head[0] = *g.nfree;
  slide_streams(g, t, w, wi, warps, window, first, gone, status);
}

__global__ void __cluster_dims__(kOneCtas, 1, 1) __launch_bounds__(kOneThreads)
    slide_one_kernel(PoolGeom g, PageTab t, int window, int first, int32_t* gone, int32_t* status, PageWs w) {
  griddep_launch();
  griddep_wait();
  cg::cluster_group cl = cg::this_cluster();
  const int nfree = *g.nfree;
  cluster_zero(g, w, cl.block_rank() * kOneThreads + threadIdx.x);
  cl.sync();
  slide_streams(g, t, w, (threadIdx.x >> 5) * kOneCtas + cl.block_rank(), kOneCtas * kOneThreads / 32, window, first, gone,
                status);
  cl.sync();
  cluster_push(cl, g, w, nfree);
}

// ---- accepted drafts ------------------------------------------------------------------------------
// kvc_page_compact's steps for lists that name a few tokens behind `base` unmoved ones, a warp a stream: few rows move
// and few entries are looked at, so the plan, the move and the new tables are a chain of some six reads, and two
// launches (or one cluster, barriers between) do instead of four.
//   plan  the path checked, the first row that moves, the destination pages that are shared (refs are read only here)
//   move  fresh pages numbered in stream order, rows moved, entries, counts and lengths set
struct Paths {
  const int32_t *path, *n_path, *n_q;
  int T;
  __device__ __forceinline__ int drafts(int b) const { return n_q ? min(max(n_q[b], 0), T) : T; }
};

__device__ __forceinline__ void accept_plan(const PoolGeom& g, const PageTab& t, const Paths& x, const PageWs& w, int s,
                                            int32_t* status) {
  const int lane = threadIdx.x & 31, b = s / t.Hkv % t.B;
  const int n = t.len[s], nq = x.drafts(b), np = x.n_path[b], base = n - nq, m = base + np;
  const int32_t* path = x.path + (size_t)b * x.T;
  const int32_t* row = t.table + (size_t)s * t.maxp;
  int32_t* to = w.newtab + (size_t)s * t.maxp;
  const bool badlen = n < 0 || n > ((long long)t.maxp << g.lp);
  bool bad = badlen || base < 0 || np < 0 || np > nq;
  int k0 = np;  // the first draft that moves
  if (!bad) {
    for (int k = lane; k < np; k += 32) {
      const int v = path[k], next = k + 1 < np ? path[k + 1] : nq;
      bad |= v < k || v >= next;
      if (v != k && k < k0) k0 = k;
    }
    k0 = __reduce_min_sync(kFull, k0);
    bad = __any_sync(kFull, bad);
  }
  if (bad && lane == 0) status_or(status, badlen ? KVC_STATUS_BAD_PAGE : KVC_STATUS_BAD_INDEX);
  int need = 0, first = base + k0;
  if (!bad) {
    bool missing = false, shared0 = false;
    const int e = pages_of(n, g.lp), pe = k0 < np ? pages_of(m, g.lp) : 0, p0 = first >> g.lp;
    for (int i = p0 + lane; i < e; i += 32) {
      const int p = row[i];
      const bool ok = page_ok(g, p);
      missing |= !ok;
      if (i < pe) {
        const bool shared = ok && g.refs[p] > 1;
        to[i] = shared ? -1 : p;
        need += shared;
        shared0 |= shared && i == p0;
      }
    }
    need = warp_sum_i(need);
    if (__any_sync(kFull, shared0)) first = p0 << g.lp;  // with its page replaced, the unmoved rows go along
    bad = __any_sync(kFull, missing);
    if (bad && lane == 0) status_or(status, KVC_STATUS_BAD_PAGE);
  }
  if (lane == 0) {
    w.need[s] = bad ? 0 : need;
    w.plan[s] = make_int4(first, m, n, bad ? kCompactBad : k0 < np ? kCompactMoves : 0);
  }
}

// Rows [first, m) of a stream by a warp, 16 tokens at a time: a lane holds four of their code vectors (16 bytes) and a
// token's K or V scales. A batch is read before it is written, and lies before every later batch's sources.
template <int D>
__device__ __forceinline__ void accept_rows(const PoolGeom& g, const int32_t* row, const int32_t* to, const int32_t* path,
                                            int base, int first, int m) {
  constexpr int kVec = D / 16, kAt = 32 / kVec, kTok = 16, U = kTok / kAt;  // vectors of a token (K, then V)
  const int lane = threadIdx.x & 31, lmask = (1 << g.lp) - 1, v = lane % kVec, kv = v / (kVec / 2);
  auto code = [&](int page, int tok) {
    return reinterpret_cast<uint4*>(block_of(g, page, (tok & lmask) >> 4) + piece_off(D, 2 * kv) + (tok & 15) * (D / 2)) +
           v % (kVec / 2);
  };
  auto scale = [&](int page, int tok) {
    return block_of(g, page, (tok & lmask) >> 4) + piece_off(D, 1 + 2 * (lane >> 4)) + (tok & 15) * (D / 16);
  };
  for (int k0 = first; k0 < m; k0 += kTok) {
    const int mine = k0 + (lane & 15);
    const int src = mine >= m ? -1 : mine < base ? mine : base + path[mine - base];
    const int ps = src >= 0 ? row[src >> g.lp] : 0, pd = src >= 0 ? to[mine >> g.lp] : 0;
    uint4 c[U];
    uint64_t sc = 0;
    if (src >= 0) {
      if constexpr (D == 128)
        sc = *reinterpret_cast<const uint64_t*>(scale(ps, src));
      else
        sc = *reinterpret_cast<const uint32_t*>(scale(ps, src));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = u * kAt + lane / kVec;
      const int sj = __shfl_sync(kFull, src, j), pj = __shfl_sync(kFull, ps, j);
      if (sj >= 0) c[u] = *code(pj, sj);
    }
    __syncwarp();
    if (src >= 0) {
      if constexpr (D == 128)
        *reinterpret_cast<uint64_t*>(scale(pd, mine)) = sc;
      else
        *reinterpret_cast<uint32_t*>(scale(pd, mine)) = (uint32_t)sc;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = u * kAt + lane / kVec;
      const int pj = __shfl_sync(kFull, pd, j);
      if (k0 + j < m) *code(pj, k0 + j) = c[u];
    }
    __syncwarp();
  }
}

// before: the pages that the streams before this one take
template <int D>
__device__ __forceinline__ void accept_move(const PoolGeom& g, const PageTab& t, const Paths& x, const PageWs& w, int s,
                                            int4 plan, int need, int before, int nfree, int32_t* status) {
  if (plan.w & kCompactBad) return;
  const int lane = threadIdx.x & 31, b = s / t.Hkv % t.B, first = plan.x, m = plan.y, n = plan.z;
  int32_t* row = t.table + (size_t)s * t.maxp;
  int32_t* to = w.newtab + (size_t)s * t.maxp;
  const int pe = pages_of(m, g.lp);
  if (need) {
    int at = nfree - 1 - before;
    bool lost = false;
    for (int i0 = first >> g.lp; i0 < pe; i0 += 32) {
      const int i = i0 + lane;
      const bool want = i < pe && to[i] < 0;
      const unsigned mask = __ballot_sync(kFull, want);
      if (want) {
        const int p = g.free_list[at - __popc(mask & ((1u << lane) - 1))];
        if (page_ok(g, p))
          to[i] = p;
        else
          lost = true;
      }
      at -= __popc(mask);
    }
    if (__any_sync(kFull, lost)) {  // a damaged free list: the stream is left alone
      if (lane == 0) status_or(status, KVC_STATUS_BAD_PAGE);
      return;
    }
    __syncwarp();
  }
  if (plan.w & kCompactMoves) {
    accept_rows<D>(g, row, to, x.path + (size_t)b * x.T, n - x.drafts(b), first, m);
    if (need)
      for (int i = (first >> g.lp) + lane; i < pe; i += 32) {
        const int old = row[i], p = to[i];
        if (p != old) {
          row[i] = p;
          g.refs[p] = 1;
          drop_page(g, w, old, nullptr);
        }
      }
  }
  for (int i = pe + lane; i < pages_of(n, g.lp); i += 32) {
    drop_page(g, w, row[i], nullptr);
    row[i] = -1;
  }
  if (lane == 0) t.len[s] = m;
}

constexpr int kAcceptWarps = 8;
__global__ void __launch_bounds__(32 * kAcceptWarps) accept_plan_kernel(PoolGeom g, PageTab t, Paths x, int32_t* status,
                                                                       PageWs w) {
  griddep_launch();
  griddep_wait();
  const int s = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    w.head[0] = *g.nfree;
    w.head[1] = 0;
  }
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < (g.npages + 31) / 32; i += gridDim.x * blockDim.x) w.gone[i] = 0u;
  if (s < t.S) accept_plan(g, t, x, w, s, status);
}

// The pages that the streams before s take, and all: by 32 * kAcceptWarps threads.
__device__ __forceinline__ void accept_needs(const PageWs& w, int S, int s0, int* sm, int* before, int* total) {
  int b = 0, all = 0;
  for (int i = threadIdx.x; i < S; i += 32 * kAcceptWarps) {
    const int v = w.need[i];
    all += v;
    if (i < s0) b += v;
  }
  *before = *total = 0;
  if (!__syncthreads_or(all)) return;  // nearly always
  *total = block_sum(all, sm);
  *before = block_sum(b, sm);
}

template <int D>
__global__ void __launch_bounds__(32 * kAcceptWarps) accept_move_kernel(PoolGeom g, PageTab t, Paths x, int32_t* status,
                                                                       PageWs w) {
  __shared__ int sm[8];
  griddep_launch();
  griddep_wait();
  const int s0 = blockIdx.x * kAcceptWarps, s = s0 + (threadIdx.x >> 5), nfree = w.head[0];
  const int4 plan = s < t.S ? w.plan[s] : make_int4(0, 0, 0, kCompactBad);
  int before, total;
  accept_needs(w, t.S, s0, sm, &before, &total);
  const bool none = total > 0 && (total > nfree || nfree > g.npages);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (none) status_or(status, KVC_STATUS_NO_PAGES);
    w.head[1] = none ? 0 : total;
  }
  if (none || s >= t.S) return;
  if (total)
    for (int i = s0; i < s; ++i) before += w.need[i];
  accept_move<D>(g, t, x, w, s, plan, w.need[s], before, nfree, status);
}

// Up to kAcceptOne streams: a warp of the cluster has one.
constexpr int kAcceptOne = kOneCtas * kOneThreads / 32;
template <int D>
__global__ void __cluster_dims__(kOneCtas, 1, 1) __launch_bounds__(kOneThreads)
    accept_one_kernel(PoolGeom g, PageTab t, Paths x, int32_t* status, PageWs w) {
  __shared__ int sm[kOneThreads / 32];
  griddep_launch();
  griddep_wait();
  cg::cluster_group cl = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, s = warp * kOneCtas + cl.block_rank(), nfree = *g.nfree;
  cluster_zero(g, w, cl.block_rank() * kOneThreads + threadIdx.x);
  if (s < t.S) accept_plan(g, t, x, w, s, status);
  cl.sync();
  // every stream's need, a thread each
  const int v = (int)threadIdx.x < t.S ? __ldcg(&w.need[threadIdx.x]) : 0;
  int before = 0, total = 0;
  if (__syncthreads_or(v)) {  // hardly ever
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sm[warp] = incl;
    __syncthreads();
    total = warp_sum_i(sm[lane]);
    for (int i = 0; i < kOneThreads / 32; ++i)
      if (i < (s >> 5)) before += sm[i];
    if (s < t.S) {  // the streams before s in its group of 32
      const int y = (s & ~31) + lane < s ? __ldcg(&w.need[(s & ~31) + lane]) : 0;
      before += warp_sum_i(y);
    }
  }
  const bool none = total > 0 && (total > nfree || nfree > g.npages);
  if (cl.block_rank() == 0 && threadIdx.x == 0 && none) status_or(status, KVC_STATUS_NO_PAGES);
  if (none) return;  // every CTA of the cluster alike
  if (s < t.S) accept_move<D>(g, t, x, w, s, w.plan[s], w.need[s], before, nfree, status);
  cl.sync();
  cluster_push(cl, g, w, nfree - total);
}

bool one_fits(const PoolGeom& g, const PageTab& t, const PageTab& o) {
  return g.npages <= kOnePages && (long long)t.S * t.maxp <= kOneEntries && (long long)o.S * o.maxp <= kOneEntries &&
         t.B <= kOneSeqs && o.B <= kOneSeqs;
}

int push_grid(const PoolGeom& g) { return ((g.npages + 31) / 32 + kPushWords - 1) / kPushWords; }

// After a compaction's moves: rows and lengths of a stream, by a warp; its replaced pages and those behind the
// kept rows counted down.
__device__ __forceinline__ void compact_finish(const PoolGeom& g, const PageTab& t, const PageWs& w, int s) {
  const int lane = threadIdx.x & 31;
  const int4 plan = w.plan[s];  // first row written, kept, length, flags
  if (plan.w & kCompactBad) return;
  int32_t* row = t.table + (size_t)s * t.maxp;
  const int32_t* to = w.newtab + (size_t)s * t.maxp;
  const int pe = pages_of(plan.y, g.lp);
  if (w.need[s]) {
    bool lost = false;  // a mark that the free list held no page for
    for (int i = (plan.x >> g.lp) + lane; i < pe; i += 32) lost |= to[i] < 0;
    if (__any_sync(kFull, lost)) return;
    for (int i = (plan.x >> g.lp) + lane; i < pe; i += 32) {
      const int old = row[i], p = to[i];
      if (p != old) {
        row[i] = p;
        g.refs[p] = 1;
        drop_page(g, w, old, nullptr);
      }
    }
  }
  for (int i = pe + lane; i < pages_of(plan.z, g.lp); i += 32) {
    drop_page(g, w, row[i], nullptr);
    row[i] = -1;
  }
  if (lane == 0) t.len[s] = plan.y;
}

// head[1] < 0: too few pages, nothing happened.
__global__ void __launch_bounds__(256) finish_kernel(PoolGeom g, PageTab t, PageWs w) {
  griddep_launch();
  griddep_wait();
  const int s = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (s < t.S && w.head[1] >= 0) compact_finish(g, t, w, s);
}

__global__ void __cluster_dims__(kOneCtas, 1, 1) __launch_bounds__(kOneThreads)
    finish_one_kernel(PoolGeom g, PageTab t, PageWs w) {
  griddep_launch();
  griddep_wait();
  cg::cluster_group cl = cg::this_cluster();
  const int total = w.head[1];
  if (total < 0) return;
  for (int s = (threadIdx.x >> 5) * kOneCtas + cl.block_rank(); s < t.S; s += kOneCtas * kOneThreads / 32)
    compact_finish(g, t, w, s);
  cl.sync();
  cluster_push(cl, g, w, w.head[0] - total);
}
}  // namespace

int page_finish_compact(const PoolGeom& g, const PageTab& t, const PageWs& w, cudaStream_t s) {
  constexpr int kStreams = 64;  // one launch less; with 288 streams the eight SMs take 11.5 us, the two kernels 10
  if (t.S <= kStreams && g.npages <= kOnePages)
    return launch_pdl(finish_one_kernel, dim3(kOneCtas), dim3(kOneThreads), 0, s, false, g, t, w) == cudaSuccess
               ? KVC_OK
               : KVC_ERR_LAUNCH;
  if (launch_pdl(finish_kernel, dim3((t.S + 7) / 8), dim3(256), 0, s, false, g, t, w) != cudaSuccess)
    return KVC_ERR_LAUNCH;
  return page_push(g, w, s);
}

int page_push(const PoolGeom& g, const PageWs& w, cudaStream_t s) {
  return launch_pdl(push_kernel, dim3(push_grid(g)), dim3(kPushThreads), 0, s, false, g, w) == cudaSuccess ? KVC_OK
                                                                                                          : KVC_ERR_LAUNCH;
}

int launch_page_init(const PoolGeom& g, const PageTab* t, cudaStream_t s) {
  PageTab none = {};
  const PageTab& x = t ? *t : none;
  long long n = (long long)x.S * x.maxp;
  if (n < g.npages) n = g.npages;
  if (n < x.S) n = x.S;
  long long grid = (n + 255) / 256;
  if (grid > 4096) grid = 4096;
  return launch_pdl(init_kernel, dim3((unsigned)grid), dim3(256), 0, s, false, g, x) == cudaSuccess ? KVC_OK
                                                                                                   : KVC_ERR_LAUNCH;
}

int launch_page_extend(const PoolGeom& g, const PageTab& t, const int32_t* add, int add_all, int32_t* start,
                       int32_t* status, const PageWs& w, cudaStream_t s) {
  if (t.S <= kOneStreams)
    return launch_pdl(extend_one_kernel, dim3(kOneCtas), dim3(kOneThreads), 0, s, false, g, t, add, add_all, start,
                      status) == cudaSuccess
               ? KVC_OK
               : KVC_ERR_LAUNCH;
  if (launch_pdl(extend_plan_kernel, dim3((t.S + kPlanThreads - 1) / kPlanThreads), dim3(kPlanThreads), 0, s, false, g,
                 t, add, add_all, status, w) != cudaSuccess)
    return KVC_ERR_LAUNCH;
  if (launch_pdl(extend_assign_kernel, dim3((t.S + kAssignStreams - 1) / kAssignStreams), dim3(kAssignThreads), 0, s,
                 false, g, t, add, add_all, start, status, w) != cudaSuccess)
    return KVC_ERR_LAUNCH;
  return KVC_OK;
}

int launch_page_free(const PoolGeom& g, const PageTab& t, const int32_t* drop, int drop_all, int32_t* status,
                     const PageWs& w, cudaStream_t s) {
  if (one_fits(g, t, t))
    return launch_pdl(free_one_kernel, dim3(kOneCtas), dim3(kOneThreads), 0, s, false, g, t, drop, drop_all, status,
                      w) == cudaSuccess
               ? KVC_OK
               : KVC_ERR_LAUNCH;
  if (cudaMemsetAsync(w.head, 0, w.zero_bytes, s) != cudaSuccess) return KVC_ERR_LAUNCH;
  if (launch_pdl(free_kernel, dim3((t.S + 7) / 8), dim3(256), 0, s, false, g, t, drop, drop_all, status, w) !=
      cudaSuccess)
    return KVC_ERR_LAUNCH;
  return page_push(g, w, s);
}

int launch_page_slide(const PoolGeom& g, const PageTab& t, int window, int sinks, int32_t* gone, int32_t* status,
                      const PageWs& w, cudaStream_t s) {
  const int first = (int)(((long long)sinks + (1 << g.lp) - 1) >> g.lp);
  if (t.S <= kSlideOne && g.npages <= kOnePages)
    return launch_pdl(slide_one_kernel, dim3(kOneCtas), dim3(kOneThreads), 0, s, false, g, t, window, first, gone, status,
                      w) == cudaSuccess
               ? KVC_OK
               : KVC_ERR_LAUNCH;
  if (cudaMemsetAsync(w.head, 0, w.zero_bytes, s) != cudaSuccess) return KVC_ERR_LAUNCH;
  const int per = 8 * kSlideStreams;
  if (launch_pdl(slide_kernel, dim3((t.S + per - 1) / per), dim3(256), 0, s, false, g, t, window, first, gone, status, w) !=
      cudaSuccess)
    return KVC_ERR_LAUNCH;
  return page_push(g, w, s);
}

int launch_page_accept(const PoolGeom& g, const PageTab& t, int T, const int32_t* path, const int32_t* n_path,
                       const int32_t* n_q, int32_t* status, const PageWs& w, cudaStream_t s) {
  const Paths x{path, n_path, n_q, T};
  if (t.S <= kAcceptOne && g.npages <= kOnePages)
    return launch_pdl(g.D == 128 ? accept_one_kernel<128> : accept_one_kernel<64>, dim3(kOneCtas), dim3(kOneThreads), 0, s,
                      false, g, t, x, status, w) == cudaSuccess
               ? KVC_OK
               : KVC_ERR_LAUNCH;
  const dim3 grid((t.S + kAcceptWarps - 1) / kAcceptWarps), block(32 * kAcceptWarps);
  if (launch_pdl(accept_plan_kernel, grid, block, 0, s, false, g, t, x, status, w) != cudaSuccess) return KVC_ERR_LAUNCH;
  if (launch_pdl(g.D == 128 ? accept_move_kernel<128> : accept_move_kernel<64>, grid, block, 0, s, false, g, t, x, status,
                 w) != cudaSuccess)
    return KVC_ERR_LAUNCH;
  return page_push(g, w, s);
}

int launch_page_fork(const PoolGeom& g, const PageTab& t, const int32_t* parent, const PageTab& out, int32_t* status,
                     const PageWs& w, cudaStream_t s) {
  if (one_fits(g, t, out))
    return launch_pdl(fork_one_kernel, dim3(kOneCtas), dim3(kOneThreads), 0, s, false, g, t, parent, out, status, w) ==
                   cudaSuccess
               ? KVC_OK
               : KVC_ERR_LAUNCH;
  if (cudaMemsetAsync(w.head, 0, w.zero_bytes, s) != cudaSuccess) return KVC_ERR_LAUNCH;
  if (launch_pdl(fork_kernel, dim3((t.S + out.S + 7) / 8), dim3(256), 0, s, false, g, t, parent, out, status, w) !=
      cudaSuccess)
    return KVC_ERR_LAUNCH;
  return page_push(g, w, s);
}

}  // namespace kvc
