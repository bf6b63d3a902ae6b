// page_ops.cu -- pages of the 4-bit cache taken, shared, copied on write and given back.
//
// Every result is a function of the arguments alone: pages are taken from the free list's end in
// stream order, counted with integer atomics (whose order cannot show), and given back in the order
// of their numbers through a bitmap. A call that cannot get all its pages changes nothing.
#include "page.cuh"

namespace kvc {
namespace {

constexpr int kCopyFlag = 1 << 30;
constexpr int kPlanThreads = 256;   // streams per planning CTA
constexpr int kAssignStreams = 32;  // streams per assigning CTA
constexpr int kAssignThreads = 256;
constexpr int kPushThreads = 256;
constexpr int kPushWords = 1024;  // bitmap words per giving-back CTA

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

// Pages each stream takes: the fresh ones behind its last page and, when that page is partly filled
// and shared, a copy of it. Of the streams that share a page and all write to it, the lowest sequence
// keeps it; the sharers of a page are sequences of the same layer and head (forks keep it so), found
// by comparing that page's number over the sequences, for shared last pages only.
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(PoolGeom g, PageTab t, const int32_t* add,
                                                                  int add_all, int32_t* status, PageWs w) {
  __shared__ int sm[8];
  griddep_wait();
  const int s = blockIdx.x * kPlanThreads + threadIdx.x;
  int need = 0;
  if (s < t.S) {
    const int h = s % t.Hkv, b = s / t.Hkv % t.B, l = s / (t.Hkv * t.B);
    const int a = add ? add[b] : add_all;
    int n;
    if (!extend_wants(g, t, s, a, &n, status)) {
      need = -1;
    } else if (a > 0) {
      need = pages_of(n + a, g.lp) - pages_of(n, g.lp);
      if (n & ((1 << g.lp) - 1)) {
        const int p = t.table[(size_t)s * t.maxp + (n >> g.lp)];
        if (!page_ok(g, p)) {
          status_or(status, KVC_STATUS_BAD_PAGE);
          need = -1;
        } else {
          const int r = g.refs[p];
          if (r > 1) {
            int writers = 0, lowest = b;
            for (int o = 0; o < t.B; ++o) {
              const int so = (l * t.B + o) * t.Hkv + h;
              const int ao = add ? add[o] : add_all, no = t.len[so];
              if (ao <= 0 || no <= 0 || no + (long long)ao > ((long long)t.maxp << g.lp) || !(no & ((1 << g.lp) - 1))) continue;
              if (t.table[(size_t)so * t.maxp + (no >> g.lp)] != p) continue;
              ++writers;
              if (o < lowest) lowest = o;
            }
            if (!(lowest == b && writers >= r)) need = (need + 1) | kCopyFlag;
          }
        }
      }
    }
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

__device__ __forceinline__ void copy_page(const PoolGeom& g, int dst, int src, int lane, int lanes) {
  const size_t bytes = (size_t)blk_bytes(g.D) << (g.lp - 4);
  uint4* d = reinterpret_cast<uint4*>(g.data + (size_t)dst * bytes);
  const uint4* x = reinterpret_cast<const uint4*>(g.data + (size_t)src * bytes);
  const int n = (int)(bytes / 16);
  for (int i = lane; i < n; i += 4 * lanes) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * lanes < n) v[u] = x[i + u * lanes];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * lanes < n) d[i + u * lanes] = v[u];
  }
}

// The pages handed out: 32 streams a CTA, a warp per stream in turn; the copies go with them.
__global__ void __launch_bounds__(kAssignThreads) extend_assign_kernel(PoolGeom g, PageTab t, const int32_t* add,
                                                                      int add_all, int32_t* start, int32_t* status,
                                                                      PageWs w) {
  __shared__ int sm[8];
  griddep_wait();
  const int s0 = blockIdx.x * kAssignStreams, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  int incl = s0 + lane < t.S ? need_of(w, s0 + lane) : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  for (int i = warp; i < kAssignStreams; i += kAssignThreads / 32) {
    const int s = s0 + i;
    if (s >= t.S) break;
    const int need = w.need[s];
    if (none || need < 0) {
      if (lane == 0 && start) start[s] = -1;
      continue;
    }
    const int b = s / t.Hkv % t.B;
    const int a = add ? add[b] : add_all, n = t.len[s];
    const int end = __shfl_sync(kFull, incl, i);
    const int k = need & ~kCopyFlag;
    const int copy = need & kCopyFlag ? 1 : 0;
    int at = nfree - 1 - (before + end - k);  // free-list slot of the stream's first page
    int32_t* row = t.table + (size_t)s * t.maxp;
    if (copy) {
      const int old = row[n >> g.lp], p = g.free_list[at];
      if (page_ok(g, p)) copy_page(g, p, old, lane, 32);
      __syncwarp();
      if (lane == 0) {
        row[n >> g.lp] = p;
        if (page_ok(g, p)) g.refs[p] = 1;
        atomicSub(&g.refs[old], 1);
      }
    }
    const int first = pages_of(n, g.lp);
    for (int j = lane; j < k - copy; j += 32) {
      const int p = g.free_list[at - copy - j];
      row[first + j] = p;
      if (page_ok(g, p)) g.refs[p] = 1;
    }
    __syncwarp();
    if (lane == 0) {
      t.len[s] = n + a;
      if (start) start[s] = n;
    }
  }
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

// The marked pages join the free list in the order of their numbers. Each CTA counts the marks before
// its words itself (the bitmap is small and in L2), so no CTA waits for another.
__global__ void __launch_bounds__(kPushThreads) push_kernel(PoolGeom g, PageWs w) {
  __shared__ int sm[8];
  griddep_wait();
  const int words = (g.npages + 31) / 32, w0 = blockIdx.x * kPushWords;
  int c = 0;
  const uint4* g4 = reinterpret_cast<const uint4*>(w.gone);
  for (int i = threadIdx.x; i < w0 / 4; i += kPushThreads) {
    const uint4 v = g4[i];
    c += __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
  }
  const int base = block_sum(c, sm);
  // this CTA's words, four neighbours a thread
  uint32_t m[4];
  int mine = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = w0 + 4 * threadIdx.x + u;
    m[u] = i < words ? w.gone[i] : 0u;
    mine += __popc(m[u]);
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  __syncthreads();
  if (lane == 31) sm[warp] = incl;
  __syncthreads();
  int at = base + incl - mine, all = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < warp) at += sm[i];
    all += sm[i];
  }
  const int nfree = w.head[0] - (w.head[2] ? 0 : w.head[1]);  // what the call took is off the list's end
#pragma unroll
  for (int u = 0; u < 4; ++u)
    for (uint32_t v = m[u]; v; v &= v - 1) {
      const int to = nfree + at++;
      if (to >= 0 && to < g.npages) g.free_list[to] = (w0 + 4 * threadIdx.x + u) * 32 + __ffs(v) - 1;
    }
  if (w0 + kPushWords >= words && threadIdx.x == 0) *g.nfree = nfree + base + all;
}

int push_grid(const PoolGeom& g) { return ((g.npages + 31) / 32 + kPushWords - 1) / kPushWords; }

}  // namespace

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
  if (cudaMemsetAsync(w.head, 0, w.zero_bytes, s) != cudaSuccess) return KVC_ERR_LAUNCH;
  if (launch_pdl(free_kernel, dim3((t.S + 7) / 8), dim3(256), 0, s, false, g, t, drop, drop_all, status, w) !=
      cudaSuccess)
    return KVC_ERR_LAUNCH;
  return page_push(g, w, s);
}

int launch_page_fork(const PoolGeom& g, const PageTab& t, const int32_t* parent, const PageTab& out, int32_t* status,
                     const PageWs& w, cudaStream_t s) {
  if (cudaMemsetAsync(w.head, 0, w.zero_bytes, s) != cudaSuccess) return KVC_ERR_LAUNCH;
  if (launch_pdl(fork_kernel, dim3((t.S + out.S + 7) / 8), dim3(256), 0, s, false, g, t, parent, out, status, w) !=
      cudaSuccess)
    return KVC_ERR_LAUNCH;
  return page_push(g, w, s);
}

}  // namespace kvc
