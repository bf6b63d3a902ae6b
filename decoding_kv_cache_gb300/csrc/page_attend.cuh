// page_attend.cuh -- what the kernels of kvc_page_attend share: the streams' work units and their split
// over the CTAs, partial results, and small helpers.
#pragma once

#include <type_traits>

#include "page.cuh"
#include "tc_ptx.cuh"

namespace kvc {

constexpr float kOff = 10.f;   // probabilities are held times 2^10 (fp16's range is used below the maximum too)
constexpr float kRaise = 5.f;  // a reference may lag the maximum by 2^5: 2^15 at most, inside fp16

struct AttendPlan {
  int unit;    // tokens of a work unit
  int lead;    // units that beginning a stream's part counts for, when the work is split
  int nrb;     // row blocks per stream
  int rb, lrb;  // rows per block (a power of two) and its logarithm
  int G;
  int nvs;     // streams * nrb
  FastDiv by_nrb, by_hkv, by_G;
  int grid;    // CTAs of the main kernel
  int whole;   // a CTA takes a whole stream: no parts, no second kernel
  int ctas;    // under SeenArgs, whole: a cluster of so many CTAs does
  float* part;  // [grid][2][rb][D] (tcgen05 kernels: [grid][2][D][rb], under SeenArgs in part_at's order)
  float2* ml;   // [grid][2][rb] (reference, sum)
  int2* span;   // [nvs] first and last CTA of a stream's units (streams with units only; negative: that CTA gave up)
};

struct Stream {  // what a (stream, row block) has to see
  int s, b, h, len, nq, r0, rows, vis;
  // Under SeenArgs the tokens that no row of the block sees, between the sinks and the windows, are left out in
  // whole 16-token blocks: len, vis and every token number count without them, and token v lies in the cache at
  // real(v). With skip > 0 the sinks end at or before `at` and every row's window begins at or behind it.
  int at, skip, sinks;
  __device__ __forceinline__ int real(int v) const { return v < at ? v : v + skip; }
};

struct Causal {};  // what the rows of kvc_page_attend see: SeenArgs' place there
template <typename M>
constexpr bool kPart = !std::is_same<M, Causal>::value;

template <typename M>
__device__ __forceinline__ Stream stream_of(const AttendArgs& a, const AttendPlan& p, const M& m, int vs, bool report) {
  Stream x;
  x.s = p.by_nrb.div(vs);
  x.r0 = (vs - x.s * p.nrb) * p.rb;
  x.b = p.by_hkv.div(x.s);
  x.h = x.s - x.b * a.t.Hkv;
  x.len = a.t.len[x.s];
  x.nq = a.n_q ? min(max(a.n_q[x.b], 0), a.T) : a.T;
  if (x.len < 0 || x.len > ((long long)a.t.maxp << a.g.lp)) {
    if (report) status_or(a.status, KVC_STATUS_BAD_PAGE);
    x.len = 0;
  }
  x.rows = max(0, min(p.rb, x.nq * p.G - x.r0));
  const int tmax = min(p.by_G.div(x.r0 + p.rb - 1), x.nq - 1);
  x.vis = x.rows ? max(0, x.len - x.nq + tmax + 1) : 0;
  if constexpr (kPart<M>) {
    const int base = x.len - x.nq;
    if (m.mask && x.rows) x.vis = x.len;
    int lo = max(0, base + (m.depth ? 0 : p.by_G.div(x.r0)) - m.window + 1);  // no row's window begins before it
    if (m.mask) lo = min(lo, max(base, 0));  // of the own tokens any may be seen
    const int sinks = min(m.sinks, lo);
    x.at = (sinks + kBlkTok - 1) & -kBlkTok;
    x.skip = x.vis ? max(0, (lo & -kBlkTok) - x.at) : 0;
    x.sinks = x.skip ? sinks : m.sinks;
    x.len -= x.skip;
    x.vis -= x.skip;
  }
  return x;
}
// Row r of a stream's block: its query token and, with it, offsets in q and out.
__device__ __forceinline__ long long q_row(const AttendArgs& a, const AttendPlan& p, const Stream& x, int r) {
  const int t = p.by_G.div(r);
  return x.b * a.qs.b + t * a.qs.t + (x.h * p.G + r - t * p.G) * a.qs.h;
}
__device__ __forceinline__ size_t out_row(const AttendArgs& a, const AttendPlan& p, const Stream& x, int r) {
  const int t = p.by_G.div(r);
  return ((size_t)x.b * a.T + t) * a.Hq + x.h * p.G + r - t * p.G;
}
// tokens that row r sees
__device__ __forceinline__ int seen_by(const AttendPlan& p, const Stream& x, int r) {
  return min(max(x.len - x.nq + p.by_G.div(r) + 1, 0), x.vis);
}
// Under SeenArgs row r sees the tokens below x.sinks and those from lo on, up to hi, and under a mask the own tokens,
// from `base` on, whose bits its words have set.
struct RowSeen {
  int lo, hi;
};
__device__ __forceinline__ RowSeen row_seen(const AttendArgs& a, const AttendPlan& p, const SeenArgs& m, const Stream& x,
                                            int r) {
  const int base = x.len - x.nq, i = p.by_G.div(r);
  const int d = m.depth ? min(max(m.depth[(size_t)x.b * a.T + i], 0), x.nq - 1) : i;
  return RowSeen{max(0, base + d - m.window + 1), m.mask ? max(base, 0) : seen_by(p, x, r)};
}
// Every row of the block sees all tokens of [lo, hi).
__device__ __forceinline__ RowSeen all_see(const AttendPlan& p, const SeenArgs& m, const Stream& x) {
  const int base = x.len - x.nq, last = m.depth ? x.nq - 1 : min(p.by_G.div(x.r0 + p.rb - 1), x.nq - 1);
  return RowSeen{max(0, base + last - m.window + 1), m.mask ? max(base, 0) : seen_by(p, x, x.r0)};
}
__device__ __forceinline__ const uint32_t* mask_words(const AttendArgs& a, const AttendPlan& p, const SeenArgs& m,
                                                      const Stream& x, int r) {
  return m.mask + ((size_t)x.b * a.T + p.by_G.div(r)) * m.words;
}
__device__ __forceinline__ int units_of(const AttendPlan& p, const Stream& x) { return (x.vis + p.unit - 1) / p.unit; }
__device__ __forceinline__ int cost_of(const AttendPlan& p, const Stream& x) { return x.vis ? units_of(p, x) + p.lead : 0; }

// Cost, in units, before each thread's run of streams, of it (own) and in all (block of kThr threads; every thread calls).
template <int kThr, typename M>
__device__ __forceinline__ int scan_units(const AttendArgs& a, const AttendPlan& p, const M& m, int* sm, int per,
                                          int* total, int* own = nullptr) {
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int vs = threadIdx.x * per + i;
    if (vs < p.nvs) mine += cost_of(p, stream_of(a, p, m, vs, false));
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if ((threadIdx.x & 31) >= o) incl += v;
  }
  if ((threadIdx.x & 31) == 31) sm[threadIdx.x >> 5] = incl;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kThr / 32; ++i) {
    const int v = sm[i];
    if (i < (int)(threadIdx.x >> 5)) base += v;
    all += v;
  }
  *total = all;
  if (own) *own = mine;
  return base + incl - mine;
}

// CTA i of `grid` takes [first(i), first(i + 1)) of the cost W, units and streams' leads: the first W % grid CTAs one more than the others.
struct Split {
  int q, rem;
  __device__ __forceinline__ Split(int W, int grid) : q(W / grid), rem(W % grid) {}
  __device__ __forceinline__ int first(int i) const { return i * q + min(i, rem); }
  __device__ __forceinline__ int owner(int u) const {
    const int big = rem * (q + 1);
    return u < big ? u / (q + 1) : rem + (u - big) / q;
  }
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                   tc::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ uint32_t hmul2(uint32_t x, uint32_t y) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Under SeenArgs a row's probability of a token that it does not see is 0, whatever the token's bytes: a V scale that the
// store does not write (NaN, below zero) counts as zero.
__device__ __forceinline__ uint32_t at_least2(uint32_t x, uint32_t least) {  // the other operand where one is no number
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&least));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t no_nan2(uint32_t x) { return at_least2(x, 0u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// two fp32 operations in one issue
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 w, x, y;\n"
      " mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// One poll of a barrier in line; the waiting out of line, so that the loops stay short. A poll suspends the
// thread for as long as the hardware likes, so the waits are bounded by the clock (false when they give up), and
// the vote keeps a warp together: no lane may leave a loop whose other lanes then wait for it.
constexpr uint64_t kWaitNs = 1000000000;
__device__ __forceinline__ uint64_t clock_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;\n" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool mbar_ready(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(tc::smem_u32(bar)), "r"(parity)
      : "memory");
  return done;
}
// by whole warps; gave_up() says that nothing will come any more
template <typename F>
__device__ __forceinline__ bool mbar_wait_until(uint64_t* bar, uint32_t parity, F&& gave_up) {
  uint64_t since = 0;
  while (!__any_sync(kFull, gave_up())) {
    for (int i = 0; i < 256; ++i)
      if (__all_sync(kFull, mbar_ready(bar, parity))) return true;
    const uint64_t now = clock_ns();
    if (since == 0) since = now;
    if (__any_sync(kFull, now - since > kWaitNs)) return false;
  }
  return false;
}
__device__ __noinline__ static bool mbar_wait_far(uint64_t* bar, uint32_t parity) {
  return mbar_wait_until(bar, parity, [] { return false; });
}

// The kernels for many query rows (tcgen05): 128 rows a block, under SeenArgs 128 or 256.
constexpr int kTcRows = 128, kTcUnit = 128;
int launch_attend_tc(const AttendArgs& a, const AttendPlan& p, cudaStream_t s);
int launch_attend_rows(const AttendArgs& a, const AttendPlan& p, const SeenArgs& m, cudaStream_t s);

// Where the tcgen05 kernel under SeenArgs leaves channel k of a part's row: eight channels of a row together, the rows
// side by side, so that a thread with a row moves 32 bytes at a time and a warp one run of 1 KB (a channel's rows side by
// side, 4 bytes a thread: 64 drafts x 7 rows 70.5 us and not 69.0, 16 x 5 over 8 x 8 x 32768 123.5 and not 122.3).
template <int ROWS>
__device__ __forceinline__ int part_at(int k, int row) {
  return ((k >> 3) * ROWS + row) * 8 + (k & 7);
}
__device__ __forceinline__ void st_f8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void ld_f8(float* v, const float* p) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p));
}

}  // namespace kvc
