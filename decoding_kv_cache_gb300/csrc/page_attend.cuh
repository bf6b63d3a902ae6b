// page_attend.cuh -- what the kernels of kvc_page_attend share: the streams' work units and their split
// over the CTAs, partial results, and small helpers.
#pragma once

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
  float* part;  // [grid][2][rb][D] (tcgen05 kernel: [grid][2][D][rb])
  float2* ml;   // [grid][2][rb] (reference, sum)
  int2* span;   // [nvs] first and last CTA of a stream's units (streams with units only; negative: that CTA gave up)
};

struct Stream {  // what a (stream, row block) has to see
  int s, b, h, len, nq, r0, rows, vis;
};

__device__ __forceinline__ Stream stream_of(const AttendArgs& a, const AttendPlan& p, int vs, bool report) {
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
__device__ __forceinline__ int units_of(const AttendPlan& p, const Stream& x) { return (x.vis + p.unit - 1) / p.unit; }
__device__ __forceinline__ int cost_of(const AttendPlan& p, const Stream& x) { return x.vis ? units_of(p, x) + p.lead : 0; }

// Cost, in units, before each thread's run of streams and in all (block of kThr threads; every thread calls).
template <int kThr>
__device__ __forceinline__ int scan_units(const AttendArgs& a, const AttendPlan& p, int* sm, int per, int* total) {
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int vs = threadIdx.x * per + i;
    if (vs < p.nvs) mine += cost_of(p, stream_of(a, p, vs, false));
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

// The kernel for many query rows (tcgen05, 128 rows a block).
constexpr int kTcRows = 128, kTcUnit = 128;
int launch_attend_tc(const AttendArgs& a, const AttendPlan& p, cudaStream_t s);

}  // namespace kvc
