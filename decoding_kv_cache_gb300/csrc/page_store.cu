// page_store.cu -- rows into the paged 4-bit cache and back out of it.
//
// A group of 16 channels x of a row, with the pool's tensor scale ts:
//   scale = e4m3(clamp(max|x| / (6 ts), 2^-9, 448)), round to nearest even
//   code  = the e2m1 nearest to x / (scale ts), ties to the even code, beyond 6: 6
// Both decisions are those of the exact quotient. 16-bit inputs meet borders exactly and often, and a
// quotient rounded to fp32 first would fall to a neighbour's side: the scale's quotient is truncated
// and its lowest bit set when anything was cut off (so rounding it again to e4m3 is the exact
// quotient's rounding), and the code counts the borders b with |x| > b * (scale ts), b and the scale
// having three and four bits, which makes the product exact when ts is a power of two.
// A thread owns a group: two 16-byte loads (bf16), 8 bytes of codes, 1 of scale. Memory-bound:
// 2.56 bytes a value moved for bf16.
#include "page.cuh"

namespace kvc {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]) {
  constexpr int per = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < 16 / per; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int u = 0; u < per; ++u) x[i * per + u] = to_f32(e[u]);
  }
}

// codes (8 bytes, even channel in the low nibble) and scale of one group
__device__ __forceinline__ uint2 quantise16(const float (&x)[16], float ts, uint32_t* scale) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));  // a NaN takes no part
  const float den = 6.f * ts;
  float want = __fdiv_rz(amax, den);
  if (__fmaf_rn(-want, den, amax) != 0.f && want < 448.f) want = __uint_as_float(__float_as_uint(want) | 1u);
  want = fminf(fmaxf(want, 0.001953125f), 448.f);
  const uint32_t sb = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
  *scale = sb;
  const float step = e4m3_f32(sb) * ts;
  const float b0 = 0.25f * step, b1 = 0.75f * step, b2 = 1.25f * step, b3 = 1.75f * step, b4 = 2.5f * step,
              b5 = 3.5f * step, b6 = 5.f * step;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float a = fabsf(x[i]);
    uint32_t c = (a > b0) + (a >= b1) + (a > b2) + (a >= b3) + (a > b4) + (a >= b5) + (a > b6);
    c |= x[i] < 0.f ? 8u : 0u;
    w[i / 8] |= c << (4 * (i % 8));
  }
  return make_uint2(w[0], w[1]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) store_kernel(StoreArgs a) {
  griddep_wait();
  constexpr int kGroups = D / 16;
  const long long item = (long long)blockIdx.x * (kThreads / kGroups) + threadIdx.x / kGroups;
  const int grp = threadIdx.x % kGroups;
  const long long rows = (long long)a.t.S * a.T;
  if (item >= 2 * rows) return;
  const int kv = item >= rows;
  const long long r = item - (kv ? rows : 0);
  const int s = (int)(r / a.T), tok = (int)(r % a.T);
  const int h = s % a.t.Hkv, b = s / a.t.Hkv;
  if (a.n && tok >= a.n[b]) return;
  const int st = a.start[s];
  if (st < 0) return;  // the extension did not take place
  const long long pos = (long long)st + tok;
  if (pos >= a.t.len[s] || pos >= ((long long)a.t.maxp << a.g.lp)) {
    status_or(a.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  const int p = a.t.table[(size_t)s * a.t.maxp + (pos >> a.g.lp)];
  if (!page_ok(a.g, p) || a.g.refs[p] != 1) {
    status_or(a.status, KVC_STATUS_BAD_PAGE);
    return;
  }
  const RowStrides& xs = a.xs[kv];
  float x[16];
  load16(static_cast<const T*>(a.x[kv]) + b * xs.b + tok * xs.t + h * xs.h + 16 * grp, x);
  uint32_t sc;
  const uint2 c = quantise16(x, a.g.ts[kv], &sc);
  const int in = (int)(pos & ((1 << a.g.lp) - 1));
  uint8_t* blk = block_of(a.g, p, in >> 4);
  *reinterpret_cast<uint2*>(blk + piece_off(D, 2 * kv) + (in & 15) * (D / 2) + 8 * grp) = c;
  blk[piece_off(D, 2 * kv + 1) + (in & 15) * (D / 16) + grp] = (uint8_t)sc;
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&x)[16]) {
  constexpr int per = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < 16 / per; ++i) {
    uint4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int u = 0; u < per; ++u) e[u] = from_f32<T>(x[i * per + u]);
    reinterpret_cast<uint4*>(p)[i] = v;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(ReadArgs a) {
  griddep_wait();
  constexpr int kGroups = D / 16;
  const long long rows = (long long)a.t.S * a.count;
  const long long item = (long long)blockIdx.x * (kThreads / kGroups) + threadIdx.x / kGroups;
  const int grp = threadIdx.x % kGroups;
  const int both = a.out[0] && a.out[1];
  if (item >= (both ? 2 * rows : rows)) return;
  const int kv = both ? item >= rows : a.out[0] == nullptr;
  const long long r = both && kv ? item - rows : item;
  const int s = (int)(r / a.count), i = (int)(r % a.count);
  const int f = a.first ? a.first[s] : a.first_all;
  const long long pos = (long long)f + i;
  if (f < 0 || pos >= a.t.len[s] || pos >= ((long long)a.t.maxp << a.g.lp)) return;
  const int p = a.t.table[(size_t)s * a.t.maxp + (pos >> a.g.lp)];
  if (!page_ok(a.g, p)) {
    status_or(a.status, KVC_STATUS_BAD_PAGE);
    return;
  }
  const int in = (int)(pos & ((1 << a.g.lp) - 1));
  const uint8_t* blk = block_of(a.g, p, in >> 4);
  const uint2 c = *reinterpret_cast<const uint2*>(blk + piece_off(D, 2 * kv) + (in & 15) * (D / 2) + 8 * grp);
  const float step = e4m3_f32(blk[piece_off(D, 2 * kv + 1) + (in & 15) * (D / 16) + grp]) * a.g.ts[kv];
  float x[16];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t v[4];
    e2m1x8_f16(u ? c.y : c.x, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = f16x2_f32(v[e]);
      x[8 * u + 2 * e] = y.x * step;
      x[8 * u + 2 * e + 1] = y.y * step;
    }
  }
  store16(static_cast<T*>(a.out[kv]) + ((size_t)s * a.ncap + i) * D + 16 * grp, x);
}

template <typename A>
int go(void (*k)(A), const A& a, long long items, int D, cudaStream_t s) {
  const long long per = kThreads / (D / 16);
  const long long grid = (items + per - 1) / per;
  if (grid > 0x7fffffffLL) return KVC_ERR_TOO_LARGE;
  return launch_pdl(k, dim3((unsigned)grid), dim3(kThreads), 0, s, false, a) == cudaSuccess ? KVC_OK : KVC_ERR_LAUNCH;
}

}  // namespace

int launch_page_store(const StoreArgs& a, int dtype, cudaStream_t s) {
  const long long items = 2LL * a.t.S * a.T;
  if (dtype == KVC_BF16)
    return go(a.g.D == 128 ? store_kernel<__nv_bfloat16, 128> : store_kernel<__nv_bfloat16, 64>, a, items, a.g.D, s);
  return go(a.g.D == 128 ? store_kernel<float, 128> : store_kernel<float, 64>, a, items, a.g.D, s);
}

int launch_page_read(const ReadArgs& a, int dtype, cudaStream_t s) {
  const long long items = (a.out[0] && a.out[1] ? 2LL : 1LL) * a.t.S * a.count;
  if (dtype == KVC_BF16)
    return go(a.g.D == 128 ? read_kernel<__nv_bfloat16, 128> : read_kernel<__nv_bfloat16, 64>, a, items, a.g.D, s);
  return go(a.g.D == 128 ? read_kernel<float, 128> : read_kernel<float, 64>, a, items, a.g.D, s);
}

}  // namespace kvc
