// page_store.cu -- rows into the paged 4-bit cache and back out of it.
//
// A group of 16 channels x of a row, with the pool's tensor scale ts:
//   scale = e4m3(clamp(max|x| / (6 ts), 2^-9, 448)), round to nearest even
//   code  = the e2m1 nearest to x / (scale ts), ties to the even code, beyond 6: 6
// Both decisions are those of the exact quotient by the fp32 numbers 6 ts and scale ts. 16-bit inputs
// meet borders exactly and often, and a quotient rounded to fp32 first would fall to a neighbour's side:
// the scale's quotient is truncated and its lowest bit set when anything was cut off (so rounding it
// again to e4m3 is the exact quotient's rounding); the code is found by halving, each border b by the
// sign of fma(-b, scale ts, |x|), which is that of the exact difference.
// For bf16 rows and ts a power of two there is a shorter way. With integers X <= 255 and m <= 15 every
// quotient decided here is X 2^k / 6 (a scale) or X 2^k / m (a code): it either is a border or misses it by
// more than 2^-10.7 of it, and the borders between codes are multiples of 1/4. So products with rounded
// reciprocals (off by less than 2^-20), rounded to 12 bits for the scale and to a multiple of 2^-13 for the
// codes (an fma onto 1536, taken off again), lie on the quotient's side of every border, and on it where the
// quotient does; the hardware's e4m3 and e2m1 conversions then decide as the exact quotients would.
// A thread owns a group: two 16-byte loads (bf16), 8 bytes of codes, 1 of scale. Memory-bound:
// 2.56 bytes a value moved for bf16.
#include "page.cuh"

namespace kvc {
namespace {

constexpr int kThreads = 256;

// 16 values of a row as they lie in memory
template <typename T>
struct Raw {
  uint4 v[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void unpack16(const Raw<T>& r, float (&x)[16]) {
  const T* e = reinterpret_cast<const T*>(r.v);
#pragma unroll
  for (int u = 0; u < 16; ++u) x[u] = to_f32(e[u]);
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN wins
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Codes (8 bytes, even channel in the low nibble) and scale of one group; NaNs count as 0, and what rounds to
// zero has no sign.
__device__ __forceinline__ uint2 quantise16(float (&x)[16], float ts, uint32_t* scale) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (x[i] != x[i]) x[i] = 0.f;
    amax = fmaxf(amax, fabsf(x[i]));
  }
  const float den = 6.f * ts;
  float want = __fdiv_rz(amax, den);
  if (__fmaf_rn(-want, den, amax) != 0.f && want < 448.f) want = __uint_as_float(__float_as_uint(want) | 1u);
  want = fminf(fmaxf(want, 0.001953125f), 448.f);
  const uint32_t sb = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
  *scale = sb;
  const float step = e4m3_f32(sb) * ts;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = fabsf(x[i]);
    const bool c2 = __fmaf_rn(-1.75f, step, v) >= 0.f;
    const bool c1 = __fmaf_rn(c2 ? -3.5f : -0.75f, step, v) >= 0.f;
    const bool c0 = __fmaf_rn(c2 ? (c1 ? -5.f : -2.5f) : (c1 ? -1.25f : -0.25f), step, v) > 0.f;
    uint32_t c = (c2 ? 4u : 0u) | (c1 ? 2u : 0u) | (c0 ? 1u : 0u);
    if (c) c |= __float_as_uint(x[i]) >> 28 & 8u;
    w[i / 8] |= c << (4 * (i % 8));
  }
  return make_uint2(w[0], w[1]);
}

// The short way (see above): inv6 = 1 / (6 ts), ts a power of two.
__device__ __forceinline__ uint2 quantise16_snap(const uint4 (&raw)[2], float ts, float inv6, uint32_t* scale) {
  uint32_t h[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
  auto pair = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); };
  __nv_bfloat162 m = __habs2(pair(h[0]));
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(pair(h[i])));
  float amax = max_nan(__low2float(m), __high2float(m));
  if (amax != amax) {
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((h[i] & 0x7fffu) > 0x7f80u) h[i] &= 0xffff0000u;
      if ((h[i] & 0x7fff0000u) > 0x7f800000u) h[i] &= 0xffffu;
      amax = fmaxf(amax, fmaxf(fabsf(__low2float(pair(h[i]))), fabsf(__high2float(pair(h[i])))));
    }
  }
  float want = fminf(fmaxf(amax * inv6, 0.001953125f), 448.f);
  want = __uint_as_float((__float_as_uint(want) + 0x400u) & ~0x7ffu);
  const uint32_t sb = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
  *scale = sb;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(e4m3_f32(sb) * ts));
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float y[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t v = h[4 * i + u];
      y[2 * u] = __fadd_rn(__fmaf_rn(__uint_as_float(v << 16), r, 1536.f), -1536.f);
      y[2 * u + 1] = __fadd_rn(__fmaf_rn(__uint_as_float(v & 0xffff0000u), r, 1536.f), -1536.f);
    }
    asm("{\n .reg .b8 b0, b1, b2, b3;\n cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n mov.b32 %0, {b0, b1, b2, b3};\n}\n"
        : "=r"(w[i])
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    const uint32_t some = (w[i] | w[i] >> 1 | w[i] >> 2) & 0x11111111u;  // codes that are not zero
    w[i] &= 0x77777777u | some << 3;
  }
  return make_uint2(w[0], w[1]);
}

// Where an item (a row of K or V: K's rows first) lies.
template <typename Index>
struct Item {
  int kv, s, tok;
  __device__ __forceinline__ Item(Index item, Index rows, const FastDiv& by_T, bool both, int only) {
    kv = both ? item >= rows : only;
    const Index r = both && kv ? item - rows : item;
    s = sizeof(Index) == 4 ? by_T.div((int)r) : (int)(r / by_T.d);
    tok = (int)(r - (Index)s * (Index)by_T.d);
  }
};

// A thread takes one group of a row (with two, four or eight rows a thread the registers cost more warps than
// the reads in flight gain: 42.0 us stored and read back with four, 38.8 with one). Index: 32 bits wherever
// the rows fit, where no division is left.
template <typename T, int D, bool SNAP, typename Index>
__global__ void __launch_bounds__(kThreads) store_kernel(StoreArgs a) {
  griddep_launch();
  griddep_wait();
  constexpr int kGroups = D / 16, kRows = kThreads / kGroups;
  const int grp = threadIdx.x % kGroups;
  const Index rows = (Index)a.t.S * a.T, item = (Index)blockIdx.x * kRows + threadIdx.x / kGroups;
  if (item >= 2 * rows) return;
  const Item<Index> it(item, rows, a.by_T, true, 0);
  const int b = a.by_hkv.div(it.s), h = it.s - b * a.t.Hkv;
  const RowStrides& xs = it.kv ? a.xs[1] : a.xs[0];
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(it.kv ? a.x[1] : a.x[0]) + b * xs.b +
                                                    it.tok * xs.t + h * xs.h + 16 * grp);
  Raw<T> raw;  // on its way while the token's place is found
#pragma unroll
  for (int u = 0; u < (int)sizeof(T); ++u) raw.v[u] = __ldg(src + u);
  if (a.n && it.tok >= a.n[b]) return;
  const int st = a.start[it.s];
  if (st < 0) return;  // the extension did not take place
  const long long pos = (long long)st + it.tok;
  if (pos >= a.t.len[it.s] || pos >= ((long long)a.t.maxp << a.g.lp)) {
    status_or(a.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  const int p = a.t.table[(size_t)it.s * a.t.maxp + (pos >> a.g.lp)];
  if (!page_ok(a.g, p) || a.g.refs[p] != 1) {
    status_or(a.status, KVC_STATUS_BAD_PAGE);
    return;
  }
  const int in = (int)(pos & ((1 << a.g.lp) - 1));
  uint8_t* blk = block_of(a.g, p, in >> 4);
  uint32_t sc;
  uint2 c;
  const float ts = it.kv ? a.g.ts[1] : a.g.ts[0];
  if constexpr (SNAP) {
    c = quantise16_snap(raw.v, ts, it.kv ? a.inv6[1] : a.inv6[0], &sc);
  } else {
    float x[16];
    unpack16<T>(raw, x);
    c = quantise16(x, ts, &sc);
  }
  *reinterpret_cast<uint2*>(blk + (it.kv ? piece_off(D, 2) : 0) + (in & 15) * (D / 2) + 8 * grp) = c;
  blk[(it.kv ? piece_off(D, 3) : piece_off(D, 1)) + (in & 15) * (D / 16) + grp] = (uint8_t)sc;
}

template <typename T, int D, typename Index>
__global__ void __launch_bounds__(kThreads) read_kernel(ReadArgs a) {
  griddep_launch();
  griddep_wait();
  constexpr int kGroups = D / 16, kRows = kThreads / kGroups;
  const int grp = threadIdx.x % kGroups;
  const bool both = a.out[0] && a.out[1];
  const Index rows = (Index)a.t.S * a.count, item = (Index)blockIdx.x * kRows + threadIdx.x / kGroups;
  if (item >= (both ? 2 * rows : rows)) return;
  const Item<Index> it(item, rows, a.by_count, both, a.out[0] == nullptr);
  const int f = a.first ? a.first[it.s] : a.first_all;
  const long long pos = (long long)f + it.tok;
  if (f < 0 || pos >= a.t.len[it.s] || pos >= ((long long)a.t.maxp << a.g.lp)) return;
  const int p = a.t.table[(size_t)it.s * a.t.maxp + (pos >> a.g.lp)];
  if (!page_ok(a.g, p)) {
    status_or(a.status, KVC_STATUS_BAD_PAGE);
    return;
  }
  const int in = (int)(pos & ((1 << a.g.lp) - 1));
  const uint8_t* blk = block_of(a.g, p, in >> 4);
  const uint2 c = *reinterpret_cast<const uint2*>(blk + (it.kv ? piece_off(D, 2) : 0) + (in & 15) * (D / 2) + 8 * grp);
  const float step = e4m3_f32(blk[(it.kv ? piece_off(D, 3) : piece_off(D, 1)) + (in & 15) * (D / 16) + grp]) *
                     (it.kv ? a.g.ts[1] : a.g.ts[0]);
  Raw<T> y;
  T* e = reinterpret_cast<T*>(y.v);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t v[4];
    e2m1x8_f16(u ? c.y : c.x, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 z = f16x2_f32(v[k]);
      e[8 * u + 2 * k] = from_f32<T>(z.x * step);
      e[8 * u + 2 * k + 1] = from_f32<T>(z.y * step);
    }
  }
  uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(it.kv ? a.out[1] : a.out[0]) + ((size_t)it.s * a.ncap + it.tok) * D +
                                       16 * grp);
#pragma unroll
  for (int u = 0; u < (int)sizeof(T); ++u) __stcs(to + u, y.v[u]);
}

template <typename A>
int go(void (*k)(A), const A& a, long long items, int groups, cudaStream_t s) {
  const long long per = kThreads / groups, grid = (items + per - 1) / per;
  if (grid > 0x7fffffffLL) return KVC_ERR_TOO_LARGE;
  return launch_pdl(k, dim3((unsigned)grid), dim3(kThreads), 0, s, false, a) == cudaSuccess ? KVC_OK : KVC_ERR_LAUNCH;
}

// The last CTA's items are indexed too: fewer than kThreads beyond the end.
bool fits32(long long items) { return items + kThreads < (1LL << 31); }
bool power_of_two(float x) { return (__builtin_bit_cast(uint32_t, x) & 0x7fffffu) == 0; }

template <typename T, int D, bool SNAP>
int store(const StoreArgs& a, cudaStream_t s) {
  const long long items = 2LL * a.t.S * a.T;
  if (fits32(items))
    return go(store_kernel<T, D, SNAP, unsigned>, a, items, D / 16, s);
  return go(store_kernel<T, D, SNAP, long long>, a, items, D / 16, s);
}

template <int D>
int store(const StoreArgs& a, int dtype, cudaStream_t s) {
  if (dtype == KVC_F32) return store<float, D, false>(a, s);
  return power_of_two(a.g.ts[0]) && power_of_two(a.g.ts[1]) ? store<__nv_bfloat16, D, true>(a, s)
                                                            : store<__nv_bfloat16, D, false>(a, s);
}

template <typename T, int D>
int read(const ReadArgs& a, cudaStream_t s) {
  const long long items = (a.out[0] && a.out[1] ? 2LL : 1LL) * a.t.S * a.count;
  if (fits32(items))
    return go(read_kernel<T, D, unsigned>, a, items, D / 16, s);
  return go(read_kernel<T, D, long long>, a, items, D / 16, s);
}

}  // namespace

int launch_page_store(const StoreArgs& a, int dtype, cudaStream_t s) {
  return a.g.D == 128 ? store<128>(a, dtype, s) : store<64>(a, dtype, s);
}

int launch_page_read(const ReadArgs& a, int dtype, cudaStream_t s) {
  if (dtype == KVC_BF16) return a.g.D == 128 ? read<__nv_bfloat16, 128>(a, s) : read<__nv_bfloat16, 64>(a, s);
  return a.g.D == 128 ? read<float, 128>(a, s) : read<float, 64>(a, s);
}

}  // namespace kvc
