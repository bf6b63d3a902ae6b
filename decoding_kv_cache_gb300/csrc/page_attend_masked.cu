// page_attend_masked.cu -- attention over the paged 4-bit cache where a query sees part of the tokens: a window and the
// first tokens, and of its own step's drafts its ancestors. First form: a warp a query row, a token at a time.
#include "page_attend.cuh"

namespace kvc {
namespace {

constexpr int kWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) attend_masked_kernel(AttendArgs a, SeenArgs m, int rows) {
  griddep_wait();
  const int r = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= rows) return;
  constexpr int E = D / 32;
  const int hq = r % a.Hq, i = r / a.Hq % a.T, b = r / a.Hq / a.T, h = hq / (a.Hq / a.t.Hkv), s = b * a.t.Hkv + h;
  int len = a.t.len[s];
  const int nq = a.n_q ? min(max(a.n_q[b], 0), a.T) : a.T;
  if (i >= nq) return;
  if (len < 0 || len > ((long long)a.t.maxp << a.g.lp)) {
    if (lane == 0) status_or(a.status, KVC_STATUS_BAD_PAGE);
    len = 0;
  }
  const int base = len - nq;
  const size_t at = ((size_t)b * a.T + i);
  const int pos = base + (m.depth ? min(max(m.depth[at], 0), nq - 1) : i);
  const T* qp = static_cast<const T*>(a.q) + b * a.qs.b + i * a.qs.t + hq * a.qs.h + E * lane;
  float q[E], o[E], mx = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = to_f32(qp[e]) * a.scale, o[e] = 0.f;
  for (int j = 0; j < len; ++j) {
    const int u = j - base;
    if (u >= 0 && m.mask ? !(m.mask[at * m.words + (u >> 5)] >> (u & 31) & 1)
                         : (u > i && !m.mask) || !(j < m.sinks || j > pos - m.window)) {
      if (u < 0 && j == m.sinks && pos - m.window > j) j = min(pos - m.window, base - 1);
      continue;
    }
    const int id = a.t.table[(size_t)s * a.t.maxp + (j >> a.g.lp)];
    if (!page_ok(a.g, id)) {
      if (lane == 0) status_or(a.status, KVC_STATUS_BAD_PAGE);
      continue;
    }
    const uint8_t* blk = block_of(a.g, id, (j & ((1 << a.g.lp) - 1)) >> 4);
    auto value = [&](int kv, int c) {
      const uint8_t* codes = blk + piece_off(D, 2 * kv) + (j & 15) * (D / 2);
      const uint8_t* sc = blk + piece_off(D, 2 * kv + 1) + (j & 15) * (D / 16);
      uint32_t r4[4];
      e2m1x8_f16(codes[c >> 1], r4);
      const float2 v = f16x2_f32(r4[0]);
      return (c & 1 ? v.y : v.x) * e4m3_f32(sc[c >> 4]);
    };
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) dot = fmaf(q[e], value(0, E * lane + e), dot);
#pragma unroll
    for (int x = 16; x; x >>= 1) dot += __shfl_xor_sync(kFull, dot, x);
    const float to = fmaxf(mx, dot), c = to == -INFINITY ? 1.f : __expf(mx - to), p = to == -INFINITY ? 0.f : __expf(dot - to);
    mx = to;
    l = l * c + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * value(1, E * lane + e);
  }
  T* op = static_cast<T*>(a.out) + (at * a.Hq + hq) * D + E * lane;
#pragma unroll
  for (int e = 0; e < E; ++e) op[e] = from_f32<T>(l == 0.f ? 0.f : o[e] * (a.g.ts[1] / l));
  if (a.lse && lane == 0) a.lse[at * a.Hq + hq] = l == 0.f ? -INFINITY : mx + logf(l);
}

template <typename T, int D>
int run(const AttendArgs& a, const SeenArgs& m, cudaStream_t s) {
  const long long rows = (long long)a.t.B * a.T * a.Hq;
  return launch_pdl(attend_masked_kernel<T, D>, dim3((unsigned)((rows + kWarps - 1) / kWarps)), dim3(32 * kWarps), 0, s,
                    false, a, m, (int)rows) == cudaSuccess
             ? KVC_OK
             : KVC_ERR_LAUNCH;
}

}  // namespace

size_t attend_masked_ws_bytes(const PoolGeom& g, const PageTab& t, int Hq, int T, const SeenArgs&) {
  AttendArgs a = {};
  a.g = g;
  a.t = t;
  a.Hq = Hq;
  a.T = T;
  return attend_fits(a) ? 256 : 0;
}

int launch_page_attend_masked(const AttendArgs& a, const SeenArgs& m, int dtype, cudaStream_t s) {
  if (dtype == KVC_BF16) return a.g.D == 128 ? run<__nv_bfloat16, 128>(a, m, s) : run<__nv_bfloat16, 64>(a, m, s);
  return a.g.D == 128 ? run<float, 128>(a, m, s) : run<float, 64>(a, m, s);
}

}  // namespace kvc
