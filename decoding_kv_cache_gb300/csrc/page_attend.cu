// page_attend.cu -- attention over the paged 4-bit cache.
//
// T new queries of each sequence (already stored in the cache) over its streams' tokens: query i of n_q
// sees the first len - n_q + i + 1 tokens of its KV head;
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j),  lse = log sum_j p_j,
// and a query that sees no token gets out = 0 and lse = -inf. Running maximum and sum in fp32.
#include "page.cuh"

namespace kvc {
namespace {

// One warp per query row; each lane owns D/32 channels.
template <typename T, int D>
__global__ void __launch_bounds__(128) attend_simple_kernel(AttendArgs a) {
  griddep_wait();
  constexpr int E = D / 32;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int G = a.Hq / a.t.Hkv;
  if (row >= a.t.B * a.T * a.Hq) return;
  const int hq = row % a.Hq, t = row / a.Hq % a.T, b = row / (a.Hq * a.T);
  const int nq = a.n_q ? min(max(a.n_q[b], 0), a.T) : a.T;
  if (t >= nq) return;
  const int s = b * a.t.Hkv + hq / G;
  const int len = a.t.len[s];
  int seen = len - nq + t + 1;
  if (len < 0 || len > ((long long)a.t.maxp << a.g.lp)) {
    if (lane == 0) status_or(a.status, KVC_STATUS_BAD_PAGE);
    seen = 0;
  }
  const T* qp = static_cast<const T*>(a.q) + b * a.qs.b + t * a.qs.t + hq * a.qs.h + lane * E;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = to_f32(qp[e]) * a.scale;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < seen; ++j) {
    const int p = a.t.table[(size_t)s * a.t.maxp + (j >> a.g.lp)];
    if (!page_ok(a.g, p)) {
      if (lane == 0) status_or(a.status, KVC_STATUS_BAD_PAGE);
      continue;
    }
    const int in = j & ((1 << a.g.lp) - 1);
    const uint8_t* blk = block_of(a.g, p, in >> 4);
    float kv[2][E];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint8_t* c = blk + piece_off(D, 2 * w) + (in & 15) * (D / 2) + lane * (E / 2);
      const float sc = e4m3_f32(blk[piece_off(D, 2 * w + 1) + (in & 15) * (D / 16) + lane * E / 16]);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const float2 x = f16x2_f32(e2m1x2_f16x2(c[e]));
        kv[w][2 * e] = x.x * sc;
        kv[w][2 * e + 1] = x.y * sc;
      }
    }
    float d = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) d += q[e] * kv[0][e];
    d = warp_sum(d);
    const float mn = fmaxf(m, d), c = expf(m - mn), x = expf(d - mn);
    l = l * c + x;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + x * kv[1][e];
    m = mn;
  }
  const float inv = l > 0.f ? a.g.ts[1] / l : 0.f;
  T* op = static_cast<T*>(a.out) + (size_t)row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) op[e] = from_f32<T>(o[e] * inv);
  if (a.lse && lane == 0) a.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t attend_ws_bytes(int, int, int, int, int) { return 256; }

int launch_page_attend(const AttendArgs& a, int dtype, cudaStream_t s) {
  const long long rows = (long long)a.t.B * a.T * a.Hq;
  const dim3 grid((unsigned)((rows + 3) / 4));
  cudaError_t e;
  if (dtype == KVC_BF16)
    e = launch_pdl(a.g.D == 128 ? attend_simple_kernel<__nv_bfloat16, 128> : attend_simple_kernel<__nv_bfloat16, 64>,
                   grid, dim3(128), 0, s, false, a);
  else
    e = launch_pdl(a.g.D == 128 ? attend_simple_kernel<float, 128> : attend_simple_kernel<float, 64>, grid, dim3(128),
                   0, s, false, a);
  return e == cudaSuccess ? KVC_OK : KVC_ERR_LAUNCH;
}

}  // namespace kvc
