// page_attend.cu -- attention over the paged 4-bit cache.
//
// T new queries of each sequence (already stored in the cache) over its streams' tokens: query i of n_q
// sees the first len - n_q + i + 1 tokens of its KV head;
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j),  lse = log sum_j p_j,
// and a query that sees no token gets out = 0 and lse = -inf. One pass over the cache with a running
// maximum and sum in fp32.
//
// A KV head's R = T * Hq/Hkv query rows are taken 8 * NT at a time (a row block). The tokens lie on the
// m axis of mma.sync m16n8k16 and the rows on its n axis (S^T = K Q^T, then O^T = V^T P^T), so eight rows
// fill a tile and the 4-bit operand is decoded straight into A fragments in registers: a lane reads its
// tokens' codes with one vector load, two codes become an fp16 pair by one conversion and one multiply by
// their scale (exact: at most six significant bits), and P^T's fragment is S^T's transposed by movmatrix.
// Why mma.sync: with at most 8 * NT rows the contraction needs a few percent of the tensor peak; what has
// to keep up with memory is the decoding, and tcgen05 would need the decoded tile written to shared or
// tensor memory first. (Probed on this chip: conversion and multiply of 32 code pairs take 14 ns of an SM's
// issue; masks and shifts to 4-bit integers with an fma 27 ns.)
//
// Work is split by tokens over all CTAs of one wave, whatever the streams' lengths: the 64-token units of
// all streams form one list, each stream led by a few units' worth of starting cost, and every CTA takes an
// equal run of it. A stream cut by a CTA border leaves partial (max, sum, O) rows in the workspace; the combine
// kernel merges them (and writes the rows of empty streams). In a CTA each of the four warps takes every fourth
// 32-token chunk with its own two-stage ring of bulk copies; nothing but the end of a stream's part
// synchronises them.
#include "page_attend.cuh"

namespace kvc {
namespace {

constexpr int kWarps = 4;
constexpr int kUnit = 64;    // tokens of a work unit
constexpr int kChunk32 = 32;  // tokens of a ring stage
constexpr int kStages = 2;
constexpr int kMaxGridSMs = 160;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
template <int D, int NT>
struct Smem {
  static constexpr int kStage = 2 * blk_bytes(D);  // 32 tokens
  static constexpr int kRows = 8 * NT;
  static constexpr int kMerge = kRows * D * 4 + kRows * 8;  // one warp's O^T, references and sums
  static constexpr int bytes = kWarps * kStages * kStage + 2 * kMerge;
};

// Rows per thread in the accumulators: of tile nt, rows 2t and 2t+1 (t = lane % 4); channels
// CPV*g + 2 mt (+1), g = lane / 4.
template <typename T, int D, int NT, int PARTS, int MINB>
__global__ void __launch_bounds__(32 * kWarps, MINB) attend_kernel(AttendArgs a, AttendPlan p) {
  using SM = Smem<D, NT>;
  constexpr int KS = D / 16;   // k steps of Q K^T and m tiles of V^T
  constexpr int CPL = D / 4;   // channels of a lane in K
  constexpr int CPV = D / 8;   // channels of a lane in V
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kWarps][kStages];
  __shared__ uint32_t oks[kWarps][kStages];
  __shared__ int sm_scan[kWarps], sm_first[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * kStages * SM::kStage;
  float* merge = reinterpret_cast<float*>(smem + kWarps * kStages * SM::kStage);
  if (lane == 0) {
    // test-only fault (kvc_debug_fault 2): a barrier of the first CTA waits for one arrival more than it gets
    for (int i = 0; i < kStages; ++i) tc::mbar_init(&bars[warp][i], a.fault && blockIdx.x + warp + i == 0 ? 2 : 1);
    tc::mbar_fence_init();
  }
  griddep_wait();

  // this CTA's units, and the stream its first one lies in
  int vs = blockIdx.x, base = 0, ca = 0, left = 1;  // whole: `left` becomes the stream's units
  Split split(0, 1);
  if (!p.whole) {
    const int per = (p.nvs + 32 * kWarps - 1) / (32 * kWarps);
    int W;
    int before = scan_units<32 * kWarps>(a, p, sm_scan, per, &W);
    split = Split(W, p.grid);
    const int w0 = split.first(blockIdx.x), w1 = split.first(blockIdx.x + 1);
    if (w0 >= w1) return;
    for (int i = 0; i < per; ++i) {
      const int v = threadIdx.x * per + i;
      if (v >= p.nvs) break;
      const int u = cost_of(p, stream_of(a, p, v, false));
      if (before <= w0 && w0 < before + u) {
        sm_first[0] = v;
        sm_first[1] = before;
      }
      before += u;
    }
    __syncthreads();
    vs = sm_first[0];
    base = sm_first[1];  // cost before the stream
    ca = w0 - base;
    left = w1 - w0;
  } else {
    const Stream x = stream_of(a, p, vs, threadIdx.x == 0);
    left = units_of(p, x);
    if (left == 0)  // rows that see nothing
      for (int e = threadIdx.x; e < x.rows * D; e += 32 * kWarps) {
        const size_t at = out_row(a, p, x, x.r0 + e / D);
        static_cast<T*>(a.out)[at * D + e % D] = from_f32<T>(0.f);
        if (a.lse && e % D == 0) a.lse[at] = -INFINITY;
      }
    __syncwarp();  // the barriers of this warp's ring are visible to its lanes
  }
  uint32_t n = 0;  // chunks this warp has waited for
  bool alive = true;

  for (int C; left > 0; ++vs, ca = 0, base += C) {
    const Stream x = stream_of(a, p, vs, true);
    C = cost_of(p, x);
    if (C == 0) continue;
    const int cb = min(C, ca + left), ua = max(ca - p.lead, 0), ub = max(cb - p.lead, 0), U = C - p.lead;
    left -= cb - ca;
    if (ub == ua) continue;  // only the stream's leading cost
    const int c1 = min(2 * ub, (x.vis + kChunk32 - 1) / kChunk32);  // chunks [2 ua, c1) of the stream
    const int c0 = 2 * ua + warp;
    const int mine = c1 > c0 ? (c1 - c0 + kWarps - 1) / kWarps : 0;
    const int32_t* row = a.t.table + (size_t)x.s * a.t.maxp;

    // Where this warp's next 32 chunks lie, one a lane (two blocks apart where a page is half a chunk): the
    // lane that knows a chunk's place issues its copy.
    const uint8_t* src[2];
    auto locate = [&](int i) {
      const int tok = (c0 + kWarps * (i + lane)) * kChunk32;
      const int q0 = tok >> a.g.lp, q1 = (tok + 16) >> a.g.lp;
      const bool want = i + lane < mine, want1 = want && tok + 16 < x.vis;
      const int id0 = want ? row[q0] : 0;
      const int id1 = a.g.lp > 4 || !want1 ? id0 : row[q1];
      const int blk = (tok & ((1 << a.g.lp) - 1)) >> 4;
      src[0] = page_ok(a.g, id0) ? block_of(a.g, id0, blk) : nullptr;
      src[1] = want1 && page_ok(a.g, id1) ? (a.g.lp > 4 ? src[0] + blk_bytes(D) : block_of(a.g, id1, 0)) : nullptr;
      if (want && (!src[0] || (want1 && !src[1]))) status_or(a.status, KVC_STATUS_BAD_PAGE);
    };
    auto issue = [&](int i, int st) {  // chunk i of this warp into stage st
      if ((i & 31) == 0) locate(i);
      if (lane == (i & 31)) {
        uint8_t* dst = ring + st * SM::kStage;
        uint64_t* bar = &bars[warp][st];
        oks[warp][st] = (src[0] ? 1u : 0u) | (src[1] ? 2u : 0u);
        if (src[1] == src[0] + blk_bytes(D)) {
          tc::mbar_expect_tx(bar, 2 * blk_bytes(D));
          bulk_load(dst, src[0], 2 * blk_bytes(D), bar);
        } else {
          tc::mbar_expect_tx(bar, (src[0] ? blk_bytes(D) : 0) + (src[1] ? blk_bytes(D) : 0));
          if (src[0]) bulk_load(dst, src[0], blk_bytes(D), bar);
          if (src[1]) bulk_load(dst + blk_bytes(D), src[1], blk_bytes(D), bar);
        }
      }
    };
    for (int i = 0; i < kStages && i < mine && alive; ++i) issue(i, (n + i) % kStages);

    // the query rows as B fragments: k step i, k = 2t,2t+1 -> channels CPL t + 4 i + 0,1 and
    // k = 2t+8,2t+9 -> + 2,3. Each row is brought to [256, 512) by a power of two. bf16 values are then exact in
    // fp16 from 2^-25 of the row's largest on, smaller ones off by at most 2^-33 of it (fp16's smallest step is
    // 2^-24); fp32 values are split in two terms, 22 bits of 24.
    uint32_t qf[NT][PARTS][KS][2];
    float f[NT][2];  // rows 2t, 2t+1: scale * log2 e over that power
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = x.r0 + nt * 8 + g;
      const bool in = nt * 8 + g < x.rows;
      float v[CPL];
      float mx = 0.f;
      if (in) {
        const T* qp = static_cast<const T*>(a.q) + q_row(a, p, x, r) + CPL * t;
        constexpr int per16 = 16 / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < CPL / per16; ++i) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(qp) + i);
          const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
          for (int u = 0; u < per16; ++u) v[i * per16 + u] = to_f32(e[u]);
        }
#pragma unroll
        for (int i = 0; i < CPL; ++i) mx = fmaxf(mx, fabsf(v[i]));
      } else {
#pragma unroll
        for (int i = 0; i < CPL; ++i) v[i] = 0.f;
      }
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      const int ex = max((int)(__float_as_uint(mx) >> 23), 24);
      const float mul = __uint_as_float((uint32_t)(262 - ex) << 23);
      const float inv = __uint_as_float((uint32_t)(ex - 8) << 23) * (a.scale * kLog2e);
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float lo = v[4 * i + 2 * u] * mul, hi = v[4 * i + 2 * u + 1] * mul;
          const uint32_t w = pack2(lo, hi);
          qf[nt][0][i][u] = w;
          if constexpr (PARTS == 2) {
            const float2 b = f16x2_f32(w);
            qf[nt][1][i][u] = pack2(lo - b.x, hi - b.y);
          }
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[nt][e] = __shfl_sync(kFull, inv, 8 * t + 4 * e);
        const int rr = nt * 8 + 2 * t + e;
        lim[nt][e] = rr < x.rows ? seen_by(p, x, x.r0 + rr) : x.vis;
      }
    }
    const int minlim = seen_by(p, x, x.r0);

    float o[NT][KS][4];
    float ref[NT][2], l[NT][2];  // reference minus kOff (0 until a token is seen), this lane's part of the sum
    float top[NT][2];            // how far over it a logit may lie: -inf until a token is seen
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ref[nt][e] = 0.f;
        l[nt][e] = 0.f;
        top[nt][e] = -INFINITY;
      }
    }

    for (int i = 0; i < mine && alive; ++i, ++n) {
      const int st = n % kStages;
      if (!__all_sync(kFull, mbar_ready(&bars[warp][st], (n / kStages) & 1)) &&
          !mbar_wait_far(&bars[warp][st], (n / kStages) & 1)) {
        // nothing more is issued; the copies in flight get a second, bounded wait
        if (lane == 0) status_or(a.status, KVC_STATUS_TIMEOUT);
        alive = false;
        for (int k = 1; k < kStages && i + k < mine; ++k)
          (void)mbar_wait_far(&bars[warp][(n + k) % kStages], ((n + k) / kStages) & 1);
        break;
      }
      const uint8_t* buf = ring + st * SM::kStage;
      const int tok0 = (c0 + kWarps * i) * kChunk32;
      const uint32_t ok = *reinterpret_cast<volatile uint32_t*>(&oks[warp][st]);

      // S^T of the two 16-token blocks
      float sc[2][NT][4];
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const uint8_t* kb = buf + blk * blk_bytes(D);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[blk][nt][e] = 0.f;
        uint32_t w[2][CPL / 8], s2[2][2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint8_t* kr = kb + (g + 8 * half) * (D / 2) + t * (CPL / 2);
          const uint8_t* sr = kb + piece_off(D, 1) + (g + 8 * half) * (D / 16);
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(kr);
            w[half][0] = v.x, w[half][1] = v.y, w[half][2] = v.z, w[half][3] = v.w;
            const uint32_t two = e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(sr + 2 * t));
            s2[half][0] = __byte_perm(two, two, 0x1010);
            s2[half][1] = __byte_perm(two, two, 0x3232);
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(kr);
            w[half][0] = v.x, w[half][1] = v.y;
            const uint32_t two = e4m3x2_f16x2(sr[t]);
            s2[half][0] = s2[half][1] = __byte_perm(two, two, 0x1010);
          }
        }
#pragma unroll
        for (int j = 0; j < CPL / 8; ++j) {  // a word: two k steps
          uint32_t k0[4], k1[4];
          e2m1x8_f16(w[0][j], k0);
          e2m1x8_f16(w[1][j], k1);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int ks = 2 * j + e, sg = D == 128 ? ks / 4 : 0;
            const uint32_t af[4] = {hmul2(k0[2 * e], s2[0][sg]), hmul2(k1[2 * e], s2[1][sg]),
                                    hmul2(k0[2 * e + 1], s2[0][sg]), hmul2(k1[2 * e + 1], s2[1][sg])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int q = 0; q < PARTS; ++q) mma16816(sc[blk][nt], af, qf[nt][q][ks][0], qf[nt][q][ks][1]);
          }
        }
      }

      // logits in base 2 over the reference; what a row does not see is -inf
      const bool masked = tok0 + kChunk32 > minlim || ok != 3;
      float2 y[2][NT][2];  // rows 2t, 2t+1 of token g (first) and g + 8
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            y[blk][nt][h] = fma2(make_float2(sc[blk][nt][2 * h], sc[blk][nt][2 * h + 1]), make_float2(f[nt][0], f[nt][1]),
                                 make_float2(-ref[nt][0], -ref[nt][1]));
      if (masked) {
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int tok = tok0 + 16 * blk + g + 8 * h;
              if (tok >= lim[nt][0] || !(ok >> blk & 1)) y[blk][nt][h].x = -INFINITY;
              if (tok >= lim[nt][1] || !(ok >> blk & 1)) y[blk][nt][h].y = -INFINITY;
            }
      }
      // raise the references where a logit passes them by more than 2^(kOff + kRaise)
      float2 mx[NT];
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mx[nt].x = fmaxf(fmaxf(y[0][nt][0].x, y[0][nt][1].x), fmaxf(y[1][nt][0].x, y[1][nt][1].x));
        mx[nt].y = fmaxf(fmaxf(y[0][nt][0].y, y[0][nt][1].y), fmaxf(y[1][nt][0].y, y[1][nt][1].y));
        raise |= mx[nt].x > top[nt][0] || mx[nt].y > top[nt][1];
      }
      if (__any_sync(kFull, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = e ? mx[nt].y : mx[nt].x;
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
            if (m > top[nt][e] - kRaise) {
              const float up = m - kOff, c = top[nt][e] == -INFINITY ? 1.f : ex2(-up);
              ref[nt][e] += up;
              top[nt][e] = kOff + kRaise;
              l[nt][e] *= c;
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                o[nt][k][e] *= c;
                o[nt][k][e + 2] *= c;
              }
#pragma unroll
              for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int h = 0; h < 2; ++h) (e ? y[blk][nt][h].y : y[blk][nt][h].x) -= up;
            }
          }
      }
      // P^T fragments. A probability is rounded to fp16, once, for bf16 outputs: 2^-11 relative at most, token by
      // token, against the output's own 2^-8; two terms would double the products. For fp32 outputs a second term
      // holds what the first cut off. The sum adds the unrounded ones.
      uint32_t pf[2][NT][PARTS][2];
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float2 pr = make_float2(ex2(y[blk][nt][half].x), ex2(y[blk][nt][half].y));
            const float2 sum = add2(make_float2(l[nt][0], l[nt][1]), pr);
            l[nt][0] = sum.x;
            l[nt][1] = sum.y;
            const uint32_t w = pack2(pr.x, pr.y);
            pf[blk][nt][0][half] = transpose8x8(w);
            if constexpr (PARTS == 2) {
              const float2 b = f16x2_f32(w);
              pf[blk][nt][1][half] = transpose8x8(pack2(pr.x - b.x, pr.y - b.y));
            }
          }

      // O^T += V^T P^T
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const uint8_t* vb = buf + blk * blk_bytes(D) + piece_off(D, 2);
        const uint8_t* sb = buf + blk * blk_bytes(D) + piece_off(D, 3);
        uint32_t w[4][CPV / 8], s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tk = 2 * t + (e & 1) + (e >= 2 ? 8 : 0);
          const uint8_t* vr = vb + tk * (D / 2) + g * (CPV / 2);
          if constexpr (D == 128) {
            const uint2 v = *reinterpret_cast<const uint2*>(vr);
            w[e][0] = v.x, w[e][1] = v.y;
            s[e] = sb[tk * 8 + g];
          } else {
            w[e][0] = *reinterpret_cast<const uint32_t*>(vr);
            s[e] = sb[tk * 4 + (g >> 1)];
          }
        }
        if (masked) {  // behind the last visible token lies anything: a zero scale keeps it out of 0 * NaN
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (tok0 + 16 * blk + 2 * t + (e & 1) + (e >= 2 ? 8 : 0) >= x.vis || !(ok >> blk & 1)) s[e] = 0;
        }
        const uint32_t s01 = e4m3x2_f16x2(__byte_perm(s[0], s[1], 0x3340)), s23 = e4m3x2_f16x2(__byte_perm(s[2], s[3], 0x3340));
#pragma unroll
        for (int j = 0; j < CPV / 8; ++j) {
          uint32_t e01[4], o01[4], e23[4], o23[4];
          constexpr uint32_t m = 0x0f0f0f0fu;
          e2m1x8_f16((w[0][j] & m) | (w[1][j] << 4 & ~m), e01);
          e2m1x8_f16((w[0][j] >> 4 & m) | (w[1][j] & ~m), o01);
          e2m1x8_f16((w[2][j] & m) | (w[3][j] << 4 & ~m), e23);
          e2m1x8_f16((w[2][j] >> 4 & m) | (w[3][j] & ~m), o23);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t af[4] = {hmul2(e01[e], s01), hmul2(o01[e], s01), hmul2(e23[e], s23), hmul2(o23[e], s23)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int q = 0; q < PARTS; ++q) mma16816(o[nt][4 * j + e], af, pf[blk][nt][q][0], pf[blk][nt][q][1]);
          }
        }
      }
      __syncwarp();  // every lane is done with the stage
      if (i + kStages < mine) issue(i + kStages, st);
    }

    // a row's sum over the eight lanes that hold its tokens
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], 16);
      }
    // the four warps' parts into warp 0: 2, 3 to 0, 1, then 1 to 0
    for (int gap = 2; gap; gap >>= 1) {
      float* mb = merge + (warp & (gap - 1)) * (SM::kMerge / 4);
      float2* ml = reinterpret_cast<float2*>(mb + SM::kRows * D);
      if (warp >= gap && warp < 2 * gap) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (g == 0) {
            ml[nt * 8 + 2 * t] = make_float2(ref[nt][0], l[nt][0]);
            ml[nt * 8 + 2 * t + 1] = make_float2(ref[nt][1], l[nt][1]);
          }
#pragma unroll
          for (int k = 0; k < KS; ++k)
            *reinterpret_cast<float4*>(mb + ((nt * KS + k) * 32 + lane) * 4) =
                make_float4(o[nt][k][0], o[nt][k][1], o[nt][k][2], o[nt][k][3]);
        }
      }
      __syncthreads();
      if (warp < gap) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float ca[2], cb[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 y = ml[nt * 8 + 2 * t + e];
            const float m = y.y > 0.f ? (l[nt][e] > 0.f ? fmaxf(ref[nt][e], y.x) : y.x) : ref[nt][e];
            ca[e] = l[nt][e] > 0.f ? ex2(ref[nt][e] - m) : 0.f;
            cb[e] = y.y > 0.f ? ex2(y.x - m) : 0.f;
            if (isnan(l[nt][e]) || isnan(y.y)) ca[e] = NAN;
            l[nt][e] = l[nt][e] * ca[e] + y.y * cb[e];
            ref[nt][e] = m;
          }
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const float4 y = *reinterpret_cast<const float4*>(mb + ((nt * KS + k) * 32 + lane) * 4);
            o[nt][k][0] = o[nt][k][0] * ca[0] + y.x * cb[0];
            o[nt][k][1] = o[nt][k][1] * ca[1] + y.y * cb[1];
            o[nt][k][2] = o[nt][k][2] * ca[0] + y.z * cb[0];
            o[nt][k][3] = o[nt][k][3] * ca[1] + y.w * cb[1];
          }
        }
      }
      __syncthreads();
    }
    if (warp == 0) {
      const bool whole = ua == 0 && ub == U;
      // who holds the stream's parts, for the combine kernel
      if (!p.whole && ua == 0 && lane == 0) p.span[vs] = make_int2(blockIdx.x, whole ? (int)blockIdx.x : split.owner(base + C - 1));
      const size_t slot = (size_t)blockIdx.x * 2 + (ua == 0 ? 1 : 0);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = nt * 8 + 2 * t + e;
          if (rr >= x.rows) continue;
          if (whole) {
            const size_t at = out_row(a, p, x, x.r0 + rr);
            const float inv = l[nt][e] == 0.f ? 0.f : a.g.ts[1] / l[nt][e];
            T* op = static_cast<T*>(a.out) + at * D + CPV * g;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              op[2 * k] = from_f32<T>(o[nt][k][e] * inv);
              op[2 * k + 1] = from_f32<T>(o[nt][k][e + 2] * inv);
            }
            if (a.lse && g == 0)
              a.lse[at] = l[nt][e] == 0.f ? -INFINITY : (ref[nt][e] + log2f(l[nt][e])) * 0.6931471805599453f;
          } else {
            float* op = p.part + (slot * SM::kRows + rr) * D + CPV * g;
#pragma unroll
            for (int k = 0; k < KS; ++k) *reinterpret_cast<float2*>(op + 2 * k) = make_float2(o[nt][k][e], o[nt][k][e + 2]);
            if (g == 0) p.ml[slot * SM::kRows + rr] = make_float2(ref[nt][e], l[nt][e]);
          }
        }
    }
  }
}

// A row's merged parts, E channels a lane.
template <int E>
struct Merged {
  float o[E], l = 0.f, m = -INFINITY;
  __device__ __forceinline__ Merged() {
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
  }
  __device__ __forceinline__ void add(float y_m, float y_l, const float* y) {
    if (y_l == 0.f) return;
    const float to = l == 0.f ? y_m : fmaxf(m, y_m);
    const float c0 = l == 0.f ? 0.f : ex2(m - to), c1 = ex2(y_m - to);
    l = l * c0 + y_l * c1;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * c0 + y[e] * c1;
    m = to;
  }
};

// Rows whose stream several CTAs shared, and rows of streams without tokens: a CTA per row, its warps taking
// every fourth part, four at a time.
constexpr int kCombThreads = 128, kCombWarps = kCombThreads / 32;
template <typename T, int D>
__global__ void __launch_bounds__(kCombThreads) combine_kernel(AttendArgs a, AttendPlan p) {
  __shared__ float sm_o[kCombWarps][D];
  __shared__ float2 sm_ml[kCombWarps];
  griddep_launch();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int vs = blockIdx.x >> p.lrb, rr = blockIdx.x & (p.rb - 1);
  const int2 span = p.span[vs];  // read beside the length; undefined for a stream without units
  const Stream x = stream_of(a, p, vs, threadIdx.x == 0 && rr == 0);
  if (rr >= x.rows) return;
  const size_t at = out_row(a, p, x, x.r0 + rr);
  T* op = static_cast<T*>(a.out) + at * D;
  constexpr int E = D / 32, N = 4;
  if (x.vis == 0) {
    if (warp) return;
#pragma unroll
    for (int e = 0; e < E; ++e) op[lane * E + e] = from_f32<T>(0.f);
    if (a.lse && lane == 0) a.lse[at] = -INFINITY;
    return;
  }
  if (span.x == span.y) return;  // written by that CTA
  Merged<E> r;
  for (int c0 = span.x + warp; c0 <= span.y; c0 += N * kCombWarps) {
    float2 ml[N];
    float y[N][E];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * kCombWarps;
      ml[i] = make_float2(0.f, 0.f);
      if (c > span.y) continue;
      // the first CTA's part begins at the stream's first unit, the others' behind it
      const size_t row = ((size_t)c * 2 + (c == span.x ? 1 : 0)) * p.rb + rr;
      ml[i] = p.ml[row];
      const float* src = p.part + row * D + lane * E;
      if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        y[i][0] = v.x, y[i][1] = v.y, y[i][2] = v.z, y[i][3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        y[i][0] = v.x, y[i][1] = v.y;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) r.add(ml[i].x, ml[i].y, y[i]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = r.o[e];
  if (lane == 0) sm_ml[warp] = make_float2(r.m, r.l);
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int w = 1; w < kCombWarps; ++w) r.add(sm_ml[w].x, sm_ml[w].y, &sm_o[w][lane * E]);
  const float inv = r.l == 0.f ? 0.f : a.g.ts[1] / r.l;
#pragma unroll
  for (int e = 0; e < E; ++e) op[lane * E + e] = from_f32<T>(r.o[e] * inv);
  if (a.lse && lane == 0) a.lse[at] = r.l == 0.f ? -INFINITY : (r.m + log2f(r.l)) * 0.6931471805599453f;
}

// The tcgen05 kernel's parts lie with the rows contiguous: a thread a row, 16 channels a CTA.
template <typename T, int D>
__global__ void __launch_bounds__(kTcRows) combine_tc_kernel(AttendArgs a, AttendPlan p) {
  griddep_launch();
  griddep_wait();
  constexpr int C = 16, kPer = D / C;
  const int vs = blockIdx.x / kPer, c0 = blockIdx.x % kPer * C, rr = threadIdx.x;
  const int2 span = p.span[vs];
  const Stream x = stream_of(a, p, vs, rr == 0);
  const bool given_up = x.vis && span.x < 0;
  if (rr >= x.rows || (x.vis && span.x == span.y && !given_up)) return;
  float o[C], l = 0.f, m = -INFINITY;
#pragma unroll
  for (int e = 0; e < C; ++e) o[e] = 0.f;
  if (x.vis && !given_up) {
    constexpr int N = 4;  // parts whose reads are in flight at once
    for (int c1 = span.x; c1 <= span.y; c1 += N) {
      float2 ml[N];
      float y[N][C];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = min(c1 + i, span.y);
        const size_t slot = (size_t)c * 2 + (c == span.x ? 1 : 0);
        ml[i] = p.ml[slot * kTcRows + rr];
        const float* src = p.part + (slot * D + c0) * kTcRows + rr;
#pragma unroll
        for (int e = 0; e < C; ++e) y[i][e] = src[e * kTcRows];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (c1 + i > span.y || ml[i].y == 0.f) continue;
        const float to = l == 0.f ? ml[i].x : fmaxf(m, ml[i].x);
        const float k0 = l == 0.f ? 0.f : ex2(m - to), k1 = ex2(ml[i].x - to);
        l = l * k0 + ml[i].y * k1;
#pragma unroll
        for (int e = 0; e < C; ++e) o[e] = o[e] * k0 + y[i][e] * k1;
        m = to;
      }
    }
  }
  const size_t at = out_row(a, p, x, x.r0 + rr);
  const float inv = l == 0.f ? 0.f : a.g.ts[1] / l;
  alignas(16) T y[C];
#pragma unroll
  for (int e = 0; e < C; ++e) y[e] = from_f32<T>(o[e] * inv);
  uint4* op = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + at * D + c0);
#pragma unroll
  for (int e = 0; e < (int)sizeof(y) / 16; ++e) op[e] = reinterpret_cast<const uint4*>(y)[e];
  if (a.lse && c0 == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Row tiles of 8 a block takes: one covers the decode step of up to 8 query heads per KV head; more rows
// share the decoding of a chunk. From kTcMin rows on bf16 queries go to the tcgen05 kernel (32 streams of 8192
// tokens: 16 rows 24.4 us here and 36.6 there, 24 rows 39.2 and 37.3 with four tiles a block here).
constexpr int kTcMin = 17;
// What beginning a stream's part costs, in units (query rows read, the ring or pipeline filled, results merged):
// counted when the work is split, so that a CTA with two parts gets less (64 new tokens over 4 x 8192: 46.7 us
// with none, 43.1 with 5; 16 x 8 heads of up to 1000 tokens 13.0 and 10.8 us with 3).
constexpr int kTcLead = 5, kLead = 3;
// Tables of at most kWholeCap tokens: a CTA takes a whole stream, which saves the search for its units and the
// second kernel (8 heads x 256 tokens: 6.9 us split, 5.9 whole; x 2048: 8.5 and 18.7). With two streams an SM
// and more that pays up to kWholeCapMany tokens (512 heads x 256: 16.8 and 9.3 us; x 2048: 43 and 37.5).
constexpr int kWholeCap = 512, kWholeCapMany = 2048;
constexpr int tiles_for(int R) { return R <= 8 ? 1 : 2; }
constexpr int min_blocks(int nt, int parts) { return nt * parts == 1 ? 4 : nt * parts == 2 ? 3 : 2; }

AttendPlan make_plan(const AttendArgs& a, int parts, int sms, size_t* bytes) {
  AttendPlan p = {};
  p.G = a.Hq / a.t.Hkv;
  const int R = p.G * a.T, nt = tiles_for(R);
  const bool tc = parts == 1 && R >= kTcMin;
  p.unit = tc ? kTcUnit : kUnit;
  p.lead = tc ? kTcLead : kLead;
  p.rb = tc ? kTcRows : 8 * nt;
  p.nrb = (R + p.rb - 1) / p.rb;
  p.nvs = a.t.S * p.nrb;
  p.by_nrb = FastDiv::make(p.nrb);
  p.by_hkv = FastDiv::make(a.t.Hkv);
  p.by_G = FastDiv::make(p.G);
  while ((1 << p.lrb) < p.rb) ++p.lrb;
  sms = sms < kMaxGridSMs ? sms : kMaxGridSMs;
  p.grid = sms * (tc ? 1 : min_blocks(nt, parts));
  const long long cap = (long long)a.t.maxp << a.g.lp;
  const long long cost = (long long)p.nvs * ((cap + p.unit - 1) / p.unit + p.lead);  // if every stream is full
  if (cost < p.grid) p.grid = (int)cost;
  if (!tc && cap <= (p.nvs >= 2 * sms ? kWholeCapMany : kWholeCap)) {
    p.whole = 1;
    p.lead = 0;
    p.grid = p.nvs;
    if (bytes) *bytes = 256;
    return p;
  }
  const size_t slots = (size_t)p.grid * 2 * p.rb;
  const size_t ml = (slots * sizeof(float2) + 255) & ~(size_t)255;
  const size_t span = ((size_t)p.nvs * sizeof(int2) + 255) & ~(size_t)255;
  p.ml = static_cast<float2*>(a.ws);
  p.span = reinterpret_cast<int2*>(static_cast<char*>(a.ws) + ml);
  p.part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + ml + span);
  if (bytes) *bytes = ml + span + slots * a.g.D * sizeof(float);
  return p;
}

template <typename T, int D, int NT, int PARTS>
int go(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  auto k = attend_kernel<T, D, NT, PARTS, min_blocks(NT, PARTS)>;
  constexpr int smem = Smem<D, NT>::bytes;
  if (smem > 47 * 1024 &&  // beyond the default, beside the kernel's static part
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return KVC_ERR_LAUNCH;
  return launch_pdl(k, dim3(p.grid), dim3(32 * kWarps), smem, s, false, a, p) == cudaSuccess ? KVC_OK : KVC_ERR_LAUNCH;
}

template <typename T, int D, int PARTS>
int run(const AttendArgs& a, int sms, cudaStream_t s) {
  const AttendPlan p = make_plan(a, PARTS, sms, nullptr);
  int rc = KVC_ERR_INVALID_ARG;
  switch (p.rb / 8) {
    case 1: rc = go<T, D, 1, PARTS>(a, p, s); break;
    case 2: rc = go<T, D, 2, PARTS>(a, p, s); break;
    case kTcRows / 8:
      if constexpr (PARTS == 1) rc = launch_attend_tc(a, p, s);
      break;
  }
  if (rc || p.whole) return rc;
  const long long rows = (long long)p.nvs * p.rb;
  if constexpr (PARTS == 1)
    if (p.rb == kTcRows)
      return launch_pdl(combine_tc_kernel<T, D>, dim3((unsigned)(p.nvs * (D / 16))), dim3(kTcRows), 0, s, false, a, p) ==
                     cudaSuccess
                 ? KVC_OK
                 : KVC_ERR_LAUNCH;
  return launch_pdl(combine_kernel<T, D>, dim3((unsigned)rows), dim3(kCombThreads), 0, s, false, a, p) == cudaSuccess
             ? KVC_OK
             : KVC_ERR_LAUNCH;
}

}  // namespace

bool attend_fits(const AttendArgs& a) {  // work units and rows are counted in 32 bits
  const int R = a.Hq / a.t.Hkv * a.T, rb = 8 * tiles_for(R);
  const long long nvs = (long long)a.t.S * ((R + rb - 1) / rb);
  return nvs * rb <= 0x7fffffffLL && nvs * ((((long long)a.t.maxp << a.g.lp) + kUnit - 1) / kUnit + kTcLead) <= 0x7fffffffLL;
}

size_t attend_ws_bytes(const PoolGeom& g, const PageTab& t, int Hq, int T) {
  AttendArgs a = {};
  a.g = g;
  a.t = t;
  a.Hq = Hq;
  a.T = T;
  if (!attend_fits(a)) return 0;
  size_t most = 0;
  for (int parts = 1; parts <= 2; ++parts) {
    size_t n;
    make_plan(a, parts, kMaxGridSMs, &n);
    most = n > most ? n : most;
  }
  return most;
}

int launch_page_attend(const AttendArgs& a, int dtype, cudaStream_t s) {
  int dev, sms;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return KVC_ERR_LAUNCH;
  if (dtype == KVC_BF16) return a.g.D == 128 ? run<__nv_bfloat16, 128, 1>(a, sms, s) : run<__nv_bfloat16, 64, 1>(a, sms, s);
  return a.g.D == 128 ? run<float, 128, 2>(a, sms, s) : run<float, 64, 2>(a, sms, s);
}

}  // namespace kvc
