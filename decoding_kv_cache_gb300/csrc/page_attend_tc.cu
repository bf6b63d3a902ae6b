// page_attend_tc.cu -- attention of many query rows (a prompt's chunk, a verified tree) over the paged
// 4-bit cache, on the tcgen05 tensor cores (bf16 queries).
//
// A CTA takes 128 query rows of a KV head and a run of its 128-token units. Per unit: 4 * 128 * 128 * D
// operations, S = Q K^T and O += P V, both kind::f16 with M = 128 rows on the tensor-memory lanes.
// The cache's codes become fp16 exactly (page.cuh), so decoding costs no precision; queries are brought to
// fp16 by a power of two per row (bf16 values exact from 2^-25 of the row's largest on, below that off by at
// most 2^-33 of it); a probability is rounded to fp16 once, 2^-11 relative against the bf16 output's 2^-8.
//
//   producer  (warp 16)     a unit's blocks by bulk copies into a three-stage ring of raw bytes
//   decoders  (warps 8-15)  four warps K, four V: a thread a token, codes and scales to fp16 rows in the
//                           128-byte-swizzled layout, two stages each. V's tile [token][channel] is the
//                           second product's B operand as it lies, channels contiguous (MN-major).
//   issuer    (warp 17)     S_i = Q K_i, then P_{i-1} V_{i-1}
//   softmax   (warps 0-7)   two groups, a unit's first and last 64 tokens, each with its own O and running
//                           maximum and sum (a thread a row): neither waits for the other. S has two
//                           buffers, so the next unit's logits lie ready. P replaces S in tensor memory
//                           (fp16, the A operand). O is rescaled in place, and only when a row's maximum
//                           has risen by more than 2^kRaise.
//
// At a part's end the groups' O are merged and written (whole streams) or left for the combine kernel.
// All waits are bounded; a role that gives up raises KVC_STATUS_TIMEOUT and the others follow.
#include "page_attend.cuh"
#include "page_attend_tc.cuh"
#include "score_tc.cuh"

namespace kvc {
namespace {

constexpr int kSoftWarps = 8, kDecWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + kDecWarps + 2);
constexpr int kRaw = 3;   // stages of raw units
constexpr int kTiles = 2;  // stages of decoded tiles
constexpr uint32_t kTmemCols = 512, kColO = 256;
constexpr int kHalfTok = kTcUnit / 2;  // a softmax group's tokens of a unit

template <int D>
struct Lay {
  static constexpr int kHalf = 128 * 128;             // 128 rows of 64 fp16
  static constexpr int kTile = D / 64 * kHalf;        // a decoded K or V unit, or Q
  static constexpr int kRawBytes = 8 * blk_bytes(D);  // a unit as it lies in the pages
  static constexpr int oK = kTile, oV = oK + kTiles * kTile, oRaw = oV + kTiles * kTile;
  static constexpr int bytes = oRaw + kRaw * kRawBytes + 1024;
};

// Why no wait for a phase's parity can find its barrier two phases off, parts of one unit included (tests/barrier_model.py):
//   raw_*, k_*, v_*  a stage is filled again only when all who wait for it have given it back, in the order of the units
//   s_full, p_full   the next S of a buffer is issued behind P V of the unit in it, so after the waiting softmax warps' P, and
//                    the next P there needs an S that the waiting issuer issues
//   pv_done          by the softmax within a part, for the unit before the one in hand, whose Q K was issued behind the P V of
//                    the unit before that: its commit covers both
//   part_done        once a part, by every warp of the group
//   q_full, merge    the softmax warps stage a part's queries when all of them have met at the end of the part before
struct Bars {
  uint64_t raw_full[kRaw], raw_empty[kRaw], k_full[kTiles], k_empty[kTiles], v_full[kTiles], v_empty[kTiles];
  uint64_t s_full[2], p_full[2][2], pv_done[2], part_done[2];  // p_full: S buffer, group (a group may be a unit ahead)
  uint64_t q_full, merge, drain;
};

// A token's codes and scales to a row of fp16 in the swizzled tile; zero: the row stands for nothing.
// Lanes hold neighbouring tokens, whose 16-byte code vectors lie D/2 bytes apart: each lane begins at another
// vector of its row, so that eight lanes' reads fall on eight different bank groups (with all lanes at the
// same vector, four of them met on one: the shared memory, which the first product reads too, is what
// bounds this kernel). Their stores, of different chunks, still differ in every chunk's low bits.
template <int D>
__device__ __forceinline__ void decode_row(const uint8_t* codes, const uint8_t* scales, uint8_t* tile, int j, bool zero) {
  constexpr int V = D / 32;  // code vectors of a row
  // the tile is 1024-byte aligned: 16-byte chunk c of row j lies at (row + (j & 7) 16) ^ c 16
  const uint32_t row = tc::smem_u32(tile) + j * 128 + ((j & 7) << 4);
#pragma unroll
  for (int q = 0; q < V; ++q) {
    const int c = (q + (D == 128 ? j >> 1 : j >> 2)) & (V - 1);  // 32 channels: two scale groups, four chunks
    const uint4 w4 = reinterpret_cast<const uint4*>(codes)[c];
    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
    const uint32_t two = zero ? 0u : e4m3x2_f16x2(reinterpret_cast<const uint16_t*>(scales)[c]);
    const uint32_t s2[2] = {__byte_perm(two, two, 0x1010), __byte_perm(two, two, 0x3232)};
    const uint32_t at = (row ^ ((c & 1) << 6)) + (c >> 1) * Lay<D>::kHalf;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t r[4];
      e2m1x8_f16(w[i], r);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at ^ (i << 4)), "r"(hmul2(r[0], s2[i >> 1])),
                   "r"(hmul2(r[1], s2[i >> 1])), "r"(hmul2(r[2], s2[i >> 1])), "r"(hmul2(r[3], s2[i >> 1]))
                   : "memory");
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) attend_tc_kernel(AttendArgs a, AttendPlan p) {
  using L = Lay<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot, raw_ok[kRaw], unit_ok[4];
  __shared__ int sm_scan[kThreads / 32], sm_first[2];
  __shared__ int abort_flag, parts_done;
  __shared__ uint32_t raw_issued;  // units the producer has asked for
  __shared__ float row_f[kTcRows];
  __shared__ float2 row_ml[2][kTcRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    abort_flag = parts_done = 0;
    for (int i = 0; i < kRaw; ++i) {
      tc::mbar_init(&bars.raw_full[i], 1);
      tc::mbar_init(&bars.raw_empty[i], kDecWarps);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.k_full[i], kDecWarps / 2);
      tc::mbar_init(&bars.v_full[i], kDecWarps / 2);
      tc::mbar_init(&bars.k_empty[i], 1);
      tc::mbar_init(&bars.v_empty[i], 1);
      // test-only fault (kvc_debug_fault 2): the first CTA's second unit waits for an arrival that nothing makes
      tc::mbar_init(&bars.s_full[i], a.fault && blockIdx.x == 0 && i == 1 ? 2 : 1);
      tc::mbar_init(&bars.pv_done[i], 1);
      tc::mbar_init(&bars.part_done[i], 1);
      tc::mbar_init(&bars.p_full[i][0], 4);
      tc::mbar_init(&bars.p_full[i][1], 4);
    }
    tc::mbar_init(&bars.q_full, kSoftWarps);
    tc::mbar_init(&bars.merge, kSoftWarps);
    tc::mbar_init(&bars.drain, 1);
    tc::mbar_fence_init();
  }
  griddep_wait();
  const int per = (p.nvs + kThreads - 1) / kThreads;
  int W;
  int before = scan_units<kThreads>(a, p, Causal{}, sm_scan, per, &W);
  const Split split(W, p.grid);
  const int w0 = split.first(blockIdx.x), w1 = split.first(blockIdx.x + 1);
  if (w0 >= w1) return;
  for (int i = 0; i < per; ++i) {
    const int vs = threadIdx.x * per + i;
    if (vs >= p.nvs) break;
    const int u = cost_of(p, stream_of(a, p, Causal{}, vs, false));
    if (before <= w0 && w0 < before + u) {
      sm_first[0] = vs;
      sm_first[1] = before;
    }
    before += u;
  }
  if (warp == 17) tc::tmem_alloc(&tmem_slot, kTmemCols);
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  volatile int* ab = &abort_flag;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(kFull, mbar_ready(bar, parity)) || wait_slow(bar, parity, ab, a.status);
  };

  // Every role walks the same parts: f(stream, vs, first unit, end unit, units of the stream, cost before them).
  // A stream begins with `lead` units of cost and no work, so that a CTA that begins another stream gets less.
  auto parts = [&](auto&& f) {
    int vs = sm_first[0], base = sm_first[1], left = w1 - w0, ca = w0 - base;
    for (int C; left > 0; ++vs, ca = 0, base += C) {
      const Stream x = stream_of(a, p, Causal{}, vs, false);
      C = cost_of(p, x);
      if (C == 0) continue;
      const int cb = min(C, ca + left), ua = max(ca - p.lead, 0), ub = max(cb - p.lead, 0);
      left -= cb - ca;
      if (ub > ua && !f(x, vs, ua, ub, C - p.lead, base + p.lead)) return;
    }
  };

  if (warp == 16) {
    // ---- producer ------------------------------------------------------------------------------
    uint32_t n = 0;
    parts([&](const Stream& x, int, int ua, int ub, int, int) {
      const int32_t* row = a.t.table + (size_t)x.s * a.t.maxp;
      const int run = a.g.lp >= 7 ? 8 : 1 << (a.g.lp - 4);  // blocks that lie side by side
      auto id_of = [&](int u) {
        const int tok = u * kTcUnit + (lane & 7) * 16;
        return lane < 8 && lane % run == 0 && u < ub && tok < x.vis ? row[tok >> a.g.lp] : -1;
      };
      int id = id_of(ua);
      for (int u = ua; u < ub; ++u, ++n) {
        const int s = n % kRaw, tok = u * kTcUnit;
        const int nblk = min(8, (x.vis - tok + 15) >> 4);
        const bool lead = lane < nblk && lane % run == 0;
        const int cnt = lead ? min(run, nblk - lane) : 0;
        const bool ok = lead && page_ok(a.g, id);
        if (lead && !ok) status_or(a.status, KVC_STATUS_BAD_PAGE);
        const uint32_t bytes = __reduce_add_sync(kFull, ok ? cnt * blk_bytes(D) : 0);
        const uint32_t mask = __reduce_or_sync(kFull, ok ? ((1u << cnt) - 1) << lane : 0u);
        const uint8_t* src = ok ? block_of(a.g, id, ((tok & ((1 << a.g.lp) - 1)) >> 4)) : nullptr;
        id = id_of(u + 1);
        if (!wait(&bars.raw_empty[s], ((n / kRaw) & 1) ^ 1)) return false;
        if (lane == 0) {
          raw_ok[s] = mask;
          tc::mbar_expect_tx(&bars.raw_full[s], bytes);
        }
        __syncwarp();
        if (ok)
          bulk_load(smem + L::oRaw + s * L::kRawBytes + lane * blk_bytes(D), src, cnt * blk_bytes(D), &bars.raw_full[s]);
      }
      return true;
    });
    if (lane == 0) raw_issued = n;
  } else if (warp == 17) {
    // ---- issuer --------------------------------------------------------------------------------
    // the whole warp walks the loop, so that addresses stay in uniform registers; one lane issues
    constexpr uint32_t id_qk = idesc_f16(128, kTcUnit, false), id_pv = idesc_f16(128, D, true);
    const uint64_t dq = tc::desc_k_sw128(tc::smem_u32(smem)), dk = tc::desc_k_sw128(tc::smem_u32(smem + L::oK)),
                   dv = desc_mn_sw128(tc::smem_u32(smem + L::oV), L::kHalf);
    const bool leader = elect_one();
    uint32_t nk = 0, nv = 0, seg = 0;
    parts([&](const Stream&, int, int ua, int ub, int, int) {
      const int m = ub - ua;
      if (!wait(&bars.q_full, seg++ & 1)) return false;
      for (int i = 0; i <= m; ++i) {
        if (i < m) {
          const int t = nk & 1;
          if (!wait(&bars.k_full[t], (nk >> 1) & 1)) return false;
          tc::fence_after_sync();
          if (leader) {
            const uint64_t d = dk + (uint64_t)(t * (L::kTile >> 4));
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              constexpr int step = 32 >> 4;
              const uint64_t at = (j >> 2) * (L::kHalf >> 4) + (j & 3) * step;
              umma_ss(tmem + t * 128, dq + at, d + at, id_qk, j > 0);
            }
            tc::umma_commit(&bars.k_empty[t]);
            tc::umma_commit(&bars.s_full[t]);
          }
          __syncwarp();
          ++nk;
        }
        if (i > 0) {
          const int t = nv & 1;
          if (!wait(&bars.v_full[t], (nv >> 1) & 1)) return false;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (!wait(&bars.p_full[t][w], (nv >> 1) & 1)) return false;
            tc::fence_after_sync();
            if (leader) {
              const uint64_t d = dv + (uint64_t)(t * (L::kTile >> 4) + w * (kHalfTok * 128 >> 4));
#pragma unroll
              for (int j = 0; j < kHalfTok / 16; ++j)
                umma_ts(tmem + kColO + w * 128, tmem + t * 128 + w * kHalfTok + 8 * j, d + j * (2048 >> 4), id_pv,
                        i > 1 || j > 0);
              tc::umma_commit(&bars.pv_done[w]);
              if (i == m) tc::umma_commit(&bars.part_done[w]);
            }
            __syncwarp();
          }
          if (leader) tc::umma_commit(&bars.v_empty[t]);
          __syncwarp();
          ++nv;
        }
      }
      return true;
    });
  } else if (warp >= kSoftWarps) {
    // ---- decoders ------------------------------------------------------------------------------
    const int kv = (warp - kSoftWarps) >> 2, j = threadIdx.x & 127;
    uint64_t* full = kv ? bars.v_full : bars.k_full;
    uint64_t* empty = kv ? bars.v_empty : bars.k_empty;
    uint32_t n = 0;
    parts([&](const Stream& x, int, int ua, int ub, int, int) {
      for (int u = ua; u < ub; ++u, ++n) {
        const int s = n % kRaw, t = n & 1;
        if (!wait(&bars.raw_full[s], (n / kRaw) & 1) || !wait(&empty[t], ((n >> 1) & 1) ^ 1)) return false;
        const uint32_t ok = *reinterpret_cast<volatile uint32_t*>(&raw_ok[s]);
        const uint8_t* blk = smem + L::oRaw + s * L::kRawBytes + (j >> 4) * blk_bytes(D);
        // behind the last visible token lies anything: V rows of zero keep it out of 0 * NaN
        const bool zero = u * kTcUnit + j >= x.vis || !(ok >> (j >> 4) & 1);
        decode_row<D>(blk + (kv ? piece_off(D, 2) : 0) + (j & 15) * (D / 2),
                      blk + (kv ? piece_off(D, 3) : piece_off(D, 1)) + (j & 15) * (D / 16),
                      smem + (kv ? L::oV : L::oK) + t * L::kTile, j, zero);
        if (kv == 0 && j == 0) unit_ok[n & 3] = ok;
        fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[t]);
          mbar_arrive(&bars.raw_empty[s]);
        }
      }
      return true;
    });
  } else {
    // ---- softmax -------------------------------------------------------------------------------
    const int w = warp >> 2, rr = threadIdx.x & 127;  // group, row
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's quarter of the lanes
    const uint32_t tO = tmem + kColO + w * 128 + lanes;
    uint32_t n = 0, seg = 0;  // units so far
    parts([&](const Stream& x, int vs, int ua, int ub, int U, int base) {
      const int m = ub - ua;
      {
        // the query rows, each brought to [256, 512) by a power of two, with the scale's sign, so that maxima of dot products are maxima of logits. A warp takes 16 rows, D/8 lanes
        // a row, all of its reads in flight at once.
        constexpr int kLanes = D / 8, kAt = 32 / kLanes, kBatch = 16 / kAt;  // lanes of a row, rows at a time, reads in flight
        const int i = lane % kLanes;
#pragma unroll 1
        for (int k0 = 0; k0 < 16 / kAt; k0 += kBatch) {
          uint4 v[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int q = warp * 16 + (k0 + k) * kAt + lane / kLanes;
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (q < x.rows)
              v[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + q_row(a, p, x, x.r0 + q)) + i);
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int q = warp * 16 + (k0 + k) * kAt + lane / kLanes;
            const T* e = reinterpret_cast<const T*>(&v[k]);
            float mx = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) mx = fmaxf(mx, fabsf(to_f32(e[c])));
#pragma unroll
            for (int c = kLanes / 2; c; c >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, c));
            const int ex = max((int)(__float_as_uint(mx) >> 23), 24);
            const float mul = copysignf(__uint_as_float((uint32_t)(262 - ex) << 23), a.scale);
            if (i == 0) row_f[q] = __uint_as_float((uint32_t)(ex - 8) << 23) * (fabsf(a.scale) * kLog2e);
            uint32_t o[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] = pack2(to_f32(e[2 * c]) * mul, to_f32(e[2 * c + 1]) * mul);
            *reinterpret_cast<uint4*>(smem + (i >> 3) * L::kHalf + q * 128 + (((i & 7) ^ (q & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.q_full);
      }
      const int lim = rr < x.rows ? seen_by(p, x, x.r0 + rr) : x.vis;
      const int minlim = seen_by(p, x, x.r0);
      float ref = 0.f, l = 0.f;
      bool none = true;
      // the query rows' factors were written before q_full, which precedes every s_full
      float f = 0.f;
      for (int i = 0; i < m; ++i, ++n) {
        const uint32_t tS = tmem + (n & 1) * 128 + w * kHalfTok + lanes;
        if (!wait(&bars.s_full[n & 1], (n >> 1) & 1)) return false;
        tc::fence_after_sync();
        f = *reinterpret_cast<volatile float*>(&row_f[rr]);
        const int tok0 = (ua + i) * kTcUnit + w * kHalfTok;
        const uint32_t ok = *reinterpret_cast<volatile uint32_t*>(&unit_ok[n & 3]) >> (4 * w) & 0xf;
        const bool masked = tok0 + kHalfTok > minlim || ok != 0xf;
        float mx = -INFINITY;
        {
          uint32_t r[2][32];
          tc::tmem_ld32_async(tS, r[0]);
          tc::tmem_ld32_async(tS + 32, r[1]);
          tc::tmem_wait();
          tc::tmem_regs_ready(r[0]);
          tc::tmem_regs_ready(r[1]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[h][k]);
            if (masked) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (tok0 + 32 * h + k >= lim || !(ok >> (2 * h + (k >> 4)) & 1)) v[k] = -INFINITY;
            }
            mx = fmaxf(mx, tree_max32_3(v));
          }
        }
        mx *= f;
        if (mx != mx) mx = -INFINITY;  // -inf * 0
        const bool raise = none ? mx > -INFINITY : mx > ref + (kOff + kRaise);
        if (__any_sync(kFull, raise)) {
          float c = 1.f;
          if (mx > -INFINITY && (none || mx > ref + kOff)) {
            const float to = mx - kOff;
            c = none ? 1.f : ex2(ref - to);
            none = false;
            ref = to;
            l *= c;
          }
          if (i > 0 && __any_sync(kFull, c != 1.f)) {  // O holds the part's earlier units
            if (!wait(&bars.pv_done[w], (n - 1) & 1)) return false;
            tc::fence_after_sync();
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              uint32_t o[16];
              asm volatile(
                  "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
                  "tcgen05.wait::ld.sync.aligned;\n"
                  : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]),
                    "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
                  : "r"(tO + 16 * k));
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * c);
              tmem_st16(tO + 16 * k, o);
            }
          }
        }
        // P over S, 16 tokens at a time with the next 16 logits on their way: columns [0, 8 c + 8) are written
        // when S's [0, 16 c + 16) have been read
        const float2 f2 = make_float2(f, f), ref2 = make_float2(-ref, -ref);
        float2 l2 = make_float2(0.f, 0.f), l3 = l2;
        uint32_t s0[16], s1[16];
        auto probabilities = [&](uint32_t (&v)[16], int c, auto with_mask) {
          uint32_t o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float2 y = fma2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), f2, ref2);
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            if constexpr (decltype(with_mask)::value) {
              const bool blk = ok >> c & 1;
              if (tok0 + 16 * c + 2 * k >= lim || !blk) y.x = 0.f;
              if (tok0 + 16 * c + 2 * k + 1 >= lim || !blk) y.y = 0.f;
            }
            if (k & 1)
              l3 = add2(l3, y);
            else
              l2 = add2(l2, y);
            o[k] = pack2(y.x, y.y);
          }
          asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(tS + 8 * c),
                       "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                       : "memory");
        };
        auto sweep = [&](auto with_mask) {
          tmem_ld16(tS, s0);
#pragma unroll 1
          for (int c = 0; c < kHalfTok / 16; c += 2) {
            tc::tmem_wait();
            tc::tmem_regs_ready(s0);
            tmem_ld16(tS + 16 * c + 16, s1);
            probabilities(s0, c, with_mask);
            tc::tmem_wait();
            tc::tmem_regs_ready(s1);
            if (c + 2 < kHalfTok / 16) tmem_ld16(tS + 16 * c + 32, s0);
            probabilities(s1, c + 1, with_mask);
          }
        };
        if (masked)
          sweep(std::true_type());
        else
          sweep(std::false_type());
        l += (l2.x + l2.y) + (l3.x + l3.y);
        tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[n & 1][w]);
      }
      // ---- the groups' results together. A wait for a phase's parity tells it from the phase two before only once the one
      // between is over, and this group may be a unit ahead of the issuer: a barrier of its own, once a part.
      if (!wait(&bars.part_done[w], seg >> 1 & 1)) return false;  // seg counts the merges, two a part
      tc::fence_after_sync();
      row_ml[w][rr] = make_float2(ref, l);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.merge);
      if (!wait(&bars.merge, seg & 1)) return false;
      tc::fence_after_sync();
      const float2 y0 = row_ml[0][rr], y1 = row_ml[1][rr];
      const float mm = y1.y > 0.f ? (y0.y > 0.f ? fmaxf(y0.x, y1.x) : y1.x) : y0.x;
      float c0 = y0.y > 0.f ? ex2(y0.x - mm) : 0.f, c1 = y1.y > 0.f ? ex2(y1.x - mm) : 0.f;
      if (y0.y != y0.y || y1.y != y1.y) c0 = NAN;
      const float ll = y0.y * c0 + y1.y * c1;
      const bool whole = ua == 0 && ub == U;
      if (ua == 0 && threadIdx.x == 0)
        p.span[vs] = make_int2(blockIdx.x, whole ? (int)blockIdx.x : split.owner(base + U - 1));
      const size_t at = out_row(a, p, x, x.r0 + rr);
      const size_t slot = (size_t)blockIdx.x * 2 + (ua == 0 ? 1 : 0), prow = slot * kTcRows + rr;
      const float inv = ll == 0.f ? 0.f : a.g.ts[1] / ll;
      constexpr int kCols = D / 2;  // each group writes half of the channels
#pragma unroll 1
      for (int k = w * kCols; k < (w + 1) * kCols; k += 16) {
        uint32_t o0[16], o1[16];
        tmem_ld16(tmem + kColO + lanes + k, o0);
        tmem_ld16(tmem + kColO + lanes + k + 128, o1);
        tc::tmem_wait();
        tc::tmem_regs_ready(o0);
        tc::tmem_regs_ready(o1);
        float o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = fmaf(__uint_as_float(o1[e]), c1, __uint_as_float(o0[e]) * c0);
        if (rr < x.rows) {
          if (whole) {
            alignas(16) T y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = from_f32<T>(o[e] * inv);
            uint4* op = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + at * D + k);
            op[0] = reinterpret_cast<const uint4*>(y)[0];
            op[1] = reinterpret_cast<const uint4*>(y)[1];
          } else {  // rows contiguous: a warp's store is one line
            float* op = p.part + (slot * D + k) * kTcRows + rr;
#pragma unroll
            for (int e = 0; e < 16; ++e) op[e * kTcRows] = o[e];
          }
        }
      }
      if (w == 0 && rr < x.rows) {
        if (whole) {
          if (a.lse) a.lse[at] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
        } else {
          p.ml[prow] = make_float2(mm, ll);
        }
      }
      // both groups have read O, and every product on this Q is done, before the next part begins
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.merge);
      if (!wait(&bars.merge, (seg & 1) ^ 1)) return false;
      seg += 2;
      if (threadIdx.x == 0) parts_done = seg / 2;
      return true;
    });
  }
  __syncwarp();
  tc::fence_before_sync();
  if (__syncthreads_or(*ab)) {
    // a role gave up and the others followed: what this CTA leaves undone must not be taken for what lay in the
    // workspace. Streams that begin here hold no part at all, those that began before nothing of this CTA's.
    int i = 0;
    parts([&](const Stream&, int vs, int ua, int, int, int) {
      if (i++ < parts_done) return true;
      if (ua == 0 && threadIdx.x == 0) p.span[vs] = make_int2(-1, -1);
      if (threadIdx.x < kTcRows)
        p.ml[((size_t)blockIdx.x * 2 + (ua == 0 ? 1 : 0)) * kTcRows + threadIdx.x] = make_float2(0.f, 0.f);
      return true;
    });
    // copies and products under way end before their memory goes
    if (warp == 16)
      for (uint32_t n = raw_issued > kRaw ? raw_issued - kRaw : 0; n < raw_issued; ++n)
        (void)mbar_wait_far(&bars.raw_full[n % kRaw], (n / kRaw) & 1);
    if (warp == 17) {
      if (elect_one()) tc::umma_commit(&bars.drain);  // the lane that issued the products
      __syncwarp();
      (void)mbar_wait_far(&bars.drain, 0);
    }
    __syncthreads();
  }
  if (warp == 17) tc::tmem_dealloc(tmem, kTmemCols);
}

template <typename T, int D>
int go(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  auto k = attend_tc_kernel<T, D>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::bytes) != cudaSuccess)
    return KVC_ERR_LAUNCH;
  return launch_pdl(k, dim3(p.grid), dim3(kThreads), Lay<D>::bytes, s, false, a, p) == cudaSuccess ? KVC_OK
                                                                                                   : KVC_ERR_LAUNCH;
}

}  // namespace

int launch_attend_tc(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  return a.g.D == 128 ? go<__nv_bfloat16, 128>(a, p, s) : go<__nv_bfloat16, 64>(a, p, s);
}

}  // namespace kvc
