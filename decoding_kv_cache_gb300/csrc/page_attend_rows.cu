// page_attend_rows.cu -- kvc_page_attend_masked for many query rows (a prompt's chunk, a drafted tree), on the tcgen05
// tensor cores (bf16 queries).
//
// A CTA takes RT tiles of 128 query rows of a KV head and a run of its 128-token units; S = Q K^T and O += P V are
// kind::f16 with M = 128 rows on the tensor-memory lanes. Codes become fp16 exactly (page.cuh); queries are brought to
// fp16 by a power of two per row (bf16 values exact from 2^-25 of the row's largest on, below that off by at most 2^-33
// of it); a probability is rounded to fp16 once, 2^-11 relative against the bf16 output's 2^-8.
//
//   decoders  a part's query rows to fp16 (the first part's are the softmax warps' work), for RT = 2 in place; then half of the warps K, half V:
//             codes and scales from global memory straight to registers ahead of time, four lanes a token, and as fp16
//             into the 128-byte-swizzled tiles (two stages each). V's tile [token][channel] is the second product's B
//             operand as it lies (MN-major).
//   issuers   the products
//   softmax   two groups, a thread a row. RT = 2: a row tile each. While one group's tile is in its softmax the tensor
//             cores work on the other's: P V of a unit, then Q K of the next into the same columns. RT = 1: a unit's first
//             and last 64 tokens each, with their own O, reference and sum, S double-buffered, O merged at the part's end.
// Both shapes decode a unit once; a 256-row block does so for twice the products.
//
// The softmax works on 64 tokens at a time (a step). Probabilities are formed against the reference at hand without
// looking for a maximum first; the sums of 32 tell whether one was too large (32 of at most 2^kOff sum to 2^15, and none
// passes fp16's largest number while the sum does not). Then, as for a part's first tokens and where a row does not see
// all of them, the step is read again 32 tokens at a time, the reference raised to their maximum (by a whole power of two)
// and what was summed so far rescaled. That path lies behind the straight one: instructions between those that always
// run cost as much as they would run (in line and per element: 870 cycles a chunk of 32, 480 without). P replaces S in
// tensor memory.
//
// What bounds it. RT = 1: some 2000 cycles a unit, of which the tensor cores need 1024; a softmax warp's chain (logits from
// tensor memory 400, 64 exponentials and what belongs to them 1000, P back and handed on 600) at 0.72 of the SM's issue
// (80 rows over 64 x 32768 tokens: 124 us, 0.36 of the copy peak, 0.36 of the tensor peak on the rows there are). RT = 2:
// some 3500 cycles a unit of 256 rows, 2048 of them the tensor cores': a tile's softmax (1700) and its products (1400) take
// turns, the other tile's lie beside them (a prompt's 1024 tokens under a window of 2048, 2 x 8 heads: 81 us, 0.45 of the
// tensor peak). At each CTA's beginning 5 us, at its end and between two parts some 3 us.
//
// All waits are bounded; a role that gives up raises KVC_STATUS_TIMEOUT and the others follow.
#include "page_attend.cuh"
#include "page_attend_tc.cuh"
#include "score_tc.cuh"

namespace kvc {
namespace {

// Roles and the registers of their threads. Every role is a chain of dependent steps, so what counts is how many warps
// share its work; the shares of registers stay within what the block is launched with.
template <int RT>
struct Roles;
constexpr bool fits(int soft, int dec, int soft_regs, int dec_regs, int issue_regs) {  // a split above the launch's total never ends
  const int warps = soft + dec + 4, regs = 65536 / (32 * warps) / 8 * 8;
  return soft * soft_regs + dec * dec_regs + 4 * issue_regs <= warps * regs;
}
template <>
struct Roles<1> {  // 896 threads with 72 registers (64512): 2 x 128 x 120 + 4 x 128 x 56 + 128 x 32 = 63488
  static constexpr int kSoft = 8, kDec = 16, kSoftRegs = 120, kDecRegs = 56, kIssueRegs = 32;
  static_assert(fits(kSoft, kDec, kSoftRegs, kDecRegs, kIssueRegs), "registers");
};
template <>
struct Roles<2> {  // 640 threads with 96 registers (61440): 2 x 128 x 144 + 2 x 128 x 72 + 128 x 48 = 61440
  static constexpr int kSoft = 8, kDec = 8, kSoftRegs = 144, kDecRegs = 72, kIssueRegs = 48;
  static_assert(fits(kSoft, kDec, kSoftRegs, kDecRegs, kIssueRegs), "registers");
};
template <int RT>
constexpr int kThreadsOf = 32 * (Roles<RT>::kSoft + Roles<RT>::kDec + 4);  // the issuers' warpgroup is not filled
template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}
constexpr int kTiles = 2;  // stages of decoded tiles
constexpr uint32_t kTmemCols = 512, kColO = 256;
constexpr int kStep = 64, kChunk = 32;  // tokens of a softmax step, and of its slow path at a time
constexpr float kMost = 65504.f;

template <int D, int RT>
struct Lay {
  static constexpr int kHalf = 128 * 128;       // 128 rows of 64 fp16
  static constexpr int kTile = D / 64 * kHalf;  // a decoded K or V unit, or a Q tile
  static constexpr int oK = RT * kTile, oV = oK + kTiles * kTile;
  static constexpr int bytes = oV + kTiles * kTile + 1024;
};

// A wait for a phase's parity tells that phase from the one two before or two behind it only where the barrier cannot be that
// far from it. Why it cannot, parts of one unit included (tests/barrier_model.py runs all of them in any order):
//   k_full, v_full   a stage is filled again only when it is free, and it is so by the products that the waiting issuer issues
//   s_full           by stage (RT = 2: by row tile, and the second's by stage): the next S there needs the waiting softmax
//                    warps' P, and for the K decoders, who take it for "the tile is free", their next keys
//   v_empty          the next products on a stage need those who wait for this: its V decoders, its softmax and, RT = 1, its
//                    Q K; and Q K of a unit is issued when the unit two before is over, so the softmax finds at most one open
//   p_full, pv_done  the next phase needs an S that the waiting issuer issues; a product on the waiting softmax warps' next P
//   merge            all who wait arrive at every phase
//   q_full           who issues Q K waits for it, and the next phase needs q_empty, its own commit. P V reads no queries, and
//                    while it waits for a P those of two more parts may come: who issues P V does not wait for q_full.
//   q_empty          every decoder warp waits for it, and only then arrives at the q_full that the next phase needs
struct Bars {
  uint64_t k_full[kTiles], v_full[kTiles], v_empty[kTiles];
  // RT = 1: by S buffer, which is the tile's stage; 2: of the first row tile, and of the second by the stage. The last one
  // over K's tile says that it is free.
  uint64_t s_full[3], p_full[2];
  uint64_t pv_done[2];  // RT = 2: a part's last P V, by row tile
  uint64_t q_full, q_empty, merge, drain;
};

// A decoder lane's share of a unit: V vectors of 16 bytes of codes and their two scales each.
template <int D, int kTokens>
struct Share {  // of kTokens tokens a warp
  static constexpr int kLanes = D / 32;           // lanes of a token
  static constexpr int kTok = 32 / kLanes;        // tokens between two of a lane's vectors
  static constexpr int V = kTokens / kTok;        // vectors a lane
  uint4 c[V];
  uint32_t s[V];
};

__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint32_t ld_stream2(const void* p) {
  uint32_t r;
  asm volatile("ld.global.nc.u16 %0, [%1];\n" : "=r"(r) : "l"(p));
  return r;
}

// Which of the 32 tokens from tok0 on row rr sees; ok's low bits tell the two 16-token blocks that are there.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }
__device__ __forceinline__ uint32_t row_bits(const AttendArgs& a, const AttendPlan& p, const SeenArgs& m, const Stream& x,
                                          int rr, int lo, int hi, int tok0, uint32_t ok) {
  uint32_t v = (below(x.sinks - tok0) | ~below(lo - tok0)) & below(hi - tok0);
  const int base = x.len - x.nq, u = tok0 - base;
  if (m.mask && rr < x.rows && u > -32) {
    const uint32_t* w = mask_words(a, p, m, x, x.r0 + rr);
    auto word = [&](int i) { return i >= 0 && i < m.words ? w[i] : 0u; };
    // 32 bits from bit u on; bits before the first are the base's
    v |= __funnelshift_r(word(u >> 5), word((u >> 5) + 1), u & 31) & below(x.vis - tok0);
  }
  return v & ((ok & 1 ? 0xffffu : 0u) | (ok & 2 ? 0xffff0000u : 0u));
}

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kThreadsOf<RT>, 1) attend_rows_kernel(AttendArgs a, AttendPlan p, SeenArgs seen) {
  using L = Lay<D, RT>;
  constexpr int kRows = RT * 128, kThreads = kThreadsOf<RT>;
  constexpr int kSoftWarps = Roles<RT>::kSoft, kDecWarps = Roles<RT>::kDec;
  constexpr int kIssuer = kSoftWarps + kDecWarps, kIssuers = RT == 1 ? 2 : 1;  // first warp, warps
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ uint64_t unit_ok[4];  // a byte a K warp: its blocks
  __shared__ int sm_scan[kThreads / 32], sm_first[2];
  __shared__ int abort_flag, parts_done[2];
  // The rows' factors, by part. When those of part s are written, its predecessor's last Q K is over. RT = 2: before that Q K
  // was issued, part s - 2's last P was there, so its factors had been read: two parts' are alive. RT = 1: the P of the unit two
  // before was, which in parts of one unit is part s - 3's: three are alive.
  constexpr int kFactors = RT == 1 ? 4 : 2;
  __shared__ float row_f[kFactors][kRows];
  __shared__ float2 row_ml[RT == 1 ? 2 : 1][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    abort_flag = parts_done[0] = parts_done[1] = 0;
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.k_full[i], kDecWarps / 2);
      tc::mbar_init(&bars.v_full[i], kDecWarps / 2);
      tc::mbar_init(&bars.v_empty[i], 1);
      // test-only fault (kvc_debug_fault 2): a wait of the first CTA is for an arrival that nothing makes
      tc::mbar_init(&bars.s_full[i], a.fault && blockIdx.x == 0 && i == 1 ? 2 : 1);
      tc::mbar_init(&bars.s_full[2], 1);
      tc::mbar_init(&bars.pv_done[i], 1);
      tc::mbar_init(&bars.p_full[i], kSoftWarps / RT);
    }
    tc::mbar_init(&bars.q_full, kDecWarps);
    tc::mbar_init(&bars.q_empty, 1);
    tc::mbar_init(&bars.merge, kSoftWarps);
    tc::mbar_init(&bars.drain, kIssuers);
    tc::mbar_fence_init();
  }
  griddep_wait();
  const int per = (p.nvs + kThreads - 1) / kThreads;
  int W;
  int mine;
  int before = scan_units<kThreads>(a, p, seen, sm_scan, per, &W, &mine);
  const Split split(W, p.grid);
  const int w0 = split.first(blockIdx.x), w1 = split.first(blockIdx.x + 1);
  if (w0 >= w1) return;
  for (int i = 0; i < per && before <= w0; ++i) {
    const int vs = threadIdx.x * per + i;
    if (vs >= p.nvs) break;
    const int u = per == 1 ? mine : cost_of(p, stream_of(a, p, seen, vs, false));
    if (w0 < before + u) {
      sm_first[0] = vs;
      sm_first[1] = before;
      break;
    }
    before += u;
  }
  if (warp == kIssuer) tc::tmem_alloc(&tmem_slot, kTmemCols);
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  volatile int* ab = &abort_flag;
  // In line, and short: a function call has no place between roles that hold different numbers of registers. The clock,
  // which takes long to read, and the other roles' flag are looked at every 64 polls.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    uint64_t since = 0;
#pragma unroll 1
    for (uint32_t i = 1; !__all_sync(kFull, mbar_ready(bar, parity)); ++i)
      if (i % 64 == 0) {
        const uint64_t now = clock_ns();
        if (since == 0) since = now;
        if (__any_sync(kFull, *ab != 0)) return false;
        if (__any_sync(kFull, now - since > kWaitNs)) {
          status_or(a.status, KVC_STATUS_TIMEOUT);
          *ab = 1;
          return false;
        }
      }
    return true;
  };

  // Every role walks the same parts: f(stream, vs, first unit, end unit, units of the stream, cost before them).
  // A stream begins with `lead` units of cost and no work, so that a CTA that begins another stream gets less.
  auto parts = [&](auto&& f) {
    int vs = sm_first[0], base = sm_first[1], left = w1 - w0, ca = w0 - base;
    for (int C; left > 0; ++vs, ca = 0, base += C) {
      const Stream x = stream_of(a, p, seen, vs, false);
      C = cost_of(p, x);
      if (C == 0) continue;
      const int cb = min(C, ca + left), ua = max(ca - p.lead, 0), ub = max(cb - p.lead, 0);
      left -= cb - ca;
      if (ub > ua && !f(x, vs, ua, ub, C - p.lead, base + p.lead)) return;
    }
  };

  using std::integral_constant;
  // A part's query rows, by warp `by` of `of`: each is brought to [256, 512) by a power of two, with the scale's sign, so that
  // maxima of dot products are maxima of logits. RT = 1: D/8 lanes take a row, all of a warp's reads into registers, under way
  // before the products on the part before are over. RT = 2: they are four times as many, and are copied to the places of
  // their 16-byte chunks, all at once; from there four lanes take a row, each every fourth chunk, those of odd rows the second
  // of two first, so that eight lanes find different banks. (A prompt's 1024 tokens 80.8 us so and 84.6 by registers, four
  // reads at a time; 16 x 5 rows over 8 x 8 x 32768 124.6 and 123.0.)
  auto queries = [&](const Stream& x, uint32_t seg, int by, auto of) {
    static_assert(sizeof(T) == 2, "bf16");
    constexpr int kQRows = kRows / decltype(of)::value, kChunks = D / 8, kAt = 32 / kChunks;
    const int q0 = by * kQRows;
    auto place = [&](int q, int c) { return smem + (q >> 7) * L::kTile + (c >> 3) * L::kHalf + (q & 127) * 128 + (((c & 7) ^ (q & 7)) << 4); };
    // the row's power of two from its largest magnitude's bits, and what undoes it
    auto factor = [&](int q, uint32_t top, bool one) {
      const int ex = max((int)(max(top & 0xffffu, top >> 16) >> 7), 24);
      if (one) row_f[seg % kFactors][q] = __uint_as_float((uint32_t)(ex - 8) << 23) * (fabsf(a.scale) * kLog2e);
      return copysignf(__uint_as_float((uint32_t)(262 - ex) << 23), a.scale);
    };
    auto top_of = [](uint32_t top, const uint4& w) {  // two magnitudes at a time: bf16 bits without the sign, in their order
      constexpr uint32_t m = 0x7fff7fffu;
      return __vmaxu2(__vmaxu2(top, __vmaxu2(w.x & m, w.y & m)), __vmaxu2(w.z & m, w.w & m));
    };
    auto times = [](const uint4& w, float mul) {
      auto two = [&](uint32_t v) { return pack2(__uint_as_float(v << 16) * mul, __uint_as_float(v & 0xffff0000u) * mul); };
      return make_uint4(two(w.x), two(w.y), two(w.z), two(w.w));
    };
    auto from = [&](int q, int c) { return static_cast<const T*>(a.q) + (q < x.rows ? q_row(a, p, x, x.r0 + q) : 0) + 8 * c; };
    // the products on the part before read its queries no more
    auto free = [&] { return seg == 0 || wait(&bars.q_empty, (seg - 1) & 1); };
    if constexpr (RT == 1) {
      const int c = lane % kChunks;
      uint4 v[kQRows / kAt];
#pragma unroll
      for (int k = 0; k < kQRows / kAt; ++k) {
        const int q = q0 + k * kAt + lane / kChunks;
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (q < x.rows) v[k] = __ldg(reinterpret_cast<const uint4*>(from(q, c)));
      }
      if (!free()) return false;
#pragma unroll
      for (int k = 0; k < kQRows / kAt; ++k) {
        const int q = q0 + k * kAt + lane / kChunks;
        uint32_t top = top_of(0u, v[k]);
#pragma unroll
        for (int o = kChunks / 2; o; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(kFull, top, o));
        *reinterpret_cast<uint4*>(place(q, c)) = times(v[k], factor(q, top, c == 0));
      }
    } else {
      if (!free()) return false;
#pragma unroll 4
      for (int k = 0; k < kQRows; k += kAt) {
        const int q = q0 + k + lane / kChunks, c = lane % kChunks;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(tc::smem_u32(place(q, c))), "l"(from(q, c)),
                     "r"(q < x.rows ? 16 : 0)
                     : "memory");
      }
      asm volatile("cp.async.wait_all;\n" ::: "memory");
      __syncwarp();
#pragma unroll 2
      for (int k = 0; k < kQRows; k += 8) {
        const int q = q0 + k + lane / 4, c0 = lane & 3;
        uint4 v[kChunks / 4];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kChunks / 4; ++j) {
          v[j] = *reinterpret_cast<const uint4*>(place(q, c0 + 4 * (j ^ (q & 1))));
          top = top_of(top, v[j]);
        }
        top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 2));
        const float mul = factor(q, top, c0 == 0);
#pragma unroll
        for (int j = 0; j < kChunks / 4; ++j) *reinterpret_cast<uint4*>(place(q, c0 + 4 * (j ^ (q & 1)))) = times(v[j], mul);
      }
    }
    fence_async();
    __syncwarp();
    if (lane < kDecWarps / decltype(of)::value) mbar_arrive(&bars.q_full);  // as many arrivals by either role
    return true;
  };

  if (warp >= kIssuer) {
    regs_down<Roles<RT>::kIssueRegs>();
    if (warp < kIssuer + kIssuers) {
    // ---- issuers -------------------------------------------------------------------------------
    // A product costs some 50 cycles to issue and a wait or commit 100 to 300, so there are as few of those as can be. A
    // warp's products run in the order of their issue, which is all that keeps Q K from overwriting a P. RT = 1: two
    // warps share the work; one issues Q K, into a buffer of S once P V has read the last P in it, the other P V (one warp
    // for both: 134 us and not 131 for 16 x 5 rows over 8 x 8 x 32768 tokens). RT = 2: one (a warp a row tile: 112 us and not 96 for a
    // prompt's 1024 tokens). The whole warp walks the loop, so that addresses stay in uniform registers; one lane issues.
    constexpr uint32_t id_qk = idesc_f16(128, kTcUnit, false), id_pv = idesc_f16(128, D, true);
    const uint64_t dq = tc::desc_k_sw128(tc::smem_u32(smem)), dk = tc::desc_k_sw128(tc::smem_u32(smem + L::oK)),
                   dv = desc_mn_sw128(tc::smem_u32(smem + L::oV), L::kHalf);
    const bool leader = elect_one();
    const int iw = warp - kIssuer;
    uint32_t nk = 0, nv = 0, seg = 0;
    auto qk = [&](uint32_t cols, int tile, int t) {  // S of row tile `tile` with the keys of stage t
      const uint64_t q = dq + (uint64_t)(tile * (L::kTile >> 4)), d = dk + (uint64_t)(t * (L::kTile >> 4));
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const uint64_t at = (j >> 2) * (L::kHalf >> 4) + (j & 3) * (32 >> 4);
        umma_ss(tmem + cols, q + at, d + at, id_qk, j > 0);
      }
    };
    auto pv = [&](uint32_t o, uint32_t pcol, int tok, int ntok, int t, bool acc) {  // O += P V, tokens [tok, tok + ntok) of stage t
      const uint64_t d = dv + (uint64_t)(t * (L::kTile >> 4) + (tok * 128 >> 4));
#pragma unroll
      for (int j = 0; j < ntok / 16; ++j)
        umma_ts(tmem + o, tmem + pcol + 8 * j, d + j * (2048 >> 4), id_pv, acc || j > 0);
    };
    parts([&](const Stream&, int, int ua, int ub, int, int) {
      const int m = ub - ua;
      if ((RT == 2 || iw == 0) && !wait(&bars.q_full, seg++ & 1)) return false;
      if constexpr (RT == 2) {
        for (int i = 0; i <= m; ++i) {  // unit i - 1's second product and unit i's first, a row tile after the other
          const int tk = nk & 1, tv = nv & 1;
          if (i > 0 && !wait(&bars.v_full[tv], (nv >> 1) & 1)) return false;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (i > 0 && !wait(&bars.p_full[w], nv & 1)) return false;
            if (w == 0 && i < m && !wait(&bars.k_full[tk], (nk >> 1) & 1)) return false;
            tc::fence_after_sync();
            if (leader) {
              if (i > 0) {
                pv(kColO + w * 128, w * 128, 0, kTcUnit, tv, i > 1);
                if (w == 1) tc::umma_commit(&bars.v_empty[tv]);
                if (i == m) tc::umma_commit(&bars.pv_done[w]);
              }
              if (i < m) {
                qk(w * 128, w, tk);
                tc::umma_commit(w == 0 ? &bars.s_full[0] : &bars.s_full[1 + tk]);
                if (w == 1 && i == m - 1) tc::umma_commit(&bars.q_empty);
              }
            }
            __syncwarp();
          }
          if (i > 0) ++nv;
          if (i < m) ++nk;
        }
      } else if (iw == 0) {
        for (int i = 0; i < m; ++i, ++nk) {
          const int t = nk & 1;
          if (!wait(&bars.k_full[t], (nk >> 1) & 1) || !wait(&bars.v_empty[t], ((nk >> 1) & 1) ^ 1)) return false;
          tc::fence_after_sync();
          if (leader) {
            qk(t * 128, 0, t);
            tc::umma_commit(&bars.s_full[t]);
            if (i == m - 1) tc::umma_commit(&bars.q_empty);
          }
          __syncwarp();
        }
      } else {
        for (int i = 0; i < m; ++i, ++nv) {
          const int t = nv & 1;
          if (!wait(&bars.v_full[t], (nv >> 1) & 1) || !wait(&bars.p_full[t], (nv >> 1) & 1)) return false;
          tc::fence_after_sync();
          if (leader) {
#pragma unroll
            for (int w = 0; w < 2; ++w) pv(kColO + w * 128, t * 128 + w * kStep, w * kStep, kStep, t, i > 0);
            tc::umma_commit(&bars.v_empty[t]);
          }
          __syncwarp();
        }
      }
      return true;
    });
    }
  } else if (warp >= kSoftWarps) {
    regs_down<Roles<RT>::kDecRegs>();
    // ---- decoders ------------------------------------------------------------------------------
    constexpr int kPer = kDecWarps / 2, kTokens = kTcUnit / kPer, kBlks = kTokens / kBlkTok;  // warps, tokens and blocks of one
    using Sh = Share<D, kTokens>;
    const int dw = warp - kSoftWarps, kv = dw / kPer, wd = dw % kPer;  // K or V; tokens of the unit
    uint64_t* full = kv ? bars.v_full : bars.k_full;
    uint64_t* empty = kv ? bars.v_empty : &bars.s_full[RT - 1];
    // A lane has 32 channels, chunk c of a row, of tokens r + kTok * i: a warp's loads are contiguous. Its four 16-byte
    // stores of a vector go chunk by chunk; with c & 2 in another order, so that eight lanes' stores fall on different
    // banks (their rows' chunks c and c + 2 lie a multiple of 128 bytes apart).
    const int r = lane / Sh::kLanes, c = lane % Sh::kLanes, turn = c & 2;
    const uint32_t scale0 = turn ? 0x3232u : 0x1010u, scale1 = turn ? 0x1010u : 0x3232u;
    uint32_t st_at[4];
    {
      const int row = wd * kTokens + r;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st_at[i] = tc::smem_u32(smem + (kv ? L::oV : L::oK)) + (c >> 1) * L::kHalf + row * 128 +
                   ((((c & 1) * 4 + (i ^ turn)) ^ (row & 7)) << 4);
    }
    const uint8_t* codes = a.g.data + (kv ? piece_off(D, 2) : 0) + (r & 15) * (D / 2) + c * 16;
    const uint8_t* scales = a.g.data + (kv ? piece_off(D, 3) : piece_off(D, 1)) + (r & 15) * (D / 16) + c * 2;
    const int pmask = (1 << a.g.lp) - 1;
    const uint32_t least = kv ? 0u : 0xfc00fc00u;  // a V scale that is no number or below zero counts as zero
    uint32_t n = 0, seg = 0;
    parts([&](const Stream& x, int, int ua, int ub, int, int) {
      const int32_t* row = a.t.table + (size_t)x.s * a.t.maxp;
      // page numbers of 16 units and more at a time, a block a lane, and those of as many units behind them
      constexpr int kAhead = 32 / kBlks;
      auto tok_of = [&](int u, int b) { return u * kTcUnit + wd * kTokens + b * kBlkTok; };
      auto read_ids = [&](int u0) {
        const int u = u0 + lane / kBlks, tok = tok_of(u, lane % kBlks);
        const bool want = u < ub && tok < x.vis;
        const int id = want ? row[x.real(tok) >> a.g.lp] : -1;
        return want && !page_ok(a.g, id) ? -2 : id;
      };
      int ibase = ua, ids = read_ids(ua), ids_next = read_ids(ua + kAhead);
      auto load = [&](Sh& v, uint32_t& ok, int u) {
        if (u >= ub) return;
        if (u - ibase >= kAhead) {
          ids = ids_next;
          ibase += kAhead;
          ids_next = read_ids(ibase + kAhead);
        }
        ok = 0;
#pragma unroll
        for (int b = 0; b < kBlks; ++b) {
          const int id = __shfl_sync(kFull, ids, (u - ibase) * kBlks + b);
          const int tok = x.real(tok_of(u, b));
          const uint32_t blk = ((uint32_t)id << (a.g.lp - 4)) + ((tok & pmask) >> 4);  // of the pool's, below 2^32
          const uint64_t at = (uint64_t)blk * (uint32_t)blk_bytes(D);
          if (id >= 0) ok |= 1u << b;
          if (id == -2 && kv == 0 && lane == 0) status_or(a.status, KVC_STATUS_BAD_PAGE);
#pragma unroll
          for (int k = 0; k < Sh::V / kBlks; ++k) {
            const int i = b * (Sh::V / kBlks) + k;
            v.c[i] = id >= 0 ? ld_stream16(codes + at + k * Sh::kTok * (D / 2)) : make_uint4(0u, 0u, 0u, 0u);
            v.s[i] = id >= 0 ? ld_stream2(scales + at + k * Sh::kTok * (D / 16)) : 0u;
          }
        }
      };
      auto decode = [&](const Sh& v, uint32_t ok) {
        const int t = n & 1;
        if (!wait(&empty[t], ((n >> 1) & 1) ^ 1)) return false;
#pragma unroll
        for (int i = 0; i < Sh::V; ++i) {
          uint32_t w[4] = {v.c[i].x, v.c[i].y, v.c[i].z, v.c[i].w};
          if (D == 128 && turn) {
            const uint32_t y = w[0], z = w[1];
            w[0] = w[2], w[1] = w[3], w[2] = y, w[3] = z;
          }
          const uint32_t two = at_least2(e4m3x2_f16x2(v.s[i]), least);
          const uint32_t s2[2] = {__byte_perm(two, two, scale0), __byte_perm(two, two, scale1)};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h[4];
            e2m1x8_f16(w[k], h);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(st_at[k] + t * L::kTile + i * Sh::kTok * 128),
                         "r"(hmul2(h[0], s2[k >> 1])), "r"(hmul2(h[1], s2[k >> 1])), "r"(hmul2(h[2], s2[k >> 1])),
                         "r"(hmul2(h[3], s2[k >> 1]))
                         : "memory");
          }
        }
        if (kv == 0 && lane == 0) reinterpret_cast<uint8_t*>(&unit_ok[n & 3])[wd] = (uint8_t)ok;
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[t]);
        ++n;
        return true;
      };
      // rows two units ahead of their decoding, one for RT = 2, whose units take twice as long
      Sh v0, v1;
      uint32_t ok0 = 0, ok1 = 0;
      load(v0, ok0, ua);
      if (RT == 1) load(v1, ok1, ua + 1);
      // the first part's are the softmax warps' work
      if (seg > 0 && !queries(x, seg, dw, integral_constant<int, kDecWarps>())) return false;
      ++seg;
      for (int u = ua; u < ub; u += RT == 1 ? 2 : 1) {
        if (!decode(v0, ok0)) return false;
        load(v0, ok0, u + (RT == 1 ? 2 : 1));
        if (RT == 1 && u + 1 < ub) {
          if (!decode(v1, ok1)) return false;
          load(v1, ok1, u + 3);
        }
      }
      return true;
    });
  } else {
    regs_up<Roles<RT>::kSoftRegs>();
    // ---- softmax -------------------------------------------------------------------------------
    const int w = warp >> 2, rt = threadIdx.x & 127, rr = RT == 2 ? threadIdx.x : rt;  // group, row of its tile, of the block
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;                                // this warp's quarter of the lanes
    const uint32_t tO = tmem + kColO + w * 128 + lanes;
    uint32_t n = 0, seg = 0;  // units so far
    parts([&](const Stream& x, int vs, int ua, int ub, int U, int base) {
      const int m = ub - ua;
      if (seg == 0 && !queries(x, 0, warp, integral_constant<int, kSoftWarps>())) return false;
      int lim = x.vis, lo = 0;
      if (rr < x.rows) {
        const RowSeen y = row_seen(a, p, seen, x, x.r0 + rr);
        lo = y.lo;
        lim = y.hi;
        if (seen.mask) {  // for the units with the own tokens, the part's last
          const uint32_t* words = mask_words(a, p, seen, x, x.r0 + rr);
          asm volatile("prefetch.global.L1 [%0];\n" ::"l"(words));
          asm volatile("prefetch.global.L1 [%0];\n" ::"l"(words + seen.words - 1));
        }
      }
      const RowSeen all = all_see(p, seen, x);
      float ref = 0.f, l = 0.f, f = 0.f;
      bool none = true, fresh = true;  // the row has seen no token; one of the warp's rows has not
      for (int i = 0; i < m; ++i, ++n) {
        const uint32_t tS = tmem + lanes + (RT == 2 ? w * 128 : (n & 1) * 128 + w * kStep);
        if (!(RT == 2 && w == 0 ? wait(&bars.s_full[0], n & 1) : wait(&bars.s_full[RT - 1 + (n & 1)], (n >> 1) & 1))) return false;
        tc::fence_after_sync();
        // the factors were written before q_full, which precedes every s_full
        if (i == 0) f = *reinterpret_cast<volatile float*>(&row_f[seg % kFactors][rr]);
        // the unit's blocks that are there: one or two a byte, nearly always all
        using Word = typename std::conditional<kDecWarps == 16, uint64_t, uint32_t>::type;
        const Word by = *reinterpret_cast<volatile Word*>(&unit_ok[n & 3]);
        uint32_t blocks = 0xff;
        if (by != (kDecWarps == 16 ? (Word)0x0101010101010101ull : (Word)0x03030303u))
          blocks = kDecWarps == 16 ? (uint32_t)(by * 0x0102040810204080ull >> 56) : (uint32_t)by * 0x01041040u >> 24;
        // every row sees every token, and nearly always the reference holds: one straight run, the next chunk's logits on
        // their way
        uint32_t s[2][32];
        tc::tmem_ld32_async(tS, s[0]);
        if (RT == 1) tc::tmem_ld32_async(tS + kChunk, s[1]);
#pragma unroll
        for (int h = 0; h < RT; ++h) {
          const int part = RT == 2 ? h : w, tok0 = (ua + i) * kTcUnit + part * kStep;
          const uint32_t ok = blocks >> 4 * part & 15;
          bool slow = fresh || ok != 15 || tok0 + kStep > all.hi || (tok0 < all.lo && tok0 + kStep > x.sinks);
          const float2 f2 = make_float2(f, f), ref2 = make_float2(-ref, -ref);
          uint32_t o[2][16];
          float l2[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (RT == 2 || e == 0) {
              tc::tmem_wait();
              tc::tmem_regs_ready(s[e]);
              if (RT == 1) tc::tmem_regs_ready(s[1]);
            }
            if (RT == 2 && 2 * h + e < 3) tc::tmem_ld32_async(tS + (2 * h + e + 1) * kChunk, s[e ^ 1]);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float2 y = fma2(make_float2(__uint_as_float(s[e][2 * k]), __uint_as_float(s[e][2 * k + 1])), f2, ref2);
              y.x = ex2(y.x);
              y.y = ex2(y.y);
              sum[k & 1] = add2(sum[k & 1], y);
              o[e][k] = pack2(y.x, y.y);
            }
            sum[0] = add2(sum[0], sum[1]);
            l2[e] = sum[0].x + sum[0].y;
          }
          slow = __any_sync(kFull, slow || !(l2[0] <= kMost && l2[1] <= kMost));
          if (!slow) {
            l += l2[0] + l2[1];
            tmem_st16(tS + h * (kStep / 2), o[0]);
            tmem_st16(tS + h * (kStep / 2) + 16, o[1]);
          }
          if (__builtin_expect(slow, 0)) {
            if (h + 1 < RT) {  // the load under way is over before anything else has the registers
              tc::tmem_wait();
              tc::tmem_regs_ready(s[0]);
            }
            // A chunk at a time: what the row sees of it, its maximum, the reference raised where that passes it by more
            // than kOff, what was summed so far rescaled, and the probabilities.
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
              const int c = 2 * h + e;  // of the unit's chunks in this group's columns
              const uint32_t bits = row_bits(a, p, seen, x, rr, lo, lim, tok0 + e * kChunk, ok >> 2 * e);
              uint32_t z[32];
              tc::tmem_ld32_async(tS + c * kChunk, z);
              tc::tmem_wait();
              tc::tmem_regs_ready(z);
              float y[32], m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                y[k] = bits >> k & 1 ? fmaf(__uint_as_float(z[k]), f, -ref) : -INFINITY;
                m4[k & 3] = fmaxf(m4[k & 3], y[k]);
              }
              const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
              float up = 0.f, down = 1.f;
              if (none ? mx > -INFINITY : mx > kOff) {
                up = ceilf(mx) - kOff;
                if (!none) down = ex2(-up);
                none = false;
                ref += up;
                l *= down;
              }
              if (__any_sync(kFull, down != 1.f)) {
                // O holds the part's earlier units, and P this one's earlier chunks
                if (RT == 1 && i > 0 && !wait(&bars.v_empty[(n - 1) & 1], ((n - 1) >> 1) & 1)) return false;
                tmem_st_wait();
                tc::fence_after_sync();
                if (i > 0)
#pragma unroll 1
                  for (int k = 0; k < D / 16; ++k) scale_cols16(tO + 16 * k, down);
#pragma unroll 1
                for (int k = 0; k < c; ++k) scale_halves16(tS + 16 * k, down);
                tmem_st_wait();
              }
              uint32_t o[16];
              float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float p0 = ex2(y[2 * k] - up), p1 = ex2(y[2 * k + 1] - up);
                sum[k & 1] = add2(sum[k & 1], make_float2(p0, p1));
                o[k] = pack2(p0, p1);
              }
              l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
              tmem_st16(tS + c * (kChunk / 2), o);
            }
            fresh = __any_sync(kFull, none);
          }
        }
        tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[RT == 2 ? w : n & 1]);
      }
      // the last product is done (RT = 1: the one two units before was, or S would not have been written)
      if (!(RT == 2 ? wait(&bars.pv_done[w], seg & 1) : wait(&bars.v_empty[(n - 1) & 1], ((n - 1) >> 1) & 1))) return false;
      tc::fence_after_sync();
      const bool whole = ua == 0 && ub == U;
      if (ua == 0 && threadIdx.x == 0)
        p.span[vs] = make_int2(blockIdx.x, whole ? (int)blockIdx.x : split.owner(base + U - 1));
      const size_t at = out_row(a, p, x, x.r0 + rr);
      const size_t slot = (size_t)blockIdx.x * 2 + (ua == 0 ? 1 : 0), prow = slot * kRows + rr;
      float mm = ref, ll = l, c0 = 1.f, c1 = 0.f;
      if constexpr (RT == 1) {  // the groups' results together
        row_ml[w][rt] = make_float2(ref, l);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.merge);
        if (!wait(&bars.merge, 0)) return false;
        tc::fence_after_sync();
        const float2 y0 = row_ml[0][rt], y1 = row_ml[1][rt];
        mm = y1.y > 0.f ? (y0.y > 0.f ? fmaxf(y0.x, y1.x) : y1.x) : y0.x;
        c0 = y0.y > 0.f ? ex2(y0.x - mm) : 0.f, c1 = y1.y > 0.f ? ex2(y1.x - mm) : 0.f;
        if (y0.y != y0.y || y1.y != y1.y) c0 = NAN;
        ll = y0.y * c0 + y1.y * c1;
      }
      const float inv = ll == 0.f ? 0.f : a.g.ts[1] / ll;
      constexpr int kCols = RT == 2 ? D : D / 2;  // RT = 1: each group writes half of the channels
      const int k0 = RT == 2 ? 0 : w * kCols;
#pragma unroll 1
      for (int k = k0; k < k0 + kCols; k += 32) {
        uint32_t o0[32], o1[RT == 1 ? 32 : 1];
        tc::tmem_ld32_async(tmem + kColO + (RT == 2 ? w * 128 : 0) + lanes + k, o0);
        if constexpr (RT == 1) tc::tmem_ld32_async(tmem + kColO + 128 + lanes + k, o1);
        tc::tmem_wait();
        tc::tmem_regs_ready(o0);
        if constexpr (RT == 1) tc::tmem_regs_ready(o1);
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if constexpr (RT == 1)
            o[e] = fmaf(__uint_as_float(o1[e]), c1, __uint_as_float(o0[e]) * c0);
          else
            o[e] = __uint_as_float(o0[e]);
        if (rr < x.rows) {
          if (whole) {
            alignas(16) T y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = from_f32<T>(o[e] * inv);
            uint4* op = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + at * D + k);
#pragma unroll
            for (int e = 0; e < 4; ++e) op[e] = reinterpret_cast<const uint4*>(y)[e];
          } else {
            float* op = p.part + slot * D * kRows + part_at<kRows>(k, rr);
#pragma unroll
            for (int e = 0; e < 4; ++e) st_f8(op + part_at<kRows>(8 * e, 0), o + 8 * e);
          }
        }
      }
      if ((RT == 2 || w == 0) && rr < x.rows) {
        if (whole) {
          if (a.lse) a.lse[at] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
        } else {
          p.ml[prow] = make_float2(mm, ll);
        }
      }
      // O is read by no thread any more before the next part's products write it (RT = 2: those wait for this group's
      // probabilities)
      tc::fence_before_sync();
      if constexpr (RT == 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.merge);
        if (!wait(&bars.merge, 1)) return false;
      }
      ++seg;
      if (rt == 0) parts_done[w] = seg;
      return true;
    });
  }
  __syncwarp();
  tc::fence_before_sync();
  if (__syncthreads_or(*ab)) {
    // a role gave up and the others followed: what this CTA leaves undone must not be taken for what lay in the
    // workspace. Streams that begin here hold no part at all, those that began before nothing of this CTA's.
    if (warp < kSoftWarps) {  // they have the registers for it, and a thread a row
      static_assert(32 * kSoftWarps >= kRows, "a thread a row");
      const int done = min(parts_done[0], parts_done[1]);
      int i = 0;
      parts([&](const Stream&, int vs, int ua, int, int, int) {
        if (i++ < done) return true;
        if (ua == 0 && threadIdx.x == 0) p.span[vs] = make_int2(-1, -1);
        if (threadIdx.x < kRows)
          p.ml[((size_t)blockIdx.x * 2 + (ua == 0 ? 1 : 0)) * kRows + threadIdx.x] = make_float2(0.f, 0.f);
        return true;
      });
    }
    // products under way end before their memory goes
    if (warp >= kIssuer && warp < kIssuer + kIssuers) {
      if (elect_one()) tc::umma_commit(&bars.drain);  // the lane that issued the products
      __syncwarp();
      const uint64_t since = clock_ns();
      while (!__all_sync(kFull, mbar_ready(&bars.drain, 0)) && !__any_sync(kFull, clock_ns() - since > kWaitNs)) {
      }
    }
    __syncthreads();
  }
  if (warp == kIssuer) tc::tmem_dealloc(tmem, kTmemCols);
}

template <typename T, int D, int RT>
int go(const AttendArgs& a, const AttendPlan& p, const SeenArgs& m, cudaStream_t s) {
  auto k = attend_rows_kernel<T, D, RT>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D, RT>::bytes) != cudaSuccess)
    return KVC_ERR_LAUNCH;
  return launch_pdl(k, dim3(p.grid), dim3(kThreadsOf<RT>), Lay<D, RT>::bytes, s, false, a, p, m) == cudaSuccess ? KVC_OK
                                                                                                         : KVC_ERR_LAUNCH;
}

}  // namespace

int launch_attend_rows(const AttendArgs& a, const AttendPlan& p, const SeenArgs& m, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (p.rb == kTcRows) return a.g.D == 128 ? go<B, 128, 1>(a, p, m, s) : go<B, 64, 1>(a, p, m, s);
  return a.g.D == 128 ? go<B, 128, 2>(a, p, m, s) : go<B, 64, 2>(a, p, m, s);
}

}  // namespace kvc
