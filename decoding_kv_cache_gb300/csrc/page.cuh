// page.cuh -- the paged 4-bit cache: geometry, the block format and its decoding.
//
// A page holds `page` tokens (a power of two, 16..256) of one KV head of one layer as a run of
// 16-token blocks; a block is 18 D bytes, every piece of it 16-byte aligned:
//   K codes  [16][D/2]   two e2m1 codes a byte, the even channel in the low nibble
//   K scales [16][D/16]  one e4m3 scale per 16 channels
//   V codes  [16][D/2]
//   V scales [16][D/16]
// A code stands for ts * scale * e2m1(code), ts = the pool's k_scale or v_scale. Keeping a block's
// four pieces side by side makes any run of blocks one contiguous copy, and a token's 4.5 bits a
// value are read from a single place. scale * e2m1 has at most six significant bits and lies in
// [2^-10, 2688]: it is exact in fp16, which is what the attention kernels multiply.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kvc_internal.cuh"

namespace kvc {

constexpr int kBlkTok = 16;  // tokens of a block
constexpr int kPageMax = 256;

struct PoolGeom {
  int D, lp, npages;  // head dimension, log2(tokens per page), pages
  float ts[2];        // k_scale, v_scale
  uint8_t* data;
  int32_t* refs;
  int32_t* free_list;
  int32_t* nfree;
};
struct PageTab {
  int L, B, Hkv, S, maxp;  // S = L * B * Hkv streams
  int32_t* table;          // [S][maxp]
  int32_t* len;            // [S]
};

// Division of 0 <= n < 2^31 by a fixed d >= 1 (Granlund and Montgomery: with 2^s >= d and m = ceil(2^(31+s) / d)
// the product n m / 2^(31+s) exceeds n / d by less than 1 / d).
struct FastDiv {
  uint32_t m;
  int sh, d;
  static FastDiv make(int d) {
    int s = 0;
    while ((1LL << s) < d) ++s;
    return FastDiv{(uint32_t)(((1ULL << (31 + s)) + d - 1) / d), 31 + s, d};
  }
  __device__ __forceinline__ int div(int n) const { return (int)(((unsigned long long)(uint32_t)n * m) >> sh); }
};

// Workspace of the page operators (kvc_page_workspace_size).
struct PageWs {
  int32_t* head;     // [0] nfree on entry, [1] pages the call took (compaction; -1: too few)
  uint32_t* gone;    // one bit per page: its last reference went in this call
  int32_t* need;     // [S] pages a stream takes (bit 30: its last page is copied)
  int32_t* sums;     // [ceil(S/256)] their sums
  int4* plan;        // [S] compaction: first row written, kept, length, flags
  int32_t* newtab;   // [2][S][maxp] compaction: the destination pages (-1: one to be taken), for K and V
  size_t zero_bytes;
};

__host__ __device__ constexpr int blk_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int piece_off(int D, int piece) {  // K codes, K scales, V codes, V scales
  return piece == 0 ? 0 : piece == 1 ? 8 * D : piece == 2 ? 9 * D : 17 * D;
}

__device__ __forceinline__ uint8_t* block_of(const PoolGeom& g, int page_id, int blk_in_page) {
  return g.data + ((size_t)page_id * (size_t)(1 << (g.lp - 4)) + blk_in_page) * (size_t)blk_bytes(g.D);
}
__device__ __forceinline__ bool page_ok(const PoolGeom& g, int id) { return (unsigned)id < (unsigned)g.npages; }
__host__ __device__ __forceinline__ int pages_of(int n, int lp) { return (int)(((long long)n + (1 << lp) - 1) >> lp); }

// the four bytes of a word (eight e2m1 codes) to four fp16 pairs, a byte's low nibble in the low half
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b1;\n cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// two e4m3 scales to fp16, the low byte in the low half
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ float2 f16x2_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float e4m3_f32(uint32_t b) { return f16x2_f32(e4m3x2_f16x2(b)).x; }

enum { kCompactBad = 1, kCompactMoves = 2 };  // PageWs::plan.w

// ---- launchers (arguments already validated) ---------------------------------------------------
int page_push(const PoolGeom& g, const PageWs& w, cudaStream_t s);                              // marked pages to the free list
int page_finish_compact(const PoolGeom& g, const PageTab& t, const PageWs& w, cudaStream_t s);  // and what a compaction leaves
int launch_page_init(const PoolGeom& g, const PageTab* t, cudaStream_t s);
int launch_page_extend(const PoolGeom& g, const PageTab& t, const int32_t* add, int add_all, int32_t* start,
                       int32_t* status, const PageWs& w, cudaStream_t s);
int launch_page_free(const PoolGeom& g, const PageTab& t, const int32_t* drop, int drop_all, int32_t* status,
                     const PageWs& w, cudaStream_t s);
int launch_page_fork(const PoolGeom& g, const PageTab& t, const int32_t* parent, const PageTab& out, int32_t* status,
                     const PageWs& w, cudaStream_t s);
int launch_page_compact(const PoolGeom& g, const PageTab& t, const int32_t* kept_idx, const int32_t* kept_len,
                        int stride, int per_seq, int32_t* status, const PageWs& w, cudaStream_t s);
int launch_page_slide(const PoolGeom& g, const PageTab& t, int window, int sinks, int32_t* gone, int32_t* status,
                      const PageWs& w, cudaStream_t s);
int launch_page_accept(const PoolGeom& g, const PageTab& t, int T, const int32_t* path, const int32_t* n_path,
                       const int32_t* n_q, int32_t* status, const PageWs& w, cudaStream_t s);
int launch_tree_mask(int B, int T, const int32_t* parent, const int32_t* n_q, int window, uint32_t* mask, int32_t* depth,
                     int32_t* status, cudaStream_t s);
int launch_tree_verify(int B, int T, const int32_t* parent, const int32_t* draft, const int32_t* target,
                       const int32_t* n_q, int32_t* path, int32_t* n_path, int32_t* next, int32_t* status, cudaStream_t s);

struct RowStrides {  // in elements
  long long b, t, h;
};
struct StoreArgs {
  PoolGeom g;
  PageTab t;
  const void* x[2];  // K, V rows
  RowStrides xs[2];
  int T;
  FastDiv by_T, by_hkv;
  float inv6[2];  // 1 / (6 k_scale), 1 / (6 v_scale)
  const int32_t* n;      // [B] or null
  const int32_t* start;  // [S]
  int32_t* status;
};
int launch_page_store(const StoreArgs& a, int dtype, cudaStream_t s);
struct ReadArgs {
  PoolGeom g;
  PageTab t;
  void* out[2];  // K, V: [S][ncap][D], either may be null
  const int32_t* first;
  int first_all, count;
  FastDiv by_count;
  long long ncap;
  int32_t* status;
};
int launch_page_read(const ReadArgs& a, int dtype, cudaStream_t s);

struct AttendArgs {
  PoolGeom g;
  PageTab t;  // one layer
  const void* q;
  RowStrides qs;
  void* out;   // [B][T][Hq][D]
  float* lse;  // [B][T][Hq] or null
  int Hq, T;
  const int32_t* n_q;  // [B] or null
  float scale;         // of the dot products, k_scale included
  int32_t* status;
  void* ws;
  int fault;  // kvc_debug_fault 2 (0 in normal use)
};
// What a query of kvc_page_attend_masked sees; all but sinks, window <= kSeenAll (longer than any stream).
constexpr int kSeenAll = 1 << 30;
struct SeenArgs {
  int window, sinks;     // kSeenAll: no window
  const uint32_t* mask;  // [B][T][words] or null
  const int32_t* depth;  // [B][T] or null
  int words;
};
bool attend_fits(const AttendArgs& a);
size_t attend_ws_bytes(const PoolGeom& g, const PageTab& t, int Hq, int T);
int launch_page_attend(const AttendArgs& a, int dtype, cudaStream_t s);
size_t attend_masked_ws_bytes(const PoolGeom& g, const PageTab& t, int Hq, int T, const SeenArgs& m);
int launch_page_attend_masked(const AttendArgs& a, const SeenArgs& m, int dtype, cudaStream_t s);

}  // namespace kvc
