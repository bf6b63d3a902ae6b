// page_attend_tc.cuh -- what the tcgen05 kernels of the paged attention share: waits that follow a role which gave up,
// descriptors, products and tensor-memory moves.
#pragma once

#include "page_attend.cuh"

namespace kvc {

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(tc::smem_u32(bar)) : "memory");
}
// The first poll in line, the waiting out of it (the roles' loops stay short: five warps of different roles
// share an SM quarter's instruction cache). Gives up as soon as another role has.
__device__ __noinline__ static bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  if (mbar_wait_until(bar, parity, [&] { return *abort_flag != 0; })) return true;
  if (!*abort_flag) status_or(status, KVC_STATUS_TIMEOUT);
  *abort_flag = 1;
  return false;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

// fp16 A and B, fp32 accumulator; b_mn: B lies with its N dimension contiguous
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// B operand with channels contiguous: 128-byte rows of 64 channels, a row per token, 8-token groups 1024
// bytes apart (stride offset), the next 64 channels `next64` bytes on (leading offset)
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t next64) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(next64 >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  tc::umma_bf16(d, a, b, idesc, acc);  // kind::f16; the descriptor names the types
}
// A from tensor memory: lane = row, a 32-bit column two reduction elements
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// 16 columns of this thread's lane, without waiting
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 16 columns of this thread's lane: fp32 numbers, or fp16 pairs, times c. The thread's own stores before it are done.
__device__ __forceinline__ void scale_cols16(uint32_t taddr, float c) {
  uint32_t o[16];
  tmem_ld16(taddr, o);
  tc::tmem_wait();
  tc::tmem_regs_ready(o);
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * c);
  tmem_st16(taddr, o);
}
__device__ __forceinline__ void scale_halves16(uint32_t taddr, float c) {  // c may lie below fp16's numbers
  uint32_t o[16];
  tmem_ld16(taddr, o);
  tc::tmem_wait();
  tc::tmem_regs_ready(o);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float2 v = f16x2_f32(o[e]);
    o[e] = pack2(v.x * c, v.y * c);
  }
  tmem_st16(taddr, o);
}

}  // namespace kvc
