// fd_tcgen05.cuh -- fifth-generation tensor core primitives shared by the
// tcgen05 kernels (fd_split_tc.cu, fd_prefill.cuh): descriptors, product
// issue, tensor-memory loads and stores, fences, operand layouts.
#pragma once

#include "fd_split_mma.cuh"

namespace fd {
namespace tc {

using mma::smem_u32;

// Shared-memory matrix descriptor: 128-byte swizzle, start address, leading
// and stride byte offsets (bytes, multiples of 16), descriptor version 1.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Instruction descriptor, kind::f16: f16 (or bf16) A and B, f32 accumulator, A
// K-major, B K-major (b_mn = 0) or MN-major (b_mn = 1), M x N.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn, int bf16 = 0) {
  return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// The same, issued by the lane whose `lead` is set while the whole warp runs
// the code around it: no branch, and descriptors in uniform registers.
__device__ __forceinline__ void umma_lead(uint32_t lead, uint32_t d, uint64_t a, uint64_t b,
                                          uint32_t idesc, int acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}

// With A in tensor memory (16-bit pairs, two to a column).
__device__ __forceinline__ void umma_ts_lead(uint32_t lead, uint32_t d, uint32_t a, uint64_t b,
                                             uint32_t idesc, int acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void umma_commit_lead(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// Arrives on `bar` once every tcgen05.mma this thread issued so far is done.
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// generic-proxy shared-memory writes -> visible to the tensor core
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Non-blocking test of a barrier phase.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

#define TC_REGS32(r, o)                                                                    \
  "=r"(r[o + 0]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]),          \
      "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7]), "=r"(r[o + 8]), "=r"(r[o + 9]),      \
      "=r"(r[o + 10]), "=r"(r[o + 11]), "=r"(r[o + 12]), "=r"(r[o + 13]), "=r"(r[o + 14]), \
      "=r"(r[o + 15]), "=r"(r[o + 16]), "=r"(r[o + 17]), "=r"(r[o + 18]), "=r"(r[o + 19]), \
      "=r"(r[o + 20]), "=r"(r[o + 21]), "=r"(r[o + 22]), "=r"(r[o + 23]), "=r"(r[o + 24]), \
      "=r"(r[o + 25]), "=r"(r[o + 26]), "=r"(r[o + 27]), "=r"(r[o + 28]), "=r"(r[o + 29]), \
      "=r"(r[o + 30]), "=r"(r[o + 31])
#define TC_FREGS32(v, o)                                                                  \
  "f"(v[o + 0]), "f"(v[o + 1]), "f"(v[o + 2]), "f"(v[o + 3]), "f"(v[o + 4]), "f"(v[o + 5]), \
      "f"(v[o + 6]), "f"(v[o + 7]), "f"(v[o + 8]), "f"(v[o + 9]), "f"(v[o + 10]),           \
      "f"(v[o + 11]), "f"(v[o + 12]), "f"(v[o + 13]), "f"(v[o + 14]), "f"(v[o + 15]),       \
      "f"(v[o + 16]), "f"(v[o + 17]), "f"(v[o + 18]), "f"(v[o + 19]), "f"(v[o + 20]),       \
      "f"(v[o + 21]), "f"(v[o + 22]), "f"(v[o + 23]), "f"(v[o + 24]), "f"(v[o + 25]),       \
      "f"(v[o + 26]), "f"(v[o + 27]), "f"(v[o + 28]), "f"(v[o + 29]), "f"(v[o + 30]),       \
      "f"(v[o + 31])
#define TC_LIST32                                                                        \
  "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23," \
  "%24,%25,%26,%27,%28,%29,%30,%31}"
#define TC_LIST32_1                                                                        \
  "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24," \
  "%25,%26,%27,%28,%29,%30,%31,%32}"

// 32 columns of this thread's accumulator row.  M = 128: lane l of the warp's
// lane quarter, columns [c, c + 32).  M = 64 (rows in lanes 0..15 of each
// quarter): lanes 0..15 read columns [c, c + 32) of rows 0..15 and lanes
// 16..31 columns [c + 64, c + 96) of the same rows.
template <int M>
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  if constexpr (M == 128) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " TC_LIST32 ", [%32];"
                 : TC_REGS32(r, 0)
                 : "r"(taddr));
  } else {
    asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x32.b32 " TC_LIST32 ", [%32], 64;"
                 : TC_REGS32(r, 0)
                 : "r"(taddr));
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

template <int M>
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  if constexpr (M == 128) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], " TC_LIST32_1 ";" ::"r"(taddr),
                 TC_FREGS32(v, 0)
                 : "memory");
  } else {
    asm volatile("tcgen05.st.sync.aligned.16x32bx2.x32.b32 [%0], 64, " TC_LIST32_1 ";" ::"r"(taddr),
                 TC_FREGS32(v, 0)
                 : "memory");
  }
}

// 16 columns of 32-bit words, M = 128 layout.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Operand layouts (byte offsets inside a buffer), 128-byte swizzle: the
// 16-byte chunk index inside a 128-byte row is XORed with the row index mod 8.
//   K-major [rows][K] f16: blocks of 64 K-elements, each rows x 128 bytes.
__device__ __forceinline__ uint32_t kmajor_chunk(uint32_t rows, int r, int c16) {
  return (uint32_t)(c16 >> 3) * rows * 128u + (uint32_t)r * 128u +
         ((uint32_t)((c16 & 7) ^ (r & 7)) << 4);
}
//   MN-major V [tile tokens][128 dims] f16: dims in two 64-dim atoms of
//   tile x 128 bytes, tokens in groups of 8 rows of 128 bytes, 1 KB apart.
__device__ __forceinline__ uint32_t vmn_chunk(uint32_t tile, int t, int c16) {
  return (uint32_t)(c16 >> 3) * tile * 128u + (uint32_t)(t >> 3) * 1024u +
         (uint32_t)(t & 7) * 128u + ((uint32_t)((c16 & 7) ^ (t & 7)) << 4);
}

}  // namespace tc
}  // namespace fd
