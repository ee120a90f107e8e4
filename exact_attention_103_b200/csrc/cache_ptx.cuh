// cache_ptx.cuh -- inline-PTX wrappers that only the attention over the paged cache uses,
// beside those of sm100_ptx.cuh.
#pragma once
#include "sm100_ptx.cuh"

namespace attn {

// 4-D tiled bulk-tensor load into this CTA's shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                            int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::"
      "cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}

// Shared-memory matrix descriptor with 64-byte swizzle (layout type 4): rows of 64 bytes,
// 16-byte units permuted over groups of 8 rows (512 bytes).
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
  d |= 1ull << 46;
  d |= 4ull << 61;
  return d;
}

// Packed fp32 arithmetic with every operand per element: y = x * a + b.
__device__ __forceinline__ void ffma2_vv(float& y0, float& y1, float x0, float x1, float a0, float a1, float b0,
                                         float b1) {
  asm("{\n\t.reg .b64 xa, aa, ba, ya;\n\t"
      "mov.b64 xa, {%2, %3};\n\tmov.b64 aa, {%4, %5};\n\tmov.b64 ba, {%6, %7};\n\t"
      "fma.rn.f32x2 ya, xa, aa, ba;\n\tmov.b64 {%0, %1}, ya;\n\t}"
      : "=f"(y0), "=f"(y1)
      : "f"(x0), "f"(x1), "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// Two values rounded to 4 significant bits (Veltkamp's splitting: t = (2^20 + 1) x, t - (t - x)).
// t is one fma, 2^20 x + x: a product would be contracted with the subtraction behind it.
__device__ __forceinline__ void upper4_x2(float& h0, float& h1, float x0, float x1) {
  float t0, t1, u0, u1;
  ffma2_bv(t0, t1, x0, x1, 1048576.f, x0, x1);
  fsub2(u0, u1, t0, t1, x0, x1);
  fsub2(h0, h1, t0, t1, u0, u1);
}

// Four non-negative values below 2^16 as three E5M2 terms each, one byte per value and term.  E5M2 is
// the upper byte of fp16: each value is rounded to fp16 (2^-11), the first two terms are upper bytes cut
// off, what they leave is exact in fp16, and the last is rounded.  The first leaves less than 2^-2 of the
// value's power of two, the second less than 2^-5, the third at most 2^-9, or half of E5M2's smallest
// step, 2^-17.  A NaN stays one in the first term.
__device__ __forceinline__ uint32_t fp16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t less_upper_bytes(uint32_t x) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(x & 0xff00ff00u));
  return r;
}
__device__ __forceinline__ void split_e5m2x4(float x0, float x1, float x2, float x3, uint32_t& t1, uint32_t& t2, uint32_t& t3) {
  const uint32_t a = fp16_pair(x0, x1), b = fp16_pair(x2, x3);
  const uint32_t ar = less_upper_bytes(a), br = less_upper_bytes(b);
  // half of the last term's step, carried into its upper byte; halves of fp16 numbers never
  // overflow into one another, as what is left is small
  const uint32_t as = less_upper_bytes(ar) + 0x00800080u, bs = less_upper_bytes(br) + 0x00800080u;
  t1 = __byte_perm(a, b, 0x7531);
  t2 = __byte_perm(ar, br, 0x7531);
  t3 = __byte_perm(as, bs, 0x7531);
}

// 16 columns of this warp's 32 lanes, complete on return (as tmem_ld_x8 and its wider forms).
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr) : "memory");
}

// 16 of this warp's lanes (the first, or from 16 on), two column groups: thread i < 16 has lane i's
// columns from taddr on, thread 16 + i the same lane's from taddr + N on (N registers each).
__device__ __forceinline__ void tmem_ld_duo(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16], 16;\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr) : "memory");
}
// The same of the first 16 lanes and of the lanes behind them, 32 columns each.
__device__ __forceinline__ void tmem_ld_duo_both(uint32_t taddr, uint32_t (&r)[32], uint32_t (&q)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64], 32;\n\t"
               "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65], 32;\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15]), "=r"(q[16]), "=r"(q[17]), "=r"(q[18]), "=r"(q[19]), "=r"(q[20]), "=r"(q[21]), "=r"(q[22]), "=r"(q[23]), "=r"(q[24]), "=r"(q[25]), "=r"(q[26]), "=r"(q[27]), "=r"(q[28]), "=r"(q[29]), "=r"(q[30]), "=r"(q[31])
               : "r"(taddr), "r"(taddr + (16u << 16)) : "memory");
}
__device__ __forceinline__ void tmem_st_duo(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x32bx2.x8.b32 [%0], 8, {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}

}  // namespace attn
