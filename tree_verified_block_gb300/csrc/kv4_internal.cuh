// Shared by the kernels on 4-bit K/V caches (glance_kv4): the row format, host
// checks of a view, and the conversions between codes, scales and values.
//
// A row (one slot of one kv head of K or V) is 128 codes of 4 bits in 64 bytes
// and 8 e4m3 scales, one per 16 elements. A code has 2 significant bits and a
// scale 4, so code * scale has at most 6 and lies in [2^-10, 2688] or is 0:
// f16 (and bf16) hold it exactly. Only the fp32 global factor needs rounding.
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include "glance_internal.cuh"

namespace glance {

// status words of the units added after the first five families; each one is
// reported with a family (api.cu)
GLANCE_DECLARE_STATUS_WORD(status_kv4)
GLANCE_DECLARE_STATUS_WORD(status_kv4_attention)
GLANCE_DECLARE_STATUS_WORD(status_rope)

constexpr int kKv4D = 128;           // head_dim
constexpr int kKv4CodeBytes = 64;    // codes of one row
constexpr int kKv4ScaleBytes = 8;    // scales of one row
constexpr int kKv4MaxCap = 1 << 30;  // slots per head
constexpr int kKv4MaxHeads = 1024;   // kv heads

// Checks of one view, shared by the 4-bit calls.
inline glance_status check_kv4(const char* who, const glance_kv4& x, int rows, int index) {
  if (!x.k || !x.k_scale || !x.v || !x.v_scale || !x.t_len)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: null array in view %d", who, index);
  if (x.head_dim != kKv4D)
    return fail(GLANCE_ERR_UNSUPPORTED, "%s: 4-bit caches need head_dim 128 (view %d)", who, index);
  if (x.n_kv_heads < 1 || x.n_kv_heads > kKv4MaxHeads || x.t_cap < rows || x.head_stride < x.t_cap || (x.head_stride & 1))
    return fail(GLANCE_ERR_INVALID_ARG,
                "%s: need 1 <= n_kv_heads <= %d, t_cap >= rows and an even head_stride >= t_cap (view %d)", who, kKv4MaxHeads,
                index);
  if (x.t_cap > kKv4MaxCap) return fail(GLANCE_ERR_UNSUPPORTED, "%s: t_cap too large (view %d)", who, index);
  if (!aligned16(x.k) || !aligned16(x.k_scale) || !aligned16(x.v) || !aligned16(x.v_scale))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: codes and scales must be 16-byte aligned (view %d)", who, index);
  const float lo = 8.6736174e-19f, hi = 1.1529215e18f;  // 2^-60, 2^60
  if (!(x.k_global >= lo && x.k_global <= hi) || !(x.v_global >= lo && x.v_global <= hi))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: k_global and v_global must be in [2^-60, 2^60] (view %d)", who, index);
  return GLANCE_OK;
}

}  // namespace glance

namespace glance_dev {

// Eight codes (one word, element 0 in the lowest bits) as four pairs of f16,
// elements (0, 1), (2, 3), (4, 5), (6, 7): the hardware conversion, exact.
__device__ __forceinline__ void codes8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two e4m3 scales (the low 16 bits of w, the first in the lower byte) as f16, exact.
__device__ __forceinline__ uint32_t scales2_to_f16(uint32_t w) {
  uint32_t h;
  asm("{\n .reg .b16 t, u;\n mov.b32 {t, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Eight fp32 values as codes (nearest even, at most 6 in magnitude), the first in the lowest bits.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// An fp32 value >= 0 as an e4m3 scale (nearest even, at most 448).
__device__ __forceinline__ uint32_t scale1(float s) {
  uint32_t r;
  asm("{\n .reg .b16 t, z;\n mov.b16 z, 0;\n cvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n mov.b32 %0, {t, z};\n}\n"
      : "=r"(r)
      : "f"(s), "f"(0.f));
  return r;
}

// tcgen05.wait::ld tied to the 32 registers of a load before it, so that no
// use of them can be moved in front of the wait.
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// 32 lanes x 64 columns with the wait in the same statement, so that no use of
// a register can be moved in front of it.
__device__ __forceinline__ void tmem_row64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
}

// 32 lanes x 16 columns, likewise.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// f16 codes as bf16 times 2^-112: both formats have the sign on top, and a
// shift by three puts the exponent's five bits and the mantissa's top in place
// (a code has one fraction bit, so nothing falls out). Exact.
__device__ __forceinline__ uint32_t f16_codes_to_bf16(uint32_t h) {
  return ((h >> 3) & 0x0FFF0FFFu) | (h & 0x80008000u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Two fp32 values in one register pair, each operation as on one; but a mul_f2
// whose only use is an add_f2 becomes one fused operation (seen with nvcc 13.0):
// where the product's rounding counts, __fmul_rn on each half.
__device__ __forceinline__ unsigned long long pair_f2(float lo, float hi) {
  unsigned long long v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void split_f2(unsigned long long v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma_f2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ unsigned long long add_f2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long mul_f2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 16 bytes global -> shared without registers; a thread waits for its own copies.
__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

}  // namespace glance_dev
