// Device helpers of the attention over a paged cache: copies into shared memory,
// conversions, exponentials.
#pragma once

#include "fo_device.cuh"
#include "fo_ops.h"

namespace fo_ops {

using fo::smem_u32;

constexpr uint64_t kWaitNs = 2000000000ull;   // every wait's bound
constexpr float kLazy = 8.f;                  // growth of a row's maximum (base 2) that is let pass

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts_f(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ float lds_f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(a));
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^(a - b), and 0 for b = -infinity (a row that has seen nothing).
__device__ __forceinline__ float ex2_below(float a, float b) { return b == -INFINITY ? 0.f : ex2(a - b); }
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 bytes (exactly) as two f16.
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of_e4m3_high(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// A weight is 2^(s f - m), with the product unrounded and m the rounded product of
// the largest score. Past 2^31 that rounding alone is more than a power of two in
// fp32 holds, and for f16 weights (of up to 2^15 without it) from 2^24 on. With
// this power of two on f and m, m stays below 2^30 (2^23). Scores so large then
// differ by more than a weight's range, or (from 2^23 on) by less than what their
// sums' roundings leave open.
template <bool F16>
__device__ __forceinline__ float held_back(float m) {
  const int over = (int)(__float_as_uint(m) >> 23 & 0xffu) - (127 + (F16 ? 22 : 29));
  return over > 0 ? __uint_as_float((uint32_t)(127 - over) << 23) : 1.f;
}

// The sign bits of the halves (or, of e4m3, bytes) that are no finite numbers.
template <bool E8>
__device__ __forceinline__ uint32_t odd_of(uint32_t w) {
  return E8 ? ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u : ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
template <bool E8>
__device__ __forceinline__ uint32_t odd_of(const uint4& v) { return odd_of<E8>(v.x) | odd_of<E8>(v.y) | odd_of<E8>(v.z) | odd_of<E8>(v.w); }
// Zeros in their places.
template <bool E8>
__device__ __forceinline__ uint32_t even_of(uint32_t w) {
  const uint32_t odd = odd_of<E8>(w);
  return w & ~((odd >> (E8 ? 7 : 15)) * (E8 ? 0xffu : 0xffffu));
}
template <bool E8>
__device__ __forceinline__ uint4 even_of(const uint4& v) { return make_uint4(even_of<E8>(v.x), even_of<E8>(v.y), even_of<E8>(v.z), even_of<E8>(v.w)); }
__device__ __forceinline__ bool odd_of(float v) { return !(fabsf(v) <= 3.402823466e38f); }

// ln of the sum, from a maximum in base 2.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.f || l != l ? m * 0.69314718055994531f + logf(l) : -INFINITY; 
}
// Maximum of three (a NaN is dropped).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

}  // namespace fo_ops
