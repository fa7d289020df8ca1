// Host-side checks and device helpers shared by the operators between the
// residual stream and the attention (norm, quantisation, 8-bit product,
// rotary positions) and by those on a paged cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <utility>

#include "fo_internal.h"

namespace fo_ops {

constexpr int kMaxR = FO_MAX_R;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// R non-null pointers of `align` bytes' alignment.
inline fo_status check_array(int R, const void* const* a, size_t align) {
  if (!a) return FO_ERR_INVALID_ARG;
  for (int r = 0; r < R; ++r) {
    if (!a[r]) return FO_ERR_INVALID_ARG;
    if (!aligned(a[r], align)) return FO_ERR_ALIGN;
  }
  return FO_OK;
}
inline bool all_aligned(int R, const void* const* a, size_t align) {
  if (a)
    for (int r = 0; r < R; ++r)
      if (!aligned(a[r], align)) return false;
  return true;
}

// The device addresses of one call, gathered so that the driver is asked
// about all of them in one go, after every other check.
struct PtrList {
  const void* p[16 * kMaxR];
  int n = 0;
  void add(const void* q) {
    if (q) p[n++] = q;
  }
  void add(int R, const void* const* a) {
    if (a)
      for (int r = 0; r < R; ++r)
        if (r == 0 || a[r] != a[r - 1]) add(a[r]);
  }
};

// The SMs of the current device; FO_ERR_UNSUPPORTED when it is no sm_103.
inline fo_status device_sms(int* sms) { return fo_internal_device_sms(sms); }
// fo_check_device_pointers on the list.
fo_status check_device(const PtrList& l, fo_stream_t stream);
// An initialised rotary description's fields (fo_rope.cu).
fo_status check_rope_desc(const fo_rope_desc* d);
// After a launch that returned `e`: FO_OK or FO_ERR_CUDA, with FO_LOG's line.
fo_status launched(cudaError_t e, const char* what, int R, int64_t rows, int64_t cols, int grid, int threads);

// Launches `kern` so that it may start while the kernel before it in the
// stream still runs its last blocks (programmatic dependent launch): it sets
// itself up and then waits, in grid_wait(), until that kernel has ended and
// its writes can be seen. cluster = 0: no cluster.
template <typename... A, typename... B>
cudaError_t launch_after(void (*kern)(A...), dim3 grid, int threads, int smem, int cluster, cudaStream_t s, B&&... args) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<B>(args)...);
}

// ------------------------------------------------------------- device side

// Lets the next kernel of the stream start once every block has come here;
// it waits for this one's end by itself.
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Waits until the kernels before this one have ended. Comes before the first
// access to global memory of every thread.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Loads of values that may be used again. (The read-only path, __ldg, is for
// what nobody writes while the kernel exists; a kernel that starts before the
// one ahead of it has ended exists while its inputs are written.)
__device__ __forceinline__ float load1(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 load4(const float* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load4(const __nv_bfloat16* p) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// n / d for n < 2^31 by a multiplication (Granlund and Montgomery's: with s the
// bits of d - 1, m = floor(2^32 (2^s - d) / d) + 1, the quotient is
// (floor(m n / 2^32) + n) / 2^s). The hardware has no integer division; the
// compiler's takes some 30 dependent instructions.
struct Divisor {
  uint32_t d, m, s;
  void set(uint32_t divisor) {
    d = divisor;
    for (s = 0; (1ull << s) < d; ++s) {
    }
    m = (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

constexpr float kE4M3Top = 448.f;
constexpr float kLeastScale = 1.17549435e-38f;   // 2^-126

// Maximum that hands a NaN on (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float max_nan3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Largest magnitude of N values, NaN if one is NaN.
template <int N>
__device__ __forceinline__ float amax_of(const float (&v)[N]) {
  float m = fabsf(v[0]);
  if constexpr (N % 2 == 0) m = max_nan(m, fabsf(v[1]));
#pragma unroll
  for (int j = N % 2 == 0 ? 2 : 1; j < N; j += 2) m = max_nan3(m, fabsf(v[j]), fabsf(v[j + 1]));
  return m;
}

// Packed fp32 pairs (each half rounded as the scalar instruction would).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair_of(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f32x2 pair_of(uint32_t a, uint32_t b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void halves(f32x2 r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A block's scale: the product with the rounded 1/448, within a last place of
// the quotient.
__device__ __forceinline__ float scale_of(float amax) { return max_nan(amax * (1.f / kE4M3Top), kLeastScale); }
// v / scale rounded to nearest: the products with the reciprocal's two parts,
// hi from the approximate instruction (1 ulp) less a last place, lo what is
// left of 1 / scale, positive so that a zero keeps its sign; together they are
// 2^-45 off. In packed pairs that is as many instructions as products with hi
// alone took one by one, and a value on the border between two 8-bit numbers
// goes to the even one: with hi alone 2% of fp32 values on and beside borders went to
// the other one. Under an infinite scale finite values are zeros.
template <int N>
__device__ __forceinline__ void divide_by(float scale, float (&v)[N]) {
  float hi;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(hi) : "f"(scale));
  const bool finite = scale <= 3.402823466e38f;
  if (finite) hi = __uint_as_float(__float_as_uint(hi) - 1u);
  const float e = fmaf(finite ? -scale : 0.f, hi, 1.f), lo = e * hi, low = fmaf(e, lo, lo);
  const f32x2 hi2 = pair_of(hi, hi), lo2 = pair_of(low, low);
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const f32x2 x = pair_of(v[j], v[j + 1]);
    halves(fma2(x, hi2, mul2(x, lo2)), v[j], v[j + 1]);
  }
}

// Two / four values in 8 bits, the first in the lowest byte. Rounded to
// nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// 16 bytes <-> the fp32 values they hold.
template <typename T>
struct Vec16;
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {   // over LANES neighbouring lanes
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

}  // namespace fo_ops
