// Product of e4m3 matrices with a scale for each block of 128 of the
// reduction.
#include <stdio.h>
#include <string.h>

#include "fo_ops.h"

namespace fo_ops {
namespace {

struct GemmParams {
  const uint8_t* A[kMaxR];
  const uint8_t* W[kMaxR];
  const float* sA[kMaxR];
  const float* sW[kMaxR];
  void* Y[kMaxR];
  int64_t M, N, K;
  int32_t kblocks;
  bool f32;
};

__device__ __forceinline__ float from_e4m3(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// 64 x 64 of Y a block, 4 x 4 a thread, 32 of the reduction a step.
__global__ void __launch_bounds__(256) gemm_fp8_kernel(const __grid_constant__ GemmParams p) {
  __shared__ float a[32][65], w[32][65];
  const int r = blockIdx.z, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
  float sum[4][4] = {};
  for (int b = 0; b < p.kblocks; ++b) {
    float part[4][4] = {};
    for (int64_t k0 = (int64_t)b * 128; k0 < (int64_t)b * 128 + 128 && k0 < p.K; k0 += 32) {
      __syncthreads();
      for (int i = threadIdx.x; i < 64 * 32; i += 256) {
        const int row = i >> 5, k = i & 31;
        a[k][row] = m0 + row < p.M && k0 + k < p.K ? from_e4m3(p.A[r][(m0 + row) * p.K + k0 + k]) : 0.f;
        w[k][row] = n0 + row < p.N && k0 + k < p.K ? from_e4m3(p.W[r][(n0 + row) * p.K + k0 + k]) : 0.f;
      }
      __syncthreads();
#pragma unroll 8
      for (int k = 0; k < 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(a[k][ty * 4 + i], w[k][tx * 4 + j], part[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (m < p.M && n < p.N)
          sum[i][j] = fmaf(part[i][j], p.sA[r][m * p.kblocks + b] * p.sW[r][n / 128 * p.kblocks + b], sum[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= p.M || n >= p.N) continue;
      if (p.f32) static_cast<float*>(p.Y[r])[m * p.N + n] = sum[i][j];
      else static_cast<__nv_bfloat16*>(p.Y[r])[m * p.N + n] = __float2bfloat16_rn(sum[i][j]);
    }
}

fo_status check_desc(const fo_gemm_fp8_desc* d, int64_t M) {
  if (!d) return FO_ERR_INVALID_ARG;
  if (d->R < 1 || d->R > kMaxR) return FO_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (d->reserved[i]) return FO_ERR_INVALID_ARG;
  if (M < 0 || M > (1 << 21) || d->N < 1 || d->N > (1 << 21) || d->K < 1 || d->K > (1 << 21)) return FO_ERR_SHAPE;
  if (d->out_dtype != FO_BF16 && d->out_dtype != FO_F32) return FO_ERR_DTYPE;
  if (d->K % 16) return FO_ERR_ALIGN;   // rows of A and W start on 16 bytes
  return FO_OK;
}

}  // namespace

fo_status launched(const char* what, int R, int64_t rows, int64_t cols, int grid, int threads) {
  const cudaError_t e = cudaGetLastError();
  if (fo_log_enabled())
    fprintf(stderr, "[flashoverlap] %s R=%d rows=%lld cols=%lld: %d blocks of %d: %s\n", what, R, (long long)rows,
            (long long)cols, grid, threads, cudaGetErrorString(e));
  return e == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

fo_status check_device(const PtrList& l, fo_stream_t stream) {
  return fo_internal_check_device_ptrs(l.n, l.p, stream);
}

}  // namespace fo_ops

extern "C" fo_status fo_gemm_fp8_workspace(const fo_gemm_fp8_desc* d, int64_t M, size_t* bytes) {
  const fo_status st = fo_ops::check_desc(d, M);
  if (st) return st;
  if (!bytes) return FO_ERR_INVALID_ARG;
  *bytes = sizeof(fo_ws_header);
  return FO_OK;
}

extern "C" fo_status fo_ops_workspace_init(void* ws, size_t bytes, fo_stream_t stream) {
  if (!ws || bytes < sizeof(fo_ws_header)) return FO_ERR_INVALID_ARG;
  if (!fo_ops::aligned(ws, 16)) return FO_ERR_ALIGN;
  if (cudaMemsetAsync(ws, 0, bytes, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return FO_ERR_CUDA;
  }
  return FO_OK;
}

extern "C" fo_status fo_ops_status_query(void* ws, fo_stream_t stream, int32_t info[4]) {
  if (!ws) return FO_ERR_INVALID_ARG;
  int32_t got[4] = {0, 0, 0, 0};
  const cudaStream_t s = (cudaStream_t)stream;
  bool ok = cudaMemcpyAsync(got, ws, sizeof(got), cudaMemcpyDeviceToHost, s) == cudaSuccess &&
            cudaStreamSynchronize(s) == cudaSuccess;
  if (ok && got[0])
    ok = cudaMemsetAsync(ws, 0, sizeof(fo_ws_header), s) == cudaSuccess && cudaStreamSynchronize(s) == cudaSuccess;
  if (!ok) {
    cudaGetLastError();
    return FO_ERR_CUDA;
  }
  if (info) memcpy(info, got, sizeof(got));
  return (fo_status)got[0];
}

extern "C" fo_status fo_gemm_fp8(const fo_gemm_fp8_desc* d, int64_t M, const void* const* A, const float* const* sA,
                                 const void* const* W, const float* const* sW, void* const* Y, void* ws,
                                 fo_stream_t stream) {
  using namespace fo_ops;
  fo_status st = check_desc(d, M);
  if (st) return st;
  if (!ws) return FO_ERR_INVALID_ARG;
  if (!aligned(ws, 16)) return FO_ERR_ALIGN;
  if (M == 0) return FO_OK;
  const int R = d->R;
  typedef const void* const* P;
  if ((st = check_array(R, A, 16)) || (st = check_array(R, W, 16)) || (st = check_array(R, (P)Y, 16)) ||
      (st = check_array(R, (P)sA, 4)) || (st = check_array(R, (P)sW, 4)))
    return st;
  int sms;
  if ((st = device_sms(&sms))) return st;
  PtrList l;
  l.add(R, A), l.add(R, (P)sA), l.add(R, W), l.add(R, (P)sW), l.add(R, (P)Y), l.add(ws);
  if ((st = check_device(l, stream))) return st;
  GemmParams k;
  memset(&k, 0, sizeof(k));
  for (int r = 0; r < R; ++r) {
    k.A[r] = static_cast<const uint8_t*>(A[r]);
    k.W[r] = static_cast<const uint8_t*>(W[r]);
    k.sA[r] = sA[r];
    k.sW[r] = sW[r];
    k.Y[r] = Y[r];
  }
  k.M = M;
  k.N = d->N;
  k.K = d->K;
  k.kblocks = (int32_t)((d->K + 127) / 128);
  k.f32 = d->out_dtype == FO_F32;
  const dim3 grid((unsigned)((d->N + 63) / 64), (unsigned)((M + 63) / 64), R);
  gemm_fp8_kernel<<<grid, 256, 0, (cudaStream_t)stream>>>(k);
  return launched("gemm_fp8", R, M, d->N, grid.x * grid.y, 256);
}
