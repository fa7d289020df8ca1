// Quantisation to e4m3 with one scale for 128 values of a row, or for each
// 128 x 128 block (with the transposed copy).
#include <string.h>

#include "fo_ops.h"

namespace fo_ops {
namespace {

struct QuantParams {
  const void* x[kMaxR];
  uint8_t* q[kMaxR];
  float* scale[kMaxR];
  uint8_t* qt[kMaxR];
  float* scale_t[kMaxR];
  int64_t rows, cols;
  int32_t groups, row_blocks;
};

// One warp for each group of 128 values of a row.
template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const __grid_constant__ QuantParams p) {
  const int lane = threadIdx.x & 31, r = blockIdx.y;
  const int64_t n = p.rows * p.groups;
  for (int64_t g = blockIdx.x * 8ll + (threadIdx.x >> 5); g < n; g += gridDim.x * 8ll) {
    const int64_t row = g / p.groups;
    const int64_t c0 = (g - row * p.groups) * FO_FP8_BLOCK;
    const T* x = static_cast<const T*>(p.x[r]) + row * p.cols;
    float v[4], amax = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + lane + 32 * j;
      v[j] = c < p.cols ? to_f(x[c]) : 0.f;
      amax = max_nan(amax, fabsf(v[j]));
    }
    const float scale = scale_of(lanes_max<32>(amax)), inv = 1.f / scale;
    uint8_t* q = p.q[r] + row * p.cols;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + lane + 32 * j;
      if (c < p.cols) q[c] = (uint8_t)e4m3x2(v[j] * inv, 0.f);
    }
    if (lane == 0) p.scale[r][g] = scale;
  }
}

// One block for each 128 x 128 block: warp w holds rows w, w + 8, ...
template <typename T>
__global__ void __launch_bounds__(256) quant_blocks_kernel(const __grid_constant__ QuantParams p) {
  __shared__ float smem[8];
  __shared__ uint8_t tile[128][132];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.z;
  const int64_t r0 = (int64_t)blockIdx.y * 128, c0 = (int64_t)blockIdx.x * 128;
  float v[16][4], amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = r0 + warp + 8 * i, c = c0 + lane + 32 * j;
      v[i][j] = row < p.rows && c < p.cols ? to_f(static_cast<const T*>(p.x[r])[row * p.cols + c]) : 0.f;
      amax = max_nan(amax, fabsf(v[i][j]));
    }
  amax = lanes_max<32>(amax);
  if (lane == 0) smem[warp] = amax;
  __syncthreads();
  const float scale = scale_of(lanes_max<32>(smem[lane & 7])), inv = 1.f / scale;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = r0 + warp + 8 * i, c = c0 + lane + 32 * j;
      const uint8_t b = (uint8_t)e4m3x2(v[i][j] * inv, 0.f);
      if (row < p.rows && c < p.cols) p.q[r][row * p.cols + c] = b;
      tile[lane + 32 * j][warp + 8 * i] = b;
    }
  if (threadIdx.x == 0) {
    p.scale[r][(int64_t)blockIdx.y * p.groups + blockIdx.x] = scale;
    if (p.qt[r]) p.scale_t[r][(int64_t)blockIdx.x * p.row_blocks + blockIdx.y] = scale;
  }
  if (!p.qt[r]) return;
  __syncthreads();
  for (int i = 0; i < 16; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + warp + 8 * i, row = r0 + lane + 32 * j;
      if (row < p.rows && c < p.cols) p.qt[r][c * p.rows + row] = tile[warp + 8 * i][lane + 32 * j];
    }
}

}  // namespace
}  // namespace fo_ops

extern "C" fo_status fo_quant_fp8(int32_t R, int64_t rows, int64_t cols, int32_t dtype, int32_t block_rows,
                                  const void* const* x, void* const* q, float* const* scale, void* const* qt,
                                  float* const* scale_t, fo_stream_t stream) {
  using namespace fo_ops;
  if (R < 1 || R > kMaxR || (block_rows != 1 && block_rows != FO_FP8_BLOCK)) return FO_ERR_INVALID_ARG;
  if (!qt != !scale_t || (qt && block_rows == 1)) return FO_ERR_INVALID_ARG;
  // A grid has at most 65535 blocks in y: block rows of the matrix.
  if (rows < 0 || rows > (int64_t)65535 * 128 || cols < 1 || cols > (int64_t)INT32_MAX - 128) return FO_ERR_SHAPE;
  if (dtype != FO_BF16 && dtype != FO_F32) return FO_ERR_DTYPE;
  if (rows == 0) return FO_OK;
  const size_t es = dtype == FO_BF16 ? 2 : 4;
  typedef const void* const* A;
  fo_status st;
  if ((st = check_array(R, x, es)) || (st = check_array(R, (A)q, 1)) || (st = check_array(R, (A)scale, 4)) ||
      (qt && ((st = check_array(R, (A)qt, 1)) || (st = check_array(R, (A)scale_t, 4)))))
    return st;
  int sms;
  if ((st = device_sms(&sms))) return st;
  PtrList l;
  l.add(R, x), l.add(R, (A)q), l.add(R, (A)scale), l.add(R, (A)qt), l.add(R, (A)scale_t);
  if ((st = check_device(l, stream))) return st;
  QuantParams k;
  memset(&k, 0, sizeof(k));
  for (int r = 0; r < R; ++r) {
    k.x[r] = x[r];
    k.q[r] = static_cast<uint8_t*>(q[r]);
    k.scale[r] = scale[r];
    k.qt[r] = qt ? static_cast<uint8_t*>(qt[r]) : nullptr;
    k.scale_t[r] = scale_t ? scale_t[r] : nullptr;
  }
  k.rows = rows;
  k.cols = cols;
  k.groups = (int32_t)((cols + FO_FP8_BLOCK - 1) / FO_FP8_BLOCK);
  k.row_blocks = (int32_t)((rows + FO_FP8_BLOCK - 1) / FO_FP8_BLOCK);
  const cudaStream_t s = (cudaStream_t)stream;
  if (block_rows == 1) {
    const int64_t want = (rows * k.groups + 7) / 8;
    const dim3 grid((unsigned)(want < 65536 ? want : 65536), R);
    if (dtype == FO_BF16) quant_rows_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(k);
    else quant_rows_kernel<float><<<grid, 256, 0, s>>>(k);
    return launched("quant_rows", R, rows, cols, grid.x, 256);
  }
  const dim3 grid(k.groups, k.row_blocks, R);
  if (dtype == FO_BF16) quant_blocks_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(k);
  else quant_blocks_kernel<float><<<grid, 256, 0, s>>>(k);
  return launched("quant_blocks", R, rows, cols, grid.x * grid.y, 256);
}
