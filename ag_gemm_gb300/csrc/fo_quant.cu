// Quantisation to e4m3 with one scale for 128 values of a row, or for each
// 128 x 128 block (with the transposed copy). Bandwidth-bound: each value is
// read once, in 16-byte pieces, and written once (twice with the copy).
#include <string.h>

#include <type_traits>

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
  int32_t pieces;   // quant_rows_wide_kernel: warp-wide pieces of a row
  Divisor by_groups;   // quant_rows_kernel: where there are less than 2^31 groups
  int32_t copy8;    // quant_blocks_wide_kernel: the copy's lines start on 8 bytes
};

// Four neighbouring values of a row as they are read, VEC at an access (the
// most that rows and tensors start on). They are converted where they are
// used: a conversion behind the load would wait for it.
template <typename T, int VEC>
struct Four {
  static constexpr bool kWords = sizeof(T) == 2 && VEC > 1;
  typename std::conditional<kWords, uint32_t, T>::type raw[kWords ? 2 : 4];
  __device__ __forceinline__ void load(const T* p, int n) {   // n of them, the others zero
    if constexpr (kWords) {
      raw[0] = raw[1] = 0;
      if constexpr (VEC == 4) {
        if (n > 0) {
          const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
          raw[0] = u.x, raw[1] = u.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (2 * j < n) raw[j] = __ldcs(reinterpret_cast<const unsigned int*>(p) + j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) from_f(0.f, raw[j]);
      if constexpr (VEC == 4) {
        if (n > 0) {
          const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
          raw[0] = v.x, raw[1] = v.y, raw[2] = v.z, raw[3] = v.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < n) raw[j] = p[j];
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    if constexpr (kWords) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        f[2 * j] = __uint_as_float(raw[j] << 16), f[2 * j + 1] = __uint_as_float(raw[j] & 0xffff0000u);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = to_f(raw[j]);
    }
  }
};

// A warp stores a line of n <= 128 bytes that starts anywhere, lane l holding
// its bytes 4 l .. 4 l + 3, in the 4-byte words of memory, each put together
// from two lanes' words; single bytes where a word is not the line's alone.
__device__ __forceinline__ void store_line(uint8_t* line, uint32_t mine, int lane, int n) {
  const int off = (int)(reinterpret_cast<uintptr_t>(line) & 3u);   // the same in every lane
  int at = 4 * lane;
  uint32_t v = mine;
  if (off) {   // lane l has the word of memory that begins at byte 4 l + 4 - off
    const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);   // (lane 31's is not stored whole)
    const uint32_t first = __shfl_sync(0xffffffffu, mine, 0);
    at += 4 - off;
    v = __byte_perm(mine, next, 0x7654u - 0x1111u * (uint32_t)off);
    if (lane < 4 - off && lane < n) line[lane] = (uint8_t)(first >> (8 * lane));
  }
  if (at + 4 <= n) {
    *reinterpret_cast<uint32_t*>(line + at) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (at + j < n) line[at + j] = (uint8_t)(v >> (8 * j));
  }
}

// One warp for each group of 128 values of a row, kUnroll groups at a time
// with all loads first (rows that do not start on 16 bytes). 8191 x 4098 bf16:
// 36 us; 8191 x 4095: 39 (with accesses of one value and byte stores 45).
template <typename T, int VEC>
__global__ void __launch_bounds__(256) quant_rows_kernel(const __grid_constant__ QuantParams p) {
  constexpr int kUnroll = 4;
  const int lane = threadIdx.x & 31, r = blockIdx.y;
  const int64_t n = p.rows * p.groups, step = gridDim.x * 8ll;
  grid_release();
  grid_wait();
  for (int64_t g = blockIdx.x * 8ll + (threadIdx.x >> 5); g < n; g += step * kUnroll) {
    Four<T, VEC> x[kUnroll];
    int64_t row[kUnroll];
    int c0[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int64_t u = g + i * step;
      row[i] = p.by_groups.d ? (int64_t)p.by_groups((uint32_t)u) : u / p.groups;
      c0[i] = (int)(u - row[i] * p.groups) * FO_FP8_BLOCK;
      const int left = u < n ? (int)(p.cols - c0[i]) - 4 * lane : 0;
      x[i].load(static_cast<const T*>(p.x[r]) + row[i] * p.cols + c0[i] + 4 * lane, left);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int64_t u = g + i * step;
      if (u >= n) break;
      float v[4];
      x[i].get(v);
      const float scale = scale_of(lanes_max<32>(amax_of(v)));
      divide_by(scale, v);
      const int left = (int)(p.cols - c0[i]);
      store_line(p.q[r] + row[i] * p.cols + c0[i], e4m3x4(v[0], v[1], v[2], v[3]), lane,
                 left < FO_FP8_BLOCK ? left : FO_FP8_BLOCK);
      if (lane == 0) p.scale[r][u] = scale;
    }
  }
}

// 8192 x 4096 bf16 (102 MB): 16.5 us, 6.2 TB/s. A warp takes kUnroll pieces of
// 32 lanes x 16 bytes at a time, all loads first; a group's scale is the
// maximum over the 16 (bf16) or 32 lanes that hold it. A piece never crosses a row (rows of whole groups are one long
// row to this kernel).
// ONE: there is one such long row and a warp for every kUnroll pieces.
template <typename T, bool ONE>
__global__ void __launch_bounds__(256) quant_rows_wide_kernel(const __grid_constant__ QuantParams p) {
  constexpr int E = Vec16<T>::N, kCols = 32 * E, kUnroll = 2, kLanes = FO_FP8_BLOCK / E;
  const int lane = threadIdx.x & 31, r = blockIdx.y;
  const int64_t n = p.rows * p.pieces, step = ONE ? 8 : (int64_t)gridDim.x * 8;
  grid_release();
  grid_wait();
  for (int64_t w = (int64_t)blockIdx.x * (ONE ? 8 * kUnroll : 8) + (threadIdx.x >> 5);; w += step * kUnroll) {
    if (!ONE && w >= n) break;
    uint4 raw[kUnroll];
    int64_t row[kUnroll];
    int col[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int64_t u = w + i * step;
      // (A 64-bit division costs as much as the rest of a piece.)
      row[i] = ONE || p.rows == 1 ? 0 : n <= UINT32_MAX ? (int64_t)((uint32_t)u / (uint32_t)p.pieces) : u / p.pieces;
      col[i] = (int)(u - row[i] * p.pieces) * kCols + lane * E;
      raw[i] = make_uint4(0, 0, 0, 0);
      if ((ONE || u < n) && col[i] < p.cols)
        raw[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.x[r]) + row[i] * p.cols + col[i]));
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      float v[E];
      Vec16<T>::unpack(raw[i], v);
      const float scale = scale_of(lanes_max<kLanes>(amax_of(v)));
      if ((!ONE && w + i * step >= n) || col[i] >= p.cols) continue;
      divide_by(scale, v);
      uint8_t* q = p.q[r] + row[i] * p.cols + col[i];
      if constexpr (E == 8)
        *reinterpret_cast<uint2*>(q) = make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
      else
        *reinterpret_cast<uint32_t*>(q) = e4m3x4(v[0], v[1], v[2], v[3]);
      if (lane % kLanes == 0) p.scale[r][row[i] * p.groups + col[i] / FO_FP8_BLOCK] = scale;
    }
    if (ONE) break;
  }
}

// Four words of four bytes each, transposed: byte j of word i becomes byte i
// of word j.
__device__ __forceinline__ void transpose4(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  const uint32_t ab_lo = __byte_perm(a, b, 0x5140), ab_hi = __byte_perm(a, b, 0x7362);
  const uint32_t cd_lo = __byte_perm(c, d, 0x5140), cd_hi = __byte_perm(c, d, 0x7362);
  a = __byte_perm(ab_lo, cd_lo, 0x5410);
  b = __byte_perm(ab_lo, cd_lo, 0x7632);
  c = __byte_perm(ab_hi, cd_hi, 0x5410);
  d = __byte_perm(ab_hi, cd_hi, 0x7632);
}

// One block for each 128 x 128 block (rows that do not start on 16 bytes):
// warp w has rows 16 w .. 16 w + 15, lane l columns 4 l .. 4 l + 3, so its
// bytes of a row are a word, and those of four rows, transposed, are words of
// the copy's lines. 8191 x 4098 bf16 with the copy: 43 us, 8191 x 4095: 55
// (with accesses of one value and byte stores 78).
template <typename T, int VEC>
__global__ void __launch_bounds__(256) quant_blocks_kernel(const __grid_constant__ QuantParams p) {
  __shared__ float smem[8];
  __shared__ uint32_t tile[128 * 32];   // [column][word of four rows, mixed with the column]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.z;
  const int64_t r0 = (int64_t)blockIdx.y * 128, c0 = (int64_t)blockIdx.x * 128;
  const int rows = (int)min((int64_t)128, p.rows - r0), cols = (int)min((int64_t)128, p.cols - c0);
  Four<T, VEC> x[16];
  grid_release();
  grid_wait();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int row = warp * 16 + i;
    x[i].load(static_cast<const T*>(p.x[r]) + (r0 + (row < rows ? row : 0)) * p.cols + c0 + 4 * lane,
              row < rows ? cols - 4 * lane : 0);
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float v[4];
    x[i].get(v);
    amax = max_nan(amax, amax_of(v));
  }
  amax = lanes_max<32>(amax);
  if (lane == 0) smem[warp] = amax;
  __syncthreads();
  const float scale = scale_of(lanes_max<8>(smem[lane & 7]));
  if (threadIdx.x == 0) {
    p.scale[r][(int64_t)blockIdx.y * p.groups + blockIdx.x] = scale;
    if (p.qt[r]) p.scale_t[r][(int64_t)blockIdx.x * p.row_blocks + blockIdx.y] = scale;
  }
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[4];
      x[4 * g + i].get(v);
      divide_by(scale, v);
      b[i] = e4m3x4(v[0], v[1], v[2], v[3]);
      const int row = warp * 16 + 4 * g + i;
      if (row < rows) store_line(p.q[r] + (r0 + row) * p.cols + c0, b[i], lane, cols);
    }
    transpose4(b[0], b[1], b[2], b[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) tile[(4 * lane + j) * 32 + ((4 * warp + g) ^ lane)] = b[j];
  }
  if (!p.qt[r]) return;
  __syncthreads();
#pragma unroll 4
  for (int c = warp; c < cols; c += 8)
    store_line(p.qt[r] + (c0 + c) * p.rows + r0, tile[c * 32 + (lane ^ (c >> 2))], lane, rows);
}

// Largest magnitude of the values in N x 16 bytes, NaN if one is NaN. Those of
// bf16, as 15-bit numbers, have the order of their values, with infinity above
// the finite ones and NaN above infinity: two at a time as they are read, in
// two thirds of the instructions that their fp32 forms take (12288 x 4096 with
// the copy: 33.8 us, 36.4 from the fp32 forms; but rows, with 8 values a
// thread, 17.1 against 16.6).
template <typename T, int N>
__device__ __forceinline__ float amax_raw(const uint4 (&raw)[N]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t a = __vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu);
      const uint32_t b = __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu);
      m = __vmaxu2(m, __vmaxu2(a, b));
    }
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  } else {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float v[4];
      Vec16<float>::unpack(raw[i], v);
      m = max_nan(m, amax_of(v));
    }
    return m;
  }
}

// 12288 x 4096 bf16 with the copy (201 MB): 33.8 us, 6.0 TB/s (223 us with bytes
// loaded and stored one by one). The stores are marked as streaming, since a
// weight's copies are read much later, and the copy's are 16 bytes wide where
// its lines allow it: 36.0 us with plain stores of 8 bytes, 34.7 with
// streaming ones of 8. One block for each 128 x 128 block, a thread
// for 8 neighbouring columns of 8 neighbouring rows: the rows' loads are whole 256-byte (fp32: 512-byte)
// runs, and the thread can transpose its 8 x 8 bytes by itself. The copy's
// lines of 128 bytes are put together in shared memory, in 8-byte pieces
// whose place is mixed with the column, so that neither the writes nor the
// reads meet in a bank.
// COPY: 0 none, 8 the copy's lines start on 8 bytes or anywhere, 16 on 16.
template <typename T, int COPY>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) quant_blocks_wide_kernel(const __grid_constant__ QuantParams p) {
  constexpr int V = 8 / Vec16<T>::N;   // 16-byte loads for 8 values
  __shared__ float smem[8];
  __shared__ uint2 tile[COPY ? 128 * 16 : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.z;
  const int64_t r0 = (int64_t)blockIdx.y * 128, c0 = (int64_t)blockIdx.x * 128;
  const int rg = tid >> 4, cg = tid & 15;   // groups of 8 rows, of 8 columns
  const int64_t row0 = r0 + rg * 8, col = c0 + cg * 8;
  const bool in = col < p.cols;   // whole groups: the columns are a multiple of 8
  grid_release();
  grid_wait();
  uint4 raw[8][V];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      raw[i][k] = make_uint4(0, 0, 0, 0);
      if (in && row0 + i < p.rows)
        raw[i][k] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.x[r]) + (row0 + i) * p.cols + col) + k);
    }
  const float amax = lanes_max<32>(amax_raw<T>(reinterpret_cast<const uint4(&)[8 * V]>(raw)));
  if (lane == 0) smem[warp] = amax;
  __syncthreads();
  const float scale = scale_of(lanes_max<8>(smem[lane & 7]));
  uint32_t lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    if constexpr (V == 1) {
      Vec16<T>::unpack(raw[i][0], reinterpret_cast<float(&)[Vec16<T>::N]>(v));
    } else {
      Vec16<T>::unpack(raw[i][0], reinterpret_cast<float(&)[Vec16<T>::N]>(v[0]));
      Vec16<T>::unpack(raw[i][V - 1], reinterpret_cast<float(&)[Vec16<T>::N]>(v[4]));
    }
    divide_by(scale, v);
    lo[i] = e4m3x4(v[0], v[1], v[2], v[3]);
    hi[i] = e4m3x4(v[4], v[5], v[6], v[7]);
    if (in && row0 + i < p.rows)
      __stcs(reinterpret_cast<uint2*>(p.q[r] + (row0 + i) * p.cols + col), make_uint2(lo[i], hi[i]));
  }
  if (tid == 0) {
    p.scale[r][(int64_t)blockIdx.y * p.groups + blockIdx.x] = scale;
    if (COPY) p.scale_t[r][(int64_t)blockIdx.x * p.row_blocks + blockIdx.y] = scale;
  }
  if constexpr (COPY != 0) {
    transpose4(lo[0], lo[1], lo[2], lo[3]);   // columns 0-3 of rows 0-3
    transpose4(lo[4], lo[5], lo[6], lo[7]);   // of rows 4-7
    transpose4(hi[0], hi[1], hi[2], hi[3]);   // columns 4-7
    transpose4(hi[4], hi[5], hi[6], hi[7]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      tile[(cg * 8 + j) * 16 + (rg ^ cg)] = make_uint2(lo[j], lo[j + 4]);
      tile[(cg * 8 + 4 + j) * 16 + (rg ^ cg)] = make_uint2(hi[j], hi[j + 4]);
    }
    __syncthreads();
    if constexpr (COPY == 16) {   // eight threads store a line of the copy
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = i * 32 + (tid >> 3), g = (tid & 7) * 2;
        const int64_t row = r0 + g * 8;
        if (c0 + c < p.cols && row < p.rows) {
          const uint2 a = tile[c * 16 + (g ^ (c >> 3))], b = tile[c * 16 + ((g + 1) ^ (c >> 3))];
          __stcs(reinterpret_cast<uint4*>(p.qt[r] + (c0 + c) * p.rows + row), make_uint4(a.x, a.y, b.x, b.y));
        }
      }
    } else if (p.copy8) {   // sixteen threads
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = i * 16 + rg;
        const int64_t row = r0 + cg * 8;
        if (c0 + c < p.cols && row < p.rows)
          __stcs(reinterpret_cast<uint2*>(p.qt[r] + (c0 + c) * p.rows + row), tile[c * 16 + (cg ^ (c >> 3))]);
      }
    } else {
      const int n = (int)min((int64_t)128, p.rows - r0);   // bytes of a line
#pragma unroll 4
      for (int c = warp; c < 128; c += 8) {
        if (c0 + c >= p.cols) break;
        const uint2 u = tile[c * 16 + ((lane >> 1) ^ (c >> 3))];
        store_line(p.qt[r] + (c0 + c) * p.rows + r0, lane & 1 ? u.y : u.x, lane, n);
      }
    }
  }
}

// The kernels for rows off the 16-byte grid, `vec` values an access.
template <typename T>
auto rows_any(int vec) {
  if constexpr (sizeof(T) == 4) return vec == 4 ? quant_rows_kernel<T, 4> : quant_rows_kernel<T, 1>;
  else return vec == 4 ? quant_rows_kernel<T, 4> : vec == 2 ? quant_rows_kernel<T, 2> : quant_rows_kernel<T, 1>;
}
template <typename T>
auto blocks_any(int vec) {
  if constexpr (sizeof(T) == 4) return vec == 4 ? quant_blocks_kernel<T, 4> : quant_blocks_kernel<T, 1>;
  else return vec == 4 ? quant_blocks_kernel<T, 4> : vec == 2 ? quant_blocks_kernel<T, 2> : quant_blocks_kernel<T, 1>;
}
template <typename T>
auto blocks_wide(int copy) {
  return copy == 16 ? quant_blocks_wide_kernel<T, 16> : copy ? quant_blocks_wide_kernel<T, 8> : quant_blocks_wide_kernel<T, 0>;
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
  if (rows < 0 || rows > (block_rows == 1 ? (int64_t)INT32_MAX : (int64_t)65535 * 128) || cols < 1 || cols > (int64_t)INT32_MAX - 1024) return FO_ERR_SHAPE;
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
  const bool bf16 = dtype == FO_BF16;
  const bool wide = (cols * es) % 16 == 0 && all_aligned(R, x, 16) && all_aligned(R, (A)q, 8);
  int vec = 4;
  while (cols % vec || !all_aligned(R, x, vec * es)) vec /= 2;
  cudaError_t e;
  if (block_rows == 1) {
    if (!wide) {
      if (rows * k.groups < INT32_MAX - 65536 * 32) k.by_groups.set((uint32_t)k.groups);
      // (Few groups: a warp each.)
      const int64_t n = rows * k.groups, want = n >= 16384 ? (n + 31) / 32 : (n + 7) / 8;
      const dim3 grid((unsigned)(want < 65536 ? want : 65536), R);
      e = launch_after(bf16 ? rows_any<__nv_bfloat16>(vec) : rows_any<float>(vec), grid, 256, 0, 0, s, k);
      return launched(e, "quant_rows", R, rows, cols, grid.x, 256);
    }
    const int piece = bf16 ? 256 : 128;
    if (cols % FO_FP8_BLOCK == 0 && rows * cols <= INT32_MAX - 1024) {   // groups back to back: one long row
      k.cols = rows * cols;
      k.groups = (int32_t)(k.cols / FO_FP8_BLOCK);
      k.rows = 1;
    }
    k.pieces = (int32_t)((k.cols + piece - 1) / piece);
    // A warp for two pieces (20.0 us for 8192 x 4096 bf16; four: 21.2, eight:
    // 21.7), few pieces: a warp each.
    const int64_t n = k.rows * k.pieces, want = n >= 4096 ? (n + 15) / 16 : (n + 7) / 8;
    const bool one = k.rows == 1 && n >= 4096;
    const dim3 grid((unsigned)(one || want < 65536 ? want : 65536), R);
    void (*kern)(const QuantParams) =
        one ? (bf16 ? quant_rows_wide_kernel<__nv_bfloat16, true> : quant_rows_wide_kernel<float, true>)
            : (bf16 ? quant_rows_wide_kernel<__nv_bfloat16, false> : quant_rows_wide_kernel<float, false>);
    e = launch_after(kern, grid, 256, 0, 0, s, k);
    return launched(e, "quant_rows wide", R, rows, cols, grid.x, 256);
  }
  const dim3 grid(k.groups, k.row_blocks, R);
  const bool wide_blocks = wide && cols % 8 == 0;
  const int copy = !qt ? 0 : rows % 16 == 0 && all_aligned(R, (A)qt, 16) ? 16 : 8;
  k.copy8 = rows % 8 == 0 && all_aligned(R, (A)qt, 8);
  void (*kern)(const QuantParams) =
      !wide_blocks ? (bf16 ? blocks_any<__nv_bfloat16>(vec) : blocks_any<float>(vec))
      : bf16       ? blocks_wide<__nv_bfloat16>(copy)
                   : blocks_wide<float>(copy);
  e = launch_after(kern, grid, 256, 0, 0, s, k);
  return launched(e, wide_blocks ? "quant_blocks wide" : "quant_blocks", R, rows, cols, grid.x * grid.y, 256);
}
