// Quantisation to e4m3 with one scale for 128 values of a row, or for each
// 128 x 128 block (with the transposed copy). Bandwidth-bound: each value is
// read once, in 16-byte pieces, and written once (twice with the copy).
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
  int32_t pieces;   // quant_rows_wide_kernel: warp-wide pieces of a row
  int32_t copy8;    // quant_blocks_wide_kernel: the copy's lines start on 8 bytes
};

// One warp for each group of 128 values of a row (rows that do not start on
// 16 bytes).
template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const __grid_constant__ QuantParams p) {
  const int lane = threadIdx.x & 31, r = blockIdx.y;
  const int64_t n = p.rows * p.groups;
  grid_release();
  grid_wait();
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
    const float scale = scale_of(lanes_max<32>(amax)), inv = inverse_of(scale);
    uint8_t* q = p.q[r] + row * p.cols;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + lane + 32 * j;
      if (c < p.cols) q[c] = (uint8_t)e4m3x2(v[j] * inv, 0.f);
    }
    if (lane == 0) p.scale[r][g] = scale;
  }
}

// 8192 x 4096 bf16 (102 MB): 16.3 us, 6.2 TB/s. A warp takes kUnroll pieces of
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
      const float scale = scale_of(lanes_max<kLanes>(amax_of(v))), inv = inverse_of(scale);
      if ((!ONE && w + i * step >= n) || col[i] >= p.cols) continue;
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] *= inv;
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

// One block for each 128 x 128 block: warp w holds rows w, w + 8, ... (rows
// that do not start on 16 bytes).
template <typename T>
__global__ void __launch_bounds__(256) quant_blocks_kernel(const __grid_constant__ QuantParams p) {
  __shared__ float smem[8];
  __shared__ uint8_t tile[128][132];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.z;
  const int64_t r0 = (int64_t)blockIdx.y * 128, c0 = (int64_t)blockIdx.x * 128;
  float v[16][4], amax = 0.f;
  grid_release();
  grid_wait();
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
  const float scale = scale_of(lanes_max<32>(smem[lane & 7])), inv = inverse_of(scale);
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

// 12288 x 4096 bf16 with the copy (201 MB): 33.7 us, 6.0 TB/s (223 us with bytes
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
__global__ void __launch_bounds__(256) quant_blocks_wide_kernel(const __grid_constant__ QuantParams p) {
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
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float v[Vec16<T>::N];
      Vec16<T>::unpack(raw[i][k], v);
      amax = max_nan(amax, amax_of(v));
    }
  amax = lanes_max<32>(amax);
  if (lane == 0) smem[warp] = amax;
  __syncthreads();
  const float scale = scale_of(lanes_max<8>(smem[lane & 7])), inv = inverse_of(scale);
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
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= inv;
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
      // A warp stores a line in the 4-byte words of memory, each put together
      // from two words of the tile; bytes where a word is not the line's alone.
      const int n = (int)min((int64_t)128, p.rows - r0);   // bytes of a line
#pragma unroll 4
      for (int c = warp; c < 128; c += 8) {
        if (c0 + c >= p.cols) break;
        uint8_t* const line = p.qt[r] + (c0 + c) * p.rows + r0;
        const int off = (int)(reinterpret_cast<uintptr_t>(line) & 3u);
        auto word = [&](int k) -> uint32_t {   // bytes 4 k .. 4 k + 3 of the line
          const uint2 u = tile[c * 16 + ((k >> 1) ^ (c >> 3))];
          return k & 1 ? u.y : u.x;
        };
        const uint32_t mine = word(lane);
        const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);   // (lane 31's is not stored whole)
        // Lane l has the word of memory that begins at byte 4 l + 4 - off (4 l
        // where the line starts on a word).
        const int at = off ? 4 * lane + 4 - off : 4 * lane;
        const uint32_t v = off ? __byte_perm(mine, next, 0x7654u - 0x1111u * (uint32_t)off) : mine;
        if (at + 4 <= n) {
          *reinterpret_cast<uint32_t*>(line + at) = v;
        } else {
#pragma unroll
          for (int j = 0; j < 3; ++j)
            if (at + j < n) line[at + j] = (uint8_t)(v >> (8 * j));
        }
        const uint32_t first = __shfl_sync(0xffffffffu, mine, 0);
        if (lane < 4 - off && off && lane < n) line[lane] = (uint8_t)(first >> (8 * lane));
      }
    }
  }
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
  cudaError_t e;
  if (block_rows == 1) {
    if (!wide) {
      const int64_t want = (rows * k.groups + 7) / 8;
      const dim3 grid((unsigned)(want < 65536 ? want : 65536), R);
      e = launch_after(bf16 ? quant_rows_kernel<__nv_bfloat16> : quant_rows_kernel<float>, grid, 256, 0, 0, s, k);
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
      !wide_blocks ? (bf16 ? quant_blocks_kernel<__nv_bfloat16> : quant_blocks_kernel<float>)
      : bf16       ? blocks_wide<__nv_bfloat16>(copy)
                   : blocks_wide<float>(copy);
  e = launch_after(kern, grid, 256, 0, 0, s, k);
  return launched(e, wide_blocks ? "quant_blocks wide" : "quant_blocks", R, rows, cols, grid.x * grid.y, 256);
}
