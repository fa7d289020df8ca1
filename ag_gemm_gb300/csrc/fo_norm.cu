// RMSNorm with the residual's addition, its output in 16/32 bits, in 8 bits
// with one scale for 128 columns, or both; and its gradient.
//
// Both are bound by memory: a row is read once, held in registers while its
// sum of squares (its product with the gradient) goes round the block, and
// written once. A block has one row at a time; several blocks an SM keep the
// loads going while others wait for their sums. Sums, scales and quotients
// are fp32, each output is rounded once; the sum of squares is a tree over a
// thread's at most 32 values, its warp and the block, so it repeats bit for bit.
#include <string.h>

#include <type_traits>

#include "fo_ops.h"

namespace fo_ops {
namespace {

struct NormParams {
  const void* x[kMaxR];
  const void* res[kMaxR];
  void* h[kMaxR];
  void* y[kMaxR];
  uint8_t* q[kMaxR];
  float* scale[kMaxR];
  float* rstd[kMaxR];
  const void* w;
  int64_t rows;   // of a shard
  int32_t H, groups;
  float eps, w_offset, inv_H;
  bool has_res, has_h, has_y, has_q, has_rstd, w_f32;
};

// Where a thread's values lie. An access has VEC neighbouring values, the most
// that rows and tensors start on. With 16-byte accesses each lane holds E =
// VEC neighbouring columns of a chunk of 32 * E, else E = 4 in 4 / VEC pieces
// that are 32 * VEC apart (each access still covers whole sectors). Either way
// a group of 128 columns belongs to one warp, or to one half of it, so its
// maximum never leaves the warp.
// FULL: the row is exactly the block's chunks, so no column is beyond it.
template <typename T, int VEC, bool FULL>
struct Chunk {
  static constexpr bool WIDE = VEC == Vec16<T>::N;
  static constexpr int E = WIDE ? VEC : 4;
  static constexpr int COLS = 32 * E;
  static constexpr int GROUP_LANES = 128 / E;
  static __device__ __forceinline__ int col(int chunk, int lane, int j) {
    return chunk * COLS + j / VEC * 32 * VEC + lane * VEC + j % VEC;
  }
  static __device__ __forceinline__ void load(const T* p, int chunk, int lane, int H, float (&f)[E]) {
    if constexpr (WIDE) {
      const int c = col(chunk, lane, 0);
      uint4 u = make_uint4(0, 0, 0, 0);
      if (FULL || c < H) u = *reinterpret_cast<const uint4*>(p + c);
      Vec16<T>::unpack(u, f);
    } else {
#pragma unroll
      for (int j = 0; j < E; j += VEC) {
        const int c = col(chunk, lane, j);
        if constexpr (VEC == 1) f[j] = FULL || c < H ? to_f(p[c]) : 0.f;
        else load_some(p + c, FULL || c < H, &f[j]);
      }
    }
  }
  // VEC > 1 values, zeros when not `in`.
  static __device__ __forceinline__ void load_some(const __nv_bfloat16* p, bool in, float* f) {
    uint32_t w[VEC < 2 ? 1 : VEC / 2] = {};
    if (in) {
      if constexpr (VEC >= 4) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
          const uint2 u = load4(p + i);
          w[i / 2] = u.x, w[i / 2 + 1] = u.y;
        }
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  static __device__ __forceinline__ void load_some(const float* p, bool in, float* f) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = 0.f;
    if (in) {
      if constexpr (VEC >= 4) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
          const float4 v = load4(p + i);
          f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = p[i];
      }
    }
  }
  static __device__ __forceinline__ void store(T* p, int chunk, int lane, int H, const float (&f)[E]) {
    if constexpr (WIDE) {
      const int c = col(chunk, lane, 0);
      if (FULL || c < H) *reinterpret_cast<uint4*>(p + c) = Vec16<T>::pack(f);
    } else if constexpr (VEC == 1) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int c = col(chunk, lane, j);
        if (FULL || c < H) from_f(f[j], p[c]);
      }
    } else {   // bf16
#pragma unroll
      for (int j = 0; j < E; j += VEC) {
        const int c = col(chunk, lane, j);
        uint32_t w[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(f[j + i], f[j + i + 1]);
          w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
        if (c < H) {
          if constexpr (VEC == 4) *reinterpret_cast<uint2*>(p + c) = make_uint2(w[0], w[1]);
          else *reinterpret_cast<uint32_t*>(p + c) = w[0];
        }
      }
    }
  }
  static __device__ __forceinline__ void store_e4m3(uint8_t* p, int chunk, int lane, int H, const float (&f)[E]) {
#pragma unroll
    for (int j = 0; j < E; j += VEC) {
      const int c = col(chunk, lane, j);
      if (FULL || c < H) {
        if constexpr (VEC == 8)
          *reinterpret_cast<uint2*>(p + c) = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
        else if constexpr (VEC == 4)
          *reinterpret_cast<uint32_t*>(p + c) = e4m3x4(f[0], f[1], f[2], f[3]);
        else if constexpr (VEC == 2)
          *reinterpret_cast<uint16_t*>(p + c) = (uint16_t)e4m3x2(f[j], f[j + 1]);
        else
          p[c] = (uint8_t)e4m3x2(f[j], 0.f);
      }
    }
  }
  // The chunk's weights plus the offset, zero beyond H.
  static __device__ __forceinline__ void load_w(const void* w, bool f32, float offset, int chunk, int lane, int H,
                                                float (&f)[E]) {
    if constexpr (VEC == 1) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int c = col(chunk, lane, j);
        f[j] = !FULL && c >= H ? 0.f
                      : offset + (f32 ? static_cast<const float*>(w)[c]
                                      : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; j += VEC) {
        const int c = col(chunk, lane, j);
        if (f32) load_some(static_cast<const float*>(w) + c, FULL || c < H, &f[j]);
        else load_some(static_cast<const __nv_bfloat16*>(w) + c, FULL || c < H, &f[j]);
      }
      if (offset != 0.f) {
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (FULL || col(chunk, lane, j) < H) f[j] += offset;
      }
    }
  }
};

// Sum over the block's nw <= NW warps, the same in every thread. `smem`: nw
// floats, which no thread may write again before the next barrier.
template <int NW>
__device__ __forceinline__ float block_sum(float v, float* smem, int nw) {
  v = warp_sum(v);
  if constexpr (NW == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) smem[warp] = v;
  __syncthreads();
  return warp_sum(lane < nw ? smem[lane] : 0.f);
}

// Blocks have no more warps than their row needs (8191 x 4098 bf16, 33 chunks
// of 4 a thread: 78 us with 9 warps, 114 with 16; 8191 x 1280: 12.9 us with 5,
// 18.2 with 8), but for the widest rows, where the number of warps would be one
// register too many (2000 x 20001: 130 us with 32 warps, 240 with 20).
template <int NW, int C>
constexpr bool kAllWarps = NW == 32 && C == 8;

// 8192 x 4096 bf16 with residual and 8-bit output (236 MB): 39.0 us, 6.0 TB/s.
// Three fifths of the issue slots are taken, so instructions count: no 64-bit
// division, packed products, no bounds checks on full rows. Six blocks
// of 8 warps on an SM: 1.5 us less than the five that the compiler's own
// choice of registers leaves, 4 less than rows on 4 warps, 15 less than on 16.
template <typename T, int VEC, int NW, int C, bool FULL>
__global__ void __launch_bounds__(NW * 32, NW == 8 ? 6 : NW == 16 ? (C <= 2 ? 3 : 2) : 1) rmsnorm_kernel(const __grid_constant__ NormParams p) {
  using K = Chunk<T, VEC, FULL>;
  __shared__ float smem[2][32];   // by turns: a barrier a row is enough
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nw = FULL || kAllWarps<NW, C> ? NW : (int)blockDim.x >> 5;
  const int r = blockIdx.y;
  grid_release();
  grid_wait();
  int turn = 0;
  for (int64_t at = blockIdx.x; at < p.rows; at += gridDim.x, turn ^= 1) {
    const int64_t off = at * p.H;
    float s[C][K::E];
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) K::load(static_cast<const T*>(p.x[r]) + off, c * nw + warp, lane, p.H, s[c]);
    if (p.has_res) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float t[K::E];
        K::load(static_cast<const T*>(p.res[r]) + off, c * nw + warp, lane, p.H, t);
#pragma unroll
        for (int j = 0; j < K::E; ++j) s[c][j] += t[j];
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int j = 0; j < K::E; ++j) sum = fmaf(s[c][j], s[c][j], sum);
    }
    if (p.has_h) {
#pragma unroll
      for (int c = 0; c < C; ++c) K::store(static_cast<T*>(p.h[r]) + off, c * nw + warp, lane, p.H, s[c]);
    }
    const float rstd = rsqrtf(fmaf(block_sum<NW>(sum, smem[turn], nw), p.inv_H, p.eps));
    if (p.has_rstd && threadIdx.x == 0) p.rstd[r][at] = rstd;
    if (!p.has_y && !p.has_q) continue;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int chunk = c * nw + warp;
      float w[K::E];
      K::load_w(p.w, p.w_f32, p.w_offset, chunk, lane, p.H, w);
#pragma unroll
      for (int j = 0; j < K::E; j += 2)
        halves(mul2(mul2(pair_of(s[c][j], s[c][j + 1]), pair_of(rstd, rstd)), pair_of(w[j], w[j + 1])), s[c][j], s[c][j + 1]);
      if (p.has_y) K::store(static_cast<T*>(p.y[r]) + off, chunk, lane, p.H, s[c]);
      if (p.has_q) {
        const float scale = scale_of(lanes_max<K::GROUP_LANES>(amax_of(s[c])));
        divide_by(scale, s[c]);
        K::store_e4m3(p.q[r] + off, chunk, lane, p.H, s[c]);
        const int group = K::col(chunk, lane, 0) / FO_FP8_BLOCK;
        if (lane % K::GROUP_LANES == 0 && group < p.groups) p.scale[r][at * p.groups + group] = scale;
      }
    }
  }
}

struct NormBwdParams {
  const void* dy[kMaxR];
  const void* dh[kMaxR];
  const void* h[kMaxR];
  const float* rstd[kMaxR];
  void* dx[kMaxR];
  const void* w;
  float* part;   // [gridDim.x][H] partial sums of dweight
  int64_t rows, total;
  int32_t H;
  float w_offset, inv_H;
  bool has_dh, has_dw, w_f32;
};

// Blocks of the backward kernel on an SM: sixteen warps' worth, or 32 where a
// thread has one chunk (of four warps or more: fewer leave too many partial sums).
constexpr int bwd_per_sm(int nw, int c) { return c == 1 && nw >= 4 ? 32 / nw : nw <= 16 ? 16 / nw : 1; }

// 16, 8 or 4 bytes to shared memory in the background, or zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from, bool in) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(in ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at), "l"(from), "n"(BYTES), "r"(in ? BYTES : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {   // all but the N newest groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, int VEC, int NW, int C>
struct BwdCfg {
  static constexpr int E = Chunk<T, VEC, false>::E;
  static constexpr int kPiece = VEC * (int)sizeof(T);   // bytes of an access
  static constexpr int kPart = C * E * (int)sizeof(T);  // of a thread's part of a row of one input
  static constexpr bool kAhead = kPiece >= 4 && NW <= 16 && kPart <= 64;
  static constexpr int kRows = kPart <= 16 && NW >= 8 ? 4 : kPart <= 32 ? 3 : 2;   // the row in hand and those loaded in the background
  static constexpr bool kNext = !kAhead && NW <= 16 && C * E <= 8;
  static constexpr bool kHold = NW <= 16 && !(kAhead && C * E > 16);   // this row's values
  static constexpr bool kWeights = kNext || (kAhead && C * E <= 16);     // held
  // Bytes of one input's row, and of all, with nw warps.
  static constexpr __host__ __device__ int slot(int nw) { return nw * 32 * kPart; }
  static constexpr int smem(int nw) { return kAhead ? kRows * 3 * slot(nw) : 0; }
};

// A block takes every gridDim.x-th row and keeps its columns' share of the
// weight's gradient in registers. Where a thread's part of a row is at most 64
// bytes, in accesses of 4 or more, the next rows come in the background, each
// thread its own pieces, so that the loads go on through a row's barrier
// (8191 x 4098 bf16: 69 us, 185 without; 4000 x 8192 fp32: 81, 120); such
// blocks have no more warps than their rows need (8191 x 1280 bf16: 20 us,
// 31 with the next power of two and half as many blocks). The weights stay in
// registers too where a thread has at most 16 values; with 32 it reads them,
// and in the second pass the row in shared memory, again (2556 x 8704 bf16:
// 51 us, 83 from L2). At most 8 values of odd rows: the weights, and the next
// row's values in registers (8191 x 4095 bf16: 96 us, 161 without). Else, with
// up to 16 warps, this row's values; else nothing, and the second pass reads
// the row from L2.
// 8192 x 4096 bf16 with the residual's gradient (268 MB): 45.7 us with the
// sum below, 5.9 TB/s (48.5 with partial sums stored value by value). With the next row in registers instead of three in
// shared memory 53 us; three blocks an SM instead of two 64 us.
template <typename T, int VEC, int NW, int C, bool FULL>
__global__ void __launch_bounds__(NW * 32, bwd_per_sm(NW, C)) rmsnorm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  using K = Chunk<T, VEC, FULL>;
  using Cfg = BwdCfg<T, VEC, NW, C>;
  constexpr int E = K::E;
  constexpr bool kAhead = Cfg::kAhead, kNext = Cfg::kNext, kHold = Cfg::kHold, kWeights = Cfg::kWeights;
  __shared__ float smem[2][32];   // by turns: a barrier a row is enough
  extern __shared__ uint4 ring_mem[];   // kAhead: [row % Cfg::kRows][input][chunk][piece of E values][thread]
  uint8_t* const ring = reinterpret_cast<uint8_t*>(ring_mem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nw = FULL || !kAhead ? NW : (int)blockDim.x >> 5;
  grid_release();
  grid_wait();
  float w[kWeights ? C : 1][E], dw[C][E];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (kWeights) K::load_w(p.w, p.w_f32, p.w_offset, c * nw + warp, lane, p.H, w[c]);
#pragma unroll
    for (int j = 0; j < E; ++j) dw[c][j] = 0.f;
  }
  // (A 64-bit division costs as much as a third of a row.)
  auto rank_of = [&](int64_t row) -> int {
    return p.total == p.rows ? 0 : p.total <= UINT32_MAX ? (int)((uint32_t)row / (uint32_t)p.rows) : (int)(row / p.rows);
  };
  auto fetch = [&](int64_t row, int slot) {
    if (row < p.total) {
      const int r = rank_of(row);
      const int64_t off = (row - r * p.rows) * p.H;
      uint8_t* const to = ring + slot * 3 * Cfg::slot(nw) + threadIdx.x * Cfg::kPiece;
#pragma unroll
      for (int i = 0; i < C * E / VEC; ++i) {
        const int col = K::col(i / (E / VEC) * nw + warp, lane, i % (E / VEC) * VEC), n = i * nw * 32 * Cfg::kPiece;
        const bool in = FULL || col < p.H;
        const int64_t at = off + (in ? col : 0);
        copy_async<Cfg::kPiece>(to + n, static_cast<const T*>(p.dy[r]) + at, in);
        copy_async<Cfg::kPiece>(to + Cfg::slot(nw) + n, static_cast<const T*>(p.h[r]) + at, in);
        if (p.has_dh) copy_async<Cfg::kPiece>(to + 2 * Cfg::slot(nw) + n, static_cast<const T*>(p.dh[r]) + at, in);
      }
    }
    copies_end();   // a group for every row, empty ones too: the waits count them
  };
  auto piece = [&](int slot, int input, int c, float (&v)[E]) {
    if constexpr (kAhead) {
#pragma unroll
      for (int j = 0; j < E; j += VEC) {
        const uint8_t* const at = ring + (slot * 3 + input) * Cfg::slot(nw) +
                                  ((c * (E / VEC) + j / VEC) * nw * 32 + threadIdx.x) * Cfg::kPiece;
        if constexpr (Cfg::kPiece == 16) {
          Vec16<T>::unpack(*reinterpret_cast<const uint4*>(at), v);
        } else if constexpr (sizeof(T) == 4) {
          v[j] = *reinterpret_cast<const float*>(at);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; i += 2) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(at)[i / 2];
            v[j + i] = __uint_as_float(w << 16), v[j + i + 1] = __uint_as_float(w & 0xffff0000u);
          }
        }
      }
    }
  };
  if constexpr (kAhead) {
#pragma unroll
    for (int i = 0; i < Cfg::kRows - 1; ++i) fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
  }
  // kNext: the row after this one, as it was read (converted, each value would be waited for).
  T nu[kNext ? C : 1][E], nh[kNext ? C : 1][E], nt[kNext ? C : 1][E];
  auto next = [&](int64_t row) {
    if constexpr (kNext)
      if (row < p.total) {
        const int r = rank_of(row);
        const int64_t off = (row - r * p.rows) * p.H;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < E; ++j) {
            const int col = K::col(c * nw + warp, lane, j);
            if (col < p.H) {
              nu[c][j] = static_cast<const T*>(p.dy[r])[off + col];
              nh[c][j] = static_cast<const T*>(p.h[r])[off + col];
              if (p.has_dh) nt[c][j] = static_cast<const T*>(p.dh[r])[off + col];
            }
          }
      }
  };
  if constexpr (kNext) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < E; ++j) from_f(0.f, nu[c][j]), from_f(0.f, nh[c][j]), from_f(0.f, nt[c][j]);   // beyond H
  }
  next(blockIdx.x);
  int slot = 0, turn = 0;
  for (int64_t row = blockIdx.x; row < p.total; row += gridDim.x, turn ^= 1) {
    const int r = rank_of(row);
    const int64_t at = row - r * p.rows, off = at * p.H;
    const T* const dy = static_cast<const T*>(p.dy[r]) + off;
    const T* const hp = static_cast<const T*>(p.h[r]) + off;
    const float rstd = p.rstd[r][at];
    if constexpr (kAhead) {
      // The slot of the row before this one is free: this thread has read its
      // pieces, and no other thread reads them.
      fetch(row + (int64_t)(Cfg::kRows - 1) * gridDim.x, slot == 0 ? Cfg::kRows - 1 : slot - 1);
      copies_wait<Cfg::kRows - 1>();
    }
    float h[kHold ? C : 1][E], u[kHold ? C : 1][E], t[kNext ? C : 1][E];
    float sum = 0.f;
    if constexpr (kNext) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < E; ++j) u[c][j] = to_f(nu[c][j]), h[c][j] = to_f(nh[c][j]), t[c][j] = to_f(nt[c][j]);
      next(row + gridDim.x);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float(&uc)[E] = u[kHold ? c : 0];
      float(&hc)[E] = h[kHold ? c : 0];
      if constexpr (kAhead) {
        piece(slot, 0, c, uc);
        piece(slot, 1, c, hc);
      } else if constexpr (!kNext) {
        K::load(dy, c * nw + warp, lane, p.H, uc);
        K::load(hp, c * nw + warp, lane, p.H, hc);
      }
      if constexpr (!kWeights) K::load_w(p.w, p.w_f32, p.w_offset, c * nw + warp, lane, p.H, w[0]);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        dw[c][j] = fmaf(uc[j] * rstd, hc[j], dw[c][j]);
        uc[j] *= w[kWeights ? c : 0][j];
        sum = fmaf(uc[j], hc[j], sum);
      }
    }
    const float k = block_sum<NW>(sum, smem[turn], nw) * p.inv_H * rstd * rstd * rstd;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float(&uc)[E] = u[kHold ? c : 0];
      float(&hc)[E] = h[kHold ? c : 0];
      if constexpr (!kHold) {
        if constexpr (kAhead) {
          piece(slot, 0, c, uc);
          piece(slot, 1, c, hc);
        } else {
          K::load(dy, c * nw + warp, lane, p.H, uc);
          K::load(hp, c * nw + warp, lane, p.H, hc);
        }
        K::load_w(p.w, p.w_f32, p.w_offset, c * nw + warp, lane, p.H, w[0]);
#pragma unroll
        for (int j = 0; j < E; ++j) uc[j] *= w[0][j];
      }
      float d[E];
#pragma unroll
      for (int j = 0; j < E; ++j) d[j] = rstd * uc[j] - hc[j] * k;
      if (p.has_dh) {
        float(&tc)[E] = t[kNext ? c : 0];
        if constexpr (kAhead) piece(slot, 2, c, tc);
        else if constexpr (!kNext) K::load(static_cast<const T*>(p.dh[r]) + off, c * nw + warp, lane, p.H, tc);
#pragma unroll
        for (int j = 0; j < E; ++j) d[j] += tc[j];
      }
      K::store(static_cast<T*>(p.dx[r]) + off, c * nw + warp, lane, p.H, d);
    }
    slot = slot + 1 == Cfg::kRows ? 0 : slot + 1;
  }
  if (p.has_dw) {   // (one value a store, a sector of memory would be written eight times over)
    float* const part = p.part + (int64_t)blockIdx.x * p.H;
    constexpr int kStore = VEC >= 4 ? 4 : VEC;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < E; j += kStore) {
        const int col = K::col(c * nw + warp, lane, j);
        if (FULL || col < p.H) {
          if constexpr (kStore == 4)
            *reinterpret_cast<float4*>(part + col) = make_float4(dw[c][j], dw[c][j + 1], dw[c][j + 2], dw[c][j + 3]);
          else if constexpr (kStore == 2)
            *reinterpret_cast<float2*>(part + col) = make_float2(dw[c][j], dw[c][j + 1]);
          else
            part[col] = dw[c][j];
        }
      }
  }
}

// dweight[c] = sum of the blocks' partial sums. A block has COLS columns; a
// warp adds every (warps * 32 / COLS)th block's for them, 32 / COLS at a time,
// then the lanes' and the warps' sums are added in order. As many loads in
// flight as there are: the loads' latency is what counts (8192 x 4096 bf16,
// 304 partial sums: 3.5 us of the backward pass with 32 warps, 8 with eight),
// and no more warps than there are sums for (18 x 4096: 5.4 us both kernels,
// 6.7 with 32 warps).
template <int COLS>
__global__ void __launch_bounds__(1024) dweight_kernel(const float* part, int blocks, int H, float* dw) {
  constexpr int kSub = 32 / COLS;
  __shared__ float smem[32][COLS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (int)blockDim.x >> 5;
  const int c = blockIdx.x * COLS + lane % COLS;
  float s = 0.f;
  grid_release();
  grid_wait();
  if (c < H) {
#pragma unroll 10
    for (int b = warp * kSub + lane / COLS; b < blocks; b += warps * kSub) s += part[(int64_t)b * H + c];
  }
#pragma unroll
  for (int o = COLS; o < 32; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane < COLS) smem[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && lane < COLS && c < H) {
    for (int k = 1; k < warps; ++k) s += smem[k][lane];
    dw[c] = s;
  }
}

fo_status check_desc(const fo_norm_desc* d, int64_t rows) {
  if (!d) return FO_ERR_INVALID_ARG;
  if (d->R < 1 || d->R > kMaxR || d->reserved[0] || d->reserved[1]) return FO_ERR_INVALID_ARG;
  if (d->H < 1 || d->H > FO_NORM_MAX_H || rows < 0 || rows > INT32_MAX) return FO_ERR_SHAPE;
  if ((d->dtype != FO_BF16 && d->dtype != FO_F32) || (d->w_dtype != FO_BF16 && d->w_dtype != FO_F32))
    return FO_ERR_DTYPE;
  if (!(d->eps >= 0.f) || !(d->w_offset == d->w_offset)) return FO_ERR_INVALID_ARG;
  return FO_OK;
}

size_t elem(int32_t dtype) { return dtype == FO_BF16 ? 2 : 4; }

// Chunks of a thread for rows of n chunks, the warps that cover them, and
// the warps that a kernel is compiled for.
int chunks_for(int n) { return n <= 8 ? 1 : n <= 32 ? 2 : n <= 128 ? 4 : 8; }
int warps_for(int n) { return (n + chunks_for(n) - 1) / chunks_for(n); }
int most_warps(int n) { return n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : n <= 16 ? 8 : n <= 64 ? 16 : 32; }
// Blocks of the backward pass (its partial sums are one row each).
// At least four rows each where that leaves a block for every SM: more
// blocks' partial sums would cost more than the rows (2529 x 128: 9.5 us with
// as many blocks as fit).
int bwd_blocks(int64_t total, int nw, int c) {
  const int64_t most = bwd_per_sm(nw, c) * FO_GB300_SMS, least = total < FO_GB300_SMS ? total : FO_GB300_SMS;
  const int64_t want = total / 4 > least ? total / 4 : least;
  return (int)(want < most ? want : most);
}

template <int N>
using Int = std::integral_constant<int, N>;

// Calls f.template operator()<T, VEC, NW, C, FULL>(n) for rows of n chunks:
// one chunk a thread while 8 warps suffice, then up to 32 warps and up to 8
// chunks.
template <typename T, int VEC, typename F>
fo_status by_width(int H, F&& f) {
  using K = Chunk<T, VEC, false>;
  constexpr int kCols = K::COLS;
  const int n = (H + kCols - 1) / kCols;
  auto go = [&](auto nw, auto c) -> fo_status {
    constexpr int NW = decltype(nw)::value, C = decltype(c)::value;
    if constexpr (K::WIDE)
      if (H == NW * C * kCols) return f.template operator()<T, VEC, NW, C, true>(n);
    return f.template operator()<T, VEC, NW, C, false>(n);
  };
  if (n <= 1) return go(Int<1>(), Int<1>());
  if (n <= 2) return go(Int<2>(), Int<1>());
  if (n <= 4) return go(Int<4>(), Int<1>());
  if (n <= 8) return go(Int<8>(), Int<1>());
  if (n <= 16) return go(Int<8>(), Int<2>());
  if (n <= 32) return go(Int<16>(), Int<2>());
  if (n <= 64) return go(Int<16>(), Int<4>());
  if (n <= 128) return go(Int<32>(), Int<4>());
  if constexpr (kCols * 128 < FO_NORM_MAX_H) return go(Int<32>(), Int<8>());
  return FO_ERR_SHAPE;
}
// The values that an access may have: rows of H and every tensor start on them.
struct Width {
  int vec;
  Width(int most, int H) : vec(most) { fit((uintptr_t)(unsigned)H); }
  void fit(uintptr_t at) {   // `at`: in elements
    while (at % vec) vec /= 2;
  }
  void add(int R, const void* const* a, int size) {
    for (int r = 0; a && r < R; ++r) fit(reinterpret_cast<uintptr_t>(a[r]) / size);
  }
};
template <typename F>
fo_status by_type(int32_t dtype, int vec, int H, F&& f) {
  if (dtype == FO_F32) return vec == 4 ? by_width<float, 4>(H, f) : by_width<float, 1>(H, f);
  return vec == 8   ? by_width<__nv_bfloat16, 8>(H, f)
         : vec == 4 ? by_width<__nv_bfloat16, 4>(H, f)
         : vec == 2 ? by_width<__nv_bfloat16, 2>(H, f)
                    : by_width<__nv_bfloat16, 1>(H, f);
}

struct LaunchFwd {
  const NormParams& k;
  cudaStream_t s;
  int R;
  template <typename T, int VEC, int NW, int C, bool FULL>
  fo_status operator()(int n) const {
    const int nw = kAllWarps<NW, C> ? NW : warps_for(n);
    // The GPU starts about a block a nanosecond, which is longer than a narrow
    // row takes: its blocks take several, as many blocks as an SM holds, twice
    // that from five warps on (16384 x 512 bf16: 8.1 us, 17.1 with a block for
    // every row; 16384 x 128: 5.4 and 17.1; 8191 x 1280: 8.7 and 10.1).
    int64_t blocks = k.rows;
    if (C == 1) {
      const int64_t most = (int64_t)FO_GB300_SMS * (nw == 1 ? 32 : nw <= 4 ? 64 / nw : 128 / nw) / R;
      if (blocks > most) blocks = most;
    }
    const dim3 grid((unsigned)blocks, R);
    return launched(launch_after(rmsnorm_kernel<T, VEC, NW, C, FULL>, grid, nw * 32, 0, 0, s, k), "rmsnorm", R, k.rows, k.H, (int)blocks, nw * 32);
  }
};
struct LaunchBwd {
  const NormBwdParams& k;
  cudaStream_t s;
  int R;
  int* blocks;
  template <typename T, int VEC, int NW, int C, bool FULL>
  fo_status operator()(int n) const {
    const int nw = BwdCfg<T, VEC, NW, C>::kAhead ? warps_for(n) : NW;
    const int grid = *blocks = bwd_blocks(k.total, nw, C);
    const int smem = BwdCfg<T, VEC, NW, C>::smem(nw);
    auto kern = rmsnorm_bwd_kernel<T, VEC, NW, C, FULL>;
    // Leave for what the kernel's most warps take, whatever this call takes: the
    // leave is the process's, and another thread's launch may lie behind it.
    constexpr int most = BwdCfg<T, VEC, NW, C>::smem(NW);
    static_assert(most <= 232448 - 1024, "shared memory per block");
    if (most > 47 * 1024) {   // (with the static part, beyond what needs no leave)
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) return launched(e, "rmsnorm_bwd", R, k.rows, k.H, grid, nw * 32);
    }
    return launched(launch_after(kern, dim3(grid), nw * 32, smem, 0, s, k), "rmsnorm_bwd", R, k.rows, k.H, grid, nw * 32);
  }
};

}  // namespace
}  // namespace fo_ops

extern "C" fo_status fo_rmsnorm(const fo_norm_desc* d, int64_t rows, const void* const* x,
                                const void* const* residual, const void* weight, void* const* h, void* const* y,
                                void* const* q, float* const* scale, float* const* rstd, fo_stream_t stream) {
  using namespace fo_ops;
  fo_status st = check_desc(d, rows);
  if (st) return st;
  if (!weight || (!h && !y && !q && !rstd) || (!q != !scale)) return FO_ERR_INVALID_ARG;
  if (rows == 0) return FO_OK;
  const int R = d->R;
  const size_t es = elem(d->dtype);
  typedef const void* const* A;
  if ((st = check_array(R, x, es)) || (residual && (st = check_array(R, residual, es))) ||
      (h && (st = check_array(R, (A)h, es))) || (y && (st = check_array(R, (A)y, es))) ||
      (q && ((st = check_array(R, (A)q, 1)) || (st = check_array(R, (A)scale, 4)))) ||
      (rstd && (st = check_array(R, (A)rstd, 4))))
    return st;
  if (!aligned(weight, elem(d->w_dtype))) return FO_ERR_ALIGN;
  int sms;
  if ((st = device_sms(&sms))) return st;
  PtrList l;
  l.add(R, x), l.add(R, residual), l.add(R, (A)h), l.add(R, (A)y), l.add(R, (A)q), l.add(R, (A)scale);
  l.add(R, (A)rstd), l.add(weight);
  if ((st = check_device(l, stream))) return st;
  NormParams k;
  memset(&k, 0, sizeof(k));
  for (int r = 0; r < R; ++r) {
    k.x[r] = x[r];
    k.res[r] = residual ? residual[r] : nullptr;
    k.h[r] = h ? h[r] : nullptr;
    k.y[r] = y ? y[r] : nullptr;
    k.q[r] = q ? static_cast<uint8_t*>(q[r]) : nullptr;
    k.scale[r] = scale ? scale[r] : nullptr;
    k.rstd[r] = rstd ? rstd[r] : nullptr;
  }
  k.w = weight;
  k.rows = rows;
  k.H = d->H;
  k.groups = (d->H + FO_FP8_BLOCK - 1) / FO_FP8_BLOCK;
  k.eps = d->eps;
  k.w_offset = d->w_offset;
  k.inv_H = 1.f / (float)d->H;
  k.has_res = residual, k.has_h = h, k.has_y = y, k.has_q = q, k.has_rstd = rstd;
  k.w_f32 = d->w_dtype == FO_F32;
  const int es_i = (int)es;
  Width v(16 / es_i, d->H);
  if (!aligned(weight, 16)) v.add(1, &weight, (int)elem(d->w_dtype));   // (no access is wider)
  v.add(R, x, es_i), v.add(R, residual, es_i), v.add(R, (A)h, es_i), v.add(R, (A)y, es_i), v.add(R, (A)q, 1);
  return by_type(d->dtype, v.vec, d->H, LaunchFwd{k, (cudaStream_t)stream, R});
}

extern "C" fo_status fo_rmsnorm_bwd_workspace(const fo_norm_desc* d, int64_t rows, size_t* bytes) {
  using namespace fo_ops;
  const fo_status st = check_desc(d, rows);
  if (st) return st;
  if (!bytes) return FO_ERR_INVALID_ARG;
  // Enough for rows on the 16-byte grid (chunks of 256 or 128 columns) and off
  // it (of 128), with as many warps as the rows need and with the kernel's most.
  const int cols[2] = {d->dtype == FO_BF16 ? 256 : 128, 128};
  size_t n = 0;
  for (const int c : cols) {
    const int chunks = (d->H + c - 1) / c;
    for (const int w : {warps_for(chunks), most_warps(chunks)}) {
      const size_t b = (size_t)bwd_blocks(rows * d->R, w, chunks_for(chunks)) * (size_t)d->H * sizeof(float);
      n = b > n ? b : n;
    }
  }
  *bytes = n ? n : 16;
  return FO_OK;
}

extern "C" fo_status fo_rmsnorm_bwd(const fo_norm_desc* d, int64_t rows, const void* const* dy,
                                    const void* const* dh, const void* const* h, const void* weight,
                                    const float* const* rstd, void* const* dx, float* dweight, void* ws,
                                    fo_stream_t stream) {
  using namespace fo_ops;
  fo_status st = check_desc(d, rows);
  if (st) return st;
  if (!weight || (dweight && !ws)) return FO_ERR_INVALID_ARG;
  const int R = d->R;
  const size_t es = elem(d->dtype);
  typedef const void* const* A;
  if (rows > 0 && ((st = check_array(R, dy, es)) || (dh && (st = check_array(R, dh, es))) ||
                   (st = check_array(R, h, es)) || (st = check_array(R, (A)rstd, 4)) ||
                   (st = check_array(R, (A)dx, es))))
    return st;
  if (!aligned(weight, elem(d->w_dtype)) || !aligned(dweight, 4) || !aligned(ws, 16)) return FO_ERR_ALIGN;
  int sms;
  if ((st = device_sms(&sms))) return st;
  PtrList l;
  if (rows > 0) l.add(R, dy), l.add(R, dh), l.add(R, h), l.add(R, (A)rstd), l.add(R, (A)dx), l.add(weight);
  l.add(dweight), l.add(ws);
  if ((st = check_device(l, stream))) return st;
  const cudaStream_t s = (cudaStream_t)stream;
  if (rows == 0) {   // an empty sum
    if (dweight && cudaMemsetAsync(dweight, 0, (size_t)d->H * 4, s) != cudaSuccess) {
      cudaGetLastError();
      return FO_ERR_CUDA;
    }
    return FO_OK;
  }
  NormBwdParams k;
  memset(&k, 0, sizeof(k));
  for (int r = 0; r < R; ++r) {
    k.dy[r] = dy[r];
    k.dh[r] = dh ? dh[r] : nullptr;
    k.h[r] = h[r];
    k.rstd[r] = rstd[r];
    k.dx[r] = dx[r];
  }
  k.w = weight;
  k.part = static_cast<float*>(ws);
  k.rows = rows;
  k.total = rows * R;
  k.H = d->H;
  k.w_offset = d->w_offset;
  k.inv_H = 1.f / (float)d->H;
  k.has_dh = dh, k.has_dw = dweight;
  k.w_f32 = d->w_dtype == FO_F32;
  const int es_i = (int)es;
  Width v(16 / es_i, d->H);
  if (!aligned(weight, 16)) v.add(1, &weight, (int)elem(d->w_dtype));   // (no access is wider)
  v.add(R, dy, es_i), v.add(R, dh, es_i), v.add(R, h, es_i), v.add(R, (A)dx, es_i);
  int grid = 0;
  if ((st = by_type(d->dtype, v.vec, d->H, LaunchBwd{k, s, R, &grid}))) return st;
  if (!dweight) return FO_OK;
  // Slices of 8 columns where 32 would make few blocks.
  const int cols = d->H >= 32 * FO_GB300_SMS / 2 ? 32 : 8, slices = (d->H + cols - 1) / cols;
  int warps = (grid + 4 * (32 / cols) - 1) / (4 * (32 / cols));
  warps = warps < 2 ? 2 : warps > 32 ? 32 : warps;
  auto kern = cols == 32 ? dweight_kernel<32> : dweight_kernel<8>;
  return launched(launch_after(kern, dim3(slices), warps * 32, 0, 0, s, (const float*)k.part, grid, d->H, dweight),
                  "rmsnorm_dweight", R, grid, d->H, slices, warps * 32);
}
