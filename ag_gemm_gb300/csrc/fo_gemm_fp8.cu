// Product of e4m3 matrices with a scale for each block of 128 of the
// reduction, on the tensor cores (tcgen05.mma.kind::f8f6f4, fp32 accumulators
// in tensor memory):
//   Y[m][n] = sum_b sA[m][b] sW[n/128][b] P_b[m][n],  P_b the plain product
//   over block b.
// The scales change with b, so no accumulator may run over the whole
// reduction: each P_b (one stage of 128 reduction bytes) goes into a tensor
// memory buffer of its own, and warps add it, scaled, into fp32 registers
// while the tensor core fills the next buffer.
//
// Two kernels share the work by size (choose() below says which):
//   wide    256 x 256 tiles on CTA pairs, persistent: many rows, tensor-bound;
//   narrow  128 weight rows x 16..128 rows of A on one CTA, the operands'
//           roles swapped (the weight is the MMA's 128-row operand, so few
//           rows of A cost few columns), the reduction split over a cluster:
//           few rows, bound by the stream of weights.
#include <cudaTypedefs.h>
#include <stdio.h>
#include <string.h>

#include "fo_device.cuh"
#include "fo_ops.h"

namespace fo_ops {
namespace {

using namespace fo;

constexpr uint64_t kWaitNs = 2000000000ull;   // every wait's bound
constexpr int kBlockK = FO_FP8_BLOCK;         // reduction bytes a stage

struct GemmParams {
  CUtensorMap tmA[kMaxR];   // A_r [M x K] bytes
  CUtensorMap tmW[kMaxR];   // W_r [N x K] bytes
  const float* sA[kMaxR];
  const float* sW[kMaxR];
  void* Y[kMaxR];
  int32_t* status;
  int32_t R, M, N, kblocks, nblocks;   // nblocks: 128-row blocks of W
  int32_t tiles_m, tiles_n;
  int32_t f32, vec;                    // vec: rows of Y start on 16 bytes
};

// kind::f8f6f4 instruction descriptor: D fp32 (bits 4-5 = 1), A and B e4m3
// (bits 7-9 and 10-12 = 0), both K-major, N >> 3 (bits 17-22), M >> 4 (bits
// 24-28).
__host__ __device__ constexpr uint32_t idesc_fp8(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <int CG>
__device__ __forceinline__ void mma_fp8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One arrival on an mbarrier of this cluster. Release at CTA scope: what it
// guards, tensor memory that has been read into registers
// (tcgen05.wait::ld), is no memory that a wider fence would order, and the
// cluster-wide release waits for every outstanding store: with it each block
// of the reduction took about four times as long.
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
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

// ------------------------------------------------------------------- wide

namespace wide {

// 12 warps: 0 TMA producer, 1 MMAs (the pair's leader) and TMEM, 2-3 idle,
// 4-11 accumulate: a warp's 32 rows (its TMEM lane quarter) x 128 columns,
// 128 fp32 sums a thread. The registers come from the first warpgroup: 384 x
// 168 at launch = 128 x 56 + 256 x 224.
constexpr int kThreads = 384;
constexpr int kStages = 6;
constexpr int kTile = 256;
constexpr uint32_t kOperand = 128 * kBlockK;          // 16 KB: this CTA's 128 rows of A, or its half of W's 256
constexpr uint32_t kStageBytes = 2 * kOperand;
constexpr int kSmem = 1024 + kStages * (int)kStageBytes + 256;
static_assert(kSmem <= 232448, "shared memory per CTA");
constexpr int kPanel = 8;   // row tiles that go through all column tiles together (their A stays in L2)

struct Tile {
  int r, mt, nt;
};
__device__ __forceinline__ Tile decode(const GemmParams& p, int L) {
  const int per = p.tiles_m * p.tiles_n;
  Tile t;
  t.r = L / per;
  const int i = L - t.r * per;
  const int panel = i / (kPanel * p.tiles_n);
  const int rows = min(kPanel, p.tiles_m - panel * kPanel);
  const int j = i - panel * kPanel * p.tiles_n;
  t.nt = j / rows;
  t.mt = panel * kPanel + j - t.nt * rows;
  return t;
}

template <bool F32>
__device__ __forceinline__ void store_row(const GemmParams& p, int r, int m, int n0, const f32x2 (&acc)[64]) {
  if (m >= p.M || n0 >= p.N) return;
  const int left = p.N - n0;
  if constexpr (F32) {
    float* y = static_cast<float*>(p.Y[r]) + (int64_t)m * p.N + n0;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      float v[4];
      halves(acc[2 * c], v[0], v[1]);
      halves(acc[2 * c + 1], v[2], v[3]);
      if (p.vec && 4 * c + 4 <= left) {
        *reinterpret_cast<float4*>(y + 4 * c) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * c + j < left) y[4 * c + j] = v[j];
      }
    }
  } else {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.Y[r]) + (int64_t)m * p.N + n0;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) halves(acc[4 * c + j], v[2 * j], v[2 * j + 1]);
      if (p.vec && 8 * c + 8 <= left) {
        *reinterpret_cast<uint4*>(y + 8 * c) = Vec16<__nv_bfloat16>::pack(v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (8 * c + j < left) y[8 * c + j] = __float2bfloat16_rn(v[j]);
      }
    }
  }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads, 1) gemm_fp8_wide_kernel(const __grid_constant__ GemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sBar = base + kStages * kStageBytes;
  auto full_bar = [&](int i) { return sBar + 8u * i; };
  auto empty_bar = [&](int i) { return sBar + 8u * (kStages + i); };
  auto tfull_bar = [&](uint32_t a) { return sBar + 8u * (2 * kStages + a); };
  auto tempty_bar = [&](uint32_t a) { return sBar + 8u * (2 * kStages + 2 + a); };
  const uint32_t done_bar = sBar + 8u * (2 * kStages + 4);
  const uint32_t slot = sBar + 8u * (2 * kStages + 5);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + (slot - base));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + (slot - base) + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t prank = cluster_ctarank();
  const bool leader = prank == 0;
  const int unit = (int)(blockIdx.x >> 1), units = (int)(gridDim.x >> 1);
  const int total = p.R * p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full_bar(i), 1);
      mbar_init(empty_bar(i), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 16);   // eight warps of each CTA
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc<2>(slot, 512);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------- producer
      uint32_t it = 0, ph = 0;
      int st = 0;
      bool ok = true;
      for (int L = unit; L < total && ok; L += units) {
        const Tile t = decode(p, L);
        const int m0 = t.mt * kTile + (int)prank * 128, n0 = t.nt * kTile + (int)prank * 128;
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          if (!mbar_wait(empty_bar(st), ph ^ 1u, abort_flag, kWaitNs)) {
            ok = false;
            break;
          }
          const uint32_t fb = mapa_shared(full_bar(st), 0);
          if (leader) mbar_arrive_expect_tx(full_bar(st), 2 * kStageBytes);   // both CTAs' loads
          const uint32_t sa = base + st * kStageBytes;
          tma_load_2d_pair(sa, &p.tmA[t.r], fb, kb * kBlockK, m0);
          tma_load_2d_pair(sa + kOperand, &p.tmW[t.r], fb, kb * kBlockK, n0);
          if (++st == kStages) st = 0, ph ^= 1u;
        }
      }
      // Every load still in flight lands before the CTA may exit.
      volatile int never = 0;
      if (leader) {
        for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0u; j < it; ++j)
          mbar_wait(full_bar(j % kStages), (j / kStages) & 1u, &never, 100000000ull);
      } else if (*abort_flag) {
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 200000ull) __nanosleep(1000);
      }
      if (*abort_flag) record_error(p.status, FO_ERR_TIMEOUT, -1, -1, 0);
    } else if (warp == 1 && lane == 0 && leader) {
      // ------------------------------------------------------------ MMAs
      uint32_t it = 0, ph = 0;
      int st = 0;
      bool ok = true;
      constexpr uint32_t id = idesc_fp8(256, 256);
      for (int L = unit; L < total && ok; L += units) {
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const uint32_t a = it & 1u;
          if (!mbar_wait(tempty_bar(a), ((it >> 1) & 1u) ^ 1u, abort_flag, kWaitNs) ||
              !mbar_wait(full_bar(st), ph, abort_flag, kWaitNs)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base + st * kStageBytes;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_fp8<2>(tmem + a * 256u, smem_desc_sw128(sa + k * 32u, 16, 1024),
                       smem_desc_sw128(sa + kOperand + k * 32u, 16, 1024), id, k > 0 ? 1u : 0u);
          tc_commit_pair_multicast(empty_bar(st), 0x3);
          tc_commit_pair_multicast(tfull_bar(a), 0x3);
          if (++st == kStages) st = 0, ph ^= 1u;
        }
      }
      // Every issued MMA completes before TMEM is released.
      tc_commit<2>(done_bar);
      volatile int never = 0;
      mbar_wait(done_bar, 0, &never, 100000000ull);
    }
  } else {
    // ---------------------------------------------------------- accumulate
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_col = ((uint32_t)(q * 32) << 16) + (uint32_t)half * 128u;
    const uint32_t free0 = mapa_shared(tempty_bar(0), 0), free1 = mapa_shared(tempty_bar(1), 0);
    uint32_t it = 0;
    bool ok = true;
    for (int L = unit; L < total && ok; L += units) {
      const Tile t = decode(p, L);
      const int m = t.mt * kTile + (int)prank * 128 + q * 32 + lane;
      const int n0 = t.nt * kTile + half * 128, nb = n0 / 128;
      // The row's and the columns' scales of a block are loaded a block ahead.
      const bool in = m < p.M && nb < p.nblocks;
      const float* sa = p.sA[t.r] + (int64_t)(in ? m : 0) * p.kblocks;
      const float* sw = p.sW[t.r] + (int64_t)(in ? nb : 0) * p.kblocks;
      float a_next = __ldg(sa), w_next = __ldg(sw);
      f32x2 acc[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = 0ull;
      for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
        const float s = a_next * w_next;
        const f32x2 s2 = pair_of(s, s);
        if (kb + 1 < p.kblocks) a_next = __ldg(sa + kb + 1), w_next = __ldg(sw + kb + 1);
        const uint32_t b = it & 1u;
        if (!mbar_wait(tfull_bar(b), (it >> 1) & 1u, abort_flag, kWaitNs)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = tmem + lane_col + b * 256u;
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          uint32_t v[2][32];
          tmem_ld32(at + c * 32, v[0]);
          tmem_ld32(at + c * 32 + 32, v[1]);
          tmem_ld_wait();
          reg_fence(v[0]);
          reg_fence(v[1]);
          if (c == 2) {   // the buffer has been read: the tensor core may fill it again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at(b ? free1 : free0);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j)
            acc[c * 16 + j] = fma2(pair_of(v[j >> 4][(2 * j) & 31], v[j >> 4][(2 * j + 1) & 31]), s2, acc[c * 16 + j]);
        }
      }
      if (ok) store_row<F32>(p, t.r, m, n0, acc);
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();   // neither CTA leaves while the pair still uses its memory
  if (warp == 1) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc<2>(tmem, 512);
  }
}

}  // namespace wide

// ----------------------------------------------------------------- narrow

namespace narrow {

// 6 warps: 0 TMA producer, 1 MMAs and TMEM, 2-5 accumulate (TN fp32 sums a
// thread: lane = weight row, register = row of A). Two CTAs fit on an SM.
constexpr int kThreads = 192;
constexpr uint32_t kWBytes = 128 * kBlockK;

template <int TN>
struct Cfg {
  static constexpr uint32_t kXBytes = TN * kBlockK;
  static constexpr uint32_t kStageBytes = kWBytes + kXBytes;
  static constexpr int kStages = TN <= 32 ? 5 : TN <= 64 ? 4 : 3;
  static constexpr int kBufs = TN <= 64 ? 4 : 2;                      // TMEM buffers of TN columns
  static constexpr uint32_t kCols = TN * kBufs < 64 ? 64 : TN * kBufs;   // allocated: a power of two
  static constexpr uint32_t kRing = kStages * kStageBytes;
};

// Beside the ring: barriers, and the scales of kScaleBlocks blocks of the
// reduction at a time ([blocks][TN], the product of both; rows padded to
// spread the banks).
constexpr int kScaleBlocks = 32;
template <int TN>
constexpr int smem_bytes() {
  return 1024 + (int)Cfg<TN>::kRing + 256 + kScaleBlocks * (TN + 4) * 4;
}

template <int TN>
__global__ void __launch_bounds__(kThreads) gemm_fp8_narrow_kernel(const __grid_constant__ GemmParams p, int split) {
  using C = Cfg<TN>;
  constexpr int S = C::kStages, NB = C::kBufs;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sBar = base + C::kRing;
  auto full_bar = [&](int i) { return sBar + 8u * i; };
  auto empty_bar = [&](int i) { return sBar + 8u * (S + i); };
  auto tfull_bar = [&](uint32_t a) { return sBar + 8u * (2 * S + a); };
  auto tempty_bar = [&](uint32_t a) { return sBar + 8u * (2 * S + NB + a); };
  const uint32_t done_bar = sBar + 8u * (2 * S + 2 * NB);
  const uint32_t slot = done_bar + 8u;
  static_assert(8 * (2 * S + 2 * NB + 2) <= 256, "barriers");
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + (slot - base));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + (slot - base) + 4);
  float* const sScale = reinterpret_cast<float*>(gbase + C::kRing + 256);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // blockIdx.x: share of the reduction (the cluster's rank), .y: block of 128
  // weight rows, .z: rank and tile of A's rows.
  const int part = (int)blockIdx.x, nb = (int)blockIdx.y;
  const int r = (int)blockIdx.z / p.tiles_m, m0 = ((int)blockIdx.z % p.tiles_m) * TN;
  const int kb0 = (int)((int64_t)p.kblocks * part / split), kb1 = (int)((int64_t)p.kblocks * (part + 1) / split);
  const int blocks = kb1 - kb0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full_bar(i), 1);
      mbar_init(empty_bar(i), 1);
    }
    for (int a = 0; a < NB; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc<1>(slot, C::kCols);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  float acc[TN];
  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------------- producer
      int i = 0;
      for (; i < blocks; ++i) {
        const int st = i % S;
        if (!mbar_wait(empty_bar(st), ((uint32_t)(i / S) & 1u) ^ 1u, abort_flag, kWaitNs)) break;
        mbar_arrive_expect_tx(full_bar(st), C::kStageBytes);
        const uint32_t sw = base + st * C::kStageBytes;
        tma_load_2d(sw, &p.tmW[r], full_bar(st), (kb0 + i) * kBlockK, nb * 128);
        tma_load_2d(sw + kWBytes, &p.tmA[r], full_bar(st), (kb0 + i) * kBlockK, m0);
      }
      // Every load still in flight lands before the ring is used again.
      volatile int never = 0;
      for (int j = i > S ? i - S : 0; j < i; ++j)
        mbar_wait(full_bar(j % S), (uint32_t)(j / S) & 1u, &never, 100000000ull);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMAs
      constexpr uint32_t id = idesc_fp8(128, TN);
      for (int i = 0; i < blocks; ++i) {
        const int st = i % S;
        const uint32_t a = (uint32_t)i % NB;
        if (!mbar_wait(tempty_bar(a), ((uint32_t)(i / NB) & 1u) ^ 1u, abort_flag, kWaitNs) ||
            !mbar_wait(full_bar(st), (uint32_t)(i / S) & 1u, abort_flag, kWaitNs))
          break;
        tc_fence_after();
        const uint32_t sw = base + st * C::kStageBytes;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_fp8<1>(tmem + a * TN, smem_desc_sw128(sw + k * 32u, 16, 1024),
                     smem_desc_sw128(sw + kWBytes + k * 32u, 16, 1024), id, k > 0 ? 1u : 0u);
        tc_commit<1>(empty_bar(st));
        tc_commit<1>(tfull_bar(a));
      }
      tc_commit<1>(done_bar);
      volatile int never = 0;
      mbar_wait(done_bar, 0, &never, 100000000ull);
    }
  } else {
    // ---------------------------------------------------------- accumulate
    const int q = warp & 3, tid = threadIdx.x - 64;
    auto load_scales = [&](int first) {
#pragma unroll 4
      for (int i = tid; i < kScaleBlocks * TN; i += 128) {
        const int c = i / kScaleBlocks, b = i % kScaleBlocks;   // neighbours: neighbouring blocks of a row
        const int m = m0 + c, kb = kb0 + first + b;
        if (m < p.M && kb < kb1)
          sScale[b * (TN + 4) + c] = __ldg(p.sA[r] + (int64_t)m * p.kblocks + kb) *
                                     __ldg(p.sW[r] + (int64_t)nb * p.kblocks + kb);
        else
          sScale[b * (TN + 4) + c] = 0.f;
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
    };
#pragma unroll
    for (int c = 0; c < TN; ++c) acc[c] = 0.f;
    for (int i = 0; i < blocks; ++i) {
      if (i % kScaleBlocks == 0) {
        if (i) asm volatile("bar.sync 1, 128;" ::: "memory");   // the last scales have been read
        load_scales(i);
      }
      const uint32_t a = (uint32_t)i % NB;
      // (After a wait that ran out the loop goes on, for the barriers' sake:
      // the waits that follow return at once.)
      mbar_wait(tfull_bar(a), (uint32_t)(i / NB) & 1u, abort_flag, kWaitNs);
      tc_fence_after();
      const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + a * TN;
      const float4* s4 = reinterpret_cast<const float4*>(sScale + (i % kScaleBlocks) * (TN + 4));
      if constexpr (TN == 16) {
        uint32_t v[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
              "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
            : "r"(at));
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(v[j]));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(a));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 s = s4[j];
          acc[4 * j] = fmaf(__uint_as_float(v[4 * j]), s.x, acc[4 * j]);
          acc[4 * j + 1] = fmaf(__uint_as_float(v[4 * j + 1]), s.y, acc[4 * j + 1]);
          acc[4 * j + 2] = fmaf(__uint_as_float(v[4 * j + 2]), s.z, acc[4 * j + 2]);
          acc[4 * j + 3] = fmaf(__uint_as_float(v[4 * j + 3]), s.w, acc[4 * j + 3]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < TN; c += 32) {
          uint32_t v[32];
          tmem_ld32(at + c, v);
          tmem_ld_wait();
          reg_fence(v);
          if (c + 32 == TN) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(a));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 s = s4[c / 4 + j];
            acc[c + 4 * j] = fmaf(__uint_as_float(v[4 * j]), s.x, acc[c + 4 * j]);
            acc[c + 4 * j + 1] = fmaf(__uint_as_float(v[4 * j + 1]), s.y, acc[c + 4 * j + 1]);
            acc[c + 4 * j + 2] = fmaf(__uint_as_float(v[4 * j + 2]), s.z, acc[c + 4 * j + 2]);
            acc[c + 4 * j + 3] = fmaf(__uint_as_float(v[4 * j + 3]), s.w, acc[c + 4 * j + 3]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();   // loads and MMAs are done: the ring is free
  if (warp == 1) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc<1>(tmem, C::kCols);
  }
  if (threadIdx.x == 0 && *abort_flag) record_error(p.status, FO_ERR_TIMEOUT, -1, -1, 0);

  // The sums of the cluster's CTAs meet in shared memory, [TN][128] each in
  // the ring's place; every CTA adds and stores its share of A's rows, in
  // the order of the reduction.
  float* const sSum = reinterpret_cast<float*>(gbase);
  static_assert(C::kRing >= TN * 128 * 4, "the sums fit into the ring");
  if (warp >= 2) {
    const int row = (warp & 3) * 32 + lane;
#pragma unroll
    for (int c = 0; c < TN; ++c) sSum[c * 128 + row] = acc[c];
  }
  __syncwarp();
  if (split > 1) cluster_sync_all();
  else __syncthreads();
  const int rows = min(TN, p.M - m0);
  const int c0 = rows * part / split, c1 = rows * (part + 1) / split;
  for (int i = c0 * 128 + (int)threadIdx.x; i < c1 * 128; i += kThreads) {
    const int c = i >> 7, n = nb * 128 + (i & 127);
    float s = 0.f;
    if (split > 1) {
      for (int k = 0; k < split; ++k) {
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(base + 4u * (uint32_t)i, k)) : "memory");
        s += v;
      }
    } else {
      s = sSum[i];
    }
    if (n < p.N) {
      const int64_t at = (int64_t)(m0 + c) * p.N + n;
      if (p.f32) static_cast<float*>(p.Y[r])[at] = s;
      else static_cast<__nv_bfloat16*>(p.Y[r])[at] = __float2bfloat16_rn(s);
    }
  }
  __syncwarp();
  if (split > 1) cluster_sync_all();   // no CTA leaves while another reads its sums
}

template <int TN>
cudaError_t launch(const GemmParams& k, int split, cudaStream_t s, int* grid_out) {
  constexpr int smem = smem_bytes<TN>();
  auto kern = gemm_fp8_narrow_kernel<TN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(split, k.nblocks, k.tiles_m * k.R);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = split;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  *grid_out = split * k.nblocks * k.tiles_m * k.R;
  return cudaLaunchKernelEx(&cfg, kern, k, split);
}

}  // namespace narrow

struct Choice {
  int tn, split;   // tn 0: wide
};

// Which kernel, and how it is cut.
Choice choose(int R, int64_t M, int64_t N, int64_t kblocks) {
  Choice c;
  const int64_t pairs = R * ((M + 255) / 256) * ((N + 255) / 256);
  if (M > 128 && pairs >= 38) return {0, 1};
  c.tn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const int64_t tiles = R * ((M + c.tn - 1) / c.tn) * ((N + 127) / 128);
  c.split = 1;
  while (c.split < 8 && tiles * c.split * 2 <= 2 * FO_GB300_SMS && kblocks >= 4 * c.split) c.split *= 2;
  return c;
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

// [rows x cols] bytes, boxes of 128 columns x `box` rows; what lies outside
// reads as zero.
bool encode(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint32_t box) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols};
  cuuint32_t size[2] = {128, box};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, size, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  memset(static_cast<void*>(&k), 0, sizeof(k));
  k.kblocks = (int32_t)((d->K + kBlockK - 1) / kBlockK);
  k.nblocks = (int32_t)((d->N + 127) / 128);
  const Choice c = choose(R, M, d->N, k.kblocks);
  for (int r = 0; r < R; ++r) {
    if (r && A[r] == A[r - 1]) k.tmA[r] = k.tmA[r - 1];
    else if (!encode(&k.tmA[r], A[r], (uint64_t)d->K, (uint64_t)M, c.tn ? c.tn : 128)) return FO_ERR_CUDA;
    if (!encode(&k.tmW[r], W[r], (uint64_t)d->K, (uint64_t)d->N, 128)) return FO_ERR_CUDA;
    k.sA[r] = sA[r];
    k.sW[r] = sW[r];
    k.Y[r] = Y[r];
  }
  k.status = static_cast<int32_t*>(ws);
  k.R = R;
  k.M = (int32_t)M;
  k.N = (int32_t)d->N;
  k.f32 = d->out_dtype == FO_F32;
  k.vec = (d->N * (k.f32 ? 4 : 2)) % 16 == 0;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  int grid = 0, threads = 0;
  if (c.tn == 0) {
    k.tiles_m = (int32_t)((M + 255) / 256);
    k.tiles_n = (int32_t)((d->N + 255) / 256);
    const int64_t total = (int64_t)R * k.tiles_m * k.tiles_n;
    if (total > INT32_MAX / 2) return FO_ERR_SHAPE;
    auto kern = k.f32 ? wide::gemm_fp8_wide_kernel<true> : wide::gemm_fp8_wide_kernel<false>;
    threads = wide::kThreads;
    grid = 2 * (int)(total < sms / 2 ? total : sms / 2);
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, wide::kSmem);
    if (e == cudaSuccess) {
      cudaLaunchConfig_t cfg;
      memset(&cfg, 0, sizeof(cfg));
      cfg.gridDim = dim3(grid);
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = wide::kSmem;
      cfg.stream = s;
      cudaLaunchAttribute at;
      at.id = cudaLaunchAttributeClusterDimension;
      at.val.clusterDim.x = 2;
      at.val.clusterDim.y = at.val.clusterDim.z = 1;
      cfg.attrs = &at;
      cfg.numAttrs = 1;
      e = cudaLaunchKernelEx(&cfg, kern, k);
    }
  } else {
    k.tiles_m = (int32_t)((M + c.tn - 1) / c.tn);
    k.tiles_n = k.nblocks;
    threads = narrow::kThreads;
    switch (c.tn) {
      case 16: e = narrow::launch<16>(k, c.split, s, &grid); break;
      case 32: e = narrow::launch<32>(k, c.split, s, &grid); break;
      case 64: e = narrow::launch<64>(k, c.split, s, &grid); break;
      default: e = narrow::launch<128>(k, c.split, s, &grid); break;
    }
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FO_ERR_CUDA;
  }
  return launched(c.tn ? "gemm_fp8 narrow" : "gemm_fp8 wide", R, M, d->N, grid, threads);
}
