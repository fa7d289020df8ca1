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
//   wide    256 x 256 (or 128) tiles on CTA pairs, persistent: many rows, tensor-bound
//           (8 ranks of 8192 x 1536 x 4096: 276 us, 2.99 PFLOP/s, 68% of the
//           tensor pipe's cycles; in a loop for seconds, under the power cap,
//           311 us);
//   narrow  128 weight rows x 16..64 rows of A on one CTA, the operands'
//           roles swapped (the weight is the MMA's 128-row operand, so few
//           rows of A cost few columns), the reduction split over a cluster:
//           few rows, bound by the stream of weights (4 x 12288 x 4096 from
//           HBM: 10.6 us, 4.7 TB/s, of which 3 us are start and end).
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
  CUtensorMap tmY[kMaxR];   // Y_r [M x N] (where its rows start on 16 bytes)
  const float* sA[kMaxR];
  const float* sW[kMaxR];
  void* Y[kMaxR];
  int32_t* status;
  int32_t R, M, N, kblocks, nblocks;   // nblocks: 128-row blocks of W
  int32_t tiles_m, tiles_n;
  Divisor per_rank, per_panel, last_panel;   // wide: tiles of a rank, of a panel, rows of the last panel
  int32_t f32;
  int32_t vec, row8, row4;             // rows of Y start on 16, 8, 4 bytes
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

// 32 lanes x 16 consecutive columns (tmem_ld32's layout).
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(at));
}

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one;
}

// mbar_wait without a look at the clock on the common path (the clock is
// first read after 64 tries).
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 63u) == 0) {
      if (*abort_flag) return false;
      const uint64_t t = globaltimer();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitNs) {
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// ------------------------------------------------------------------- wide

namespace wide {

// 12 warps: 0 TMA producer, 1 MMAs (the pair's leader) and TMEM, 2-3 idle,
// 4-11 accumulate: a warp's 32 rows (its TMEM lane quarter) x 128 columns,
// 128 fp32 sums a thread. The registers come from the first warpgroup: 384 x
// 168 at launch = 128 x 56 + 256 x 224.
//
// A block of the reduction is 512 cycles of the tensor core. Two buffers of
// 256 columns leave 1024 from the start of a buffer's MMAs to its next ones,
// so that commit, wake-up, reads and release have to fit in 512: the second
// half of a buffer is loaded while the first is being added, and the buffer
// is released before the last additions. A finished tile goes through shared
// memory to TMA stores (rows stored straight from registers took 6000 cycles
// a tile); scales are loaded a block ahead, across tiles too.
//
// Tiles of 128 columns keep four buffers and 64 sums a thread. For the same
// work they take a third longer (4096 x 4096 x 4096: 60.5 us, 54.0 with 256
// columns, which leave a sixth of their waves empty), so choose() takes them
// where tiles of 256 would leave more than that idle (256 x 9728 x 4096:
// 12.0 us, 15.5 with 256; 4 ranks of 3836 x 64 x 13216: 27.9 us and 38.9).
constexpr int kThreads = 384;
constexpr int kTile = 256;                            // rows
constexpr uint32_t kOutBuf = 32 * 128;                // a warp's piece of the output: 32 rows x 128 bytes
template <int TN>
struct Cfg {
  static constexpr int kStages = TN == 256 ? 5 : 6;
  static constexpr int kBufs = 512 / TN;                                // TMEM buffers of TN columns
  static constexpr int kCols = TN / 2;                                  // a warp's columns
  static constexpr uint32_t kOperandA = 128 * kBlockK;                  // this CTA's 128 rows of A
  static constexpr uint32_t kStageBytes = kOperandA + kCols * kBlockK;  // and its half of W's TN rows
  static constexpr uint32_t kOffOut = kStages * kStageBytes;
  static constexpr uint32_t kOffBar = kOffOut + 16 * kOutBuf;
  static constexpr int kSmem = 1024 + (int)kOffBar + 256;
  static_assert(kSmem <= 232448, "shared memory per CTA");
  static_assert(8 * (2 * kStages + 2 * kBufs + 2) <= 256, "barriers");
};
constexpr int kPanel = 8;   // row tiles that go through all column tiles together (their A stays in L2)

struct Tile {
  int r, mt, nt;
};
__device__ __forceinline__ Tile decode(const GemmParams& p, int L) {
  Tile t;
  t.r = (int)p.per_rank((uint32_t)L);
  const uint32_t i = (uint32_t)L - (uint32_t)t.r * p.per_rank.d;
  const uint32_t panel = p.per_panel(i), j = i - panel * p.per_panel.d;
  const bool full = (int)panel * kPanel + kPanel <= p.tiles_m;
  t.nt = (int)(full ? j / kPanel : p.last_panel(j));
  t.mt = (int)(panel * kPanel + j) - t.nt * (full ? kPanel : (int)p.last_panel.d);
  return t;
}

// 32 words a lane (a row of 128 bytes) into a 32 x 128 byte buffer, 16-byte
// chunk j of row i at chunk j ^ (i % 8): the TMA's 128-byte swizzle, and free
// of bank conflicts.
__device__ __forceinline__ void stage_row(uint32_t buf, int lane, const uint32_t (&w)[32]) {
  const uint32_t row = buf + (uint32_t)lane * 128u;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((uint32_t)(j ^ (lane & 7)) << 4)),
                 "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                 : "memory");
}
__device__ __forceinline__ uint32_t staged_word(uint32_t buf, int row, int word) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];"
               : "=r"(v)
               : "r"(buf + (uint32_t)row * 128u + ((uint32_t)((word >> 2) ^ (row & 7)) << 4) + (uint32_t)(word & 3) * 4u)
               : "memory");
  return v;
}

// A warp's 32 rows x COLS columns at (m, n) of Y_r, through its two buffers.
template <bool F32, int COLS>
__device__ __forceinline__ void store_part(const GemmParams& p, int r, int m, int n, uint32_t bufs, int lane,
                                           const f32x2 (&acc)[COLS / 2]) {
  if (m >= p.M || n >= p.N) return;
  constexpr int kBytes = F32 ? 4 : 2, kCols = 128 / kBytes, kParts = COLS / kCols;   // columns in 128 bytes
#pragma unroll
  for (int h0 = 0; h0 < kParts; h0 += 2) {   // both buffers, then their stores behind one fence
    if (lane == 0) bulk_wait_read<0>();   // the buffers' last stores have read them
    __syncwarp();
#pragma unroll
    for (int h = h0; h < h0 + 2 && h < kParts; ++h) {
      uint32_t w[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float lo, hi;
        if constexpr (F32) {
          halves(acc[h * 16 + j / 2], lo, hi);
          w[j] = __float_as_uint(j & 1 ? hi : lo);
        } else {
          halves(acc[h * 32 + j], lo, hi);
          const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
          w[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      stage_row(bufs + (uint32_t)(h & 1) * kOutBuf, lane, w);
    }
    if (p.vec) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (n + h0 * kCols < p.N) tma_store_2d(&p.tmY[r], bufs, n + h0 * kCols, m);   // clipped at Y's edges
        if (h0 + 1 < kParts && n + h0 * kCols + kCols < p.N) tma_store_2d(&p.tmY[r], bufs + kOutBuf, n + h0 * kCols + kCols, m);
        bulk_commit();
      }
    } else {   // rows of Y that no TMA store can start on: lanes along the columns
      __syncwarp();
      for (int h = h0; h < h0 + 2 && h < kParts; ++h) {
        const uint32_t buf = bufs + (uint32_t)(h & 1) * kOutBuf;
        const int c0 = n + h * kCols;
        uint8_t* const y = static_cast<uint8_t*>(p.Y[r]) + ((int64_t)m * p.N + c0) * kBytes;
        const int64_t ld = (int64_t)p.N * kBytes;
        if (p.row8) {   // 8 bytes a lane, two rows at a time
          const int col = c0 + (lane & 15) * (8 / kBytes);
#pragma unroll 8
          for (int i = lane >> 4; i < 32; i += 2) {
            const uint32_t lo = staged_word(buf, i, 2 * (lane & 15)), hi = staged_word(buf, i, 2 * (lane & 15) + 1);
            if (m + i < p.M && col < p.N) *reinterpret_cast<uint2*>(y + i * ld + (lane & 15) * 8) = make_uint2(lo, hi);
          }
        } else if (F32 || p.row4) {   // 4 bytes
          const int col = c0 + lane * (4 / kBytes);
#pragma unroll 8
          for (int i = 0; i < 32; ++i) {
            const uint32_t v = staged_word(buf, i, lane);
            if (m + i < p.M && col < p.N) *reinterpret_cast<uint32_t*>(y + i * ld + lane * 4) = v;
          }
        } else {
          const int col = c0 + 2 * lane;
#pragma unroll 8
          for (int i = 0; i < 32; ++i) {
            const uint32_t v = staged_word(buf, i, lane);
            uint16_t* const to = reinterpret_cast<uint16_t*>(y + i * ld + lane * 4);
            if (m + i < p.M && col < p.N) to[0] = (uint16_t)v;
            if (m + i < p.M && col + 1 < p.N) to[1] = (uint16_t)(v >> 16);
          }
        }
      }
      __syncwarp();
    }
  }
}

template <bool F32, int TN>
__global__ void __launch_bounds__(kThreads, 1) gemm_fp8_wide_kernel(const __grid_constant__ GemmParams p) {
  using C = Cfg<TN>;
  constexpr int kStages = C::kStages, NB = C::kBufs;
  constexpr uint32_t kStageBytes = C::kStageBytes;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sBar = base + C::kOffBar;
  auto full_bar = [&](uint32_t i) { return sBar + 8u * i; };
  auto empty_bar = [&](uint32_t i) { return sBar + 8u * (kStages + i); };
  auto tfull_bar = [&](uint32_t a) { return sBar + 8u * (2 * kStages + a); };
  auto tempty_bar = [&](uint32_t a) { return sBar + 8u * (2 * kStages + NB + a); };
  const uint32_t done_bar = sBar + 8u * (2 * kStages + 2 * NB);
  const uint32_t slot = done_bar + 8u;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + (slot - base));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + (slot - base) + 4);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t prank = cluster_ctarank();
  const bool leader = prank == 0;
  const int unit = (int)(blockIdx.x >> 1), units = (int)(gridDim.x >> 1);
  const int total = p.R * p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full_bar(i), 1);
      mbar_init(empty_bar(i), 1);
    }
    for (int a = 0; a < NB; ++a) {
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
  grid_release();
  grid_wait();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------- producer
      uint32_t it = 0, ph = 0;
      int st = 0;
      bool ok = true;
      for (int L = unit; L < total && ok; L += units) {
        const Tile t = decode(p, L);
        const int m0 = t.mt * kTile + (int)prank * 128, n0 = t.nt * TN + (int)prank * C::kCols;
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          if (!wait_bar(empty_bar(st), ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t fb = mapa_shared(full_bar(st), 0);
          if (leader) mbar_arrive_expect_tx(full_bar(st), 2 * kStageBytes);   // both CTAs' loads
          const uint32_t sa = base + st * kStageBytes;
          tma_load_2d_pair(sa, &p.tmA[t.r], fb, kb * kBlockK, m0);
          tma_load_2d_pair(sa + C::kOperandA, &p.tmW[t.r], fb, kb * kBlockK, n0);
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
    } else if (warp == 1 && leader) {
      // ------------------------------------------------------------ MMAs
      // The whole warp runs the loop and one elected lane issues: descriptors
      // and barrier addresses are then the same in every lane for the
      // compiler too and stay in uniform registers, where the MMA wants them.
      // (From a loop of one lane's own, each MMA took 85 cycles to issue.)
      constexpr uint32_t id = idesc_fp8(256, TN);
      const uint64_t a0 = smem_desc_sw128(base, 16, 1024), w0 = smem_desc_sw128(base + C::kOperandA, 16, 1024);
      uint32_t st = 0, ph = 0, b = 0, bph = 1;
      bool ok = true;
      for (int L = unit; L < total && ok; L += units) {
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!__all_sync(0xffffffffu,
                          wait_bar(tempty_bar(b), bph, abort_flag) && wait_bar(full_bar(st), ph, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t da = a0 + st * (kStageBytes >> 4), dw = w0 + st * (kStageBytes >> 4);
            const uint32_t d = tmem + b * (uint32_t)TN;
            mma_fp8<2>(d, da, dw, id, 0);
            mma_fp8<2>(d, da + 2, dw + 2, id, 1);   // 32 bytes further along the rows
            mma_fp8<2>(d, da + 4, dw + 4, id, 1);
            mma_fp8<2>(d, da + 6, dw + 6, id, 1);
            tc_commit_pair_multicast(tfull_bar(b), 0x3);
            tc_commit_pair_multicast(empty_bar(st), 0x3);
          }
          __syncwarp();
          if (++st == kStages) st = 0, ph ^= 1u;
          if (++b == NB) b = 0, bph ^= 1u;
        }
      }
      // Every issued MMA completes before TMEM is released.
      if (elect_one()) {
        tc_commit<2>(done_bar);
        volatile int never = 0;
        mbar_wait(done_bar, 0, &never, 100000000ull);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- accumulate
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int q = warp & 3, h = (warp - 4) >> 2;
    const uint32_t at0 = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * C::kCols);
    const uint32_t bufs = base + C::kOffOut + (uint32_t)(warp - 4) * 2 * kOutBuf;
    const uint32_t free0 = mapa_shared(tempty_bar(0), 0);
    uint32_t it = 0;
    bool ok = true;
    // The scales of the row and of the columns' block, by block of the
    // reduction; what lies outside reads the first ones and is not stored.
    const float *sa = nullptr, *sw = nullptr;
    auto scales_of = [&](int L) {
      const Tile t = decode(p, L);
      const int m = t.mt * kTile + (int)prank * 128 + q * 32 + lane, nb = t.nt * (TN / 128) + h * C::kCols / 128;
      sa = p.sA[t.r] + (int64_t)(m < p.M ? m : 0) * p.kblocks;
      sw = p.sW[t.r] + (int64_t)(nb < p.nblocks ? nb : 0) * p.kblocks;
    };
    float a_next = 0.f, w_next = 0.f;
    if (unit < total) {
      scales_of(unit);
      a_next = load1(sa), w_next = load1(sw);
    }
    for (int L = unit; L < total && ok; L += units) {
      f32x2 acc[C::kCols / 2];
#pragma unroll
      for (int c = 0; c < C::kCols / 2; ++c) acc[c] = 0ull;
      for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
        const float s = a_next * w_next;
        const f32x2 s2 = pair_of(s, s);
        if (kb + 1 < p.kblocks) {
          a_next = load1(sa + kb + 1), w_next = load1(sw + kb + 1);
        } else if (L + units < total) {
          scales_of(L + units);
          a_next = load1(sa), w_next = load1(sw);
        }
        const uint32_t b = it % NB;
        if (!wait_bar(tfull_bar(b), (it / NB) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = at0 + b * (uint32_t)TN;
        auto add = [&](int c, const uint32_t(&v)[32]) {
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c * 16 + j] = fma2(pair_of(v[2 * j], v[2 * j + 1]), s2, acc[c * 16 + j]);
        };
        uint32_t v0[32], v1[32];
        tmem_ld32(at, v0);
        tmem_ld32(at + 32, v1);
        tmem_ld_wait();
        reg_fence(v0);
        reg_fence(v1);
        if constexpr (TN == 256) {
          add(0, v0);
          tmem_ld32(at + 64, v0);
          add(1, v1);
          tmem_ld32(at + 96, v1);
          tmem_ld_wait();
          reg_fence(v0);
          reg_fence(v1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(free0 + b * 8u);   // read: the tensor core may fill it again
        add(C::kCols / 32 - 2, v0);
        add(C::kCols / 32 - 1, v1);
      }
      if (ok) {
        const Tile t = decode(p, L);
        store_part<F32, C::kCols>(p, t.r, t.mt * kTile + (int)prank * 128 + q * 32, t.nt * TN + h * C::kCols, bufs, lane, acc);
      }
    }
    if (lane == 0) bulk_wait<0>();   // the stores are done with shared memory
    __syncwarp();
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
constexpr int kScaleBlocks = 32;   // blocks whose scales are in shared memory at a time
constexpr int kMaxSplit = 8;       // CTAs that share a reduction (portable cluster size)

// Blocks of weights that a CTA asks for while the kernel before it ends (4 x
// 12288 x 4096 from HBM, back to back: none 11.8 us, four 10.7, sixteen 11.6).
constexpr int kPrefetchBlocks = 4;

__device__ __forceinline__ void prefetch_box(const CUtensorMap* map, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

template <int TN>
struct Cfg {
  static constexpr uint32_t kXBytes = TN * kBlockK;
  static constexpr uint32_t kStageBytes = kWBytes + kXBytes;
  static constexpr int kStages = TN <= 16 ? 5 : 4;
  static constexpr int kBufs = 4;                                        // TMEM buffers of TN columns
  static constexpr uint32_t kCols = TN * kBufs < 64 ? 64 : TN * kBufs;   // allocated: a power of two
  static constexpr uint32_t kRing = kStages * kStageBytes;
  static constexpr int kScaleLd = TN + 4;   // [block][row of A], padded to spread the banks
  static constexpr uint32_t kScales = kScaleBlocks * kScaleLd * 4;
  static constexpr uint32_t kOffBar = kRing;
  static constexpr uint32_t kOffScale = kOffBar + 256;
  static constexpr int kSmem = 1024 + (int)(kOffScale + kScales);
  static_assert(TN * 128 * 4 <= kRing, "a CTA's sums fit in the ring's place");
};

template <int TN>
__global__ void __launch_bounds__(kThreads) gemm_fp8_narrow_kernel(const __grid_constant__ GemmParams p, int split) {
  using C = Cfg<TN>;
  constexpr int S = C::kStages, NB = C::kBufs;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sBar = base + C::kOffBar;
  auto full_bar = [&](uint32_t i) { return sBar + 8u * i; };
  auto empty_bar = [&](uint32_t i) { return sBar + 8u * (S + i); };
  auto tfull_bar = [&](uint32_t a) { return sBar + 8u * (2 * S + a); };
  auto tempty_bar = [&](uint32_t a) { return sBar + 8u * (2 * S + NB + a); };
  const uint32_t done_bar = sBar + 8u * (2 * S + 2 * NB);
  const uint32_t slot = done_bar + 8u;
  static_assert(8 * (2 * S + 2 * NB + 2) <= 256, "barriers");
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + (slot - base));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + (slot - base) + 4);
  float* const sScale = reinterpret_cast<float*>(gbase + C::kOffScale);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  // blockIdx.x: share of the reduction (the cluster's rank), .y: block of 128
  // weight rows, .z: rank and tile of A's rows.
  const int part = (int)blockIdx.x, nb = (int)blockIdx.y;
  const int r = (int)blockIdx.z / p.tiles_m, m0 = ((int)blockIdx.z % p.tiles_m) * TN;
  const int kb0 = p.kblocks * part / split, kb1 = p.kblocks * (part + 1) / split;
  const int blocks = kb1 - kb0;
  const int rows = min(TN, p.M - m0);
  const int share = (rows + split - 1) / split;   // rows of A that one CTA adds up and stores

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
  // While the kernel before this one ends, the CTA's first weights come into
  // L2: a hint that reads nothing, so it need not wait. (From every tile of A's
  // rows the same hints would queue for the same lines.)
  if (warp == 0 && m0 == 0 && elect_one())
    for (int i = 0; i < blocks && i < kPrefetchBlocks; ++i) prefetch_box(&p.tmW[r], (kb0 + i) * kBlockK, nb * 128);
  __syncwarp();
  grid_wait();
  __syncwarp();

  f32x2 acc[TN / 2];
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t st = 0, ph = 1;
    int i = 0;
    for (; i < blocks; ++i) {
      if (!__all_sync(0xffffffffu, wait_bar(empty_bar(st), ph, abort_flag))) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(full_bar(st), C::kStageBytes);
        const uint32_t sw = base + st * C::kStageBytes;
        tma_load_2d(sw, &p.tmW[r], full_bar(st), (kb0 + i) * kBlockK, nb * 128);
        tma_load_2d(sw + kWBytes, &p.tmA[r], full_bar(st), (kb0 + i) * kBlockK, m0);
      }
      __syncwarp();
      if (++st == S) st = 0, ph ^= 1u;
    }
    // Every load still in flight lands before the ring is used again.
    volatile int never = 0;
    for (int j = i > S ? i - S : 0; j < i; ++j)
      mbar_wait(full_bar(j % S), (uint32_t)(j / S) & 1u, &never, 100000000ull);
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMAs
    // (The whole warp, one lane issuing: see the wide kernel.)
    constexpr uint32_t id = idesc_fp8(128, TN);
    const uint64_t w0 = smem_desc_sw128(base, 16, 1024), x0 = smem_desc_sw128(base + kWBytes, 16, 1024);
    uint32_t st = 0, a = 0, ph = 0, aph = 1;
    for (int i = 0; i < blocks; ++i) {
      if (!__all_sync(0xffffffffu, wait_bar(tempty_bar(a), aph, abort_flag) && wait_bar(full_bar(st), ph, abort_flag)))
        break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dw = w0 + st * (C::kStageBytes >> 4), dx = x0 + st * (C::kStageBytes >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_fp8<1>(tmem + a * TN, dw + 2 * k, dx + 2 * k, id, k > 0 ? 1u : 0u);
        tc_commit<1>(tfull_bar(a));
        tc_commit<1>(empty_bar(st));
      }
      __syncwarp();
      if (++st == S) st = 0, ph ^= 1u;
      if (++a == NB) a = 0, aph ^= 1u;
    }
    if (elect_one()) {
      tc_commit<1>(done_bar);
      volatile int never = 0;
      mbar_wait(done_bar, 0, &never, 100000000ull);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- accumulate
    const int q = warp & 3;
    // Scales of blocks first .. first + 31: lane = block, so a warp reads 128
    // neighbouring bytes of a row's scales.
    auto load_scales = [&](int first) {
      const int kb = kb0 + first + lane;
      const bool in = kb < kb1;
      const float w = in ? load1(p.sW[r] + (int64_t)nb * p.kblocks + kb) : 0.f;
      const float* sa = p.sA[r] + (int64_t)m0 * p.kblocks + kb;
#pragma unroll
      for (int c = warp - 2; c < TN; c += 4)
        sScale[lane * C::kScaleLd + c] = in && c < rows ? w * load1(sa + (int64_t)c * p.kblocks) : 0.f;
      asm volatile("bar.sync 1, 128;" ::: "memory");
    };
#pragma unroll
    for (int c = 0; c < TN / 2; ++c) acc[c] = 0ull;
    int a = 0;
    uint32_t aph = 0;
    for (int i = 0; i < blocks; ++i) {
      const int at_scale = i % kScaleBlocks;
      if (at_scale == 0) {
        if (i) asm volatile("bar.sync 1, 128;" ::: "memory");   // the last scales have been read
        load_scales(i);
      }
      // (After a wait that ran out the loop goes on, for the barriers' sake:
      // the waits that follow return at once.)
      wait_bar(tfull_bar(a), aph, abort_flag);
      tc_fence_after();
      const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + a * TN;
      const ulonglong2* s4 = reinterpret_cast<const ulonglong2*>(sScale + at_scale * C::kScaleLd);
      constexpr int W = TN < 32 ? TN : 32;
#pragma unroll
      for (int c = 0; c < TN; c += W) {
        uint32_t v[W];
        if constexpr (TN == 16) tmem_ld16(at, v);
        else tmem_ld32(at + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < W; ++j) asm volatile("" : "+r"(v[j]));
        if (c + W == TN) {   // the buffer has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty_bar(a));
        }
#pragma unroll
        for (int j = 0; j < W / 4; ++j) {
          const ulonglong2 s = s4[c / 4 + j];
          acc[c / 2 + 2 * j] = fma2(pair_of(v[4 * j], v[4 * j + 1]), s.x, acc[c / 2 + 2 * j]);
          acc[c / 2 + 2 * j + 1] = fma2(pair_of(v[4 * j + 2], v[4 * j + 3]), s.y, acc[c / 2 + 2 * j + 1]);
        }
      }
      if (++a == NB) a = 0, aph ^= 1u;
    }
  }
  tc_fence_before();
  __syncthreads();   // loads and MMAs are done: the ring is free
  // Only now may the next kernel's blocks come: earlier ones would wait beside
  // this kernel's, two to an SM, and leave other SMs idle when they start
  // (333 x 1000 x 1744 back to back: 8.6 us instead of 6.8).
  grid_release();
  if (warp == 1) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc<1>(tmem, C::kCols);
  }
  if (threadIdx.x == 0 && *abort_flag) record_error(p.status, FO_ERR_TIMEOUT, -1, -1, 0);
  // The CTA's sums into its shared memory, [row of A][128 weight rows]; then
  // every CTA of the cluster adds up its share of A's rows from all of them,
  // in the order of the reduction, and stores them.
  if (warp >= 2) {
    float* mine = reinterpret_cast<float*>(gbase) + (warp & 3) * 32 + lane;
#pragma unroll
    for (int c = 0; c < TN; c += 2) halves(acc[c / 2], mine[c * 128], mine[c * 128 + 128]);
  }
  __syncwarp();
  if (split > 1) cluster_sync_all();
  else __syncthreads();
  const int n = nb * 128 + lane * 4;
  for (int j = warp; j < share && part * share + j < rows; j += kThreads / 32) {
    const int c = part * share + j;
    const uint32_t at = base + (uint32_t)(c * 128 + lane * 4) * 4u;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (split > 1) {
#pragma unroll 4
      for (int k = 0; k < split; ++k) {
        float4 u;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(u.x), "=f"(u.y), "=f"(u.z), "=f"(u.w)
                     : "r"(mapa_shared(at, (uint32_t)k))
                     : "memory");
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
    } else {
      v = *reinterpret_cast<const float4*>(gbase + (c * 128 + lane * 4) * 4);
    }
    const int64_t to = (int64_t)(m0 + c) * p.N + n;
    const float f[4] = {v.x, v.y, v.z, v.w};
    if (p.f32) {
      float* y = static_cast<float*>(p.Y[r]) + to;
      if (p.vec && n + 4 <= p.N) {
        *reinterpret_cast<float4*>(y) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < p.N) y[i] = f[i];
      }
    } else {
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.Y[r]) + to;
      if (p.vec && n + 4 <= p.N) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(y) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < p.N) y[i] = __float2bfloat16_rn(f[i]);
      }
    }
  }
  __syncwarp();
  if (split > 1) cluster_sync_all();   // no CTA leaves while another reads its sums
}

template <int TN>
cudaError_t launch(const GemmParams& k, int split, cudaStream_t s, int* grid_out) {
  auto kern = gemm_fp8_narrow_kernel<TN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<TN>::kSmem);
  if (e != cudaSuccess) return e;
  *grid_out = split * k.nblocks * k.tiles_m * k.R;
  return launch_after(kern, dim3(split, k.nblocks, k.tiles_m * k.R), kThreads, Cfg<TN>::kSmem, split, s, k, split);
}

}  // namespace narrow

namespace wide {

template <int TN>
cudaError_t launch(const GemmParams& k, int grid, cudaStream_t s) {
  auto kern = k.f32 ? gemm_fp8_wide_kernel<true, TN> : gemm_fp8_wide_kernel<false, TN>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<TN>::kSmem);
  return e != cudaSuccess ? e : launch_after(kern, dim3(grid), kThreads, Cfg<TN>::kSmem, 2, s, k);
}

}  // namespace wide

struct Choice {
  int tn, split;   // tn 0: wide, with tiles of `split` columns
};

// Which kernel, and how it is cut: the cheapest by a model of the time in ns,
// fitted to GB300 runs (operands in L2):
//   wide    3500 + waves of 76 tiles x (345 a block + 1200), with tiles of
//           128 columns 3300 + waves x (240 a block + 1000)
//   narrow  a start and an end for each wave, 10 for each tile of A's rows (all
//           of them read the same weights at once), then per block of a CTA's
//           share one time when it has the SM for itself and one when two share
//           it; a split adds the cluster's barriers and sums, and its clusters
//           fill the GPU less well.
// Both sides, measured: 128 x 12288 x 4096 wide 16.5 us, narrow 20.8 us; 128 x
// 4096 x 4096 wide 16.2 us, narrow 10.1 us (64 rows, split 4); 333 x 1000 x
// 1744 wide 11.1 us, narrow 6.8 us (32 rows, no split; split 3: 7.7 us); 4 x
// 12288 x 4096 8.9 us split in 3, 9.1 us whole; 1 x 4096 x 4096 5.5 us split in
// 4, 9.1 us whole; 6765 x 64 x 1104 wide (128) 5.6 us, narrow 8.5; 2729 x 64 x
// 9952 11.2 us split in 6, 17.0 in 8 (43 clusters, of which 30 fit).
Choice choose(int R, int64_t M, int64_t N, int64_t kblocks) {
  const int64_t pairs = FO_GB300_SMS / 2, rows_w = R * ((M + 255) / 256);
  Choice best = {0, 256};
  int64_t least = 3500 + (rows_w * ((N + 255) / 256) + pairs - 1) / pairs * (kblocks * 345 + 1200);
  const int64_t half = 3300 + (rows_w * ((N + 127) / 128) + pairs - 1) / pairs * (kblocks * 240 + 1000);
  if (half < least) least = half, best.split = 128;
  static const struct {
    int tn, fixed, alone, shared;
  } kNarrow[3] = {{16, 3300, 180, 400}, {32, 4350, 190, 320}, {64, 4900, 280, 520}};
  // CTAs that the GPU holds in whole clusters of 1 .. 8: one an SM (the runtime's
  // occupancy query), and two (where more than these took another wave).
  static const int kAlone[narrow::kMaxSplit] = {152, 152, 138, 144, 140, 138, 105, 120};
  static const int kShared[narrow::kMaxSplit] = {304, 304, 288, 288, 280, 276, 210, 240};
  for (const auto& v : kNarrow) {
    if (v.tn > 16 && v.tn >= 2 * M) break;   // more than half of the columns would be empty
    const int64_t tiles_m = (M + v.tn - 1) / v.tn, tiles = R * tiles_m * ((N + 127) / 128);
    if (tiles > 64 * FO_GB300_SMS) continue;   // long past the point where wide wins
    for (int64_t k = 1; k <= narrow::kMaxSplit && k <= kblocks; ++k) {
      const int64_t slots = kShared[k - 1], alone = kAlone[k - 1];
      const int64_t full = tiles * k / slots, rest = tiles * k % slots;
      const int64_t block = full * v.shared + (rest == 0 ? 0 : rest <= alone ? v.alone : v.shared);
      const int64_t waves = full + (rest ? 1 : 0);
      const int64_t cost = waves * v.fixed + tiles_m * 10 + (k > 1 ? 1200 : 0) + (kblocks + k - 1) / k * block;
      if (cost < least) least = cost, best = {v.tn, (int)k};
    }
  }
  return best;
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

// [rows x cols] values of `es` bytes, boxes of 128 bytes x `box` rows; what
// lies outside reads as zero and is not written.
bool encode(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint32_t box, int es = 1) {
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
  cuuint64_t strides[1] = {cols * es};
  cuuint32_t size[2] = {128u / es, box};
  cuuint32_t each[2] = {1, 1};
  const CUtensorMapDataType type = es == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  return fn(m, type, 2, const_cast<void*>(ptr), dims, strides, size, each,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

fo_status launched(cudaError_t e, const char* what, int R, int64_t rows, int64_t cols, int grid, int threads) {
  if (e != cudaSuccess) cudaGetLastError();
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
  k.f32 = d->out_dtype == FO_F32;
  const int es = k.f32 ? 4 : 2;
  k.vec = (d->N * es) % 16 == 0;
  k.row8 = (d->N * es) % 8 == 0;
  k.row4 = (d->N * es) % 4 == 0;
  for (int r = 0; r < R; ++r) {
    if (c.tn == 0 && k.vec && !encode(&k.tmY[r], Y[r], (uint64_t)d->N, (uint64_t)M, 32, es)) return FO_ERR_CUDA;
    if (r && A[r] == A[r - 1]) k.tmA[r] = k.tmA[r - 1];
    else if (!encode(&k.tmA[r], A[r], (uint64_t)d->K, (uint64_t)M, c.tn ? c.tn : 128)) return FO_ERR_CUDA;
    if (!encode(&k.tmW[r], W[r], (uint64_t)d->K, (uint64_t)d->N, c.tn ? 128 : c.split / 2)) return FO_ERR_CUDA;
    k.sA[r] = sA[r];
    k.sW[r] = sW[r];
    k.Y[r] = Y[r];
  }
  k.status = static_cast<int32_t*>(ws);
  k.R = R;
  k.M = (int32_t)M;
  k.N = (int32_t)d->N;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  int grid = 0, threads = 0;
  if (c.tn == 0) {
    k.tiles_m = (int32_t)((M + 255) / 256);
    k.tiles_n = (int32_t)((d->N + c.split - 1) / c.split);
    k.per_rank.set((uint32_t)(k.tiles_m * k.tiles_n));
    k.per_panel.set((uint32_t)(wide::kPanel * k.tiles_n));
    k.last_panel.set((uint32_t)(k.tiles_m % wide::kPanel ? k.tiles_m % wide::kPanel : wide::kPanel));
    const int64_t total = (int64_t)R * k.tiles_m * k.tiles_n;
    if (total > INT32_MAX / 2) return FO_ERR_SHAPE;
    threads = wide::kThreads;
    grid = 2 * (int)(total < sms / 2 ? total : sms / 2);
    e = c.split == 256 ? wide::launch<256>(k, grid, s) : wide::launch<128>(k, grid, s);
  } else {
    k.tiles_m = (int32_t)((M + c.tn - 1) / c.tn);
    k.tiles_n = k.nblocks;
    threads = narrow::kThreads;
    switch (c.tn) {
      case 16: e = narrow::launch<16>(k, c.split, s, &grid); break;
      case 32: e = narrow::launch<32>(k, c.split, s, &grid); break;
      default: e = narrow::launch<64>(k, c.split, s, &grid); break;
    }
  }
  return launched(e, c.tn ? "gemm_fp8 narrow" : "gemm_fp8 wide", R, M, d->N, grid, threads);
}
