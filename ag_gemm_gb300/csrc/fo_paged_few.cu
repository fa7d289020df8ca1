// Attention of a few new tokens a sequence over a paged cache: the cache's
// length is split.
//
// Reading the visible keys and values once is what a call cannot do without:
// 4 D flops for 4 D bytes (bf16), times the query heads that share a key head.
// So a unit of work is a sequence's key head with all rows (new tokens x heads
// of the group) that read it, up to 16 of them. Keys are the rows of the
// products and a unit's rows their columns, eight at a time:
//     S^T [16 keys x 8 rows] = K Q^T,   O^T [16 of D x 8 rows] += V^T P^T
// (mma.sync m16n8k16; tcgen05's 128 x 8 at least would have every tile's
// scores and weights cross between warps for 8 rows' work, and the eight rows
// of this form take 9% of even its rate). P's transposition in between is one
// movmatrix for 8 x 8. With the rows as the 16-row operand instead, half of
// what a decode step multiplies was padding, and the sums took twice the
// registers.
//
// The tiles of all units (the visible ones alone) form one line, in the order
// sequence, rank, head, tile; the line is cut into equal pieces, one for each
// block, so that every SM reads the same bytes whatever the lengths. A block
// finds its piece from the lengths on the device: a captured call may be
// replayed with other ones. In a block, one warp has TMA bring the tiles into a
// ring, running ahead over units and sequences (when each warp loaded for
// itself, two thirds of the instructions were that); each of four others takes
// 32 or 64 keys of a tile and keeps its own maximum, sum and output in
// registers. At a unit's end, or the piece's, the warps' parts are joined through
// shared memory. A unit cut between blocks is joined by the last of them to arrive,
// the parts in the blocks' order (16 at a time), so results repeat.
//
// An 8-bit cache's e4m3 values become f16, which holds them exactly; queries
// and weights are f16 then, the queries' rows times powers of two, the weights
// times their values' scales over a running power of two.
//
// Bound by bandwidth: 64 contexts of up to 8192 with 32 + 8 heads (1.34 GB of
// keys and values) take 203 us, 6.6 TB/s or 97% of a copy's; one of 131072 91
// us (87%: the join of 38 parts a head, and the start); 32 of up to 16384 in 8
// bits 123 us (84%). Eight of up to 512 take 10 us: the launch and look-ups,
// a tile, the join, each waiting for the one before (pieces of at least two or
// four tiles, with fewer blocks and joins, took 15.4 and 16.3 us, not 11.0). A
// third block an SM spilled (407 us for the 64 contexts).
#include <math.h>

#include <algorithm>

#include "fo_paged.h"
#include "fo_paged_tiles.cuh"

namespace fo_ops {
namespace {

using namespace fo;

constexpr int kRadix = 16;             // parts joined at a time

template <int D, bool E8, int NT>
struct Few {
  static constexpr int kKeys = few_keys(E8), kStep = 4 * kKeys;   // keys of a tile: of a warp, of all
  static constexpr int kM = kKeys / 16;
  static constexpr int kRow = D * (E8 ? 1 : 2);             // bytes of a key
  static constexpr int kWidth = kRow < 128 ? kRow : 128;    // of a box
  static constexpr int kCuts = kRow / kWidth;
  static constexpr int kSlot = kStep * kRow;                // a tile's keys, or its values
  static constexpr int kSlots = 98304 / kSlot;
  static constexpr int kRows = 8 * NT;
  static constexpr int kPart = kRows * (D + 2);             // floats of a part: output, maxima, sums
  // Shared memory: ring, scales, rows being joined (four of a warp at a time,
  // apart so that a warp's columns meet no bank twice), (m, l) of each warp,
  // barriers.
  static constexpr int kOffScale = kSlots * kSlot;
  static constexpr int kApart = D + 8;
  static constexpr int kOffJoin = kOffScale + (E8 ? kSlots * kStep * 4 : 0);
  static constexpr int kOffStat = kOffJoin + 3 * 4 * kApart * 4;
  static constexpr int kOffBar = kOffStat + 4 * 8 * NT * 8;
  static constexpr int kOffMisc = kOffBar + 2 * kSlots * 8;
  static constexpr int kSmem = 1024 + kOffMisc + 64;
  static_assert(kSlots >= 2 && kFewBlocks * (kSmem + 1024) <= 233472, "blocks an SM");
};

// Where a block is on the line of tiles.
template <int STEP>
struct Walk {
  int b, r, h, t, tiles;        // sequence, rank and key head, tile of the unit, tiles of a unit
  Seq s;
  int lo, sinks_end, early, late;
  __device__ __forceinline__ void of(const Batch& batch, int window, int sinks) {
    s = sequence(batch, b);
    const Sight v = sight_of(max(s.base, 0), window, sinks);
    lo = v.lo;
    sinks_end = v.sinks_end;
    early = (sinks_end + STEP - 1) / STEP;
    late = max(lo / STEP, early);
    tiles = s.n ? max(early + (s.end + STEP - 1) / STEP - late, 1) : 0;
  }
  __device__ __forceinline__ int first_key() const { return (t < early ? t : t - early + late) * STEP; }
  // Whether a new token may see one of the `n` tokens from key on.
  __device__ __forceinline__ bool any(int key, int n) const { return key < s.end && (key < sinks_end || key + n > lo); }
  __device__ __forceinline__ void next(const FewParams& p) {
    if (++t < tiles) return;
    t = 0;
    if (++h < p.heads_k) return;
    h = 0;
    if (++r < p.R) return;
    r = 0;
    do {
      if (++b >= p.batch.seqs) return;
      of(p.batch, p.window, p.sinks);
    } while (!tiles);
  }
};

__device__ __forceinline__ uint32_t transposed(uint32_t v) {   // 8 x 8 of 16 bits
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

template <int D, bool E8, int NT>
__global__ void __launch_bounds__(kFewThreads, kFewBlocks) few_kernel(const __grid_constant__ FewParams p) {
  using C = Few<D, E8, NT>;
  constexpr int kKeys = C::kKeys, kM = C::kM;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbase + C::kOffMisc);
  int* const misc = reinterpret_cast<int*>(gbase + C::kOffMisc);   // [0] abort, [1] flag, [2] sequence, [4..5] its first tile
  const uint32_t full = base + C::kOffBar, empty = full + C::kSlots * 8;
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) mbar_init(full + i * 8, 1), mbar_init(empty + i * 8, 4);
    *abort_flag = 0;
    misc[2] = -1;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  grid_release();
  grid_wait();

  // The line's length, and the sequence that this block's piece begins in. A
  // thread adds up a run of sequences.
  const int units = p.R * p.heads_k;
  long long total, x0, x1, piece;
  Walk<C::kStep> cw;
  {
    const int run = (p.batch.seqs + 127) / 128, first = tid < 128 ? tid * run : p.batch.seqs, last = min(first + run, p.batch.seqs);
    long long mine = 0;
    for (cw.b = first; cw.b < last; ++cw.b) cw.of(p.batch, p.window, p.sinks), mine += (long long)cw.tiles * units;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    long long* const sums = reinterpret_cast<long long*>(gbase + C::kOffStat);
    if (lane == 31 && warp < 4) sums[warp] = upto;
    __syncthreads();
    total = 0;
    for (int w = 0; w < 4; ++w) {
      if (w < warp) upto += sums[w];   // (warp 4 adds up none)
      total += sums[w];
    }
    piece = (total + gridDim.x - 1) / gridDim.x;   // (none has work where the line is empty)
    x0 = blockIdx.x * piece;
    x1 = min(x0 + piece, total);
    long long at = upto - mine;
    if (x0 < x1 && at <= x0 && x0 < upto) {
      for (cw.b = first;; ++cw.b) {
        cw.of(p.batch, p.window, p.sinks);
        const long long here = (long long)cw.tiles * units;
        if (x0 < at + here) break;
        at += here;
      }
      misc[2] = cw.b;
      *reinterpret_cast<long long*>(misc + 4) = at;
    }
    __syncthreads();
  }
  if (x0 >= x1) return;
  {
    cw.b = misc[2];
    cw.of(p.batch, p.window, p.sinks);
    const long long off = x0 - *reinterpret_cast<long long*>(misc + 4);
    const int u = (int)(off / cw.tiles);
    cw.t = (int)(off - (long long)u * cw.tiles);
    cw.r = u / p.heads_k;
    cw.h = u - cw.r * p.heads_k;
  }
  __syncthreads();

  // Of the 2 x 128 registers that a pair of threads is launched with, the four
  // computing warps take 208.
  if (warp >= 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp > 4) return;
    // ---- loads, a lane for each box: `box` tokens x 128 bytes
    const int boxes = 1 << p.boxes_log2, box = lane & (boxes - 1), cut = lane >> p.boxes_log2;
    const bool mine = cut < C::kCuts;
    const uint32_t to = base + cut * (C::kStep * 128) + box * p.box * C::kWidth;
    int slot = 0, round = 0;
    // The page of this lane's box in the tile that cw is at; -1 where none is
    // needed.
    auto page_of = [&]() -> int {
      const int key = cw.first_key() + box * p.box;
      if (!mine || !cw.any(key, p.box)) return -1;
      const int id = p.batch.table[(long long)cw.b * p.batch.cols + (key >> p.batch.shift)];
      if (id >= 0 && id < p.batch.pages) return id;
      report(p.batch, cw.b, kBadPage, id);
      return -1;
    };
    int id = page_of();
    long long left = x1 - x0;
    for (; left > 0; --left) {
      // What no page holds is read from behind the last one: zeros.
      const int z = id >= 0 ? id * p.heads_k + cw.h : p.batch.pages * p.heads_k, r = cw.r;
      const int y = (cw.first_key() + box * p.box) & ((1 << p.batch.shift) - 1);
      uint32_t bytes = C::kSlot;
      if constexpr (E8) bytes += __popc(__ballot_sync(0xffffffffu, mine && id >= 0)) * p.box * 4;
      // The next tile's pages are looked up meanwhile.
      cw.next(p);
      if (left > 1) id = page_of();
      bool ok = true;
#pragma unroll
      for (int value = 0; value < 2; ++value) {
        if (round > 0 && !(ok = mbar_wait(empty + slot * 8, (round - 1) & 1, abort_flag, kWaitNs))) break;
        const uint32_t bar = full + slot * 8;
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (mine) {
          tma_load_3d(to + slot * C::kSlot, value ? &p.v[r] : &p.k[r], bar, cut * 64, y, z);
          if constexpr (E8)
            if (z < p.batch.pages * p.heads_k)
              bulk_load(base + C::kOffScale + (slot * C::kStep + box * p.box) * 4,
                        (value ? p.vs[r] : p.ks[r]) + ((long long)z << p.batch.shift) + y, p.box * 4, bar);
        }
        if (++slot == C::kSlots) slot = 0, ++round;
      }
      if (!ok) break;
    }
    if (*abort_flag) {   // what is still on its way lands before the block may end
      volatile int never = 0;
      for (int i = 0; i < C::kSlots && (round || i < slot); ++i) {
        const int at = slot - 1 - i, wrapped = at < 0;
        mbar_wait(full + (wrapped ? at + C::kSlots : at) * 8, (round - wrapped) & 1, &never, 100000000ull);
      }
    }
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  int cslot = 0, cround = 0;
  // The slot that has been read is free again.
  auto done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + cslot * 8);
    if (++cslot == C::kSlots) cslot = 0, ++cround;
  };
  // The four warps that compute.
  auto meet = [&]() { asm volatile("barrier.sync 1, 128;" ::: "memory"); };

  for (long long x = x0; x < x1;) {
    // ---- a unit, or what of it is in this piece
    const int here = (int)min((long long)(cw.tiles - cw.t), x1 - x);
    const long long unit = x - cw.t;
    const bool whole = here == cw.tiles;
    const int tiles = cw.tiles, r = cw.r, h = cw.h, real = cw.s.n * p.group;
    const Seq s = cw.s;
    // Queries: the columns' fragments, row g of each eight.
    uint32_t qf[D / 16][NT][2];
    int pos[NT][2], lo[NT][2];          // of rows 2 c and 2 c + 1
    float qscale[NT][2];                // with what their scores are to be multiplied
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int rho = i * 8 + g, token = rho / p.group, head = rho - token * p.group;
      const bool is = rho < real;
      const __nv_bfloat16* const q = p.q[r] + (long long)(is ? s.row + token : 0) * p.ld_q + (h * p.group + head) * D;
      float mine = p.scale_log2;
      if constexpr (!E8) {
        // Elements in the order that 16-byte pieces of a key give them.
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (is) v = *reinterpret_cast<const uint4*>(q + (k >> 1) * 64 + (2 * c + (k & 1)) * 8);
          qf[2 * k][i][0] = v.x, qf[2 * k][i][1] = v.y, qf[2 * k + 1][i][0] = v.z, qf[2 * k + 1][i][1] = v.w;
        }
      } else {
        // The row times a power of two that brings its largest magnitude to
        // [128, 256) (or less: see least_exponent). What that makes smaller
        // than f16's least normal number is 2^-21 of the largest.
        constexpr int kEach = D / 4;   // elements of a thread
        uint4 v[kEach / 8];
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < kEach / 8; ++k) {
          v[k] = make_uint4(0, 0, 0, 0);
          if (is) v[k] = *reinterpret_cast<const uint4*>(q + c * kEach + k * 8);
          float f[8];
          Vec16<__nv_bfloat16>::unpack(v[k], f);
          top = max_nan(top, amax_of(f));
        }
        top = lanes_max<4>(top);
        const uint32_t exponent = min(max(__float_as_uint(top) >> 23, p.least_exponent), 254u);
        const float by = top <= 3.4e38f ? __uint_as_float((261u - exponent) << 23) : 1.f;
        mine *= 1.f / by;
#pragma unroll
        for (int k = 0; k < kEach / 4; ++k) {
          const uint32_t w0 = (k & 1) ? v[k / 2].z : v[k / 2].x, w1 = (k & 1) ? v[k / 2].w : v[k / 2].y;
          const float f0 = __uint_as_float(w0 << 16) * by, f1 = __uint_as_float(w0 & 0xffff0000u) * by;
          const float f2 = __uint_as_float(w1 << 16) * by, f3 = __uint_as_float(w1 & 0xffff0000u) * by;
          qf[k][i][0] = f16x2(f0, f1), qf[k][i][1] = f16x2(f2, f3);
        }
      }
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int mine_rho = i * 8 + 2 * c + a;
        pos[i][a] = mine_rho < real ? s.base + mine_rho / p.group : -1;
        lo[i][a] = sight_of(max(pos[i][a], 0), p.window, p.sinks).lo;
        qscale[i][a] = __shfl_sync(0xffffffffu, mine, (2 * c + a) * 4);
      }
    }
    float o[D / 16][NT][4], m[NT][2], l[NT][2];   // m: of the scores as they are, before their factor
    float sigma = 0.f, sigma_inv = 0.f;   // what the values' scales are divided by (a power of two), and its reciprocal
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      m[i][0] = m[i][1] = -INFINITY, l[i][0] = l[i][1] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
    }
    const uint32_t scales = base + C::kOffScale + warp * kKeys * 4;
    const int lo_last = sight_of(max(s.base + s.n - 1, 0), p.window, p.sinks).lo;

    for (int n = 0; n < here; ++n, cw.t += n < here ? 1 : 0) {
      const int key = cw.first_key() + warp * kKeys;
      if (!cw.any(key, kKeys)) {   // (other warps' keys)
        for (int value = 0; value < 2; ++value) {
          mbar_wait(full + cslot * 8, cround & 1, abort_flag, kWaitNs);
          done();
        }
        continue;
      }
      // All of a tile's keys seen by all rows?
      const bool part = !(key + kKeys - 1 <= s.base && (key >= lo_last || key + kKeys <= p.sinks));
      float sc[kM][NT][4];   // keys 16 i + g (and + 8) x rows 2 c, 2 c + 1
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) sc[i][t][0] = sc[i][t][1] = sc[i][t][2] = sc[i][t][3] = 0.f;
      mbar_wait(full + cslot * 8, cround & 1, abort_flag, kWaitNs);
      {
        const uint32_t at = base + cslot * C::kSlot + warp * kKeys * C::kWidth;
        if constexpr (!E8) {
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint4 v[kM][2];
#pragma unroll
            for (int i = 0; i < kM; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                v[i][e] = lds128(at + (k >> 1) * (C::kStep * 128) + (16 * i + 8 * e + g) * 128 + (((2 * c + (k & 1)) ^ g) << 4));
            // (Sums in turn: one after the other they would wait for each product.)
#pragma unroll
            for (int i = 0; i < kM; ++i)
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                const uint32_t a[4] = {v[i][0].x, v[i][1].x, v[i][0].y, v[i][1].y};
                mma16816<false>(sc[i][t], a, qf[2 * k][t][0], qf[2 * k][t][1]);
              }
#pragma unroll
            for (int i = 0; i < kM; ++i)
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                const uint32_t a[4] = {v[i][0].z, v[i][1].z, v[i][0].w, v[i][1].w};
                mma16816<false>(sc[i][t], a, qf[2 * k + 1][t][0], qf[2 * k + 1][t][1]);
              }
          }
        } else {
#pragma unroll
          for (int k = 0; k < D / 64; ++k)
#pragma unroll
            for (int i0 = 0; i0 < kM; i0 += 2) {
              uint4 v[2][2];
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int row = 16 * (i0 + i) + 8 * e + g;
                  v[i][e] = lds128(D == 128 ? at + row * 128 + (((2 * c + k) ^ g) << 4) : at + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
                }
#pragma unroll
              for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t w0 = e == 0 ? v[i][0].x : e == 1 ? v[i][0].y : e == 2 ? v[i][0].z : v[i][0].w;
                  const uint32_t w1 = e == 0 ? v[i][1].x : e == 1 ? v[i][1].y : e == 2 ? v[i][1].z : v[i][1].w;
                  const uint32_t a[4] = {f16x2_of_e4m3(w0), f16x2_of_e4m3(w1), f16x2_of_e4m3_high(w0), f16x2_of_e4m3_high(w1)};
#pragma unroll
                  for (int t = 0; t < NT; ++t) mma16816<true>(sc[i0 + i][t], a, qf[4 * k + e][t][0], qf[4 * k + e][t][1]);
                }
            }
#pragma unroll
          for (int i = 0; i < kM; ++i) {
            const float k0 = lds_f(scales + cslot * (C::kStep * 4) + (16 * i + g) * 4), k1 = lds_f(scales + cslot * (C::kStep * 4) + (16 * i + 8 + g) * 4);
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[i][t][0] *= k0, sc[i][t][1] *= k0, sc[i][t][2] *= k1, sc[i][t][3] *= k1;
          }
        }
      }
      done();
      if (part) {
#pragma unroll
        for (int i = 0; i < kM; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = key + 16 * i + g + 8 * (e >> 1), a = e & 1;
              if (at > pos[t][a] || (at < lo[t][a] && at >= p.sinks)) sc[i][t][e] = -INFINITY;
            }
      }
      // The running maximum moves when it grows by more than kLazy; a smaller
      // growth leaves weights of up to 2^kLazy, which the last division cancels.
      bool grown = false;
      float by[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          float mx = fmaxf(sc[0][t][a], sc[0][t][2 + a]);
#pragma unroll
          for (int i = 1; i < kM; ++i) mx = max3(mx, sc[i][t][a], sc[i][t][2 + a]);
#pragma unroll
          for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          by[t][a] = 1.f;
          if ((mx - m[t][a]) * qscale[t][a] > kLazy) {   // (false for -infinity less itself)
            by[t][a] = ex2((m[t][a] - mx) * qscale[t][a]);
            m[t][a] = mx;
            l[t][a] *= by[t][a];
            grown = true;
          }
        }
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            o[j][t][0] *= by[t][0], o[j][t][1] *= by[t][1], o[j][t][2] *= by[t][0], o[j][t][3] *= by[t][1];
      }
      mbar_wait(full + cslot * 8, cround & 1, abort_flag, kWaitNs);
      // Where some rows see a value and others do not, a weight of zero times an
      // infinity or a NaN would be NaN: such elements are added to the rows that
      // see them (weights are positive) and zeros in the product.
      if (part && s.n > 1) {
        const uint32_t at = base + cslot * C::kSlot + warp * kKeys * C::kWidth;
        const uint32_t by_key = scales + cslot * (C::kStep * 4);
        auto seen = [&](int k) { return k < s.end && (k >= cw.lo || k < cw.sinks_end); };
        constexpr int kPieces = C::kRow / 16;
        auto piece_at = [&](int x) {   // of 16 bytes; x / kPieces is the key
          const int row = x / kPieces, piece = x % kPieces;
          return at + (piece >> 3) * (C::kStep * 128) + row * C::kWidth + (piece & 7) * 16;
        };
        uint32_t odd = 0;
#pragma unroll 4
        for (int x = lane; x < kKeys * kPieces; x += 32)
          if (seen(key + x / kPieces)) odd |= odd_of<E8>(lds128(piece_at(x)));
        if constexpr (E8)
          for (int k = lane; k < kKeys; k += 32) odd |= seen(key + k) && odd_of(lds_f(by_key + k * 4));
        if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
          for (int k = 0; k < kKeys; ++k) {
            if (!seen(key + k)) continue;
            float scale = 1.f;
            if constexpr (E8) scale = lds_f(by_key + k * 4);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float v;
                if constexpr (E8) {
                  const int d = (D / 8) * g + 2 * j + e, piece = D == 128 ? (d >> 4) ^ (k & 7) : (d >> 4) ^ ((k >> 1) & 3);
                  const uint32_t two = f16x2_of_e4m3(lds_u8(at + k * C::kWidth + piece * 16 + (d & 15)));
                  v = __half2float(__ushort_as_half((unsigned short)two)) * scale;
                } else {
                  const int d = 16 * j + 8 * e + g;
                  v = __uint_as_float(lds_u16(at + (d >> 6) * (C::kStep * 128) + k * 128 + ((((d >> 3) & 7) ^ (k & 7)) << 4) + (d & 7) * 2) << 16);
                }
                if (odd_of(v))
#pragma unroll
                  for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int a = 0; a < 2; ++a)
                      if (key + k <= pos[t][a] && (key + k >= lo[t][a] || key + k < p.sinks)) o[j][t][2 * e + a] += v;
              }
          }
          __syncwarp();
          for (int x = lane; x < kKeys * kPieces; x += 32) sts128(piece_at(x), even_of<E8>(lds128(piece_at(x))));
          if constexpr (E8)
            for (int k = lane; k < kKeys; k += 32)
              if (odd_of(lds_f(by_key + k * 4))) sts_f(by_key + k * 4, 0.f);
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
      if constexpr (E8) {
        // Weights times the values' scales over sigma, the largest scale so
        // far: at most 2^(kLazy + 7) in f16.
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < kKeys / 32; ++e) {
          const int at = key + lane + 32 * e;
          if (at < s.end && (at >= cw.lo || at < cw.sinks_end))
            top = max(top, __float_as_uint(lds_f(scales + cslot * (C::kStep * 4) + (lane + 32 * e) * 4)) & 0x7fffffffu);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (__uint_as_float(top) > sigma * 128.f || sigma == 0.f) {
          const uint32_t exponent = min(max((top + 0x7fffffu) >> 23, 9u), 253u);
          const float to = __uint_as_float((exponent - 7u) << 23), less = sigma == 0.f ? 1.f : sigma / to;
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int t = 0; t < NT; ++t) o[j][t][0] *= less, o[j][t][1] *= less, o[j][t][2] *= less, o[j][t][3] *= less;
          sigma = to;
          sigma_inv = 1.f / to;
        }
      }
      uint32_t pf[kM][NT][2];
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v_scale = 1.f;
          if constexpr (E8) v_scale = lds_f(scales + cslot * (C::kStep * 4) + (16 * i + 8 * e + g) * 4) * sigma_inv;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            // (The difference first: a score's product with its factor, unrounded, less
            // the maximum's, rounded, is no small number where scores are huge.)
            const float down0 = m[t][0] == -INFINITY ? 0.f : m[t][0], down1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
            float w0 = ex2((sc[i][t][2 * e] - down0) * qscale[t][0]), w1 = ex2((sc[i][t][2 * e + 1] - down1) * qscale[t][1]);
            l[t][0] += w0, l[t][1] += w1;
            if constexpr (E8) {
              w0 = part && w0 == 0.f ? 0.f : w0 * v_scale;
              w1 = part && w1 == 0.f ? 0.f : w1 * v_scale;
              pf[i][t][e] = transposed(f16x2(w0, w1));
            } else {
              pf[i][t][e] = transposed(bf16x2(w0, w1));
            }
          }
        }
      {
        const uint32_t at = base + cslot * C::kSlot + warp * kKeys * C::kWidth;
        // Places that no row sees may hold NaN: their values count as zeros.
        auto seen = [&](int k) { return k < s.end && (k >= cw.lo || k < cw.sinks_end); };
#pragma unroll
        for (int i = 0; i < kM; ++i) {
          if constexpr (!E8) {
            const int row = 16 * i + (lane & 7) + (lane >> 4) * 8;
            uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
            if (part)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int k = key + 16 * i + 2 * c + 8 * e;
                keep[e] = (seen(k) ? 0xffffu : 0u) | (seen(k + 1) ? 0xffff0000u : 0u);
              }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              uint32_t v[4];
              const int piece16 = 2 * j + ((lane >> 3) & 1);
              ldsm4_t(at + (piece16 >> 3) * (C::kStep * 128) + row * 128 + (((piece16 & 7) ^ (row & 7)) << 4), v);
              if (part) v[0] &= keep[0], v[1] &= keep[0], v[2] &= keep[1], v[3] &= keep[1];
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816<false>(o[j][t], v, pf[i][t][0], pf[i][t][1]);
            }
          } else {
            // A thread's values of D: D / 8 neighbours for its g, two for each
            // product; keys 2 c, 2 c + 1, 2 c + 8 and 2 c + 9.
            constexpr int kWords = D / 32;
            uint32_t w[4][kWords];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int row = 16 * i + 2 * c + (e & 1) + (e >> 1) * 8;
              if constexpr (D == 128) {
                const uint4 v = lds128(at + row * 128 + ((g ^ (row & 7)) << 4));
                w[e][0] = v.x, w[e][1] = v.y, w[e][2] = v.z, w[e][3] = v.w;
              } else {
                const uint2 v = lds64(at + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
                w[e][0] = v.x, w[e][1] = v.y;
              }
              if (part && !seen(key + row))
#pragma unroll
                for (int k = 0; k < kWords; ++k) w[e][k] = 0;
            }
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
              const uint32_t a01 = __byte_perm(w[0][k], w[1][k], 0x5140), a23 = __byte_perm(w[0][k], w[1][k], 0x7362);
              const uint32_t b01 = __byte_perm(w[2][k], w[3][k], 0x5140), b23 = __byte_perm(w[2][k], w[3][k], 0x7362);
              const uint32_t x[4] = {f16x2_of_e4m3(a01), f16x2_of_e4m3_high(a01), f16x2_of_e4m3(b01), f16x2_of_e4m3_high(b01)};
              const uint32_t y[4] = {f16x2_of_e4m3(a23), f16x2_of_e4m3_high(a23), f16x2_of_e4m3(b23), f16x2_of_e4m3_high(b23)};
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                mma16816<true>(o[2 * k][t], x, pf[i][t][0], pf[i][t][1]);
                mma16816<true>(o[2 * k + 1][t], y, pf[i][t][0], pf[i][t][1]);
              }
            }
          }
        }
      }
      done();
    }
    x += here;
    cw.next(p);

    // ---- the warps' parts together, four rows of a warp at a time, and out
    auto part_of = [&](int block, bool first) { return p.part + ((long long)block * 2 + (first ? 1 : 0)) * C::kPart; };
    const int first = (int)(unit / piece), shares = (int)((unit + tiles - 1) / piece) - first + 1;
    float2* const stat = reinterpret_cast<float2*>(gbase + C::kOffStat);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int a = 0; a < 2; ++a) {
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[t][a] += __shfl_xor_sync(0xffffffffu, l[t][a], d);
        m[t][a] *= qscale[t][a];
        if (g == 0) stat[(warp * NT + t) * 8 + 2 * c + a] = make_float2(m[t][a], l[t][a]);
      }
    meet();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t > 0 && real <= 8 * t) break;   // (no rows)
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmaxf(top, stat[(k * NT + t) * 8 + 2 * c + a].x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = stat[(k * NT + t) * 8 + 2 * c + a];
          sum += ex2_below(v.x, top) * v.y;
        }
        const float by = ex2_below(m[t][a], top) * (E8 ? sigma : 1.f);
        // Where this thread's values of D lie.
        auto d_of = [&](int j, int e) { return E8 ? (D / 8) * g + 2 * j + e : 16 * j + 8 * e + g; };
        float* const buf = reinterpret_cast<float*>(gbase + C::kOffJoin);
        if (warp > 0) {
          float* const to = buf + (warp - 1) * 4 * C::kApart + c * C::kApart;
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) to[d_of(j, e)] = o[j][t][2 * e + a] * by;
        }
        meet();
        if (warp == 0) {
          float* const mine = buf;   // (the first other warp's)
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = o[j][t][2 * e + a] * by;
#pragma unroll
              for (int k = 1; k < 4; ++k) v += buf[(k - 1) * 4 * C::kApart + c * C::kApart + d_of(j, e)];
              mine[c * C::kApart + d_of(j, e)] = v;
            }
          __syncwarp();
          // Eight lanes a row.
          constexpr int kEach = D / 8;
          const int mine_row = lane >> 3, rho = t * 8 + 2 * mine_row + a;
          const float top_of = __shfl_sync(0xffffffffu, top, mine_row), sum_of = __shfl_sync(0xffffffffu, sum, mine_row);
          if (rho < real) {
            const float* const from = mine + mine_row * C::kApart + (lane & 7) * kEach;
            if (whole) {
              const int token = rho / p.group, head = h * p.group + rho - token * p.group;
              const float inv = top_of == -INFINITY ? 0.f : 1.f / sum_of;
              __nv_bfloat16* const to = p.o[r] + (long long)(s.row + token) * p.ld_o + head * D + (lane & 7) * kEach;
#pragma unroll
              for (int k = 0; k < kEach; k += 8) {
                const float4 u = *reinterpret_cast<const float4*>(from + k), v = *reinterpret_cast<const float4*>(from + k + 4);
                *reinterpret_cast<uint4*>(to + k) = make_uint4(bf16x2(u.x * inv, u.y * inv), bf16x2(u.z * inv, u.w * inv),
                                                               bf16x2(v.x * inv, v.y * inv), bf16x2(v.z * inv, v.w * inv));
              }
              if (p.lse[r] && (lane & 7) == 0) p.lse[r][(long long)(s.row + token) * p.heads_q + head] = lse_of(top_of, sum_of);
            } else {
              float* const to = part_of(blockIdx.x, (int)blockIdx.x == first);
#pragma unroll
              for (int k = 0; k < kEach; k += 4)
                *reinterpret_cast<float4*>(to + rho * D + (lane & 7) * kEach + k) = *reinterpret_cast<const float4*>(from + k);
              if ((lane & 7) == 0) to[C::kRows * D + rho] = top_of, to[C::kRows * (D + 1) + rho] = sum_of;
            }
          }
        }
        meet();
      }
    }
    if (whole) continue;

    // ---- a unit that other blocks share
    // Adds one to a counter; true for the last of n, which finds it at zero again.
    auto last_of = [&](uint32_t* counter, int n) {
      __threadfence();
      meet();
      if (tid == 0) {
        const bool is = fo::atom_add_acq_rel_u32(counter, 1u) == (uint32_t)n - 1u;
        if (is) *counter = 0u;
        misc[1] = is;
      }
      meet();
      const bool is = misc[1];
      if (is) __threadfence();
      return is;
    };
    // Parts of `n` blocks, `step` apart, together: a warp for a row.
    auto join = [&](int block, int step, int n, bool finish) {
      constexpr int kEach = D / 32;
      for (int rho = warp; rho < real; rho += 4) {
        float mi = -INFINITY, li = 0.f;
        if (lane < n) {
          const float* const from = part_of(block + lane * step, block + lane * step == first);
          mi = __ldcg(from + C::kRows * D + rho), li = __ldcg(from + C::kRows * (D + 1) + rho);
        }
        float top = mi;
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float fi = lane < n ? ex2_below(mi, top) : 0.f, sum = warp_sum(fi * li);
        float acc[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) acc[e] = 0.f;
        for (int k0 = 0; k0 < n; k0 += 8) {
          float v[8][kEach];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (k0 + k >= n) break;
            const int from_block = block + (k0 + k) * step;
            const float* const from = part_of(from_block, from_block == first) + rho * D + lane * kEach;
            if constexpr (kEach == 4) {
              const float4 f = __ldcg(reinterpret_cast<const float4*>(from));
              v[k][0] = f.x, v[k][1] = f.y, v[k][2] = f.z, v[k][3] = f.w;
            } else {
              const float2 f = __ldcg(reinterpret_cast<const float2*>(from));
              v[k][0] = f.x, v[k][1] = f.y;
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (k0 + k >= n) break;
            const float f = __shfl_sync(0xffffffffu, fi, k0 + k);
#pragma unroll
            for (int e = 0; e < kEach; ++e) acc[e] = fmaf(f, v[k][e], acc[e]);
          }
        }
        if (finish) {
          const int token = rho / p.group, head = h * p.group + rho - token * p.group;
          const float by = top == -INFINITY ? 0.f : 1.f / sum;
          __nv_bfloat16* const to = p.o[r] + (long long)(s.row + token) * p.ld_o + head * D + lane * kEach;
          if constexpr (kEach == 4)
            *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2(acc[0] * by, acc[1] * by), bf16x2(acc[2] * by, acc[3] * by));
          else
            *reinterpret_cast<uint32_t*>(to) = bf16x2(acc[0] * by, acc[1] * by);
          if (p.lse[r] && lane == 0) p.lse[r][(long long)(s.row + token) * p.heads_q + head] = lse_of(top, sum);
        } else {
          float* const to = part_of(block, block == first);
#pragma unroll
          for (int e = 0; e < kEach; ++e) to[rho * D + lane * kEach + e] = acc[e];
          if (lane == 0) to[C::kRows * D + rho] = top, to[C::kRows * (D + 1) + rho] = sum;
        }
      }
    };
    const int set = ((int)blockIdx.x - first) / kRadix, lead = first + set * kRadix, members = min(kRadix, shares - set * kRadix);
    if (last_of(p.count + lead * 3 + (set == 0 ? 1 : 0), members)) {
      join(lead, 1, members, shares <= kRadix);
      if (shares > kRadix) {
        const int sets = (shares + kRadix - 1) / kRadix;
        if (last_of(p.count + first * 3 + 2, sets)) join(first, kRadix, sets, true);
      }
    }
    meet();
  }
  if (tid == 0 && *abort_flag) fo::record_error(p.batch.status, FO_ERR_TIMEOUT, -1, -1, 0);
}

template <int D, bool E8, int NT>
fo_status launch(FewParams& k, int sms, cudaStream_t s) {
  using C = Few<D, E8, NT>;
  auto kern = few_kernel<D, E8, NT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return launched(e, "paged attention", k.R, k.batch.rows, D, 0, kFewThreads);
  const int blocks = std::min(sms, FO_GB300_SMS) * kFewBlocks;
  return launched(launch_after(kern, dim3(blocks), kFewThreads, C::kSmem, 0, s, k), "paged attention", k.R, k.batch.rows, D, blocks,
                  kFewThreads);
}
template <int D>
fo_status launch_for(FewParams& k, bool wide, bool eight, int sms, cudaStream_t s) {
  if (eight) return wide ? launch<D, true, 2>(k, sms, s) : launch<D, true, 1>(k, sms, s);
  return wide ? launch<D, false, 2>(k, sms, s) : launch<D, false, 1>(k, sms, s);
}

}  // namespace

fo_status attend_few(FewParams& k, int D, bool wide, bool eight, int sms, cudaStream_t s) {
  return D == 128 ? launch_for<128>(k, wide, eight, sms, s) : launch_for<64>(k, wide, eight, sms, s);
}

}  // namespace fo_ops
