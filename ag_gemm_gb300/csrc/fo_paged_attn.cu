// Attention of a batch's new tokens over a paged cache of keys and values.
#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "fo_paged.h"
#include "fo_paged_tiles.cuh"

namespace fo_ops {
namespace {

using namespace fo;

// ---- few new tokens a sequence: the cache's length is split
//
// Reading the visible keys and values once is what a call cannot do without:
// 4 D flops for 4 D bytes (bf16), times the query heads that share a key head.
// So a unit of work is a sequence's key head with all rows (new tokens x heads
// of the group) that read it, up to 64 of them, as the 16-row operand of
// mma.sync; tcgen05 takes 128 rows, and the 8 to 16 that a decode step has
// leave even this path's rate (a quarter of tcgen05's) 85% idle.
//
// The tiles of all units (kStep keys, the visible ones alone) form one line, in
// the order sequence, rank, head, tile; the line is cut into equal pieces, one
// for each of two blocks an SM, so that every SM reads the same bytes whatever
// the lengths. A block finds its piece from the lengths on the device: a captured call may
// be replayed with other ones. In a block, each of four warps takes 32 of a
// tile's keys (64 in 8 bits) (with more than 16 rows, two or four warps share the keys and
// part the rows), has TMA bring them into a ring of its own, and keeps its own
// maximum, sum and output in registers: no barrier in the stream of tiles. At
// a unit's end, or the piece's, the warps' parts are joined through shared
// memory. A unit cut between blocks is joined by the last of them to arrive,
// the parts in the blocks' order (16 at a time), so results repeat.

constexpr int kFewThreads = 128;
constexpr int kRadix = 16;             // parts joined at a time
constexpr int kPerSm = 2;              // blocks

struct FewParams {
  CUtensorMap k[kMaxR];   // [pages * heads_k][page][D]; boxes of 128 bytes x `box` tokens
  CUtensorMap v[kMaxR];
  const float* ks[kMaxR];
  const float* vs[kMaxR];
  const __nv_bfloat16* q[kMaxR];
  __nv_bfloat16* o[kMaxR];
  float* lse[kMaxR];
  int64_t ld_q, ld_o;
  Batch batch;
  int32_t R, heads_q, heads_k, group, window, sinks;
  int32_t box;            // tokens of a box: a page's, or a warp's tile's
  int32_t boxes_log2;     // of a warp's tile
  int32_t least;          // tiles of a piece, at least
  float scale_log2;
  float* part;            // [blocks][2][rows * (D + 2)]
  uint32_t* count;        // [blocks][3], zero between calls
};

template <int D, bool E8, int MT>
struct Few {
  static constexpr int kKeys = E8 ? 64 : 32;                // a warp's keys of a tile
  static constexpr int kRow = D * (E8 ? 1 : 2);             // bytes of a key
  static constexpr int kWidth = kRow < 128 ? kRow : 128;    // of a box
  static constexpr int kCuts = kRow / kWidth;
  static constexpr int kSlot = kKeys * kRow;
  static constexpr int kRing = 24576;                       // bytes of a warp
  static constexpr int kGroups = 4 / MT;                    // warps with keys of their own
  static constexpr int kStep = kKeys * kGroups;             // keys of a tile
  static constexpr int kSlots = kRing * MT / kSlot;
  // Warps that share keys: a slot is filled again this much later than it is
  // read, so that the one that loads need not wait for the others.
  static constexpr int kLag = MT > 1 ? 2 : 0;
  static constexpr int kRows = 16 * MT;
  static constexpr int kPart = kRows * (D + 2);             // floats of a part: output, maxima, sums
  // Shared memory: rings, scales, rows being joined, (m, l) of each warp, barriers.
  static constexpr int kOffScale = 4 * kRing;
  static constexpr int kOffJoin = kOffScale + (E8 ? kGroups * kSlots * kKeys * 4 : 0);
  static constexpr int kOffStat = kOffJoin + (4 - MT) * 8 * D * 4;
  static constexpr int kOffBar = kOffStat + 4 * 16 * 8;
  static constexpr int kOffMisc = kOffBar + 2 * kGroups * kSlots * 8;
  static constexpr int kSmem = 1024 + kOffMisc + 64;
  static_assert(kPerSm * (kSmem + 1024) <= 233472, "blocks an SM");
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

template <int D, bool E8, int MT>
__global__ void __launch_bounds__(kFewThreads, kPerSm) few_kernel(const __grid_constant__ FewParams p) {
  using C = Few<D, E8, MT>;
  constexpr int kKeys = C::kKeys;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int kg = warp / MT, mt = warp % MT;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbase + C::kOffMisc);
  int* const misc = reinterpret_cast<int*>(gbase + C::kOffMisc);   // [0] abort, [1] flag, [2] sequence, [4..5] its first tile
  const uint32_t full = base + C::kOffBar + kg * C::kSlots * 8, empty = full + C::kGroups * C::kSlots * 8;
  const uint32_t ring = base + kg * (C::kRing * MT), scales = base + C::kOffScale + kg * C::kSlots * kKeys * 4;
  if (tid == 0) {
    for (int i = 0; i < C::kGroups * C::kSlots; ++i) {
      mbar_init(base + C::kOffBar + i * 8, 1);
      mbar_init(base + C::kOffBar + (C::kGroups * C::kSlots + i) * 8, MT);
    }
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
    const int run = (p.batch.seqs + kFewThreads - 1) / kFewThreads, first = tid * run, last = min(first + run, p.batch.seqs);
    long long mine = 0;
    for (cw.b = first; cw.b < last; ++cw.b) cw.of(p.batch, p.window, p.sinks), mine += (long long)cw.tiles * units;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    long long* const sums = reinterpret_cast<long long*>(gbase + C::kOffStat);
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    total = 0;
    for (int w = 0; w < 4; ++w) {
      if (w < warp) upto += sums[w];
      total += sums[w];
    }
    piece = max((total + gridDim.x - 1) / gridDim.x, (long long)p.least);
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

  // ---- loads: by the first warp of those that share keys
  Walk<C::kStep> pw = cw;
  long long pleft = x1 - x0;
  int pslot = 0, pround = 0, page_b = -1, page_t = 0, page_of = -1;
  bool value = false;   // the next load is of values
  auto seek = [&]() {
    while (pleft > 0 && !pw.any(pw.first_key() + kg * kKeys, kKeys)) pw.next(p), --pleft;
  };
  auto issue = [&]() {
    if (pleft <= 0) return;
    if (!value && (pw.b != page_b || (uint32_t)(pw.t - page_t) >= 32u >> p.boxes_log2)) {
      // Page numbers of the next tiles, a lane for a box.
      page_b = pw.b;
      page_t = pw.t;
      page_of = -1;
      const int t = pw.t + (lane >> p.boxes_log2);
      const int key = (t < pw.early ? t : t - pw.early + pw.late) * C::kStep + kg * kKeys + (lane & ((1 << p.boxes_log2) - 1)) * p.box;
      if (t < pw.tiles && pw.any(key, p.box)) {
        const int id = p.batch.table[(long long)pw.b * p.batch.cols + (key >> p.batch.shift)];
        if (id < 0 || id >= p.batch.pages) report(p.batch, pw.b, kBadPage, id);
        else page_of = id;
      }
    }
    // Lane i < boxes: box i.
    const int id = __shfl_sync(0xffffffffu, page_of, (((pw.t - page_t) << p.boxes_log2) + lane) & 31);
    if (MT > 1 && pround > 0) mbar_wait(empty + pslot * 8, (pround - 1) & 1, abort_flag, kWaitNs);
    const uint32_t bar = full + pslot * 8;
    const bool mine = lane < 1 << p.boxes_log2;
    uint32_t bytes = C::kSlot;
    if constexpr (E8) bytes += __popc(__ballot_sync(0xffffffffu, mine && id >= 0)) * p.box * 4;
    if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
    __syncwarp();
    if (mine) {
      // What no page holds is read from behind the last one: zeros.
      const int z = id >= 0 ? id * p.heads_k + pw.h : p.batch.pages * p.heads_k;
      const int y = (pw.first_key() + kg * kKeys + lane * p.box) & ((1 << p.batch.shift) - 1);
      const CUtensorMap* const map = value ? &p.v[pw.r] : &p.k[pw.r];
#pragma unroll
      for (int cut = 0; cut < C::kCuts; ++cut)
        tma_load_3d(ring + pslot * C::kSlot + cut * kKeys * 128 + lane * p.box * C::kWidth, map, bar, cut * 64, y, z);
      if constexpr (E8)
        if (id >= 0)
          bulk_load(scales + (pslot * kKeys + lane * p.box) * 4, (value ? p.vs[pw.r] : p.ks[pw.r]) + ((long long)z << p.batch.shift) + y,
                    p.box * 4, bar);
    }
    if (value) pw.next(p), --pleft, seek();
    value = !value;
    if (++pslot == C::kSlots) pslot = 0, ++pround;
  };
  int cslot = 0, cround = 0;
  // The slot that has been read is free again.
  auto done = [&]() {
    __syncwarp();
    if (MT > 1 && lane == 0) mbar_arrive(empty + cslot * 8);
    if (++cslot == C::kSlots) cslot = 0, ++cround;
    if (mt == 0) issue();
  };
  if (mt == 0) {
    seek();
    for (int i = 0; i < C::kSlots - C::kLag; ++i) issue();
  }

  for (long long x = x0; x < x1;) {
    // ---- a unit, or what of it is in this piece
    const int here = (int)min((long long)(cw.tiles - cw.t), x1 - x);
    const long long unit = x - cw.t;
    const bool whole = here == cw.tiles;
    const int tiles = cw.tiles, r = cw.r, h = cw.h, real = cw.s.n * p.group;
    const Seq s = cw.s;
    int row[2], pos[2], lo[2];
    uint32_t qf[D / 16][4];
    float qscale[2] = {p.scale_log2, p.scale_log2};   // with what the scores are to be multiplied
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rho = mt * 16 + g + 8 * i, token = rho / p.group, head = rho - token * p.group;
      const bool is = rho < real;
      row[i] = is ? s.row + token : -1;
      pos[i] = is ? s.base + token : -1;
      lo[i] = sight_of(max(pos[i], 0), p.window, p.sinks).lo;
      const __nv_bfloat16* const q = p.q[r] + (long long)max(row[i], 0) * p.ld_q + (h * p.group + head) * D;
      if constexpr (!E8) {
        // Elements in the order that 16-byte pieces of a key give them.
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (is) v = *reinterpret_cast<const uint4*>(q + (k >> 1) * 64 + (2 * c + (k & 1)) * 8);
          qf[2 * k][i] = v.x, qf[2 * k][2 + i] = v.y, qf[2 * k + 1][i] = v.z, qf[2 * k + 1][2 + i] = v.w;
        }
      } else {
        // In f16, which e4m3 values are exactly: the row times a power of two
        // that brings its largest magnitude to [128, 256). What that makes
        // smaller than f16's least normal number is 2^-21 of the largest.
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
        const uint32_t exponent = min(max(__float_as_uint(top) >> 23, 8u), 254u);
        const float by = top <= 3.4e38f ? __uint_as_float((261u - exponent) << 23) : 1.f;
        qscale[i] *= 1.f / by;
#pragma unroll
        for (int k = 0; k < kEach / 4; ++k) {
          const uint32_t w0 = (k & 1) ? v[k / 2].z : v[k / 2].x, w1 = (k & 1) ? v[k / 2].w : v[k / 2].y;
          const float f0 = __uint_as_float(w0 << 16) * by, f1 = __uint_as_float(w0 & 0xffff0000u) * by;
          const float f2 = __uint_as_float(w1 << 16) * by, f3 = __uint_as_float(w1 & 0xffff0000u) * by;
          qf[k][i] = f16x2(f0, f1), qf[k][2 + i] = f16x2(f2, f3);
        }
      }
    }
    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float sigma = 0.f, sigma_inv = 0.f;   // what the values' scales are divided by (a power of two), and its reciprocal
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    const int lo_last = sight_of(max(s.base + s.n - 1, 0), p.window, p.sinks).lo;

    for (int i = 0; i < here; ++i, cw.t += i < here ? 1 : 0) {
      const int key = cw.first_key() + kg * kKeys;
      if (!cw.any(key, kKeys)) continue;
      // All of a tile's keys seen by all rows?
      const bool part = !(key + kKeys - 1 <= s.base && (key >= lo_last || key + kKeys <= p.sinks));
      constexpr int kJ = kKeys / 8;   // eights of keys
      float sc[kJ][4];
#pragma unroll
      for (int j = 0; j < kJ; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
      mbar_wait(full + cslot * 8, cround & 1, abort_flag, kWaitNs);
      {
        const uint32_t at = ring + cslot * C::kSlot;
        if constexpr (!E8) {
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint4 v[kJ];
#pragma unroll
            for (int j = 0; j < kJ; ++j)
              v[j] = lds128(at + (k >> 1) * (kKeys * 128) + (8 * j + g) * 128 + (((2 * c + (k & 1)) ^ g) << 4));
            // (Four sums in turn: one after the other they would wait for each product.)
#pragma unroll
            for (int j = 0; j < kJ; ++j) mma16816<false>(sc[j], qf[2 * k], v[j].x, v[j].y);
#pragma unroll
            for (int j = 0; j < kJ; ++j) mma16816<false>(sc[j], qf[2 * k + 1], v[j].z, v[j].w);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kJ / 4 * (D / 64); ++k) {
            const int j0 = k / (D / 64) * 4, half = k % (D / 64);
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int n = 8 * (j0 + j) + g;
              v[j] = lds128(D == 128 ? at + n * 128 + (((2 * c + half) ^ g) << 4) : at + n * 64 + ((c ^ ((n >> 1) & 3)) << 4));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t w = e == 0 ? v[j].x : e == 1 ? v[j].y : e == 2 ? v[j].z : v[j].w;
                mma16816<true>(sc[j0 + j], qf[4 * half + e], f16x2_of_e4m3(w), f16x2_of_e4m3_high(w));
              }
            }
          }
        }
        if constexpr (E8) {
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            const uint2 k2 = lds64(scales + cslot * (kKeys * 4) + (8 * j + 2 * c) * 4);
            const float k0 = __uint_as_float(k2.x), k1 = __uint_as_float(k2.y);
            sc[j][0] *= k0, sc[j][1] *= k1, sc[j][2] *= k0, sc[j][3] *= k1;
          }
        }
      }
      done();
      if (part) {
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = key + 8 * j + 2 * c + (e & 1), a = e >> 1;
            if (at > pos[a] || (at < lo[a] && at >= p.sinks)) sc[j][e] = -INFINITY;
          }
      }
      // The running maximum moves when it grows by more than kLazy; a smaller
      // growth leaves weights of up to 2^kLazy, which the last division cancels.
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        float mx = fmaxf(sc[0][2 * a], sc[0][2 * a + 1]);
#pragma unroll
        for (int j = 1; j < kJ; ++j) mx = fmaxf(mx, fmaxf(sc[j][2 * a], sc[j][2 * a + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * qscale[a];
        const bool grows = mx > m[a] + kLazy || (m[a] == -INFINITY && mx > m[a]);
        if (__any_sync(0xffffffffu, grows)) {
          const float to = grows ? mx : m[a], by = grows ? ex2_below(m[a], to) : 1.f;
          m[a] = to;
          l[a] *= by;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) o[j][2 * a] *= by, o[j][2 * a + 1] *= by;
        }
      }
      uint32_t pf[kJ / 2][4];
      mbar_wait(full + cslot * 8, cround & 1, abort_flag, kWaitNs);
      if constexpr (E8) {
        // Weights times the values' scales over sigma, the largest scale so
        // far: at most 2^(kLazy + 7) in f16.
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < kKeys / 32; ++e) {
          const int at = key + lane + 32 * e;
          if (at < s.end && (at >= cw.lo || at < cw.sinks_end))
            top = max(top, __float_as_uint(lds_f(scales + cslot * (kKeys * 4) + (lane + 32 * e) * 4)) & 0x7fffffffu);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (__uint_as_float(top) > sigma * 128.f || sigma == 0.f) {
          const uint32_t exponent = min(max((top + 0x7fffffu) >> 23, 9u), 253u);
          const float to = __uint_as_float((exponent - 7u) << 23), by = sigma == 0.f ? 0.f : sigma / to;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) o[j][0] *= by, o[j][1] *= by, o[j][2] *= by, o[j][3] *= by;
          sigma = to;
          sigma_inv = 1.f / to;
        }
      }
      const float down[2] = {m[0] == -INFINITY ? 0.f : -m[0], m[1] == -INFINITY ? 0.f : -m[1]};
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        float2 by = make_float2(1.f, 1.f);
        if constexpr (E8) {
          const uint2 v2 = lds64(scales + cslot * (kKeys * 4) + (8 * j + 2 * c) * 4);
          by = make_float2(__uint_as_float(v2.x) * sigma_inv, __uint_as_float(v2.y) * sigma_inv);
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          float w0 = ex2(fmaf(sc[j][2 * a], qscale[a], down[a])), w1 = ex2(fmaf(sc[j][2 * a + 1], qscale[a], down[a]));
          l[a] += w0 + w1;
          if constexpr (E8) {
            w0 = part && w0 == 0.f ? 0.f : w0 * by.x;
            w1 = part && w1 == 0.f ? 0.f : w1 * by.y;
            pf[j >> 1][(j & 1) * 2 + a] = f16x2(w0, w1);
          } else {
            pf[j >> 1][(j & 1) * 2 + a] = bf16x2(w0, w1);
          }
        }
      }
      {
        const uint32_t at = ring + cslot * C::kSlot;
        // Places that no row sees may hold NaN: their values count as zeros.
        auto seen = [&](int k) { return k < s.end && (k >= cw.lo || k < cw.sinks_end); };
#pragma unroll
        for (int kk = 0; kk < kJ / 2; ++kk) {
          if constexpr (!E8) {
            const int n = kk * 16 + (lane & 15);
            uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
            if (part)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int k = key + kk * 16 + 2 * c + 8 * e;
                keep[e] = (seen(k) ? 0xffffu : 0u) | (seen(k + 1) ? 0xffff0000u : 0u);
              }
#pragma unroll
            for (int j = 0; j < D / 8; j += 2) {
              uint32_t v[4];
              const int piece16 = j + (lane >> 4);
              ldsm4_t(at + (piece16 >> 3) * (kKeys * 128) + n * 128 + (((piece16 & 7) ^ (n & 7)) << 4), v);
              if (part) v[0] &= keep[0], v[1] &= keep[1], v[2] &= keep[0], v[3] &= keep[1];
              mma16816<false>(o[j], pf[kk], v[0], v[1]);
              mma16816<false>(o[j + 1], pf[kk], v[2], v[3]);
            }
          } else {
            // A thread's columns: D / 8 neighbours for its g, one for each
            // product; keys 2 c, 2 c + 1, 2 c + 8 and 2 c + 9.
            constexpr int kWords = D / 32;
            uint32_t w[4][kWords];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int n = kk * 16 + 2 * c + (e & 1) + (e >> 1) * 8;
              if constexpr (D == 128) {
                const uint4 v = lds128(at + n * 128 + ((g ^ (n & 7)) << 4));
                w[e][0] = v.x, w[e][1] = v.y, w[e][2] = v.z, w[e][3] = v.w;
              } else {
                const uint2 v = lds64(at + n * 64 + (((g >> 1) ^ ((n >> 1) & 3)) << 4) + (g & 1) * 8);
                w[e][0] = v.x, w[e][1] = v.y;
              }
              if (part && !seen(key + n))
#pragma unroll
                for (int i2 = 0; i2 < kWords; ++i2) w[e][i2] = 0;
            }
#pragma unroll
            for (int i2 = 0; i2 < kWords; ++i2) {
              const uint32_t a01 = __byte_perm(w[0][i2], w[1][i2], 0x5140), a23 = __byte_perm(w[0][i2], w[1][i2], 0x7362);
              const uint32_t b01 = __byte_perm(w[2][i2], w[3][i2], 0x5140), b23 = __byte_perm(w[2][i2], w[3][i2], 0x7362);
              mma16816<true>(o[4 * i2], pf[kk], f16x2_of_e4m3(a01), f16x2_of_e4m3(b01));
              mma16816<true>(o[4 * i2 + 1], pf[kk], f16x2_of_e4m3_high(a01), f16x2_of_e4m3_high(b01));
              mma16816<true>(o[4 * i2 + 2], pf[kk], f16x2_of_e4m3(a23), f16x2_of_e4m3(b23));
              mma16816<true>(o[4 * i2 + 3], pf[kk], f16x2_of_e4m3_high(a23), f16x2_of_e4m3_high(b23));
            }
          }
        }
      }
      done();
    }
    x += here;
    cw.next(p);

    // ---- the warps' parts together
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      l[a] += __shfl_xor_sync(0xffffffffu, l[a], 1);
      l[a] += __shfl_xor_sync(0xffffffffu, l[a], 2);
    }
    const float own = E8 ? sigma : 1.f;
    if constexpr (C::kGroups > 1) {
      float2* const stat = reinterpret_cast<float2*>(gbase + C::kOffStat);
      float* const buf = reinterpret_cast<float*>(gbase + C::kOffJoin);
      if (c == 0) stat[warp * 16 + g] = make_float2(m[0], l[0]), stat[warp * 16 + g + 8] = make_float2(m[1], l[1]);
      __syncthreads();
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        if (MT == 1 && a == 1 && real <= 8) break;   // (the second half's rows are none)
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < C::kGroups; ++k) top = fmaxf(top, stat[(k * MT + mt) * 16 + g + 8 * a].x);
#pragma unroll
        for (int k = 0; k < C::kGroups; ++k) {
          const float2 v = stat[(k * MT + mt) * 16 + g + 8 * a];
          sum += ex2_below(v.x, top) * v.y;
        }
        const float by = ex2_below(m[a], top) * own;
        m[a] = top;
        l[a] = sum;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][2 * a] *= by, o[j][2 * a + 1] *= by;
        if (kg > 0) {
          float2* const to = reinterpret_cast<float2*>(buf + ((kg - 1) * MT + mt) * 8 * D) + lane;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) to[j * 32] = make_float2(o[j][2 * a], o[j][2 * a + 1]);
        }
        __syncthreads();
        if (kg == 0) {
#pragma unroll
          for (int k = 1; k < C::kGroups; ++k) {
            const float2* const from = reinterpret_cast<const float2*>(buf + ((k - 1) * MT + mt) * 8 * D) + lane;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
              const float2 v = from[j * 32];
              o[j][2 * a] += v.x, o[j][2 * a + 1] += v.y;
            }
          }
        }
        __syncthreads();
      }
    } else if (E8) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j) o[j][0] *= own, o[j][1] *= own, o[j][2] *= own, o[j][3] *= own;
    }

    if (whole) {
      if (kg == 0) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          if (row[a] < 0) continue;
          const int rho = mt * 16 + g + 8 * a, head = h * p.group + rho % p.group;
          const float by = m[a] == -INFINITY ? 0.f : 1.f / l[a];
          __nv_bfloat16* const to = p.o[r] + (long long)row[a] * p.ld_o + head * D;
          if constexpr (!E8) {
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
              *reinterpret_cast<uint32_t*>(to + 8 * j + 2 * c) = bf16x2(o[j][2 * a] * by, o[j][2 * a + 1] * by);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < D / 8; j += 8) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = bf16x2(o[j + 2 * i][2 * a + e] * by, o[j + 2 * i + 1][2 * a + e] * by);
                *reinterpret_cast<uint4*>(to + (D / 8) * (2 * c + e) + j) = make_uint4(w[0], w[1], w[2], w[3]);
              }
          }
          if (p.lse[r] && c == 0) p.lse[r][(long long)row[a] * p.heads_q + head] = lse_of(m[a], l[a]);
        }
      }
      continue;
    }

    // ---- a unit that other blocks share
    auto part_of = [&](int block, bool first) { return p.part + ((long long)block * 2 + (first ? 1 : 0)) * C::kPart; };
    const int first = (int)(unit / piece), shares = (int)((unit + tiles - 1) / piece) - first + 1;
    if (kg == 0) {
      float* const to = part_of(blockIdx.x, (int)blockIdx.x == first);
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int rho = mt * 16 + g + 8 * a;
        if (rho >= real) continue;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          if constexpr (!E8)
            *reinterpret_cast<float2*>(to + rho * D + 8 * j + 2 * c) = make_float2(o[j][2 * a], o[j][2 * a + 1]);
          else
#pragma unroll
            for (int e = 0; e < 2; ++e) to[rho * D + (D / 8) * (2 * c + e) + j] = o[j][2 * a + e];
        }
        if (c == 0) to[C::kRows * D + rho] = m[a], to[C::kRows * (D + 1) + rho] = l[a];
      }
    }
    // Adds one to a counter; true for the last of n, which finds it at zero again.
    auto last_of = [&](uint32_t* counter, int n) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const bool is = fo::atom_add_acq_rel_u32(counter, 1u) == (uint32_t)n - 1u;
        if (is) *counter = 0u;
        misc[1] = is;
      }
      __syncthreads();
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
    __syncthreads();
  }
  if (tid == 0 && *abort_flag && p.batch.status) fo::record_error(p.batch.status, FO_ERR_TIMEOUT, -1, -1, 0);
}

// Rows of a unit that the split kernel takes: 16 a warp, four warps.
constexpr int kFewRows = 64;
constexpr int kMostBlocks = kPerSm * FO_GB300_SMS;
constexpr size_t kCountBytes = (kMostBlocks * 3 * 4 + 255) / 256 * 256;
int row_tiles(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }
size_t few_bytes(const fo_paged_desc* d, int64_t rows) {
  return 256 + kCountBytes + (size_t)kMostBlocks * 2 * 16 * row_tiles(rows) * (d->head_dim + 2) * 4;
}

template <int D, bool E8, int MT>
fo_status launch_few(FewParams& k, int sms, cudaStream_t s) {
  auto kern = few_kernel<D, E8, MT>;
  constexpr int smem = Few<D, E8, MT>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return launched(e, "paged attention", k.R, k.batch.rows, D, 0, kFewThreads);
  const int blocks = std::min(sms, FO_GB300_SMS) * kPerSm;
  return launched(launch_after(kern, dim3(blocks), kFewThreads, smem, 0, s, k), "paged attention", k.R, k.batch.rows, D, blocks,
                  kFewThreads);
}
template <int D, bool E8>
fo_status launch_few(FewParams& k, int mt, int sms, cudaStream_t s) {
  return mt == 1 ? launch_few<D, E8, 1>(k, sms, s) : mt == 2 ? launch_few<D, E8, 2>(k, sms, s) : launch_few<D, E8, 4>(k, sms, s);
}

}  // namespace
}  // namespace fo_ops

extern "C" fo_status fo_paged_attention_workspace(const fo_paged_desc* d, int32_t seqs, int64_t rows, int32_t max_new,
                                                  size_t* bytes) {
  const fo_status st = fo_ops::check_paged(d);
  if (st) return st;
  if (!bytes) return FO_ERR_INVALID_ARG;
  if (seqs < 0 || rows < 0 || rows > INT32_MAX || max_new < 1) return FO_ERR_SHAPE;
  const int64_t most = (int64_t)max_new * (d->heads_q / d->heads_k);
  *bytes = fo_ops::few_bytes(d, most < fo_ops::kFewRows ? most : fo_ops::kFewRows);
  if (most > fo_ops::kFewRows) *bytes = std::max(*bytes, fo_ops::prompt_bytes(seqs));
  return FO_OK;
}

extern "C" fo_status fo_paged_attention(const fo_paged_desc* d, const fo_paged_batch* b, int64_t rows, const void* const* q,
                                        const int64_t ld[2], const void* const* k_cache, const void* const* v_cache,
                                        const float* const* k_scale, const float* const* v_scale, void* const* o,
                                        float* const* lse, void* ws, fo_stream_t stream) {
  using namespace fo_ops;
  fo_status st = check_paged(d);
  if (st || (st = check_batch(d, b, rows))) return st;
  if (!ld || !ws) return FO_ERR_INVALID_ARG;
  const bool eight = d->cache_dtype == FO_CACHE_E4M3;
  if (!eight && (k_scale || v_scale)) return FO_ERR_INVALID_ARG;
  const int64_t wide = (int64_t)d->heads_q * d->head_dim;
  if (ld[0] < wide || ld[1] < wide) return FO_ERR_SHAPE;
  if (ld[0] % 8 || ld[1] % 8 || !aligned(ws, 16)) return FO_ERR_ALIGN;
  if (rows == 0 || b->seqs == 0) return FO_OK;
  typedef const void* const* A;
  const int R = d->R;
  if ((st = check_array(R, q, 16)) || (st = check_array(R, (A)o, 16)) || (st = check_array(R, k_cache, 16)) ||
      (st = check_array(R, v_cache, 16)) || (lse && (st = check_array(R, (A)lse, 4))))
    return st;
  if (eight && ((st = check_array(R, (A)k_scale, 16)) || (st = check_array(R, (A)v_scale, 16)))) return st;
  int sms;
  if ((st = device_sms(&sms))) return st;
  PtrList l;
  l.add(R, q), l.add(R, (A)o), l.add(R, k_cache), l.add(R, v_cache), l.add(R, (A)lse);
  if (eight) l.add(R, (A)k_scale), l.add(R, (A)v_scale);
  l.add(b->lengths), l.add(b->starts), l.add(b->table), l.add(ws);
  if ((st = check_device(l, stream))) return st;
  const float scale = d->scale > 0.f ? d->scale : (float)(1.0 / sqrt((double)d->head_dim));
  const int64_t unit_rows = (int64_t)b->max_new * (d->heads_q / d->heads_k);
  if (unit_rows <= kFewRows) {
    FewParams f;
    memset(static_cast<void*>(&f), 0, sizeof(f));
    const int keys = eight ? Few<128, true, 1>::kKeys : Few<128, false, 1>::kKeys;
    f.box = std::min(d->page, keys);
    for (f.boxes_log2 = 0; f.box << f.boxes_log2 < keys; ++f.boxes_log2) {
    }
    for (int r = 0; r < R; ++r) {
      if (!encode_pages(&f.k[r], k_cache[r], d, b->pages, f.box) || !encode_pages(&f.v[r], v_cache[r], d, b->pages, f.box)) return FO_ERR_CUDA;
      f.ks[r] = eight ? k_scale[r] : nullptr;
      f.vs[r] = eight ? v_scale[r] : nullptr;
      f.q[r] = static_cast<const __nv_bfloat16*>(q[r]);
      f.o[r] = static_cast<__nv_bfloat16*>(o[r]);
      f.lse[r] = lse ? lse[r] : nullptr;
    }
    f.ld_q = ld[0];
    f.ld_o = ld[1];
    f.batch = batch_of(d, b, rows, ws);
    f.R = R;
    f.heads_q = d->heads_q;
    f.heads_k = d->heads_k;
    f.group = d->heads_q / d->heads_k;
    f.window = d->window;
    f.sinks = d->sinks;
    f.least = 1;
    f.scale_log2 = scale * 1.4426950408889634f;
    f.count = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + 256);
    f.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256 + kCountBytes);
    const int mt = row_tiles(unit_rows);
    const cudaStream_t s = (cudaStream_t)stream;
    if (d->head_dim == 128) return eight ? launch_few<128, true>(f, mt, sms, s) : launch_few<128, false>(f, mt, sms, s);
    return eight ? launch_few<64, true>(f, mt, sms, s) : launch_few<64, false>(f, mt, sms, s);
  }
  PagedCall c;
  c.d = d, c.b = b, c.rows = rows, c.ld = ld;
  c.q = q, c.k = k_cache, c.v = v_cache, c.ks = k_scale, c.vs = v_scale, c.o = o, c.lse = lse;
  c.ws = static_cast<uint8_t*>(ws);
  c.scale_log2 = scale * 1.4426950408889634f;
  c.sms = sms;
  return attend_prompts(c, (cudaStream_t)stream);
}
