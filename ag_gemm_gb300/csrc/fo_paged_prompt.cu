// Attention of prompts over a paged cache: many new tokens a sequence, on
// tcgen05.
//
// The rows that read a key head are its group's heads of every new token,
// tokens outermost; 128 of them (as many whole tokens as fit) are a tile, and
// a block works on two tiles at a time over the same keys and values, 128 a
// step. While the tensor core sums one tile's weights times values and
// computes its next scores (1024 cycles of bf16 at D = 128), the other tile's
// softmax runs; a thread has a row of its own, so no row needs another
// thread. Per step and tile:
//     S = Q K^T        in TMEM, 128 columns
//     P = 2^(S - m)    in 16 bits over the same columns, by the tile's four warps
//     O += P V         in TMEM, D columns, P read from TMEM
// The running maximum m moves when it grows by more than 2^8 (smaller growth
// is cancelled by the division at the end); only then O is read and rescaled.
//
// Warps: 0 loads (and deals items), 1 issues the products, 2 and 3 put zeros
// in the place of values that nobody sees, 4-7 and 8-11 are the tiles'
// softmax. With an 8-bit cache 12-15 turn its bytes into f16 (which holds
// e4m3 exactly): queries and weights are f16 then, the keys' scales multiply
// the scores' columns and the values' the weights.
//
// A first kernel of one block adds up the sequences' tile pairs; blocks take
// pairs from a counter, the last (under the causal mask the costliest) first.
#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "fo_paged.h"
#include "fo_paged_tiles.cuh"

namespace fo_ops {
namespace {

using namespace fo;

constexpr int kTile = 128;           // rows of a tile, keys of a step
constexpr int kScaleSlots = 4;       // steps whose scales are in shared memory
constexpr int kHeadsTogether = 8;    // key heads whose pairs are dealt together: their keys and values stay in L2

struct PromptParams {
  CUtensorMap q[kMaxR];   // [rows][heads_q][D]; boxes of 64 x group x tokens
  CUtensorMap k[kMaxR];   // [pages * heads_k][page][D]; boxes of at most 128 bytes x `box` tokens
  CUtensorMap v[kMaxR];
  const float* ks[kMaxR];
  const float* vs[kMaxR];
  __nv_bfloat16* o[kMaxR];
  float* lse[kMaxR];
  int64_t ld_o;
  Batch batch;
  int32_t R, heads_q, heads_k, group, tokens;   // tokens: of a tile
  int32_t window, sinks, box;
  float scale_log2;
  int64_t* before;        // [seqs + 1]: pairs of the sequences before
  uint32_t* next;         // items dealt
};

// Pairs of tiles before each sequence, and the deal's counter at zero.
__global__ void __launch_bounds__(1024) prompt_plan_kernel(const __grid_constant__ PromptParams p) {
  __shared__ long long sums[32];
  grid_release();
  grid_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.batch.seqs + 1023) / 1024, first = min(tid * run, p.batch.seqs), last = min(first + run, p.batch.seqs);
  const int each = 2 * p.tokens;
  long long mine = 0;
  for (int b = first; b < last; ++b) mine += (sequence(p.batch, b).n + each - 1) / each;
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += sums[w];
  long long at = upto - mine;
  for (int b = first; b < last; ++b) {
    p.before[b] = at;
    at += (sequence(p.batch, b).n + each - 1) / each;
  }
  if (tid == 1023) p.before[p.batch.seqs] = upto, *p.next = 0;
}

template <int D, bool E8>
struct Prompt {
  static constexpr int kThreads = E8 ? 512 : 384;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kRawBytes = kTile * D;
  static constexpr int kCuts = D / 64;               // 128-byte columns of a 16-bit tile
  static constexpr int kStages = E8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);
  static constexpr int kRaws = E8 ? (D == 128 ? 3 : 4) : 0;
  static constexpr int kOffRing = 2 * kTileBytes;    // after the two tiles of queries
  static constexpr int kOffRaw = kOffRing + kStages * kTileBytes;
  static constexpr int kOffScale = kOffRaw + kRaws * kRawBytes;
  static constexpr int kOffRow = kOffScale + (E8 ? kScaleSlots * 2 * kTile * 4 : 0);   // the rows' factors, two items
  static constexpr int kOffItem = kOffRow + (E8 ? 2 * 2 * kTile * 4 : 0);
  static constexpr int kOffBar = kOffItem + 2 * 32;
  static constexpr int kBars = 2 * kStages + 2 * kRaws + 24;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kSmem = 1024 + kOffMisc + 16;
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr uint32_t kS = 0, kO = 256;        // TMEM columns of the first tile's scores and output
};

// An item, as the warps get it.
struct Item {
  int r, h, b, row, n, base, end, token;   // token: the pair's first
};
// The steps of a pair: blocks of 128 keys that one of its rows sees.
struct Steps {
  int lo[2], sinks_end[2], end[2];   // of each tile's first row; tokens before `end` are seen by its last
  int early, late, n;
  __device__ __forceinline__ void of(const Item& it, int tokens, int window, int sinks) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int first = it.token + t * tokens, last = min(first + tokens, it.n) - 1;
      const Sight v = sight_of(max(it.base + first, 0), window, sinks);
      lo[t] = v.lo, sinks_end[t] = v.sinks_end;
      end[t] = first < it.n ? max(it.base + last + 1, 0) : 0;
    }
    const int far = max(end[0], end[1]);
    early = (min(max(sinks_end[0], end[1] ? sinks_end[1] : 0), far) + kTile - 1) / kTile;
    late = max(lo[0] / kTile, early);
    n = far ? early + max((far + kTile - 1) / kTile - late, 0) : 0;
  }
  __device__ __forceinline__ int block(int i) const { return i < early ? i : i - early + late; }
  __device__ __forceinline__ bool active(int t, int i) const {
    const int key = block(i) * kTile;
    const int lo_t = t ? lo[1] : lo[0], sinks_t = t ? sinks_end[1] : sinks_end[0], end_t = t ? end[1] : end[0];
    return i < n && key < end_t && (key < sinks_t || key + kTile > lo_t);
  }
  // Whether a row of the pair may see the key.
  __device__ __forceinline__ bool any(int key) const {
    return key < max(end[0], end[1]) && (key >= lo[0] || key < max(sinks_end[0], sinks_end[1]));
  }
  // Whether a block holds a key that no row of the pair sees.
  __device__ __forceinline__ bool dirty(int i) const {
    const int key = block(i) * kTile;
    return key + kTile > max(end[0], end[1]) || (key < lo[0] && key + kTile > max(sinks_end[0], sinks_end[1]));
  }
};

// kind::f16 instruction descriptor: fp32 sums, bf16 (or f16) operands, B
// K-major (scores) or MN-major (weighted sum), 128 x n.
__host__ __device__ constexpr uint32_t idesc(bool f16, bool b_mn, int n) {
  return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kTile >> 4) << 24);
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ uint32_t elected() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
  return is;
}
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// Sixteen columns of a thread's row.
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// The lowest n bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

template <int D, bool E8>
__global__ void __launch_bounds__(Prompt<D, E8>::kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
  using C = Prompt<D, E8>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return base + C::kOffBar + 8u * (uint32_t)i; };
  enum : int {
    kFull = 0, kEmpty = C::kStages, kRawFull = 2 * C::kStages, kRawEmpty = kRawFull + C::kRaws,
    kQFull = kRawEmpty + C::kRaws, kQReady, kQEmpty, kSFull, kPFull = kSFull + 2, kOFull = kPFull + 2, kOFree = kOFull + 2,
    kDirty = kOFree + 2, kClean, kItemFull, kItemFree = kItemFull + 2, kDrain = kItemFree + 2, kLast
  };
  static_assert(kLast <= C::kBars, "barriers");
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbase + C::kOffMisc);
  volatile uint32_t* const tmem_at = reinterpret_cast<volatile uint32_t*>(gbase + C::kOffMisc + 4);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(bar(kFull + i), E8 ? 4 : 1), mbar_init(bar(kEmpty + i), 1);
    for (int i = 0; i < C::kRaws; ++i) mbar_init(bar(kRawFull + i), 1), mbar_init(bar(kRawEmpty + i), 4);
    mbar_init(bar(kQFull), 1);
    mbar_init(bar(kQReady), 4);
    mbar_init(bar(kQEmpty), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kSFull + t), 1);
      mbar_init(bar(kPFull + t), 4);
      mbar_init(bar(kOFull + t), 1);
      mbar_init(bar(kOFree + t), 4);
      mbar_init(bar(kItemFull + t), 1);
      mbar_init(bar(kItemFree + t), E8 ? 15 : 11);   // issuer, cleaners, softmax and converting warps
    }
    mbar_init(bar(kDirty), 1);
    mbar_init(bar(kClean), 2);
    mbar_init(bar(kDrain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc<1>(base + C::kOffMisc + 4, 512);
    tmem_relinquish<1>();
  }
  grid_release();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  grid_wait();

  // Items go from warp 0 to the others through two slots.
  volatile int* const slots = reinterpret_cast<volatile int*>(gbase + C::kOffItem);
  auto take = [&](int n, Item& it) -> bool {   // false: no more
    const int sl = n & 1;
    if (!mbar_wait(bar(kItemFull + sl), (uint32_t)(n >> 1) & 1u, abort_flag, kWaitNs)) return false;
    volatile int* const s = slots + sl * 8;
    it.r = s[0], it.h = s[1], it.b = s[2], it.row = s[3], it.n = s[4], it.base = s[5], it.end = s[6], it.token = s[7];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kItemFree + sl));
    return it.r >= 0;
  };
  Item it;
  Steps st;
  if (warp < 4) {
    if constexpr (E8) fewer_registers<72>();
    else fewer_registers<104>();
  }

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    const long long pairs = p.before[p.batch.seqs];
    const int units = p.R * p.heads_k;
    const long long total = pairs * units;
    uint32_t n_load = 0;   // tiles of keys and values loaded so far
    bool ok = true;
    int n = 0;
    constexpr int kFrom = E8 ? kRawFull : kFull, kBack = E8 ? kRawEmpty : kEmpty, kRing = E8 ? C::kRaws : C::kStages;
    uint32_t at_slot = 0, at_round = 0;
    for (; ok; ++n) {
      const int sl = n & 1;
      if (!mbar_wait(bar(kItemFree + sl), ((uint32_t)(n >> 1) & 1u) ^ 1u, abort_flag, kWaitNs)) break;
      unsigned L32 = 0;
      if (lane == 0) L32 = atomicAdd(p.next, 1u);
      const long long L = __shfl_sync(0xffffffffu, L32, 0);
      it.r = -1, it.h = it.b = it.row = it.n = it.base = it.end = it.token = 0;
      if (L < total) {
        const long long set = L / (pairs * kHeadsTogether), rem = L - set * pairs * kHeadsTogether;
        const int width = min(kHeadsTogether, units - (int)set * kHeadsTogether);
        const long long pr = rem / width;
        const int u = (int)set * kHeadsTogether + (int)(rem - pr * width);
        const long long pair = pairs - 1 - pr;
        int lo = 0, hi = p.batch.seqs;   // before[lo] <= pair < before[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (p.before[mid] <= pair) lo = mid;
          else hi = mid;
        }
        const Seq s = sequence(p.batch, lo);
        it.r = u / p.heads_k, it.h = u - it.r * p.heads_k, it.b = lo;
        it.row = s.row, it.n = s.n, it.base = s.base, it.end = s.end;
        it.token = (int)(pair - p.before[lo]) * 2 * p.tokens;
      }
      if (lane == 0) {
        volatile int* const s = slots + sl * 8;
        s[0] = it.r, s[1] = it.h, s[2] = it.b, s[3] = it.row, s[4] = it.n, s[5] = it.base, s[6] = it.end, s[7] = it.token;
        mbar_arrive(bar(kItemFull + sl));
      }
      __syncwarp();
      if (it.r < 0) break;
      st.of(it, p.tokens, p.window, p.sinks);
      if (!mbar_wait(bar(kQEmpty), (uint32_t)(n & 1) ^ 1u, abort_flag, kWaitNs)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(kQFull), 2 * C::kCuts * p.tokens * p.group * 128);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int cut = 0; cut < C::kCuts; ++cut)
            tma_load_3d(base + t * C::kTileBytes + cut * (kTile * 128), &p.q[it.r], bar(kQFull), cut * 64, it.h * p.group,
                        it.row + it.token + t * p.tokens);
      }
      const int boxes = kTile / p.box;
      for (int i = 0; i < st.n && ok; ++i) {
        const int key = st.block(i) * kTile;
        // A lane for each box of tokens: its page.
        int id = -1;
        const int mine = key + lane * p.box;
        if (lane < boxes) {
          const int far = max(st.end[0], st.end[1]);
          if (mine < far && (mine < max(st.sinks_end[0], st.sinks_end[1]) || mine + p.box > st.lo[0])) {
            id = p.batch.table[(long long)it.b * p.batch.cols + (mine >> p.batch.shift)];
            if (id < 0 || id >= p.batch.pages) {
              report(p.batch, it.b, kBadPage, id);
              id = -1;
            }
          }
        }
        const int z = id >= 0 ? id * p.heads_k + it.h : p.batch.pages * p.heads_k, y = mine & ((1 << p.batch.shift) - 1);
#pragma unroll
        for (int value = 0; value < 2; ++value) {
          if (n_load >= kRing && !mbar_wait(bar(kBack + at_slot), (at_round - 1) & 1, abort_flag, kWaitNs)) {
            ok = false;
            break;
          }
          const uint32_t full = bar(kFrom + at_slot);
          if (lane == 0) mbar_arrive_expect_tx(full, E8 ? C::kRawBytes : C::kTileBytes);
          __syncwarp();
          if (lane < boxes) {
            const CUtensorMap* const map = value ? &p.v[it.r] : &p.k[it.r];
            const int row = lane * p.box;
            if constexpr (E8) {
              tma_load_3d(base + C::kOffRaw + at_slot * C::kRawBytes + row * D, map, full, 0, y, z);
            } else {
              const uint32_t dst = base + C::kOffRing + at_slot * C::kTileBytes;
#pragma unroll
              for (int cut = 0; cut < C::kCuts; ++cut)
                // Keys: [cut][128 keys]; values: [64 keys][cut][64 keys of them].
                tma_load_3d(value ? dst + (row >> 6) * (C::kTileBytes / 2) + cut * 8192 + (row & 63) * 128
                                  : dst + cut * (kTile * 128) + row * 128,
                            map, full, cut * 64, y, z);
            }
          }
          ++n_load;
          if (++at_slot == kRing) at_slot = 0, ++at_round;
        }
      }
    }
    // What is still on its way lands before the block may end.
    volatile int never = 0;
    if (*abort_flag) {
      for (int i = 0; i < kRing && (uint32_t)i < n_load; ++i) {
        at_slot = at_slot ? at_slot - 1 : (--at_round, kRing - 1);
        mbar_wait(bar(kFrom + at_slot), at_round & 1, &never, 100000000ull);
      }
      if (n > 0) mbar_wait(bar(kQFull), (n - 1) & 1, &never, 100000000ull);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    uint32_t n_tile = 0;       // number of the item's first tile of keys, of all items
    uint32_t soft[2] = {0, 0}; // steps of each tile so far
    uint32_t cleaned = 0, outs[2] = {0, 0};
    const uint32_t one = elected();
    bool ok = true;
    auto stage_of = [&](uint32_t i) { return i % (uint32_t)C::kStages; };
    auto full = [&](uint32_t i) { return mbar_wait(bar(kFull + stage_of(i)), (i / (uint32_t)C::kStages) & 1u, abort_flag, kWaitNs); };
    for (int n = 0; ok; ++n) {
      if (!take(n, it)) break;
      st.of(it, p.tokens, p.window, p.sinks);
      if (!mbar_wait(bar(E8 ? kQReady : kQFull), (uint32_t)n & 1u, abort_flag, kWaitNs)) break;
      tc_fence_after();
      int from[2], last[2], scoring = 0;   // each tile's first and last step
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        from[t] = 0, last[t] = st.n - 1;
        while (from[t] < st.n && !st.active(t, from[t])) ++from[t];
        while (last[t] >= 0 && !st.active(t, last[t])) --last[t];
        scoring += last[t] >= 0;
      }
      if (scoring == 0 && one) tc_commit<1>(bar(kQEmpty));
      // The scores of tile t's step i; with the last of them the queries are
      // free, with the second tile's the keys.
      auto scores = [&](int t, int i) -> bool {
        const uint32_t k = n_tile + 2u * (uint32_t)i;
        if (!full(k)) return false;
        tc_fence_after();
        if (i == last[t]) --scoring;
        if (one) {
          const uint32_t a = base + t * C::kTileBytes, b = base + C::kOffRing + stage_of(k) * C::kTileBytes;
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const uint32_t off = (uint32_t)(e >> 2) * (kTile * 128) + (uint32_t)(e & 3) * 32u;
            tc_mma<1, false>(tmem + C::kS + t * 128, smem_desc_sw128(a + off, 16, 1024), smem_desc_sw128(b + off, 16, 1024),
                             idesc(E8, false, kTile), e > 0 ? 1u : 0u);
          }
          tc_commit<1>(bar(kSFull + t));
          if (t == 1 || !st.active(1, i)) tc_commit<1>(bar(kEmpty + stage_of(k)));
          if (i == last[t] && scoring == 0) tc_commit<1>(bar(kQEmpty));
        }
        __syncwarp();
        return true;
      };
      // Both tiles' first scores, unless one begins later: then in its turn.
      bool begun[2] = {from[0] < st.n && from[0] <= from[1], from[1] < st.n && from[1] <= from[0]}, first[2] = {true, true};
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (ok && begun[t]) ok = scores(t, from[t]);
      for (int i = 0; i < st.n && ok; ++i) {
        const uint32_t v = n_tile + 2u * (uint32_t)i + 1u;
        const bool dirty = !E8 && st.dirty(i);
        if (dirty) {
          if (!(ok = full(v))) break;
          if (one) mbar_arrive(bar(kDirty));
          __syncwarp();
        }
        bool waited = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || !st.active(t, i)) continue;
          if (!begun[t]) {
            begun[t] = true;
            if (!(ok = scores(t, i))) continue;
          }
          ok = mbar_wait(bar(kPFull + t), soft[t] & 1u, abort_flag, kWaitNs) &&
               (!first[t] || mbar_wait(bar(kOFree + t), (outs[t] & 1u) ^ 1u, abort_flag, kWaitNs));
          if (ok && !waited) {
            waited = true;
            ok = full(v) && (!dirty || mbar_wait(bar(kClean), cleaned & 1u, abort_flag, kWaitNs));
          }
          if (!ok) continue;
          ++soft[t];
          tc_fence_after();
          if (one) {
            const uint32_t b = base + C::kOffRing + stage_of(v) * C::kTileBytes;
#pragma unroll
            for (int e = 0; e < kTile / 16; ++e)
              mma_ts(tmem + C::kO + t * D, tmem + C::kS + t * 128 + e * 8,
                     smem_desc_sw128(b + (uint32_t)(e >> 2) * (C::kTileBytes / 2) + (uint32_t)(e & 3) * 2048u, 8192, 1024),
                     idesc(E8, true, D), !first[t] || e > 0 ? 1u : 0u);
            if (t == 1 || !st.active(1, i)) tc_commit<1>(bar(kEmpty + stage_of(v)));
            if (i == last[t]) tc_commit<1>(bar(kOFull + t));
          }
          __syncwarp();
          first[t] = false;
          if (i == last[t]) {
            ++outs[t];
          } else if (st.active(t, i + 1)) {
            ok = scores(t, i + 1);
          } else {
            begun[t] = false;   // (between first tokens and window)
          }
        }
        if (dirty) ++cleaned;
      }
      n_tile += 2u * (uint32_t)st.n;
    }
    // Every product has ended before TMEM is given back.
    volatile int never = 0;
    if (one) tc_commit<1>(bar(kDrain));
    __syncwarp();
    mbar_wait(bar(kDrain), 0, &never, 100000000ull);
  } else if (warp < 4) {
    // ------------------------------------------------------------ values that nobody sees
    uint32_t n_tile = 0, asked = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!take(n, it)) break;
      if constexpr (!E8) {
        st.of(it, p.tokens, p.window, p.sinks);
        for (int i = 0; i < st.n; ++i) {
          if (!st.dirty(i)) continue;
          const uint32_t v = n_tile + 2u * (uint32_t)i + 1u, stage = v % (uint32_t)C::kStages;
          // The issuer calls for each of them: only then is the stage's phase known.
          if (!mbar_wait(bar(kDirty), asked++ & 1u, abort_flag, kWaitNs) ||
              !mbar_wait(bar(kFull + stage), (v / (uint32_t)C::kStages) & 1u, abort_flag, kWaitNs)) {
            ok = false;
            break;
          }
          const int key = st.block(i) * kTile;
          uint8_t* const at = gbase + C::kOffRing + stage * C::kTileBytes;
          // Eight lanes a row of 128 bytes.
          for (int row = (warp - 2) * 4 + (lane >> 3); row < kTile; row += 8) {
            if (st.any(key + row)) continue;
#pragma unroll
            for (int cut = 0; cut < C::kCuts; ++cut)
              *reinterpret_cast<uint4*>(at + (row >> 6) * (C::kTileBytes / 2) + cut * 8192 + (row & 63) * 128 + (lane & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kClean));
        }
        n_tile += 2u * (uint32_t)st.n;
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax
    if constexpr (E8) more_registers<184>();
    else more_registers<200>();
    const int t = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + C::kS + t * 128, o_at = tmem + lanes + C::kO + t * D;
    uint32_t step = 0, outs = 0;   // this tile's steps and outputs so far
    uint32_t n_step = 0;           // steps of the items before
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!take(n, it)) break;
      st.of(it, p.tokens, p.window, p.sinks);
      const int token = it.token + t * p.tokens + row / p.group;
      const bool real = row < p.tokens * p.group && token < it.n;
      const int pos = real ? it.base + token : -1, lo = sight_of(max(pos, 0), p.window, p.sinks).lo;
      // Blocks all of whose keys all of the tile's rows see need no mask.
      const int first_pos = it.base + it.token + t * p.tokens;
      const int last_lo = sight_of(max(first_pos + p.tokens - 1, 0), p.window, p.sinks).lo;
      float m = -INFINITY, l = 0.f, factor = p.scale_log2, sigma = 0.f, sigma_inv = 0.f;
      bool any = false;
      for (int i = 0; i < st.n && ok; ++i) {
        if (!st.active(t, i)) continue;
        const int key = st.block(i) * kTile;
        if (!mbar_wait(bar(kSFull + t), step & 1u, abort_flag, kWaitNs)) {
          ok = false;
          break;
        }
        ++step;
        tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int e = 0; e < 4; ++e) tmem_ld32(s_at + 32 * e, v[e]);
        const float* const ks = reinterpret_cast<const float*>(gbase + C::kOffScale) + ((n_step + i) % kScaleSlots) * 2 * kTile;
        if constexpr (E8)
          if (!any) factor = p.scale_log2 * reinterpret_cast<const float*>(gbase + C::kOffRow)[((n & 1) * 2 + t) * kTile + row];
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 4; ++e) reg_fence(v[e]);
        if constexpr (E8) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 f = *reinterpret_cast<const float4*>(ks + e * 32 + k);
              float a, b;
              halves(mul2(pair_of(v[e][k], v[e][k + 1]), pair_of(f.x, f.y)), a, b);
              v[e][k] = __float_as_uint(a), v[e][k + 1] = __float_as_uint(b);
              halves(mul2(pair_of(v[e][k + 2], v[e][k + 3]), pair_of(f.z, f.w)), a, b);
              v[e][k + 2] = __float_as_uint(a), v[e][k + 3] = __float_as_uint(b);
            }
        }
        if (key + kTile - 1 > first_pos || !(key >= last_lo || key + kTile <= p.sinks)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = key + 32 * e;
            const uint32_t seen = low_bits(pos + 1 - at) & (~low_bits(lo - at) | low_bits(p.sinks - at));
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(seen >> k & 1u)) v[e][k] = 0xff800000u;   // -infinity
          }
        }
        float tops[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) tops[k] = -INFINITY;
#pragma unroll
        for (int k = 0; k < 64; ++k)
          tops[k & 7] = max3(tops[k & 7], __uint_as_float(v[k >> 4][(2 * k) & 31]), __uint_as_float(v[k >> 4][(2 * k + 1) & 31]));
        const float top = max3(max3(tops[0], tops[1], tops[2]), max3(tops[3], tops[4], tops[5]), fmaxf(tops[6], tops[7])) * factor;
        const bool grows = top > m + kLazy || (m == -INFINITY && top > m);
        float by = 1.f;
        if (grows) by = ex2_below(m, top), l *= by, m = top;
        if constexpr (E8) {
          // The values' scales over sigma, as for single tokens; sigma is one
          // for all rows.
          float mx = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at = key + lane + 32 * k;
            if (st.any(at)) mx = fmaxf(mx, ks[kTile + lane + 32 * k]);
          }
          const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(mx) & 0x7fffffffu);
          if (__uint_as_float(bits) > sigma * 128.f || sigma == 0.f) {
            const uint32_t exponent = min(max((bits + 0x7fffffu) >> 23, 9u), 253u);
            const float to = __uint_as_float((exponent - 7u) << 23);
            by *= sigma == 0.f ? 0.f : sigma / to;
            sigma = to;
            sigma_inv = 1.f / to;
          }
        }
        if (any && __any_sync(0xffffffffu, by != 1.f)) {
          // (These scores come after the sums before them in the issuer's
          // order: those are done.)
          const f32x2 by2 = pair_of(by, by);
#pragma unroll
          for (int e = 0; e < D / 32; ++e) {
            uint32_t o[32];
            tmem_ld32(o_at + 32 * e, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float a, b;
              halves(mul2(pair_of(o[k], o[k + 1]), by2), a, b);
              o[k] = __float_as_uint(a), o[k + 1] = __float_as_uint(b);
            }
            tmem_st32(o_at + 32 * e, o);
          }
        }
        any = true;
        const float down = m == -INFINITY ? 0.f : -m;
        const f32x2 factor2 = pair_of(factor, factor), down2 = pair_of(down, down);
        f32x2 sums[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float x[4];
            halves(fma2(pair_of(v[e][k], v[e][k + 1]), factor2, down2), x[0], x[1]);
            halves(fma2(pair_of(v[e][k + 2], v[e][k + 3]), factor2, down2), x[2], x[3]);
#pragma unroll
            for (int a = 0; a < 4; ++a) x[a] = ex2(x[a]);
            sums[(k >> 1) & 2] = add2(sums[(k >> 1) & 2], pair_of(x[0], x[1]));
            sums[((k >> 1) & 2) + 1] = add2(sums[((k >> 1) & 2) + 1], pair_of(x[2], x[3]));
            if constexpr (E8) {
              const float4 f = *reinterpret_cast<const float4*>(ks + kTile + 32 * e + k);
              w[k / 2] = f16x2(x[0] * f.x * sigma_inv, x[1] * f.y * sigma_inv);
              w[k / 2 + 1] = f16x2(x[2] * f.z * sigma_inv, x[3] * f.w * sigma_inv);
            } else {
              w[k / 2] = bf16x2(x[0], x[1]), w[k / 2 + 1] = bf16x2(x[2], x[3]);
            }
          }
          tmem_st16(s_at + 16 * e, w);
        }
        float s0, s1, s2, s3;
        halves(add2(sums[0], sums[1]), s0, s1);
        halves(add2(sums[2], sums[3]), s2, s3);
        l += (s0 + s1) + (s2 + s3);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull + t));
      }
      if (!ok) break;
      n_step += st.n;
      // ---- the rows' results
      if (any) {
        if (!mbar_wait(bar(kOFull + t), outs & 1u, abort_flag, kWaitNs)) break;
        ++outs;
        tc_fence_after();
      }
      uint32_t w[D / 2];
      const bool none = m == -INFINITY && l == 0.f;   // (O holds nothing then, or zeros)
      const float by = E8 ? sigma / l : 1.f / l;
#pragma unroll
      for (int e = 0; e < D / 2; ++e) w[e] = 0u;
      if (any) {
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          uint32_t o[32];
          tmem_ld32(o_at + 32 * e, o);
          tmem_ld_wait();
          reg_fence(o);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            w[16 * e + k] = none ? 0u : bf16x2(__uint_as_float(o[2 * k]) * by, __uint_as_float(o[2 * k + 1]) * by);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kOFree + t));
      }
      if (real) {
        const int64_t out = it.row + token;
        const int head = it.h * p.group + row % p.group;
        uint4* const to = reinterpret_cast<uint4*>(p.o[it.r] + out * p.ld_o + head * D);
#pragma unroll
        for (int e = 0; e < D / 8; ++e) to[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        if (p.lse[it.r]) p.lse[it.r][out * p.heads_q + head] = lse_of(m, l);
      }
    }
  } else {
    // ------------------------------------------------------------ 8 bits to f16
    if constexpr (E8) {
      fewer_registers<72>();
      const int tid = threadIdx.x - 384;   // a thread for a row (of queries) or key
      uint32_t n_tile = 0, n_step = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        if (!take(n, it)) break;
        st.of(it, p.tokens, p.window, p.sinks);
        if (!mbar_wait(bar(kQFull), (uint32_t)n & 1u, abort_flag, kWaitNs)) break;
        // The queries, each row times a power of two that brings its largest
        // magnitude to [128, 256); in place.
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          const uint32_t at = base + t * C::kTileBytes + tid * 128;
          float top = 0.f;
#pragma unroll 4
          for (int k = 0; k < D / 8; ++k) {
            float f[8];
            Vec16<__nv_bfloat16>::unpack(lds128(at + (k >> 3) * (kTile * 128) + (((k & 7) ^ (tid & 7)) << 4)), f);
            top = max_nan(top, amax_of(f));
          }
          const uint32_t exponent = min(max(__float_as_uint(top) >> 23, 8u), 254u);
          const float by = top <= 3.4e38f ? __uint_as_float((261u - exponent) << 23) : 1.f;
          reinterpret_cast<float*>(gbase + C::kOffRow)[((n & 1) * 2 + t) * kTile + tid] = 1.f / by;
#pragma unroll 4
          for (int k = 0; k < D / 8; ++k) {
            const uint32_t a = at + (k >> 3) * (kTile * 128) + (((k & 7) ^ (tid & 7)) << 4);
            float f[8];
            Vec16<__nv_bfloat16>::unpack(lds128(a), f);
            sts128(a, make_uint4(f16x2(f[0] * by, f[1] * by), f16x2(f[2] * by, f[3] * by), f16x2(f[4] * by, f[5] * by),
                                 f16x2(f[6] * by, f[7] * by)));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kQReady));
        for (int i = 0; i < st.n && ok; ++i) {
          const int key = st.block(i) * kTile + tid;
          const bool seen = st.any(key);
          float scale[2] = {0.f, 0.f};
          if (seen) {
            const int id = p.batch.table[(long long)it.b * p.batch.cols + (key >> p.batch.shift)];
            if (id >= 0 && id < p.batch.pages) {
              const long long at = ((long long)(id * p.heads_k + it.h) << p.batch.shift) + (key & ((1 << p.batch.shift) - 1));
              scale[0] = p.ks[it.r][at], scale[1] = p.vs[it.r][at];
            }
          }
#pragma unroll 1
          for (int value = 0; value < 2; ++value) {
            const uint32_t x = n_tile + 2u * (uint32_t)i + (uint32_t)value;
            const uint32_t rs = x % (uint32_t)C::kRaws, ss = x % (uint32_t)C::kStages;
            if (!mbar_wait(bar(kRawFull + rs), (x / (uint32_t)C::kRaws) & 1u, abort_flag, kWaitNs) ||
                (x >= (uint32_t)C::kStages &&
                 !mbar_wait(bar(kEmpty + ss), (x / (uint32_t)C::kStages - 1u) & 1u, abort_flag, kWaitNs))) {
              ok = false;
              break;
            }
            if (value == 0) {
              float* const to = reinterpret_cast<float*>(gbase + C::kOffScale) + ((n_step + i) % kScaleSlots) * 2 * kTile + tid;
              to[0] = scale[0], to[kTile] = scale[1];
            }
            // Sixteen bytes a time: lanes side by side in a key's bytes, so
            // that reads and writes meet no bank twice.
            const uint32_t from = base + C::kOffRaw + rs * C::kRawBytes, to = base + C::kOffRing + ss * C::kTileBytes;
            constexpr int kPieces = D / 16;
#pragma unroll 4
            for (int k = tid; k < kTile * kPieces; k += kTile) {
              const int row = k / kPieces, piece = k % kPieces;
              const uint4 v = lds128(D == 128 ? from + row * 128 + ((piece ^ (row & 7)) << 4) : from + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
              uint4 a = make_uint4(f16x2_of_e4m3(v.x), f16x2_of_e4m3_high(v.x), f16x2_of_e4m3(v.y), f16x2_of_e4m3_high(v.y));
              uint4 b = make_uint4(f16x2_of_e4m3(v.z), f16x2_of_e4m3_high(v.z), f16x2_of_e4m3(v.w), f16x2_of_e4m3_high(v.w));
              if (value && !st.any(st.block(i) * kTile + row)) a = b = make_uint4(0, 0, 0, 0);
              const int cut = piece >> 2, c16 = (piece & 3) * 2;
              const uint32_t at = value ? to + (row >> 6) * (C::kTileBytes / 2) + cut * 8192 + (row & 63) * 128
                                        : to + cut * (kTile * 128) + row * 128;
              sts128(at + ((c16 ^ (row & 7)) << 4), a);
              sts128(at + (((c16 + 1) ^ (row & 7)) << 4), b);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kRawEmpty + rs)), mbar_arrive(bar(kFull + ss));
          }
        }
        n_tile += 2u * (uint32_t)st.n;
        n_step += (uint32_t)st.n;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc<1>(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) record_error(p.batch.status, FO_ERR_TIMEOUT, -1, -1, 0);
}

template <int D, bool E8>
fo_status launch_prompt(PromptParams& k, int sms, cudaStream_t s) {
  using C = Prompt<D, E8>;
  auto kern = prompt_kernel<D, E8>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  fo_status st = launched(e, "paged prompt", k.R, k.batch.rows, D, 0, C::kThreads);
  if (st || (st = launched(launch_after(prompt_plan_kernel, dim3(1), 1024, 0, 0, s, k), "paged prompt plan", k.R, k.batch.rows, D, 1, 1024)))
    return st;
  // No more blocks than pairs there can be.
  const int64_t pairs = (k.batch.rows / (2 * k.tokens) + k.batch.seqs) * (int64_t)(k.R * k.heads_k);
  const int blocks = (int)std::min<int64_t>(pairs, sms);
  return launched(launch_after(kern, dim3(blocks), C::kThreads, C::kSmem, 0, s, k), "paged prompt", k.R, k.batch.rows, D, blocks, C::kThreads);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

}  // namespace

bool encode_pages(CUtensorMap* m, const void* p, const fo_paged_desc* d, int64_t pages, int box) {
  const auto fn = encoder();
  if (!fn) return false;
  const bool eight = d->cache_dtype == FO_CACHE_E4M3;
  const cuuint64_t row = (cuuint64_t)d->head_dim * (eight ? 1 : 2);
  const cuuint64_t dims[3] = {(cuuint64_t)d->head_dim, (cuuint64_t)d->page, (cuuint64_t)(pages * d->heads_k)};
  const cuuint64_t strides[2] = {row, row * d->page};
  const cuuint32_t boxes[3] = {eight ? (cuuint32_t)d->head_dim : 64u, (cuuint32_t)box, 1u}, steps[3] = {1, 1, 1};
  return fn(m, eight ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides,
            boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, row < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_rows(CUtensorMap* m, const void* p, int64_t rows, int64_t ld, int heads, int D, int box_heads, int box_rows) {
  const auto fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows}, strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
  const cuuint32_t boxes[3] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, steps[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace: header, the deal's counter, pairs before each sequence.
size_t prompt_bytes(int32_t seqs) { return 256 + ((size_t)seqs + 1) * 8; }

fo_status attend_prompts(const PagedCall& c, cudaStream_t s) {
  const fo_paged_desc* const d = c.d;
  const bool eight = d->cache_dtype == FO_CACHE_E4M3;
  PromptParams k;
  memset(static_cast<void*>(&k), 0, sizeof(k));
  static_assert(sizeof(k) <= 32764, "kernel parameters");
  k.group = d->heads_q / d->heads_k;
  k.tokens = kTile / k.group;
  k.box = std::min(d->page, 64);
  for (int r = 0; r < d->R; ++r) {
    if (!encode_rows(&k.q[r], c.q[r], c.rows, c.ld[0], d->heads_q, d->head_dim, k.group, k.tokens) ||
        !encode_pages(&k.k[r], c.k[r], d, c.b->pages, k.box) || !encode_pages(&k.v[r], c.v[r], d, c.b->pages, k.box))
      return FO_ERR_CUDA;
    k.ks[r] = eight ? c.ks[r] : nullptr;
    k.vs[r] = eight ? c.vs[r] : nullptr;
    k.o[r] = static_cast<__nv_bfloat16*>(c.o[r]);
    k.lse[r] = c.lse ? c.lse[r] : nullptr;
  }
  k.ld_o = c.ld[1];
  k.batch = batch_of(d, c.b, c.rows, c.ws);
  k.R = d->R;
  k.heads_q = d->heads_q;
  k.heads_k = d->heads_k;
  k.window = d->window;
  k.sinks = d->sinks;
  k.scale_log2 = c.scale_log2;
  k.next = reinterpret_cast<uint32_t*>(c.ws + 128);
  k.before = reinterpret_cast<int64_t*>(c.ws + 256);
  if (d->head_dim == 128) return eight ? launch_prompt<128, true>(k, c.sms, s) : launch_prompt<128, false>(k, c.sms, s);
  return eight ? launch_prompt<64, true>(k, c.sms, s) : launch_prompt<64, false>(k, c.sms, s);
}

}  // namespace fo_ops
