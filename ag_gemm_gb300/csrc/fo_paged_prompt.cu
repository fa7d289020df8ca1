// Attention of prompts over a paged cache: many new tokens a sequence, on
// tcgen05.
//
// The rows that read a key head are its group's heads of every new token,
// tokens outermost; 128 of them (as many whole tokens as fit) are a tile, and
// a block works on two tiles at a time over the same keys and values, 128 a
// step. While the tensor core sums one tile's weights times values and
// computes its next scores (1024 cycles of bf16 at D = 128), the other tile's
// softmax runs. Per step and tile:
//     S = Q K^T        in TMEM, 128 columns
//     P = 2^(S - m)    in 16 bits over the same columns, by the tile's four warps
//     O += P V         in TMEM, D columns, P read from TMEM
// A thread has a row of its own, so no row needs another thread. The running
// maximum m moves when it grows by more than 2^8 (smaller growth is cancelled
// by the division at the end); only then O is read and rescaled.
//
// Warps: 0 loads (and deals items), 1 and 2 issue the tiles' products (one
// issuer for both fell behind: a wait for a barrier that is ready takes it 150
// cycles), 3 puts zeros in the place of values that nobody sees, 4-7 and 8-11
// are the tiles' softmax. With an 8-bit cache 12-15 turn its bytes into f16,
// and queries and weights are f16 too. Keys stay exact, and the softmax
// multiplies scores with their scales: with the scales in the keys, each
// rounded to 2^-11 of it, lse was off by 1e-4 where fp32's 1e-7 could be had,
// for 84 us in place of 92 (8-bit chunks). Values are turned times their scale
// over a power of two for each 32, which the softmax puts on their weights; what
// that rounds, 2^-11 of a value, is less than the result's own 2^-8.
//
// A first kernel of one block lists the items; blocks take them from a
// counter, the last (under the causal mask the costliest) first. A third joins
// the parts of pairs of tiles that were cut.
//
// 8 ranks of 8192 tokens with 4 heads, causal, take 395 us (393 to 402 from one
// GB300 to another), 1.39 PFLOP/s of the products that are seen: a step of two tiles takes
// some 3000 cycles, 2048 of them the tensor core's, since a tile's softmax with
// what it waits for is longer than the other tile's products. 8192 tokens with a
// window of 1024 + 4 and 32 + 8 heads take 141 us (to 148), 0.92 PFLOP/s: items of
// ten or eleven steps, whose ends and starts are not hidden (two tiles' scores
// and outputs fill TMEM), and a fifth of the products masked. Begun with the first
// 64 keys' weights, the weighted sum made the one 392 us and the other 146. The
// loop's length counts: rescaling written out for all columns, which seldom runs,
// cost the one 4 us, and a branch around weights of 32 keys that no row sees 10.
// Chunks of up to 1030 tokens of 8 bits, D = 64, take 84 us, D = 128 108: at D =
// 64 the exponentials are as long as both products. The first case from an 8-bit
// cache takes 547 us, the second 208; in bf16 with D = 64, 317 and 119.
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
  uint32_t least_exponent;
  int32_t sms;
  int64_t* before;        // [seqs + 1]: pairs of the sequences before
  uint32_t* next;         // [0] items dealt, [1] items of a key head, [2] parts of it, [3] cut pairs of it, [4] blocks of 32 rows of the largest
  struct Record* items;   // [most_items]
  long long most_items;
  float* part;            // [most parts][2 * kTile * (D + 2)]
  struct Record* cut;     // [kMostParts]: the first part of each pair that is cut, of a key head
};

// An item: a pair of tiles, or some of its steps.
struct Record {
  int32_t b, row, n, base, token;   // token: the pair's first
  int32_t from, to;                 // steps
  int32_t slot, parts;              // the pair's first part, its parts (1: the item is the whole pair)
  int32_t part;
  int32_t at, pad;                  // of a cut pair, while it is planned: its first item
};
// As the warps get it.
struct Item {
  int r, h, b, row, n, base, token, from, to, slot, parts, part;
};
// The steps of a pair: blocks of 128 keys that one of its rows sees.
struct Steps {
  int lo[2], sinks_end[2], end[2];   // of each tile's first row; tokens before `end` are seen by its last
  int early, late, n;
  template <typename T>
  __device__ __forceinline__ void of(const T& it, int tokens, int window, int sinks) {
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


// ---- the plan: one block lists the items of a key head.
//
// A pair of more steps than an SM's share of one and a half times what is still
// to be dealt (but never of fewer than an even share among twice the SMs) is cut
// into parts, which a third kernel joins: without that a few long pairs (chunks of
// prompts on long prefixes, drafted tokens) left most of the GPU idle. What is
// dealt early may be long, so few pairs are cut: with twice the SMs' even share
// as the limit of all, 8-bit chunks took 92 us, not 84, and 40 rows over 65536
// tokens 42, not 36 (64 contexts of up to 8192, on the other hand, 105, not 110).
constexpr int kLeastSteps = 4;
constexpr int kSharesPerSm = 2;
// Parts of pairs that are cut, at most: sum of ceil(n / L) over pairs of n > L
// steps, with L at least the sum of n over kSharesPerSm * SMs.
static_assert(kMostParts == 2 * kSharesPerSm * FO_GB300_SMS, "parts");

// Of 1024 threads: the sum of those up to this one, and of all.
__device__ __forceinline__ long long block_scan(long long mine, long long* sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](long long v) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  mine = scan(mine);
  __syncthreads();
  if (lane == 31) sums[warp] = mine;
  __syncthreads();
  const long long warps = scan(sums[lane]);
  *total = __shfl_sync(0xffffffffu, warps, 31);
  const long long before = __shfl_sync(0xffffffffu, warps, (warp + 31) & 31);
  return mine + (warp ? before : 0);
}

__global__ void __launch_bounds__(1024) prompt_plan_kernel(const __grid_constant__ PromptParams p) {
  __shared__ long long sums[32];
  __shared__ int largest;
  __shared__ int few[1025];   // pairs before each of up to 1024 sequences: looked up here, not in global memory
  if (threadIdx.x == 0) largest = 0;
  grid_release();
  grid_wait();
  const int tid = threadIdx.x, each = 2 * p.tokens;
  long long pairs, steps, items, parts, cuts;
  const bool in_few = p.batch.seqs <= 1024 && p.batch.rows < 1 << 30;
  {
    const int run = (p.batch.seqs + 1023) / 1024, first = min(tid * run, p.batch.seqs), last = min(first + run, p.batch.seqs);
    long long mine = 0;
    for (int b = first; b < last; ++b) mine += (sequence(p.batch, b).n + each - 1) / each;
    long long at = block_scan(mine, sums, &pairs) - mine;
    if (in_few) {
      if (tid < p.batch.seqs) few[tid] = (int)at;
      if (tid == 0) few[p.batch.seqs] = (int)pairs;
    } else {
      for (int b = first; b < last; ++b) {
        p.before[b] = at;
        at += (sequence(p.batch, b).n + each - 1) / each;
      }
      if (tid == 0) p.before[p.batch.seqs] = pairs;
    }
    __syncthreads();
  }
  // More rows than the call's: only starts that fall can say so.
  const bool bad = pairs > p.most_items;
  if (bad) pairs = 0;
  auto before = [&](int b) { return in_few ? (long long)few[b] : p.before[b]; };
  // A thread's run of pairs, from the last on; a visit to each.
  const long long run = (pairs + 1023) / 1024, first = min(tid * run, pairs), last = min(first + run, pairs);
  Record own;
  int own_n = -1;   // of a run of one, which is looked at once
  auto visit = [&](auto&& f) {
    if (first >= last) return;
    if (own_n >= 0) {
      f(own, own_n);
      return;
    }
    int lo = 0, hi = p.batch.seqs;   // before(lo) <= pair < before(hi)
    const long long start = pairs - 1 - first;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before(mid) <= start) lo = mid;
      else hi = mid;
    }
    Seq s = sequence(p.batch, lo);
    Record it;
    Steps st;
    for (long long e = first; e < last; ++e) {
      const long long pair = pairs - 1 - e;
      while (pair < before(lo)) s = sequence(p.batch, --lo);
      it.b = lo, it.row = s.row, it.n = s.n, it.base = s.base;
      it.token = (int)(pair - before(lo)) * each;
      st.of(it, p.tokens, p.window, p.sinks);
      if (run == 1) own = it, own_n = st.n;
      f(it, st.n);
    }
  };
  long long mine = 0;
  visit([&](Record&, int n) { mine += max(n, 1); });
  const long long dealt = block_scan(mine, sums, &steps) - mine, shares = (long long)kSharesPerSm * p.sms;
  const long long least = max((steps * p.R * p.heads_k + shares - 1) / shares, (long long)kLeastSteps);
  long long left = 0;   // steps from a pair on
  auto parts_of = [&](int n) {
    const long long most = max(3 * left * p.R * p.heads_k / (2 * p.sms), least);
    left -= max(n, 1);
    return n > most ? (int)((n + most - 1) / most) : 1;
  };
  // Items, and in the upper half of the number parts; cut pairs by themselves.
  long long my_items = 0, my_parts = 0;
  left = steps - dealt;
  visit([&](Record&, int n) {
    const int k = parts_of(n);
    my_items += k;
    my_parts += k > 1 ? ((long long)k << 32) + 1 : 0;
  });
  long long at = block_scan(my_items, sums, &items) - my_items, both = block_scan(my_parts, sums, &parts) - my_parts;
  cuts = parts & 0xffffffffll, parts >>= 32;
  long long cut = both & 0xffffffffll, slot = both >> 32;
  left = steps - dealt;
  visit([&](Record& it, int n) {
    const int k = parts_of(n);
    it.parts = k, it.part = 0;
    it.slot = (int)slot;
    it.from = 0, it.to = n;
    if (k > 1) {
      it.at = (int)at;
      if (cut < kMostParts) p.cut[cut] = it;
      ++cut, slot += k;
      atomicMax(&largest, it.n - it.token <= p.tokens ? ((it.n - it.token) * p.group + 31) / 32 : 2 * kTile / 32);
    } else if (at < p.most_items) {
      p.items[at] = it;
    }
    at += k;
  });
  // A warp for a cut pair's items: one of many parts is as many items.
  __syncthreads();
  for (long long c = tid >> 5; c < (items <= p.most_items ? cuts : 0); c += 32) {
    Record it = p.cut[c];
    const int n = it.to, k = it.parts, q = n / k, more = n - q * k;   // the first `more` have a step more
    for (int i = tid & 31; i < k; i += 32) {
      it.part = i;
      it.from = i * q + min(i, more), it.to = it.from + q + (i < more);
      p.items[it.at + i] = it;
    }
  }
  if (tid == 0) {
    if (bad || items > p.most_items) report(p.batch, 0, kBadStarts, p.batch.rows);
    p.next[0] = 0;
    p.next[1] = items > p.most_items ? 0u : (uint32_t)items;
    p.next[2] = (uint32_t)parts;
    p.next[3] = items > p.most_items ? 0u : (uint32_t)cuts;
    p.next[4] = (uint32_t)largest;
  }
}

template <int D, bool E8>
struct Prompt {
  static constexpr int kThreads = E8 ? 512 : 384;
  static constexpr int kConverters = 4;              // warps
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kRawBytes = kTile * D;
  static constexpr int kCuts = D / 64;               // 128-byte columns of a 16-bit tile
  static constexpr int kStages = E8 ? (D == 128 ? 3 : 6) : (D == 128 ? 4 : 8);
  static constexpr int kRaws = E8 ? (D == 128 ? 3 : 4) : 0;
  // Steps whose scales are in shared memory. Keys of step i + kScaleSlots are
  // turned once the last reader has released their stage, which was a product's
  // that followed the softmax of step i.
  static constexpr int kScaleSlots = kStages / 2 + 1;
  static constexpr int kScaleBytes = (kTile + 4) * 4;   // the keys', the values' powers of two
  static constexpr int kOffRing = 2 * kTileBytes;    // after the two tiles of queries
  static constexpr int kOffRaw = kOffRing + kStages * kTileBytes;
  static constexpr int kOffScale = kOffRaw + kRaws * kRawBytes;
  static constexpr int kOffRow = kOffScale + (E8 ? kScaleSlots * kScaleBytes : 0);   // the rows' factors (exponents of two), two items
  static constexpr int kOffItem = kOffRow + (E8 ? 2 * 2 * kTile : 0);
  static constexpr int kOffOut = (kOffItem + 2 * 48 + 127) / 128 * 128;   // results on their way out: a warp's 32 rows x 64 bytes
  static constexpr int kOffBar = kOffOut + 8 * 2048;
  static constexpr int kBars = 3 * kStages + 2 * kRaws + 26;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kSmem = 1024 + kOffMisc + 16;
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr uint32_t kS = 0, kO = 256;        // TMEM columns of the first tile's scores and output
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
// Two f16 times two others.
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
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
    kReady = kOFree + 2, kItemFull = kReady + C::kStages, kItemFree = kItemFull + 2, kDrain = kItemFree + 2, kTurn = kDrain + 2, kLast = kTurn + 2
  };
  static_assert(kLast <= C::kBars, "barriers");
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbase + C::kOffMisc);
  volatile uint32_t* const tmem_at = reinterpret_cast<volatile uint32_t*>(gbase + C::kOffMisc + 4);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(bar(kFull + i), E8 ? C::kConverters : 1), mbar_init(bar(kEmpty + i), 2), mbar_init(bar(kReady + i), 1);
    for (int i = 0; i < C::kRaws; ++i) mbar_init(bar(kRawFull + i), 1), mbar_init(bar(kRawEmpty + i), C::kConverters);
    mbar_init(bar(kQFull), 1);
    mbar_init(bar(kQReady), C::kConverters);
    mbar_init(bar(kQEmpty), 2);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kSFull + t), 1);
      mbar_init(bar(kPFull + t), 4);
      mbar_init(bar(kOFull + t), 1);
      mbar_init(bar(kOFree + t), 4);
      mbar_init(bar(kItemFull + t), 1);
      mbar_init(bar(kDrain + t), 1);
      mbar_init(bar(kTurn + t), 1);
      mbar_init(bar(kItemFree + t), C::kThreads / 32 - 1);   // all warps but the first
    }
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
    volatile int* const s = slots + sl * 12;
    it.r = s[0], it.h = s[1], it.b = s[2], it.row = s[3], it.n = s[4], it.base = s[5], it.token = s[6];
    it.from = s[7], it.to = s[8], it.slot = s[9], it.parts = s[10], it.part = s[11];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kItemFree + sl));
    return it.r >= 0;
  };
  Item it;
  Steps st;
  // (What two warpgroups take more, the others leave.)
  if (warp < 4) fewer_registers<E8 ? 72 : 104>();

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    const long long items = p.next[1], parts = p.next[2];
    const int units = p.R * p.heads_k;
    const long long total = items * units;
    uint32_t n_load = 0;   // tiles of keys and values loaded so far
    bool ok = true;
    int n = 0;
    constexpr int kFrom = E8 ? kRawFull : kFull, kBack = E8 ? kRawEmpty : kEmpty, kRing = E8 ? C::kRaws : C::kStages;
    uint32_t at_slot = 0, at_round = 0;
    for (; ok; ++n) {
      const int sl = n & 1;
      if (!mbar_wait(bar(kItemFree + sl), ((uint32_t)(n >> 1) & 1u) ^ 1u, abort_flag, kWaitNs)) break;
      unsigned L32 = blockIdx.x;   // (the first without a look at the counter)
      if (n > 0 && lane == 0) L32 = atomicAdd(p.next, 1u) + gridDim.x;
      const long long L = __shfl_sync(0xffffffffu, L32, 0);
      it.r = -1;
      if (L < total) {
        const long long set = L / (items * kHeadsTogether), rem = L - set * items * kHeadsTogether;
        const int width = min(kHeadsTogether, units - (int)set * kHeadsTogether);
        const int at = (int)(rem / width), u = (int)set * kHeadsTogether + (int)(rem - (long long)at * width);
        const Record rec = p.items[at];
        it.r = u / p.heads_k, it.h = u - it.r * p.heads_k, it.b = rec.b;
        it.row = rec.row, it.n = rec.n, it.base = rec.base, it.token = rec.token;
        it.from = rec.from, it.to = rec.to, it.parts = rec.parts, it.part = rec.part;
        it.slot = (int)(u * parts) + rec.slot;
      }
      if (lane == 0) {
        volatile int* const s = slots + sl * 12;
        s[0] = it.r;
        if (it.r >= 0) {
          s[1] = it.h, s[2] = it.b, s[3] = it.row, s[4] = it.n, s[5] = it.base, s[6] = it.token;
          s[7] = it.from, s[8] = it.to, s[9] = it.slot, s[10] = it.parts, s[11] = it.part;
        }
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
      // The page of this lane's box of tokens in a step's keys; -1: not needed.
      const int far = max(st.end[0], st.end[1]), sinks_end = max(st.sinks_end[0], st.sinks_end[1]);
      auto page_of = [&](int i) -> int {
        const int key = st.block(i) * kTile + lane * p.box;
        if (lane >= boxes || key >= far || (key >= sinks_end && key + p.box <= st.lo[0])) return -1;
        const int id = p.batch.table[(long long)it.b * p.batch.cols + (key >> p.batch.shift)];
        if (id >= 0 && id < p.batch.pages) return id;
        report(p.batch, it.b, kBadPage, id);
        return -1;
      };
      int next_id = it.from < it.to ? page_of(it.from) : -1;
      for (int i = it.from; i < it.to && ok; ++i) {
        const int id = next_id;
        if (i + 1 < it.to) next_id = page_of(i + 1);
        const int z = id >= 0 ? id * p.heads_k + it.h : p.batch.pages * p.heads_k;
        const int y = (st.block(i) * kTile + lane * p.box) & ((1 << p.batch.shift) - 1);
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
  } else if (warp < 3) {
    // ------------------------------------------------------------ products, a warp for each tile
    const int t = warp - 1;
    uint32_t n_tile = 0;                         // number of the item's first tile of keys, of all items
    uint32_t soft = 0, outs = 0, turns = 0;      // steps, outputs, turns so far
    const uint32_t one = elected();
    bool ok = true;
    auto full = [&](int which, uint32_t i) {
      return mbar_wait(bar(which + i % (uint32_t)C::kStages), (i / (uint32_t)C::kStages) & 1u, abort_flag, kWaitNs);
    };
    // The tiles take turns, each with its weighted sum and its next scores:
    // mixed in the tensor pipe they would end together, and so would their
    // softmax, instead of one beside the other's products.
    auto my_turn = [&]() { return mbar_wait(bar(kTurn + t), (turns++ & 1u) ^ (t == 0 ? 1u : 0u), abort_flag, kWaitNs); };
    auto your_turn = [&]() {
      if (one) mbar_arrive(bar(kTurn + (t ^ 1)));
      __syncwarp();
    };
    const uint64_t q_desc = smem_desc_sw128(base + t * C::kTileBytes, 16, 1024);
    const uint64_t k_desc = smem_desc_sw128(base + C::kOffRing, 16, 1024), v_desc = smem_desc_sw128(base + C::kOffRing, 8192, 1024);
    const uint32_t s_col = tmem + C::kS + t * 128, o_col = tmem + C::kO + t * D;
    for (int n = 0; ok; ++n) {
      if (!take(n, it)) break;
      st.of(it, p.tokens, p.window, p.sinks);
      const int steps = it.to - it.from;
      if (!(ok = mbar_wait(bar(E8 ? kQReady : kQFull), (uint32_t)n & 1u, abort_flag, kWaitNs))) break;
      tc_fence_after();
      // Of 32 steps at a time, a lane for each: which this tile takes part in.
      uint32_t mine = 0;
      auto look = [&](int i) {
        const int at = it.from + i + lane;
        mine = __ballot_sync(0xffffffffu, at < it.to && st.active(t, at));
      };
      int last = -1;   // this tile's last step
      for (int i = 0; i < steps; i += 32) {
        look(i);
        if (mine) last = i + 31 - __clz(mine);
      }
      if (last < 0 && one) mbar_arrive(bar(kQEmpty));
      // The scores of step i, whose keys have been waited for. The other tile's
      // turn is called for with half of them to go: it takes as long to come.
      auto scores = [&](int i, bool call) {
        const uint32_t k = n_tile + 2u * (uint32_t)i;
        if (one) {
          const uint64_t b = k_desc + (uint64_t)((k % (uint32_t)C::kStages) * (C::kTileBytes >> 4));
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const uint64_t off = (uint64_t)(((e >> 2) * (kTile * 128) + (e & 3) * 32) >> 4);
            tc_mma<1, false>(s_col, q_desc + off, b + off, idesc(E8, false, kTile), e > 0 ? 1u : 0u);
            if (e == D / 32 - 1 && call) mbar_arrive(bar(kTurn + (t ^ 1)));
          }
          tc_commit<1>(bar(kSFull + t));
          tc_commit<1>(bar(kEmpty + k % (uint32_t)C::kStages));
          if (i == last) tc_commit<1>(bar(kQEmpty));
        }
        __syncwarp();
      };
      bool begun = false, first = true;   // this step's scores are under way; no output yet
      for (int i = 0; i < steps; ++i) {
        if ((i & 31) == 0) look(i);
        const uint32_t bit = 1u << (i & 31), v = n_tile + 2u * (uint32_t)i + 1u;
        if (!(mine & bit)) {   // the stages are the other tile's alone (but each is released in its turn)
          for (uint32_t x = v - 1u; ok && x <= v; ++x) {
            ok = full(kFull, x);
            if (ok && one) mbar_arrive(bar(kEmpty + x % (uint32_t)C::kStages));
            __syncwarp();
          }
          if (!ok || !(ok = my_turn())) break;
          your_turn();
          continue;
        }
        if (!begun) {
          if (!(ok = full(kFull, v - 1u))) break;
          tc_fence_after();
          scores(i, false);
        }
        // The next scores come with this step's sum, unless the tile passes
        // over steps (between first tokens and window) or they are the next
        // 32's: then in their turn.
        begun = bit << 1 & mine;
        if (!(ok = full(E8 ? kFull : kReady, v) && (!first || mbar_wait(bar(kOFree + t), (outs & 1u) ^ 1u, abort_flag, kWaitNs)) &&
                   (!begun || full(kFull, v + 1u)) && mbar_wait(bar(kPFull + t), soft & 1u, abort_flag, kWaitNs) && my_turn()))
          break;
        ++soft;
        tc_fence_after();
        if (one) {
          const uint64_t b = v_desc + (uint64_t)((v % (uint32_t)C::kStages) * (C::kTileBytes >> 4));
#pragma unroll
          for (int e = 0; e < kTile / 16; ++e)
            mma_ts(o_col, s_col + e * 8, b + (uint64_t)(((e >> 2) * (C::kTileBytes / 2) + (e & 3) * 2048) >> 4),
                   idesc(E8, true, D), e > 0 || !first ? 1u : 0u);
          tc_commit<1>(bar(kEmpty + v % (uint32_t)C::kStages));
          if (i == last) tc_commit<1>(bar(kOFull + t));
        }
        __syncwarp();
        first = false;
        if (begun) scores(i + 1, true);
        else your_turn();
      }
      outs += last >= 0;
      n_tile += 2u * (uint32_t)steps;
    }
    // Every product has ended before TMEM is given back.
    volatile int never = 0;
    if (one) tc_commit<1>(bar(kDrain + t));
    __syncwarp();
    mbar_wait(bar(kDrain + t), 0, &never, 100000000ull);
  } else if (warp == 3 && E8) {
    // ------------------------------------------------------------ (nothing to do: 8-bit values are cleaned as they are turned)
    for (int n = 0; take(n, it); ++n) {
    }
  } else if (warp == 3 || warp >= 12) {
    if constexpr (E8) fewer_registers<72>();
    if constexpr (!E8) {
      // ---------------------------------------------------------- values that nobody sees
      uint32_t n_tile = 0;
      for (int n = 0, ok = 1; ok; ++n) {
        if (!take(n, it)) break;
        st.of(it, p.tokens, p.window, p.sinks);
        for (int i = it.from; i < it.to; ++i) {
          const uint32_t v = n_tile + 2u * (uint32_t)(i - it.from) + 1u, stage = v % (uint32_t)C::kStages;
          if (!(ok = mbar_wait(bar(kFull + stage), (v / (uint32_t)C::kStages) & 1u, abort_flag, kWaitNs))) break;
          if (st.dirty(i)) {
            const int key = st.block(i) * kTile;
            uint8_t* const at = gbase + C::kOffRing + stage * C::kTileBytes;
            // Eight lanes a row of 128 bytes.
            for (int row = lane >> 3; row < kTile; row += 4) {
              if (st.any(key + row)) continue;
#pragma unroll
              for (int cut = 0; cut < C::kCuts; ++cut)
                *reinterpret_cast<uint4*>(at + (row >> 6) * (C::kTileBytes / 2) + cut * 8192 + (row & 63) * 128 + (lane & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(bar(kReady + stage));
        }
        n_tile += 2u * (uint32_t)(it.to - it.from);
      }
    } else {
      // ---------------------------------------------------------- 8 bits to f16
      const int tid = (warp - 12) * 32 + lane;   // a thread for a row (of queries) or key
      uint32_t n_tile = 0, n_step = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        if (!take(n, it)) break;
        st.of(it, p.tokens, p.window, p.sinks);
        if (!mbar_wait(bar(kQFull), (uint32_t)n & 1u, abort_flag, kWaitNs)) break;
        // The queries, each row times a power of two that brings its largest
        // magnitude to [128, 256) (or less: see least_exponent); in place.
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          const int row = tid;
          const uint32_t at = base + t * C::kTileBytes + row * 128;
          float top = 0.f;
#pragma unroll 8
          for (int k = 0; k < D / 8; ++k) {
            float f[8];
            Vec16<__nv_bfloat16>::unpack(lds128(at + (k >> 3) * (kTile * 128) + (((k & 7) ^ (row & 7)) << 4)), f);
            top = max_nan(top, amax_of(f));
          }
          const uint32_t exponent = min(max(__float_as_uint(top) >> 23, p.least_exponent), 254u);
          const float by = top <= 3.4e38f ? __uint_as_float((261u - exponent) << 23) : 1.f;
          gbase[C::kOffRow + ((n & 1) * 2 + t) * kTile + row] = (uint8_t)(top <= 3.4e38f ? exponent - 7u : 127u);   // of 1 / by
#pragma unroll 8
          for (int k = 0; k < D / 8; ++k) {
            const uint32_t a = at + (k >> 3) * (kTile * 128) + (((k & 7) ^ (row & 7)) << 4);
            float f[8];
            Vec16<__nv_bfloat16>::unpack(lds128(a), f);
            sts128(a, make_uint4(f16x2(f[0] * by, f[1] * by), f16x2(f[2] * by, f[3] * by), f16x2(f[4] * by, f[5] * by),
                                 f16x2(f[6] * by, f[7] * by)));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kQReady));
        // A key's place in the scales (its page looked up), and its scales: of
        // the next step while this one's bytes are turned.
        auto place_of = [&](int i) -> long long {
          const int key = st.block(i) * kTile + tid;
          if (i >= it.to || !st.any(key)) return -1;
          const int id = p.batch.table[(long long)it.b * p.batch.cols + (key >> p.batch.shift)];
          if (id < 0 || id >= p.batch.pages) return -1;
          return ((long long)(id * p.heads_k + it.h) << p.batch.shift) + (key & ((1 << p.batch.shift) - 1));
        };
        auto scale_of = [&](const float* from, long long at) { return at >= 0 ? from[at] : 0.f; };
        long long next = place_of(it.from);
        float k_scale = scale_of(p.ks[it.r], next), v_scale = scale_of(p.vs[it.r], next);
        for (int i = it.from; i < it.to && ok; ++i) {
          const bool seen = st.any(st.block(i) * kTile + tid);
          // 2^-7 times a power of two not below the scales of the warp's 32 values:
          // scales over it are at most 128, values at most 57344, and where f16's
          // least steps begin, 2^-31 of the largest value is lost. It goes out with
          // the keys: the softmax reads it when it has the step's scores, which
          // wait for the keys alone.
          const uint32_t top = __reduce_max_sync(0xffffffffu, seen ? __float_as_uint(v_scale) & 0x7fffffffu : 0u);
          const uint32_t exponent = max((top + 0x7fffffu) >> 23, 40u) - 7u;
          next = place_of(i + 1);
          float k_next = 0.f, v_next = 0.f;
#pragma unroll 1
          for (int value = 0; value < 2; ++value) {
            const uint32_t x = n_tile + 2u * (uint32_t)(i - it.from) + (uint32_t)value;
            const uint32_t rs = x % (uint32_t)C::kRaws, ss = x % (uint32_t)C::kStages;
            if (!mbar_wait(bar(kRawFull + rs), (x / (uint32_t)C::kRaws) & 1u, abort_flag, kWaitNs) ||
                (x >= (uint32_t)C::kStages &&
                 !mbar_wait(bar(kEmpty + ss), (x / (uint32_t)C::kStages - 1u) & 1u, abort_flag, kWaitNs))) {
              ok = false;
              break;
            }
            if (value) k_next = scale_of(p.ks[it.r], next), v_next = scale_of(p.vs[it.r], next);
            // Keys stay as they are (f16 holds them), and the softmax multiplies
            // with their scales. Values are multiplied here, with their scale
            // over the power of two, which the softmax puts on their weights.
            uint32_t by = 0;
            if (value) {
              const float scale = v_scale * __uint_as_float((254u - exponent) << 23);
              by = f16x2(scale, scale);
            } else {
              float* const scales = reinterpret_cast<float*>(gbase + C::kOffScale + ((n_step + i - it.from) % C::kScaleSlots) * C::kScaleBytes);
              scales[tid] = seen ? k_scale : 0.f;
              if (lane == 0) scales[kTile + (tid >> 5)] = __uint_as_float(exponent << 23);
            }
            // A thread's key, sixteen bytes a time (the swizzle has neighbours'
            // in other banks).
            const uint32_t from = base + C::kOffRaw + rs * C::kRawBytes, to = base + C::kOffRing + ss * C::kTileBytes;
            const uint32_t row_at = value ? to + (tid >> 6) * (C::kTileBytes / 2) + (tid & 63) * 128 : to + tid * 128;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint4 u = lds128(D == 128 ? from + tid * 128 + ((k ^ (tid & 7)) << 4) : from + tid * 64 + ((k ^ ((tid >> 1) & 3)) << 4));
              uint32_t w[8] = {f16x2_of_e4m3(u.x), f16x2_of_e4m3_high(u.x), f16x2_of_e4m3(u.y), f16x2_of_e4m3_high(u.y),
                               f16x2_of_e4m3(u.z), f16x2_of_e4m3_high(u.z), f16x2_of_e4m3(u.w), f16x2_of_e4m3_high(u.w)};
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = value ? mul_f16(w[e], by) : w[e];
              const uint32_t at = row_at + (k >> 2) * (value ? 8192 : kTile * 128);
              const int c16 = (k & 3) * 2;
              sts128(at + ((c16 ^ (tid & 7)) << 4), seen ? make_uint4(w[0], w[1], w[2], w[3]) : make_uint4(0, 0, 0, 0));
              sts128(at + (((c16 + 1) ^ (tid & 7)) << 4), seen ? make_uint4(w[4], w[5], w[6], w[7]) : make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kRawEmpty + rs)), mbar_arrive(bar(kFull + ss));
          }
          k_scale = k_next, v_scale = v_next;
        }
        n_tile += 2u * (uint32_t)(it.to - it.from);
        n_step += (uint32_t)(it.to - it.from);
      }
    }
  } else {
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
      const int tile_token = it.token + t * p.tokens, token = tile_token + row / p.group;
      const bool real = row < p.tokens * p.group && token < it.n;
      const int pos = real ? it.base + token : -1, lo = sight_of(max(pos, 0), p.window, p.sinks).lo;
      // Blocks all of whose keys all of the tile's rows see need no mask.
      const int first_pos = it.base + tile_token;
      const int last_lo = sight_of(max(first_pos + p.tokens - 1, 0), p.window, p.sinks).lo;
      float m = -INFINITY, l = 0.f, row_factor = p.scale_log2, sigma = 0.f;
      bool any = false;
      for (int i = it.from; i < it.to; ++i) {
        if (!st.active(t, i)) continue;
        const int key = st.block(i) * kTile;
        if (!(ok = mbar_wait(bar(kSFull + t), step & 1u, abort_flag, kWaitNs))) break;
        ++step;
        tc_fence_after();
        uint32_t v[4][32];   // the row's scores
#pragma unroll
        for (int e = 0; e < 4; ++e) tmem_ld32(s_at + 32 * e, v[e]);
        // In 8 bits: the keys' scales, and of each 32 values the power of two
        // that they are still to be multiplied with.
        const uint32_t scales = base + C::kOffScale + (E8 ? (n_step + i - it.from) % C::kScaleSlots * C::kScaleBytes : 0);
        if constexpr (E8)
          if (!any) row_factor = p.scale_log2 * __uint_as_float((uint32_t)gbase[C::kOffRow + ((n & 1) * 2 + t) * kTile + row] << 23);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 4; ++e) reg_fence(v[e]);
        if constexpr (E8) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const uint4 by = lds128(scales + (32 * e + k) * 4);
              float a[4];
              halves(mul2(pair_of(v[e][k], v[e][k + 1]), pair_of(by.x, by.y)), a[0], a[1]);
              halves(mul2(pair_of(v[e][k + 2], v[e][k + 3]), pair_of(by.z, by.w)), a[2], a[3]);
#pragma unroll
              for (int j = 0; j < 4; ++j) v[e][k + j] = __float_as_uint(a[j]);
            }
        }
        if (key + kTile - 1 > first_pos || !(key >= last_lo || key + kTile <= p.sinks)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = key + 32 * e;
            const uint32_t seen = low_bits(pos + 1 - at) & (~low_bits(lo - at) | low_bits(p.sinks - at));
            if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(seen >> k & 1u)) v[e][k] = 0xff800000u;   // -infinity
          }
        }
        float top = -INFINITY;
        {
          float tops[8];   // two chains for each 32 keys
#pragma unroll
          for (int k = 0; k < 8; ++k) tops[k] = max3(__uint_as_float(v[k >> 1][2 * (k & 1)]), __uint_as_float(v[k >> 1][2 * (k & 1) + 1]), -INFINITY);
#pragma unroll
          for (int k = 4; k < 32; k += 2)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              tops[2 * e + (k >> 1 & 1)] = max3(tops[2 * e + (k >> 1 & 1)], __uint_as_float(v[e][k]), __uint_as_float(v[e][k + 1]));
          top = max3(max3(tops[0], tops[1], tops[2]), max3(tops[3], tops[4], tops[5]), fmaxf(tops[6], tops[7])) * row_factor;
        }
        float pow2[4];
        float by = 1.f;   // what O is rescaled with
        if (top > m + kLazy || (m == -INFINITY && top > m)) {
          by = ex2_below(m, top);
          l *= by;
          m = top;
        }
        if constexpr (E8) {
          // Weights are kept over sigma, 2^-7 times the largest power of two of
          // the values so far (so they stay below 2^15 in f16); it is one for
          // all rows.
          const uint4 u = lds128(scales + kTile * 4);
          pow2[0] = __uint_as_float(u.x), pow2[1] = __uint_as_float(u.y), pow2[2] = __uint_as_float(u.z), pow2[3] = __uint_as_float(u.w);
          const float mx = fmaxf(fmaxf(pow2[0], pow2[1]), fmaxf(pow2[2], pow2[3])) * 0.0078125f;
          if (mx > sigma) {
            by *= sigma == 0.f ? 0.f : sigma / mx;
            sigma = mx;
          }
        }
        // Weights, over the scores' first 64 columns (the row's scores are in
        // registers), and their sum.
        // (Held back anew each step, which costs up to 1%; kept from when m moves
        // 2%; the difference of scores first, as for few tokens, 4% at D = 64.)
        const float less = held_back<E8>(m);
        const float factor = m == -INFINITY ? row_factor : row_factor * less, down = m == -INFINITY ? 0.f : -m * less;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // In 8 bits what multiplies a value is its weight times its 32's
          // power of two over sigma, which goes into the exponent; the sum is
          // of the weights alone. (Below 2^-60 nothing is left of them in f16.)
          const int lift = E8 ? max((int)(__float_as_uint(pow2[e]) >> 23) - (int)(__float_as_uint(sigma) >> 23), -60) : 0;
          const f32x2 factor2 = pair_of(factor, factor), down2 = pair_of(down + (float)lift, down + (float)lift);
          f32x2 sums[2] = {0ull, 0ull};
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float f[4];
            halves(fma2(pair_of(v[e][k], v[e][k + 1]), factor2, down2), f[0], f[1]);
            halves(fma2(pair_of(v[e][k + 2], v[e][k + 3]), factor2, down2), f[2], f[3]);
#pragma unroll
            for (int a = 0; a < 4; ++a) f[a] = ex2(f[a]);
            sums[0] = add2(sums[0], pair_of(f[0], f[1]));
            sums[1] = add2(sums[1], pair_of(f[2], f[3]));
            w[k / 2] = E8 ? f16x2(f[0], f[1]) : bf16x2(f[0], f[1]);
            w[k / 2 + 1] = E8 ? f16x2(f[2], f[3]) : bf16x2(f[2], f[3]);
          }
          tmem_st16(s_at + 16 * e, w);
          float s0, s1;
          halves(add2(sums[0], sums[1]), s0, s1);
          sum = E8 ? fmaf(s0 + s1, __uint_as_float((uint32_t)(127 - lift) << 23), sum) : sum + (s0 + s1);
        }
        if (any && __any_sync(0xffffffffu, by != 1.f)) {
          // (These scores come after the sums before them in the issuer's
          // order: those are done.) Seldom, so in a loop: see above.
          const f32x2 by2 = pair_of(by, by);
#pragma unroll 1
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
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull + t));
        l += sum;
        any = true;
      }
      if (!ok) break;
      n_step += it.to - it.from;
      // ---- the rows' results
      if (any) {
        if (!mbar_wait(bar(kOFull + t), outs & 1u, abort_flag, kWaitNs)) break;
        ++outs;
        tc_fence_after();
      }
      const int64_t out = it.row + token;
      const int head = it.h * p.group + row % p.group;
      // Half a line of a row (32 columns) at a time, into global memory by way of
      // shared memory: a thread's own row would be 16 bytes of each of 32 rows
      // an access. The loops over columns stay loops: code that runs once an
      // item is fetched each time.
      const long long mine_at = real ? out * p.ld_o + head * D : -1;
      auto store = [&](int e, const uint32_t (&w)[16]) {
        const uint32_t buf = base + C::kOffOut + (warp - 4) * 2048;
#pragma unroll
        for (int k = 0; k < 4; ++k) sts128(buf + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4), make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = k * 8 + (lane >> 2), piece = lane & 3;
          const long long at = __shfl_sync(0xffffffffu, mine_at, r);
          const uint4 u = lds128(buf + r * 64 + ((piece ^ (r >> 1 & 3)) << 4));
          if (at >= 0) *reinterpret_cast<uint4*>(p.o[it.r] + at + e * 32 + piece * 8) = u;
        }
        __syncwarp();
      };
      if (it.parts == 1) {
        const bool none = m == -INFINITY && l == 0.f;   // (O holds nothing then, or zeros)
        const float by = E8 ? sigma / l : 1.f / l;
#pragma unroll 1
        for (int e = 0; e < D / 32; ++e) {
          uint32_t o[32], w[16];
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
          if (any) {
            tmem_ld32(o_at + 32 * e, o);
            tmem_ld_wait();
            reg_fence(o);
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = none ? 0u : bf16x2(__uint_as_float(o[2 * k]) * by, __uint_as_float(o[2 * k + 1]) * by);
          store(e, w);
        }
        if (any) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kOFree + t));
        }
        if (real && p.lse[it.r]) p.lse[it.r][out * p.heads_q + head] = lse_of(m, l);
        continue;
      }
      // A part: four columns of all rows side by side, then maxima and sums.
      constexpr int rows = 2 * kTile;
      const int place = t * kTile + row;
      auto part_of = [&](int i) { return p.part + (int64_t)(it.slot + i) * rows * (D + 2); };
      const int stat = D * rows + place;
      if (any) {
        float4* const to = reinterpret_cast<float4*>(part_of(it.part)) + place;
        const float by = E8 ? sigma : 1.f;
#pragma unroll 1
        for (int e = 0; e < D / 32; ++e) {
          uint32_t o[32];
          tmem_ld32(o_at + 32 * e, o);
          tmem_ld_wait();
          reg_fence(o);
          if (real)
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              to[(8 * e + k / 4) * rows] = make_float4(__uint_as_float(o[k]) * by, __uint_as_float(o[k + 1]) * by,
                                                       __uint_as_float(o[k + 2]) * by, __uint_as_float(o[k + 3]) * by);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kOFree + t));
      }
      if (real) part_of(it.part)[stat] = m, part_of(it.part)[stat + rows] = l;
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

// Parts of a cut pair together, in an order of their own. A lane has a row's 32
// columns. Up to eight parts are one warp's, and a block has the pair's eight
// blocks of rows; more are dealt to a block's eight warps, whose sums meet in
// shared memory. (With eight warps to a row's parts always, chunks of prompts,
// of two or three parts a pair, took 36 us here, not 16; with one warp, the
// parts of 17 contexts of 4100 tokens and 40 rows 18 us, not 9.) Few rows are
// dealt to all warps too: their blocks would be too few.
constexpr int kJoinWays = 8;
static_assert(kJoinWays * 32 == 2 * kTile, "a warp for a block of rows");
template <int D>
__global__ void __launch_bounds__(32 * kJoinWays) prompt_join_kernel(const __grid_constant__ PromptParams p) {
  __shared__ float4 sums[kJoinWays][32][9];
  __shared__ float tops[kJoinWays][32], totals[kJoinWays][32];
  grid_release();
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int rows = 2 * kTile, E = D / 32;
  // (All of them are fewer than kMostParts.)
  const int parts = (int)p.next[2], units = p.R * p.heads_k, all = units * (int)p.next[3], most = all * E * (int)p.next[4];
  const long long step = (long long)rows * (D + 2);
  for (int x = blockIdx.x; x < most; x += gridDim.x) {
    const int y = x % all, z = x / all, e = z % E, u = y % units;
    const Record it = p.cut[y / units];
    const bool split = it.parts > kJoinWays || (it.n - it.token) * p.group <= 2 * 32;
    if (!split && z >= E) continue;
    const int first_row = (split ? z / E : warp) * 32, r = u / p.heads_k, h = u - r * p.heads_k;
    auto token_of = [&](int place) { return it.token + place / kTile * p.tokens + place % kTile / p.group; };
    auto real = [&](int place) { return place % kTile < p.tokens * p.group && token_of(place) < it.n; };
    auto write = [&](int place, int column, const float4& o, float inv) {
      *reinterpret_cast<uint2*>(p.o[r] + ((long long)it.row + token_of(place)) * p.ld_o + (h * p.group + place % kTile % p.group) * D + column) =
          make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
    };
    auto write_lse = [&](int place, float top, float total) {
      if (p.lse[r] && e == 0)
        p.lse[r][((long long)it.row + token_of(place)) * p.heads_q + h * p.group + place % kTile % p.group] = lse_of(top, total);
    };
    if (!real(first_row)) continue;   // (nor any after it)
    const int place = first_row + lane, by = split ? kJoinWays : 1;
    const float* const first = p.part + (int64_t)(u * parts + it.slot) * step;
    float top = -INFINITY, total = 0.f;
    float4 acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (real(place)) {
      const float* const stat = first + D * rows + place;
#pragma unroll 8
      for (int i = split ? warp : 0; i < it.parts; i += by) top = fmaxf(top, stat[i * step]);
#pragma unroll 1
      for (int i0 = split ? warp : 0; i0 < it.parts; i0 += 2 * by) {
        float m[2], l[2];
        float4 v[2][8];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool there = i0 + j * by < it.parts;
          const float* const at = stat + (i0 + j * by) * step;
          m[j] = there ? at[0] : -INFINITY, l[j] = there ? at[rows] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // (A part that was not written is read all the same: the columns are on
          // their way with the sums, not after them.)
          const bool there = i0 + j * by < it.parts;
          const float4* const from = reinterpret_cast<const float4*>(first + (i0 + j * by) * step) + 8 * e * rows + place;
#pragma unroll
          for (int k = 0; k < 8; ++k) v[j][k] = there ? from[k * rows] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float f = ex2_below(m[j], top);
          if (m[j] == -INFINITY && l[j] == 0.f) continue;
          total = fmaf(f, l[j], total);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            acc[k].x = fmaf(f, v[j][k].x, acc[k].x), acc[k].y = fmaf(f, v[j][k].y, acc[k].y);
            acc[k].z = fmaf(f, v[j][k].z, acc[k].z), acc[k].w = fmaf(f, v[j][k].w, acc[k].w);
          }
        }
      }
    }
    if (!split) {
      if (real(place)) {
        const float inv = top == -INFINITY && total == 0.f ? 0.f : 1.f / total;
#pragma unroll
        for (int k = 0; k < 8; ++k) write(place, 32 * e + 4 * k, acc[k], inv);
        write_lse(place, top, total);
      }
      continue;
    }
    __syncthreads();
    tops[warp][lane] = top, totals[warp][lane] = total;
#pragma unroll
    for (int k = 0; k < 8; ++k) sums[warp][lane][k] = acc[k];
    __syncthreads();
    // A thread for four of a row's columns.
    const int mine = threadIdx.x >> 3, quad = threadIdx.x & 7;
    if (real(first_row + mine)) {
      top = -INFINITY, total = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kJoinWays; ++w) top = fmaxf(top, tops[w][mine]);
#pragma unroll
      for (int w = 0; w < kJoinWays; ++w) {
        const float m = tops[w][mine], l = totals[w][mine];
        if (m == -INFINITY && l == 0.f) continue;
        const float f = ex2_below(m, top);
        const float4 v = sums[w][mine][quad];
        total = fmaf(f, l, total);
        o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
      }
      write(first_row + mine, 32 * e + 4 * quad, o, top == -INFINITY && total == 0.f ? 0.f : 1.f / total);
      if (quad == 0) write_lse(first_row + mine, top, total);
    }
  }
}

template <int D, bool E8>
fo_status launch_prompt(PromptParams& k, int sms, cudaStream_t s) {
  using C = Prompt<D, E8>;
  auto kern = prompt_kernel<D, E8>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  fo_status st = launched(e, "paged prompt", k.R, k.batch.rows, D, 0, C::kThreads);
  if (st || (st = launched(launch_after(prompt_plan_kernel, dim3(1), 1024, 0, 0, s, k), "paged prompt plan", k.R, k.batch.rows, D, 1, 1024)))
    return st;
  if ((st = launched(launch_after(kern, dim3(sms), C::kThreads, C::kSmem, 0, s, k), "paged prompt", k.R, k.batch.rows, D, sms, C::kThreads))) return st;
  return launched(launch_after(prompt_join_kernel<D>, dim3(4 * sms), 32 * kJoinWays, 0, 0, s, k), "paged prompt join", k.R, k.batch.rows, D, 4 * sms, 32 * kJoinWays);
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

// Workspace: header, deal, (the other kernel's counters,) pairs before each
// sequence, items, cut pairs, parts.
namespace {
struct PromptPlaces {
  size_t before, items, cut, part, bytes;
  int64_t most_items;
  PromptPlaces(const fo_paged_desc* d, int64_t seqs, int64_t rows) {
    const int tokens = kTile / (d->heads_q / d->heads_k);
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    most_items = rows / (2 * tokens) + seqs + kMostParts;
    before = kScratchAt;
    items = before + up((size_t)(seqs + 1) * 8);
    cut = items + up((size_t)most_items * sizeof(Record));
    part = cut + up((size_t)kMostParts * sizeof(Record));
    bytes = part + (size_t)kMostParts * 2 * kTile * (d->head_dim + 2) * 4;
  }
};
}  // namespace
size_t prompt_bytes(const fo_paged_desc* d, int32_t seqs, int64_t rows) {
  return PromptPlaces(d, seqs, rows).bytes;
}

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
  k.least_exponent = least_exponent(c.scale_log2);
  const PromptPlaces at(d, c.b->seqs, c.rows);
  k.sms = std::min(c.sms, FO_GB300_SMS);
  k.next = reinterpret_cast<uint32_t*>(c.ws + 128);
  k.cut = reinterpret_cast<Record*>(c.ws + at.cut);
  k.before = reinterpret_cast<int64_t*>(c.ws + at.before);
  k.items = reinterpret_cast<Record*>(c.ws + at.items);
  k.most_items = at.most_items;
  k.part = reinterpret_cast<float*>(c.ws + at.part);
  if (d->head_dim == 128) return eight ? launch_prompt<128, true>(k, c.sms, s) : launch_prompt<128, false>(k, c.sms, s);
  return eight ? launch_prompt<64, true>(k, c.sms, s) : launch_prompt<64, false>(k, c.sms, s);
}

}  // namespace fo_ops
