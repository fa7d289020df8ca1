// What the operators on a paged cache share: host checks, the kernels' view of
// a batch, and who sees whom.
#pragma once

#include <math.h>

#include <algorithm>

#include "fo_device.cuh"
#include "fo_ops.h"

namespace fo_ops {

// A call's sequences as kernels see them.
struct Batch {
  const int32_t* lengths;
  const int32_t* starts;
  const int32_t* table;
  int64_t cols;        // entries of a row of the table
  int32_t seqs, rows, max_new;
  int32_t pages;
  int32_t shift;       // log2 of the page's tokens
  int32_t* status;     // workspace's status word, or NULL
};

// One sequence: its first row, its new tokens (0 where there is nothing to
// do), the first one's position, and the end of what the last one sees.
struct Seq {
  int32_t row, n, base, end;
};

enum : int32_t { kBadPage = 1, kBadCount = 2, kBadStarts = 3, kBadLength = 4 };

__device__ __forceinline__ void report(const Batch& b, int seq, int what, int value) {
  if (b.status) fo::record_error(b.status, FO_ERR_SHAPE, seq, what, value);
}

// Sequence `seq` of the batch, checked: rows lie within the call's, positions
// within the table's row.
__device__ __forceinline__ Seq sequence(const Batch& b, int seq) {
  Seq s;
  const int32_t len = max(b.lengths[seq], 0);
  s.row = seq;
  s.n = 1;
  if (b.starts) {
    const int32_t first = b.starts[seq], last = b.starts[seq + 1];
    s.row = first;
    s.n = last - first;
    if (first < 0 || last < first || last > b.rows) {
      report(b, seq, kBadStarts, last);
      s.row = s.n = 0;
    }
  }
  if ((int64_t)len > b.cols << b.shift) {
    report(b, seq, kBadLength, len);
    s.n = 0;
  }
  s.base = len - s.n;
  if (s.n > b.max_new) {
    report(b, seq, kBadCount, s.n);
    s.n = b.max_new;
  }
  s.end = max(s.base + s.n, 0);
  return s;
}

// Tokens that a row at position p sees: those below `sinks_end` and those in
// [lo, p]; the two do not overlap.
struct Sight {
  int32_t lo, sinks_end;
};
__device__ __forceinline__ Sight sight_of(int p, int window, int sinks) {
  Sight s;
  s.lo = window && p >= window ? p - window + 1 : 0;
  s.sinks_end = min(sinks, s.lo);
  return s;
}

// Host side (fo_kv_append.cu).
fo_status check_paged(const fo_paged_desc* d);
fo_status check_batch(const fo_paged_desc* d, const fo_paged_batch* b, int64_t rows);
Batch batch_of(const fo_paged_desc* d, const fo_paged_batch* b, int64_t rows, void* ws);

// Workspace: header and deal (256 bytes), then the counters of few tokens'
// kernel, zero between calls, then scratch that either kind of call uses.
constexpr int kFewThreads = 256, kFewBlocks = 2;   // blocks an SM
constexpr int kMostParts = 4 * FO_GB300_SMS;       // of the prompts' kernel
constexpr size_t kFewCountBytes = (kFewBlocks * FO_GB300_SMS * 3 * 4 + 255) / 256 * 256;
constexpr size_t kScratchAt = 256 + kFewCountBytes;

// With an 8-bit cache a query's row is multiplied by 2^(134 - e), e the exponent
// of its largest magnitude, and its scores by scale_log2 over that. The least e,
// taken for rows of smaller ones (zeros, say): it leaves that factor a normal
// number. Were it zero, a hidden key's -infinity would become NaN. Elements that
// f16 then rounds, by up to 2^-25, change a score of keys below 2^25 by less
// than 2^-110.
inline uint32_t least_exponent(float scale_log2) { return (uint32_t)std::max(8, 8 - ilogbf(scale_log2)); }

// A checked call of fo_paged_attention.
struct PagedCall {
  const fo_paged_desc* d;
  const fo_paged_batch* b;
  int64_t rows;
  const int64_t* ld;
  const void *const *q, *const *k, *const *v;
  const float *const *ks, *const *vs;
  void* const* o;
  float* const* lse;
  uint8_t* ws;
  float scale_log2;
  int sms;
};
// Few new tokens a sequence (fo_paged_few.cu): up to 8 or 16 rows of a key head.
constexpr int few_keys(bool eight) { return eight ? 64 : 32; }   // of a warp's, of a tile
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
  int32_t box;            // tokens of a box: a page's, or a tile's
  int32_t boxes_log2;     // of a tile
  float scale_log2;
  uint32_t least_exponent;
  float* part;            // [blocks][2][8 or 16 * (D + 2)]
  uint32_t* count;        // [blocks][3], zero between calls
};

fo_status attend_few(FewParams& k, int D, bool wide, bool eight, int sms, cudaStream_t s);   // wide: more than 8 rows
// Many new tokens a sequence (fo_paged_prompt.cu).
fo_status attend_prompts(const PagedCall& c, cudaStream_t s);
size_t prompt_bytes(const fo_paged_desc* d, int32_t seqs, int64_t rows);
// Tensor maps (fo_paged_prompt.cu): pages of keys or values as [pages *
// heads_k][page][D], in boxes of at most 128 bytes x `box` tokens, swizzled by
// their own width; bf16 rows as [rows][heads][D], in boxes of 64 x heads x rows.
bool encode_pages(CUtensorMap* m, const void* p, const fo_paged_desc* d, int64_t pages, int box);
bool encode_rows(CUtensorMap* m, const void* p, int64_t rows, int64_t ld, int heads, int D, int box_heads, int box_rows);

}  // namespace fo_ops
