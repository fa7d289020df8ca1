// New tokens' keys and values into a paged cache, turned by their rotary
// positions on the way, and their queries turned. Bandwidth-bound: each value
// is read once and written once.
#include <math.h>
#include <string.h>

#include "fo_paged.h"

namespace fo_ops {
namespace {

struct AppendParams {
  const __nv_bfloat16* in[3][kMaxR];
  __nv_bfloat16* q_out[kMaxR];
  void* cache[2][kMaxR];
  float* scale[2][kMaxR];
  int64_t ld[4];
  const void* positions;
  int32_t pos_bytes;
  Batch batch;
  int32_t heads_q, heads_k, D, rot, half, eight;
  float factor;
  uint64_t turns[64];
};

// The sequence of a row: the last one that starts at or before it.
__device__ __forceinline__ int sequence_of(const Batch& b, int row) {
  if (!b.starts) return row < b.seqs ? row : -1;
  if (row < b.starts[0] || row >= b.starts[b.seqs]) return -1;
  int lo = 0, hi = b.seqs;   // starts[lo] <= row < starts[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (b.starts[mid] <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float2 cs[64];
  grid_release();
  grid_wait();
  const int row = blockIdx.x, r = blockIdx.y;
  const int b = sequence_of(p.batch, row);
  if (b < 0) return;
  const Seq s = sequence(p.batch, b);
  const int i = row - s.row;
  if (i < 0 || i >= s.n) return;
  const int pos = s.base + i;
  int page = -1;
  if (pos >= 0) {
    page = p.batch.table[(int64_t)b * p.batch.cols + (pos >> p.batch.shift)];
    if (page < 0 || page >= p.batch.pages) {
      if (threadIdx.x == 0) report(p.batch, b, kBadPage, page);
      page = -1;
    }
  }
  if (threadIdx.x < p.rot / 2) {
    const int64_t at = !p.positions        ? pos
                       : p.pos_bytes == 8 ? static_cast<const int64_t*>(p.positions)[row]
                                          : (int64_t) static_cast<const int32_t*>(p.positions)[row];
    float sn, c;
    sincospif((float)(int64_t)((uint64_t)at * p.turns[threadIdx.x]) * 1.08420217e-19f, &sn, &c);   // 2^-63: half turns
    cs[threadIdx.x] = make_float2(c * p.factor, sn * p.factor);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, all = p.heads_q + 2 * p.heads_k, pairs = p.rot / 2;
  for (int h = threadIdx.x >> 5; h < all; h += 8) {
    const int part = h < p.heads_q ? 0 : h < p.heads_q + p.heads_k ? 1 : 2;
    const int head = part == 0 ? h : part == 1 ? h - p.heads_q : h - p.heads_q - p.heads_k;
    if (part && page < 0) continue;
    const __nv_bfloat16* x = p.in[part][r] + row * p.ld[part] + head * p.D;
    float v[4];
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = lane + 32 * k;
      v[k] = 0.f;
      if (e >= p.D) continue;
      v[k] = to_f(x[e]);
      if (part < 2 && e < p.rot) {
        const int pair = p.half ? (e < pairs ? e : e - pairs) : e / 2;
        const bool second = p.half ? e >= pairs : e & 1;
        const int other = p.half ? (second ? e - pairs : e + pairs) : e ^ 1;
        const float w = to_f(x[other]);
        v[k] = second ? v[k] * cs[pair].x + w * cs[pair].y : v[k] * cs[pair].x - w * cs[pair].y;
      }
      top = max_nan(top, fabsf(v[k]));
    }
    __syncwarp();   // (in place: all of the head is read before it is written)
    const int64_t slot = ((int64_t)page * p.heads_k + head << p.batch.shift) + (pos & ((1 << p.batch.shift) - 1));
    if (part && p.eight) {
      const float scale = scale_of(lanes_max<32>(top));
      if (lane == 0) p.scale[part - 1][r][slot] = scale;
      divide_by(scale, v);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = lane + 32 * k;
      if (e >= p.D) continue;
      if (part == 0)
        from_f(v[k], p.q_out[r][row * p.ld[3] + head * p.D + e]);
      else if (p.eight)
        static_cast<uint8_t*>(p.cache[part - 1][r])[slot * p.D + e] = (uint8_t)e4m3x2(v[k], 0.f);
      else
        from_f(v[k], static_cast<__nv_bfloat16*>(p.cache[part - 1][r])[slot * p.D + e]);
    }
  }
}

}  // namespace

fo_status check_paged(const fo_paged_desc* d) {
  if (!d || d->R < 1 || d->R > FO_MAX_R || d->reserved[0] || d->reserved[1] || d->reserved[2]) return FO_ERR_INVALID_ARG;
  if (d->heads_k < 1 || d->heads_q < 1 || d->heads_q > 65536 || d->heads_q % d->heads_k ||
      d->heads_q / d->heads_k > FO_PAGED_MAX_GROUP)
    return FO_ERR_SHAPE;
  if (d->head_dim != 64 && d->head_dim != 128) return FO_ERR_SHAPE;
  if (d->page < 16 || d->page > 256 || (d->page & (d->page - 1))) return FO_ERR_SHAPE;
  if (d->cache_dtype != FO_CACHE_BF16 && d->cache_dtype != FO_CACHE_E4M3) return FO_ERR_DTYPE;
  if (d->window < 0 || d->sinks < 0) return FO_ERR_INVALID_ARG;
  if (!(d->scale >= 0.f) || !isfinite(d->scale)) return FO_ERR_INVALID_ARG;
  return FO_OK;
}

fo_status check_batch(const fo_paged_desc* d, const fo_paged_batch* b, int64_t rows) {
  if (!b) return FO_ERR_INVALID_ARG;
  if (rows < 0 || rows > INT32_MAX || b->seqs < 0 || b->max_new < 1) return FO_ERR_SHAPE;
  if (b->pages < 1 || b->pages > INT32_MAX / d->heads_k || b->table_cols < 1 || b->table_cols > INT32_MAX / d->page)
    return FO_ERR_SHAPE;
  if (!b->starts && (b->max_new != 1 || b->seqs > rows)) return FO_ERR_SHAPE;
  if ((int64_t)b->seqs * d->R * d->heads_k > INT32_MAX) return FO_ERR_SHAPE;
  if (b->seqs && rows) {
    if (!b->lengths || !b->table) return FO_ERR_INVALID_ARG;
    if (!aligned(b->lengths, 4) || !aligned(b->starts, 4) || !aligned(b->table, 4)) return FO_ERR_ALIGN;
  }
  return FO_OK;
}

Batch batch_of(const fo_paged_desc* d, const fo_paged_batch* b, int64_t rows, void* ws) {
  Batch k;
  k.lengths = b->lengths;
  k.starts = b->starts;
  k.table = b->table;
  k.cols = b->table_cols;
  k.seqs = b->seqs;
  k.rows = (int32_t)rows;
  k.max_new = b->max_new;
  k.pages = (int32_t)b->pages;
  for (k.shift = 4; 1 << k.shift < d->page; ++k.shift) {
  }
  k.status = static_cast<int32_t*>(ws);
  return k;
}

}  // namespace fo_ops

extern "C" fo_status fo_kv_append(const fo_paged_desc* d, const fo_rope_desc* rope, const fo_paged_batch* b, int64_t rows,
                                  const void* positions, int32_t pos_bytes, const void* const* q, const void* const* k,
                                  const void* const* v, void* const* q_out, const int64_t ld[4], void* const* k_cache,
                                  void* const* v_cache, float* const* k_scale, float* const* v_scale, void* ws,
                                  fo_stream_t stream) {
  using namespace fo_ops;
  fo_status st = check_paged(d);
  if (st || (st = check_batch(d, b, rows))) return st;
  if (rope && ((st = check_rope_desc(rope)) || rope->ready != 1)) return st ? st : FO_ERR_INVALID_ARG;
  if (rope && (rope->R != d->R || rope->heads_q != d->heads_q || rope->heads_k != d->heads_k ||
               rope->heads_v != d->heads_k || rope->head_dim != d->head_dim || rope->dtype != FO_BF16))
    return FO_ERR_INVALID_ARG;
  if (!ld || (positions && pos_bytes != 4 && pos_bytes != 8)) return FO_ERR_INVALID_ARG;
  const bool eight = d->cache_dtype == FO_CACHE_E4M3;
  if (!eight && (k_scale || v_scale)) return FO_ERR_INVALID_ARG;
  const int64_t wide_q = (int64_t)d->heads_q * d->head_dim, wide_k = (int64_t)d->heads_k * d->head_dim;
  if (ld[0] < wide_q || ld[1] < wide_k || ld[2] < wide_k || ld[3] < wide_q) return FO_ERR_SHAPE;
  if (positions && !aligned(positions, pos_bytes)) return FO_ERR_ALIGN;
  if (ws && !aligned(ws, 16)) return FO_ERR_ALIGN;
  if (rows == 0 || b->seqs == 0) return FO_OK;
  typedef const void* const* A;
  const int R = d->R;
  if ((st = check_array(R, q, 2)) || (st = check_array(R, k, 2)) || (st = check_array(R, v, 2)) ||
      (st = check_array(R, (A)q_out, 2)) || (st = check_array(R, (A)k_cache, 16)) || (st = check_array(R, (A)v_cache, 16)))
    return st;
  if (eight && ((st = check_array(R, (A)k_scale, 16)) || (st = check_array(R, (A)v_scale, 16)))) return st;
  int sms;
  if ((st = device_sms(&sms))) return st;
  PtrList l;
  l.add(R, q), l.add(R, k), l.add(R, v), l.add(R, (A)q_out), l.add(R, (A)k_cache), l.add(R, (A)v_cache);
  if (eight) l.add(R, (A)k_scale), l.add(R, (A)v_scale);
  l.add(positions), l.add(b->lengths), l.add(b->starts), l.add(b->table), l.add(ws);
  if ((st = check_device(l, stream))) return st;
  AppendParams p;
  memset(&p, 0, sizeof(p));
  for (int r = 0; r < R; ++r) {
    p.in[0][r] = static_cast<const __nv_bfloat16*>(q[r]);
    p.in[1][r] = static_cast<const __nv_bfloat16*>(k[r]);
    p.in[2][r] = static_cast<const __nv_bfloat16*>(v[r]);
    p.q_out[r] = static_cast<__nv_bfloat16*>(q_out[r]);
    p.cache[0][r] = k_cache[r];
    p.cache[1][r] = v_cache[r];
    p.scale[0][r] = eight ? k_scale[r] : nullptr;
    p.scale[1][r] = eight ? v_scale[r] : nullptr;
  }
  memcpy(p.ld, ld, sizeof(p.ld));
  p.positions = positions;
  p.pos_bytes = pos_bytes;
  p.batch = batch_of(d, b, rows, ws);
  p.heads_q = d->heads_q;
  p.heads_k = d->heads_k;
  p.D = d->head_dim;
  p.eight = eight;
  if (rope) {
    p.rot = rope->rot_dim;
    p.half = rope->layout == FO_ROPE_HALF;
    p.factor = rope->factor;
    memcpy(p.turns, rope->turns, sizeof(p.turns));
  }
  const dim3 grid((unsigned)rows, R);
  return launched(launch_after(append_kernel, grid, 256, 0, 0, (cudaStream_t)stream, p), "kv append", R, rows, d->head_dim,
                  (int)rows, 256);
}
