// New tokens' keys and values into a paged cache, turned by their rotary
// positions on the way, and their queries turned. Bandwidth-bound: each value
// is read once and written once.
#include <math.h>
#include <string.h>

#include <algorithm>

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
  int32_t heads[3];   // of q, k and v
  int32_t D, rot, half, eight, R;
  int32_t heads_each, ranks_each;   // that a thread goes through
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

// Where a row's token goes.
struct Place {
  int pos;       // in its sequence
  int page, at;  // page (-1: it is not kept) and place in it
};
// False for a row that no sequence has.
__device__ __forceinline__ bool place_of(const Batch& batch, int row, bool tell, Place* to) {
  const int b = sequence_of(batch, row);
  if (b < 0) return false;
  const Seq s = sequence(batch, b);
  const int i = row - s.row;
  if (i < 0 || i >= s.n) return false;
  to->pos = s.base + i;
  to->page = -1;
  to->at = to->pos & ((1 << batch.shift) - 1);
  if (to->pos >= 0) {
    to->page = batch.table[(int64_t)b * batch.cols + (to->pos >> batch.shift)];
    if (to->page < 0 || to->page >= batch.pages) {
      if (tell) report(batch, b, kBadPage, to->page);
      to->page = -1;
    }
  }
  return true;
}
// cos and sin (times the factor) of a pair at a position, as fo_rope has them.
__device__ __forceinline__ float2 turn_of(const AppendParams& p, int row, int pos, uint64_t turns) {
  const int64_t at = !p.positions        ? pos
                     : p.pos_bytes == 8 ? static_cast<const int64_t*>(p.positions)[row]
                                        : (int64_t) static_cast<const int32_t*>(p.positions)[row];
  float s, c;
  sincospif((float)(int64_t)((uint64_t)at * turns) * 1.08420217e-19f, &s, &c);   // 2^-63: half turns
  return make_float2(c * p.factor, s * p.factor);
}

// A pair turned, with fo_rope's roundings.
__device__ __forceinline__ float2 turn_pair(float u, float w, float c, float s) {
  return make_float2(fmaf(u, c, -(w * s)), fmaf(w, c, u * s));
}

// Rows, heads and halves on the 16-byte grid. A thread has a token and two
// pieces of eight elements in every head: in the half layout those that are
// turned together, else neighbours' (the threads beyond the turned pieces copy
// the rest). It computes its angles once and goes through its share of the
// heads, four at a time with all loads first; a head's lanes are neighbours,
// so its largest magnitude takes two or three shuffles.
// Bandwidth-bound: 8192 tokens of 8 ranks with 4 + 4 + 4 heads (403 MB) take
// 63 us, 6.4 TB/s, element by element (below) 321; 5015 tokens of 32 + 8 + 8
// heads into 8 bits (113 MB) 26.5 us, element by element 80.
template <bool HALF, bool E8, bool RANKS>
__global__ void __launch_bounds__(256, 3) append_wide_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kHeads = 4, V = 8;
  __shared__ uint64_t turns[64];   // (lane by lane from the parameters each would be an access of its own)
  if (threadIdx.x < p.rot / 2) turns[threadIdx.x] = p.turns[threadIdx.x];
  __syncthreads();
  grid_release();
  grid_wait();
  const int whole = p.D / V, lanes = whole / 2, tok = threadIdx.x / lanes, i = threadIdx.x - tok * lanes;
  const int64_t row64 = (int64_t)blockIdx.x * (256 / lanes) + tok;
  Place place;
  if (row64 >= p.batch.rows || !place_of(p.batch, (int)row64, i == 0, &place)) return;
  const int row = (int)row64;
  // The token's lanes: they go the same way, others of the warp may not.
  const uint32_t together = ((1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
  const int pieces = p.rot / V / (HALF ? 2 : 1);   // of the first half; of all that is turned
  const bool turn_a = i < pieces, turn_b = HALF ? turn_a : i + lanes < pieces;
  const int a = !HALF || turn_a ? i : i + pieces, b = !HALF ? i + lanes : turn_a ? i + pieces : i + lanes;
  float c[V], s[V];   // HALF: by element; else the first four for piece a, the others for b
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int pair = HALF ? i * V + j : j < V / 2 ? a * (V / 2) + j : b * (V / 2) + j - V / 2;
    const float2 cs = 2 * pair < p.rot ? turn_of(p, row, place.pos, turns[pair]) : make_float2(0.f, 0.f);
    c[j] = cs.x, s[j] = cs.y;
  }
  const int first_r = RANKS ? (int)blockIdx.z * p.ranks_each : (int)blockIdx.z;
  const int last_r = RANKS ? min(p.R, first_r + p.ranks_each) : first_r + 1;
  for (int r = first_r; RANKS ? r < last_r : r == first_r; ++r) {
    int h0 = (int)blockIdx.y * p.heads_each, h1 = h0 + p.heads_each;   // this block's heads, counted from each part's first
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      const int first = max(h0, 0), last = min(h1, p.heads[part]);
      h0 -= p.heads[part], h1 -= p.heads[part];
      if (first >= last || (part && place.page < 0)) continue;
      const int pa = (part < 2 ? a : i) * V, pb = (part < 2 ? b : i + lanes) * V;
      const __nv_bfloat16* in = p.in[part][r] + row * p.ld[part] + first * p.D;
      // Elements from one head to the next where it goes to.
      const int64_t step = part ? (int64_t)p.D << p.batch.shift : p.D;
      const int64_t slot = ((int64_t)place.page * p.heads[1] + first << p.batch.shift) + place.at;
      __nv_bfloat16* out = part ? static_cast<__nv_bfloat16*>(p.cache[part - 1][r]) + slot * p.D
                                : p.q_out[r] + row * p.ld[3] + first * p.D;
      uint8_t* out8 = part ? static_cast<uint8_t*>(p.cache[part - 1][r]) + slot * p.D : nullptr;
      float* scale = part && E8 ? p.scale[part - 1][r] + slot : nullptr;
      for (int n = last - first; n > 0; n -= kHeads, in += kHeads * p.D) {
        uint4 x[kHeads], y[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
          if (k < n) {
            x[k] = *reinterpret_cast<const uint4*>(in + k * p.D + pa);
            y[k] = *reinterpret_cast<const uint4*>(in + k * p.D + pb);
          }
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
          if (k < n) {
            const bool eight = part && E8, turned = part < 2;
            if (eight || (turned && (turn_a || turn_b))) {
              float u[V], w[V];
              Vec16<__nv_bfloat16>::unpack(x[k], u);
              Vec16<__nv_bfloat16>::unpack(y[k], w);
              if (turned) {
                if constexpr (HALF) {
                  if (turn_a) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                      const float2 z = turn_pair(u[j], w[j], c[j], s[j]);
                      u[j] = z.x, w[j] = z.y;
                    }
                  }
                } else {
                  auto turn = [&](float (&z)[V], int at) {
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) {
                      const float2 y = turn_pair(z[2 * j], z[2 * j + 1], c[at + j], s[at + j]);
                      z[2 * j] = y.x, z[2 * j + 1] = y.y;
                    }
                  };
                  if (turn_a) turn(u, 0);
                  if (turn_b) turn(w, V / 2);
                }
              }
              if (eight) {
                float top = max_nan(amax_of(u), amax_of(w));
                for (int o = lanes / 2; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(together, top, o));
                const float by = scale_of(top);
                if (i == 0) scale[(int64_t)k << p.batch.shift] = by;
                divide_by(by, u);
                divide_by(by, w);
                *reinterpret_cast<uint2*>(out8 + k * step + pa) = make_uint2(e4m3x4(u[0], u[1], u[2], u[3]), e4m3x4(u[4], u[5], u[6], u[7]));
                *reinterpret_cast<uint2*>(out8 + k * step + pb) = make_uint2(e4m3x4(w[0], w[1], w[2], w[3]), e4m3x4(w[4], w[5], w[6], w[7]));
                continue;
              }
              x[k] = Vec16<__nv_bfloat16>::pack(u);
              y[k] = Vec16<__nv_bfloat16>::pack(w);
            }
            *reinterpret_cast<uint4*>(out + k * step + pa) = x[k];
            *reinterpret_cast<uint4*>(out + k * step + pb) = y[k];
          }
        if (part && E8) out8 += kHeads * step, scale += (int64_t)kHeads << p.batch.shift;
        else out += kHeads * step;
      }
    }
  }
}

// Rows, heads or halves that are not on that grid: a block for a row and rank,
// a warp for a head, element by element.
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float2 cs[64];
  grid_release();
  grid_wait();
  const int row = blockIdx.x, r = blockIdx.y;
  Place place;
  if (!place_of(p.batch, row, threadIdx.x == 0, &place)) return;
  const int page = place.page, pos = place.pos;
  if (threadIdx.x < p.rot / 2) cs[threadIdx.x] = turn_of(p, row, pos, p.turns[threadIdx.x]);
  __syncthreads();
  const int lane = threadIdx.x & 31, all = p.heads[0] + 2 * p.heads[1], pairs = p.rot / 2;
  for (int h = threadIdx.x >> 5; h < all; h += 8) {
    const int part = h < p.heads[0] ? 0 : h < p.heads[0] + p.heads[1] ? 1 : 2;
    const int head = part == 0 ? h : part == 1 ? h - p.heads[0] : h - p.heads[0] - p.heads[1];
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
        v[k] = second ? turn_pair(w, v[k], cs[pair].x, cs[pair].y).y : turn_pair(v[k], w, cs[pair].x, cs[pair].y).x;
      }
      top = max_nan(top, fabsf(v[k]));
    }
    __syncwarp();   // (in place: all of the head is read before it is written)
    const int64_t slot = ((int64_t)page * p.heads[1] + head << p.batch.shift) + place.at;
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
  if (!(d->scale >= 0.f) || !isfinite(d->scale * 1.4426950408889634f)) return FO_ERR_INVALID_ARG;   // (in base 2, as it is used)
  return FO_OK;
}

fo_status check_batch(const fo_paged_desc* d, const fo_paged_batch* b, int64_t rows) {
  if (!b) return FO_ERR_INVALID_ARG;
  if (rows < 0 || rows > INT32_MAX || b->seqs < 0 || b->max_new < 1) return FO_ERR_SHAPE;
  if (b->pages < 1 || b->pages > INT32_MAX / d->heads_k || b->table_cols < 1 || b->table_cols > (1 << 30) / d->page)
    return FO_ERR_SHAPE;   // (positions, and a tile beyond them, are 32-bit numbers)
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
  p.heads[0] = d->heads_q;
  p.heads[1] = p.heads[2] = d->heads_k;
  p.R = R;
  p.D = d->head_dim;
  p.eight = eight;
  if (rope) {
    p.rot = rope->rot_dim;
    p.half = rope->layout == FO_ROPE_HALF;
    p.factor = rope->factor;
    memcpy(p.turns, rope->turns, sizeof(p.turns));
  }
  const cudaStream_t at = (cudaStream_t)stream;
  bool wide = p.rot % (p.half ? 16 : 8) == 0 && all_aligned(R, q, 16) && all_aligned(R, k, 16) && all_aligned(R, v, 16) &&
              all_aligned(R, (A)q_out, 16);
  for (int j = 0; j < 4; ++j) wide = wide && ld[j] % 8 == 0;
  if (!wide) {
    const dim3 grid((unsigned)rows, R);
    return launched(launch_after(append_kernel, grid, 256, 0, 0, at, p), "kv append, by elements", R, rows, d->head_dim, (int)rows, 256);
  }
  // Heads for a thread: all of a rank's, unless that leaves the GPU short of
  // threads; with few heads a rank, those of several ranks, so that at least 8
  // share the angles (which take as long as four heads).
  const int all = p.heads[0] + 2 * p.heads[1], tokens = 256 / (p.D / 16);
  const int64_t blocks = (rows + tokens - 1) / tokens, enough = 4 * FO_GB300_SMS;
  p.ranks_each = 1;
  while (p.ranks_each < R && p.ranks_each * all < 8 && blocks * R >= enough * p.ranks_each) p.ranks_each *= 2;
  const int64_t cuts = std::min<int64_t>((enough + blocks * R - 1) / (blocks * R), (all + 3) / 4);
  p.heads_each = (int)((all + cuts - 1) / cuts);
  const dim3 grid((unsigned)blocks, (unsigned)((all + p.heads_each - 1) / p.heads_each), (unsigned)((R + p.ranks_each - 1) / p.ranks_each));
  const bool several = p.ranks_each > 1;
  auto kern = p.half ? (eight ? (several ? append_wide_kernel<true, true, true> : append_wide_kernel<true, true, false>)
                              : (several ? append_wide_kernel<true, false, true> : append_wide_kernel<true, false, false>))
                     : (eight ? (several ? append_wide_kernel<false, true, true> : append_wide_kernel<false, true, false>)
                              : (several ? append_wide_kernel<false, false, true> : append_wide_kernel<false, false, false>));
  return launched(launch_after(kern, grid, 256, 0, 0, at, p), "kv append", R, rows, d->head_dim, grid.x * grid.y * grid.z, 256);
}
