// Attention of a batch's new tokens over a paged cache of keys and values.
#include <math.h>
#include <string.h>

#include "fo_paged.h"

namespace fo_ops {
namespace {

struct PagedParams {
  const __nv_bfloat16* q[kMaxR];
  const void* k[kMaxR];
  const void* v[kMaxR];
  const float* ks[kMaxR];
  const float* vs[kMaxR];
  __nv_bfloat16* o[kMaxR];
  float* lse[kMaxR];
  int64_t ld_q, ld_o;
  Batch batch;
  int32_t heads_q, heads_k, group, D, eight, window, sinks;
  float scale;
};

// A warp for a row's head: key by key, the head's values over the lanes.
__global__ void __launch_bounds__(128) row_kernel(const __grid_constant__ PagedParams p) {
  grid_release();
  grid_wait();
  const int lane = threadIdx.x & 31, h = blockIdx.y * 4 + (threadIdx.x >> 5), r = blockIdx.z;
  if (h >= p.heads_q) return;
  const int each = p.D / 32, mask = (1 << p.batch.shift) - 1;
  for (int b = blockIdx.x; b < p.batch.seqs; b += gridDim.x) {
    const Seq s = sequence(p.batch, b);
    if (s.n > p.batch.max_new) report(p.batch, b, kBadCount, s.n);
    for (int i = 0; i < min(s.n, p.batch.max_new); ++i) {
      const int64_t row = s.row + i;
      const int pos = s.base() + i;
      const Sight see = sight_of(pos, p.window, p.sinks);
      float q[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
      for (int k = 0; k < each; ++k) q[k] = to_f(p.q[r][row * p.ld_q + h * p.D + lane + 32 * k]) * p.scale;
      for (int j = 0; j <= pos; ++j) {
        if (j >= see.sinks_end && j < see.lo) j = see.lo;
        const int page = p.batch.table[(int64_t)b * p.batch.cols + (j >> p.batch.shift)];
        if (page < 0 || page >= p.batch.pages) {
          report(p.batch, b, kBadPage, page);
          continue;
        }
        const int64_t slot = ((int64_t)page * p.heads_k + h / p.group << p.batch.shift) + (j & mask);
        float kv[2][4];
        for (int c = 0; c < 2; ++c) {
          const void* base = c ? p.v[r] : p.k[r];
          const float scale = p.eight ? (c ? p.vs[r] : p.ks[r])[slot] : 1.f;
          for (int k = 0; k < each; ++k) {
            const int64_t at = slot * p.D + lane + 32 * k;
            kv[c][k] = p.eight ? (float)static_cast<const __nv_fp8_e4m3*>(base)[at] * scale
                               : to_f(static_cast<const __nv_bfloat16*>(base)[at]);
          }
        }
        float d = 0.f;
        for (int k = 0; k < each; ++k) d = fmaf(q[k], kv[0][k], d);
        d = warp_sum(d);
        const float top = fmaxf(m, d), keep = m == -INFINITY ? 0.f : expf(m - top), w = expf(d - top);
        m = top;
        l = l * keep + w;
        for (int k = 0; k < each; ++k) acc[k] = fmaf(w, kv[1][k], acc[k] * keep);
      }
      for (int k = 0; k < each; ++k)
        from_f(m == -INFINITY ? 0.f : acc[k] / l, p.o[r][row * p.ld_o + h * p.D + lane + 32 * k]);
      if (p.lse[r] && lane == 0) p.lse[r][row * p.heads_q + h] = m == -INFINITY ? -INFINITY : m + logf(l);
    }
  }
}

}  // namespace
}  // namespace fo_ops

extern "C" fo_status fo_paged_attention_workspace(const fo_paged_desc* d, int32_t seqs, int64_t rows, int32_t max_new,
                                                  size_t* bytes) {
  const fo_status st = fo_ops::check_paged(d);
  if (st) return st;
  if (!bytes) return FO_ERR_INVALID_ARG;
  if (seqs < 0 || rows < 0 || rows > INT32_MAX || max_new < 1) return FO_ERR_SHAPE;
  *bytes = sizeof(fo_ws_header);
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
  PagedParams p;
  memset(&p, 0, sizeof(p));
  for (int r = 0; r < R; ++r) {
    p.q[r] = static_cast<const __nv_bfloat16*>(q[r]);
    p.k[r] = k_cache[r];
    p.v[r] = v_cache[r];
    p.ks[r] = eight ? k_scale[r] : nullptr;
    p.vs[r] = eight ? v_scale[r] : nullptr;
    p.o[r] = static_cast<__nv_bfloat16*>(o[r]);
    p.lse[r] = lse ? lse[r] : nullptr;
  }
  p.ld_q = ld[0];
  p.ld_o = ld[1];
  p.batch = batch_of(d, b, rows, ws);
  p.heads_q = d->heads_q;
  p.heads_k = d->heads_k;
  p.group = d->heads_q / d->heads_k;
  p.D = d->head_dim;
  p.eight = eight;
  p.window = d->window;
  p.sinks = d->sinks;
  p.scale = d->scale > 0.f ? d->scale : (float)(1.0 / sqrt((double)d->head_dim));
  const dim3 grid(b->seqs, (d->heads_q + 3) / 4, R);
  return launched(launch_after(row_kernel, grid, 128, 0, 0, (cudaStream_t)stream, p), "paged attention", R, rows, wide,
                  b->seqs, 128);
}
