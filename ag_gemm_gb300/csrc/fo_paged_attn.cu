// Attention of a batch's new tokens over a paged cache of keys and values: the
// calls. The kernels are in fo_paged_few.cu and fo_paged_prompt.cu.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "fo_paged.h"

namespace fo_ops {
namespace {

// Rows of a key head (new tokens x heads of its group) that the split kernel
// takes. More are the prompts' kernel's, whose tiles have 128: 17 contexts of
// up to 4100 on two ranks with 24, 40 and 64 rows take it 40, 43 and 44 us, and
// took the split kernel (with two and four warps to a warp's keys) 53, 73 and
// 89. With 16 rows the split kernel takes 41 to 45 us, the prompts' 40, from an 8-bit
// cache 44 and 49; over 64 contexts of up to 8192, with two key heads 80 and 107,
// with four 128 and 147.
constexpr int kFewRows = 16;
size_t few_bytes(const fo_paged_desc* d) {
  return kScratchAt + (size_t)kFewBlocks * FO_GB300_SMS * 2 * kFewRows * (d->head_dim + 2) * 4;
}

}  // namespace
}  // namespace fo_ops

extern "C" fo_status fo_paged_attention_workspace(const fo_paged_desc* d, int32_t seqs, int64_t rows, int32_t max_new,
                                                  size_t* bytes) {
  const fo_status st = fo_ops::check_paged(d);
  if (st) return st;
  if (!bytes) return FO_ERR_INVALID_ARG;
  if (seqs < 0 || rows < 0 || rows > INT32_MAX || max_new < 1) return FO_ERR_SHAPE;
  const bool prompts = (int64_t)max_new * (d->heads_q / d->heads_k) > fo_ops::kFewRows;
  *bytes = prompts ? std::max(fo_ops::few_bytes(d), fo_ops::prompt_bytes(d, seqs, rows)) : fo_ops::few_bytes(d);
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
    const int step = 4 * few_keys(eight);
    f.box = std::min(d->page, step);
    for (f.boxes_log2 = 0; f.box << f.boxes_log2 < step; ++f.boxes_log2) {
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
    f.scale_log2 = scale * 1.4426950408889634f;
    f.least_exponent = least_exponent(f.scale_log2);
    f.count = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + 256);
    f.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kScratchAt);
    return attend_few(f, d->head_dim, unit_rows > 8, eight, sms, (cudaStream_t)stream);
  }
  PagedCall c;
  c.d = d, c.b = b, c.rows = rows, c.ld = ld;
  c.q = q, c.k = k_cache, c.v = v_cache, c.ks = k_scale, c.vs = v_scale, c.o = o, c.lse = lse;
  c.ws = static_cast<uint8_t*>(ws);
  c.scale_log2 = scale * 1.4426950408889634f;
  c.sms = sms;
  return attend_prompts(c, (cudaStream_t)stream);
}
