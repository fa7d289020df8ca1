// Rotary positions on Q and K, V copied: packed rows to parted ones or back,
// or in place. Bandwidth-bound: each element is read and written once.
#include <math.h>
#include <string.h>

#include "fo_ops.h"

namespace fo_ops {
namespace {

struct RopeParams {
  const void* in[3][kMaxR];
  void* out[3][kMaxR];
  int64_t ld_in[3], ld_out[3];
  const void* positions;
  int64_t rows;
  int32_t pos_bytes;
  int32_t heads[3];
  int32_t D, rot;
  int32_t half;       // layout
  int32_t R;
  int32_t lanes, tokens;              // threads for a token, tokens a block
  int32_t heads_each, ranks_each;     // heads and ranks a thread goes through
  float factor, sign;
  uint64_t turns[FO_ROPE_MAX_DIM / 2];
};

// cos and sin (times the factor) of position * turns: the product modulo
// 2^64 is the angle's fraction of a turn, exact but for the frequency's own
// last bit; as a signed number it lies in [-1/2, 1/2).
__device__ __forceinline__ float2 rotation(const RopeParams& p, int64_t pos, uint64_t turns) {
  const int64_t frac = (int64_t)((uint64_t)pos * turns);
  float s, c;
  sincospif((float)frac * 1.08420217e-19f, &s, &c);   // 2^-63: half turns
  return make_float2(c * p.factor, s * p.factor * p.sign);
}

__device__ __forceinline__ int64_t position_of(const RopeParams& p, int64_t t) {
  if (!p.positions) return t;
  return p.pos_bytes == 8 ? static_cast<const int64_t*>(p.positions)[t]
                          : (int64_t)static_cast<const int32_t*>(p.positions)[t];
}

// V values of type T as one access.
template <int BYTES>
struct Bits;
template <>
struct Bits<2> { typedef uint16_t type; };
template <>
struct Bits<4> { typedef uint32_t type; };
template <>
struct Bits<8> { typedef uint2 type; };
template <>
struct Bits<16> { typedef uint4 type; };
template <typename T, int V>
union Piece {
  typename Bits<sizeof(T) * V>::type bits;
  T v[V];
  __device__ __forceinline__ Piece() {}
  __device__ __forceinline__ void load(const T* p) { bits = *reinterpret_cast<const decltype(bits)*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<decltype(bits)*>(p) = bits; }
};

// A thread has a token and two pieces of V elements in every head, computes
// its own angles once and goes through its share of the ranks and heads,
// kHeads at a time with all loads first. The pieces of a rotated head: in the half layout
// piece i of the first half and of the second (V pairs); interleaved, pieces
// i and i + lanes (V / 2 pairs each); the threads beyond the rotated pieces
// copy the head's rest, two pieces each. Heads of V: pieces i and i + lanes.
// V is the widest access that the sizes, strides and addresses allow (at
// least a pair where pairs are neighbours).
// Eight ranks' packed rows of 8192 x 12 heads of 128, bf16 (403 MB): 62 us,
// 6.5 TB/s; with V's heads in a loop of their own, two loads at a time, and
// 98 registers 101 us, one element at a time 193 us.
template <typename T, int V, bool HALF, bool RANKS>
__global__ void __launch_bounds__(256, 3) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kHeads = 4;
  // (Read lane by lane from the parameters, the frequencies would be one
  // access to the constant cache for each.)
  __shared__ uint64_t turns[FO_ROPE_MAX_DIM / 2];
  if (threadIdx.x < p.rot / 2) turns[threadIdx.x] = p.turns[threadIdx.x];
  __syncthreads();
  grid_release();
  grid_wait();
  const int lanes = p.lanes, tok = threadIdx.x / lanes, i = threadIdx.x - tok * lanes;
  const int64_t t = (int64_t)blockIdx.x * p.tokens + tok;
  if (tok >= p.tokens || t >= p.rows) return;
  const int pieces = p.rot / V / (HALF ? 2 : 1);   // of the first half; of all that is rotated
  const int whole = p.D / V;
  // This thread's pieces of a rotated head, and whether they are rotated.
  const bool turn_a = i < pieces, turn_b = HALF ? turn_a : i + lanes < pieces;
  const int a = !HALF || turn_a ? i : i + pieces;
  const int b = !HALF ? i + lanes : turn_a ? i + pieces : i + lanes;
  const bool two = b < whole;
  float c[V], s[V];   // HALF: by element; else the first V / 2 for piece a, the others for b
  const int64_t pos = position_of(p, t);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int pair = HALF ? i * V + j : j < V / 2 ? a * (V / 2) + j : b * (V / 2) + j - V / 2;
    const float2 cs = 2 * pair < p.rot ? rotation(p, pos, turns[pair]) : make_float2(0.f, 0.f);
    c[j] = cs.x, s[j] = cs.y;
  }
  // (A loop over one rank alone costs a tenth of the kernel: registers.)
  const int first_r = RANKS ? (int)blockIdx.z * p.ranks_each : (int)blockIdx.z;
  const int last_r = RANKS ? min(p.R, first_r + p.ranks_each) : first_r + 1;
  for (int r = first_r; RANKS ? r < last_r : r == first_r; ++r) {
    int h0 = (int)blockIdx.y * p.heads_each, h1 = h0 + p.heads_each;   // this block's heads, counted from each part's first
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      const int first = max(h0, 0), last = min(h1, p.heads[part]);
      h0 -= p.heads[part], h1 -= p.heads[part];
      if (first >= last) continue;
      const bool turned = part < 2;
      const int pa = (turned ? a : i) * V, pb = (turned ? b : i + lanes) * V;
      const bool has_b = turned ? two : i + lanes < whole;
      const T* in = static_cast<const T*>(p.in[part][r]) + t * p.ld_in[part] + first * p.D;
      T* out = static_cast<T*>(p.out[part][r]) + t * p.ld_out[part] + first * p.D;
      const bool moves = in != out;   // in place, what is not rotated stays
      for (int n = last - first; n > 0; n -= kHeads, in += kHeads * p.D, out += kHeads * p.D) {
        Piece<T, V> x[kHeads], y[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
          if (k < n) {
            x[k].load(in + k * p.D + pa);
            if (has_b) y[k].load(in + k * p.D + pb);
          }
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
          if (k < n) {
            if (turned) {
              if constexpr (HALF) {
                if (turn_a) {
#pragma unroll
                  for (int j = 0; j < V; ++j) {
                    const float u = to_f(x[k].v[j]), w = to_f(y[k].v[j]);
                    from_f(u * c[j] - w * s[j], x[k].v[j]);
                    from_f(w * c[j] + u * s[j], y[k].v[j]);
                  }
                }
              } else {
                auto turn = [&](Piece<T, V>& z, int at) {
#pragma unroll
                  for (int j = 0; j < V / 2; ++j) {
                    const float u = to_f(z.v[2 * j]), w = to_f(z.v[2 * j + 1]);
                    from_f(u * c[at + j] - w * s[at + j], z.v[2 * j]);
                    from_f(w * c[at + j] + u * s[at + j], z.v[2 * j + 1]);
                  }
                };
                if (turn_a) turn(x[k], 0);
                if (turn_b) turn(y[k], V / 2);
              }
            }
            if (moves || (turned && turn_a)) x[k].store(out + k * p.D + pa);
            if (has_b && (moves || (turned && turn_b))) y[k].store(out + k * p.D + pb);
          }
      }
    }
  }
}

template <typename T, int V, bool HALF>
fo_status launch_as(RopeParams& k, int R, cudaStream_t s) {
  // Lanes for a token: two pieces each. Heads for a thread: all of a rank's,
  // unless that leaves the GPU short of threads; with few heads a rank, those
  // of several ranks, so that at least 8 share the angles (which take as long
  // as four heads).
  k.R = R;
  k.lanes = (k.D / V + 1) / 2;
  k.tokens = 256 / k.lanes;
  const int all = k.heads[0] + k.heads[1] + k.heads[2];
  const int64_t blocks = (k.rows + k.tokens - 1) / k.tokens;
  const int64_t enough = 4 * FO_GB300_SMS;
  k.ranks_each = 1;
  while (k.ranks_each < R && k.ranks_each * all < 8 && blocks * R >= enough * k.ranks_each) k.ranks_each *= 2;
  int64_t cuts = (enough + blocks * R - 1) / (blocks * R);
  if (cuts > (all + 3) / 4) cuts = (all + 3) / 4;
  k.heads_each = (int)((all + cuts - 1) / cuts);
  const dim3 grid((unsigned)blocks, (unsigned)((all + k.heads_each - 1) / k.heads_each),
                  (unsigned)((R + k.ranks_each - 1) / k.ranks_each));
  auto kern = k.ranks_each > 1 ? rope_kernel<T, V, HALF, true> : rope_kernel<T, V, HALF, false>;
  return launched(launch_after(kern, grid, 256, 0, 0, s, k), "rope", R, k.rows, k.D, grid.x * grid.y, 256);
}
template <typename T>
fo_status launch_with(RopeParams& k, int R, int v, cudaStream_t s) {
  constexpr int kMost = 16 / sizeof(T);
  if (k.half) {
    if (v == kMost) return launch_as<T, kMost, true>(k, R, s);
    if (kMost == 8 && v == 4) return launch_as<T, 4, true>(k, R, s);
    if (v >= 2) return launch_as<T, 2, true>(k, R, s);
    return launch_as<T, 1, true>(k, R, s);
  }
  if (v == kMost) return launch_as<T, kMost, false>(k, R, s);
  if (kMost == 8 && v == 4) return launch_as<T, 4, false>(k, R, s);
  return launch_as<T, 2, false>(k, R, s);
}

// A head whose pairs are neighbours but do not start on a pair's address
// (odd head dimensions): one element at a time, a block for a row and rank.
template <typename T>
__global__ void __launch_bounds__(256) rope_single_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 rot[FO_ROPE_MAX_DIM / 2];
  const int64_t t = blockIdx.x;
  const int r = blockIdx.y, pairs = p.rot / 2;
  grid_release();
  grid_wait();
  if (threadIdx.x < pairs) rot[threadIdx.x] = rotation(p, position_of(p, t), p.turns[threadIdx.x]);
  __syncthreads();
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    if (!p.heads[part]) continue;
    const T* in = static_cast<const T*>(p.in[part][r]) + t * p.ld_in[part];
    T* out = static_cast<T*>(p.out[part][r]) + t * p.ld_out[part];
    const int per_head = part == 2 ? p.D : pairs + p.D - p.rot;
    for (int i = threadIdx.x; i < p.heads[part] * per_head; i += 256) {
      const int head = i / per_head, k = i - head * per_head;
      const int at = head * p.D;
      if (part == 2) {
        out[at + k] = in[at + k];
      } else if (k >= pairs) {
        out[at + k + pairs] = in[at + k + pairs];
      } else {
        const int ia = at + 2 * k, ib = ia + 1;
        const float a = to_f(in[ia]), b = to_f(in[ib]);
        from_f(a * rot[k].x - b * rot[k].y, out[ia]);
        from_f(b * rot[k].x + a * rot[k].y, out[ib]);
      }
    }
  }
}

}  // namespace
}  // namespace fo_ops

// What fo_rope_init and every call look at: a caller may have changed the
// description since.
fo_status fo_ops::check_rope_desc(const fo_rope_desc* d) {
  if (d->R < 1 || d->R > FO_MAX_R || d->reserved) return FO_ERR_INVALID_ARG;
  if (d->head_dim < 1 || d->head_dim > FO_ROPE_MAX_DIM || d->rot_dim < 2 || d->rot_dim % 2 ||
      d->rot_dim > d->head_dim || d->heads_q < 1 || d->heads_k < 0 || d->heads_v < 0 || d->heads_q > 65536 ||
      d->heads_k > 65536 || d->heads_v > 65536)
    return FO_ERR_SHAPE;
  if (d->dtype != FO_BF16 && d->dtype != FO_F32) return FO_ERR_DTYPE;
  if (d->layout != FO_ROPE_HALF && d->layout != FO_ROPE_INTERLEAVED) return FO_ERR_INVALID_ARG;
  if (d->scaling < FO_ROPE_SCALE_NONE || d->scaling > FO_ROPE_SCALE_PARTS) return FO_ERR_INVALID_ARG;
  if (!(d->base > 1.0) || !isfinite(d->base)) return FO_ERR_INVALID_ARG;
  const bool mixed = d->scaling == FO_ROPE_SCALE_WAVELENGTH || d->scaling == FO_ROPE_SCALE_PARTS;
  if (d->scaling != FO_ROPE_SCALE_NONE && (!(d->stretch >= 1.0) || !isfinite(d->stretch))) return FO_ERR_INVALID_ARG;
  if (mixed && (!(d->trained >= 1.0) || !isfinite(d->trained) || !(d->slow > 0.0) || !(d->fast > d->slow) ||
                !isfinite(d->fast)))
    return FO_ERR_INVALID_ARG;
  return FO_OK;
}

extern "C" fo_status fo_rope_init(fo_rope_desc* d) {
  if (!d) return FO_ERR_INVALID_ARG;
  d->ready = 0;
  if (const fo_status st = fo_ops::check_rope_desc(d)) return st;
  const bool mixed = d->scaling == FO_ROPE_SCALE_WAVELENGTH || d->scaling == FO_ROPE_SCALE_PARTS;
  const double two_pi = 6.283185307179586476925286766559;
  const int pairs = d->rot_dim / 2;
  // PARTS: the (real) pair indices that make `fast` and `slow` turns.
  double lo = 0.0, hi = 0.0;
  if (d->scaling == FO_ROPE_SCALE_PARTS) {
    lo = floor(d->rot_dim * log(d->trained / (two_pi * d->fast)) / (2.0 * log(d->base)));
    hi = ceil(d->rot_dim * log(d->trained / (two_pi * d->slow)) / (2.0 * log(d->base)));
    lo = fmax(lo, 0.0);
    hi = fmin(hi, d->rot_dim - 1.0);
  }
  memset(d->turns, 0, sizeof(d->turns));
  for (int i = 0; i < pairs; ++i) {
    double f = pow(d->base, -2.0 * i / d->rot_dim);
    if (d->scaling == FO_ROPE_SCALE_LINEAR) f /= d->stretch;
    if (mixed) {
      const double k = d->scaling == FO_ROPE_SCALE_WAVELENGTH
                           ? (d->trained * f / two_pi - d->slow) / (d->fast - d->slow)
                           : 1.0 - (i - lo) / fmax(hi - lo, 0.001);
      const double kc = fmin(fmax(k, 0.0), 1.0);
      f = kc * f + (1.0 - kc) * f / d->stretch;
    }
    d->turns[i] = (uint64_t)ldexp(f / two_pi, 64);   // below 2^62: f <= 1
  }
  d->factor = d->scaling == FO_ROPE_SCALE_PARTS ? (float)(0.1 * log(d->stretch) + 1.0) : 1.f;
  d->ready = 1;
  return FO_OK;
}

extern "C" fo_status fo_rope(const fo_rope_desc* d, int64_t rows, const void* positions, int32_t pos_bytes,
                             const void* const* q_in, const void* const* k_in, const void* const* v_in,
                             const int64_t ld_in[3], void* const* q_out, void* const* k_out, void* const* v_out,
                             const int64_t ld_out[3], int32_t inverse, fo_stream_t stream) {
  using namespace fo_ops;
  if (!d || d->ready != 1 || !ld_in || !ld_out) return FO_ERR_INVALID_ARG;
  fo_status st;
  if ((st = check_rope_desc(d))) return st;
  if ((inverse != 0 && inverse != 1) || (positions && pos_bytes != 4 && pos_bytes != 8)) return FO_ERR_INVALID_ARG;
  if (rows < 0 || rows > INT32_MAX) return FO_ERR_SHAPE;
  const int R = d->R;
  const size_t es = d->dtype == FO_BF16 ? 2 : 4;
  typedef const void* const* A;
  const int32_t heads[3] = {d->heads_q, d->heads_k, d->heads_v};
  const A in[3] = {q_in, k_in, v_in}, out[3] = {(A)q_out, (A)k_out, (A)v_out};
  for (int j = 0; j < 3; ++j) {
    if (!heads[j]) continue;
    if (ld_in[j] < (int64_t)heads[j] * d->head_dim || ld_out[j] < (int64_t)heads[j] * d->head_dim)
      return FO_ERR_SHAPE;
    if (rows && ((st = check_array(R, in[j], es)) || (st = check_array(R, out[j], es)))) return st;
  }
  if (positions && !aligned(positions, pos_bytes)) return FO_ERR_ALIGN;
  if (rows == 0) return FO_OK;
  int sms;
  if ((st = device_sms(&sms))) return st;
  PtrList l;
  for (int j = 0; j < 3; ++j)
    if (heads[j]) l.add(R, in[j]), l.add(R, out[j]);
  l.add(positions);
  if ((st = check_device(l, stream))) return st;
  RopeParams k;
  memset(&k, 0, sizeof(k));
  for (int j = 0; j < 3; ++j) {
    if (!heads[j]) continue;
    k.heads[j] = heads[j];
    k.ld_in[j] = ld_in[j];
    k.ld_out[j] = ld_out[j];
    for (int r = 0; r < R; ++r) k.in[j][r] = in[j][r], k.out[j][r] = const_cast<void*>(out[j][r]);
  }
  k.positions = positions;
  k.pos_bytes = pos_bytes;
  k.rows = rows;
  k.D = d->head_dim;
  k.rot = d->rot_dim;
  k.half = d->layout == FO_ROPE_HALF;
  k.factor = d->factor;
  k.sign = inverse ? -1.f : 1.f;
  memcpy(k.turns, d->turns, sizeof(k.turns));
  const cudaStream_t s = (cudaStream_t)stream;
  // The widest piece of V elements that every head, half and row starts on.
  int v = (int)(16 / es);
  for (; v > 1; v /= 2) {
    bool fits = d->head_dim % v == 0 && d->rot_dim % (k.half ? 2 * v : v) == 0;
    for (int j = 0; j < 3 && fits; ++j)
      if (heads[j])
        fits = ld_in[j] % v == 0 && ld_out[j] % v == 0 && all_aligned(R, in[j], v * es) && all_aligned(R, out[j], v * es);
    if (fits) break;
  }
  if (!k.half && v < 2) {
    const dim3 grid((unsigned)rows, R);
    auto kern = d->dtype == FO_BF16 ? rope_single_kernel<__nv_bfloat16> : rope_single_kernel<float>;
    return launched(launch_after(kern, grid, 256, 0, 0, s, k), "rope single", R, rows, d->head_dim, (int)rows, 256);
  }
  return d->dtype == FO_BF16 ? launch_with<__nv_bfloat16>(k, R, v, s) : launch_with<float>(k, R, v, s);
}
