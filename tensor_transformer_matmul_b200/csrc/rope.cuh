// Rotary positions: the frequency table, and the rotation of rows of heads, alone or while the
// rows are appended to a paged key/value cache.
//   pair i of a row at position n:  (x1, x2) -> m (x1 cos a - x2 sin a, x1 sin a + x2 cos a),
//   a = n w_i;  the gradient is the transpose, the same with -a.
#pragma once

#include <cmath>

#include "tp_common.cuh"

namespace tp {
namespace rope {

struct Rows {
  const void* p;
  int64_t ts, hs;   // token and head strides, elements
};

// w_i / 2 pi of every pair, in 64 bits: positions are multiplied by it and reduced to one turn.
static __global__ void freqs_kernel(tp_rope_desc d, double* freqs) {
  const int half = d.rot_dim / 2;
  constexpr double kTurn = 6.283185307179586476925286766559;
  const double R = d.rot_dim;
  double base = d.base;
  if (d.scaling == TP_ROPE_NTK && d.rot_dim > 2) base *= pow(d.factor, R / (R - 2.0));
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < half; i += gridDim.x * blockDim.x) {
    double w = pow(base, -2.0 * i / R);
    if (d.scaling == TP_ROPE_LINEAR) w /= d.factor;
    if (d.scaling == TP_ROPE_BY_PARTS) {
      const double r = d.orig_len * w / kTurn;
      const double g = fmin(1.0, fmax(0.0, (r - d.beta_slow) / (d.beta_fast - d.beta_slow)));
      w = g * w + (1.0 - g) * w / d.factor;
    }
    freqs[i] = w / kTurn;
  }
}

// cos and sin of the angle pos * w: the turns are reduced in 64 bits, so a far position costs
// no accuracy; what is left is at most half a turn and keeps fp32's relative accuracy.
__device__ __forceinline__ void cos_sin(int32_t pos, double f, float m, float& c, float& s) {
  const double t = static_cast<double>(pos) * f;
  sincospif(static_cast<float>(2.0 * (t - rint(t))), &s, &c);
  c *= m;
  s *= m;
}

struct Args {
  const double* freqs;
  const int32_t* positions;
  int64_t T;
  int heads, hd, half, interleaved;
  float m, sign;     // magnitude; +1 forward, -1 gradient
  Rows x, out;
};

// One thread per pair (or per dim that passes through) of a row.
template <typename T>
__global__ void __launch_bounds__(256) rotate_kernel(Args a) {
  pdl_wait();
  pdl_trigger();
  const int per = a.hd - a.half;
  const int64_t n = a.T * a.heads * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int e = static_cast<int>(i % per);
    const int64_t row = i / per;
    const int64_t t = row / a.heads, j = row - t * a.heads;
    const T* x = static_cast<const T*>(a.x.p) + t * a.x.ts + j * a.x.hs;
    T* o = static_cast<T*>(const_cast<void*>(a.out.p)) + t * a.out.ts + j * a.out.hs;
    if (e >= a.half) {
      o[e + a.half] = x[e + a.half];
      continue;
    }
    float c, s;
    cos_sin(a.positions[t], a.freqs[e], a.m, c, s);
    s *= a.sign;
    const int e1 = a.interleaved ? 2 * e : e, e2 = a.interleaved ? 2 * e + 1 : e + a.half;
    const float x1 = to_f(x[e1]), x2 = to_f(x[e2]);
    o[e1] = from_f<T>(x1 * c - x2 * s);
    o[e2] = from_f<T>(x1 * s + x2 * c);
  }
}

inline tp_status check_desc(const tp_rope_desc* d) {
  if (!d) return set_error(TP_ERR_INVALID_ARG, "rope desc is null");
  if (d->rot_dim < 2 || d->rot_dim % 2 || d->rot_dim > 1024)
    return set_error(TP_ERR_SHAPE, "rot_dim must be even, in [2, 1024]");
  if (d->layout != TP_ROPE_HALF && d->layout != TP_ROPE_INTERLEAVED)
    return set_error(TP_ERR_INVALID_ARG, "unknown rope layout");
  if (d->scaling < TP_ROPE_PLAIN || d->scaling > TP_ROPE_BY_PARTS)
    return set_error(TP_ERR_INVALID_ARG, "unknown rope scaling");
  if (d->flags != 0) return set_error(TP_ERR_INVALID_ARG, "unknown flags");
  if (!(d->base > 0.0) || !std::isfinite(d->base))
    return set_error(TP_ERR_INVALID_ARG, "base must be finite and > 0");
  if (d->scaling != TP_ROPE_PLAIN && (!(d->factor > 0.0) || !std::isfinite(d->factor)))
    return set_error(TP_ERR_INVALID_ARG, "factor must be finite and > 0");
  if (d->scaling == TP_ROPE_BY_PARTS &&
      (!(d->orig_len > 0.0) || !std::isfinite(d->orig_len) || !std::isfinite(d->beta_fast) ||
       !std::isfinite(d->beta_slow) || !(d->beta_fast > d->beta_slow)))
    return set_error(TP_ERR_INVALID_ARG, "by-parts scaling needs orig_len > 0 and beta_fast > beta_slow");
  if (!(d->magnitude >= 0.0) || !std::isfinite(d->magnitude))
    return set_error(TP_ERR_INVALID_ARG, "magnitude must be finite and >= 0");
  return TP_OK;
}

inline float magnitude_of(const tp_rope_desc* d) {
  if (d->magnitude > 0.0) return static_cast<float>(d->magnitude);
  return d->scaling == TP_ROPE_BY_PARTS ? static_cast<float>(1.0 + 0.1 * std::log(d->factor)) : 1.f;
}

// Rows of ``heads`` heads over T tokens: pointer and element alignment, strides that are not
// negative, and (``written``) rows that do not overlap each other.
inline tp_status check_rows(const tp_head_rows* r, int64_t T, int heads, int hd, int eb,
                            bool written, const char* name) {
  if (!r || !r->data) return set_error(TP_ERR_INVALID_ARG, std::string(name) + " is null");
  if (reinterpret_cast<uintptr_t>(r->data) % eb)
    return set_error(TP_ERR_INVALID_ARG, std::string(name) + " is not aligned to its elements");
  if (r->token_stride < 0 || r->head_stride < 0)
    return set_error(TP_ERR_INVALID_ARG, std::string(name) + ": strides must be >= 0");
  // offsets are 64-bit; the farthest must stay in an address
  const int64_t kFar = int64_t(1) << 56;
  if ((T > 1 && r->token_stride > kFar / T) || (heads > 1 && r->head_stride > kFar / heads))
    return set_error(TP_ERR_INVALID_ARG, std::string(name) + ": stride too large");
  if (written) {
    const int64_t lo = r->token_stride < r->head_stride ? r->token_stride : r->head_stride;
    const int64_t hi = r->token_stride < r->head_stride ? r->head_stride : r->token_stride;
    const int64_t n_lo = r->token_stride < r->head_stride ? T : heads;
    const int64_t n_hi = r->token_stride < r->head_stride ? heads : T;
    const bool bad = (n_lo > 1 && lo < hd) || (n_hi > 1 && hi < (n_lo > 1 ? lo * (n_lo - 1) : 0) + hd);
    if (bad) return set_error(TP_ERR_INVALID_ARG, std::string(name) + ": its rows overlap");
  }
  return TP_OK;
}

// out may be x itself (same strides), not x with other strides
inline tp_status check_pair(const tp_head_rows* x, const tp_head_rows* o, const char* name) {
  if (x->data == o->data && (x->token_stride != o->token_stride || x->head_stride != o->head_stride))
    return set_error(TP_ERR_INVALID_ARG, std::string(name) + " in place needs the input's strides");
  return TP_OK;
}

inline unsigned grid_for(int64_t threads) {
  const int64_t most = static_cast<int64_t>(num_sms()) * 16;
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(threads, 256), most)));
}

inline tp_status launch(const Args& a, int dtype, cudaStream_t s) {
  ProfScope prof(s, "rope");
  const unsigned g = grid_for(a.T * a.heads * (a.hd - a.half));
  if (dtype == TP_BF16)
    TP_LAUNCH_PDL(rotate_kernel<__nv_bfloat16>, dim3(g), dim3(256), 0, s, a);
  else
    TP_LAUNCH_PDL(rotate_kernel<float>, dim3(g), dim3(256), 0, s, a);
  return TP_OK;
}

}  // namespace rope
}  // namespace tp
