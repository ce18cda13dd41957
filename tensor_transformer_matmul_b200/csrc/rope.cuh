// Rotary positions: the frequency table, and the rotation of rows of heads, alone or while the
// rows are appended to a paged key/value cache.
//   pair i of a row at position n:  (x1, x2) -> m (x1 cos a - x2 sin a, x1 sin a + x2 cos a),
//   a = n w_i;  the gradient is the transpose, the same with -a.
#pragma once

#include <algorithm>
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

// Where a token's rows come from and go: n rows of x to out, and with a cache (kAppend) its k and v
// rows to a slot.  ``Cache`` gives heads() per token and slot(t, err) -> element offset or -1.
struct NoCache {
  Rows k, v;
  void *kp, *vp;
  int64_t head_stride;
  int n_kv;
  __device__ __forceinline__ int64_t slot(int64_t, bool) const { return -1; }
};

// 16-byte vectors: an item is one vector of a row (interleaved pairs, or dims that pass through) or
// two, half a rotation apart.  A thread takes the same item of kRows rows of a token: their loads
// are issued together, and the sines and cosines (about 40 instructions a pair, in 64 bits up to
// the reduced angle) are shared by the rows, computed while the loads fly.  Bound by the bytes
// moved, each once.
template <typename T, int kVecs, int kRows, typename Cache>
__global__ void __launch_bounds__(256) rotate_rows_kernel(const __grid_constant__ Args a,
                                                          const __grid_constant__ Cache c,
                                                          int pass_items) {
  constexpr int VE = 16 / sizeof(T), kPairs = VE * kVecs / 2;
  pdl_wait();
  pdl_trigger();
  const int turn_items = a.half * 2 / (VE * kVecs), items = turn_items + pass_items;
  const int rows = a.heads + 2 * c.n_kv, groups = (rows + kRows - 1) / kRows;
  const uint32_t per = static_cast<uint32_t>(groups) * items;
  const int64_t n = a.T * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = n <= UINT32_MAX ? static_cast<uint32_t>(i) / per : i / per;
    const uint32_t in = static_cast<uint32_t>(i - t * per);
    const int r = in / static_cast<uint32_t>(items), e = in - r * items;
    const bool turn = e < turn_items;
    const int d = turn ? e * VE : 2 * a.half + (e - turn_items) * VE;
    const int vecs = turn ? kVecs : 1;
    const int32_t pos = turn ? a.positions[t] : 0;
    const int64_t slot = c.n_kv > 0 ? c.slot(t, in == 0) : -1;
    uint4 x[kRows][kVecs];
    T* to[kRows];
    bool is_v[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      int j = r + k * groups;
      to[k] = nullptr;
      is_v[k] = false;
      if (j >= rows) continue;
      const T* from;
      if (j < a.heads) {
        from = static_cast<const T*>(a.x.p) + t * a.x.ts + j * a.x.hs + d;
        to[k] = static_cast<T*>(const_cast<void*>(a.out.p)) + t * a.out.ts + j * a.out.hs + d;
      } else {
        if (slot < 0) continue;
        j -= a.heads;
        is_v[k] = j >= c.n_kv;
        j -= is_v[k] ? c.n_kv : 0;
        const Rows& src = is_v[k] ? c.v : c.k;
        from = static_cast<const T*>(src.p) + t * src.ts + j * src.hs + d;
        to[k] = static_cast<T*>(is_v[k] ? c.vp : c.kp) + slot + j * c.head_stride + d;
      }
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (v < vecs) x[k][v] = *reinterpret_cast<const uint4*>(from + v * a.half);
    }
    float co[kPairs], si[kPairs];
    if (turn) {
#pragma unroll
      for (int q = 0; q < kPairs; ++q) {
        cos_sin(pos, a.freqs[e * kPairs + q], a.m, co[q], si[q]);
        si[q] *= a.sign;
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (!to[k]) continue;
      if (turn && !is_v[k]) {
        T y[VE * kVecs];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) *reinterpret_cast<uint4*>(y + v * VE) = x[k][v];
#pragma unroll
        for (int q = 0; q < kPairs; ++q) {
          const int e1 = kVecs == 2 ? q : 2 * q, e2 = kVecs == 2 ? VE + q : 2 * q + 1;
          const float x1 = to_f(y[e1]), x2 = to_f(y[e2]);
          y[e1] = from_f<T>(x1 * co[q] - x2 * si[q]);
          y[e2] = from_f<T>(x1 * si[q] + x2 * co[q]);
        }
#pragma unroll
        for (int v = 0; v < kVecs; ++v) x[k][v] = *reinterpret_cast<const uint4*>(y + v * VE);
      }
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (v < vecs) *reinterpret_cast<uint4*>(to[k] + v * a.half) = x[k][v];
    }
  }
}

// One thread per pair, or per dim that passes through: rows that 16-byte vectors do not fit.
template <typename T, typename Cache>
__global__ void __launch_bounds__(256) rotate_elements_kernel(const __grid_constant__ Args a,
                                                              const __grid_constant__ Cache c) {
  pdl_wait();
  pdl_trigger();
  const int per = a.hd - a.half, rows = a.heads + 2 * c.n_kv;
  const int64_t n = a.T * rows * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int e = static_cast<int>(i % per);
    const int64_t row = i / per, t = row / rows;
    int j = static_cast<int>(row - t * rows);
    const T* x;
    T* o;
    bool turn = a.half > 0;
    if (j < a.heads) {
      x = static_cast<const T*>(a.x.p) + t * a.x.ts + j * a.x.hs;
      o = static_cast<T*>(const_cast<void*>(a.out.p)) + t * a.out.ts + j * a.out.hs;
    } else {
      const int64_t slot = c.slot(t, e == 0);
      if (slot < 0) continue;
      j -= a.heads;
      const bool is_v = j >= c.n_kv;
      j -= is_v ? c.n_kv : 0;
      const Rows& src = is_v ? c.v : c.k;
      x = static_cast<const T*>(src.p) + t * src.ts + j * src.hs;
      o = static_cast<T*>(is_v ? c.vp : c.kp) + slot + j * c.head_stride;
      if (is_v) turn = false;
    }
    if (!turn) {   // a row that moves as it is: both dims of a pair
      if (e < a.half) o[e] = x[e];
      o[e + a.half] = x[e + a.half];
      continue;
    }
    if (e >= a.half) {
      o[e + a.half] = x[e + a.half];
      continue;
    }
    float co, si;
    cos_sin(a.positions[t], a.freqs[e], a.m, co, si);
    si *= a.sign;
    const int e1 = a.interleaved ? 2 * e : e, e2 = a.interleaved ? 2 * e + 1 : e + a.half;
    const float x1 = to_f(x[e1]), x2 = to_f(x[e2]);
    o[e1] = from_f<T>(x1 * co - x2 * si);
    o[e2] = from_f<T>(x1 * si + x2 * co);
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

inline bool vector_rows(const Rows& r, int64_t unit) {
  return !(reinterpret_cast<uintptr_t>(r.p) & 15) && r.ts % unit == 0 && r.hs % unit == 0;
}

// ``vectors``: the cache's rows (if any) fit 16-byte vectors.
template <typename T, typename Cache>
inline tp_status launch_rows(const Args& a, const Cache& c, bool vectors, cudaStream_t s) {
  constexpr int VE = 16 / sizeof(T);
  const int vecs = a.interleaved ? 1 : 2, rot = 2 * a.half;
  const int64_t rows = a.heads + 2 * c.n_kv;
  if (a.heads > 0) vectors = vectors && vector_rows(a.x, VE) && vector_rows(a.out, VE);
  if (vectors && rot % (VE * vecs) == 0 && (a.hd - rot) % VE == 0) {
    // in place the dims that pass through stay where they are
    const int pass = c.n_kv == 0 && a.x.p == a.out.p ? 0 : (a.hd - rot) / VE;
    const int64_t items = rot / (VE * vecs) + pass;
    // four rows to a thread once that fills the GPU; one row each is faster for a few tokens
    // (64 tokens of 80 rows of 128 bf16 dims: see the figures at the entry point)
    const bool many = a.T * ceil_div(rows, 4) * items >= static_cast<int64_t>(num_sms()) * 512;
    const int64_t n = a.T * ceil_div(rows, many ? 4 : 1) * items;
    const unsigned g = static_cast<unsigned>(std::min<int64_t>(ceil_div(n, 256), 1 << 24));
#define TP_ROTATE(V, R) \
  TP_LAUNCH_PDL((rotate_rows_kernel<T, V, R, Cache>), dim3(g), dim3(256), 0, s, a, c, pass)
    if (a.interleaved) {
      if (many) TP_ROTATE(1, 4); else TP_ROTATE(1, 1);
    } else {
      if (many) TP_ROTATE(2, 4); else TP_ROTATE(2, 1);
    }
#undef TP_ROTATE
    return TP_OK;
  }
  const int64_t n = a.T * rows * (a.hd - a.half);
  const unsigned g = static_cast<unsigned>(std::min<int64_t>(ceil_div(n, 256), num_sms() * 16));
  TP_LAUNCH_PDL((rotate_elements_kernel<T, Cache>), dim3(g), dim3(256), 0, s, a, c);
  return TP_OK;
}

}  // namespace rope
}  // namespace tp
