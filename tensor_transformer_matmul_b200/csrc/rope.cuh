// Rotary positions: the frequency table, and the rotation of rows of heads, alone or while the
// rows are appended to a paged key/value cache.
//   pair i of a row at position n:  (x1, x2) -> m (x1 cos a - x2 sin a, x1 sin a + x2 cos a),
//   a = n w_i;  the gradient is the transpose, the same with -a.
#pragma once

#include <algorithm>
#include <cmath>

#include "sm100.cuh"
#include "tp_common.cuh"

namespace tp {

// 16 bytes into shared memory; zeros where ``take`` is false (src is then not read)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
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

// A warp's share: a slice of a token's rows, ``step`` of them at once.
struct Share {
  int slices, rows, step, items;
};
constexpr int kRotateWarps = 4, kRotateSteps = 24, kRotateRing = 8;

// The vectors that rows move in: 16 bytes, or 8 where halves of a rotation are no multiple of 16.
template <int kBytes> struct Vec;
template <> struct Vec<16> {
  using type = uint4;
  __device__ __forceinline__ static void copy(uint32_t dst, const void* src) { copy16(dst, src, true); }
  __device__ __forceinline__ static type lds(uint32_t a) { return lds16(a); }
};
template <> struct Vec<8> {
  using type = uint2;
  __device__ __forceinline__ static void copy(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
  }
  __device__ __forceinline__ static type lds(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
    return r;
  }
};

// Vectors: an item is one vector of a row (interleaved pairs, or dims that pass through) or
// two, half a rotation apart.  A warp has a slice of a token's rows, a lane the same item of every
// step-th row.  The vectors are copied asynchronously into a ring of shared memory, eight of a lane
// in flight, each lane reading back what it copied itself; while the first ones fly the warp
// computes the token's sines and cosines (64-bit products up to the reduced angle), each once, for
// all rows of the slice.  No warp waits for another.  Bound by the bytes moved.
template <typename T, int kVecs, int kBytes, typename Cache>
__global__ void __launch_bounds__(kRotateWarps * 32) rotate_rows_kernel(
    const __grid_constant__ Args a, const __grid_constant__ Cache c, const __grid_constant__ Share sh) {
  using V = typename Vec<kBytes>::type;
  constexpr int VE = kBytes / sizeof(T), kPairs = VE * kVecs / 2, kDepth = kRotateRing / kVecs;
  constexpr int kWide = kPairs < 4 ? 2 : 4;
  extern __shared__ __align__(16) char smem[];           // [warp][ring][32] vectors, [warp][2][half]
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, turn_items = a.half * 2 / (VE * kVecs);
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kRotateWarps + warp;
  const int64_t t = w / sh.slices;
  if (t >= a.T) return;
  const int slice = static_cast<int>(w - t * sh.slices);
  const uint32_t ring = sm100::smem_addr(smem) + warp * kRotateRing * 512 + lane * 16;
  float* s_cos = reinterpret_cast<float*>(smem + kRotateWarps * kRotateRing * 512) + warp * 2 * a.half;
  float* s_sin = s_cos + a.half;
  const int all = a.heads + 2 * c.n_kv, r_begin = slice * sh.rows, r_end = min(all, r_begin + sh.rows);
  const int steps = (r_end - r_begin + sh.step - 1) / sh.step;
  int64_t slot = -1;
  for (int e0 = 0; e0 < sh.items; e0 += 32) {            // (rows of more than 32 items)
    const int q = sh.items > 32 ? 0 : lane / sh.items;
    const int e = sh.items > 32 ? e0 + lane : lane - q * sh.items;
    const bool pair = e < turn_items;
    const int d = pair ? e * VE : 2 * a.half + (e - turn_items) * VE;
    const int r0 = r_begin + q, r1 = q < sh.step && e < sh.items ? r_end : 0;
    const T* xq = static_cast<const T*>(a.x.p) + t * a.x.ts + d;
    const T* xk = static_cast<const T*>(c.k.p) + t * c.k.ts + d;
    const T* xv = static_cast<const T*>(c.v.p) + t * c.v.ts + d;
    auto issue = [&](int s) {
      const int row = r0 + s * sh.step, j = row - a.heads;
      const T* from = j < 0 ? xq + row * a.x.hs : j < c.n_kv ? xk + j * c.k.hs : xv + (j - c.n_kv) * c.v.hs;
      const uint32_t to = ring + (s % kDepth) * (kVecs * 512);
      if (row < r1) {
        Vec<kBytes>::copy(to, from);
        if (kVecs == 2 && pair) Vec<kBytes>::copy(to + 512, from + a.half);
      }
      copy_commit();
    };
#pragma unroll
    for (int s = 0; s < kDepth; ++s) issue(s);
    if (e0 == 0) {
      if (a.half > 0) {
        const int32_t pos = a.positions[t];
        for (int i = lane; i < a.half; i += 32) {
          float y, z;
          cos_sin(pos, a.freqs[i], a.m, y, z);
          s_cos[i] = y;
          s_sin[i] = z * a.sign;
        }
      }
      if (c.n_kv > 0) slot = c.slot(t, lane == 0 && slice == 0);
      __syncwarp();
    }
    float co[kPairs], si[kPairs];
    if (pair) {
#pragma unroll
      for (int i = 0; i < kPairs; i += kWide) {
        if constexpr (kWide == 2) {
          *reinterpret_cast<float2*>(co + i) = *reinterpret_cast<const float2*>(s_cos + e * kPairs + i);
          *reinterpret_cast<float2*>(si + i) = *reinterpret_cast<const float2*>(s_sin + e * kPairs + i);
        } else {
          *reinterpret_cast<float4*>(co + i) = *reinterpret_cast<const float4*>(s_cos + e * kPairs + i);
          *reinterpret_cast<float4*>(si + i) = *reinterpret_cast<const float4*>(s_sin + e * kPairs + i);
        }
      }
    }
    T* oq = static_cast<T*>(const_cast<void*>(a.out.p)) + t * a.out.ts + d;
    T* ok = static_cast<T*>(c.kp) + slot + d;
    T* ov = static_cast<T*>(c.vp) + slot + d;
    for (int s = 0; s < steps; ++s) {
      const int row = r0 + s * sh.step, j = row - a.heads;
      copy_wait<kDepth - 1>();
      if (row < r1 && (j < 0 || slot >= 0)) {
        const uint32_t at = ring + (s % kDepth) * (kVecs * 512);
        V x[kVecs];
        x[0] = Vec<kBytes>::lds(at);
        if (kVecs == 2 && pair) x[kVecs - 1] = Vec<kBytes>::lds(at + 512);
        T* to = j < 0 ? oq + row * a.out.hs : j < c.n_kv ? ok + j * c.head_stride
                                                         : ov + (j - c.n_kv) * c.head_stride;
        if (pair && j < c.n_kv) {
          alignas(16) T y[VE * kVecs];
#pragma unroll
          for (int v = 0; v < kVecs; ++v) *reinterpret_cast<V*>(y + v * VE) = x[v];
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            const int e1 = kVecs == 2 ? i : 2 * i, e2 = kVecs == 2 ? VE + i : 2 * i + 1;
            const float x1 = to_f(y[e1]), x2 = to_f(y[e2]);
            y[e1] = from_f<T>(x1 * co[i] - x2 * si[i]);
            y[e2] = from_f<T>(x1 * si[i] + x2 * co[i]);
          }
#pragma unroll
          for (int v = 0; v < kVecs; ++v) x[v] = *reinterpret_cast<const V*>(y + v * VE);
        }
        *reinterpret_cast<V*>(to) = x[0];
        if (kVecs == 2 && pair) *reinterpret_cast<V*>(to + a.half) = x[kVecs - 1];
      }
      issue(s + kDepth);
    }
    copy_wait<0>();
  }
}

// One thread per pair, or per dim that passes through: rows that no vector fits.  Every pair computes
// its own angle, a product in 64 bits, and its sines: bound by those (4096 tokens of 72 heads of 128
// dims from an odd start: 124 us in bf16 and 122 in fp32, 31 in 16-byte vectors; 1715 tokens of 80
// heads of 50 dims, 34 of them rotated: 32 us).
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

// rows that start on a multiple of ``bytes``
inline bool vector_rows(const Rows& r, int eb, int bytes) {
  return !(reinterpret_cast<uintptr_t>(r.p) % bytes) && r.ts * eb % bytes == 0 && r.hs * eb % bytes == 0;
}
inline bool vector_rows(const NoCache&, int, int) { return true; }

template <typename T, typename Cache>
inline tp_status launch_rows(const Args& a, const Cache& c, cudaStream_t s) {
  const int vecs = a.interleaved ? 1 : 2, rot = 2 * a.half, eb = static_cast<int>(sizeof(T));
  const int64_t rows = a.heads + 2 * c.n_kv;
  // 16-byte vectors where they fit, 8-byte ones for the halves they do not (a head of 80 bf16 dims, 40
  // of them rotated: 1715 tokens of 80 rows 18 us, 52 by elements)
  auto fits = [&](int bytes) {
    const int VE = bytes / eb;
    return rot % (VE * vecs) == 0 && (a.hd - rot) % VE == 0 && vector_rows(c, eb, bytes) &&
           (a.heads == 0 || (vector_rows(a.x, eb, bytes) && vector_rows(a.out, eb, bytes)));
  };
  const int bytes = fits(16) ? 16 : !a.interleaved && fits(8) ? 8 : 0;
  if (bytes) {
    const int VE = bytes / eb;
    // in place the dims that pass through stay where they are
    const int pass = c.n_kv == 0 && a.x.p == a.out.p ? 0 : (a.hd - rot) / VE;
    const int64_t items = rot / (VE * vecs) + pass;
    // Slices of at most 24 steps of a warp's rows (the angles' cost is then small), and of fewer
    // where the GPU would have less than 8 warps an SM (24 are no faster: 2051 tokens of 16 fp32 rows
    // of 96 dims 7.7 and 8.1 us, 6300 tokens of 40 bf16 rows of 128 dims 26.5 and 27.6 us).
    Share sh;
    sh.items = static_cast<int>(items);
    sh.step = items >= 32 ? 1 : static_cast<int>(32 / items);
    const int64_t steps = ceil_div(rows, sh.step);
    const int64_t slices = std::max(ceil_div(steps, kRotateSteps),
                                    std::min(steps, ceil_div(num_sms() * 8, a.T)));
    sh.rows = static_cast<int>(ceil_div(steps, slices)) * sh.step;
    sh.slices = static_cast<int>(ceil_div(rows, sh.rows));
    const int64_t blocks = ceil_div(a.T * sh.slices, kRotateWarps);
    if (blocks > INT32_MAX) return set_error(TP_ERR_SHAPE, "too many rows");
    const dim3 g(static_cast<unsigned>(blocks)), threads(kRotateWarps * 32);
    const size_t smem = static_cast<size_t>(kRotateWarps) * (kRotateRing * 512 + a.half * 8);
    if (a.interleaved)
      TP_LAUNCH_PDL((rotate_rows_kernel<T, 1, 16, Cache>), g, threads, smem, s, a, c, sh);
    else if (bytes == 16)
      TP_LAUNCH_PDL((rotate_rows_kernel<T, 2, 16, Cache>), g, threads, smem, s, a, c, sh);
    else
      TP_LAUNCH_PDL((rotate_rows_kernel<T, 2, 8, Cache>), g, threads, smem, s, a, c, sh);
    return TP_OK;
  }
  const int64_t n = a.T * rows * (a.hd - a.half);
  const unsigned g = static_cast<unsigned>(std::min<int64_t>(ceil_div(n, 256), num_sms() * 16));
  TP_LAUNCH_PDL((rotate_elements_kernel<T, Cache>), dim3(g), dim3(256), 0, s, a, c);
  return TP_OK;
}

}  // namespace rope
}  // namespace tp
