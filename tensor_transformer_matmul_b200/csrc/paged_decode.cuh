// Attention of one new token per sequence over a paged key/value cache.
//
// Mathematics: one pass over a sequence's keys with the running maximum m and sum l of its softmax:
// o = sum_n e^(z_n - m) v_n / l.  Parts of a sequence are joined by (m, l, o): each part's weight is
// e^(m_part - m).  m, l, scores and o are fp32 throughout.
//
// What bounds it: every key and value is read once and used by the query heads of its group, a few
// operations per byte, so the cache's bytes do.  The kernel is built around keeping loads in flight:
//   * A warp takes 32 keys at a time and stages them itself with 16-byte asynchronous copies into
//     its own part of shared memory, so no warp waits for another in the loop, and a page may end
//     anywhere (a row's address is looked up per key, one table entry per lane).
//   * bf16: scores are K q^T and the output V^T p^T with 16 x 8 x 16 matrix instructions, keys or
//     dims as the rows and the group's heads as the 8 columns, so a group of 8 heads wastes
//     nothing.  The order of the dims inside a product is free: a lane's 16 bytes of a row are its
//     operands of two instructions as they lie; values are paired over two keys by byte permutes.
//     Larger instructions (tcgen05, 64 rows or more) would need the rows staged in the layouts that
//     their descriptors know and gain nothing on a stream that memory bounds.
//   * fp32: products in fp32 on the SIMT units;
//     groups of more than four heads use the matrix instructions on numbers cut into three.
//
// Split: a unit is 32 keys of one (sequence, KV head, tile of query heads); the units of the whole
// batch lie in one line, cut into equal runs, one per block of a grid that fills the GPU once.  So
// one long sequence and a ragged batch load every SM alike, whatever the lengths (which only the
// device knows).  A run that holds the whole of a (sequence, head) writes its output; the others
// leave (m, l, o) for join_kernel.  Caches of short rows use one block per (sequence, head) and no
// second launch.
//
// Measured (64 query / 8 KV heads of 128 bf16 dims, from DRAM): 32 ragged sequences of up to 16384
// keys 198 us, 6.2 TB/s; one of 131071 91 us, 5.9 TB/s; 16 ragged of up to 4096 30 us, 4.9 TB/s (one
// wave of unequal blocks); one of 200 4.7 us (latency of the lookups and copies).
#pragma once

#include "paged.cuh"
#include "sm100.cuh"

namespace tp {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kChunk = 32;       // keys of a unit

struct DecodeArgs {
  View c;
  rope::Rows q, o;
  const void *kp, *vp;
  const int32_t* lens;
  float scale;
  float* lse;
  float* score;
  // split runs
  int64_t* first;                // [b + 2]: units before a sequence, of one head tile; units of a run
  float* pm;                     // [2 * runs][heads of a tile]: maximum
  float* pl;                     // ... sum
  float* po;                     // ... [hd]: output before the division
  float* z;                      // [b][n_kv][cap][zw]: scores, for the weights (may be null)
  int64_t min_units;
  int runs, tiles, zw;           // blocks; head tiles of a group; columns of z
};

// D += A B of 16 x 8 x 16, bf16 with fp32 sums
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
constexpr uint32_t kLeftOut = 0x7fc0dead;   // in place of a score: a NaN that no operation returns
constexpr float kSlack = 5.5f;
// e^(x - m): by the hardware's 2^x (relative error 2^-22; results below 2^-126 are zeros) of the
// difference, which is rounded once where scores in base 2 would be rounded at their full size
__device__ __forceinline__ float exp_above(float x, float m) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((x - m) * kLog2e));
  return y;
}
// maximum that scores are taken relative to: an all -infinity maximum gives weights of 0, not NaN
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

// A staged row is kept with its 16-byte chunks permuted (chunk index xor this): every access below,
// eight lanes at a time, then touches all banks once.
__device__ __forceinline__ int swizzle(int row) { return (((row >> 2) ^ row) & 1) << 2 | (row & 2); }

// ---- the ways to multiply; lane = 4 g + t ----
// bf16: NT tiles of 8 heads; a step is 16 keys.  A lane's scores: keys g and g + 8, heads
// 8 nt + 2 t and the next.
template <int HDP_, int NT>
struct Mma {
  using T = __nv_bfloat16;
  static constexpr int HDP = HDP_, kHeads = 8 * NT, kStep = 16, kOwn = 2 * NT, kKeys = 2;
  static constexpr int kRowBytes = HDP * 2, kStages = 2;
  static constexpr int kShared = 0;                 // block-wide and per-warp scratch
  static constexpr bool kRedo = false, kRedoApart = true;
  static constexpr int kWarpShared = 0;
  uint32_t q[HDP / 32][NT][4];
  float acc[HDP / 16][NT][4];

  __device__ __forceinline__ static int head(int i, int t) { return (i >> 1) * 8 + 2 * t + (i & 1); }
  __device__ __forceinline__ void load_q(const T* qp, int64_t hs, int heads, int hd, char*, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int c = 0; c < HDP / 32; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint4 r = make_uint4(0, 0, 0, 0);
        if (n * 8 + g < heads && c * 32 + t * 8 < hd)
          r = *reinterpret_cast<const uint4*>(qp + (n * 8 + g) * hs + c * 32 + t * 8);
        q[c][n][0] = r.x; q[c][n][1] = r.y; q[c][n][2] = r.z; q[c][n][3] = r.w;
      }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < HDP / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][n][r] = 0.f;
  }
  __device__ __forceinline__ void scores(uint32_t kbuf, float (&z)[kOwn][kKeys], float scale, char*, int lane) {
    // row g (and g + 8), chunk 4 c + t: the swizzle exchanges even and odd c of a lane
    const int g = lane >> 2, t = lane & 3, flip = ((g >> 2) ^ g) & 1;
    const uint32_t at = kbuf + g * kRowBytes + (t ^ (g & 2)) * 16;
    const uint32_t even = at + flip * 64, odd = at + (flip ^ 1) * 64;
    float s[NT][4], u[NT][4];                          // two chains of sums
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[n][r] = u[n][r] = 0.f;
#pragma unroll
    for (int c = 0; c < HDP / 32; ++c) {
      const uint32_t k = (c & 1 ? odd : even) + (c & ~1) * 64;
      const uint4 x = lds16(k), y = lds16(k + 8 * kRowBytes);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816(s[n], x.x, y.x, x.y, y.y, q[c][n][0], q[c][n][1]);
        mma16816(u[n], x.z, y.z, x.w, y.w, q[c][n][2], q[c][n][3]);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) z[2 * n + i][k] = (s[n][2 * k + i] + u[n][2 * k + i]) * scale;
  }
  // key k's scores into its row (columns behind the group's last head hold anything)
  __device__ __forceinline__ static void keep_scores(float* to, const float (&z)[kOwn][kKeys], int k,
                                                     int t, int room) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (8 * n + 2 * t < room)
        *reinterpret_cast<float2*>(to + 8 * n + 2 * t) = make_float2(z[2 * n][k], z[2 * n + 1][k]);
  }
  __device__ __forceinline__ void rescale(const float (&corr)[kOwn]) {
#pragma unroll
    for (int i = 0; i < HDP / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][n][r] *= corr[2 * n + (r & 1)];
  }
  // The weights enter the product as two bf16 parts, value and remainder (2^-17 of a weight is
  // left): with one part alone the output's error would grow from its own rounding's 0.0017 to
  // about 0.0020, and the second product costs nothing on a stream that memory bounds.
  __device__ __forceinline__ void add_values(uint32_t vbuf, const float (&p)[kOwn][kKeys], char*, int lane) {
    // rows 2 t, 2 t + 1 and 8 further, chunk 8 v + g
    const int g = lane >> 2, t = lane & 3, sw = ((t & 2) << 1) | ((t & 1) << 1);
    const uint32_t row0 = vbuf + 2 * t * kRowBytes + (g ^ sw) * 16;
    const uint32_t row1 = vbuf + (2 * t + 1) * kRowBytes + (g ^ sw ^ 4) * 16;
    uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float a = p[2 * n][k], b = p[2 * n + 1][k];
        const uint32_t w = pack_bf16x2(a, b);
        hi[n][k] = transpose8x8(w);
        lo[n][k] = transpose8x8(pack_bf16x2(a - bf16lo(w), b - bf16hi(w)));
      }
#pragma unroll
    for (int v = 0; v < HDP / 64; ++v) {
      uint32_t r[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 x = lds16((k & 1 ? row1 : row0) + (k >> 1) * 8 * kRowBytes + v * 128);
        r[k][0] = x.x; r[k][1] = x.y; r[k][2] = x.z; r[k][3] = x.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = __byte_perm(r[0][i], r[1][i], 0x5410), a1 = __byte_perm(r[0][i], r[1][i], 0x7632);
        const uint32_t a2 = __byte_perm(r[2][i], r[3][i], 0x5410), a3 = __byte_perm(r[2][i], r[3][i], 0x7632);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816(acc[4 * v + i][n], a0, a1, a2, a3, hi[n][0], hi[n][1]);
          mma16816(acc[4 * v + i][n], a0, a1, a2, a3, lo[n][0], lo[n][1]);
        }
      }
    }
  }
  // out: [kHeads][HDP] floats
  __device__ __forceinline__ void store(float* out, int lane) const {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < HDP / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int d = (i >> 2) * 64 + g * 8 + 2 * (i & 3);
          *reinterpret_cast<float2*>(out + (n * 8 + 2 * t + h) * HDP + d) =
              make_float2(acc[i][n][h], acc[i][n][2 + h]);
        }
  }
};

// Two fp32 numbers as the sums of three bf16 numbers each (every remainder is exact; numbers that
// round to an infinite bf16, from 3.3962e38 on, have no parts).
__device__ __forceinline__ void cut3(float a, float b, uint32_t (&w)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    w[i] = pack_bf16x2(a, b);
    a -= bf16lo(w[i]);
    b -= bf16hi(w[i]);
  }
}

// fp32 on the same instructions: a number is the sum of three bf16 numbers, the second at most 2^-8 and
// the third at most 2^-17 of it, and of the nine products of two sums the six largest are taken; what is
// left out is at most 2^-24 of the product (all of an fp32 rounding; two numbers of the same 1 + 2^-8 -
// 2^-17 reach it).  Parts end at 2^-133: numbers below 2^-109 lose last places.  The instructions' own sums are cut off, not rounded, so they run over
// one step or 16 dims only, and fp32 additions join them.  A cut costs 5.5 instructions a number once,
// plain fp32 products one a head.  Layout as above with four dims to 16 bytes; the queries' parts lie
// in shared memory as the lanes' operands.
template <int HDP_, int NT>
struct MmaF32 {
  using T = float;
  static constexpr int HDP = HDP_, kHeads = 8 * NT, kStep = 16, kOwn = 2 * NT, kKeys = 2;
  static constexpr int kRowBytes = HDP * 4, kStages = 1;
  static constexpr int kShared = HDP / 16 * NT * 3 * 256;      // [16 dims][tile][part][lane] pairs
  static constexpr int kWarpShared = 0;
  static constexpr bool kRedo = true, kRedoApart = true;
  float acc[HDP / 16][NT][4];

  __device__ __forceinline__ static int head(int i, int t) { return (i >> 1) * 8 + 2 * t + (i & 1); }
  // (every warp writes the same values and reads behind its own stores, so no order of the warps
  // matters; shares and a barrier put the warps in step: 16 x 4000 keys 76.2 -> 78.1 us)
  __device__ __forceinline__ void load_q(const T* qp, int64_t hs, int heads, int hd, char* sq, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int c0 = 0; c0 < HDP / 16; c0 += 8 / NT) {    // eight loads in flight
      float4 x[8 / NT][NT];
#pragma unroll
      for (int c = 0; c < 8 / NT; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int d = (c0 + c) * 16 + t * 4;
          x[c][n] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c0 + c < HDP / 16 && n * 8 + g < heads && d < hd)
            x[c][n] = *reinterpret_cast<const float4*>(qp + (n * 8 + g) * hs + d);
        }
#pragma unroll
      for (int c = 0; c < 8 / NT; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (c0 + c >= HDP / 16) continue;
          uint32_t lo[3], hi[3];
          cut3(x[c][n].x, x[c][n].y, lo);
          cut3(x[c][n].z, x[c][n].w, hi);
#pragma unroll
          for (int i = 0; i < 3; ++i)
            *reinterpret_cast<uint2*>(sq + (((c0 + c) * NT + n) * 3 + i) * 256 + lane * 8) = make_uint2(lo[i], hi[i]);
        }
    }
    __syncwarp();
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < HDP / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][n][r] = 0.f;
  }
  __device__ __forceinline__ void scores(uint32_t kbuf, float (&z)[kOwn][kKeys], float scale, char* sq, int lane) {
    const int g = lane >> 2, t = lane & 3, flip = ((g >> 2) ^ g) & 1;
    const uint32_t at = kbuf + g * kRowBytes + (t ^ (g & 2)) * 16;
    const uint32_t even = at + flip * 64, odd = at + (flip ^ 1) * 64;
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[n][r] = 0.f;
#pragma unroll
    for (int c = 0; c < HDP / 16; ++c) {
      const uint32_t k = (c & 1 ? odd : even) + (c & ~1) * 64;
      const uint4 x = lds16(k), y = lds16(k + 8 * kRowBytes);
      uint32_t x0[3], x1[3], y0[3], y1[3];
      cut3(__uint_as_float(x.x), __uint_as_float(x.y), x0);
      cut3(__uint_as_float(x.z), __uint_as_float(x.w), x1);
      cut3(__uint_as_float(y.x), __uint_as_float(y.y), y0);
      cut3(__uint_as_float(y.z), __uint_as_float(y.w), y1);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint2 q[3];
#pragma unroll
        for (int i = 0; i < 3; ++i)
          q[i] = *reinterpret_cast<const uint2*>(sq + ((c * NT + n) * 3 + i) * 256 + lane * 8);
        // (part of the key, part of the query), the smallest first
        float u[4] = {0.f, 0.f, 0.f, 0.f};
        mma16816(u, x0[2], y0[2], x1[2], y1[2], q[0].x, q[0].y);
        mma16816(u, x0[0], y0[0], x1[0], y1[0], q[2].x, q[2].y);
        mma16816(u, x0[1], y0[1], x1[1], y1[1], q[1].x, q[1].y);
        mma16816(u, x0[1], y0[1], x1[1], y1[1], q[0].x, q[0].y);
        mma16816(u, x0[0], y0[0], x1[0], y1[0], q[1].x, q[1].y);
        mma16816(u, x0[0], y0[0], x1[0], y1[0], q[0].x, q[0].y);
#pragma unroll
        for (int r = 0; r < 4; ++r) s[n][r] += u[r];
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) z[2 * n + i][k] = s[n][2 * k + i] * scale;
  }
  // An infinite number has no parts: scores that came out as NaN are taken again in plain fp32.
  __device__ __noinline__ static void redo_scores(uint32_t kbuf, float (&z)[kOwn][kKeys], float scale,
                                                  const T* qp, int64_t hs, int heads, int hd, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int k = 0; k < kKeys; ++k) {
        if (head(i, t) >= heads) continue;
        const int row = g + 8 * k;
        float s = 0.f;
        for (int d = 0; d < hd; d += 4) {
          const uint4 x = lds16(kbuf + row * kRowBytes + ((d >> 2) ^ swizzle(row)) * 16);
          const float4 y = *reinterpret_cast<const float4*>(qp + head(i, t) * hs + d);
          s = fmaf(__uint_as_float(x.x), y.x, s);
          s = fmaf(__uint_as_float(x.y), y.y, s);
          s = fmaf(__uint_as_float(x.z), y.z, s);
          s = fmaf(__uint_as_float(x.w), y.w, s);
        }
        z[i][k] = s * scale;
      }
  }
  __device__ __forceinline__ static void keep_scores(float* to, const float (&z)[kOwn][kKeys], int k,
                                                     int t, int room) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (8 * n + 2 * t < room)
        *reinterpret_cast<float2*>(to + 8 * n + 2 * t) = make_float2(z[2 * n][k], z[2 * n + 1][k]);
  }
  __device__ __forceinline__ void rescale(const float (&corr)[kOwn]) {
#pragma unroll
    for (int i = 0; i < HDP / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][n][r] *= corr[2 * n + (r & 1)];
  }
  __device__ __forceinline__ void add_values(uint32_t vbuf, const float (&p)[kOwn][kKeys], char*, int lane) {
    const int g = lane >> 2, t = lane & 3, sw = ((t & 2) << 1) | ((t & 1) << 1);
    const uint32_t row0 = vbuf + 2 * t * kRowBytes + (g ^ sw) * 16;
    const uint32_t row1 = vbuf + (2 * t + 1) * kRowBytes + (g ^ sw ^ 4) * 16;
    uint32_t w[NT][2][3];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        cut3(p[2 * n][k], p[2 * n + 1][k], w[n][k]);
#pragma unroll
        for (int i = 0; i < 3; ++i) w[n][k][i] = transpose8x8(w[n][k][i]);
      }
#pragma unroll
    for (int v = 0; v < HDP / 32; ++v) {
      float r[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 x = lds16((k & 1 ? row1 : row0) + (k >> 1) * 8 * kRowBytes + v * 128);
        r[k][0] = __uint_as_float(x.x); r[k][1] = __uint_as_float(x.y);
        r[k][2] = __uint_as_float(x.z); r[k][3] = __uint_as_float(x.w);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t a0[3], a1[3], a2[3], a3[3];
        cut3(r[0][2 * i], r[1][2 * i], a0);
        cut3(r[0][2 * i + 1], r[1][2 * i + 1], a1);
        cut3(r[2][2 * i], r[3][2 * i], a2);
        cut3(r[2][2 * i + 1], r[3][2 * i + 1], a3);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float to[4] = {0.f, 0.f, 0.f, 0.f};
          mma16816(to, a0[2], a1[2], a2[2], a3[2], w[n][0][0], w[n][1][0]);
          mma16816(to, a0[0], a1[0], a2[0], a3[0], w[n][0][2], w[n][1][2]);
          mma16816(to, a0[1], a1[1], a2[1], a3[1], w[n][0][1], w[n][1][1]);
          mma16816(to, a0[1], a1[1], a2[1], a3[1], w[n][0][0], w[n][1][0]);
          mma16816(to, a0[0], a1[0], a2[0], a3[0], w[n][0][1], w[n][1][1]);
          mma16816(to, a0[0], a1[0], a2[0], a3[0], w[n][0][0], w[n][1][0]);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[2 * v + i][n][r] += to[r];
        }
      }
    }
  }
  __device__ __forceinline__ void store(float* out, int lane) const {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < HDP / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int d = (i >> 1) * 32 + g * 4 + 2 * (i & 1);
          *reinterpret_cast<float2*>(out + (n * 8 + 2 * t + h) * HDP + d) =
              make_float2(acc[i][n][h], acc[i][n][2 + h]);
        }
  }
};

// fp32: G heads (1 or 4); a step is 8 keys.  Four lanes share a key's dims and then its heads:
// a lane's scores: key g, head t (G == 1: all four the same).  A lane owns four
// dims of the output (HDP 256: eight; HDP 64: of every other key).
template <int HDP_, int G>
struct Simt {
  using T = float;
  static constexpr int HDP = HDP_, kHeads = G, kStep = 8, kOwn = G >= 4 ? G / 4 : 1, kKeys = 1;
  static constexpr int kRowBytes = HDP * 4, kStages = 2;
  static constexpr int kShared = G * HDP * 4;
  static constexpr bool kRedo = false, kRedoApart = false;
  static constexpr int kWarpShared = 8 * G * 4;
  static constexpr int kLanes = HDP / 4 < 32 ? HDP / 4 : 32;   // lanes of a row of V
  static constexpr int kRows = 32 / kLanes;                    // rows of a copy of V
  static constexpr int kCols = HDP / 4 / kLanes;               // 16-byte columns of a lane
  float acc[G][kCols][4];

  __device__ __forceinline__ static int head(int i, int t) { return G >= 4 ? t * kOwn + i : 0; }
  // the block's queries in shared memory (every warp writes the same values and reads behind its own
  // stores; shares and a barrier: 16 x 4000 keys, four heads a group, 63.3 -> 67.3 us)
  __device__ __forceinline__ void load_q(const T* qp, int64_t hs, int heads, int hd, char* sq, int lane) {
    float* s = reinterpret_cast<float*>(sq);
    for (int i = lane; i < G * HDP; i += 32) {
      const int h = i / HDP, d = i % HDP;
      s[i] = h < heads && d < hd ? qp[h * hs + d] : 0.f;
    }
    __syncwarp();
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int h = 0; h < G; ++h)
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[h][c][r] = 0.f;
  }
  __device__ __forceinline__ void scores(uint32_t kbuf, float (&z)[kOwn][kKeys], float scale, char* sq, int lane) {
    const int g = lane >> 2, t = lane & 3, flip = ((g >> 2) ^ g) & 1;
    const uint32_t at = kbuf + g * kRowBytes + (t ^ (g & 2)) * 16;
    const uint32_t even = at + flip * 64, odd = at + (flip ^ 1) * 64;
    const uint32_t qa = sm100::smem_addr(sq) + t * 16;
    float s[G];
#pragma unroll
    for (int h = 0; h < G; ++h) s[h] = 0.f;
#pragma unroll 4
    for (int c = 0; c < HDP / 16; ++c) {
      const uint4 x = lds16((c & 1 ? odd : even) + (c & ~1) * 64);
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const uint4 y = lds16(qa + (h * HDP + c * 16) * 4);
        s[h] = fmaf(__uint_as_float(x.x), __uint_as_float(y.x), s[h]);
        s[h] = fmaf(__uint_as_float(x.y), __uint_as_float(y.y), s[h]);
        s[h] = fmaf(__uint_as_float(x.z), __uint_as_float(y.z), s[h]);
        s[h] = fmaf(__uint_as_float(x.w), __uint_as_float(y.w), s[h]);
      }
    }
    if constexpr (G == 1) {
      s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);
      s[0] += __shfl_xor_sync(0xffffffffu, s[0], 2);
      z[0][0] = s[0] * scale;
    } else {
      // halves of the heads change hands: after two exchanges a lane has the sums of its own
      float u[G / 2];
#pragma unroll
      for (int h = 0; h < G / 2; ++h) {
        const float give = t & 2 ? s[h] : s[h + G / 2], have = t & 2 ? s[h + G / 2] : s[h];
        u[h] = have + __shfl_xor_sync(0xffffffffu, give, 2);
      }
#pragma unroll
      for (int h = 0; h < G / 4; ++h) {
        const float give = t & 1 ? u[h] : u[h + G / 4], have = t & 1 ? u[h + G / 4] : u[h];
        z[h][0] = (have + __shfl_xor_sync(0xffffffffu, give, 1)) * scale;
      }
    }
  }
  __device__ __forceinline__ static void keep_scores(float* to, const float (&z)[kOwn][kKeys], int k,
                                                     int t, int room) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (head(i, t) < room && (G >= 4 || t == 0)) to[head(i, t)] = z[i][k];
  }
  __device__ __forceinline__ void rescale(const float (&corr)[kOwn]) {
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float f = __shfl_sync(0xffffffffu, corr[G >= 4 ? h % kOwn : 0], G >= 4 ? h / kOwn : 0);
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[h][c][r] *= f;
    }
  }
  __device__ __forceinline__ void add_values(uint32_t vbuf, const float (&p)[kOwn][kKeys], char* sp, int lane) {
    float* s = reinterpret_cast<float*>(sp);      // [G][8 keys]
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (G >= 4 || (lane & 3) == 0) s[head(i, lane & 3) * 8 + (lane >> 2)] = p[i][0];
    __syncwarp();
    const int sub = lane / kLanes;
#pragma unroll
    for (int r = 0; r < 8 / kRows; ++r) {
      const int row = r * kRows + sub;
      const uint32_t at = vbuf + row * kRowBytes + ((lane % kLanes) ^ swizzle(row)) * 16;
      float w[G];
#pragma unroll
      for (int h = 0; h < G; ++h) w[h] = s[h * 8 + row];
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const uint4 x = lds16(at + c * kLanes * 16);
#pragma unroll
        for (int h = 0; h < G; ++h) {
          acc[h][c][0] = fmaf(w[h], __uint_as_float(x.x), acc[h][c][0]);
          acc[h][c][1] = fmaf(w[h], __uint_as_float(x.y), acc[h][c][1]);
          acc[h][c][2] = fmaf(w[h], __uint_as_float(x.z), acc[h][c][2]);
          acc[h][c][3] = fmaf(w[h], __uint_as_float(x.w), acc[h][c][3]);
        }
      }
    }
  }
  __device__ __forceinline__ void store(float* out, int lane) {
#pragma unroll
    for (int h = 0; h < G; ++h)
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if constexpr (kRows == 2) acc[h][c][r] += __shfl_xor_sync(0xffffffffu, acc[h][c][r], 16);
        if (lane < kLanes)
          *reinterpret_cast<float4*>(out + h * HDP + (c * kLanes + lane) * 4) =
              make_float4(acc[h][c][0], acc[h][c][1], acc[h][c][2], acc[h][c][3]);
      }
  }
};

// shared memory of a warp's ring: two steps of keys and values, or one (kStages) where a step computes
// long enough for twice the warps to keep the memory busy
template <typename E>
constexpr int ring_bytes() { return 2 * E::kStages * E::kStep * E::kRowBytes; }
// Warps of a block that has a row to itself (192 KB of rings, the SM's whole), warps of a block of a
// split launch, and how many of these share an SM.
constexpr int kRings = 192 * 1024;
constexpr int whole_warps(int ring) { return ring * 12 <= kRings ? 12 : kRings / ring; }
constexpr int whole_blocks(int rings) { return rings * 2 <= kRings ? 2 : 1; }   // at least, on an SM
constexpr int split_warps(int ring) { return ring * 6 <= kRings ? 6 : kRings / ring; }
constexpr int split_blocks(int ring) {
  return kRings / (split_warps(ring) * ring) < 3 ? kRings / (split_warps(ring) * ring) : 3;
}
template <typename E>
constexpr int decode_smem(int warps) {
  return warps * (ring_bytes<E>() + E::kWarpShared) + E::kShared + warps * E::kHeads * 8;
}

// Outputs are summed with weights of up to e^kSlack before the division, and as sums of bf16 parts:
// values near the largest number overflow there although their mean does not, and an infinite value
// meets a second part of either sign or of 0.  A warp whose sums lie beyond kFarthest (or are not
// numbers) takes those heads again in plain fp32 (redo_values), with weights that add up to 2^-14:
// then no part exceeds kFarthest, nor does the sum of all parts (444 runs of 6 warps of two halves
// each, or 12 warps) reach 2^127, and what is infinite or NaN in o is so in sum_n w_n v_n.
constexpr float kFarthest = 20769187434139310514121985316880384.f;    // 2^114
constexpr float kRedoShift = 9.7040605f;                               // 14 log 2
template <int A, int B, int C>
__device__ __forceinline__ bool beyond(const float (&acc)[A][B][C]) {
  bool far = false;
#pragma unroll
  for (int i = 0; i < A; ++i)
#pragma unroll
    for (int n = 0; n < B; ++n)
#pragma unroll
      for (int r = 0; r < C; ++r) far |= !(fabsf(acc[i][n][r]) <= kFarthest);
  return far;
}
// out [heads][HDP], sm, sl: the warp's sums, maxima and sums of weights of its keys of k0 .. k1-1.  Not
// made for speed: with an infinite value in every key 32 ragged sequences up to 16384 take 4.0 ms instead
// of 0.2, one of 131071 keys 1.8 ms instead of 0.1 (heads one after another over all keys: 6.5 and 2.9).
template <typename E, int W>
__device__ __forceinline__ void redo_values(const DecodeArgs& a, int64_t seq, int g, int j0, int heads,
                                            int k0, int k1, float* out, float* sm, float* sl) {
  using T = typename E::T;
  constexpr int kDims = E::HDP / 32, kUnit = 16 / sizeof(T);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* qp = static_cast<const T*>(a.q.p) + seq * a.q.ts + j0 * a.q.hs;
  const T* kp = static_cast<const T*>(a.kp) + g * a.c.head_stride;
  const T* vp = static_cast<const T*>(a.vp) + g * a.c.head_stride;
  const int32_t* table = a.c.tables + seq * a.c.max_pages;
  const int hd = a.c.hd;
  // the heads to take again; out, sm and sl hold their sums from here on
  uint32_t again = 0;
  for (int h = 0; h < heads; ++h) {
    const float m = sm[h], l = sl[h];
    bool far = false;
    for (int d = lane; d < hd; d += 32) far |= !(fabsf(out[h * E::HDP + d]) <= kFarthest);
    // (without a sum there is no softmax, or NaN for every dim)
    if (!__any_sync(0xffffffffu, far) || !(l > 0.f)) continue;
    again |= 1u << h;
    for (int d = lane; d < hd; d += 32) out[h * E::HDP + d] = 0.f;
    __syncwarp();
    if (lane == 0) sm[h] = m + logf(l) + kRedoShift, sl[h] = 0.f;
    __syncwarp();
  }
  for (int first = (k0 / kChunk + warp) * kChunk; first < k1; first += W * kChunk) {
    // a lane's key: its score and weight; then all keys' values, a lane the dims it keeps
    const int key = first + lane, pi = key / a.c.page_size;
    const int64_t page = key < k1 ? table[pi] : -1;
    const bool in = page >= 0 && page < a.c.n_pages;
    const int64_t row = in ? page * a.c.page_stride + (key - pi * a.c.page_size) * a.c.slot_stride : 0;
    const uint32_t mask = __ballot_sync(0xffffffffu, in);
    for (uint32_t left = again; left; left &= left - 1) {
      const int h = __ffs(left) - 1;
      float w = 0.f;
      if (in) {
        float z = 0.f;
#pragma unroll 4
        for (int d = 0; d < hd; d += kUnit) {
          alignas(16) T x[kUnit], y[kUnit];
          *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(qp + h * a.q.hs + d);
          *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(kp + row + d);
#pragma unroll
          for (int i = 0; i < kUnit; ++i) z = fmaf(to_f(x[i]), to_f(y[i]), z);
        }
        w = exp_above(z * a.scale, sm[h]);
      }
      float acc[kDims], sum = w;
#pragma unroll
      for (int c = 0; c < kDims; ++c) acc[c] = 0.f;
      constexpr int kRows = 8;              // whose loads fly together
      for (int r = 0; r < kChunk; r += kRows) {
        T v[kRows][kDims];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          const int64_t from = __shfl_sync(0xffffffffu, row, r + k);
#pragma unroll
          for (int c = 0; c < kDims; ++c)
            v[k][c] = ((mask >> (r + k)) & 1u) && c * 32 + lane < hd ? vp[from + c * 32 + lane] : from_f<T>(0.f);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          const float f = __shfl_sync(0xffffffffu, w, r + k);
#pragma unroll
          for (int c = 0; c < kDims; ++c) acc[c] = fmaf(f, to_f(v[k][c]), acc[c]);
        }
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
#pragma unroll
      for (int c = 0; c < kDims; ++c)
        if (c * 32 + lane < hd) out[h * E::HDP + c * 32 + lane] += acc[c];
      if (lane == 0) sl[h] += sum;
      __syncwarp();
    }
  }
}

// As a call where the engine has registers to spare for one; within the kernel for the SIMT engines (one
// head a group, 64 dims, runs: 42.2 us without it, 44.3 with a call, 42.6 within).
template <typename E, int W>
__device__ __noinline__ void redo_apart(const DecodeArgs& a, int64_t seq, int g, int j0, int heads, int k0,
                                        int k1, float* out, float* sm, float* sl) {
  redo_values<E, W>(a, seq, g, j0, heads, k0, k1, out, sm, sl);
}

// Keys k0 .. k1-1 of (sequence, KV head g), heads j0 .. j0+heads-1: this warp's share of them.
// On return the accumulators are in the warp's ring, its maxima and sums in sm / sl; true where an
// accumulator lies beyond kFarthest.
template <typename E, int W>
__device__ __forceinline__ bool warp_pass(const DecodeArgs& a, E& e, int64_t seq, int g, int j0,
                                          int heads, int k0, int k1, char* ring, char* wsh,
                                          char* bsh, float* sm, float* sl, int warp, int lane) {
  using T = typename E::T;
  constexpr int NS = kChunk / E::kStep, kBuf = E::kStep * E::kRowBytes, kUnit = 16 / sizeof(T);
  const int t = lane & 3, g8 = lane >> 2, hd = a.c.hd;
  const T* kp = static_cast<const T*>(a.kp);
  const T* vp = static_cast<const T*>(a.vp);
  const uint32_t buf = sm100::smem_addr(ring);
  const int32_t* table = a.c.tables + seq * a.c.max_pages;
  const T* kl = kp + g * a.c.head_stride + (lane & 7) * kUnit;
  const T* vl = vp + g * a.c.head_stride + (lane & 7) * kUnit;
  const int left = hd - (lane & 7) * kUnit;      // dims from this lane's first chunk on

  // a key's scores, from this tile's heads on; columns left there
  const int room = a.zw - (j0 - g * a.c.group);
  auto z_row = [&](int key) {
    return a.z + ((seq * a.c.n_kv + g) * a.c.cap + key) * a.zw + (j0 - g * a.c.group);
  };
  // a lane looks up the row of one key of a chunk: its table entry first, its offset a chunk later
  struct Entry {
    int32_t page;
    uint32_t slot;
  };
  auto entry_of = [&](int key) -> Entry {
    const uint32_t pi = static_cast<uint32_t>(key) / static_cast<uint32_t>(a.c.page_size);
    return {key < k1 ? table[pi] : -1, key - pi * static_cast<uint32_t>(a.c.page_size)};
  };
  auto row_of = [&](int key, const Entry& x, uint32_t& mask) -> int64_t {
    const bool in = x.page >= 0 && x.page < a.c.n_pages;
    if (!in && key < k1) record_device_error(a.c.err, DEVERR_INDEX);
    mask = __ballot_sync(0xffffffffu, in);
    return in ? x.page * a.c.page_stride + x.slot * a.c.slot_stride : 0;
  };
  // Step s of the chunk whose rows the lanes hold.  Rows without a page are zeros (offset 0 is an
  // address of the pool, and nothing is read), so are the dims that pad a row.
  // Eight lanes copy 128 consecutive bytes of a row, so that every request is a whole line of L2
  // (with 32 and 64 bytes of a row to a request the kernel stopped at 4.6 TB/s).
  // Keys (kv 0), values (kv 1) or both, each a group.
  auto issue = [&](int64_t row, uint32_t mask, int s, int first, int last) {
    constexpr int kPtrs = E::kStep / 4, kLines = E::kRowBytes / 128;
    const int j = lane >> 3;
    const uint32_t to = buf + (s % E::kStages) * 2 * kBuf + j * E::kRowBytes;
    const uint32_t to0 = to + ((lane & 7) ^ swizzle(j)) * 16, to1 = to + ((lane & 7) ^ swizzle(j + 4)) * 16;
    int64_t off[kPtrs];
    bool in[kPtrs];
#pragma unroll
    for (int i = 0; i < kPtrs; ++i) {
      off[i] = __shfl_sync(0xffffffffu, row, s * E::kStep + 4 * i + j);
      in[i] = (mask >> (s * E::kStep + 4 * i + j)) & 1u;
    }
#pragma unroll
    for (int kv = first; kv <= last; ++kv) {
#pragma unroll
      for (int i = 0; i < kPtrs; ++i)
#pragma unroll
        for (int c = 0; c < kLines; ++c)
          copy16((i & 1 ? to1 : to0) + kv * kBuf + 4 * i * E::kRowBytes + c * 128,
                 (kv ? vl : kl) + off[i] + c * 8 * kUnit, in[i] && c * 8 * kUnit < left);
      copy_commit();
    }
  };

  float m[E::kOwn], l[E::kOwn];
#pragma unroll
  for (int i = 0; i < E::kOwn; ++i) m[i] = -INFINITY, l[i] = 0.f;
  e.clear();
  bool seen = false;

  int chunk = k0 / kChunk + warp;
  const int end = (k1 + kChunk - 1) / kChunk;
  const T* qp = static_cast<const T*>(a.q.p) + seq * a.q.ts + j0 * a.q.hs;
  if constexpr (E::kShared == 0) e.load_q(qp, a.q.hs, heads, hd, bsh, lane);
  int64_t row = 0;
  uint32_t mask = 0;
  Entry entry{-1, 0};
  if (chunk < end) {
    const int key = chunk * kChunk + lane;
    row = row_of(key, entry_of(key), mask);
#pragma unroll
    for (int s = 0; s < E::kStages; ++s) issue(row, mask, s, 0, 1);
    if (chunk + W < end) entry = entry_of(key + W * kChunk);
  }
  // queries that go to shared memory: while the first rows are on their way
  if constexpr (E::kShared > 0) e.load_q(qp, a.q.hs, heads, hd, bsh, lane);
  for (; chunk < end; chunk += W) {
    const bool more = chunk + W < end;
    int64_t row_n = 0;
    uint32_t mask_n = 0;
    // what follows in the freed buffers: keys, values or both of the step kStages later
    auto issue_next = [&](int s, int first, int last) {
      const int ahead = s + E::kStages;
      __syncwarp();                               // every lane has read what was there
      if (ahead < NS) {
        issue(row, mask, ahead, first, last);
      } else if (more) {
        if (ahead == NS && first == 0) {
          const int key = (chunk + W) * kChunk + lane;
          row_n = row_of(key, entry, mask_n);
          if (chunk + 2 * W < end) entry = entry_of(key + W * kChunk);
        }
        issue(row_n, mask_n, ahead - NS, first, last);
      } else {
        for (int kv = first; kv <= last; ++kv) copy_commit();
      }
    };
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const uint32_t kb = buf + (s % E::kStages) * 2 * kBuf;
      constexpr int kPending = 2 * E::kStages - 1;   // groups in flight behind the one waited for
      constexpr uint32_t kAll = (1u << E::kStep) - 1u;
      const uint32_t live = (mask >> (s * E::kStep)) & kAll;
      copy_wait<kPending>();                      // this step's keys are there
      __syncwarp();
      if (live) {
        seen = true;
        float z[E::kOwn][E::kKeys];
        e.scores(kb, z, a.scale, bsh, lane);
        if constexpr (E::kRedo) {
          bool nan = false;
#pragma unroll
          for (int i = 0; i < E::kOwn; ++i)
#pragma unroll
            for (int k = 0; k < E::kKeys; ++k) nan |= z[i][k] != z[i][k];
          if (__any_sync(0xffffffffu, nan))
            E::redo_scores(kb, z, a.scale, qp, a.q.hs, heads, hd, lane);
        }
        if (a.z != nullptr) {
#pragma unroll
          for (int k = 0; k < E::kKeys; ++k)
            if ((live >> (g8 + 8 * k)) & 1u) e.keep_scores(z_row(chunk * kChunk + s * E::kStep + g8 + 8 * k), z, k, t, room);
        }
        if (live != kAll) {
#pragma unroll
          for (int k = 0; k < E::kKeys; ++k)
            if (!((live >> (g8 + 8 * k)) & 1u)) {
#pragma unroll
              for (int i = 0; i < E::kOwn; ++i) z[i][k] = -INFINITY;
            }
        }
        // The scores are taken relative to a maximum that grows only where one exceeds it by more
        // than kSlack: weights up to e^kSlack lose nothing in fp32, and most steps need no
        // exchange between lanes and no rescaling.
        bool grew = false;
#pragma unroll
        for (int i = 0; i < E::kOwn; ++i)
#pragma unroll
          for (int k = 0; k < E::kKeys; ++k) grew |= z[i][k] > m[i] + kSlack;
        if (__any_sync(0xffffffffu, grew)) {
          float corr[E::kOwn];
#pragma unroll
          for (int i = 0; i < E::kOwn; ++i) {
            float x = z[i][0];
            if constexpr (E::kKeys == 2) x = fmaxf(x, z[i][1]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float mn = fmaxf(m[i], x);
            corr[i] = exp_above(m[i], base_of(mn));
            m[i] = mn;
            l[i] *= corr[i];
          }
          e.rescale(corr);
        }
#pragma unroll
        for (int i = 0; i < E::kOwn; ++i)
#pragma unroll
          for (int k = 0; k < E::kKeys; ++k) {
            z[i][k] = exp_above(z[i][k], base_of(m[i]));
            l[i] += z[i][k];
          }
        if constexpr (E::kStages == 1) issue_next(s, 0, 0);
        copy_wait<2 * E::kStages - 2 + (E::kStages == 1)>();   // and its values
        __syncwarp();
        e.add_values(kb + kBuf, z, wsh, lane);
      }
      if constexpr (E::kStages == 1) {
        if (!live) issue_next(s, 0, 0);
        copy_wait<1>();                           // (nothing lands in the values' buffer any more)
        issue_next(s, 1, 1);
      } else {
        copy_wait<2>();
        issue_next(s, 0, 1);
      }
      if (a.z != nullptr && live != kAll && lane < E::kStep && !((live >> lane) & 1u)) {
        const int key = chunk * kChunk + s * E::kStep + lane;
        if (key < k1) *z_row(key) = __uint_as_float(kLeftOut);
      }
    }
    row = row_n;
    mask = mask_n;
  }
  copy_wait<0>();
  __syncwarp();
#pragma unroll
  for (int i = 0; i < E::kOwn; ++i) {
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
    if (g8 == 0 && (E::kHeads >= 4 || t == 0)) {
      sm[E::head(i, t)] = m[i];
      // a sum of 0: no key, or keys whose scores are all -infinity, which have no softmax.  The
      // second is marked by a negative sum.
      sl[E::head(i, t)] = seen && l[i] == 0.f ? -1.f : l[i];
    }
  }
  const bool far = __any_sync(0xffffffffu, beyond(e.acc));
  e.store(reinterpret_cast<float*>(ring), lane);
  __syncwarp();
  return far;
}

// Weight of a part with maximum pm and sum pl where the joined maximum is m.
__device__ __forceinline__ float part_weight(float pm, float pl, float m) {
  return pl == 0.f || pl == -1.f ? 0.f : exp_above(pm, base_of(m));
}

template <typename T>
__device__ __forceinline__ void store4(T* p, float a, float b, float c, float d) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
  else
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

// 1 / l of a joined sum; none < 0: keys without a softmax (NaN), no keys at all: 0
__device__ __forceinline__ float inverse_sum(float l, bool none) {
  return l == 0.f ? (none ? NAN : 0.f) : 1.f / l;
}

// The weights that the group's heads gave to keys first, first + stride, ...: e^(z - lse), heads in
// order.  s_lse: those of the first kWeightHeads heads (lse has all).
constexpr int kWeightHeads = 64;
__device__ __forceinline__ void add_weights(const DecodeArgs& a, int64_t seq, int g, int n,
                                            const float* s_lse, const float* lse, int first, int stride) {
  constexpr int kKeys = 4;       // keys of a thread whose loads fly together
  const int64_t row = (seq * a.c.n_kv + g) * a.c.cap;
  for (int i0 = first; i0 < n; i0 += kKeys * stride) {
    float w[kKeys], old[kKeys];
    bool take[kKeys];
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
      take[k] = i0 + k * stride < n;
      w[k] = 0.f;
      old[k] = take[k] ? a.score[row + i0 + k * stride] : 0.f;
    }
#pragma unroll 2
    for (int h = 0; h < a.c.group; h += 4) {
      float4 x[kKeys];
#pragma unroll
      for (int k = 0; k < kKeys; ++k)
        if (i0 + k * stride < n)
          x[k] = *reinterpret_cast<const float4*>(a.z + (row + i0 + k * stride) * a.zw + h);
#pragma unroll
      for (int k = 0; k < kKeys; ++k) {
        if (!take[k]) continue;
        if (h == 0) take[k] = __float_as_uint(x[k].x) != kLeftOut;
        const float v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (h + r < a.c.group)
            w[k] += exp_above(v[r], h + r < kWeightHeads ? s_lse[h + r] : lse[h + r]);
      }
    }
#pragma unroll
    for (int k = 0; k < kKeys; ++k)
      if (take[k]) a.score[row + i0 + k * stride] = old[k] + w[k];
  }
}

// Joins the warps' parts of keys k0 .. k1-1 and writes the output (slot < 0) or a part.
template <typename E, int W>
__device__ __forceinline__ void block_piece(const DecodeArgs& a, E& e, int64_t seq, int g, int ht,
                                            int k0, int k1, int64_t slot, char* smem) {
  using T = typename E::T;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  char* ring = smem + warp * ring_bytes<E>();
  char* wsh = smem + W * ring_bytes<E>() + warp * E::kWarpShared;
  char* bsh = smem + W * (ring_bytes<E>() + E::kWarpShared);
  float* sm = reinterpret_cast<float*>(bsh + E::kShared);
  float* sl = sm + W * E::kHeads;
  const int j0 = g * a.c.group + ht * E::kHeads;
  const int heads = min(E::kHeads, a.c.group - ht * E::kHeads);
  const int hd = a.c.hd;
  const int busy = min(W, (k1 - k0 + kChunk - 1) / kChunk);     // warps that get keys
  if (warp < busy) {
    float *m = sm + warp * E::kHeads, *l = sl + warp * E::kHeads, *out = reinterpret_cast<float*>(ring);
    if (warp_pass<E, W>(a, e, seq, g, j0, heads, k0, k1, ring, wsh, bsh, m, l, warp, lane)) {
      if constexpr (E::kRedoApart) redo_apart<E, W>(a, seq, g, j0, heads, k0, k1, out, m, l);
      else redo_values<E, W>(a, seq, g, j0, heads, k0, k1, out, m, l);
    }
  }
  __syncthreads();
  const int cols = hd / 4;
  for (int i = tid; i < heads * cols; i += W * 32) {
    const int h = i / cols, d = (i - h * cols) * 4;
    float mx = -INFINITY;
    bool none = false;
#pragma unroll
    for (int w = 0; w < W; ++w)
      if (w < busy) mx = fmaxf(mx, sm[w * E::kHeads + h]);
    float l = 0.f;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w >= busy) break;
      const float pl = sl[w * E::kHeads + h], f = part_weight(sm[w * E::kHeads + h], pl, mx);
      none |= pl == -1.f;
      if (pl == 0.f || pl == -1.f) continue;
      const float4 x = *reinterpret_cast<const float4*>(smem + w * ring_bytes<E>() + (h * E::HDP + d) * 4);
      l = fmaf(pl, f, l);
      s.x = fmaf(x.x, f, s.x); s.y = fmaf(x.y, f, s.y);
      s.z = fmaf(x.z, f, s.z); s.w = fmaf(x.w, f, s.w);
    }
    if (slot < 0) {
      const float inv = inverse_sum(l, none);
      T* o = static_cast<T*>(const_cast<void*>(a.o.p)) + seq * a.o.ts + (j0 + h) * a.o.hs + d;
      store4(o, s.x * inv, s.y * inv, s.z * inv, s.w * inv);
      if (d == 0) a.lse[seq * a.c.n_q + j0 + h] = mx + logf(l);
    } else {
      *reinterpret_cast<float4*>(a.po + (slot * E::kHeads + h) * hd + d) = s;
      if (d == 0) {
        a.pm[slot * E::kHeads + h] = mx;
        a.pl[slot * E::kHeads + h] = l == 0.f && none ? -1.f : l;
      }
    }
  }
  __syncthreads();
}

// One block per (head tile, KV head, sequence).
template <typename E, int W>
__global__ void __launch_bounds__(W * 32, whole_blocks(W * ring_bytes<E>())) decode_whole_kernel(const __grid_constant__ DecodeArgs a) {
  extern __shared__ __align__(128) char smem[];
  pdl_wait();
  pdl_trigger();
  const int64_t seq = blockIdx.y;
  const int n = static_cast<int>(a.c.keys(a.lens, seq));
  if (blockIdx.x == 0 && threadIdx.x == 0 && n != a.lens[seq]) record_device_error(a.c.err, DEVERR_INDEX);
  E e;
  const int g = blockIdx.x / a.tiles;
  block_piece<E, W>(a, e, seq, g, blockIdx.x % a.tiles, 0, n, -1, smem);
  // the scores that this block left behind, as weights, where it has all heads of the group
  if (a.z != nullptr && a.tiles == 1) {
    const float* lse = a.lse + seq * a.c.n_q + g * a.c.group;
    float* s_lse = reinterpret_cast<float*>(smem);
    for (int h = threadIdx.x; h < a.c.group; h += blockDim.x) s_lse[h] = lse[h];
    __syncthreads();
    add_weights(a, seq, g, n, s_lse, lse, threadIdx.x, blockDim.x);
  }
}

// a / b for a >= 0, b > 0; most quotients here fit the quicker 32-bit division
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// One block per run of units.  A run that ends one row of keys and begins the next passes over two
// parts, one after the other; where there are few rows (a quarter of the runs at most) every row is
// given a whole number of runs instead, its last one partly empty, and no run has two parts (3 x 1123
// fp32 keys, 24 rows on 296 runs: 22.9 -> 17.8 us; 16 x 4000, 128 rows on 148 runs, would lose: 76 -> 95).
template <typename E>
__global__ void __launch_bounds__(split_warps(ring_bytes<E>()) * 32, split_blocks(ring_bytes<E>()))
    decode_split_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int W = split_warps(ring_bytes<E>());
  extern __shared__ __align__(128) char smem[];
  __shared__ int64_t s_sum[2][W], s_seq, s_first;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t tiles = static_cast<int64_t>(a.c.n_kv) * a.tiles;
  const int64_t per_thread = (a.c.b + W * 32 - 1) / (W * 32);
  const int64_t q0 = min(tid * per_thread, a.c.b), q1 = min(q0 + per_thread, a.c.b);
  int64_t grain = 1;                             // a row's units are a multiple of this
  auto chunks = [&](int64_t seq) {
    const int64_t n = (a.c.keys(a.lens, seq) + kChunk - 1) / kChunk;
    return grain == 1 ? n : quotient(n + grain - 1, grain) * grain;
  };
  // units of this thread's sequences, before them, and of all
  int64_t sum, before, total;
  auto count = [&](int64_t* s_part) {
    sum = 0;
    for (int64_t s = q0; s < q1; ++s) sum += chunks(s);
    int64_t x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_part[warp] = x;
    __syncthreads();
    before = x - sum;
    total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) before += s_part[w];
      total += s_part[w];
    }
  };
  count(s_sum[0]);
  // units of a run: at least min_units, so that short work is not cut into parts that cost more to
  // join than to compute
  const int64_t rows = a.c.b * tiles;
  const bool aligned = rows * 4 <= a.runs;
  const int64_t cuts = aligned ? a.runs - rows : a.runs;
  const int64_t per = max(quotient(total * tiles + cuts - 1, cuts), a.min_units);
  if (aligned) {
    grain = per;
    count(s_sum[1]);
  }
  const int64_t units = total * tiles;
  const int64_t u0 = blockIdx.x * per, u1 = min(u0 + per, units);
  if (blockIdx.x == 0) {
    int64_t at = before;
    for (int64_t s = q0; s < q1; ++s) {
      a.first[s] = at;
      at += chunks(s);
      if (a.c.keys(a.lens, s) != a.lens[s]) record_device_error(a.c.err, DEVERR_INDEX);
    }
    if (tid == 0) {
      a.first[a.c.b] = total;
      a.first[a.c.b + 1] = per;
    }
  }
  if (u0 >= units) return;
  if (sum > 0 && before * tiles <= u0 && u0 < (before + sum) * tiles) {
    int64_t s = q0, at = before;
    while ((at + chunks(s)) * tiles <= u0) at += chunks(s++);
    s_seq = s;
    s_first = at;
  }
  __syncthreads();
  int64_t seq = s_seq, first = s_first * tiles, u = u0;
  E e;
  while (u < u1) {
    const int64_t n = chunks(seq);
    if (n == 0 || u >= first + n * tiles) {
      first += n * tiles;
      ++seq;
      continue;
    }
    const int64_t tile = quotient(u - first, n), begin = first + tile * n;
    const int64_t stop = min(begin + n, u1);
    const int k0 = static_cast<int>(u - begin) * kChunk;
    const int k1 = static_cast<int>(min((stop - begin) * kChunk, a.c.keys(a.lens, seq)));
    const bool whole = u == begin && stop == begin + n;
    block_piece<E, W>(a, e, seq, static_cast<int>(tile / a.tiles), static_cast<int>(tile % a.tiles), k0,
                      k1, whole ? -1 : 2 * static_cast<int64_t>(blockIdx.x) + (u == u0 ? 0 : 1), smem);
    u = stop;
  }
}

// One block per (query head, sequence) that was cut: its parts, in the order of its keys.  It reads
// little and waits for what it reads, so everything that one step of 32 parts needs is loaded at
// once: each lane one part's maximum and sum, each warp eight parts' outputs.
template <typename T, int kHeads>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ DecodeArgs a) {
  __shared__ float4 s_o[4][64];
  pdl_wait();
  pdl_trigger();
  const int j = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hd = a.c.hd;
  const int64_t seq = blockIdx.y, tiles = static_cast<int64_t>(a.c.n_kv) * a.tiles;
  const int64_t f = a.first[seq], n = a.first[seq + 1] - f, per = a.first[a.c.b + 1];
  const int g = j / a.c.group, ht = (j - g * a.c.group) / kHeads, h = (j - g * a.c.group) % kHeads;
  const int64_t u0 = f * tiles + (static_cast<int64_t>(g) * a.tiles + ht) * n, u1 = u0 + n;
  T* o = static_cast<T*>(const_cast<void*>(a.o.p)) + seq * a.o.ts + j * a.o.hs;
  if (n == 0) {
    for (int d = tid * 4; d < hd; d += 512) store4(o + d, 0.f, 0.f, 0.f, 0.f);
    if (tid == 0) a.lse[seq * a.c.n_q + j] = -INFINITY;
    return;
  }
  const int64_t c0 = quotient(u0, per), c1 = quotient(u1 - 1, per);
  if (c0 == c1) return;
  const int parts = static_cast<int>(c1 - c0) + 1;
  const int64_t slot0 = (2 * c0 + (u0 > c0 * per ? 1 : 0)) * kHeads + h, slot1 = 2 * (c0 + 1) * kHeads + h;
  auto slot = [&](int c) { return c == 0 ? slot0 : slot1 + (c - 1) * (2 * kHeads); };
  float mx = -INFINITY, l = 0.f;
  bool none = false;
  float4 s[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int b = 0; b < parts; b += 32) {
    float4 x[2][8];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int d = (r * 32 + lane) * 4;
      if (d >= hd) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = b + warp + 4 * k;
        if (c < parts) x[r][k] = *reinterpret_cast<const float4*>(a.po + slot(c) * hd + d);
      }
    }
    const bool mine = b + lane < parts;
    const float pm = mine ? a.pm[slot(b + lane)] : -INFINITY, pl = mine ? a.pl[slot(b + lane)] : 0.f;
    float mn = fmaxf(mx, pm);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, i));
    const float keep = exp_above(mx, base_of(mn)), w = part_weight(pm, pl, mn);
    mx = mn;
    none |= pl == -1.f;
    l = l * keep + (pl == 0.f || pl == -1.f ? 0.f : pl * w);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if ((r * 32 + lane) * 4 >= hd) continue;
      s[r].x *= keep; s[r].y *= keep; s[r].z *= keep; s[r].w *= keep;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float f = __shfl_sync(0xffffffffu, w, warp + 4 * k);
      if (b + warp + 4 * k >= parts) continue;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if ((r * 32 + lane) * 4 >= hd) continue;
        s[r].x = fmaf(x[r][k].x, f, s[r].x); s[r].y = fmaf(x[r][k].y, f, s[r].y);
        s[r].z = fmaf(x[r][k].z, f, s[r].z); s[r].w = fmaf(x[r][k].w, f, s[r].w);
      }
    }
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
  const float inv = inverse_sum(l, __any_sync(0xffffffffu, none));
  s_o[warp][lane] = s[0];
  s_o[warp][32 + lane] = s[1];
  __syncthreads();
  if (tid * 4 < hd) {
    float4 x = s_o[0][tid];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      x.x += s_o[w][tid].x; x.y += s_o[w][tid].y;
      x.z += s_o[w][tid].z; x.w += s_o[w][tid].w;
    }
    store4(o + tid * 4, x.x * inv, x.y * inv, x.z * inv, x.w * inv);
  }
  if (tid == 0) a.lse[seq * a.c.n_q + j] = mx + logf(l);
}

// score += the group's weights of each key, for the cut rows and the tiled groups.
static __global__ void __launch_bounds__(256) weights_kernel(const __grid_constant__ DecodeArgs a) {
  __shared__ float s_lse[kWeightHeads];
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y;
  const int64_t seq = blockIdx.z;
  const int n = static_cast<int>(a.c.keys(a.lens, seq));
  const float* lse = a.lse + seq * a.c.n_q + g * a.c.group;
  for (int h = threadIdx.x; h < min(a.c.group, kWeightHeads); h += 256) s_lse[h] = lse[h];
  __syncthreads();
  add_weights(a, seq, g, n, s_lse, lse, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

}  // namespace paged
}  // namespace tp
