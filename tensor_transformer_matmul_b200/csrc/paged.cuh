// The paged key/value cache: append, decode attention over it, eviction by accumulated weight.
#pragma once

#include <algorithm>

#include "rope.cuh"
#include "tp_common.cuh"

namespace tp {
namespace paged {

// Device view of a cache: addressing and the bounds that every index is checked against.
struct View {
  int64_t page_stride, head_stride, slot_stride;
  int64_t n_pages, max_pages, cap;    // cap: slots of a table row
  int64_t b;
  int n_q, n_kv, group, hd, page_size;
  const int32_t* tables;
  uint32_t* err;

  // element offset of (sequence, head, slot n), -1 when the table has no page of the pool there
  __device__ __forceinline__ int64_t at(int64_t seq, int g, int64_t n) const {
    const int64_t pi = n / page_size;
    const int64_t page = tables[seq * max_pages + pi];
    if (page < 0 || page >= n_pages) return -1;
    return page * page_stride + g * head_stride + (n - pi * page_size) * slot_stride;
  }
  // keys of a sequence, as far as its table goes
  __device__ __forceinline__ int64_t keys(const int32_t* lens, int64_t seq) const {
    const int64_t n = lens[seq];
    return n < 0 ? 0 : (n > cap ? cap : n);
  }
};

inline tp_status check_desc(const tp_paged_desc* d, View* v) {
  if (!d) return set_error(TP_ERR_INVALID_ARG, "desc is null");
  if (d->b < 0 || d->b > 65535) return set_error(TP_ERR_SHAPE, "b must be in [0, 65535]");
  if (d->n_q < 1 || d->n_kv < 1) return set_error(TP_ERR_SHAPE, "n_q and n_kv must be >= 1");
  if (d->n_q % d->n_kv) return set_error(TP_ERR_SHAPE, "n_kv must divide n_q");
  if (d->n_q > 65535) return set_error(TP_ERR_SHAPE, "n_q must be <= 65535");
  if (d->head_dim < 8 || d->head_dim > 256 || d->head_dim % 8)
    return set_error(TP_ERR_SHAPE, "head_dim must be a multiple of 8 in [8, 256]");
  if (d->dtype != TP_F32 && d->dtype != TP_BF16) return set_error(TP_ERR_INVALID_ARG, "dtype");
  if (d->flags != 0) return set_error(TP_ERR_INVALID_ARG, "unknown flags");
  if (d->page_size < 1 || d->n_pages < 1 || d->n_pages > INT32_MAX || d->max_pages < 1)
    return set_error(TP_ERR_SHAPE, "page_size, n_pages and max_pages must be >= 1");
  // (slots, and what a kernel adds to them for its steps, are 32-bit numbers)
  if (d->max_pages > (1 << 30) / d->page_size)
    return set_error(TP_ERR_SHAPE, "max_pages * page_size must be <= 2^30");
  if (!(d->scale >= 0.f) || !std::isfinite(d->scale))
    return set_error(TP_ERR_INVALID_ARG, "scale must be finite and >= 0");
  v->b = d->b;
  v->n_pages = d->n_pages;
  v->max_pages = d->max_pages;
  v->cap = d->max_pages * d->page_size;
  v->n_q = d->n_q; v->n_kv = d->n_kv; v->group = d->n_q / d->n_kv; v->hd = d->head_dim;
  v->page_size = d->page_size;
  v->page_stride = d->page_stride; v->head_stride = d->head_stride; v->slot_stride = d->slot_stride;
  if (!d->page_stride && !d->head_stride && !d->slot_stride) {
    v->slot_stride = d->head_dim;
    v->head_stride = v->slot_stride * d->page_size;
    v->page_stride = v->head_stride * d->n_kv;
  }
  const int64_t unit = 16 / elem_bytes(d->dtype);
  // the three strides must not make two slots overlap: sort them and let each cover the ones below
  struct Dim { int64_t n, st; } dim[3] = {{d->n_pages, v->page_stride}, {d->n_kv, v->head_stride},
                                          {d->page_size, v->slot_stride}};
  std::sort(dim, dim + 3, [](const Dim& a, const Dim& b) { return a.st < b.st; });
  int64_t span = d->head_dim;
  for (const Dim& x : dim) {
    if (x.st < 0 || x.st % unit) return set_error(TP_ERR_INVALID_ARG, "strides must be multiples of 16 bytes");
    if (x.n == 1) continue;
    if (x.st < span) return set_error(TP_ERR_INVALID_ARG, "the strides make slots of the cache overlap");
    if (x.st > (int64_t(1) << 56) / x.n) return set_error(TP_ERR_SHAPE, "the cache is too large");
    span += x.st * (x.n - 1);
  }
  v->tables = nullptr;
  v->err = nullptr;
  return TP_OK;
}

inline float scale_of(const tp_paged_desc* d) {
  return d->scale > 0.f ? d->scale : 1.0f / sqrtf(static_cast<float>(d->head_dim));
}

inline tp_status check_pages(const void* k, const void* v, const void* tables) {
  if (!k || !v || !tables) return set_error(TP_ERR_INVALID_ARG, "null pointer");
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15)
    return set_error(TP_ERR_INVALID_ARG, "k_pages and v_pages must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(tables) & 3)
    return set_error(TP_ERR_INVALID_ARG, "tables must be 4-byte aligned");
  return TP_OK;
}

// ---------------------------------------------------------------------------------- append
// The cache as the destination of a token's k and v rows (rope.cuh moves them).
struct Target {
  rope::Rows k, v;
  void *kp, *vp;
  int64_t head_stride;
  int n_kv;
  View c;
  const int32_t* seq_ids;
  const int32_t* slots;
  __device__ __forceinline__ int64_t slot(int64_t t, bool report) const {
    const int64_t n = slots[t];
    if (n < 0) return -1;
    const int64_t seq = seq_ids ? seq_ids[t] : t;
    const int64_t off = seq >= 0 && seq < c.b && n < c.cap ? c.at(seq, 0, n) : -1;
    if (off < 0 && report) record_device_error(c.err, DEVERR_INDEX);
    return off;
  }
};

inline bool vector_rows(const Target& t, int eb, int bytes) {   // (the cache's strides fit 16)
  return rope::vector_rows(t.k, eb, bytes) && rope::vector_rows(t.v, eb, bytes);
}

// ---------------------------------------------------------------------------------- evict
struct EvictArgs {
  View c;
  float* score;
  const int32_t* lens;
  int32_t* new_lens;
  int32_t* keep_out;    // may be null
  int32_t* keep;        // [b][n_kv][budget]
  int32_t* cut;         // [b][n_kv]: 1 where the sequence is longer than the budget
  int32_t* new_ws;      // [b]
  int budget, recent, room, strips;
  void *kp, *vp;
};

// A score as an unsigned number of the same order: NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t rank_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kEvictThreads = 1024, kEvictWarps = kEvictThreads / 32;
constexpr int kEvictRoom = 50000;      // scores that a block keeps in shared memory

// Sum over the threads before this one; s_warp: kEvictWarps ints.
__device__ __forceinline__ int sum_before(int v, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  return (warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0) + x - v;
}

// One block per (KV head, sequence).  The scores are read once into shared memory (rows longer than
// kEvictRoom: from L2 each time).  Three passes find the smallest score that stays, by 12, 10 and 10
// bits: counts by digit (12 bits spread the scores' few octaves over enough counters), and a sum
// over the digits from above.  Then every warp has a run of slots: it counts what stays of it, and
// with the counts before it writes the kept slots in order, of the scores equal to the smallest the
// first ones.  Bound by the latency of its steps; the rows it selects cost far more to move.
static __global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ float s_score[];
  __shared__ int s_hist[4096 + 2 * 1024], s_warp[3][kEvictWarps], s_above[kEvictWarps], s_ties[kEvictWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_want;
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t seq = blockIdx.y, sg = seq * a.c.n_kv + g;
  const int n = static_cast<int>(a.c.keys(a.lens, seq)), budget = a.budget;
  if (tid == 0 && n != a.lens[seq]) record_device_error(a.c.err, DEVERR_INDEX);
  float* score = a.score + sg * a.c.cap;
  int32_t* keep = a.keep + sg * budget;
  int32_t* out = a.keep_out ? a.keep_out + sg * budget : nullptr;
  if (tid == 0) {
    a.cut[sg] = n > budget;
    if (g == 0) a.new_ws[seq] = min(n, budget);
  }
  if (n <= budget) {
    if (out)
      for (int i = tid; i < budget; i += kEvictThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int old = n - a.recent;             // candidates: slots 0 .. old-1
  const int pick = budget - a.recent;       // how many of them stay (< old)
  const bool held = n <= a.room;
  for (int i = tid; i < 4096 + 2 * 1024; i += kEvictThreads) s_hist[i] = 0;
  if (held) {
    for (int i0 = tid; i0 < n; i0 += 8 * kEvictThreads) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i0 + k * kEvictThreads < n) x[k] = score[i0 + k * kEvictThreads];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i0 + k * kEvictThreads < n) s_score[i0 + k * kEvictThreads] = x[k];
    }
  }
  const float* from = held ? s_score : score;
  __syncthreads();
  uint32_t prefix = 0;
  int want = pick;
  if (pick > 0) {
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      constexpr int kShift[3] = {20, 10, 0}, kFirst[3] = {0, 4096, 4096 + 1024};
      const int shift = kShift[p], per = p == 0 ? 4 : 1;
      const uint32_t digits = p == 0 ? 4096 : 1024, mask = p == 0 ? 0u : 0xffffffffu << (p == 1 ? 20 : 10);
      int* hist = s_hist + kFirst[p];
      for (int i0 = warp * 32; i0 < old; i0 += kEvictThreads) {
        const int i = i0 + lane;
        const uint32_t u = i < old ? rank_of(from[i]) : 0u;
        const bool in = i < old && (u & mask) == prefix;
        const uint32_t d = in ? (u >> shift) & (digits - 1) : digits;
        int same;
        __match_all_sync(0xffffffffu, d, &same);       // equal scores: one count for the warp
        if (in && (!same || lane == 0)) atomicAdd(&hist[d], same ? 32 : 1);
      }
      __syncthreads();
      // this thread's digits, from above; the one whose sum from above reaches ``want``
      int c[4], sum = 0;
      const int top = static_cast<int>(digits) - 1 - tid * per;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < per) sum += c[k] = hist[top - k];
      int before = sum_before(sum, s_warp[p]);
      if (before < want && before + sum >= want) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k >= per) break;
          if (before < want && before + c[k] >= want) {
            s_prefix = prefix | static_cast<uint32_t>(top - k) << shift;
            s_want = want - before;
          }
          before += c[k];
        }
      }
      __syncthreads();
      prefix = s_prefix;
      want = s_want;
    }
  }
  // above the threshold: all; equal to it: the first ``want`` by slot
  const int run = (old + kEvictThreads - 1) / kEvictThreads * 32, begin = min(warp * run, old),
            end = min(begin + run, old);
  int above = 0, ties = 0;
  for (int i = begin + lane; i < end; i += 32) {
    const uint32_t u = rank_of(from[i]);
    above += u > prefix;
    ties += u == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) s_above[warp] = above, s_ties[warp] = ties;
  __syncthreads();
  int at = 0, tie = 0;
  for (int w = 0; w < warp; ++w) at += s_above[w], tie += s_ties[w];
  at += min(tie, want);
  for (int i0 = begin; i0 < end && pick > 0; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t u = i < end ? rank_of(from[i]) : 0u;
    const uint32_t same = __ballot_sync(0xffffffffu, i < end && u == prefix), below = (1u << lane) - 1u;
    const bool stays = i < end && (u > prefix || (u == prefix && tie + __popc(same & below) < want));
    const uint32_t all = __ballot_sync(0xffffffffu, stays);
    if (stays) {
      const int j = at + __popc(all & below);
      keep[j] = i;
      if (out) out[j] = i;
      if (held) score[j] = from[i];
    }
    at += __popc(all);
    tie += __popc(same);
  }
  for (int i = tid; i < a.recent; i += kEvictThreads) {
    keep[pick + i] = old + i;
    if (out) out[pick + i] = old + i;
    if (held) score[pick + i] = from[old + i];
  }
  if (held) return;
  // the kept scores move down in place: a kept score never moves up, and what a step writes was
  // read by it or by an earlier one
  __syncthreads();
  for (int j0 = 0; j0 < budget; j0 += kEvictThreads) {
    const int j = j0 + tid;
    const float v = j < budget ? score[keep[j]] : 0.f;
    __syncthreads();
    if (j < budget) score[j] = v;
    __syncthreads();
  }
}

// One block per (KV head, sequence, K or V, 128-byte strip of a row): the kept rows' strips move
// down in place, chunks of 32 rows dealt to the warps in turn, each with a ring of kMoveDepth of them
// in shared memory.  Row j comes from slot keep[j] >= j: a round's chunks are written once they and
// all before them were read, and rows that were written are never read again, so reading ahead needs
// nothing but that order.  Bound by the bytes: each kept row is read and written once, by whole lines
// of L2.  Eight warps: one alone moves about 8 GB/s, so few strips need many, and for many strips
// the barrier of a round costs little (8 heads of 128 bf16 dims, 1 / 2 / 4 / 8 / 16 warps: 30000
// keys of one sequence cut to 20000 388 / 229 / 142 / 116 / 108 us, 32 sequences of 4000 cut to
// 2000 87 / 87 / 81 / 76 / 82 us).
constexpr int kMoveWarps = 8, kMoveDepth = 3;
constexpr int kMoveRing = kMoveDepth * (4096 + 256);       // bytes of a warp: rows and where they go
static __global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(const __grid_constant__ EvictArgs a,
                                                                            int eb) {
  extern __shared__ __align__(128) char smem[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = blockIdx.x, g = blockIdx.y;
  const int64_t seq = blockIdx.z, sg = seq * a.c.n_kv + g;
  if (part == 0 && g == 0 && threadIdx.x == 0) a.new_lens[seq] = a.new_ws[seq];
  if (!a.cut[sg]) return;
  const int32_t* keep = a.keep + sg * a.budget;
  const int32_t* table = a.c.tables + seq * a.c.max_pages;
  const int col = (part >> 1) * 128 + (lane & 7) * 16, sub = lane >> 3, budget = a.budget;
  char* base = static_cast<char*>(part & 1 ? a.vp : a.kp) + g * a.c.head_stride * eb + col;
  const bool mine = col < a.c.hd * eb;
  char* own = smem + warp * kMoveRing;
  const uint32_t ring = sm100::smem_addr(own) + lane * 16;
  int64_t* s_to = reinterpret_cast<int64_t*>(own + kMoveDepth * 4096);    // [kMoveDepth][32] byte offsets
  const int rounds = (budget + 32 * kMoveWarps - 1) / (32 * kMoveWarps);                // of a chunk per warp
  const uint32_t page_size = static_cast<uint32_t>(a.c.page_size);
  auto offset = [&](int slot, int32_t page) -> int64_t {
    const int in = slot - static_cast<int>(static_cast<uint32_t>(slot) / page_size * page_size);
    return (page * a.c.page_stride + in * a.c.slot_stride) * eb;
  };
  auto valid = [&](int32_t page) { return page >= 0 && page < a.c.n_pages; };
  // The lookups of four of the warp's chunks at once, two and one turns of the loop ahead of their use: a lane's
  // slots first, then the pages of where its rows come from and go.
  struct Rows4 {
    int slot[4];
    int32_t from[4], to[4];
  };
  auto load_slots = [&](int c, Rows4& x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = ((c + k) * kMoveWarps + warp) * 32 + lane;
      x.slot[k] = j < budget ? keep[j] : -1;
    }
  };
  auto load_pages = [&](int c, Rows4& x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = ((c + k) * kMoveWarps + warp) * 32 + lane;
      const bool moves = x.slot[k] > j;                // (a row that stays is left alone)
      x.from[k] = moves ? table[static_cast<uint32_t>(x.slot[k]) / page_size] : 0;
      x.to[k] = moves ? table[static_cast<uint32_t>(j) / page_size] : 0;
    }
  };
  Rows4 now, next;
  load_slots(0, now);
  load_pages(0, now);
  load_slots(4, next);
#pragma unroll 1
  for (int c = 0; c < rounds + kMoveDepth; c += 4) {
    Rows4 after;
    load_slots(c + 8, after);
    load_pages(c + 4, next);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int in = c + k, out = in - kMoveDepth, j = (in * kMoveWarps + warp) * 32 + lane;
      const uint32_t at = ring + (in % kMoveDepth) * 4096;
      int64_t* to = s_to + (in % kMoveDepth) * 32;
      if (out >= 0 && out < rounds) {
        copy_wait<kMoveDepth - 1>();
        __syncthreads();                  // the round's copies have landed
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t row = to[4 * i + sub];
          if (row >= 0 && mine) *reinterpret_cast<uint4*>(base + row) = lds16(at + i * 512);
        }
        __syncwarp();
      }
      if (in < rounds) {
        int64_t from = -1, dest = -1;
        if (now.slot[k] > j) {
          if (valid(now.from[k]) && valid(now.to[k])) {
            from = offset(now.slot[k], now.from[k]);
            dest = offset(j, now.to[k]);
          } else {
            record_device_error(a.c.err, DEVERR_INDEX);
          }
        }
        to[lane] = dest;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t row = __shfl_sync(0xffffffffu, from, 4 * i + sub);
          if (row >= 0 && mine) copy16(at + i * 512, base + row, true);
        }
      }
      copy_commit();
    }
    now = next;
    next = after;
  }
  copy_wait<0>();
}

}  // namespace paged
}  // namespace tp
