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
  if (d->max_pages > (INT32_MAX - 1024) / d->page_size)
    return set_error(TP_ERR_SHAPE, "max_pages * page_size must fit in 31 bits");
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
  int budget, recent;
  void *kp, *vp;
};

// A score as an unsigned number of the same order: NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t rank_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kEvictThreads = 1024;

// exclusive sum over the block's threads; *total gets the whole
__device__ __forceinline__ int block_scan(int v, int* total, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int nw = blockDim.x >> 5;
    int w = lane < nw ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < nw) s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[(blockDim.x >> 5) - 1];
  const int before = warp > 0 ? s_warp[warp - 1] : 0;
  __syncthreads();
  return before + x - v;
}

// One block per (KV head, sequence): the budget-recent largest scores by a radix search of the
// threshold (8 bits a pass, counted in shared memory), then their slots in order, ties from the
// lowest; the kept scores move down in chunks (a chunk is read before it is written, and a kept
// score never moves up).
static __global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(EvictArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int s_hist[256], s_warp[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_want;
  const int g = blockIdx.x, tid = threadIdx.x;
  const int64_t seq = blockIdx.y, sg = seq * a.c.n_kv + g;
  const int64_t n64 = a.c.keys(a.lens, seq);
  if (tid == 0 && n64 != a.lens[seq]) record_device_error(a.c.err, DEVERR_INDEX);
  const int n = static_cast<int>(n64), budget = a.budget;
  float* score = a.score + sg * a.c.cap;
  int32_t* keep = a.keep + sg * budget;
  int32_t* out = a.keep_out ? a.keep_out + sg * budget : nullptr;
  if (tid == 0) {
    a.cut[sg] = n > budget;
    if (g == 0) a.new_ws[seq] = min(n, budget);
  }
  if (n <= budget) {
    if (out)
      for (int i = tid; i < budget; i += blockDim.x) out[i] = i < n ? i : -1;
    return;
  }
  const int old = n - a.recent;             // candidates: slots 0 .. old-1
  const int pick = budget - a.recent;       // how many of them stay (< old)
  uint32_t prefix = 0;
  int want = pick;
  if (pick > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += blockDim.x) s_hist[i] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int i = tid; i < old; i += blockDim.x) {
        const uint32_t u = rank_of(score[i]);
        if ((u & mask) == prefix) atomicAdd(&s_hist[(u >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int left = want, d = 255;
        while (d > 0 && s_hist[d] < left) left -= s_hist[d--];
        s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
        s_want = left;
      }
      __syncthreads();
      prefix = s_prefix;
      want = s_want;
      __syncthreads();
    }
  }
  // above the threshold: all; equal to it: the first ``want`` by slot
  int kept = 0, ties = 0;
  for (int i0 = 0; i0 < old && pick > 0; i0 += blockDim.x) {
    const int i = i0 + tid;
    const uint32_t u = i < old ? rank_of(score[i]) : 0u;
    const int tie = i < old && u == prefix;
    int n_tie, n_keep;
    const int t = ties + block_scan(tie, &n_tie, s_warp);
    const int k = i < old && (u > prefix || (tie && t < want));
    const int at = kept + block_scan(k, &n_keep, s_warp);
    if (k) keep[at] = i;
    ties += n_tie;
    kept += n_keep;
  }
  for (int i = tid; i < a.recent; i += blockDim.x) keep[pick + i] = old + i;
  __syncthreads();
  for (int j0 = 0; j0 < budget; j0 += blockDim.x) {
    const int j = j0 + tid;
    float v = 0.f;
    int from = 0;
    if (j < budget) {
      from = keep[j];
      v = score[from];
      if (out) out[j] = from;
    }
    __syncthreads();
    if (j < budget) score[j] = v;
  }
}

// One block per (16-byte column pair of K or V, KV head, sequence): the kept rows' columns move
// down chunk by chunk.  Row j comes from slot keep[j] >= j, so rows written by earlier chunks are
// never read again, and a chunk is read before it is written.
static __global__ void __launch_bounds__(256) evict_move_kernel(EvictArgs a, int eb) {
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y, tid = threadIdx.x;
  const int64_t seq = blockIdx.z, sg = seq * a.c.n_kv + g;
  const int units = a.c.hd * eb / 16;                 // 16-byte columns of a row
  if (blockIdx.x == 0 && g == 0 && tid == 0) a.new_lens[seq] = a.new_ws[seq];
  if (!a.cut[sg]) return;
  const int32_t* keep = a.keep + sg * a.budget;
  char* base = static_cast<char*>(blockIdx.x < units ? a.kp : a.vp);
  const int col = (blockIdx.x % units) * 16;
  for (int j0 = 0; j0 < a.budget; j0 += 256) {
    const int j = j0 + tid;
    uint4 x;
    int64_t to = -1;
    if (j < a.budget && keep[j] != j) {
      const int64_t from = a.c.at(seq, g, keep[j]);
      to = a.c.at(seq, g, j);
      if (from < 0 || to < 0) {
        record_device_error(a.c.err, DEVERR_INDEX);
        to = -1;
      } else {
        x = *reinterpret_cast<const uint4*>(base + from * eb + col);
      }
    }
    __syncthreads();
    if (to >= 0) *reinterpret_cast<uint4*>(base + to * eb + col) = x;
  }
}

}  // namespace paged
}  // namespace tp
