// Rotary positions and the paged key/value cache: argument checks and launches.
#include <atomic>

#include "paged.cuh"
#include "paged_decode.cuh"

using tp::set_error;

namespace {

tp_status check_freqs(const void* freqs) {
  if (!freqs) return set_error(TP_ERR_INVALID_ARG, "freqs is null");
  if (reinterpret_cast<uintptr_t>(freqs) & 7)
    return set_error(TP_ERR_INVALID_ARG, "freqs must be 8-byte aligned");
  return TP_OK;
}

tp_status check_ints(const void* p, const char* name) {
  if (!p) return set_error(TP_ERR_INVALID_ARG, std::string(name) + " is null");
  if (reinterpret_cast<uintptr_t>(p) & 3)
    return set_error(TP_ERR_INVALID_ARG, std::string(name) + " must be 4-byte aligned");
  return TP_OK;
}

tp_status check_vec_rows(const tp_head_rows* r, int64_t T, int heads, int hd, int eb, bool written,
                         const char* name) {
  tp_status st = tp::rope::check_rows(r, T, heads, hd, eb, written, name);
  if (st != TP_OK) return st;
  const int64_t unit = 16 / eb;
  if ((reinterpret_cast<uintptr_t>(r->data) & 15) || r->token_stride % unit || r->head_stride % unit)
    return set_error(TP_ERR_INVALID_ARG,
                     std::string(name) + ": rows must be 16-byte aligned, strides multiples of 16 bytes");
  return TP_OK;
}

tp::rope::Rows rows_of(const tp_head_rows* r) { return {r->data, r->token_stride, r->head_stride}; }

// ---- decode attention: which kernel, and its workspace ----
// fp32 groups of up to this many heads multiply on the SIMT units (16 x 4000 keys, 4 heads of 128 dims
// to a group: 63 us, 71 on the matrix instructions; 3 x 1123 keys, 8 heads: 33 and 23 us)
constexpr int kSimtHeads = 4;

// heads of a tile and blocks of a split launch per SM: of the padded head size and the group
struct DecodePlan {
  int hdp, heads, tiles, runs;
  bool whole;
};

DecodePlan decode_plan(const tp::paged::View& c, int dtype) {
  DecodePlan p;
  p.hdp = c.hd <= 64 ? 64 : c.hd <= 128 ? 128 : 256;
  if (dtype == TP_BF16) p.heads = c.group > 8 && p.hdp < 256 ? 16 : 8;
  else p.heads = c.group == 1 ? 1 : c.group <= kSimtHeads ? 4 : c.group > 8 && p.hdp < 256 ? 16 : 8;
  p.tiles = static_cast<int>(tp::ceil_div(c.group, p.heads));
  // One block per (sequence, KV head, head tile) or runs of equal length?  A block alone streams
  // about 0.1 TB/s; a split launch costs about 5 us more (the cuts' joins, a second kernel) but no
  // row, however long, then holds the others up.  The host knows the rows' room, not their lengths,
  // so whole rows are for room that one block reads in 8 us, or in 25 us where there are enough
  // blocks to keep a third of the SMs busy.  Measured on 64 / 8 bf16 heads of 128 dims, whole and
  // split: 1 x 700 keys 7.8 / 9.8 us, 1 x 1000 9.6 / 10.0, 1 x 1500 11.7 / 10.1, 1 x 4000 24.8 / 13.2,
  // 16 ragged up to 1500 15 / 22, 16 up to 4096 30 / 35, 64 up to 700 27 / 40.
  const int64_t blocks = c.b * c.n_kv * p.tiles;
  // (An fp32 group computes two or four times as long per byte: 3 x 1123 keys of 64 / 8 fp32 heads of
  // 128 dims 23.5 us whole, 17.8 split; 16 x 4000 of 32 / 8 heads of 64 dims 55 and 39 us.)
  const int64_t row = c.cap * c.hd * 2 * tp::elem_bytes(dtype) * (dtype == TP_F32 && p.heads > 1 ? p.heads > 4 ? 4 : 2 : 1);
  p.whole = row <= (5 << 17) || (row <= (5 << 19) && blocks * 3 >= tp::num_sms());
  p.runs = tp::num_sms() * tp::paged::split_blocks(128 * p.hdp);   // (all engines' rings)
  return p;
}

// columns of a key's kept scores: the group's heads, in 16-byte vectors
int score_columns(const tp::paged::View& c) { return static_cast<int>(tp::round_up(c.group, 4)); }

// Arrays of the room of every table row: of ``columns`` floats a slot and KV head.  More bytes than
// an address has are refused, before a size wraps around.
tp_status check_room(const tp::paged::View& c, int columns) {
  const double bytes = 4.0 * static_cast<double>(c.b) * c.n_kv * static_cast<double>(c.cap) * columns;
  if (bytes > static_cast<double>(int64_t(1) << 56))
    return set_error(TP_ERR_SHAPE, "b * n_kv * max_pages * page_size scores are too many");
  return TP_OK;
}

struct DecodeWs {
  size_t lse, first, pm, pl, po, z, total;
};
DecodeWs decode_ws(const tp::paged::View& c, int dtype, bool with_score) {
  const DecodePlan p = decode_plan(c, dtype);
  DecodeWs w{};
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t x = at; at += tp::align256(bytes); return x; };
  const size_t parts = p.whole ? 0 : static_cast<size_t>(2) * p.runs * p.heads;
  w.lse = take(static_cast<size_t>(c.b) * c.n_q * 4);
  w.first = take(p.whole ? 0 : static_cast<size_t>(c.b + 2) * 8);
  w.pm = take(parts * 4);
  w.pl = take(parts * 4);
  w.po = take(parts * c.hd * 4);
  w.z = take(with_score ? static_cast<size_t>(c.b) * c.n_kv * c.cap * score_columns(c) * 4 : 0);
  w.total = at;
  return w;
}

// Lets a kernel use ``bytes`` of dynamic shared memory; done: per device, whether it may already
// (host threads may meet here: setting the limit twice is the same as once).
using Done = std::atomic<bool>[64];
template <typename K>
tp_status allow_smem(K* kern, int bytes, Done& done) {
  int dev = 0;
  TP_CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 64 && done[dev].load(std::memory_order_acquire)) return TP_OK;
  TP_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  if (dev < 64) done[dev].store(true, std::memory_order_release);
  return TP_OK;
}

template <typename E, int W>
tp_status launch_whole(const tp::paged::DecodeArgs& a, dim3 grid, cudaStream_t s) {
  constexpr int smem = tp::paged::decode_smem<E>(W);
  auto* whole = tp::paged::decode_whole_kernel<E, W>;
  static Done done;
  const tp_status st = allow_smem(whole, smem, done);
  if (st != TP_OK) return st;
  TP_LAUNCH_PDL(whole, grid, dim3(W * 32), smem, s, a);
  return TP_OK;
}

template <typename E>
tp_status launch_decode(const tp::paged::DecodeArgs& a, const DecodePlan& p, cudaStream_t s) {
  using namespace tp::paged;
  static_assert(ring_bytes<E>() == 128 * E::HDP, "decode_plan's");
  constexpr int kWhole = whole_warps(ring_bytes<E>()), kSplit = split_warps(ring_bytes<E>());
  tp::ProfScope prof(s, "attn_decode_paged");
  if (p.whole) {
    // no more warps than the row's room has units, so that blocks of short rows share an SM
    const int64_t units = tp::ceil_div(a.c.cap, kChunk);
    const dim3 grid(static_cast<unsigned>(a.c.n_kv * a.tiles), static_cast<unsigned>(a.c.b));
    if (units <= 4) return launch_whole<E, 4>(a, grid, s);
    if (units <= 8 && kWhole > 8) return launch_whole<E, 8 < kWhole ? 8 : kWhole>(a, grid, s);
    return launch_whole<E, kWhole>(a, grid, s);
  }
  constexpr int smem = decode_smem<E>(kSplit);
  auto* split = decode_split_kernel<E>;
  static Done done;
  const tp_status st = allow_smem(split, smem, done);
  if (st != TP_OK) return st;
  TP_LAUNCH_PDL(split, dim3(static_cast<unsigned>(a.runs)), dim3(kSplit * 32), smem, s, a);
  auto* join = join_kernel<typename E::T, E::kHeads>;
  TP_LAUNCH_PDL(join, dim3(static_cast<unsigned>(a.c.n_q), static_cast<unsigned>(a.c.b)), dim3(128), 0, s, a);
  return TP_OK;
}

size_t evict_ws(const tp::paged::View& c, int64_t budget) {
  const size_t heads = static_cast<size_t>(c.b) * c.n_kv;
  return tp::align256(heads * budget * 4) + tp::align256(heads * 4) +
         tp::align256(static_cast<size_t>(c.b) * 4);
}

}  // namespace

extern "C" tp_status tp_rope_freqs(const tp_rope_desc* desc, void* freqs, void* stream) {
  tp::clear_error();
  tp_status st = tp::rope::check_desc(desc);
  if (st != TP_OK) return st;
  if ((st = check_freqs(freqs)) != TP_OK) return st;
  tp::rope::freqs_kernel<<<1, 128, 0, static_cast<cudaStream_t>(stream)>>>(
      *desc, static_cast<double*>(freqs));
  TP_LAUNCH_CHECK();
  return TP_OK;
}

extern "C" tp_status tp_rope(const tp_rope_desc* desc, int32_t dtype, int64_t T, int32_t n_heads,
                             int32_t head_dim, const tp_head_rows* x, const void* positions,
                             const void* freqs, int32_t inverse, const tp_head_rows* out,
                             void* stream) {
  tp::clear_error();
  tp_status st = tp::rope::check_desc(desc);
  if (st != TP_OK) return st;
  if (dtype != TP_F32 && dtype != TP_BF16) return set_error(TP_ERR_INVALID_ARG, "dtype");
  if (T < 0 || n_heads < 0 || n_heads > 65535)
    return set_error(TP_ERR_SHAPE, "T must be >= 0 and n_heads in [0, 65535]");
  if (head_dim < desc->rot_dim || head_dim > 1024)
    return set_error(TP_ERR_SHAPE, "head_dim must be in [rot_dim, 1024]");
  if (T > INT32_MAX) return set_error(TP_ERR_SHAPE, "T must fit in 31 bits");
  if (T == 0 || n_heads == 0) return TP_OK;
  const int eb = tp::elem_bytes(dtype);
  if ((st = tp::rope::check_rows(x, T, n_heads, head_dim, eb, false, "x")) != TP_OK ||
      (st = tp::rope::check_rows(out, T, n_heads, head_dim, eb, true, "out")) != TP_OK ||
      (st = tp::rope::check_pair(x, out, "out")) != TP_OK ||
      (st = check_ints(positions, "positions")) != TP_OK || (st = check_freqs(freqs)) != TP_OK)
    return st;
  tp::rope::Args a{};
  a.freqs = static_cast<const double*>(freqs);
  a.positions = static_cast<const int32_t*>(positions);
  a.T = T;
  a.heads = n_heads;
  a.hd = head_dim;
  a.half = desc->rot_dim / 2;
  a.interleaved = desc->layout == TP_ROPE_INTERLEAVED;
  a.m = tp::rope::magnitude_of(desc);
  a.sign = inverse ? -1.f : 1.f;
  a.x = rows_of(x);
  a.out = rows_of(out);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  tp::ProfScope prof(s, "rope");
  const tp::rope::NoCache none{};
  return dtype == TP_BF16 ? tp::rope::launch_rows<__nv_bfloat16>(a, none, s)
                          : tp::rope::launch_rows<float>(a, none, s);
}

extern "C" tp_status tp_kv_append_paged(const tp_paged_desc* desc, int64_t T, const void* seq_ids,
                                        const void* slots, const void* tables,
                                        const tp_head_rows* k, const tp_head_rows* v,
                                        const tp_rope_desc* rope, const void* freqs,
                                        const void* positions, const tp_head_rows* q,
                                        const tp_head_rows* q_out, void* k_pages, void* v_pages,
                                        void* stream) {
  tp::clear_error();
  tp::paged::Target c{};
  tp::rope::Args a{};
  tp_status st = tp::paged::check_desc(desc, &c.c);
  if (st != TP_OK) return st;
  if (T < 0 || T > INT32_MAX) return set_error(TP_ERR_SHAPE, "T must be >= 0 and fit in 31 bits");
  if (!seq_ids && T > desc->b) return set_error(TP_ERR_SHAPE, "without seq_ids T must be <= b");
  if (rope) {
    if ((st = tp::rope::check_desc(rope)) != TP_OK) return st;
    if (rope->rot_dim > desc->head_dim) return set_error(TP_ERR_SHAPE, "rot_dim must be <= head_dim");
  }
  if (!rope && q) return set_error(TP_ERR_INVALID_ARG, "q is rotated: it needs a rope desc");
  if (!q != !q_out) return set_error(TP_ERR_INVALID_ARG, "q and q_out come together");
  if (T == 0) return TP_OK;
  const int eb = tp::elem_bytes(desc->dtype);
  if (k_pages && k_pages == v_pages)
    return set_error(TP_ERR_INVALID_ARG, "k_pages and v_pages are the same pool");
  if ((st = tp::paged::check_pages(k_pages, v_pages, tables)) != TP_OK ||
      (st = check_ints(slots, "slots")) != TP_OK ||
      (st = tp::rope::check_rows(k, T, desc->n_kv, desc->head_dim, eb, false, "k")) != TP_OK ||
      (st = tp::rope::check_rows(v, T, desc->n_kv, desc->head_dim, eb, false, "v")) != TP_OK)
    return st;
  if (seq_ids && (st = check_ints(seq_ids, "seq_ids")) != TP_OK) return st;
  if (rope && (st = check_freqs(freqs)) != TP_OK) return st;
  if (positions && (st = check_ints(positions, "positions")) != TP_OK) return st;
  if (q && ((st = tp::rope::check_rows(q, T, desc->n_q, desc->head_dim, eb, false, "q")) != TP_OK ||
            (st = tp::rope::check_rows(q_out, T, desc->n_q, desc->head_dim, eb, true, "q_out")) != TP_OK ||
            (st = tp::rope::check_pair(q, q_out, "q_out")) != TP_OK))
    return st;
  c.c.tables = static_cast<const int32_t*>(tables);
  c.c.err = tp::device_error_word();
  c.seq_ids = static_cast<const int32_t*>(seq_ids);
  c.slots = static_cast<const int32_t*>(slots);
  c.k = rows_of(k);
  c.v = rows_of(v);
  c.kp = k_pages;
  c.vp = v_pages;
  c.head_stride = c.c.head_stride;
  c.n_kv = desc->n_kv;
  a.T = T;
  a.hd = desc->head_dim;
  a.sign = 1.f;
  if (rope) {
    a.freqs = static_cast<const double*>(freqs);
    a.positions = static_cast<const int32_t*>(positions ? positions : slots);
    a.half = rope->rot_dim / 2;
    a.interleaved = rope->layout == TP_ROPE_INTERLEAVED;
    a.m = tp::rope::magnitude_of(rope);
  }
  if (q) {
    a.heads = desc->n_q;
    a.x = rows_of(q);
    a.out = rows_of(q_out);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  tp::ProfScope prof(s, "kv_append");
  return desc->dtype == TP_BF16 ? tp::rope::launch_rows<__nv_bfloat16>(a, c, s)
                                : tp::rope::launch_rows<float>(a, c, s);
}

extern "C" size_t tp_attn_decode_paged_workspace(const tp_paged_desc* desc, int32_t with_score) {
  tp::clear_error();
  tp::paged::View c;
  if (tp::paged::check_desc(desc, &c) != TP_OK) return 0;
  if (with_score && check_room(c, score_columns(c)) != TP_OK) return 0;
  return decode_ws(c, desc->dtype, with_score != 0).total;
}

extern "C" tp_status tp_attn_decode_paged(const tp_paged_desc* desc, const tp_head_rows* q,
                                          const void* k_pages, const void* v_pages,
                                          const void* tables, const void* lens,
                                          const tp_head_rows* o, void* lse, void* score,
                                          void* workspace, size_t ws_bytes, void* stream) {
  tp::clear_error();
  tp::paged::DecodeArgs a{};
  tp_status st = tp::paged::check_desc(desc, &a.c);
  if (st != TP_OK) return st;
  if (score && (st = check_room(a.c, score_columns(a.c))) != TP_OK) return st;
  if (desc->b == 0) return TP_OK;
  const int eb = tp::elem_bytes(desc->dtype);
  if ((st = tp::paged::check_pages(k_pages, v_pages, tables)) != TP_OK ||
      (st = check_ints(lens, "lens")) != TP_OK ||
      (st = check_vec_rows(q, desc->b, desc->n_q, desc->head_dim, eb, false, "q")) != TP_OK ||
      (st = check_vec_rows(o, desc->b, desc->n_q, desc->head_dim, eb, true, "o")) != TP_OK)
    return st;
  if (lse && (st = check_ints(lse, "lse")) != TP_OK) return st;
  if (score && (st = check_ints(score, "score")) != TP_OK) return st;
  if (!workspace) return set_error(TP_ERR_INVALID_ARG, "workspace is null");
  if (reinterpret_cast<uintptr_t>(workspace) & 15)
    return set_error(TP_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  const DecodeWs w = decode_ws(a.c, desc->dtype, score != nullptr);
  if (ws_bytes < w.total) return set_error(TP_ERR_WORKSPACE, "workspace too small");
  a.c.tables = static_cast<const int32_t*>(tables);
  a.c.err = tp::device_error_word();
  a.q = rows_of(q);
  a.o = rows_of(o);
  a.kp = k_pages;
  a.vp = v_pages;
  a.lens = static_cast<const int32_t*>(lens);
  a.scale = tp::paged::scale_of(desc);
  const DecodePlan p = decode_plan(a.c, desc->dtype);
  char* ws = static_cast<char*>(workspace);
  a.lse = static_cast<float*>(lse ? lse : ws + w.lse);
  a.score = static_cast<float*>(score);
  a.first = reinterpret_cast<int64_t*>(ws + w.first);
  a.pm = reinterpret_cast<float*>(ws + w.pm);
  a.pl = reinterpret_cast<float*>(ws + w.pl);
  a.po = reinterpret_cast<float*>(ws + w.po);
  a.z = score ? reinterpret_cast<float*>(ws + w.z) : nullptr;
  a.zw = score_columns(a.c);
  a.tiles = p.tiles;
  a.runs = p.runs;
  a.min_units = 4;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  using tp::paged::Mma;
  using tp::paged::MmaF32;
  using tp::paged::Simt;
#define TP_DECODE(H)                                                                             \
  (desc->dtype == TP_BF16                                                                        \
       ? (p.heads == 8 ? launch_decode<Mma<H, 1>>(a, p, s)                                       \
                       : launch_decode<Mma<H, H == 256 ? 1 : 2>>(a, p, s))                       \
       : (p.heads == 1 ? launch_decode<Simt<H, 1>>(a, p, s)                                      \
                       : p.heads == 4 ? launch_decode<Simt<H, 4>>(a, p, s)                       \
                       : p.heads == 8 ? launch_decode<MmaF32<H, 1>>(a, p, s)                     \
                                      : launch_decode<MmaF32<H, H == 256 ? 1 : 2>>(a, p, s)))
  st = p.hdp == 64 ? TP_DECODE(64) : p.hdp == 128 ? TP_DECODE(128) : TP_DECODE(256);
#undef TP_DECODE
  if (st != TP_OK || !score || (p.whole && p.tiles == 1)) return st;
  tp::ProfScope prof(s, "attn_score_paged");
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(tp::ceil_div(a.c.cap, 512), 256)),
                  static_cast<unsigned>(desc->n_kv), static_cast<unsigned>(desc->b));
  TP_LAUNCH_PDL(tp::paged::weights_kernel, grid, dim3(256), 0, s, a);
  return TP_OK;
}

extern "C" size_t tp_kv_evict_paged_workspace(const tp_paged_desc* desc, int32_t budget) {
  tp::clear_error();
  tp::paged::View c;
  if (tp::paged::check_desc(desc, &c) != TP_OK || check_room(c, 1) != TP_OK) return 0;
  return budget >= 1 && budget <= c.cap ? evict_ws(c, budget) : 0;
}

extern "C" tp_status tp_kv_evict_paged(const tp_paged_desc* desc, void* score, const void* lens,
                                       int32_t budget, int32_t recent, void* k_pages,
                                       void* v_pages, const void* tables, void* new_lens,
                                       void* keep, void* workspace, size_t ws_bytes,
                                       void* stream) {
  tp::clear_error();
  tp::paged::EvictArgs a{};
  tp_status st = tp::paged::check_desc(desc, &a.c);
  if (st != TP_OK || (st = check_room(a.c, 1)) != TP_OK) return st;
  if (budget < 1 || budget > a.c.cap)
    return set_error(TP_ERR_SHAPE, "budget must be in [1, max_pages * page_size]");
  if (recent < 0 || recent > budget) return set_error(TP_ERR_SHAPE, "recent must be in [0, budget]");
  if (desc->b == 0) return TP_OK;
  if (k_pages && k_pages == v_pages)
    return set_error(TP_ERR_INVALID_ARG, "k_pages and v_pages are the same pool");
  if ((st = tp::paged::check_pages(k_pages, v_pages, tables)) != TP_OK ||
      (st = check_ints(score, "score")) != TP_OK || (st = check_ints(lens, "lens")) != TP_OK ||
      (st = check_ints(new_lens, "new_lens")) != TP_OK)
    return st;
  if (keep && (st = check_ints(keep, "keep")) != TP_OK) return st;
  if (!workspace) return set_error(TP_ERR_INVALID_ARG, "workspace is null");
  if (reinterpret_cast<uintptr_t>(workspace) & 15)
    return set_error(TP_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  if (ws_bytes < evict_ws(a.c, budget)) return set_error(TP_ERR_WORKSPACE, "workspace too small");
  const size_t heads = static_cast<size_t>(a.c.b) * a.c.n_kv;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.c.tables = static_cast<const int32_t*>(tables);
  a.c.err = tp::device_error_word();
  a.score = static_cast<float*>(score);
  a.lens = static_cast<const int32_t*>(lens);
  a.new_lens = static_cast<int32_t*>(new_lens);
  a.keep_out = static_cast<int32_t*>(keep);
  a.keep = reinterpret_cast<int32_t*>(w);
  w += tp::align256(heads * budget * 4);
  a.cut = reinterpret_cast<int32_t*>(w);
  w += tp::align256(heads * 4);
  a.new_ws = reinterpret_cast<int32_t*>(w);
  a.budget = budget;
  a.recent = recent;
  a.kp = k_pages;
  a.vp = v_pages;
  const int eb = tp::elem_bytes(desc->dtype);
  a.room = static_cast<int>(std::min<int64_t>(a.c.cap, tp::paged::kEvictRoom));
  a.strips = static_cast<int>(tp::ceil_div(static_cast<int64_t>(desc->head_dim) * eb, 128));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  {
    tp::ProfScope prof(s, "kv_evict_select");
    static Done done;
    if ((st = allow_smem(tp::paged::evict_select_kernel, tp::paged::kEvictRoom * 4, done)) != TP_OK) return st;
    const int smem = a.room * 4;
    TP_LAUNCH_PDL(tp::paged::evict_select_kernel,
                  dim3(static_cast<unsigned>(desc->n_kv), static_cast<unsigned>(desc->b)),
                  dim3(tp::paged::kEvictThreads), smem, s, a);
  }
  tp::ProfScope prof(s, "kv_evict_move");
  const dim3 grid(static_cast<unsigned>(2 * a.strips), static_cast<unsigned>(desc->n_kv),
                  static_cast<unsigned>(desc->b));
  constexpr int smem = tp::paged::kMoveWarps * tp::paged::kMoveRing;
  static Done done;
  if ((st = allow_smem(tp::paged::evict_move_kernel, smem, done)) != TP_OK) return st;
  TP_LAUNCH_PDL(tp::paged::evict_move_kernel, grid, dim3(tp::paged::kMoveWarps * 32), smem, s, a, eb);
  return TP_OK;
}
