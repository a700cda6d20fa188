// Rotary positions: q and k rotated alone, or on the way into the paged cache
// (sm_103a).
//
// A head's first rot = 2 n dims are n pairs: pair j is dims (j, j + n), or (2 j, 2 j + 1)
// when adjacent.  With (c, s) = table[position on the pair's axis, j]:
//   y1 = x1 c - x2 s,   y2 = x2 c + x1 s
// every product and sum rounded to fp32 (never contracted), so that a result is a
// function of its inputs alone: fp16 results are rounded once from there, 8-bit codes
// follow the 8-bit write's rule on the fp32 values.  Dims from rot on are copied.
//
// Why a table and not the angles: a program's frequencies, their rescaling for long
// contexts and a magnitude are then all in it, and codes stay reproducible, which
// cosines of two implementations are not.  It costs 8 bytes a pair and token, 2 % of a
// token of 32/8 heads.
//
// What bounds it: HBM for prompts: 16 of 1..4096 tokens of 32/8 heads into the fp16 cache
// 107 us, 6.65 TB/s (a copy's rate is 6.77); 4 x 4096 with three axes, without a cache, 53 us,
// 6.3 TB/s.  A step of single tokens is a chain of dependent loads (sequence, position, table
// and block id): 64 tokens of 40 heads 3.4 us.  The 8-bit cache's kernels are in rope_q8.cuh.
#include <initializer_list>

#include "rope.cuh"

namespace pkv {
namespace rope {

// ---- rows: rotary alone, and the fp16 cache ----------------------------------------------
// One warp per (token, up to 16 of its heads' rows), 4 rows a pass: the rows are loaded before
// the warp knows the token's sequence, position, cosines and block, whose loads depend on
// one another.  A prompt's warps are many enough to cover that chain (28 on an SM, at 72
// registers), and a step's single tokens are spread over many warps by their heads.  Measured
// on the way, 4 x 4096 tokens of 32/8 heads: code for one axis and for several apart 53 us for
// three axes instead of 67; warps that walk 8 tokens with the next one's rows under way 59
// (127 registers); parts of 32 rows 62.
constexpr int kRowWarps = 4;
constexpr int kPasses = 4;             // of 4 rows each, at most

template <bool CACHE, bool ADJACENT, int AXES>
__global__ void __launch_bounds__(kRowWarps * 32, 7) rope_rows_kernel(const RowParams p) {
  // a programmatic dependent of the stream's previous kernel, and the next one may
  // place its CTAs while this grid runs: each reads after its wait
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t max_context = static_cast<int64_t>(p.max_blocks) * p.block_size;
  if (CACHE && blockIdx.x == gridDim.x - 1) {   // a CTA that looks at every entry once, used or not
    if (blockIdx.y == 0)
      for (int s = threadIdx.x; s < p.num_seqs; s += kRowWarps * 32)
        packed_seq(p.query_start, p.context_lens, s, p.num_tokens, max_context, p.dev_err, true);
    return;
  }
  const int64_t i64 = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (i64 >= p.num_tokens) return;
  const int i = static_cast<int>(i64);
  const int row0 = blockIdx.y * p.part_rows + (lane >> 3);
  const int rows = min(p.num_q_heads + (CACHE ? 2 : 1) * p.num_kv_heads, (blockIdx.y + 1) * p.part_rows);
  const Chunks ch(lane & 7, p.rot.n);
  const int q_end = p.num_q_heads, k_end = q_end + p.num_kv_heads;

  int32_t pos[AXES];
  if (!CACHE) load_positions(p.rot, i, 0, pos);
  // plain loads: q and k may be rotated in place
  uint4 xa[kPasses], xb[kPasses];
  const __half* from_q = p.q + i * p.q_stride;
  const __half* from_k = p.k + i * p.k_stride;
  const __half* from_v = CACHE ? p.v + i * p.v_stride : nullptr;
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int row = row0 + 4 * u;
    if (row >= rows) continue;
    const __half* from = row < q_end               ? from_q + row * kHeadDim
                         : !CACHE || row < k_end ? from_k + (row - q_end) * kHeadDim
                                                 : from_v + (row - k_end) * kHeadDim;
    const uint4* at = reinterpret_cast<const uint4*>(from);
    xa[u] = at[ch.a];
    xb[u] = at[ch.b];
  }

  int64_t slot = 0;
  if (CACHE) {
    const int s = find_unit_seq(p.query_start, p.num_seqs, i, 1, 0);
    const PackedSeq q = packed_seq(p.query_start, p.context_lens, s, p.num_tokens, max_context,
                                   p.dev_err, false);
    if (!q.ok || i < q.row0 || i >= q.row0 + q.n) return;
    const int place = q.ctx - q.n + (i - q.row0);
    load_positions(p.rot, i, place, pos);
    const int lb = place / p.block_size;
    const int32_t blk = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks + lb);
    slot = blk >= 0 && blk < p.num_blocks
               ? static_cast<int64_t>(blk) * p.block_size + (place - lb * p.block_size)
               : -1;
  }
  if (!on_table(p.rot, pos)) {
    if (lane == 0) report(p.dev_err, PKV_DEV_BAD_POSITION);
    return;
  }
  float4 cs[4];
  if (ch.turns) load_turn<ADJACENT>(p.rot, ch, pos, cs);
  if (slot < 0 && lane == 0) report(p.dev_err, PKV_DEV_BAD_BLOCK_ID);

  const int64_t kv_row = slot * p.num_kv_heads * kHeadDim;
  __half* to_q = p.q_out + i * p.q_out_stride;
  __half* to_k = CACHE ? p.k_cache + kv_row : p.k_out + i * p.k_out_stride;
  __half* to_v = p.v_cache + kv_row;
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int row = row0 + 4 * u;
    if (row >= rows) continue;
    if (ch.turns && (!CACHE || row < k_end)) {
      float a[8], b[8];
      widen(xa[u], a);
      widen(xb[u], b);
      rotate<ADJACENT>(a, b, cs);
      xa[u] = narrow(a);
      xb[u] = narrow(b);
    }
    if (row >= q_end && slot < 0) continue;
    __half* to = row < q_end               ? to_q + row * kHeadDim
                 : !CACHE || row < k_end ? to_k + (row - q_end) * kHeadDim
                                         : to_v + (row - k_end) * kHeadDim;
    reinterpret_cast<uint4*>(to)[ch.a] = xa[u];
    reinterpret_cast<uint4*>(to)[ch.b] = xb[u];
  }
}

// ---- host -------------------------------------------------------------------------------

bool misaligned(int bytes, std::initializer_list<const void*> ptrs) {
  uintptr_t all = 0;
  for (const void* p : ptrs) all |= reinterpret_cast<uintptr_t>(p);
  return all & (bytes - 1);
}

// the rotation's arguments, checked
int make_rotation(Rotation* r, const int32_t* positions, int num_axes, const uint8_t* axes,
                  const float* table, int64_t table_rows, int rot_dim, int num_tokens) {
  if (num_axes < 1 || table_rows <= 0 || rot_dim <= 0) return PKV_ERR_INVALID_ARG;
  if (num_axes > kMaxAxes || rot_dim > kHeadDim || rot_dim % 16 || table_rows > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  *r = {};
  r->n = rot_dim / 2;
  r->num_axes = num_axes;   // all are looked at, whatever axes the pairs follow
  if (axes)
    for (int j = 0; j < r->n; ++j) {
      if (axes[j] >= num_axes) return PKV_ERR_INVALID_ARG;
      r->axis[j >> 4] |= static_cast<uint32_t>(axes[j]) << 2 * (j & 15);
    }
  r->in_twos = 1;
  for (int j = 0; axes && j < r->n; j += 2) r->in_twos &= axes[j] == axes[j + 1];
  r->table = table;
  r->positions = positions;
  r->table_rows = table_rows;
  r->num_tokens = num_tokens;
  if (!positions) {   // on every axis the place in the sequence: one axis
    r->num_axes = r->in_twos = 1;
    for (uint32_t& w : r->axis) w = 0;
  }
  return PKV_OK;
}

bool bad_stride(int64_t stride) { return stride < 0 || stride % 8; }

template <bool CACHE>
int launch_rows(RowParams& p, bool adjacent, void* stream) {
  const int64_t rows = p.num_q_heads + (CACHE ? 2ll : 1ll) * p.num_kv_heads;
  // parts of even length; shorter ones where they leave SMs with less than 16 warps
  int64_t parts = (rows + 4 * kPasses - 1) / (4 * kPasses);
  if (p.num_tokens * parts < 152 * 16) parts = (rows + 7) / 8;
  p.part_rows = static_cast<int>((rows + 4 * parts - 1) / (4 * parts) * 4);
  parts = (rows + p.part_rows - 1) / p.part_rows;
  if (parts > 65535) return PKV_ERR_UNSUPPORTED;
  const dim3 grid((static_cast<unsigned>(p.num_tokens) + kRowWarps - 1) / kRowWarps + CACHE,
                  static_cast<unsigned>(parts));
  const auto go = [&](auto kernel) { return launch(kernel, grid, kRowWarps * 32, stream, p); };
  if (p.rot.num_axes == 1)
    return adjacent ? go(rope_rows_kernel<CACHE, true, 1>) : go(rope_rows_kernel<CACHE, false, 1>);
  return adjacent ? go(rope_rows_kernel<CACHE, true, kMaxAxes>)
                  : go(rope_rows_kernel<CACHE, false, kMaxAxes>);
}

}  // namespace rope
}  // namespace pkv

extern "C" int pkv_rotary_embedding(void* q_out, void* k_out, const void* q, const void* k,
                                    int64_t q_out_stride, int64_t k_out_stride, int64_t q_stride,
                                    int64_t k_stride, const int32_t* positions, int num_axes,
                                    const uint8_t* axes, const float* table, int64_t table_rows,
                                    int rot_dim, int adjacent, int num_tokens, int num_q_heads,
                                    int num_kv_heads, int head_dim, int32_t* dev_err,
                                    void* stream) {
  using namespace pkv::rope;
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads < 0) return PKV_ERR_INVALID_ARG;
  if (head_dim != kHeadDim || num_q_heads > (1 << 20) || num_kv_heads > (1 << 20))
    return PKV_ERR_UNSUPPORTED;
  RowParams p = {};
  const int rc = make_rotation(&p.rot, positions, num_axes, axes, table, table_rows, rot_dim, num_tokens);
  if (rc != PKV_OK) return rc;
  if (num_tokens == 0) return PKV_OK;
  if (!q_out || !q || !positions || !table || (num_kv_heads > 0 && (!k_out || !k)))
    return PKV_ERR_INVALID_ARG;
  if (misaligned(16, {q_out, k_out, q, k, table}) || misaligned(4, {positions}) ||
      bad_stride(q_stride) || bad_stride(k_stride) || bad_stride(q_out_stride) ||
      bad_stride(k_out_stride))
    return PKV_ERR_INVALID_ARG;
  if (num_tokens > 1 && (q_out_stride < static_cast<int64_t>(num_q_heads) * kHeadDim ||
                         k_out_stride < static_cast<int64_t>(num_kv_heads) * kHeadDim))
    return PKV_ERR_INVALID_ARG;
  p.q_out = static_cast<__half*>(q_out);
  p.k_out = static_cast<__half*>(k_out);
  p.q = static_cast<const __half*>(q);
  p.k = static_cast<const __half*>(k);
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.dev_err = dev_err;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  return launch_rows<false>(p, adjacent != 0, stream);
}

namespace pkv {
namespace rope {
namespace {

// the arguments that both caches share, checked; PKV_OK with p->num_tokens 0: nothing to do
int make_append(RowParams* p, void* q_out, const void* q, const void* k, const void* v,
                int64_t q_out_stride, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                const int32_t* query_start, const int32_t* block_tables,
                const int32_t* context_lens, const void* k_cache, const void* v_cache,
                const int32_t* positions, int num_axes, const uint8_t* axes, const float* table,
                int64_t table_rows, int rot_dim, int num_tokens, int num_seqs, int num_q_heads,
                int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                int max_blocks, int32_t* dev_err) {
  if (num_tokens < 0 || num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_blocks <= 0 || max_blocks <= 0 || block_size <= 0)
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kHeadDim || num_q_heads > (1 << 20) || num_kv_heads > (1 << 20) ||
      num_blocks > INT32_MAX / block_size ||
      static_cast<int64_t>(max_blocks) * block_size > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  *p = {};
  const int rc = make_rotation(&p->rot, positions, num_axes, axes, table, table_rows, rot_dim, num_tokens);
  if (rc != PKV_OK) return rc;
  if (num_tokens == 0 || num_seqs == 0) return PKV_OK;
  if (!q_out || !q || !k || !v || !query_start || !block_tables || !context_lens || !k_cache ||
      !v_cache || !table)
    return PKV_ERR_INVALID_ARG;
  if (misaligned(16, {q_out, q, k, v, k_cache, v_cache, table}) ||
      misaligned(4, {query_start, block_tables, context_lens, positions}) ||
      bad_stride(q_stride) || bad_stride(k_stride) || bad_stride(v_stride) ||
      bad_stride(q_out_stride))
    return PKV_ERR_INVALID_ARG;
  if (num_tokens > 1 && q_out_stride < static_cast<int64_t>(num_q_heads) * kHeadDim)
    return PKV_ERR_INVALID_ARG;
  p->q_out = static_cast<__half*>(q_out);
  p->q = static_cast<const __half*>(q);
  p->k = static_cast<const __half*>(k);
  p->v = static_cast<const __half*>(v);
  p->q_out_stride = q_out_stride;
  p->q_stride = q_stride;
  p->k_stride = k_stride;
  p->v_stride = v_stride;
  p->query_start = query_start;
  p->context_lens = context_lens;
  p->block_tables = block_tables;
  p->dev_err = dev_err;
  p->num_blocks = num_blocks;
  p->num_tokens = num_tokens;
  p->num_seqs = num_seqs;
  p->num_q_heads = num_q_heads;
  p->num_kv_heads = num_kv_heads;
  p->block_size = block_size;
  p->max_blocks = max_blocks;
  return PKV_OK;
}

}  // namespace
}  // namespace rope
}  // namespace pkv

extern "C" int pkv_rope_and_cache(void* q_out, const void* q, const void* k, const void* v,
                                  int64_t q_out_stride, int64_t q_stride, int64_t k_stride,
                                  int64_t v_stride, const int32_t* query_start,
                                  const int32_t* block_tables, const int32_t* context_lens,
                                  void* k_cache, void* v_cache, const int32_t* positions,
                                  int num_axes, const uint8_t* axes, const float* table,
                                  int64_t table_rows, int rot_dim, int adjacent, int num_tokens,
                                  int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                  int block_size, int64_t num_blocks, int max_blocks_per_seq,
                                  int32_t* dev_err, void* stream) {
  using namespace pkv::rope;
  RowParams p;
  const int rc = make_append(&p, q_out, q, k, v, q_out_stride, q_stride, k_stride, v_stride,
                             query_start, block_tables, context_lens, k_cache, v_cache, positions,
                             num_axes, axes, table, table_rows, rot_dim, num_tokens, num_seqs,
                             num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                             max_blocks_per_seq, dev_err);
  if (rc != PKV_OK || p.num_tokens == 0) return rc;
  p.k_cache = static_cast<__half*>(k_cache);
  p.v_cache = static_cast<__half*>(v_cache);
  return launch_rows<true>(p, adjacent != 0, stream);
}

extern "C" int pkv_rope_and_cache_q8(void* q_out, const void* q, const void* k, const void* v,
                                     int64_t q_out_stride, int64_t q_stride, int64_t k_stride,
                                     int64_t v_stride, const int32_t* query_start,
                                     const int32_t* block_tables, const int32_t* context_lens,
                                     void* k_cache, void* v_cache, float* k_scale,
                                     float* v_scale, int code, const int32_t* positions,
                                     int num_axes, const uint8_t* axes, const float* table,
                                     int64_t table_rows, int rot_dim, int adjacent,
                                     int num_tokens, int num_seqs, int num_q_heads,
                                     int num_kv_heads, int head_dim, int block_size,
                                     int64_t num_blocks, int max_blocks_per_seq, int scale_stride,
                                     int32_t* dev_err, void* stream) {
  using namespace pkv::rope;
  if (scale_stride < num_kv_heads || (code != PKV_CODE_INT8 && code != PKV_CODE_E4M3))
    return PKV_ERR_INVALID_ARG;
  Q8Params p;
  const int rc = make_append(&p.r, q_out, q, k, v, q_out_stride, q_stride, k_stride, v_stride,
                             query_start, block_tables, context_lens, k_cache, v_cache, positions,
                             num_axes, axes, table, table_rows, rot_dim, num_tokens, num_seqs,
                             num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                             max_blocks_per_seq, dev_err);
  if (rc != PKV_OK) return rc;
  if (!(block_size == 8 || block_size == 16 || block_size == 32 || block_size == 64))
    return PKV_ERR_UNSUPPORTED;
  if (p.r.num_tokens == 0) return PKV_OK;
  if (!k_scale || !v_scale || misaligned(4, {k_scale, v_scale})) return PKV_ERR_INVALID_ARG;
  p.k_codes = static_cast<uint8_t*>(k_cache);
  p.v_codes = static_cast<uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.scale_stride = scale_stride;
  // A step's way holds up to 16 rows of a head, the long chunks' a whole block's whatever is new
  // of it.  Of 32/8 heads, in blocks of 8, 16, 32 and 64: 128 x 4 tokens 6.2 us against 8, 10, 14
  // and 23; 64 x 15 9.4 to 10 against 8.5, 9, 11 and 16; 256 x 30 45, 50, 55 and 55 against 40,
  // 42, 49 and 82.
  const int few = std::max(8, block_size / 2);   // tokens a sequence
  const bool step = num_tokens < static_cast<int64_t>(few) * num_seqs;
  const int64_t heads = num_q_heads + 2ll * num_kv_heads;
  const int64_t units =
      step ? num_tokens : static_cast<int64_t>(num_tokens) / block_size + 2ll * num_seqs;
  // A token's heads share its cosines and the search for its place: they are cut apart where
  // that makes no more than two rounds of CTAs (blocks of 8 and 16 and single warps: about two).
  // Prompts of 32/8 and 32/32 heads: four rounds are 3 to 6 % slower; 32-token blocks, 32/32
  // heads: 46 us of two, as three 50; 8-token blocks, 2 x 3000 of 32/8: 30 us of three, as one
  // and a half 34.  Steps of 32/32 heads: 1024 tokens 12 us, in CTAs of 16 heads 17.  Few long
  // chunks: 64 rows of 32/8 heads in 64-token blocks 4.6 us, in CTAs of 16 heads 22, of 4 heads 8.4.
  const int64_t least =   // 4 heads for each of a step's warps, one for each team of a chunk's
      step ? 4 * kQ8Warps : block_size == 64 ? 1 : block_size == 32 ? 2 : kQ8Warps;
  const int64_t rounds = 2 * 152 * (step ? 8 : 4);
  // of two units to spare for a sequence one is empty
  const int64_t likely = std::max<int64_t>(1, step ? units : units - num_seqs);
  const bool teams = !step && block_size > 16;
  const int64_t parts = std::max<int64_t>(1, (rounds + (teams ? 0 : likely - 1)) / likely);
  const int64_t per = (heads + parts * least - 1) / (parts * least) * least;
  p.heads_per_cta = static_cast<int>(per);
  p.heads_per_warp = static_cast<int>((per + kQ8Warps - 1) / kQ8Warps);
  if (units >= INT32_MAX || (heads + per - 1) / per > 65535) return PKV_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(units + 1), static_cast<unsigned>((heads + per - 1) / per));
  return (code == PKV_CODE_INT8 ? launch_q8_int8 : launch_q8_e4m3)(p, step, adjacent != 0, block_size,
                                                                   grid, stream);
}
