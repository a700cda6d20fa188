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
// What bounds it: HBM for prompts; a step of single tokens is a chain of dependent loads
// (sequence, position, table and block id, scale).
#include <climits>

#include "q8_device.cuh"

namespace pkv {
namespace rope {

constexpr int kHeadDim = 128;
constexpr int kMaxAxes = 4;

struct Rotation {
  const float* table;          // [table_rows, n, 2]: cosine, sine
  const int32_t* positions;    // [num_axes, num_tokens], nullptr: the place in the sequence
  int64_t table_rows;
  int64_t num_tokens;
  int num_axes;
  int n;                       // pairs, a multiple of 8
  uint32_t axis[4];            // two bits a pair
};

struct RowParams {
  Rotation rot;
  __half *q_out, *k_out;       // k_out: rotary alone
  const __half *q, *k, *v;
  int64_t q_out_stride, k_out_stride, q_stride, k_stride, v_stride;   // halves, token to token
  __half *k_cache, *v_cache;
  const int32_t *query_start, *context_lens, *block_tables;
  int32_t* dev_err;
  int64_t num_blocks;
  int num_tokens, num_seqs, num_q_heads, num_kv_heads, block_size, max_blocks;
};

// A row of a head is worked by 8 lanes, two 16-byte chunks each: a rotating lane c holds
// chunks c and c + n / 8, which for pairs half a part apart are both halves of 8 pairs
// and for adjacent pairs 4 whole pairs each; the other lanes hold neighbours.
struct Chunks {
  int a, b;
  bool turns;
  __device__ __forceinline__ Chunks(int c, int n) {
    const int lanes = n >> 3;
    turns = c < lanes;
    a = turns ? c : 2 * c;       // 2 lanes + 2 (c - lanes)
    b = turns ? c + lanes : 2 * c + 1;
  }
};

// a token's positions on the axes; false: one lies outside the table
__device__ __forceinline__ bool load_positions(const Rotation& r, int64_t token, int place,
                                               int32_t (&pos)[kMaxAxes]) {
  bool ok = true;
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) {
    pos[a] = place;
    if (r.positions && a < r.num_axes) pos[a] = __ldg(r.positions + a * r.num_tokens + token);
    if (a < r.num_axes) ok = ok && pos[a] >= 0 && pos[a] < r.table_rows;
  }
  return ok;
}

// cosines and sines of the lane's 8 pairs (rotating lanes)
template <bool ADJACENT>
__device__ __forceinline__ void load_turn(const Rotation& r, const Chunks& ch,
                                          const int32_t (&pos)[kMaxAxes], float2 (&cs)[8]) {
  const int p0 = ADJACENT ? 4 * ch.a : 8 * ch.a, p1 = ADJACENT ? 4 * ch.b : p0 + 4;
  if (r.num_axes == 1) {
    const float* row = r.table + static_cast<int64_t>(pos[0]) * r.n * 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(row + 2 * (i < 2 ? p0 : p1)) + (i & 1));
      cs[2 * i] = make_float2(w.x, w.y);
      cs[2 * i + 1] = make_float2(w.z, w.w);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int p = (e < 4 ? p0 : p1) + (e & 3);
      const int w = p >> 4;
      const uint32_t word = w & 2 ? (w & 1 ? r.axis[3] : r.axis[2]) : (w & 1 ? r.axis[1] : r.axis[0]);
      const uint32_t a = word >> (2 * (p & 15)) & 3;
      const int32_t at = a & 2 ? (a & 1 ? pos[3] : pos[2]) : (a & 1 ? pos[1] : pos[0]);
      cs[e] = __ldg(reinterpret_cast<const float2*>(r.table) + static_cast<int64_t>(at) * r.n + p);
    }
  }
}

// 8 fp16 values of a chunk
__device__ __forceinline__ void widen(uint4 w, float (&f)[8]) {
  const float2 a = half2_to_float2(w.x), b = half2_to_float2(w.y);
  const float2 c = half2_to_float2(w.z), d = half2_to_float2(w.w);
  f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  f[4] = c.x, f[5] = c.y, f[6] = d.x, f[7] = d.y;
}
__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
  return make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]),
                    pack_half2(f[6], f[7]));
}

__device__ __forceinline__ void turn(float& x1, float& x2, float2 cs) {
  const float y1 = __fsub_rn(__fmul_rn(x1, cs.x), __fmul_rn(x2, cs.y));
  x2 = __fadd_rn(__fmul_rn(x2, cs.x), __fmul_rn(x1, cs.y));
  x1 = y1;
}

// the lane's two chunks, widened and rotated
template <bool ADJACENT>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float2 (&cs)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (!ADJACENT)
      turn(a[e], b[e], cs[e]);
    else if (e < 4)
      turn(a[2 * e], a[2 * e + 1], cs[e]);
    else
      turn(b[2 * e - 8], b[2 * e - 7], cs[e]);
  }
}

// ---- rows: rotary alone, and the fp16 cache ----------------------------------------------
// One warp per (token, 16 of its heads' rows), 4 rows a pass: the rows are loaded before
// the warp knows the token's sequence, position, cosines and block, whose loads depend on
// one another.  A prompt's warps are many enough to cover that chain, and a step's single
// tokens are spread over many warps by their heads; a warp for a whole token would walk 3
// to 8 times as many rows in turn.
constexpr int kRowWarps = 4;
constexpr int kPasses = 4;             // of 4 rows each
constexpr int kPartRows = 4 * kPasses;

template <bool CACHE, bool ADJACENT>
__global__ void __launch_bounds__(kRowWarps * 32) rope_rows_kernel(const RowParams p) {
  // a programmatic dependent of the stream's previous kernel, and the next one may
  // place its CTAs while this grid runs: each reads after its wait
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t max_context = static_cast<int64_t>(p.max_blocks) * p.block_size;
  if (CACHE && blockIdx.x == 0 && blockIdx.y == 0)   // every entry is looked at once, used or not
    for (int s = threadIdx.x; s < p.num_seqs; s += kRowWarps * 32)
      packed_seq(p.query_start, p.context_lens, s, p.num_tokens, max_context, p.dev_err, true);
  const int i = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (i >= p.num_tokens) return;
  const int rows = p.num_q_heads + (CACHE ? 2 : 1) * p.num_kv_heads;
  const int row0 = blockIdx.y * kPartRows + (lane >> 3);
  const Chunks ch(lane & 7, p.rot.n);

  // plain loads: q and k may be rotated in place
  uint4 xa[kPasses], xb[kPasses];
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int row = row0 + 4 * u;
    if (row >= rows) continue;
    const int head = row < p.num_q_heads ? row : (row - p.num_q_heads) % p.num_kv_heads;
    const __half* from = row < p.num_q_heads                      ? p.q + i * p.q_stride
                         : row < p.num_q_heads + p.num_kv_heads ? p.k + i * p.k_stride
                                                                : p.v + i * p.v_stride;
    const uint4* at = reinterpret_cast<const uint4*>(from + head * kHeadDim);
    xa[u] = at[ch.a];
    xb[u] = at[ch.b];
  }

  int place = 0;
  int64_t slot = -1;
  if (CACHE) {
    const int s = find_unit_seq(p.query_start, p.num_seqs, i, 1, 0);
    const PackedSeq q = packed_seq(p.query_start, p.context_lens, s, p.num_tokens, max_context,
                                   p.dev_err, false);
    if (!q.ok || i < q.row0 || i >= q.row0 + q.n) return;
    place = q.ctx - q.n + (i - q.row0);
    const int lb = place / p.block_size;
    const int32_t blk = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks + lb);
    if (blk >= 0 && blk < p.num_blocks)
      slot = static_cast<int64_t>(blk) * p.block_size + (place - lb * p.block_size);
    else if (lane == 0)
      report(p.dev_err, PKV_DEV_BAD_BLOCK_ID);
  }
  int32_t pos[kMaxAxes];
  if (!load_positions(p.rot, i, place, pos)) {
    if (lane == 0) report(p.dev_err, PKV_DEV_BAD_POSITION);
    return;
  }
  float2 cs[8];
  if (ch.turns) load_turn<ADJACENT>(p.rot, ch, pos, cs);

#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int row = row0 + 4 * u;
    if (row >= rows) continue;
    const bool is_q = row < p.num_q_heads, is_k = !is_q && row < p.num_q_heads + p.num_kv_heads;
    const int head = is_q ? row : (row - p.num_q_heads) % p.num_kv_heads;
    if (ch.turns && (is_q || is_k)) {
      float a[8], b[8];
      widen(xa[u], a);
      widen(xb[u], b);
      rotate<ADJACENT>(a, b, cs);
      xa[u] = narrow(a);
      xb[u] = narrow(b);
    }
    __half* to;
    if (is_q) {
      to = p.q_out + i * p.q_out_stride + head * kHeadDim;
    } else if (!CACHE) {
      to = p.k_out + i * p.k_out_stride + head * kHeadDim;
    } else {
      if (slot < 0) continue;
      to = (is_k ? p.k_cache : p.v_cache) + (slot * p.num_kv_heads + head) * kHeadDim;
    }
    reinterpret_cast<uint4*>(to)[ch.a] = xa[u];
    reinterpret_cast<uint4*>(to)[ch.b] = xb[u];
  }
}

// ---- the 8-bit cache ---------------------------------------------------------------------
struct Q8Params {
  RowParams r;                 // k_out, k_cache and v_cache unused
  uint8_t *k_codes, *v_codes;
  float *k_scale, *v_scale;    // [num_blocks, scale_stride]
  int scale_stride;
  int by_token;                // units are tokens, see below
};

// The new rows of one block of one sequence.
struct Piece {
  int s, row0;      // its sequence; the packed row that would be the block's row 0
  int base, r0, r1; // place of the block's row 0; new rows [r0, r1)
  int64_t blk;      // -1: no valid id
};

// Units are cut in one of two ways.  Long chunks: the write's units of BS rows, numbered
// without a prefix sum, two to spare for each sequence.  Steps (fewer than 4 tokens a
// sequence): every token is a unit, and the first new one of its block takes the
// block's others along; no unit is empty when each sequence brings one.
template <int BS>
__device__ __forceinline__ bool find_piece(const Q8Params& qp, Piece& c) {
  const RowParams& p = qp.r;
  const int unit = blockIdx.x, per = qp.by_token ? 1 : BS, slack = qp.by_token ? 0 : 2;
  c.s = find_unit_seq(p.query_start, p.num_seqs, unit, per, slack);
  const PackedSeq q = packed_seq(p.query_start, p.context_lens, c.s, p.num_tokens,
                                 static_cast<int64_t>(p.max_blocks) * BS, p.dev_err, false);
  if (!q.ok || q.n == 0) return false;
  const int start = q.ctx - q.n;
  int64_t lb;
  if (qp.by_token) {
    const int nth = unit - q.row0;
    if (nth < 0 || nth >= q.n || (nth > 0 && (start + nth) % BS != 0)) return false;
    lb = (start + nth) / BS;
  } else {
    const int nth = unit - unit_base(p.query_start, c.s, BS, 2);
    lb = start / BS + static_cast<int64_t>(nth);
    if (nth < 0 || lb * BS >= q.ctx) return false;
  }
  c.base = static_cast<int>(lb) * BS;
  c.r0 = max(start - c.base, 0);
  c.r1 = min(q.ctx - c.base, BS);
  c.row0 = q.row0 + c.base - start;
  const int32_t blk = __ldg(p.block_tables + static_cast<int64_t>(c.s) * p.max_blocks + lb);
  c.blk = blk >= 0 && blk < p.num_blocks ? blk : -1;
  return true;
}

// Heads are numbered q, k, v.  `lanes`: the lanes that share a block and head (32, or 8
// when each group of 8 lanes has a head of its own and one row).  The rotated values are
// computed twice, for the maximum and for the codes: held in 32 bits they would take
// twice the registers of the fp16 rows, and the table's lines are in L1.
template <class Code, int BS, bool ADJACENT, bool STEP>
__device__ __forceinline__ void append_head(const Q8Params& qp, const Piece& c, int head,
                                            bool valid) {
  constexpr int kRows = STEP ? 1 : BS / 4;   // rows of a lane
  const RowParams& p = qp.r;
  const int lane = threadIdx.x & 31;
  const Chunks ch(lane & 7, p.rot.n);
  const bool is_q = head < p.num_q_heads, is_v = head >= p.num_q_heads + p.num_kv_heads;
  const int g = is_q ? head : (head - p.num_q_heads) % p.num_kv_heads;
  const int64_t in_stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
  const __half* src = (is_q ? p.q : is_v ? p.v : p.k) + g * kHeadDim;
  const auto row_of = [&](int u) { return STEP ? c.r0 : 4 * u + (lane >> 3); };
  const auto in_range = [&](int u) { return valid && row_of(u) >= c.r0 && row_of(u) < c.r1; };

  uint4 xa[kRows], xb[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    if (!in_range(u)) continue;
    const uint4* at = reinterpret_cast<const uint4*>(src + (c.row0 + row_of(u)) * in_stride);
    xa[u] = at[ch.a];
    xb[u] = at[ch.b];
  }
  const int64_t row_elems = static_cast<int64_t>(p.num_kv_heads) * kHeadDim;
  uint8_t* dst = (is_v ? qp.v_codes : qp.k_codes) + c.blk * BS * row_elems + g * kHeadDim;
  float* scale_at = (is_v ? qp.v_scale : qp.k_scale) + c.blk * qp.scale_stride + g;
  const bool stores = valid && !is_q && c.blk >= 0;
  const float before = stores && c.r0 > 0 ? *scale_at : 0.f;

  // row u's values in 32 bits; false: it is left out
  const auto values = [&](int u, float (&a)[8], float (&b)[8]) {
    const int r = row_of(u);
    int32_t pos[kMaxAxes];
    if (!load_positions(p.rot, c.row0 + r, c.base + r, pos)) return false;
    widen(xa[u], a);
    widen(xb[u], b);
    if (!is_v && ch.turns) {
      float2 cs[8];
      load_turn<ADJACENT>(p.rot, ch, pos, cs);
      rotate<ADJACENT>(a, b, cs);
    }
    return true;
  };

  // the largest magnitude: as unsigned integers the bits of |y| order as |y| does, and
  // those of infinities and NaN lie above
  constexpr uint32_t kInf = 0x7f800000u;
  uint32_t top = 0, all = 0;   // of the finite ones, of all
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    if (!in_range(u)) continue;
    float a[8], b[8];
    if (!values(u, a, b)) {
      if ((lane & 7) == 0) report(p.dev_err, PKV_DEV_BAD_POSITION);
      continue;
    }
    if (is_q) {
      uint4* to = reinterpret_cast<uint4*>(
          p.q_out + (c.row0 + row_of(u)) * p.q_out_stride + g * kHeadDim);
      to[ch.a] = narrow(a);
      to[ch.b] = narrow(b);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t m = __float_as_uint(a[e]) & 0x7fffffffu, n = __float_as_uint(b[e]) & 0x7fffffffu;
        all = max(all, max(m, n));
        top = max(top, max(m < kInf ? m : 0u, n < kInf ? n : 0u));
      }
    }
  }
  if (all >= kInf && stores) report(p.dev_err, PKV_DEV_NONFINITE);
  if (STEP) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  } else {
    top = __reduce_max_sync(0xffffffffu, top);
  }
  if (!is_q && valid && c.blk < 0 && (lane & 7) == 0) report(p.dev_err, PKV_DEV_BAD_BLOCK_ID);
  const float scale = fmaxf(before, __fdiv_rn(__uint_as_float(top), Code::kMax));
  const float inv = scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
  if (stores && scale > before && c.r0 > 0) {   // earlier rows of the block, under the grown scale
    const float ratio = __fdiv_rn(before, scale);
    for (int r = STEP ? 0 : lane >> 3; r < c.r0; r += STEP ? 1 : 4) {
      uint4* at = reinterpret_cast<uint4*>(dst + r * row_elems) + (lane & 7);
      const uint4 w = *at;
      uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float f[4];
        Code::decode4(in[e], f);
        in[e] = Code::encode4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
      }
      *at = make_uint4(in[0], in[1], in[2], in[3]);
    }
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    if (!in_range(u) || !stores) continue;
    float a[8], b[8];
    if (!values(u, a, b)) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) {   // what is not finite is stored as 0
      a[e] = fabsf(a[e]) < INFINITY ? a[e] * inv : 0.f;
      b[e] = fabsf(b[e]) < INFINITY ? b[e] * inv : 0.f;
    }
    uint8_t* to = dst + row_of(u) * row_elems;
    *reinterpret_cast<uint2*>(to + 8 * ch.a) =
        make_uint2(Code::encode4(a[0], a[1], a[2], a[3]), Code::encode4(a[4], a[5], a[6], a[7]));
    *reinterpret_cast<uint2*>(to + 8 * ch.b) =
        make_uint2(Code::encode4(b[0], b[1], b[2], b[3]), Code::encode4(b[4], b[5], b[6], b[7]));
  }
  __syncwarp();   // every lane has read the earlier scale
  if (stores && (STEP ? (lane & 7) == 0 : lane == 0)) *scale_at = scale;
}

// One CTA per (unit, heads), a warp for 4 heads by tokens (side by side where the piece is
// a single row, in turn otherwise), else for one.
constexpr int kQ8Warps = 4;

template <class Code, int BS, bool ADJACENT>
__global__ void __launch_bounds__(kQ8Warps * 32) rope_q8_kernel(const Q8Params qp) {
  const RowParams& p = qp.r;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && blockIdx.y == 0)   // every entry is looked at once, used or not
    for (int s = threadIdx.x; s < p.num_seqs; s += kQ8Warps * 32)
      packed_seq(p.query_start, p.context_lens, s, p.num_tokens,
                 static_cast<int64_t>(p.max_blocks) * BS, p.dev_err, true);
  Piece c;
  if (!find_piece<BS>(qp, c)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  if (!qp.by_token) {
    const int head = blockIdx.y * kQ8Warps + warp;
    if (head < heads) append_head<Code, BS, ADJACENT, false>(qp, c, head, true);
    return;
  }
  const int first = (blockIdx.y * kQ8Warps + warp) * 4;
  if (c.r1 - c.r0 == 1) {
    const int head = first + (lane >> 3);
    append_head<Code, BS, ADJACENT, true>(qp, c, min(head, heads - 1), head < heads);
  } else {
#pragma unroll 1
    for (int h = first; h < min(first + 4, heads); ++h)
      append_head<Code, BS, ADJACENT, false>(qp, c, h, true);
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
  r->num_axes = axes ? num_axes : 1;
  if (axes)
    for (int j = 0; j < r->n; ++j) {
      if (axes[j] >= num_axes) return PKV_ERR_INVALID_ARG;
      r->axis[j >> 4] |= static_cast<uint32_t>(axes[j]) << 2 * (j & 15);
    }
  r->table = table;
  r->positions = positions;
  r->table_rows = table_rows;
  r->num_tokens = num_tokens;
  // on every axis the place in the sequence: one axis
  if (!positions) r->num_axes = 1;
  return PKV_OK;
}

bool bad_stride(int64_t stride) { return stride < 0 || stride % 8; }

template <class... P>
int launch(void (*kernel)(const P...), dim3 grid, int threads, void* stream, const P&... p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p...) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <bool CACHE>
int launch_rows(const RowParams& p, bool adjacent, void* stream) {
  const int rows = p.num_q_heads + (CACHE ? 2 : 1) * p.num_kv_heads;
  const int64_t parts = (static_cast<int64_t>(rows) + kPartRows - 1) / kPartRows;
  if (parts > 65535) return PKV_ERR_UNSUPPORTED;
  const dim3 grid((static_cast<unsigned>(p.num_tokens) + kRowWarps - 1) / kRowWarps,
                  static_cast<unsigned>(parts));
  return adjacent ? launch(rope_rows_kernel<CACHE, true>, grid, kRowWarps * 32, stream, p)
                  : launch(rope_rows_kernel<CACHE, false>, grid, kRowWarps * 32, stream, p);
}

template <class Code, bool ADJACENT>
int launch_q8(const Q8Params& p, int block_size, dim3 grid, void* stream) {
  constexpr int kThreads = kQ8Warps * 32;
  switch (block_size) {
    case 8: return launch(rope_q8_kernel<Code, 8, ADJACENT>, grid, kThreads, stream, p);
    case 16: return launch(rope_q8_kernel<Code, 16, ADJACENT>, grid, kThreads, stream, p);
    case 32: return launch(rope_q8_kernel<Code, 32, ADJACENT>, grid, kThreads, stream, p);
    default: return launch(rope_q8_kernel<Code, 64, ADJACENT>, grid, kThreads, stream, p);
  }
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
  p.by_token = num_tokens < 4ll * num_seqs;
  const int64_t heads = num_q_heads + 2ll * num_kv_heads;
  const int64_t units = p.by_token ? num_tokens
                                   : static_cast<int64_t>(num_tokens) / block_size + 2ll * num_seqs;
  const int64_t per = p.by_token ? 4 * kQ8Warps : kQ8Warps;
  if (units > INT32_MAX || (heads + per - 1) / per > 65535) return PKV_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>((heads + per - 1) / per));
  if (code == PKV_CODE_INT8)
    return adjacent ? launch_q8<pkv::Int8Code, true>(p, block_size, grid, stream)
                    : launch_q8<pkv::Int8Code, false>(p, block_size, grid, stream);
  return adjacent ? launch_q8<pkv::E4m3Code, true>(p, block_size, grid, stream)
                  : launch_q8<pkv::E4m3Code, false>(p, block_size, grid, stream);
}
