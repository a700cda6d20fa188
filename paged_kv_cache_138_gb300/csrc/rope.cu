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
#include <algorithm>
#include <cfloat>
#include <climits>
#include <initializer_list>

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
  int in_twos;                 // pairs 2 i and 2 i + 1 always follow one axis
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
  int part_rows;               // of a warp of rope_rows_kernel
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

// a token's positions on the axes (AXES: 1, or kMaxAxes with num_axes of them in use)
template <int AXES>
__device__ __forceinline__ void load_positions(const Rotation& r, int64_t token, int place,
                                               int32_t (&pos)[AXES]) {
#pragma unroll
  for (int a = 0; a < AXES; ++a) {
    pos[a] = place;
    if (r.positions && (a == 0 || a < r.num_axes)) pos[a] = __ldg(r.positions + a * r.num_tokens + token);
  }
}
// false: one lies outside the table
template <int AXES>
__device__ __forceinline__ bool on_table(const Rotation& r, const int32_t (&pos)[AXES]) {
  bool ok = true;
#pragma unroll
  for (int a = 0; a < AXES; ++a)
    if (a == 0 || a < r.num_axes) ok = ok && static_cast<uint32_t>(pos[a]) < static_cast<uint32_t>(r.table_rows);
  return ok;
}

// Cosines and sines of the lane's 8 pairs (rotating lanes), as packed arithmetic takes them:
// pairs 2 i and 2 i + 1 are (c, c', s, s').
template <bool ADJACENT, int AXES>
__device__ __forceinline__ void load_turn(const Rotation& r, const Chunks& ch,
                                          const int32_t (&pos)[AXES], float4 (&cs)[4]) {
  const int p0 = ADJACENT ? 4 * ch.a : 8 * ch.a, p1 = ADJACENT ? 4 * ch.b : p0 + 4;
  const float2* table = reinterpret_cast<const float2*>(r.table);
  if (AXES == 1) {
    const float4* row = reinterpret_cast<const float4*>(table + static_cast<int64_t>(pos[0]) * r.n);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 w = __ldg(row + (i < 2 ? p0 : p1) / 2 + (i & 1));
      cs[i] = make_float4(w.x, w.z, w.y, w.w);
    }
    return;
  }
  // the axes of the first and the last four pairs, two bits each
  const auto word = [&](int p) {
    const uint32_t lo = p & 16 ? r.axis[1] : r.axis[0], hi = p & 16 ? r.axis[3] : r.axis[2];
    return (p & 32 ? hi : lo) >> (2 * (p & 15));
  };
  const uint32_t axes0 = word(p0), axes1 = ADJACENT ? word(p1) : axes0 >> 8;
  const auto at = [&](int e) {   // the table's entry of the lane's pair e
    const uint32_t a = (e < 4 ? axes0 : axes1) >> (2 * (e & 3));
    const int32_t lo = a & 1 ? pos[1 % AXES] : pos[0], hi = a & 1 ? pos[3 % AXES] : pos[2 % AXES];
    return table + static_cast<int64_t>(a & 2 ? hi : lo) * r.n + (e < 4 ? p0 : p1) + (e & 3);
  };
  if (r.in_twos) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(at(2 * i)));
      cs[i] = make_float4(w.x, w.z, w.y, w.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 w = __ldg(at(2 * i)), v = __ldg(at(2 * i + 1));
      cs[i] = make_float4(w.x, v.x, w.y, v.y);
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

// two pairs at a time: (x1 c - x2 s, x2 c + x1 s), each product and sum rounded by itself.
// The sums stay scalar: packed ones were contracted with the packed products.
__device__ __forceinline__ void turn2(float& x1, float& y1, float& x2, float& y2, float4 cs) {
  const float2 a = make_float2(x1, y1), b = make_float2(x2, y2);
  const float2 c = make_float2(cs.x, cs.y), s = make_float2(cs.z, cs.w);
  const float2 ac = fmul2(a, c), bs = fmul2(b, s), bc = fmul2(b, c), as = fmul2(a, s);
  x1 = __fsub_rn(ac.x, bs.x), y1 = __fsub_rn(ac.y, bs.y);
  x2 = __fadd_rn(bc.x, as.x), y2 = __fadd_rn(bc.y, as.y);
}

// the lane's two chunks, widened and rotated
template <bool ADJACENT>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float4 (&cs)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!ADJACENT) {
      turn2(a[2 * i], a[2 * i + 1], b[2 * i], b[2 * i + 1], cs[i]);
    } else {
      float* f = i < 2 ? a + 4 * i : b + 4 * i - 8;
      turn2(f[0], f[2], f[1], f[3], cs[i]);
    }
  }
}

// ---- rows: rotary alone, and the fp16 cache ----------------------------------------------
// One warp per (token, up to 16 of its heads' rows), 4 rows a pass: the rows are loaded before
// the warp knows the token's sequence, position, cosines and block, whose loads depend on
// one another.  A prompt's warps are many enough to cover that chain (24 on an SM), and a
// step's single tokens are spread over many warps by their heads.
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

// ---- the 8-bit cache ---------------------------------------------------------------------
struct Q8Params {
  RowParams r;                 // k_out, k_cache and v_cache unused
  uint8_t *k_codes, *v_codes;
  float *k_scale, *v_scale;    // [num_blocks, scale_stride]
  int scale_stride;
  int by_token;                // units are tokens, see below
  int heads_per_cta;           // a multiple of 4 kQ8Warps
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

// Where a head's rows come from and its codes go; heads are numbered q, k, v.
struct HeadAt {
  bool is_q, is_v;
  int g;
  const __half* src;     // its row of packed row 0
  int64_t stride;
  uint8_t* dst;          // its codes of the block's row 0
  float* scale;
  __device__ __forceinline__ HeadAt(const Q8Params& qp, const Piece& c, int block_size, int head) {
    const RowParams& p = qp.r;
    is_q = head < p.num_q_heads;
    is_v = head >= p.num_q_heads + p.num_kv_heads;
    g = is_q ? head : is_v ? head - p.num_q_heads - p.num_kv_heads : head - p.num_q_heads;
    src = (is_q ? p.q : is_v ? p.v : p.k) + g * kHeadDim;
    stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
    dst = (is_v ? qp.v_codes : qp.k_codes) +
          (c.blk * block_size * p.num_kv_heads + g) * kHeadDim;
    scale = (is_v ? qp.v_scale : qp.k_scale) + c.blk * qp.scale_stride + g;
  }
};

constexpr uint32_t kInf = 0x7f800000u;

// the largest magnitude of a chunk, NaN above all: as unsigned integers the bits of what is
// not negative order as the numbers do
__device__ __forceinline__ float top_of(float m, const float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(f[e]), "f"(f[e + 1]));
  return m;
}
__device__ __forceinline__ float top2(float a, float b) {
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(a), "f"(b));
  return a;
}
__device__ __forceinline__ void drop_nonfinite(float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = fabsf(f[e]) < INFINITY ? f[e] : 0.f;
}

// Codes are 0 under a scale whose inverse would pass fp32's range (rotated values can be as
// small as a table makes them; fp16 ones cannot).
__device__ __forceinline__ float inverse_of(float scale) {
  return scale >= FLT_MIN ? __fdiv_rn(1.f, scale) : 0.f;
}

// codes of a chunk: no value times inv passes the largest code by more than a rounding
template <class Code>
__device__ __forceinline__ uint2 code8(const float (&f)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 lo = fmul2(make_float2(f[4 * h], f[4 * h + 1]), make_float2(inv, inv));
    const float2 hi = fmul2(make_float2(f[4 * h + 2], f[4 * h + 3]), make_float2(inv, inv));
    w[h] = Code::near4(lo, hi);
  }
  return make_uint2(w[0], w[1]);
}
struct Int8Near : Int8Code {
  // to the nearest integer, ties to even, by a sum whose last place is 1: its low byte is
  // the code (9 instructions instead of 24 with conversions and limits)
  static __device__ __forceinline__ uint32_t near4(float2 a, float2 b) {
    const auto near = [](float y) { return __float_as_uint(__fadd_rn(y, 12582912.f)); };
    return __byte_perm(__byte_perm(near(a.x), near(a.y), 0x0040),
                       __byte_perm(near(b.x), near(b.y), 0x0040), 0x5410);
  }
};
struct E4m3Near : E4m3Code {
  static __device__ __forceinline__ uint32_t near4(float2 a, float2 b) {
    return encode4(a.x, a.y, b.x, b.y);
  }
};

// 16 codes of a row under a scale that has grown
template <class Code>
__device__ __forceinline__ void recode16(uint8_t* at, float ratio) {
  const uint4 w = *reinterpret_cast<uint4*>(at);
  uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float f[4];
    Code::decode4(in[e], f);
    in[e] = Code::encode4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
  }
  *reinterpret_cast<uint4*>(at) = make_uint4(in[0], in[1], in[2], in[3]);
}

// Pieces of a single row (a decoded token): each 8 lanes take a head of their own.
template <class Code, int BS, bool ADJACENT, int AXES>
__device__ __forceinline__ void append_row(const Q8Params& qp, const Piece& c, int first, int last) {
  const RowParams& p = qp.r;
  const int lane = threadIdx.x & 31, token = c.row0 + c.r0;
  const Chunks ch(lane & 7, p.rot.n);
  const int64_t row_elems = static_cast<int64_t>(p.num_kv_heads) * kHeadDim;
  int32_t pos[AXES];
  load_positions(p.rot, token, c.base + c.r0, pos);
  const bool ok = on_table(p.rot, pos);
  if (!ok && lane == 0) report(p.dev_err, PKV_DEV_BAD_POSITION);
  float4 cs[4];
  if (ok && ch.turns) load_turn<ADJACENT>(p.rot, ch, pos, cs);
#pragma unroll 1
  for (int h0 = first; h0 < last; h0 += 4) {
    const bool valid = h0 + (lane >> 3) < last && ok;
    const HeadAt at(qp, c, BS, min(h0 + (lane >> 3), last - 1));
    const bool stores = valid && !at.is_q && c.blk >= 0;
    uint4 xa = make_uint4(0u, 0u, 0u, 0u), xb = xa;
    if (valid) {
      const uint4* from = reinterpret_cast<const uint4*>(at.src + token * at.stride);
      xa = from[ch.a];
      xb = from[ch.b];
    }
    const float before = stores && c.r0 > 0 ? *at.scale : 0.f;
    float a[8], b[8];
    widen(xa, a);
    widen(xb, b);
    if (valid && !at.is_v && ch.turns) rotate<ADJACENT>(a, b, cs);
    if (valid && at.is_q) {
      uint4* to = reinterpret_cast<uint4*>(p.q_out + token * p.q_out_stride + at.g * kHeadDim);
      to[ch.a] = narrow(a);
      to[ch.b] = narrow(b);
    }
    uint32_t top = __float_as_uint(top_of(top_of(0.f, a), b));
    if (__any_sync(0xffffffffu, stores && top >= kInf)) {
      if (stores && top >= kInf) report(p.dev_err, PKV_DEV_NONFINITE);
      drop_nonfinite(a);
      drop_nonfinite(b);
      top = __float_as_uint(top_of(top_of(0.f, a), b));
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float scale = fmaxf(before, __fdiv_rn(__uint_as_float(top), Code::kMax));
    const float inv = inverse_of(scale);
    if (stores) {
      if (scale > before && c.r0 > 0) {   // earlier rows of the block
        const float ratio = __fdiv_rn(before, scale);
        for (int r = 0; r < c.r0; ++r) recode16<Code>(at.dst + r * row_elems + 16 * (lane & 7), ratio);
      }
      uint8_t* to = at.dst + c.r0 * row_elems;
      *reinterpret_cast<uint2*>(to + 8 * ch.a) = code8<Code>(a, inv);
      *reinterpret_cast<uint2*>(to + 8 * ch.b) = code8<Code>(b, inv);
    }
    __syncwarp();   // every lane has read the earlier scale
    if (stores && (lane & 7) == 0) *at.scale = scale;
  }
}

// Pieces of several rows: a warp holds 16 rows of the block (8 of 8-row blocks), 4 a
// pass, and walks the heads, the CTA's rows' cosines and sines in shared memory (read again
// for every head from L1, strided, they bounded the kernel: prompts 203 us instead of 110).  A
// block of 32 or 64 rows is a team of 2 or 4 warps, which join their maxima.  The rotated
// values stay in 32 bits from the maximum to the codes, while the next head's rows are under
// way; computed twice instead, at 96 registers, they took 10 to 20 % longer.  Four CTAs an SM
// (128 registers) for teams, three (0: left to the compiler) where a warp is alone and keeps its cosines in
// registers: 32-token blocks 48 us (three CTAs: 54), 16-token blocks 110 us (four: 113).
constexpr int kQ8Warps = 4;
constexpr int kWarpRows = 16;

// The rows' cosines and sines in shared memory: 8 lanes of a row read a 16-byte chunk each at
// a time, chunk i of the 4 of lane c lying at i XOR (c / 2), in 8 different banks.
__device__ __forceinline__ int turn_at(int row, int c, int i) { return (row * 8 + c) * 4 + (i ^ (c >> 1)); }

// read where it is used: as a loop invariant it would take 64 registers
__device__ __forceinline__ float4 read_turn(const float4* at) {
  float4 w;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(w.x), "=f"(w.y), "=f"(w.z), "=f"(w.w)
               : "r"(smem_u32(at)));
  return w;
}

template <class Code, int BS, bool ADJACENT, int AXES>
__device__ __forceinline__ void append_rows(const Q8Params& qp, const Piece& c, int first, int last,
                                            uint32_t (&tops)[2][kQ8Warps], float4 (&table)[BS * 32]) {
  constexpr int kRows = BS < kWarpRows ? BS : kWarpRows, kPass = kRows / 4;
  constexpr int kTeam = BS / kRows, kTeams = kQ8Warps / kTeam;
  const RowParams& p = qp.r;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / kTeam, own = kRows * (warp % kTeam) + (lane >> 3);
  const Chunks ch(lane & 7, p.rot.n);
  const int64_t row_elems = static_cast<int64_t>(p.num_kv_heads) * kHeadDim;

  // bit u: the pass's row is one of the piece and has a place in the table; the others are zeros
  uint32_t in = 0;
#pragma unroll
  for (int u = 0; u < kPass; ++u) {
    const int r = own + 4 * u;
    if (r >= c.r0 && r < c.r1) {
      int32_t pos[AXES];
      load_positions(p.rot, c.row0 + r, c.base + r, pos);
      if (on_table(p.rot, pos)) in |= 1u << u;
    }
  }
  uint4 xa[kPass], xb[kPass];
  const auto load = [&](const HeadAt& at) {
    const __half* row = at.src + (c.row0 + own) * at.stride;
#pragma unroll
    for (int u = 0; u < kPass; ++u, row += 4 * at.stride) {
      xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
      if (in >> u & 1) {
        xa[u] = reinterpret_cast<const uint4*>(row)[ch.a];
        xb[u] = reinterpret_cast<const uint4*>(row)[ch.b];
      }
    }
  };
  int head = first + team;
  HeadAt next(qp, c, BS, min(head, last - 1));
  if (head < last) load(next);
#pragma unroll 1
  for (int r = threadIdx.x >> 3; r < BS; r += kQ8Warps * 4) {
    if (r < c.r0 || r >= c.r1) continue;
    int32_t pos[AXES];
    load_positions(p.rot, c.row0 + r, c.base + r, pos);
    if (!on_table(p.rot, pos)) {
      report(p.dev_err, PKV_DEV_BAD_POSITION);
    } else if (ch.turns) {
      float4 cs[4];
      load_turn<ADJACENT>(p.rot, ch, pos, cs);
#pragma unroll
      for (int i = 0; i < 4; ++i) table[turn_at(r, lane & 7, i)] = cs[i];
    }
  }
  __syncthreads();
  int turns = 0;               // of the team's exchange
  const auto join = [&](uint32_t top) {
    top = __reduce_max_sync(0xffffffffu, top);
    if (kTeam > 1) {
      if (lane == 0) tops[turns & 1][warp] = top;
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(kTeam * 32) : "memory");
#pragma unroll
      for (int w = 0; w < kTeam; ++w) top = max(top, tops[turns & 1][team * kTeam + w]);
      ++turns;
    }
    return top;
  };
#pragma unroll 1
  for (; head < last; head += kTeams) {
    const HeadAt at = next;
    const bool stores = !at.is_q && c.blk >= 0;
    const float before = stores && c.r0 > 0 ? *at.scale : 0.f;
    float a[kPass][8], b[kPass][8];
#pragma unroll
    for (int u = 0; u < kPass; ++u) {
      widen(xa[u], a[u]);
      widen(xb[u], b[u]);
    }
    if (head + kTeams < last) {
      next = HeadAt(qp, c, BS, head + kTeams);
      load(next);
    }
    if (!at.is_v && ch.turns)
#pragma unroll
      for (int u = 0; u < kPass; ++u) {   // rows that are not in hold zeros, whatever turns them
        float4 cs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4* from = table + turn_at(own + 4 * u, lane & 7, i);
          cs[i] = kTeam > 1 ? read_turn(from) : *from;
        }
        rotate<ADJACENT>(a[u], b[u], cs);
      }
    if (at.is_q) {
      __half* out = p.q_out + (c.row0 + own) * p.q_out_stride + at.g * kHeadDim;
#pragma unroll
      for (int u = 0; u < kPass; ++u, out += 4 * p.q_out_stride) {
        const uint4 ya = narrow(a[u]), yb = narrow(b[u]);
        if (in >> u & 1) {
          reinterpret_cast<uint4*>(out)[ch.a] = ya;
          reinterpret_cast<uint4*>(out)[ch.b] = yb;
        }
      }
      continue;
    }
    if (!stores) continue;
    const auto largest = [&]() {
      float m = 0.f;
#pragma unroll
      for (int u = 0; u < kPass; ++u) {
        const float t = top_of(top_of(0.f, a[u]), b[u]);
        if (in >> u & 1) m = top2(m, t);
      }
      return join(__float_as_uint(m));
    };
    uint32_t top = largest();
    if (top >= kInf) {
      if (lane == 0) report(p.dev_err, PKV_DEV_NONFINITE);
#pragma unroll
      for (int u = 0; u < kPass; ++u) {
        drop_nonfinite(a[u]);
        drop_nonfinite(b[u]);
      }
      top = largest();
    }
    const float scale = fmaxf(before, __fdiv_rn(__uint_as_float(top), Code::kMax));
    const float inv = inverse_of(scale);
    if (scale > before && c.r0 > 0) {   // earlier rows of the block, under the grown scale
      const float ratio = __fdiv_rn(before, scale);
      for (int r = own; r < min(c.r0, kRows * (warp % kTeam) + kRows); r += 4)
        recode16<Code>(at.dst + r * row_elems + 16 * (lane & 7), ratio);
    }
    uint8_t* to = at.dst + own * row_elems;
#pragma unroll
    for (int u = 0; u < kPass; ++u, to += 4 * row_elems) {
      const uint2 ya = code8<Code>(a[u], inv), yb = code8<Code>(b[u], inv);
      if (in >> u & 1) {
        *reinterpret_cast<uint2*>(to + 8 * ch.a) = ya;
        *reinterpret_cast<uint2*>(to + 8 * ch.b) = yb;
      }
    }
    __syncwarp();   // every lane has read the earlier scale (every warp, before they joined)
    if (lane == 0 && warp % kTeam == 0) *at.scale = scale;
  }
}

// One CTA per (unit, range of heads).
template <class Code, int BS, bool ADJACENT, int AXES>
__global__ void __launch_bounds__(kQ8Warps * 32, BS > 16 ? 4 : 0) rope_q8_kernel(const Q8Params qp) {
  const RowParams& p = qp.r;
  __shared__ uint32_t tops[2][kQ8Warps];
  __shared__ float4 table[BS * 32];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == gridDim.x - 1) {   // a CTA that looks at every entry once, used or not
    if (blockIdx.y == 0)
      for (int s = threadIdx.x; s < p.num_seqs; s += kQ8Warps * 32)
        packed_seq(p.query_start, p.context_lens, s, p.num_tokens,
                   static_cast<int64_t>(p.max_blocks) * BS, p.dev_err, true);
    return;
  }
  Piece c;
  if (!find_piece<BS>(qp, c)) return;
  if (c.blk < 0 && threadIdx.x == 0) report(p.dev_err, PKV_DEV_BAD_BLOCK_ID);
  const int first = blockIdx.y * qp.heads_per_cta;
  const int last = min(first + qp.heads_per_cta, p.num_q_heads + 2 * p.num_kv_heads);
  if (c.r1 - c.r0 == 1) {
    const int per = qp.heads_per_cta / kQ8Warps, warp = threadIdx.x >> 5;
    append_row<Code, BS, ADJACENT, AXES>(qp, c, first + warp * per, min(last, first + (warp + 1) * per));
  } else {
    append_rows<Code, BS, ADJACENT, AXES>(qp, c, first, last, tops, table);
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

template <class... P>
int launch(void (*kernel)(P...), dim3 grid, int threads, void* stream, const P&... p) {
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

template <class Code, bool ADJACENT, int AXES>
int launch_q8(const Q8Params& p, int block_size, dim3 grid, void* stream) {
  const auto go = [&](auto kernel) { return launch(kernel, grid, kQ8Warps * 32, stream, p); };
  switch (block_size) {
    case 8: return go(rope_q8_kernel<Code, 8, ADJACENT, AXES>);
    case 16: return go(rope_q8_kernel<Code, 16, ADJACENT, AXES>);
    case 32: return go(rope_q8_kernel<Code, 32, ADJACENT, AXES>);
    default: return go(rope_q8_kernel<Code, 64, ADJACENT, AXES>);
  }
}

template <class Code>
int launch_q8(const Q8Params& p, bool adjacent, int block_size, dim3 grid, void* stream) {
  if (p.r.rot.num_axes == 1)
    return adjacent ? launch_q8<Code, true, 1>(p, block_size, grid, stream)
                    : launch_q8<Code, false, 1>(p, block_size, grid, stream);
  return adjacent ? launch_q8<Code, true, kMaxAxes>(p, block_size, grid, stream)
                  : launch_q8<Code, false, kMaxAxes>(p, block_size, grid, stream);
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
  // a step's heads are spread over as many warps as there are; a prompt's stay together, as
  // they share cosines and sines, as long as there are two rounds of CTAs (four are 3 to 6 %
  // slower on prompts of 32/8 and 32/32 heads)
  constexpr int64_t kLeast = 4 * kQ8Warps, kRounds = 152 * 4 * 2;
  const int64_t parts = p.by_token ? heads : (kRounds + units - 1) / units;
  const int64_t per = std::max(kLeast, (heads + parts * kLeast - 1) / (parts * kLeast) * kLeast);
  p.heads_per_cta = static_cast<int>(per);
  if (units >= INT32_MAX || (heads + per - 1) / per > 65535) return PKV_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(units + 1), static_cast<unsigned>((heads + per - 1) / per));
  return code == PKV_CODE_INT8 ? launch_q8<Int8Near>(p, adjacent != 0, block_size, grid, stream)
                               : launch_q8<E4m3Near>(p, adjacent != 0, block_size, grid, stream);
}
