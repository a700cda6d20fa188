// Rotary positions on the way into the 8-bit cache: the kernels, instantiated for each code in
// rope_q8_int8.cu and rope_q8_e4m3.cu.  What they compute is stated in rope.cu and, for the
// codes, in q8_cache.cu.
//
// What bounds them: HBM and latency for prompts, 16 of 1..4096 tokens of 32/8 heads, half of
// each head rotated, e4m3: 110 us, 5.9 TB/s; 4 of 100..2500 tokens of 32/32 heads in blocks of
// 32, three axes, int8: 46 us, 5.1 TB/s (16 warps an SM, each some 400 instructions for 4 KB).
// A step of 256 tokens of 32/8 heads 4.6 us, a chain of dependent loads, where no block's scale
// grows.  Where every one does, earlier rows are coded anew one after another, a load behind the
// store before it: at row 15 of 16 16 us (int8; e4m3 10), at row 63 of 64 53 (25).
#pragma once

#include <cfloat>

#include "rope.cuh"

namespace pkv {
namespace rope {

// The new rows of one block of one sequence.
struct Piece {
  int s, row0;      // its sequence; the packed row that would be the block's row 0
  int nth;          // of a step's units of the piece (0 of long chunks')
  int base, r0, r1; // place of the block's row 0; new rows [r0, r1)
  int64_t blk;      // -1: no valid id
};

// Units are cut in one of two ways.  Long chunks: the write's units of BS rows, numbered
// without a prefix sum, two to spare for each sequence.  Steps (few tokens a
// sequence on average): every token is a unit, and the units of a piece share its heads.
template <int BS, bool STEP>
__device__ __forceinline__ bool find_piece(const Q8Params& qp, Piece& c) {
  const RowParams& p = qp.r;
  const int unit = blockIdx.x, per = STEP ? 1 : BS, slack = STEP ? 0 : 2;
  c.s = find_unit_seq(p.query_start, p.num_seqs, unit, per, slack);
  const PackedSeq q = packed_seq(p.query_start, p.context_lens, c.s, p.num_tokens,
                                 static_cast<int64_t>(p.max_blocks) * BS, p.dev_err, false);
  if (!q.ok || q.n == 0) return false;
  const int start = q.ctx - q.n;
  int64_t lb;
  if (STEP) {
    const int nth = unit - q.row0;
    if (nth < 0 || nth >= q.n) return false;
    lb = (start + nth) / BS;
    c.nth = start + nth - max(start, static_cast<int>(lb) * BS);
  } else {
    const int nth = unit - unit_base(p.query_start, c.s, BS, 2);
    lb = start / BS + static_cast<int64_t>(nth);
    if (nth < 0 || lb * BS >= q.ctx) return false;
    c.nth = 0;
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

// The barrier of a team of two warps, or of all four.  Numbers that the compiler sees: with one
// in a register a CTA holds all 16 barriers, and an SM has room for half as many CTAs (a step
// of 256 tokens 5.4 us instead of 4.6).
__device__ __forceinline__ void join_team(int team, bool all) {
  if (all)
    asm volatile("bar.sync 1, 128;" ::: "memory");
  else if (team == 0)
    asm volatile("bar.sync 1, 64;" ::: "memory");
  else
    asm volatile("bar.sync 2, 64;" ::: "memory");
}

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
    const bool there = h0 + (lane >> 3) < last, valid = there && ok;
    const HeadAt at(qp, c, BS, min(h0 + (lane >> 3), last - 1));
    // a token that is left out still starts its block's scale, at 0: it would be its last owner's
    const bool scales = there && !at.is_q && c.blk >= 0, stores = scales && ok;
    uint4 xa = make_uint4(0u, 0u, 0u, 0u), xb = xa;
    if (valid) {
      const uint4* from = reinterpret_cast<const uint4*>(at.src + token * at.stride);
      xa = from[ch.a];
      xb = from[ch.b];
    }
    const float before = scales && c.r0 > 0 ? *at.scale : 0.f;
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
    if (scales && (lane & 7) == 0) *at.scale = scale;
  }
}

// More than 16 rows in a step, one after another and twice, for the maximum and for the codes:
// what is in registers then does not depend on how many there are.
template <class Code, bool ADJACENT, int AXES>
struct StepHead {
  const Q8Params& qp;
  const Piece& c;
  const HeadAt at;
  const Chunks ch;
  const bool stores;
  uint32_t top = 0;      // the largest of the finite values as bits

  __device__ __forceinline__ StepHead(const Q8Params& params, const Piece& piece, int block_size, int head)
      : qp(params), c(piece), at(params, piece, block_size, head), ch(threadIdx.x & 7, params.r.rot.n),
        stores(!at.is_q && piece.blk >= 0) {}
  // row r's values in 32 bits; false: it is left out
  __device__ __forceinline__ bool values(int r, float (&a)[8], float (&b)[8]) const {
    const RowParams& p = qp.r;
    const uint4* from = reinterpret_cast<const uint4*>(at.src + (c.row0 + r) * at.stride);
    const uint4 xa = from[ch.a], xb = from[ch.b];
    int32_t pos[AXES];
    load_positions(p.rot, c.row0 + r, c.base + r, pos);
    if (!on_table(p.rot, pos)) return false;
    widen(xa, a);
    widen(xb, b);
    if (!at.is_v && ch.turns) {
      float4 cs[4];
      load_turn<ADJACENT>(p.rot, ch, pos, cs);
      rotate<ADJACENT>(a, b, cs);
    }
    return true;
  }
  // rows own, own + every, ..: q's to their place, what is stored to its maximum
  __device__ __forceinline__ void look(int own, int every) {
    const RowParams& p = qp.r;
    uint32_t all = 0;
#pragma unroll 1
    for (int r = c.r0 + own; r < c.r1; r += every) {
      float a[8], b[8];
      if (!values(r, a, b)) {
        report(p.dev_err, PKV_DEV_BAD_POSITION);
      } else if (at.is_q) {
        uint4* to = reinterpret_cast<uint4*>(p.q_out + (c.row0 + r) * p.q_out_stride + at.g * kHeadDim);
        to[ch.a] = narrow(a);
        to[ch.b] = narrow(b);
      } else {
        all = max(all, __float_as_uint(top_of(top_of(0.f, a), b)));
        drop_nonfinite(a);
        drop_nonfinite(b);
        top = max(top, __float_as_uint(top_of(top_of(0.f, a), b)));
      }
    }
    if (stores && all >= kInf) report(p.dev_err, PKV_DEV_NONFINITE);
  }
  // and their codes, under the maximum of all of them; the block's scale
  __device__ __forceinline__ float code(int own, int every, float before) const {
    const int64_t row_elems = static_cast<int64_t>(qp.r.num_kv_heads) * kHeadDim;
    const float scale = fmaxf(before, __fdiv_rn(__uint_as_float(top), Code::kMax));
    const float inv = inverse_of(scale);
    if (scale > before && c.r0 > 0) {   // earlier rows of the block
      const float ratio = __fdiv_rn(before, scale);
      for (int r = own; r < c.r0; r += every)
        recode16<Code>(at.dst + r * row_elems + 16 * (threadIdx.x & 7), ratio);
    }
#pragma unroll 1
    for (int r = c.r0 + own; r < c.r1; r += every) {
      float a[8], b[8];
      if (!values(r, a, b)) continue;
      drop_nonfinite(a);
      drop_nonfinite(b);
      uint8_t* to = at.dst + r * row_elems;
      *reinterpret_cast<uint2*>(to + 8 * ch.a) = code8<Code>(a, inv);
      *reinterpret_cast<uint2*>(to + 8 * ch.b) = code8<Code>(b, inv);
    }
    return scale;
  }
};

// Up to 16 rows: a head is a team of 1, 2 or 4 warps, 8 lanes a row, whose values stay in
// registers from the maximum to the codes; unit j of n takes each n-th group of heads.
template <class Code, int BS, bool ADJACENT, int AXES>
__device__ __forceinline__ void append_held(const Q8Params& qp, const Piece& c, int first, int last,
                                            uint32_t (&tops)[2][kQ8Warps]) {
  const RowParams& p = qp.r;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = c.r1 - c.r0;
  const int shift = n <= 4 ? 0 : n <= 8 ? 1 : 2, warps = 1 << shift, teams = kQ8Warps >> shift;
  const int team = warp >> shift, own = (warp & (warps - 1)) * 4 + (lane >> 3);
  const Chunks ch(lane & 7, p.rot.n);
  const int64_t row_elems = static_cast<int64_t>(p.num_kv_heads) * kHeadDim;
  const int row = c.row0 + c.r0 + own;   // packed
  bool in = own < n;
  float4 cs[4];
  if (in) {
    int32_t pos[AXES];
    load_positions(p.rot, row, c.base + c.r0 + own, pos);
    in = on_table(p.rot, pos);
    if (!in) report(p.dev_err, PKV_DEV_BAD_POSITION);
    if (in && ch.turns) load_turn<ADJACENT>(p.rot, ch, pos, cs);
  }
  int turns = 0;
#pragma unroll 1
  for (int h = first + c.nth * teams + team; h < last; h += n * teams) {
    const HeadAt at(qp, c, BS, h);
    const bool stores = !at.is_q && c.blk >= 0;
    uint4 xa = make_uint4(0u, 0u, 0u, 0u), xb = xa;
    if (in) {
      const uint4* from = reinterpret_cast<const uint4*>(at.src + row * at.stride);
      xa = from[ch.a];
      xb = from[ch.b];
    }
    const float before = stores && c.r0 > 0 ? *at.scale : 0.f;
    float a[8], b[8];
    widen(xa, a);
    widen(xb, b);
    if (in && !at.is_v && ch.turns) rotate<ADJACENT>(a, b, cs);
    if (at.is_q) {
      if (in) {
        uint4* to = reinterpret_cast<uint4*>(p.q_out + row * p.q_out_stride + at.g * kHeadDim);
        to[ch.a] = narrow(a);
        to[ch.b] = narrow(b);
      }
      continue;
    }
    if (!stores) continue;
    uint32_t top = __float_as_uint(top_of(top_of(0.f, a), b));
    if (top >= kInf) {
      report(p.dev_err, PKV_DEV_NONFINITE);
      drop_nonfinite(a);
      drop_nonfinite(b);
      top = __float_as_uint(top_of(top_of(0.f, a), b));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (shift > 0) {
      if (lane == 0) tops[turns & 1][warp] = top;
      join_team(team, shift == 2);
      for (int w = 0; w < warps; ++w) top = max(top, tops[turns & 1][team * warps + w]);
      ++turns;
    }
    const float scale = fmaxf(before, __fdiv_rn(__uint_as_float(top), Code::kMax));
    const float inv = inverse_of(scale);
    if (scale > before && c.r0 > 0) {   // earlier rows of the block
      const float ratio = __fdiv_rn(before, scale);
      for (int r = own; r < c.r0; r += 4 << shift)
        recode16<Code>(at.dst + r * row_elems + 16 * (lane & 7), ratio);
    }
    if (in) {
      uint8_t* to = at.dst + (c.r0 + own) * row_elems;
      *reinterpret_cast<uint2*>(to + 8 * ch.a) = code8<Code>(a, inv);
      *reinterpret_cast<uint2*>(to + 8 * ch.b) = code8<Code>(b, inv);
    }
    __syncwarp();   // every lane has read the earlier scale (every warp, before they joined)
    if (lane == 0 && (warp & (warps - 1)) == 0) *at.scale = scale;
  }
}

// More than 16 rows: 16 at a time, one for each 8 lanes of the CTA, twice; of the CTA's heads,
// unit j takes each (r1 - r0)-th from j on.  With 255 single tokens a chunk of 250 takes 2.6 us
// (16-token blocks) to 4.2 (64) more; done by a unit a block, 18 to 82.
template <class Code, int BS, bool ADJACENT, int AXES>
__device__ __forceinline__ void append_shared(const Q8Params& qp, const Piece& c, int first, int last,
                                              uint32_t (&tops)[2][kQ8Warps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, own = threadIdx.x >> 3;
  int turns = 0;
#pragma unroll 1
  for (int h = first + c.nth; h < last; h += c.r1 - c.r0) {
    StepHead<Code, ADJACENT, AXES> head(qp, c, BS, h);
    const float before = head.stores && c.r0 > 0 ? *head.at.scale : 0.f;
    head.look(own, kQ8Warps * 4);
    if (!head.stores) continue;
    const uint32_t top = __reduce_max_sync(0xffffffffu, head.top);
    if (lane == 0) tops[turns & 1][warp] = top;
    __syncthreads();   // and every thread has read the earlier scale
    head.top = top;
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) head.top = max(head.top, tops[turns & 1][w]);
    ++turns;
    const float scale = head.code(own, kQ8Warps * 4, before);
    if (threadIdx.x == 0) *head.at.scale = scale;
  }
}

// Pieces of several rows: a warp holds 16 rows of the block (8 of 8-row blocks), 4 a
// pass, and walks the heads, the CTA's rows' cosines and sines in shared memory (read again
// for every head from L1, strided, they bounded the kernel: prompts 203 us instead of 110).  A
// block of 32 or 64 rows is a team of 2 or 4 warps, which join their maxima.  The rotated
// values stay in 32 bits from the maximum to the codes, while the next head's rows are under
// way; computed twice instead, at 96 registers, they took 10 to 20 % longer.  Four CTAs an SM
// (128 registers) for teams, three (0: left to the compiler) where a warp is alone and keeps
// its cosines in registers: 32-token blocks 46 us (three CTAs: 54), 16-token blocks 110 us (four: 113).
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
      join_team(team, kTeam == kQ8Warps);
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

// One CTA per (unit, range of heads).  A step's code without that of long pieces takes half
// the registers, so that its CTAs are all there at once.
template <class Code, int BS, bool ADJACENT, int AXES, bool STEP>
__global__ void __launch_bounds__(kQ8Warps * 32, STEP ? (AXES == 1 ? 8 : 6) : BS > 16 ? 4 : 0)
    rope_q8_kernel(const Q8Params qp) {
  const RowParams& p = qp.r;
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
  if (!find_piece<BS, STEP>(qp, c)) return;
  if (c.blk < 0 && threadIdx.x == 0) report(p.dev_err, PKV_DEV_BAD_BLOCK_ID);
  const int first = blockIdx.y * qp.heads_per_cta;
  const int last = min(first + qp.heads_per_cta, p.num_q_heads + 2 * p.num_kv_heads);
  // the warp's heads
  const int from = first + (threadIdx.x >> 5) * qp.heads_per_warp;
  const int to = min(last, from + qp.heads_per_warp);
  if (c.r1 - c.r0 == 1) {
    append_row<Code, BS, ADJACENT, AXES>(qp, c, from, to);
    return;
  }
  __shared__ uint32_t tops[2][kQ8Warps];
  if constexpr (STEP) {
    if (BS <= 16 || c.r1 - c.r0 <= 16)
      append_held<Code, BS, ADJACENT, AXES>(qp, c, first, last, tops);
    else
      append_shared<Code, BS, ADJACENT, AXES>(qp, c, first, last, tops);
  } else {
    __shared__ float4 table[BS * 32];
    append_rows<Code, BS, ADJACENT, AXES>(qp, c, first, last, tops, table);
  }
}

// ---- host -------------------------------------------------------------------------------

template <class Code, bool ADJACENT, int AXES, bool STEP>
int launch_q8(const Q8Params& p, int block_size, dim3 grid, void* stream) {
  const auto go = [&](auto kernel) { return launch(kernel, grid, kQ8Warps * 32, stream, p); };
  switch (block_size) {
    case 8: return go(rope_q8_kernel<Code, 8, ADJACENT, AXES, STEP>);
    case 16: return go(rope_q8_kernel<Code, 16, ADJACENT, AXES, STEP>);
    case 32: return go(rope_q8_kernel<Code, 32, ADJACENT, AXES, STEP>);
    default: return go(rope_q8_kernel<Code, 64, ADJACENT, AXES, STEP>);
  }
}

template <class Code, bool STEP>
int launch_q8(const Q8Params& p, bool adjacent, int block_size, dim3 grid, void* stream) {
  if (p.r.rot.num_axes == 1)
    return adjacent ? launch_q8<Code, true, 1, STEP>(p, block_size, grid, stream)
                    : launch_q8<Code, false, 1, STEP>(p, block_size, grid, stream);
  return adjacent ? launch_q8<Code, true, kMaxAxes, STEP>(p, block_size, grid, stream)
                  : launch_q8<Code, false, kMaxAxes, STEP>(p, block_size, grid, stream);
}

template <class Code>
int launch_q8_of(const Q8Params& p, bool step, bool adjacent, int block_size, dim3 grid, void* stream) {
  return step ? launch_q8<Code, true>(p, adjacent, block_size, grid, stream)
              : launch_q8<Code, false>(p, adjacent, block_size, grid, stream);
}

}  // namespace rope
}  // namespace pkv
