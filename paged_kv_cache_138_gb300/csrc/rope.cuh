// What the rotary kernels share (fp16 rows and the 8-bit cache): parameters, the rotation,
// the launch.
#pragma once

#include <algorithm>
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

constexpr int kQ8Warps = 4;     // of a CTA of the 8-bit kernels
struct Q8Params {
  RowParams r;                 // k_out, k_cache and v_cache unused
  uint8_t *k_codes, *v_codes;
  float *k_scale, *v_scale;    // [num_blocks, scale_stride]
  int scale_stride;
  int heads_per_cta, heads_per_warp;   // of single rows
};

// launches of the 8-bit kernels, a translation unit each
int launch_q8_int8(const Q8Params& p, bool step, bool adjacent, int block_size, dim3 grid, void* stream);
int launch_q8_e4m3(const Q8Params& p, bool step, bool adjacent, int block_size, dim3 grid, void* stream);

template <class... P>
inline int launch(void (*kernel)(P...), dim3 grid, int threads, void* stream, const P&... p) {
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

}  // namespace rope
}  // namespace pkv
