// Single-token decode attention over the 8-bit paged cache (sm_103a).
//
// out[s,h] = softmax(scale * q[s,h] . K_s^T) V_s over L = context_lens[s]
// tokens, with K_s[t] = code * k_scale[block of t, KV head] and V likewise
// (codes int8 or e4m3, [num_blocks, BS, Hkv, 128] bytes).
//
// The bytes are half the fp16 cache's, so the arithmetic per byte doubles and
// the work is laid out for the fewest instructions a token:
//  * Tokens and dims are the rows of the matrix products, the (at most 8)
//    query heads of a KV head their columns: S^T = K q^T takes 8 and
//    O^T += V^T P^T another 8 mma.m16n8k16 for 16 tokens, half of what query
//    heads as rows would, and no accumulator is padding for 8 heads.
//  * Which dims a lane multiplies in which step is free as long as q agrees,
//    so a lane takes 32 consecutive dims of its token (two 16-byte reads), and
//    for V 16 consecutive dims of its four tokens.  Under the TMA's 128-byte
//    swizzle both patterns are free of bank conflicts.
//  * Codes become fp16 exactly: int8 by placing the byte under the exponent of
//    1024 and subtracting, e4m3 by its conversion.  The scales never touch the
//    values: a block's K scale multiplies its scores, its V scale enters the
//    weight's exponent, w = 2^(x + log2 v_scale - m2), under a unit 2^m2 from a
//    running maximum of its own.  So w keeps fp16's full precision for the tokens
//    that make up the result whatever the scales are: it is off by half a step, 2^-11,
//    or by 2^-32 of the largest.  l sums 2^(x - m) in fp32, without the V scales,
//    so not the rounded weights: a row that one token dominates is off by 2^-11.
//  * 32 tokens a stage (4 KB of K, 4 KB of V), 4 warps with a private 2-stage
//    TMA ring each and 3 CTAs an SM: 192 KB in flight, as the fp16 kernel.
//  * Splits and their fp32 partials are the fp16 kernel's.
//  * What bounds it: HBM.  64 x 4096 of 32 heads, int8 (2.15 GB): 317 us, 6.8 TB/s, the
//    rate of a plain copy (327 on another card); the same copies without the arithmetic take 319.  256 x 4096 of
//    32/8 heads, e4m3: 328-339 us (332 without the arithmetic).  Two contexts of 100k-131k tokens:
//    92 us, 5.2 TB/s: 83-85 us of it here (3.6 rounds of CTAs), the rest the merge.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "attention_kernel.cuh"
#include "q8_device.cuh"

namespace pkv {
namespace attn {

// the fp16 launches' host helpers (paged_attention.cu)
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
bool supported_block_size(int bs);
int seq_stride_for(int num_seqs);

constexpr int kQ8Tile = 32;                      // tokens per stage
constexpr int kQ8HalfBytes = kQ8Tile * kHeadDim; // K or V of a stage
static_assert(2 * kQ8HalfBytes == kStageBytes, "the stage layout of Smem");

struct Q8Params {
  Params p;
  const float* k_scale;   // [num_blocks, scale_stride]
  const float* v_scale;
  int scale_stride;
};

// four codes of one row as two packed fp16 pairs (exact)
struct Int8Half {
  static __device__ __forceinline__ uint32_t bias(uint32_t w) { return w ^ 0x80808080u; }
  // bytes of w (biased by 128): 1024 + u, minus 1152 = the code
  static __device__ __forceinline__ uint32_t pair(uint32_t w, uint32_t sel) {
    const uint32_t h = __byte_perm(w, 0x64646464u, sel);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ uint32_t lo(uint32_t w) { return pair(w, 0x4140); }
  static __device__ __forceinline__ uint32_t hi(uint32_t w) { return pair(w, 0x4342); }
  // K keeps the bias: a byte alone in a half is the subnormal u 2^-24, and the scores start at
  // -128 2^-24 sum q instead of 0.  The sums are then of the size of 255 sum |q| at most,
  // whatever the codes are, and 8 steps round them by 2^-23 each: 2^-12 of a code for each
  // product, where the code itself is off by up to a half.  So nothing is lost even in a
  // block whose scale an outlier sets (under V, where tokens average out, it would count).
  static constexpr float kScoreUnit = 16777216.f, kScoreBias = -128.f / 16777216.f;
  static __device__ __forceinline__ uint32_t k_lo(uint32_t w) { return __byte_perm(w, 0u, 0x4140); }
  static __device__ __forceinline__ uint32_t k_hi(uint32_t w) { return __byte_perm(w, 0u, 0x4342); }
};
struct E4m3Half {
  static __device__ __forceinline__ uint32_t bias(uint32_t w) { return w; }
  static __device__ __forceinline__ uint32_t lo(uint32_t w) { return E4m3Code::half2_of(w & 0xffffu); }
  static __device__ __forceinline__ uint32_t hi(uint32_t w) { return E4m3Code::half2_of(w >> 16); }
  static constexpr float kScoreUnit = 1.f, kScoreBias = 0.f;
  static __device__ __forceinline__ uint32_t k_lo(uint32_t w) { return lo(w); }
  static __device__ __forceinline__ uint32_t k_hi(uint32_t w) { return hi(w); }
};

__device__ __forceinline__ uint4 q8_chunk(const uint8_t* half, int row, int c) {
  return *reinterpret_cast<const uint4*>(half + row * 128 + ((c ^ (row & 7)) << 4));
}

// transpose an 8x8 fp16 matrix held one row per four lanes
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Online-softmax state of the lane's two query heads (2 (lane % 4) + {0, 1}).
// O is in units of 2^m2; rows of the MMA are dims 16 (lane / 4) + {2 i, 2 i + 1}.
struct Q8State {
  float m[2], m2[2], l[2];
  float o[8][4];
};

// The unit of the fp16 weights and of O is 2^-7 of the running maximum, so that the weights
// fill fp16's range: at most 2^(7 + kRescaleThreshold), and what rounds to 0 is below 2^-32
// of the maximum (2^-25 with the maximum itself for a unit).
constexpr float kHeadroom = 7.f;
static_assert(kHeadroom + kRescaleThreshold <= 15.f, "weights in fp16's range");
constexpr float kNoMax = -1e30f;    // below every exponent, and finite: x - m is never inf - inf
constexpr int kLeftOut = 0x7fc0dead;  // in place of a K scale: the block has no valid id (a NaN
                                      // that no arithmetic makes)

// One stage of 32 tokens.  ks[j] / lv[j]: K scale * scale * log2 e and
// log2 of the V scale of box j (boxes of BS, at most 32, tokens).
template <class Half, int BOXES>
__device__ __forceinline__ void q8_tile(const uint8_t* st, const uint32_t (&qb)[8][2],
                                        const float (&s0)[2],
                                        const float (&ks)[BOXES], const float (&lv)[BOXES],
                                        int valid, int lane, Q8State& a) {
  constexpr unsigned kFull = 0xffffffffu;
  const int r = lane >> 2, c = lane & 3;
  float x[2][4];   // [16-token half][token r head 0, head 1, token r + 8 head 0, head 1]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float s[4] = {s0[0], s0[1], s0[0], s0[1]};
    const int t0 = 16 * h + r, t1 = t0 + 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 w0 = q8_chunk(st, t0, 2 * c + i);
      const uint4 w1 = q8_chunk(st, t1, 2 * c + i);
      const uint32_t u0[4] = {w0.x, w0.y, w0.z, w0.w}, u1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t b0 = Half::bias(u0[j]), b1 = Half::bias(u1[j]);
        mma_16816_full(s, Half::k_lo(b0), Half::k_lo(b1), Half::k_hi(b0), Half::k_hi(b1),
                       qb[4 * i + j][0], qb[4 * i + j][1]);
      }
    }
    const float k0 = ks[16 * h * BOXES / kQ8Tile], k1 = ks[(16 * h + 8) * BOXES / kQ8Tile];
    const bool in0 = t0 < valid && __float_as_int(k0) != kLeftOut;
    const bool in1 = t1 < valid && __float_as_int(k1) != kLeftOut;
    x[h][0] = in0 ? s[0] * k0 : -INFINITY;
    x[h][1] = in0 ? s[1] * k0 : -INFINITY;
    x[h][2] = in1 ? s[2] * k1 : -INFINITY;
    x[h][3] = in1 ? s[3] * k1 : -INFINITY;
  }
  // lv of the lane's tokens: a box never ends inside 8 tokens
  const float lv4[2][2] = {{lv[0], lv[8 * BOXES / kQ8Tile]},
                           {lv[16 * BOXES / kQ8Tile], lv[24 * BOXES / kQ8Tile]}};
  // the maxima move only when a token passes one by more than 2^8: most tiles
  // take one vote and no exchange
  float bm[2], bm2[2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    bm[n] = fmaxf(fmaxf(x[0][n], x[0][2 + n]), fmaxf(x[1][n], x[1][2 + n]));
    bm2[n] = fmaxf(fmaxf(x[0][n] + lv4[0][0], x[0][2 + n] + lv4[0][1]),
                   fmaxf(x[1][n] + lv4[1][0], x[1][2 + n] + lv4[1][1]));
  }
  const bool moves = bm[0] > a.m[0] + kRescaleThreshold || bm[1] > a.m[1] + kRescaleThreshold ||
                     bm2[0] > a.m2[0] + (kHeadroom + kRescaleThreshold) ||
                     bm2[1] > a.m2[1] + (kHeadroom + kRescaleThreshold);
  if (__any_sync(kFull, moves)) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        bm[n] = fmaxf(bm[n], __shfl_xor_sync(kFull, bm[n], o));
        bm2[n] = fmaxf(bm2[n], __shfl_xor_sync(kFull, bm2[n], o));
      }
      if (bm[n] > a.m[n] + kRescaleThreshold) {
        a.l[n] *= exp2_approx(a.m[n] - bm[n]);
        a.m[n] = bm[n];
      }
      if (bm2[n] > a.m2[n] + (kHeadroom + kRescaleThreshold)) {
        const float unit = bm2[n] - kHeadroom;
        const float alpha = exp2_approx(a.m2[n] - unit);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a.o[i][n] *= alpha;
          a.o[i][2 + n] *= alpha;
        }
        a.m2[n] = unit;
      }
    }
  }
  uint32_t pb[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = i & 1;
      a.l[n] += exp2_approx(x[h][i] - a.m[n]);
      w[i] = exp2_approx(x[h][i] + lv4[h][i >> 1] - a.m2[n]);
    }
    pb[h][0] = movmatrix(pack_half2(w[0], w[1]));
    pb[h][1] = movmatrix(pack_half2(w[2], w[3]));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t t[4][4];   // tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of the half, 16 dims each
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 w = q8_chunk(st + kQ8HalfBytes, 16 * h + 2 * c + (k & 1) + 8 * (k >> 1), r);
      t[k][0] = w.x;
      t[k][1] = w.y;
      t[k][2] = w.z;
      t[k][3] = w.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a01 = Half::bias(__byte_perm(t[0][j], t[1][j], 0x5140));
      const uint32_t b01 = Half::bias(__byte_perm(t[2][j], t[3][j], 0x5140));
      mma_16816_full(a.o[2 * j], Half::lo(a01), Half::hi(a01), Half::lo(b01), Half::hi(b01),
                     pb[h][0], pb[h][1]);
      const uint32_t a23 = Half::bias(__byte_perm(t[0][j], t[1][j], 0x7362));
      const uint32_t b23 = Half::bias(__byte_perm(t[2][j], t[3][j], 0x7362));
      mma_16816_full(a.o[2 * j + 1], Half::lo(a23), Half::hi(a23), Half::lo(b23), Half::hi(b23),
                     pb[h][0], pb[h][1]);
    }
  }
}

// fp16 output of dims d .. d + 3 of a row: 0 where every token was left out (a sum of 0),
// NaN where the sum is NaN
__device__ __forceinline__ void store_q8_out4(__half* o, float den, float4 num) {
  const bool none = den == 0.f;
  uint2 u;
  u.x = pack_half2(none ? 0.f : num.x / den, none ? 0.f : num.y / den);
  u.y = pack_half2(none ? 0.f : num.z / den, none ? 0.f : num.w / den);
  *reinterpret_cast<uint2*>(o) = u;
}

// One CTA per (KV head, sequence, split); warp w streams tiles w, w + 4, ...
template <class Half, int BS, bool CLEAR>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    paged_attention_q8_kernel(const __grid_constant__ CUtensorMap tmap_k,
                              const __grid_constant__ CUtensorMap tmap_v, const Q8Params qp) {
  constexpr unsigned kFull = 0xffffffffu;
  constexpr int kBoxes = BS < kQ8Tile ? kQ8Tile / BS : 1;   // per stage
  constexpr int kBoxTok = kQ8Tile / kBoxes;
  constexpr int kMaxTiles = kMaxPartitionTiles * kTile / kQ8Tile / kWarps;   // of a warp
  constexpr int kSlots = (kMaxTiles * kBoxes + 31) / 32;
  // launched as a programmatic dependent of the stream's previous kernel
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Params& p = qp.p;
  uint8_t* smem = aligned_smem();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.x, split = blockIdx.z;
  const int y = blockIdx.y;
  const int s = (p.rank_by_length && blockIdx.z == gridDim.z - 1)
                    ? ranked_sequence(p, smem, zigzag_rank(y, p.num_seqs))
                    : static_cast<int>(static_cast<int64_t>(y) * p.seq_stride % p.num_seqs);
  const int G = p.num_q_heads / p.num_kv_heads;
  const int L = clamp_context<BS>(p, s, threadIdx.x == 0 && g == 0 && split == 0);
  if (L == 0) {
    if (split == 0) {
      __half* o = p.out + (static_cast<int64_t>(s) * p.num_q_heads + g * G) * kHeadDim;
      for (int i = threadIdx.x; i < G * kHeadDim; i += kThreads) o[i] = __float2half_rn(0.f);
    }
    return;
  }
  const int split_tok = p.partition_tiles * kTile;
  const int64_t first64 = static_cast<int64_t>(split) * split_tok;
  if (first64 >= L) return;
  const int first = static_cast<int>(first64);
  const int nsplit = (L - 1) / split_tok + 1;
  const int tiles = (min(split_tok, L - first) + kQ8Tile - 1) / kQ8Tile;
  const int mine = warp < tiles ? (tiles - warp + kWarps - 1) / kWarps : 0;

  // block ids of the warp's boxes, box b of its tile k at lane (k boxes + b) % 32;
  // a block out of range, or past the context, is read from past the cache's
  // last row, where the copy engine fills zeros
  const int64_t oob = p.num_blocks * BS;
  int32_t row[kSlots];
  float ksv[kSlots], lvv[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int box = i * 32 + lane;
    const int tok = first + ((box / kBoxes) * kWarps + warp) * kQ8Tile + (box % kBoxes) * kBoxTok;
    row[i] = static_cast<int32_t>(oob);
    ksv[i] = 0.f;
    lvv[i] = -INFINITY;
    if (box < mine * kBoxes && static_cast<unsigned>(tok) < static_cast<unsigned>(L)) {
      const int32_t b = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks + tok / BS);
      if (b < 0 || b >= p.num_blocks) {
        report(p.dev_err, PKV_DEV_BAD_BLOCK_ID);
        ksv[i] = __int_as_float(kLeftOut);   // its tokens are left out
      } else {
        row[i] = b * BS + tok % BS;
        const int64_t at = static_cast<int64_t>(b) * qp.scale_stride + g;
        ksv[i] = __ldg(qp.k_scale + at) * p.scale_log2 * Half::kScoreUnit;
        lvv[i] = __log2f(__ldg(qp.v_scale + at));
      }
    }
  }
  uint8_t* ring = smem + Smem::stages + warp * kStages * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Smem::bars) + warp * kStages;
  if (lane == 0) {
    if (warp == 0) {
      prefetch_tmap(&tmap_k);
      prefetch_tmap(&tmap_v);
    }
    for (int j = 0; j < kStages; ++j) mbar_init(&bars[j], 1);
    fence_barrier_init();
  }
  __syncwarp();
  const auto issue = [&](int k) {   // the whole warp; lane 0 starts the copies
    int32_t r[kBoxes];
#pragma unroll
    for (int b = 0; b < kBoxes; ++b) {
      const int box = k * kBoxes + b;
      int32_t v = row[0];
#pragma unroll
      for (int i = 1; i < kSlots; ++i) v = (box >> 5) == i ? row[i] : v;
      r[b] = __shfl_sync(kFull, v, box & 31);
    }
    if (lane == 0) {
      uint64_t* bar = &bars[k % kStages];
      uint8_t* st = ring + (k % kStages) * kStageBytes;
      mbar_arrive_expect_tx(bar, kStageBytes);
#pragma unroll
      for (int b = 0; b < kBoxes; ++b) {
        tma_load_3d(st + b * kBoxTok * kHeadDim, &tmap_k, 0, g, r[b], bar);
        tma_load_3d(st + kQ8HalfBytes + b * kBoxTok * kHeadDim, &tmap_v, 0, g, r[b], bar);
      }
    }
  };
  int issued = min(kStages, mine);
#pragma unroll
  for (int k = 0; k < kStages; ++k)
    if (k < issued) issue(k);

  // q as the products' B fragments: head lane / 4, dims 32 (lane % 4) + 4 step ..
  uint32_t qb[8][2];
  {
    const int h = lane >> 2;
    const uint2* src = reinterpret_cast<const uint2*>(
        p.q + (static_cast<int64_t>(s) * p.num_q_heads + g * G + h) * kHeadDim + 32 * (lane & 3));
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint2 w = h < G ? __ldg(src + k) : make_uint2(0u, 0u);
      qb[k][0] = w.x;
      qb[k][1] = w.y;
    }
  }

  // where the scores of the lane's two heads start (e4m3: 0, and NaN for a q that is not
  // finite: its scores, were they all -inf, would else look like a head without tokens)
  float s0[2];
  {
    float sum = 0.f;   // of head lane / 4 over the lane's 32 dims, then over the four lanes
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += sum_half2(qb[k][0]) + sum_half2(qb[k][1]);
    sum += __shfl_xor_sync(kFull, sum, 1);
    sum += __shfl_xor_sync(kFull, sum, 2);
#pragma unroll
    for (int n = 0; n < 2; ++n)
      s0[n] = __shfl_sync(kFull, sum, 4 * (2 * (lane & 3) + n)) * Half::kScoreBias;
  }

  Q8State a;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    a.m[n] = a.m2[n] = kNoMax;
    a.l[n] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) a.o[i][0] = a.o[i][1] = a.o[i][2] = a.o[i][3] = 0.f;

  const auto landed = [&](int k) {
    return warp_wait(&bars[k % kStages], (k / kStages) & 1, p.dev_err);
  };
  bool ok = true;
  int k = 0;
  for (; k < issued; ++k) {
    ok = landed(k);
    if (!ok) break;
    const uint8_t* st = ring + (k % kStages) * kStageBytes;
    float ks[kBoxes], lv[kBoxes];
#pragma unroll
    for (int b = 0; b < kBoxes; ++b) {
      const int box = k * kBoxes + b;
      float vk = ksv[0], vl = lvv[0];
#pragma unroll
      for (int i = 1; i < kSlots; ++i) {
        vk = (box >> 5) == i ? ksv[i] : vk;
        vl = (box >> 5) == i ? lvv[i] : vl;
      }
      ks[b] = __shfl_sync(kFull, vk, box & 31);
      lv[b] = __shfl_sync(kFull, vl, box & 31);
    }
    const int valid = L - first - (k * kWarps + warp) * kQ8Tile;
    if (CLEAR && valid < kQ8Tile) {
      // rows past the context may hold any byte, and e4m3 has NaN codes: 0 * NaN
      // would poison the sums
      for (int i = lane; i < (kQ8Tile - valid) * 8; i += 32)
        st_shared_zero16(smem_u32(st) + kQ8HalfBytes + valid * kHeadDim + i * 16);
      fence_proxy_async_smem();
      __syncwarp();
    }
    q8_tile<Half, kBoxes>(st, qb, s0, ks, lv, valid, lane, a);
    __syncwarp();
    if (issued < mine) {
      issue(issued);
      ++issued;
    }
  }
  // after a wait that gave up its copies and those behind them are still on their way into the
  // ring: they get a bounded wait each before the shared memory goes to another CTA
  for (; !ok && k < issued; ++k) landed(k);
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) a.l[n] += __shfl_xor_sync(kFull, a.l[n], o);

  // after a wait that gave up: no merge (it reuses the rings), no store
  if (__syncthreads_or(!ok)) return;
  float* ml = reinterpret_cast<float*>(smem + Smem::ml);
  float* ob = reinterpret_cast<float*>(smem + Smem::stages);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int h = 2 * (lane & 3) + n;
    if (h >= G) continue;
    // O from units of 2^m2 (the V scales in them) to units of 2^m
    const float f = exp2_approx(a.m2[n] - a.m[n]);
    if (lane < 4) {
      ml[(warp * 16 + h) * 2] = a.m[n];
      ml[(warp * 16 + h) * 2 + 1] = a.l[n];
    }
    float* orow = ob + (warp * 16 + h) * kHeadDim + 16 * (lane >> 2);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float2*>(orow + 2 * i) = make_float2(a.o[i][n] * f, a.o[i][2 + n] * f);
  }
  __syncthreads();
  merge_warps(ml, ob, G, [&](int gi, int d, float M, float den, float4 num) {
    const int64_t orow = static_cast<int64_t>(s) * p.num_q_heads + g * G + gi;
    if (nsplit == 1)
      store_q8_out4(p.out + orow * kHeadDim + d, den, num);
    else
      store_partial(p, orow, split, d, M, den, num);
  });
}

// Log-sum-exp merge of a row's splits by ROW_WARPS warps: warp w takes splits w,
// w + ROW_WARPS, ..., their sums join in warp order.  A CTA (8 warps) a row against a warp
// a row (whole calls, int8, 32/8 heads unless said): 118 splits of 64 rows 92 us instead
// of 133, 16 splits (8 x 8000, e4m3) 32.3 and 36.1, 8 splits 33.9 and 36.5 (16 x 4096),
// 16.3 and 18.3 (8 x 4096, 8/8, its 67 MB in L2); 4 splits 35.1 and 34.9 (32 x 2048), 2 splits 38.0 and 35.1
// (64 x 1024): a CTA for each of 2048 rows costs more than it reads.
constexpr int kWideSplits = 8;   // a CTA a row from here on
constexpr int kMergeWarps = 8;
template <int ROW_WARPS>
__global__ void __launch_bounds__(kMergeWarps * 32) q8_merge_kernel(const Params p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kRows = kMergeWarps / ROW_WARPS;   // of a CTA
  static_assert(ROW_WARPS == 1 || kRows == 1, "one row's sums meet in shared memory at most");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + warp / ROW_WARPS;
  if (row >= static_cast<int64_t>(p.num_seqs) * p.num_q_heads) return;
  const int s = static_cast<int>(row / p.num_q_heads);
  const int cap = p.max_blocks * p.block_size;
  const int L = max(0, min(__ldg(p.context_lens + s), cap));
  const int n = splits_for_tiles(p, (L + kTile - 1) / kTile);
  if (n <= 1) return;   // written by its only split
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + row * p.max_splits;
  const float4* po = reinterpret_cast<const float4*>(p.part_o) + row * p.max_splits * 32 + lane;
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, ml[i].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
#pragma unroll (ROW_WARPS == 1 ? 4 : 8)
  for (int i = warp % ROW_WARPS; i < n; i += ROW_WARPS) {
    const float2 w = ml[i];
    const float4 v = po[static_cast<int64_t>(i) * 32];
    const float c = exp2_approx(w.x - M);
    num.x += c * v.x;
    num.y += c * v.y;
    num.z += c * v.z;
    num.w += c * v.w;
    den += c * w.y;
  }
  if (ROW_WARPS > 1) {
    __shared__ float4 part[ROW_WARPS][32];
    __shared__ float dens[ROW_WARPS];
    part[warp][lane] = num;
    if (lane == 0) dens[warp] = den;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < ROW_WARPS; ++w) {
      const float4 v = part[w][lane];
      num.x += v.x;
      num.y += v.y;
      num.z += v.z;
      num.w += v.w;
      den += dens[w];
    }
  }
  store_q8_out4(p.out + row * kHeadDim + 4 * lane, den, num);
}

// The cache as [num_blocks * BS rows, Hkv, 128 bytes]; a box is min(BS, 32)
// rows of one head under the 128-byte swizzle.
bool make_q8_map(CUtensorMap* map, const void* base, int num_kv_heads, int64_t num_blocks,
                 int block_size) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(num_kv_heads),
                        static_cast<cuuint64_t>(num_blocks) * block_size};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim),
                           static_cast<cuuint64_t>(num_kv_heads) * kHeadDim};
  cuuint32_t box[3] = {kHeadDim, 1, static_cast<cuuint32_t>(std::min(block_size, kQ8Tile))};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Half, int BS, bool CLEAR>
int launch_q8(const CUtensorMap& mk, const CUtensorMap& mv, const Q8Params& qp, int splits,
              cudaStream_t st) {
  static std::atomic<uint8_t> opted_in[64];
  const int rc = opt_in_smem(paged_attention_q8_kernel<Half, BS, CLEAR>, opted_in);
  if (rc != PKV_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(qp.p.num_kv_heads, qp.p.num_seqs, splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem::alloc;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_attention_q8_kernel<Half, BS, CLEAR>, mk, mv, qp) ==
                 cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

template <class Half, bool CLEAR>
int launch_q8_bs(int block_size, const CUtensorMap& mk, const CUtensorMap& mv, const Q8Params& qp,
                 int splits, cudaStream_t st) {
  switch (block_size) {
    case 8: return launch_q8<Half, 8, CLEAR>(mk, mv, qp, splits, st);
    case 16: return launch_q8<Half, 16, CLEAR>(mk, mv, qp, splits, st);
    case 32: return launch_q8<Half, 32, CLEAR>(mk, mv, qp, splits, st);
    default: return launch_q8<Half, 64, CLEAR>(mk, mv, qp, splits, st);
  }
}

}  // namespace attn
}  // namespace pkv

extern "C" int pkv_paged_attention_decode_q8(void* out, const void* q, const void* k_cache,
                                             const void* v_cache, const float* k_scale,
                                             const float* v_scale, int code,
                                             const int32_t* block_tables,
                                             const int32_t* context_lens, int num_seqs,
                                             int num_q_heads, int num_kv_heads, int head_dim,
                                             int block_size, int64_t num_blocks,
                                             int max_blocks_per_seq, int scale_stride,
                                             float scale, void* workspace, size_t workspace_bytes,
                                             int32_t* dev_err, void* stream) {
  using namespace pkv::attn;
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0 || scale_stride < num_kv_heads)
    return PKV_ERR_INVALID_ARG;
  if (code != PKV_CODE_INT8 && code != PKV_CODE_E4M3) return PKV_ERR_INVALID_ARG;
  if (head_dim != kHeadDim || !supported_block_size(block_size)) return PKV_ERR_UNSUPPORTED;
  if (num_q_heads % num_kv_heads != 0) return PKV_ERR_UNSUPPORTED;
  const int G = num_q_heads / num_kv_heads;
  if (G != 1 && G != 2 && G != 4 && G != 8) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables ||
      !context_lens)
    return PKV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
       reinterpret_cast<uintptr_t>(workspace)) &
      15)
    return PKV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 7)
    return PKV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3)
    return PKV_ERR_INVALID_ARG;
  if (num_blocks > INT32_MAX / block_size || num_seqs > 65535 || num_kv_heads > 65535)
    return PKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_blocks_per_seq) * block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  const size_t need = pkv_paged_attention_workspace_bytes(num_seqs, num_q_heads,
                                                          max_blocks_per_seq, block_size, head_dim);
  if (need > 0 && (!workspace || workspace_bytes < need)) return PKV_ERR_INVALID_ARG;
  const int partition =
      partition_tiles_for(num_seqs, num_kv_heads, max_blocks_per_seq, block_size);
  const int splits = max_splits_for(max_blocks_per_seq, block_size, partition);
  if (splits > 65535) return PKV_ERR_UNSUPPORTED;

  Q8Params qp = {};
  Params& p = qp.p;
  p.out = static_cast<__half*>(out);
  p.q = static_cast<const __half*>(q);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.max_splits = splits;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = need ? p.part_o + static_cast<size_t>(num_seqs) * num_q_heads * splits * kHeadDim
                   : nullptr;
  p.dev_err = dev_err;
  p.num_blocks = num_blocks;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks = max_blocks_per_seq;
  p.block_size = block_size;
  p.seq_stride = seq_stride_for(num_seqs);
  {
    // as the fp16 launch: the last split plane in zigzag order of length
    const int64_t table_tiles =
        tiles_for_tokens(static_cast<int64_t>(max_blocks_per_seq) * block_size);
    const int64_t last_plane_tiles = table_tiles - static_cast<int64_t>(splits - 1) * partition;
    p.rank_by_length = num_seqs <= kMaxRankedSeqs && 2 * last_plane_tiles >= partition;
  }
  p.partition_tiles = partition;
  // an infinite scale makes every score infinite or NaN: NaN for all, as every score of
  // -inf would look like a head without tokens
  p.scale_log2 = std::isfinite(scale) ? scale * 1.4426950408889634f : NAN;
  qp.k_scale = k_scale;
  qp.v_scale = v_scale;
  qp.scale_stride = scale_stride;

  CUtensorMap mk, mv;
  if (!make_q8_map(&mk, k_cache, num_kv_heads, num_blocks, block_size) ||
      !make_q8_map(&mv, v_cache, num_kv_heads, num_blocks, block_size))
    return PKV_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rc = code == PKV_CODE_INT8
                     ? launch_q8_bs<Int8Half, false>(block_size, mk, mv, qp, splits, st)
                     : launch_q8_bs<E4m3Half, true>(block_size, mk, mv, qp, splits, st);
  if (rc != PKV_OK) return rc;
  if (p.max_splits <= 1) return PKV_OK;
  const int64_t rows = static_cast<int64_t>(num_seqs) * num_q_heads;
  const bool wide = p.max_splits >= kWideSplits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(wide ? rows : (rows + kMergeWarps - 1) / kMergeWarps));
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, wide ? q8_merge_kernel<kMergeWarps> : q8_merge_kernel<1>, p) ==
                 cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}
