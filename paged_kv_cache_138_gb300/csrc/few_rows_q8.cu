// Causal attention of a few rows a sequence over the 8-bit paged cache (sm_103a): draft
// tokens that are checked, short chunks, single tokens.
//
//   out[i, h] = sum_{t <= pos} softmax_t(scale <q[i, h], K[t, g]>) V[t, g]
// as in prompt_q8.cu, whose products take 128 query rows at a time whatever there are, and
// whose widened tiles pass through shared memory.  Here tokens and dims are the rows of
// mma.m16n8k16 and the query rows its columns, 8 or 16 of them: codes are read from shared
// memory once, widened in registers, exactly, and each fragment meets one or two groups of
// 8 columns.
//  * A unit is (8 or 16 rows of one KV head of one sequence, a split of its context).  Its 4
//    warps stream 32 tokens each at a time (4 KB of K, 4 KB of V) through private rings of two
//    stages; three CTAs an SM have 192 KB under way.
//  * Which dims a lane multiplies in which step is free as long as q agrees: a lane takes
//    32 consecutive dims of its token (two 16-byte reads), and for V 16 consecutive dims
//    of its four tokens; under the 128-byte swizzle both are free of bank conflicts.
//  * Scales as in prompt_q8.cu: K's multiplies scores, V's enters the weight's exponent, and
//    is divided out of the sum.
//  * The warps' maxima, sums and outputs join in shared memory, splits in
//    prompt_merge_kernel.
//  * What bounds it: HBM for 8 columns, 256 x 1 rows over 4096 of 32/8 heads 330-337 us (the
//    single-token kernel 328-342); 64 x 2 rows 103-106 us, 80 of them the bytes', the rest the last
//    round of CTAs and the merge; arithmetic for 16, 64 x 4 rows 119-125 us (prompt_q8.cu
//    132-144).  32 columns took 166 us (64 x 8 rows; prompt_q8.cu 130-142): the products
//    of warps alone take as long as the copies then, with two CTAs an SM to hide them.
#include "prompt_q8.cuh"

namespace pkv {
namespace prompt_q8 {

namespace {

constexpr int kStepTok = 32;                        // tokens of a stage
constexpr int kHalfStage = kStepTok * kHeadDim;     // K or V of it
constexpr int kStageBytes = 2 * kHalfStage;
constexpr int kWarps = 4, kFewThreads = kWarps * 32, kFewStages = 2;
constexpr int kRings = kWarps * kFewStages * kStageBytes;
constexpr int kFewCtas = 3;                         // of an SM

template <int COLS>
struct FewSmem {
  static constexpr int bars = kRings;                          // u64 [warps][stages]
  static constexpr int ml = bars + kWarps * kFewStages * 8;    // float2 [warps][COLS]
  static constexpr int alloc = ml + kWarps * COLS * 8 + 1024;  // 1024: alignment
  static_assert(kWarps * COLS * kHeadDim * 4 <= kRings, "the warps' outputs meet in the rings");
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}
// transpose an 8x8 fp16 matrix held one row per four lanes
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint4 chunk_of(const uint8_t* half, int row, int c) {
  return *reinterpret_cast<const uint4*>(half + row * 128 + ((c ^ (row & 7)) << 4));
}

// 8 columns: the lane's two are 2 (lane % 4) + {0, 1}, its dims 16 (lane / 4) + {2 i, 2 i + 1}
struct Column8 {
  float m[2], l[2];
  float o[8][4];
};

// Registers bound the CTAs of an SM: a column group's q takes 16, its state 36.
template <class Wide, int BS, int GROUPS>
__global__ void __launch_bounds__(kFewThreads, kFewCtas)
    few_rows_q8_kernel(const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const Q8Params qp) {
  constexpr unsigned kFull = 0xffffffffu;
  constexpr int kCols = 8 * GROUPS;
  constexpr int kBoxes = BS < kStepTok ? kStepTok / BS : 1;   // per stage
  constexpr int kBoxTok = kStepTok / kBoxes;
  constexpr int kBatch = 32 / kBoxes;                         // stages whose boxes fill a warp
  using Smem = FewSmem<kCols>;
  const Params& p = qp.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t max_context = static_cast<int64_t>(p.max_blocks) * BS;
  // a programmatic dependent of the stream's previous kernel
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // every entry is looked at once, used or not, where seldom a unit is (see few_rows_plan)
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == 0)
    for (int s = threadIdx.x; s < p.num_seqs; s += kFewThreads)
      packed_seq(p.query_start, p.context_lens, s, p.num_tokens, max_context, p.dev_err, true);

  // ---- the unit -----------------------------------------------------------------------------
  const int shift = p.group_shift, per = kCols >> shift;   // tokens of a unit
  const int unit = blockIdx.x / p.num_kv_heads, g = blockIdx.x % p.num_kv_heads;
  const int s = find_unit_seq(p.query_start, p.num_seqs, unit, per, 1);
  const PackedSeq seq = packed_seq(p.query_start, p.context_lens, s, p.num_tokens, max_context,
                                   p.dev_err, false);
  const int nth = unit - unit_base(p.query_start, s, per, 1);
  if (!seq.ok || nth < 0 || static_cast<int64_t>(nth) * per >= seq.n) return;
  const int tok0 = nth * per, toks = min(per, seq.n - tok0);
  const int pos0 = seq.ctx - seq.n + tok0;             // of the unit's first token
  const int64_t split_tok = static_cast<int64_t>(p.split_tiles) * kTile;
  const int64_t first64 = blockIdx.y * split_tok;
  if (first64 >= pos0 + toks) return;                  // its last token sees pos0 + toks
  const int first = static_cast<int>(first64);
  const int end = static_cast<int>(min(first64 + split_tok, static_cast<int64_t>(pos0 + toks)));
  const int steps = (end - first + kStepTok - 1) / kStepTok;
  const int mine = warp < steps ? (steps - warp + kWarps - 1) / kWarps : 0;

  // ---- copies -------------------------------------------------------------------------------
  // Block ids and scales come a batch of 32 boxes at a time, ids a batch ahead, scales
  // when the batch's first copy starts, two stages before they are used.
  const auto first_token = [&](int k) { return first + (k * kWarps + warp) * kStepTok; };
  const auto ids_of = [&](int b) {   // -1 past the unit's tokens
    const int k = b * kBatch + lane / kBoxes;
    const int64_t tok = static_cast<int64_t>(first) + (static_cast<int64_t>(k) * kWarps + warp) * kStepTok +
                        lane % kBoxes * kBoxTok;
    return k < mine && tok < seq.ctx
               ? __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks + tok / BS)
               : -1;
  };
  const auto scales_of = [&](int32_t id) {
    if (id < 0 || id >= p.num_blocks) return make_float2(0.f, 0.f);
    const int64_t at = static_cast<int64_t>(id) * qp.scale_stride + g;
    return make_float2(__ldg(qp.k_scale + at), __ldg(qp.v_scale + at));
  };
  int32_t ids = ids_of(0), ids1 = ids_of(1);
  float2 loaded = make_float2(0.f, 0.f);
  BlockScale sc = {1.f, 0.f, 1.f};
  uint8_t* ring = smem + warp * kFewStages * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Smem::bars) + warp * kFewStages;
  if (lane == 0) {
    if (warp == 0) {
      prefetch_tmap(&tmap_k);
      prefetch_tmap(&tmap_v);
    }
    for (int j = 0; j < kFewStages; ++j) mbar_init(&bars[j], 1);
    fence_barrier_init();
  }
  __syncwarp();
  const auto issue = [&](int k) {   // the whole warp
    const int in_batch = k % kBatch;
    if (in_batch == 0) {
      if (k > 0) {
        ids = ids1;
        ids1 = ids_of(k / kBatch + 1);
      }
      loaded = scales_of(ids);
    }
    const int32_t id = __shfl_sync(kFull, ids, in_batch * kBoxes + lane % kBoxes);
    const int tok = first_token(k) + lane % kBoxes * kBoxTok;
    int row = static_cast<int>(p.num_blocks * BS);   // past the last row: zeros
    if (id >= 0 && id < p.num_blocks)
      row = id * BS + tok % BS;
    else if (lane < kBoxes && tok < seq.ctx)
      report(p.dev_err, PKV_DEV_BAD_BLOCK_ID);
    uint64_t* b = &bars[k % kFewStages];
    uint8_t* st = ring + (k % kFewStages) * kStageBytes;
    if (lane == 0) mbar_arrive_expect_tx(b, kStageBytes);
    __syncwarp();
    if (lane < kBoxes) {
      tma_load_3d(st + lane * kBoxTok * kHeadDim, &tmap_k, 0, g, row, b);
      tma_load_3d(st + kHalfStage + lane * kBoxTok * kHeadDim, &tmap_v, 0, g, row, b);
    }
  };
  int issued = min(kFewStages, mine);
#pragma unroll
  for (int k = 0; k < kFewStages; ++k)
    if (k < issued) issue(k);

  // q as the products' B fragments: column lane / 4 of each group, dims 32 (lane % 4) + 4 step ..
  uint32_t qb[GROUPS][8][2];
#pragma unroll
  for (int c = 0; c < GROUPS; ++c) {
    const int n = 8 * c + (lane >> 2), tok = n >> shift;
    const uint2* src = reinterpret_cast<const uint2*>(
        qp.q + ((static_cast<int64_t>(seq.row0) + tok0 + tok) * p.num_q_heads + (g << shift) +
                (n & ((1 << shift) - 1))) * kHeadDim + 32 * (lane & 3));
    // a negative scale negates q, so that a row's maximum is the largest score either way
    const uint32_t sign = p.idesc_qk & kNegateA ? 0x80008000u : 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint2 w = tok < toks ? __ldg(src + k) : make_uint2(0u, 0u);
      qb[c][k][0] = w.x ^ sign;
      qb[c][k][1] = w.y ^ sign;
    }
  }

  Column8 col[GROUPS];
#pragma unroll
  for (int c = 0; c < GROUPS; ++c) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      col[c].m[n] = kNoMax;
      col[c].l[n] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) col[c].o[i][0] = col[c].o[i][1] = col[c].o[i][2] = col[c].o[i][3] = 0.f;
  }

  // ---- one stage of 32 tokens -----------------------------------------------------------------
  const auto process = [&](int k) {
    const uint8_t* st = ring + (k % kFewStages) * kStageBytes;
    const int r = lane >> 2, c4 = lane & 3, t0 = first_token(k);
    if (t0 + kStepTok > seq.ctx) {
      // codes past the context may be any bytes, NaN among them: 0 * NaN would poison a sum
      for (int i = lane; i < (t0 + kStepTok - max(seq.ctx, t0)) * 8; i += 32)
        st_shared_zero16(smem_u32(st) + kHalfStage + (max(seq.ctx, t0) - t0) * kHeadDim + i * 16);
      fence_proxy_async_smem();
      __syncwarp();
    }
    // scales of the lane's tokens r, r + 8 of either half: a box never ends inside 8 tokens
    BlockScale bs[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int src = (k % kBatch) * kBoxes + 8 * e * kBoxes / kStepTok;
      bs[e].k = __shfl_sync(kFull, sc.k, src);
      bs[e].v = __shfl_sync(kFull, sc.v, src);
      bs[e].inv = __shfl_sync(kFull, sc.inv, src);
    }
    float x[GROUPS][2][4];   // [16-token half][token r columns 0, 1, token r + 8 columns 0, 1]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < GROUPS; ++c) x[c][h][0] = x[c][h][1] = x[c][h][2] = x[c][h][3] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 w0 = chunk_of(st, 16 * h + r, 2 * c4 + i);
        const uint4 w1 = chunk_of(st, 16 * h + r + 8, 2 * c4 + i);
        const uint32_t u0[4] = {w0.x, w0.y, w0.z, w0.w}, u1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint2 a = Wide::four(u0[j]), b = Wide::four(u1[j]);
#pragma unroll
          for (int c = 0; c < GROUPS; ++c) mma_16816(x[c][h], a.x, b.x, a.y, b.y, qb[c][4 * i + j]);
        }
      }
#pragma unroll
      for (int c = 0; c < GROUPS; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[c][h][e] = fmaf(x[c][h][e], bs[2 * h + (e >> 1)].k, bs[2 * h + (e >> 1)].v);
    }
    if (t0 + kStepTok > min(pos0 + 1, end)) {   // some column does not see all of it
#pragma unroll
      for (int c = 0; c < GROUPS; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = t0 + 16 * h + r + 8 * (e >> 1);
            const int last = pos0 + ((8 * c + 2 * c4 + (e & 1)) >> shift);
            if (t > last || t >= end) x[c][h][e] = -INFINITY;
          }
    }
    uint32_t pb[GROUPS][2][2];
#pragma unroll
    for (int c = 0; c < GROUPS; ++c) {
      Column8& a = col[c];
      float top[2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
        top[n] = fmaxf(fmaxf(x[c][0][n], x[c][0][2 + n]), fmaxf(x[c][1][n], x[c][1][2 + n]));
      // the maxima move only when a token passes one by more than 2^8
      const bool moves = top[0] > a.m[0] + (kHeadroom + kRescale) ||
                         top[1] > a.m[1] + (kHeadroom + kRescale);
      if (__any_sync(kFull, moves)) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top[n] = fmaxf(top[n], __shfl_xor_sync(kFull, top[n], o));
          if (top[n] > a.m[n] + (kHeadroom + kRescale)) {
            const float unit = top[n] - kHeadroom, alpha = exp2_approx(a.m[n] - unit);
            a.l[n] *= alpha;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              a.o[i][n] *= alpha;
              a.o[i][2 + n] *= alpha;
            }
            a.m[n] = unit;
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = exp2_approx(x[c][h][e] - a.m[e & 1]);
          a.l[e & 1] = fmaf(w[e], bs[2 * h + (e >> 1)].inv, a.l[e & 1]);
        }
        pb[c][h][0] = transpose8(pack_half2(w[0], w[1]));
        pb[c][h][1] = transpose8(pack_half2(w[2], w[3]));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t t[4][4];   // tokens 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9 of the half, 16 dims each
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = chunk_of(st + kHalfStage, 16 * h + 2 * c4 + (i & 1) + 8 * (i >> 1), r);
        t[i][0] = w.x;
        t[i][1] = w.y;
        t[i][2] = w.z;
        t[i][3] = w.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const uint32_t sel = d ? 0x7362 : 0x5140;
          const uint2 a = Wide::four(__byte_perm(t[0][j], t[1][j], sel));
          const uint2 b = Wide::four(__byte_perm(t[2][j], t[3][j], sel));
#pragma unroll
          for (int c = 0; c < GROUPS; ++c)
            mma_16816(col[c].o[2 * j + d], a.x, a.y, b.x, b.y, pb[c][h]);
        }
    }
  };

  const auto landed = [&](int k) {
    return warp_wait(&bars[k % kFewStages], (k / kFewStages) & 1, p.dev_err);
  };
  bool ok = true;
  int k = 0;
#pragma unroll 1
  for (; k < issued; ++k) {
    if (k % kBatch == 0) sc = block_scale(loaded.x, loaded.y, p.scale_log2);
    ok = landed(k);
    if (!ok) break;
    process(k);
    fence_proxy_async_smem();   // the stage is read before the copy engine writes it again
    __syncwarp();
    if (issued < mine) {
      issue(issued);
      ++issued;
    }
  }
  // after a wait that gave up its copies and those behind them are still on their way into the
  // ring: they get a bounded wait each before the shared memory goes to another CTA
  for (; !ok && k < issued; ++k) landed(k);
  // after a wait that gave up: no merge (it reuses the rings), no store
  if (__syncthreads_or(!ok)) return;

  // ---- the warps' results, joined -----------------------------------------------------------
  float2* ml = reinterpret_cast<float2*>(smem + Smem::ml);
  float* ob = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int c = 0; c < GROUPS; ++c)
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float l = col[c].l[n];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(kFull, l, o);
      const int at = warp * kCols + 8 * c + 2 * (lane & 3) + n;
      if (lane < 4) ml[at] = make_float2(col[c].m[n], l);
      float* row = ob + at * kHeadDim + 16 * (lane >> 2);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float2*>(row + 2 * i) = make_float2(col[c].o[i][n], col[c].o[i][2 + n]);
    }
  __syncthreads();
#pragma unroll 1
  for (int n = warp; n < toks << shift; n += kWarps) {
    const int tok = n >> shift, pos = pos0 + tok;
    // rows whose tokens one unit covers are written, others leave a partial
    const bool whole = pos / kTile < p.split_tiles;
    if (whole ? blockIdx.y > 0 : pos < first) continue;
    float M = ml[n].x;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, ml[w * kCols + n].x);
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 e = ml[w * kCols + n];
      const float4 v = *reinterpret_cast<const float4*>(ob + (w * kCols + n) * kHeadDim + 4 * lane);
      const float f = exp2_approx(e.x - M);
      num.x += f * v.x;
      num.y += f * v.y;
      num.z += f * v.z;
      num.w += f * v.w;
      den += f * e.y;
    }
    const int64_t row = (static_cast<int64_t>(seq.row0) + tok0 + tok) * p.num_q_heads +
                        (g << shift) + (n & ((1 << shift) - 1));
    if (whole) {
      const float inv = 1.f / den;   // a sum of 0 (all scores -inf): the definition's NaN
      *reinterpret_cast<uint2*>(p.out + row * kHeadDim + 4 * lane) =
          make_uint2(pack_half2(num.x * inv, num.y * inv), pack_half2(num.z * inv, num.w * inv));
    } else {
      const int64_t at = row * p.splits + blockIdx.y;
      *reinterpret_cast<float4*>(p.part_o + at * kHeadDim + 4 * lane) = num;
      if (lane == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(M, den);
    }
  }
}

// codes [rows, heads, 128 bytes], a box is min(BS, 32) rows of a head
bool make_few_map(CUtensorMap* map, const void* base, int heads, int64_t rows, int block_size) {
  auto fn = attn::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {kHeadDim, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {kHeadDim, static_cast<cuuint64_t>(heads) * kHeadDim};
  cuuint32_t box[3] = {kHeadDim, 1, static_cast<cuuint32_t>(std::min(block_size, kStepTok))};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Wide, int BS, int GROUPS>
int launch(const CUtensorMap& mk, const CUtensorMap& mv, const Q8Params& qp, dim3 grid,
           cudaStream_t st) {
  static std::atomic<uint8_t> opted_in[64];
  constexpr int kAlloc = FewSmem<8 * GROUPS>::alloc;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  if (dev < 0 || dev >= 64 || !opted_in[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(few_rows_q8_kernel<Wide, BS, GROUPS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kAlloc) != cudaSuccess)
      return PKV_ERR_CUDA;
    if (dev >= 0 && dev < 64) opted_in[dev].store(1, std::memory_order_release);
  }
  return launch_dependent(few_rows_q8_kernel<Wide, BS, GROUPS>, grid, kFewThreads, kAlloc, st, mk,
                          mv, qp);
}

template <class Wide, int GROUPS>
int launch_any(int block_size, const CUtensorMap& mk, const CUtensorMap& mv, const Q8Params& qp,
               dim3 grid, cudaStream_t st) {
  switch (block_size) {
    case 8: return launch<Wide, 8, GROUPS>(mk, mv, qp, grid, st);
    case 16: return launch<Wide, 16, GROUPS>(mk, mv, qp, grid, st);
    case 32: return launch<Wide, 32, GROUPS>(mk, mv, qp, grid, st);
    default: return launch<Wide, 64, GROUPS>(mk, mv, qp, grid, st);
  }
}

}  // namespace

Plan few_rows_plan(int num_tokens, int num_seqs, int num_kv_heads, int group_shift,
                   int64_t max_context) {
  Plan plan = {};
  const int64_t rows = static_cast<int64_t>(num_tokens) << group_shift;
  plan.columns = rows <= 8ll * num_seqs ? 8 : 16;
  const int per = plan.columns >> group_shift;
  plan.units = num_tokens / per + static_cast<int64_t>(num_seqs);
  // Splits: one round of CTAs where the units leave places, else two rounds and more (three
  // or more are no faster), of at least 512 tokens each.
  const int64_t places = kSms * kFewCtas;
  const int64_t ctas = std::max<int64_t>(num_seqs, num_tokens / per) * num_kv_heads;
  const int64_t tiles = (max_context + kTile - 1) / kTile;
  const int64_t fill = 2 * ctas <= places ? places / ctas : (2 * places + ctas - 1) / ctas;
  const int64_t want = std::min(fill, std::max<int64_t>(1, tiles / 4));
  const int64_t each = (tiles + want - 1) / want;
  plan.split_tiles = static_cast<int>(each);
  plan.splits = static_cast<int>((tiles + each - 1) / each);
  return plan;
}

int launch_few_rows(const Q8Params& qp, const Plan& plan, int code, int block_size,
                    const void* k_cache, const void* v_cache, cudaStream_t st) {
  CUtensorMap mk, mv;
  const int64_t rows = qp.p.num_blocks * block_size;
  if (!make_few_map(&mk, k_cache, qp.p.num_kv_heads, rows, block_size) ||
      !make_few_map(&mv, v_cache, qp.p.num_kv_heads, rows, block_size))
    return PKV_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>(plan.units * qp.p.num_kv_heads), plan.splits);
  const auto go = [&](auto wide) {
    using Wide = decltype(wide);
    return plan.columns == 8 ? launch_any<Wide, 1>(block_size, mk, mv, qp, grid, st)
                             : launch_any<Wide, 2>(block_size, mk, mv, qp, grid, st);
  };
  return code == PKV_CODE_INT8 ? go(Int8Wide()) : go(E4m3Wide());
}

}  // namespace prompt_q8
}  // namespace pkv
