// Causal attention of whole prompts and prompt chunks (sm_103a, tcgen05).
//
// For packed row i of sequence s (position pos, query head h, KV head g):
//   out[i, h] = sum_{t <= pos} softmax_t(scale <q[i, h], K[t, g]>) V[t, g]
// with K and V either in the paged fp16 cache (context_lens[s] tokens, the
// packed rows the last of them) or packed like q.
//
// How:
//  * A unit of work is 256 rows of one KV head: 256 / group tokens with the
//    group's query heads side by side, so that grouped heads share every K and V
//    tile and the tiles along the diagonal are short.  Two query tiles of 128
//    rows take turns: while one's 128 x 128 products run on the tensor core the
//    other's softmax runs on the CUDA cores.
//  * S = Q K^T (operands in shared memory) and O += P V (P in tensor memory, over
//    the scores it came from) accumulate in fp32 in tensor memory: 2 x 128 columns
//    of scores and 2 x 128 of outputs, all 512.
//  * One softmax thread owns a row of scores.  Its running maximum moves only when
//    a score passes it by more than 2^8, so O is rescaled in few tiles.  The weights
//    are rounded to fp16 for the product with V, by half a step, 2^-11, or by 2^-32 of
//    the largest (see kHeadroom).  Their sum is fp32 and takes them unrounded: the
//    rounded ones would have to be widened again, 64 conversions more a thread and tile,
//    and would spare only a row that one token dominates, which is now off by 2^-11.
//  * K and V come through a ring of four 32 KB tiles, by TMA: a box for each block
//    (paged) or for 128 tokens (packed).
//  * What bounds it: in steady state a turn (128 tokens for 256 rows) takes 2300
//    cycles, of which the tensor core is busy 2048; a unit adds some 4000 at its
//    ends.  16,384 tokens of 32/8 heads: 1180-1310 us in short runs, 1.68-1.86 PFLOP/s
//    (the measured cuBLAS burst is 1.96), 1370-1460 us in loops of seconds, where the
//    chip is at its power limit; 4 x 4096 of 32 heads: 345-371 us, 1.48-1.59, and 402-405.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "q8_device.cuh"

namespace pkv {
namespace attn {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
}
namespace prompt {

constexpr int kHeadDim = 128;
constexpr int kTile = 128;                       // rows of a query tile, tokens of a KV tile
constexpr int kHalfBytes = kTile * 128;          // 128 rows x 64 dims, 128-byte swizzle
constexpr int kTileBytes = 2 * kHalfBytes;
constexpr int kStages = 4;                       // KV tiles in shared memory
constexpr int kThreads = 384;                    // 2 softmax warpgroups; 2 copy, MMA and work warps
// Registers a thread after the split: 256 * 224 + 128 * 56 = 384 * 168, what the
// CTA was launched with (a softmax thread holds a row of 128 scores).
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 224, kOtherRegs = 56;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");
constexpr int kCopyWarp = 8, kMmaWarp = 9, kWorkWarp = 10, kCopyVWarp = 11;
constexpr int kReaders = 11;                     // warps that read a unit's description
constexpr float kRescale = 8.f;                  // log2 units
// The weights' unit is 2^-7 of the running maximum, so that they fill fp16's range: at most
// 2^(7 + kRescale), and what rounds to 0 is below 2^-32 of the maximum.  With the maximum
// itself for a unit, 65,536 tokens 25 to 29 log2 units below one lost all their share of
// the output, 2^-10, which their sum kept.
constexpr float kHeadroom = 7.f;
static_assert(kHeadroom + kRescale <= 15.f, "weights in fp16's range");
constexpr float kNoMax = -1e30f;
constexpr uint32_t kWaitLimit = 1u << 31;        // cycles a wait may take, a second: some wait
                                                 // for a whole unit (see kMaxContext)

struct Smem {
  static constexpr int q = 0;                            // two query tiles
  static constexpr int kv = q + 2 * kTileBytes;
  static constexpr int stage = kv + kStages * kTileBytes;  // output rows, 4 KB a softmax warp
  static constexpr int lm = stage + 8 * 4096;            // float2 [128]: sums and maxima of a
                                                         // row that both warpgroups work on
  static constexpr int bars = lm + kTile * 8;
  static constexpr int q_full = bars;                    // [2]
  static constexpr int q_empty = q_full + 16;            // [2] the tile's last score product is done
  static constexpr int kv_full = q_empty + 16;           // [kStages]
  static constexpr int kv_empty = kv_full + 8 * kStages; // [kStages]
  static constexpr int s_full = kv_empty + 8 * kStages;  // [2] scores of a tile are in TMEM
  static constexpr int p_full = s_full + 16;             // [2][2] a half's weights are in TMEM
  static constexpr int o_full = p_full + 32;             // [2] the tile's output is complete
  static constexpr int lm_full = o_full + 16;            // lm is written
  static constexpr int lm_free = lm_full + 8;            // and read, tile 1's output too
  static constexpr int raw = lm_free + 8;                // a V tile to be cleaned has landed
  static constexpr int unit_full = raw + 8;              // the next unit is described
  static constexpr int unit_empty = unit_full + 8;       // and every warp has read it
  static constexpr int stolen = unit_empty + 8;          // the scheduler's answer is there
  static constexpr int drained = stolen + 8;
  static constexpr int answer = (drained + 16 + 15) / 16 * 16;
  static constexpr int unit = answer + 16;
  static constexpr int tmem = unit + 64;
  static constexpr int gave_up = tmem + 4;               // a wait did
  static constexpr int nonfinite = tmem + 8;             // [2] the last odd and even unit in whose
                                                         // V some values were set to zero
  static constexpr int total = tmem + 16;
  static constexpr int alloc = total + 1024;
  static_assert(alloc <= 227 * 1024, "shared memory of one CTA");
};

// A KV tile in shared memory is made of 1 KB atoms of 8 tokens x 64 dims (128-byte
// swizzle).  Paged: the atoms of both halves of the dims lie side by side, 8 tokens
// after 8 tokens, so that one box brings a whole block (half the boxes, whose number
// bounds the copies of 16-token blocks).  Packed: one half, then the other, as two
// boxes of 128 tokens (packed rows start anywhere, not at multiples of 8).
template <int BS>
struct KvLayout {
  static constexpr uint32_t kHalf = BS ? 1024 : kHalfBytes;   // to the other half of the dims
  static constexpr uint32_t kEight = BS ? 2048 : 1024;        // to the next 8 tokens
};

// TMEM columns: scores (overwritten by the fp16 weights) and outputs of the two tiles
constexpr uint32_t kColS = 0, kColO = 256;

struct Params {
  __half* out;
  const __half* v;
  const int32_t* query_start;
  const int32_t* context_lens;   // nullptr: K and V are packed like q
  const int32_t* block_tables;
  float* part_o;                 // [rows, splits, 128]
  float* part_ml;                // [rows, splits, 2]
  int32_t* dev_err;
  int64_t num_blocks;
  int num_tokens, num_seqs, num_q_heads, num_kv_heads, max_blocks;
  int group_shift;               // log2(num_q_heads / num_kv_heads)
  int split_tiles;               // KV tiles a unit covers at most
  int splits;
  float scale_log2;              // |scale| log2 e
  uint32_t idesc_qk;
};

// ---- tcgen05 ------------------------------------------------------------------------
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11,"
      " %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29,"
      " %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10,"
      " %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28,"
      " %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(void* smem_dst, const void* tmap, int c0, int c1, int c2,
                                            int c3, int c4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4),
      "r"(smem_u32(bar))
      : "memory");
}

// store a box from shared memory; the buffer may be written again after bulk_wait_read()
__device__ __forceinline__ void tma_store_3d(const void* tmap, const void* smem_src, int c0, int c1,
                                             int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(smem_u32(smem_src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 w;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "r"(addr)
               : "memory");
  return w;
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w.x), "r"(w.y), "r"(w.z),
               "r"(w.w)
               : "memory");
}
__device__ __forceinline__ __half2 u32_as_half2(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }
__device__ __forceinline__ uint32_t half2_as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Shared-memory operand descriptor, 128-byte swizzle.  K-major (Q, K): rows of
// 128 bytes, 8-row groups `stride` apart.  MN-major (V): 64-dim chunks
// `lead` apart, 8-token groups `stride` apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | static_cast<uint64_t>(lead >> 4) << 16 |
         static_cast<uint64_t>(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

constexpr uint32_t kIdescBase = 1u << 4                       // fp32 accumulators, fp16 operands
                                | (kTile / 8) << 17 | (kTile / 16) << 24;
constexpr uint32_t kIdescPv = kIdescBase | 1u << 16;          // V is MN-major
constexpr uint32_t kNegateA = 1u << 13;

// A piece of work: two query tiles of 128 rows of one KV head, row r of a tile
// being token r / group, query head g * group + r % group, and the KV tiles
// [begin, end) each attends to, taken from the last to the first: the masked
// tiles come while the last unit's output is still being written, and both
// query tiles end together.  Tile 0 holds the later tokens (its longer stretch
// starts first).
// A unit with rows in one tile only (a short chunk, the rest of a prompt) is a
// pair: both warpgroups work on tile 0's rows, on every other KV tile each, and
// the first joins the two results.  Alone a tile waits for its own products and
// weights in turn, 3100 cycles a KV tile; a pair takes 1200 to 2000 (copies of
// 16-token blocks).
struct alignas(16) Unit {
  int row0, n, ctx, s;   // the sequence (see PackedSeq) and its index
  int g, split;
  int tok0[2];           // first token of each tile (among the sequence's packed rows)
  int end[2];
  int begin, last;       // KV tiles of the unit; last == begin: no more work
  int pair;
  __device__ __forceinline__ bool has(int x) const { return pair || end[x] > begin; }
};
static_assert(sizeof(Unit) <= 64 && sizeof(Unit) % 16 == 0, "a unit's place in shared memory");

__device__ __forceinline__ bool make_unit(const Params& p, int bx, int by, int64_t max_context,
                                          Unit& u) {
  const int per = 2 * kTile >> p.group_shift;   // tokens of a unit
  const int units = gridDim.x / p.num_kv_heads;
  // later rows of a prompt see more tokens: start with them
  const int unit = units - 1 - bx / p.num_kv_heads;
  u.g = bx % p.num_kv_heads;
  u.split = by;
  u.s = find_unit_seq(p.query_start, p.num_seqs, unit, per, 1);
  const PackedSeq q = packed_seq(p.query_start, p.context_lens, u.s, p.num_tokens, max_context,
                                 p.dev_err, false);
  u.row0 = q.row0;
  u.n = q.n;
  u.ctx = q.ctx;
  const int nth = unit - unit_base(p.query_start, u.s, per, 1);
  u.begin = u.last = by * p.split_tiles;
  if (!q.ok || nth < 0 || static_cast<int64_t>(nth) * per >= q.n) return false;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    u.tok0[x] = nth * per + (1 - x) * (kTile >> p.group_shift);
    const int tok_end = min(q.n, u.tok0[x] + (kTile >> p.group_shift));
    u.end[x] = u.begin;
    if (tok_end > u.tok0[x]) {
      const int last_pos = q.ctx - q.n + tok_end - 1;
      u.end[x] = max(u.begin, min(u.begin + p.split_tiles, last_pos / kTile + 1));
    }
    u.last = max(u.last, u.end[x]);
  }
  u.pair = (u.end[0] == u.begin || u.end[1] == u.begin) && u.last - u.begin >= 2;
  if (u.pair) {
    u.tok0[0] = u.tok0[1] = u.end[0] > u.begin ? u.tok0[0] : u.tok0[1];
    u.end[0] = u.last;
    u.end[1] = u.begin;
  }
  return u.last > u.begin;
}

// Tokens of a KV tile that some row of the unit does not see have a weight of 0
// there, and 0 * NaN must not reach a sum.  So before the product their V is made
// finite in shared memory: tokens that no row of the unit sees, those past the
// context among them (whatever the copy brings there; a paged block wholly past
// the context is read from past the cache's last row, where the copy engine fills
// zeros), become zeros; the others are searched for infinities and NaN, which
// become zeros too and are added to the rows that see them at the end (add_nonfinite).
// The search costs 1 % (in one run, 4 x 4096 of 32 heads 356 us, 351 without; 16 x 512 of
// 32/8 47.2 and 45.9).  The warp that copies V does it: in the work warp, which has the time,
// 64 prompts of 128 take 40.6 us instead of 36.6; one tile late, under the next
// copy, 4 x 4096 takes 361.
template <int BS>
struct Masked {
  int seen, unseen, end;   // tokens of the tile: [seen, unseen) by some rows, [unseen, end) by none
  __device__ __forceinline__ Masked(const Unit& u, int group_shift, int j) {
    const int at = u.ctx - u.n - j * kTile;   // the first packed row's place in the tile
    unseen = min(kTile, at + min(u.n, u.tok0[0] + (kTile >> group_shift)));
    seen = min(unseen, max(0, at + (j < u.end[1] ? u.tok0[1] : u.tok0[0]) + 1));
    const int valid = u.ctx - j * kTile;
    end = BS ? min(kTile, (valid + BS - 1) / (BS ? BS : 1) * BS) : kTile;
  }
  __device__ __forceinline__ bool any() const { return seen < end; }
};

// infinities and NaN of a pair become zeros
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  if ((w & 0x7c00u) == 0x7c00u) w &= 0xffff0000u;
  if ((w & 0x7c000000u) == 0x7c000000u) w &= 0x0000ffffu;
  return w;
}

// The infinities and NaN that Masked took out of the unit's V are added to the output in
// tensor memory (a whole warp, a row each lane): the row that sees a token has a positive
// weight for it.  Seldom run, so it is short and reads V again, token after token.
template <int BS>
__device__ __forceinline__ void add_nonfinite(const Params& p, const Unit& u, uint32_t o_at, int pos,
                                           int end) {
  const int per = kTile >> p.group_shift;
  const int from = max(u.begin * kTile, u.ctx - u.n + u.tok0[1] + 1);
  const int to = min(end * kTile, u.ctx - u.n + min(u.n, u.tok0[0] + per));
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t o[32];
    tmem_ld32(o_at + 32 * c, o);
    wait_ld();
#pragma unroll 1
    for (int t = from; t < to; ++t) {
      int64_t row = static_cast<int64_t>(u.row0) + t;
      if (BS) {
        const int32_t id = __ldg(p.block_tables + static_cast<int64_t>(u.s) * p.max_blocks +
                                 t / (BS ? BS : 1));
        if (id < 0 || id >= p.num_blocks) continue;   // read as zeros
        row = static_cast<int64_t>(id) * BS + t % (BS ? BS : 1);
      }
      const uint4* v = reinterpret_cast<const uint4*>(
          p.v + (row * p.num_kv_heads + u.g) * kHeadDim + 32 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w4 = __ldg(v + i);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t rest = w[e] ^ finite2(w[e]);   // the bits that were taken out
          const float2 f = half2_to_float2(rest);
          if (t <= pos) {
            o[8 * i + 2 * e] = __float_as_uint(__uint_as_float(o[8 * i + 2 * e]) + f.x);
            o[8 * i + 2 * e + 1] = __float_as_uint(__uint_as_float(o[8 * i + 2 * e + 1]) + f.y);
          }
        }
      }
    }
    tmem_st32(o_at + 32 * c, o);
  }
  wait_st();
}

// BS: block size of the paged cache, 0 for packed K and V.
//
// One CTA per SM.  Its warps: two softmax warpgroups (one per query tile, one
// thread per row), two copy warps (TMA; Q and K, and V), a warp that issues the matrix
// products and one that fetches work: the grid has a CTA for every unit, and a CTA that
// runs takes the place of CTAs that have not started (clusterlaunchcontrol), so
// that the next unit's copies and first products run beside the last
// unit's softmax and output, and units of any length balance themselves.
template <int BS>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tmap_q,
                            const __grid_constant__ CUtensorMap tmap_k,
                            const __grid_constant__ CUtensorMap tmap_v,
                            const __grid_constant__ CUtensorMap tmap_o, const Params p) {
  using Kv = KvLayout<BS>;
  constexpr unsigned kFull = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  // the same in every lane, which the compiler learns from the shuffle
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int64_t max_context = BS ? static_cast<int64_t>(p.max_blocks) * BS : INT32_MAX;
  const auto bar = [&](int at, int i) { return reinterpret_cast<uint64_t*>(smem + at) + i; };
  volatile uint32_t* gave_up = reinterpret_cast<volatile uint32_t*>(smem + Smem::gave_up);
  volatile int* nonfinite = reinterpret_cast<volatile int*>(smem + Smem::nonfinite);
  const auto wait = [&](uint64_t* b, uint32_t parity) {
    return flag_wait(b, parity, gave_up, kWaitLimit);
  };
  if (warp == kCopyWarp && lane == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Smem::q_full, i), 1);
      mbar_init(bar(Smem::q_empty, i), 1);
      mbar_init(bar(Smem::s_full, i), 1);
      mbar_init(bar(Smem::p_full, 2 * i), 4);
      mbar_init(bar(Smem::p_full, 2 * i + 1), 4);
      mbar_init(bar(Smem::o_full, i), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(Smem::kv_full, i), 1);
      mbar_init(bar(Smem::kv_empty, i), 1);
    }
    mbar_init(bar(Smem::lm_full, 0), 4);
    mbar_init(bar(Smem::lm_free, 0), 4);
    mbar_init(bar(Smem::raw, 0), 1);
    mbar_init(bar(Smem::unit_full, 0), 1);
    mbar_init(bar(Smem::unit_empty, 0), kReaders);
    mbar_init(bar(Smem::stolen, 0), 1);
    mbar_init(bar(Smem::drained, 0), 1);
    *gave_up = 0;
    nonfinite[0] = nonfinite[1] = -1;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(smem + Smem::tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // launched as a programmatic dependent of the stream's previous kernel: nothing is
  // read before this wait, which returns once that kernel's writes are visible
  asm volatile("griddepcontrol.wait;" ::: "memory");
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Smem::tmem);

  // the k-th unit, read by a whole warp; false: no more work, or a wait gave up
  const auto next_unit = [&](int k, Unit& u) {
    if (!wait(bar(Smem::unit_full, 0), k & 1)) return false;
    u = *reinterpret_cast<const Unit*>(smem + Smem::unit);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(Smem::unit_empty, 0));
    return u.last > u.begin;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kCopyWarp || warp == kCopyVWarp) {
      // ---- copies: K and V of each tile through a ring of kStages -----------------------------
      // One warp brings Q and K, one V: both count through the whole sequence.  A warp starts
      // a box of 16 rows every 73 cycles.
      const int mine = warp == kCopyVWarp;
      constexpr int kBoxes = BS ? kTile / (BS ? BS : 1) : 1;
      static_assert((kStages & (kStages - 1)) == 0, "ring positions by shifts");
      int base = 0, nraw = 0;                 // the unit's first place in the ring, cleaned tiles
      int raw_st = -1;                        // the stage of a tile that is to be cleaned
      uint32_t q_seen = 0, q_parity = 0;      // bit x: Q copies of tile x so far
      uint32_t kv_seen = 0, kv_parity = 0;    // bit st: this warp's copies into a stage
      bool ok = true;
      Unit u;
      for (int k = 0; ok && next_unit(k, u); ++k) {
        const int n = u.last - u.begin;
        // the block id of this lane's part of tile j (paged): loaded a tile ahead
        const auto id_of = [&](int j) {
          const int tok = j * kTile + lane * BS;
          return BS && lane < kBoxes && j >= u.begin && tok < u.ctx
                     ? __ldg(p.block_tables + static_cast<int64_t>(u.s) * p.max_blocks +
                             tok / (BS ? BS : 1))
                     : -1;
        };
        int32_t id = id_of(u.last - 1);
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
          const int j = u.last - 1 - i;
          const int32_t next_id = id_of(j - 1);
          // where the tile's K or V comes in the ring: V after its K, in a pair after the
          // next tile's K
          const int at = !u.pair ? 2 * i + mine
                         : mine  ? (i + 1 < n ? 2 * i + 2 : 2 * n - 1)
                                 : max(0, 2 * i - 1);
          const int st = (base + at) & (kStages - 1), round = (base + at) / kStages;
          int row = u.row0 + j * kTile;
          if (BS) {
            row = static_cast<int>(p.num_blocks * BS);   // past the last row: zeros
            if (id >= 0 && id < p.num_blocks)
              row = id * BS;
            else if (lane < kBoxes && j * kTile + lane * BS < u.ctx)
              report(p.dev_err, PKV_DEV_BAD_BLOCK_ID);
          }
          id = next_id;
          if (round > 0) ok = wait(bar(Smem::kv_empty, st), (round - 1) & 1);
          if (!ok) break;
          kv_seen |= 1u << st;
          kv_parity = (kv_parity & ~(1u << st)) | (round & 1) << st;
          const Masked<BS> masked(u, p.group_shift, j);
          const bool raw = mine && masked.any();
          uint64_t* b = raw ? bar(Smem::raw, 0) : bar(Smem::kv_full, st);
          uint8_t* dst = smem + Smem::kv + st * kTileBytes;
          if (raw) raw_st = st;
          if (lane == 0) mbar_arrive_expect_tx(b, kTileBytes);
          __syncwarp();
          if (lane < kBoxes) {
            const CUtensorMap* m = mine ? &tmap_v : &tmap_k;
            if (BS) {
              tma_load_5d(dst + lane * (kTileBytes / kBoxes), m, 0, 0, 0, row >> 3, u.g, b);
            } else {
              tma_load_3d(dst, m, 0, u.g, row, b);
              tma_load_3d(dst + kHalfBytes, m, 64, u.g, row, b);
            }
          }
          if (raw) {   // the tile may be used once its masked tokens are finite
            ok = wait(b, nraw & 1);
            if (!ok) break;
            ++nraw;
            const uint32_t to = smem_u32(dst);
            const auto chunk = [&](int c) {   // 16 bytes: token c / 16, dims 8 (c % 16)
              const int r = c >> 4;
              return to + (c & 8 ? Kv::kHalf : 0) + (r >> 3) * Kv::kEight + (r & 7) * 128 +
                     (c & 7) * 16;
            };
            // 0 * x adds a zero, and for an infinity or NaN a NaN
            const __half2 zero = __floats2half2_rn(0.f, 0.f);
            __half2 acc[4] = {zero, zero, zero, zero};
#pragma unroll 4
            for (int c = masked.seen * 16 + lane; c < masked.unseen * 16; c += 32) {
              const uint4 w = ld_shared16(chunk(c));
              acc[0] = __hfma2(u32_as_half2(w.x), zero, acc[0]);
              acc[1] = __hfma2(u32_as_half2(w.y), zero, acc[1]);
              acc[2] = __hfma2(u32_as_half2(w.z), zero, acc[2]);
              acc[3] = __hfma2(u32_as_half2(w.w), zero, acc[3]);
            }
            if (__any_sync(kFull, half2_as_u32(acc[0]) | half2_as_u32(acc[1]) | half2_as_u32(acc[2]) |
                                      half2_as_u32(acc[3]))) {
#pragma unroll 1
              for (int c = masked.seen * 16 + lane; c < masked.unseen * 16; c += 32) {
                const uint4 w = ld_shared16(chunk(c));
                st_shared16(chunk(c), make_uint4(finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w)));
              }
              if (lane == 0) nonfinite[k & 1] = k;
            }
            for (int c = masked.unseen * 16 + lane; c < masked.end * 16; c += 32)
              st_shared_zero16(chunk(c));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(Smem::kv_full, st));
            raw_st = -1;
          }
          if (i == 0 && !mine) {
#pragma unroll 1
            for (int x = 0; x < 2 && ok; ++x) {
              if ((x ? u.end[1] : u.end[0]) == u.begin) continue;
              if (q_seen >> x & 1)
                ok = wait(bar(Smem::q_empty, x), (q_parity >> x & 1) ^ 1);
              if (!ok) break;
              q_seen |= 1u << x;
              q_parity ^= 1u << x;
              if (lane == 0) {
                uint64_t* qb = bar(Smem::q_full, x);
                uint8_t* to = smem + Smem::q + x * kTileBytes;
                mbar_arrive_expect_tx(qb, kTileBytes);
                for (int h = 0; h < 2; ++h)
                  tma_load_3d(to + h * kHalfBytes, &tmap_q, 64 * h, u.g << p.group_shift,
                              u.row0 + (x ? u.tok0[1] : u.tok0[0]), qb);
              }
            }
          }
        }
        base += 2 * n;
      }
      // a wait gave up: let this warp's copies land before the CTA goes (that of a tile to be
      // cleaned counts on a barrier of its own)
      if (__any_sync(kFull, *gave_up)) {
        if (raw_st >= 0) wait(bar(Smem::raw, 0), nraw & 1);
#pragma unroll 1
        for (int i = 0; i < kStages; ++i)
          if ((kv_seen >> i & 1) && i != raw_st) wait(bar(Smem::kv_full, i), kv_parity >> i & 1);
#pragma unroll 1
        for (int x = 0; x < 2; ++x)
          if (q_seen >> x & 1) wait(bar(Smem::q_full, x), (q_parity >> x & 1) ^ 1);
      }
    } else if (warp == kMmaWarp) {
      // ---- matrix products: the warp runs together, one elected lane issues ------------------
      // (operands stay in uniform registers that way; a loop of one diverged lane took 85
      // cycles to issue a product that runs for 64).  The tensor core holds some 7 products
      // in its queue, and a wait takes 30 cycles even when what it waits for is there: the
      // waits for K and V are kept out of the stretch between one tile's products and the
      // other's weights.  One warp issues for both tiles, a whole batch at a time: with a
      // warp for each their products alternate, end together and the tiles fall into step
      // (3400 cycles a pair of tiles instead of 2800).
      struct Ring {
        int st;
        uint32_t round;
        __device__ __forceinline__ Ring after() const {
          return st + 1 == kStages ? Ring{0, round + 1} : Ring{st + 1, round};
        }
      };
      const uint32_t s_col = tmem + kColS, o_col = tmem + kColO;
      const uint64_t q_desc = operand_desc(smem_u32(smem + Smem::q), 16, 1024);
      const uint64_t k_desc = operand_desc(smem_u32(smem + Smem::kv), 16, Kv::kEight);
      const uint64_t v_desc = operand_desc(smem_u32(smem + Smem::kv), Kv::kHalf, Kv::kEight);
      const auto full = [&](Ring r) { return wait(bar(Smem::kv_full, r.st), r.round & 1); };
      const auto commit = [&](uint64_t* b) {
        if (elect_one()) mma_commit(b);
        __syncwarp();
      };
      // O_x += P_x V over the first (h0) and last 64 tokens, S_x = Q_x K^T
      const auto pv4 = [&](int x, int half, uint64_t vd, bool acc) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kk = 4 * half + i;
          mma_ts(o_col + x * kTile, s_col + x * kTile + 8 * kk, vd + kk * (2 * Kv::kEight >> 4),
                 kIdescPv, acc || i > 0);
        }
      };
      const auto qk8 = [&](int x, uint64_t qd, uint64_t kd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t step = (i & 3) * 32;
          mma_ss(s_col + x * kTile, qd + (((i >> 2) * kHalfBytes + step) >> 4),
                 kd + (((i >> 2) * Kv::kHalf + step) >> 4), p.idesc_qk, i > 0);
        }
        mma_commit(bar(Smem::s_full, x));
      };
      const auto k_at = [&](Ring r) { return k_desc + r.st * (kTileBytes >> 4); };
      const auto v_at = [&](Ring r) { return v_desc + r.st * (kTileBytes >> 4); };
      Ring ring = {0, 0};             // of the next tile to take
      uint32_t q_parity = 0, p_parity = 0;   // bit x: of tile x's next query tile, weights
      bool ok = true;
      Unit u;
      for (int k = 0; ok && next_unit(k, u); ++k) {
        if (u.pair) {
          const int n = u.last - u.begin;
          ok = wait(bar(Smem::q_full, 0), q_parity & 1);
          q_parity ^= 1u;
#pragma unroll 1
          for (int i = -2; i < n && ok; ++i) {   // tile i's weights, tile i + 2's scores
            const int x = i & 1;
            const bool more = i + 2 < n;
            const Ring rv = ring, rk = i < 0 ? ring : ring.after();
            if (i >= 0) {
              ok = full(rv) && wait(bar(Smem::p_full, 2 * x), p_parity >> x & 1);
              if (!ok) break;
              fence_after();
              if (elect_one()) pv4(x, 0, v_at(rv), i >= 2);
              __syncwarp();
            }
            if (more) ok = full(rk);
            if (i >= 0) {
              ok = wait(bar(Smem::p_full, 2 * x + 1), p_parity >> x & 1) && ok;
              p_parity ^= 1u << x;
              fence_after();
            }
            if (!ok) break;
            if (elect_one()) {
              if (i >= 0) pv4(x, 1, v_at(rv), true);
              if (more)
                qk8(x, q_desc, k_at(rk));
              else
                mma_commit(bar(Smem::o_full, x));
              if (i + 3 == n) mma_commit(bar(Smem::q_empty, 0));
              if (i >= 0) mma_commit(bar(Smem::kv_empty, rv.st));
              if (more) mma_commit(bar(Smem::kv_empty, rk.st));
            }
            __syncwarp();
            ring = more ? rk.after() : rk;
          }
          continue;
        }
        bool v_there = false;
        // turn j: tile j - 1's K gives scores, tile j's weights meet their V
        // (j == u.last: only the first scores; j == u.begin: only the last outputs)
        int j = u.last;
        const int both = min(u.end[0], u.end[1]);
        while (j >= u.begin && ok) {
          const Ring rv = ring, rk = j == u.last ? ring : ring.after();
          if (j < both && j > u.begin) {
            // both tiles in full swing
            if (!v_there) ok = full(rv);
            const uint64_t vd = v_at(rv), kd = k_at(rk);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              ok = wait(bar(Smem::p_full, 2 * x), p_parity >> x & 1) && ok;
              fence_after();
              if (elect_one()) pv4(x, 0, vd, j + 1 < u.end[x]);
              __syncwarp();
              if (x == 0) ok = full(rk) && ok;
              ok = wait(bar(Smem::p_full, 2 * x + 1), p_parity >> x & 1) && ok;
              if (!ok) break;
              fence_after();
              if (elect_one()) {
                pv4(x, 1, vd, true);
                qk8(x, q_desc + x * (kTileBytes >> 4), kd);
              }
              __syncwarp();
              if (x == 0) {           // V of tile j - 1, if it is there already
                const Ring r2 = rk.after();
                v_there = __all_sync(kFull, mbar_test_wait(bar(Smem::kv_full, r2.st), r2.round & 1));
              }
            }
            if (!ok) break;
            p_parity ^= 3u;
            if (elect_one()) {
              if (j == u.begin + 1) {
                mma_commit(bar(Smem::q_empty, 0));
                mma_commit(bar(Smem::q_empty, 1));
              }
              mma_commit(bar(Smem::kv_empty, rv.st));
              mma_commit(bar(Smem::kv_empty, rk.st));
            }
            __syncwarp();
            ring = rk.after();
            --j;
            continue;
          }
          // a turn in which a tile starts, ends or has no part
          const bool first = j == u.last, more = j > u.begin;
          if (!first && !v_there) ok = full(rv);
          v_there = false;
          if (more && ok) ok = full(rk);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || u.end[x] == u.begin || j > u.end[x]) continue;
            const bool starts = j == u.end[x];
            if (starts) {
              ok = wait(bar(Smem::q_full, x), q_parity >> x & 1);
              if (!ok) continue;
              q_parity ^= 1u << x;
            } else {
              ok = wait(bar(Smem::p_full, 2 * x), p_parity >> x & 1) &&
                   wait(bar(Smem::p_full, 2 * x + 1), p_parity >> x & 1);
              if (!ok) continue;
              p_parity ^= 1u << x;
              fence_after();
            }
            if (elect_one()) {
              if (!starts) {
                pv4(x, 0, v_at(rv), j + 1 < u.end[x]);
                pv4(x, 1, v_at(rv), true);
              }
              if (more) {
                qk8(x, q_desc + x * (kTileBytes >> 4), k_at(rk));
                if (j == u.begin + 1) mma_commit(bar(Smem::q_empty, x));
              } else {
                mma_commit(bar(Smem::o_full, x));
              }
            }
            __syncwarp();
          }
          if (!first) {
            commit(bar(Smem::kv_empty, rv.st));
            ring = rk;
          }
          if (more) {
            commit(bar(Smem::kv_empty, rk.st));
            ring = rk.after();
          }
          --j;
        }
      }
      // every product has completed before the tensor memory is given back
      commit(bar(Smem::drained, 0));
      wait(bar(Smem::drained, 0), 0);
    } else if (warp == kWorkWarp) {
      // ---- work: the CTA's own unit, then those of CTAs that have not started -------------
      if (blockIdx.x == 0 && blockIdx.y == 0)   // every entry is looked at once, used or not
#pragma unroll 1
        for (int s = lane; s < p.num_seqs; s += 32)
          packed_seq(p.query_start, p.context_lens, s, p.num_tokens, max_context, p.dev_err, true);
      int bx = blockIdx.x, by = blockIdx.y;
      bool ok = true;
      int published = 0;
      for (int tries = 0; ok; ++tries) {
        Unit u;
        const bool work = bx >= 0 && make_unit(p, bx, by, max_context, u);
        if (bx < 0) u.begin = u.last = 0;   // tells the readers to stop
        if (work || bx < 0) {
          if (lane == 0) {
            *reinterpret_cast<Unit*>(smem + Smem::unit) = u;
            mbar_arrive(bar(Smem::unit_full, 0));
          }
          __syncwarp();
          if (bx < 0) break;
          ok = wait(bar(Smem::unit_empty, 0), published & 1);
          ++published;
          if (!ok) break;
        }
        if (lane == 0) {
          fence_proxy_async_smem();   // the last answer has been read
          mbar_arrive_expect_tx(bar(Smem::stolen, 0), 16);
          asm volatile(
              "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
              " [%0], [%1];" ::"r"(smem_u32(smem + Smem::answer)),
              "r"(smem_u32(bar(Smem::stolen, 0)))
              : "memory");
        }
        __syncwarp();
        ok = wait(bar(Smem::stolen, 0), tries & 1);
        if (!ok) {   // the answer may still come: another wait before the CTA goes
          wait(bar(Smem::stolen, 0), tries & 1);
          break;
        }
        uint32_t got, ax, ay;
        asm volatile(
            "{\n .reg .pred p;\n .reg .b128 h;\n .reg .b32 z, w;\n ld.shared.b128 h, [%3];\n"
            " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n"
            " selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n"
            " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, z, w}, h;\n"
            "}\n"
            : "=r"(got), "=r"(ax), "=r"(ay)
            : "r"(smem_u32(smem + Smem::answer))
            : "memory");
        __syncwarp();
        bx = got ? static_cast<int>(ax) : -1;
        by = static_cast<int>(ay);
      }
    }
  } else {
    // ---- softmax: one thread per query row ------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = warp >> 2;
    const int r = threadIdx.x & (kTile - 1);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + kColS + x * kTile;
    const uint32_t o_at = tmem + lanes + kColO + x * kTile;
    const float sc = p.scale_log2;
    int ns = 0, npair = 0;      // score tiles and pairs taken
    int turn[2] = {0, 0};       // outputs of either tile so far
    bool ok = true;
    Unit u;
    for (int k = 0; ok && next_unit(k, u); ++k) {
      const int o_turn[2] = {turn[0], turn[1]};
      turn[0] += u.has(0);
      turn[1] += u.has(1);
      if (!u.has(x)) continue;
      const int tok = u.tok0[x] + (r >> p.group_shift);
      const int pos0 = u.ctx - u.n + u.tok0[x];             // of the tile's first row
      const int pos = min(u.ctx - u.n + tok, u.ctx - 1);
      float m = kNoMax;   // log2 of the weights' unit
      float2 l2 = make_float2(0.f, 0.f);
      const int step = u.pair ? 2 : 1, top = u.pair ? u.last - 1 - x : u.end[x] - 1;
      for (int j = top; j >= u.begin; j -= step) {
        ok = wait(bar(Smem::s_full, x), ns & 1);
        if (!ok) break;
        ++ns;
        fence_after();
        if (j * kTile + kTile - 1 > pos0) {
          // some row of the tile does not see all of it: mask the scores in place, 32 columns
          // at a time
          const int see = pos - j * kTile;                    // columns 0 .. see
          const int all = __shfl_sync(kFull, see, 0);         // lane 0 sees the fewest
#pragma unroll 1
          for (int q = max(0, all + 1) & ~31; q < kTile; q += 32) {
            uint32_t v[32];
            tmem_ld32(s_at + q, v);
            wait_ld();
            const int left = see - q;
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = c <= left ? v[c] : 0xff800000u;
            tmem_st32(s_at + q, v);
          }
          wait_st();
        }
        float s[kTile];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, reinterpret_cast<uint32_t*>(s + 32 * c));
        wait_ld();
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < kTile - 4; c += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], s[c + i], s[c + 4 + i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], s[kTile - 4 + i]);
        const float bm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        // the maximum moves only when a score passes it by more than 2^8
        const bool moves = bm > m + (kHeadroom + kRescale);
        if (__any_sync(kFull, moves)) {
          const float nm = moves ? bm - kHeadroom : m;
          const float alpha = exp2_approx(m - nm);
          m = nm;
          l2 = fmul2(l2, make_float2(alpha, alpha));
          if (j != top) {
            // the scores of a tile follow the product of the one before it: O is at rest
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld32(o_at + 32 * c, o);
              wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(o_at + 32 * c, o);
            }
          }
        }
        const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-m, -m);
#pragma unroll
        for (int c = 0; c < 2; ++c) {   // the products start on the first half's weights
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float2 e = ffma2(make_float2(s[64 * c + 2 * i], s[64 * c + 2 * i + 1]), sc2, nm2);
            e.x = exp2_approx(e.x);
            e.y = exp2_approx(e.y);
            w[i] = pack_half2(e.x, e.y);
            l2 = ffma2(e, make_float2(1.f, 1.f), l2);
          }
          tmem_st32(s_at + 32 * c, w);
          wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(Smem::p_full, 2 * x + c));
        }
      }
      if (!ok) break;
      float l = l2.x + l2.y, other = 0.f;   // other: the second warpgroup's share of a pair
      if (u.pair) {
        float2* lm = reinterpret_cast<float2*>(smem + Smem::lm) + r;
        if (x == 1) {
          *lm = make_float2(l, m);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(Smem::lm_full, 0));
          // its output may go once the first warpgroup has read it
          ok = wait(bar(Smem::lm_free, 0), npair & 1);
          ++npair;
          continue;
        }
        ok = wait(bar(Smem::lm_full, 0), npair & 1) && wait(bar(Smem::o_full, 1), o_turn[1] & 1);
        if (!ok) break;
        ++npair;
        const float2 b = *lm;
        const float M = fmaxf(m, b.y), ca = exp2_approx(m - M), cb = exp2_approx(b.y - M);
        l = l * ca + b.x * cb;
        m = M;
        l2.x = ca;          // weights of the two outputs
        other = cb;
      }
      ok = wait(bar(Smem::o_full, x), o_turn[x] & 1);
      if (!ok) break;
      fence_after();
      if (nonfinite[k & 1] == k)
        add_nonfinite<BS>(p, u, o_at, pos, u.pair ? u.last : u.end[x]);
      const int head = (u.g << p.group_shift) + (r & ((1 << p.group_shift) - 1));
      const int64_t row = (static_cast<int64_t>(u.row0) + tok) * p.num_q_heads + head;
      const bool mine = tok < u.n;
      // rows whose tokens one unit covers are written, others leave a partial
      const bool whole = pos / kTile < p.split_tiles;
      const bool direct = mine && whole && u.split == 0;
      const bool part = mine && !whole && pos / kTile >= u.begin;
      // a row sees itself at least: its sum is 0 only if all its scores are -inf, and then the
      // definition's NaN comes out (0 * inf)
      const float inv = 1.f / l;
      const float mul = u.pair ? l2.x : 1.f;
      // 32 columns of the output, in units of 2^m
      const auto take = [&](int col, uint32_t* o) {
        tmem_ld32(o_at + col, o);
        if (u.pair) {
          uint32_t o1[32];
          tmem_ld32(o_at + kTile + col, o1);
          wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = __float_as_uint(__uint_as_float(o[i]) * mul + __uint_as_float(o1[i]) * other);
        } else {
          wait_ld();
        }
      };
      const int64_t at = row * p.splits + u.split;
      const uint32_t mine32 = __ballot_sync(kFull, direct);
      // rows leave through the warp's 4 KB of shared memory, 64 dims at a time (16-byte
      // chunk index XOR row % 8, as the copy engine reads them), while the warp goes on to
      // the next unit; stores of its own took 3700 cycles a tile (a row for each thread) or
      // 2700 (whole lines)
      uint4* box = reinterpret_cast<uint4*>(smem + Smem::stage + warp * 4096);
      if (mine32) {
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          if (lane == 0) bulk_wait_read();   // the last rows have left the buffer
          __syncwarp();
#pragma unroll 1
          for (int d = 0; d < 2; ++d) {
            uint32_t o[32];
            take(64 * c + 32 * d, o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                h[e] = pack_half2(__uint_as_float(o[8 * i + 2 * e]) * inv,
                                  __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
              box[lane * 8 + ((4 * d + i) ^ (lane & 7))] = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (mine32 == kFull) {
            if (lane == 0)
              tma_store_3d(&tmap_o, box, 64 * c, u.g << p.group_shift,
                           u.row0 + u.tok0[x] + ((warp & 3) * 32 >> p.group_shift));
          } else {   // the sequence's last rows: only those
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              const int rr = 4 * i + (lane >> 3), ch = lane & 7;
              const int64_t to = __shfl_sync(kFull, row, rr);
              if (mine32 >> rr & 1)
                *reinterpret_cast<uint4*>(p.out + to * kHeadDim + 64 * c + 8 * ch) =
                    box[rr * 8 + (ch ^ (rr & 7))];
            }
            __syncwarp();
          }
        }
      }
      if (__any_sync(kFull, part)) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          take(32 * c, o);
          uint4* dst = reinterpret_cast<uint4*>(p.part_o + at * kHeadDim + 32 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (part) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (part) {
        p.part_ml[2 * at] = m;
        p.part_ml[2 * at + 1] = l;
      }
      fence_before();   // O is read: the next unit's products may overwrite it once its weights are there
      if (u.pair) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Smem::lm_free, 0));
      }
    }
    if (lane == 0) bulk_wait();
  }
  fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *gave_up) report(p.dev_err, PKV_DEV_WAIT_TIMEOUT);
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Log-sum-exp merge of the rows that several units covered: one warp per row.
constexpr int kMergeRows = 8;
__global__ void __launch_bounds__(kMergeRows * 32)
    prompt_merge_kernel(const Params p, int64_t max_context) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeRows + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(p.num_tokens) * p.num_q_heads) return;
  const int i = static_cast<int>(row / p.num_q_heads);
  const int s = find_unit_seq(p.query_start, p.num_seqs, i, 1, 0);
  const PackedSeq q = packed_seq(p.query_start, p.context_lens, s, p.num_tokens, max_context,
                                 p.dev_err, false);
  if (!q.ok || i < q.row0 || i >= q.row0 + q.n) return;
  const int tile = (q.ctx - q.n + i - q.row0) / kTile;
  const int n = tile / p.split_tiles + 1;
  if (n == 1) return;
  const float* ml = p.part_ml + row * p.splits * 2;
  const float4* po = reinterpret_cast<const float4*>(p.part_o + row * p.splits * kHeadDim);
  float M = kNoMax;
  for (int k = lane; k < n; k += 32) M = fmaxf(M, ml[2 * k]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
#pragma unroll 4
  for (int k = 0; k < n; ++k) {
    const float c = exp2_approx(ml[2 * k] - M);
    const float4 v = po[k * (kHeadDim / 4) + lane];
    num.x += c * v.x;
    num.y += c * v.y;
    num.z += c * v.z;
    num.w += c * v.w;
    den += c * ml[2 * k + 1];
  }
  const float inv = 1.f / den;   // 0 only if all scores are -inf: NaN, see above
  uint2 w;
  w.x = pack_half2(num.x * inv, num.y * inv);
  w.y = pack_half2(num.z * inv, num.w * inv);
  *reinterpret_cast<uint2*>(p.out + row * kHeadDim + 4 * lane) = w;
}

// ---- host -------------------------------------------------------------------------------

// [rows, heads, 128] fp16, boxes of box_rows rows x box_heads heads x 64 dims
bool make_map(CUtensorMap* map, const void* base, int heads, int64_t rows, int box_heads,
              int box_rows) {
  auto fn = attn::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {kHeadDim, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {kHeadDim * 2, static_cast<cuuint64_t>(heads) * kHeadDim * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// a programmatic dependent launch: see the waits at the kernels' entries
template <class Kernel, class... Args>
int launch_dependent(Kernel kernel, dim3 grid, int threads, int smem, cudaStream_t st,
                     const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// the cache as [head][8 tokens][half][token of 8][64 dims]: a box is a block of one head,
// laid down as KvLayout wants it
bool make_block_map(CUtensorMap* map, const void* base, int heads, int64_t rows, int block_size) {
  auto fn = attn::encode_fn();
  if (!fn) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(heads) * kHeadDim * 2;
  cuuint64_t dims[5] = {64, 8, 2, static_cast<cuuint64_t>(rows) / 8, static_cast<cuuint64_t>(heads)};
  cuuint64_t strides[4] = {row, 128, 8 * row, kHeadDim * 2};
  cuuint32_t box[5] = {64, 8, 2, static_cast<cuuint32_t>(block_size) / 8, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BS>
int launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
           const CUtensorMap& mo, const Params& p, int64_t units, cudaStream_t st) {
  static std::atomic<uint8_t> opted_in[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  if (dev < 0 || dev >= 64 || !opted_in[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(prompt_attention_kernel<BS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Smem::alloc) != cudaSuccess)
      return PKV_ERR_CUDA;
    if (dev >= 0 && dev < 64) opted_in[dev].store(1, std::memory_order_release);
  }
  return launch_dependent(prompt_attention_kernel<BS>,
                          dim3(static_cast<unsigned>(units * p.num_kv_heads), p.splits), kThreads,
                          Smem::alloc, st, mq, mk, mv, mo, p);
}

int group_shift_of(int num_q_heads, int num_kv_heads) {
  if (num_q_heads % num_kv_heads) return -1;
  switch (num_q_heads / num_kv_heads) {
    case 1: return 0;
    case 2: return 1;
    case 4: return 2;
    case 8: return 3;
    default: return -1;
  }
}

// Splits of the key axis: 1 unless the units alone leave SMs idle; then two units
// for each SM, of at least 8 KV tiles.
constexpr int kSms = 152;
constexpr int kMinSplitTiles = 8;
// The longest context: a warp that waits for a whole unit of it stays within half the waits'
// limit.  128 tokens take 2300 cycles, 3100 in the slowest unit (one tile alone, see Unit).
constexpr int64_t kMaxContext = 1 << 25;
static_assert(kMaxContext / kTile * 3100 <= kWaitLimit / 2, "a unit of the longest context");
int64_t units_for(int num_tokens, int num_seqs, int group_shift) {
  return num_tokens / (2 * kTile >> group_shift) + static_cast<int64_t>(num_seqs);
}
int splits_for(int64_t ctas, int64_t max_context, int* split_tiles) {
  const int64_t tiles = (max_context + kTile - 1) / kTile;
  const int64_t fill = ctas < kSms ? 2 * kSms / std::max<int64_t>(ctas, 1) : 1;
  const int64_t want = std::min(fill, std::max<int64_t>(1, tiles / kMinSplitTiles));
  const int64_t per = (tiles + want - 1) / want;
  *split_tiles = static_cast<int>(per);
  return static_cast<int>((tiles + per - 1) / per);
}

int run(void* out, const void* q, const void* k, const void* v, const int32_t* block_tables,
        const int32_t* context_lens, const int32_t* query_start, int num_tokens, int num_seqs,
        int num_q_heads, int num_kv_heads, int block_size, int64_t num_blocks, int max_blocks,
        float scale, void* workspace, size_t workspace_bytes, int32_t* dev_err, void* stream) {
  const int shift = group_shift_of(num_q_heads, num_kv_heads);
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!out || !q || !k || !v || !query_start) return PKV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(q) |
       reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
       reinterpret_cast<uintptr_t>(workspace)) &
      15)
    return PKV_ERR_INVALID_ARG;
  const bool paged = block_size > 0;
  const int64_t units = units_for(num_tokens, num_seqs, shift);
  if (units * num_kv_heads > INT32_MAX || num_q_heads > 65535) return PKV_ERR_UNSUPPORTED;
  Params p = {};
  p.splits = 1;
  p.split_tiles = INT32_MAX / kTile;
  if (paged)
    p.splits = splits_for(units * num_kv_heads, static_cast<int64_t>(max_blocks) * block_size,
                          &p.split_tiles);
  if (p.splits > 1) {
    const size_t rows = static_cast<size_t>(num_tokens) * num_q_heads;
    if (!workspace || workspace_bytes < rows * p.splits * (kHeadDim + 2) * sizeof(float))
      return PKV_ERR_INVALID_ARG;
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = p.part_o + rows * p.splits * kHeadDim;
  }
  p.out = static_cast<__half*>(out);
  p.v = static_cast<const __half*>(v);
  p.query_start = query_start;
  p.context_lens = context_lens;
  p.block_tables = block_tables;
  p.dev_err = dev_err;
  p.num_blocks = num_blocks;
  p.num_tokens = num_tokens;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks = max_blocks;
  p.group_shift = shift;
  // a negative scale negates Q in the product, so that a row's maximum is the
  // largest score either way; a scale of 0 keeps masked scores at -infinity (and a
  // NaN stays one: std::max returns its first argument then)
  p.idesc_qk = kIdescBase | (scale < 0.f ? kNegateA : 0u);
  p.scale_log2 = std::max((scale < 0.f ? -scale : scale) * 1.4426950408889634f, 1e-30f);

  CUtensorMap mq, mk, mv, mo;
  const int64_t rows = num_blocks * block_size;
  if (!make_map(&mq, q, num_q_heads, num_tokens, 1 << shift, kTile >> shift) ||
      !make_map(&mo, out, num_q_heads, num_tokens, 1 << shift, 32 >> shift) ||
      !(paged ? make_block_map(&mk, k, num_kv_heads, rows, block_size) &&
                    make_block_map(&mv, v, num_kv_heads, rows, block_size)
              : make_map(&mk, k, num_kv_heads, num_tokens, 1, kTile) &&
                    make_map(&mv, v, num_kv_heads, num_tokens, 1, kTile)))
    return PKV_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int rc;
  switch (block_size) {
    case 0: rc = launch<0>(mq, mk, mv, mo, p, units, st); break;
    case 8: rc = launch<8>(mq, mk, mv, mo, p, units, st); break;
    case 16: rc = launch<16>(mq, mk, mv, mo, p, units, st); break;
    case 32: rc = launch<32>(mq, mk, mv, mo, p, units, st); break;
    default: rc = launch<64>(mq, mk, mv, mo, p, units, st); break;
  }
  if (rc != PKV_OK || p.splits == 1) return rc;
  const int64_t all = static_cast<int64_t>(num_tokens) * num_q_heads;
  return launch_dependent(prompt_merge_kernel,
                          dim3(static_cast<unsigned>((all + kMergeRows - 1) / kMergeRows)),
                          kMergeRows * 32, 0, st, p, static_cast<int64_t>(max_blocks) * block_size);
}

}  // namespace prompt
}  // namespace pkv

extern "C" size_t pkv_paged_attention_prefill_workspace_bytes(int num_tokens, int num_seqs,
                                                              int num_q_heads, int num_kv_heads,
                                                              int max_blocks_per_seq,
                                                              int block_size) {
  using namespace pkv::prompt;
  if (num_tokens <= 0 || num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      max_blocks_per_seq <= 0 || block_size <= 0)
    return 0;
  const int shift = group_shift_of(num_q_heads, num_kv_heads);
  if (shift < 0) return 0;
  int per = 0;
  const int splits = splits_for(units_for(num_tokens, num_seqs, shift) * num_kv_heads,
                                static_cast<int64_t>(max_blocks_per_seq) * block_size, &per);
  return splits > 1 ? static_cast<size_t>(num_tokens) * num_q_heads * splits * (kHeadDim + 2) *
                          sizeof(float)
                    : 0;
}

extern "C" int pkv_paged_attention_prefill(void* out, const void* q, const void* k_cache,
                                           const void* v_cache, const int32_t* block_tables,
                                           const int32_t* context_lens,
                                           const int32_t* query_start, int num_tokens,
                                           int num_seqs, int num_q_heads, int num_kv_heads,
                                           int head_dim, int block_size, int64_t num_blocks,
                                           int max_blocks_per_seq, float scale, void* workspace,
                                           size_t workspace_bytes, int32_t* dev_err,
                                           void* stream) {
  using namespace pkv::prompt;
  if (num_tokens < 0 || num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0)
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kHeadDim ||
      !(block_size == 8 || block_size == 16 || block_size == 32 || block_size == 64))
    return PKV_ERR_UNSUPPORTED;
  if (group_shift_of(num_q_heads, num_kv_heads) < 0) return PKV_ERR_UNSUPPORTED;
  if (num_tokens > INT32_MAX - 2 * kTile || num_blocks > INT32_MAX / block_size ||
      static_cast<int64_t>(max_blocks_per_seq) * block_size > kMaxContext)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs > 0 && num_tokens > 0 && (!block_tables || !context_lens)) return PKV_ERR_INVALID_ARG;
  return run(out, q, k_cache, v_cache, block_tables, context_lens, query_start, num_tokens,
             num_seqs, num_q_heads, num_kv_heads, block_size, num_blocks, max_blocks_per_seq, scale,
             workspace, workspace_bytes, dev_err, stream);
}

extern "C" int pkv_prompt_attention(void* out, const void* q, const void* k, const void* v,
                                    const int32_t* query_start, int num_tokens, int num_seqs,
                                    int num_q_heads, int num_kv_heads, int head_dim, float scale,
                                    int32_t* dev_err, void* stream) {
  using namespace pkv::prompt;
  if (num_tokens < 0 || num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0)
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kHeadDim || group_shift_of(num_q_heads, num_kv_heads) < 0)
    return PKV_ERR_UNSUPPORTED;
  if (num_tokens > kMaxContext) return PKV_ERR_UNSUPPORTED;
  return run(out, q, k, v, nullptr, nullptr, query_start, num_tokens, num_seqs, num_q_heads,
             num_kv_heads, 0, 0, 0, scale, nullptr, 0, dev_err, stream);
}
