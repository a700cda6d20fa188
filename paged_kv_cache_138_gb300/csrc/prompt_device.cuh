// What the prompt attention kernels share (fp16 and 8-bit cache): tcgen05 and TMA wrappers,
// the units of work, launch helpers.
#pragma once

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

// TILES: query tiles of a unit, 2, or 1 where units have rows in one tile only
template <int TILES = 2>
__device__ __forceinline__ bool make_unit(const Params& p, int bx, int by, int64_t max_context,
                                          Unit& u) {
  const int per = TILES * kTile >> p.group_shift;   // tokens of a unit
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
    u.tok0[x] = nth * per + (TILES - 1 - x) * (kTile >> p.group_shift);
    const int tok_end = min(q.n, u.tok0[x] + (kTile >> p.group_shift));
    u.end[x] = u.begin;
    if (tok_end > u.tok0[x] && x < TILES) {
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

// ---- host -------------------------------------------------------------------------------

// [rows, heads, 128] fp16, boxes of box_rows rows x box_heads heads x 64 dims
inline bool make_map(CUtensorMap* map, const void* base, int heads, int64_t rows, int box_heads,
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
inline int launch_dependent(Kernel kernel, dim3 grid, int threads, int smem, cudaStream_t st,
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

inline int group_shift_of(int num_q_heads, int num_kv_heads) {
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
inline int64_t units_for(int num_tokens, int num_seqs, int group_shift, int tiles = 2) {
  return num_tokens / (tiles * kTile >> group_shift) + static_cast<int64_t>(num_seqs);
}
inline int splits_for(int64_t ctas, int64_t max_context, int* split_tiles) {
  const int64_t tiles = (max_context + kTile - 1) / kTile;
  const int64_t fill = ctas < kSms ? 2 * kSms / std::max<int64_t>(ctas, 1) : 1;
  const int64_t want = std::min(fill, std::max<int64_t>(1, tiles / kMinSplitTiles));
  const int64_t per = (tiles + want - 1) / want;
  *split_tiles = static_cast<int>(per);
  return static_cast<int>((tiles + per - 1) / per);
}

// the log-sum-exp merge of rows that several units covered (prompt_attention.cu)
int launch_merge(const Params& p, int64_t max_context, cudaStream_t st);

}  // namespace prompt
}  // namespace pkv
