// Causal attention of prompts and prompt chunks over the 8-bit paged cache (sm_103a,
// tcgen05).
//
// For packed row i of sequence s (position pos, query head h, KV head g):
//   out[i, h] = sum_{t <= pos} softmax_t(scale <q[i, h], K[t, g]>) V[t, g]
// with K[t] = code * k_scale[block of t, g] and V likewise (codes int8 or e4m3).
//
// The units of work, the two query tiles that take turns, the places in tensor memory and
// the softmax are those of the prompt attention over the fp16 cache.  What differs:
//  * Codes come by TMA through a ring of three 16 KB tiles (five where units have one query
//    tile); a warpgroup widens them to fp16, exactly (int8 by placing the byte under the
//    exponent of 1024 and subtracting, e4m3 by its conversion), into a ring of three 32 KB
//    tiles in the layout that the products read.  An 8-bit product would need q and the
//    weights in 8 bits.
//  * The scales never touch the values.  A block's K scale multiplies its scores
//    (columns of one block lie together, so that it is one factor for 8 or 16 columns of
//    a row); its V scale enters the weight's exponent, w = 2^(x + log2 v_scale - m), and
//    the running maximum m is that of x + log2 v_scale.  So a weight keeps fp16's
//    precision whatever the scales are: off by half a step, 2^-11, or by 2^-32 of the largest
//    (see kHeadroom).  The softmax's sum takes them unrounded and divided by the scale
//    again, a block's sum at a time.
//  * Output rows leave through 2 KB a warp (the fp16 kernel: 4), which makes room for the
//    third ring stage of each kind.
//  * What bounds it: a query tile's softmax (1550 cycles a tile of 128 tokens, 500 of its
//    scheduler's instructions being the widening's) and its own products (1024) follow one
//    another, 2800 cycles a turn where the tensor core is busy for 2048.  16,384 tokens of 32/8
//    heads, int8: 1283-1305 us in short runs, 1363-1391 in loops of seconds, 1.58-1.71 PFLOP/s
//    (fp16 cache: 1180-1310 and 1370-1460); 16 x 2048 413-422 us, e4m3 399-405 (fp16 376-385); 8 of
//    64..512 rows behind 2048, 32 heads, e4m3: 94 us.  4 x 5..8 rows over 30k of 32/8 heads,
//    int8: 80 us, 3.2 TB/s: a tile of codes is widened in 1000 cycles, 550 of them instructions
//    of one warp a scheduler.  Tried and not kept: two warpgroups that widen, in turn or one
//    tile together (the softmax has 24 registers less; no faster), the next codes read ahead
//    of the widening (their place comes free later: 10 % slower with few rows).
#include <cmath>

#include "prompt_q8.cuh"

namespace pkv {
namespace prompt_q8 {

constexpr int kStages = 3;                       // fp16 tiles in shared memory
constexpr int kRawBytes = kTile * kHeadDim;
constexpr int kThreads = 512;                    // 2 softmax warpgroups; 2 copy, MMA and work
                                                 // warps; a widening warpgroup
// Registers a thread after the split: 256 * 200 + 256 * 56 = 512 * 128, what the CTA was
// launched with (a softmax thread holds a row of 128 scores).
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 200, kOtherRegs = 56;
static_assert(256 * kSoftmaxRegs + 256 * kOtherRegs <= kThreads * kLaunchRegs, "register split");
constexpr int kCopyWarp = 8, kMmaWarp = 9, kWorkWarp = 10, kCopyVWarp = 11, kWidenWarp = 12;
// The next unit is asked for when this one's last tiles are about to be copied.  Asked for as
// soon as a unit began, a CTA with a long one kept another from those that had none: 16 x 32
// rows over 4096 78 us instead of 48, 4 x 70..563 over 0..16,000 337 for 273, 16 x 2048 430 for
// 420 (2, 4 and 8 tiles ahead are alike).
constexpr int kAhead = 4;
constexpr int kReaders = 15;                     // warps that read a unit's description
// Scale entries of a tile, one for each `gran` tokens, in a ring: a tile's are written
// before its K is waited for and read until its weights are done.  K of the tile kSlots
// further on cannot be under way by then: the copies that are not yet read number kRaw at
// most, the widened tiles that are not yet used kStages, 8 copies of K and V or 4 tiles in all.
constexpr int kSlots = 8;
template <int BS>
struct Scales {
  static constexpr int gran = BS < 16 ? BS : 16;
  static constexpr int n = kTile / gran;           // entries of a tile
  static constexpr int bytes = 3 * n * 4;          // K factors, log2 of V scales, their inverses
};

// TILES: query tiles of a unit.  Units of one tile (few rows a sequence) have two more places
// for codes where the second tile would be: what bounds them is how much is under way.
template <int TILES>
struct Layout {
  static constexpr int kRaw = TILES == 2 ? 3 : 5;        // tiles of codes
  static_assert(kRaw + kStages <= 8 && kSlots >= 8, "see kSlots");
  static constexpr int q = 0;                            // query tiles
  static constexpr int kv = q + TILES * kTileBytes;
  static constexpr int raw = kv + kStages * kTileBytes;
  static constexpr int stage = raw + kRaw * kRawBytes;   // output rows, 2 KB a softmax warp
  static constexpr int lm = stage + 8 * 2048;            // float2 [128]: sums and maxima of a
                                                         // row that both warpgroups work on
  static constexpr int scales = lm + kTile * 8;
  static constexpr int bars = scales + kSlots * Scales<8>::bytes;
  static constexpr int q_full = bars;                    // [2]
  static constexpr int q_empty = q_full + 16;            // [2] the tile's last score product is done
  static constexpr int raw_full = q_empty + 16;          // [kRaw]
  static constexpr int raw_empty = raw_full + 8 * kRaw;  // [kRaw]
  static constexpr int kv_full = raw_empty + 8 * kRaw;   // [kStages]
  static constexpr int kv_empty = kv_full + 8 * kStages; // [kStages]
  static constexpr int sc_full = kv_empty + 8 * kStages; // [kSlots] a tile's scales are there
  static constexpr int s_full = sc_full + 8 * kSlots;    // [2] scores of a tile are in TMEM
  static constexpr int p_full = s_full + 16;             // [2][2] a half's weights are in TMEM
  static constexpr int o_full = p_full + 32;             // [2] the tile's output is complete
  static constexpr int lm_full = o_full + 16;            // lm is written
  static constexpr int lm_free = lm_full + 8;            // and read, tile 1's output too
  static constexpr int unit_full = lm_free + 8;          // the next unit is described
  static constexpr int unit_empty = unit_full + 8;       // and every warp has read it
  static constexpr int near_end = unit_empty + 8;        // most of a unit's copies are under way
  static constexpr int stolen = near_end + 8;            // the scheduler's answer is there
  static constexpr int drained = stolen + 8;
  static constexpr int answer = (drained + 8 + 15) / 16 * 16;
  static constexpr int unit = answer + 16;
  static constexpr int tmem = unit + 64;
  static constexpr int gave_up = tmem + 4;               // a wait did
  static constexpr int alloc = tmem + 16;
  static_assert(alloc <= 227 * 1024, "shared memory of one CTA");
};

// an fp16 tile: both halves of the dims one after the other, 1 KB atoms of 8 tokens x 64
// dims (128-byte swizzle)
constexpr uint32_t kHalf = kHalfBytes, kEight = 1024;

// The tile (counted from the unit's last) and kind of the at-th copy of a unit of n tiles:
// K and V of each tile in turn; in a pair V after the next tile's K.
struct CopyAt {
  int tile;
  bool v;
};
__device__ __forceinline__ CopyAt copy_at(int at, int n, bool pair) {
  if (!pair) return {at >> 1, (at & 1) != 0};
  if (at == 2 * n - 1) return {n - 1, true};
  if (at & 1) return {(at + 1) >> 1, false};
  return at ? CopyAt{(at - 2) >> 1, true} : CopyAt{0, false};
}

template <int N>
struct RingOf {
  int st;
  uint32_t round;
  __device__ __forceinline__ RingOf after() const {
    return st + 1 == N ? RingOf{0, round + 1} : RingOf{st + 1, round};
  }
};
using Ring = RingOf<kStages>;

template <class Wide, int BS, int TILES>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_q8_kernel(const __grid_constant__ CUtensorMap tmap_q,
                     const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v,
                     const __grid_constant__ CUtensorMap tmap_o, const Q8Params qp) {
  using Sc = Scales<BS>;
  using Smem = Layout<TILES>;
  constexpr int kRaw = Smem::kRaw;
  constexpr unsigned kFull = 0xffffffffu;
  const Params& p = qp.p;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {   // the swizzles count on it, and nothing is left to align by hand
    report(p.dev_err, PKV_DEV_WAIT_TIMEOUT);
    return;
  }
  // the same in every lane, which the compiler learns from the shuffle
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int64_t max_context = static_cast<int64_t>(p.max_blocks) * BS;
  const auto bar = [&](int at, int i) { return reinterpret_cast<uint64_t*>(smem + at) + i; };
  volatile uint32_t* gave_up = reinterpret_cast<volatile uint32_t*>(smem + Smem::gave_up);
  const auto wait = [&](uint64_t* b, uint32_t parity) {
    return flag_wait(b, parity, gave_up, kWaitLimit);
  };
  // the scales of tile slot t: factors at [0, n), logs at [n, 2 n), inverses at [2 n, 3 n)
  const auto scales_at = [&](uint32_t t) {
    return reinterpret_cast<float*>(smem + Smem::scales) + (t & (kSlots - 1)) * 3 * Sc::n;
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
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(bar(Smem::raw_full, i), 1);
      mbar_init(bar(Smem::raw_empty, i), 4);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(Smem::kv_full, i), 4);
      mbar_init(bar(Smem::kv_empty, i), 1);
    }
    for (int i = 0; i < kSlots; ++i) mbar_init(bar(Smem::sc_full, i), 1);
    mbar_init(bar(Smem::lm_full, 0), 4);
    mbar_init(bar(Smem::lm_free, 0), 4);
    mbar_init(bar(Smem::unit_full, 0), 1);
    mbar_init(bar(Smem::unit_empty, 0), kReaders);
    mbar_init(bar(Smem::near_end, 0), 1);
    mbar_init(bar(Smem::stolen, 0), 1);
    mbar_init(bar(Smem::drained, 0), 1);
    *gave_up = 0;
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
      // ---- copies: codes of K and V of each tile through a ring of kRaw -----------------------
      // One warp brings Q, K and the scales of both, one V: both count through the whole
      // sequence.
      const int mine = warp == kCopyVWarp;
      constexpr int kBoxes = kTile / BS, kBatch = 32 / kBoxes;
      uint32_t base = 0, tiles = 0;           // the unit's first place in the ring, its first tile
      uint32_t q_seen = 0, q_parity = 0;      // bit x: Q copies of tile x so far
      uint32_t raw_seen = 0, raw_parity = 0;  // bit st: this warp's copies into a stage
      bool ok = true;
      Unit u;
      for (int k = 0; ok && next_unit(k, u); ++k) {
        const int n = u.last - u.begin;
        // Block ids and scales come a batch of 32 boxes at a time (a box a lane), ids two
        // batches ahead and scales one: loaded tile by tile, one ahead, their latency was the
        // time of a tile (3100 cycles with few rows).
        const auto ids_of = [&](int b) {   // -1 past the context
          const int i = b * kBatch + lane / kBoxes;
          const int tok = (u.last - 1 - i) * kTile + lane % kBoxes * BS;
          return i < n && tok < u.ctx
                     ? __ldg(p.block_tables + static_cast<int64_t>(u.s) * p.max_blocks + tok / BS)
                     : -1;
        };
        const auto scales_of = [&](int32_t id) {
          if (mine || id < 0 || id >= p.num_blocks) return make_float2(0.f, 0.f);
          const int64_t at = static_cast<int64_t>(id) * qp.scale_stride + u.g;
          return make_float2(__ldg(qp.k_scale + at), __ldg(qp.v_scale + at));
        };
        int32_t ids = ids_of(0), ids1 = ids_of(1), ids2 = -1;
        float2 scs = scales_of(ids), scs1 = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
          const int j = u.last - 1 - i, in_batch = i % kBatch;
          if (!mine && i == max(0, n - kAhead) && lane == 0) mbar_arrive(bar(Smem::near_end, 0));
          if (in_batch == 0) {
            if (i > 0) {
              ids = ids1;
              ids1 = ids2;
              scs = scs1;
            }
            ids2 = ids_of(i / kBatch + 2);
            scs1 = scales_of(ids1);
          }
          // this lane's box of the tile
          const int32_t id = __shfl_sync(kFull, ids, in_batch * kBoxes + lane % kBoxes);
          // where the tile's K or V comes in the ring (see CopyAt)
          const int at = !u.pair ? 2 * i + mine
                         : mine  ? (i + 1 < n ? 2 * i + 2 : 2 * n - 1)
                                 : max(0, 2 * i - 1);
          const uint32_t round = (base + at) / kRaw, st = (base + at) % kRaw;
          int row = static_cast<int>(p.num_blocks * BS);   // past the last row: zeros
          if (id >= 0 && id < p.num_blocks)
            row = id * BS;
          else if (lane < kBoxes && j * kTile + lane * BS < u.ctx)
            report(p.dev_err, PKV_DEV_BAD_BLOCK_ID);
          if (round > 0) ok = wait(bar(Smem::raw_empty, st), (round - 1) & 1);
          if (!ok) break;
          raw_seen |= 1u << st;
          raw_parity = (raw_parity & ~(1u << st)) | (round & 1) << st;
          uint64_t* b = bar(Smem::raw_full, st);
          uint8_t* dst = smem + Smem::raw + st * kRawBytes;
          if (lane == 0) mbar_arrive_expect_tx(b, kRawBytes);
          __syncwarp();
          if (lane < kBoxes)
            tma_load_3d(dst + lane * (kRawBytes / kBoxes), mine ? &tmap_v : &tmap_k, 0, u.g, row, b);
          if (!mine) {
            const float k_sc = __shfl_sync(kFull, scs.x, in_batch * kBoxes + lane % kBoxes);
            const float v_sc = __shfl_sync(kFull, scs.y, in_batch * kBoxes + lane % kBoxes);
            if (lane < kBoxes) {
              const BlockScale b = block_scale(k_sc, v_sc, p.scale_log2);
              float* to = scales_at(tiles + i);
#pragma unroll
              for (int e = 0; e < BS / Sc::gran; ++e) {
                const int c = lane * (BS / Sc::gran) + e;
                to[c] = b.k;
                to[Sc::n + c] = b.v;
                to[2 * Sc::n + c] = b.inv;
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(Smem::sc_full, (tiles + i) & (kSlots - 1)));
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
        tiles += n;
      }
      // a wait gave up: let this warp's copies land before the CTA goes
      if (__any_sync(kFull, *gave_up)) {
#pragma unroll 1
        for (int i = 0; i < kRaw; ++i)
          if (raw_seen >> i & 1) wait(bar(Smem::raw_full, i), raw_parity >> i & 1);
#pragma unroll 1
        for (int x = 0; x < 2; ++x)
          if (q_seen >> x & 1) wait(bar(Smem::q_full, x), (q_parity >> x & 1) ^ 1);
      }
    } else if (warp >= kWidenWarp) {
      // ---- widening: a lane takes a token's 128 codes of each tile ----------------------------
      // 8 lanes are 8 tokens, whose 16-byte chunks the swizzle lays in 8 different banks,
      // among the codes (8 chunks a token) as among the fp16 values (twice 8).
      const int token = (warp - kWidenWarp) * 32 + lane;
      const uint32_t from = smem_u32(smem + Smem::raw) + token * kHeadDim;
      const uint32_t to = smem_u32(smem + Smem::kv) + (token >> 3) * kEight + (token & 7) * 128;
      const uint32_t x7 = (token & 7) << 4;
      Ring ring = {0, 0};
      RingOf<kRaw> raw = {0, 0};
      bool ok = true;
      Unit u;
      for (int k = 0; ok && next_unit(k, u); ++k) {
        const int n = u.last - u.begin;
#pragma unroll 1
        for (int at = 0; at < 2 * n; ++at, ring = ring.after(), raw = raw.after()) {
          ok = wait(bar(Smem::raw_full, raw.st), raw.round & 1);
          if (!ok) break;
          uint4 w[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            w[c] = ld_shared16(from + raw.st * kRawBytes + ((c << 4) ^ x7));
          // the codes are in registers before the copy engine may write their place again: an
          // arrival alone does not wait for reads (other tiles' codes came out, 8 tokens x 16
          // dims now and then)
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(Smem::raw_empty, raw.st));
          // a weight of 0 must not meet a NaN: codes past the context are any bytes
          const int tile = u.last - 1 - copy_at(at, n, u.pair).tile;
          if (tile * kTile + token >= u.ctx)
#pragma unroll
            for (int c = 0; c < 8; ++c) w[c] = make_uint4(0u, 0u, 0u, 0u);
          if (ring.round > 0) ok = wait(bar(Smem::kv_empty, ring.st), (ring.round - 1) & 1);
          if (!ok) break;
          const uint32_t dst = to + ring.st * kTileBytes;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint2 a = Wide::four(w[c].x), b = Wide::four(w[c].y);
            const uint2 d = Wide::four(w[c].z), e = Wide::four(w[c].w);
            const uint32_t half = dst + (c >> 2) * kHalf;
            st_shared16(half + (((c & 3) << 5) ^ x7), make_uint4(a.x, a.y, b.x, b.y));
            st_shared16(half + (((c & 3) << 5 | 16) ^ x7), make_uint4(d.x, d.y, e.x, e.y));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(Smem::kv_full, ring.st));
        }
      }
    } else if (warp == kMmaWarp) {
      // ---- matrix products: the warp runs together, one elected lane issues; the order and
      // the waits are those of the fp16 kernel --------------------------------------------------
      const uint32_t s_col = tmem + kColS, o_col = tmem + kColO;
      const uint64_t q_desc = operand_desc(smem_u32(smem + Smem::q), 16, 1024);
      const uint64_t k_desc = operand_desc(smem_u32(smem + Smem::kv), 16, kEight);
      const uint64_t v_desc = operand_desc(smem_u32(smem + Smem::kv), kHalf, kEight);
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
          mma_ts(o_col + x * kTile, s_col + x * kTile + 8 * kk, vd + kk * (2 * kEight >> 4),
                 kIdescPv, acc || i > 0);
        }
      };
      const auto qk8 = [&](int x, uint64_t qd, uint64_t kd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t step = (i & 3) * 32;
          mma_ss(s_col + x * kTile, qd + (((i >> 2) * kHalfBytes + step) >> 4),
                 kd + (((i >> 2) * kHalf + step) >> 4), p.idesc_qk, i > 0);
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
                // the widening of the next K waits for this V's place in the ring
                if (x == 1) mma_commit(bar(Smem::kv_empty, rv.st));
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
        const bool work = bx >= 0 && make_unit<TILES>(p, bx, by, max_context, u);
        if (bx < 0) u.begin = u.last = 0;   // tells the readers to stop
        if (work || bx < 0) {
          if (lane == 0) {
            *reinterpret_cast<Unit*>(smem + Smem::unit) = u;
            mbar_arrive(bar(Smem::unit_full, 0));
          }
          __syncwarp();
          if (bx < 0) break;
          ok = wait(bar(Smem::unit_empty, 0), published & 1) &&
               wait(bar(Smem::near_end, 0), published & 1);
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
    int ns = 0, npair = 0;      // score tiles and pairs taken
    uint32_t tiles = 0;         // the unit's first tile
    int turn[2] = {0, 0};       // outputs of either tile so far
    bool ok = true;
    Unit u;
    for (int k = 0; ok && next_unit(k, u); ++k) {
      const int o_turn[2] = {turn[0], turn[1]};
      const uint32_t tile0 = tiles;
      turn[0] += u.has(0);
      turn[1] += u.has(1);
      tiles += u.last - u.begin;
      if (!u.has(x)) continue;
      const int tok = u.tok0[x] + (r >> p.group_shift);
      const int pos0 = u.ctx - u.n + u.tok0[x];             // of the tile's first row
      const int pos = min(u.ctx - u.n + tok, u.ctx - 1);
      const bool rows = u.tok0[x] + ((warp & 3) * 32 >> p.group_shift) < u.n;
      float m = kNoMax;   // log2 of the weights' unit
      float2 l2 = make_float2(0.f, 0.f);
      const int step = u.pair ? 2 : 1, top = u.pair ? u.last - 1 - x : u.end[x] - 1;
      for (int j = top; j >= u.begin; j -= step) {
        const uint32_t slot = tile0 + (u.last - 1 - j);
        ok = wait(bar(Smem::sc_full, slot & (kSlots - 1)), slot / kSlots & 1);
        if (!ok) break;
        // K's factors and the logarithms of V's scales, read while the scores are under way
        const float4* scale4 = reinterpret_cast<const float4*>(scales_at(slot));
        constexpr bool kHeld = Sc::n == 8;   // 16 registers; with 8-token blocks read twice
        float4 held[kHeld ? 4 : 1];
        if (kHeld)
#pragma unroll
          for (int e = 0; e < 4; ++e) held[kHeld ? e : 0] = scale4[e];
        ok = wait(bar(Smem::s_full, x), ns & 1);
        if (!ok) break;
        ++ns;
        if (!rows) {   // none of the warp's rows is a token's: whatever the weights are, nobody reads
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(Smem::p_full, 2 * x));
            mbar_arrive(bar(Smem::p_full, 2 * x + 1));
          }
          continue;
        }
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
        // the largest x + log2 v_scale, an entry's columns at a time
        float bm[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int e4 = 0; e4 < Sc::n / 4; ++e4) {
          const float4 f4 = kHeld ? held[kHeld ? e4 : 0] : scale4[e4];
          const float4 g4 = kHeld ? held[kHeld ? Sc::n / 4 + e4 : 0] : scale4[Sc::n / 4 + e4];
          const float f[4] = {f4.x, f4.y, f4.z, f4.w}, g[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float* t = s + (4 * e4 + e) * Sc::gran;
            float a = max3(t[0], t[1], t[2]), b = max3(t[3], t[4], t[5]);
#pragma unroll
            for (int i = 6; i + 3 < Sc::gran; i += 4) {
              a = max3(a, t[i], t[i + 1]);
              b = max3(b, t[i + 2], t[i + 3]);
            }
            a = max3(a, t[Sc::gran - 2], t[Sc::gran - 1]);
            bm[e & 1] = fmaxf(bm[e & 1], fmaf(fmaxf(a, b), f[e], g[e]));
          }
        }
        const float top_x = fmaxf(bm[0], bm[1]);
        // the maximum moves only when a score passes it by more than 2^8
        const bool moves = top_x > m + (kHeadroom + kRescale);
        if (__any_sync(kFull, moves)) {
          const float nm = moves ? top_x - kHeadroom : m;
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
#pragma unroll
        for (int c = 0; c < 2; ++c) {   // the products start on the first half's weights
          uint32_t w[32];
#pragma unroll
          for (int e4 = 0; e4 < Sc::n / 8; ++e4) {
            const int at = c * (Sc::n / 8) + e4;
            const float4 f4 = kHeld ? held[kHeld ? at : 0] : scale4[at];
            const float4 g4 = kHeld ? held[kHeld ? Sc::n / 4 + at : 0] : scale4[Sc::n / 4 + at];
            const float4 h4 = scale4[Sc::n / 2 + at];
            const float f[4] = {f4.x, f4.y, f4.z, f4.w}, g[4] = {g4.x, g4.y, g4.z, g4.w};
            const float h[4] = {h4.x, h4.y, h4.z, h4.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float off = g[q] - m;
              const float2 f2 = make_float2(f[q], f[q]), off2 = make_float2(off, off);
              float2 sum = make_float2(0.f, 0.f);
#pragma unroll
              for (int i = 0; i < Sc::gran / 2; ++i) {
                const int col = (4 * e4 + q) * Sc::gran + 2 * i;   // of the half
                float2 e = ffma2(make_float2(s[64 * c + col], s[64 * c + col + 1]), f2, off2);
                e.x = exp2_approx(e.x);
                e.y = exp2_approx(e.y);
                w[col / 2] = pack_half2(e.x, e.y);
                sum = i ? ffma2(e, make_float2(1.f, 1.f), sum) : e;
              }
              l2 = ffma2(sum, make_float2(h[q], h[q]), l2);
            }
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
      // rows leave through the warp's 2 KB of shared memory, 32 dims at a time (16-byte
      // chunk index XOR row / 2 % 4, as the copy engine reads 64-byte rows), while the warp
      // goes on to the next unit
      uint4* box = reinterpret_cast<uint4*>(smem + Smem::stage + warp * 2048);
      if (mine32) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          take(32 * c, o);
          if (lane == 0) bulk_wait_read();   // the last rows have left the buffer
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              h[e] = pack_half2(__uint_as_float(o[8 * i + 2 * e]) * inv,
                                __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
            box[lane * 4 + (i ^ (lane >> 1 & 3))] = make_uint4(h[0], h[1], h[2], h[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (mine32 == kFull) {
            if (lane == 0)
              tma_store_3d(&tmap_o, box, 32 * c, u.g << p.group_shift,
                           u.row0 + u.tok0[x] + ((warp & 3) * 32 >> p.group_shift));
          } else {   // the sequence's last rows: only those
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const int rr = 8 * i + (lane >> 2), ch = lane & 3;
              const int64_t to = __shfl_sync(kFull, row, rr);
              if (mine32 >> rr & 1)
                *reinterpret_cast<uint4*>(p.out + to * kHeadDim + 32 * c + 8 * ch) =
                    box[rr * 4 + (ch ^ (rr >> 1 & 3))];
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

// ---- host -------------------------------------------------------------------------------

// codes [rows, heads, 128 bytes], a box is a block of one head
bool make_code_map(CUtensorMap* map, const void* base, int heads, int64_t rows, int block_size) {
  auto fn = attn::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {kHeadDim, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {kHeadDim, static_cast<cuuint64_t>(heads) * kHeadDim};
  cuuint32_t box[3] = {kHeadDim, 1, static_cast<cuuint32_t>(block_size)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// output rows, boxes of 32 rows x 32 dims
bool make_out_map(CUtensorMap* map, void* base, int heads, int64_t rows, int group) {
  auto fn = attn::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {kHeadDim, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {kHeadDim * 2, static_cast<cuuint64_t>(heads) * kHeadDim * 2};
  cuuint32_t box[3] = {32, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(32 / group)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap q, k, v, out;
};

template <class Wide, int BS, int TILES>
int launch(const Maps& m, const Q8Params& qp, dim3 grid, cudaStream_t st) {
  static std::atomic<uint8_t> opted_in[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  if (dev < 0 || dev >= 64 || !opted_in[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(prompt_q8_kernel<Wide, BS, TILES>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Layout<TILES>::alloc) != cudaSuccess)
      return PKV_ERR_CUDA;
    if (dev >= 0 && dev < 64) opted_in[dev].store(1, std::memory_order_release);
  }
  return launch_dependent(prompt_q8_kernel<Wide, BS, TILES>, grid, kThreads, Layout<TILES>::alloc,
                          st, m.q, m.k, m.v, m.out, qp);
}

template <class Wide, int TILES>
int launch_any(int block_size, const Maps& m, const Q8Params& qp, dim3 grid, cudaStream_t st) {
  switch (block_size) {
    case 8: return launch<Wide, 8, TILES>(m, qp, grid, st);
    case 16: return launch<Wide, 16, TILES>(m, qp, grid, st);
    case 32: return launch<Wide, 32, TILES>(m, qp, grid, st);
    default: return launch<Wide, 64, TILES>(m, qp, grid, st);
  }
}

// a warp that waits for a whole unit of the longest context: see kMaxContext (a tile takes
// 2000 to 3000 cycles)
static_assert(kMaxContext / kTile * 4000 <= kWaitLimit / 2, "a unit of the longest context");

// Splits of the key axis for units of one query tile, by a model of the time in key tiles
// (1.2 us): a unit takes its tiles and one to four (128 rows), partials what they write and
// read, the merge four.  What counts is the sum for contexts that are all as long as the
// table and for contexts of every length up to it, where a unit is half as long on average
// and the last one ends half a unit late.  int8, 32/8 heads, against two units for each SM by
// the largest number of units that there can be: 4 x 8 rows over 32,760 81 us (92), 4 x 5..8 over
// 30k to 32.7k 80 (78), 1 x 20 over 32k 34 (43), 16 x 16 over 0..16,000 98 (133), 7 x 7..56 over
// 0..16,000 62 (67), 4 x 32 over 16,384, e4m3, 54 (47).  Units of two tiles keep that rule: by the
// model 4 x 200 over 8000 took 132 us (121), 1 x 200 over 3000 40 (31).
void cut_axis(Plan* plan, int num_tokens, int num_seqs, int num_kv_heads, int group_shift,
              int64_t max_context) {
  const int64_t all = (max_context + kTile - 1) / kTile;
  const double units = static_cast<double>(num_seqs) * num_kv_heads;   // mostly one a sequence
  const double rows = static_cast<double>(num_tokens) * (num_kv_heads << group_shift);
  // as many as fill the SMs three times, eight at least, of two tiles or more
  const int64_t most = std::min(std::max<int64_t>(1, all / 2),
                                std::max<int64_t>(8, static_cast<int64_t>(3 * kSms / units)));
  double least = 0;
  for (int64_t s = 1; s <= most; ++s) {
    const int64_t per = (all + s - 1) / s, splits = (all + per - 1) / per;
    const double unit = per + 1 + 3 * rows / (units * kTile);
    const double alike = std::ceil(units * splits / kSms) * unit;
    const double mixed = std::max(unit, units * splits * unit / (2 * kSms) + unit / 2);
    // 1040 bytes a row and split, 8.2 MB in a tile's time
    const double time = alike + mixed + (splits > 1 ? 2 * (4 + rows * splits / 7900) : 0);
    if (s > 1 && time >= least) continue;
    least = time;
    plan->splits = static_cast<int>(splits);
    plan->split_tiles = static_cast<int>(per);
  }
}

Plan plan_of(int num_tokens, int num_seqs, int num_kv_heads, int group_shift, int64_t max_context) {
  const int64_t rows = static_cast<int64_t>(num_tokens) << group_shift;   // of a KV head
  // Both kernels work for any batch; the rules go by the average sequence, since the host knows
  // no lengths.  16 rows, 64 x 4096 tokens, e4m3: 119 us and 132 here; 32 rows: 168 and 130.
  // Contexts of one tile whose units are all there at once take less time in the other kernel
  // (5 of 7..63 rows, 8 heads 5.8 us and 8.9 here; 4 x 64 of 32/8 heads, more units than places,
  // 14 and 9.3).  A long chunk among single tokens pays for the average: its units of 16 rows
  // each stream the whole context (255 single tokens over 1000 and 700 rows over 16k of 32/8
  // heads, int8, 1006 us, as two calls 256; 63 single tokens and 100 rows over 4096 145 and 132).
  const int64_t few = (rows / 16 + num_seqs) * num_kv_heads;   // units of the other kernel
  if (rows <= 16ll * num_seqs || (max_context <= kTile && few <= 3 * kSms))
    return few_rows_plan(num_tokens, num_seqs, num_kv_heads, group_shift, max_context);
  Plan plan = {};
  plan.tiles = rows <= static_cast<int64_t>(num_seqs) * kTile ? 1 : 2;
  plan.units = units_for(num_tokens, num_seqs, group_shift, plan.tiles);
  if (plan.tiles == 1)
    cut_axis(&plan, num_tokens, num_seqs, num_kv_heads, group_shift, max_context);
  else
    plan.splits = splits_for(plan.units * num_kv_heads, max_context, &plan.split_tiles);
  return plan;
}

size_t partial_bytes(const Plan& plan, int num_tokens, int num_q_heads) {
  return plan.splits > 1 ? static_cast<size_t>(num_tokens) * num_q_heads * plan.splits *
                               (kHeadDim + 2) * sizeof(float)
                         : 0;
}

}  // namespace prompt_q8
}  // namespace pkv

extern "C" int pkv_paged_attention_prefill_q8(
    void* out, const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
    const float* v_scale, int code, const int32_t* block_tables, const int32_t* context_lens,
    const int32_t* query_start, int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, int64_t num_blocks, int max_blocks_per_seq, int scale_stride,
    float scale, void* workspace, size_t workspace_bytes, int32_t* dev_err, void* stream) {
  using namespace pkv::prompt_q8;
  if (num_tokens < 0 || num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0 || scale_stride < num_kv_heads ||
      (code != PKV_CODE_INT8 && code != PKV_CODE_E4M3))
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kHeadDim ||
      !(block_size == 8 || block_size == 16 || block_size == 32 || block_size == 64))
    return PKV_ERR_UNSUPPORTED;
  const int shift = group_shift_of(num_q_heads, num_kv_heads);
  if (shift < 0) return PKV_ERR_UNSUPPORTED;
  const int64_t max_context = static_cast<int64_t>(max_blocks_per_seq) * block_size;
  if (num_tokens > INT32_MAX - 2 * kTile || num_blocks > INT32_MAX / block_size ||
      max_context > kMaxContext)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables ||
      !context_lens || !query_start)
    return PKV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(q) |
       reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
       reinterpret_cast<uintptr_t>(workspace)) &
          15 ||
      (reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3)
    return PKV_ERR_INVALID_ARG;
  const Plan plan = plan_of(num_tokens, num_seqs, num_kv_heads, shift, max_context);
  if (plan.units * num_kv_heads > INT32_MAX || num_q_heads > 65535 || plan.splits > 65535)
    return PKV_ERR_UNSUPPORTED;
  Q8Params qp = {};
  Params& p = qp.p;
  p.splits = plan.splits;
  p.split_tiles = plan.split_tiles;
  if (p.splits > 1) {
    if (!workspace || workspace_bytes < partial_bytes(plan, num_tokens, num_q_heads))
      return PKV_ERR_INVALID_ARG;
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = p.part_o + static_cast<size_t>(num_tokens) * num_q_heads * p.splits * kHeadDim;
  }
  p.out = static_cast<__half*>(out);
  qp.q = static_cast<const __half*>(q);
  p.query_start = query_start;
  p.context_lens = context_lens;
  p.block_tables = block_tables;
  p.dev_err = dev_err;
  p.num_blocks = num_blocks;
  p.num_tokens = num_tokens;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks = max_blocks_per_seq;
  p.group_shift = shift;
  // a negative scale negates Q in the product, so that a row's maximum is the largest score
  // either way
  p.idesc_qk = kIdescBase | (scale < 0.f ? kNegateA : 0u);
  p.scale_log2 = (scale < 0.f ? -scale : scale) * 1.4426950408889634f;
  qp.k_scale = k_scale;
  qp.v_scale = v_scale;
  qp.scale_stride = scale_stride;

  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int rc;
  if (plan.columns) {
    rc = launch_few_rows(qp, plan, code, block_size, k_cache, v_cache, st);
  } else {
    Maps m;
    const int64_t rows = num_blocks * block_size;
    if (!make_map(&m.q, q, num_q_heads, num_tokens, 1 << shift, kTile >> shift) ||
        !make_out_map(&m.out, out, num_q_heads, num_tokens, 1 << shift) ||
        !make_code_map(&m.k, k_cache, num_kv_heads, rows, block_size) ||
        !make_code_map(&m.v, v_cache, num_kv_heads, rows, block_size))
      return PKV_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(plan.units * num_kv_heads), p.splits);
    const auto go = [&](auto wide) {
      using Wide = decltype(wide);
      return plan.tiles == 1 ? launch_any<Wide, 1>(block_size, m, qp, grid, st)
                             : launch_any<Wide, 2>(block_size, m, qp, grid, st);
    };
    rc = code == PKV_CODE_INT8 ? go(Int8Wide()) : go(E4m3Wide());
  }
  if (rc != PKV_OK || p.splits == 1) return rc;
  return launch_merge(p, max_context, st);
}

extern "C" size_t pkv_paged_attention_prefill_q8_workspace_bytes(int num_tokens, int num_seqs,
                                                                 int num_q_heads,
                                                                 int num_kv_heads,
                                                                 int max_blocks_per_seq,
                                                                 int block_size) {
  using namespace pkv::prompt_q8;
  if (num_tokens <= 0 || num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      max_blocks_per_seq <= 0 || block_size <= 0)
    return 0;
  const int shift = group_shift_of(num_q_heads, num_kv_heads);
  if (shift < 0) return 0;
  return partial_bytes(plan_of(num_tokens, num_seqs, num_kv_heads, shift,
                               static_cast<int64_t>(max_blocks_per_seq) * block_size),
                       num_tokens, num_q_heads);
}
