// The 8-bit cache's codes, and the packed-batch metadata the prompt and
// 8-bit-cache kernels share.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// ---- packed batches ----------------------------------------------------------------
// Sequence s owns rows query_start[s] .. query_start[s + 1] - 1 of a packed
// [num_tokens, ...] tensor: the last n_s of its context_lens[s] tokens.
struct PackedSeq {
  int row0;   // first packed row
  int n;      // packed rows
  int ctx;    // tokens of the context, the packed ones included
  bool ok;    // the entries describe rows inside the tensor and a context that holds them
};

__device__ __forceinline__ PackedSeq packed_seq(const int32_t* query_start,
                                                const int32_t* context_lens, int s,
                                                int num_tokens, int64_t max_context,
                                                int32_t* dev_err, bool may_report) {
  PackedSeq q;
  q.row0 = __ldg(query_start + s);
  const int end = __ldg(query_start + s + 1);
  q.n = end - q.row0;
  q.ok = q.row0 >= 0 && end >= q.row0 && end <= num_tokens;
  if (!q.ok && may_report) report(dev_err, PKV_DEV_BAD_QUERY_RANGE);
  q.ctx = q.n;
  if (q.ok && context_lens) {
    q.ctx = __ldg(context_lens + s);
    if (q.ctx < q.n || q.ctx > max_context) {
      if (may_report) report(dev_err, PKV_DEV_BAD_CONTEXT_LEN);
      q.ok = false;
    }
  }
  return q;
}

// The batch is cut into units of `per` rows, each inside one sequence: those
// of sequence s are numbered from query_start[s] / per + slack * s.  That
// leaves room for every sequence's units (floor(b / per) - floor(a / per) +
// slack units between neighbours) without a prefix sum over the batch.
// Returns the last s with base(s) <= unit: a 32-way search by one warp.
__device__ __forceinline__ int unit_base(const int32_t* query_start, int s, int per, int slack) {
  return __ldg(query_start + s) / per + slack * s;
}
__device__ __forceinline__ int find_unit_seq(const int32_t* query_start, int num_seqs, int unit,
                                             int per, int slack) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = num_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool le = lane == 0 || (at < hi && unit_base(query_start, at, per, slack) <= unit);
    const unsigned b = __ballot_sync(0xffffffffu, le);
    // leading run of lanes that hold (entries out of order end it early)
    const int run = b == 0xffffffffu ? 32 : __ffs(~b) - 1;
    lo += (run - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// ---- waits ------------------------------------------------------------------------
// Bounded waits of a whole warp on an mbarrier: one vote decides, so that no lane
// branches by itself, and the limit is counted in clock cycles, which are quick to
// read.  A barrier that is through already costs 30 cycles so, 90 with each lane
// branching and a look at the global timer.
constexpr uint32_t kCopyWaitLimit = 1u << 30;   // half a second

// true: through; false: more than limit cycles have passed
__device__ __forceinline__ bool vote_wait(uint64_t* bar, uint32_t parity, uint32_t limit) {
  constexpr unsigned kAll = 0xffffffffu;
  if (__all_sync(kAll, mbar_try_wait(bar, parity))) return true;
  const uint32_t t0 = clock();
  while (!__all_sync(kAll, mbar_try_wait(bar, parity)))
    if (__any_sync(kAll, static_cast<uint32_t>(clock()) - t0 > limit)) return false;
  return true;
}

// a wait that gives up is reported
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* dev_err,
                                          uint32_t limit = kCopyWaitLimit) {
  const bool through = vote_wait(bar, parity, limit);
  if (!through) report(dev_err, PKV_DEV_WAIT_TIMEOUT);
  return through;
}

// With short code: a wait that gives up only raises a flag in shared memory, which the
// CTA reports at its end.  The prompt kernel has some 45 waits, and code counts: what is
// not in the instruction cache costs some 100 cycles for 8 instructions, and a unit's
// first and last steps run code that the steps between have pushed out (the kernel
// shrunk from 77 to 56 KB ran 5 % faster on prompts of 2048 tokens).
__device__ __forceinline__ bool flag_wait(uint64_t* bar, uint32_t parity,
                                          volatile uint32_t* gave_up, uint32_t limit) {
  const bool through = vote_wait(bar, parity, limit);
  if (!through) *gave_up = 1;
  return through;
}

// ---- codes ------------------------------------------------------------------------
// A code c of a block and KV head stands for c * scale.  int8: -127..127;
// e4m3: the finite values, at most 448 in magnitude.
struct Int8Code {
  static constexpr float kMax = 127.f;
  // codes nearest to four values, ties to even
  static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    const auto one = [](float y) {
      return static_cast<uint32_t>(max(-127, min(127, __float2int_rn(y)))) & 0xffu;
    };
    return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
  }
  static __device__ __forceinline__ void decode4(uint32_t w, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = static_cast<float>(static_cast<int8_t>((w >> (8 * i)) & 0xffu));
  }
};

struct E4m3Code {
  static constexpr float kMax = 448.f;
  static __device__ __forceinline__ uint32_t pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    return pair(a, b) | pair(c, d) << 16;
  }
  static __device__ __forceinline__ uint32_t half2_of(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
    return r;
  }
  static __device__ __forceinline__ void decode4(uint32_t w, float (&f)[4]) {
    const float2 lo = half2_to_float2(half2_of(w & 0xffffu));
    const float2 hi = half2_to_float2(half2_of(w >> 16));
    f[0] = lo.x;
    f[1] = lo.y;
    f[2] = hi.x;
    f[3] = hi.y;
  }
};

}  // namespace pkv
