// What the two kernels of attention over the 8-bit cache share: parameters, exact widening of
// codes, a block's scales as they enter the softmax.
#pragma once

#include "prompt_device.cuh"

namespace pkv {
namespace prompt_q8 {

using namespace prompt;

struct Q8Params {
  Params p;                // v unused
  const float* k_scale;    // [num_blocks, scale_stride]
  const float* v_scale;
  const __half* q;
  int scale_stride;
};

// V scales from here down count as this one, 0 among them: what such a block adds to an output,
// 448 * 2^-60 at most, is nothing in fp16, while its weights, 2^60 times what meets the codes,
// count in the softmax's sum.  Scales of fp16 values are 0 or from 2^-33 on (2^-24 / 448).  With
// 2^-33 for the least, e4m3 codes above 256 under a scale of 0 came out as 2^-24.
constexpr float kLeastScale = 1.f / (1ull << 60), kLeastLog = -60.f;

// four codes as two packed fp16 pairs, exactly
struct Int8Wide {
  static __device__ __forceinline__ uint32_t pair(uint32_t w, uint32_t sel) {
    // bytes biased by 128: 1024 + u, minus 1152 = the code
    const __half2 h = u32_as_half2(__byte_perm(w, 0x64646464u, sel));
    return half2_as_u32(__hsub2(h, __half2half2(__ushort_as_half(0x6480))));
  }
  static __device__ __forceinline__ uint2 four(uint32_t w) {
    w ^= 0x80808080u;
    return make_uint2(pair(w, 0x4140), pair(w, 0x4342));
  }
};
struct E4m3Wide {
  static __device__ __forceinline__ uint2 four(uint32_t w) {
    return make_uint2(E4m3Code::half2_of(w & 0xffffu), E4m3Code::half2_of(w >> 16));
  }
};

// A block's scales in the softmax: x = score * k + v in log2 units is the exponent of the
// weight that meets V's codes, and that weight times inv the one that counts in the sum.
struct BlockScale {
  float k, v, inv;
};
__device__ __forceinline__ BlockScale block_scale(float k_scale, float v_scale, float scale_log2) {
  // a factor of 0 would turn a masked -infinity into a NaN (a scale that is not a number
  // stays one)
  const float f = k_scale * scale_log2, v = fmaxf(v_scale, kLeastScale);
  return {f < 1e-30f ? 1e-30f : f, v_scale <= kLeastScale ? kLeastLog : __log2f(v), __frcp_rn(v)};
}

// How a call is cut: by the kernel in prompt_q8.cu (columns 0), or the one for few rows a
// sequence (few_rows_q8.cu) with 8 or 16 rows of a KV head a unit.
struct Plan {
  int columns;
  int tiles;         // query tiles of a unit (columns 0)
  int64_t units;     // of one KV head, an upper bound
  int splits, split_tiles;
};
Plan few_rows_plan(int num_tokens, int num_seqs, int num_kv_heads, int group_shift,
                   int64_t max_context);
int launch_few_rows(const Q8Params& qp, const Plan& plan, int code, int block_size,
                    const void* k_cache, const void* v_cache, cudaStream_t st);

}  // namespace prompt_q8
}  // namespace pkv
