// The 8-bit cache write: new fp16 K/V rows of a packed batch are coded into
// the blocks their positions fall in, one fp32 scale for each (block, KV head).
//
// For a block and head with new rows x and, when the block already holds rows
// of the sequence, the scale s0 they were coded under (0 otherwise):
//   s = max(s0, max|x| / M),  M = 127 (int8) or 448 (e4m3)
//   code(x) = nearest(x * (1 / s)), ties to even; one fp32 product
//   where s > s0, each earlier code c becomes nearest(c * (s0 / s))
// 1 / s, s0 / s and max|x| / M are IEEE fp32 quotients, so the codes are a
// function of the inputs alone, whatever the batch around them.
//
// What bounds it: HBM for prompts (16 of 1..4096 tokens, 8 heads, e4m3: 178 MB in 29.5 us,
// 6.0 TB/s with the launch); a step of single tokens (64 x 40 heads) is a chain of
// dependent loads, batch entry, block id, scale, row: 6.6 us.
#include <climits>

#include "q8_device.cuh"

namespace pkv {
namespace q8 {

constexpr int kHeadDim = 128;
constexpr int kWarps = 4;

struct WriteParams {
  const __half *k, *v;            // [num_tokens, Hkv, 128]
  uint8_t *k_cache, *v_cache;     // [num_blocks, bs, Hkv, 128]
  float *k_scale, *v_scale;       // [num_blocks, scale_stride]
  const int32_t* query_start;
  const int32_t* context_lens;
  const int32_t* block_tables;
  int32_t* dev_err;
  int64_t num_blocks;
  int num_tokens, num_seqs, num_kv_heads, max_blocks, scale_stride;
};

// One warp per (block of a sequence, KV head, K or V): the head's new rows of
// the block stay in registers between the maximum and the coding, 16 lanes to
// a row (16 bytes in, 8 out for each lane), so every input byte is read once.
template <class Code, int BS>
__global__ void __launch_bounds__(kWarps * 32) write_q8_kernel(const WriteParams p) {
  constexpr int kPasses = BS / 2;   // two rows a pass
  const int lane = threadIdx.x & 31;
  // a programmatic dependent of the stream's previous kernel, and the next one (the
  // attention) may place its CTAs while this grid runs: each reads after its wait
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && blockIdx.y == 0)   // every entry is looked at once, used or not
    for (int s = threadIdx.x; s < p.num_seqs; s += kWarps * 32)
      packed_seq(p.query_start, p.context_lens, s, p.num_tokens,
                 static_cast<int64_t>(p.max_blocks) * BS, p.dev_err, true);
  const int item = blockIdx.y * kWarps + (threadIdx.x >> 5);
  if (item >= 2 * p.num_kv_heads) return;
  const bool is_v = item >= p.num_kv_heads;
  const int g = is_v ? item - p.num_kv_heads : item;

  const int unit = blockIdx.x;
  const int s = find_unit_seq(p.query_start, p.num_seqs, unit, BS, 2);
  const PackedSeq seq = packed_seq(p.query_start, p.context_lens, s, p.num_tokens,
                                   static_cast<int64_t>(p.max_blocks) * BS, p.dev_err, false);
  if (!seq.ok || seq.n == 0) return;
  const int nth = unit - unit_base(p.query_start, s, BS, 2);
  const int start = seq.ctx - seq.n;
  const int64_t lb = start / BS + static_cast<int64_t>(nth);
  if (nth < 0 || lb * BS >= seq.ctx) return;
  const int base = static_cast<int>(lb) * BS;   // position of the block's row 0
  const int r0 = max(start - base, 0), r1 = min(seq.ctx - base, BS);
  const int32_t blk = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks + lb);
  if (blk < 0 || blk >= p.num_blocks) {
    if (lane == 0) report(p.dev_err, PKV_DEV_BAD_BLOCK_ID);
    return;
  }

  const int sub = lane >> 4, c = lane & 15;
  const int64_t row_elems = static_cast<int64_t>(p.num_kv_heads) * kHeadDim;
  const __half* src = (is_v ? p.v : p.k) +
                      (static_cast<int64_t>(seq.row0) + base - start) * row_elems + g * kHeadDim +
                      c * 8;
  uint8_t* dst = (is_v ? p.v_cache : p.k_cache) + static_cast<int64_t>(blk) * BS * row_elems +
                 g * kHeadDim + c * 8;
  float* scale_at =
      (is_v ? p.v_scale : p.k_scale) + static_cast<int64_t>(blk) * p.scale_stride + g;

  const float before = r0 > 0 ? *scale_at : 0.f;
  uint4 x[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = 2 * i + sub;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r >= r0 && r < r1) x[i] = __ldg(reinterpret_cast<const uint4*>(src + r * row_elems));
  }
  // |x| of fp16 orders as its bits do; 0x7c00 and above is not finite
  uint32_t top2 = 0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    top2 = __vmaxu2(top2, x[i].x & 0x7fff7fffu);
    top2 = __vmaxu2(top2, x[i].y & 0x7fff7fffu);
    top2 = __vmaxu2(top2, x[i].z & 0x7fff7fffu);
    top2 = __vmaxu2(top2, x[i].w & 0x7fff7fffu);
  }
  uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
  if (top >= 0x7c00u) {   // infinities and NaN are reported and stored as 0
    if (lane == 0) report(p.dev_err, PKV_DEV_NONFINITE);
    const auto drop = [](uint32_t w) {
      if ((w & 0x7c00u) == 0x7c00u) w &= 0xffff0000u;
      if ((w & 0x7c000000u) == 0x7c000000u) w &= 0x0000ffffu;
      return w;
    };
    top2 = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      x[i].x = drop(x[i].x);
      x[i].y = drop(x[i].y);
      x[i].z = drop(x[i].z);
      x[i].w = drop(x[i].w);
      top2 = __vmaxu2(top2, x[i].x & 0x7fff7fffu);
      top2 = __vmaxu2(top2, x[i].y & 0x7fff7fffu);
      top2 = __vmaxu2(top2, x[i].z & 0x7fff7fffu);
      top2 = __vmaxu2(top2, x[i].w & 0x7fff7fffu);
    }
    top = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
  }
  const float amax = __half2float(__ushort_as_half(static_cast<unsigned short>(top)));
  const float scale = fmaxf(before, __fdiv_rn(amax, Code::kMax));
  const float inv = scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;

  if (scale > before && r0 > 0) {   // earlier rows of the block, under the grown scale
    const float ratio = __fdiv_rn(before, scale);
    for (int r = sub; r < r0; r += 2) {
      uint2* at = reinterpret_cast<uint2*>(dst + r * row_elems);
      uint2 w = *at;
      float f[4], h[4];
      Code::decode4(w.x, f);
      Code::decode4(w.y, h);
      w.x = Code::encode4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
      w.y = Code::encode4(h[0] * ratio, h[1] * ratio, h[2] * ratio, h[3] * ratio);
      *at = w;
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = 2 * i + sub;
    if (r < r0 || r >= r1) continue;
    const float2 a = half2_to_float2(x[i].x), b = half2_to_float2(x[i].y);
    const float2 d = half2_to_float2(x[i].z), e = half2_to_float2(x[i].w);
    uint2 w;
    w.x = Code::encode4(a.x * inv, a.y * inv, b.x * inv, b.y * inv);
    w.y = Code::encode4(d.x * inv, d.y * inv, e.x * inv, e.y * inv);
    *reinterpret_cast<uint2*>(dst + r * row_elems) = w;
  }
  __syncwarp();   // every lane has read the earlier scale
  if (lane == 0) *scale_at = scale;
}

template <class Code>
int launch_write(const WriteParams& p, int block_size, int64_t units, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(units), (2 * p.num_kv_heads + kWarps - 1) / kWarps);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t rc;
  switch (block_size) {
    case 8: rc = cudaLaunchKernelEx(&cfg, write_q8_kernel<Code, 8>, p); break;
    case 16: rc = cudaLaunchKernelEx(&cfg, write_q8_kernel<Code, 16>, p); break;
    case 32: rc = cudaLaunchKernelEx(&cfg, write_q8_kernel<Code, 32>, p); break;
    default: rc = cudaLaunchKernelEx(&cfg, write_q8_kernel<Code, 64>, p); break;
  }
  return rc == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace q8
}  // namespace pkv

extern "C" int pkv_reshape_and_cache_q8(const void* k, const void* v, const int32_t* query_start,
                                        const int32_t* block_tables, const int32_t* context_lens,
                                        void* k_cache, void* v_cache, float* k_scale,
                                        float* v_scale, int code, int num_tokens, int num_seqs,
                                        int num_kv_heads, int head_dim, int block_size,
                                        int64_t num_blocks, int max_blocks_per_seq,
                                        int scale_stride, int32_t* dev_err, void* stream) {
  using namespace pkv::q8;
  if (num_tokens < 0 || num_seqs < 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0 || scale_stride < num_kv_heads)
    return PKV_ERR_INVALID_ARG;
  if (code != PKV_CODE_INT8 && code != PKV_CODE_E4M3) return PKV_ERR_INVALID_ARG;
  if (head_dim != kHeadDim ||
      !(block_size == 8 || block_size == 16 || block_size == 32 || block_size == 64))
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!k || !v || !query_start || !block_tables || !context_lens || !k_cache || !v_cache ||
      !k_scale || !v_scale)
    return PKV_ERR_INVALID_ARG;
  const uintptr_t align = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
                          reinterpret_cast<uintptr_t>(k_cache) |
                          reinterpret_cast<uintptr_t>(v_cache);
  if ((align & 15) || ((reinterpret_cast<uintptr_t>(k_scale) |
                        reinterpret_cast<uintptr_t>(v_scale)) & 3))
    return PKV_ERR_INVALID_ARG;
  if (num_kv_heads > 65535 || num_blocks > INT32_MAX / block_size ||
      static_cast<int64_t>(max_blocks_per_seq) * block_size > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  const int64_t units = static_cast<int64_t>(num_tokens) / block_size + 2 * int64_t(num_seqs);
  if (units > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  WriteParams p;
  p.k = static_cast<const __half*>(k);
  p.v = static_cast<const __half*>(v);
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.query_start = query_start;
  p.context_lens = context_lens;
  p.block_tables = block_tables;
  p.dev_err = dev_err;
  p.num_blocks = num_blocks;
  p.num_tokens = num_tokens;
  p.num_seqs = num_seqs;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks = max_blocks_per_seq;
  p.scale_stride = scale_stride;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return code == PKV_CODE_INT8 ? launch_write<pkv::Int8Code>(p, block_size, units, st)
                               : launch_write<pkv::E4m3Code>(p, block_size, units, st);
}
