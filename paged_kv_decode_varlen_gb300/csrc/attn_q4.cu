// Attention over 4-bit pages: one CTA per (query token, kv head), one warp
// per query head of the group.  Each lane scores one key of 32, the warp
// updates its running maximum and sum, and every lane accumulates 4 dims.
#include <math.h>

#include "internal.h"
#include "q4.cuh"

namespace pa {
namespace {

__device__ __forceinline__ float q4_value(const uint8_t* slab, int t, int d) {
  const int g = d / 32, w = d % 32 / 8, j = d % 8;
  const uint32_t word = *reinterpret_cast<const uint32_t*>(slab + q4_code_at(t, g) + 4 * w);
  const uint32_t dz = *reinterpret_cast<const uint32_t*>(slab + q4_scale_at(t, g));
  const uint4 v = q4_word_values(word, dz);
  const uint32_t pair = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
  return (j & 1) ? bf16hi(pair) : bf16lo(pair);
}

__global__ void __launch_bounds__(128) attn_q4_kernel(const AttnQ4Params p) {
  pdl_launch_dependents();
  pdl_wait();
  const int tok = blockIdx.x, kvh = blockIdx.y;
  const int lane = threadIdx.x & 31, head = kvh * kGroup + (threadIdx.x >> 5);
  int lo = 0, hi = p.num_reqs - 1;  // the last request that starts at or before tok
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.qo_indptr[mid] <= tok) lo = mid; else hi = mid - 1;
  }
  const int r = lo;
  if (p.qo_indptr[r + 1] - p.qo_indptr[r] == 1) return;  // a decode row
  const int n_keys = p.seq_lens[r] - (p.qo_indptr[r + 1] - tok) + 1;
  const uint16_t* q = p.q + ((size_t)tok * p.num_q_heads + head) * kHeadDim;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int t0 = 0; t0 < n_keys; t0 += 32) {
    const int t = t0 + lane;
    int blk = -1;
    if (t < n_keys && t / kPage < p.max_blocks_per_req) {
      blk = p.block_tables[(size_t)r * p.max_blocks_per_req + t / kPage];
      if (blk < 0 || blk >= p.num_blocks) {
        record_error(p.err, PA_ERR_DEVICE_INDEX);
        blk = -1;
      }
    }
    float s = -INFINITY;
    if (blk >= 0) {
      const uint8_t* slab = p.k_cache + ((size_t)blk * p.num_kv_heads + kvh) * kQ4Slab;
      float a = 0.f;
      for (int d = 0; d < kHeadDim; ++d) a = fmaf(__uint_as_float((uint32_t)q[d] << 16), q4_value(slab, t % kPage, d), a);
      s = a * p.scale_log2;
    }
    float mt = s;
    for (int i = 16; i > 0; i >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, i));
    mt = fmaxf(mt, m);
    if (mt == -INFINITY) continue;
    const float corr = fast_exp2(m - mt);
    const float w = blk >= 0 ? fast_exp2(s - mt) : 0.f;
    m = mt;
    l = l * corr + w;
    for (int i = 0; i < 4; ++i) o[i] *= corr;
    for (int j = 0; j < 32; ++j) {
      const int b = __shfl_sync(0xffffffffu, blk, j);
      const float wj = __shfl_sync(0xffffffffu, w, j);
      if (b < 0) continue;
      const uint8_t* slab = p.v_cache + ((size_t)b * p.num_kv_heads + kvh) * kQ4Slab;
      for (int i = 0; i < 4; ++i) o[i] = fmaf(wj, q4_value(slab, (t0 + j) % kPage, 4 * lane + i), o[i]);
    }
  }
  for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const size_t row = (size_t)tok * p.num_q_heads + head;
  *reinterpret_cast<uint2*>(p.out + row * kHeadDim + 4 * lane) =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (p.lse && lane == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t launch_attn_q4(const AttnQ4Params& p, int total_q, cudaStream_t stream) {
  return launch_pdl(attn_q4_kernel, dim3(total_q, p.num_kv_heads), dim3(128), 0, stream, p);
}

}  // namespace pa
