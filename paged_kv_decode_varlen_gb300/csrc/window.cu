// Attention with a sliding window and first tokens that stay visible, over the
// paged cache.
//
// What is computed: the query at position p sees keys t <= p with t < sink_tokens or
// t > p - window; softmax attention over these in binary32, the running maximum and
// sum in the log2 domain.
//
// One warp per (query token, kv head): the 4 heads of the group, 4 dims per lane.
#include <math.h>

#include "internal.h"

#include "common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float4 load4(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}

__global__ void __launch_bounds__(kThreads) window_kernel(const WindowParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (u >= (int64_t)p.total_q * p.num_kv_heads) return;
  const int tok = (int)(u / p.num_kv_heads), kvh = (int)(u % p.num_kv_heads);
  int r = tok, n = 1, j = 0;
  if (p.qo_indptr) {
    int lo = 0, hi = p.num_reqs - 1;
    while (lo < hi) {  // the last request whose queries begin at or before tok
      const int mid = (lo + hi + 1) >> 1;
      if (p.qo_indptr[mid] <= tok) lo = mid; else hi = mid - 1;
    }
    r = lo;
    j = tok - p.qo_indptr[r];
    n = p.qo_indptr[r + 1] - p.qo_indptr[r];
  }
  if (n <= kWindowDecodeQueries) return;  // a row of the decode kernel
  int L = p.seq_lens[r];
  if (L < 0 || L > PA_MAX_SEQ_LEN || (L + kPage - 1) / kPage > p.max_blocks_per_req || (L > 0 && n > L)) {
    if (lane == 0) record_error(p.err, PA_ERR_DEVICE_INDEX);
    L = 0;
  }
  const int pos = L - n + j;
  const size_t row = (size_t)tok * p.num_q_heads + kvh * kGroup;
  float4 q[kGroup], o[kGroup];
  float m[kGroup], l[kGroup];
#pragma unroll
  for (int g = 0; g < kGroup; ++g) {
    q[g] = load4(p.q + (row + g) * kHeadDim + 4 * lane);
    q[g] = make_float4(q[g].x * p.scale_log2, q[g].y * p.scale_log2, q[g].z * p.scale_log2, q[g].w * p.scale_log2);
    o[g] = make_float4(0.f, 0.f, 0.f, 0.f);
    m[g] = -INFINITY;
    l[g] = 0.f;
  }
  const int keys = L > 0 ? pos + 1 : 0;
  const int low = max(pos - p.window + 1, 0);  // first key of the window
  for (int t = 0; t < keys; ++t) {
    if (t >= p.sink_tokens && t < low) t = low;
    const int id = p.block_tables[(size_t)r * p.max_blocks_per_req + t / kPage];
    if (id < 0 || id >= p.num_blocks) {
      if (lane == 0) record_error(p.err, PA_ERR_DEVICE_INDEX);
      continue;
    }
    const size_t at = (((size_t)id * p.num_kv_heads + kvh) * kPage + t % kPage) * kHeadDim + 4 * lane;
    const float4 k = load4(p.k_cache + at), v = load4(p.v_cache + at);
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      float s = q[g].x * k.x + q[g].y * k.y + q[g].z * k.z + q[g].w * k.w;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      if (s > m[g]) {
        const float c = exp2f(m[g] - s);  // m = -inf -> 0
        m[g] = s;
        l[g] *= c;
        o[g] = make_float4(o[g].x * c, o[g].y * c, o[g].z * c, o[g].w * c);
      }
      const float w = exp2f(s - (m[g] == -INFINITY ? 0.f : m[g]));
      l[g] += w;
      o[g] = make_float4(fmaf(w, v.x, o[g].x), fmaf(w, v.y, o[g].y), fmaf(w, v.z, o[g].z), fmaf(w, v.w, o[g].w));
    }
  }
#pragma unroll
  for (int g = 0; g < kGroup; ++g) {
    const float inv = l[g] == 0.f ? 0.f : 1.f / l[g];
    const uint2 w = make_uint2(pack_bf16x2(o[g].x * inv, o[g].y * inv), pack_bf16x2(o[g].z * inv, o[g].w * inv));
    *reinterpret_cast<uint2*>(p.out + (row + g) * kHeadDim + 4 * lane) = w;
    if (p.lse && lane == 0) p.lse[row + g] = l[g] == 0.f ? -INFINITY : (m[g] == -INFINITY ? 0.f : m[g]) * kLn2 + logf(l[g]);
  }
}

}  // namespace

cudaError_t launch_window(const WindowParams& p, cudaStream_t stream) {
  const int64_t warps = (int64_t)p.total_q * p.num_kv_heads;
  if (warps == 0) return cudaSuccess;
  const int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
  return launch_pdl(window_kernel, dim3((unsigned)grid), dim3(kThreads), 0, stream, p);
}

}  // namespace pa
