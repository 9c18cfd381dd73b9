// Norms of queries and keys for each head and the rotation by their positions, in
// one pass; with the append, keys and values go to their slots of the pools.
//
// What is computed, for a head's row x of 128 values: y = x / sqrt(mean x^2 + eps) *
// weight, and pairs (a, b) of y turned by the angle position * speed.  Everything in
// binary32, rounded once to bf16.
//
// Angles.  A speed comes as the fraction of a turn per position in units of 2^-64
// (pa_rope_turns); position times that in 64-bit integers, whose overflow drops whole
// turns, is the angle to 2^-64 of a turn times the position.  Its upper 32 bits, as
// a signed fraction of half a turn, go to sincospif: no range reduction, and as exact
// at position 2^20 as at 1.
//
// Bound: HBM for many tokens (a token with 32 + 8 + 8 heads reads and writes 12 KiB
// each), latency for few.
#include "internal.h"

#include "common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;  // per row, 16 dims each: [8 c, 8 c + 8) and [64 + 8 c, 64 + 8 c + 8)
constexpr int kSlots = kThreads / kLanes;
constexpr int kMaxTok = 32;  // tokens per CTA

__device__ __forceinline__ void unpack8(const uint4& x, float* f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo(w[i]);
    f[2 * i + 1] = bf16hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

template <bool kAppend, bool kInter>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const RopeParams p, int tok_per_cta) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float2 cs[kMaxTok][kHeadDim / 2];  // cos, sin of (token, pair)
  const int half = p.rotary_dim / 2;
  const int64_t tok0 = (int64_t)blockIdx.x * tok_per_cta;
  const int n_tok = (int)min((int64_t)tok_per_cta, p.n_tokens - tok0);
  for (int i = threadIdx.x; i < n_tok * half; i += kThreads) {
    const int t = i / half, j = i - t * half;
    const uint64_t a = (uint64_t)(int64_t)p.positions[tok0 + t] * p.turns[j];
    float s, c;
    sincospif((float)(int32_t)(a >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: of half a turn
    cs[t][j] = make_float2(c, s);
  }
  __syncthreads();
  const int rows = p.num_q_heads + (kAppend ? 2 : 1) * p.num_kv_heads;
  const int c = threadIdx.x % kLanes;
  const unsigned lanes = 0xffu << (threadIdx.x & 24);  // of this row
  for (int u = threadIdx.x / kLanes; u < n_tok * rows; u += kSlots) {
    const int t = u / rows, h = u - t * rows;
    const int64_t tok = tok0 + t;
    const bool is_q = h < p.num_q_heads, is_v = h >= p.num_q_heads + p.num_kv_heads;
    const int hk = is_q ? h : is_v ? h - p.num_q_heads - p.num_kv_heads : h - p.num_q_heads;
    const uint16_t* src = (is_q ? p.q + tok * p.q_stride : is_v ? p.v + tok * p.v_stride : p.k + tok * p.k_stride) +
                          (size_t)hk * kHeadDim;
    uint16_t* dst;
    if (is_q) {
      dst = p.q_out + (tok * p.num_q_heads + hk) * kHeadDim;
    } else if constexpr (kAppend) {
      const int64_t slot = p.slot_mapping[tok];
      if (slot < 0) continue;
      const int64_t block = slot / kPage;
      if (block >= p.num_blocks) {
        if (c == 0) record_error(p.err, PA_ERR_DEVICE_INDEX);
        continue;
      }
      dst = (is_v ? p.v_cache : p.k_cache) + ((block * p.num_kv_heads + hk) * kPage + slot % kPage) * kHeadDim;
    } else {
      dst = p.k_out + (tok * p.num_kv_heads + hk) * kHeadDim;
    }
    uint4 lo = *reinterpret_cast<const uint4*>(src + 8 * c);
    uint4 hi = *reinterpret_cast<const uint4*>(src + 64 + 8 * c);
    if (!is_v) {
      float y[16];
      unpack8(lo, y);
      unpack8(hi, y + 8);
      const float* weight = is_q ? p.q_weight : p.k_weight;
      if (weight) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(lanes, ss, o);
        const float r = 1.f / sqrtf(ss * (1.f / kHeadDim) + p.eps);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] *= r * weight[(i < 8 ? 8 * c : 56 + 8 * c) + i];
      }
      float z[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int d = (i < 8 ? 8 * c : 56 + 8 * c) + i;
        z[i] = y[i];
        if constexpr (kInter) {
          if (d < p.rotary_dim) {
            const float2 w = cs[t][d / 2];
            z[i] = (i & 1) ? fmaf(y[i], w.x, y[i ^ 1] * w.y) : fmaf(y[i], w.x, -y[i ^ 1] * w.y);
          }
        }
      }
      if constexpr (!kInter) {
        // dims come in chunks of 8, chunk e = c or 8 + c; its partner lies half / 8
        // chunks away
        const int far = half / 8;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int e = 8 * s + c;
          const bool low = e < far, turned = e < 2 * far;
          const int pe = !turned ? e : low ? e + far : e - far;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int from = (threadIdx.x & 24) + (pe & 7);
            const float p0 = __shfl_sync(lanes, y[i], from), p1 = __shfl_sync(lanes, y[8 + i], from);
            const float other = pe >> 3 ? p1 : p0;
            if (turned) {
              const float2 w = cs[t][(low ? e : pe) * 8 + i];
              z[8 * s + i] = fmaf(y[8 * s + i], w.x, low ? -other * w.y : other * w.y);
            }
          }
        }
      }
      lo = pack8(z);
      hi = pack8(z + 8);
    }
    *reinterpret_cast<uint4*>(dst + 8 * c) = lo;
    *reinterpret_cast<uint4*>(dst + 64 + 8 * c) = hi;
  }
}

}  // namespace

cudaError_t launch_norm_rope(const RopeParams& p, bool append, bool interleaved, cudaStream_t stream) {
  const int rows = p.num_q_heads + (append ? 2 : 1) * p.num_kv_heads;
  const int per = rows >= kSlots ? 1 : kSlots / rows;
  const dim3 grid((unsigned)((p.n_tokens + per - 1) / per));
  if (append)
    return interleaved ? launch_pdl(norm_rope_kernel<true, true>, grid, dim3(kThreads), 0, stream, p, per)
                       : launch_pdl(norm_rope_kernel<true, false>, grid, dim3(kThreads), 0, stream, p, per);
  return interleaved ? launch_pdl(norm_rope_kernel<false, true>, grid, dim3(kThreads), 0, stream, p, per)
                     : launch_pdl(norm_rope_kernel<false, false>, grid, dim3(kThreads), 0, stream, p, per);
}

}  // namespace pa
