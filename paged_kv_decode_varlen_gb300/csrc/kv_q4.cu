// 4-bit pages: quantising new K/V rows into their slots, and reading rows
// back as bf16.
//
// Quantisation of a group of 32 values (binary32 operations, each rounded to
// nearest even): lo, hi = min, max; D = bf16(16 ((hi - lo) / 15)); Z =
// bf16(lo - D); code = rint(16 ((x - Z) / D) - 16) clamped to [0, 15], 0 when
// D is 0.  The codes are taken against the rounded D and Z, so their rounding
// only shifts the grid's ends (by at most 2^-9 of |lo| + 2 D) and adds no
// error of its own inside it.
//
// Both kernels move bytes: a (token, kv head) row is 256 B of bf16 and 80 B of
// a page, for K and for V.  Sixteen threads take one row, eight dims (one code
// word) each: 16-byte accesses on the bf16 side, 64 contiguous bytes of codes
// and 16 of scales on the other.
#include "internal.h"
#include "q4.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kLanesPerRow = kHeadDim / 8;  // 16: one code word each
constexpr int kRowsPerCta = kThreads / kLanesPerRow;

// One lane's 8 values -> its code word and its group's (D, Z) word; the
// group's 32 values lie in 4 adjacent lanes of `mask`.
__device__ __forceinline__ void quantize8_q4(const uint4& x, unsigned mask, uint32_t& codes, uint32_t& dz) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo(w[i]);
    v[2 * i + 1] = bf16hi(w[i]);
  }
  float lo = v[0], hi = v[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, v[i]);
    hi = fmaxf(hi, v[i]);
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(mask, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, o));
  }
  const __nv_bfloat16 db = __float2bfloat16_rn(__fmul_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f), 16.f));
  const float d = __bfloat162float(db);
  const __nv_bfloat16 zb = __float2bfloat16_rn(__fsub_rn(lo, d));
  const float z = __bfloat162float(zb);
  codes = 0u;
  if (d != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = rintf(__fmul_rn(__fdiv_rn(__fsub_rn(v[i], z), d), 16.f) - 16.f);
      codes |= (uint32_t)fminf(fmaxf(c, 0.f), 15.f) << (4 * (i >> 1) + 16 * (i & 1));
    }
  }
  dz = (uint32_t)__bfloat16_as_ushort(db) | ((uint32_t)__bfloat16_as_ushort(zb) << 16);
}

__global__ void __launch_bounds__(kThreads) kv_append_q4_kernel(const AppendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t rows = p.n_tokens * p.num_kv_heads;
  const int64_t stride = (int64_t)gridDim.x * kRowsPerCta;
  const int l = threadIdx.x % kLanesPerRow;
  const unsigned mask = 0xffffu << (threadIdx.x & 16);  // the 16 lanes of this row
  uint8_t* kc = reinterpret_cast<uint8_t*>(p.k_cache);
  uint8_t* vc = reinterpret_cast<uint8_t*>(p.v_cache);
  for (int64_t row = (int64_t)blockIdx.x * kRowsPerCta + threadIdx.x / kLanesPerRow; row < rows; row += stride) {
    const int64_t tok = row / p.num_kv_heads;
    const int h = (int)(row % p.num_kv_heads);
    const int64_t slot = p.slot_mapping[tok];
    if (slot < 0) continue;
    const int64_t block = slot / kPage;
    const int t = (int)(slot % kPage);
    if (block >= p.num_blocks) {
      if (l == 0) record_error(p.err, PA_ERR_DEVICE_INDEX);
      continue;
    }
    const size_t slab = ((size_t)block * p.num_kv_heads + h) * kQ4Slab;
    const size_t code_at = slab + q4_code_at(t, l >> 2) + 4 * (l & 3);
    const size_t scale_at = slab + q4_scale_at(t, l >> 2);
    const uint4 kx = reinterpret_cast<const uint4*>(p.k_new + row * kHeadDim)[l];
    const uint4 vx = reinterpret_cast<const uint4*>(p.v_new + row * kHeadDim)[l];
    uint32_t codes, dz;
    quantize8_q4(kx, mask, codes, dz);
    *reinterpret_cast<uint32_t*>(kc + code_at) = codes;
    if ((l & 3) == 0) *reinterpret_cast<uint32_t*>(kc + scale_at) = dz;
    quantize8_q4(vx, mask, codes, dz);
    *reinterpret_cast<uint32_t*>(vc + code_at) = codes;
    if ((l & 3) == 0) *reinterpret_cast<uint32_t*>(vc + scale_at) = dz;
  }
}

__global__ void __launch_bounds__(kThreads) kv_read_q4_kernel(const ReadParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t rows = p.n_tokens * p.num_kv_heads;
  const int64_t stride = (int64_t)gridDim.x * kRowsPerCta;
  const int l = threadIdx.x % kLanesPerRow;
  for (int64_t row = (int64_t)blockIdx.x * kRowsPerCta + threadIdx.x / kLanesPerRow; row < rows; row += stride) {
    const int64_t tok = row / p.num_kv_heads;
    const int h = (int)(row % p.num_kv_heads);
    const int64_t slot = p.slot_mapping[tok];
    const int64_t block = slot / kPage;
    uint4 kx = make_uint4(0u, 0u, 0u, 0u), vx = kx;
    if (slot >= 0 && block < p.num_blocks) {
      const int t = (int)(slot % kPage);
      const size_t slab = ((size_t)block * p.num_kv_heads + h) * kQ4Slab;
      const size_t code_at = slab + q4_code_at(t, l >> 2) + 4 * (l & 3);
      const size_t scale_at = slab + q4_scale_at(t, l >> 2);
      kx = q4_word_values(*reinterpret_cast<const uint32_t*>(p.k_cache + code_at),
                          *reinterpret_cast<const uint32_t*>(p.k_cache + scale_at));
      vx = q4_word_values(*reinterpret_cast<const uint32_t*>(p.v_cache + code_at),
                          *reinterpret_cast<const uint32_t*>(p.v_cache + scale_at));
    } else if (slot >= 0 && l == 0) {
      record_error(p.err, PA_ERR_DEVICE_INDEX);
    }
    reinterpret_cast<uint4*>(p.k_out + row * kHeadDim)[l] = kx;
    reinterpret_cast<uint4*>(p.v_out + row * kHeadDim)[l] = vx;
  }
}

unsigned grid_for(int64_t rows) {
  const int64_t g = (rows + kRowsPerCta - 1) / kRowsPerCta;
  return (unsigned)(g > 65535 ? 65535 : g);
}

}  // namespace

cudaError_t launch_kv_append_q4(const AppendParams& p, cudaStream_t stream) {
  return launch_pdl(kv_append_q4_kernel, dim3(grid_for(p.n_tokens * p.num_kv_heads)), dim3(kThreads), 0, stream, p);
}

cudaError_t launch_kv_read_q4(const ReadParams& p, cudaStream_t stream) {
  return launch_pdl(kv_read_q4_kernel, dim3(grid_for(p.n_tokens * p.num_kv_heads)), dim3(kThreads), 0, stream, p);
}

}  // namespace pa
