// 4-bit pages: quantising new K/V rows into their slots, and reading rows
// back as bf16.
//
// Quantisation of a group of 32 values (binary32 operations, each rounded to
// nearest even): lo, hi = min, max; D = bf16(16 ((hi - lo) / 15)); Z =
// bf16(lo - D); code = rint(16 ((x - Z) / D) - 16) clamped to [0, 15], 0 when
// D is 0.  The codes are taken against the rounded D and Z, so their rounding
// only shifts the grid's ends and adds no error of its own inside it.  A bf16 is
// off by at most 2^-8 of the number: the lowest grid value, Z + D, lies within
// 2^-8 |lo - D| of lo, the highest, Z + 31/16 D, within that and 2^-8 (hi - lo)
// of hi, as 15/16 D is hi - lo but for D's rounding (binary32's aside).
//
// Both kernels move bytes: a (token, kv head) row is 256 B of bf16 and 80 B of
// a page, for K and for V.  Read back, sixteen threads take one row, eight dims
// (one code word) each: 16-byte accesses on the bf16 side, 64 contiguous bytes of
// codes and 16 of scales on the other, kRows rows per thread in flight, since one
// row is a chain of two loads (its slot, its bytes).  Written, eight threads take
// a row, two code words each: what a group needs once (its range, D, Z, the
// reciprocal) and a row (its slot, its place) is then done by half as many threads
// (7,021 tokens, 8 kv heads, written and read back: 17.2 us against 20.1 with
// sixteen; 64 tokens 3.7 against 3.5).  What bounds that side: warps wait for their
// own row's loads (the first stall), as a thread has one row and 46 % of the warp
// slots are taken; the schedulers issue 63 % of the time.
#include "internal.h"
#include "q4.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kLanesPerRow = kHeadDim / 8;  // 16: one code word each
constexpr int kRowsPerPass = kThreads / kLanesPerRow;
constexpr int kWriteLanes = kHeadDim / 16;  // 8: two code words each
constexpr int kWriteRows = kThreads / kWriteLanes;

// The least and greatest of a group's 32 values: 16 in each of 2 adjacent
// lanes, as bf16 pairs.  Across lanes both travel in one word, (least,
// -greatest), of which the lesser is kept.
__device__ __forceinline__ void group_range(const uint4& x, const uint4& y, float& lo, float& hi) {
  auto b2 = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
  const __nv_bfloat162 mn = __hmin2(__hmin2(__hmin2(b2(x.x), b2(x.y)), __hmin2(b2(x.z), b2(x.w))),
                                    __hmin2(__hmin2(b2(y.x), b2(y.y)), __hmin2(b2(y.z), b2(y.w))));
  const __nv_bfloat162 mx = __hmax2(__hmax2(__hmax2(b2(x.x), b2(x.y)), __hmax2(b2(x.z), b2(x.w))),
                                    __hmax2(__hmax2(b2(y.x), b2(y.y)), __hmax2(b2(y.z), b2(y.w))));
  __nv_bfloat162 m = __halves2bfloat162(__hmin(mn.x, mn.y), __hneg(__hmax(mx.x, mx.y)));
  m = __hmin2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  lo = __bfloat162float(m.x);
  hi = -__bfloat162float(m.y);
}

// One lane's 16 values -> its two code words and its group's (D, Z) word.
__device__ __forceinline__ void quantize16_q4(const uint4& x, const uint4& y, uint32_t (&codes)[2], uint32_t& dz) {
  float lo, hi;
  group_range(x, y, lo, hi);
  const __nv_bfloat16 db = __float2bfloat16_rn(__fmul_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f), 16.f));
  const __nv_bfloat16 zb = __float2bfloat16_rn(__fsub_rn(lo, __bfloat162float(db)));
  dz = (uint32_t)__bfloat16_as_ushort(db) | ((uint32_t)__bfloat16_as_ushort(zb) << 16);
  const float d = __bfloat162float(db) * 0.0625f, z = __bfloat162float(zb);  // a sixteenth of D: the step
  const uint32_t w[2][4] = {{x.x, x.y, x.z, x.w}, {y.x, y.y, y.z, y.w}};
  // n = (x - Z) / step rounded to an integer is 16 more than the code.  Clamped
  // to [16, 31], it is rounded by adding 1.5 x 2^23 (binary32 keeps no fraction
  // there) and left in the sum's low bits; four sums b_i = K + 16 + c_i add up to
  // sum 16^i c_i and a constant.
  constexpr uint32_t kBase = (0x4b400000u + 16u) * 0x1111u;
  uint32_t half[2][2] = {{0u, 0u}, {0u, 0u}};  // per word: even and odd dims' codes
  if (d >= 7.8886091e-31f && d <= 1.2676506e+30f) {  // 2^-100 .. 2^100: x - Z is between 0 and 48 steps
    // (x - Z) / step rounded to nearest, from r = 1 / step rounded to nearest:
    // one correction of t r by the exact remainder (Markstein, "Computation of
    // elementary functions on the IBM RISC System/6000 processor", 1990).  A
    // group shares the reciprocal, and pairs of values the instructions, which
    // count (7,021 tokens, when sixteen threads took a row: 24 us with a division
    // per value, 17.6 with this and no pairs, 12.5 so).
    const float r = __frcp_rn(d);
    const float2 r2 = make_float2(r, r), nd2 = make_float2(-d, -d), nz2 = make_float2(-z, -z);
    const float2 magic = make_float2(12582912.f, 12582912.f);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const float2 t = __fadd2_rn(bf16x2_to_f2(w[c][i]), nz2);
        float2 q = __fmul2_rn(t, r2);
        q = __ffma2_rn(__ffma2_rn(q, nd2, t), r2, q);
        q = make_float2(fminf(fmaxf(q.x, 16.f), 31.f), fminf(fmaxf(q.y, 16.f), 31.f));
        q = __fadd2_rn(q, magic);
        half[c][0] = half[c][0] * 16u + __float_as_uint(q.x);
        half[c][1] = half[c][1] * 16u + __float_as_uint(q.y);
      }
      half[c][0] -= kBase;
      half[c][1] -= kBase;
    }
  } else if (d != 0.f) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      uint32_t p = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i == j) p = w[j >> 2][j & 3];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float v = e ? bf16hi(p) : bf16lo(p);
        // 16 ((x - Z) / D): the quotient by D, as a step may be too small for binary32
        const float n = __fmul_rn(__fdiv_rn(__fsub_rn(v, z), __bfloat162float(db)), 16.f);
        const uint32_t code = (__float_as_uint(__fadd_rn(fminf(fmaxf(n, 16.f), 31.f), 12582912.f)) & 15u) << (4 * (i & 3));
        if (i < 4) half[0][e] |= code; else half[1][e] |= code;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) codes[c] = (half[c][0] & 0xffffu) | (half[c][1] << 16);
}

// Row indices fit 32 bits: 2^31 rows of bf16 would be 512 GiB.
struct Row {
  uint32_t row;   // token * kv heads + head
  uint32_t tok;
  int head;
  bool exists;
};
template <int kRows>
__device__ __forceinline__ Row row_of(int u, uint32_t rows, int num_kv_heads) {
  Row x;
  x.row = (blockIdx.x * kRows + u) * kRowsPerPass + threadIdx.x / kLanesPerRow;
  x.exists = x.row < rows;
  x.tok = x.row / (uint32_t)num_kv_heads;
  x.head = (int)(x.row - x.tok * (uint32_t)num_kv_heads);
  return x;
}

__global__ void __launch_bounds__(kThreads) kv_append_q4_kernel(const AppendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t row = blockIdx.x * kWriteRows + threadIdx.x / kWriteLanes;
  const bool exists = row < (uint32_t)(p.n_tokens * p.num_kv_heads);
  const uint32_t tok = row / (uint32_t)p.num_kv_heads;
  const int head = (int)(row - tok * (uint32_t)p.num_kv_heads);
  // the lane's words of its group: word and word + 2 (with its neighbour's 32
  // contiguous bytes per load)
  const int l = threadIdx.x % kWriteLanes, group = l >> 1, word = l & 1;
  int64_t slot = -1;
  uint4 k0, k1, v0, v1;
  k0 = k1 = v0 = v1 = make_uint4(0u, 0u, 0u, 0u);
  if (exists) {
    slot = p.slot_mapping[tok];
    const uint4* k = reinterpret_cast<const uint4*>(p.k_new + (size_t)row * kHeadDim) + 4 * group + word;
    const uint4* v = reinterpret_cast<const uint4*>(p.v_new + (size_t)row * kHeadDim) + 4 * group + word;
    k0 = load_cs(k);
    k1 = load_cs(k + 2);
    v0 = load_cs(v);
    v1 = load_cs(v + 2);
  }
  if (__all_sync(0xffffffffu, slot < 0)) return;
  uint32_t kcode[2], kdz, vcode[2], vdz;  // (whole warp: the groups' shuffles)
  quantize16_q4(k0, k1, kcode, kdz);
  quantize16_q4(v0, v1, vcode, vdz);
  if (slot < 0) return;
  const int64_t block = slot / kPage;
  if (block >= p.num_blocks) {
    if (l == 0) record_error(p.err, PA_ERR_DEVICE_INDEX);
    return;
  }
  const int t = (int)(slot % kPage);
  const size_t slab = ((size_t)block * p.num_kv_heads + head) * kQ4Slab;
  const size_t code_at = slab + q4_code_at(t, group) + 4 * word, scale_at = slab + q4_scale_at(t, group);
  uint8_t* kc = reinterpret_cast<uint8_t*>(p.k_cache);
  uint8_t* vc = reinterpret_cast<uint8_t*>(p.v_cache);
  *reinterpret_cast<uint32_t*>(kc + code_at) = kcode[0];
  *reinterpret_cast<uint32_t*>(kc + code_at + 8) = kcode[1];
  *reinterpret_cast<uint32_t*>(vc + code_at) = vcode[0];
  *reinterpret_cast<uint32_t*>(vc + code_at + 8) = vcode[1];
  if (word == 0) {
    *reinterpret_cast<uint32_t*>(kc + scale_at) = kdz;
    *reinterpret_cast<uint32_t*>(vc + scale_at) = vdz;
  }
}

template <int kRows>
__global__ void __launch_bounds__(kThreads) kv_read_q4_kernel(const ReadParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t rows = (uint32_t)(p.n_tokens * p.num_kv_heads);
  const int l = threadIdx.x % kLanesPerRow;
  int64_t slot[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const Row x = row_of<kRows>(u, rows, p.num_kv_heads);
    slot[u] = x.exists ? p.slot_mapping[x.tok] : -1;
  }
  // codes and (D, Z) of K and of V; a slot outside the pool reads as zeros
  uint32_t w[kRows][4];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const Row x = row_of<kRows>(u, rows, p.num_kv_heads);
    const int64_t block = slot[u] / kPage;
    w[u][0] = w[u][1] = w[u][2] = w[u][3] = 0u;
    if (slot[u] >= 0 && block < p.num_blocks) {
      const int t = (int)(slot[u] % kPage);
      const size_t slab = ((size_t)block * p.num_kv_heads + x.head) * kQ4Slab;
      const size_t code_at = slab + q4_code_at(t, l >> 2) + 4 * (l & 3);
      const size_t scale_at = slab + q4_scale_at(t, l >> 2);
      w[u][0] = load_cg(reinterpret_cast<const uint32_t*>(p.k_cache + code_at));
      w[u][1] = load_cg(reinterpret_cast<const uint32_t*>(p.k_cache + scale_at));
      w[u][2] = load_cg(reinterpret_cast<const uint32_t*>(p.v_cache + code_at));
      w[u][3] = load_cg(reinterpret_cast<const uint32_t*>(p.v_cache + scale_at));
    } else if (slot[u] >= 0 && l == 0) {
      record_error(p.err, PA_ERR_DEVICE_INDEX);
    }
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const Row x = row_of<kRows>(u, rows, p.num_kv_heads);
    if (!x.exists) continue;
    __stcs(reinterpret_cast<uint4*>(p.k_out + (size_t)x.row * kHeadDim) + l, q4_word_values(w[u][0], w[u][1]));
    __stcs(reinterpret_cast<uint4*>(p.v_out + (size_t)x.row * kHeadDim) + l, q4_word_values(w[u][2], w[u][3]));
  }
}

template <int kRows>
dim3 grid_for(int64_t rows) {
  return dim3((unsigned)((rows + kRows * kRowsPerPass - 1) / (kRows * kRowsPerPass)));
}

}  // namespace

// The read-back takes four rows per thread, for their loads in flight together,
// only when there are CTAs enough for every SM several times over; before that
// more CTAs are worth more (8 heads, captured: 4096 tokens 6.5 us with one row per
// thread, 7.6 with four; 8192 tokens 10.7 and 10.2; 16384 tokens 18.9 and 16.5;
// 131072 tokens 134 and 110).
constexpr int64_t kFewRows = 65536;

cudaError_t launch_kv_append_q4(const AppendParams& p, cudaStream_t stream) {
  const int64_t rows = p.n_tokens * p.num_kv_heads;
  return launch_pdl(kv_append_q4_kernel, dim3((unsigned)((rows + kWriteRows - 1) / kWriteRows)), dim3(kThreads), 0, stream,
                    p);
}

cudaError_t launch_kv_read_q4(const ReadParams& p, cudaStream_t stream) {
  const int64_t rows = p.n_tokens * p.num_kv_heads;
  if (rows <= kFewRows) return launch_pdl(kv_read_q4_kernel<1>, grid_for<1>(rows), dim3(kThreads), 0, stream, p);
  return launch_pdl(kv_read_q4_kernel<4>, grid_for<4>(rows), dim3(kThreads), 0, stream, p);
}

}  // namespace pa
