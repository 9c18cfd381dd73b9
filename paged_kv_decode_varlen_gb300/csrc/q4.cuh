// The q4 page format: device helpers shared by the kernels that write, read
// and attend to 4-bit pages.
//
// A (block, kv head) slab of kQ4Slab bytes holds 16 tokens: 64 bytes of codes
// per token, then per (token, group of 32 dims) a bf16 pair D, Z.  A code c
// in 0 .. 15 stands for bf16(Z + D (1 + c / 16)), rounded once (to nearest
// even).  The four bits become the top mantissa bits of a bf16 in [1, 2), so
// one packed bf16 FMA gives two values, and they are what the tensor cores
// take: no wider copy of a page is made anywhere.
//
// Place of a code: token t's group g lies at 64 t + 16 (g ^ ((t >> 1) & 3)),
// so the 8 rows of 16 bytes that one 8 x 8 shared-memory matrix load takes
// (8 tokens, one group) fall into 8 different groups of four banks.  In its
// 32-bit word w, dim 32 g + 8 w + 2 i sits at bit 4 i and dim 32 g + 8 w +
// 2 i + 1 at bit 16 + 4 i: one shift and one masked insert give a pair of
// neighbouring dims.
#pragma once

#include <math.h>

#include "common.cuh"

namespace pa {

constexpr int kQ4Groups = kHeadDim / 32;             // scale groups of a row
constexpr int kQ4Row = kHeadDim / 2;                 // code bytes of a token
constexpr int kQ4Codes = kPage * kQ4Row;             // code bytes of a slab
constexpr int kQ4Slab = PA_Q4_SLAB_BYTES;
static_assert(kQ4Slab == kQ4Codes + kPage * kQ4Groups * 4 && kQ4Slab % 16 == 0, "codes, then (D, Z) pairs");

// Loads of what an earlier kernel of the stream may have written (a pool, new
// rows, partial results), as the coherent loads that they have to be: a q4 kernel
// is launched while the one before it may still run, so ld.global.nc, which wants
// memory that nobody writes while the kernel runs, might give what was there
// before.  Volatile, so that none is moved above the wait for that kernel; they
// pass L1, which none of them would use twice.  (.cs: read once.)
__device__ __forceinline__ uint32_t load_cg(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 load_cg(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float load_cg(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 load_cg(const float4* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_cs(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// The greater of two, NaN if one is: merging parts, a NaN of one shows in all.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// log2 sum_t 2^(s_t) from a maximum (or any reference) and the sum of weights
// against it; -inf without a weight (the sum of a row that has one is never 0),
// NaN where a score was.
__device__ __forceinline__ float lse_log2(float m, float l) { return l == 0.f ? -INFINITY : m + log2f(l); }

// Byte of token t's 16 code bytes of group g, and of its (D, Z) pair.
__device__ __forceinline__ int q4_code_at(int t, int g) { return t * kQ4Row + ((g ^ ((t >> 1) & 3)) << 4); }
__device__ __forceinline__ int q4_scale_at(int t, int g) { return kQ4Codes + (t * kQ4Groups + g) * 4; }

// Pair i (0 .. 3) of a code word as bf16x2 bits: 1 + c / 16 of dims 2 i and
// 2 i + 1 of the word's eight.
template <int i>
__device__ __forceinline__ uint32_t q4_unit_pair(uint32_t w) {
  const uint32_t s = i == 0 ? w << 3 : w >> (i == 0 ? 0 : 4 * i - 3);
  uint32_t u;  // (s & mask) | one in one instruction
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(u) : "r"(s), "r"(0x00780078u), "r"(0x3f803f80u));
  return u;
}

__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// A (D, Z) word -> (D, D) and (Z, Z); as moves of halves, which the FMA can take
// as an operand's halves (a byte permute it cannot: 2.7 % of a long decode).
__device__ __forceinline__ uint32_t q4_dup_d(uint32_t dz) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(r) : "r"(dz));
  return r;
}
__device__ __forceinline__ uint32_t q4_dup_z(uint32_t dz) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(r) : "r"(dz));
  return r;
}

// The eight values of a code word, as four bf16 pairs in dim order.
__device__ __forceinline__ uint4 q4_word_values(uint32_t w, uint32_t dz) {
  const uint32_t d = q4_dup_d(dz), z = q4_dup_z(dz);
  return make_uint4(bf16x2_fma(q4_unit_pair<0>(w), d, z), bf16x2_fma(q4_unit_pair<1>(w), d, z),
                    bf16x2_fma(q4_unit_pair<2>(w), d, z), bf16x2_fma(q4_unit_pair<3>(w), d, z));
}

}  // namespace pa
