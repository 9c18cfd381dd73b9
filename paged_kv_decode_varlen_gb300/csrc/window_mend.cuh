// Attention with a window where values are not finite.
//
// A query that does not see a value has weight 0 for it, but 0 times an infinity or a NaN is
// a NaN.  Values that no query of a row sees are cleared before the products; where some
// queries see one and others do not, the outputs of the others are NaN.  (And a weight that
// goes into the product as two bf16 of opposite signs makes a NaN of an infinity.)  So
// outputs that are not finite are looked at again, which costs little where there are none:
// mend_row computes them from the keys that their query sees and no others.  8 prompts behind
// a window of 512 take 102.4 us (100.8 without), 80 rows of 5 queries 59.6 (59.4).  Taking
// such values out of the operands, by the warp that clears, and adding them to the outputs
// that see them at the end: 103.6; looking at V's pages in the decode kernel's loop: 62.4.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "q4.cuh"  // load_cg

namespace pa {

// Scores of a query (lane: dims 4 lane .. + 3 of q) and the page at `rows`, key t0 + k each,
// handed to use(k, score) for keys that the query at `pos` sees.
template <class F>
__device__ __forceinline__ void page_scores(const uint16_t* rows, float4 q, int t0, int pos, int window, int sinks, F use) {
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int k = 0; k < kPage; ++k) {
    const uint2 x = load_cg(reinterpret_cast<const uint2*>(rows + k * kHeadDim) + lane);
    float s = q.x * bf16lo(x.x) + q.y * bf16hi(x.x) + q.z * bf16lo(x.y) + q.w * bf16hi(x.y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int t = t0 + k;
    if (t <= pos && (t < sinks || t > pos - window)) use(k, s);
  }
}

// y: 4 dims (of this lane) of the output of a query at `pos`, its q (128 bf16), over pages 0 ..
// n - 1, page v + (v < lead ? lo : hi) of `table` each, of kv head kvh.  Those that are not
// finite, again, unless the query's scores are not.  Whole warp.
static __device__ __noinline__ float4 mend_row(const WindowParams& p, float4 y, const uint16_t* q, const int32_t* table,
                                               int kvh, int lead, int lo, int hi, int n, int pos) {
  const int lane = threadIdx.x & 31;
  const uint2 x = load_cg(reinterpret_cast<const uint2*>(q) + lane);
  const float4 qs = make_float4(bf16lo(x.x) * p.scale_log2, bf16hi(x.x) * p.scale_log2, bf16lo(x.y) * p.scale_log2,
                                bf16hi(x.y) * p.scale_log2);
  auto pages = [&](auto use) {  // every page with a block: its first token, its slab's offset
    for (int v = 0; v < n; ++v) {
      const int page = v + (v < lead ? lo : hi), block = table[page];
      if (block >= 0 && block < p.num_blocks)
        use(page * kPage, ((size_t)block * p.num_kv_heads + kvh) * (kPage * kHeadDim));
    }
  };
  float m = -INFINITY, l = 0.f;
  pages([&](int t0, size_t at) {
    page_scores(p.k_cache + at, qs, t0, pos, p.window, p.sink_tokens, [&](int, float s) {
      const float top = fmaxf(m, s);
      l = top == -INFINITY ? l : l * fast_exp2(m - top) + fast_exp2(s - top);
      m = top;
    });
  });
  if (!(l > 0.f && l < INFINITY)) return y;
  const float inv = 1.f / l;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  pages([&](int t0, size_t at) {
    page_scores(p.k_cache + at, qs, t0, pos, p.window, p.sink_tokens, [&](int k, float s) {
      const float w = fast_exp2(s - m) * inv;
      const uint2 v = load_cg(reinterpret_cast<const uint2*>(p.v_cache + at + k * kHeadDim) + lane);
      o = make_float4(fmaf(w, bf16lo(v.x), o.x), fmaf(w, bf16hi(v.x), o.y), fmaf(w, bf16lo(v.y), o.z),
                      fmaf(w, bf16hi(v.y), o.w));
    });
  });
  auto or_again = [](float was, float now) { return fabsf(was) < INFINITY ? was : now; };
  return make_float4(or_again(y.x, o.x), or_again(y.y, o.y), or_again(y.z, o.z), or_again(y.w, o.w));
}

// The same of 4 dims in bf16, in place.
__device__ __forceinline__ void mend_out(const WindowParams& p, uint16_t* out, const uint16_t* q, const int32_t* table,
                                         int kvh, int lead, int lo, int hi, int n, int pos) {
  uint2* at = reinterpret_cast<uint2*>(out) + (threadIdx.x & 31);
  const uint2 x = load_cg(at);
  const float4 y = make_float4(bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y));
  if (!__any_sync(0xffffffffu, !(fabsf(y.x) < INFINITY && fabsf(y.y) < INFINITY && fabsf(y.z) < INFINITY && fabsf(y.w) < INFINITY)))
    return;
  const float4 z = mend_row(p, y, q, table, kvh, lead, lo, hi, n, pos);
  *at = make_uint2(pack_bf16x2(z.x, z.y), pack_bf16x2(z.z, z.w));
}

}  // namespace pa
