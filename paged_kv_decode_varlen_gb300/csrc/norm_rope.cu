// Norms of queries and keys for each head and the rotation by their positions, in
// one pass; with the append, keys and values go to their slots of the pools.
//
// What is computed, for a head's row x of 128 values: y = x / sqrt(mean x^2 + eps) *
// weight, and pairs (a, b) of y turned by the angle position * speed.  Everything in
// binary32, rounded once to bf16.
//
// Angles.  A speed comes as the fraction of a turn per position in units of 2^-64
// (pa_rope_turns); position times that in 64-bit integers, whose overflow drops whole
// turns, is off by what the speed is (2^-52 of it, from binary64) times the position, and
// by nothing else: 2^-34 of a turn at position 2^20 for a speed of one radian.  Its upper 32
// bits, less the nearest quarter turn, go to sincospif as a signed fraction of half a turn,
// without a range reduction: what binary32 leaves of it, 2^-28 of a turn, is the larger error
// at every position.
//
// Work.  A unit is a token and up to kHeads of its kv heads, with the 4 query heads of
// each.  A warp takes units in turn: its lane 0 keeps the rows of the next kStages units
// on their way to shared memory by bulk copies (three a unit: q, k, v), so that what is
// in flight does not depend on how far the warp's arithmetic is.  8 lanes hold a row, 16
// dims each, four rows at a time.  A unit's angles are computed once, two a lane, and
// handed around by shuffles: each lane keeps the cosines and sines of its own dims in
// registers for all rows.
// Bound: HBM for many tokens (a token with 32 + 8 + 8 heads reads and writes 12 KiB
// each), latency for few.
#include "internal.h"

#include <type_traits>

#include "common.cuh"

namespace pa {
namespace {

// (8191 tokens of 32 + 8 + 8 heads, 34.8 us, 5.6 TB/s.  Rows loaded by the lanes that
// compute them, up to 12 ahead, 44 to 57 us: registers for what is in flight cost warps;
// one unit in flight and 16 warps 35.5, three and 6 warps 38.9.)
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kCtas = 2;    // resident per SM
constexpr int kStages = 2;  // units in flight per warp
constexpr int kHeads = 8;   // kv heads of a unit

// How dims pair up.  kFull: dim i with 64 + i.  kPairs: 2 i with 2 i + 1.  kPart: i with i
// + half, for i < half < 64 (half 0: nothing is rotated).
enum class Mode { kFull, kPairs, kPart };

// Lane c of a row's 8 holds dims [8 c, 8 c + 8) and [64 + 8 c, 64 + 8 c + 8): in pairs f[0
// .. 3] and f[4 .. 7].
__device__ __forceinline__ void unpack(const uint4& lo, const uint4& hi, float2 (&f)[8]) {
  f[0] = bf16x2_to_f2(lo.x); f[1] = bf16x2_to_f2(lo.y); f[2] = bf16x2_to_f2(lo.z); f[3] = bf16x2_to_f2(lo.w);
  f[4] = bf16x2_to_f2(hi.x); f[5] = bf16x2_to_f2(hi.y); f[6] = bf16x2_to_f2(hi.z); f[7] = bf16x2_to_f2(hi.w);
}
__device__ __forceinline__ uint4 pack4(const float2* f) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                    pack_bf16x2(f[3].x, f[3].y));
}
__device__ __forceinline__ float2 shfl2(float2 v, int from) {
  return make_float2(__shfl_sync(0xffffffffu, v.x, from), __shfl_sync(0xffffffffu, v.y, from));
}

// cos and sin of pair j's angle at `pos`; (1, 0) for a pair that is not rotated.
__device__ __forceinline__ float2 angle(const RopeParams& p, int pos, int j, int half) {
  float2 r = make_float2(1.f, 0.f);
  if (j >= 0 && j < half) {
    const uint32_t a = (uint32_t)(((uint64_t)(int64_t)pos * p.turns[j]) >> 32);
    // what is left of it to the nearest quarter turn: 30 bits, of which a float keeps 24
    const uint32_t quarter = (a + (1u << 29)) >> 30;
    float c, s;
    sincospif((float)(int32_t)(a - (quarter << 30)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: of half a turn
    r.x = (quarter & 1u) ? s : c;
    r.y = (quarter & 1u) ? c : s;
    if ((quarter + 1u) & 2u) r.x = -r.x;  // cos of the second and third quarter
    if (quarter & 2u) r.y = -r.y;
  }
  return r;
}

// The angles of a lane's dims.  kFull: of dims 8 c + i (and 64 + 8 c + i), pairs (2 u, 2 u +
// 1) of i in c[u], s[u].  kPairs: of the pair f[u].  kPart: c[u], s[u] for f[u]; the sine's
// sign is that of its partner's share.
template <Mode kMode>
struct Angles {
  static constexpr int kN = kMode == Mode::kPart ? 8 : 4;
  float2 c[kN], s[kN];
};

template <Mode kMode>
__device__ __forceinline__ void make_angles(const RopeParams& p, int pos, Angles<kMode>& t) {
  const int lane = threadIdx.x & 31, r = lane >> 3, c = lane & 7, half = p.rotary_dim / 2;
  if constexpr (kMode == Mode::kFull) {
    // pairs 8 c + 2 r, + 1 here; lane (u, c) has those of c[u], s[u]
    const float2 a = angle(p, pos, 8 * c + 2 * r, half), b = angle(p, pos, 8 * c + 2 * r + 1, half);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      t.c[u] = shfl2(make_float2(a.x, b.x), 8 * u + c);
      t.s[u] = shfl2(make_float2(a.y, b.y), 8 * u + c);
    }
  } else if constexpr (kMode == Mode::kPairs) {
    // f[u] (u < 4) is pair 4 c + u, f[4 + u] pair 32 + 4 c + u: as c[u], s[u] = (that, this one's)
    const float2 a = angle(p, pos, 4 * c + r, half), b = angle(p, pos, 32 + 4 * c + r, half);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      t.c[u] = shfl2(make_float2(a.x, b.x), 8 * u + c);
      t.s[u] = shfl2(make_float2(a.y, b.y), 8 * u + c);
    }
  } else {
    // chunks of 8 dims, e = c and 8 + c; with far = half / 8 chunk e < far pairs with e + far
    const int far = half / 8;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int e = 8 * x + c;
      const int j = e < far ? 8 * e : e < 2 * far ? 8 * (e - far) : -64;  // first pair of the chunk
      const float2 a = angle(p, pos, j + 2 * r, half), b = angle(p, pos, j + 2 * r + 1, half);
      const float sign = e < far ? -1.f : 1.f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        t.c[4 * x + u] = shfl2(make_float2(a.x, b.x), 8 * u + c);
        t.s[4 * x + u] = shfl2(make_float2(sign * a.y, sign * b.y), 8 * u + c);
      }
    }
  }
}

// Dims from 2 half on stay as they are: a product with cos 0 and sin 0 would make NaN of an
// infinity.  (half is a multiple of 8, so a lane's chunk of 8 dims is rotated or not as a
// whole.)
template <Mode kMode>
__device__ __forceinline__ void rotate(float2 (&f)[8], const Angles<kMode>& t, int half) {
  auto neg = [](float2 v) { return make_float2(-v.x, -v.y); };
  if constexpr (kMode == Mode::kFull) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float2 a = f[u], b = f[4 + u];
      f[u] = __ffma2_rn(a, t.c[u], neg(__fmul2_rn(b, t.s[u])));
      f[4 + u] = __ffma2_rn(b, t.c[u], __fmul2_rn(a, t.s[u]));
    }
  } else if constexpr (kMode == Mode::kPairs) {
    const int first = 4 * (threadIdx.x & 7);  // pair of f[0]; f[4]'s is 32 further
    const bool turned[2] = {first < half, 32 + first < half};
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float c = u < 4 ? t.c[u & 3].x : t.c[u & 3].y, s = u < 4 ? t.s[u & 3].x : t.s[u & 3].y;
      const float a = f[u].x, b = f[u].y;
      if (turned[u >> 2]) f[u] = make_float2(fmaf(a, c, -b * s), fmaf(b, c, a * s));
    }
  } else {
    const int lane = threadIdx.x & 31, c = lane & 7, far = half / 8;
    float2 other[8];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int e = 8 * x + c;
      const int pe = e < far ? e + far : e < 2 * far ? e - far : e;  // the partner's chunk
      const int from = (lane & 24) + (pe & 7);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 a = shfl2(f[u], from), b = shfl2(f[4 + u], from);
        other[4 * x + u] = pe >= 8 ? b : a;
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (8 * (u >> 2) + c < 2 * far) f[u] = __ffma2_rn(f[u], t.c[u], __fmul2_rn(other[u], t.s[u]));
  }
}

// The weights of a lane's dims.
__device__ __forceinline__ void load_weight(const float* w, float2 (&f)[8]) {
  const int c = threadIdx.x & 7;
#pragma unroll
  for (int u = 0; u < 8; ++u)
    f[u] = w ? reinterpret_cast<const float2*>(w)[(u < 4 ? 4 * c : 28 + 4 * c) + u] : make_float2(1.f, 1.f);
}

// A row's 16 dims of this lane, normalised (weights w) and rotated.
template <Mode kMode, bool kNorm>
__device__ __forceinline__ void row16(uint4& lo, uint4& hi, const float2 (&w)[8], const Angles<kMode>& t, int half,
                                      float eps) {
  float2 f[8];
  unpack(lo, hi, f);
  if constexpr (kNorm) {
    float2 s2 = __fmul2_rn(f[0], f[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) s2 = __ffma2_rn(f[i], f[i], s2);
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // (a Newton step: without it, and with angles to 2^-24 of half a turn, twice as many of
    // the results were rounded to the other neighbour as the formula's)
    const float v = fmaf(ss, 1.f / kHeadDim, eps);
    float q = rsqrtf(v);
    const float r = fmaf(-v * q, q, 1.f);
    if (fabsf(r) < 1.f) q = fmaf(0.5f * q, r, q);  // (not of a zero or an infinity)
    const float2 q2 = make_float2(q, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fmul2_rn(__fmul2_rn(f[i], w[i]), q2);
  }
  rotate<kMode>(f, t, half);
  lo = pack4(f);
  hi = pack4(f + 4);
}

// n rows of 256 bytes from shared memory (row i at src + 256 i) to dst + i * step
// elements, on the way normalised with `weight` (null: not) and rotated.
template <Mode kMode>
__device__ __forceinline__ void rows_through(const uint8_t* src, int n, uint16_t* dst, size_t step, const float* weight,
                                             const Angles<kMode>& t, int half, float eps) {
  const int lane = threadIdx.x & 31, r = lane >> 3, c = lane & 7;
  const uint8_t* s = src + r * (kHeadDim * 2) + 16 * c;
  uint16_t* d = dst + r * step + 8 * c;
  auto go = [&](auto norm) {
    float2 w[8];
    if constexpr (decltype(norm)::value) load_weight(weight, w);
#pragma unroll 2
    for (int i = 0; i < n; i += 4, s += 4 * kHeadDim * 2, d += 4 * step) {
      const bool live = i + r < n;
      uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
      if (live) {
        lo = *reinterpret_cast<const uint4*>(s);
        hi = *reinterpret_cast<const uint4*>(s + 128);
      }
      row16<kMode, decltype(norm)::value>(lo, hi, w, t, half, eps);
      if (live) {
        *reinterpret_cast<uint4*>(d) = lo;
        *reinterpret_cast<uint4*>(d + 64) = hi;
      }
    }
  };
  if (weight) go(std::true_type{}); else go(std::false_type{});
}

template <bool kAppend>
struct __align__(128) Smem {
  uint8_t rows[kWarps][kStages][kHeads * (kGroup + (kAppend ? 2 : 1)) * kHeadDim * 2];
  uint64_t full[kWarps][kStages];
};

template <bool kAppend, Mode kMode>
__global__ void __launch_bounds__(kThreads, kCtas) norm_rope_kernel(const RopeParams p, int heads) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<kAppend>& sm = *reinterpret_cast<Smem<kAppend>*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[warp][s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait();
  const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, half = p.rotary_dim / 2;
  const int shares = (Hkv + heads - 1) / heads;  // units of a token
  const int64_t units = p.n_tokens * shares, stride = (int64_t)gridDim.x * kWarps;
  const int64_t first = (int64_t)blockIdx.x * kWarps + warp;
  constexpr int kRow = kHeadDim * 2;
  // unit u (the warp's k-th) on its way: q's rows, then k's, then v's (lane 0)
  auto issue = [&](int64_t u, int k) {
    if (u >= units) return;
    const int64_t tok = u / shares;
    const int h0 = (int)(u - tok * shares) * heads, n = min(heads, Hkv - h0);
    uint64_t* bar = &sm.full[warp][k % kStages];
    uint8_t* dst = sm.rows[warp][k % kStages];
    mbar_arrive_expect_tx(bar, n * (kGroup + (kAppend ? 2 : 1)) * kRow);
    bulk_g2s(dst, p.q + tok * p.q_stride + (size_t)h0 * kGroup * kHeadDim, n * kGroup * kRow, bar);
    bulk_g2s(dst + n * kGroup * kRow, p.k + tok * p.k_stride + (size_t)h0 * kHeadDim, n * kRow, bar);
    if constexpr (kAppend)
      bulk_g2s(dst + n * (kGroup + 1) * kRow, p.v + tok * p.v_stride + (size_t)h0 * kHeadDim, n * kRow, bar);
  };
  if (lane == 0)
    for (int k = 0; k < kStages; ++k) issue(first + k * stride, k);
  int k = 0;
  for (int64_t u = first; u < units; u += stride, ++k) {
    const int64_t tok = u / shares;
    const int h0 = (int)(u - tok * shares) * heads, n = min(heads, Hkv - h0);
    int64_t slot = 0;
    if constexpr (kAppend) slot = p.slot_mapping[tok];
    Angles<kMode> t;
    make_angles(p, p.rotary_dim > 0 ? p.positions[tok] : 0, t);
    if (!mbar_wait_bounded(&sm.full[warp][k % kStages], (uint32_t)(k / kStages) & 1u)) {
      record_error(p.err, PA_ERR_DEVICE_TIMEOUT);
      // the copies in flight land before the warp leaves (bounded)
      for (int j = k + 1; j < k + kStages; ++j)
        if (first + j * stride < units) mbar_wait_bounded(&sm.full[warp][j % kStages], (uint32_t)(j / kStages) & 1u);
      return;
    }
    const uint8_t* rows = sm.rows[warp][k % kStages];
    rows_through(rows, n * kGroup, p.q_out + (tok * Hq + (size_t)h0 * kGroup) * kHeadDim, kHeadDim, p.q_weight, t, half,
                 p.eps);
    rows += n * kGroup * kRow;
    if constexpr (!kAppend) {
      rows_through(rows, n, p.k_out + (tok * Hkv + h0) * kHeadDim, kHeadDim, p.k_weight, t, half, p.eps);
    } else {
      const int64_t block = slot / kPage;
      if (slot >= 0 && block < p.num_blocks) {
        // a page's heads lie a slab apart
        const size_t at = ((block * Hkv + h0) * kPage + slot % kPage) * kHeadDim;
        constexpr size_t kStep = kPage * kHeadDim;
        rows_through(rows, n, p.k_cache + at, kStep, p.k_weight, t, half, p.eps);
        const int r = lane >> 4, c = lane & 15;
        for (int i = r; i < n; i += 2)
          *reinterpret_cast<uint4*>(p.v_cache + at + i * kStep + 8 * c) =
              *reinterpret_cast<const uint4*>(rows + (n + i) * kRow + 16 * c);
      } else if (slot >= 0 && lane == 0) {
        record_error(p.err, PA_ERR_DEVICE_INDEX);
      }
    }
    __syncwarp();  // every lane has read the unit
    if (lane == 0) {
      fence_proxy_async_smem();
      issue(u + kStages * stride, k + kStages);
    }
  }
}

std::atomic<bool> g_attr_set[2][3][kMaxDevices];

template <bool kAppend, Mode kMode>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  constexpr int64_t kResident = 152 * kCtas * kWarps;  // warps that the SMs hold at once
  constexpr size_t kBytes = sizeof(Smem<kAppend>);
  static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "resident CTAs");
  const cudaError_t e = set_smem_limit_once((const void*)norm_rope_kernel<kAppend, kMode>, (int)kBytes,
                                            g_attr_set[kAppend][(int)kMode]);
  if (e != cudaSuccess) return e;
  // as many kv heads a unit as leave a unit to every warp
  int heads = kHeads;
  while (heads > 1 && p.n_tokens * ((p.num_kv_heads + heads - 1) / heads) < kResident) heads /= 2;
  const int64_t units = p.n_tokens * ((p.num_kv_heads + heads - 1) / heads);
  const int64_t warps = units < kResident ? units : kResident;
  return launch_pdl(norm_rope_kernel<kAppend, kMode>, dim3((unsigned)((warps + kWarps - 1) / kWarps)), dim3(kThreads),
                    kBytes, stream, p, heads);
}

template <bool kAppend>
cudaError_t launch_mode(const RopeParams& p, bool interleaved, cudaStream_t stream) {
  if (interleaved) return launch<kAppend, Mode::kPairs>(p, stream);
  if (p.rotary_dim == kHeadDim) return launch<kAppend, Mode::kFull>(p, stream);
  return launch<kAppend, Mode::kPart>(p, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeParams& p, bool append, bool interleaved, cudaStream_t stream) {
  return append ? launch_mode<true>(p, interleaved, stream) : launch_mode<false>(p, interleaved, stream);
}

}  // namespace pa
