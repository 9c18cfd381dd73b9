// Flash-decode over 4-bit pages (rows with one query token).
//
// What is computed: for a decode row and each of the 4 query heads of a kv
// head, s_t = sm_scale <q, K_t> over the row's keys, out = sum_t p_t V_t /
// sum_t p_t with p_t = 2^(s_t log2 e - m), K_t and V_t the bf16 values of the
// page's codes (q4.cuh).
//
// Work.  As in the bf16 decode kernel the rows' pages are laid end to end for
// each kv head and cut into equal segments, one CTA of 16 warps per SM and
// segment; each warp streams its sixteenth of the segment through a ring of
// its own (two 1280-byte bulk copies per page), so warps never wait for one
// another.  A row cut between warps is put together in shared memory by the
// last of them to finish, a row cut between CTAs in the workspace by the last
// CTA.
//
// Arithmetic.  A page is 16 tokens, the M of one mma.m16n8k16, and the four
// heads fill half of its N: 8 products give the page's scores, 8 the page's
// part of the output, and the 4 KiB of values exist only as the products' A
// operands, in registers.  (The 5th-generation tensor cores take their
// operands from shared or tensor memory, so the values would have to be
// written out and read again, and M = 128 keys would need 8 pages per product;
// the products here are 7 % of the issue slots.)  Codes arrive in operand
// order through 8 x 8 matrix loads: K straight (a lane gets 8 dims of a
// token), V transposed (a lane gets 4 dims of two tokens), so that one shift,
// one insert and one packed FMA turn each pair of codes into an operand half.
//   Columns 2 h and 2 h + 1 of the second product carry the weight of head h
// as two bf16, its leading 8 bits and the rest, which the idle half of N takes
// for nothing: the weights keep 16 bits, scores, sums and output stay in
// binary32.
#include <math.h>
#include <stddef.h>

#include "internal.h"
#include "q4.cuh"

namespace pa {
namespace {

constexpr int kWarps = kQ4Warps;
constexpr int kThreads = kWarps * 32;
#ifndef Q4_PAIR
#define Q4_PAIR 2
#endif
#ifndef Q4_STAGES
#define Q4_STAGES 2
#endif
constexpr int kPair = Q4_PAIR;  // pages per stage
constexpr int kStages = Q4_STAGES;  // stages in flight per warp
constexpr float kRescaleSlack = 8.f;  // the running max is re-based when it grows by more than 2^8

struct Item {        // one row's pages within this CTA's segment
  int32_t q_start;  // first page of the item in the segment
  int32_t n;        // pages of the item in the segment
  int32_t p0;       // row page index of the item's first page
  int32_t r;        // request
  int32_t L;        // its seq_len
  int32_t tok;      // its query token
  int32_t A;        // stream position of the row's page 0
};

struct __align__(128) Smem {
  uint8_t ring[kWarps][kStages][kPair][2][kQ4Slab];  // two pages per stage, K slab and V slab
  // a warp's part of its first item, 16 values per lane; the part of its last
  // one goes where its ring was
  float4 part_o[kWarps][4][32];
  float part_m[kWarps][2][kGroup], part_l[kWarps][2][kGroup];
  uint64_t full[kWarps][kStages];
  int32_t ids[kQ4MaxPagesPerCta];
  Item items[kQ4MaxItemsPerCta];
  int arrived[kQ4MaxItemsPerCta];  // warps done with their part of the item
  int n_items;
};
static_assert(sizeof(float4) * 4 * 32 <= sizeof(Smem::ring[0]), "a part fits a warp's ring");
static_assert(sizeof(Smem) <= 227 * 1024, "one CTA per SM");
static_assert(kQ4Slab % 128 == 0, "matrix-load rows of a slab meet the banks as laid out in q4.cuh");

__device__ __forceinline__ float4* part_of(Smem& sm, int warp, int slot) {
  return slot == 0 ? &sm.part_o[warp][0][0] : reinterpret_cast<float4*>(sm.ring[warp]);
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 8 x 8 matrix of b16 held as a fragment -> the fragment of its transpose
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// D (16 x 8 fp32) += A (16 x 16 bf16) B (16 x 8 bf16)
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t at(const uint4& v, int g) { return g == 0 ? v.x : g == 1 ? v.y : g == 2 ? v.z : v.w; }

// An output row (head of this lane, 16 dims per lane as described at the
// kernel's epilogue) as bf16: lanes r and r ^ 1 hold the even and the odd dims
// of the same words and exchange halves, so each stores 8 neighbouring dims of
// two groups.
__device__ __forceinline__ void store_row(uint16_t* row, const float (&o)[16], int r) {
  const bool odd = r & 1;
  float mine[8], other[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mine[i] = odd ? o[8 + i] : o[i];
    other[i] = __shfl_xor_sync(0xffffffffu, odd ? o[i] : o[8 + i], 4);
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = mine[4 * g + i], b = other[4 * g + i];
      w[i] = odd ? pack_bf16x2(b, a) : pack_bf16x2(a, b);
    }
    *reinterpret_cast<uint4*>(row + 32 * (g + (odd ? 2 : 0)) + 8 * (r >> 1)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Running log-sum-exp merge of parts of one head (16 values per lane).
struct Merge {
  float m = -INFINITY, l = 0.f;
  float o[16] = {};
  // a part with maximum (or lse) m2, weight sum l2 and values x
  __device__ __forceinline__ void add(float m2, float l2, const float4 (&x)[4]) {
    const float mn = fmaxf(m, m2);
    if (mn == -INFINITY) return;
    const float f = fast_exp2(m - mn), f2 = fast_exp2(m2 - mn);
    l = l * f + l2 * f2;
    m = mn;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[4 * i] = fmaf(f2, x[i].x, o[4 * i] * f);
      o[4 * i + 1] = fmaf(f2, x[i].y, o[4 * i + 1] * f);
      o[4 * i + 2] = fmaf(f2, x[i].z, o[4 * i + 2] * f);
      o[4 * i + 3] = fmaf(f2, x[i].w, o[4 * i + 3] * f);
    }
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    decode_q4_kernel(const DecodeParams p, const __grid_constant__ DecodePlan plan) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int b = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hkv = p.num_kv_heads;
  const int kvh = b % Hkv, sidx = b / Hkv;
  const int S0 = sidx * plan.seg;
  const int npg = min(plan.total, S0 + plan.seg) - S0;  // pages of this CTA's segment
  if (npg <= 0) return;
  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[w][s], 1);
    fence_mbar_init();
  }
  for (int i = tid; i < kQ4MaxItemsPerCta; i += kThreads) sm.arrived[i] = 0;
  // ---- item table of the segment (one warp, 32 rows per round); it comes
  // from the kernel parameters alone, so it is built before the wait for the
  // previous kernel
  if (warp == 1) {
    int base_q = 0, n_it = 0;
    for (int k0 = 0; k0 < kQ4MaxItemsPerCta; k0 += 32) {
      const int item = plan.first_row[sidx] + k0 + lane;
      const bool exists = item < plan.n_rows;
      int r = 0, L = 0, size = 0, tok = 0;
      const int p0 = (k0 + lane == 0) ? plan.first_page[sidx] : 0;
      if (exists) {
        r = plan.rows[item];
        L = plan.seq[item];
        tok = plan.tok[item];
        size = max((L + kPage - 1) / kPage - p0, 0);
      }
      int incl = size;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const int start = base_q + incl - size;
      const bool in_seg = size > 0 && start < npg;
      if (in_seg) {
        Item& it = sm.items[k0 + lane];
        it.q_start = start;
        it.n = min(size, npg - start);
        it.p0 = p0;
        it.r = r;
        it.L = L;
        it.tok = tok;
        it.A = S0 + start - p0;
      }
      const unsigned covered = __ballot_sync(0xffffffffu, in_seg);
      const int lead = (~covered == 0u) ? 32 : (__ffs((int)~covered) - 1);
      n_it = k0 + lead;
      base_q += __shfl_sync(0xffffffffu, incl, 31);
      if (lead < 32 || base_q >= npg) break;
    }
    if (lane == 0) {
      if (base_q < npg) record_error(p.err, PA_ERR_DEVICE_INDEX);  // metadata differ from the plan
      sm.n_items = n_it;
    }
  }
  __syncthreads();
  pdl_wait();
  const int n_items = sm.n_items;
  if (n_items == 0) return;  // nothing covered (recorded above); no copy was issued
  // ---- block ids of the segment's pages; a page with an id outside the pool
  // (or past the table) is recorded and skipped
  const int n_cov = sm.items[n_items - 1].q_start + sm.items[n_items - 1].n;
  int ok = 1;
  for (int q = tid; q < n_cov; q += kThreads) {
    int lo = 0, hi = n_items - 1;
    while (lo < hi) {  // last item with q_start <= q
      const int mid = (lo + hi + 1) >> 1;
      if (sm.items[mid].q_start <= q) lo = mid; else hi = mid - 1;
    }
    int32_t blk = -1;
    const Item& it = sm.items[lo];
    const int page = it.p0 + (q - it.q_start);
    if (page < p.max_blocks_per_req) blk = p.block_tables[(size_t)it.r * p.max_blocks_per_req + page];
    if (blk < 0 || blk >= p.num_blocks) {
      record_error(p.err, PA_ERR_DEVICE_INDEX);
      blk = -1;
      ok = 0;
    }
    sm.ids[q] = blk;
  }
  const bool ids_ok = __syncthreads_and(ok) != 0;

  // ---- this warp's pages [a, e) of the segment
  const int sw = plan.seg / kWarps;
  const int a = warp * sw, e = min(a + sw, n_cov);
  if (a >= e) return;
  int k = 0;  // the item holding page a
  {
    int lo = 0, hi = n_items - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sm.items[mid].q_start <= a) lo = mid; else hi = mid - 1;
    }
    k = lo;
  }
  const uint8_t* kbase = reinterpret_cast<const uint8_t*>(p.k_cache);
  const uint8_t* vbase = reinterpret_cast<const uint8_t*>(p.v_cache);
  // Pages a + 2 i and a + 2 i + 1 -> stage i % kStages.  Lanes 0 .. 3 issue the
  // K and V slab of the two pages; a page with a bad id is fetched from block 0
  // and does not count.
  const int n_pairs = (e - a + kPair - 1) / kPair;
  auto issue = [&](int i) {
    if (lane < 2 * kPair) {
      const int s = i % kStages, q = a + kPair * i + (lane >> 1);
      if (lane == 0) mbar_arrive_expect_tx(&sm.full[warp][s], (kPair == 2 && q + 1 < e ? 4 : 2) * kQ4Slab);
      if (q < e) {
        const size_t off = ((size_t)max(sm.ids[q], 0) * Hkv + kvh) * kQ4Slab;
        bulk_g2s(sm.ring[warp][s][lane >> 1][lane & 1], ((lane & 1) ? vbase : kbase) + off, kQ4Slab, &sm.full[warp][s]);
      }
    }
  };
  for (int i = 0; i < min(n_pairs, kStages); ++i) issue(i);

  const int r = lane >> 2;   // token slot (r, r + 8) in the scores; dim row in the output
  const int cq = lane & 3;   // the lane's head in scores and output
  // matrix-load address of lane l: matrix (group) l / 8, row (token) l % 8
  const uint32_t ld_at = (uint32_t)q4_code_at(lane & 7, lane >> 3);
  int issued = min(n_pairs, kStages);
  bool gave_up = false;

  for (; k < n_items; ++k) {
    const Item it = sm.items[k];
    const int i0 = max(it.q_start, a), i1 = min(it.q_start + it.n, e);
    if (i0 >= i1) break;  // past this warp's pages
    const int pages_r = (it.L + kPage - 1) / kPage;
    const int tail = it.L - (pages_r - 1) * kPage;  // tokens of the row's last page
    const int q_last = it.q_start + (pages_r - 1 - it.p0);
    // q as the first product's B operand: column 2 h holds head h (column
    // 2 h + 1 zeros); k step (g, e) takes dims 32 g + 8 cq + 4 e .. + 3
    uint4 qb[4];
    {
      const uint16_t* qrow =
          p.q + ((size_t)it.tok * p.num_q_heads + (size_t)kvh * kGroup + (lane >> 3)) * kHeadDim + 8 * cq;
#pragma unroll
      for (int g = 0; g < 4; ++g)
        qb[g] = (r & 1) ? make_uint4(0u, 0u, 0u, 0u) : *reinterpret_cast<const uint4*>(qrow + 32 * g);
    }
    float acc[4][2][4];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[g][x][i] = 0.f;
    // running max of head cq (the same in its 8 lanes), minus it (0 before
    // the first key), and the sum of this lane's own weights
    float m = -INFINITY, nm = 0.f, l = 0.f;

    for (int q = i0; q < i1;) {
      const int j = q - a, i = j / kPair, s = i % kStages;
      if (!mbar_wait_bounded(&sm.full[warp][s], (uint32_t)(i / kStages) & 1u)) {
        record_error(p.err, PA_ERR_DEVICE_TIMEOUT);
        gave_up = true;
        break;
      }
      // two pages at once where the pair lies in the row, else one: page 0 is
      // q, page 1 its neighbour in the stage, of which no token counts then
      const int half = kPair == 2 ? j & 1 : 0, n = (kPair == 2 && half == 0 && q + 1 < i1) ? 2 : 1;
      int live[kPair];  // tokens of each page that count
      live[0] = q == q_last ? tail : kPage;
      if (kPair == 2) live[kPair - 1] = n == 1 ? 0 : q + 1 == q_last ? tail : kPage;
      if (!ids_ok) {
        if (sm.ids[q] < 0) live[0] = 0;
        if (n == 2 && sm.ids[q + 1] < 0) live[kPair - 1] = 0;
      }
      const uint32_t st = smem_addr(sm.ring[warp][s][half]), step = half ? 0u - 2 * kQ4Slab : 2u * kQ4Slab;
      // ---- scores: tokens r and r + 8 of head cq, of both pages
      float sc[2 * kPair];
#pragma unroll
      for (int u = 0; u < kPair; ++u) {
        const uint32_t ks = st + u * step;
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t ka[4], kb[4];
        ldmatrix4(ka, ks + ld_at);
        ldmatrix4(kb, ks + ld_at + 8 * kQ4Row);
        const uint4 za = lds128(ks + kQ4Codes + 16 * r), zb = lds128(ks + kQ4Codes + 16 * (r + 8));
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t da = q4_dup_d(at(za, g)), oa = q4_dup_z(at(za, g));
          const uint32_t db = q4_dup_d(at(zb, g)), ob = q4_dup_z(at(zb, g));
          mma16816(c, bf16x2_fma(q4_unit_pair<0>(ka[g]), da, oa), bf16x2_fma(q4_unit_pair<0>(kb[g]), db, ob),
                   bf16x2_fma(q4_unit_pair<1>(ka[g]), da, oa), bf16x2_fma(q4_unit_pair<1>(kb[g]), db, ob), qb[g].x,
                   qb[g].y);
          mma16816(c, bf16x2_fma(q4_unit_pair<2>(ka[g]), da, oa), bf16x2_fma(q4_unit_pair<2>(kb[g]), db, ob),
                   bf16x2_fma(q4_unit_pair<3>(ka[g]), da, oa), bf16x2_fma(q4_unit_pair<3>(kb[g]), db, ob), qb[g].z,
                   qb[g].w);
        }
        sc[2 * u] = c[0] * p.scale_log2;
        sc[2 * u + 1] = c[2] * p.scale_log2;
      }
      const bool whole = live[0] == kPage && live[kPair - 1] == kPage;
      if (!whole) {
#pragma unroll
        for (int u = 0; u < kPair; ++u) {
          if (r >= live[u]) sc[2 * u] = -INFINITY;
          if (r + 8 >= live[u]) sc[2 * u + 1] = -INFINITY;
        }
      }
      float mx = fmaxf(sc[0], sc[1]);
      if (kPair == 2) mx = fmaxf(mx, fmaxf(sc[2 * kPair - 2], sc[2 * kPair - 1]));
      if (__any_sync(0xffffffffu, mx > m + kRescaleSlack)) {  // rare after the first pages
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (mx > m + kRescaleSlack) {
          const float corr = fast_exp2(m - mx);  // m = -inf -> 0
          m = mx;
          nm = -mx;
          l *= corr;
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int y = 0; y < 4; ++y) acc[g][x][y] *= corr;
        }
      }
      // weights as two bf16 each (leading bits, rest), transposed into the
      // second product's B operand
      uint32_t pb[2 * kPair];
#pragma unroll
      for (int u = 0; u < 2 * kPair; ++u) {
        const float w = fast_exp2(sc[u] + nm);
        l += w;
        const float h = __uint_as_float(__float_as_uint(w) & 0xffff0000u);
        pb[u] = movmatrix_trans(pack_bf16x2(h, w - h));
      }
      // ---- output: dims of row r of each group's words, tokens 2 cq, 2 cq +
      // 1 and the same + 8
#pragma unroll
      for (int u = 0; u < kPair; ++u) {
        const uint32_t vs = st + u * step + kQ4Slab;
        uint32_t va[4], vb[4];
        ldmatrix4_trans(va, vs + ld_at);
        ldmatrix4_trans(vb, vs + ld_at + 8 * kQ4Row);
        const uint32_t sp = vs + kQ4Codes + 32 * cq;
        uint4 z0 = lds128(sp), z1 = lds128(sp + 16), z2 = lds128(sp + 128), z3 = lds128(sp + 144);
        if (!whole) {  // a token that does not count has weight 0: its values must be finite
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          if (2 * cq >= live[u]) z0 = zero;
          if (2 * cq + 1 >= live[u]) z1 = zero;
          if (2 * cq + 8 >= live[u]) z2 = zero;
          if (2 * cq + 9 >= live[u]) z3 = zero;
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t da = __byte_perm(at(z0, g), at(z1, g), 0x5410), oa = __byte_perm(at(z0, g), at(z1, g), 0x7632);
          const uint32_t db = __byte_perm(at(z2, g), at(z3, g), 0x5410), ob = __byte_perm(at(z2, g), at(z3, g), 0x7632);
          mma16816(acc[g][0], bf16x2_fma(q4_unit_pair<0>(va[g]), da, oa), bf16x2_fma(q4_unit_pair<1>(va[g]), da, oa),
                   bf16x2_fma(q4_unit_pair<0>(vb[g]), db, ob), bf16x2_fma(q4_unit_pair<1>(vb[g]), db, ob), pb[2 * u],
                   pb[2 * u + 1]);
          mma16816(acc[g][1], bf16x2_fma(q4_unit_pair<2>(va[g]), da, oa), bf16x2_fma(q4_unit_pair<3>(va[g]), da, oa),
                   bf16x2_fma(q4_unit_pair<2>(vb[g]), db, ob), bf16x2_fma(q4_unit_pair<3>(vb[g]), db, ob), pb[2 * u],
                   pb[2 * u + 1]);
        }
      }
      q += n;
      // the pair is done with: refill its stage
      if ((q - a) % kPair == 0) {
        __syncwarp();
        if (issued < n_pairs) {
          fence_proxy_async_smem();
          issue(issued);
          ++issued;
        }
      }
    }
    if (gave_up) break;

    // ---- this warp's part of the item: head cq, value 4 g + i is dim 32 g +
    // 8 (r / 2) + r % 2 + 2 i, unnormalised
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float4 x[4];
#pragma unroll
    for (int g = 0; g < 4; ++g)
      x[g] = make_float4(acc[g][0][0] + acc[g][0][1], acc[g][0][2] + acc[g][0][3], acc[g][1][0] + acc[g][1][1],
                         acc[g][1][2] + acc[g][1][3]);
    Merge mg;
    const int wf = it.q_start / sw, wl = (it.q_start + it.n - 1) / sw;  // warps holding the item
    if (wf == wl) {
      mg.add(m, l, x);
    } else {
      const int slot = it.q_start <= a ? 0 : 1;  // the warp's first item, or its last
      float4* mine = part_of(sm, warp, slot);
      __syncwarp();  // every lane has read the ring
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[32 * i + lane] = x[i];
      if (r == 0) {
        sm.part_m[warp][slot][cq] = m;
        sm.part_l[warp][slot][cq] = l;
      }
      __syncwarp();
      int last = 0;
      if (lane == 0) {
        __threadfence_block();
        last = atomicAdd(&sm.arrived[k], 1) == wl - wf;
        __threadfence_block();
      }
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      for (int w = wf; w <= wl; ++w) {  // in page order, whichever warp came last
        const int sl = it.q_start <= w * sw ? 0 : 1;
        float4 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = part_of(sm, w, sl)[32 * i + lane];
        mg.add(sm.part_m[w][sl][cq], sm.part_l[w][sl][cq], y);
      }
    }
    const size_t orow = (size_t)it.tok * p.num_q_heads + kvh * kGroup + cq;
    if (it.p0 != 0 || it.n != pages_r) {
      // the row is cut between CTAs: publish this one's piece; the last CTA
      // to do so merges them
      const float inv = mg.l > 0.f ? 1.f / mg.l : 0.f;
      const float lse2 = mg.l > 0.f ? mg.m + log2f(mg.l) : -INFINITY;
      const int b0 = it.A / plan.seg, b1 = (it.A + pages_r - 1) / plan.seg;  // segments holding the row
      auto piece_at = [&](int bb) {
        const int j = (bb == b0 && b0 * plan.seg < it.A) ? 1 : 0;  // a segment's last item, or its first
        return ((size_t)(bb * Hkv + kvh) * 2 + j) * kGroup;
      };
      const size_t mine = piece_at(sidx);
      if ((int64_t)(mine + kGroup) > p.piece_slots) {  // the host sized the workspace for fewer pieces
        if (lane == 0) record_error(p.err, PA_ERR_DEVICE_INDEX);
        continue;
      }
      float4* dst = reinterpret_cast<float4*>(p.piece_o + mine * kHeadDim);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dst[32 * i + lane] =
            make_float4(mg.o[4 * i] * inv, mg.o[4 * i + 1] * inv, mg.o[4 * i + 2] * inv, mg.o[4 * i + 3] * inv);
      if (r == 0) p.piece_lse[mine + cq] = lse2;
      __syncwarp();  // every lane's writes precede lane 0's release
      int last = 0;
      if (lane == 0) {
        int* cnt = p.counters + (size_t)it.r * Hkv + kvh;
        last = atom_add_acq_rel_gpu(cnt, 1) == b1 - b0;
        if (last) *cnt = 0;  // every piece has arrived: ready for the next call
      }
      __syncwarp();  // lane 0's acquire orders the reads below
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      Merge all;
      for (int bb = b0; bb <= b1; ++bb) {
        const size_t src = piece_at(bb);
        const float4* y4 = reinterpret_cast<const float4*>(p.piece_o + src * kHeadDim);
        float4 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __ldcg(y4 + 32 * i + lane);
        all.add(__ldcg(p.piece_lse + src + cq), 1.f, y);
      }
      mg = all;
    }
    const float inv = mg.l > 0.f ? 1.f / mg.l : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) mg.o[i] *= inv;
    store_row(p.out + orow * kHeadDim, mg.o, r);
    if (p.lse && r == 0) p.lse[orow] = mg.l > 0.f ? (mg.m + log2f(mg.l)) * kLn2 : -INFINITY;
  }

  if (gave_up && lane == 0) {
    // a wait ran out: let the last copies issued into each stage land
    // (bounded), then leave
    for (int i = max(0, issued - kStages); i < issued; ++i)
      mbar_wait_bounded(&sm.full[warp][i % kStages], (uint32_t)(i / kStages) & 1u);
  }
}

std::atomic<bool> g_attr_set[kMaxDevices];

}  // namespace

cudaError_t launch_decode_q4(const DecodeParams& p, const DecodePlan& plan, int grid, bool overlap,
                             cudaStream_t stream) {
  const cudaError_t e = set_smem_limit_once((const void*)decode_q4_kernel, (int)sizeof(Smem), g_attr_set);
  if (e != cudaSuccess) return e;
  return launch_maybe_pdl(overlap, decode_q4_kernel, dim3(grid), dim3(kThreads), sizeof(Smem), stream, p, plan);
}

}  // namespace pa
