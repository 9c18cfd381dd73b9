// Flash-decode over 4-bit pages: rows with one query token, and rows with a
// few (verify rows).
//
// What is computed: query j of a row with n queries and L keys attends to keys
// 0 .. L - n + j; for each of the 4 query heads of a kv head, s_t = sm_scale
// <q, K_t>, out = sum_t p_t V_t / sum_t p_t with p_t = 2^(s_t log2 e - m), K_t
// and V_t the bf16 values of the page's codes (q4.cuh).
//
// Work.  As in the bf16 decode kernel the rows' pages are laid end to end for
// each kv head and cut into equal segments, one CTA per SM and segment; each
// warp streams its share of the segment through a ring of its own (asynchronous
// copies, two pages at a time), so warps never wait for one another.  A
// row cut between warps is put together in shared memory by the last of them
// to finish, a row cut between CTAs in the workspace by the last CTA; parts are
// always added in page order, so results do not depend on who came last.
//
// Arithmetic.  A page is 16 tokens, the M of one mma.m16n8k16, and four heads
// of two queries are its N: 8 products give a page's scores for 8 (query, head)
// columns, 8 its part of the output, and the 4 KiB of values exist only as the
// products' A operands, in registers, whatever the number of queries.  (The
// 5th-generation tensor cores take their operands from shared or tensor memory,
// so the values would have to be written out and read again, and M = 128 keys
// would need 8 pages per product.)  Codes arrive in operand order through 8 x 8
// matrix loads: K straight (a lane gets 8 dims of a token), V transposed (a
// lane gets 4 dims of two tokens), so that one shift, one insert and one packed
// FMA turn each pair of codes into an operand half.
//   With one query the columns of the second product come in pairs: the weight
// of a head as two bf16, its leading 8 bits and the rest, so that the idle half
// of N keeps 16 bits of every weight.  With several queries the weights are
// rounded to bf16.  Scores, sums and outputs stay in binary32.
//
// Bound.  The SMs, before memory: one does 12 to 13 pages of a kv head per us,
// ~155 cycles each, whether 88 or 152 of them run (64 rows of 2176 tokens, 8 kv
// heads: a step of 41 us, 4.9 TB/s in the page loop; one row of 131072 tokens:
// 39 us).  A page takes some 350 instructions, 164 of them on the ALU pipe, 128
// for the shift and the insert of each pair of codes; in the loop the schedulers
// issue ~70 % of the time and that pipe is ~65 % busy.  16 warps instead of 12
// take the same time.  With 5 queries it is some 490 instructions, and two warps
// per scheduler wait for one another's fixed latencies (issuing 47 % of the time):
// 70 us for the step of those 64 rows.
#include <math.h>
#include <stddef.h>

#include <chrono>

#include "internal.h"
#include "q4.cuh"

namespace pa {
namespace {

constexpr int kPair = 2;     // pages per stage
constexpr float kRescaleSlack = 8.f;  // the running max is re-based when it grows by more than 2^8
constexpr float kNoMax = 3.402823466e38f;  // the greatest binary32: any score is above its negative

struct Item {        // one row's pages within this CTA's segment
  int32_t q_start;  // first page of the item in the segment
  int32_t n;        // pages of the item in the segment
  int32_t p0;       // row page index of the item's first page
  int32_t r;        // request
  int32_t L;        // its seq_len
  int32_t tok;      // its first query token
  int32_t nq;       // its query tokens
  int32_t A;        // stream position of the row's page 0
};

// kTiles: 8-column tiles (two queries of 4 heads each); 0: one query, weights
// as two bf16.
template <int kTiles>
struct Shape {
  static constexpr bool kOne = kTiles == 0;
  static constexpr int kT = kOne ? 1 : kTiles;
  static constexpr int kCols = kOne ? 1 : 2;       // (query, head) columns per lane and tile
  static constexpr int kVec = kCols * 4;           // float4 of output values per lane and tile
  static constexpr int kTileCols = kOne ? 4 : 8;   // columns of a tile
  static constexpr int kWarps = q4_decode_warps(kTiles);
  // pages computed at once (several queries: one, for shorter code and no spilled
  // registers, 70.5 us against 71.6 for 64 rows of 5 queries and 2300 tokens)
  static constexpr int kU = kOne ? 2 : 1;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kPartBytes = kT * kVec * 32 * 16;
  static constexpr int kStages = 2;                // stages in flight per warp (a power of two)
  static constexpr int kRingBytes = kStages * kPair * 2 * kQ4Slab;
};

template <int kTiles>
struct __align__(128) Smem {
  using S = Shape<kTiles>;
  // per warp: two pages per stage, K slab and V slab; its last item's part
  // takes the ring's place at the end
  uint8_t ring[S::kWarps][S::kRingBytes > S::kPartBytes ? S::kRingBytes : S::kPartBytes];
  uint8_t part[S::kWarps][S::kPartBytes];  // a warp's part of its first item
  float part_m[S::kWarps][2][S::kT * S::kTileCols], part_l[S::kWarps][2][S::kT * S::kTileCols];
  int32_t ids[kQ4MaxPagesPerCta];
  Item items[kQ4MaxItemsPerCta];
  int arrived[kQ4MaxItemsPerCta];  // warps done with their part of the item
  int n_items;
};
static_assert(sizeof(Smem<0>) <= 227 * 1024 && sizeof(Smem<2>) <= 227 * 1024 && sizeof(Smem<3>) <= 227 * 1024,
              "one CTA per SM");
static_assert(kQ4Slab % 128 == 0 && Shape<3>::kPartBytes % 128 == 0,
              "matrix-load rows of a slab meet the banks as laid out in q4.cuh");

// A warp's part (slot 0: of its first item, 1: of its last), [tile][vector][lane].
template <int kTiles>
__device__ __forceinline__ float4* part_of(Smem<kTiles>& sm, int warp, int slot) {
  return reinterpret_cast<float4*>(slot == 0 ? sm.part[warp] : sm.ring[warp]);
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
__device__ __forceinline__ void store_row(uint16_t* row, const float (&o)[16], int r, bool used) {
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
    if (used)
      *reinterpret_cast<uint4*>(row + 32 * (g + (odd ? 2 : 0)) + 8 * (r >> 1)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// One tile's columns of this lane: maximum, weight sum and 16 unnormalised
// values per column (vector v = 4 col + group: 4 dims).
template <int kCols>
struct Part {
  float m[kCols], l[kCols];
  float4 o[4 * kCols];
};

// Log-sum-exp merge of n parts, in order.  m_at(i, c), l_at(i, c): maximum (-inf:
// nothing counts, NaN: nor does any other part) and weight sum of column c of
// this lane in part i; row(i): the part's vectors of
// this lane at stride 32.  The loads of a batch of parts are all in flight
// before any is used.
template <int kCols, class M, class L, class Row>
__device__ __forceinline__ void merge_parts(Part<kCols>& out, int n, int lane, M&& m_at, L&& l_at, Row&& row) {
#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    out.m[c] = -INFINITY;
    out.l[c] = 0.f;
  }
#pragma unroll
  for (int v = 0; v < 4 * kCols; ++v) out.o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = kCols == 1 ? 4 : 2;
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    float4 x[kBatch][4 * kCols];
    float mi[kBatch][kCols], li[kBatch][kCols];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = min(i0 + u, n - 1);
      const float4* src = row(i);
#pragma unroll
      for (int v = 0; v < 4 * kCols; ++v) x[u][v] = src[32 * v + lane];
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        mi[u][c] = i0 + u < n ? m_at(i, c) : -INFINITY;
        li[u][c] = l_at(i, c);
      }
    }
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      float mx = out.m[c];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) mx = max_nan(mx, mi[u][c]);
      if (mx == -INFINITY) continue;  // every part so far is empty
      const float f = fast_exp2(out.m[c] - mx);  // -inf -> 0
      out.m[c] = mx;
      out.l[c] *= f;
#pragma unroll
      for (int v = 4 * c; v < 4 * c + 4; ++v)
        out.o[v] = make_float4(out.o[v].x * f, out.o[v].y * f, out.o[v].z * f, out.o[v].w * f);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float w = fast_exp2(mi[u][c] - mx);
        out.l[c] = fmaf(w, li[u][c], out.l[c]);
#pragma unroll
        for (int v = 4 * c; v < 4 * c + 4; ++v) {
          out.o[v].x = fmaf(w, x[u][v].x, out.o[v].x);
          out.o[v].y = fmaf(w, x[u][v].y, out.o[v].y);
          out.o[v].z = fmaf(w, x[u][v].z, out.o[v].z);
          out.o[v].w = fmaf(w, x[u][v].w, out.o[v].w);
        }
      }
    }
  }
}

template <int kTiles, class Plan>
__global__ void __launch_bounds__(Shape<kTiles>::kThreads, 1)
    decode_q4_kernel(const DecodeParams p, const __grid_constant__ Plan plan) {
  using S = Shape<kTiles>;
  constexpr int kThreads = S::kThreads, kWarps = S::kWarps, kT = S::kT, kCols = S::kCols, kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<kTiles>& sm = *reinterpret_cast<Smem<kTiles>*>(smem_raw);
  const int b = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hkv = p.num_kv_heads;
  const int kvh = b % Hkv, sidx = b / Hkv;
  const int S0 = sidx * plan.seg;
  const int npg = min(plan.total, S0 + plan.seg) - S0;  // pages of this CTA's segment (by_row: at most)
  if (npg <= 0) return;
  for (int i = tid; i < kQ4MaxItemsPerCta; i += kThreads) sm.arrived[i] = 0;
  // ---- item table of the segment (one warp, 32 rows per round); it comes
  // from the kernel parameters alone, so it is built before the wait for the
  // previous kernel
  if (warp == 1) {
    const int2 at = plan.start[sidx];  // first row and its first page
    int base_q = 0, n_it = 0;
    for (int k0 = 0; k0 < kQ4MaxItemsPerCta; k0 += 32) {
      const int item = at.x + k0 + lane;
      const int p0 = (k0 + lane == 0) ? at.y : 0;
      int4 row = make_int4(0, 0, 0, 0);  // request, seq_len, first query token, queries
      int size = 0;
      if (item < plan.n_rows && (!plan.by_row || item == at.x)) {
        row = plan.row[item];
        size = max((row.y + kPage - 1) / kPage - p0, 0);
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
        it.r = row.x;
        it.L = row.y;
        it.tok = row.z;
        it.nq = row.w;
        it.A = S0 + start - p0;
      }
      const unsigned covered = __ballot_sync(0xffffffffu, in_seg);
      const int lead = (~covered == 0u) ? 32 : (__ffs((int)~covered) - 1);
      n_it = k0 + lead;
      base_q += __shfl_sync(0xffffffffu, incl, 31);
      if (lead < 32 || base_q >= npg) break;
    }
    if (lane == 0) {
      if (base_q < npg && !plan.by_row) record_error(p.err, PA_ERR_DEVICE_INDEX);  // not planned on the host
      sm.n_items = n_it;
    }
  }
  __syncthreads();
  // Beside a tile kernel (p.beside) this launch starts once every CTA of that
  // kernel has passed its own wait, so the kernels before it are complete;
  // waiting here would wait for the tile kernel itself.
  if (!p.beside) pdl_wait();
  const int n_items = sm.n_items;
  if (n_items == 0) return;  // nothing covered (recorded above)
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
  // slab of the page `half` of stage s: K, then V one slab further
  auto slab_at = [&](int s, int half) { return sm.ring[warp] + (s * kPair + half) * (2 * kQ4Slab); };
  // Pages a + 2 i and a + 2 i + 1 -> stage i % kStages, one copy group per call
  // (empty past the end).  A lane copies bytes 512 c + 16 lane of each page's
  // two slabs laid end to end; a page with a bad id is fetched from block 0 and
  // does not count.  (One bulk copy per slab instead: 246 us against 230 for 8
  // rows of 131072 tokens; copies of 1280 bytes start too slowly.)
  const int n_pairs = (e - a + kPair - 1) / kPair;
  auto issue = [&](int i) {
#pragma unroll
    for (int h = 0; h < kPair; ++h) {
      const int q = a + kPair * i + h;
      if (q < e) {
        const size_t off = ((size_t)max(sm.ids[q], 0) * Hkv + kvh) * kQ4Slab + 16 * lane;
        const uint8_t* ks = kbase + off;
        const uint8_t* vs = vbase + off;
        const uint32_t dst = smem_addr(slab_at(i % kStages, h)) + 16 * lane;
        static_assert(kQ4Slab == 1280, "five copies per lane, the third from both slabs");
        copy16(dst, ks);
        copy16(dst + 512, ks + 512);
        copy16(dst + 1024, lane < 16 ? ks + 1024 : vs - 256);
        copy16(dst + 1536, vs + 256);
        copy16(dst + 2048, vs + 768);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) issue(i);

  // The pieces of a row cut between CTAs lie in the workspace: segments b0 ..
  // b1 hold the row, and each CTA's piece of it is its last item's or its
  // first's.  The pieces that have arrived are counted in a word beside the
  // first one, tag << 16 | count.  Every CTA of the row makes sure before it
  // adds its piece that the word carries this launch's tag, so what the workspace
  // held before (from calls of other shapes, or not cleared) does not matter.
  constexpr int kSlots = q4_piece_slots(kTiles);
  auto first_seg = [&](const Item& it) { return it.A / plan.seg; };
  auto piece_at = [&](const Item& it, int bb) {
    const int b0 = first_seg(it);
    return ((size_t)(bb * Hkv + kvh) * 2 + ((bb == b0 && b0 * plan.seg < it.A) ? 1 : 0)) * kSlots;
  };
  auto cut = [&](const Item& it) { return it.p0 != 0 || it.n != (it.L + kPage - 1) / kPage; };
  // (the host sized the workspace: never false)
  auto piece_fits = [&](const Item& it) { return (int64_t)(piece_at(it, sidx) + kSlots) <= p.piece_slots; };
  auto word_of = [&](const Item& it) {
    return reinterpret_cast<unsigned long long*>(p.piece_lse + piece_at(it, first_seg(it)) + kSlots - 2);
  };
  if (lane < 2 && n_items > lane) {  // (while the first pages are on their way)
    const Item& it = sm.items[lane == 0 ? n_items - 1 : 0];
    if (it.q_start / sw == warp && cut(it) && piece_fits(it)) {  // the item's first warp
      unsigned long long* word = word_of(it);
      const unsigned long long was = *reinterpret_cast<volatile unsigned long long*>(word);
      if (was >> 16 != plan.tag) atomicCAS(word, was, (unsigned long long)plan.tag << 16);
    }
  }
  __syncwarp();

  const int r = lane >> 2;   // token slot (r, r + 8) in the scores; dim row in the output
  const int cq = lane & 3;   // the lane's columns in scores and output: head cq, or 2 cq and 2 cq + 1
  // matrix-load address of lane l: matrix (group) l / 8, row (token) l % 8
  const uint32_t ld_at = (uint32_t)q4_code_at(lane & 7, lane >> 3);

  for (; k < n_items; ++k) {
    const Item it = sm.items[k];
    const int i0 = max(it.q_start, a), i1 = min(it.q_start + it.n, e);
    if (i0 >= i1) break;  // past this warp's pages
    const int L = it.L, nq = it.nq;
    const int page0 = it.p0 - it.q_start;  // row page of segment page q: page0 + q
    // keys the lane's columns of tile y see (columns past the last query: all)
    auto sees = [&](int y) { return S::kOne ? L : min(L - nq + 2 * y + (cq >> 1) + 1, L); };
    // q as the first product's B operand: column n of tile y is query 2 y + n
    // / 4, head n % 4 (one query: column 2 h is head h, column 2 h + 1 zeros);
    // k step (g, e) takes dims 32 g + 8 cq + 4 e .. + 3
    uint4 qb[kT][4];
#pragma unroll
    for (int y = 0; y < kT; ++y) {
      const int query = S::kOne ? 0 : 2 * y + (r >> 2), head = S::kOne ? r >> 1 : r & 3;
      const bool used = S::kOne ? (r & 1) == 0 : query < nq;
      const uint16_t* qrow =
          p.q + ((size_t)(it.tok + (used ? query : 0)) * p.num_q_heads + (size_t)kvh * kGroup + head) * kHeadDim + 8 * cq;
#pragma unroll
      for (int g = 0; g < 4; ++g)
        qb[y][g] = used ? *reinterpret_cast<const uint4*>(qrow + 32 * g) : make_uint4(0u, 0u, 0u, 0u);
    }
    float acc[kT][4][2][4];
#pragma unroll
    for (int y = 0; y < kT; ++y)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[y][g][x][i] = 0.f;
    // per column: minus the running max (the same in the column's 8 lanes; a
    // huge number before the first key, so that nothing weighs anything) and
    // the sum of this lane's own weights
    float nm[kT][kCols], l[kT][kCols];
#pragma unroll
    for (int y = 0; y < kT; ++y)
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        nm[y][c] = kNoMax;
        l[y][c] = 0.f;
      }

    for (int q = i0; q < i1;) {
      const int j = q - a, i = j / kPair, s = i % kStages;
      cp_async_wait<kStages - 1>();  // this lane's copies of pair i
      __syncwarp();                  // and the others'
      // two pages at once where the pair lies in the row, else one: page 0 is
      // q, page 1 its neighbour in the stage, of which no token counts then
      const int half = j & 1, n = (S::kU == 2 && half == 0 && q + 1 < i1) ? 2 : 1;
      int pos[kPair];  // row position of each page's first token (L: the page does not count)
      pos[0] = (page0 + q) * kPage;
      pos[1] = n == 1 ? L : pos[0] + kPage;
      if (!ids_ok) {
        if (sm.ids[q] < 0) pos[0] = L;
        if (n == 2 && sm.ids[q + 1] < 0) pos[1] = L;
      }
      // every token of both pages counts for every column
      const bool whole = (S::kU == 2 ? max(pos[0], pos[1]) : pos[0]) + kPage <= L - nq + 1;
      const uint32_t st = smem_addr(slab_at(s, half)), step = half ? 0u - 2 * kQ4Slab : 2u * kQ4Slab;
      // ---- scores: tokens r and r + 8 of the lane's columns, of both pages
      float sc[kT][kCols][2 * S::kU];
#pragma unroll
      for (int u = 0; u < S::kU; ++u) {
        const uint32_t ks = st + u * step;
        float c[kT][4];
#pragma unroll
        for (int y = 0; y < kT; ++y) c[y][0] = c[y][1] = c[y][2] = c[y][3] = 0.f;
        float c2[kT][4];  // a second accumulator: two shorter chains of products
#pragma unroll
        for (int y = 0; y < kT; ++y) c2[y][0] = c2[y][1] = c2[y][2] = c2[y][3] = 0.f;
        uint32_t ka[4], kb[4];
        ldmatrix4(ka, ks + ld_at);
        ldmatrix4(kb, ks + ld_at + 8 * kQ4Row);
        const uint4 za = lds128(ks + kQ4Codes + 16 * r), zb = lds128(ks + kQ4Codes + 16 * (r + 8));
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t da = q4_dup_d(at(za, g)), oa = q4_dup_z(at(za, g));
          const uint32_t db = q4_dup_d(at(zb, g)), ob = q4_dup_z(at(zb, g));
          const uint32_t a0 = bf16x2_fma(q4_unit_pair<0>(ka[g]), da, oa), a1 = bf16x2_fma(q4_unit_pair<0>(kb[g]), db, ob);
          const uint32_t a2 = bf16x2_fma(q4_unit_pair<1>(ka[g]), da, oa), a3 = bf16x2_fma(q4_unit_pair<1>(kb[g]), db, ob);
          const uint32_t a4 = bf16x2_fma(q4_unit_pair<2>(ka[g]), da, oa), a5 = bf16x2_fma(q4_unit_pair<2>(kb[g]), db, ob);
          const uint32_t a6 = bf16x2_fma(q4_unit_pair<3>(ka[g]), da, oa), a7 = bf16x2_fma(q4_unit_pair<3>(kb[g]), db, ob);
#pragma unroll
          for (int y = 0; y < kT; ++y) {
            mma16816(c[y], a0, a1, a2, a3, qb[y][g].x, qb[y][g].y);
            mma16816(c2[y], a4, a5, a6, a7, qb[y][g].z, qb[y][g].w);
          }
        }
#pragma unroll
        for (int y = 0; y < kT; ++y)
#pragma unroll
          for (int x = 0; x < kCols; ++x) {
            sc[y][x][2 * u] = (c[y][x] + c2[y][x]) * p.scale_log2;
            sc[y][x][2 * u + 1] = (c[y][2 + x] + c2[y][2 + x]) * p.scale_log2;
          }
      }
      if (!whole) {
#pragma unroll
        for (int y = 0; y < kT; ++y) {
          const int vis = sees(y);
#pragma unroll
          for (int u = 0; u < S::kU; ++u)
#pragma unroll
            for (int x = 0; x < kCols; ++x) {
              if (pos[u] + r >= vis) sc[y][x][2 * u] = -INFINITY;
              if (pos[u] + r + 8 >= vis) sc[y][x][2 * u + 1] = -INFINITY;
            }
        }
      }
      float mx[kT][kCols];
      bool grow = false;
#pragma unroll
      for (int y = 0; y < kT; ++y)
#pragma unroll
        for (int x = 0; x < kCols; ++x) {
          mx[y][x] = fmaxf(sc[y][x][0], sc[y][x][1]);
          if constexpr (S::kU == 2) mx[y][x] = fmaxf(mx[y][x], fmaxf(sc[y][x][2], sc[y][x][3]));
          grow = grow || mx[y][x] + nm[y][x] > kRescaleSlack;
        }
      if (__any_sync(0xffffffffu, grow)) {  // rare after the first pages
#pragma unroll
        for (int y = 0; y < kT; ++y)
#pragma unroll
          for (int x = 0; x < kCols; ++x) {
            float t = mx[y][x];
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
            if (t + nm[y][x] > kRescaleSlack) {
              const float corr = fast_exp2(-nm[y][x] - t);  // the first time 0
              nm[y][x] = -t;
              l[y][x] *= corr;
#pragma unroll
              for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int v = 0; v < 4; ++v)
                    if (S::kOne || (v & 1) == x) acc[y][g][h][v] *= corr;
            }
          }
      }
      // weights, transposed into the second product's B operand
      uint32_t pb[kT][2 * S::kU];
#pragma unroll
      for (int y = 0; y < kT; ++y)
#pragma unroll
        for (int u = 0; u < 2 * S::kU; ++u) {
          const float w0 = fast_exp2(sc[y][0][u] + nm[y][0]);
          l[y][0] += w0;
          if constexpr (S::kOne) {  // leading bits, rest
            const float h = __uint_as_float(__float_as_uint(w0) & 0xffff0000u);
            pb[y][u] = movmatrix_trans(pack_bf16x2(h, w0 - h));
          } else {
            const float w1 = fast_exp2(sc[y][kCols - 1][u] + nm[y][kCols - 1]);
            l[y][kCols - 1] += w1;
            pb[y][u] = movmatrix_trans(pack_bf16x2(w0, w1));
          }
        }
      // ---- output: dims of row r of each group's words, tokens 2 cq, 2 cq +
      // 1 and the same + 8
#pragma unroll
      for (int u = 0; u < S::kU; ++u) {
        const uint32_t vs = st + u * step + kQ4Slab;
        uint32_t va[4], vb[4];
        ldmatrix4_trans(va, vs + ld_at);
        ldmatrix4_trans(vb, vs + ld_at + 8 * kQ4Row);
        const uint32_t sp = vs + kQ4Codes + 32 * cq;
        uint4 z0 = lds128(sp), z1 = lds128(sp + 16), z2 = lds128(sp + 128), z3 = lds128(sp + 144);
        if (!whole) {  // a token past the end has weight 0: its values must be finite
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          const int left = L - pos[u];
          if (2 * cq >= left) z0 = zero;
          if (2 * cq + 1 >= left) z1 = zero;
          if (2 * cq + 8 >= left) z2 = zero;
          if (2 * cq + 9 >= left) z3 = zero;
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t da = __byte_perm(at(z0, g), at(z1, g), 0x5410), oa = __byte_perm(at(z0, g), at(z1, g), 0x7632);
          const uint32_t db = __byte_perm(at(z2, g), at(z3, g), 0x5410), ob = __byte_perm(at(z2, g), at(z3, g), 0x7632);
          const uint32_t a0 = bf16x2_fma(q4_unit_pair<0>(va[g]), da, oa), a1 = bf16x2_fma(q4_unit_pair<1>(va[g]), da, oa);
          const uint32_t a2 = bf16x2_fma(q4_unit_pair<0>(vb[g]), db, ob), a3 = bf16x2_fma(q4_unit_pair<1>(vb[g]), db, ob);
          const uint32_t a4 = bf16x2_fma(q4_unit_pair<2>(va[g]), da, oa), a5 = bf16x2_fma(q4_unit_pair<3>(va[g]), da, oa);
          const uint32_t a6 = bf16x2_fma(q4_unit_pair<2>(vb[g]), db, ob), a7 = bf16x2_fma(q4_unit_pair<3>(vb[g]), db, ob);
#pragma unroll
          for (int y = 0; y < kT; ++y) {
            mma16816(acc[y][g][0], a0, a1, a2, a3, pb[y][2 * u], pb[y][2 * u + 1]);
            mma16816(acc[y][g][1], a4, a5, a6, a7, pb[y][2 * u], pb[y][2 * u + 1]);
          }
        }
      }
      q += n;
      // the pair is done with: refill its stage
      if ((q - a) % kPair == 0) {
        __syncwarp();
        issue((q - a) / kPair - 1 + kStages);
      }
    }

    // ---- this warp's part of the item: in a column, value 4 g + i is dim 32 g
    // + 8 (r / 2) + r % 2 + 2 i, unnormalised
    Part<kCols> own[kT];
#pragma unroll
    for (int y = 0; y < kT; ++y)
#pragma unroll
      for (int x = 0; x < kCols; ++x) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) l[y][x] += __shfl_xor_sync(0xffffffffu, l[y][x], o);
        // (without a maximum the sum is 0, or NaN from scores that were NaN)
        own[y].m[x] = nm[y][x] == kNoMax ? l[y][x] - INFINITY : -nm[y][x];
        own[y].l[x] = l[y][x];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float(&c)[2][4] = acc[y][g];
          own[y].o[4 * x + g] = S::kOne ? make_float4(c[0][0] + c[0][1], c[0][2] + c[0][3], c[1][0] + c[1][1],
                                                      c[1][2] + c[1][3])
                                        : make_float4(c[0][x], c[0][2 + x], c[1][x], c[1][2 + x]);
        }
      }
    const bool is_cut = cut(it);  // between CTAs
    const int wf = it.q_start / sw, wl = (it.q_start + it.n - 1) / sw;  // warps holding the item
    if (wf != wl) {
      const int slot = it.q_start <= a ? 0 : 1;  // the warp's first item, or its last
      float4* mine = part_of(sm, warp, slot);
      __syncwarp();  // every lane has read the ring
#pragma unroll
      for (int y = 0; y < kT; ++y) {
#pragma unroll
        for (int v = 0; v < S::kVec; ++v) mine[(y * S::kVec + v) * 32 + lane] = own[y].o[v];
        if (r == 0) {
#pragma unroll
          for (int x = 0; x < kCols; ++x) {
            sm.part_m[warp][slot][y * S::kTileCols + kCols * cq + x] = own[y].m[x];
            sm.part_l[warp][slot][y * S::kTileCols + kCols * cq + x] = own[y].l[x];
          }
        }
      }
      __syncwarp();
      int last = 0;
      if (lane == 0) {
        __threadfence_block();
        last = atomicAdd(&sm.arrived[k], 1) == wl - wf;
        __threadfence_block();
      }
      __syncwarp();  // lane 0's fence orders every lane's reads of the parts below (a shuffle orders no memory)
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
    }
    const int b0 = first_seg(it), b1 = (it.A + (L + kPage - 1) / kPage - 1) / plan.seg;
    if (is_cut && !piece_fits(it)) {
      if (lane == 0) record_error(p.err, PA_ERR_DEVICE_INDEX);
      continue;
    }
    auto output = [&](int y, const Part<kCols>& v) {
#pragma unroll
      for (int x = 0; x < kCols; ++x) {
        const int col = kCols * cq + x;  // of the tile
        const int query = S::kOne ? 0 : 2 * y + (col >> 2), head = S::kOne ? col : col & 3;
        const float inv = v.l[x] == 0.f ? 0.f : 1.f / v.l[x];
        float o[16];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          o[4 * g] = v.o[4 * x + g].x * inv;
          o[4 * g + 1] = v.o[4 * x + g].y * inv;
          o[4 * g + 2] = v.o[4 * x + g].z * inv;
          o[4 * g + 3] = v.o[4 * x + g].w * inv;
        }
        const size_t orow = (size_t)(it.tok + query) * p.num_q_heads + kvh * kGroup + head;
        store_row(p.out + orow * kHeadDim, o, r, query < nq);
        if (p.lse && r == 0 && query < nq)
          p.lse[orow] = lse_log2(v.m[x], v.l[x]) * kLn2;
      }
    };
#pragma unroll
    for (int y = 0; y < kT; ++y) {
      if (wf != wl)  // in page order, whichever warp came last
        merge_parts<kCols>(
            own[y], wl - wf + 1, lane,
            [&](int i, int c) {
              return sm.part_m[wf + i][it.q_start <= (wf + i) * sw ? 0 : 1][y * S::kTileCols + kCols * cq + c];
            },
            [&](int i, int c) {
              return sm.part_l[wf + i][it.q_start <= (wf + i) * sw ? 0 : 1][y * S::kTileCols + kCols * cq + c];
            },
            [&](int i) { return part_of(sm, wf + i, it.q_start <= (wf + i) * sw ? 0 : 1) + y * S::kVec * 32; });
      if (!is_cut) {
        output(y, own[y]);
        continue;
      }
      const size_t mine = piece_at(it, sidx) + y * S::kTileCols;
      float4* dst = reinterpret_cast<float4*>(p.piece_o + mine * kHeadDim);
#pragma unroll
      for (int x = 0; x < kCols; ++x) {
        const float inv = own[y].l[x] == 0.f ? 0.f : 1.f / own[y].l[x];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float4 v = own[y].o[4 * x + g];
          dst[(4 * x + g) * 32 + lane] = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        }
        if (r == 0)
          p.piece_lse[mine + kCols * cq + x] = lse_log2(own[y].m[x], own[y].l[x]);
      }
    }
    if (!is_cut) continue;
    __syncwarp();  // every lane's writes precede lane 0's release
    int last = 0;
    if (lane == 0) {
      unsigned long long* word = word_of(it);
      last = (int)(atom_add64_acq_rel_gpu(word, 1ull) & 0xffffu) == b1 - b0;
      if (last) *word = 0;  // every piece has arrived: ready for the next replay with this tag
    }
    __syncwarp();  // lane 0's acquire orders the reads below
    if (!__shfl_sync(0xffffffffu, last, 0)) continue;
#pragma unroll 1
    for (int y = 0; y < kT; ++y) {
      Part<kCols> all;
      merge_parts<kCols>(
          all, b1 - b0 + 1, lane,
          [&](int i, int c) { return load_cg(p.piece_lse + piece_at(it, b0 + i) + y * S::kTileCols + kCols * cq + c); },
          [&](int, int) { return 1.f; },
          [&](int i) {
            return reinterpret_cast<const float4*>(p.piece_o + (piece_at(it, b0 + i) + y * S::kTileCols) * kHeadDim);
          });
      output(y, all);
    }
  }
  // beside a tile kernel: this launch completes after it (the last thing that
  // the warps with pages do; one of them is enough)
  if (p.beside) pdl_wait();
}

std::atomic<bool> g_attr_set[6][kMaxDevices];

template <int kTiles, class Plan>
cudaError_t launch(const DecodeParams& p, const Plan& plan, int grid, bool overlap, std::atomic<bool>* done,
                   cudaStream_t stream) {
  constexpr int kSmem = (int)sizeof(Smem<kTiles>);
  const cudaError_t e = set_smem_limit_once((const void*)decode_q4_kernel<kTiles, Plan>, kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_maybe_pdl(overlap, decode_q4_kernel<kTiles, Plan>, dim3(grid), dim3(Shape<kTiles>::kThreads), kSmem,
                          stream, p, plan);
}

// The plan in a parameter block of the size it needs, 24 KiB or 3: four short
// rows 7.1 us with the small one against 7.2 to 7.3, and up to 1.4 us less on the
// host; most batches fit it.
template <int kTiles>
cudaError_t launch_tiles(const DecodeParams& p, const DecodePlan& plan, const int32_t* n_q, int grid, bool by_row,
                         bool overlap, std::atomic<bool>* done, cudaStream_t stream) {
  const int segs = grid / p.num_kv_heads;
  auto fill = [&](auto& d) {
    d.n_rows = plan.n_rows;
    d.seg = plan.seg;
    d.total = plan.total;
    d.by_row = by_row ? 1 : 0;
    d.tag = next_tag();
    for (int i = 0; i < plan.n_rows; ++i) d.row[i] = make_int4(plan.rows[i], plan.seq[i], plan.tok[i], n_q[i]);
    for (int i = 0; i < segs; ++i) d.start[i] = make_int2(plan.first_row[i], plan.first_page[i]);
  };
  if (plan.n_rows <= 128 && segs <= 160) {
    Q4Plan<128, 160> small;
    fill(small);
    return launch<kTiles>(p, small, grid, overlap, done, stream);
  }
  static thread_local Q4Plan<kPlanMaxRows, kPlanMaxCtas> large;
  fill(large);
  return launch<kTiles>(p, large, grid, overlap, done + kMaxDevices, stream);
}

}  // namespace

// A tag that no earlier launch of this process has had, and that other data
// are as good as never: 47 bits of a scrambled count (the finalizer of the
// splitmix64 generator), never 0.
uint64_t next_tag() {
  static std::atomic<uint64_t> count{
      (uint64_t)std::chrono::system_clock::now().time_since_epoch().count()};
  uint64_t z = count.fetch_add(1, std::memory_order_relaxed) * 0x9e3779b97f4a7c15ull;
  z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
  z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
  z ^= z >> 31;
  return z >> 17 | uint64_t(1) << 47;
}

cudaError_t launch_decode_q4(const DecodeParams& p, const DecodePlan& plan, const int32_t* n_q, int tiles, int grid,
                             bool by_row, bool overlap, cudaStream_t stream) {
  std::atomic<bool>* done = &g_attr_set[0][0];
  if (tiles == 0) return launch_tiles<0>(p, plan, n_q, grid, by_row, overlap, done, stream);
  if (tiles <= 2) return launch_tiles<2>(p, plan, n_q, grid, by_row, overlap, done + 2 * kMaxDevices, stream);
  return launch_tiles<3>(p, plan, n_q, grid, by_row, overlap, done + 4 * kMaxDevices, stream);
}

}  // namespace pa
