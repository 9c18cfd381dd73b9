// Decode with a sliding window: rows of 1 to 6 queries over the pages they see.
//
// What is computed: the query at position p sees keys t <= p with t < sinks or t > p -
// window; softmax attention over these.  Scores, maxima, sums and outputs in
// binary32; log2 domain.
//
// Work.  A row's visible pages (leading ones, then the window's) are counted through,
// and for each kv head all rows' pages form one stream that is cut into equal segments,
// one for each gang of a CTA's warps (one gang, or two where rows are many and short);
// with few rows each row is cut into pieces of its own instead, so that no CTA needs the
// other rows' lengths.  The plan is made on the device from the
// lengths (one load per row and a scan), so the launch depends on scalars alone.
//
// Bound: HBM (2 FMA per byte of K and V and query).  A segment's pages go to the gang's
// consumer warps in turn; each warp keeps its next ones in flight in a ring of its own, by
// asynchronous 16-byte copies that place the 16-byte chunks of a row of 64 dims at c ^
// (row mod 8), so that matrix loads meet no bank twice.
//   Products: mma.sync m16n8k16 with keys as M.  A page is 16 keys: S^T = K Q^T has
// M = 16 keys, N = 8 columns (a column is a query and one of the 4 heads of the group),
// O^T += V^T P^T has M = 16 dims, so K and V are the A operands as they lie in shared
// memory, and a page costs 16 products per 8 columns.  tcgen05 would want 64 or 128 keys
// or rows at once: with 4 to 24 rows it would wait for 8 pages and idle on 80 % of its
// M.
//   The weights of one query fill half of N = 8, those of two queries one of two
// column tiles; the other half takes what their rounding to bf16 left (16 bits in all).
// Three queries and more are rounded to bf16 once, as the tile kernel rounds them.
//   Maxima are looked at only when a score exceeds its column's reference by 2^8
// (one vote a page), so sums stay far inside binary32.
//   At a row's end each consumer warp leaves its partial sums in shared memory and goes
// on with the next row; two or three merging warps put them together behind it.  A row cut between
// CTAs leaves one partial per CTA in the workspace; the last CTA to arrive at the row's
// count merges them in order: results do not depend on timing.  The counts carry a tag of the
// launch, which every CTA of the row makes sure of before it adds to one, so that what the
// workspace held before does not matter: the pieces of batches of other sizes lie where the
// counts of this one do.  Both merges work out
// what each part counts for all columns at once, a lane a column, and then add up several
// columns' sums at a time: a column after another, each with its own reductions and
// loads, a row of 5 queries kept a CTA for 6 us (80 rows of 5 queries, 1024 keys: 76.3 us;
// 69.1 with the first, 61.5 with both and a row's q fetched by copies all in flight, 59.1
// with three merging warps for two).
//
// Measured (GB300, in a graph, bytes of the pages seen over time): 64 rows of 1 query,
// 1028 keys 47.5 us; 80 rows of 1, 2, 4, 5 queries, 4096 keys 6.8, 6.8, 6.6, 6.5 TB/s.
// Of seven and more queries the products would take the time (5.3 TB/s): the tile kernel's.
#include <math.h>
#include <stddef.h>

#include <algorithm>

#include "internal.h"
#include "q4.cuh"  // load_cg, max_nan, lse_log2
#include "window.cuh"
#include "window_mend.cuh"

namespace pa {
namespace {

constexpr float kSlack = 8.f;        // log2 of the largest weight against a column's reference
constexpr int kOStride = kHeadDim + 4;  // floats between columns of a partial: stores meet no bank twice
constexpr int kQStride = kHeadDim + 8;  // bf16 between rows of q: matrix loads meet no bank twice

// NT: tiles of 8 columns (2 queries).  Consumer warps, pages in flight of each, and
// partial buffers fill the shared memory; up to 8 warps in all a thread has 255 registers,
// which three tiles need, up to 12 it has 168.  Measured (with two merging warps), 80 rows,
// 1024 keys, us: 2 tiles, 8 warps x 2 pages 63.8, 7 x 2 63.9, 5 x 4 65.3; 3 tiles, 4 x 4
// 67.8, 4 x 3 68.9, 5 x 3 70.9, 5 x 2 71.9.  Two warps that share a ring's pages and split
// the columns load each page's fragments twice: 111 for 85.6 then.
template <int NT, int kGangs>
struct Cfg {
  static constexpr int kQueries = NT == 1 ? 1 : 2 * NT;
  static constexpr int kCols = kQueries * kGroup;
  static constexpr int kWarps = NT <= 2 ? 8 : 4;
  static constexpr int kStages = NT <= 2 ? 2 : 4;
  static constexpr int kBufs = NT == 1 ? 2 : 1;
  static constexpr bool kQRegs = NT <= 2;  // q's fragments kept in registers
  // the CTA's warps as kGangs gangs, each with a segment, merging warps and a q of its own
  static constexpr int kGang = kWarps / kGangs;                          // consumer warps of a gang
  static constexpr int kMergeWarps = kGangs == 2 ? 1 : NT == 1 ? 2 : 3;  // every so many-th column each
  static constexpr int kThreads = (kWarps + kGangs * (kMergeWarps + 1)) * 32;
  static_assert(kMergeWarps <= kWindowMergeWarps && kGangs <= kWindowGangs, "counts, pieces");
};

template <int NT, int kGangs>
struct __align__(1024) Smem {
  using C = Cfg<NT, kGangs>;
  uint8_t page[C::kWarps][C::kStages][4][kPage * 128];  // K dims 0-63, 64-127, V dims 0-63, 64-127
  uint16_t q[kGangs][2][8 * NT][kQStride];  // a row's q by column (columns without a query: anything)
  float o[C::kBufs][C::kWarps][C::kCols][kOStride];
  float m[C::kBufs][C::kWarps][C::kCols], l[C::kBufs][C::kWarps][C::kCols];
  uint64_t q_full[kGangs][2], q_free[kGangs][2];
  uint64_t part_full[kGangs][C::kBufs], part_free[kGangs][C::kBufs];
  int start[kPlanMaxRows + 1];  // pages of the rows before
  int len[kPlanMaxRows], tok[kPlanMaxRows];
  uint8_t n_q[kPlanMaxRows];
  int scan[32];
  int abort;
};

// (The loop is a function of its own: code at every wait's place that the instruction
// caches need not take along.)
__device__ __noinline__ bool wait_on(int* abort, uint64_t* bar, uint32_t parity, int* err) {
  const unsigned long long t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*reinterpret_cast<volatile int*>(abort)) return false;
      if (globaltimer() - t0 > kWaitLimitNs) {
        record_error(err, PA_ERR_DEVICE_TIMEOUT);
        *reinterpret_cast<volatile int*>(abort) = 1;
        return false;
      }
    }
  }
}
template <class S>
__device__ __forceinline__ bool wait(S& sm, uint64_t* bar, uint32_t parity, int* err) {
  return mbar_try_wait(bar, parity) || wait_on(&sm.abort, bar, parity, err);
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A row's part of a CTA's pages.
struct Item {
  int r, L, n, tok;  // request, its keys, queries, first query token
  int i0, i1;        // pages of the CTA (counted from its first)
  int v0;            // which of the row's visible pages page i0 is
  int count;         // the row's visible pages
  int s0, pieces;    // the first segment that holds any of them; how many do
  int slot;          // 0: the CTA's first row, 1: another
};

// The rows of a CTA's segment, one after another.  pieces > 0: each row is cut into
// that many segments of its own (at most; of 8 pages at least).
template <int NT, int kGangs>
struct Rows {
  const WindowParams& p;
  const Smem<NT, kGangs>& sm;
  int S, E, seg, d, per_row, sidx;
  __device__ __forceinline__ Rows(const WindowParams& p_, const Smem<NT, kGangs>& sm_, int S_, int E_, int seg_, int d_, int per,
                                  int sidx_)
      : p(p_), sm(sm_), S(S_), E(E_), seg(seg_), d(d_), per_row(per), sidx(sidx_) {}
  __device__ __forceinline__ bool next(Item& it) {
    while (d < p.rows) {
      const int a = sm.start[d], b = sm.start[d + 1];
      if (a >= E) return false;
      if (b > S && b > a) {
        it.r = p.row0 + d;
        it.L = sm.len[d];
        it.n = sm.n_q[d];
        it.tok = sm.tok[d];
        it.i0 = max(a, S) - S;
        it.i1 = min(b, E) - S;
        it.v0 = max(S - a, 0);
        it.count = b - a;
        if (per_row) {
          it.s0 = sidx / per_row * per_row;
          it.pieces = (b - a + seg - 1) / seg;
          it.slot = 0;
          d = p.rows - 1;  // the CTA has one row
        } else {
          it.s0 = a / seg;
          it.pieces = (b - 1) / seg - it.s0 + 1;
          it.slot = a < S || a == sidx * seg ? 0 : 1;
        }
        ++d;
        return true;
      }
      ++d;
    }
    return false;
  }
};

// Row d of the launch: its pages (0: nothing to do), queries, first query token; L < 0
// in a padding row whose output this launch writes.
struct RowInfo {
  int pages, L, n, tok;
};
template <int NT, int kGangs>
__device__ __forceinline__ RowInfo row_info(const WindowParams& p, int d, bool first_cta) {
  const int r = p.row0 + d;
  RowInfo x{0, 0, 1, r};
  if (p.qo_indptr) {
    x.tok = p.qo_indptr[r];
    x.n = p.qo_indptr[r + 1] - x.tok;
  }
  x.L = p.seq_lens[r];
  if (x.n < 1 || x.n > kWindowDecodeQueries) return x;  // no row of this kernel
  if (x.tok < 0 || x.tok > p.total_q - x.n) {  // (not what the host copy says)
    if (first_cta) record_error(p.err, PA_ERR_DEVICE_INDEX);
    return x;
  }
  if (x.L < x.n || x.L > PA_MAX_SEQ_LEN || (x.L + kPage - 1) / kPage > p.max_blocks_per_req || x.n > Cfg<NT, kGangs>::kQueries) {
    if (x.L != 0 && first_cta) record_error(p.err, PA_ERR_DEVICE_INDEX);
    x.L = -1;  // padding
    return x;
  }
  x.pages = seen_pages(x.L, x.n, p.window, p.sink_tokens).count();
  return x;
}

template <int NT, int kGangs>
__global__ void __launch_bounds__(Cfg<NT, kGangs>::kThreads, 1)
    decode_window_kernel(const __grid_constant__ WindowParams p) {
  using C = Cfg<NT, kGangs>;
  extern __shared__ uint8_t smem_raw[];
  Smem<NT, kGangs>& sm = *reinterpret_cast<Smem<NT, kGangs>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // the warp's gang: consumers, then merging warps, then the warps that fetch q
  const int past = warp - C::kWarps, fetch = past - kGangs * C::kMergeWarps;
  const int gang = past < 0 ? warp / C::kGang : fetch < 0 ? past / C::kMergeWarps : fetch;
  const int Hkv = p.num_kv_heads, kvh = (int)blockIdx.x % Hkv, sidx = (int)blockIdx.x / Hkv * kGangs + gang;
  const int nseg = (int)gridDim.x / Hkv * kGangs;
  if (tid == 0) {
    for (int x = 0; x < kGangs; ++x) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sm.q_full[x][b], 1);
        mbar_init(&sm.q_free[x][b], C::kGang);
      }
      for (int b = 0; b < C::kBufs; ++b) {
        mbar_init(&sm.part_full[x][b], C::kGang);
        mbar_init(&sm.part_free[x][b], C::kMergeWarps);
      }
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  // ---- the plan: every row's pages, laid end to end
  const int per_row = kGangs == 1 ? p.per_row : 0, per = kGangs == 1 ? per_row : 1;  // (per: > 0 where it divides)
  int total = 0, S, E, seg, d0 = 0;
  constexpr int kPer = (kPlanMaxRows + C::kThreads - 1) / C::kThreads;
  if (per_row > 0) {
    // rows cut into per_row segments: this CTA has one row
    const int d = sidx / per;
    if (d >= p.rows) return;
    if (tid == 0) {
      const RowInfo x = row_info<NT, kGangs>(p, d, kvh == 0 && sidx == d * per_row);
      sm.start[d] = 0;
      sm.start[d + 1] = x.pages;
      sm.len[d] = x.L;
      sm.tok[d] = x.tok;
      sm.n_q[d] = (uint8_t)x.n;
    }
    __syncthreads();
    total = sm.start[d + 1];
    seg = max(8, (total + per - 1) / per);
    S = (sidx - d * per_row) * seg;
    E = min(S + seg, total);
    d0 = d;
    if (total == 0 && sm.len[d] <= 0 && sidx == d * per_row) {  // padding: defined outputs
      const size_t row = (size_t)sm.tok[d] * p.num_q_heads + kvh * kGroup;
      if (!p.qo_indptr) {
        if (tid < kGroup * kHeadDim * 2 / 16)
          reinterpret_cast<uint4*>(p.out + row * kHeadDim)[tid] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse && tid < kGroup) p.lse[row + tid] = -INFINITY;
      }
    }
    if (S >= E) return;
  } else {
    int own = 0, pages[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = tid * kPer + i;
      pages[i] = 0;
      if (d < p.rows) {
        const RowInfo x = row_info<NT, kGangs>(p, d, blockIdx.x == 0);
        pages[i] = x.pages;
        sm.len[d] = x.L;
        sm.tok[d] = x.tok;
        sm.n_q[d] = (uint8_t)x.n;
        if (x.pages == 0 && x.L <= 0 && !p.qo_indptr && (int)blockIdx.x / Hkv == d % (nseg / kGangs)) {  // padding: defined outputs
          const size_t row = (size_t)x.tok * p.num_q_heads + kvh * kGroup;
          uint4* o = reinterpret_cast<uint4*>(p.out + row * kHeadDim);
          for (int j = 0; j < kGroup * kHeadDim * 2 / 16; ++j) o[j] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse)
            for (int g = 0; g < kGroup; ++g) p.lse[row + g] = -INFINITY;
        }
      }
      own += pages[i];
    }
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    int before = incl - own;
#pragma unroll
    for (int w = 0; w < C::kThreads / 32; ++w) {
      const int y = sm.scan[w];
      before += w < warp ? y : 0;
      total += y;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = tid * kPer + i;
      if (d < p.rows) sm.start[d] = before;
      before += pages[i];
      if (d == p.rows - 1) sm.start[p.rows] = before;
    }
    __syncthreads();
    seg = max(8, (total + nseg - 1) / nseg);
    S = sidx * seg;
    E = min(S + seg, total);
    if (S >= E) return;
    int lo = 0, hi = p.rows - 1;  // the last row that starts at or before S
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sm.start[mid] <= S) lo = mid; else hi = mid - 1;
    }
    d0 = lo;
  }
  const int n_pages = E - S;
  Rows<NT, kGangs> rows(p, sm, S, E, seg, d0, per_row, sidx);
  Item it;

  if (fetch >= 0) {
    // --------------------------------------------------- each row's queries
    for (int n_item = 0; rows.next(it); ++n_item) {
      const int b = n_item & 1;
      if (n_item >= 2 && !__all_sync(0xffffffffu, wait(sm, &sm.q_free[gang][b], ((n_item >> 1) - 1) & 1, p.err))) return;
      for (int i = lane; i < it.n * kGroup * (kHeadDim / 8); i += 32) {  // all in flight at once
        const int col = i / (kHeadDim / 8), ch = i % (kHeadDim / 8);
        const uint16_t* src = p.q + ((size_t)(it.tok + col / kGroup) * p.num_q_heads + kvh * kGroup + col % kGroup) * kHeadDim;
        cp_async16(&sm.q[gang][b][col][8 * ch], src + 8 * ch);
      }
      cp_async_commit();
      cp_async_wait<0>();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[gang][b]);
    }
  } else if (warp < C::kWarps) {
    // ----------------------------------------------------------- consumers
    // The warp's pages are i = gw + kGang k, k = 0 .. n_own - 1.  Slabs of 32 of them by
    // lane, a batch ahead: which (block, kv head); -1: outside the pool
    const int gw = warp % C::kGang;
    const int n_own = (n_pages - gw + C::kGang - 1) / C::kGang;
    auto load_ids = [&](int k0) -> int {
      const int i = gw + C::kGang * (k0 + lane);
      if (i >= n_pages) return 0;
      int lo = d0, hi = per_row ? d0 : p.rows - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sm.start[mid] <= S + i) lo = mid; else hi = mid - 1;
      }
      const Seen seen = seen_pages(sm.len[lo], sm.n_q[lo], p.window, p.sink_tokens);
      const int page = seen.page(S + i - sm.start[lo]);
      const int b = p.block_tables[(size_t)(p.row0 + lo) * p.max_blocks_per_req + page];
      if (b < 0 || b >= p.num_blocks) {
        record_error(p.err, PA_ERR_DEVICE_INDEX);
        return -1;
      }
      return b;
    };
    int ids = load_ids(0), ids_next = load_ids(32);  // of batches kb, kb + 1 (kb: of the page being issued)
    uint32_t bad = 0;  // bit k mod 32: page k (of the last ones issued) is outside the pool
    // lane's 16-byte chunk of every second row of a slab: row r0 + 2 j, chunk ch of its 16
    const int r0 = lane >> 4, ch = lane & 15;
    // page k into stage k mod kStages (one group of copies, empty past the end)
    auto issue = [&](int k) {
      if (k < n_own) {
        if (k > 0 && (k & 31) == 0) {
          ids = ids_next;
          ids_next = load_ids(k + 32);
        }
        const int b = __shfl_sync(0xffffffffu, ids, k & 31);
        bad = (bad & ~(1u << (k & 31))) | (b < 0 ? 1u << (k & 31) : 0u);
        if (b >= 0) {
          const size_t at = ((size_t)b * Hkv + kvh) * (kPage * kHeadDim) + lane * 8;
          uint8_t* dst = sm.page[warp][k % C::kStages][ch >> 3];
#pragma unroll
          for (int j = 0; j < kPage / 2; ++j) {
            const int row = r0 + 2 * j;
            const int to = row * 128 + (((ch & 7) ^ (row & 7)) << 4);
            cp_async16(dst + to, p.k_cache + at + j * 2 * kHeadDim);
            cp_async16(dst + 2 * kPage * 128 + to, p.v_cache + at + j * 2 * kHeadDim);
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < C::kStages; ++k) issue(k);
    int k = 0;
    const int g = lane >> 2, c = lane & 3;  // fragments: key or dim g (and g + 8), columns 2 c, 2 c + 1
    // matrix loads: lane's row of a page and 16-byte chunk parity, K and V
    const int k_row = (lane & 7) + ((lane >> 3) & 1) * 8, k_ch = lane >> 4;
    const int v_row = (lane & 7) + (lane >> 4) * 8, v_ch = (lane >> 3) & 1;
    for (int n_item = 0; rows.next(it); ++n_item) {
      const int qb = n_item & 1;
      if (!__all_sync(0xffffffffu, wait(sm, &sm.q_full[gang][qb], (n_item >> 1) & 1, p.err))) break;
      // q as the B operand, columns 8 t .. 8 t + 7 (matrix loads: column lane mod 8, dims
      // 32 y + 8 (lane / 8) on).  One query: columns 4 .. 7 again (for what rounding
      // leaves); two: tile 1 is tile 0
      auto q_at = [&](int t, int y) {
        const int col = it.n == 1 ? lane & 3 : it.n == 2 && t == 1 ? lane & 7 : 8 * t + (lane & 7);
        return smem_addr(&sm.q[gang][qb][col][32 * y + 8 * (lane >> 3)]);
      };
      uint32_t qf[C::kQRegs ? NT : 1][4][4];
      if constexpr (C::kQRegs) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int y = 0; y < 4; ++y) ldsm4(qf[t][y], q_at(t, y));
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_free[gang][qb]);
      }
      const Seen seen = seen_pages(it.L, it.n, p.window, p.sink_tokens);
      const int p0 = it.L - it.n;  // position of the first query
      const int low = max(p0 - p.window + 1, 0);
      float m[NT][2], l[NT][2], o[8][NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        m[t][0] = m[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int y = 0; y < 4; ++y) o[mt][t][y] = 0.f;
      }
      const int k_first = k;
      for (int i; (i = gw + C::kGang * k) < it.i1; ++k) {
        cp_async_wait<C::kStages - 1>();
        __syncwarp();  // every lane's copies have landed
        if ((bad >> (k & 31)) & 1u) {
          issue(k + C::kStages);
          continue;
        }
        const uint32_t kb = smem_addr(sm.page[warp][k % C::kStages][0]), vb = kb + 2 * kPage * 128;
        float sc[NT][4];
        {
          float s2[NT][4];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int y = 0; y < 4; ++y) sc[t][y] = s2[t][y] = 0.f;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t a[2][4], qx[C::kQRegs ? 1 : NT][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int ks = 2 * y + e;
              ldsm4(a[e], kb + (ks >> 2) * (kPage * 128) + k_row * 128 + (((2 * (ks & 3) + k_ch) ^ (k_row & 7)) << 4));
            }
            if constexpr (!C::kQRegs) {
#pragma unroll
              for (int t = 0; t < NT; ++t) ldsm4(qx[t], q_at(t, y));
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint32_t(&f)[4] = C::kQRegs ? qf[C::kQRegs ? t : 0][y] : qx[C::kQRegs ? 0 : t];
              mma(sc[t], a[0], f[0], f[1]);
              mma(s2[t], a[1], f[2], f[3]);
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int y = 0; y < 4; ++y) sc[t][y] = (sc[t][y] + s2[t][y]) * p.scale_log2;
        }
        // keys of the page that a query does not see
        const int t0 = seen.page(it.v0 + i - it.i0) * kPage;
        const bool edge = !(t0 + kPage - 1 <= p0 && (t0 + kPage - 1 < p.sink_tokens || t0 > it.L - 1 - p.window));
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;  // V's keys 2 c, 2 c + 1 and those + 8
        if (edge) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            // the query of the lane's two columns
            const int j = it.n == 1 ? 0 : it.n == 2 ? (c >> 1) : 2 * t + (c >> 1);
            const int at = p0 + j;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int key = t0 + g + 8 * y;
              if (key > at || (key >= p.sink_tokens && key <= at - p.window)) sc[t][2 * y] = sc[t][2 * y + 1] = -INFINITY;
            }
          }
          auto visible = [&](int key) { return key < it.L && (key < p.sink_tokens || key >= low); };
          keep0 = (visible(t0 + 2 * c) ? 0xffffu : 0u) | (visible(t0 + 2 * c + 1) ? 0xffff0000u : 0u);
          keep1 = (visible(t0 + 2 * c + 8) ? 0xffffu : 0u) | (visible(t0 + 2 * c + 9) ? 0xffff0000u : 0u);
        }
        bool grow = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            grow = grow || fmaxf(sc[t][e], sc[t][2 + e]) > m[t][e] + kSlack;  // (any score, while m is -inf)
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(sc[t][e], sc[t][2 + e]);
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
              const bool up = x > m[t][e] + kSlack;  // (by itself: other columns do not matter)
              const float corr = up ? fast_exp2(m[t][e] - x) : 1.f;  // m = -inf -> 0
              if (up) m[t][e] = x;
              l[t][e] *= corr;
#pragma unroll
              for (int mt = 0; mt < 8; ++mt) {
                o[mt][t][e] *= corr;
                o[mt][t][2 + e] *= corr;
              }
            }
        }
        uint32_t pf[NT][2];
        {
          uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float mm = m[t][y & 1];
              w[y] = fast_exp2(sc[t][y] - (mm == -INFINITY ? 0.f : mm));
            }
            l[t][0] += w[0] + w[2];
            l[t][1] += w[1] + w[3];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              hi[t][y] = pack_bf16x2(w[2 * y], w[2 * y + 1]);
              lo[t][y] = pack_bf16x2(w[2 * y] - bf16lo(hi[t][y]), w[2 * y + 1] - bf16hi(hi[t][y]));
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const bool rest = (it.n == 1 && t == 0 && c >= 2) || (it.n == 2 && t == 1);
#pragma unroll
            for (int y = 0; y < 2; ++y) pf[t][y] = transpose8(rest ? lo[t][y] : hi[t][y]);
          }
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          uint32_t a[4];
          ldsm4_t(a, vb + (mt >> 2) * (kPage * 128) + v_row * 128 + (((2 * (mt & 3) + v_ch) ^ (v_row & 7)) << 4));
          if (edge) {
            a[0] &= keep0;
            a[1] &= keep0;
            a[2] &= keep1;
            a[3] &= keep1;
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) mma(o[mt][t], a, pf[t][0], pf[t][1]);
        }
        __syncwarp();  // every lane has read the page
        issue(k + C::kStages);
      }
      if constexpr (!C::kQRegs) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_free[gang][qb]);
      }
      // ---- the warp's part of the row
      const int buf = n_item % C::kBufs;
      if (n_item >= C::kBufs &&
          !__all_sync(0xffffffffu, wait(sm, &sm.part_free[gang][buf], ((n_item / C::kBufs) - 1) & 1, p.err)))
        break;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], w);
      const bool had = k > k_first;
      if (it.n == 1) {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int y = 0; y < 4; ++y) o[mt][0][y] += __shfl_xor_sync(0xffffffffu, o[mt][0][y], 2);
      } else if (NT > 1 && it.n == 2) {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int y = 0; y < 4; ++y) o[mt][0][y] += o[mt][NT > 1 ? 1 : 0][y];
      }
      const int cols = it.n * kGroup;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = 8 * t + 2 * c + e;
          if (col < cols) {
            if (had) {
#pragma unroll
              for (int mt = 0; mt < 8; ++mt) {
                sm.o[buf][warp][col][16 * mt + g] = o[mt][t][e];
                sm.o[buf][warp][col][16 * mt + 8 + g] = o[mt][t][2 + e];
              }
            }
            if (g == 0) {
              sm.m[buf][warp][col] = m[t][e];
              sm.l[buf][warp][col] = l[t][e];
            }
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.part_full[gang][buf]);
    }
    cp_async_wait<0>();  // (none is left but after a wait that gave up)
  } else {
    // -------------------------------------------------------------- merging
    // The warp has every second or third column, h0 + kMergeWarps j.  What a column's
    // parts count is worked out by lane j; their sums are then added up kAt columns at a
    // time.
    constexpr int kMergeWarps = C::kMergeWarps, kAt = NT == 1 && kMergeWarps == 2 ? 2 : 4;
    const int h0 = (warp - C::kWarps) % C::kMergeWarps, w0 = gang * C::kGang;
    for (int n_item = 0; rows.next(it); ++n_item) {
      const int buf = n_item % C::kBufs;
      // (a row cut between CTAs: no other is cut at the end of its first segment)
      unsigned long long* word = p.words + ((size_t)it.s0 * Hkv + kvh) * kWindowMergeWarps + h0;
      if (it.pieces > 1 && lane == 0) {  // (while the row's pages are on their way)
        const unsigned long long was = *reinterpret_cast<volatile unsigned long long*>(word);
        if (was >> 16 != p.tag) atomicCAS(word, was, (unsigned long long)p.tag << 16);
      }
      if (!__all_sync(0xffffffffu, wait(sm, &sm.part_full[gang][buf], (n_item / C::kBufs) & 1, p.err))) return;
      const size_t mine = ((size_t)(sidx * Hkv + kvh) * 2 + it.slot) * p.piece_cols;
      const int n_col = (kGroup * it.n - h0 + kMergeWarps - 1) / kMergeWarps;  // columns of the warp
      const int own = h0 + kMergeWarps * min(lane, n_col - 1);  // the lane's column
      auto out_row = [&](int col) {
        return (size_t)(it.tok + col / kGroup) * p.num_q_heads + kvh * kGroup + col % kGroup;
      };
      float f[C::kGang], M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < C::kGang; ++w) {
        f[w] = sm.m[buf][w0 + w][own];
        M = fmaxf(M, f[w]);
      }
#pragma unroll
      for (int w = 0; w < C::kGang; ++w) {
        f[w] = fast_exp2(f[w] - (M == -INFINITY ? 0.f : M));  // -inf -> 0
        L = fmaf(f[w], sm.l[buf][w0 + w][own], L);                 // (0 x NaN: a NaN of a part without a maximum shows)
      }
      const float inv = L == 0.f ? 0.f : (L != L ? L : 1.f / L);
#pragma unroll
      for (int w = 0; w < C::kGang; ++w) f[w] *= inv;
      const float lse = lse_log2(M == -INFINITY ? 0.f : M, L);
      if (lane < n_col) {
        if (it.pieces > 1) p.piece_lse[mine + own] = lse;
        else if (p.lse) p.lse[out_row(own)] = lse * kLn2;
      }
      // columns whose output is not finite: see window_mend.cuh
      uint32_t odd = 0;
      auto look = [&](int j, const float4& v) {
        const float z = fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, v.w * 0.f)));
        if (z != 0.f) odd |= 1u << j;
      };
      auto mend = [&]() {
        uint32_t todo = __reduce_or_sync(0xffffffffu, odd);
        if (todo == 0u) return;
        const Seen seen = seen_pages(it.L, it.n, p.window, p.sink_tokens);
        for (; todo != 0u; todo &= todo - 1u) {
          const int col = h0 + kMergeWarps * (__ffs((int)todo) - 1);
          mend_out(p, p.out + out_row(col) * kHeadDim, p.q + out_row(col) * kHeadDim,
                   p.block_tables + (size_t)it.r * p.max_blocks_per_req, kvh, seen.lead, 0, seen.first - seen.lead, seen.count(),
                   it.L - it.n + col / kGroup);
        }
      };
      for (int j0 = 0; j0 < n_col; j0 += kAt) {
        float4 a[kAt];
#pragma unroll
        for (int u = 0; u < kAt; ++u) {
          const int j = min(j0 + u, n_col - 1);
          a[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < C::kGang; ++w) {
            const float fw = __shfl_sync(0xffffffffu, f[w], j);
            const float4 x = *reinterpret_cast<const float4*>(&sm.o[buf][w0 + w][h0 + kMergeWarps * j][4 * lane]);
            if (fw != 0.f)  // (a part that had no page left nothing there)
              a[u] = make_float4(fmaf(fw, x.x, a[u].x), fmaf(fw, x.y, a[u].y), fmaf(fw, x.z, a[u].z), fmaf(fw, x.w, a[u].w));
          }
        }
#pragma unroll
        for (int u = 0; u < kAt; ++u) {
          if (j0 + u >= n_col) break;
          const int col = h0 + kMergeWarps * (j0 + u);
          if (it.pieces == 1) look(j0 + u, a[u]);
          if (it.pieces == 1)
            *reinterpret_cast<uint2*>(p.out + out_row(col) * kHeadDim + 4 * lane) =
                make_uint2(pack_bf16x2(a[u].x, a[u].y), pack_bf16x2(a[u].z, a[u].w));
          else
            *reinterpret_cast<float4*>(p.piece_o + (mine + col) * kHeadDim + 4 * lane) = a[u];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.part_free[gang][buf]);
      if (it.pieces == 1) {
        mend();
        continue;
      }
      // the row is cut between CTAs: the last of them to get here merges its pieces
      int last = 0;
      if (lane == 0) {
        last = (int)(atom_add64_acq_rel_gpu(word, 1ull) & 0xffffu) == it.pieces - 1;
        if (last) *word = (unsigned long long)p.tag << 16;  // ready for the next replay with this tag
      }
      __syncwarp();  // lane 0's acquire orders the reads below
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      // piece x lies with segment s0 + x, as its CTA's first row but for a row that
      // begins inside the segment
      const int first = !per_row && sm.start[it.r - p.row0] != it.s0 * seg ? 1 : 0;
      auto slot = [&](int x) {
        return ((size_t)((it.s0 + x) * Hkv + kvh) * 2 + (x == 0 ? first : 0)) * p.piece_cols;
      };
      constexpr int kMany = NT == 1 ? kAt : NT == 2 ? 4 : 8;  // columns at a time, of two pieces each
      float e[kMany][2];
      float4 y[kMany][2];
      auto fetch = [&](int j0, int x0) {
#pragma unroll
        for (int u = 0; u < kMany; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            e[u][v] = -INFINITY;
            y[u][v] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x0 + v < it.pieces) {
              const size_t at = slot(x0 + v) + h0 + kMergeWarps * min(j0 + u, n_col - 1);
              e[u][v] = load_cg(p.piece_lse + at);
              y[u][v] = load_cg(reinterpret_cast<const float4*>(p.piece_o + at * kHeadDim + 4 * lane));
            }
          }
      };
      fetch(0, 0);
      float top = -INFINITY, sum = 0.f;  // of the lane's column
      for (int x0 = 0; x0 < it.pieces; x0 += 4) {
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = x0 + u < it.pieces ? load_cg(p.piece_lse + slot(x0 + u) + own) : -INFINITY;
        const float mx = max_nan(max_nan(top, max_nan(x[0], x[1])), max_nan(x[2], x[3]));
        if (mx == -INFINITY) continue;
        sum *= fast_exp2(top - mx);
#pragma unroll
        for (int u = 0; u < 4; ++u) sum += fast_exp2(x[u] - mx);
        top = mx;
      }
      if (p.lse && lane < n_col) p.lse[out_row(own)] = lse_log2(top, sum) * kLn2;
      const float over = sum == 0.f ? 0.f : 1.f / sum;
      const float base = top == -INFINITY ? 0.f : top;
      for (int j0 = 0; j0 < n_col; j0 += kMany) {
        float4 a[kMany];
#pragma unroll
        for (int u = 0; u < kMany; ++u) a[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x0 = 0; x0 < it.pieces; x0 += 2) {
          if (j0 > 0 || x0 > 0) fetch(j0, x0);
#pragma unroll
          for (int u = 0; u < kMany; ++u)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const int j = min(j0 + u, n_col - 1);
              const float fu = fast_exp2(e[u][v] - __shfl_sync(0xffffffffu, base, j)) * __shfl_sync(0xffffffffu, over, j);
              const float4& x = y[u][v];
              a[u] = make_float4(fmaf(fu, x.x, a[u].x), fmaf(fu, x.y, a[u].y), fmaf(fu, x.z, a[u].z), fmaf(fu, x.w, a[u].w));
            }
        }
#pragma unroll
        for (int u = 0; u < kMany; ++u) {
          if (j0 + u >= n_col) break;
          look(j0 + u, a[u]);
          *reinterpret_cast<uint2*>(p.out + out_row(h0 + kMergeWarps * (j0 + u)) * kHeadDim + 4 * lane) =
              make_uint2(pack_bf16x2(a[u].x, a[u].y), pack_bf16x2(a[u].z, a[u].w));
        }
      }
      mend();
    }
  }
}

std::atomic<bool> g_attr_set[3][2][kMaxDevices];

template <int NT, int kGangs>
cudaError_t launch(const WindowParams& p, int grid, cudaStream_t stream) {
  constexpr size_t kBytes = sizeof(Smem<NT, kGangs>) + 1024;  // + slack to align the base
  static_assert(kBytes <= 232448, "shared memory per CTA");
  const cudaError_t e = set_smem_limit_once((const void*)decode_window_kernel<NT, kGangs>, (int)kBytes, g_attr_set[NT - 1][kGangs - 1]);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_window_kernel<NT, kGangs>, dim3((unsigned)grid), dim3(Cfg<NT, kGangs>::kThreads), kBytes, stream, p);
}

}  // namespace

cudaError_t launch_decode_window(const WindowParams& p, int queries, int grid, cudaStream_t stream) {
  // Two gangs a CTA where rows are many and short: a row's start and end take a gang 1.3 us,
  // and two do them side by side.  Measured, us, one gang and two.  Rows of one query, more
  // than three a segment: 1000 of 100 keys 95.9 and 85.4, 143 of 100 20.8 and 17.4, 100 of 64
  // 14.4 and 13.1, 58 of 300 15.0 and 14.6, 58 of 1024 44.5 and 44.7; fewer (20 of 300) 10.1 and
  // 14.2.  Rows of three and four: 179 of 149 23.8 and 20.9, 100 of 64 22.5 and 19.8, 100 of 300
  // 30.2 and 31.5.  Rows of five and six would have two warps a gang: 80 of 1024 65.9 and 69.2.
  const int64_t pages = std::min<int64_t>(p.max_blocks_per_req, (int64_t)p.window / kPage + p.sink_tokens / kPage + 3);
  const bool two = p.per_row == 0 && p.rows > 3 * (grid / p.num_kv_heads) && pages <= (queries == 1 ? 32 : 14);
  if (queries == 1) return two ? launch<1, 2>(p, grid, stream) : launch<1, 1>(p, grid, stream);
  if (queries <= 4) return two ? launch<2, 2>(p, grid, stream) : launch<2, 1>(p, grid, stream);
  return launch<3, 1>(p, grid, stream);
}

}  // namespace pa
