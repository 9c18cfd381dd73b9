// Tensor-core tiles of attention with a sliding window: rows with more than six
// queries (prompt chunks).
//
// What is computed: the query at position p sees keys t <= p with t < sinks or t > p -
// window; scores, softmax and output as in decode_window.cu.
//
// Work.  A job is up to 64 query tokens of a row for one kv head: two query tiles A and
// B of 32 tokens x 4 heads = 128 rows, the M of one tcgen05.mma each (a job of up to 32
// has A alone).  The pages that any of its queries sees (leading ones, then from the
// first query's window on) are counted through and go in key tiles of 128 (8 pages), so a
// job costs its window and its own length, not its context.  The jobs' key tiles are
// laid end to end and cut into one equal share per SM (a job counts some tiles more, for
// its start and end), so that no SM waits for the others with whole jobs still to
// run.  A CTA runs its share without a barrier between jobs: rings, phases and buffers are
// indexed by running counts.  A job that is cut leaves a part per CTA in the workspace,
// which merge_window_kernel puts together.  Where whole jobs end about as soon, they are
// dealt out whole (an instantiation of its own: the other's code costs the loops 2 %).
//
// Warps.  0-3 and 4-7: softmax of A and B, one thread per row (tensor-memory lane =
// row).  8 and 9: issue the score products of A and of B (8 also copies Q by TMA and owns
// the tensor memory), 10 and 11 the PV products, so that the waits of one kind do not hold
// up the other.  12 and 13: copy K and V by tiled TMA, a page's half of 64 dims per box.
// 14: clears V's rows that no query of the job sees, whose weight is 0 but which may hold
// infinities or NaN (only key tiles at the ends have any).
//
// Tensor memory: per query tile two score buffers of 64 keys and the output, 128
// columns; that is all 512.  Scores are made 64 keys at a time (a sub-tile) and a
// sub-tile's weights (bf16 pairs, the A operand of the PV product) overwrite its scores:
// the scores of sub-tile i + 1 are there when the softmax has finished sub-tile i, and
// those of i + 2 follow the PV product of i.  The softmax takes the scores once, 32
// columns at a time, against a reference that is re-based only when weights get large.
// Weights are rounded to bf16, as the tensor cores take them; their sum is kept in
// binary32 from the unrounded ones, as are scores, maxima and outputs.
//
// Bound and measured (GB300).  Per sub-tile of both query tiles the tensor pipe is busy for
// 1281 cycles: 2 x 256 of PV, 2 x 384 of scores (64 keys at a time a product reads Q's 4 KB
// and K's 2 KB from shared memory, 48 cycles at 128 B, for 32 cycles of arithmetic; 128
// keys at a time would take 256, but then one buffer has to do, and 1089 busy cycles became
// 2500 in all).  A sub-tile takes 1360 cycles in the middle of a job; a job costs about 3 us
// beside (its first sub-tile's maximum, masks at both ends, the output), a launch 10 us
// (152 CTAs fetch their first 30 MB at once).  Softmax of a row by two threads of 32 columns
// each was slower (1120 ns a sub-tile for 870), as were scores, weights and PV from one warp
// (67.2 us for 65.7, 19 jobs of 64 queries x 8 heads over 4160 keys; 61.4 now).  Most of
// what a job costs beside is code that runs once in it and is not in the instruction
// caches: every path laid out a second time shows.  A second buffer for Q, three stages of K
// and V for four and the output staged in the Q that is done with was slower too (109.7 us
// for 100.4 on those prompts): the softmax warps are what a job's ends wait for.
//
// Every wait is bounded; on a timeout the CTA records the error, lets its copies and
// products finish (bounded), frees its tensor memory and returns.
#include <math.h>
#include <stddef.h>

#include <type_traits>

#include "internal.h"
#include "q4.cuh"  // lse_log2, load_cg, bf16x2_fma
#include "tc.cuh"
#include "window.cuh"
#include "window_mend.cuh"

namespace pa {
namespace {

using namespace tc;

constexpr int kTok = kPrefillQTile;  // query tokens of a tile
constexpr int kRows = kTok * kGroup;
constexpr int kKeys = kTcKeyTile;
constexpr int kPagesPerTile = kKeys / kPage;
constexpr int kSub = 64;          // keys of a score product and of a stage
constexpr int kPagesPerSub = kSub / kPage;
constexpr int kHalf = 128 * 128;  // a query tile: 128 rows x 64 bf16
constexpr int kTileBytes = 2 * kHalf;
constexpr int kSubHalf = kSub * 128;  // 64 keys x 64 bf16
constexpr int kSubBytes = 2 * kSubHalf;
constexpr int kPageHalfBytes = kPage * 128;
constexpr int kStages = 4;  // of K and of V
constexpr int kBad = 16;      // entries of the flags below: more than stages and sub-tiles on their way
constexpr int kScoreWarp = 8, kPvWarp = 10, kKWarp = 12, kVWarp = 13, kClearWarp = 14;  // (+ 1: tile B)
constexpr int kThreads = 15 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 for tile B
// The sum of 64 weights above which their row's reference is raised: binary32 and bf16 hold
// larger ones as exactly, so it only keeps far from their ends; at 2^10 a row whose first
// sub-tile shows it few keys re-bases more often.
constexpr float kMaxSum = 65536.f;
constexpr int kOutTok = kQ4OutTok;          // query tokens of a softmax warp
constexpr uint32_t kIdescS = idesc_bf16_f32(kRows, kSub, false);
constexpr uint32_t kIdescO = idesc_bf16_f32(kRows, kHeadDim, true);
static_assert(kRows == 128 && kKeys == 128 && kWindowTileTokens == 2 * kTok, "tile shape");
static_assert(kOutTok * kGroup == 32 && 4 * kOutTok == kTok, "a softmax warp's 32 rows are whole tokens");

struct __align__(1024) Smem {
  uint8_t q[2][kTileBytes];
  uint8_t k[kStages][kSubBytes];
  uint8_t v[kStages][kSubBytes];
  uint8_t out[8][32 * 128];  // a softmax warp's rows on their way out, 64 dims at a time
  uint64_t q_full, q_free;   // a job's Q has landed; its last scores are done
  uint64_t o_free[2];        // the softmax warps have read a job's output
  uint64_t k_full[kStages], k_empty[kStages];
  uint64_t v_full[kStages], v_ready[kStages], v_empty[kStages];  // landed; cleared; read
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // per query tile and buffer: phase i / 2 for sub-tile i
  uint64_t drained[4];  // every product issued by a warp has completed
  uint8_t bad_k[kBad][kPagesPerSub], bad_v[kBad][kPagesPerSub];  // pages outside the pool, of a sub-tile
  uint32_t tmem;
  int abort;
  int odd;  // some output is not finite
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;  // + slack to align the base
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

// (The loop is a function of its own: at every wait's place it would be more code than the
// instruction caches take along.  8 prompts behind a window of 512 took 118.7 us for
// 107.1; the output by a rolled-up loop made that 103.)
__device__ __noinline__ bool wait_on(Smem& sm, uint64_t* bar, uint32_t parity, int* err) {
  const unsigned long long t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*reinterpret_cast<volatile int*>(&sm.abort)) return false;
      if (globaltimer() - t0 > kWaitLimitNs) {
        record_error(err, PA_ERR_DEVICE_TIMEOUT);
        *reinterpret_cast<volatile int*>(&sm.abort) = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait(Smem& sm, uint64_t* bar, uint32_t parity, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_on(sm, bar, parity, err);
}

struct Job {
  int32_t tok0;  // first query token of the job
  int32_t nq;    // its query tokens (1 .. 64)
  int32_t kvh;
  int32_t pos0;  // position of the first
  const int32_t* table;
  // this CTA's part of the pages that any of its queries sees: page v of them is page v + (v
  // < lead ? lo : hi) of the row
  int32_t lead, lo, hi;
  int32_t n_pages;         // to the job's end
  int32_t n_tiles, n_sub;  // key tiles; sub-tiles of 64 keys (for both query tiles)
  int32_t n_x;             // query tiles
  int32_t u;               // (kCut) the job
  __device__ __forceinline__ int page(int v) const { return v + (v < lead ? lo : hi); }
};

// The CTA's jobs.  kCut: its share of all key tiles, from start[b] to start[b + 1], whose
// first and last job may be cut.  Else job b of every round of gridDim.x whole jobs, in reverse order on odd
// rounds (the items come longest first).
template <bool kCut>
struct Jobs {
  const WindowParams& p;
  const WindowItems& items;
  int k, odd;  // kCut: the share's jobs given; else the jobs of the rounds before
  __device__ __forceinline__ Jobs(const WindowParams& p_, const WindowItems& items_) : p(p_), items(items_), k(0), odd(0) {}
  __device__ __forceinline__ bool next(Job& job) {
    const int b = (int)blockIdx.x;
    int u;
    if constexpr (kCut) {
      const int2 s0 = items.start[b], s1 = items.start[b + 1];
      const int n = s1.x - s0.x + (s1.y > 0 ? 1 : 0);
      if (k >= n) return false;
      u = s0.x + k++;
    } else {
      const int n = items.count * p.num_kv_heads, G = (int)gridDim.x;
      u = k + (odd ? G - 1 - b : b);
      if (u >= n) {  // (a last round that has no job for this CTA)
        k = n;
        return false;
      }
      k += G;
      odd ^= 1;
    }
    const int it = u / p.num_kv_heads;
    const int4 item = items.item[it];  // request, first query token, its position, queries
    job.tok0 = item.y;
    job.nq = item.w;
    job.kvh = u - it * p.num_kv_heads;
    job.pos0 = item.z;
    job.table = p.block_tables + (size_t)item.x * p.max_blocks_per_req;
    const Seen seen = seen_pages(item.z + item.w, item.w, p.window, p.sink_tokens);
    job.n_pages = seen.count();
    job.n_x = job.nq > kTok ? 2 : 1;
    job.lead = seen.lead;
    job.lo = 0;
    job.hi = seen.first - seen.lead;
    job.n_tiles = (job.n_pages + kPagesPerTile - 1) / kPagesPerTile;
    job.n_sub = (job.n_pages + kPagesPerSub - 1) / kPagesPerSub;
    if constexpr (kCut) {
      const int2 s0 = items.start[b], s1 = items.start[b + 1];
      job.u = u;
      if (u == s1.x) {
        job.n_tiles = s1.y;
        job.n_sub = min(job.n_sub, 2 * s1.y);
      }
      if (u == s0.x) {  // from key tile s0.y on
        const int v = s0.y * kPagesPerTile;
        job.n_pages -= v;
        job.lead -= v;
        job.lo += v;
        job.hi += v;
        job.n_tiles -= s0.y;
        job.n_sub -= 2 * s0.y;
      }
    }
    return true;
  }
  // Whether the job given last is cut.
  __device__ __forceinline__ bool cut(const Job& job) const {
    const int2 s0 = items.start[blockIdx.x], s1 = items.start[blockIdx.x + 1];
    return (job.u == s0.x && s0.y > 0) || (job.u == s1.x && s1.y > 0);
  }
  // Where its part goes: with the CTA's first job or its last.
  __device__ __forceinline__ int slot() const { return 2 * (int)blockIdx.x + (k > 1 ? 1 : 0); }
};

// Bits n .. 31 (n clamped to 0 .. 32).
__device__ __forceinline__ uint32_t bits_from(int n) { return n <= 0 ? 0xffffffffu : n >= 32 ? 0u : 0xffffffffu << n; }

// The keys of a page at position t0 that a query at `pos` sees, as bits 0 .. 15.
__device__ __forceinline__ uint32_t page_seen(int t0, int pos, int window, int sinks) {
  return ~bits_from(pos - t0 + 1) & (bits_from(pos - window + 1 - t0) | ~bits_from(sinks - t0)) & 0xffffu;
}

// The job's sub-tiles of the window of whose keys every query from position a to b sees all:
// x .. y - 1.
__device__ __forceinline__ int2 whole_subs(const Job& job, int a, int b, int window) {
  // first and last page (of the job's count) of which they do
  const int lo = max(job.lead, ((b - window) >> 4) + 1 - job.hi);  // its first key > b - window
  const int hi = min(job.n_pages, ((a + 1) >> 4) - job.hi) - 1;    // its last key <= a
  static_assert(kPage == 16, "positions to pages");
  return make_int2((max(lo, 0) + kPagesPerSub - 1) / kPagesPerSub, (hi + 1) / kPagesPerSub);
}

// Pool rows of 32 of a job's pages, one per lane (eight sub-tiles); pages past the end
// repeat the last one (hidden, and V's cleared); -1: outside the pool.
__device__ __forceinline__ int load_group(const Job& job, int g, int num_kv_heads, int64_t num_blocks, int* err) {
  const int v = 32 * g + (int)(threadIdx.x & 31);
  if (v >= job.n_sub * kPagesPerSub) return 0;
  const int b = job.table[job.page(min(v, job.n_pages - 1))];
  if (b < 0 || b >= num_blocks) {
    record_error(err, PA_ERR_DEVICE_INDEX);
    return -1;
  }
  return (b * num_kv_heads + job.kvh) * kPage;
}

// The weights of 32 scores against a reference -nm, in pairs of bf16, and their sums.
__device__ __forceinline__ void weigh(const uint32_t (&c)[32], uint32_t (&w)[16], float2 (&s2)[2], float scale, float nm) {
  const float2 sc2 = make_float2(scale, scale), nm2 = make_float2(nm, nm);
#pragma unroll
  for (int y = 0; y < 16; ++y) {
    const float2 d = __ffma2_rn(make_float2(__uint_as_float(c[2 * y]), __uint_as_float(c[2 * y + 1])), sc2, nm2);
    const float2 e = make_float2(fast_exp2(d.x), fast_exp2(d.y));
    s2[y & 1] = __fadd2_rn(s2[y & 1], e);
    w[y] = pack_bf16x2(e.x, e.y);
  }
}

// Copies of K (is_k) or V, a sub-tile per stage, two lanes a page; block ids one group or
// job ahead.
template <bool kCut>
__device__ __forceinline__ void copy_tiles(Smem& sm, const WindowParams& p, const WindowItems& items, bool is_k,
                                           const CUtensorMap* map) {
  const int lane = threadIdx.x & 31;
  uint64_t* full = is_k ? sm.k_full : sm.v_full;
  uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
  Jobs<kCut> jobs(p, items);
  Job job, after;
  bool more = jobs.next(job), ok = true;
  int R = 0;  // sub-tiles so far
  int cur = more ? load_group(job, 0, p.num_kv_heads, p.num_blocks, p.err) : 0;
  while (more && ok) {
    int next = load_group(job, 1, p.num_kv_heads, p.num_blocks, p.err), first = 0;
    for (int i = 0; i < job.n_sub; ++i, ++R) {
      const int s = R % kStages;
      if (i > 0 && (i & 7) == 0) {
        cur = next;
        next = load_group(job, (i >> 3) + 1, p.num_kv_heads, p.num_blocks, p.err);
      }
      if (i == job.n_sub - 1) {
        more = jobs.next(after);
        if (more) first = load_group(after, 0, p.num_kv_heads, p.num_blocks, p.err);
      }
      const int row = __shfl_sync(0xffffffffu, cur, ((i & 7) << 2) + ((lane >> 1) & 3));
      ok = R < kStages ? is_k || R > 0 || __all_sync(0xffffffffu, wait(sm, &sm.k_full[0], 0, p.err))
                       : __all_sync(0xffffffffu, wait(sm, &empty[s], ((R / kStages) - 1) & 1, p.err));
      if (!ok) break;
      if (lane < 2 * kPagesPerSub && !(lane & 1)) (is_k ? sm.bad_k : sm.bad_v)[R % kBad][lane >> 1] = row < 0;
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(&full[s], kSubBytes);
      __syncwarp();
      uint8_t* dst = is_k ? sm.k[s] : sm.v[s];
      if (lane < 2 * kPagesPerSub)
        tma_load_2d(dst + (lane & 1) * kSubHalf + (lane >> 1) * kPageHalfBytes, map, 64 * (lane & 1), max(row, 0), &full[s]);
    }
    job = after;
    cur = first;
  }
  if (!ok)  // gave up: the copies in flight land before the CTA leaves (bounded)
    for (int r = max(0, R - kStages); r < R; ++r) mbar_wait_bounded(&full[r % kStages], (r / kStages) & 1);
}

// The outputs (or parts) of the CTA's jobs that are not finite, again (see window_mend.cuh), a row
// at a time and warp.  Out of line: few registers are alive where it is called.
template <bool kCut>
__device__ __noinline__ void mend_jobs(const WindowParams& p, const WindowItems& items) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Jobs<kCut> jobs(p, items);
  Job job;
  while (jobs.next(job)) {
    const int n = min(job.n_pages, job.n_sub * kPagesPerSub);
    const bool is_cut = kCut && jobs.cut(job);
    const size_t part = kCut ? (size_t)jobs.slot() * 2 * kRows : 0;
    for (int i = warp; i < kGroup * job.nq; i += kThreads / 32) {
      const int pos = job.pos0 + (i >> 2);
      const size_t at = ((size_t)(job.tok0 + (i >> 2)) * p.num_q_heads + job.kvh * kGroup + (i & 3)) * kHeadDim;
      if (is_cut) {  // (tile B's rows lie behind tile A's)
        float4* o = reinterpret_cast<float4*>(p.part_o + (part + (i & ~(kRows - 1))) * kHeadDim) + lane * kRows + (i & (kRows - 1));
        const float4 y = load_cg(o);
        if (__any_sync(0xffffffffu, fmaf(y.x, 0.f, fmaf(y.y, 0.f, fmaf(y.z, 0.f, y.w * 0.f))) != 0.f))
          *o = mend_row(p, y, p.q + at, job.table, job.kvh, job.lead, job.lo, job.hi, n, pos);
      } else {
        mend_out(p, p.out + at, p.q + at, job.table, job.kvh, job.lead, job.lo, job.hi, n, pos);
      }
    }
  }
}

template <bool kCut>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_window_kernel(const __grid_constant__ WindowParams p, const __grid_constant__ WindowItems items,
                          const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap out_map,
                          const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (warp == kScoreWarp && lane == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_free, 2);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 2);
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_ready[s], 1);
      mbar_init(&sm.v_empty[s], 2);
    }
    for (int x = 0; x < 2; ++x) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sm.s_full[x][b], 1);
        mbar_init(&sm.p_full[x][b], kRows);
        mbar_init(&sm.pv_done[x][b], 1);
      }
      mbar_init(&sm.o_free[x], kRows);
    }
    for (int w = 0; w < 4; ++w) mbar_init(&sm.drained[w], 1);
    sm.abort = 0;
    sm.odd = 0;
    fence_mbar_init();
  }
  if (warp == kScoreWarp) {
    __syncwarp();
    tmem_alloc(&sm.tmem, kTmemCols);
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sm.tmem;
  // nothing above touches what an earlier kernel may write (the jobs come with the
  // parameters)
  pdl_wait();
  pdl_launch_dependents();

  if (warp == kKWarp || warp == kVWarp) {
    const CUtensorMap* map = warp == kKWarp ? &k_map : &v_map;
    if (lane == 0) prefetch_tensormap(map);
    copy_tiles<kCut>(sm, p, items, warp == kKWarp, map);
  } else if (warp == kClearWarp) {
    // ------------------------------------------- V's rows that no query sees
    Jobs<kCut> jobs(p, items);
    Job job;
    int R = 0;
    bool ok = true;
    while (ok && jobs.next(job)) {
      const int keys = job.pos0 + job.nq, low = max(job.pos0 - p.window + 1, 0);
      for (int i = 0; i < job.n_sub; ++i, ++R) {
        const int s = R % kStages;
        ok = __all_sync(0xffffffffu, wait(sm, &sm.v_full[s], (R / kStages) & 1, p.err));
        if (!ok) break;
        bool cleared = false;
#pragma unroll 1
        for (int y = 0; y < kSub / 32; ++y) {
          const int row = 32 * y + lane, v = i * kPagesPerSub + row / kPage;
          const int t = job.page(v) * kPage + row % kPage;
          const bool hide = v >= job.n_pages || t >= keys || (t >= p.sink_tokens && t < low) ||
                            reinterpret_cast<volatile uint8_t*>(sm.bad_v[R % kBad])[row / kPage];
          if (hide) {
            uint4* d = reinterpret_cast<uint4*>(sm.v[s] + row * 128);
#pragma unroll
            for (int c = 0; c < 8; ++c) d[c] = d[c + kSubHalf / 16] = make_uint4(0u, 0u, 0u, 0u);
            cleared = true;
          }
        }
        if (cleared) fence_proxy_async_smem();  // the products read the tile through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.v_ready[s]);
      }
    }
  } else if (warp >= kScoreWarp) {
    // --------------------------------------------------------- MMA issuers
    // The whole warp runs this (so that descriptors and addresses are warp-uniform
    // values) and one elected lane issues.  Scores and PV products of a query tile come
    // from two warps, so that neither's waits delay the other's products.
    const int x = (warp - kScoreWarp) & 1;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t t_s = tm + kColS + x * kKeys, t_o = tm + kColO + x * kHeadDim;
    auto arrived = [&](uint64_t* bar, int phase) {
      return __all_sync(0xffffffffu, wait(sm, bar, (uint32_t)phase & 1u, p.err)) != 0;
    };
    // two barriers, looked at together
    auto both = [&](uint64_t* bar0, int phase0, uint64_t* bar1, int phase1) {
      const bool a = mbar_try_wait(bar0, (uint32_t)phase0 & 1u), b = mbar_try_wait(bar1, (uint32_t)phase1 & 1u);
      if (__all_sync(0xffffffffu, a && b)) return true;
      return arrived(bar0, phase0) && arrived(bar1, phase1);
    };
    // a job without this tile: every phase is waited for in turn all the same (a wait by
    // parity tells a phase only from its neighbours), and every stage given back
    auto pass = [&](uint64_t* full, uint64_t* empty, int phase) {
      const bool there = arrived(full, phase);
      if (there && lane == 0) mbar_arrive(empty);
      __syncwarp();
      return there;
    };
    Jobs<kCut> jobs(p, items);
    Job job;
    bool more = jobs.next(job), ok = true;
    int R0 = 0, I0 = 0;  // running counts: sub-tiles, this query tile's
    if (warp < kPvWarp) {
      const uint64_t q_desc = desc_sw128(smem_addr(sm.q[0]), 16, 1024) + (uint32_t)x * (kTileBytes >> 4);
      const uint64_t k_desc = desc_sw128(smem_addr(sm.k[0]), 16, 1024);
      auto load_q = [&](const Job& job) {
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.q_full, job.n_x * kTileBytes);
          for (int y = 0; y < job.n_x; ++y) {
            tma_load_3d(sm.q[y], &q_map, 0, job.kvh * kGroup, job.tok0 + y * kTok, &sm.q_full);
            tma_load_3d(sm.q[y] + kHalf, &q_map, 64, job.kvh * kGroup, job.tok0 + y * kTok, &sm.q_full);
          }
        }
        __syncwarp();
      };
      int n_job = 0, n_q = 0;
      while (more && ok) {
        if (x == 0) {  // Q, after the last scores of the job before
          ok = n_job == 0 || arrived(&sm.q_free, n_job - 1);
          if (!ok) break;
          load_q(job);
          n_q += 1;
        }
        if (x < job.n_x) {
          ok = arrived(&sm.q_full, n_job);
          for (int i = 0; ok && i < job.n_sub; ++i) {
            // scores of sub-tile i: its keys are there, and the PV product of the sub-tile
            // whose weights lie where they go is done
            const int R = R0 + i, s = R % kStages, I = I0 + i, b = I & 1;
            ok = I < 2 ? arrived(&sm.k_full[s], R / kStages)
                       : both(&sm.k_full[s], R / kStages, &sm.pv_done[x][b], (I >> 1) - 1);
            if (!ok) break;
            const uint64_t kd = k_desc + (uint32_t)s * (kSubBytes >> 4);
            const uint32_t on = elect_one();
            fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < kHeadDim / 16; ++ks) {
              // 64-dim half, 16-dim step in it
              mma_ss_if(on, t_s + b * kSub, q_desc + (((ks >> 2) * kHalf + (ks & 3) * 32) >> 4),
                        kd + (((ks >> 2) * kSubHalf + (ks & 3) * 32) >> 4), kIdescS, ks > 0);
            }
            commit_if(on, &sm.s_full[x][b]);
            commit_if(on, &sm.k_empty[s]);
            if (i == job.n_sub - 1) commit_if(on, &sm.q_free);
          }
          I0 += job.n_sub;
        } else {
          ok = pass(&sm.q_full, &sm.q_free, n_job);
          for (int R = R0; ok && R < R0 + job.n_sub; ++R) ok = pass(&sm.k_full[R % kStages], &sm.k_empty[R % kStages], R / kStages);
        }
        R0 += job.n_sub;
        n_job += 1;
        more = jobs.next(job);
      }
      if (n_q > 0) mbar_wait_bounded(&sm.q_full, (uint32_t)(n_q - 1) & 1u);  // Q has landed before the CTA leaves
    } else {
      const uint64_t v_desc = desc_sw128(smem_addr(sm.v[0]), kSubHalf, 1024);
      int n_own = 0;
      while (more && ok) {
        if (x < job.n_x) {
          // the first product overwrites the output of this tile's job before
          ok = n_own == 0 || arrived(&sm.o_free[x], n_own - 1);
          for (int i = 0; ok && i < job.n_sub; ++i) {
            const int R = R0 + i, s = R % kStages, I = I0 + i, b = I & 1;
            ok = both(&sm.v_ready[s], R / kStages, &sm.p_full[x][b], I >> 1);
            if (!ok) break;
            const uint64_t vd = v_desc + (uint32_t)s * (kSubBytes >> 4);
            const uint32_t on = elect_one();
            fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < kSub / 16; ++ks)  // 16 keys: two 8-row groups of V, 8 columns of weight pairs
              mma_ts_if(on, t_o, t_s + b * kSub + 8 * ks, vd + (uint32_t)ks * (2 * 1024 >> 4), kIdescO,
                        (i > 0 || ks > 0) ? 1u : 0u);
            commit_if(on, &sm.pv_done[x][b]);
            commit_if(on, &sm.v_empty[s]);
          }
          I0 += job.n_sub;
          n_own += 1;
        } else {
          for (int R = R0; ok && R < R0 + job.n_sub; ++R) ok = pass(&sm.v_ready[R % kStages], &sm.v_empty[R % kStages], R / kStages);
        }
        R0 += job.n_sub;
        more = jobs.next(job);
      }
    }
    // every product issued has completed before the tensor memory is freed (a commit
    // tracks all of the warp's)
    commit_if(elect_one(), &sm.drained[warp - kScoreWarp]);
    mbar_wait_bounded(&sm.drained[warp - kScoreWarp], 0);
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    const int x = warp >> 2;
    const int row = threadIdx.x & 127;  // 4 * token + head in group
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_o = lane_base + kColO + x * kHeadDim;
    const float scale = p.scale_log2;  // not 0 (see the launch)
    const uint32_t hide = scale >= 0.f ? 0xff800000u : 0x7f800000u;  // scales to -inf
    int R0 = 0, I0 = 0;  // running counts: sub-tiles, this query tile's
    Jobs<kCut> jobs(p, items);
    Job job;
    bool more = jobs.next(job), ok = true;
    while (more) {
      if (x >= job.n_x) {
        R0 += job.n_sub;
        more = jobs.next(job);
        continue;
      }
      const int a = job.pos0 + x * kTok, b = min(a + kTok, job.pos0 + job.nq) - 1;  // the tile's positions
      const int pos = a + (row >> 2);
      const int2 whole = whole_subs(job, a, b, p.window);
      float m_run = -INFINITY, l_run = 0.f;
      for (int i = 0; i < job.n_sub; ++i) {
        const int I = I0 + i;
        const uint32_t t_s = lane_base + kColS + x * kKeys + (I & 1) * kSub;
        ok = __all_sync(0xffffffffu, wait(sm, &sm.s_full[x][I & 1], (I >> 1) & 1, p.err));
        if (!ok) break;
        fence_after_sync();
        // bytes of its 4 pages
        const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(sm.bad_k[(R0 + i) % kBad]);
        // The weights are taken against the row's reference m_run.  Only when their sum
        // shows that it lies too low are the scores read again for their maximum, m_run
        // re-based to it and the output rescaled: rare after a row's first keys.
        uint32_t c[2][32], w[2][16];
        float sum = 0.f;
        // what the row does not see hidden
        auto hide_some = [&](int h) {
          uint32_t see = 0u;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int v = i * kPagesPerSub + 2 * h + e;
            if (v < job.n_pages && ((bad >> (8 * (2 * h + e))) & 0xffu) == 0u)
              see |= page_seen(job.page(v) * kPage, pos, p.window, p.sink_tokens) << (16 * e);
          }
          if (__all_sync(0xffffffffu, see == 0xffffffffu)) return;  // (half of the time)
#pragma unroll
          for (int y = 0; y < 32; ++y)
            if (!((see >> y) & 1u)) c[h][y] = hide;
        };
        auto weights = [&](auto some) {
          const float nm = (m_run == -INFINITY) ? 0.f : -m_run;
          float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          tmem_ld32_async(t_s, c[0]);
          wait_ld(c[0]);
          tmem_ld32_async(t_s + 32, c[1]);
          if (decltype(some)::value) hide_some(0);
          weigh(c[0], w[0], s2, scale, nm);
          wait_ld(c[1]);
          if (decltype(some)::value) hide_some(1);
          weigh(c[1], w[1], s2, scale, nm);
          s2[0] = __fadd2_rn(s2[0], s2[1]);
          sum = s2[0].x + s2[0].y;
        };
        const bool some = i < whole.x || i >= whole.y || bad != 0u;
        bool low = true;
        if (i > 0) {
          if (some) weights(std::true_type{});
          else weights(std::false_type{});
          low = sum > kMaxSum || m_run == -INFINITY;
        }
        if (__any_sync(0xffffffffu, low)) {
          float mt = __uint_as_float(hide);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tmem_ld32_async(t_s + 32 * h, c[h]);
            wait_ld(c[h]);
            if (some) hide_some(h);
#pragma unroll
            for (int y = 0; y < 32; ++y)
              mt = scale >= 0.f ? fmaxf(mt, __uint_as_float(c[h][y])) : fminf(mt, __uint_as_float(c[h][y]));
          }
          mt *= scale;
          const bool grow = low && mt > m_run;
          const float corr = grow ? fast_exp2(m_run - mt) : 1.f;  // m_run = -inf -> 0
          if (grow) m_run = mt;
          l_run *= corr;
          if (i > 0) {  // O is stable once PV of the sub-tile before is done
            ok = __all_sync(0xffffffffu, wait(sm, &sm.pv_done[x][(I - 1) & 1], ((I - 1) >> 1) & 1, p.err));
            if (!ok) break;
            fence_after_sync();
            rescale(t_o, t_s, 0, true, corr);
          }
          const float nm = (m_run == -INFINITY) ? 0.f : -m_run;
          float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          weigh(c[0], w[0], s2, scale, nm);
          weigh(c[1], w[1], s2, scale, nm);
          s2[0] = __fadd2_rn(s2[0], s2[1]);
          sum = s2[0].x + s2[0].y;
        }
        store16(t_s, w[0]);  // weights over scores already read
        store16(t_s + 16, w[1]);
        l_run += sum;
        wait_st();
        fence_before_sync();  // the tensor-memory accesses above precede the arrive
        mbar_arrive(&sm.p_full[x][I & 1]);
      }
      if (!ok) break;
      const int I1 = I0 + job.n_sub - 1;
      const bool is_cut = kCut && jobs.cut(job);
      const int slot = kCut ? jobs.slot() : 0;
      Job after;  // (the next one, while the last product runs)
      more = jobs.next(after);
      if (!__all_sync(0xffffffffu, wait(sm, &sm.pv_done[x][I1 & 1], (I1 >> 1) & 1, p.err))) break;
      fence_after_sync();
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      float lse = lse_log2(m_run, l_run);
      const int tok = x * kTok + (row >> 2);
      const int tok_w = x * kTok + kOutTok * (warp & 3);  // the warp's first token
      if (is_cut) {
        // the row's part, 4 dims of 32 rows at a time
        const size_t at = ((size_t)slot * 2 + x) * kRows;
        float4* dst = reinterpret_cast<float4*>(p.part_o + at * kHeadDim) + row;
        float zero = 0.f;  // 0 times every value: NaN where one is not finite
#pragma unroll 1
        for (int c = 0; c < kHeadDim / 16; ++c) {
          uint32_t o[16];
          load16(t_o + 16 * c, o);
#pragma unroll
          for (int y = 0; y < 16; ++y) zero = fmaf(__uint_as_float(o[y]), 0.f, zero);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            dst[(4 * c + y) * kRows] =
                make_float4(__uint_as_float(o[4 * y]) * inv, __uint_as_float(o[4 * y + 1]) * inv,
                            __uint_as_float(o[4 * y + 2]) * inv, __uint_as_float(o[4 * y + 3]) * inv);
        }
        fence_before_sync();  // the tensor-memory reads above precede the arrive
        mbar_arrive(&sm.o_free[x]);
        p.part_lse[at + row] = lse;
        if (zero != 0.f && tok < job.nq) *reinterpret_cast<volatile int*>(&sm.odd) = 1;
      } else {
        // The output, 64 dims at a time, through shared memory (128-byte swizzle) and out
        // by TMA, the warp's 8 tokens x 4 heads x 64 dims.
        uint8_t* stg = sm.out[warp];
        uint32_t zero = 0u;  // 0 times every value, in pairs: 0 or NaN
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          if (lane == 0) bulk_wait_read();  // what was staged before has been read
          __syncwarp();
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t o[32];
            tmem_ld32_async(t_o + 64 * h + 32 * c, o);
            wait_ld(o);
            uint32_t w[16];
#pragma unroll
            for (int y = 0; y < 16; ++y)
              w[y] = pack_bf16x2(__uint_as_float(o[2 * y]) * inv, __uint_as_float(o[2 * y + 1]) * inv);
#pragma unroll
            for (int y = 0; y < 16; ++y) zero = bf16x2_fma(w[y], 0u, zero);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              *reinterpret_cast<uint4*>(stg + lane * 128 + (((4 * c + y) ^ (lane & 7)) << 4)) =
                  make_uint4(w[4 * y], w[4 * y + 1], w[4 * y + 2], w[4 * y + 3]);
          }
          if (h == 1) {
            fence_before_sync();  // the tensor-memory reads above precede the arrive
            mbar_arrive(&sm.o_free[x]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (tok_w + kOutTok <= job.nq) {
            if (lane == 0) {
              tma_store_3d(&out_map, stg, 64 * h, job.kvh * kGroup, job.tok0 + tok_w);
              bulk_commit();
            }
          } else {  // the row's last tokens
#pragma unroll 1
            for (int i = lane >> 3; i < kGroup * (job.nq - tok_w); i += 4) {
              const size_t at = (size_t)(job.tok0 + tok_w + (i >> 2)) * p.num_q_heads + job.kvh * kGroup + (i & 3);
              *reinterpret_cast<uint4*>(p.out + at * kHeadDim + 64 * h + 8 * (lane & 7)) =
                  *reinterpret_cast<const uint4*>(stg + 128 * i + (((lane ^ i) & 7) << 4));
            }
            __syncwarp();  // (read before the next 64 dims go there)
          }
        }
        if ((zero & 0x7fff7fffu) != 0u && tok < job.nq) *reinterpret_cast<volatile int*>(&sm.odd) = 1;
        if (p.lse && tok < job.nq)
          p.lse[(size_t)(job.tok0 + tok) * p.num_q_heads + job.kvh * kGroup + (row & 3)] = lse * kLn2;
      }
      R0 += job.n_sub;
      I0 += job.n_sub;
      job = after;
    }
    if (lane == 0) bulk_wait_all();  // the stores have been written
    __syncwarp();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == kScoreWarp) tmem_dealloc(tmem, kTmemCols);
  if (sm.odd && !sm.abort) mend_jobs<kCut>(p, items);  // (rare)
}

// The outputs of cut jobs: the log-sum-exp merge of their parts, in order.  A CTA takes 32
// dims of a query tile's 128 rows, a thread 16 dims of a row.  The parts lie as 4 dims of
// neighbouring rows, so a warp reads 512 bytes at once.
__global__ void __launch_bounds__(256) merge_window_kernel(const __grid_constant__ WindowParams p,
                                                           const __grid_constant__ WindowCuts cuts) {
  pdl_launch_dependents();
  pdl_wait();
  const WindowCut cut = cuts.cut[blockIdx.x];
  const int x = blockIdx.y, row = threadIdx.x & 127, tok = x * kTok + (row >> 2);
  if (x * kTok >= cut.nq) return;
  // rows of part i: with CTA b0's last job, unless that is its first; the others with their
  // CTAs' first
  auto at = [&](int i) { return ((size_t)(i == 0 ? cut.slot0 : 2 * (cut.b0 + i)) * 2 + x) * kRows; };
  float m = -INFINITY;
#pragma unroll 4
  for (int i = 0; i < cut.parts; ++i) m = max_nan(m, load_cg(p.part_lse + at(i) + row));
  const float ref = m == -INFINITY ? 0.f : m;
  const int c = blockIdx.z * 8 + 4 * (threadIdx.x >> 7);  // dims 4 c .. 4 c + 15
  float l = 0.f;
  float4 o[4];
#pragma unroll
  for (int y = 0; y < 4; ++y) o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < cut.parts; ++i) {
    const float w = fast_exp2(load_cg(p.part_lse + at(i) + row) - ref);
    const float4* src = reinterpret_cast<const float4*>(p.part_o + at(i) * kHeadDim) + c * kRows + row;
    l += w;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const float4 a = load_cg(src + y * kRows);
      o[y] = make_float4(fmaf(w, a.x, o[y].x), fmaf(w, a.y, o[y].y), fmaf(w, a.z, o[y].z), fmaf(w, a.w, o[y].w));
    }
  }
  if (tok >= cut.nq) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const size_t orow = (size_t)(cut.tok0 + tok) * p.num_q_heads + cut.kvh * kGroup + (row & 3);
#pragma unroll
  for (int y = 0; y < 4; y += 2)
    *reinterpret_cast<uint4*>(p.out + orow * kHeadDim + 4 * (c + y)) =
        make_uint4(pack_bf16x2(o[y].x * inv, o[y].y * inv), pack_bf16x2(o[y].z * inv, o[y].w * inv),
                   pack_bf16x2(o[y + 1].x * inv, o[y + 1].y * inv), pack_bf16x2(o[y + 1].z * inv, o[y + 1].w * inv));
  if (p.lse && c == 0) p.lse[orow] = lse_log2(ref, l) * kLn2;
}

std::atomic<bool> g_attr_set[2][kMaxDevices];

template <bool kCut>
cudaError_t launch(const WindowParams& p, const WindowItems& items, const TcMaps& maps, const CUtensorMap& out_map, int ctas,
                   cudaStream_t stream) {
  const cudaError_t e = set_smem_limit_once((const void*)prefill_window_kernel<kCut>, (int)kSmemBytes, g_attr_set[kCut]);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefill_window_kernel<kCut>, dim3((unsigned)ctas), dim3(kThreads), kSmemBytes, stream, p, items, maps.q,
                    out_map, maps.k, maps.v);
}

}  // namespace

cudaError_t launch_prefill_window(const WindowParams& p, const WindowItems& items, bool cut, const TcMaps& maps,
                                  const CUtensorMap& out_map, int ctas, cudaStream_t stream) {
  // a zero scale (every score 0) as 2^-100, so that a hidden score scales to -inf:
  // scores of q and k whose products stay below 2^40 are below 2^-60 then and weigh 1
  // as before
  WindowParams pp = p;
  if (pp.scale_log2 == 0.f) pp.scale_log2 = 7.888609e-31f;
  return cut ? launch<true>(pp, items, maps, out_map, ctas, stream) : launch<false>(pp, items, maps, out_map, ctas, stream);
}

cudaError_t launch_merge_window(const WindowParams& p, const WindowCuts& cuts, int n, cudaStream_t stream) {
  return launch_pdl(merge_window_kernel, dim3((unsigned)n, 2, 4), dim3(256), 0, stream, p, cuts);
}

}  // namespace pa
