// Tensor-core tiles of attention with a sliding window: rows with more than eight
// queries (prompt chunks).
//
// What is computed: the query at position p sees keys t <= p with t < sinks or t > p -
// window; scores, softmax and output as in decode_window.cu.
//
// Work.  A job is up to 64 query tokens of a row for one kv head: two query tiles A and
// B of 32 tokens x 4 heads = 128 rows, the M of one tcgen05.mma each (a job of up to 32
// has A alone).  The pages that any of its queries sees (leading ones, then from the
// first query's window on) are counted through and go in key tiles of 128 (8 pages), so a
// job costs its window and its own length, not its context.  One CTA per SM runs its
// share of the jobs one after another without a barrier between them: rings, phases and
// buffers are indexed by running counts.
//
// Warps.  0-3 and 4-7: softmax of A and B, one thread per row (tensor-memory lane =
// row).  8 and 9: issue the products of A and of B (8 also copies Q by TMA and owns the
// tensor memory).  10 and 11: copy K and V by tiled TMA, a page's half of 64 dims per
// box.  12: clears V's rows that no query of the job sees, whose weight is 0 but which may
// hold infinities or NaN (only key tiles at the ends have any).
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
// Every wait is bounded; on a timeout the CTA records the error, lets its copies and
// products finish (bounded), frees its tensor memory and returns.
#include <math.h>
#include <stddef.h>

#include "internal.h"
#include "q4.cuh"  // lse_log2
#include "tc.cuh"
#include "window.cuh"

namespace pa {
namespace {

using namespace tc;

constexpr int kTok = kPrefillQTile;  // query tokens of a tile
constexpr int kRows = kTok * kGroup;
constexpr int kKeys = kTcKeyTile;
constexpr int kPagesPerTile = kKeys / kPage;
constexpr int kHalf = 128 * 128;  // 128 rows x 64 bf16
constexpr int kTileBytes = 2 * kHalf;
constexpr int kPageHalfBytes = kPage * 128;
constexpr int kStages = 2;  // of K and of V
constexpr int kMmaWarp = 8, kKWarp = 10, kVWarp = 11, kClearWarp = 12;  // (kMmaWarp + 1: tile B)
constexpr int kThreads = 13 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 for tile B
constexpr float kMaxSum = 1024.f;           // of 32 weights, before their row's reference is raised
constexpr int kOutTok = kQ4OutTok;          // query tokens of a softmax warp
constexpr int kSub = 64;                    // keys of a score product
constexpr int kPagesPerSub = kSub / kPage;
constexpr uint32_t kIdescS = idesc_bf16_f32(kRows, kSub, false);
constexpr uint32_t kIdescO = idesc_bf16_f32(kRows, kHeadDim, true);
static_assert(kRows == 128 && kKeys == 128 && kWindowTileTokens == 2 * kTok, "tile shape");
static_assert(kOutTok * kGroup == 32 && 4 * kOutTok == kTok, "a softmax warp's 32 rows are whole tokens");

struct __align__(1024) Smem {
  uint8_t q[2][kTileBytes];
  uint8_t k[kStages][kTileBytes];
  uint8_t v[kStages][kTileBytes];
  uint8_t out[8][32 * 128];  // a softmax warp's rows on their way out, 64 dims at a time
  uint64_t q_full, q_free;   // a job's Q has landed; its last scores are done
  uint64_t o_free[2];        // the softmax warps have read a job's output
  uint64_t k_full[kStages], k_empty[kStages];
  uint64_t v_full[kStages], v_ready[kStages], v_empty[kStages];  // landed; cleared; read
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // per query tile and buffer: phase i / 2 for sub-tile i
  uint64_t drained[2];  // every product issued by a query tile's warp has completed
  uint8_t bad_k[8][kPagesPerTile], bad_v[8][kPagesPerTile];  // of key tile j mod 8: pages outside the pool
  uint32_t tmem;
  int abort;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;  // + slack to align the base
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

__device__ __forceinline__ bool wait(Smem& sm, uint64_t* bar, uint32_t parity, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
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

struct Job {
  int32_t tok0;  // first query token of the job
  int32_t nq;    // its query tokens (1 .. 64)
  int32_t kvh;
  int32_t pos0;  // position of the first
  const int32_t* table;
  Seen seen;               // pages that any of its queries sees
  int32_t n_pages;         // how many
  int32_t n_tiles, n_sub;  // key tiles; sub-tiles of 64 keys (for both query tiles)
  int32_t n_x;             // query tiles
};

// The CTA's jobs: job b of every round of gridDim.x jobs, in reverse order on odd rounds
// (the items come longest first).
struct Jobs {
  const WindowParams& p;
  const WindowItems& items;
  int base, odd;
  __device__ __forceinline__ Jobs(const WindowParams& p_, const WindowItems& items_) : p(p_), items(items_), base(0), odd(0) {}
  __device__ __forceinline__ bool next(Job& job) {
    const int n = items.count * p.num_kv_heads, G = (int)gridDim.x;
    const int u = base + (odd ? G - 1 - (int)blockIdx.x : (int)blockIdx.x);
    if (u >= n) {  // (a last round that has no job for this CTA)
      base = n;
      return false;
    }
    base += G;
    odd ^= 1;
    const int it = u / p.num_kv_heads;
    const int4 item = items.item[it];  // request, first query token, its position, queries
    job.tok0 = item.y;
    job.nq = item.w;
    job.kvh = u - it * p.num_kv_heads;
    job.pos0 = item.z;
    job.table = p.block_tables + (size_t)item.x * p.max_blocks_per_req;
    job.seen = seen_pages(item.z + item.w, item.w, p.window, p.sink_tokens);
    job.n_pages = job.seen.count();
    job.n_tiles = (job.n_pages + kPagesPerTile - 1) / kPagesPerTile;
    job.n_sub = (job.n_pages + kPagesPerSub - 1) / kPagesPerSub;
    job.n_x = job.nq > kTok ? 2 : 1;
    return true;
  }
};

// Bits n .. 31 (n clamped to 0 .. 32).
__device__ __forceinline__ uint32_t bits_from(int n) { return n <= 0 ? 0xffffffffu : n >= 32 ? 0u : 0xffffffffu << n; }

// The keys of a page at position t0 that a query at `pos` sees, as bits 0 .. 15.
__device__ __forceinline__ uint32_t page_seen(int t0, int pos, int window, int sinks) {
  return ~bits_from(pos - t0 + 1) & (bits_from(pos - window + 1 - t0) | ~bits_from(sinks - t0)) & 0xffffu;
}

// Whether every query from position a to b sees every key of the pages v0 .. v1.
__device__ __forceinline__ bool all_seen(const Seen& seen, int v0, int v1, int a, int b, int window, int sinks) {
  const int first = seen.page(v0) * kPage, last = seen.page(v1) * kPage + kPage - 1;
  return last <= a && (first > b - window || last < sinks);
}

// Copies of K (is_k) or V: key tile by key tile, 8 lanes a page each.  J0: the CTA's key
// tiles before the job's.  False after a timeout.
__device__ __forceinline__ bool copy_tiles(Smem& sm, const Job& job, bool is_k, const CUtensorMap* map, int J0,
                                           int& last_issued, int num_kv_heads, int64_t num_blocks, int* err) {
  const int lane = threadIdx.x & 31;
  // pool rows four tiles at a time, one group ahead: lane l holds page l % 8 of tile 4 g +
  // l / 8; pages past the end repeat the last one (hidden, and V's cleared)
  auto load_group = [&](int g) -> int {
    const int t = 4 * g + (lane >> 3);
    if (t >= job.n_tiles) return 0;
    const int b = job.table[job.seen.page(min(t * kPagesPerTile + (lane & 7), job.n_pages - 1))];
    if (b < 0 || b >= num_blocks) {
      record_error(err, PA_ERR_DEVICE_INDEX);
      return -1;
    }
    return (b * num_kv_heads + job.kvh) * kPage;
  };
  int cur = load_group(0), next = load_group(1);
  uint64_t* full = is_k ? sm.k_full : sm.v_full;
  uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
  for (int j = 0; j < job.n_tiles; ++j) {
    const int J = J0 + j, s = J % kStages;
    if (j > 0 && (j & 3) == 0) {
      cur = next;
      next = load_group((j >> 2) + 1);
    }
    const int row = __shfl_sync(0xffffffffu, cur, ((j & 3) << 3) + (lane & 7));
    if (J >= kStages && !__all_sync(0xffffffffu, wait(sm, &empty[s], ((J / kStages) - 1) & 1, err))) return false;
    if (lane < kPagesPerTile) (is_k ? sm.bad_k : sm.bad_v)[J & 7][lane] = row < 0;
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(&full[s], kTileBytes);
    __syncwarp();
    uint8_t* dst = is_k ? sm.k[s] : sm.v[s];
    if (lane < kPagesPerTile) {
      const int off = lane * kPageHalfBytes;
      tma_load_2d(dst + off, map, 0, max(row, 0), &full[s]);
      tma_load_2d(dst + kHalf + off, map, 64, max(row, 0), &full[s]);
    }
    last_issued = J;
  }
  return true;
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_window_kernel(const WindowParams p, const __grid_constant__ WindowItems items,
                          const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap out_map,
                          const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (warp == kMmaWarp && lane == 0) {
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
      mbar_init(&sm.drained[x], 1);
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
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
    const bool is_k = warp == kKWarp;
    const CUtensorMap* map = is_k ? &k_map : &v_map;
    if (lane == 0) prefetch_tensormap(map);
    Jobs jobs(p, items);
    Job job;
    int J0 = 0, last = -1;
    bool ok = true;
    while (jobs.next(job) && (ok = copy_tiles(sm, job, is_k, map, J0, last, p.num_kv_heads, p.num_blocks, p.err)))
      J0 += job.n_tiles;
    if (!ok)  // gave up: the copies in flight land before the CTA leaves (bounded)
      for (int J = max(0, last - kStages + 1); J <= last; ++J)
        mbar_wait_bounded(&(is_k ? sm.k_full : sm.v_full)[J % kStages], (J / kStages) & 1);
  } else if (warp == kClearWarp) {
    // ------------------------------------------- V's rows that no query sees
    Jobs jobs(p, items);
    Job job;
    int J0 = 0;
    bool ok = true;
    while (ok && jobs.next(job)) {
      const int keys = job.pos0 + job.nq, low = max(job.pos0 - p.window + 1, 0);
      for (int j = 0; j < job.n_tiles; ++j) {
        const int J = J0 + j, s = J % kStages;
        ok = __all_sync(0xffffffffu, wait(sm, &sm.v_full[s], (J / kStages) & 1, p.err));
        if (!ok) break;
        bool cleared = false;
#pragma unroll 1
        for (int y = 0; y < kKeys / 32; ++y) {
          const int row = 32 * y + lane, v = j * kPagesPerTile + row / kPage;
          const int t = job.seen.page(v) * kPage + row % kPage;
          const bool hide = v >= job.n_pages || t >= keys || (t >= p.sink_tokens && t < low) ||
                            reinterpret_cast<volatile uint8_t*>(sm.bad_v[J & 7])[row / kPage];
          if (hide) {
            uint4* d = reinterpret_cast<uint4*>(sm.v[s] + row * 128);
#pragma unroll
            for (int c = 0; c < 8; ++c) d[c] = d[c + kHalf / 16] = make_uint4(0u, 0u, 0u, 0u);
            cleared = true;
          }
        }
        if (cleared) fence_proxy_async_smem();  // the products read the tile through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.v_ready[s]);
      }
      J0 += job.n_tiles;
    }
  } else if (warp >= kMmaWarp) {
    // --------------------------------------------------------- MMA issuers
    // The whole warp runs this (so that descriptors and addresses are warp-uniform
    // values) and one elected lane issues.
    const int x = warp - kMmaWarp;
    const uint64_t q_desc = desc_sw128(smem_addr(sm.q[0]), 16, 1024) + (uint32_t)x * (kTileBytes >> 4);
    const uint64_t k_desc = desc_sw128(smem_addr(sm.k[0]), 16, 1024);
    const uint64_t v_desc = desc_sw128(smem_addr(sm.v[0]), kHalf, 1024);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t t_s = tm + kColS + x * kKeys, t_o = tm + kColO + x * kHeadDim;
    auto arrived = [&](uint64_t* bar, int phase) {
      return __all_sync(0xffffffffu, wait(sm, bar, (uint32_t)phase & 1u, p.err)) != 0;
    };
    // running counts: key tiles, jobs, this query tile's sub-tiles and jobs, Qs loaded
    int J0 = 0, n_job = 0, I0 = 0, n_own = 0, n_q = 0;
    // Q of a job: after the last scores of the job before
    auto load_q = [&](const Job& job) {
      n_q += 1;
      if (elect_one()) {
        mbar_arrive_expect_tx(&sm.q_full, job.n_x * kTileBytes);
        for (int y = 0; y < job.n_x; ++y) {
          tma_load_3d(sm.q[y], &q_map, 0, job.kvh * kGroup, job.tok0 + y * kTok, &sm.q_full);
          tma_load_3d(sm.q[y] + kHalf, &q_map, 64, job.kvh * kGroup, job.tok0 + y * kTok, &sm.q_full);
        }
      }
      __syncwarp();
    };
    Jobs jobs(p, items);
    Job job, next;
    bool more = jobs.next(job), ok = true;
    if (x == 0 && more) load_q(job);
    while (more && ok) {
      if (x < job.n_x) {
        const int n_sub = job.n_sub;
        // scores of sub-tile i: 64 keys, half i & 1 of the job's key tile i / 2
        auto issue_s = [&](int i) {
          const int J = J0 + (i >> 1), b = (I0 + i) & 1;
          const uint64_t kd = k_desc + (uint32_t)(J % kStages) * (kTileBytes >> 4) + (uint32_t)(i & 1) * (kSub * 128 >> 4);
          const uint32_t on = elect_one();
          fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < kHeadDim / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;  // 64-dim half, 16-dim step in it
            mma_ss_if(on, t_s + b * kSub, q_desc + off, kd + off, kIdescS, ks > 0);
          }
          commit_if(on, &sm.s_full[x][b]);
          if ((i & 1) || i == n_sub - 1) commit_if(on, &sm.k_empty[J % kStages]);  // the tile's last use here
          if (i == n_sub - 1) commit_if(on, &sm.q_free);
        };
        auto issue_pv = [&](int i) {
          const int J = J0 + (i >> 1), b = (I0 + i) & 1;
          const uint64_t vd = v_desc + (uint32_t)(J % kStages) * (kTileBytes >> 4);
          const uint32_t on = elect_one();
          fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < kSub / 16; ++ks)  // 16 keys: two 8-row groups of V, 8 columns of weight pairs
            mma_ts_if(on, t_o, t_s + b * kSub + 8 * ks, vd + (uint32_t)((i & 1) * (kSub / 16) + ks) * (2 * 1024 >> 4),
                      kIdescO, (i > 0 || ks > 0) ? 1u : 0u);
          commit_if(on, &sm.pv_done[x][b]);
          if ((i & 1) || i == n_sub - 1) commit_if(on, &sm.v_empty[J % kStages]);
        };
        // before the scores of sub-tile i: its key tile, and the PV product of the
        // sub-tile whose weights lie where they go
        auto may_score = [&](int i) {
          const int J = J0 + (i >> 1), I = I0 + i;
          return ((i & 1) || arrived(&sm.k_full[J % kStages], J / kStages)) &&
                 (I < 2 || arrived(&sm.pv_done[x][I & 1], (I >> 1) - 1));
        };
        ok = ok && arrived(&sm.q_full, n_job);
        for (int i = 0; ok && i < min(n_sub, 2); ++i)
          if ((ok = may_score(i))) issue_s(i);
        more = jobs.next(next);
        // the first PV product overwrites the output of this tile's job before
        ok = ok && (n_own == 0 || arrived(&sm.o_free[x], n_own - 1));
        for (int i = 0; ok && i < n_sub; ++i) {
          const int J = J0 + (i >> 1), I = I0 + i;
          if (x == 0 && more && i == n_sub - 1) {  // the next job's Q, while the softmax has the last scores
            ok = arrived(&sm.q_free, n_job);
            if (!ok) break;
            load_q(next);
          }
          ok = ((i & 1) || arrived(&sm.v_ready[J % kStages], J / kStages)) && arrived(&sm.p_full[x][I & 1], I >> 1);
          if (!ok) break;
          issue_pv(i);
          if (i + 2 < n_sub && (ok = may_score(i + 2))) issue_s(i + 2);
        }
        I0 += n_sub;
        n_own += 1;
      } else {
        // a job without this tile: every phase is waited for in turn all the same (a
        // wait by parity tells a phase only from its neighbours), and every stage
        // given back
        auto pass = [&](uint64_t* full, uint64_t* empty, int phase) {
          ok = ok && arrived(full, phase);
          if (ok && lane == 0) mbar_arrive(empty);
          __syncwarp();
        };
        pass(&sm.q_full, &sm.q_free, n_job);
        for (int j = 0; j < job.n_tiles; ++j) {
          const int J = J0 + j;
          pass(&sm.k_full[J % kStages], &sm.k_empty[J % kStages], J / kStages);
          pass(&sm.v_ready[J % kStages], &sm.v_empty[J % kStages], J / kStages);
        }
        more = jobs.next(next);
      }
      J0 += job.n_tiles;
      n_job += 1;
      job = next;
    }
    // every product issued has completed before the tensor memory is freed (a commit
    // tracks all of them), and Q has landed before the CTA leaves
    commit_if(elect_one(), &sm.drained[x]);
    mbar_wait_bounded(&sm.drained[x], 0);
    if (n_q > 0) mbar_wait_bounded(&sm.q_full, (uint32_t)(n_q - 1) & 1u);
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    const int x = warp >> 2;
    const int row = threadIdx.x & 127;  // 4 * token + head in group
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_o = lane_base + kColO + x * kHeadDim;
    const float scale = p.scale_log2;  // not 0 (see the launch)
    int J0 = 0, I0 = 0;  // running counts: key tiles, this query tile's sub-tiles
    Jobs jobs(p, items);
    Job job;
    bool more = jobs.next(job), ok = true;
    while (more) {
      if (x >= job.n_x) {
        J0 += job.n_tiles;
        more = jobs.next(job);
        continue;
      }
      const int a = job.pos0 + x * kTok, b = min(a + kTok, job.pos0 + job.nq) - 1;  // the tile's positions
      const int pos = a + (row >> 2);
      float m_run = -INFINITY, l_run = 0.f;
      for (int i = 0; i < job.n_sub; ++i) {
        const int I = I0 + i;
        const uint32_t t_s = lane_base + kColS + x * kKeys + (I & 1) * kSub;
        ok = __all_sync(0xffffffffu, wait(sm, &sm.s_full[x][I & 1], (I >> 1) & 1, p.err));
        if (!ok) break;
        fence_after_sync();
        // bytes of its 4 pages
        const uint32_t bad =
            reinterpret_cast<volatile uint32_t*>(sm.bad_k[(J0 + (i >> 1)) & 7])[i & 1];
        const int v0 = i * kPagesPerSub;
        const bool masked = v0 + kPagesPerSub > job.n_pages || bad != 0u ||
                            !all_seen(job.seen, v0, v0 + kPagesPerSub - 1, a, b, p.window, p.sink_tokens);
        const uint32_t hide = scale >= 0.f ? 0xff800000u : 0x7f800000u;  // scales to -inf
        // One pass over the scores, 32 keys at a time, the next ones' load in flight.
        // The weights are taken against the row's reference m_run first; only when
        // their sum shows that it lies too low (or there is none yet) the maximum is
        // looked for, m_run re-based to it, and the output and the weights stored so
        // far rescaled.  After a row's first keys that is rare.
        float2 ls = make_float2(0.f, 0.f);
        uint32_t buf[2][32];
        tmem_ld32_async(t_s, buf[0]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t(&c)[32] = buf[h & 1];
          wait_ld(c);
          if (h < 1) tmem_ld32_async(t_s + 32 * (h + 1), buf[(h + 1) & 1]);
          if (masked) {
            uint32_t see = 0u;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int v = v0 + 2 * h + e;
              if (v < job.n_pages && ((bad >> (8 * (2 * h + e))) & 0xffu) == 0u)
                see |= page_seen(job.seen.page(v) * kPage, pos, p.window, p.sink_tokens) << (16 * e);
            }
#pragma unroll
            for (int y = 0; y < 32; ++y)
              if (!((see >> y) & 1u)) c[y] = hide;
          }
          uint32_t w[16];
          float2 sum;
          for (bool again = false;; again = true) {
            const float nm = (m_run == -INFINITY) ? 0.f : -m_run;
            const float2 sc2 = make_float2(scale, scale), nm2 = make_float2(nm, nm);
            float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              const float2 d = __ffma2_rn(make_float2(__uint_as_float(c[2 * y]), __uint_as_float(c[2 * y + 1])), sc2, nm2);
              const float2 e = make_float2(fast_exp2(d.x), fast_exp2(d.y));
              s2[y & 1] = __fadd2_rn(s2[y & 1], e);
              w[y] = pack_bf16x2(e.x, e.y);
            }
            sum = __fadd2_rn(s2[0], s2[1]);
            const bool low = sum.x + sum.y > kMaxSum || m_run == -INFINITY;
            if (again || !__any_sync(0xffffffffu, low)) break;
            if (h < 1) wait_ld(buf[(h + 1) & 1]);  // nothing in flight across the call
            float mt = -INFINITY;
#pragma unroll
            for (int y = 0; y < 32; ++y) mt = fmaxf(mt, __uint_as_float(c[y]) * scale);
            const bool grow = low && mt > m_run;
            const float corr = grow ? fast_exp2(m_run - mt) : 1.f;  // m_run = -inf -> 0
            if (grow) m_run = mt;
            l_run *= corr;
            ls = __fmul2_rn(ls, make_float2(corr, corr));
            if (i > 0) {  // O is stable once PV of the sub-tile before is done
              ok = __all_sync(0xffffffffu, wait(sm, &sm.pv_done[x][(I - 1) & 1], ((I - 1) >> 1) & 1, p.err));
              if (!ok) break;
              fence_after_sync();
            }
            rescale(t_o, t_s, h, i > 0, corr);
          }
          ls = __fadd2_rn(ls, sum);
          store16(t_s + 16 * h, w);  // weights over scores already read
        }
        if (!ok) break;
        l_run += ls.x + ls.y;
        wait_st();
        fence_before_sync();  // the tensor-memory accesses above precede the arrive
        mbar_arrive(&sm.p_full[x][I & 1]);
      }
      if (!ok) break;
      const int I1 = I0 + job.n_sub - 1;
      if (!__all_sync(0xffffffffu, wait(sm, &sm.pv_done[x][I1 & 1], (I1 >> 1) & 1, p.err))) break;
      fence_after_sync();
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      // The output, 64 dims at a time, through shared memory (128-byte swizzle) and out
      // by TMA, the warp's 8 tokens x 4 heads x 64 dims.
      const int tok = x * kTok + (row >> 2);
      const int tok_w = x * kTok + kOutTok * (warp & 3);  // the warp's first token
      uint8_t* stg = sm.out[warp];
      uint32_t o[2][32];
      tmem_ld32_async(t_o, o[0]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (lane == 0) bulk_wait_read();  // what was staged before has been read
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          wait_ld(o[c]);
          if (h == 0 || c == 0) tmem_ld32_async(t_o + 64 * h + 32 * (c + 1), o[c ^ 1]);
          uint32_t w[16];
#pragma unroll
          for (int y = 0; y < 16; ++y)
            w[y] = pack_bf16x2(__uint_as_float(o[c][2 * y]) * inv, __uint_as_float(o[c][2 * y + 1]) * inv);
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
      if (p.lse && tok < job.nq)
        p.lse[(size_t)(job.tok0 + tok) * p.num_q_heads + job.kvh * kGroup + (row & 3)] = lse_log2(m_run, l_run) * kLn2;
      J0 += job.n_tiles;
      I0 += job.n_sub;
      more = jobs.next(job);
    }
    if (lane == 0) bulk_wait_all();  // the stores have been written
    __syncwarp();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

std::atomic<bool> g_attr_set[kMaxDevices];

}  // namespace

cudaError_t launch_prefill_window(const WindowParams& p, const WindowItems& items, const TcMaps& maps,
                                  const CUtensorMap& out_map, int ctas, cudaStream_t stream) {
  if (items.count <= 0) return cudaSuccess;
  // a zero scale (every score 0) as 2^-100, so that a hidden score scales to -inf:
  // scores of q and k whose products stay below 2^40 are below 2^-60 then and weigh 1
  // as before
  WindowParams pp = p;
  if (pp.scale_log2 == 0.f) pp.scale_log2 = 7.888609e-31f;
  const cudaError_t e = set_smem_limit_once((const void*)prefill_window_kernel, (int)kSmemBytes, g_attr_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefill_window_kernel, dim3((unsigned)ctas), dim3(kThreads), kSmemBytes, stream, pp, items, maps.q,
                    out_map, maps.k, maps.v);
}

}  // namespace pa
