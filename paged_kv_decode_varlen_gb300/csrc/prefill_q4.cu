// Tensor-core tiles of attention over 4-bit pages: rows with several query
// tokens (prompt chunks, verify rows).
//
// What is computed: query j of a row with h cached tokens sits at position
// h + j and attends to keys 0 .. h + j; scores, softmax and output as in
// decode_q4.cu, keys and values the bf16 numbers that the codes stand for.
//
// Work.  A job is up to 64 query tokens of a row for one kv head: two query tiles
// A and B of 32 tokens x 4 heads = 128 rows, the M of one tcgen05.mma each (B is
// left out of a job of up to 32, which the host also makes of longer rows where
// jobs of 64 would leave SMs idle), against key tiles of 128 (8 pages).  One CTA
// per SM runs its share of the jobs one after another without a barrier between
// them: rings, phases and buffers are indexed by running counts, so the next
// job's Q, first key tiles and first scores are made while the softmax warps
// finish this one (8 prompts of 100 to 1000 tokens, 32 heads: 44.0 us, where a
// CTA per job took 56).  The two tiles share every dequantised K and V tile.
//   Bound.  Per key tile of 128 the products take 2560 cycles of the tensor
// cores, the instructions of all warps some 2330 of the schedulers'; the whole
// takes some 3400 (4 chunks of 512 tokens, 4096 to 8192 keys: 174 us, 1115
// TFLOP/s, 24 us of it uneven work: 256 whole jobs on 152 SMs, the busiest of
// which has 91 key tiles, the mean 77.5): a warp that issues products or turns
// scores into weights waits for its turn among four on a scheduler.  The loops of
// the three roles fill the instruction cache, so code counts: a third slot of
// read-ahead in the producers costs 5 % of the prompts' time, two loops kept apart
// in the issuing warps save 8 % against a merged one.
//
// Warps.  0-3 and 4-7: softmax of A and B, one thread per row (tensor-memory
// lane = row).  8 and 9: issue the products of A and of B (8 also copies Q by
// TMA and owns the tensor memory).  10-15: producers.  A unit of their work is
// one page's K or V slab: each lane reads two 16-byte pieces of codes (tokens t
// and t + 8 of one group) and their (D, Z), two units ahead, and writes 64
// bf16 values into the 128-byte-swizzled operand tile.  A key tile is 16 units,
// dealt out to the six warps in turn.  (Dequantised once per CTA in registers: a
// second copy of the cache in bf16 is never made.)
//   With the schedulers busy an issuing warp is slow (some 20 cycles per
// instruction), so each query tile has its own, in a fixed order of few waits: one
// warp that polled for whichever product was ready took 3000 cycles per round of
// four.
//
// Tensor memory: per query tile two score buffers of 64 keys and the output,
// 128 columns; that is all 512.  Scores are therefore made 64 keys at a time
// (a sub-tile), and a sub-tile's weights (bf16 pairs, the A operand of the PV
// product) overwrite its scores: the scores of sub-tile i + 1 are there when
// the softmax has finished sub-tile i, and those of i + 2 follow the PV product
// of i.  (With one buffer of 128 keys each score product waited for the PV
// product before it: 206 us for the late chunks against 186 at that step,
// although 64 columns of B make a score product read its Q tile at the shared
// memory's limit, 48 cycles for 32.)  The softmax takes the scores once, 32
// columns at a time, against a reference that is re-based only when weights get
// large.  Weights are rounded to bf16, as the tensor cores take them; their sum
// is kept in binary32 from the unrounded ones, as are scores, maxima and outputs.
//
// Every wait is bounded; on a timeout the CTA records the error, lets its
// copies and products finish (bounded), frees its tensor memory and returns.
#include <math.h>
#include <stddef.h>

#include "internal.h"
#include "q4.cuh"
#include "tc.cuh"

namespace pa {
namespace {

using namespace tc;

constexpr int kTok = kPrefillQTile;          // query tokens of a tile
constexpr int kRows = kTok * kGroup;         // 128
constexpr int kKeys = kTcKeyTile;            // 128 keys per tile
constexpr int kPagesPerTile = kKeys / kPage;
constexpr int kHalf = 128 * 128;             // 128 rows x 64 bf16
constexpr int kTileBytes = 2 * kHalf;
constexpr int kKStages = 2, kVStages = 2;
constexpr int kMmaWarp = 8, kProducer0 = 10, kProducers = 6;  // (kMmaWarp + 1: tile B)
constexpr int kThreads = (kProducer0 + kProducers) * 32;
constexpr int kUnits = 2 * kPagesPerTile;    // slabs of a key tile
constexpr int kAhead = 2;                    // units a producer warp reads ahead
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;   // + 128 for tile B
constexpr float kMaxSum = 1024.f;  // of 32 weights, before their row's reference is raised
constexpr int kOutTok = kQ4OutTok;           // query tokens of a softmax warp
constexpr int kSub = 64;                     // keys of a score product
constexpr uint32_t kIdescS = idesc_bf16_f32(kRows, kSub, false);
constexpr uint32_t kIdescO = idesc_bf16_f32(kRows, kHeadDim, true);
static_assert(kRows == 128 && kKeys == 128 && kQ4TileTokens == 2 * kTok, "tile shape");
static_assert(kOutTok * kGroup == 32 && 4 * kOutTok == kTok, "a softmax warp's 32 rows are whole tokens");
static_assert(2 * 32 * 16 == kQ4Codes, "two pieces of codes per lane");
static_assert(kKStages == kVStages, "one ring depth");

struct __align__(1024) Smem {
  uint8_t q[2][kTileBytes];
  uint8_t k[kKStages][kTileBytes];
  uint8_t v[kVStages][kTileBytes];
  uint8_t out[8][32 * 128];  // a softmax warp's rows on their way out, 64 dims at a time
  uint64_t q_full, q_free;  // a job's Q has landed; its last scores are done
  uint64_t o_free[2];       // the softmax warps have read a job's output
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // per query tile and buffer: phase i / 2 for sub-tile i
  uint64_t drained[2];  // every product issued by a query tile's warp has completed
  uint64_t bad[8];   // byte u of entry j % 8: page u of key tile j has a block id outside the pool
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

// 1 in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one;
}

// tc::mma_bf16, tc::mma_bf16_ts and tc::commit by the lanes with `on` set,
// without a branch: run by a whole warp whose control flow is warp-uniform, the
// descriptors stay uniform registers and a product is one instruction (in a
// branch of one lane they cost six, and with the schedulers busy a group of
// eight took 890 cycles to issue against 514 to run).
__device__ __forceinline__ void mma_ss_if(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(on)
      : "memory");
}

// Waits for this thread's tensor-memory loads; `r` is bound to the wait.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  tmem_bind32(r);
}
// 16 columns of this thread's lane, without a wait (wait_st) / with its wait
__device__ __forceinline__ void store16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// A row's maximum grew (rare): scales its output columns, and the weights of
// the tile's first `quarters` quarters already stored, by corr.  Whole warp;
// out of line to keep its registers off the softmax loop.
__device__ __noinline__ void rescale(uint32_t t_o, uint32_t t_p, int quarters, bool has_o, float corr) {
  wait_st();
  if (has_o) {
#pragma unroll 1
    for (int c = 0; c < kHeadDim; c += 16) {
      uint32_t o[16];
      load16(t_o + c, o);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
      store16(t_o + c, o);
    }
  }
#pragma unroll 1
  for (int c = 0; c < 16 * quarters; c += 16) {
    uint32_t w[16];
    load16(t_p + c, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(bf16lo(w[i]) * corr, bf16hi(w[i]) * corr);
    store16(t_p + c, w);
  }
  wait_st();
}

// A box of a tensor map from shared to global memory, in the thread's current
// group of bulk copies; groups; and waits for all of the thread's groups to have
// read shared memory / to have been written.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(smem_addr(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

struct Job {  // (split: positions and keys from the range's first key on)
  int32_t tok0;  // first query token of the job
  int32_t nq;    // its query tokens (1 .. 64)
  int32_t kvh;
  int32_t pos0;  // position of the first
  int32_t keys;  // keys its last query sees
  const int32_t* table;
  int32_t n_tiles, n_sub;  // key tiles; sub-tiles of 64 keys (for both query tiles)
  int32_t n_x;             // query tiles
};

// The CTA's jobs: job b of every round of gridDim.x jobs, in reverse order on
// odd rounds (the items come longest first).  kSplit: job b, the only round.
template <class Items, bool kSplit>
struct Jobs {
  const PrefillParams& p;
  const Items& items;
  int base, odd;
  __device__ __forceinline__ Jobs(const PrefillParams& p_, const Items& items_) : p(p_), items(items_), base(0), odd(0) {}
  __device__ __forceinline__ bool next(Job& job) {
    if (kSplit && base > 0) return false;  // one job per CTA
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
    job.nq = kSplit ? item.w & 0xff : item.w;
    job.kvh = u - it * p.num_kv_heads;
    job.pos0 = item.z;
    job.keys = item.z + job.nq;
    job.table = p.block_tables + (size_t)item.x * p.max_blocks_per_req;
    if constexpr (kSplit) {
      const int key0 = (item.w >> 8) * items.split.tiles * kKeys;
      job.pos0 -= key0;
      job.keys = min(job.keys - key0, items.split.tiles * kKeys);
      job.table += key0 / kPage;
    }
    job.n_tiles = (job.keys + kKeys - 1) / kKeys;
    job.n_sub = (job.keys + kSub - 1) / kSub;
    job.n_x = job.nq > kTok ? 2 : 1;
    return true;
  }
};

// Producer warp w: units w, w + 6, ... of the job (unit u: key tile u / 16, K
// pages 0 .. 7, then V pages 0 .. 7); J0: the CTA's key tiles before the job's.
// False after a timeout.
__device__ __forceinline__ bool produce(Smem& sm, const Job& job, int w, int J0, const uint8_t* k_cache,
                                        const uint8_t* v_cache, int num_kv_heads, int64_t num_blocks, int* err) {
  const int lane = threadIdx.x & 31;
  const int t = lane >> 2, g = (lane & 3) ^ ((t >> 1) & 3);  // tokens t and t + 8 of group g
  const int last_page = (job.keys - 1) / kPage;
  const int n_units = job.n_tiles * kUnits;
  // block id of the warp's unit n (lane l of a batch: unit 32 B + l), a batch
  // ahead; -1: past the row's keys, -2: outside the pool
  auto load_ids = [&](int n0) -> int {
    const int u = w + kProducers * (n0 + lane);
    const int page = (u / kUnits) * kPagesPerTile + (u & (kPagesPerTile - 1));
    if (u >= n_units || page > last_page) return -1;
    const int32_t b = job.table[page];
    if (b < 0 || b >= num_blocks) {
      record_error(err, PA_ERR_DEVICE_INDEX);
      return -2;
    }
    return b;
  };
  int ids = load_ids(0), ids_next = load_ids(32);
  // Row t of a page, 16-byte chunk c of its 64-dim half at c ^ (t & 7).  The
  // words of groups 2 and 3 are taken in the order 2, 3, 0, 1, so that the eight
  // lanes of a store phase (2 tokens x 4 groups) meet eight chunks.
  const int swap = g & 2;
  uint32_t at[4];
#pragma unroll
  for (int x = 0; x < 4; ++x)
    at[x] = (g >> 1) * kHalf + t * 128 + (((((g & 1) << 2) + (x ^ swap)) ^ (t & 7)) << 4);
  const uint32_t code_at = 16 * lane + 4 * swap, dz_at = q4_scale_at(t, g);
  uint2 code[kAhead][2][2];  // per piece: words 0, 1 and words 2, 3 (in the order taken)
  uint32_t dz[kAhead][2];
  bool bad[kAhead];
  // unit n into slot d; a key past the end, or of a page outside the pool, becomes 0
  auto fetch = [&](int n, int d) {
    if (n > 0 && (n & 31) == 0) {
      ids = ids_next;
      ids_next = load_ids(n + 32);
    }
    const int id = __shfl_sync(0xffffffffu, ids, n & 31);
    const int u = w + kProducers * n;
    const int left = job.keys - ((u / kUnits) * kPagesPerTile + (u & (kPagesPerTile - 1))) * kPage;
    const uint8_t* slab =
        ((u & kPagesPerTile) ? v_cache : k_cache) + ((size_t)max(id, 0) * num_kv_heads + job.kvh) * kQ4Slab;
    bad[d] = id == -2;
    auto load = [&](int y) {  // tokens t + 8 y
      code[d][y][0] = load_cg(reinterpret_cast<const uint2*>(slab + 512 * y + code_at));
      code[d][y][1] = load_cg(reinterpret_cast<const uint2*>(slab + 512 * y + (code_at ^ 8u)));
      dz[d][y] = load_cg(reinterpret_cast<const uint32_t*>(slab + 8 * 4 * kQ4Groups * y + dz_at));
    };
    if (id >= 0 && left >= kPage) {
      load(0);
      load(1);
      return;
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      code[d][y][0] = code[d][y][1] = make_uint2(0u, 0u);
      dz[d][y] = 0u;
      if (id >= 0 && t + 8 * y < left) load(y);
    }
  };
#pragma unroll
  for (int d = 0; d < kAhead; ++d) fetch(d, d);
  for (int n0 = 0; w + kProducers * n0 < n_units; n0 += kAhead) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const int n = n0 + d, u = w + kProducers * n;
      if (u >= n_units) return true;
      const int j = J0 + u / kUnits, pg = u & (kPagesPerTile - 1), s = j % kKStages;
      const bool is_v = u & kPagesPerTile;
      if (!is_v && lane == 0) reinterpret_cast<volatile uint8_t*>(&sm.bad[j & 7])[pg] = bad[d];
      if (j >= kKStages &&
          !__all_sync(0xffffffffu, wait(sm, is_v ? &sm.v_empty[s] : &sm.k_empty[s], ((j / kKStages) - 1) & 1, err)))
        return false;
      const uint32_t dst = smem_addr(is_v ? sm.v[s] : sm.k[s]) + pg * (kPage * 128);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t z = dz[d][y];
        const uint32_t word[4] = {code[d][y][0].x, code[d][y][0].y, code[d][y][1].x, code[d][y][1].y};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint4 val = q4_word_values(word[x], z);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + y * (8 * 128) + at[x]), "r"(val.x),
                       "r"(val.y), "r"(val.z), "r"(val.w)
                       : "memory");
        }
      }
      fetch(n + kAhead, d);
      fence_proxy_async_smem();  // the products read the tile through the async proxy
      __syncwarp();
      if (lane == 0) mbar_arrive(is_v ? &sm.v_full[s] : &sm.k_full[s]);
    }
  }
  return true;
}

template <class Items, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_q4_kernel(const PrefillParams p, const __grid_constant__ Items items,
                      const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap out_map) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // roles by warp: hardware warp 0 is role 8 (the issuing warps first: 43.7 us
  // against 44.3 for the prompts above; a role keeps its warp number modulo 4,
  // which names its tensor-memory lanes)
  const int warp = __shfl_sync(0xffffffffu, (((int)threadIdx.x >> 5) + kMmaWarp) & 15, 0), lane = threadIdx.x & 31;
  if (warp == kMmaWarp && lane == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_free, 2);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&sm.k_full[s], kPagesPerTile);
      mbar_init(&sm.k_empty[s], 2);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&sm.v_full[s], kPagesPerTile);
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
  // nothing above touches what an earlier kernel may write (the jobs come with
  // the parameters)
  pdl_wait();
  pdl_launch_dependents();

  if (warp >= kProducer0) {
    Jobs<Items, kSplit> jobs(p, items);
    Job job;
    int J0 = 0;
    while (jobs.next(job) &&
           produce(sm, job, warp - kProducer0, J0, reinterpret_cast<const uint8_t*>(p.k_cache),
                   reinterpret_cast<const uint8_t*>(p.v_cache), p.num_kv_heads, p.num_blocks, p.err))
      J0 += job.n_tiles;
  } else if (warp >= kMmaWarp) {
    // --------------------------------------------------------- MMA issuers
    // The whole warp runs this (so that descriptors and addresses are
    // warp-uniform values) and one elected lane issues.
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
    Jobs<Items, kSplit> jobs(p, items);
    Job job, next;
    bool more = jobs.next(job), ok = true;
    if (x == 0 && more) load_q(job);
    while (more && ok) {
      if (x < job.n_x) {
        const int n_sub = job.n_sub;
        // scores of sub-tile i: 64 keys, half i & 1 of the job's key tile i / 2
        auto issue_s = [&](int i) {
          const int J = J0 + (i >> 1), b = (I0 + i) & 1;
          const uint64_t kd = k_desc + (uint32_t)(J % kKStages) * (kTileBytes >> 4) + (uint32_t)(i & 1) * (kSub * 128 >> 4);
          const uint32_t on = elect_one();
          fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < kHeadDim / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;  // 64-dim half, 16-dim step in it
            mma_ss_if(on, t_s + b * kSub, q_desc + off, kd + off, kIdescS, ks > 0);
          }
          commit_if(on, &sm.s_full[x][b]);
          if ((i & 1) || i == n_sub - 1) commit_if(on, &sm.k_empty[J % kKStages]);  // the tile's last use here
          if (i == n_sub - 1) commit_if(on, &sm.q_free);
        };
        auto issue_pv = [&](int i) {
          const int J = J0 + (i >> 1), b = (I0 + i) & 1;
          const uint64_t vd = v_desc + (uint32_t)(J % kVStages) * (kTileBytes >> 4);
          const uint32_t on = elect_one();
          fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < kSub / 16; ++ks)  // 16 keys: two 8-row groups of V, 8 columns of weight pairs
            mma_ts_if(on, t_o, t_s + b * kSub + 8 * ks, vd + (uint32_t)((i & 1) * (kSub / 16) + ks) * (2 * 1024 >> 4),
                      kIdescO, (i > 0 || ks > 0) ? 1u : 0u);
          commit_if(on, &sm.pv_done[x][b]);
          if ((i & 1) || i == n_sub - 1) commit_if(on, &sm.v_empty[J % kVStages]);
        };
        // before the scores of sub-tile i: its key tile, and the PV product of
        // the sub-tile whose weights lie where they go
        auto may_score = [&](int i) {
          const int J = J0 + (i >> 1), I = I0 + i;
          return ((i & 1) || arrived(&sm.k_full[J % kKStages], J / kKStages)) &&
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
          ok = ((i & 1) || arrived(&sm.v_full[J % kVStages], J / kVStages)) && arrived(&sm.p_full[x][I & 1], I >> 1);
          if (!ok) break;
          issue_pv(i);
          if (i + 2 < n_sub && (ok = may_score(i + 2))) issue_s(i + 2);
        }
        I0 += n_sub;
        n_own += 1;
      } else {
        // a job without this tile: every phase is waited for in turn all the
        // same (a wait by parity tells a phase only from its neighbours), and
        // every stage given back
        auto pass = [&](uint64_t* full, uint64_t* empty, int phase) {
          ok = ok && arrived(full, phase);
          if (ok && lane == 0) mbar_arrive(empty);
          __syncwarp();
        };
        pass(&sm.q_full, &sm.q_free, n_job);
        for (int j = 0; j < job.n_tiles; ++j) {
          const int J = J0 + j;
          pass(&sm.k_full[J % kKStages], &sm.k_empty[J % kKStages], J / kKStages);
          pass(&sm.v_full[J % kVStages], &sm.v_empty[J % kVStages], J / kVStages);
        }
        more = jobs.next(next);
      }
      J0 += job.n_tiles;
      n_job += 1;
      job = next;
    }
    // every product issued has completed before the tensor memory is freed (a
    // commit tracks all of them), and Q has landed before the CTA leaves
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
    Jobs<Items, kSplit> jobs(p, items);
    Job job;
    bool more = jobs.next(job), ok = true;
    while (more) {
      if (x >= job.n_x) {
        J0 += job.n_tiles;
        more = jobs.next(job);
        continue;
      }
      const int pos = job.pos0 + x * kTok + (row >> 2);
      float m_run = -INFINITY, l_run = 0.f;
      for (int i = 0; i < job.n_sub; ++i) {
        const int I = I0 + i;
        const uint32_t t_s = lane_base + kColS + x * kKeys + (I & 1) * kSub;
        ok = __all_sync(0xffffffffu, wait(sm, &sm.s_full[x][I & 1], (I >> 1) & 1, p.err));
        if (!ok) break;
        fence_after_sync();
        const int kbase = i * kSub;
        // bytes of its 4 pages
        const uint32_t bad = reinterpret_cast<volatile uint32_t*>(&sm.bad[(J0 + (i >> 1)) & 7])[i & 1];
        // hidden keys: after the row's position, past the end, of a bad page
        const bool masked = kbase + kSub - 1 > job.pos0 + x * kTok || kbase + kSub > job.keys || bad != 0u;
        const int seen = min(pos, job.keys - 1) - kbase + 1;  // keys of the sub-tile before the first hidden one
        const uint32_t hide = scale >= 0.f ? 0xff800000u : 0x7f800000u;  // scales to -inf
        // One pass over the scores, 32 keys at a time, the next ones' load in
        // flight.  The weights are taken against the row's reference m_run first;
        // only when their sum shows that it lies too low (or there is none yet)
        // the maximum is looked for, m_run re-based to it, and the output and the
        // weights stored so far rescaled.  After a row's first keys that is rare.
        float2 ls = make_float2(0.f, 0.f);
        uint32_t buf[2][32];
        tmem_ld32_async(t_s, buf[0]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t(&c)[32] = buf[h & 1];
          wait_ld(c);
          if (h < 1) tmem_ld32_async(t_s + 32 * (h + 1), buf[(h + 1) & 1]);
          if (masked) {
            const uint32_t pages = bad >> (16 * h);  // bytes of pages 2 h and 2 h + 1
#pragma unroll
            for (int y = 0; y < 32; ++y)
              if (32 * h + y >= seen || (pages & (y < 16 ? 0xffu : 0xff00u))) c[y] = hide;
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
      if constexpr (kSplit) {
        // the row's part of this key range, 4 dims of 32 rows at a time
        const size_t at = (size_t)blockIdx.x * items.split.rows + x * kRows;
        float4* dst = reinterpret_cast<float4*>(items.split.piece_o + at * kHeadDim) + row;
#pragma unroll 1
        for (int c = 0; c < kHeadDim / 16; ++c) {
          uint32_t o[16];
          load16(t_o + 16 * c, o);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            dst[(4 * c + y) * kRows] =
                make_float4(__uint_as_float(o[4 * y]) * inv, __uint_as_float(o[4 * y + 1]) * inv,
                            __uint_as_float(o[4 * y + 2]) * inv, __uint_as_float(o[4 * y + 3]) * inv);
        }
        fence_before_sync();  // the tensor-memory reads above precede the arrive
        mbar_arrive(&sm.o_free[x]);
        items.split.piece_lse[at + row] = lse_log2(m_run, l_run);
      } else {
        // The output, 64 dims at a time, through shared memory (128-byte swizzle)
        // and out by TMA, the warp's 8 tokens x 4 heads x 64 dims.  (Stored by the
        // threads, 16 bytes of a row each, an instruction touches 32 lines: a job's
        // end took 6000 cycles against 2600, the prompts above 52 us against 47.)
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
          }
        }
        if (p.lse && tok < job.nq)
          p.lse[(size_t)(job.tok0 + tok) * p.num_q_heads + job.kvh * kGroup + (row & 3)] =
              lse_log2(m_run, l_run) * kLn2;
      }
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

// The outputs of split items: the log-sum-exp merge of their key ranges' parts,
// in order.  A CTA takes 32 dims of a query tile's 128 rows, a thread 16 dims of a
// row.  The parts lie as 4 dims of neighbouring rows, so a warp reads 512 bytes at
// once; the ranges' weights are shared by the CTA, so that nothing but the parts'
// loads, four ranges at a time, stands in the way of the sums.
template <class Items>
__global__ void __launch_bounds__(256) merge_q4_kernel(const PrefillParams p, const __grid_constant__ Items items) {
  __shared__ float weight[kQ4MaxRanges][kRows];
  pdl_launch_dependents();
  pdl_wait();
  const int u = blockIdx.x, x = blockIdx.y, row = threadIdx.x & 127;
  const int it = u / p.num_kv_heads, kvh = u - it * p.num_kv_heads;
  const int4 item = items.item[it];
  const int nq = item.w & 0xff, tok = x * kTok + (row >> 2);
  if (item.w >> 8 || x * kTok >= nq) return;  // not the item's first range, no such query tile
  const int n_tiles = (item.z + nq + kKeys - 1) / kKeys;
  const int n = (n_tiles + items.split.tiles - 1) / items.split.tiles;
  const size_t stride = (size_t)p.num_kv_heads * items.split.rows;  // rows from a range to the next
  const size_t at = (size_t)u * items.split.rows + x * kRows;
  const size_t orow = (size_t)(item.y + tok) * p.num_q_heads + kvh * kGroup + (row & 3);
  if (threadIdx.x < kRows) {
    const float* lse = items.split.piece_lse + at + row;
    float m = -INFINITY;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float v = load_cg(lse + i * stride);
      weight[i][row] = v;
      m = max_nan(m, v);
    }
    float l = 0.f;
    for (int i = 0; i < n; ++i) {
      const float w = m == -INFINITY ? 0.f : fast_exp2(weight[i][row] - m);
      weight[i][row] = w;
      l += w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = 0; i < n; ++i) weight[i][row] *= inv;
    if (p.lse && blockIdx.z == 0 && tok < nq) p.lse[orow] = lse_log2(m, l) * kLn2;
  }
  __syncthreads();
  const int c = blockIdx.z * 8 + 4 * (threadIdx.x >> 7);  // dims 4 c .. 4 c + 15
  const float4* src = reinterpret_cast<const float4*>(items.split.piece_o + at * kHeadDim) + c * kRows + row;
  float4 o[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float w = weight[i][row];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float4 a = load_cg(src + i * stride * (kHeadDim / 4) + v * kRows);
      o[v] = make_float4(fmaf(w, a.x, o[v].x), fmaf(w, a.y, o[v].y), fmaf(w, a.z, o[v].z), fmaf(w, a.w, o[v].w));
    }
  }
  if (tok >= nq) return;
#pragma unroll
  for (int v = 0; v < 4; v += 2)
    *reinterpret_cast<uint4*>(p.out + orow * kHeadDim + 4 * (c + v)) =
        make_uint4(pack_bf16x2(o[v].x, o[v].y), pack_bf16x2(o[v].z, o[v].w), pack_bf16x2(o[v + 1].x, o[v + 1].y),
                   pack_bf16x2(o[v + 1].z, o[v + 1].w));
}

std::atomic<bool> g_attr_set[3][kMaxDevices];

template <int N>
const Q4Items<N>& fill(int count, const int4* rows, const Q4Split& split) {
  static thread_local Q4Items<N> d;
  d.count = count;
  d.split = split;
  for (int i = 0; i < count; ++i) d.item[i] = rows[i];
  return d;
}

template <int N, bool kSplit>
cudaError_t launch(const PrefillParams& p, int count, const int4* rows, const Q4Split& split, const Q4Maps& maps, int ctas,
                   std::atomic<bool>* done, cudaStream_t stream) {
  auto kernel = prefill_q4_kernel<Q4Items<N>, kSplit>;
  const cudaError_t e = set_smem_limit_once((const void*)kernel, (int)kSmemBytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3((unsigned)ctas), dim3(kThreads), kSmemBytes, stream, p, fill<N>(count, rows, split),
                    maps.q, maps.out);
}

}  // namespace

cudaError_t launch_prefill_q4(const PrefillParams& p, int count, const int4* rows, const Q4Split& split,
                              const Q4Maps& maps, int ctas, cudaStream_t stream) {
  if (count <= 0) return cudaSuccess;
  // a zero scale (every score 0) as 2^-100, so that a hidden score scales to
  // -inf: scores of q and k whose products stay below 2^40 are below 2^-60 then
  // and weigh 1 as before
  PrefillParams pp = p;
  if (pp.scale_log2 == 0.f) pp.scale_log2 = 7.888609e-31f;
  if (split.tiles > 0) {
    if (count > kQ4FewItems) return cudaErrorInvalidValue;
    return launch<kQ4FewItems, true>(pp, count, rows, split, maps, ctas, g_attr_set[2], stream);
  }
  // (parameters of the size needed, as in the decode launch)
  if (count <= kQ4FewItems) return launch<kQ4FewItems, false>(pp, count, rows, split, maps, ctas, g_attr_set[0], stream);
  return launch<kMaxPrefillItems, false>(pp, count, rows, split, maps, ctas, g_attr_set[1], stream);
}

cudaError_t launch_merge_q4(const PrefillParams& p, int count, const int4* rows, const Q4Split& split,
                            cudaStream_t stream) {
  if (count <= 0) return cudaSuccess;
  if (count > kQ4FewItems) return cudaErrorInvalidValue;
  return launch_pdl(merge_q4_kernel<Q4Items<kQ4FewItems>>,
                    dim3((unsigned)(count * p.num_kv_heads), (unsigned)(split.rows / kRows), 4), dim3(256), 0, stream, p,
                    fill<kQ4FewItems>(count, rows, split));
}

}  // namespace pa
