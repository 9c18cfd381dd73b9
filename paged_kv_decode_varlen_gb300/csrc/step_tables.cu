// A step's block tables, slots, positions and query offsets from the requests'
// lengths.
//
// What is computed: exclusive sums over the requests of their new tokens, of the
// pages these need (ceil((c + n) / 16) - ceil(c / 16)) and of the pages given back,
// and from them every token's, granted page's and returned page's place: three
// flat lists, each entry of which finds its request by a search in the sums.
//
// Bound: latency.  The lists are short (a decode step of 64 requests moves 3 KB, a
// step of 8 Ki tokens 130 KB), so what counts is one launch and few dependent round
// trips: lengths -> sums -> ring or table entry -> store.  Every CTA of the launch
// makes all sums for itself from the lengths (R <= 1024: one load of each array
// per thread) and takes its share of the three lists; no CTA waits for another.
// The last one to arrive at a count writes what may lie where the others still had
// to read (lengths, ring state), so that these outputs may be their inputs.
#include "internal.h"

#include "common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// One request's step.
struct Row {
  int cached, n;        // tokens before, new tokens
  int had, has;         // pages before, after
  int a_lo, a_hi;       // pages given back: [a_lo, a_hi), then [b_lo, b_hi)
  int b_lo, b_hi;
  int seq, first;       // what it holds after the step
  __device__ __forceinline__ int granted() const { return has - had; }
  __device__ __forceinline__ int back() const { return a_hi - a_lo + (b_hi - b_lo); }
};

// `wait`: every row is taken as one that brings nothing.
__device__ __forceinline__ Row row_of(const TablesParams& p, int r, bool wait, bool* bad) {
  Row w;
  const int raw = p.new_tokens[r], c = p.cached_lens[r];
  const int first = p.first_page ? max(p.first_page[r], 0) : 0;
  const int c_max = min(p.max_blocks_per_req, PA_MAX_SEQ_LEN / kPage) * kPage;
  const bool c_bad = c < 0 || c > c_max;
  const bool n_bad = !c_bad && raw > c_max - c;
  if (bad) *bad = c_bad || n_bad;
  w.cached = c_bad ? 0 : c;
  w.n = (c_bad || n_bad || wait) ? 0 : max(raw, 0);
  const bool ended = raw < 0 && !c_bad && !wait;
  w.had = (w.cached + kPage - 1) / kPage;
  w.has = (w.cached + w.n + kPage - 1) / kPage;
  const int sinks = p.window > 0 ? (int)(((int64_t)p.sink_tokens + kPage - 1) / kPage) : 0;
  const int keep = max(sinks, p.shared_pages);
  w.a_lo = w.a_hi = w.b_lo = w.b_hi = 0;
  w.seq = w.cached + w.n;
  w.first = first;
  const int from = max(first, keep);
  if (ended) {
    w.a_lo = min(p.shared_pages, w.had);
    w.a_hi = max(w.a_lo, min(keep, w.had));
    w.b_lo = min(from, w.had);
    w.b_hi = w.had;
    w.seq = 0;
    w.first = 0;
  } else if (p.window > 0 && w.n > 0) {
    const int upto = min(max(w.cached - p.window + 1, 0) / kPage, w.had);  // (window >= 1: no overflow)
    if (upto > from) {
      w.b_lo = from;
      w.b_hi = upto;
      w.first = upto;
    }
  }
  return w;
}

struct Sums {
  int64_t tok, grant, back;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.tok + b.tok, a.grant + b.grant, a.back + b.back};
}

struct Smem {
  Sums warp[kWarps];
  // start of each thread's first request in the three lists, and their ends
  int tok[kThreads + 1], grant[kThreads + 1], back[kThreads + 1];
  int last;
};

// The thread whose requests hold entry i of a list: the last with start <= i among
// `n` threads (of equal starts, the one that holds anything).
__device__ __forceinline__ int find(const int* start, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads, 1) step_tables_kernel(const TablesParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ Smem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = p.num_reqs, per = (R + kThreads - 1) / kThreads;  // consecutive requests per thread
  const int r0 = min(tid * per, R), r1 = min(r0 + per, R);
  const int head = p.free_state[0], count = p.free_state[1], cap = p.num_blocks;
  // ---- sums over the requests
  Sums own{0, 0, 0};
  bool any_bad = false;
  for (int r = r0; r < r1; ++r) {
    bool bad;
    const Row w = row_of(p, r, false, &bad);
    any_bad = any_bad || bad;
    own = own + Sums{w.n, w.granted(), w.back()};
  }
  Sums incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums y{__shfl_up_sync(0xffffffffu, incl.tok, o), __shfl_up_sync(0xffffffffu, incl.grant, o),
                 __shfl_up_sync(0xffffffffu, incl.back, o)};
    if (lane >= o) incl = incl + y;
  }
  if (lane == 31) sm.warp[warp] = incl;
  __syncthreads();
  Sums before{0, 0, 0}, all{0, 0, 0};
#pragma unroll 8
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = all;
    all = all + sm.warp[w];
  }
  before = before + incl;  // (inclusive)
  const bool state_bad = head < 0 || head >= cap || count < 0 || count > cap;
  const int64_t left = max((int64_t)count - all.grant, (int64_t)0);
  // nothing is done where it could not be done in bounds
  const bool wait = state_bad || all.tok > p.n_tokens || left + all.back > cap;
  const int total = wait ? 0 : (int)all.tok, grants = wait ? 0 : (int)all.grant, backs = wait ? 0 : (int)all.back;
  const int given = state_bad ? 0 : min(grants, count);  // ids the ring can give
  if (blockIdx.x == 0 && any_bad) record_error(p.err, PA_ERR_DEVICE_INDEX);
  if (blockIdx.x == 0 && tid == 0) {
    if (wait) record_error(p.err, PA_ERR_DEVICE_INDEX);
    else if (given < grants) record_error(p.err, PA_ERR_DEVICE_NO_BLOCKS);
  }
  sm.tok[tid] = wait ? 0 : (int)(before.tok - own.tok);
  sm.grant[tid] = wait ? 0 : (int)(before.grant - own.grant);
  sm.back[tid] = wait ? 0 : (int)(before.back - own.back);
  __syncthreads();
  const int used = (R + max(per, 1) - 1) / max(per, 1);  // threads that hold requests
  const int step = (int)gridDim.x * kThreads, i0 = (int)blockIdx.x * kThreads + tid;
  // id of grant g, -1 if there is none
  auto granted_id = [&](int g) -> int {
    if (g >= given) return -1;
    uint32_t at = (uint32_t)head + (uint32_t)g;  // < 2 cap < 2^32
    at -= at >= (uint32_t)cap ? (uint32_t)cap : 0u;
    const int id = p.free_ring[at];
    if (id < 0 || id >= cap) {
      record_error(p.err, PA_ERR_DEVICE_INDEX);
      return -1;
    }
    return id;
  };
  // ---- tokens
  for (int i = i0; i < p.n_tokens; i += step) {
    int64_t slot = -1;
    int pos = 0;
    if (i < total) {
      const int t = find(sm.tok, used, i);
      int r = t * per, s = sm.tok[t], g = sm.grant[t];
      Row w = row_of(p, r, false, nullptr);
      while (i >= s + w.n) {  // (ends: the thread's requests hold entry i)
        s += w.n;
        g += w.granted();
        w = row_of(p, ++r, false, nullptr);
      }
      pos = w.cached + (i - s);
      const int page = pos / kPage;
      const int id = page >= w.had ? granted_id(g + page - w.had) : p.block_tables[(size_t)r * p.max_blocks_per_req + page];
      if (id >= 0) slot = (int64_t)id * kPage + pos % kPage;
    }
    p.slot_mapping[i] = slot;
    p.positions[i] = pos;
  }
  // ---- pages granted
  for (int i = i0; i < grants; i += step) {
    const int t = find(sm.grant, used, i);
    int r = t * per, s = sm.grant[t];
    Row w = row_of(p, r, false, nullptr);
    while (i >= s + w.granted()) {
      s += w.granted();
      w = row_of(p, ++r, false, nullptr);
    }
    p.block_tables[(size_t)r * p.max_blocks_per_req + w.had + (i - s)] = granted_id(i);
  }
  // ---- pages given back (their entries are no granted ones)
  for (int i = i0; i < backs; i += step) {
    const int t = find(sm.back, used, i);
    int r = t * per, s = sm.back[t];
    Row w = row_of(p, r, false, nullptr);
    while (i >= s + w.back()) {
      s += w.back();
      w = row_of(p, ++r, false, nullptr);
    }
    const int a = w.a_hi - w.a_lo;
    const int page = i - s < a ? w.a_lo + (i - s) : w.b_lo + (i - s - a);
    p.free_ring[((int64_t)head + count + i) % cap] = p.block_tables[(size_t)r * p.max_blocks_per_req + page];
  }
  // ---- offsets
  if (blockIdx.x == 0) {
    int s = sm.tok[tid];
    for (int r = r0; r < r1; ++r) {
      p.qo_indptr[r] = s;
      s += wait ? 0 : row_of(p, r, false, nullptr).n;
    }
    if (tid == 0) p.qo_indptr[R] = total;
  }
  // ---- what the other CTAs read: written by the last one to get here
  __syncthreads();
  if (tid == 0) {
    sm.last = 1;
    if (gridDim.x > 1) {
      sm.last = atom_add_acq_rel_gpu(p.arrived, 1) == (int)gridDim.x - 1;
      if (sm.last) *p.arrived = 0;
    }
  }
  __syncthreads();
  if (!sm.last) return;
  for (int r = r0; r < r1; ++r) {
    const Row w = row_of(p, r, wait, nullptr);
    p.seq_lens[r] = w.seq;
    if (p.first_page_out) p.first_page_out[r] = w.first;
  }
  if (tid == 0) {
    p.free_state_out[0] = wait ? head : (int)(((int64_t)head + given) % cap);
    p.free_state_out[1] = wait ? count : count - given + backs;
  }
}

}  // namespace

cudaError_t launch_step_tables(const TablesParams& p, cudaStream_t stream) {
  const int64_t work = p.n_tokens > p.num_reqs ? p.n_tokens : p.num_reqs;
  int64_t grid = (work + kThreads - 1) / kThreads;
  grid = grid < 1 ? 1 : grid > 128 ? 128 : grid;
  return launch_pdl(step_tables_kernel, dim3((unsigned)grid), dim3(kThreads), 0, stream, p);
}

}  // namespace pa
