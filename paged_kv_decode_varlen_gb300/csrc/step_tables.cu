// A step's block tables, slots, positions and query offsets from the requests'
// lengths.
//
// What is computed: exclusive sums over the requests of their new tokens, of the
// pages these need (ceil((c + n) / 16) - ceil(c / 16)) and of the pages given back,
// and from them every token's, granted page's and returned page's place.
//
// Bound: latency.  A decode step of 64 requests moves 3 KB, a step of 8 Ki tokens 130
// KB, so what counts is one launch and few dependent round trips: lengths -> sums ->
// ring or table entry -> store.  Every CTA of the launch makes all sums for itself from
// the lengths and takes its share of the work; no CTA waits for another.
//   A thread has one request (kMany: several, one after another).  A request of at most
// one new token and one returned page is seen to by its own thread, whose table entry
// is fetched while the sums are made.  The tokens and pages of the others are three flat
// lists, each entry of which finds its request by a search in the sums: a prompt of
// thousands of tokens is spread over all threads.
//   Where an output is the array it is made from (lengths, ring state, first pages), the
// last CTA to arrive at a count writes it, as the others may still have to read it.
//   Table entries that are no blocks (pages that the ring could not grant) are not given
// back.  They come up only after the ring has run out, so places in the ring are taken as if
// there were none; where one is found, the last CTA to have given its pages back puts the
// real ids side by side by itself, and writes the ring's state (1000 requests and
// 8 Ki tokens 8.2 us with the arrivals ahead of the lists of tokens and grants, 8.4 behind
// them, 7.4 without).
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace pa {
namespace {

// One request's step.
struct Row {
  int cached, n;   // tokens before, new tokens
  int had, has;    // pages before, after
  int a_lo, a_hi;  // pages given back: [a_lo, a_hi), then [b_lo, b_hi)
  int b_lo, b_hi;
  int seq, first;  // what it holds after the step
  bool bad, ended;
  __device__ __forceinline__ int granted() const { return has - had; }
  __device__ __forceinline__ int back() const { return a_hi - a_lo + (b_hi - b_lo); }
};

// raw: the request's entry of new_tokens; wait: it is taken as one that brings nothing.
__device__ __forceinline__ Row row_of(const TablesParams& p, int raw, int c, int first, bool wait) {
  Row w;
  first = max(first, 0);
  const int c_max = min(p.max_blocks_per_req, PA_MAX_SEQ_LEN / kPage) * kPage;
  const bool c_bad = c < 0 || c > c_max;
  w.bad = c_bad || raw > c_max - c;  // (c_max - c does not overflow where c is not bad)
  w.cached = c_bad ? 0 : c;
  w.n = (w.bad || wait) ? 0 : max(raw, 0);
  w.ended = raw < 0 && !c_bad && !wait;
  w.had = (w.cached + kPage - 1) / kPage;
  w.has = (w.cached + w.n + kPage - 1) / kPage;
  const int sinks = p.window > 0 ? p.sink_tokens / kPage + (p.sink_tokens % kPage != 0) : 0;
  const int keep = max(sinks, p.shared_pages);
  w.a_lo = w.a_hi = w.b_lo = w.b_hi = 0;
  w.seq = w.cached + w.n;
  w.first = first;
  const int from = max(first, keep);
  if (w.ended) {
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

// The three sums; T holds them for the requests of a launch (2^20 tokens and 2^16 pages
// each at most: 32 bits for up to 1024 requests, 64 for more).
template <class T>
struct Sums {
  T tok, grant, back;
  __device__ __forceinline__ Sums operator+(const Sums& b) const { return {tok + b.tok, grant + b.grant, back + b.back}; }
};
template <class T>
__device__ __forceinline__ Sums<T> shfl_up(const Sums<T>& a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.tok, o), __shfl_up_sync(0xffffffffu, a.grant, o),
          __shfl_up_sync(0xffffffffu, a.back, o)};
}

constexpr int kMaxThreads = 1024;

template <class T>
struct Smem {
  Sums<T> warp[32];
  // start of each thread's first request in the three lists
  int tok[kMaxThreads], grant[kMaxThreads], back[kMaxThreads];
  int raw[kMaxThreads], cached[kMaxThreads], first[kMaxThreads];  // (one request per thread)
  int real;  // returned pages that have a block
  int last, holes;
};

// The thread whose requests hold entry i of a list: the last of n with start <= i.
__device__ __forceinline__ int find(const int* start, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <bool kMany>
__global__ void __launch_bounds__(kMaxThreads, 1) step_tables_kernel(const TablesParams p) {
  using T = typename std::conditional<kMany, int64_t, int32_t>::type;
  pdl_launch_dependents();
  pdl_wait();
  __shared__ Smem<T> sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_thr = (int)blockDim.x;
  const int R = p.num_reqs, per = kMany ? (R + n_thr - 1) / n_thr : 1;  // consecutive requests per thread
  const int r0 = min(tid * per, R), r1 = min(r0 + per, R);
  const int head = p.free_state[0], count = p.free_state[1], cap = p.num_blocks;
  auto load = [&](int r, bool wait) {
    return row_of(p, p.new_tokens[r], p.cached_lens[r], p.first_page ? p.first_page[r] : 0, wait);
  };
  auto in_pool = [&](int id) { return id >= 0 && id < cap; };
  // ---- sums over the requests
  Sums<T> own{0, 0, 0};
  bool any_bad = false, listed = false;  // a request for the lists
  Row mine{};  // the thread's request (!kMany)
  bool small = false;
  int entry = -1;  // its table entry of position `cached`
  if constexpr (kMany) {
    for (int r = r0; r < r1; ++r) {
      const Row w = load(r, false);
      any_bad = any_bad || w.bad;
      own = own + Sums<T>{w.n, w.granted(), w.back()};
    }
    listed = true;
  } else if (r0 < R) {
    const int raw = p.new_tokens[r0], c = p.cached_lens[r0], first = p.first_page ? p.first_page[r0] : 0;
    mine = row_of(p, raw, c, first, false);
    small = !mine.ended && mine.n <= 1 && mine.back() <= 1;
    if (small && mine.n == 1 && mine.granted() == 0)
      entry = p.block_tables[(size_t)r0 * p.max_blocks_per_req + mine.cached / kPage];
    sm.raw[tid] = raw;
    sm.cached[tid] = c;
    sm.first[tid] = first;
    any_bad = mine.bad;
    listed = !small;
    own = Sums<T>{mine.n, mine.granted(), mine.back()};
  }
  Sums<T> incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums<T> y = shfl_up(incl, o);
    if (lane >= o) incl = incl + y;
  }
  if (lane == 31) sm.warp[warp] = incl;
  const bool lists = __syncthreads_or(listed) != 0;
  Sums<T> w_incl = lane < n_thr / 32 ? sm.warp[lane] : Sums<T>{0, 0, 0};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums<T> y = shfl_up(w_incl, o);
    if (lane >= o) w_incl = w_incl + y;
  }
  auto of_lane = [&](int l) {
    return Sums<T>{__shfl_sync(0xffffffffu, w_incl.tok, l), __shfl_sync(0xffffffffu, w_incl.grant, l),
                   __shfl_sync(0xffffffffu, w_incl.back, l)};
  };
  const Sums<T> all = of_lane(31), prev = of_lane(max(warp - 1, 0));
  const Sums<T> before = (warp > 0 ? prev : Sums<T>{0, 0, 0}) + incl;  // inclusive
  const bool state_bad = head < 0 || head >= cap || count < 0 || count > cap;
  const int used = (R + per - 1) / per;  // threads that hold requests
  // entry i of a list (start: its sums; size: a request's share): its request r, whose
  // entries begin at s, and the request's first grant
  auto locate = [&](const int* start, auto size, int i, int& r, int& s, int& g, Row& w) -> bool {
    const int t = find(start, used, i);
    s = start[t];
    g = sm.grant[t];
    r = t * per;
    if constexpr (kMany) {
      w = load(r, false);
      while (i >= s + size(w)) {  // (ends: the thread's requests hold entry i)
        s += size(w);
        g += w.granted();
        w = load(++r, false);
      }
      return true;
    } else {
      w = row_of(p, sm.raw[t], sm.cached[t], sm.first[t], false);
      return w.ended || w.n > 1 || w.back() > 1;  // (not seen to by its own thread)
    }
  };
  // the id in the table entry of returned page i of all
  auto returned_id = [&](int i) -> int {
    int r, s, g;
    Row w;
    locate(sm.back, [](const Row& x) { return x.back(); }, i, r, s, g, w);
    const int a = w.a_hi - w.a_lo;
    return p.block_tables[(size_t)r * p.max_blocks_per_req + (i - s < a ? w.a_lo + (i - s) : w.b_lo + (i - s - a))];
  };
  // More pages come back than there are places: it depends on how many have a block.  (More
  // than 2^31 are refused.)
  const bool tight = !state_bad && (int64_t)count + (int64_t)all.back > cap;
  bool full = tight && (int64_t)all.back > INT32_MAX;
  if (__builtin_expect(tight && !full, 0)) {
    sm.back[tid] = (int)(before.back - own.back);
    if (tid == 0) sm.real = 0;
    __syncthreads();
    int real = 0;
    for (uint32_t i = (uint32_t)tid; i < (uint32_t)all.back; i += (uint32_t)n_thr) real += in_pool(returned_id((int)i)) ? 1 : 0;
    atomicAdd(&sm.real, real);
    __syncthreads();
    full = (int64_t)count + sm.real > cap;
  }
  // nothing is done where it could not be done in bounds
  const bool wait = state_bad || all.tok > p.n_tokens || full;
  const int total = wait ? 0 : (int)all.tok, grants = wait ? 0 : (int)all.grant;
  const int backs = wait || tight ? 0 : (int)all.back;  // (tight: by the last CTA)
  bool hole = false;                                    // a returned page without a block
  const int given = min(grants, max(count, 0));  // ids the ring can give
  if (blockIdx.x == 0 && any_bad) record_error(p.err, PA_ERR_DEVICE_INDEX);
  if (blockIdx.x == 0 && tid == 0) {
    if (wait) record_error(p.err, PA_ERR_DEVICE_INDEX);
    else if (given < grants) record_error(p.err, PA_ERR_DEVICE_NO_BLOCKS);
  }
  const int tok0 = wait ? 0 : (int)(before.tok - own.tok), grant0 = wait ? 0 : (int)(before.grant - own.grant),
            back0 = wait ? 0 : (int)(before.back - own.back);
  // the ring's place i behind its head (i <= cap)
  auto place = [&](int i) {
    const uint32_t at = (uint32_t)head + (uint32_t)i;  // < 2^32
    return at - (at >= (uint32_t)cap ? (uint32_t)cap : 0u);
  };
  // id of grant g, -1 if there is none
  auto granted_id = [&](int g) -> int {
    if (g >= given) return -1;
    const int id = p.free_ring[place(g)];
    if (id < 0 || id >= cap) {
      record_error(p.err, PA_ERR_DEVICE_INDEX);
      return -1;
    }
    return id;
  };
  auto give_back = [&](int i, int id) {
    if (in_pool(id)) {
      p.free_ring[place(count + i)] = id;
    } else {
      hole = true;
    }
  };

  if (!kMany && small && !wait && warp % (int)gridDim.x == (int)blockIdx.x) {
    // a request of its own thread; its ring entry is one more round trip only where the
    // token opens a page
    if (mine.back() == 1 && !tight)
      give_back(back0, p.block_tables[(size_t)r0 * p.max_blocks_per_req + (mine.a_hi > mine.a_lo ? mine.a_lo : mine.b_lo)]);
    if (mine.n == 1) {
      if (mine.granted() == 1) {
        entry = granted_id(grant0);
        p.block_tables[(size_t)r0 * p.max_blocks_per_req + mine.had] = entry;
      } else if (entry < 0) {
        record_error(p.err, PA_ERR_DEVICE_NO_BLOCKS);
      }
      p.slot_mapping[tok0] = entry >= 0 ? (int64_t)entry * kPage + mine.cached % kPage : -1;
      p.positions[tok0] = mine.cached;
    }
  }
  // Whether every CTA has given its pages back, and holes: arrivals in the count's lower
  // half, those of CTAs with holes in the upper.
  const bool some_back = !wait && all.back > 0;
  auto arrive = [&]() {
    const int own_hole = __syncthreads_or(hole) != 0;
    return tid == 0 ? atom_add_acq_rel_gpu(p.arrived, 1 + (own_hole << 16)) + (own_hole << 16) : 0;
  };
  // The ring's state alone waits for them, unless an output is the array it is made from
  // or places are tight: then all CTAs have to be done before anything is written
  const bool early = some_back && lists && gridDim.x > 1 && !p.in_place && !tight;
  int was = 0;
  const int step = (int)gridDim.x * n_thr, i0 = (int)blockIdx.x * n_thr + tid;
  if (lists && !wait) {
    sm.tok[tid] = tok0;
    sm.grant[tid] = grant0;
    sm.back[tid] = back0;
    __syncthreads();
    int r, s, g;
    Row w;
    for (int i = i0; i < backs; i += step)  // (their entries are no granted ones)
      if (locate(sm.back, [](const Row& x) { return x.back(); }, i, r, s, g, w)) {
        const int a = w.a_hi - w.a_lo;
        const int page = i - s < a ? w.a_lo + (i - s) : w.b_lo + (i - s - a);
        give_back(i, p.block_tables[(size_t)r * p.max_blocks_per_req + page]);
      }
    if (early) was = arrive();
    for (int i = i0; i < total; i += step) {
      if (!locate(sm.tok, [](const Row& x) { return x.n; }, i, r, s, g, w)) continue;
      const int pos = w.cached + (i - s), page = pos / kPage;
      const int id = page >= w.had ? granted_id(g + page - w.had) : p.block_tables[(size_t)r * p.max_blocks_per_req + page];
      if (id < 0 && page < w.had) record_error(p.err, PA_ERR_DEVICE_NO_BLOCKS);
      p.slot_mapping[i] = id >= 0 ? (int64_t)id * kPage + pos % kPage : -1;
      p.positions[i] = pos;
    }
    for (int i = i0; i < grants; i += step)
      if (locate(sm.grant, [](const Row& x) { return x.granted(); }, i, r, s, g, w))
        p.block_tables[(size_t)r * p.max_blocks_per_req + w.had + (i - s)] = granted_id(i);
  }
  for (int i = total + i0; i < p.n_tokens; i += step) {  // padding
    p.slot_mapping[i] = -1;
    p.positions[i] = 0;
  }
  // ---- offsets, and what follows the step
  if (blockIdx.x == 0) {
    int s = tok0;
    for (int r = r0; r < r1; ++r) {
      p.qo_indptr[r] = s;
      s += kMany ? load(r, wait).n : 0;
    }
    if (tid == 0) p.qo_indptr[R] = total;
  }
  auto lengths = [&]() {
    for (int r = r0; r < r1; ++r) {
      const Row w = kMany ? load(r, wait) : row_of(p, sm.raw[tid], sm.cached[tid], sm.first[tid], wait);
      p.seq_lens[r] = w.seq;
      if (p.first_page_out) p.first_page_out[r] = w.first;
    }
  };
  const bool late = gridDim.x > 1 && (p.in_place || some_back) && !early;
  bool last = blockIdx.x == 0, holes = false;
  if (late) was = arrive();
  if (late || early) {
    if (tid == 0) {
      sm.last = (was & 0xffff) == (int)gridDim.x - 1;
      sm.holes = was >> 16;
      if (sm.last) *p.arrived = 0;
    }
    __syncthreads();
    last = sm.last != 0;
    holes = sm.holes != 0;
  } else if (gridDim.x == 1 && (p.in_place || some_back)) {
    holes = __syncthreads_or(hole) != 0;  // (every thread has read its requests and the ring's state)
  }
  if (last) {
    int real = some_back ? (int)all.back : 0;
    if (__builtin_expect(some_back && (holes || tight), 0)) {
      // the ids of those that have a block, side by side
      sm.back[tid] = back0;
      __syncthreads();
      real = 0;
      for (uint32_t base = 0; base < (uint32_t)all.back; base += (uint32_t)n_thr) {
        const int id = base + (uint32_t)tid < (uint32_t)all.back ? returned_id((int)(base + (uint32_t)tid)) : -1;
        const uint32_t there = __ballot_sync(0xffffffffu, in_pool(id));
        if (lane == 0) sm.warp[warp].back = __popc(there);
        __syncthreads();
        int at = real + __popc(there & ((1u << lane) - 1u));
        for (int x = 0; x < n_thr / 32; ++x) {
          at += x < warp ? (int)sm.warp[x].back : 0;
          real += (int)sm.warp[x].back;
        }
        if (in_pool(id)) p.free_ring[place(count + at)] = id;
        __syncthreads();
      }
    }
    if (tid == 0) {
      p.free_state_out[0] = wait ? head : (int)place(given);
      p.free_state_out[1] = wait ? count : count - given + real;
    }
  }
  if (p.in_place ? last : blockIdx.x == 0) lengths();
}

}  // namespace

cudaError_t launch_step_tables(const TablesParams& p, cudaStream_t stream) {
  // a thread per request, and up to 1024 tokens a CTA
  const int64_t work = p.n_tokens > p.num_reqs ? p.n_tokens : p.num_reqs;
  const int threads = work <= 128 ? 128 : work <= 256 ? 256 : kMaxThreads;
  int64_t grid = (p.n_tokens + kMaxThreads - 1) / kMaxThreads;
  grid = grid < 1 ? 1 : grid > 128 ? 128 : grid;
  if (p.num_reqs > kMaxThreads)
    return launch_pdl(step_tables_kernel<true>, dim3((unsigned)grid), dim3(threads), 0, stream, p);
  return launch_pdl(step_tables_kernel<false>, dim3((unsigned)grid), dim3(threads), 0, stream, p);
}

}  // namespace pa
