// Host-side interface between the C ABI (pa_api.cu) and the kernel files.
#pragma once

#include <cuda.h>  // CUtensorMap
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "pa.h"

namespace pa {

struct AppendParams {
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int64_t* slot_mapping;
  int64_t n_tokens;
  uint16_t* k_cache;
  uint16_t* v_cache;
  int64_t num_blocks;
  int32_t num_kv_heads;
  int* err;
};

// Read-back of q4 rows by slot (zero rows for slots outside the pool).
struct ReadParams {
  const int64_t* slot_mapping;
  int64_t n_tokens;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  int64_t num_blocks;
  int32_t num_kv_heads;
  uint16_t* k_out;
  uint16_t* v_out;
  int* err;
};

struct CopyParams {
  uint16_t* k_cache;
  uint16_t* v_cache;
  int64_t num_blocks;
  const int32_t* src;
  const int32_t* dst;
  int64_t n_pairs;
  int64_t block_vecs;  // 16-byte words in one block of one cache
  int* err;
};

// Persistent decode launch plan (host-made, passed by value).  For each kv
// head the decode rows' pages are laid end to end as one stream (row d of
// the launch, then row d + 1, ...); every stream is cut into n_seg equal
// segments of seg pages.  CTA b takes kv head b % Hkv and segment b / Hkv,
// so the Hkv CTAs of a segment read the same blocks at the same time.
constexpr int kPlanMaxRows = 1024;   // decode rows per launch
constexpr int kPlanMaxCtas = 1024;   // CTAs per launch
constexpr int kDecodeMaxItemsPerCta = 64;
// Warps of the CTA-granular decode kernel (three CTAs per SM).  Workspaces
// hold kDecodeWarps pieces per CTA of the largest CTA-granular grid, which
// also covers the warp-granular launches (a third of the CTAs, kWgWarps
// pieces each).
constexpr int kDecodeWarps = 4;
// Host-planned launches whose warp segments would hold fewer pages than this
// run the CTA-granular kernel: a row cut into many short warp pieces costs
// its last piece a long merge, and few pages per warp leave its 2-page ring
// latency-bound (measured: one 2048-token row per layer 12.6 us CTA-granular
// against 18.6 us warp-granular; 32 rows 58.2 against 54.9 us).
constexpr int kMinWarpSegPages = 8;
// The warp-granular decode kernel runs one CTA of kWgWarps warps per SM,
// one warp segment per warp: the warps of an SM then share one CTA, which
// measured faster than three CTAs of four warps (the later CTAs on an SM
// streamed up to 9 % slower).  A segment may hold kWgMaxPagesPerCta pages and
// kWgMaxItemsPerCta rows.
constexpr int kWgWarps = 12;
constexpr int kWgMaxPagesPerCta = 3072;
constexpr int kWgMaxItemsPerCta = 192;
// The decode kernel over q4 pages: pages and rows a CTA's segment may hold.
constexpr int kQ4MaxPagesPerCta = 1992;
constexpr int kQ4MaxItemsPerCta = 192;
static_assert(kQ4MaxItemsPerCta % 32 == 0, "whole rounds of the item table");
// Rows of up to kQ4DecodeQueries queries run it: tiles = 0 for one query, else
// tiles of 8 columns (two queries of 4 heads): 2 for up to 4 queries, 3 for 5
// and 6.  (A fourth tile's partial results would no longer fit beside the
// rings.)
constexpr int kQ4DecodeQueries = 6;
constexpr int q4_decode_tiles(int n_q) { return n_q == 1 ? 0 : n_q <= 4 ? 2 : 3; }
// Warps per CTA: as many as registers (tiles) and shared memory leave room for.
constexpr int q4_decode_warps(int tiles) { return tiles == 0 ? 12 : 8; }
// (piece, head) slots of the workspace that a piece of a row cut between CTAs
// takes: its columns, and a 64-bit word in two of the lse slots.
constexpr int q4_piece_slots(int tiles) { return (tiles == 0 ? PA_GQA_GROUP : 8 * tiles) + 2; }
static_assert(kQ4MaxPagesPerCta % 12 == 0 && kQ4MaxPagesPerCta % 8 == 0, "whole warp segments");
// Bytes of one (page, kv head) slab of K or V in bf16 (16 tokens x 128 dims).
constexpr int kSlabBytesHost = 16 * 128 * 2;
struct DecodePlan {
  int32_t n_rows;                     // decode rows of this launch
  int32_t seg;                        // pages per segment
  int32_t total;                      // pages of one kv head's stream
  int32_t rows[kPlanMaxRows];         // request index of decode row d
  int32_t seq[kPlanMaxRows];          // its seq_len (from the host copy)
  int32_t tok[kPlanMaxRows];          // its query token (qo_indptr, from the host copy)
  int32_t first_row[kPlanMaxCtas];    // row (index d) holding a segment's first page
  int32_t first_page[kPlanMaxCtas];   // that page's index within its row
};

// The same plan as the q4 decode kernel takes it, for at most R rows and C
// segments.
template <int R, int C>
struct Q4Plan {
  int32_t n_rows, seg, total;
  int32_t by_row;  // a segment holds pages of its first row only
  uint64_t tag;    // marks this launch's words in the workspace (next_tag)
  int4 row[R];    // request, seq_len, first query token, queries
  int2 start[C];  // a segment's first row and that row's first page
};

// Decode step (self-planned launch): the kernel parameters carry only the
// padded batch size and the longest valid seq_len; each CTA plans its own
// segment from the device seq_lens, so one captured launch serves any
// lengths within these bounds.  A row costs its pages plus kStepItemCost
// stream units (the item-end merge work, in pages of streaming), and the
// stream is cut into segments of at least kStepMinSegCost units.
struct StepPlan {
  int32_t n_rows;       // rows of the padded batch (<= kPlanMaxRows)
  int32_t max_seq_len;  // rows with a longer seq_len are errors
};
constexpr int kStepItemCost = 8;
constexpr int kStepMinSegCost = 8;
template <bool kStep>
struct PlanOf {
  using type = DecodePlan;
};
template <>
struct PlanOf<true> {
  using type = StepPlan;
};

struct DecodeParams {
  const uint16_t* q;
  const uint16_t* k_cache;
  const uint16_t* v_cache;
  int64_t num_blocks;
  const int32_t* block_tables;
  int32_t max_blocks_per_req;
  const int32_t* seq_lens;
  const int32_t* qo_indptr;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  float scale_log2;      // sm_scale * log2(e)
  int32_t page_offset;   // leading pages of every row left out (a shared prefix attended elsewhere)
  const float* prefix_o;    // fp32 [prefix_n][total_q, Hq, D] normalised partials over those pages, or null
  const float* prefix_lse;  // fp32 [prefix_n][total_q, Hq] their log2-domain lse
  int32_t prefix_n;         // partials to fold in (key chunks of the prefix; 1 once merged)
  int64_t prefix_rows;      // total_q * Hq: the stride between two partials' rows
  // Prefix pass running at the same time as this launch (else null: its
  // partials are complete before the launch).  prefix_done[t * Hkv + kvh]
  // counts the key chunks of query tile t (kPrefillQTile tokens) written so
  // far; a row's fold waits for prefix_n of them.  prefix_readers counts the
  // folds done per (tile, kv head); the last of a tile's prefix_tile_rows(t)
  // readers returns both counters to zero.
  int* prefix_done;
  int* prefix_readers;
  // 1: the tile kernel launched just before runs beside this launch (a
  // prefix pass, or chunked-prefill jobs on SMs of their own).  Its CTAs
  // waited for the kernels before it and then released this launch, which
  // therefore skips its own wait at the start, and waits for that kernel at
  // its end, so that this launch completes after it (stream order).
  int32_t beside;
  int32_t total_q;
  uint16_t* out;         // bf16 [total_q, Hq, D]
  float* lse;            // [total_q, Hq] natural log, or null
  float* piece_o;        // fp32 [2 x warp segments (warp-granular) or CTAs (CTA-granular), 4, D]: the
                         // partial of a segment's first / last item
  float* piece_lse;      // fp32 [2 x the same, 4], log2 domain
  int64_t piece_slots;   // (piece, head) slots the two arrays hold; a write past them is recorded, not made
  int* counters;         // [num_reqs, Hkv] CTAs finished per item; zero between calls
  int* err;
  // decode step only: the new token of every row ([rows, Hkv, D] bf16) and
  // the pools it is appended to (the same memory as k_cache / v_cache)
  const uint16_t* k_new;
  const uint16_t* v_new;
  uint16_t* k_store;
  uint16_t* v_store;
};

// Tiled TMA maps of the tensor-core tile kernels (host-encoded, passed by
// value): q as [total_q][Hq][D] with 64 x 4 x 32 boxes, the K and V pools as
// [num_blocks * Hkv * 16][D] rows with 64 x 16 boxes, all 128-byte swizzled.
struct TcMaps {
  CUtensorMap q;
  CUtensorMap k;
  CUtensorMap v;
};

// Those of the tile kernel over q4 pages: q as above, and out as q with boxes of
// kQ4OutTok tokens, the rows that a softmax warp stores at once.
constexpr int kQ4OutTok = 32 / PA_GQA_GROUP;
struct Q4Maps {
  CUtensorMap q;
  CUtensorMap out;
};

// Prefill work items: (request, first query of the tile) pairs, passed by
// value in the kernel's parameter block.
constexpr int kMaxPrefillItems = 1536;
struct PrefillItems {
  int32_t count;
  int32_t req[kMaxPrefillItems];
  int32_t q_start[kMaxPrefillItems];
};

// Key ranges of the tile jobs over q4 pages, when few jobs would leave SMs idle:
// each item is listed once per range of `tiles` key tiles (0: whole), and each
// (listed item, kv head) leaves `rows` rows of partial outputs in piece_o (512
// bytes each) and piece_lse.
struct Q4Split {
  int32_t tiles, rows;
  float* piece_o;
  float* piece_lse;
};
// The tile kernel's items over q4 pages, up to N of them: request, first query
// token, its position, queries + 256 x key range.
template <int N>
struct Q4Items {
  int32_t count;
  int32_t pad;
  Q4Split split;
  int4 item[N];
};
constexpr int kQ4FewItems = 160;  // a batch of split items has no more
constexpr int kQ4MaxRanges = 32;

// Attention with a window: a query at position p sees keys t <= p with t <
// sink_tokens or t > p - window.
constexpr int kWindowGangs = 2;       // groups of warps of a decode CTA, at most; each has a segment
constexpr int kWindowMergeWarps = 3;  // at most; each counts a row's pieces for itself
struct WindowParams {
  const uint16_t* q;
  const uint16_t* k_cache;
  const uint16_t* v_cache;
  int64_t num_blocks;
  const int32_t* block_tables;
  int32_t max_blocks_per_req;
  const int32_t* seq_lens;
  const int32_t* qo_indptr;  // or null: row r has the one query r
  int32_t num_reqs;
  int32_t total_q;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  float scale_log2;
  int32_t window;
  int32_t sink_tokens;
  uint16_t* out;
  float* lse;
  // rows of a decode launch (at most kPlanMaxRows), and the segments that each is cut
  // into (0: all rows' pages as one stream)
  int32_t row0, rows, per_row;
  float* piece_o;      // fp32 [2 x segments, piece_cols, D] of rows cut between segments
  float* piece_lse;    // fp32 [2 x segments, piece_cols], log2 domain
  int32_t piece_cols;  // (query, head) columns of a piece
  // pieces that have arrived, of the row that is cut at segment s's end: [s, Hkv,
  // kWindowMergeWarps], tag << 16 | count
  unsigned long long* words;
  uint64_t tag;  // marks this launch's words (next_tag)
  // the tile kernel's parts of jobs cut between CTAs: [2 x CTAs][2 query tiles][128 rows]
  float* part_o;    // ... x D fp32, 4 dims of neighbouring rows side by side
  float* part_lse;  // log2 domain
  int* err;
};
// Rows of up to this many queries run the decode kernel with a window, others the tiles.
// Decode and tiles, us, 8 kv heads, rows x keys: 3 queries 80 x 256 27.5 and 30.5, 40 x 4096
// 107 and 114; 5 queries 31.0 and 31.5, 112 and 115; 8 queries 37.2 and 29.2, 130 and 115.
constexpr int kWindowDecodeQueries = 6;
// The items of a tile launch: request, first query token, its position, queries (up to
// kWindowTileTokens).
constexpr int kWindowTileTokens = 64;
constexpr int kWindowMaxSms = 256;  // (workspace sizing; more SMs are not used)
// ... and how the jobs (job u: item u / Hkv, kv head u % Hkv) are shared: whole, in
// rounds of one per CTA, or CTA b from key tile start[b].y of job start[b].x to where CTA
// b + 1 begins (no share is empty).
struct WindowItems {
  int32_t count, pad[3];
  int4 item[kMaxPrefillItems];
  int2 start[kWindowMaxSms + 1];
};
// A job that CTAs b0 .. b0 + parts - 1 have parts of, and where the first of these lies.
struct WindowCut {
  int32_t tok0, nq, kvh, b0, parts, slot0;
};
struct WindowCuts {
  WindowCut cut[kWindowMaxSms];
};

struct PrefillParams {
  const uint16_t* q;
  const uint16_t* k_cache;
  const uint16_t* v_cache;
  int64_t num_blocks;
  const int32_t* block_tables;
  int32_t max_blocks_per_req;
  const int32_t* seq_lens;
  const int32_t* qo_indptr;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  float scale_log2;
  int32_t kv_key_offset;    // keys [0, kv_key_offset) left out (a shared prefix, whole pages)
  const float* prefix_o;    // as in DecodeParams, or null
  const float* prefix_lse;
  uint16_t* out;
  float* lse;
  int* err;
};

// Shared-prefix pass: all total_q query tokens against the prefix keys
// [0, prefix_keys) of block-table row table_row, cut into key chunks of
// chunk_keys (a multiple of 64).  Chunk partials go to chunk_o / chunk_lse
// ([n_chunks][total_q][Hq] rows), merged into prefix_o / prefix_lse by the
// merge kernel.  With one chunk the CTAs write prefix_o / prefix_lse directly.
struct PrefixParams {
  const uint16_t* q;
  const uint16_t* k_cache;
  const uint16_t* v_cache;
  int64_t num_blocks;
  const int32_t* block_tables;
  int32_t max_blocks_per_req;
  int32_t table_row;
  int32_t total_q;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t prefix_keys;
  int32_t chunk_keys;
  float scale_log2;
  float* chunk_o;
  float* chunk_lse;
  float* prefix_o;
  float* prefix_lse;
  int* done;  // per (query tile, kv head): chunks written (release), or null
  int* err;
};

// A step's tables from the requests' lengths (pa_step_tables).
struct TablesParams {
  const int32_t* new_tokens;
  const int32_t* cached_lens;
  const int32_t* first_page;  // or null: zeros
  int32_t num_reqs;
  int32_t* block_tables;
  int32_t max_blocks_per_req;
  int32_t* free_ring;
  int32_t num_blocks;
  const int32_t* free_state;  // head, count
  int32_t window, sink_tokens, shared_pages;
  int32_t n_tokens;
  int32_t* seq_lens;
  int32_t* qo_indptr;
  int64_t* slot_mapping;
  int32_t* positions;
  int32_t* free_state_out;
  int32_t* first_page_out;  // or null
  int* err;
  int32_t in_place;  // an output is the array it is made from
  int* arrived;      // CTAs of the launch that are done; zero between calls
};

// Norms and rotations of queries and keys; with pools the keys and the values go
// to their slots, else the keys to k_out.
struct RopeParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;  // append only
  int64_t q_stride, k_stride, v_stride;  // elements from a token to the next
  const int32_t* positions;
  const int64_t* slot_mapping;  // append only
  int64_t n_tokens;
  const float* q_weight;  // or null: no norm
  const float* k_weight;
  float eps;
  const uint64_t* turns;
  int32_t rotary_dim;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  uint16_t* q_out;
  uint16_t* k_out;    // no append
  uint16_t* k_cache;  // append
  uint16_t* v_cache;
  int64_t num_blocks;
  int* err;
};

struct MergeParams {
  const uint16_t* o_a;
  const float* lse_a;
  const uint16_t* o_b;
  const float* lse_b;
  uint16_t* o_out;
  float* lse_out;
  int64_t rows;
  int32_t num_heads;
  int32_t head_dim;
};

// Raises the dynamic shared-memory limit of kernel `fn` to `bytes` once per
// device: done[dev] records that it was set.  Host threads may race on the
// first call of a device; each then sets the same value, which is harmless,
// and the flag is an atomic.
constexpr int kMaxDevices = 64;
inline cudaError_t set_smem_limit_once(const void* fn, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  return e;
}

// Sets the calling thread's pa_last_error_message() text and returns s.
pa_status set_error(pa_status s, const char* fmt, ...);

// Each launcher enqueues one kernel on `stream` and returns its launch error.
cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_kv_append_q8(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_kv_append_q4(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_kv_read_q4(const ReadParams& p, cudaStream_t stream);
cudaError_t launch_copy_blocks(const CopyParams& p, cudaStream_t stream);
// overlap: programmatic launch after the stream's previous kernel; diag:
// the timeout-path diagnostic instantiation (bf16 pages, warp-granular);
// cta_granular: the kernel whose 4 warps read every page of the CTA's
// segment (no prefix pass beside it), for plans with short segments; else
// the warp-granular kernel (plan in whole warp segments of kWgWarps warps)
cudaError_t launch_decode(const DecodeParams& p, const DecodePlan& plan, int grid, bool q8, bool overlap,
                          bool diag, bool cta_granular, cudaStream_t stream);
// q4 pages: rows of n_q[i] queries (i: plan row), all of the class `tiles`; a
// plan in whole warp segments of q4_decode_warps(tiles) warps
cudaError_t launch_decode_q4(const DecodeParams& p, const DecodePlan& plan, const int32_t* n_q, int tiles, int grid,
                             bool by_row, bool overlap, cudaStream_t stream);
// warp_granular: the warp-granular kernel (grid: one CTA per SM at most; no
// segment may hold more than kWgMaxItemsPerCta rows or kWgMaxPagesPerCta
// pages), else the CTA-granular one (windows of rows)
cudaError_t launch_decode_step(const DecodeParams& p, const StepPlan& plan, int grid, bool warp_granular,
                               cudaStream_t stream);
// q4 pages: (item of up to kQ4TileTokens queries, kv head) jobs on ctas CTAs;
// rows[i] is item i's (request, first query token, its position, queries + 256 x
// key range).  With key ranges: one CTA per job, at most kQ4FewItems items
cudaError_t launch_prefill_q4(const PrefillParams& p, int count, const int4* rows, const Q4Split& split,
                              const Q4Maps& maps, int ctas, cudaStream_t stream);
// ... and the outputs of split items from their ranges' parts
cudaError_t launch_merge_q4(const PrefillParams& p, int count, const int4* rows, const Q4Split& split,
                            cudaStream_t stream);
// ctas: CTAs of the launch (0: one per (item, kv head) job; fewer run
// several jobs each)
cudaError_t launch_prefill(const PrefillParams& p, const PrefillItems& items, const TcMaps& maps, int ctas,
                           cudaStream_t stream);
cudaError_t launch_prefix(const PrefixParams& p, int n_chunks, const TcMaps& maps, cudaStream_t stream);
cudaError_t launch_prefix_merge(const PrefixParams& p, int n_chunks, cudaStream_t stream);
cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream);
// A mark for the words that a launch counts in (48 bits), another one for every launch.
uint64_t next_tag();

cudaError_t launch_step_tables(const TablesParams& p, cudaStream_t stream);
cudaError_t launch_norm_rope(const RopeParams& p, bool append, bool interleaved, cudaStream_t stream);
// rows of up to `queries` queries on grid CTAs, a multiple of the kv heads
cudaError_t launch_decode_window(const WindowParams& p, int queries, int grid, cudaStream_t stream);

// the (item, kv head) jobs of rows of more queries, shared by ctas CTAs
cudaError_t launch_prefill_window(const WindowParams& p, const WindowItems& items, bool cut, const TcMaps& maps,
                                  const CUtensorMap& out_map, int ctas, cudaStream_t stream);

// ... and the outputs of n cut jobs from their parts
cudaError_t launch_merge_window(const WindowParams& p, const WindowCuts& cuts, int n, cudaStream_t stream);

// Query tile of the tensor-core tile kernels (query tokens per CTA: with the
// 4 heads of a GQA group, 128 rows = the MMA's M) and their key tile.
constexpr int kPrefillQTile = 32;
constexpr int kTcKeyTile = 128;
// Most query tokens of a job of the tile kernel over q4 pages (two MMA tiles).
constexpr int kQ4TileTokens = 2 * kPrefillQTile;
// Decode kernel: pages a CTA may hold block ids for (bounds the segment).
constexpr int kDecodeMaxPagesPerCta = 1024;

}  // namespace pa
