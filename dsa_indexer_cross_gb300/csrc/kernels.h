// Internal launch interface between the C-ABI layer (api.cu) and the kernels.
#pragma once

#include <atomic>
#include <climits>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace dsa {

// Sets Kern's maximum dynamic shared memory once per device (the attribute persists for the
// device's context, so later launches skip the driver call).
template <auto Kern>
inline cudaError_t smem_attr_once(int bytes) {
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

template <auto K>
struct Kernel {              // a kernel as an argument, where it has to be a constant
  static constexpr auto value = K;
};
// Clusters of `cluster` <= 8 CTAs of Kern that are resident at once, as the device says: fewer than the SMs' room, as a
// cluster's CTAs lie in one group of SMs (two 512-thread CTAs an SM, 304 in all: 97 clusters of three, 46 of six, 36 of
// eight).  Asked once per device and size; no bound where it cannot be told.
template <auto Kern>
inline int resident_clusters(int cluster, int threads, int smem) {
  static std::atomic<int> known[64][9];        // 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return INT_MAX;
  int n = known[dev][cluster].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(cluster);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, Kern, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = INT_MAX;
    }
    n = n > 0 ? n : 1;
    known[dev][cluster].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Layout of the 256-byte header at the start of every workspace.
struct WsHeader {
  uint32_t status;       // DEV_ERR_* bits
  uint32_t bad_count;    // number of out-of-range indices met
  uint32_t pad[62];
};
static_assert(sizeof(WsHeader) == 256, "header is 256 bytes");

// Paged latent / index-key caches: pages of kPageRows rows; row t's logical key j lives at
// cache row block_table[t * max_pages + j / kPageRows] * kPageRows + j % kPageRows and is
// valid for j < seq_len[t].  block_table == nullptr means a contiguous cache (rows ks[t] + j).
constexpr int kPageShift = 7;
constexpr int kPageRows = 1 << kPageShift;
struct PagedRows {
  const int32_t* block_table = nullptr;
  const int32_t* seq_len = nullptr;
  int max_pages = 0;
  int n_pages = 0;
};

// ---------------------------------------------------------------------------- RoPE pre-pass
// out[row] = in[row] with its last `rope` dims rotated at position pos[row / rows_per_pos];
// only dims from the first 64-dim block holding rotary dims on are written
// (rope_split_blocks gives how many leading blocks are left to the unrotated input).
cudaError_t launch_rope_rows(const void* in, void* out, const int32_t* pos, int64_t n_rows, int rows_per_pos, int d,
                             int rope, const float* cs, int n_pos, uint32_t* status, cudaStream_t st);

// ---------------------------------------------------------------------------- indexer
// Candidate buffers: per (row, key chunk) kSub sub-buffers of cap / kSub entries, one per
// lane quarter of the indexer's 128-key tiles (keys j with (j - chunk start) % 128 in
// [32 q, 32 q + 32) go to sub-buffer q, in key order).
constexpr int kSub = 4;
// Rows with at most kDirectMax keys in a chunk keep every key (no streaming threshold).
constexpr int kDirectMax = 4096;
struct IndexerPlan {
  int n_heads, head_dim, group;      // group = query rows sharing one key stream (G)
  int n_groups, n_chunks, chunk;     // key chunking of every group's range
  int cap;                           // candidate capacity per (row, chunk), multiple of 128
  int grid;                          // persistent CTAs
  int topk;
  bool unit_list;                    // the kernel reads the dense unit list (independent rows)
};

// Fills row_range[t] = (ks, ke) when valid (ks == nullptr: every range starts at 0), else
// (0, 0) and flags; group_range[g] = union of the ranges of the group's rows longer than
// trivial_len (shorter rows keep every key and are not scored), at most span_limit keys long
// (a longer union is cut there and flagged: the plan's key chunks cover span_limit keys).
// In-place transpose of the index RoPE on fp32 rows (the backward of launch_rope_rows): the
// rotated pair (a, b) of dims (d - r + i, d - r/2 + i) becomes (a c + b s, b c - a s).
cudaError_t launch_rope_rows_transpose_f32(float* x, const int32_t* pos, int64_t n_rows, int rows_per_pos, int d,
                                           int rope, const float* cs, int n_pos, uint32_t* status, cudaStream_t st);

cudaError_t launch_ranges(const int32_t* ks, const int32_t* ke, int n_q, int group, int n_kv, int max_len,
                          int trivial_len, long long span_limit, int2* row_range, int2* group_range,
                          uint32_t* status, cudaStream_t st);

// The indexer's work units, listed densely: every (group, chunk) pair whose chunk holds keys
// of the group's range, chunk-major, later groups first within a chunk, as int2 (group,
// chunk), followed by (-1, -1) up to n_groups * n_chunks entries.  The candidate counts and
// edges of every (row, chunk) pair left out are zeroed, so the final select reads them as
// empty.  One block.
cudaError_t launch_units(const int2* group_range, int n_groups, int n_chunks, int chunk_len, int group, int n_q,
                         int2* units, uint32_t* cand_cnt, uint32_t* cand_edge, cudaStream_t st);

// Bound of every pipeline wait and a test hook that stops a kernel's producer after a number
// of tiles (so the waits behind it run out); see dsa_debug_pipeline.
struct PipelineDebug {
  unsigned long long wait_ns = 2000000000ull;
  int stop_after_tiles = -1;
};
PipelineDebug pipeline_debug();

// Lightning-indexer backward (head_dim 128, n_heads a multiple of 4 up to 64): dq~ written,
// dk~ and dw accumulated (both zeroed by the caller), all fp32.  q_split / k_split: 64-dim
// blocks read from the unrotated inputs, as in launch_indexer.
cudaError_t launch_indexer_bwd(int n_q, int n_kv, int n_heads, int head_dim, int topk, const void* q_rot,
                               const void* q_in, const void* k_rot, const void* k_in, int q_split, int k_split,
                               const float* w, const int32_t* ks, const int32_t* ke, const int32_t* idx,
                               const float* d_score, float* dq, float* dk, float* dw, int grid, uint32_t* status,
                               const PipelineDebug& dbg, cudaStream_t st);

// Scores + streaming top-k candidates.  tmap_q covers rotated q as [(n_q*H_I) x d_I] bf16,
// tmap_k covers rotated k as [n_kv x d_I] bf16, both 128-byte swizzled, boxes {64, N} and
// {64, 128}.  Per (row, chunk) it leaves up to p.cap candidates in key order, their count and
// an edge key (no entry below it can be in the row's top-k; 0 when unknown) for
// launch_select.  Rows of at most trivial_len keys are not scored (count 0).
inline int rope_split_blocks(int d, int rope) { return rope > 0 ? (d - rope) / 64 : 0; }
// tmap_q / tmap_k: rotated copies; tmap_q_in / tmap_k_in: the unrotated inputs, read for the
// 64-dim blocks below q_split / k_split.
cudaError_t launch_indexer(const IndexerPlan& p, const CUtensorMap& tmap_q, const CUtensorMap& tmap_k,
                           const CUtensorMap& tmap_q_in, const CUtensorMap& tmap_k_in, int q_split, int k_split,
                           const PagedRows& pg, const float* w, int n_q, const int2* row_range,
                           const int2* group_range, int trivial_len, uint32_t* cand_key, int32_t* cand_idx,
                           uint32_t* cand_cnt, uint32_t* cand_edge, const int2* units, uint32_t* status, const PipelineDebug& dbg, cudaStream_t st);

// Exact top-k of every row from its candidates; writes offsets (ascending) and -1 padding.
// Rows of at most trivial_len keys are written as 0..L-1 without reading candidates; entries
// below the largest of a row's chunk edges are skipped.
// max_len bounds every row's length (the ranges kernel empties longer rows).
cudaError_t launch_select(int n_q, int n_chunks, int cap, int topk, int trivial_len, int max_len, const int2* row_range,
                          const uint32_t* cand_edge,
                          const uint32_t* cand_key,
                          const int32_t* cand_idx, const uint32_t* cand_cnt, int32_t* idx_out, float* score_out,
                          uint32_t* status, cudaStream_t st);

// ---------------------------------------------------------------------------- sparse attention
// Block-dense walk: an item is kDenseCols (token, head) columns, kDenseCols / H consecutive
// tokens with all H heads, and its tokens' selections over the item's key range are one
// bitmask of kDenseMaskBytes (kDenseMaskBytes * 8 / tokens bits a token).
constexpr int kDenseCols = 64;
constexpr int kDenseMaskBytes = 4096;
// Heads of the block-dense walk for this shape, or 0 for the per-token gather walk.
int sparse_attn_dense_heads(int n_heads, int n_kv, int topk);
// The block-dense pre-pass over idx, one CTA per item (hd = heads of the walk): block_range[b]
// = [min, max + 1) of the in-range latent rows the item's tokens select ((0, 0) for none),
// block_mask[b] = per token, bit o set when row min + o is selected.  Bad offsets are counted in
// status[0..1].  dense_scratch splits a scratch of sparse_attn_ws_bytes into the two arrays.
struct DenseScratch {
  int2* block_range;
  uint32_t* block_mask;
};
DenseScratch dense_scratch(void* scratch, int n_q, int hd);
cudaError_t launch_block_mask(int hd, const int32_t* idx, const int32_t* ks, int n_q, int n_kv, int topk,
                              const DenseScratch& ds, uint32_t* status, cudaStream_t st);
// Scratch bytes launch_sparse_attn needs (per-row tile counts, or per-block key ranges and
// selection bitmasks).
size_t sparse_attn_ws_bytes(int n_q, int n_heads, int n_kv, int topk);
// Rows of q (consecutive (token, head) rows) that one work item of the chosen walk reads:
// the box height of tmap_q (a paged cache always takes the gather walk).
int sparse_attn_q_box_rows(int n_heads, int n_kv, int topk, bool paged);
// tmap_kv: block-dense walk -- kv [n_kv x 576] bf16 viewed as (64 dims, n_kv rows, 9 dim
// blocks) with 128-byte swizzled boxes of {64, 64, 9} = one 64-row tile; gather walk -- kv as
// a 2-D [n_kv][576] tensor with 128-byte swizzled boxes of {64, 1} (four-row gathers).
// tmap_q: q as a 2-D [n_q * n_heads][576] tensor, 128-byte swizzled boxes of
// {64, sparse_attn_q_box_rows(...)}.
// reuse_prepass: the scratch already holds the pre-pass results (tile counts, or key ranges and
// bitmasks) for these idx and ks rows, from the previous call on the same scratch and shape.
cudaError_t launch_sparse_attn(const CUtensorMap& tmap_kv, const CUtensorMap& tmap_q, int n_q, int n_kv, int n_heads,
                               int topk, float scale, const void* kv, const int32_t* idx, const int32_t* ks,
                               const PagedRows& pg, void* out, float* lse, uint32_t* status, void* scratch,
                               cudaStream_t st, bool reuse_prepass = false);

// ---------------------------------------------------------------------------- indexer projections
// One GEMM job of the projection kernel, Y = A[T][k] . W^T in N tiles of n_tile weight rows.
//   kProjEpiBf16:        W = one matrix [n_total][k], output bf16 [T][n_total], n_tile <= 256;
//   kProjEpiLayerNormF32: W = two matrices stacked in one tile -- n_total rows (LayerNorm'd,
//                        output bf16 [T][n_total]) then n2 rows (output fp32 out2 [T][n2]) --
//                        so both share one pass over the activations; n_tile = n_total + the
//                        second matrix's box height.
enum { kProjEpiBf16 = 0, kProjEpiLayerNormF32 = 1 };
struct ProjJob {
  int n_total, k, n_tile, epi;
  void* out;
  const float* gamma;    // LayerNorm weight / bias [n_total]
  const float* beta;
  float eps;
  float* out2;           // fp32 tail outputs [T][n2]
  int n2;
};
struct ProjJobs {
  ProjJob job[2];
  int n_jobs;
  int first_unit[3];     // first unit of each job; first_unit[n_jobs] = total units
};
// ta[j]: the activations of job j ([T][k] bf16, boxes {64, 128}); tb[j]: its weights ([rows][k],
// boxes {64, rows of the tile}); tb2: the second weight matrix of the LayerNorm job.
cudaError_t launch_projections(const CUtensorMap* ta, const CUtensorMap* tb, const CUtensorMap& tb2,
                               const ProjJobs& J, int n_tokens, uint32_t* status, cudaStream_t st);

// ---------------------------------------------------------------------------- attention backward
// dq [n_q][H][576] fp32 (written), dkv [n_kv][576] fp32 (accumulated: zero it first), given the
// forward's out (bf16) and lse (fp32) and the upstream gradient dout [n_q][H][512] bf16.
cudaError_t launch_sparse_attn_bwd(int n_q, int n_kv, int n_heads, int topk, float scale, const void* q,
                                   const void* kv, const int32_t* idx, const int32_t* ks, const void* out,
                                   const float* lse, const void* dout, float* dq, float* dkv, uint32_t* status,
                                   cudaStream_t st);

// The same gradients on the block-dense walk (hd = sparse_attn_dense_heads(...) != 0), on
// tcgen05: delta [n_q * hd] fp32 scratch for D = d_out . out, scratch of sparse_attn_ws_bytes
// for the walk's pre-pass.  tmap_kv as for launch_sparse_attn's block-dense walk; tmap_q and
// tmap_do: q [n_q * hd][576] and dout [n_q * hd][512] bf16 with 128-byte swizzled boxes of
// {64, kDenseCols}.
size_t sparse_attn_bwd_dense_delta_bytes(int n_q, int n_heads);
// The same gradients on the gather walk (every other shape), on tcgen05: item = (token, 64-head
// block), each 64-slot tile of the token's selections gathered with cp.async.  delta as above;
// row_nt: n_q int32 scratch (64-slot tiles per token).
cudaError_t launch_sparse_attn_bwd_gather(const CUtensorMap& tmap_q, const CUtensorMap& tmap_do, int n_q, int n_kv,
                                          int n_heads, int topk, float scale, const void* kv, const int32_t* idx,
                                          const int32_t* ks, const void* out, const float* lse, const void* dout,
                                          float* dq, float* dkv, uint32_t* status, float* delta, int32_t* row_nt,
                                          cudaStream_t st);
// row_nt[t] = number of 64-slot tiles of idx row t up to its last index >= 0.
cudaError_t launch_row_tiles(const int32_t* idx, int n_q, int topk, int32_t* row_nt, cudaStream_t st);
cudaError_t launch_sparse_attn_bwd_dense(int hd, const CUtensorMap& tmap_kv, const CUtensorMap& tmap_q,
                                         const CUtensorMap& tmap_do, int n_q, int n_kv, int topk, float scale,
                                         const int32_t* idx, const int32_t* ks, const void* out, const float* lse,
                                         const void* dout, float* dq, float* dkv, uint32_t* status, float* delta,
                                         void* scratch, cudaStream_t st);

// Rows that share prefixes: group g's are [start[g], start[g + 1]), their common keys [0, prefix[g]); max_rows: a
// group's rows, at most or thereabouts (it chooses the kernels).
struct SharedRows {
  const int32_t* start;
  const int32_t* prefix;
  int n_groups, max_rows;
};

// ---------------------------------------------------------------------------- latent cache
// A launch whose blocks may be scheduled while the previous kernel on the stream ends (as soon as all of
// its blocks have called grid_trigger or left); every block calls grid_wait before it touches global
// memory, so launches, prologues and first waves hide behind the kernel before (32768 rows written to
// fp8, back to back on a stream: 16.1 -> 12.7 us; 8000 tokens of 64 heads turned, 26.7 -> 24.3; 300 keys
// attended, 12.3 -> 10.8).  cluster > 1: clusters of that many CTAs.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster,
                       A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  int n = 1;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// out[t, h, :rope] = the rotary dims x[t, h, :rope] turned at pos[t] (strides in elements).  One launch
// turns at most kRopeMostPairs pairs (32-bit thread numbers); a token's fit into one.
constexpr long long kRopeMostPairs = 0x7FFFFF00LL;
struct RopeApply {
  const void* x;
  void* out;
  int n_tokens, n_heads, rope;
  long long x_tok, x_head, o_tok, o_head;
  bool f32, interleaved, inverse;
};
cudaError_t launch_rope_apply(const RopeApply& a, const int32_t* pos, const float* cs, int n_pos, uint32_t* status,
                              cudaStream_t st);

// A latent cache: bf16 rows of 576 in latent, or (fp8) e4m3 codes [n_rows][512] in latent, scale
// bytes [n_rows][4] and bf16 rotary dims [n_rows][64].
struct LatentCache {
  uint8_t* latent;
  uint8_t* scale;
  uint16_t* rope;
  int n_rows;
  bool fp8;
};
// Row kv + t * kv_stride -> cache row slot[t] (negative: not stored); cs != nullptr turns the last
// 64 dims at pos[t].
cudaError_t launch_cache_write(const LatentCache& c, const void* kv, long long kv_stride, const int32_t* slot,
                               const int32_t* pos, const float* cs, int n_pos, int n_tokens, bool interleaved,
                               uint32_t* status, cudaStream_t st);
// Every row j < seq_len[t] of n_seq sequences -> out row row_start[t] + j, bf16.
cudaError_t launch_cache_read(const LatentCache& c, const PagedRows& pg, int n_seq, const int32_t* row_start, int n_out,
                              void* out, uint32_t* status, cudaStream_t st);

// Latent attention over a paged cache: every key of row t's sequence (idx == nullptr), or the
// offsets in idx [n_q][topk] (fp8 cache).  A bf16 cache is read through tmap_v, boxes {64, 64, 4},
// and tmap_kv, boxes {64, 64, 1} (up to 64 heads) or {64, 32, 9}.
// tmap_q: q as [n_q * n_heads][576], boxes {64, latent_attn_q_box_rows(n_heads)}.
// For more than 64 heads an fp8 cache's tiles go through a ring of kRing bf16 tiles per CTA pair in the
// scratch (offset and rows of that array: latent_attn_ring), which the two maps then cover instead.
constexpr int kRing = 8;
struct LatentRing {
  size_t offset;
  int rows;            // 0: none
};
LatentRing latent_attn_ring(int n_q, int n_heads, const PagedRows& pg, bool selected, int topk);
int latent_attn_q_box_rows(int n_heads);
// Whether the call over every key takes more than one CTA, and so a join.
bool latent_attn_joins(int n_q, int n_heads, const PagedRows& pg);
size_t latent_attn_ws_bytes(int n_q, int n_heads);
cudaError_t launch_latent_attn(const LatentCache& c, const CUtensorMap& tmap_kv, const CUtensorMap& tmap_v,
                               const CUtensorMap& tmap_q, const PagedRows& pg, const int32_t* idx, int n_q, int n_heads,
                               int topk, float scale, void* out, float* lse, uint32_t* status, void* scratch, cudaStream_t st,
                               const SharedRows* named = nullptr);

// w_out[t][j] = w_in[t][j] (nullptr: 0) + sum over heads of exp(scale q . kv_j - lse) of every key of row t, rows of
// both w_stride apart.  The maps are as for launch_latent_attn with at most 64 heads (tmap_q: boxes of
// key_weights_q_box_rows).
int key_weights_q_box_rows(int n_heads);
cudaError_t launch_key_weights(const LatentCache& c, const CUtensorMap& tmap_kv, const CUtensorMap& tmap_v,
                               const CUtensorMap& tmap_q, const PagedRows& pg, int n_q, int n_heads, float scale,
                               const float* lse, const float* w_in, float* w_out, long long w_stride, uint32_t* status,
                               cudaStream_t st);

// The walks (kernel launches) of such a call, those that it may have: whether a walk takes CTA pairs, the box height
// of its tmap_q, and (rows > 0) the bf16 rows in the scratch that its maps cover for an fp8 cache: the pairs' ring, or
// (walk 2, for an fp8 cache only) the staged prefixes.  Else the maps are as for launch_latent_attn.
struct SharedWalks {
  bool used[3], pair[3];
  int q_rows[3];
  size_t rows_offset[3];
  int rows[3];
};
SharedWalks latent_shared_walks(int n_q, int n_heads, int n_groups, int max_rows);
// Whether a call is better off, or no worse, without sharing: then launch_latent_attn takes it (named: the groups, for
// their checks).
bool latent_shared_alone(bool fp8, int n_q, int n_heads, const PagedRows& pg, const SharedRows& groups);
size_t latent_shared_ws_bytes(int n_q, int n_heads, int n_groups, int max_rows);
cudaError_t launch_latent_shared(const LatentCache& c, const CUtensorMap* tmap_kv, const CUtensorMap* tmap_v,
                                 const CUtensorMap* tmap_q, const PagedRows& pg, const SharedRows& groups, int n_q,
                                 int n_heads, float scale, void* out, float* lse, uint32_t* status, void* scratch,
                                 cudaStream_t st);

// ---------------------------------------------------------------------------- eviction
// Positions that stay (kept [n_seq][n_keep]), their weights and number, and their rows copied from one cache's
// pages to another's; strides in elements.
struct Evict {
  PagedRows from, to;          // (to.seq_len is not read)
  const float* weight;
  float* weight_out;           // or nullptr
  long long weight_stride, weight_out_stride;
  int32_t* kept;
  int32_t* new_len;
  int n_seq, n_keep, n_first, n_last;
};
cudaError_t launch_evict(const Evict& a, const LatentCache& src, const LatentCache& dst, uint32_t* status, cudaStream_t st);

// ---------------------------------------------------------------------------- draft verification
// Drafts taken, and the token drawn behind them, of every sequence (strides in elements between vocabulary
// rows; draft NULL: drafts without probabilities; draft_len NULL: n_draft each).
struct Verify {
  const void* target;
  const void* draft;
  const int32_t* tokens;
  const int32_t* draft_len;
  const float* u_accept;
  const float* u_sample;
  int32_t* tokens_out;
  int32_t* n_accepted;
  long long target_stride, draft_stride;
  int n_seq, n_draft, vocab;
};
cudaError_t launch_verify(const Verify& a, bool f32, uint32_t* status, cudaStream_t st);

int device_sm_count();

// ---------------------------------------------------------------------------- launch log
// While profiling is switched on (dsa_profile_enable), every kernel launch of the library is
// bracketed by a pair of CUDA events on its stream, tagged with the kernel's kind, so that a
// caller can read each launch's device time afterwards (dsa_profile_read).  Off, both calls
// do nothing.  prof_begin returns the record's slot (-1 when nothing is recorded).
enum ProfKind : int {
  kProfRope = 0, kProfRanges = 1, kProfIndexer = 2, kProfSelect = 3, kProfAttnPrep = 4, kProfAttn = 5,
  kProfAttnBwd = 6, kProfProj = 7, kProfIndexerBwd = 8, kProfCache = 9, kProfVerify = 10
};
int prof_begin(int kind, cudaStream_t st);
void prof_end(int slot, cudaStream_t st);

}  // namespace dsa
