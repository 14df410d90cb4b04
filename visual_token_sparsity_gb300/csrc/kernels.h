// Internal launch interface between the C-ABI layer (api.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sv {

// Zeroed counters behind the status word of every workspace that holds more
// than it: completion counts that each call leaves at zero.  They lie at one
// place, which nothing else uses, whatever the call and its shapes, so that
// calls may share a workspace: a count that another call's data had run over
// would never be reached.  Enough for one per (sequence, KV head) that has
// more than one split.
constexpr int kWorkspaceCounters = 4096;

// Optional per-sequence lengths of a decode batch: device int32 arrays of
// `batch` entries, nullptr = the batch-wide value for every sequence.  With
// any of them set, the batch-wide n_vis / n_text / k are capacities: strides
// of the score and index arrays, workspace sizes and split plans.
struct SeqLens {
  const int32_t* n_vis = nullptr;   // visual tokens of each sequence
  const int32_t* n_text = nullptr;  // text tokens of each sequence
  const int32_t* k = nullptr;       // selected visual tokens of each sequence
  __host__ __device__ bool any() const { return n_vis || n_text || k; }
};

// ---- retrieval scoring + top-k (retrieve.cu).  With row_done (zeroed int per
// (sequence, KV head) row) and rows that fit in shared memory, the top-k runs
// inside the scoring kernel; otherwise a separate top-k kernel follows.
// Per-sequence lengths: scores of sequence b cover its n_vis[b] tokens, its
// rows select k[b] indices and fill the rest of the k slots with -1.
cudaError_t launch_retrieve(const void* q, int R, int H, int G, const void* k_pool, int num_blocks,
                            int Hkv, int D, const int32_t* block_table, int max_blocks, int n_vis,
                            int batch, float* scores, int* status, int num_sms, int* row_done, int k,
                            int32_t* vis_idx, cudaStream_t stream, const SeqLens& lens = SeqLens{},
                            int n_text = 0);

// ---- softmax-normalised retrieval (retrieve_softmax.cu): scores of visual
// tokens = attention mass of the R x G question rows, then the row top-k
size_t retrieve_softmax_workspace_bytes(int B, int R, int H, int Hkv, int D, int n_vis, int n_text);
int retrieve_softmax_max_rows();
cudaError_t launch_retrieve_softmax(const void* q, int R, int H, float scale, const void* k_pool, int num_blocks,
                                    int Hkv, int D, const int32_t* block_table, int max_blocks, int n_vis,
                                    int n_text, int batch, const float* lse_in, int k, int32_t* vis_idx,
                                    float* scores_out, void* ws, int* status, cudaStream_t stream);

// ---- row top-k (topk.cu: one CTA per row; topk_cluster.cu: an 8-CTA cluster
// per row for long rows).  n and k are the row stride of scores and idx; with
// per-sequence lengths (rows_per_seq rows per sequence) row r uses
// lens.n_vis / lens.k of sequence r / rows_per_seq and fills its slots past
// that k with -1 (out-of-range lengths, lens.n_text beyond n_text included: the
// whole row is -1).
cudaError_t launch_topk_rows(const float* scores, int rows, int n, int k, int32_t* idx,
                             cudaStream_t stream, const SeqLens& lens = SeqLens{}, int rows_per_seq = 1,
                             int n_text = 0);
bool topk_cluster_fits(int n);
bool topk_prefers_cluster(int n);   // long rows that fit: use launch_topk_cluster
cudaError_t launch_topk_cluster(const float* scores, int rows, int n, int k, int32_t* idx,
                                cudaStream_t stream, const SeqLens& lens = SeqLens{},
                                int rows_per_seq = 1, int n_text = 0);

// ---- pack-once KV (pack.cu): selected visual + text rows of src copied to
// positions [0, k + n_text) of every sequence of dst (same Hkv and D)
cudaError_t launch_pack_kv(const void* k_src, const void* v_src, int src_blocks, const int32_t* src_bt,
                           int src_max_blocks, int n_vis, const int32_t* vis_idx, int k, int n_text,
                           void* k_dst, void* v_dst, int dst_blocks, const int32_t* dst_bt,
                           int dst_max_blocks, int batch, int Hkv, int D, int* status,
                           cudaStream_t stream);

// ---- sparse decode attention (attn.cu)
struct AttnPlan {
  int tile;
  int chunk;   // tokens per split (multiple of tile)
  int nsplit;  // splits per (sequence, KV head)
  int nsplit_max;  // upper bound of nsplit over all n' <= n_tokens
};
AttnPlan attn_plan(int B, int Hkv, int G, int n_tokens);
// kernels one attention call launches: 1 (split merge fused), or 2 (merge kernel)
int attn_kernel_count(int B, int Hkv, int G, int n_tokens);
// whether the retrieval top-k runs inside the scoring kernel (rows of n_vis keys)
bool retrieve_fuses_topk(int rows, int n_vis);

struct AttnArgs {
  const void* q;
  int H;
  float scale;
  const void* k_pool;
  const void* v_pool;
  int num_blocks, Hkv, D;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* vis_idx;
  int k_vis, n_vis, n_text, batch;   // capacities when lens has per-sequence counts
  SeqLens lens;                       // vis_idx == nullptr: lens.k is ignored (all visual tokens)
  void* out;
  float* lse;
  float* part_ml;
  float* part_o;
  int* split_done;   // zeroed int per (sequence, KV head) with splits; left zeroed after the call
  int* status;
  // fused append: one new token per (sequence, KV head), bf16 [batch][Hkv][D],
  // stored at text position n_text and attended as the last token (n_text
  // then counts the tokens before it); nullptr: plain attention
  const void* k_new = nullptr;
  const void* v_new = nullptr;
};
cudaError_t launch_sparse_attn(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_sparse_attn_mma(const AttnArgs& a, const AttnPlan& p, cudaStream_t stream);

// ---- compaction gather (prune.cu)
cudaError_t launch_gather_rows(const void* feat, int B, int N, int k, int64_t row_bytes,
                               const int32_t* idx, void* out, int* status, cudaStream_t stream,
                               const int32_t* counts = nullptr);
cudaError_t launch_threshold_select(const float* sal, int B, int N, float threshold, int32_t* idx, int32_t* count,
                                    cudaStream_t stream);

// ---- cache maintenance (evict.cu)
cudaError_t launch_kv_move_down(void* k_pool, void* v_pool, int num_blocks, int Hkv, int D,
                                const int32_t* block_table, int max_blocks, int batch,
                                int dst_pos, int src_pos, int count, int* status,
                                cudaStream_t stream);
// new tokens go to positions [pos0, pos0 + T); with per-sequence lengths
// pos0 of sequence b is lens.n_vis[b] + lens.n_text[b] (each falling back to
// n_vis / n_text), and pos0 is unused
cudaError_t launch_kv_append(void* k_pool, void* v_pool, int num_blocks, int Hkv, int D,
                             const int32_t* block_table, int max_blocks, int batch, int pos0,
                             const void* k_new, const void* v_new, int T, int* status,
                             cudaStream_t stream, const SeqLens& lens = SeqLens{}, int n_vis = 0,
                             int n_text = 0);

// ---- norm and rotation of queries and keys (norm_rope.cu).  Rows are
// token-major, [B][T] tokens of a.*_stride elements; the outputs are
// [B][heads][T][d] (encoder operands) or, with `append`, q_out [B][T][H][d]
// and the K / V pools (a.k_out, a.v_out) of the paged cache.
struct NormRopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  long long q_stride, k_stride, v_stride;
  int B, T, H, Hk;
  const uint16_t* q_weight;   // [d] or nullptr (no norm)
  const uint16_t* k_weight;
  float eps;
  const float* cos_sin;       // [n_pos][rot / 2][2]
  const int32_t* pos;         // [n_axes][B][T]
  int n_pos, rot, interleaved, n_axes;
  int sec_end[3];             // pairs [sec_end[x - 1], sec_end[x]) turn by axis x
  uint16_t* q_out;
  uint16_t* k_out;
  uint16_t* v_out;
  int* status;
  // append: where the new tokens go
  const int32_t* block_table;
  int num_blocks, max_blocks, n_vis, n_text;
  SeqLens lens;
  const int32_t* n_new;
};
cudaError_t launch_norm_rope(const NormRopeArgs& a, int d, bool append, int num_sms,
                             cudaStream_t stream);

// ---- attention of T drafted tokens over the paged cache (tree_attn.cu)
struct TreeArgs {
  const void* q;
  int T, H;
  float scale_log2;                  // > 0
  bool zero_scale;                   // the queries count as 0 times what they are
  const void* k_pool;
  const void* v_pool;
  int num_blocks, Hkv, D;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* vis_idx;
  int k_vis, n_vis, n_text, batch;   // capacities with per-sequence lengths
  SeqLens lens;
  const uint64_t* tree_mask;         // [batch][T], or nullptr: each sees itself and the earlier ones
  const int32_t* n_new;              // [batch] or nullptr
  void* out;
  float* lse;
  void* ws;                          // tree_attn_workspace_bytes
  int* status;
  // set by launch_tree_attn: query heads per KV head, tiles of query rows,
  // pieces of one row tile's work, cut units and their partial results
  int G, row_tiles, columns;
  bool by_unit;
  int* part_unit;
  float* part_ml;
  float* part_o;
};
size_t tree_attn_workspace_bytes(int B, int T, int H, int Hkv, int D, int n_tokens);
cudaError_t launch_tree_attn(const TreeArgs& a, cudaStream_t stream);

// ---- the cache in 8 bits: e4m3 pools [num_blocks][Hkv][16][D] and fp32 factors
// [num_blocks][Hkv][2], of K and of V (kv8_append.cu, kv8_retrieve.cu, kv8_attn.cu)
struct Kv8AppendArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  long long q_stride, k_stride, v_stride;
  int N, H, Hkv;                   // packed new tokens
  const int32_t* seq_start;        // [batch + 1], or nullptr: per_seq tokens each
  int per_seq;
  const uint16_t* q_weight;        // norm and rotation as in NormRopeArgs, pos [n_axes][N]
  const uint16_t* k_weight;
  float eps;
  const float* cos_sin;
  const int32_t* pos;
  int n_pos, rot, interleaved, n_axes;
  int sec_end[3];
  uint16_t* q_out;                 // [N][H][D]
  uint16_t* k_out;                 // [N][Hkv][D] or nullptr
  uint8_t* k_pool;
  uint8_t* v_pool;
  float* scales;
  const int32_t* block_table;
  int num_blocks, max_blocks, batch, n_vis, n_text;
  SeqLens lens;
  int* status;
};
cudaError_t launch_kv8_append(const Kv8AppendArgs& a, int d, int num_sms, cudaStream_t stream);

struct Kv8RetrieveArgs {
  const void* q;
  int R, H;
  const uint8_t* k_pool;
  const float* scales;
  int num_blocks, Hkv;
  const int32_t* block_table;
  int max_blocks, n_vis, n_text, k, batch;   // capacities with per-sequence lengths
  SeqLens lens;
  int32_t* vis_idx;
  float* scores;                   // [batch][Hkv][n_vis] or nullptr
  void* ws;                        // kv8_retrieve_workspace_bytes
  int* status;
};
size_t kv8_retrieve_workspace_bytes(int B, int Hkv, int D, int n_vis);
cudaError_t launch_kv8_retrieve(const Kv8RetrieveArgs& a, int D, int num_sms, cudaStream_t stream);

struct Kv8AttnArgs {
  const void* q;
  int H;
  float scale_log2;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* scales;
  int num_blocks, Hkv;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* vis_idx;
  int k_vis, n_vis, n_text, batch;
  SeqLens lens;
  void* out;
  float* lse;
  void* ws;                        // kv8_attn_workspace_bytes
  int* counters;
  int* status;
  // set by launch_kv8_attn: pieces that the work is cut into, their partial
  // results and the counters of the units that they share (nullptr: the merge
  // kernel joins them)
  int pieces, per_unit;            // (blocks of a unit, with equal counts)
  bool cut;                        // a unit may lie in several pieces
  float* part_ml;
  float* part_o;
  int* split_done;
};
size_t kv8_attn_workspace_bytes(int B, int H, int Hkv, int D, int n_tokens);
cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, int D, int num_sms, cudaStream_t stream);

// ---- causal attention of packed prompts (prompt_attn.cu)
struct PromptArgs {
  const void* q;                   // token-major rows, strides in elements
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride;
  int N, H, Hkv, batch;
  const int32_t* seq_start;        // [batch + 1]
  float scale_log2;                // > 0
  void* out;                       // [N][H][D]
  float* lse;                      // [N][H] or nullptr
  int* counters;
  int* status;
};
cudaError_t launch_prompt_attn(const PromptArgs& a, int D, int num_sms, cudaStream_t stream);

// ---- pages shared between branches (pages.cu)
constexpr int kMaxLayers = 64;   // layers of one launch
struct LayerPools {
  void* k[kMaxLayers];
  void* v[kMaxLayers];
};
struct PagesArgs {
  int32_t* ref;          // [num_pages] block-table entries that hold each page
  int32_t* n_pages;      // [batch] entries each sequence holds
  int num_pages;
  int32_t* block_table;  // [batch][max_blocks]
  int batch, max_blocks;
  int* status;
};
cudaError_t launch_pages_release(const PagesArgs& a, const int32_t* keep, cudaStream_t stream);
cudaError_t launch_pages_fork(const PagesArgs& a, const int32_t* parent, const int32_t* child, int n,
                              const int32_t* n_tok, cudaStream_t stream);
size_t pages_workspace_bytes(long long batch, long long max_blocks, long long num_pages);
// pools: n_pools groups of layers[i] layers each
cudaError_t launch_pages_reserve(const PagesArgs& a, const SeqLens& lens, int n_vis, int n_text, int T,
                                 const int32_t* n_new, const LayerPools* pools, int n_pools, const int* layers,
                                 int page_bytes, void* ws, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_accept(const LayerPools& pools, int layers, int num_blocks, int Hkv, int D,
                             const int32_t* block_table, int max_blocks, int batch, const SeqLens& lens, int n_vis,
                             int n_text, int T, const int32_t* path, int P, const int32_t* n_path, int* status,
                             cudaStream_t stream);

// ---- prefill salience (salience.cu)
cudaError_t launch_head_mean(const float* colsum, int B, int H, int N, float inv, float* out,
                             cudaStream_t stream);
// ---- summary-row salience (summary.cu)
size_t summary_smem_bytes(int N, int d, int R);
cudaError_t launch_summary_salience(const void* q, const void* k, int B, int H, int N, int d, int R,
                                    float scale, float* salience, float* colsum, cudaStream_t stream);
bool salience_head_dim_supported(int d);
// whether sv_salience_prefill streams both operands (long sequences) and how
// many kernels one call launches
bool salience_uses_long_schedule(int N, int d);
int salience_kernel_count(int N, int d);
size_t salience_workspace_bytes(int B, int H, int N, int d);
cudaError_t launch_salience(const void* q, const void* k, int B, int H, int N, int d, float scale,
                            float* salience, void* ws, int* counters, int* status, int num_sms,
                            cudaStream_t stream);

}  // namespace sv
