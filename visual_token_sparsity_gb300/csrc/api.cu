// C-ABI entry points of libsv (declared in include/sv.h): argument checks,
// workspace layout and kernel launches.  No allocation, no synchronisation
// (except sv_read_device_status), no exceptions across the boundary.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../include/sv.h"
#include "api_checks.h"
#include "kernels.h"

namespace sv {

bool pdl_enabled() {
  static const bool on = [] {
    const char* e = std::getenv("SV_PDL");
    return !(e != nullptr && e[0] == '0');
  }();
  return on;
}
int topk_max_smem_keys();
}  // namespace sv

namespace {

constexpr size_t kStatusBytes = 256;
constexpr size_t kHeadBytes = kStatusBytes + sv::kWorkspaceCounters * sizeof(int);
constexpr size_t kMaxSmemPerBlock = 232448;  // 227 KB opt-in on sm_100-family parts
thread_local char g_err[512] = "";

sv_status fail(sv_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return s;
}

sv_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return SV_OK;
  return fail(SV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int num_sms() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int* status_word(void* ws) { return static_cast<int*>(ws); }

// the zeroed counters, and what follows them: the calls' data
int* counters_of(void* ws) { return reinterpret_cast<int*>(static_cast<char*>(ws) + kStatusBytes); }
char* data_of(void* ws) { return static_cast<char*>(ws) + kHeadBytes; }

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

sv_status check_ws(void* ws, size_t have, size_t need) {
  if (!ws) return fail(SV_ERR_INVALID_ARG, "workspace pointer is NULL");
  if (!aligned16(ws)) return fail(SV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  if (have < need) return fail(SV_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", have, need);
  return SV_OK;
}

// Per-sequence lengths of a batch view (all NULL: uniform lengths).
sv::SeqLens lens_of(const sv_seq_batch* S) {
  sv::SeqLens l;
  l.n_vis = S->n_vis_seq;
  l.n_text = S->n_text_seq;
  l.k = S->k_seq;
  return l;
}

sv_status reject_lens(const sv_seq_batch* S, const char* call) {
  if (S && lens_of(S).any())
    return fail(SV_ERR_UNSUPPORTED, "%s: per-sequence lengths (n_vis_seq / n_text_seq / k_seq) are not supported",
                call);
  return SV_OK;
}

}  // namespace

namespace sv {
// Records `msg` as this thread's sv_last_error() text.
void set_error_message(const char* msg) { snprintf(g_err, sizeof(g_err), "%s", msg); }

sv_status check_cache(const sv_kv_layer* L, const sv_seq_batch* S, bool need_v) {
  if (!L || !S) return fail(SV_ERR_INVALID_ARG, "layer or batch descriptor is NULL");
  if (!L->k_pool || (need_v && !L->v_pool) || !S->block_table)
    return fail(SV_ERR_INVALID_ARG, "cache pool or block table pointer is NULL");
  if (!aligned16(L->k_pool) || (need_v && !aligned16(L->v_pool)))
    return fail(SV_ERR_INVALID_ARG, "cache pools must be 16-byte aligned");
  if (L->head_dim != 64 && L->head_dim != 128)
    return fail(SV_ERR_UNSUPPORTED, "head_dim %d not supported (64 or 128)", L->head_dim);
  if (L->num_blocks <= 0 || L->n_kv_heads <= 0)
    return fail(SV_ERR_INVALID_ARG, "num_blocks and n_kv_heads must be positive");
  if ((long long)L->num_blocks * L->n_kv_heads * SV_BLOCK_TOKENS >= 0xffffffffLL)
    return fail(SV_ERR_UNSUPPORTED, "pool has too many rows for 32-bit row ids");
  if (S->batch < 0 || S->max_blocks <= 0 || S->n_vis < 0 || S->n_text < 0)
    return fail(SV_ERR_INVALID_ARG, "negative batch or length");
  if ((long long)S->n_vis + S->n_text > (long long)S->max_blocks * SV_BLOCK_TOKENS)
    return fail(SV_ERR_INVALID_ARG, "n_vis + n_text = %d exceeds max_blocks * 16 = %d",
                S->n_vis + S->n_text, S->max_blocks * SV_BLOCK_TOKENS);
  return SV_OK;
}

sv_status check_retrieve_args(const void* q, int R, int H, const sv_kv_layer* layer, const sv_seq_batch* seqs,
                              int k, const int32_t* vis_idx) {
  sv_status s = check_cache(layer, seqs, false);
  if (s != SV_OK) return s;
  if (!q || !vis_idx) return fail(SV_ERR_INVALID_ARG, "q and vis_idx must be non-NULL");
  if (!aligned16(q)) return fail(SV_ERR_INVALID_ARG, "q must be 16-byte aligned");
  const int Hkv = layer->n_kv_heads;
  if (R <= 0 || H <= 0 || H % Hkv) return fail(SV_ERR_INVALID_ARG, "need R > 0 and H a multiple of n_kv_heads");
  if (seqs->n_vis <= 0) return fail(SV_ERR_INVALID_ARG, "no visual tokens to retrieve from");
  if (k < 1 || k > seqs->n_vis) return fail(SV_ERR_INVALID_ARG, "need 1 <= k <= n_vis (k = %d)", k);
  return SV_OK;
}
}  // namespace sv

namespace {

// ---- checks of the new-token, draft and page calls

// token-major bf16 rows `stride` elements apart
sv_status check_rows(const char* name, const void* p, int64_t stride, long long row) {
  if (!aligned16(p)) return fail(SV_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (stride < row || stride % 8)
    return fail(SV_ERR_INVALID_ARG, "%s_stride = %lld: need a multiple of 8, at least %lld", name, (long long)stride,
                row);
  return SV_OK;
}

size_t row_extent(long long tokens, int64_t stride, long long row) {
  return ((size_t)(tokens - 1) * (size_t)stride + (size_t)row) * 2;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

sv_status check_rotation(const sv_rotation* r, int d, long long n_tok) {
  if (!r) return fail(SV_ERR_INVALID_ARG, "rotation descriptor is NULL");
  if (r->rot_dim < 0 || r->rot_dim > d || r->rot_dim % 8)
    return fail(SV_ERR_INVALID_ARG, "rot_dim = %d: need a multiple of 8, at most the head dim %d", r->rot_dim, d);
  if (!(r->eps >= 0.f) || !std::isfinite(r->eps)) return fail(SV_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if ((r->q_weight && !aligned16(r->q_weight)) || (r->k_weight && !aligned16(r->k_weight)))
    return fail(SV_ERR_INVALID_ARG, "norm weights must be 16-byte aligned");
  if (n_tok > 0x7fffffffLL) return fail(SV_ERR_INVALID_ARG, "more than 2^31 tokens");
  if (r->rot_dim == 0) return SV_OK;
  if (!r->cos_sin || (!r->pos && n_tok > 0)) return fail(SV_ERR_INVALID_ARG, "cos_sin and pos must be non-NULL");
  if (!aligned16(r->cos_sin)) return fail(SV_ERR_INVALID_ARG, "cos_sin must be 16-byte aligned");
  if (r->n_pos <= 0) return fail(SV_ERR_INVALID_ARG, "n_pos must be positive");
  if (r->n_axes < 1 || r->n_axes > 3) return fail(SV_ERR_UNSUPPORTED, "n_axes = %d (1 to 3)", r->n_axes);
  if (r->n_axes > 1) {
    long long sum = 0;
    for (int x = 0; x < r->n_axes; ++x) {
      if (r->section[x] < 0) return fail(SV_ERR_INVALID_ARG, "negative section");
      sum += r->section[x];
    }
    if (sum != r->rot_dim / 2)
      return fail(SV_ERR_INVALID_ARG, "sections add up to %lld, not to rot_dim / 2 = %d", sum, r->rot_dim / 2);
  }
  return SV_OK;
}

void fill_rotation(sv::NormRopeArgs& a, const sv_rotation* r) {
  a.q_weight = static_cast<const uint16_t*>(r->q_weight);
  a.k_weight = static_cast<const uint16_t*>(r->k_weight);
  a.eps = r->eps;
  a.cos_sin = r->cos_sin; a.pos = r->pos; a.n_pos = r->n_pos;
  a.rot = r->rot_dim; a.interleaved = r->interleaved != 0; a.n_axes = r->n_axes;
  int end = 0;
  for (int x = 0; x < 3; ++x) {
    end += r->n_axes == 1 ? (x == 0 ? r->rot_dim / 2 : 0) : (x < r->n_axes ? r->section[x] : 0);
    a.sec_end[x] = end;
  }
}

// T more tokens behind n_vis + n_text fit the block table, and their positions
// (rounded up to tiles) 32 bits
sv_status check_new_tokens(const sv_seq_batch* S, int T) {
  const long long end = (long long)S->n_vis + S->n_text + T;
  if (end > (long long)S->max_blocks * SV_BLOCK_TOKENS)
    return fail(SV_ERR_INVALID_ARG, "%d new tokens overflow the block table", T);
  if (end > (1 << 30)) return fail(SV_ERR_UNSUPPORTED, "%lld tokens of a sequence: more than 2^30", end);
  return SV_OK;
}

sv_status check_layers(const sv_kv_layer* layers, int n_layers, const sv_seq_batch* seqs) {
  if (n_layers < 0 || (n_layers > 0 && !layers) || !seqs)
    return fail(SV_ERR_INVALID_ARG, "layers and seqs must be non-NULL");
  for (int l = 0; l < n_layers; ++l) {
    sv_status s = sv::check_cache(&layers[l], seqs, true);
    if (s != SV_OK) return s;
    if (layers[l].num_blocks != layers[0].num_blocks || layers[l].n_kv_heads != layers[0].n_kv_heads ||
        layers[l].head_dim != layers[0].head_dim)
      return fail(SV_ERR_INVALID_ARG, "layer %d differs in num_blocks, n_kv_heads or head_dim", l);
  }
  return SV_OK;
}

sv::LayerPools pools_of(const sv_kv_layer* layers, int n) {
  sv::LayerPools p = {};
  for (int l = 0; l < n; ++l) {
    p.k[l] = layers[l].k_pool;
    p.v[l] = layers[l].v_pool;
  }
  return p;
}

sv_status check_pages(const sv_page_pool* pool, const sv_seq_batch* seqs, void* ws, size_t ws_bytes,
                      sv::PagesArgs& a) {
  if (!pool || !seqs) return fail(SV_ERR_INVALID_ARG, "pool or batch descriptor is NULL");
  if (!pool->ref || !pool->n_pages || !seqs->block_table)
    return fail(SV_ERR_INVALID_ARG, "ref, n_pages or block table pointer is NULL");
  if (!aligned16(pool->ref)) return fail(SV_ERR_INVALID_ARG, "ref must be 16-byte aligned");
  if (pool->num_blocks <= 0 || seqs->batch < 0 || seqs->max_blocks <= 0)
    return fail(SV_ERR_INVALID_ARG, "num_blocks and max_blocks must be positive, batch >= 0");
  if (pool->num_blocks > (1 << 30) || (long long)seqs->batch * seqs->max_blocks > (1LL << 30))
    return fail(SV_ERR_UNSUPPORTED, "more than 2^30 pages or block-table entries");
  a.ref = pool->ref;
  a.n_pages = pool->n_pages;
  a.num_pages = pool->num_blocks;
  a.block_table = const_cast<int32_t*>(seqs->block_table);
  a.batch = seqs->batch;
  a.max_blocks = seqs->max_blocks;
  a.status = status_word(ws);
  return check_ws(ws, ws_bytes, sv_pages_workspace_bytes(seqs->batch, seqs->max_blocks, pool->num_blocks));
}

}  // namespace

using sv::check_cache;

extern "C" {

const char* sv_status_string(sv_status s) {
  switch (s) {
    case SV_OK: return "ok";
    case SV_ERR_INVALID_ARG: return "invalid argument";
    case SV_ERR_UNSUPPORTED: return "unsupported shape";
    case SV_ERR_CUDA: return "CUDA error";
    case SV_ERR_WORKSPACE: return "workspace too small";
    case SV_ERR_DEVICE_BOUNDS: return "device-side index out of bounds";
  }
  return "unknown status";
}

const char* sv_last_error(void) { return g_err; }

const char* sv_version(void) { return "sv 0.1 sm_103a"; }

// ------------------------------------------------------------------ sizes

size_t sv_salience_workspace_bytes(int B, int H, int N, int d) {
  if (B < 0 || H < 0 || N <= 0 || !sv::salience_head_dim_supported(d)) return kStatusBytes;
  return kHeadBytes + round256(sv::salience_workspace_bytes(B, H, N, d));
}

int sv_salience_kernel_count(int N, int d) {
  if (N <= 0 || !sv::salience_head_dim_supported(d)) return 0;
  return sv::salience_kernel_count(N, d);
}

size_t sv_topk_workspace_bytes(int rows, int n, int k) {
  (void)rows; (void)n; (void)k;
  return kStatusBytes;
}

size_t sv_prune_workspace_bytes(int B, int N, int k) {
  (void)B; (void)N; (void)k;
  return kStatusBytes;
}

size_t sv_retrieve_workspace_bytes(int B, int H, int n_kv_heads, int head_dim, int n_vis, int k) {
  (void)H; (void)head_dim; (void)k;
  if (B < 0 || n_kv_heads < 0 || n_vis < 0) return kStatusBytes;
  // status | counters | scores [B][Hkv][n_vis]
  return kHeadBytes + round256((size_t)B * n_kv_heads * n_vis * sizeof(float));
}

size_t sv_attn_workspace_bytes(int B, int H, int n_kv_heads, int head_dim, int n_tokens) {
  if (B < 0 || H <= 0 || n_kv_heads <= 0 || head_dim <= 0 || n_tokens < 0 || H % n_kv_heads)
    return kStatusBytes;
  const int G = H / n_kv_heads;
  const sv::AttnPlan p = sv::attn_plan(B, n_kv_heads, G, n_tokens);
  const size_t parts = (size_t)B * n_kv_heads * p.nsplit_max * G;
  // status | counters | (m, l) partials | o partials
  return kHeadBytes + round256(parts * 2 * sizeof(float)) + round256(parts * head_dim * sizeof(float));
}

size_t sv_evict_workspace_bytes(void) { return kStatusBytes; }

int sv_retrieve_kernel_count(int batch, int n_kv_heads, int n_vis) {
  if (n_vis <= 0) return 0;
  return sv::retrieve_fuses_topk(batch * n_kv_heads, n_vis) ? 1 : 2;
}

int sv_attn_kernel_count(int B, int H, int n_kv_heads, int n_tokens) {
  if (B <= 0 || H <= 0 || n_kv_heads <= 0 || H % n_kv_heads || n_tokens <= 0) return 0;
  return sv::attn_kernel_count(B, n_kv_heads, H / n_kv_heads, n_tokens);
}

// ------------------------------------------------------------------ prefill

sv_status sv_salience_prefill(const void* q, const void* k, int B, int H, int N, int d, float scale,
                              float* salience, void* ws, size_t ws_bytes, void* stream) {
  if (!q || !k || !salience) return fail(SV_ERR_INVALID_ARG, "q, k and salience must be non-NULL");
  if (B < 0 || H <= 0 || N <= 0) return fail(SV_ERR_INVALID_ARG, "need B >= 0, H > 0, N > 0");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(SV_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!sv::salience_head_dim_supported(d))
    return fail(SV_ERR_UNSUPPORTED, "salience head_dim %d (64, 72, 80 or 128)", d);
  if (!aligned16(q) || !aligned16(k)) return fail(SV_ERR_INVALID_ARG, "q and k must be 16-byte aligned");
  if (N > (1 << 24)) return fail(SV_ERR_UNSUPPORTED, "N = %d > 2^24 tokens", N);
  if ((long long)B * H * ((N + 127) / 128) > 0x7fffffffLL) return fail(SV_ERR_INVALID_ARG, "B * H * N too large");
  sv_status s = check_ws(ws, ws_bytes, sv_salience_workspace_bytes(B, H, N, d));
  if (s != SV_OK) return s;
  if (B == 0) return SV_OK;
  cudaError_t e = sv::launch_salience(q, k, B, H, N, d, scale, salience, data_of(ws),
                                      counters_of(ws), status_word(ws), num_sms(), static_cast<cudaStream_t>(stream));
  if (e == cudaErrorInvalidValue)
    return fail(SV_ERR_CUDA, "tensor-map encoding or launch rejected the salience operands");
  return cuda_status(e, "sv_salience_prefill");
}

size_t sv_salience_summary_workspace_bytes(int B, int H, int N, int d, int R) {
  (void)d;
  (void)R;
  if (B < 0 || H < 0 || N < 0) return kStatusBytes;
  return kHeadBytes + round256((size_t)B * H * N * sizeof(float));
}

sv_status sv_salience_summary(const void* q, const void* k, int B, int H, int N, int d, int R, float scale,
                              float* salience, void* ws, size_t ws_bytes, void* stream) {
  if (!q || !k || !salience) return fail(SV_ERR_INVALID_ARG, "q, k and salience must be non-NULL");
  if (B < 0 || H <= 0 || N <= 0) return fail(SV_ERR_INVALID_ARG, "need B >= 0, H > 0, N > 0");
  if (R < 1 || R > 16 || R > N) return fail(SV_ERR_INVALID_ARG, "need 1 <= R <= min(16, N) (R = %d)", R);
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(SV_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (d < 8 || d > 256 || d % 8) return fail(SV_ERR_UNSUPPORTED, "summary salience head_dim %d (multiple of 8, <= 256)", d);
  if (!aligned16(q) || !aligned16(k)) return fail(SV_ERR_INVALID_ARG, "q and k must be 16-byte aligned");
  if (sv::summary_smem_bytes(N, d, R) > kMaxSmemPerBlock - 4096)
    return fail(SV_ERR_UNSUPPORTED, "R * N = %d logits do not fit in shared memory", R * N);
  if ((long long)B * H > 0x7fffffffLL) return fail(SV_ERR_INVALID_ARG, "B * H too large");
  sv_status s = check_ws(ws, ws_bytes, sv_salience_summary_workspace_bytes(B, H, N, d, R));
  if (s != SV_OK) return s;
  if (B == 0) return SV_OK;
  cudaError_t e = sv::launch_summary_salience(q, k, B, H, N, d, R, scale, salience,
                                              reinterpret_cast<float*>(data_of(ws)),
                                              static_cast<cudaStream_t>(stream));
  return cuda_status(e, "sv_salience_summary");
}

sv_status sv_topk_rows(const float* scores, int rows, int n, int k, int32_t* idx, void* ws,
                       size_t ws_bytes, void* stream) {
  if (!scores || !idx) return fail(SV_ERR_INVALID_ARG, "scores and idx must be non-NULL");
  if (rows < 0 || n <= 0 || n > (1 << 24)) return fail(SV_ERR_INVALID_ARG, "need rows >= 0, 0 < n <= 2^24");
  if (k < 1 || k > n) return fail(SV_ERR_INVALID_ARG, "need 1 <= k <= n (k = %d, n = %d)", k, n);
  sv_status s = check_ws(ws, ws_bytes, sv_topk_workspace_bytes(rows, n, k));
  if (s != SV_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // long rows: a cluster of CTAs per row; otherwise one CTA per row
  const cudaError_t e = sv::topk_prefers_cluster(n)
                            ? sv::launch_topk_cluster(scores, rows, n, k, idx, st)
                            : sv::launch_topk_rows(scores, rows, n, k, idx, st);
  return cuda_status(e, "sv_topk_rows");
}

sv_status sv_prune_threshold(const float* salience, int B, int N, float threshold, const void* feat,
                             int64_t row_bytes, void* feat_out, int32_t* kept_idx, int32_t* kept_count,
                             void* ws, size_t ws_bytes, void* stream) {
  if (!salience || !kept_idx || !kept_count)
    return fail(SV_ERR_INVALID_ARG, "salience, kept_idx and kept_count must be non-NULL");
  if (B < 0 || N <= 0 || N > (1 << 24)) return fail(SV_ERR_INVALID_ARG, "need B >= 0, 0 < N <= 2^24");
  if (std::isnan(threshold)) return fail(SV_ERR_INVALID_ARG, "threshold is NaN");
  if (row_bytes < 0 || row_bytes % 16) return fail(SV_ERR_INVALID_ARG, "row_bytes must be a multiple of 16");
  if (row_bytes > 0 && (!feat || !feat_out)) return fail(SV_ERR_INVALID_ARG, "feat and feat_out must be non-NULL");
  if (row_bytes > 0 && (!aligned16(feat) || !aligned16(feat_out)))
    return fail(SV_ERR_INVALID_ARG, "feat and feat_out must be 16-byte aligned");
  sv_status s = check_ws(ws, ws_bytes, sv_prune_workspace_bytes(B, N, 1));
  if (s != SV_OK) return s;
  if (B == 0) return SV_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = sv::launch_threshold_select(salience, B, N, threshold, kept_idx, kept_count, st);
  if (e == cudaSuccess && row_bytes > 0)
    e = sv::launch_gather_rows(feat, B, N, N, row_bytes, kept_idx, feat_out, status_word(ws), st, kept_count);
  return cuda_status(e, "sv_prune_threshold");
}

sv_status sv_prune_compact(const float* salience, int B, int N, int k, const void* feat,
                           int64_t row_bytes, void* feat_out, int32_t* kept_idx, void* ws,
                           size_t ws_bytes, void* stream) {
  if (!salience || !kept_idx) return fail(SV_ERR_INVALID_ARG, "salience and kept_idx must be non-NULL");
  if (B < 0 || N <= 0 || N > (1 << 24)) return fail(SV_ERR_INVALID_ARG, "need B >= 0, 0 < N <= 2^24");
  if (k < 1 || k > N) return fail(SV_ERR_INVALID_ARG, "need 1 <= k <= N (k = %d, N = %d)", k, N);
  if (row_bytes < 0 || row_bytes % 16) return fail(SV_ERR_INVALID_ARG, "row_bytes must be a multiple of 16");
  if (row_bytes > 0 && (!feat || !feat_out)) return fail(SV_ERR_INVALID_ARG, "feat and feat_out must be non-NULL");
  if (row_bytes > 0 && (!aligned16(feat) || !aligned16(feat_out)))
    return fail(SV_ERR_INVALID_ARG, "feat and feat_out must be 16-byte aligned");
  sv_status s = check_ws(ws, ws_bytes, sv_prune_workspace_bytes(B, N, k));
  if (s != SV_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = sv::launch_topk_rows(salience, B, N, k, kept_idx, st);
  if (e == cudaSuccess && row_bytes > 0)
    e = sv::launch_gather_rows(feat, B, N, k, row_bytes, kept_idx, feat_out, status_word(ws), st);
  return cuda_status(e, "sv_prune_compact");
}

// ------------------------------------------------------------------ decode

sv_status sv_retrieve_topk(const void* q, int R, int H, const sv_kv_layer* layer,
                           const sv_seq_batch* seqs, int k, int32_t* vis_idx, float* scores,
                           void* ws, size_t ws_bytes, void* stream) {
  sv_status s = sv::check_retrieve_args(q, R, H, layer, seqs, k, vis_idx);
  if (s != SV_OK) return s;
  const int Hkv = layer->n_kv_heads;
  s = check_ws(ws, ws_bytes, sv_retrieve_workspace_bytes(seqs->batch, H, Hkv, layer->head_dim, seqs->n_vis, k));
  if (s != SV_OK) return s;
  if (seqs->batch == 0) return SV_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* sc = scores ? scores : reinterpret_cast<float*>(data_of(ws));
  cudaError_t e = sv::launch_retrieve(q, R, H, H / Hkv, layer->k_pool, layer->num_blocks, Hkv,
                                      layer->head_dim, seqs->block_table, seqs->max_blocks, seqs->n_vis,
                                      seqs->batch, sc, status_word(ws), num_sms(), counters_of(ws), k, vis_idx, st,
                                      lens_of(seqs), seqs->n_text);
  return cuda_status(e, "sv_retrieve_topk");
}

size_t sv_retrieve_softmax_workspace_bytes(int B, int R, int H, int n_kv_heads, int head_dim, int n_vis,
                                           int n_text) {
  if (B < 0 || R <= 0 || H <= 0 || n_kv_heads <= 0 || H % n_kv_heads || n_vis < 0 || n_text < 0) return kStatusBytes;
  return kHeadBytes + sv::retrieve_softmax_workspace_bytes(B, R, H, n_kv_heads, head_dim, n_vis, n_text);
}

sv_status sv_retrieve_topk_softmax(const void* q, int R, int H, float scale, const sv_kv_layer* layer,
                                   const sv_seq_batch* seqs, const float* lse, int k, int32_t* vis_idx,
                                   float* scores, void* ws, size_t ws_bytes, void* stream) {
  sv_status s = check_cache(layer, seqs, false);
  if (s != SV_OK) return s;
  s = reject_lens(seqs, "sv_retrieve_topk_softmax");
  if (s != SV_OK) return s;
  if (!q || !vis_idx) return fail(SV_ERR_INVALID_ARG, "q and vis_idx must be non-NULL");
  if (!aligned16(q)) return fail(SV_ERR_INVALID_ARG, "q must be 16-byte aligned");
  const int Hkv = layer->n_kv_heads;
  if (R <= 0 || H <= 0 || H % Hkv) return fail(SV_ERR_INVALID_ARG, "need R > 0 and H a multiple of n_kv_heads");
  if (R * (H / Hkv) > sv::retrieve_softmax_max_rows())
    return fail(SV_ERR_UNSUPPORTED, "R * (H / n_kv_heads) = %d > %d question rows per KV head", R * (H / Hkv),
                sv::retrieve_softmax_max_rows());
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(SV_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (seqs->n_vis <= 0) return fail(SV_ERR_INVALID_ARG, "no visual tokens to retrieve from");
  if (k < 1 || k > seqs->n_vis) return fail(SV_ERR_INVALID_ARG, "need 1 <= k <= n_vis (k = %d)", k);
  s = check_ws(ws, ws_bytes,
               sv_retrieve_softmax_workspace_bytes(seqs->batch, R, H, Hkv, layer->head_dim, seqs->n_vis, seqs->n_text));
  if (s != SV_OK) return s;
  if (seqs->batch == 0) return SV_OK;
  cudaError_t e = sv::launch_retrieve_softmax(q, R, H, scale, layer->k_pool, layer->num_blocks, Hkv, layer->head_dim,
                                              seqs->block_table, seqs->max_blocks, seqs->n_vis, seqs->n_text,
                                              seqs->batch, lse, k, vis_idx, scores, data_of(ws), status_word(ws),
                                              static_cast<cudaStream_t>(stream));
  return cuda_status(e, "sv_retrieve_topk_softmax");
}

}  // extern "C"

// sv_sparse_decode_attn, and with k_new / v_new the fused append of one token
// per sequence before it (sv_decode_append_attn)
static sv_status decode_attn(const char* name, const void* q, int H, float scale, const sv_kv_layer* layer,
                             const sv_seq_batch* seqs, const void* k_new, const void* v_new,
                             const int32_t* vis_idx, int k, void* out, float* lse, void* ws, size_t ws_bytes,
                             void* stream) {
  sv_status s = check_cache(layer, seqs, true);
  if (s != SV_OK) return s;
  if (!q || !out) return fail(SV_ERR_INVALID_ARG, "q and out must be non-NULL");
  if (!aligned16(q)) return fail(SV_ERR_INVALID_ARG, "q must be 16-byte aligned");
  const int Hkv = layer->n_kv_heads;
  if (H <= 0 || H % Hkv) return fail(SV_ERR_INVALID_ARG, "H must be a positive multiple of n_kv_heads");
  if (H / Hkv > 16) return fail(SV_ERR_UNSUPPORTED, "query heads per KV head %d > 16", H / Hkv);
  if (!std::isfinite(scale)) return fail(SV_ERR_INVALID_ARG, "scale must be finite");
  const bool append = k_new != nullptr || v_new != nullptr;
  if (append) {
    if (!k_new || !v_new) return fail(SV_ERR_INVALID_ARG, "k_new and v_new must be non-NULL");
    if (!aligned16(k_new) || !aligned16(v_new))
      return fail(SV_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    if ((long long)seqs->n_vis + seqs->n_text + 1 > (long long)seqs->max_blocks * SV_BLOCK_TOKENS)
      return fail(SV_ERR_INVALID_ARG, "appending a token overflows the block table");
  }
  const int k_vis = vis_idx ? k : seqs->n_vis;
  if (vis_idx && (k < 0 || k > seqs->n_vis)) return fail(SV_ERR_INVALID_ARG, "need 0 <= k <= n_vis");
  const int n_tok = k_vis + seqs->n_text + (append ? 1 : 0);
  if (n_tok <= 0) return fail(SV_ERR_INVALID_ARG, "the attended token set is empty");
  s = check_ws(ws, ws_bytes, sv_attn_workspace_bytes(seqs->batch, H, Hkv, layer->head_dim, n_tok));
  if (s != SV_OK) return s;
  if (seqs->batch == 0) return SV_OK;
  const sv::AttnPlan p = sv::attn_plan(seqs->batch, Hkv, H / Hkv, n_tok);
  const size_t parts = (size_t)seqs->batch * Hkv * p.nsplit * (H / Hkv);
  sv::AttnArgs a;
  a.q = q; a.H = H; a.scale = scale;
  a.k_pool = layer->k_pool; a.v_pool = layer->v_pool;
  a.num_blocks = layer->num_blocks; a.Hkv = Hkv; a.D = layer->head_dim;
  a.block_table = seqs->block_table; a.max_blocks = seqs->max_blocks;
  a.vis_idx = vis_idx; a.k_vis = k_vis; a.n_vis = seqs->n_vis; a.n_text = seqs->n_text;
  a.batch = seqs->batch; a.out = out; a.lse = lse;
  a.lens = lens_of(seqs);
  a.k_new = k_new; a.v_new = v_new;
  a.split_done = counters_of(ws);
  a.part_ml = reinterpret_cast<float*>(data_of(ws));
  a.part_o = reinterpret_cast<float*>(data_of(ws) + round256(parts * 2 * sizeof(float)));
  a.status = status_word(ws);
  return cuda_status(sv::launch_sparse_attn(a, static_cast<cudaStream_t>(stream)), name);
}

extern "C" {

sv_status sv_sparse_decode_attn(const void* q, int H, float scale, const sv_kv_layer* layer,
                                const sv_seq_batch* seqs, const int32_t* vis_idx, int k, void* out,
                                float* lse, void* ws, size_t ws_bytes, void* stream) {
  return decode_attn("sv_sparse_decode_attn", q, H, scale, layer, seqs, nullptr, nullptr, vis_idx, k, out, lse, ws,
                     ws_bytes, stream);
}

sv_status sv_decode_append_attn(const void* q, int H, float scale, const sv_kv_layer* layer,
                                const sv_seq_batch* seqs, const void* k_new, const void* v_new,
                                const int32_t* vis_idx, int k, void* out, float* lse, void* ws, size_t ws_bytes,
                                void* stream) {
  if (!k_new || !v_new) return fail(SV_ERR_INVALID_ARG, "k_new and v_new must be non-NULL");
  return decode_attn("sv_decode_append_attn", q, H, scale, layer, seqs, k_new, v_new, vis_idx, k, out, lse, ws,
                     ws_bytes, stream);
}

// ------------------------------------------------------------------ rounds

sv_status sv_pack_kv(const sv_kv_layer* src, const sv_seq_batch* seqs, const int32_t* vis_idx, int k,
                     const sv_kv_layer* dst, const sv_seq_batch* dst_seqs, void* ws, size_t ws_bytes,
                     void* stream) {
  sv_status s = check_cache(src, seqs, true);
  if (s != SV_OK) return s;
  s = check_cache(dst, dst_seqs, true);
  if (s != SV_OK) return s;
  s = reject_lens(seqs, "sv_pack_kv");
  if (s == SV_OK) s = reject_lens(dst_seqs, "sv_pack_kv");
  if (s != SV_OK) return s;
  if (dst->n_kv_heads != src->n_kv_heads || dst->head_dim != src->head_dim)
    return fail(SV_ERR_INVALID_ARG, "source and packed layers differ in n_kv_heads or head_dim");
  if (dst->k_pool == src->k_pool || dst->v_pool == src->v_pool)
    return fail(SV_ERR_INVALID_ARG, "the packed layer must not share pools with the source");
  const int k_vis = vis_idx ? k : seqs->n_vis;
  if (vis_idx && (k < 0 || k > seqs->n_vis)) return fail(SV_ERR_INVALID_ARG, "need 0 <= k <= n_vis");
  if (dst_seqs->batch != seqs->batch || dst_seqs->n_vis != k_vis || dst_seqs->n_text != seqs->n_text)
    return fail(SV_ERR_INVALID_ARG,
                "packed batch must have the source's batch, n_vis = k (%d) and n_text = %d", k_vis, seqs->n_text);
  s = check_ws(ws, ws_bytes, sv_evict_workspace_bytes());
  if (s != SV_OK) return s;
  cudaError_t e = sv::launch_pack_kv(src->k_pool, src->v_pool, src->num_blocks, seqs->block_table,
                                     seqs->max_blocks, seqs->n_vis, vis_idx, k_vis, seqs->n_text, dst->k_pool,
                                     dst->v_pool, dst->num_blocks, dst_seqs->block_table, dst_seqs->max_blocks,
                                     seqs->batch, src->n_kv_heads, src->head_dim, status_word(ws),
                                     static_cast<cudaStream_t>(stream));
  return cuda_status(e, "sv_pack_kv");
}

sv_status sv_evict_qa_tokens(const sv_kv_layer* layers, int n_layers, sv_seq_batch* seqs,
                             int32_t text_begin, int32_t text_end, int32_t* n_blocks_in_use,
                             void* ws, size_t ws_bytes, void* stream) {
  if (!layers || !seqs || n_layers < 0) return fail(SV_ERR_INVALID_ARG, "layers and seqs must be non-NULL");
  if (reject_lens(seqs, "sv_evict_qa_tokens") != SV_OK) return SV_ERR_UNSUPPORTED;
  if (text_begin < 0 || text_begin > text_end || text_end > seqs->n_text)
    return fail(SV_ERR_INVALID_ARG, "need 0 <= text_begin <= text_end <= n_text (%d, %d, %d)",
                text_begin, text_end, seqs->n_text);
  for (int l = 0; l < n_layers; ++l) {
    sv_status s = check_cache(&layers[l], seqs, true);
    if (s != SV_OK) return s;
  }
  sv_status s = check_ws(ws, ws_bytes, sv_evict_workspace_bytes());
  if (s != SV_OK) return s;
  const int count = seqs->n_text - text_end;   // later text tokens to move down
  if (text_end > text_begin && count > 0) {
    for (int l = 0; l < n_layers; ++l) {
      cudaError_t e = sv::launch_kv_move_down(
          layers[l].k_pool, layers[l].v_pool, layers[l].num_blocks, layers[l].n_kv_heads,
          layers[l].head_dim, seqs->block_table, seqs->max_blocks, seqs->batch,
          seqs->n_vis + text_begin, seqs->n_vis + text_end, count, status_word(ws),
          static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return cuda_status(e, "sv_evict_qa_tokens");
    }
  }
  seqs->n_text -= text_end - text_begin;
  if (n_blocks_in_use) {
    const int need = (seqs->n_vis + seqs->n_text + SV_BLOCK_TOKENS - 1) / SV_BLOCK_TOKENS;
    for (int b = 0; b < seqs->batch; ++b) n_blocks_in_use[b] = need;
  }
  return SV_OK;
}

sv_status sv_kv_append(const sv_kv_layer* layer, const sv_seq_batch* seqs, const void* k_new,
                       const void* v_new, int T, void* ws, size_t ws_bytes, void* stream) {
  sv_status s = check_cache(layer, seqs, true);
  if (s != SV_OK) return s;
  if (T < 0) return fail(SV_ERR_INVALID_ARG, "T must be >= 0");
  if (T > 0 && (!k_new || !v_new)) return fail(SV_ERR_INVALID_ARG, "k_new and v_new must be non-NULL");
  if (T > 0 && (!aligned16(k_new) || !aligned16(v_new)))
    return fail(SV_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
  if ((long long)seqs->n_vis + seqs->n_text + T > (long long)seqs->max_blocks * SV_BLOCK_TOKENS)
    return fail(SV_ERR_INVALID_ARG, "appending %d tokens overflows the block table", T);
  s = check_ws(ws, ws_bytes, sv_evict_workspace_bytes());
  if (s != SV_OK) return s;
  return cuda_status(sv::launch_kv_append(layer->k_pool, layer->v_pool, layer->num_blocks,
                                          layer->n_kv_heads, layer->head_dim, seqs->block_table,
                                          seqs->max_blocks, seqs->batch, seqs->n_vis + seqs->n_text,
                                          k_new, v_new, T, status_word(ws),
                                          static_cast<cudaStream_t>(stream), lens_of(seqs), seqs->n_vis,
                                          seqs->n_text),
                     "sv_kv_append");
}

// ------------------------------------------------------------------ new tokens, drafts and branches

sv_status sv_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int B, int N, int H,
                          int Hk, int d, const sv_rotation* rot, void* q_out, void* k_out, void* ws,
                          size_t ws_bytes, void* stream) {
  if (B < 0 || N < 0 || H <= 0 || Hk <= 0) return fail(SV_ERR_INVALID_ARG, "need B >= 0, N >= 0, H > 0, Hk > 0");
  const long long n_tok = (long long)B * N, qr = (long long)H * d, kr = (long long)Hk * d;
  if (n_tok > 0 && (!q || !k || !q_out || !k_out))
    return fail(SV_ERR_INVALID_ARG, "q, k, q_out and k_out must be non-NULL");
  if (!sv::salience_head_dim_supported(d)) return fail(SV_ERR_UNSUPPORTED, "head_dim %d (64, 72, 80 or 128)", d);
  sv_status s = check_rows("q", q, q_stride, qr);
  if (s == SV_OK) s = check_rows("k", k, k_stride, kr);
  if (s == SV_OK) s = check_rotation(rot, d, n_tok);
  if (s == SV_OK) s = check_ws(ws, ws_bytes, sv_evict_workspace_bytes());
  if (s != SV_OK) return s;
  if (!aligned16(q_out) || !aligned16(k_out))
    return fail(SV_ERR_INVALID_ARG, "q_out and k_out must be 16-byte aligned");
  if (n_tok == 0) return SV_OK;
  const size_t q_in = row_extent(n_tok, q_stride, qr), k_in = row_extent(n_tok, k_stride, kr);
  const size_t qb = (size_t)n_tok * qr * 2, kb = (size_t)n_tok * kr * 2;
  if (overlap(q_out, qb, q, q_in) || overlap(q_out, qb, k, k_in) || overlap(k_out, kb, q, q_in) ||
      overlap(k_out, kb, k, k_in) || overlap(q_out, qb, k_out, kb))
    return fail(SV_ERR_INVALID_ARG, "q_out and k_out must not overlap the inputs or one another");
  sv::NormRopeArgs a = {};
  fill_rotation(a, rot);
  a.q = static_cast<const uint16_t*>(q); a.k = static_cast<const uint16_t*>(k);
  a.q_stride = q_stride; a.k_stride = k_stride;
  a.B = B; a.T = N; a.H = H; a.Hk = Hk;
  a.q_out = static_cast<uint16_t*>(q_out); a.k_out = static_cast<uint16_t*>(k_out);
  a.status = status_word(ws);
  return cuda_status(sv::launch_norm_rope(a, d, false, num_sms(), static_cast<cudaStream_t>(stream)), "sv_qk_norm_rope");
}

sv_status sv_qk_norm_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, int T, int H, const sv_rotation* rot, const sv_kv_layer* layer,
                                 const sv_seq_batch* seqs, const int32_t* n_new, void* q_out, void* ws,
                                 size_t ws_bytes, void* stream) {
  sv_status s = check_cache(layer, seqs, true);
  if (s != SV_OK) return s;
  const int Hkv = layer->n_kv_heads, d = layer->head_dim;
  if (T < 0) return fail(SV_ERR_INVALID_ARG, "T must be >= 0");
  if (T > 0 && seqs->batch > 0 && (!q || !k || !v || !q_out))
    return fail(SV_ERR_INVALID_ARG, "q, k, v and q_out must be non-NULL");
  if (H <= 0 || H % Hkv) return fail(SV_ERR_INVALID_ARG, "H must be a positive multiple of n_kv_heads");
  s = check_new_tokens(seqs, T);
  const long long n_tok = (long long)seqs->batch * T, qr = (long long)H * d, kv = (long long)Hkv * d;
  if (s == SV_OK) s = check_rows("q", q, q_stride, qr);
  if (s == SV_OK) s = check_rows("k", k, k_stride, kv);
  if (s == SV_OK) s = check_rows("v", v, v_stride, kv);
  if (s == SV_OK) s = check_rotation(rot, d, n_tok);
  if (s == SV_OK) s = check_ws(ws, ws_bytes, sv_evict_workspace_bytes());
  if (s != SV_OK) return s;
  if (!aligned16(q_out)) return fail(SV_ERR_INVALID_ARG, "q_out must be 16-byte aligned");
  if (n_tok == 0) return SV_OK;
  const size_t qb = (size_t)n_tok * qr * 2;
  const bool in_place = q_out == q && q_stride == qr;
  if ((!in_place && overlap(q_out, qb, q, row_extent(n_tok, q_stride, qr))) ||
      overlap(q_out, qb, k, row_extent(n_tok, k_stride, kv)) || overlap(q_out, qb, v, row_extent(n_tok, v_stride, kv)))
    return fail(SV_ERR_INVALID_ARG, "q_out must be q itself or not overlap q, k and v");
  sv::NormRopeArgs a = {};
  fill_rotation(a, rot);
  a.q = static_cast<const uint16_t*>(q); a.k = static_cast<const uint16_t*>(k); a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.B = seqs->batch; a.T = T; a.H = H; a.Hk = Hkv;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_out = static_cast<uint16_t*>(layer->k_pool); a.v_out = static_cast<uint16_t*>(layer->v_pool);
  a.status = status_word(ws);
  a.block_table = seqs->block_table; a.num_blocks = layer->num_blocks; a.max_blocks = seqs->max_blocks;
  a.n_vis = seqs->n_vis; a.n_text = seqs->n_text; a.lens = lens_of(seqs); a.n_new = n_new;
  return cuda_status(sv::launch_norm_rope(a, d, true, num_sms(), static_cast<cudaStream_t>(stream)), "sv_qk_norm_rope_append");
}

size_t sv_tree_attn_workspace_bytes(int B, int T, int H, int n_kv_heads, int head_dim, int n_tokens) {
  if (B < 0 || T < 0 || H <= 0 || n_kv_heads <= 0 || H % n_kv_heads || head_dim <= 0 || n_tokens < 0)
    return kStatusBytes;
  return kHeadBytes + round256(sv::tree_attn_workspace_bytes(B, T, H, n_kv_heads, head_dim, n_tokens));
}

sv_status sv_tree_attn(const void* q, int T, int H, float scale, const sv_kv_layer* layer, const sv_seq_batch* seqs,
                       const int32_t* vis_idx, int k, const uint64_t* tree_mask, const int32_t* n_new, void* out,
                       float* lse, void* ws, size_t ws_bytes, void* stream) {
  sv_status s = check_cache(layer, seqs, true);
  if (s != SV_OK) return s;
  if (T > 0 && seqs->batch > 0 && (!q || !out)) return fail(SV_ERR_INVALID_ARG, "q and out must be non-NULL");
  if (!aligned16(q) || !aligned16(out)) return fail(SV_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(tree_mask) % 8) return fail(SV_ERR_INVALID_ARG, "tree_mask must be 8-byte aligned");
  const int Hkv = layer->n_kv_heads;
  if (H <= 0 || H % Hkv) return fail(SV_ERR_INVALID_ARG, "H must be a positive multiple of n_kv_heads");
  if (H / Hkv > 16) return fail(SV_ERR_UNSUPPORTED, "query heads per KV head %d > 16", H / Hkv);
  if (!(scale >= 0.f) || !std::isfinite(scale * 1.4426950408889634f))
    return fail(SV_ERR_INVALID_ARG, "scale must be >= 0 and finite, times log2(e) too");
  if (T < 0 || T > 65536) return fail(SV_ERR_INVALID_ARG, "need 0 <= T <= 65536 (T = %d)", T);
  if (tree_mask && T > 64) return fail(SV_ERR_UNSUPPORTED, "a tree mask holds at most 64 drafted tokens (T = %d)", T);
  s = check_new_tokens(seqs, T);
  if (s != SV_OK) return s;
  const int k_vis = vis_idx ? k : seqs->n_vis;
  if (vis_idx && (k < 0 || k > seqs->n_vis)) return fail(SV_ERR_INVALID_ARG, "need 0 <= k <= n_vis");
  if ((long long)seqs->batch * T * H > 0x7fffffffLL) return fail(SV_ERR_INVALID_ARG, "batch * T * H too large");
  const size_t out_bytes = (size_t)seqs->batch * T * H * layer->head_dim * 2;
  if (out != q && overlap(out, out_bytes, q, out_bytes))
    return fail(SV_ERR_INVALID_ARG, "out must be q itself or not overlap it");
  const long long n_tok = (long long)k_vis + seqs->n_text + T;   // <= max_blocks * 16
  if (seqs->batch * (n_tok / 128 + 1) > 0x7fffffffLL / Hkv)
    return fail(SV_ERR_UNSUPPORTED, "batch * n_kv_heads * tokens beyond 2^38");
  s = check_ws(ws, ws_bytes,
               sv_tree_attn_workspace_bytes(seqs->batch, T, H, Hkv, layer->head_dim, (int)n_tok));
  if (s != SV_OK) return s;
  if (seqs->batch == 0 || T == 0) return SV_OK;
  sv::TreeArgs a = {};
  // hidden logits are -inf, which a factor of 0 would turn into NaN: the
  // kernel takes 0 times the queries instead
  a.q = q; a.T = T; a.H = H;
  a.zero_scale = scale == 0.f;
  a.scale_log2 = a.zero_scale ? 1.f : scale * 1.4426950408889634f;
  a.k_pool = layer->k_pool; a.v_pool = layer->v_pool;
  a.num_blocks = layer->num_blocks; a.Hkv = Hkv; a.D = layer->head_dim;
  a.block_table = seqs->block_table; a.max_blocks = seqs->max_blocks;
  a.vis_idx = vis_idx; a.k_vis = k_vis; a.n_vis = seqs->n_vis; a.n_text = seqs->n_text; a.batch = seqs->batch;
  a.lens = lens_of(seqs);
  a.tree_mask = tree_mask; a.n_new = n_new;
  a.out = out; a.lse = lse;
  a.ws = data_of(ws); a.status = status_word(ws);
  return cuda_status(sv::launch_tree_attn(a, static_cast<cudaStream_t>(stream)), "sv_tree_attn");
}

sv_status sv_kv_accept(const sv_kv_layer* layers, int n_layers, const sv_seq_batch* seqs, int T, const int32_t* path,
                       int P, const int32_t* n_path, void* ws, size_t ws_bytes, void* stream) {
  sv_status s = check_layers(layers, n_layers, seqs);
  if (s != SV_OK) return s;
  if (T < 0 || P < 0 || P > T) return fail(SV_ERR_INVALID_ARG, "need 0 <= P <= T (P = %d, T = %d)", P, T);
  if (P > 64) return fail(SV_ERR_UNSUPPORTED, "an accepted path has at most 64 tokens (P = %d)", P);
  if (P > 0 && !path) return fail(SV_ERR_INVALID_ARG, "path must be non-NULL");
  s = check_new_tokens(seqs, T);
  if (s == SV_OK) s = check_ws(ws, ws_bytes, sv_evict_workspace_bytes());
  if (s != SV_OK) return s;
  for (int l0 = 0; l0 < n_layers; l0 += sv::kMaxLayers) {
    const int n = n_layers - l0 < sv::kMaxLayers ? n_layers - l0 : sv::kMaxLayers;
    const cudaError_t e = sv::launch_kv_accept(pools_of(layers + l0, n), n, layers->num_blocks, layers->n_kv_heads,
                                               layers->head_dim, seqs->block_table, seqs->max_blocks, seqs->batch,
                                               lens_of(seqs), seqs->n_vis, seqs->n_text, T, path, P, n_path,
                                               status_word(ws), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_status(e, "sv_kv_accept");
  }
  return SV_OK;
}

size_t sv_pages_workspace_bytes(int batch, int max_blocks, int num_blocks) {
  if (batch < 0 || max_blocks < 0 || num_blocks < 0) return kStatusBytes;
  return kHeadBytes + round256(sv::pages_workspace_bytes(batch, max_blocks, num_blocks));
}

sv_status sv_pages_release(const sv_page_pool* pool, const sv_seq_batch* seqs, const int32_t* keep, void* ws,
                           size_t ws_bytes, void* stream) {
  sv::PagesArgs a;
  sv_status s = check_pages(pool, seqs, ws, ws_bytes, a);
  if (s != SV_OK) return s;
  return cuda_status(sv::launch_pages_release(a, keep, static_cast<cudaStream_t>(stream)), "sv_pages_release");
}

sv_status sv_pages_fork(const sv_page_pool* pool, const sv_seq_batch* seqs, const int32_t* parent,
                        const int32_t* child, int n, const int32_t* n_tok, void* ws, size_t ws_bytes, void* stream) {
  sv::PagesArgs a;
  sv_status s = check_pages(pool, seqs, ws, ws_bytes, a);
  if (s != SV_OK) return s;
  if (n < 0) return fail(SV_ERR_INVALID_ARG, "n must be >= 0");
  if (n > 0 && (!parent || !child)) return fail(SV_ERR_INVALID_ARG, "parent and child must be non-NULL");
  return cuda_status(sv::launch_pages_fork(a, parent, child, n, n_tok, static_cast<cudaStream_t>(stream)),
                     "sv_pages_fork");
}

sv_status sv_pages_reserve(const sv_page_pool* pool, const sv_kv_layer* layers, int n_layers, const sv_seq_batch* seqs,
                           int T, const int32_t* n_new, void* ws, size_t ws_bytes, void* stream) {
  sv::PagesArgs a;
  sv_status s = check_pages(pool, seqs, ws, ws_bytes, a);
  if (s == SV_OK && n_layers != 0) s = check_layers(layers, n_layers, seqs);
  if (s != SV_OK) return s;
  if (n_layers > 0 && layers->num_blocks != pool->num_blocks)
    return fail(SV_ERR_INVALID_ARG, "the layers have %d pages, the pool %d", layers->num_blocks, pool->num_blocks);
  if (seqs->n_vis < 0 || seqs->n_text < 0 || T < 0) return fail(SV_ERR_INVALID_ARG, "negative length");
  s = check_new_tokens(seqs, T);
  if (s != SV_OK) return s;
  constexpr int kGroups = 16;
  if (n_layers > kGroups * sv::kMaxLayers)
    return fail(SV_ERR_UNSUPPORTED, "more than %d layers", kGroups * sv::kMaxLayers);
  sv::LayerPools pools[kGroups];
  int count[kGroups], groups = 0;
  for (int l0 = 0; l0 < n_layers; l0 += sv::kMaxLayers, ++groups) {
    count[groups] = n_layers - l0 < sv::kMaxLayers ? n_layers - l0 : sv::kMaxLayers;
    pools[groups] = pools_of(layers + l0, count[groups]);
  }
  const int page_bytes = n_layers > 0 ? layers->n_kv_heads * SV_BLOCK_TOKENS * layers->head_dim * 2 : 0;
  return cuda_status(sv::launch_pages_reserve(a, lens_of(seqs), seqs->n_vis, seqs->n_text, T, n_new, pools, groups,
                                              count, page_bytes, data_of(ws), num_sms(),
                                              static_cast<cudaStream_t>(stream)),
                     "sv_pages_reserve");
}

sv_status sv_read_device_status(void* ws, int clear, int32_t* status_out, void* stream) {
  if (!ws || !status_out) return fail(SV_ERR_INVALID_ARG, "ws and status_out must be non-NULL");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, ws, sizeof(v), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && clear) e = cudaMemsetAsync(ws, 0, sizeof(int32_t), st);
  if (e != cudaSuccess) return cuda_status(e, "sv_read_device_status");
  *status_out = v;
  return SV_OK;
}

}  // extern "C"
