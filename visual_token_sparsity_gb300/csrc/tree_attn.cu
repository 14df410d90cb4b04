// Attention of T drafted (or question) tokens per sequence over the paged
// cache: the selected visual tokens, the text, and of the T tokens' own keys
// (already appended behind the text) those that the tree mask lets each see.
//
//   tok(i) = vis_idx[i] (i < k), then n_vis + (i - k): text, then drafted
//   z_i = scale q . K[tok(i)], seen(i) = i < k + n_text or bit (i - k - n_text)
//   out = sum_seen exp(z_i - m) V[tok(i)] / sum_seen exp(z_i - m)
//
// One warp per query row: a lane holds D / 32 dims of q and of the output and
// keeps the running maximum and sum of the softmax.
#include "common.cuh"
#include "kernels.h"

namespace sv {

template <int D>
__global__ void __launch_bounds__(256)
tree_attn_row_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int E = D / 32;
  grid_dep_sync();
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (long long)a.batch * a.T * a.H) return;
  const int h = (int)(w % a.H);
  const int t = (int)(w / a.H % a.T), b = (int)(w / a.H / a.T);
  const int g = h / (a.H / a.Hkv);
  int nv, nt, kb;
  const bool report = lane == 0 && t == 0 && h == 0;
  bool ok = attn_lengths(a.lens, a.vis_idx != nullptr, b, a.n_vis, a.n_text, a.k_vis, report, a.status, nv, nt, kb);
  int tn = a.n_new ? __ldg(a.n_new + b) : a.T;
  if (tn < 0 || tn > a.T) {
    if (report) flag_status(a.status, kStatusBadLength);
    ok = false;
  }
  if (!ok) kb = nt = tn = 0;
  else if (t >= tn) return;
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;
  const int32_t* vrow = a.vis_idx ? a.vis_idx + ((size_t)b * a.Hkv + g) * a.k_vis : nullptr;
  const uint64_t mask = a.tree_mask ? a.tree_mask[(size_t)b * a.T + t] : 0;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.q)[(size_t)w * D + e * 32 + lane] << 16);
    o[e] = 0.f;
  }
  for (int i = 0; i < kb + nt + tn; ++i) {
    const int j = i - kb - nt;
    if (j >= 0 && !(a.tree_mask ? (mask >> j) & 1 : j <= t)) continue;
    int pos = i < kb ? (vrow ? __ldg(vrow + i) : i) : nv + (i - kb);
    if (i < kb && (pos < 0 || pos >= nv)) {
      flag_status(a.status, kStatusBadIndex);
      continue;
    }
    const int page = __ldg(bt + (pos >> 4));
    if (page < 0 || page >= a.num_blocks) {
      flag_status(a.status, kStatusBadBlock);
      continue;
    }
    const size_t row = ((((size_t)page * a.Hkv + g) << 4) + (pos & 15)) * D + lane;
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      z = fmaf(q[e], __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.k_pool)[row + 32 * e] << 16), z);
    z = warp_sum(z) * a.scale_log2;
    const float mn = fmaxf(m, z);
    const float old = m == -INFINITY ? 0.f : fast_exp2(m - mn);
    const float p = fast_exp2(z - mn);
    l = l * old + p;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = fmaf(p, __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.v_pool)[row + 32 * e] << 16),
                  o[e] * old);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int e = 0; e < E; ++e)
    static_cast<uint16_t*>(a.out)[(size_t)w * D + e * 32 + lane] = (uint16_t)f32_to_bf16_bits(o[e] * inv);
  if (a.lse != nullptr && lane == 0)
    a.lse[w] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

size_t tree_attn_workspace_bytes(int B, int T, int H, int Hkv, int D, int n_tokens) {
  (void)B; (void)T; (void)H; (void)Hkv; (void)D; (void)n_tokens;
  return 0;
}

cudaError_t launch_tree_attn(const TreeArgs& a, cudaStream_t stream) {
  const long long rows = (long long)a.batch * a.T * a.H;
  const dim3 grid((unsigned)((rows + 7) / 8));
  return launch_dependent(a.D == 128 ? tree_attn_row_kernel<128> : tree_attn_row_kernel<64>, grid, dim3(256), 0,
                          stream, a);
}

}  // namespace sv
