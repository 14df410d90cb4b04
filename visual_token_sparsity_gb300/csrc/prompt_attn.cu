// Causal attention of whole prompts: packed sequences, grouped heads, read from
// the token-major projections (slices of a fused one, for instance).
//
//   out_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j,  i and j in one sequence
#include "kernels.h"
#include "common.cuh"

namespace sv {

namespace {

constexpr int kWarps = 4;

// One query row by one warp: a lane per key for the products with K, then the
// lanes over the dims of V.  (m, l) base two.
template <int D>
__device__ __forceinline__ void attend_row(const float* qs, const uint16_t* k, long long k_stride, const uint16_t* v,
                                           long long v_stride, int n, float sl2, int lane, float& m, float& l,
                                           float (&o)[D / 32]) {
  constexpr int E = D / 32;
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane, cnt = min(32, n - j0);
    float z = -INFINITY;
    if (j < n) {
      float dot = 0.f;
      const uint4* src = reinterpret_cast<const uint4*>(k + (size_t)j * k_stride);
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = __ldg(src + c);
        const float4 a = *reinterpret_cast<const float4*>(qs + 8 * c), b = *reinterpret_cast<const float4*>(qs + 8 * c + 4);
        dot = fmaf(a.x, bf16_lo(x.x), fmaf(a.y, bf16_hi(x.x), fmaf(a.z, bf16_lo(x.y), fmaf(a.w, bf16_hi(x.y), dot))));
        dot = fmaf(b.x, bf16_lo(x.z), fmaf(b.y, bf16_hi(x.z), fmaf(b.z, bf16_lo(x.w), fmaf(b.w, bf16_hi(x.w), dot))));
      }
      z = dot * sl2;
    }
    const float mx = fmaxf(m, warp_max(z)), off = mx == -INFINITY ? 0.f : mx;
    const float alpha = m == -INFINITY ? 0.f : fast_exp2(m - off), p = j < n ? fast_exp2(z - off) : 0.f;
    m = mx;
    l = l * alpha + warp_sum(p);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= alpha;
    for (int i = 0; i < cnt; ++i) {
      const float w = __shfl_sync(0xffffffffu, p, i);
      const uint16_t* src = v + (size_t)(j0 + i) * v_stride + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(src + e));
        o[e] = fmaf(w, bf16_lo(x), o[e]);
        o[e + 1] = fmaf(w, bf16_hi(x), o[e + 1]);
      }
    }
  }
}

}  // namespace

// A warp per (token, query head).
template <int D>
__global__ void __launch_bounds__(kWarps * 32)
prompt_attn_kernel(const __grid_constant__ PromptArgs a) {
  constexpr int E = D / 32;
  __shared__ __align__(16) float qs[kWarps][D];
  grid_dep_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the starts have to ascend within the tokens; otherwise nothing is computed
  bool bad = false;
  for (int b = threadIdx.x; b <= a.batch; b += kWarps * 32) {
    const int s = __ldg(a.seq_start + b);
    bad = bad || s < 0 || s > a.N || (b > 0 && __ldg(a.seq_start + b - 1) > s);
  }
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_status(a.status, kStatusBadLength);
    return;
  }
  const long long w = (long long)blockIdx.x * kWarps + warp;
  const int t = (int)(w / a.H), h = (int)(w - (long long)t * a.H), g = h / (a.H / a.Hkv);
  if (t >= a.N || t < __ldg(a.seq_start) || t >= __ldg(a.seq_start + a.batch)) return;
  int lo = 0, hi = a.batch;                    // the last sequence that begins at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(a.seq_start + mid) <= t) lo = mid;
    else hi = mid;
  }
  const int begin = __ldg(a.seq_start + lo);
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + (size_t)t * a.q_stride + (size_t)h * D;
  for (int e = lane; e < D; e += 32) qs[warp][e] = __uint_as_float((uint32_t)q[e] << 16);
  __syncwarp();
  float m, l, o[E];
  attend_row<D>(qs[warp], static_cast<const uint16_t*>(a.k) + (size_t)begin * a.k_stride + (size_t)g * D, a.k_stride,
                static_cast<const uint16_t*>(a.v) + (size_t)begin * a.v_stride + (size_t)g * D, a.v_stride,
                t - begin + 1, a.scale_log2, lane, m, l, o);
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  const size_t row = (size_t)t * a.H + h;
#pragma unroll
  for (int e = 0; e < E; ++e) static_cast<uint16_t*>(a.out)[row * D + lane * E + e] = (uint16_t)f32_to_bf16_bits(o[e] * inv);
  if (lane == 0 && a.lse != nullptr) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

cudaError_t launch_prompt_attn(const PromptArgs& a, int D, cudaStream_t stream) {
  const long long blocks = ((long long)a.N * a.H + kWarps - 1) / kWarps;
  return launch_dependent(D == 128 ? prompt_attn_kernel<128> : prompt_attn_kernel<64>, dim3((unsigned)blocks),
                          dim3(kWarps * 32), 0, stream, a);
}

}  // namespace sv
