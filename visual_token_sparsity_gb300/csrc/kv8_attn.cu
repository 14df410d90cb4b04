// Sparse decode attention over the 8-bit cache: one query per head, the selected
// visual tokens and the text.
//
//   z_t = scale s_k[page(t)] q . K8[t],  out = sum softmax(z)_t s_v[page(t)] V8[t]
#include "kernels.h"
#include "kv8.cuh"

namespace sv {

namespace {
constexpr int kWarps = 8;
}

// A CTA per (sequence, query head); each warp takes every eighth 32 tokens.
template <int D>
__global__ void __launch_bounds__(kWarps * 32)
kv8_attn_kernel(const __grid_constant__ Kv8AttnArgs a) {
  constexpr int E = D / 32;                 // output dims of a lane
  __shared__ __align__(16) float qs[D];
  __shared__ float ml[kWarps][2];
  __shared__ float os[kWarps][D];
  grid_dep_sync();
  const int b = blockIdx.x / a.H, h = blockIdx.x - b * a.H, G = a.H / a.Hkv, g = h / G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int nv, nt, kb;
  attn_lengths(a.lens, a.vis_idx != nullptr, b, a.n_vis, a.n_text, a.k_vis, threadIdx.x == 0 && h == 0, a.status, nv,
               nt, kb);
  for (int e = threadIdx.x; e < D; e += kWarps * 32)
    qs[e] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.q)[((size_t)b * a.H + h) * D + e] << 16);
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int t0 = warp * 32; t0 < kb + nt; t0 += kWarps * 32) {
    const int t = t0 + lane;
    bool ok = t < kb + nt;
    int pos = 0;
    if (ok) {
      pos = t < kb ? t : nv + t - kb;
      if (t < kb && a.vis_idx != nullptr) {
        pos = __ldg(a.vis_idx + ((size_t)b * a.Hkv + g) * a.k_vis + t);
        if (pos < 0 || pos >= nv) {
          flag_status(a.status, kStatusBadIndex);
          ok = false;
        }
      }
    }
    size_t unit = 0;
    if (ok) {
      const int page = __ldg(a.block_table + (size_t)b * a.max_blocks + (pos >> 4));
      if (page < 0 || page >= a.num_blocks) {
        flag_status(a.status, kStatusBadBlock);
        ok = false;
      } else {
        unit = (size_t)page * a.Hkv + g;
      }
    }
    float z = -INFINITY, sv = 0.f;
    const size_t row = unit * 16 + (pos & 15);
    if (ok) {
      const float2 s = *reinterpret_cast<const float2*>(a.scales + unit * 2);
      sv = s.y;
      float dot = 0.f;
      const uint4* src = reinterpret_cast<const uint4*>(a.k_pool + row * D);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const uint4 v = __ldg(src + c);
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 lo = kv8::e4m3x2_to_float2((uint16_t)w[e]), hi = kv8::e4m3x2_to_float2((uint16_t)(w[e] >> 16));
          const float4 qq = *reinterpret_cast<const float4*>(qs + 16 * c + 4 * e);
          dot = fmaf(qq.x, lo.x, fmaf(qq.y, lo.y, fmaf(qq.z, hi.x, fmaf(qq.w, hi.y, dot))));
        }
      }
      z = dot * s.x * a.scale_log2;
    }
    const float top = warp_max(z);
    if (!__any_sync(0xffffffffu, ok)) continue;
    const float mx = fmaxf(m, top);
    const float off = mx == -INFINITY ? 0.f : mx, alpha = m == -INFINITY ? 0.f : fast_exp2(m - off);
    const float p = ok ? fast_exp2(z - off) : 0.f;
    m = mx;
    l = l * alpha + warp_sum(p);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= alpha;
    uint32_t there = __ballot_sync(0xffffffffu, ok);
    while (there) {
      const int i = __ffs(there) - 1;
      there &= there - 1;
      const float w = __shfl_sync(0xffffffffu, p, i) * __shfl_sync(0xffffffffu, sv, i);
      const size_t r = __shfl_sync(0xffffffffu, (unsigned long long)row, i);
      const uint8_t* v = a.v_pool + r * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 x = kv8::e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(v + e));
        o[e] = fmaf(w, x.x, o[e]);
        o[e + 1] = fmaf(w, x.y, o[e + 1]);
      }
    }
  }
  if (lane == 0) {
    ml[warp][0] = m;
    ml[warp][1] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) os[warp][lane * E + e] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w][0]);
  float f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = ml[w][0] == -INFINITY ? 0.f : fast_exp2(ml[w][0] - M);
    L += f[w] * ml[w][1];
  }
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
  for (int e = threadIdx.x; e < D; e += kWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += f[w] * os[w][e];
    static_cast<uint16_t*>(a.out)[(size_t)blockIdx.x * D + e] = (uint16_t)f32_to_bf16_bits(x * inv);
  }
  if (threadIdx.x == 0 && a.lse != nullptr)
    a.lse[blockIdx.x] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

size_t kv8_attn_workspace_bytes(int B, int H, int Hkv, int D, int n_tokens) {
  (void)B; (void)H; (void)Hkv; (void)D; (void)n_tokens;
  return 0;
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, int D, cudaStream_t stream) {
  return launch_dependent(D == 128 ? kv8_attn_kernel<128> : kv8_attn_kernel<64>, dim3((unsigned)a.batch * a.H),
                          dim3(kWarps * 32), 0, stream, a);
}

}  // namespace sv
