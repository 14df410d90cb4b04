// Per-head RMS norm and position rotation of queries and keys in one pass,
// into the salience operands (head-major) or straight into the paged cache.
//
//   x' = x * rsqrt(mean(x^2) + eps) * w          (each head of each token)
//   (a, c) -> (a cos - c sin, a sin + c cos)     (each of its rot / 2 pairs)
//
// Pair p turns by cos_sin[pos[axis(p)]][p]: one position per token, or up to
// three (time, row, column) that own consecutive sections of the pairs.
// Everything is fp32 between the bf16 load and the one rounding at the end.
//
// Bound by memory: every row is read once and written once, a dozen
// operations per element.  A row is d / 8 lanes of 8 elements, 32 / (d / 8)
// rows side by side in a warp; a lane's elements are the two halves of four
// pairs (rotate-half: 4 at 4j and 4 at rot/2 + 4j; interleaved or not
// rotated: 8 in a row), so no pair crosses lanes and the four (cos, sin) it
// needs are loaded once per token and reused for the warp's rows.
#include "common.cuh"
#include "kernels.h"

namespace sv {

namespace {

constexpr int kWarps = 8;
constexpr int kUnroll = 4;     // row groups in flight per warp

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void unpack4(uint2 u, float* x) {
  x[0] = bf16_lo(u.x);
  x[1] = bf16_hi(u.x);
  x[2] = bf16_lo(u.y);
  x[3] = bf16_hi(u.y);
}

}  // namespace

// One warp: kUnroll * (32 / L) consecutive rows of one token, where a token's
// rows are its H queries, Hk keys and (append) Hk values.
template <int L, bool APPEND>
__global__ void __launch_bounds__(kWarps * 32)
norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int D = 8 * L;
  constexpr int RPG = 32 / L;                 // rows side by side
  constexpr int RPW = RPG * kUnroll;
  grid_dep_sync();
  const int lane = threadIdx.x & 31;
  const int sub = lane / L, j = lane - sub * L;
  const int rows = a.H + (APPEND ? 2 : 1) * a.Hk;
  const int wpt = (rows + RPW - 1) / RPW;     // warps per token
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long tok = w / wpt;
  if (tok >= (long long)a.B * a.T) return;
  const int r0 = (int)(w - tok * wpt) * RPW;
  const int b = (int)(tok / a.T), t = (int)(tok - (long long)b * a.T);

  // where the token goes in the cache, and whether it is there at all
  int page = 0, slot = 0;
  if (APPEND) {
    SeqLens l = a.lens;
    l.k = nullptr;
    int nv, nt, kb;
    const bool ok = seq_lengths(l, b, a.n_vis, a.n_text, 0, nv, nt, kb);
    const int tn = a.n_new ? __ldg(a.n_new + b) : a.T;
    if (!ok || tn < 0 || tn > a.T) {
      if (r0 == 0 && t == 0 && lane == 0) flag_status(a.status, kStatusBadLength);
      return;
    }
    if (t >= tn) return;
    const int pos = nv + nt + t;
    page = __ldg(a.block_table + (size_t)b * a.max_blocks + (pos >> 4));
    slot = pos & 15;
    if (page < 0 || page >= a.num_blocks) {
      if (r0 == 0 && lane == 0) flag_status(a.status, kStatusBadBlock);
      page = -1;                              // the queries are still written
    }
  }

  // this lane's elements off0.. and off1.. and the four turns between them
  const int half = a.rot >> 1;
  const bool turned = 4 * j < half;
  const bool split = turned && !a.interleaved;
  const int off0 = split ? 4 * j : 8 * j;
  const int off1 = split ? half + 4 * j : 8 * j + 4;
  float cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) { cs[i] = 1.f; sn[i] = 0.f; }
  if (half > 0) {
    int p[3] = {0, 0, 0};
    bool bad = false;
#pragma unroll
    for (int x = 0; x < 3; ++x)
      if (x < a.n_axes && a.sec_end[x] > (x ? a.sec_end[x - 1] : 0)) {
        p[x] = __ldg(a.pos + ((size_t)x * a.B + b) * a.T + t);
        bad |= p[x] < 0 || p[x] >= a.n_pos;
      }
    if (bad) {
      if (r0 == 0 && lane == 0) flag_status(a.status, kStatusBadPosition);
      return;
    }
    if (turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int pr = 4 * j + i;
        const int px = pr < a.sec_end[0] ? p[0] : pr < a.sec_end[1] ? p[1] : p[2];
        const float2 v = __ldg(reinterpret_cast<const float2*>(a.cos_sin) + (size_t)px * half + pr);
        cs[i] = v.x;
        sn[i] = v.y;
      }
    }
  }

  uint2 u0[kUnroll], u1[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int r = r0 + i * RPG + sub;
    u0[i] = u1[i] = make_uint2(0u, 0u);
    if (sub < RPG && r < rows) {
      const uint16_t* src = r < a.H          ? a.q + tok * a.q_stride + (size_t)r * D
                            : r < a.H + a.Hk ? a.k + tok * a.k_stride + (size_t)(r - a.H) * D
                                             : a.v + tok * a.v_stride + (size_t)(r - a.H - a.Hk) * D;
      u0[i] = *reinterpret_cast<const uint2*>(src + off0);
      u1[i] = *reinterpret_cast<const uint2*>(src + off1);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int r = r0 + i * RPG + sub;
    const bool live = sub < RPG && r < rows;
    const bool is_q = r < a.H, is_v = r >= a.H + a.Hk;
    float x[8];
    unpack4(u0[i], x);
    unpack4(u1[i], x + 4);
    const uint16_t* wgt = is_q ? a.q_weight : a.k_weight;
    // the reduction is warp-wide: every lane takes part
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) {
      if (o >= L) continue;
      const float y = __shfl_down_sync(0xffffffffu, s, o);
      if (j + o < L) s += y;
    }
    s = __shfl_sync(0xffffffffu, s, sub < RPG ? sub * L : lane);
    if (!live) continue;
    if (!is_v) {
      if (wgt != nullptr) {
        const float inv = rsqrtf(s * (1.f / D) + a.eps);
        float g[8];
        unpack4(__ldg(reinterpret_cast<const uint2*>(wgt + off0)), g);
        unpack4(__ldg(reinterpret_cast<const uint2*>(wgt + off1)), g + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * g[e];
      }
      if (turned) {
        // rotate-half: pairs (e, e + 4); interleaved: pairs (2e, 2e + 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (split) {
            const float p = x[e], q = x[e + 4];
            x[e] = p * cs[e] - q * sn[e];
            x[e + 4] = p * sn[e] + q * cs[e];
          } else {
            const float p = x[2 * e], q = x[2 * e + 1];
            x[2 * e] = p * cs[e] - q * sn[e];
            x[2 * e + 1] = p * sn[e] + q * cs[e];
          }
        }
      }
      u0[i] = make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
      u1[i] = make_uint2(bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
    }
    uint16_t* dst;
    if (APPEND) {
      if (is_q) {
        dst = a.q_out + ((size_t)tok * a.H + r) * D;
      } else {
        if (page < 0) continue;
        const int g = is_v ? r - a.H - a.Hk : r - a.H;
        dst = (is_v ? a.v_out : a.k_out) + ((((size_t)page * a.Hk + g) << 4) + slot) * D;
      }
    } else {
      dst = is_q ? a.q_out + (((size_t)b * a.H + r) * a.T + t) * D
                 : a.k_out + (((size_t)b * a.Hk + (r - a.H)) * a.T + t) * D;
    }
    *reinterpret_cast<uint2*>(dst + off0) = u0[i];
    *reinterpret_cast<uint2*>(dst + off1) = u1[i];
  }
}

template <int L>
static cudaError_t launch_l(const NormRopeArgs& a, bool append, cudaStream_t stream) {
  const int rpw = 32 / L * kUnroll;
  const int rows = a.H + (append ? 2 : 1) * a.Hk;
  const long long warps = (long long)a.B * a.T * ((rows + rpw - 1) / rpw);
  const long long blocks = (warps + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_dependent(append ? norm_rope_kernel<L, true> : norm_rope_kernel<L, false>, dim3((unsigned)blocks),
                          dim3(kWarps * 32), 0, stream, a);
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, int d, bool append, cudaStream_t stream) {
  if ((long long)a.B * a.T == 0) return cudaSuccess;
  switch (d) {
    case 64: return launch_l<8>(a, append, stream);
    case 72: return launch_l<9>(a, append, stream);
    case 80: return launch_l<10>(a, append, stream);
    case 128: return launch_l<16>(a, append, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sv
