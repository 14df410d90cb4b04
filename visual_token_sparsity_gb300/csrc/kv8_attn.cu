// Sparse decode attention over the 8-bit cache: one query per head, the selected
// visual tokens and the text.
//
//   z_t = scale s_k[page(t)] q . K8[t],  out = sum softmax(z)_t s_v[page(t)] V8[t]
//
// Bound by the cache's bytes; what it takes beside them is turning e4m3 into
// something that multiplies.  e4m3 values are halves, and a query's bf16 elements
// are halves once its largest is brought to 2^14, so both products run on
// m16n8k16 tiles with fp32 accumulation and lose nothing but the weights' bits
// behind the eleventh:
//
//   S [16 tokens x 8 heads] = K (A) Q^T (B),   O [16 dims x 8 heads] += V^T (A) P^T (B)
//
// The order of the 16 elements that a tile sums over is free as long as both
// operands have it, and so are the tile's rows, so every lane loads 16 bytes in
// a row of its token and turns them in registers: as K, bytes (4i, 4i + 1 | 4i + 2,
// 4i + 3) are a tile's two pairs; as V, the bytes of two tokens are interleaved.
// S comes out token-major and goes back in as P^T by way of movmatrix.  Nothing
// passes through shared memory until a CTA's warps are joined.
//
// The weights carry the factor s_v of their page relative to the largest so far
// (and 2^6), the scores a reference that is raised only when one outgrows it by
// 2^8, so that most steps need no maximum.  A weight keeps its eleven bits down to
// 2^-20 of the reference and vanishes below 2^-30.
#include "kernels.h"
#include "kv8.cuh"

namespace sv {

namespace {

constexpr int kWarps = 4;
constexpr int kBlock = 32;               // tokens whose rows a warp looks up at a time
constexpr float kRaise = 8.f;            // log2: a reference is raised when a score outgrows it by more
constexpr int kFusedMerge = 16;          // splits that the last CTA joins itself

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The power of two 2^e, as fp32 bits, with 2^e <= max(|x|, |y|) < 2^(e + 1), within
// 2^-126 and 2^126.
__device__ __forceinline__ uint32_t exponent_of(float x, float y) {
  return min(max(__float_as_uint(fmaxf(fabsf(x), fabsf(y))) & 0x7f800000u, 0x00800000u), 253u << 23);
}

// 16 bytes of a row: D = 128 has two such pieces per lane of K, 64 bytes apart.
template <int D>
struct Rows {
  static constexpr int KC = D / 64;          // pieces of K per token and lane
  static constexpr int VB = D / 8;           // bytes of V per token and lane
  uint4 k[2][KC];                            // tokens r and r + 8
  uint32_t v[4][VB / 4];                     // tokens 2q, 2q + 1, 2q + 8, 2q + 9
};

}  // namespace

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 5 : 4)
kv8_attn_kernel(const __grid_constant__ Kv8AttnArgs a, int nsplit, int chunk) {
  using R = Rows<D>;
  constexpr int KS = D / 16, VW = R::VB / 4;
  extern __shared__ __align__(16) float joined[];        // [warps][G][D], then (m, l)
  __shared__ int s_last;
  grid_dep_sync();
  const int G = a.H / a.Hkv;
  const int unit = blockIdx.x / nsplit, split = blockIdx.x - unit * nsplit;
  const int b = unit / a.Hkv, g = unit - b * a.Hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, q4 = lane & 3;
  int nv, nt, kb;
  attn_lengths(a.lens, a.vis_idx != nullptr, b, a.n_vis, a.n_text, a.k_vis, threadIdx.x == 0 && g == 0 && split == 0,
               a.status, nv, nt, kb);
  const int total = kb + nt, begin = split * chunk, end = min(total, begin + chunk);
  const int32_t* list = a.vis_idx != nullptr ? a.vis_idx + ((size_t)b * a.Hkv + g) * a.k_vis : nullptr;
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;

  // ---- a block's tokens, a lane each, in three steps: position (two blocks
  // ahead), page (one ahead), row and factors
  struct Ahead {
    int pos, page;
    bool there;
  };
  auto load_pos = [&](int t0, Ahead& n) {
    const int t = t0 + lane;
    n.there = t < end;
    n.pos = t < kb ? t : nv + t - kb;
    if (n.there && t < kb && list != nullptr) n.pos = __ldg(list + t);
  };
  auto load_page = [&](int t0, Ahead& n) {
    if (n.there && t0 + lane < kb && (n.pos < 0 || n.pos >= nv)) {
      flag_status(a.status, kStatusBadIndex);
      n.there = false;
    }
    n.page = n.there ? __ldg(bt + (n.pos >> 4)) : -1;
  };
  uint32_t rid, there;
  float2 sc;
  auto load_row = [&](const Ahead& n) {
    const bool ok = n.there && n.page >= 0 && n.page < a.num_blocks;
    if (n.there && !ok) flag_status(a.status, kStatusBadBlock);
    const uint32_t u = ok ? (uint32_t)n.page * (uint32_t)a.Hkv + (uint32_t)g : 0u;
    rid = u * 16u + (uint32_t)(n.pos & 15);
    sc = ok ? __ldg(reinterpret_cast<const float2*>(a.scales) + u) : make_float2(0.f, 0.f);
    there = __ballot_sync(0xffffffffu, ok);
  };
  const int first = begin + warp * kBlock, stride = kWarps * kBlock;
  Ahead n1, n2;
  load_pos(first, n1);
  load_pos(first + stride, n2);

  // ---- the queries: each head's elements over 2^e, so that the largest lies in
  // [2^14, 2^15); those that are not finite stay what they are
  uint32_t qf[NT][KS][2];
  float qs[NT][2];              // of heads 2 q4 and 2 q4 + 1: scale log2(e) 2^e
  {
    float mine[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int h = 8 * t + r;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + ((size_t)b * a.H + (size_t)g * G + h) * D;
      uint2 x[KS];
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        x[k] = h < G ? __ldg(reinterpret_cast<const uint2*>(src + (k >> 2) * 64 + q4 * 16 + (k & 3) * 4)) : make_uint2(0u, 0u);
        top = kv8::max_finite2(kv8::max_finite2(top, x[k].x), x[k].y);
      }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^(14 - e) in two factors, as its exponent may be out of range
      const int e = (int)((top << 16) >> 23) - 127 - 14;              // (a head without a normal element: 2^-127 on)
      const float f0 = __uint_as_float((uint32_t)(127 - e / 2) << 23), f1 = __uint_as_float((uint32_t)(127 - (e - e / 2)) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[t][k][0] = half2_of(bf16_lo(x[k].x) * f0 * f1, bf16_hi(x[k].x) * f0 * f1);
        qf[t][k][1] = half2_of(bf16_lo(x[k].y) * f0 * f1, bf16_hi(x[k].y) * f0 * f1);
      }
      mine[t] = (float)e;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = (int)__shfl_sync(0xffffffffu, mine[t], (2 * q4 + i) * 4);
        qs[t][i] = a.scale_log2 * __uint_as_float((uint32_t)(127 + e / 2) << 23) * __uint_as_float((uint32_t)(127 + e - e / 2) << 23);
      }
  }

  float m[NT][2], l[NT][2], o[NT][KS][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[t][i] = -INFINITY;
      l[t][i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][j][e] = 0.f;
  }
  uint32_t vtop = 0x00800000u;      // the largest factor of V so far, rounded down to a power of two (bits)

  R x;
  auto load_k = [&](uint32_t rows, int h) {      // rows: this step's row ids, 16 h on
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t row = __shfl_sync(0xffffffffu, rows, 16 * h + 8 * i + r);
      const bool ok = (there >> (16 * h + 8 * i + r)) & 1;
#pragma unroll
      for (int c = 0; c < R::KC; ++c)
        x.k[i][c] = ok ? ld_stream16(a.k_pool + (size_t)row * D + c * 64 + q4 * 16) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  auto load_v = [&](uint32_t rows, int h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = 16 * h + 2 * q4 + (i & 1) + (i >> 1) * 8;
      const uint32_t row = __shfl_sync(0xffffffffu, rows, tok);
      const bool ok = (there >> tok) & 1;
      const uint8_t* src = a.v_pool + (size_t)row * D + r * R::VB;
      if constexpr (VW == 4) {
        const uint4 y = ok ? ld_stream16(src) : make_uint4(0u, 0u, 0u, 0u);
        x.v[i][0] = y.x; x.v[i][1] = y.y; x.v[i][2] = y.z; x.v[i][3] = y.w;
      } else {
        const uint2 y = ok ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0u, 0u);
        x.v[i][0] = y.x; x.v[i][1] = y.y;
      }
    }
  };

  load_page(first, n1);
  for (int t0 = first; t0 < end; t0 += stride) {
    load_row(n1);
    n1 = n2;
    load_page(t0 + stride, n1);
    load_pos(t0 + 2 * stride, n2);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && t0 + 16 >= end) break;
      load_k(rid, h);
      load_v(rid, h);
      const float sk0 = __shfl_sync(0xffffffffu, sc.x, 16 * h + r), sk1 = __shfl_sync(0xffffffffu, sc.x, 16 * h + 8 + r);
      const float sv0 = __shfl_sync(0xffffffffu, sc.y, 16 * h + r), sv1 = __shfl_sync(0xffffffffu, sc.y, 16 * h + 8 + r);
      const bool ok0 = (there >> (16 * h + r)) & 1, ok1 = (there >> (16 * h + 8 + r)) & 1;
      float z[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) z[t][e] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&x.k[0][k >> 2]);
        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&x.k[1][k >> 2]);
        const uint32_t y0 = w0[k & 3], y1 = w1[k & 3];
        const uint32_t a0 = kv8::e4m3x2_to_half2((uint16_t)y0), a1 = kv8::e4m3x2_to_half2((uint16_t)y1);
        const uint32_t a2 = kv8::e4m3x2_to_half2((uint16_t)(y0 >> 16)), a3 = kv8::e4m3x2_to_half2((uint16_t)(y1 >> 16));
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_f16(z[t], a0, a1, a2, a3, qf[t][k][0], qf[t][k][1]);
      }
      bool raise = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[t][e] = (e < 2 ? ok0 : ok1) ? z[t][e] * (e < 2 ? sk0 : sk1) * qs[t][e & 1] : -INFINITY;
          raise = raise || z[t][e] > m[t][e & 1] + kRaise || (m[t][e & 1] == -INFINITY && z[t][e] > -INFINITY);
        }
      raise = raise || exponent_of(sv0, sv1) > vtop;
      if (__any_sync(0xffffffffu, raise)) {
        // the factors' largest, and each head's
        const uint32_t top = __reduce_max_sync(0xffffffffu, max(vtop, exponent_of(sv0, sv1)));
        const float down = __uint_as_float(vtop) / __uint_as_float(top);
        vtop = top;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mx = fmaxf(m[t][i], fmaxf(z[t][i], z[t][i + 2]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float alpha = m[t][i] == -INFINITY ? 0.f : fast_exp2(m[t][i] - mx);
            m[t][i] = mx;
            l[t][i] *= alpha;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              o[t][j][i] *= alpha * down;
              o[t][j][i + 2] *= alpha * down;
            }
          }
      }
      // 2^6 s_v over the largest factor
      const float unit_v = __uint_as_float((254u - (vtop >> 23)) << 23);
      const float w0 = sv0 * unit_v * 64.f, w1 = sv1 * unit_v * 64.f;
      uint32_t p[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = m[t][e & 1];
          y[e] = fast_exp2(z[t][e] - (ref == -INFINITY ? 0.f : ref));
          l[t][e & 1] += y[e];
        }
        p[t][0] = transposed(half2_of(y[0] * w0, y[1] * w0));
        p[t][1] = transposed(half2_of(y[2] * w1, y[3] * w1));
      }
#pragma unroll
      for (int w = 0; w < VW; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t sel = i ? 0x7362u : 0x5140u;       // (token, next token) x two bytes
          const uint32_t lo = __byte_perm(x.v[0][w], x.v[1][w], sel), hi = __byte_perm(x.v[2][w], x.v[3][w], sel);
          const uint32_t a0 = kv8::e4m3x2_to_half2((uint16_t)lo), a1 = kv8::e4m3x2_to_half2((uint16_t)(lo >> 16));
          const uint32_t a2 = kv8::e4m3x2_to_half2((uint16_t)hi), a3 = kv8::e4m3x2_to_half2((uint16_t)(hi >> 16));
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_f16(o[t][2 * w + i], a0, a1, a2, a3, p[t][0], p[t][1]);
        }
    }
  }

  // ---- the CTA's warps joined
  const float back = __uint_as_float(vtop) * (1.f / 64.f);
  float* ml = joined + kWarps * G * D;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = 8 * t + 2 * q4 + i;
      float s = l[t][i];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      if (h < G) {
        if (r == 0) {
          ml[(warp * G + h) * 2] = m[t][i];
          ml[(warp * G + h) * 2 + 1] = s;
        }
        float* dst = joined + (warp * G + h) * D + r * R::VB;
#pragma unroll
        for (int j = 0; j < KS; ++j)
          *reinterpret_cast<float2*>(dst + 2 * j) = make_float2(o[t][j][i] * back, o[t][j][i + 2] * back);
      }
    }
  __syncthreads();
  const size_t part = ((size_t)unit * nsplit + split) * G;
  float* part_ml = reinterpret_cast<float*>(a.part_ml);
  for (int i = threadIdx.x; i < G * D; i += kWarps * 32) {
    const int h = i / D, e = i - h * D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[(w * G + h) * 2]);
    float L = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = ml[(w * G + h) * 2], f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
      // (a NaN of the sum stays even where the maximum knows nothing of it)
      L += mw == -INFINITY ? ml[(w * G + h) * 2 + 1] * 0.f : f * ml[(w * G + h) * 2 + 1];
      acc += f * joined[(w * G + h) * D + e];
    }
    if (nsplit == 1) {
      const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
      const size_t row = (size_t)b * a.H + (size_t)g * G + h;
      static_cast<uint16_t*>(a.out)[row * D + e] = (uint16_t)f32_to_bf16_bits(acc * inv);
      if (e == 0 && a.lse != nullptr) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    } else {
      a.part_o[part * D + i] = acc;
      if (e == 0) {
        part_ml[(part + h) * 2] = M;
        part_ml[(part + h) * 2 + 1] = L;
      }
    }
  }
  if (nsplit == 1 || a.split_done == nullptr) return;

  // ---- the last CTA of a (sequence, KV head) joins its splits
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(a.split_done + unit, 1) == nsplit - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  if (threadIdx.x == 0) a.split_done[unit] = 0;           // ready for the next call
  const size_t base = (size_t)unit * nsplit * G;
  for (int i = threadIdx.x; i < G * D; i += kWarps * 32) {
    const int h = i / D, e = i - h * D;
    float M = -INFINITY;
    for (int s = 0; s < nsplit; ++s) M = fmaxf(M, __ldcg(part_ml + (base + s * G + h) * 2));
    float L = 0.f, acc = 0.f;
#pragma unroll 4
    for (int s = 0; s < nsplit; ++s) {
      const float2 x2 = __ldcg(reinterpret_cast<const float2*>(part_ml) + base + s * G + h);
      const float v = __ldcg(a.part_o + (base + s * G) * D + i);
      const float f = x2.x == -INFINITY ? 0.f : fast_exp2(x2.x - M);
      L += x2.x == -INFINITY ? x2.y * 0.f : f * x2.y;
      acc += f * v;
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    const size_t row = (size_t)b * a.H + (size_t)g * G + h;
    static_cast<uint16_t*>(a.out)[row * D + e] = (uint16_t)f32_to_bf16_bits(acc * inv);
    if (e == 0 && a.lse != nullptr) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

namespace {

// Splits of a (sequence, KV head): as many CTAs as are resident at once (152 SMs
// times 5, or 4 with more than 8 heads), so that what varies is how full the
// last round is; each split costs about three steps beside its tokens.
constexpr int kSms = 152;
constexpr int kMaxSplits = 128;
int resident(int G) { return kSms * (G <= 8 ? 5 : 4); }
struct Plan {
  int nsplit, chunk;
};
Plan plan_of(long long units, int G, int n_tokens) {
  const int block = kWarps * kBlock;
  const int blocks = n_tokens > 0 ? (n_tokens + block - 1) / block : 1;
  const long long cap = resident(G);
  Plan best = {1, blocks * block};
  long long best_cost = -1;
  for (int s = 1; s <= blocks && s <= kMaxSplits; ++s) {
    if (s > 1 && (units * s > 2 * cap || units > kWorkspaceCounters)) break;
    const int per = (blocks + s - 1) / s;
    const long long ctas = units * ((blocks + per - 1) / per), rounds = (ctas + cap - 1) / cap;
    const long long cost = rounds * (per * 2 + 3);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = {(blocks + per - 1) / per, per * block};
    }
  }
  return best;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// (m, l) | O of every split: a bound that no smaller call exceeds
size_t kv8_attn_workspace_bytes(int B, int H, int Hkv, int D, int n_tokens) {
  const int G = H / Hkv;
  const long long units = (long long)B * Hkv, most = 2ll * resident(G);
  long long splits = (n_tokens + kWarps * kBlock - 1) / (kWarps * kBlock);
  splits = splits < kMaxSplits ? splits : kMaxSplits;
  long long parts = units * splits;
  parts = parts < most ? parts : most;
  return up256((size_t)parts * G * 2 * sizeof(float)) + up256((size_t)parts * G * D * sizeof(float));
}

template <int D, int NT>
static cudaError_t launch_nt(const Kv8AttnArgs& a, const Plan& p, cudaStream_t stream) {
  const int G = a.H / a.Hkv;
  const size_t smem = (size_t)kWarps * G * (D + 2) * sizeof(float);
  return launch_dependent(kv8_attn_kernel<D, NT>, dim3((unsigned)((long long)a.batch * a.Hkv * p.nsplit)),
                          dim3(kWarps * 32), smem, stream, a, p.nsplit, p.chunk);
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs& args, int D, cudaStream_t stream) {
  Kv8AttnArgs a = args;
  const int G = a.H / a.Hkv;
  const Plan p = plan_of((long long)a.batch * a.Hkv, G, a.k_vis + a.n_text);
  a.part_ml = static_cast<float*>(a.ws);
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(a.ws) +
                                      up256((size_t)a.batch * a.Hkv * p.nsplit * G * 2 * sizeof(float)));
  a.split_done = p.nsplit <= kFusedMerge ? a.counters : nullptr;
  cudaError_t e;
  if (D == 128) e = G <= 8 ? launch_nt<128, 1>(a, p, stream) : launch_nt<128, 2>(a, p, stream);
  else e = G <= 8 ? launch_nt<64, 1>(a, p, stream) : launch_nt<64, 2>(a, p, stream);
  if (e != cudaSuccess || p.nsplit <= kFusedMerge) return e;
  return launch_attn_merge(a.part_ml, a.part_o, a.batch, a.H, a.Hkv, D, p.nsplit, a.out, a.lse, stream);
}

}  // namespace sv
