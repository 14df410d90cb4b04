// Rows on their way through the per-head norm and the rotation: a lane's
// eight elements, row sums, and results next to a bf16 rounding boundary formed
// again with twice the bits (the reasons stand in norm_rope.cu).
#pragma once

#include "common.cuh"
#include "fastmath.cuh"

namespace sv {
namespace nr {

// fp32's error is 0.6 of the last bit of a pair's larger member (rms)
constexpr uint32_t kDoubt = 4;

__device__ __forceinline__ uint32_t bf16x2(uint64_t v) {
  float lo, hi;
  fm::unpack2(v, lo, hi);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) { return bf16x2(fm::pack2(lo, hi)); }

// A lane's 8 elements of a row as the first (p) and second (y) members of
// four pairs, two pairs per register pair.  INTER: 8 in a row, pairs (2e, 2e + 1);
// else 4 at off0 and 4 at off1, pairs (e, e + 4).
template <bool INTER>
struct Lane8 {
  uint4 u;
  __device__ __forceinline__ void load(const uint16_t* row, int off0, int off1) {
    if (INTER) {
      u = *reinterpret_cast<const uint4*>(row + off0);
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(row + off0), b = *reinterpret_cast<const uint2*>(row + off1);
      u = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
  __device__ __forceinline__ void store(uint16_t* row, int off0, int off1) const {
    if (INTER) {
      *reinterpret_cast<uint4*>(row + off0) = u;
    } else {
      *reinterpret_cast<uint2*>(row + off0) = make_uint2(u.x, u.y);
      *reinterpret_cast<uint2*>(row + off1) = make_uint2(u.z, u.w);
    }
  }
  __device__ __forceinline__ void unpack(uint64_t* p, uint64_t* y) const {
    if (INTER) {
      p[0] = fm::pack2(bf16_lo(u.x), bf16_lo(u.y));
      y[0] = fm::pack2(bf16_hi(u.x), bf16_hi(u.y));
      p[1] = fm::pack2(bf16_lo(u.z), bf16_lo(u.w));
      y[1] = fm::pack2(bf16_hi(u.z), bf16_hi(u.w));
    } else {
      p[0] = fm::pack2(bf16_lo(u.x), bf16_hi(u.x));
      p[1] = fm::pack2(bf16_lo(u.y), bf16_hi(u.y));
      y[0] = fm::pack2(bf16_lo(u.z), bf16_hi(u.z));
      y[1] = fm::pack2(bf16_lo(u.w), bf16_hi(u.w));
    }
  }
  __device__ __forceinline__ void pack(const uint64_t* p, const uint64_t* y) {
    if (INTER) {
      float a, b, c, d;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        fm::unpack2(p[e], a, b);
        fm::unpack2(y[e], c, d);
        (e ? u.z : u.x) = bf16x2(a, c);
        (e ? u.w : u.y) = bf16x2(b, d);
      }
    } else {
      u = make_uint4(bf16x2(p[0]), bf16x2(p[1]), bf16x2(y[0]), bf16x2(y[1]));
    }
  }
};

// The sum over a row's L lanes, in each of them: 8 and 16 by halves, 9 and 10
// around the row's circle by lanes 1, 2 and 4 further on, and the one or two
// that are left.  (Every lane takes part; those beside the rows add up to
// nothing that is used.)
template <int L>
struct RowLanes {
  static constexpr bool kCircle = (L & (L - 1)) != 0;
  uint32_t to = 0;     // the four lanes, a byte each (a shuffle uses five bits)
  __device__ __forceinline__ void set(int sub, int j, int lane) {
#pragma unroll
    for (int i = 0; i < (kCircle ? 4 : 0); ++i) {
      const int n = j + (1 << i);
      to |= (uint32_t)(sub < 32 / L ? sub * L + (n < L ? n : n - L) : lane) << (8 * i);
    }
  }
};
template <int L>
__device__ __forceinline__ float row_sum(float s, const RowLanes<L>& next) {
  if constexpr (RowLanes<L>::kCircle) {
    const float two = s + __shfl_sync(0xffffffffu, s, next.to);
    const float four = two + __shfl_sync(0xffffffffu, two, next.to >> 8);
    const float eight = four + __shfl_sync(0xffffffffu, four, next.to >> 16);
    return eight + __shfl_sync(0xffffffffu, L == 9 ? s : two, next.to >> 24);
  } else {
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  }
}

// a c + b d, times (ih + il), from about 48 bits of each.
__device__ __forceinline__ float exact_turn(float a, float b, float c, float d, float ih, float il) {
  const float h1 = __fmul_rn(a, c), h2 = __fmul_rn(b, d);
  const float s = __fadd_rn(h1, h2), t = __fadd_rn(s, -h1);
  const float e = __fadd_rn(__fadd_rn(h1, -__fadd_rn(s, -t)), __fadd_rn(h2, -t));    // of the sum
  const float lo = e + (fmaf(a, c, -h1) + fmaf(b, d, -h2));                          // and of the products
  const float r = __fmul_rn(s, ih);
  return __fadd_rn(r, fmaf(s, il, fmaf(lo, ih, fmaf(s, ih, -r))));
}

// (hi, lo) += (x, y), hi + lo holding about 48 bits.
__device__ __forceinline__ void add_exact(float& hi, float& lo, float x, float y) {
  const float s = __fadd_rn(hi, x), t = __fadd_rn(s, -hi);
  lo += __fadd_rn(__fadd_rn(hi, -__fadd_rn(s, -t)), __fadd_rn(x, -t)) + y;
  hi = s;
}

// A lane's 8 results formed again with twice the bits (one group of rows in
// thirty comes here).  The whole warp takes part.
template <int L, bool INTER>
__device__ __forceinline__ uint4 exact_row(uint4 raw, uint4 fast, const uint16_t* weight, int off0, int off1, float eps,
                                        uint64_t c0, uint64_t c1, uint64_t s0, uint64_t s1) {
  float x[8], w[8], c[4], n[4];
  auto split = [&](uint4 u, float* to) {     // first members 0-3, second 4-7
    Lane8<INTER> l;
    l.u = u;
    uint64_t p[2], y[2];
    l.unpack(p, y);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      fm::unpack2(p[e], to[2 * e], to[2 * e + 1]);
      fm::unpack2(y[e], to[4 + 2 * e], to[5 + 2 * e]);
    }
  };
  split(raw, x);
  fm::unpack2(c0, c[0], c[1]);
  fm::unpack2(c1, c[2], c[3]);
  fm::unpack2(s0, n[0], n[1]);
  fm::unpack2(s1, n[2], n[3]);
  float ih = 1.f, il = 0.f;
  if (weight != nullptr) {
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) add_exact(hi, lo, __fmul_rn(x[e], x[e]), 0.f);     // (the squares are exact)
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) {
      const float h = __shfl_xor_sync(0xffffffffu, hi, o), z = __shfl_xor_sync(0xffffffffu, lo, o);
      add_exact(hi, lo, h, z);
    }
    hi *= 1.f / (8 * L);                     // (a power of two)
    lo *= 1.f / (8 * L);
    add_exact(hi, lo, eps, 0.f);
    ih = rsqrtf(hi);
    const float q = __fmul_rn(ih, ih), a = __fmul_rn(hi, q);
    const float rest = __fadd_rn(1.f, -a) - fmaf(hi, q, -a) - fmaf(hi, fmaf(ih, ih, -q), lo * q);
    il = 0.5f * ih * rest;
    Lane8<INTER> g;
    g.load(weight, off0, off1);
    split(g.u, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(x[e], w[e]);                      // (exact)
  }
  float re[4], im[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    re[e] = exact_turn(x[e], x[4 + e], c[e], -n[e], ih, il);
    im[e] = exact_turn(x[e], x[4 + e], n[e], c[e], ih, il);
  }
  // infinities and NaN, and what overflows in between, as the short way has them
  bool fine = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) fine = fine && isfinite(re[e]) && isfinite(im[e]);
  if (!fine) return fast;
  Lane8<INTER> l;
  uint64_t p[2] = {fm::pack2(re[0], re[1]), fm::pack2(re[2], re[3])}, y[2] = {fm::pack2(im[0], im[1]), fm::pack2(im[2], im[3])};
  l.pack(p, y);
  return l.u;
}

}  // namespace nr
}  // namespace sv
