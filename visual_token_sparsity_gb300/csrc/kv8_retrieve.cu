// Query-aware retrieval from the 8-bit cache: scores of the cached visual keys
// and the selection of the k largest.
//
//   qbar = sum of the query rows and the group's heads
//   score_j = s_k[page(j)] * qbar . K8[j]            (as retrieve.cu)
//
// Scoring is bound by the keys' bytes.  e4m3 values are halves, and qbar is the
// sum of three halves (33 bits of its largest element), so a page of 16 keys
// meets them on m16n8k16 tiles with fp32 accumulation, three of the eight columns
// in use: the tensor core takes conversion's place as the unit that multiplies,
// and the products cost what they cost in one column.  Every lane loads 16 bytes
// in a row of its key; the order of a tile's elements is free.
//
// The selection is that of the exact scores.  The fp32 scores order all but the
// tokens next to the k-th one: with an error of at most e each, the k-th largest
// score is within e of the true one, so a token more than 2 e above it is in
// and one more than 2 e below it is out.  Those in between are scored again with
// 48 bits and the best of them taken, ties to the lower index.
#include "kernels.h"
#include "kv8.cuh"
#include "topk_cluster.cuh"

namespace cg = cooperative_groups;

namespace sv {

namespace {

constexpr int kScoreWarps = 8;
// |fp32 score - score| <= e = 2^-24 (272 |qbar|_max + 12 |qbar|_1) 448 s, as 448 s
// bounds a key's elements: a tile's 16 products lose at most the last of 24 bits
// beside the largest, and their sum, at most 16 of the largest, as much again (eight
// tiles, and their parts' columns); seven sums of tiles, two of columns and three
// products with factors round to 2^-24 of what is below |qbar|_1 448 s.  Two tokens
// are told apart by 2 e; twice that is taken:
constexpr float kBand = 448.f / 4194304.f;
constexpr float kBandMax = 272.f, kBandSum = 12.f;
constexpr int kListed = 1024;            // tokens next to the border that are ranked in shared memory
constexpr int kStagedKeys = 16384;       // keys of a row whose selection one CTA makes in shared memory

// hi + lo = a + b.
__device__ __forceinline__ void two_sum(float a, float b, float& hi, float& lo) {
  hi = __fadd_rn(a, b);
  const float t = __fadd_rn(hi, -a);
  lo = __fadd_rn(__fadd_rn(a, -__fadd_rn(hi, -t)), __fadd_rn(b, -t));
}
// (hi, lo) += (x, y), about 48 bits.
__device__ __forceinline__ void add48(float& hi, float& lo, float x, float y) {
  float s, e;
  two_sum(hi, x, s, e);
  e = __fadd_rn(e, __fadd_rn(lo, y));
  hi = __fadd_rn(s, e);
  lo = __fadd_rn(e, -__fadd_rn(hi, -s));
}

// An integer that orders like hi + lo, hi being the nearest float to it: hi
// decides, then lo.  (Comparing doubles would take a unit that has two lanes.)
__device__ __forceinline__ uint64_t order_key64(float hi, float lo) {
  return (uint64_t)order_key(hi) << 32 | order_key(lo);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One (sequence, KV head) row's query.
template <int D>
struct Query8 {
  float2 qbar[D];        // hi + lo
  uint16_t part[4][D];   // halves: qbar over 2^e in three parts, and 0
  float back[2];         // 2^e in two factors
  float slack;           // 272 |qbar|_max + 12 |qbar|_1
  uint32_t pad[13];
};

}  // namespace

namespace {

constexpr int kFusedRows = 16;       // query rows times heads that every scoring CTA sums itself

// The row's query from R x G rows, by threads 0 .. D - 1 of a block of at least D
// (all threads call this); the caller synchronises before it reads *o.
template <int D>
__device__ __forceinline__ void sum_query(const uint16_t* q, int R, int H, int Hkv, int row, Query8<D>* o) {
  __shared__ float part[2][D / 32];
  const int b = row / Hkv, g = row - b * Hkv, G = H / Hkv, e = threadIdx.x;
  float hi = 0.f, lo = 0.f;
  if (e < D) {
    const uint16_t* src = q + ((size_t)b * R * H + (size_t)g * G) * D + e;
    const int n = R * G;
    for (int i0 = 0; i0 < n; i0 += 8) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j, r = i / G;
        x[j] = i < n ? __uint_as_float((uint32_t)__ldg(src + ((size_t)r * H + (i - r * G)) * D) << 16) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) add48(hi, lo, x[j], 0.f);
    }
    const float a = fabsf(hi), s = warp_sum(a), top = warp_max(a);
    if ((e & 31) == 0) {
      part[0][e >> 5] = s;
      part[1][e >> 5] = top;
    }
  }
  __syncthreads();
  if (e >= D) return;
  float s = 0.f, top = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    s += part[0][i];
    top = fmaxf(top, part[1][i]);
  }
  // the largest element comes to lie in [2^14, 2^15), by two factors as 2^(14 - e) may
  // be out of range
  const int x = (int)(__float_as_uint(top) >> 23) - 127 - 14;
  const float f0 = __uint_as_float((uint32_t)(127 - x / 2) << 23), f1 = __uint_as_float((uint32_t)(127 - (x - x / 2)) << 23);
  float h = hi * f0 * f1, l = lo * f0 * f1;
  o->qbar[e] = make_float2(hi, lo);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const __half p = __float2half_rn(h);
    o->part[i][e] = __half_as_ushort(p);
    const float rest = __fadd_rn(h, -__half2float(p));          // (exact)
    h = __fadd_rn(rest, l);
    l = __fadd_rn(l, -__fadd_rn(h, -rest));
  }
  o->part[3][e] = 0;
  if (e == 0) {
    o->back[0] = __uint_as_float((uint32_t)(127 + x / 2) << 23);
    o->back[1] = __uint_as_float((uint32_t)(127 + x - x / 2) << 23);
    o->slack = kBandMax * top + kBandSum * s;
  }
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(D)
kv8_qbar_kernel(const uint16_t* __restrict__ q, int R, int H, int Hkv, Query8<D>* rows) {
  grid_dep_sync();
  sum_query<D>(q, R, H, Hkv, blockIdx.x, rows + blockIdx.x);
}

// A warp per page, one page in flight, as many warps as 48 registers allow.  SUM:
// the query's rows are few, and every CTA adds them up itself (the first of a row
// leaves the sum for the selection).
template <int D, bool SUM>
__global__ void __launch_bounds__(kScoreWarps * 32, 5)
kv8_score_kernel(const __grid_constant__ Kv8RetrieveArgs a, Query8<D>* rows, float* __restrict__ scores,
                 float* __restrict__ factors, int pages_per_cta) {
  constexpr int KS = D / 16, KC = D / 64, W = kScoreWarps;
  __shared__ __align__(16) Query8<D> query;
  grid_dep_sync();
  const int g = blockIdx.y, b = blockIdx.z, row = b * a.Hkv + g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, q4 = lane & 3;
  int nv, nt, kb;
  if (!seq_lengths(a.lens, b, a.n_vis, a.n_text, a.k, nv, nt, kb) && threadIdx.x == 0 && blockIdx.x == 0)
    flag_status(a.status, kStatusBadLength);
  const int end = min((nv + 15) / 16, ((int)blockIdx.x + 1) * pages_per_cta);
  const int first = blockIdx.x * pages_per_cta + warp;
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;

  uint4 k[2][KC];            // keys r and r + 8
  float factor = 0.f;
  bool ok = false;
  // (the page's id was asked for a page of this warp before)
  auto id_of = [&](int p) { return p < end ? __ldg(bt + p) : -1; };
  auto load = [&](int p, int page) {
    ok = page >= 0 && page < a.num_blocks;
    if (!ok) {
      if (p < end && lane == 0) flag_status(a.status, kStatusBadBlock);
      return;
    }
    const size_t unit = (size_t)page * a.Hkv + g;
    const uint8_t* src = a.k_pool + (unit * 16 + r) * D + q4 * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < KC; ++c) k[i][c] = ld_stream16(src + i * 8 * D + c * 64);
    factor = __ldg(a.scales + unit * 2);
  };
  int next = id_of(first);
  load(first, next);
  next = id_of(first + W);
  if constexpr (SUM) {
    sum_query<D>(static_cast<const uint16_t*>(a.q), a.R, a.H, a.Hkv, row, &query);
    __syncthreads();
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < (int)(sizeof(Query8<D>) / 16); i += W * 32)
        reinterpret_cast<uint4*>(rows + row)[i] = reinterpret_cast<const uint4*>(&query)[i];
  } else {
    for (int i = threadIdx.x; i < (int)(sizeof(Query8<D>) / 16); i += W * 32)
      reinterpret_cast<uint4*>(&query)[i] = reinterpret_cast<const uint4*>(rows + row)[i];
    __syncthreads();
  }
  // (the query's parts: column r of a tile is part r, the columns behind are 0)
  const uint16_t* part = &query.part[min(r, 3)][q4 * 16];
  float* out = scores + (size_t)row * a.n_vis;
  float top = 0.f;             // the largest factor
  for (int p = first; p < end; p += W) {
    float c[4] = {};
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&k[0][i >> 2]);
      const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&k[1][i >> 2]);
      const uint32_t y0 = w0[i & 3], y1 = w1[i & 3];
      const uint2 q = *reinterpret_cast<const uint2*>(part + (i >> 2) * 64 + (i & 3) * 4);
      float z[4] = {};         // (a chain of tiles would lose bits beside their running sum)
      mma_f16(z, kv8::e4m3x2_to_half2((uint16_t)y0), kv8::e4m3x2_to_half2((uint16_t)y1),
              kv8::e4m3x2_to_half2((uint16_t)(y0 >> 16)), kv8::e4m3x2_to_half2((uint16_t)(y1 >> 16)), q.x, q.y);
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = __fadd_rn(c[e], z[e]);
    }
    const bool there = ok;
    const float f = factor;
    load(p + W, next);
    next = id_of(p + 2 * W);
    // columns 0 and 1 are lane 4 r's, column 2 is its neighbour's
    const float z0 = __shfl_down_sync(0xffffffffu, c[0], 1), z1 = __shfl_down_sync(0xffffffffu, c[2], 1);
    const float s0 = c[0] + (c[1] + z0), s1 = c[2] + (c[3] + z1);
    const int pos = p * 16 + r;
    if (q4 == 0) {
      // (NaN without a sign, so that its key is the largest)
      auto value = [&](float v) {
        v = (v * query.back[0]) * (f * query.back[1]);
        return !there ? 0.f : isnan(v) ? __uint_as_float(0x7fffffffu) : v;
      };
      if (pos < nv) out[pos] = value(s0);
      if (pos + 8 < nv) out[pos + 8] = value(s1);
    }
    if (there) top = fmaxf(top, fabsf(f));
  }
  if (lane == 0) factors[((size_t)row * gridDim.x + blockIdx.x) * W + warp] = top;
}

namespace {

struct BorderShared {
  uint64_t list_v[kListed];
  int list_j[kListed];
  int sure, near, digit, above, last_j;
  unsigned long long last;
  uint32_t kth[32];
  float factor[32];
  uint32_t scan_tmp[33];
  int hist[256];
};

// The score of token j with 48 bits, by eight lanes (lane % 8 == 0 has it).
template <int D>
__device__ __forceinline__ uint64_t score48(const Kv8RetrieveArgs& a, const Query8<D>* query, int b, int g, int j, bool on,
                                          int lane) {
  float hi = 0.f, lo = 0.f, s = 0.f;
  if (on) {
    const int page = __ldg(a.block_table + (size_t)b * a.max_blocks + (j >> 4));
    if (page >= 0 && page < a.num_blocks) {
      const size_t unit = (size_t)page * a.Hkv + g;
      const int e0 = (lane & 7) * (D / 8);
      const uint8_t* src = a.k_pool + (unit * 16 + (j & 15)) * D + e0;
      s = __ldg(a.scales + unit * 2);
      uint32_t w[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(src) + i);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const float2 x = kv8::e4m3x2_to_float2((uint16_t)(w[i >> 1] >> ((i & 1) * 16)));
        const float4 q2 = __ldg(reinterpret_cast<const float4*>(&query->qbar[e0 + 2 * i]));
        float p = __fmul_rn(q2.x, x.x);
        add48(hi, lo, p, fmaf(q2.y, x.x, fmaf(q2.x, x.x, -p)));
        p = __fmul_rn(q2.z, x.y);
        add48(hi, lo, p, fmaf(q2.w, x.y, fmaf(q2.z, x.y, -p)));
      }
    }
  }
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
    // (the same sum whichever of the two lanes forms it)
    const bool upper = (lane & o) != 0;
    float x = upper ? h : hi, xl = upper ? l : lo;
    add48(x, xl, upper ? hi : h, upper ? lo : l);
    hi = x;
    lo = xl;
  }
  // times s, which need not be a power of two
  const float p = __fmul_rn(hi, s), e = __fadd_rn(fmaf(hi, s, -p), __fmul_rn(lo, s));
  two_sum(p, e, hi, lo);
  return order_key64(hi, lo);
}

// Keys [lo, hi] around a border may lie on its other side: those within the band of
// it (every selected fp32 score is at least the border's value and every other one
// below it, so that is as good a middle as the k-th score), and where the search for
// it ended with few keys in the border's bin, those of the bin and within the band of
// both its ends.  Scores or a band that are not finite: the fp32 order, ties included.
constexpr int kFew = 6;
struct Near {
  uint32_t lo, hi;
  bool wide;
};
__device__ __forceinline__ Near near_border(const TopkBorder& t, float band) {
  auto value = [](uint32_t key) {
    return (key & 0x80000000u) ? __uint_as_float(key ^ 0x80000000u) : __uint_as_float(~key);
  };
  const uint32_t bin = t.prefix | ~t.pmask, top = t.open ? bin : t.prefix;
  Near x;
  x.wide = band > 0.f && isfinite(band) && isfinite(value(t.prefix)) && isfinite(value(top));
  x.lo = x.wide ? order_key(value(t.prefix) - band) : t.prefix;
  x.hi = x.wide ? order_key(value(top) + band) : bin;
  return x;
}

// Writes the indices (first + i) of the keys that are taken in ascending order, by a
// block whose warps have stretches of 32 keys; before(n) tells how many come before
// the block's n.
template <typename Taken, typename Before>
__device__ __forceinline__ void emit_taken(int n, int first, int32_t* dst, uint32_t* scan_tmp, Taken taken, Before before) {
  const int nt = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = nt >> 5;
  const int per = ((n + 31) / 32 + nw - 1) / nw * 32, w0 = min(n, warp * per), w1 = min(n, w0 + per);
  uint32_t count = 0;
  for (int i0 = w0; i0 < w1; i0 += 32) count += __popc(__ballot_sync(0xffffffffu, i0 + lane < w1 && taken(i0 + lane)));
  if (lane == 0) scan_tmp[warp] = count;
  __syncthreads();
  uint32_t o = 0, all = 0;
  for (int w = 0; w < nw; ++w) {
    const uint32_t c = scan_tmp[w];
    o += w < warp ? c : 0u;
    all += c;
  }
  o += before(all);
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const bool take = i0 + lane < w1 && taken(i0 + lane);
    const uint32_t mask = __ballot_sync(0xffffffffu, take);
    if (take) dst[o + __popc(mask & ((1u << lane) - 1u))] = first + i0 + lane;
    o += __popc(mask);
  }
}

// This thread's part of the largest of a row's factors, and the block's.
__device__ __forceinline__ float some_factor(const float* factors, int n) {
  float x = 0.f;
  for (int i = threadIdx.x; i < n; i += blockDim.x) x = fmaxf(x, __ldcg(factors + i));
  return x;
}
__device__ __forceinline__ float largest_factor(float x, float* tmp) {
  x = warp_max(x);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = x;
  __syncthreads();
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) x = fmaxf(x, tmp[w]);
  return x;
}

// Selects the k tokens of a row, given its keys and their border.  All threads of
// the block call this.
template <int D>
__device__ __forceinline__ void select_row(const Kv8RetrieveArgs& a, const Query8<D>* query, int b, int g, int n, int k,
                                           uint32_t* keys, const TopkBorder& border, float factor, uint64_t* exact,
                                           int32_t* dst, BorderShared& sh) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const Near near = near_border(border, query->slack * kBand * factor);
  const uint32_t lo = near.lo, hi = near.hi;
  const bool wide = near.wide;
  if (tid == 0) sh.sure = sh.near = 0;
  __syncthreads();
  int in = 0;
  for (int i0 = tid; i0 < n; i0 += 4 * nt) {
    uint32_t key[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) key[j] = i0 + j * nt < n ? keys[i0 + j * nt] : 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      in += key[j] > hi;
      if (key[j] >= lo && key[j] <= hi) {
        const int at_list = atomicAdd(&sh.near, 1);
        if (at_list < kListed) sh.list_j[at_list] = i0 + j * nt;
      }
    }
  }
  in = __reduce_add_sync(0xffffffffu, in);
  if (lane == 0) atomicAdd(&sh.sure, in);
  __syncthreads();
  const int need = k - sh.sure, m = sh.near;     // of the m tokens next to the border
  bool by_value = false;                         // taken by (value, index), not all
  if (m > need) {
    const bool listed = m <= kListed;
    by_value = !listed;
    if (listed) {
      for (int i0 = warp * 4; i0 < m; i0 += nw * 4) {
        const int i = i0 + (lane >> 3);
        const int j = i < m ? sh.list_j[i] : 0;
        const uint64_t v = wide ? score48<D>(a, query, b, g, j, i < m, lane) : (uint64_t)keys[j] << 32;
        if (i < m && (lane & 7) == 0) sh.list_v[i] = v;
      }
      __syncthreads();
      for (int i = warp; i < m; i += nw) {
        const uint64_t v = sh.list_v[i];
        const int j = sh.list_j[i];
        int better = 0;
        for (int o = lane; o < m; o += 32) better += sh.list_v[o] > v || (sh.list_v[o] == v && sh.list_j[o] < j);
        better = __reduce_add_sync(0xffffffffu, better);
        if (lane == 0 && better >= need) keys[j] = 0u;             // (no score's key)
      }
    } else {
      for (int i0 = warp * 32; i0 < n; i0 += nt) {
        const uint32_t key = i0 + lane < n ? keys[i0 + lane] : 0u;
        uint32_t todo = __ballot_sync(0xffffffffu, i0 + lane < n && key >= lo && key <= hi);
        while (todo) {
          // four of them at a time
          int j = -1;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int bit = __ffs(todo) - 1;
            if (c == (lane >> 3) && bit >= 0) j = i0 + bit;
            todo &= todo - 1;
          }
          const uint64_t v = wide ? score48<D>(a, query, b, g, max(j, 0), j >= 0, lane) : (uint64_t)keys[max(j, 0)] << 32;
          if (j >= 0 && (lane & 7) == 0) exact[j] = v;
        }
      }
      // a radix selection over the 96 bits of (value, ~index)
      unsigned long long top = 0;
      uint32_t low = 0;
      int left = need;
      for (int pass = 0; pass < 12; ++pass) {
        for (int i = tid; i < 256; i += nt) sh.hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += nt) {
          const uint32_t key = keys[i];
          if (key < lo || key > hi) continue;
          const uint64_t kv = exact[i];
          const uint32_t ki = ~(uint32_t)i;
          if (pass < 8) {
            if (pass > 0 && (kv ^ top) >> (64 - 8 * pass)) continue;
            atomicAdd(&sh.hist[(kv >> (56 - 8 * pass)) & 255], 1);
          } else {
            if (kv != top || (pass > 8 && (ki ^ low) >> (32 - 8 * (pass - 8)))) continue;
            atomicAdd(&sh.hist[(ki >> (24 - 8 * (pass - 8))) & 255], 1);
          }
        }
        __syncthreads();
        if (tid == 0) {
          int sum = 0, d = 255;
          while (d > 0 && sum + sh.hist[d] < left) sum += sh.hist[d--];
          sh.digit = d;
          sh.above = sum;
        }
        __syncthreads();
        left -= sh.above;
        if (pass < 8) top |= (unsigned long long)sh.digit << (56 - 8 * pass);
        else low |= (uint32_t)sh.digit << (24 - 8 * (pass - 8));
        __syncthreads();
      }
      if (tid == 0) {
        sh.last = top;
        sh.last_j = (int)~low;
      }
    }
    __syncthreads();
  }
  auto taken = [&](int i) {
    const uint32_t key = keys[i];
    if (!by_value || key < lo || key > hi) return key >= lo;
    const uint64_t v = exact[i];
    return v > sh.last || (v == sh.last && i <= sh.last_j);
  };
  emit_taken(n, 0, dst, sh.scan_tmp, taken, [](uint32_t) { return 0u; });
}

}  // namespace

// The selection of one row per CTA.  KNOWN: the keys of rows that are too long for
// shared memory go to `far_keys`, the k largest fp32 scores have been taken
// (vis_idx), and the k-th is their smallest.
template <int D, bool KNOWN>
__global__ void __launch_bounds__(1024)
kv8_select_kernel(const __grid_constant__ Kv8RetrieveArgs a, const Query8<D>* rows, const float* __restrict__ scores,
                  const float* __restrict__ factors, int n_factors, uint64_t* __restrict__ exact,
                  uint32_t* __restrict__ far_keys) {
  extern __shared__ __align__(16) uint32_t staged[];
  __shared__ TopkShared ts;
  __shared__ BorderShared sh;
  grid_dep_sync();
  const int row = blockIdx.x, b = row / a.Hkv, g = row - b * a.Hkv;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  int n = a.n_vis, k = a.k;
  if (a.lens.any()) row_lengths(a.lens, row, a.Hkv, a.n_vis, a.k, n, k);
  int32_t* dst = a.vis_idx + (size_t)row * a.k;
  const float* src = scores + (size_t)row * a.n_vis;
  uint32_t* keys = KNOWN ? far_keys + (size_t)row * a.n_vis : staged;
  if (!KNOWN) fill_unselected(dst, k, a.k);
  if (k <= 0) return;
  float factor = some_factor(factors + (size_t)row * n_factors, n_factors);
  TopkBorder border;
  if (KNOWN) {
    uint32_t kth = 0xffffffffu;
    for (int i0 = tid; i0 < n; i0 += 8 * nt) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __ldcg(src + min(i0 + j * nt, n - 1));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + j * nt < n) keys[i0 + j * nt] = order_key(x[j]);
    }
    __syncthreads();
    for (int i0 = tid; i0 < k; i0 += 4 * nt) {
      int at[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) at[j] = __ldcg(dst + min(i0 + j * nt, k - 1));
#pragma unroll
      for (int j = 0; j < 4; ++j) kth = min(kth, keys[at[j]]);
    }
    kth = __reduce_min_sync(0xffffffffu, kth);
    if (lane == 0) sh.kth[warp] = kth;
    __syncthreads();
    for (int w = 0; w < nt / 32; ++w) kth = min(kth, sh.kth[w]);
    border = TopkBorder{kth, 0xffffffffu, 0, false};
  } else {
    border = block_topk_border(src, n, k, keys, ts, kFew);
  }
  factor = largest_factor(factor, sh.factor);
  select_row<D>(a, rows + row, b, g, n, k, keys, border, factor, exact + (size_t)row * a.n_vis, dst, sh);
}

// The same for a long row by a cluster: CTA r has its r-th slice.
template <int D>
__global__ void __cluster_dims__(kTopkClusterCtas, 1, 1) __launch_bounds__(kTopkClusterThreads)
kv8_select_cluster_kernel(const __grid_constant__ Kv8RetrieveArgs a, const Query8<D>* rows,
                          const float* __restrict__ scores, const float* __restrict__ factors, int n_factors,
                          uint64_t* __restrict__ exact_rows) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ ClusterTopkShared ts;
  __shared__ BorderShared sh;
  grid_dep_sync();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), row = blockIdx.x / kTopkClusterCtas, b = row / a.Hkv, g = row - b * a.Hkv;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  int n = a.n_vis, k = a.k;
  if (a.lens.any()) row_lengths(a.lens, row, a.Hkv, a.n_vis, a.k, n, k);
  int32_t* dst = a.vis_idx + (size_t)row * a.k;
  if (rank == 0) fill_unselected(dst, k, a.k);
  if (k <= 0) return;                        // (the whole cluster)
  const int slice = (n + kTopkClusterCtas - 1) / kTopkClusterCtas;
  const int first = min(n, rank * slice), len = min(n, first + slice) - first;
  const Query8<D>* query = rows + row;
  uint64_t* exact = exact_rows + (size_t)row * a.n_vis + first;
  float factor = some_factor(factors + (size_t)row * n_factors, n_factors);
  if (tid == 0) sh.sure = sh.near = 0;       // (the search below has barriers)
  const TopkBorder t = cluster_topk_border(scores + (size_t)row * a.n_vis + first, len, k, keys, ts, kFew);
  factor = largest_factor(factor, sh.factor);
  const Near x = near_border(t, query->slack * kBand * factor);
  const uint32_t lo = x.lo, hi = x.hi;
  const bool wide = x.wide;
  int in = 0;
  for (int i = tid; i < len; i += nt) {
    const uint32_t key = keys[i];
    in += key > hi;
    if (key >= lo && key <= hi) {
      const int at_list = atomicAdd(&sh.near, 1);
      if (at_list < kListed) sh.list_j[at_list] = i;
    }
  }
  in = __reduce_add_sync(0xffffffffu, in);
  if (lane == 0) atomicAdd(&sh.sure, in);
  cluster.sync();
  int sure = 0, m = 0, most = 0;
#pragma unroll
  for (int r = 0; r < kTopkClusterCtas; ++r) {
    const int near = *cluster.map_shared_rank(&sh.near, r);
    sure += *cluster.map_shared_rank(&sh.sure, r);
    m += near;
    most = max(most, near);
  }
  const int need = k - sure, mine = sh.near;
  bool by_value = false;
  if (m > need) {
    by_value = most > kListed;
    if (!by_value) {
      for (int i0 = warp * 4; i0 < mine; i0 += nw * 4) {
        const int i = i0 + (lane >> 3);
        const int j = i < mine ? sh.list_j[i] : 0;
        const uint64_t v = wide ? score48<D>(a, query, b, g, first + j, i < mine, lane) : (uint64_t)keys[j] << 32;
        if (i < mine && (lane & 7) == 0) sh.list_v[i] = v;
      }
      cluster.sync();
      // ranked against every CTA's list (slices are in order of index)
      for (int i = warp; i < mine; i += nw) {
        const uint64_t v = sh.list_v[i];
        const int j = sh.list_j[i];
        int better = 0;
        // (four lanes for each CTA, so that no list waits for another)
        const int r = lane >> 2;
        static_assert(kTopkClusterCtas == 8, "four lanes a CTA");
        const int theirs = *cluster.map_shared_rank(&sh.near, r);
        const uint64_t* values = cluster.map_shared_rank(&sh.list_v[0], r);
        const int* indices = cluster.map_shared_rank(&sh.list_j[0], r);
        for (int o = lane & 3; o < theirs; o += 4) {
          const uint64_t y = values[o];
          better += y > v || (y == v && (r < rank || (r == rank && indices[o] < j)));
        }
        better = __reduce_add_sync(0xffffffffu, better);
        if (lane == 0 && better >= need) keys[j] = 0u;             // (no score's key)
      }
    } else {
      for (int i0 = warp * 32; i0 < len; i0 += nt) {
        const uint32_t key = i0 + lane < len ? keys[i0 + lane] : 0u;
        uint32_t todo = __ballot_sync(0xffffffffu, i0 + lane < len && key >= lo && key <= hi);
        while (todo) {
          int j = -1;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int bit = __ffs(todo) - 1;
            if (c == (lane >> 3) && bit >= 0) j = i0 + bit;
            todo &= todo - 1;
          }
          const uint64_t v =
              wide ? score48<D>(a, query, b, g, first + max(j, 0), j >= 0, lane) : (uint64_t)keys[max(j, 0)] << 32;
          if (j >= 0 && (lane & 7) == 0) exact[j] = v;
        }
      }
      for (int i = tid; i < 512; i += nt) (&ts.hist[0][0])[i] = 0;
      unsigned long long top = 0;
      uint32_t low = 0;
      int left = need;
      cluster.sync();
      for (int pass = 0; pass < 12; ++pass) {
        int* hist = ts.hist[pass & 1];
        for (int i = tid; i < len; i += nt) {
          const uint32_t key = keys[i];
          if (key < lo || key > hi) continue;
          const uint64_t kv = exact[i];
          const uint32_t ki = ~(uint32_t)(first + i);
          if (pass < 8) {
            if (pass > 0 && (kv ^ top) >> (64 - 8 * pass)) continue;
            atomicAdd(&hist[(kv >> (56 - 8 * pass)) & 255], 1);
          } else {
            if (kv != top || (pass > 8 && (ki ^ low) >> (32 - 8 * (pass - 8)))) continue;
            atomicAdd(&hist[(ki >> (24 - 8 * (pass - 8))) & 255], 1);
          }
        }
        cluster.sync();
        for (int i = tid; i < 256; i += nt) {
          int sum = 0;
#pragma unroll
          for (int r = 0; r < kTopkClusterCtas; ++r) sum += cluster.map_shared_rank(hist, r)[i];
          ts.total[i] = sum;
          ts.hist[(pass + 1) & 1][i] = 0;            // (last read by peers before this pass's barrier)
        }
        __syncthreads();
        if (tid == 0) {
          int sum = 0, d = 255;
          while (d > 0 && sum + ts.total[d] < left) sum += ts.total[d--];
          sh.digit = d;
          sh.above = sum;
        }
        __syncthreads();
        left -= sh.above;
        if (pass < 8) top |= (unsigned long long)sh.digit << (56 - 8 * pass);
        else low |= (uint32_t)sh.digit << (24 - 8 * (pass - 8));
        __syncthreads();
      }
      if (tid == 0) {
        sh.last = top;
        sh.last_j = (int)~low;
      }
    }
    __syncthreads();
  }
  auto taken = [&](int i) {
    const uint32_t key = keys[i];
    if (!by_value || key < lo || key > hi) return key >= lo;
    const uint64_t v = exact[i];
    return v > sh.last || (v == sh.last && first + i <= sh.last_j);
  };
  emit_taken(len, first, dst, sh.scan_tmp, taken, [&](uint32_t all) {
    if (tid == 0) ts.cnt[0] = (int)all;
    cluster.sync();
    uint32_t o = 0;
#pragma unroll
    for (int r = 0; r < kTopkClusterCtas; ++r) o += r < rank ? (uint32_t)*cluster.map_shared_rank(&ts.cnt[0], r) : 0u;
    return o;
  });
  cluster.sync();     // keep this CTA's shared memory alive until every peer has read it
}

// Workspace: queries | 48-bit scores of tokens next to a crowded border | fp32
// scores | the largest factor of each scoring CTA's pages | keys of rows that are
// too long for shared memory
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
size_t kv8_retrieve_workspace_bytes(int B, int Hkv, int D, int n_vis) {
  const size_t rows = (size_t)B * Hkv;
  return up256(rows * (D == 128 ? sizeof(Query8<128>) : sizeof(Query8<64>))) + up256(rows * n_vis * sizeof(uint64_t)) +
         up256(rows * ((n_vis + 15) / 16 + kScoreWarps) * sizeof(float)) + up256(rows * n_vis * sizeof(float)) * (n_vis > kStagedKeys && !topk_cluster_fits(n_vis) ? 2 : 1);
}

template <int D, bool KNOWN>
static cudaError_t launch_select(const Kv8RetrieveArgs& a, const Query8<D>* rows, const float* scores,
                                 const float* factors, int n_factors, uint64_t* exact,
                                 uint32_t* far_keys, cudaStream_t stream) {
  auto kernel = kv8_select_kernel<D, KNOWN>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStagedKeys * 4);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int threads = KNOWN ? 1024 : a.n_vis >= 8192 ? 512 : 256;
  return launch_dependent(kernel, dim3((unsigned)(a.batch * a.Hkv)), dim3(threads),
                          KNOWN ? (size_t)0 : (size_t)a.n_vis * 4, stream, a, rows, scores, factors, n_factors, exact, far_keys);
}

template <int D>
static cudaError_t launch_select_cluster(const Kv8RetrieveArgs& a, const Query8<D>* rows, const float* scores,
                                         const float* factors, int n_factors, uint64_t* exact, cudaStream_t stream) {
  auto kernel = kv8_select_cluster_kernel<D>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int slice = (a.n_vis + kTopkClusterCtas - 1) / kTopkClusterCtas;
  return launch_dependent(kernel, dim3((unsigned)(kTopkClusterCtas * a.batch * a.Hkv)), dim3(kTopkClusterThreads),
                          (size_t)slice * sizeof(uint32_t), stream, a, rows, scores, factors, n_factors, exact);
}

template <int D>
static cudaError_t launch_d(const Kv8RetrieveArgs& a, int num_sms, cudaStream_t stream) {
  const int rows = a.batch * a.Hkv;
  char* at = static_cast<char*>(a.ws);
  auto take = [&](size_t bytes) {
    char* p = at;
    at += up256(bytes);
    return p;
  };
  Query8<D>* query = reinterpret_cast<Query8<D>*>(take((size_t)rows * sizeof(Query8<D>)));
  uint64_t* exact = reinterpret_cast<uint64_t*>(take((size_t)rows * a.n_vis * sizeof(uint64_t)));
  float* scores = reinterpret_cast<float*>(take((size_t)rows * a.n_vis * sizeof(float)));
  float* factors = reinterpret_cast<float*>(take((size_t)rows * ((a.n_vis + 15) / 16 + kScoreWarps) * sizeof(float)));
  uint32_t* far_keys = reinterpret_cast<uint32_t*>(at);      // (there where it is used)
  if (a.scores != nullptr) scores = a.scores;
  // pages per CTA: a multiple of its warps, for two rounds of resident CTAs (of 4, 5,
  // 10, 12 and 20 CTAs per SM ten are the fastest: LLaVA-NeXT batch 16 48 us at 10 and
  // more, 50 at 5; LongVILA batch 8 58, 62 at 5)
  const int pages = (a.n_vis + 15) / 16;
  const long long ctas = (long long)num_sms * 10;
  long long per = ((long long)pages * rows + ctas - 1) / ctas;
  per = (per + kScoreWarps - 1) / kScoreWarps * kScoreWarps;
  if (per > pages) per = pages;
  const long long per_row = (pages + per - 1) / per;
  // (the sums of few rows in every CTA cost less than a launch before them:
  // LongVILA batch 8, seven heads, 58 us, not 71)
  const bool sum = (long long)a.R * (a.H / a.Hkv) <= kFusedRows;
  cudaError_t e = cudaSuccess;
  if (!sum)
    e = launch_dependent(kv8_qbar_kernel<D>, dim3(rows), dim3(D), 0, stream, static_cast<const uint16_t*>(a.q), a.R, a.H,
                         a.Hkv, query);
  if (e != cudaSuccess) return e;
  e = launch_dependent(sum ? kv8_score_kernel<D, true> : kv8_score_kernel<D, false>, dim3((unsigned)per_row, a.Hkv, a.batch),
                       dim3(kScoreWarps * 32), 0, stream, a, query, scores, factors, (int)per);
  if (e != cudaSuccess) return e;
  // a CTA per row as long as rows are short, else a cluster (as topk_prefers_cluster),
  // and for rows that do not fit one either a CTA over their keys in memory
  if (a.n_vis <= kStagedKeys) return launch_select<D, false>(a, query, scores, factors, (int)per_row * kScoreWarps, exact, nullptr, stream);
  if (topk_cluster_fits(a.n_vis)) return launch_select_cluster<D>(a, query, scores, factors, (int)per_row * kScoreWarps, exact, stream);
  e = launch_topk_rows(scores, rows, a.n_vis, a.k, a.vis_idx, stream, a.lens, a.Hkv);
  if (e != cudaSuccess) return e;
  return launch_select<D, true>(a, query, scores, factors, (int)per_row * kScoreWarps, exact, far_keys, stream);
}

cudaError_t launch_kv8_retrieve(const Kv8RetrieveArgs& a, int D, int num_sms, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, num_sms, stream) : launch_d<64>(a, num_sms, stream);
}

}  // namespace sv
