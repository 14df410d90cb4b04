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
//
// Measured, keys out of L2, head dim 128: 16 sequences of 32 KV heads and 2880 keys
// 46.1 us (4.3 TB/s of keys), 8 ragged ones of 4 heads and up to 50176 keys 51.6 us
// (3.1 TB/s); 193 question rows of 28 heads over 4 and 576 keys 13.7 us.  Scoring takes
// 37 and 36 us of the first two by itself: with a page in flight in each of 40 warps an
// SM pages go by at 6.2 TB/s, and 17 % of an SM's time lies before its first page and
// behind its last.  More pages on their way are no faster (two in registers of
// 24 warps 48.3 / 54.5, of 32 warps with spills 62.7 / 61.5; two or three in a cp.async
// ring of 32 warps 51.0 / 56.8 and 56.4 / 56.7), nor are packed adds; two and four times
// the CTAs 48.8 / 56.8 and 52.6 / 65.6; equal shares of each row instead of one line
// 47.3 / 53.8.  The selection
// takes 9 and 16, a chain of some ten waits (scores, counts, pages of the tokens next
// to the border, and a cluster's barriers) that little work lies between; with a search
// by the bits of the keys the two calls were 1 and 2.4 us longer.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "kv8.cuh"
#include "topk_block.cuh"

namespace cg = cooperative_groups;

namespace sv {

namespace {

constexpr int kScoreWarps = 8, kScoreCtas = 5;   // per CTA, and CTAs per SM
// |fp32 score - score| <= e = 2^-24 (272 |qbar|_max + 12 |qbar|_1) 448 s, as 448 s
// bounds a key's elements: a tile's 16 products lose at most the last of 24 bits
// beside the largest, and their sum, at most 16 of the largest, as much again (eight
// tiles, and their parts' columns); seven sums of tiles, two of columns and three
// products with factors round to 2^-24 of what is below |qbar|_1 448 s.  Two tokens
// are told apart by 2 e; twice that is taken:
constexpr float kBand = 448.f / 4194304.f;
constexpr float kBandMax = 272.f, kBandSum = 12.f;
// Keys of a row whose selection one CTA makes.  Whole calls, head dim 128, by a CTA / by a
// cluster: 4 rows of 6000 keys 20.4 / 15.2 us, of 16384 24.9 / 18.3, of 20000 31.4 / 22.2;
// 32 rows 27.0 / 24.1, 38.5 / 31.9, 50.9 / 34.9; 128 rows 49.8 / 66.3, 73.6 / 97.0,
// 113.9 / 109.2 (and of 30000 105.6 / 139.6).  One border for all: right for many rows, late
// for few.
constexpr int kStagedKeys = 16384;
constexpr int kSliceKeys = 50176;        // keys that a CTA of a cluster keeps in shared memory

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

// Query rows times heads that every scoring CTA sums itself: 7 of LongVILA batch 8 so
// 51.6 us, by a launch before 60.4; 14 of two sequences of 3000 keys 20.3 and 14.9.
constexpr int kFusedRows = 8;

// *o from element e = threadIdx.x of a row's sum, by threads 0 .. D - 1 of a block of at
// least D (all threads call this); the caller synchronises before it reads *o.
template <int D>
__device__ __forceinline__ void write_query(float hi, float lo, Query8<D>* o) {
  __shared__ float part[2][D / 32];
  const int e = threadIdx.x;
  if (e < D) {
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
  const float f0 = __uint_as_float((uint32_t)(127 - x / 2) << 23);
  const float f1 = __uint_as_float((uint32_t)(127 - (x - x / 2)) << 23);
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

// The row's query from few rows, an element a thread.
template <int D>
__device__ __forceinline__ void sum_query(const uint16_t* q, int R, int H, int Hkv, int row, Query8<D>* o) {
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
  }
  write_query<D>(hi, lo, o);
}

}  // namespace

// The queries of rows with many: C CTAs per row of the cache, a warp per query row at a
// time, eight on their way.
constexpr int kSumWarps = 32, kSumCtas = 8;
template <int D, int C>
__device__ __forceinline__ void sum_queries(const uint16_t* __restrict__ q, int R, int H, int Hkv, Query8<D>* rows) {
  constexpr int E = D / 32, kAhead = 8, kParts = kSumWarps * 32 / D, kEach = kSumWarps / kParts, kStep = kSumWarps * C;
  __shared__ float2 sums[kSumWarps][D];
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = C > 1 ? (int)cluster.block_rank() : 0, row = blockIdx.x / C;
  const int b = row / Hkv, g = row - b * Hkv, G = H / Hkv, n = R * G;
  // query row i is head h of the group at question row r; the next one of a warp is
  // kStep further on
  int i = rank * kSumWarps + warp, r = i / G, h = i - r * G;
  const int dr = kStep / G, dh = kStep - dr * G;
  grid_dep_sync();
  const uint16_t* src = q + ((size_t)b * R * H + (size_t)g * G) * D + lane * E;
  float hi[E], lo[E];
#pragma unroll
  for (int e = 0; e < E; ++e) hi[e] = lo[e] = 0.f;
#pragma unroll 1
  while (i < n) {
    uint32_t x[kAhead][E / 2];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t* at = reinterpret_cast<const uint32_t*>(src + ((size_t)r * H + h) * D);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) x[j][e] = i < n ? __ldg(at + e) : 0u;
      i += kStep;
      r += dr;
      h += dh;
      if (h >= G) {
        h -= G;
        ++r;
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        add48(hi[2 * e], lo[2 * e], bf16_lo(x[j][e]), 0.f);
        add48(hi[2 * e + 1], lo[2 * e + 1], bf16_hi(x[j][e]), 0.f);
      }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = make_float2(hi[e], lo[e]);
  __syncthreads();
  // kParts threads an element, then one of the CTA, then one of the cluster
  const int e = threadIdx.x % D, part = threadIdx.x / D;
  float t = 0.f, l = 0.f;
#pragma unroll
  for (int w = 0; w < kEach; ++w) add48(t, l, sums[part * kEach + w][e].x, sums[part * kEach + w][e].y);
  __syncthreads();
  sums[part][e] = make_float2(t, l);
  __syncthreads();
  t = l = 0.f;
  if (threadIdx.x < D)
#pragma unroll
    for (int p = 0; p < kParts; ++p) add48(t, l, sums[p][e].x, sums[p][e].y);
  if constexpr (C > 1) {
    __syncthreads();
    if (threadIdx.x < D) sums[0][e] = make_float2(t, l);
    cluster.sync();
    if (rank == 0 && threadIdx.x < D) {
      float2 theirs[C];
#pragma unroll
      for (int c = 1; c < C; ++c) theirs[c] = *cluster.map_shared_rank(&sums[0][e], c);
#pragma unroll
      for (int c = 1; c < C; ++c) add48(t, l, theirs[c].x, theirs[c].y);
    }
    cluster.sync();                                          // (its shared memory has been read)
    if (rank != 0) return;
  }
  write_query<D>(t, l, rows + row);
}

template <int D>
__global__ void __launch_bounds__(kSumWarps * 32)
kv8_qbar_kernel(const uint16_t* __restrict__ q, int R, int H, int Hkv, Query8<D>* rows) {
  sum_queries<D, 1>(q, R, H, Hkv, rows);
}
template <int D>
__global__ void __cluster_dims__(kSumCtas, 1, 1) __launch_bounds__(kSumWarps * 32)
kv8_qbar_cluster_kernel(const uint16_t* __restrict__ q, int R, int H, int Hkv, Query8<D>* rows) {
  sum_queries<D, kSumCtas>(q, R, H, Hkv, rows);
}

// What a scoring warp leaves for the selection: the largest factor of its pages, and
// its smallest and largest score as ordered keys.
struct __align__(16) Part {
  float factor;
  uint32_t lo, hi, pad;
};

// The pages of all (sequence, KV head) rows form one line, cut evenly between the
// CTAs.  A CTA leaves a part per warp for each of its rows: one that it has all of, one
// that it goes on with (slot 0) and one that it begins and others go on with (slot 1).
struct Parts {
  Part* whole;             // [rows][kScoreWarps]
  Part* cut;               // [CTAs][2][kScoreWarps]
  int ctas;
  int pages;               // of a row, with equal counts
};

__device__ __forceinline__ uint32_t pages_of(const Kv8RetrieveArgs& a, int b) {
  int nv = 0, nt, kb;
  if (b < a.batch) seq_lengths(a.lens, b, a.n_vis, a.n_text, a.k, nv, nt, kb);
  return (uint32_t)(nv + 15) >> 4;
}
// Pages of all heads of sequences [b0, b0 + 32) up to this lane's (and its own), by a
// whole warp.
__device__ __forceinline__ uint32_t scan_pages(const Kv8RetrieveArgs& a, int b0, int lane, uint32_t& mine) {
  mine = pages_of(a, b0 + lane) * (uint32_t)a.Hkv;
  uint32_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  return inc;
}
// The line's length and, where b < batch, what lies before sequence b.
__device__ __forceinline__ uint32_t line_of(const Kv8RetrieveArgs& a, const Parts& parts, int b, int lane,
                                            uint32_t& before) {
  if (!a.lens.any()) {
    before = (uint32_t)b * (uint32_t)a.Hkv * (uint32_t)parts.pages;
    return (uint32_t)a.batch * (uint32_t)a.Hkv * (uint32_t)parts.pages;
  }
  uint32_t total = 0, mine;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const uint32_t inc = scan_pages(a, b0, lane, mine);
    if (b >= b0 && b < b0 + 32) before = total + __shfl_sync(0xffffffffu, inc - mine, b - b0);
    total += __shfl_sync(0xffffffffu, inc, 31);
  }
  return total;
}

// With many sequences of their own lengths a stretch of them to each warp: W warps' sums
// of pages.  (By each warp for itself 3001 sequences of 320 keys, 4 KV heads, 712 us a call
// instead of 358; 256 sequences 41 and 34.)
__device__ __forceinline__ bool by_stretches(const Kv8RetrieveArgs& a) { return a.lens.any() && a.batch > 32; }
__device__ __forceinline__ int stretch_of(const Kv8RetrieveArgs& a, int W) { return ((a.batch + 31) / 32 + W - 1) / W * 32; }
__device__ __forceinline__ uint32_t stretch_pages(const Kv8RetrieveArgs& a, int b0, int b1, int lane) {
  uint32_t sum = 0, mine;
  for (; b0 < b1; b0 += 32) sum += __shfl_sync(0xffffffffu, scan_pages(a, b0, lane, mine), 31);
  return sum;
}

// A warp per page, one page in flight, as many warps as 48 registers allow.  SUM:
// the query's rows are few, and every CTA adds them up itself (the first of a row
// leaves the sum for the selection).
template <int D, bool SUM>
__global__ void __launch_bounds__(kScoreWarps * 32, kScoreCtas)
kv8_score_kernel(const __grid_constant__ Kv8RetrieveArgs a, Query8<D>* rows, float* __restrict__ scores,
                 const Parts parts) {
  constexpr int KS = D / 16, KC = D / 64, W = kScoreWarps;
  __shared__ __align__(16) Query8<D> query;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, q4 = lane & 3;
  grid_dep_sync();
  uint32_t off = 0;                        // of this CTA's first page in sequence b
  int left, b = 0;
  __shared__ uint32_t stretch[W];
  {
    uint32_t before = 0, total = 0;
    if (by_stretches(a)) {
      const int each = stretch_of(a, W);
      const uint32_t sum = stretch_pages(a, warp * each, min(a.batch, (warp + 1) * each), lane);
      if (lane == 0) stretch[warp] = sum;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) total += stretch[w];
    } else {
      total = line_of(a, parts, 0, lane, before);
    }
    const uint32_t C = min((uint32_t)parts.ctas, total);
    if (blockIdx.x >= C) left = 0;
    else {
      off = kv8::piece_begin(total, blockIdx.x, C);
      left = (int)(kv8::piece_begin(total, blockIdx.x + 1, C) - off);
    }
  }
  if (!a.lens.any()) {
    const uint32_t in_seq = (uint32_t)a.Hkv * (uint32_t)parts.pages;
    if (left > 0) {
      b = (int)(off / in_seq);
      off -= (uint32_t)b * in_seq;
    }
  } else {
    for (int i = blockIdx.x * W * 32 + threadIdx.x; i < a.batch; i += gridDim.x * W * 32) {
      int nv, nt, kb;
      if (!seq_lengths(a.lens, i, a.n_vis, a.n_text, a.k, nv, nt, kb)) flag_status(a.status, kStatusBadLength);
    }
    if (by_stretches(a) && left > 0) {
      int w = 0;
      for (; w < W - 1 && off >= stretch[w]; ++w) off -= stretch[w];
      b = w * stretch_of(a, W);
    }
    for (; left > 0 && b < a.batch; b += 32) {
      uint32_t mine;
      const uint32_t inc = scan_pages(a, b, lane, mine), past = __ballot_sync(0xffffffffu, inc > off);
      if (past) {
        const int f = __ffs(past) - 1;
        off -= __shfl_sync(0xffffffffu, inc - mine, f);
        b += f;
        break;
      }
      off -= __shfl_sync(0xffffffffu, inc, 31);
    }
  }

#pragma unroll 1
  for (; left > 0; ++b, off = 0) {
    int nv, nt, kb;
    seq_lengths(a.lens, b, a.n_vis, a.n_text, a.k, nv, nt, kb);
    const int pages = (nv + 15) >> 4;
#pragma unroll 1
    while (left > 0 && off < (uint32_t)pages * (uint32_t)a.Hkv) {
      const int g = (int)(off / (uint32_t)pages), row = b * a.Hkv + g;
      const int p0 = (int)off - g * pages, end = min(pages, p0 + left);
      off += end - p0;
      left -= end - p0;
      const int first = p0 + warp;
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
      __syncthreads();                         // (the query of the row before has been read)
      if constexpr (SUM) {
        sum_query<D>(static_cast<const uint16_t*>(a.q), a.R, a.H, a.Hkv, row, &query);
        __syncthreads();
        if (p0 == 0)
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
      Part mine = {0.f, 0xffffffffu, 0u, 0u};
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
          auto put = [&](int at, float v) {
            if (at >= nv) return;
            out[at] = v;
            mine.lo = min(mine.lo, order_key(v));
            mine.hi = max(mine.hi, order_key(v));
          };
          put(pos, value(s0));
          put(pos + 8, value(s1));
        }
        if (there) mine.factor = fmaxf(mine.factor, fabsf(f));
      }
      mine.lo = __reduce_min_sync(0xffffffffu, mine.lo);
      mine.hi = __reduce_max_sync(0xffffffffu, mine.hi);
      Part* to = p0 == 0 && end == pages ? parts.whole + (size_t)row * W
                                         : parts.cut + ((size_t)blockIdx.x * 2 + (p0 == 0)) * W;
      if (lane == 0)
        *reinterpret_cast<uint4*>(to + warp) = make_uint4(__float_as_uint(mine.factor), mine.lo, mine.hi, 0u);
    }
  }
}

namespace {

constexpr int kCluster = 8, kClusterThreads = 512;   // of a long row's selection
constexpr int kBins = 2048;
constexpr int kCrowd = 320, kPasses = 4;   // a border's bin of more keys is cut again, up to so often
constexpr int kMany = 320;                 // tokens next to the border whose factors are worth a look
constexpr int kListed = 512;               // tokens next to the border that are ranked in shared memory

struct __align__(16) SelectShared {
  uint2 mine[kListed], all[kListed];       // (key, index) of this CTA's tokens next to the border, and of every CTA's
  uint64_t exact[kListed];
  uint32_t key[kListed];                   // (16-byte aligned)
  int inside[kListed];                     // those of `all` that fp32 cannot tell
  int hist[kBins], coarse[32];
  int sure, near;                          // this CTA's tokens above the border, and next to it
  int bin, count, clear, n_inside, kept, top;
  uint32_t kth, lo[32], hi[32], scan[32];
  float factor[32];
  int2 by;
};

// The first and the last CTA that scored pages of a row of n > 0 keys, in a line of
// `total` with `before` ahead of its sequence.
__device__ __forceinline__ int2 scorers_of(const Kv8RetrieveArgs& a, const Parts& parts, int row, int n, uint32_t total,
                                           uint32_t before) {
  const int b = row / a.Hkv, pages = (n + 15) >> 4;
  const uint32_t C = min((uint32_t)parts.ctas, total);
  const uint32_t start = before + (uint32_t)(row - b * a.Hkv) * (uint32_t)pages;
  return make_int2(kv8::piece_of(total, start, C), kv8::piece_of(total, start + pages - 1, C));
}
// The parts of a row together; all threads of the block call this.
__device__ __forceinline__ Part whole_row(const Parts& parts, int row, int2 by, SelectShared& sh) {
  Part x = {0.f, 0xffffffffu, 0u, 0u};
  for (int i = threadIdx.x; i < (by.y - by.x + 1) * kScoreWarps; i += blockDim.x) {
    const int c = by.x + i / kScoreWarps;
    const Part* at = by.x == by.y ? parts.whole + (size_t)row * kScoreWarps
                                  : parts.cut + ((size_t)c * 2 + (c == by.x)) * kScoreWarps;
    const uint4 y = __ldcg(reinterpret_cast<const uint4*>(at + i % kScoreWarps));
    x.factor = fmaxf(x.factor, __uint_as_float(y.x));
    x.lo = min(x.lo, y.y);
    x.hi = max(x.hi, y.z);
  }
  x.factor = warp_max(x.factor);
  x.lo = __reduce_min_sync(0xffffffffu, x.lo);
  x.hi = __reduce_max_sync(0xffffffffu, x.hi);
  if ((threadIdx.x & 31) == 0) {
    sh.factor[threadIdx.x >> 5] = x.factor;
    sh.lo[threadIdx.x >> 5] = x.lo;
    sh.hi[threadIdx.x >> 5] = x.hi;
  }
  __syncthreads();
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    x.factor = fmaxf(x.factor, sh.factor[w]);
    x.lo = min(x.lo, sh.lo[w]);
    x.hi = max(x.hi, sh.hi[w]);
  }
  return x;
}

// The score of token j with 48 bits, by eight lanes, all of which have it.
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
      float hi1 = 0.f, lo1 = 0.f;                          // (two sums side by side: each waits for its last step)
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const float2 x = kv8::e4m3x2_to_float2((uint16_t)(w[i >> 1] >> ((i & 1) * 16)));
        const float4 q2 = __ldg(reinterpret_cast<const float4*>(&query->qbar[e0 + 2 * i]));
        float p = __fmul_rn(q2.x, x.x);
        add48(hi, lo, p, fmaf(q2.y, x.x, fmaf(q2.x, x.x, -p)));
        p = __fmul_rn(q2.z, x.y);
        add48(hi1, lo1, p, fmaf(q2.w, x.y, fmaf(q2.z, x.y, -p)));
      }
      add48(hi, lo, hi1, lo1);
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

__device__ __forceinline__ float value_of(uint32_t key) {
  return (key & 0x80000000u) ? __uint_as_float(key ^ 0x80000000u) : __uint_as_float(~key);
}

// Keys [lo, hi] around a border: those above are in and those below are out.
struct Near {
  uint32_t lo, hi;
};

// Keys within the band around values [lo, hi] that the k-th score lies in.  (Every
// selected fp32 score is at least the border's value and every other one below it, so
// that is as good a middle as the k-th true score.)
__device__ __forceinline__ Near near_values(float lo, float hi, float band) {
  return Near{order_key(lo - band), order_key(hi + band)};
}

// Finds keys around the k-th largest of a row.  Scores are cut into bins of equal width
// between the smallest and the largest, so that they spread over most of them (the bits
// of a float's key put nearly all keys of a row into a few bins, and finding the border
// by them takes four rounds and more).  The bin of the k-th is cut again as long as it is
// crowded.  (x - a) * inv, rounded, ascends with x, so bins are in order; their edges are
// known to a few 2^-24 of the range and of the largest magnitude, of which 2^-19 is taken.
// Rows with scores that are not finite, or all equal: every key.
//   keys: this block's n, hist: their counts for the first cut (Cut::count); total(p): the
//   sum of *p over the row's CTAs; sync(): waits for them.
struct Cut {
  float lo, hi, inv, slop;
  bool ok;
  __device__ __forceinline__ explicit Cut(const Part& row) : lo(value_of(row.lo)), hi(value_of(row.hi)) {
    slop = fmaxf(fabsf(lo), fabsf(hi)) * (1.f / 524288.f);
    inv = (float)kBins / (hi - lo);
    ok = isfinite(hi - lo) && isfinite(inv);
  }
  __device__ __forceinline__ void count(uint32_t key, int* hist, int& above) const {
    const float t = (value_of(key) - lo) * inv;
    above += t >= (float)(kBins - 1);                       // (with the last bin's)
    if (t >= 0.f && t < (float)(kBins - 1)) atomicAdd(&hist[(int)t], 1);
  }
};
struct Bin {
  float lo, hi;
};
template <typename Total, typename Sync>
__device__ __forceinline__ Bin border_bin(const uint32_t* keys, int n, int k, Cut cut, int above,
                                          SelectShared& sh, Total total, Sync sync) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const float bottom = cut.lo, top = cut.hi;
  for (int pass = 0;; ++pass) {
    above = __reduce_add_sync(0xffffffffu, above);
    if (lane == 0 && above > 0) atomicAdd(&sh.hist[kBins - 1], above);
    // sums of 64 bins first, so that little is read from other CTAs
    __syncthreads();
    for (int i = warp; i < 32; i += nw) {
      const int c = __reduce_add_sync(0xffffffffu, sh.hist[i * 64 + lane] + sh.hist[i * 64 + 32 + lane]);
      if (lane == 0) sh.coarse[i] = c;
    }
    sync();
    if (warp == 0) {
      // the l-th of 32 counts from the top in lane l: the one that the k-th lies in
      int left = k;
      auto find = [&](int count) {
        int incl = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const int f = (__ffs(__ballot_sync(0xffffffffu, incl >= left)) - 1) & 31;
        left -= __shfl_sync(0xffffffffu, incl - count, f);
        return f;
      };
      const int from = (31 - find(total(&sh.coarse[31 - lane]))) * 64;
      const int c1 = total(&sh.hist[from + 63 - 2 * lane]), c0 = total(&sh.hist[from + 62 - 2 * lane]);
      const int f = find(c0 + c1);
      if (lane == f) {
        const bool upper = c1 >= left;
        sh.bin = from + 63 - 2 * f - (upper ? 0 : 1);
        sh.count = upper ? c1 : c0;
      }
    }
    __syncthreads();
    const int bin = sh.bin;
    const float width = 1.f / cut.inv, from = cut.lo;
    cut.lo = fmaxf(bottom, fmaf((float)bin, width, from) - cut.slop);
    cut.hi = bin == kBins - 1 ? top : fminf(top, fmaf((float)(bin + 1), width, from) + cut.slop);
    cut.inv = (float)kBins / (cut.hi - cut.lo);
    if (sh.count <= kCrowd || pass == kPasses - 1 || cut.hi - cut.lo < 8.f * cut.slop || !isfinite(cut.inv))
      return Bin{cut.lo, cut.hi};
    sync();                                                 // (the counts have been read)
    for (int i = tid; i < kBins; i += nt) sh.hist[i] = 0;
    __syncthreads();
    above = 0;
    for (int i = tid; i < n; i += nt) cut.count(keys[i], sh.hist, above);
  }
}

}  // namespace

// The selection of one row by C CTAs, CTA r having its r-th slice.  FAR: the keys of a
// slice do not fit shared memory and go to `far_keys`.
template <int D, int C, bool FAR>
__device__ __forceinline__ void select_row(const Kv8RetrieveArgs& a, const Query8<D>* rows, const float* __restrict__ scores,
                                           const Parts& parts, uint64_t* __restrict__ exact_rows,
                                           uint32_t* __restrict__ far_keys) {
  extern __shared__ __align__(16) uint32_t staged[];
  __shared__ SelectShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = C > 1 ? (int)cluster.block_rank() : 0, row = blockIdx.x / C, b = row / a.Hkv, g = row - b * a.Hkv;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  auto sync = [&] {
    if constexpr (C > 1) cluster.sync();
    else __syncthreads();
  };
  auto total = [&](const int* p) {
    if constexpr (C == 1) return *p;
    int sum = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) sum += *cluster.map_shared_rank(p, r);
    return sum;
  };
  if (tid == 0) sh.sure = sh.near = sh.clear = sh.n_inside = sh.kept = sh.top = 0;
  for (int i = tid; i < kBins; i += nt) sh.hist[i] = 0;
  // The lengths are read before the wait for the scores: that kernel writes none, and
  // let this one begin only when those before it had completed.
  // As the scoring takes them, the text's among them: a sequence with one out of range
  // has no page in the line, and nothing here may look for its scores.
  int n, nt_text, k;
  seq_lengths(a.lens, b, a.n_vis, a.n_text, a.k, n, nt_text, k);
  if (n > 0 && by_stretches(a)) {
    const int each = stretch_of(a, nw), b0 = warp * each, b1 = min(a.batch, b0 + each);
    if (b >= b0 && b < b1) {
      uint32_t mine;
      const int at = b0 + ((b - b0) & ~31);
      const uint32_t ahead = stretch_pages(a, b0, at, lane), inc = scan_pages(a, at, lane, mine);
      const uint32_t before = ahead + __shfl_sync(0xffffffffu, inc - mine, b - at);
      if (lane == 0) sh.hi[0] = before;                     // (of the stretch)
    }
    const uint32_t sum = stretch_pages(a, b0, b1, lane);
    if (lane == 0) sh.lo[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      uint32_t total = 0, before = sh.hi[0];
      for (int w = 0; w < nw; ++w) {
        total += sh.lo[w];
        before += (w + 1) * each <= b ? sh.lo[w] : 0u;
      }
      sh.by = scorers_of(a, parts, row, n, total, before);
    }
  } else if (n > 0 && warp == 0) {           // (by one warp: it looks at all sequences)
    uint32_t before = 0;
    const uint32_t total = line_of(a, parts, b, lane, before);
    if (lane == 0) sh.by = scorers_of(a, parts, row, n, total, before);
  }
  __syncthreads();
  grid_dep_sync();
  int32_t* dst = a.vis_idx + (size_t)row * a.k;
  if (rank == 0) fill_unselected(dst, k, a.k);
  if (k <= 0) return;                        // (the whole cluster)
  const int slice = (n + C - 1) / C, first = min(n, rank * slice), len = min(n, first + slice) - first;
  const float* src = scores + (size_t)row * a.n_vis + first;
  uint32_t* keys = FAR ? far_keys + (size_t)row * a.n_vis + first : staged;
  float x[8];                                // (on their way with the parts)
  auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = i0 + j * nt < len ? __ldcg(src + i0 + j * nt) : 0.f;
  };
  load(tid);
  const Query8<D>* query = rows + row;
  const Part whole = whole_row(parts, row, sh.by, sh);
  const Cut cut(whole);
  int above = 0;
  for (int i0 = tid; i0 < len;) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i0 + j * nt >= len) break;
      const uint32_t key = order_key(x[j]);
      keys[i0 + j * nt] = key;
      if (cut.ok) cut.count(key, sh.hist, above);
    }
    i0 += 8 * nt;
    load(i0);
  }
  const float some = query->slack * kBand * whole.factor;
  // without a band (or with scores that are not finite) the fp32 order decides
  const bool wide = some > 0.f && isfinite(some) && isfinite(value_of(whole.hi) - value_of(whole.lo));
  float band = wide ? some : 0.f;
  Bin bin = {0.f, 0.f};
  if (cut.ok) bin = border_bin(keys, len, k, cut, above, sh, total, sync);
  Near near = cut.ok ? near_values(bin.lo, bin.hi, band) : Near{whole.lo, whole.hi};

  // ---- the tokens next to the border, of every CTA
  int sure, m, their_sure = 0, theirs = 0;                  // (of CTA `lane`)
  auto find_near = [&] {
    int in = 0;
    for (int i0 = tid; i0 < len; i0 += 4 * nt) {
      uint32_t key[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) key[j] = i0 + j * nt < len ? keys[i0 + j * nt] : 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        in += key[j] > near.hi;
        if (key[j] >= near.lo && key[j] <= near.hi) {
          const int to = atomicAdd(&sh.near, 1);
          if (to < kListed) sh.mine[to] = make_uint2(key[j], (uint32_t)(first + i0 + j * nt));
        }
      }
    }
    in = __reduce_add_sync(0xffffffffu, in);
    if (lane == 0 && in > 0) atomicAdd(&sh.sure, in);
    sync();
    if constexpr (C > 1) {
      their_sure = lane < C ? *cluster.map_shared_rank(&sh.sure, lane) : 0;
      theirs = lane < C ? *cluster.map_shared_rank(&sh.near, lane) : 0;
      sure = __reduce_add_sync(0xffffffffu, their_sure);
      m = __reduce_add_sync(0xffffffffu, theirs);
    } else {
      sure = sh.sure;
      m = sh.near;
    }
  };
  find_near();
  if (m > kMany && cut.ok && band > 0.f) {
    // Many.  The k-th score is one of theirs, so only their factors count for the error,
    // not the largest of the row (of a page whose scores lie elsewhere).
    float factor = 0.f;
    for (int i = tid; i < len; i += nt) {
      if (keys[i] < near.lo || keys[i] > near.hi) continue;
      const int page = __ldg(a.block_table + (size_t)b * a.max_blocks + ((first + i) >> 4));
      if (page >= 0 && page < a.num_blocks) factor = fmaxf(factor, fabsf(__ldg(a.scales + ((size_t)page * a.Hkv + g) * 2)));
    }
    factor = warp_max(factor);
    if (lane == 0) atomicMax(&sh.top, __float_as_int(factor));         // (not negative)
    sync();                                                 // (and the counts have been read)
    int top = sh.top;
    if constexpr (C > 1) top = __reduce_max_sync(0xffffffffu, lane < C ? *cluster.map_shared_rank(&sh.top, lane) : 0);
    if (__int_as_float(top) < 0.5f * whole.factor) {
      band = query->slack * kBand * __int_as_float(top);
      near = near_values(bin.lo, bin.hi, band);
      if (tid == 0) sh.sure = sh.near = 0;
      __syncthreads();
      find_near();
    }
  }
  const uint32_t lo = near.lo, hi = near.hi;
  uint2* const all = C > 1 ? sh.all : sh.mine;
  int before = 0;                                           // taken by CTAs of lower rank
  if constexpr (C > 1) {
    before = __reduce_add_sync(0xffffffffu, lane < rank ? their_sure : 0);
    if (m <= kListed && warp < C) {
      const int at = __reduce_add_sync(0xffffffffu, lane < warp ? theirs : 0);
      const int count = __shfl_sync(0xffffffffu, theirs, warp);
      const uint2* from = cluster.map_shared_rank(sh.mine, warp);
      for (int i = lane; i < count; i += 32) all[at + i] = from[i];
    }
    __syncthreads();
  }
  const int need = k - sure;                                // of those m
  const bool listed = m <= kListed;
  auto drop = [&](int i) {
    const int j = (int)all[i].y - first;
    all[i].x = 0u;                                          // (no score's key)
    if (j >= 0 && j < len) keys[j] = 0u;
  };
  if (m > need && listed) {
    if (!wide) {
      // by (score, index)
      for (int i = tid; i < m; i += nt) {
        const uint2 x = all[i];
        const uint64_t v = (uint64_t)x.x << 32 | ~x.y;
        int better = 0;
        for (int o = 0; o < m; ++o) better += ((uint64_t)all[o].x << 32 | ~all[o].y) > v;
        sh.inside[i] = better;
      }
      __syncthreads();
      for (int i = tid; i < m; i += nt)
        if (sh.inside[i] >= need) drop(i);
      __syncthreads();
    } else {
      // the k-th by its fp32 score, then those within the band of it by their exact ones
      for (int i = tid; i < kListed; i += nt) sh.key[i] = i < m ? all[i].x : 0u;
      __syncthreads();
      for (int i = tid; i < m; i += nt) {
        const uint32_t key = sh.key[i];
        int above = 0, equal = 0;
#pragma unroll 4
        for (int o = 0; o < m; o += 4) {
          const uint4 y = *reinterpret_cast<const uint4*>(&sh.key[o]);
          above += (y.x > key) + (y.y > key) + (y.z > key) + (y.w > key);
          equal += (y.x == key) + (y.y == key) + (y.z == key) + (y.w == key);
        }
        if (above < need && need <= above + equal) sh.kth = key;
      }
      __syncthreads();
      const float kth = value_of(sh.kth);
      const Near close = near_values(kth, kth, band);
      for (int i = tid; i < m; i += nt) {
        const uint32_t key = all[i].x;
        if (key > close.hi) atomicAdd(&sh.clear, 1);
        else if (key >= close.lo) sh.inside[atomicAdd(&sh.n_inside, 1)] = i;
        else drop(i);
      }
      __syncthreads();
      const int open = sh.n_inside, wanted = need - sh.clear;
      if (open > wanted) {
        // (a cluster's CTAs share them out)
        for (int i0 = (warp * C + rank) * 4; i0 < ((m + 3) & ~3); i0 += nw * C * 4) {
          const int i = i0 + (lane >> 3);
          const bool on = i < m && all[i].x >= close.lo && all[i].x <= close.hi;
          if (!__any_sync(0xffffffffu, on)) continue;
          const uint64_t v = score48<D>(a, query, b, g, on ? (int)all[i].y : 0, on, lane);
          if (on && (lane & 7) < C) (C > 1 ? cluster.map_shared_rank(sh.exact, lane & 7) : sh.exact)[i] = v;
        }
        sync();
        for (int t = tid; t < open; t += nt) {
          const int i = sh.inside[t];
          const uint64_t v = sh.exact[i];
          const uint32_t j = all[i].y;
          int better = 0;
#pragma unroll 4
          for (int o = 0; o < open; ++o) {
            const int e = sh.inside[o];
            const uint64_t y = sh.exact[e];
            better += (y > v) | ((y == v) & (all[e].y < j));
          }
          if (better >= wanted) drop(i);                    // (no key is read here)
        }
        __syncthreads();
      }
    }
  } else if (m > need) {
    // too many to list: a radix selection over the 96 bits of (value, ~index)
    uint64_t* exact = exact_rows + (size_t)row * a.n_vis + first;
    for (int i0 = warp * 32; i0 < len; i0 += nt) {
      const uint32_t key = i0 + lane < len ? keys[i0 + lane] : 0u;
      uint32_t todo = __ballot_sync(0xffffffffu, i0 + lane < len && key >= lo && key <= hi);
      while (todo) {
        // four of them at a time
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
    // two histograms in turn (a cluster's CTAs read one pass's while the next fills the other)
    int* sums = sh.hist + 512;
    for (int i = tid; i < 256; i += nt) sh.hist[i] = 0;
    unsigned long long top = 0;
    uint32_t low = 0;
    int left = need;
    sync();
    for (int pass = 0; pass < 12; ++pass) {
      int* hist = sh.hist + (pass & 1) * 256;
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
      sync();
      for (int i = tid; i < 256; i += nt) {
        sums[i] = total(hist + i);
        sh.hist[((pass + 1) & 1) * 256 + i] = 0;
      }
      __syncthreads();
      if (tid == 0) {
        int sum = 0, d = 255;
        while (d > 0 && sum + sums[d] < left) sum += sums[d--];
        sh.bin = d;
        sh.count = sum;
      }
      __syncthreads();
      left -= sh.count;
      if (pass < 8) top |= (unsigned long long)sh.bin << (56 - 8 * pass);
      else low |= (uint32_t)sh.bin << (24 - 8 * (pass - 8));
      __syncthreads();
    }
    for (int i = tid; i < len; i += nt) {
      const uint32_t key = keys[i];
      if (key < lo || key > hi) continue;
      const uint64_t v = exact[i];
      if (v < top || (v == top && first + i > (int)~low)) keys[i] = 0u;
      else atomicAdd(&sh.kept, 1);
    }
    sync();
    if constexpr (C > 1)
      before += __reduce_add_sync(0xffffffffu, lane < rank ? *cluster.map_shared_rank(&sh.kept, lane) : 0);
  }
  if constexpr (C > 1) {
    if (listed) {
      // (in order of their CTAs' ranks, so those before this one's have lower indices)
      int kept = 0;
      for (int i = lane; i < m; i += 32) kept += all[i].x != 0u && (int)all[i].y < first;
      before += __reduce_add_sync(0xffffffffu, kept);
    } else if (m <= need) {
      before += __reduce_add_sync(0xffffffffu, lane < rank ? theirs : 0);   // (all of them are taken)
    }
  }

  // ---- the indices of the keys that are left, ascending: stretches of 32 to a warp
  const int per = ((len + 31) / 32 + nw - 1) / nw * 32, w0 = min(len, warp * per), w1 = min(len, w0 + per);
  auto taken = [&](int i) { return i < w1 && keys[i] >= lo; };
  uint32_t count = 0;
#pragma unroll 4
  for (int i0 = w0; i0 < w1; i0 += 32) count += __popc(__ballot_sync(0xffffffffu, taken(i0 + lane)));
  if (lane == 0) sh.scan[warp] = count;
  __syncthreads();
  uint32_t o = (uint32_t)before + __reduce_add_sync(0xffffffffu, lane < warp ? sh.scan[lane] : 0u);
#pragma unroll 4
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const bool take = taken(i0 + lane);
    const uint32_t mask = __ballot_sync(0xffffffffu, take);
    if (take) dst[o + __popc(mask & ((1u << lane) - 1u))] = first + i0 + lane;
    o += __popc(mask);
  }
  if constexpr (C > 1) cluster.sync();     // (this CTA's shared memory has been read)
}

template <int D>
__global__ void __launch_bounds__(kClusterThreads, 2)
kv8_select_kernel(const __grid_constant__ Kv8RetrieveArgs a, const Query8<D>* rows, const float* __restrict__ scores,
                  const Parts parts, uint64_t* __restrict__ exact, uint32_t* __restrict__ far_keys) {
  select_row<D, 1, false>(a, rows, scores, parts, exact, far_keys);
}
template <int D, bool FAR>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kClusterThreads, 2)
kv8_select_cluster_kernel(const __grid_constant__ Kv8RetrieveArgs a, const Query8<D>* rows,
                          const float* __restrict__ scores, const Parts parts, uint64_t* __restrict__ exact,
                          uint32_t* __restrict__ far_keys) {
  select_row<D, kCluster, FAR>(a, rows, scores, parts, exact, far_keys);
}

// Workspace: queries | 48-bit scores of tokens next to a crowded border | fp32
// scores | what each scoring warp leaves | keys of rows that are
// too long for shared memory
constexpr int kMostCtas = 1024;          // (of 152 SMs: 760)
static bool fits_cluster(int n) { return (n + kCluster - 1) / kCluster <= kSliceKeys; }
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
size_t kv8_retrieve_workspace_bytes(int B, int Hkv, int D, int n_vis) {
  const size_t rows = (size_t)B * Hkv;
  return up256(rows * (D == 128 ? sizeof(Query8<128>) : sizeof(Query8<64>))) + up256(rows * n_vis * sizeof(uint64_t)) +
         up256(rows * kScoreWarps * sizeof(Part)) + up256(kMostCtas * 2 * kScoreWarps * sizeof(Part)) +
         up256(rows * n_vis * sizeof(float)) * (n_vis > kStagedKeys && !fits_cluster(n_vis) ? 2 : 1);
}

// `kernel`: of C CTAs a row, with `most` keys in shared memory at most
template <typename Kernel, typename... Args>
static cudaError_t launch_select(Kernel kernel, bool (&attr_set)[64], int C, int most, const Kv8RetrieveArgs& a,
                                 cudaStream_t stream, Args... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (most > 0 && (dev < 0 || dev >= 64 || !attr_set[dev])) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most * 4);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  // (256 / 512 threads: 512 rows of 2880 keys 44.6 / 50.3 us, of 5000 75.1 / 76.6, of 8200
  // 123.6 / 114.4; 4 rows 12.2 / 11.8, 15.4 / 15.0, 19.2 / 18.1)
  const int threads = C > 1 || a.n_vis >= 8192 ? kClusterThreads : 256;
  const size_t smem = most > 0 ? (size_t)((a.n_vis + C - 1) / C) * 4 : 0;
  return launch_dependent(kernel, dim3((unsigned)(C * a.batch * a.Hkv)), dim3(threads), smem, stream, a, args...);
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
  Parts parts;
  parts.pages = (a.n_vis + 15) / 16;
  const long long pages = (long long)parts.pages * rows;
  parts.ctas = (int)std::min<long long>(std::min(num_sms * kScoreCtas, kMostCtas), (pages + kScoreWarps - 1) / kScoreWarps);
  parts.whole = reinterpret_cast<Part*>(take((size_t)rows * kScoreWarps * sizeof(Part)));
  parts.cut = reinterpret_cast<Part*>(take((size_t)kMostCtas * 2 * kScoreWarps * sizeof(Part)));
  uint32_t* far_keys = reinterpret_cast<uint32_t*>(at);      // (there where it is used)
  if (a.scores != nullptr) scores = a.scores;
  const bool sum = (long long)a.R * (a.H / a.Hkv) <= kFusedRows;
  // (Query rows for one key row by a CTA / by a cluster, whole calls of 576 keys: 256 rows
  // 12.3 / 13.1 us, 496 13.6 / 12.4, 1351 29.7 / 13.3, 16000 227 / 30.  Where key rows are
  // many the clusters queue: 32 key rows of 512 16.9 / 25.3, of 2048 31.3 / 27.0; 128 of 512
  // 25.4 / 60.5, of 2048 58.7 / 65.7.)
  const bool wide = (long long)a.R * (a.H / a.Hkv) >= 512 && rows <= num_sms;
  cudaError_t e = cudaSuccess;
  if (!sum)
    e = wide ? launch_dependent(kv8_qbar_cluster_kernel<D>, dim3(kSumCtas * rows), dim3(kSumWarps * 32), 0, stream,
                                static_cast<const uint16_t*>(a.q), a.R, a.H, a.Hkv, query)
             : launch_dependent(kv8_qbar_kernel<D>, dim3(rows), dim3(kSumWarps * 32), 0, stream,
                                static_cast<const uint16_t*>(a.q), a.R, a.H, a.Hkv, query);
  if (e != cudaSuccess) return e;
  e = launch_dependent(sum ? kv8_score_kernel<D, true> : kv8_score_kernel<D, false>, dim3((unsigned)parts.ctas),
                       dim3(kScoreWarps * 32), 0, stream, a, query, scores, parts);
  if (e != cudaSuccess) return e;
  // a CTA per row as long as rows are short, else a cluster
  static bool set[3][64] = {};
  if (a.n_vis <= kStagedKeys)
    return launch_select(kv8_select_kernel<D>, set[0], 1, kStagedKeys, a, stream, query, scores, parts, exact, far_keys);
  if (fits_cluster(a.n_vis))
    return launch_select(kv8_select_cluster_kernel<D, false>, set[1], kCluster, kSliceKeys, a, stream, query, scores, parts,
                         exact, far_keys);
  return launch_select(kv8_select_cluster_kernel<D, true>, set[2], kCluster, 0, a, stream, query, scores, parts, exact,
                       far_keys);
}

cudaError_t launch_kv8_retrieve(const Kv8RetrieveArgs& a, int D, int num_sms, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, num_sms, stream) : launch_d<64>(a, num_sms, stream);
}

}  // namespace sv
