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
#include "topk_block.cuh"

namespace sv {

namespace {

constexpr int kScoreWarps = 8;
// |fp32 score - score| <= e = 137 * 2^-24 |qbar|_1 448 s: eight tiles of 17 terms,
// each of which loses at most the last of 24 bits beside the largest, and the
// rounding of the sum times s; 448 s bounds a key's elements.  2 e, rounded up:
constexpr float kBand = 1.f / 32768.f;
constexpr int kListed = 1024;            // tokens next to the border that are ranked in shared memory
constexpr int kStagedKeys = 52 * 1024;   // keys in shared memory

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

__device__ __forceinline__ uint64_t order_key64(double x) {
  const uint64_t f = (uint64_t)__double_as_longlong(x + 0.0);   // (-0 to 0)
  return (f >> 63) ? ~f : (f | 0x8000000000000000ull);
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
  float back[2], l1;     // 2^e in two factors, sum of |qbar|
  uint32_t top;          // largest factor of the pages that were scored (fp32 bits)
  uint32_t pad[12];
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(D)
kv8_qbar_kernel(const uint16_t* __restrict__ q, int R, int H, int Hkv, Query8<D>* rows) {
  __shared__ float part[2][D / 32];
  grid_dep_sync();
  const int row = blockIdx.x, b = row / Hkv, g = row - b * Hkv, G = H / Hkv, e = threadIdx.x;
  float hi = 0.f, lo = 0.f;
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
  const float a = fabsf(hi);
  float s = warp_sum(a), top = warp_max(a);
  if ((e & 31) == 0) {
    part[0][e >> 5] = s;
    part[1][e >> 5] = top;
  }
  __syncthreads();
  s = 0.f;
  top = 0.f;
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
  Query8<D>* o = rows + row;
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
    o->l1 = s;
    o->top = 0u;
  }
}

// A warp per page, two pages in flight.
template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32, 4)
kv8_score_kernel(const __grid_constant__ Kv8RetrieveArgs a, Query8<D>* rows, float* __restrict__ scores,
                 int pages_per_cta) {
  constexpr int KS = D / 16, KC = D / 64;
  grid_dep_sync();
  const int g = blockIdx.y, b = blockIdx.z, row = b * a.Hkv + g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, q4 = lane & 3;
  int nv, nt, kb;
  if (!seq_lengths(a.lens, b, a.n_vis, a.n_text, a.k, nv, nt, kb) && threadIdx.x == 0 && blockIdx.x == 0)
    flag_status(a.status, kStatusBadLength);
  const int end = min((nv + 15) / 16, ((int)blockIdx.x + 1) * pages_per_cta);
  const int first = blockIdx.x * pages_per_cta + warp;
  if (first >= end) return;
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;

  struct Page {
    uint4 k[2][KC];        // keys r and r + 8
    float s;
    bool ok;
  };
  auto load = [&](int p, Page& x) {
    x.ok = false;
    if (p >= end) return;
    const int page = __ldg(bt + p);
    x.ok = page >= 0 && page < a.num_blocks;
    if (!x.ok) {
      if (lane == 0) flag_status(a.status, kStatusBadBlock);
      return;
    }
    const size_t unit = (size_t)page * a.Hkv + g;
    const uint8_t* src = a.k_pool + (unit * 16 + r) * D + q4 * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < KC; ++c) x.k[i][c] = ld_stream16(src + i * 8 * D + c * 64);
    x.s = __ldg(a.scales + unit * 2);
  };
  Page x, y;
  load(first, x);
  // (the query's parts: column r of a tile is part r, the columns behind are 0)
  uint32_t qf[KS][2];
  const Query8<D>* query = rows + row;
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const uint2 p = __ldg(reinterpret_cast<const uint2*>(&query->part[min(r, 3)][(k >> 2) * 64 + q4 * 16 + (k & 3) * 4]));
    qf[k][0] = p.x;
    qf[k][1] = p.y;
  }
  const float back0 = query->back[0], back1 = query->back[1];
  uint32_t top = 0;
  float* out = scores + (size_t)row * a.n_vis;
  auto score = [&](int p, const Page& x) {
    float c[2][4] = {};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&x.k[0][k >> 2]);
      const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&x.k[1][k >> 2]);
      const uint32_t y0 = w0[k & 3], y1 = w1[k & 3];
      mma_f16(c[k & 1], kv8::e4m3x2_to_half2((uint16_t)y0), kv8::e4m3x2_to_half2((uint16_t)y1),
              kv8::e4m3x2_to_half2((uint16_t)(y0 >> 16)), kv8::e4m3x2_to_half2((uint16_t)(y1 >> 16)), qf[k][0], qf[k][1]);
    }
    // columns 0 and 1 are lane 4 r's, column 2 is its neighbour's
    const float z0 = __shfl_down_sync(0xffffffffu, c[0][0] + c[1][0], 1), z1 = __shfl_down_sync(0xffffffffu, c[0][2] + c[1][2], 1);
    const float s0 = (c[0][0] + c[1][0]) + ((c[0][1] + c[1][1]) + z0), s1 = (c[0][2] + c[1][2]) + ((c[0][3] + c[1][3]) + z1);
    const int pos = p * 16 + r;
    if (q4 == 0) {
      // (NaN without a sign, so that its key is the largest)
      auto value = [&](float v) {
        v = (v * back0) * (x.s * back1);
        return !x.ok ? 0.f : isnan(v) ? __uint_as_float(0x7fffffffu) : v;
      };
      if (pos < nv) out[pos] = value(s0);
      if (pos + 8 < nv) out[pos + 8] = value(s1);
    }
    if (x.ok) top = max(top, __float_as_uint(fabsf(x.s)));
  };
  for (int p = first; p < end; p += 2 * kScoreWarps) {
    load(p + kScoreWarps, y);
    score(p, x);
    load(p + 2 * kScoreWarps, x);
    if (p + kScoreWarps < end) score(p + kScoreWarps, y);
  }
  if (lane == 0 && top != 0) atomicMax(&rows[row].top, top);   // (a maximum: the order does not matter)
}

namespace {

struct BorderShared {
  double list_v[kListed];
  int list_j[kListed];
  int sure, near, listed, digit, above, last_j;
  unsigned long long last;
  uint32_t kth[32];
  uint32_t scan_tmp[33];
  int hist[256];
};

// The score of token j with 48 bits, by eight lanes (lane % 8 == 0 has it).
template <int D>
__device__ __forceinline__ double score48(const Kv8RetrieveArgs& a, const Query8<D>* query, int b, int g, int j, bool on,
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
  return ((double)hi + (double)lo) * (double)s;
}

// Selects the k tokens of a row, given its keys (in shared memory) and the k-th
// largest of them.  All threads of the block call this.
template <int D>
__device__ __forceinline__ void select_row(const Kv8RetrieveArgs& a, const Query8<D>* query, int b, int g, int n, int k,
                                           uint32_t* keys, uint32_t kth, double* exact, int32_t* dst, BorderShared& sh) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const float at = (kth & 0x80000000u) ? __uint_as_float(kth ^ 0x80000000u) : __uint_as_float(~kth);
  const float band = query->l1 * (448.f * kBand) * __uint_as_float(query->top);
  // (scores or a band that are not finite: the fp32 order, ties included)
  const bool wide = band > 0.f && isfinite(band) && isfinite(at);
  const uint32_t hi = wide ? order_key(at + band) : kth, lo = wide ? order_key(at - band) : kth;
  if (tid == 0) sh.sure = sh.near = sh.listed = 0;
  __syncthreads();
  int in = 0, by = 0;
  for (int i = tid; i < n; i += nt) {
    const uint32_t key = keys[i];
    in += key > hi;
    by += key >= lo && key <= hi;
  }
  in = __reduce_add_sync(0xffffffffu, in);
  by = __reduce_add_sync(0xffffffffu, by);
  if (lane == 0) {
    atomicAdd(&sh.sure, in);
    atomicAdd(&sh.near, by);
  }
  __syncthreads();
  const int need = k - sh.sure, m = sh.near;     // of the m tokens next to the border
  bool by_value = false;                         // taken by (value, index), not all
  if (m > need) {
    const bool listed = m <= kListed;
    by_value = !listed;
    if (listed) {
      for (int i = tid; i < n; i += nt) {
        const uint32_t key = keys[i];
        if (key >= lo && key <= hi) sh.list_j[atomicAdd(&sh.listed, 1)] = i;
      }
      __syncthreads();
      for (int i0 = warp * 4; i0 < m; i0 += nw * 4) {
        const int i = i0 + (lane >> 3);
        const int j = i < m ? sh.list_j[i] : 0;
        // (exact ties of scores that are not told apart at all: by index alone)
        const double v = wide ? score48<D>(a, query, b, g, j, i < m, lane) : 0.0;
        if (i < m && (lane & 7) == 0) sh.list_v[i] = v;
      }
      __syncthreads();
      for (int i = tid; i < m; i += nt) {
        const double v = sh.list_v[i];
        const int j = sh.list_j[i];
        int better = 0;
        for (int o = 0; o < m; ++o) better += sh.list_v[o] > v || (sh.list_v[o] == v && sh.list_j[o] < j);
        if (better >= need) keys[j] = 0u;             // (no score's key)
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
          const double v = wide ? score48<D>(a, query, b, g, max(j, 0), j >= 0, lane) : 0.0;
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
          const uint64_t kv = order_key64(exact[i]);
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
    const uint64_t v = order_key64(exact[i]);
    return v > sh.last || (v == sh.last && i <= sh.last_j);
  };
  const int seg = (n + nt - 1) / nt, s0 = min(n, tid * seg), s1 = min(n, s0 + seg);
  uint32_t mine = 0;
  for (int i = s0; i < s1; ++i) mine += taken(i);
  uint32_t o = block_exclusive_scan<uint32_t>(mine, sh.scan_tmp);
  for (int i = s0; i < s1; ++i)
    if (taken(i)) dst[o++] = i;
}

}  // namespace

// The selection of one row per CTA.  KNOWN: a cluster has already taken the k
// largest fp32 scores (vis_idx), and the k-th is their smallest.
template <int D, bool KNOWN>
__global__ void __launch_bounds__(1024)
kv8_select_kernel(const __grid_constant__ Kv8RetrieveArgs a, const Query8<D>* rows, const float* __restrict__ scores,
                  double* __restrict__ exact, uint32_t* __restrict__ far_keys) {
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
  uint32_t* keys = far_keys != nullptr ? far_keys + (size_t)row * a.n_vis : staged;
  if (!KNOWN) fill_unselected(dst, k, a.k);
  if (k <= 0) return;
  uint32_t kth = 0xffffffffu;
  if (KNOWN) {
    for (int i = tid; i < k; i += nt) kth = min(kth, order_key(__ldcg(src + __ldcg(dst + i))));
    for (int i = tid; i < n; i += nt) keys[i] = order_key(__ldcg(src + i));
  } else {
    const TopkBorder t = block_topk_border(src, n, k, keys, ts);
    for (int i = tid; i < n; i += nt) {
      const uint32_t key = keys[i];
      if ((key & t.pmask) >= t.prefix) kth = min(kth, key);
    }
  }
  kth = __reduce_min_sync(0xffffffffu, kth);
  if (lane == 0) sh.kth[warp] = kth;
  __syncthreads();
  for (int w = 0; w < nt / 32; ++w) kth = min(kth, sh.kth[w]);
  select_row<D>(a, rows + row, b, g, n, k, keys, kth, exact + (size_t)row * a.n_vis, dst, sh);
}

// Workspace: queries | 48-bit scores of tokens next to a crowded border | fp32
// scores | keys of rows that are too long for shared memory
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
size_t kv8_retrieve_workspace_bytes(int B, int Hkv, int D, int n_vis) {
  const size_t rows = (size_t)B * Hkv;
  return up256(rows * (D == 128 ? sizeof(Query8<128>) : sizeof(Query8<64>))) + up256(rows * n_vis * sizeof(double)) +
         up256(rows * n_vis * sizeof(float)) * (n_vis > kStagedKeys ? 2 : 1);
}

template <int D, bool KNOWN>
static cudaError_t launch_select(const Kv8RetrieveArgs& a, const Query8<D>* rows, const float* scores, double* exact,
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
  const int threads = a.n_vis >= 16384 ? 1024 : (a.n_vis >= 8192 ? 512 : 256);
  return launch_dependent(kernel, dim3((unsigned)(a.batch * a.Hkv)), dim3(threads),
                          far_keys != nullptr ? (size_t)0 : (size_t)a.n_vis * 4, stream, a, rows, scores, exact, far_keys);
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
  double* exact = reinterpret_cast<double*>(take((size_t)rows * a.n_vis * sizeof(double)));
  float* scores = reinterpret_cast<float*>(take((size_t)rows * a.n_vis * sizeof(float)));
  uint32_t* far_keys = a.n_vis > kStagedKeys ? reinterpret_cast<uint32_t*>(at) : nullptr;
  if (a.scores != nullptr) scores = a.scores;
  cudaError_t e = launch_dependent(kv8_qbar_kernel<D>, dim3(rows), dim3(D), 0, stream,
                                   static_cast<const uint16_t*>(a.q), a.R, a.H, a.Hkv, query);
  if (e != cudaSuccess) return e;
  // pages per CTA: two per warp at a time
  const int pages = (a.n_vis + 15) / 16;
  const long long ctas = (long long)num_sms * 12;
  long long per = ((long long)pages * rows + ctas - 1) / ctas;
  per = (per + 2 * kScoreWarps - 1) / (2 * kScoreWarps) * (2 * kScoreWarps);
  if (per > pages) per = pages;
  e = launch_dependent(kv8_score_kernel<D>, dim3((unsigned)((pages + per - 1) / per), a.Hkv, a.batch),
                       dim3(kScoreWarps * 32), 0, stream, a, query, scores, (int)per);
  if (e != cudaSuccess) return e;
  // (a CTA per row as long as rows are short: as topk_prefers_cluster)
  if (!topk_prefers_cluster(a.n_vis) && far_keys == nullptr)
    return launch_select<D, false>(a, query, scores, exact, nullptr, stream);
  e = topk_prefers_cluster(a.n_vis)
          ? launch_topk_cluster(scores, rows, a.n_vis, a.k, a.vis_idx, stream, a.lens, a.Hkv)
          : launch_topk_rows(scores, rows, a.n_vis, a.k, a.vis_idx, stream, a.lens, a.Hkv);
  if (e != cudaSuccess) return e;
  return launch_select<D, true>(a, query, scores, exact, far_keys, stream);
}

cudaError_t launch_kv8_retrieve(const Kv8RetrieveArgs& a, int D, int num_sms, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, num_sms, stream) : launch_d<64>(a, num_sms, stream);
}

}  // namespace sv
