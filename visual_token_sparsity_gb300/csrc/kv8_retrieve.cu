// Query-aware retrieval from the 8-bit cache: scores of the cached visual keys
// and the selection of the k largest.
//
//   qbar = sum of the query rows and the group's heads
//   score_j = s_k[page(j)] * qbar . K8[j]            (as retrieve.cu)
//
// The selection is that of the exact scores.  The fp32 scores order all but the
// tokens next to the k-th one: with an error of at most e each, the k-th largest
// score is within e of the true one, so a token more than 2 e above it is in
// and one more than 2 e below it is out.  Those in between are scored again in
// 64 bits (where the products of 8-bit keys and sums of bf16 queries lose
// nothing in practice) and the best of them taken, ties to the lower index.
#include "kernels.h"
#include "kv8.cuh"
#include "topk_block.cuh"

namespace sv {

namespace {

constexpr int kScoreThreads = 256;
// |fp32 score - score| <= e = 67 * 2^-24 |qbar|_1 448 s: one rounding of each
// qbar element, at most 64 of a chain of products, one of the sum of two chains
// and one of the factor s; 448 s bounds a key's elements.  Twice that, and the
// roundings of the bound itself:
constexpr float kBand = 1.f / 65536.f;
constexpr int kListed = 1024;      // candidates that are ranked in shared memory

__device__ __forceinline__ uint64_t order_key64(double x) {
  const uint64_t f = (uint64_t)__double_as_longlong(x + 0.0);   // (-0 to 0)
  return (f >> 63) ? ~f : (f | 0x8000000000000000ull);
}

struct Row8 {       // of one (sequence, KV head)
  float l1;         // sum of |qbar|
  uint32_t top;     // largest factor of the pages that were scored (fp32 bits)
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(D)
kv8_qbar_kernel(const uint16_t* __restrict__ q, int R, int H, int Hkv, double* __restrict__ qbar, Row8* rows) {
  __shared__ float part[D / 32];
  grid_dep_sync();
  const int row = blockIdx.x, b = row / Hkv, g = row - b * Hkv, G = H / Hkv, e = threadIdx.x;
  double acc = 0.0;
  for (int r = 0; r < R; ++r) {
    const uint16_t* src = q + (((size_t)b * R + r) * H + (size_t)g * G) * D + e;
    for (int h = 0; h < G; ++h) acc += (double)__uint_as_float((uint32_t)src[(size_t)h * D] << 16);
  }
  qbar[(size_t)row * D + e] = acc;
  const float s = warp_sum(fabsf((float)acc));
  if ((e & 31) == 0) part[e >> 5] = s;
  __syncthreads();
  if (e == 0) {
    float l1 = 0.f;
    for (int i = 0; i < D / 32; ++i) l1 += part[i];
    rows[row] = Row8{l1, 0u};
  }
}

// A warp per page: two lanes a token.
template <int D>
__global__ void __launch_bounds__(kScoreThreads)
kv8_score_kernel(const __grid_constant__ Kv8RetrieveArgs a, const double* __restrict__ qbar, Row8* rows,
                 float* __restrict__ scores, int pages_per_cta) {
  __shared__ float qs[D];
  grid_dep_sync();
  const int g = blockIdx.y, b = blockIdx.z, row = b * a.Hkv + g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int nv, nt, kb;
  if (!seq_lengths(a.lens, b, a.n_vis, a.n_text, a.k, nv, nt, kb) && threadIdx.x == 0 && blockIdx.x == 0)
    flag_status(a.status, kStatusBadLength);
  for (int e = threadIdx.x; e < D; e += kScoreThreads) qs[e] = (float)qbar[(size_t)row * D + e];
  __syncthreads();
  const int end = min((nv + 15) / 16, ((int)blockIdx.x + 1) * pages_per_cta);
  uint32_t top = 0;
  for (int p = blockIdx.x * pages_per_cta + warp; p < end; p += kScoreThreads / 32) {
    const int page = __ldg(a.block_table + (size_t)b * a.max_blocks + p);
    const bool ok = page >= 0 && page < a.num_blocks;
    if (!ok && lane == 0) flag_status(a.status, kStatusBadBlock);
    const size_t unit = (size_t)(ok ? page : 0) * a.Hkv + g;
    const float s = __ldg(a.scales + unit * 2);
    float dot = 0.f;
    if (ok) {
      top = max(top, __float_as_uint(fabsf(s)));
      const uint4* src = reinterpret_cast<const uint4*>(a.k_pool + (unit * 16 + (lane >> 1)) * D + (lane & 1) * (D / 2));
      const float* qe = qs + (lane & 1) * (D / 2);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint4 v = __ldg(src + c);
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 lo = kv8::e4m3x2_to_float2((uint16_t)w[e]), hi = kv8::e4m3x2_to_float2((uint16_t)(w[e] >> 16));
          dot = fmaf(qe[16 * c + 4 * e], lo.x, dot);
          dot = fmaf(qe[16 * c + 4 * e + 1], lo.y, dot);
          dot = fmaf(qe[16 * c + 4 * e + 2], hi.x, dot);
          dot = fmaf(qe[16 * c + 4 * e + 3], hi.y, dot);
        }
      }
    }
    dot += __shfl_xor_sync(0xffffffffu, dot, 1);
    const int pos = p * 16 + (lane >> 1);
    if ((lane & 1) == 0 && pos < nv) scores[(size_t)row * a.n_vis + pos] = ok ? dot * s : 0.f;
  }
  if (lane == 0 && top != 0) atomicMax(&rows[row].top, top);   // (a maximum: the order does not matter)
}

// The tokens next to the k-th score, decided in 64 bits.
template <int D>
__global__ void __launch_bounds__(512)
kv8_border_kernel(const __grid_constant__ Kv8RetrieveArgs a, const double* __restrict__ qbar, const Row8* rows,
                  const float* __restrict__ scores, double* __restrict__ exact) {
  __shared__ float red[16];
  __shared__ int count[2];                 // surely in, next to the border
  __shared__ int listed;
  __shared__ double list_v[kListed];
  __shared__ int list_j[kListed];
  __shared__ unsigned long long sel_key;
  __shared__ int sel_j;
  __shared__ int hist[256];
  __shared__ int digit, above;
  __shared__ uint32_t scan_tmp[33];
  grid_dep_sync();
  const int row = blockIdx.x, b = row / a.Hkv, g = row - b * a.Hkv;
  const int tid = threadIdx.x, nt_ = blockDim.x, lane = tid & 31, warp = tid >> 5;
  int n = a.n_vis, k = a.k;
  if (a.lens.any()) row_lengths(a.lens, row, a.Hkv, a.n_vis, a.k, n, k);
  if (k <= 0 || k >= n) return;            // nothing, or everything, is selected
  const float* sc = scores + (size_t)row * a.n_vis;
  int32_t* dst = a.vis_idx + (size_t)row * a.k;
  double* ex = exact + (size_t)row * a.n_vis;
  const Row8 r8 = rows[row];
  const float band = r8.l1 * (448.f * kBand) * __uint_as_float(r8.top);
  if (!(band > 0.f) || !isfinite(band)) return;

  // the k-th largest fp32 score
  float kth = INFINITY;
  for (int i = tid; i < k; i += nt_) kth = fminf(kth, __ldcg(sc + __ldcg(dst + i)));
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) kth = fminf(kth, __shfl_xor_sync(0xffffffffu, kth, o));
  if (lane == 0) red[warp] = kth;
  if (tid < 2) count[tid] = 0;
  if (tid == 2) listed = 0;
  __syncthreads();
  kth = red[0];
  for (int w = 1; w < nt_ / 32; ++w) kth = fminf(kth, red[w]);
  const float hi = kth + band, lo = kth - band;
  auto sure = [&](float s) { return s > hi; };
  auto near = [&](float s) { return s >= lo && s <= hi; };

  int in = 0, at = 0;
  for (int i = tid; i < n; i += nt_) {
    const float s = __ldcg(sc + i);
    in += sure(s);
    at += near(s);
  }
  in = __reduce_add_sync(0xffffffffu, in);
  at = __reduce_add_sync(0xffffffffu, at);
  if (lane == 0) {
    atomicAdd(&count[0], in);
    atomicAdd(&count[1], at);
  }
  __syncthreads();
  const int need = k - count[0], m = count[1];
  if (need <= 0 || m <= need) return;       // (m < need: scores that are not finite; the fp32 choice stays)

  // their scores in 64 bits, a warp each
  for (int i0 = warp * 32; i0 < n; i0 += nt_) {
    const float s = i0 + lane < n ? __ldcg(sc + i0 + lane) : -INFINITY;
    uint32_t todo = __ballot_sync(0xffffffffu, near(s));
    while (todo) {
      const int j = i0 + __ffs(todo) - 1;
      todo &= todo - 1;
      const int page = __ldg(a.block_table + (size_t)b * a.max_blocks + (j >> 4));
      double v = 0.0;
      if (page >= 0 && page < a.num_blocks) {
        const size_t unit = (size_t)page * a.Hkv + g;
        const uint8_t* src = a.k_pool + (unit * 16 + (j & 15)) * D;
#pragma unroll
        for (int e = 0; e < D; e += 64) {
          const float2 x = kv8::e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(src + e + 2 * lane));
          const double* qe = qbar + (size_t)row * D + e + 2 * lane;
          v += qe[0] * (double)x.x + qe[1] * (double)x.y;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        v *= (double)__ldg(a.scales + unit * 2);
      }
      if (lane == 0) {
        ex[j] = v;
        if (m <= kListed) {
          const int at_list = atomicAdd(&listed, 1);
          list_v[at_list] = v;
          list_j[at_list] = j;
        }
      }
    }
  }
  __syncthreads();
  // the last one that is taken: by value, then by index
  if (m <= kListed) {
    for (int i = tid; i < m; i += nt_) {
      const double v = list_v[i];
      const int j = list_j[i];
      int better = 0;
      for (int o = 0; o < m; ++o) better += list_v[o] > v || (list_v[o] == v && list_j[o] < j);
      if (better == need - 1) {
        sel_key = order_key64(v);
        sel_j = j;
      }
    }
  } else {
    // a radix selection over the 96 bits of (value, ~index)
    unsigned long long key = 0;
    uint32_t low = 0;
    int left = need;
    for (int pass = 0; pass < 12; ++pass) {
      for (int i = tid; i < 256; i += nt_) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += nt_) {
        if (!near(__ldcg(sc + i))) continue;
        const uint64_t kv = order_key64(ex[i]);
        const uint32_t ki = ~(uint32_t)i;
        if (pass < 8) {
          if (pass > 0 && (kv ^ key) >> (64 - 8 * pass)) continue;
          atomicAdd(&hist[(kv >> (56 - 8 * pass)) & 255], 1);
        } else {
          if (kv != key || (pass > 8 && (ki ^ low) >> (32 - 8 * (pass - 8)))) continue;
          atomicAdd(&hist[(ki >> (24 - 8 * (pass - 8))) & 255], 1);
        }
      }
      __syncthreads();
      if (tid == 0) {
        int sum = 0, d = 255;
        while (sum + hist[d] < left) sum += hist[d--];
        digit = d;
        above = sum;
      }
      __syncthreads();
      left -= above;
      if (pass < 8) key |= (unsigned long long)digit << (56 - 8 * pass);
      else low |= (uint32_t)digit << (24 - 8 * (pass - 8));
      __syncthreads();
    }
    if (tid == 0) {
      sel_key = key;
      sel_j = (int)~low;
    }
  }
  __syncthreads();
  const uint64_t last = sel_key;
  const int last_j = sel_j;
  auto taken = [&](int i, float s) {
    if (!near(s)) return sure(s);
    const uint64_t v = order_key64(ex[i]);
    return v > last || (v == last && i <= last_j);
  };
  // the indices in ascending order
  const int seg = (n + nt_ - 1) / nt_, s0 = min(n, tid * seg), s1 = min(n, s0 + seg);
  uint32_t mine = 0;
  for (int i = s0; i < s1; ++i) mine += taken(i, __ldcg(sc + i));
  uint32_t o = block_exclusive_scan<uint32_t>(mine, scan_tmp);
  for (int i = s0; i < s1; ++i)
    if (taken(i, __ldcg(sc + i))) dst[o++] = i;
}

// Workspace: qbar | rows | 64-bit scores of the tokens next to the border | fp32 scores
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
size_t kv8_retrieve_workspace_bytes(int B, int Hkv, int D, int n_vis) {
  const size_t rows = (size_t)B * Hkv;
  return up256(rows * D * sizeof(double)) + up256(rows * sizeof(Row8)) + up256(rows * n_vis * sizeof(double)) +
         up256(rows * n_vis * sizeof(float));
}

template <int D>
static cudaError_t launch_d(const Kv8RetrieveArgs& a, int num_sms, cudaStream_t stream) {
  const int rows = a.batch * a.Hkv;
  char* ws = static_cast<char*>(a.ws);
  double* qbar = reinterpret_cast<double*>(ws);
  Row8* r8 = reinterpret_cast<Row8*>(ws + up256((size_t)rows * D * sizeof(double)));
  double* exact = reinterpret_cast<double*>(reinterpret_cast<char*>(r8) + up256(rows * sizeof(Row8)));
  float* scores = a.scores != nullptr ? a.scores
                                      : reinterpret_cast<float*>(reinterpret_cast<char*>(exact) +
                                                                 up256((size_t)rows * a.n_vis * sizeof(double)));
  cudaError_t e = launch_dependent(kv8_qbar_kernel<D>, dim3(rows), dim3(D), 0, stream,
                                   static_cast<const uint16_t*>(a.q), a.R, a.H, a.Hkv, qbar, r8);
  if (e != cudaSuccess) return e;
  const int pages = (a.n_vis + 15) / 16;
  long long per = ((long long)pages * rows + num_sms * 16 - 1) / (num_sms * 16);
  per = (per + 7) / 8 * 8;
  if (per > pages) per = pages;
  e = launch_dependent(kv8_score_kernel<D>, dim3((unsigned)((pages + per - 1) / per), a.Hkv, a.batch),
                       dim3(kScoreThreads), 0, stream, a, qbar, r8, scores, (int)per);
  if (e != cudaSuccess) return e;
  e = topk_prefers_cluster(a.n_vis)
          ? launch_topk_cluster(scores, rows, a.n_vis, a.k, a.vis_idx, stream, a.lens, a.Hkv)
          : launch_topk_rows(scores, rows, a.n_vis, a.k, a.vis_idx, stream, a.lens, a.Hkv);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv8_border_kernel<D>, dim3(rows), dim3(a.n_vis > 8192 ? 512 : 256), 0, stream, a, qbar, r8,
                          scores, exact);
}

cudaError_t launch_kv8_retrieve(const Kv8RetrieveArgs& a, int D, int num_sms, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, num_sms, stream) : launch_d<64>(a, num_sms, stream);
}

}  // namespace sv
