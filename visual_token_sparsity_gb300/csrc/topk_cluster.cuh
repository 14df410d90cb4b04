// The border of a row's k largest scores, found by a thread-block cluster: CTA r
// holds the r-th slice of the row's order-preserving keys in its shared memory.
// (How the passes exchange histograms stands in topk_cluster.cu.)
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "topk_block.cuh"

namespace sv {

constexpr int kTopkClusterCtas = 8;
constexpr int kTopkClusterThreads = 512;

struct ClusterTopkShared {
  int hist[2][256];    // double-buffered: peers read pass p's while pass p+1 fills the other
  int total[256];
  uint32_t scan_tmp[33];
  uint32_t red_min[32], red_max[32];
  uint32_t cta_min, cta_max;
  int sel_digit, sel_above, sel_count;
  int cnt[2];          // this CTA's (greater, equal) counts
};

// Stages keys [0, m) of this CTA's slice `src` of a row and finds the border of
// the k largest of the whole row (`few` as for block_topk_border).  All threads of
// the cluster call this.
__device__ __forceinline__ TopkBorder cluster_topk_border(const float* src, int m, int k, uint32_t* keys,
                                                          ClusterTopkShared& sh, int few = 0) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  // stage this CTA's keys (four independent loads in flight per thread) and
  // its smallest / largest key
  uint32_t lmin = 0xffffffffu, lmax = 0u;
  auto stage = [&](int i, float x) {
    const uint32_t key = order_key(x);
    keys[i] = key;
    lmin = min(lmin, key);
    lmax = max(lmax, key);
  };
  int i0 = tid;
  for (; i0 + 3 * nt < m; i0 += 4 * nt) {
    const float x0 = __ldcg(src + i0), x1 = __ldcg(src + i0 + nt);
    const float x2 = __ldcg(src + i0 + 2 * nt), x3 = __ldcg(src + i0 + 3 * nt);
    stage(i0, x0);
    stage(i0 + nt, x1);
    stage(i0 + 2 * nt, x2);
    stage(i0 + 3 * nt, x3);
  }
  for (; i0 < m; i0 += nt) stage(i0, __ldcg(src + i0));
  for (int i = tid; i < 512; i += nt) (&sh.hist[0][0])[i] = 0;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    lmin = min(lmin, __shfl_xor_sync(0xffffffffu, lmin, o));
    lmax = max(lmax, __shfl_xor_sync(0xffffffffu, lmax, o));
  }
  if (lane == 0) {
    sh.red_min[warp] = lmin;
    sh.red_max[warp] = lmax;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t a = sh.red_min[0], b = sh.red_max[0];
    for (int w = 1; w < nw; ++w) {
      a = min(a, sh.red_min[w]);
      b = max(b, sh.red_max[w]);
    }
    sh.cta_min = a;   // an empty slice contributes (max, 0): neutral
    sh.cta_max = b;
  }
  cluster.sync();
  uint32_t kmin = 0xffffffffu, kmax = 0u;
#pragma unroll
  for (int r = 0; r < kTopkClusterCtas; ++r) {
    kmin = min(kmin, *cluster.map_shared_rank(&sh.cta_min, r));
    kmax = max(kmax, *cluster.map_shared_rank(&sh.cta_max, r));
  }

  uint32_t prefix, pmask;
  int remaining = k;
  bool open = false;
  const uint32_t diff = kmin ^ kmax;
  if (diff == 0) {
    prefix = kmin;
    pmask = 0xffffffffu;
  } else {
    const int top = 31 - __clz(diff);
    pmask = top == 31 ? 0u : ~((2u << top) - 1u);
    prefix = kmin & pmask;
    int hi = top + 1;
#pragma unroll 1
    for (int pass = 0; hi > 0; ++pass) {
      const int lo = hi > 8 ? hi - 8 : 0;
      const uint32_t wmask = (1u << (hi - lo)) - 1u;
      int* hcur = sh.hist[pass & 1];
      for (int i = tid; i < m; i += nt) {
        const uint32_t key = keys[i];
        if ((key & pmask) == prefix) atomicAdd(&hcur[(key >> lo) & wmask], 1);
      }
      cluster.sync();                                   // all local histograms complete
      for (int b = tid; b < 256; b += nt) {
        int s = 0;
#pragma unroll
        for (int r = 0; r < kTopkClusterCtas; ++r) s += cluster.map_shared_rank(hcur, r)[b];
        sh.total[b] = s;
      }
      // the other buffer was last read by peers before this pass's barrier
      for (int i = tid; i < 256; i += nt) sh.hist[(pass + 1) & 1][i] = 0;
      __syncthreads();
      if (tid < 32) {
        int c[8], s = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) { c[j] = sh.total[255 - 8 * tid - j]; s += c[j]; }
        int incl = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, incl, o);
          if (tid >= o) incl += t;
        }
        const int excl = incl - s;
        if (excl < remaining && remaining <= incl) {
          int run = excl;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (run + c[j] >= remaining) {
              sh.sel_digit = 255 - 8 * tid - j;
              sh.sel_above = run;
              sh.sel_count = c[j];
              break;
            }
            run += c[j];
          }
        }
      }
      __syncthreads();
      prefix |= (uint32_t)sh.sel_digit << lo;
      pmask |= wmask << lo;
      remaining -= sh.sel_above;
      const int cnt_sel = sh.sel_count;
      __syncthreads();          // sh.total / sel_* are rewritten by the next pass
      open = cnt_sel != remaining && lo > 0;
      if (!open || cnt_sel <= few) break;
      hi = lo;
    }
  }
  return TopkBorder{prefix, pmask, remaining, open};
}

}  // namespace sv
