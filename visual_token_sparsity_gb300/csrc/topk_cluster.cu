// Row top-k for long rows on a thread-block cluster.
//
// The selection step of decode retrieval (velog.io SparseVILA summary §3.2)
// for long-video caches, where one (sequence, KV head) row holds tens of
// thousands of visual scores and a batch has only a few rows.  A cluster of
// kTopkClusterCtas CTAs owns one row; CTA r keeps the r-th slice of the row's
// order-preserving keys in its shared memory.  The cluster's smallest and
// largest keys fix the bits every key shares; each radix pass then builds a
// local 256-bin histogram of the next 8-bit window, and after a cluster
// barrier every CTA sums the cluster's histograms through distributed shared
// memory and picks the same digit (histograms are double-buffered, so one
// cluster barrier per pass is enough).  Passes stop once the selected bin
// holds exactly the keys still needed.  The output phase exchanges per-CTA
// (greater, equal) counts the same way, so the CTAs write disjoint ranges of
// the ascending index list, with ties broken towards the lower index exactly
// as in the single-CTA routine (topk_block.cuh).  The cluster barriers are
// hardware barriers over co-scheduled CTAs; nothing spins.
#include "kernels.h"
#include "topk_cluster.cuh"

namespace cg = cooperative_groups;

namespace sv {

__global__ void __cluster_dims__(kTopkClusterCtas, 1, 1) __launch_bounds__(kTopkClusterThreads)
topk_cluster_kernel(const float* __restrict__ scores, int n_cap, int k_cap, int32_t* __restrict__ idx,
                    SeqLens lens, int rows_per_seq) {
  extern __shared__ uint32_t keys[];
  __shared__ ClusterTopkShared sh;
  grid_dep_sync();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int row = blockIdx.y;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
  // this row's key count and selection size (the same for every CTA of the
  // cluster, so an empty selection leaves the cluster together)
  int n = n_cap, k = k_cap;
  if (lens.any()) row_lengths(lens, row, rows_per_seq, n_cap, k_cap, n, k);
  int32_t* dst = idx + (size_t)row * k_cap;
  if (rank == 0) fill_unselected(dst, k, k_cap);
  if (k <= 0) return;
  const int slice = (n + kTopkClusterCtas - 1) / kTopkClusterCtas;
  const int lo_i = min(n, rank * slice), hi_i = min(n, lo_i + slice);
  const int m = hi_i - lo_i;
  const float* src = scores + (size_t)row * n_cap + lo_i;

  const TopkBorder border = cluster_topk_border(src, m, k, keys, sh);
  const uint32_t prefix = border.prefix, pmask = border.pmask;
  const int remaining = border.remaining;

  // this CTA's counts, then the counts of the CTAs before it in the row
  const int seg = (m + nt - 1) / nt;
  const int s0 = min(m, tid * seg), s1 = min(m, s0 + seg);
  int gt = 0, eq = 0;
  for (int i = s0; i < s1; ++i) {
    const uint32_t kp = keys[i] & pmask;
    gt += kp > prefix;
    eq += kp == prefix;
  }
  if (tid == 0) sh.cnt[0] = sh.cnt[1] = 0;
  __syncthreads();
  int w_gt = gt, w_eq = eq;
#pragma unroll
  for (int o2 = 16; o2 >= 1; o2 >>= 1) {
    w_gt += __shfl_xor_sync(0xffffffffu, w_gt, o2);
    w_eq += __shfl_xor_sync(0xffffffffu, w_eq, o2);
  }
  if (lane == 0) { atomicAdd(&sh.cnt[0], w_gt); atomicAdd(&sh.cnt[1], w_eq); }
  cluster.sync();
  int gt_before = 0, eq_before_cta = 0;
  for (int r = 0; r < rank; ++r) {
    const int* rc = cluster.map_shared_rank(sh.cnt, r);
    gt_before += rc[0];
    eq_before_cta += rc[1];
  }
  // within the CTA: one scan of the packed (greater, equal) pair (a slice
  // holds fewer than 65536 keys)
  const uint32_t packed = block_exclusive_scan<uint32_t>(((uint32_t)gt << 16) | (uint32_t)eq, sh.scan_tmp);
  const int eq_before = (int)(packed & 0xffffu) + eq_before_cta;
  int take_eq = remaining - eq_before;
  take_eq = take_eq < 0 ? 0 : (take_eq > eq ? eq : take_eq);
  int o = gt_before + (int)(packed >> 16) + min(eq_before, remaining);
  int e = 0;
  for (int i = s0; i < s1; ++i) {
    const uint32_t kp = keys[i] & pmask;
    bool take = kp > prefix;
    if (kp == prefix) {
      take = e < take_eq;
      ++e;
    }
    if (take) dst[o++] = lo_i + i;
  }
  cluster.sync();     // keep this CTA's shared memory alive until every peer has read it
}

bool topk_cluster_fits(int n) {
  const int slice = (n + kTopkClusterCtas - 1) / kTopkClusterCtas;
  return (size_t)slice * sizeof(uint32_t) <= 200 * 1024;
}

// Short rows keep one CTA per row: below ~16K keys a cluster's barriers and
// DSMEM exchanges cost more than the 8x wider slice saves.
bool topk_prefers_cluster(int n) { return n > 16384 && topk_cluster_fits(n); }

cudaError_t launch_topk_cluster(const float* scores, int rows, int n, int k, int32_t* idx,
                                cudaStream_t stream, const SeqLens& lens, int rows_per_seq) {
  if (rows == 0) return cudaSuccess;
  const int slice = (n + kTopkClusterCtas - 1) / kTopkClusterCtas;
  const size_t smem = (size_t)slice * sizeof(uint32_t);
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(topk_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  dim3 grid(kTopkClusterCtas, rows);
  return launch_dependent(topk_cluster_kernel, grid, dim3(kTopkClusterThreads), smem, stream, scores, n, k, idx,
                          lens, rows_per_seq > 0 ? rows_per_seq : 1);
}

}  // namespace sv
