// Pages of a cache shared between branches of a conversation: release, fork,
// reserve (with private copies of shared pages), and the compaction of the
// accepted path of a draft tree.
//
// A page is free iff its reference count, the number of block-table entries
// that hold it, is zero; new pages are the lowest free ones, in (sequence,
// column) order.  There is no free list to keep in step, and the same state
// always gives the same tables.  The counts and the tables are a few KB to a
// few hundred KB and bound by latency: one launch each, one CTA where the
// order of the pages matters.  The row and page copies run over every layer in
// one launch.  Measured, replayed in a graph: release, fork and reserve of 2
// branches in a pool of 80 pages 9.4 us for the four kernels, of 32 branches of
// 211 pages each 13 us, with copies of 32 pages in 8 layers (17 MB read and
// written).  ncu, each alone with cold caches: 5.0, 5.4, 9.4 (plan) and 6.5 us
// (copies).
#include "common.cuh"
#include "kernels.h"

namespace sv {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kRefsPerThread = 16;   // reference counts a thread scans per step

// Drops one reference of `page`; a count that is already zero stays zero and
// is reported.
__device__ __forceinline__ void drop_ref(int32_t* ref, int page, int num_pages, int* status) {
  if (page < 0 || page >= num_pages) {
    flag_status(status, kStatusBadBlock);
    return;
  }
  if (atomicSub(ref + page, 1) <= 0) {
    atomicAdd(ref + page, 1);
    flag_status(status, kStatusBadBlock);
  }
}

// Exclusive sum over the block of kPlanThreads threads; `total` for all.
__device__ int block_scan(int v, int* total, int* warp_sums) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();   // the previous scan's sums have been read
  if (lane == 31) warp_sums[wid] = inc;
  __syncthreads();
  if (wid == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[31];
  return inc - v + (wid > 0 ? warp_sums[wid - 1] : 0);
}

}  // namespace

// One CTA per sequence: entries [ceil(keep / 16), held) are dropped.
__global__ void __launch_bounds__(256)
pages_release_kernel(PagesArgs a, const int32_t* __restrict__ keep) {
  grid_dep_sync();
  const int b = blockIdx.x;
  const int held = a.n_pages[b];
  const int kp = keep ? __ldg(keep + b) : 0;
  __syncthreads();                       // n_pages[b] is rewritten below
  if (kp == -1) return;
  if (held < 0 || held > a.max_blocks || kp < -1) {
    if (threadIdx.x == 0) flag_status(a.status, kStatusBadLength);
    return;
  }
  const int from = min(held, (int)(((long long)kp + 15) >> 4));
  int32_t* row = a.block_table + (size_t)b * a.max_blocks;
  for (int i = from + threadIdx.x; i < held; i += blockDim.x) {
    drop_ref(a.ref, row[i], a.num_pages, a.status);
    row[i] = -1;
  }
  if (threadIdx.x == 0) a.n_pages[b] = from;
}

// One CTA per (parent, child) pair: the child shares the parent's pages.
__global__ void __launch_bounds__(256)
pages_fork_kernel(PagesArgs a, const int32_t* __restrict__ parent, const int32_t* __restrict__ child, int n,
                  const int32_t* __restrict__ n_tok) {
  grid_dep_sync();
  const int p = __ldg(parent + blockIdx.x), c = __ldg(child + blockIdx.x);
  // A row that is a parent in this call, or already the child of an earlier
  // pair, is no child: every CTA reads the same two lists and decides alike,
  // so no row that another CTA reads is written.
  bool clash = p < 0 || p >= a.batch || c < 0 || c >= a.batch;
  for (int i = threadIdx.x; i < n; i += blockDim.x)
    clash |= __ldg(parent + i) == c || (i < (int)blockIdx.x && __ldg(child + i) == c);
  if (__syncthreads_or(clash)) {
    if (threadIdx.x == 0) flag_status(a.status, kStatusBadIndex);
    return;
  }
  const int held = a.n_pages[p], mine = a.n_pages[c];
  int take = held;
  bool ok = held >= 0 && held <= a.max_blocks && mine == 0;
  if (n_tok) {
    const int tk = __ldg(n_tok + blockIdx.x);
    ok = ok && tk >= 0 && tk <= (long long)held * 16;
    take = (int)(((long long)tk + 15) >> 4);
  }
  __syncthreads();                       // n_pages[c] is rewritten below
  if (!ok) {
    if (threadIdx.x == 0) flag_status(a.status, kStatusBadLength);
    return;
  }
  const int32_t* src = a.block_table + (size_t)p * a.max_blocks;
  int32_t* dst = a.block_table + (size_t)c * a.max_blocks;
  for (int i = threadIdx.x; i < take; i += blockDim.x) {
    const int page = src[i];
    dst[i] = page;
    if (page >= 0 && page < a.num_pages) atomicAdd(a.ref + page, 1);
    else flag_status(a.status, kStatusBadBlock);
  }
  if (threadIdx.x == 0) a.n_pages[c] = take;
}

// One CTA plans the pages that make positions [len, len + new) of every
// sequence writable: entries [held, last] get fresh pages, and held entries
// from the first written one on that are shared (count > 1 at the start of
// the call) get private ones.  plan: {number of entries, -, -, -}, then one
// {sequence, column, shared page or -1, new page} per entry.
__global__ void __launch_bounds__(kPlanThreads)
pages_plan_kernel(PagesArgs a, SeqLens lens, int n_vis, int n_text, int T, const int32_t* __restrict__ n_new,
                  int4* plan, int32_t* counts, int32_t* free_ids) {
  __shared__ int warp_sums[32];
  grid_dep_sync();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = kPlanThreads / 32;
  if (threadIdx.x == 0) plan[0] = make_int4(0, 0, 0, 0);

  // the written columns [first, last] of sequence b; false: nothing to do
  auto span = [&](int b, int& first, int& last, int& held, bool report) {
    SeqLens l = lens;
    l.k = nullptr;
    int nv, nt, kb;
    bool ok = seq_lengths(l, b, n_vis, n_text, 0, nv, nt, kb);
    const int tn = n_new ? __ldg(n_new + b) : T;
    held = a.n_pages[b];
    ok = ok && tn >= 0 && tn <= T && held >= 0 && held <= a.max_blocks;
    if (!ok && report && lane == 0) flag_status(a.status, kStatusBadLength);
    first = (nv + nt) >> 4;
    last = (nv + nt + tn - 1) >> 4;
    return ok && tn > 0;
  };
  auto shared_page = [&](int b, int col, bool report) {
    const int page = a.block_table[(size_t)b * a.max_blocks + col];
    if (page < 0 || page >= a.num_pages) {
      if (report) flag_status(a.status, kStatusBadBlock);
      return -1;
    }
    return a.ref[page] > 1 ? page : -1;
  };

  for (int b = wid; b < a.batch; b += nw) {
    int first, last, held, n = 0;
    if (span(b, first, last, held, true)) {
      for (int c0 = first; c0 < min(held, last + 1); c0 += 32) {
        const int c = c0 + lane;
        const bool cow = c < held && c <= last && shared_page(b, c, true) >= 0;
        n += __popc(__ballot_sync(0xffffffffu, cow));
      }
      n += max(0, last + 1 - held);
    }
    if (lane == 0) counts[b] = n;
  }
  __syncthreads();
  int total = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    const int v = b < a.batch ? counts[b] : 0;
    int sum;
    const int ex = block_scan(v, &sum, warp_sums);
    if (b < a.batch) counts[b] = total + ex;
    total += sum;
  }
  if (total == 0) return;
  // (a table cannot want more pages than the plan holds)
  if (total > a.num_pages) {
    if (threadIdx.x == 0) flag_status(a.status, kStatusNoPages);
    return;
  }

  // the lowest free pages
  int found = 0;
  for (int p0 = 0; p0 < a.num_pages && found < total; p0 += kPlanThreads * kRefsPerThread) {
    const int mine = p0 + threadIdx.x * kRefsPerThread;
    uint32_t zero = 0;
    if (mine + kRefsPerThread <= a.num_pages) {
#pragma unroll
      for (int i = 0; i < kRefsPerThread / 4; ++i) {
        const int4 v = *reinterpret_cast<const int4*>(a.ref + mine + 4 * i);
        zero |= ((v.x == 0 ? 1u : 0u) | (v.y == 0 ? 2u : 0u) | (v.z == 0 ? 4u : 0u) | (v.w == 0 ? 8u : 0u)) << (4 * i);
      }
    } else {
      for (int i = 0; i < kRefsPerThread; ++i)
        if (mine + i < a.num_pages && a.ref[mine + i] == 0) zero |= 1u << i;
    }
    int sum;
    int at = found + block_scan(__popc(zero), &sum, warp_sums);
    for (; zero && at < total; zero &= zero - 1) free_ids[at++] = mine + __ffs(zero) - 1;
    found += sum;
  }
  if (found < total) {
    if (threadIdx.x == 0) flag_status(a.status, kStatusNoPages);
    return;
  }
  __syncthreads();

  // entries of the plan, from the state at the start of the call
  for (int b = wid; b < a.batch; b += nw) {
    int first, last, held;
    if (!span(b, first, last, held, false)) continue;
    int at = counts[b];
    for (int c0 = first; c0 < min(held, last + 1); c0 += 32) {
      const int c = c0 + lane;
      const int page = c < held && c <= last ? shared_page(b, c, false) : -1;
      const uint32_t m = __ballot_sync(0xffffffffu, page >= 0);
      if (page >= 0) {
        const int i = at + __popc(m & ((1u << lane) - 1));
        plan[1 + i] = make_int4(b, c, page, free_ids[i]);
      }
      at += __popc(m);
    }
    for (int c = held + lane; c <= last; c += 32) {
      const int i = at + c - held;
      plan[1 + i] = make_int4(b, c, -1, free_ids[i]);
    }
    __syncwarp();
    if (lane == 0 && last + 1 > held) a.n_pages[b] = last + 1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += kPlanThreads) {
    const int4 e = plan[1 + i];
    a.block_table[(size_t)e.x * a.max_blocks + e.y] = e.w;
    if (e.z >= 0) atomicSub(a.ref + e.z, 1);
    a.ref[e.w] = 1;
  }
  if (threadIdx.x == 0) plan[0] = make_int4(total, 0, 0, 0);
}

// The planned private copies in up to kMaxLayers layers: a warp copies 2 KB
// (a page of K or V is a multiple of that) per step.
__global__ void __launch_bounds__(256)
pages_copy_kernel(const int4* __restrict__ plan, const __grid_constant__ LayerPools pools, int layers, int chunks) {
  grid_dep_sync();
  const int n = plan[0].x;
  const int lane = threadIdx.x & 31;
  const long long nwarps = (long long)gridDim.x * (blockDim.x >> 5);
  const long long units = (long long)n * layers * 2 * chunks;
  for (long long u = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); u < units; u += nwarps) {
    const int c = (int)(u % chunks);
    const long long r = u / chunks;
    const int pool = (int)(r % (2 * layers));
    const int4 e = plan[1 + r / (2 * layers)];
    if (e.z < 0) continue;
    uint4* base = static_cast<uint4*>((pool & 1) ? pools.v[pool >> 1] : pools.k[pool >> 1]);
    const uint4* src = base + ((size_t)e.z * chunks + c) * 128 + lane;
    uint4* dst = base + ((size_t)e.w * chunks + c) * 128 + lane;
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = src[32 * i];
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[32 * i] = x[i];
  }
}

// Accepted path of a draft: row base + path[i] -> row base + i, for one
// (layer, KV head, sequence) per CTA.  path ascends, so rows only move down;
// every row is loaded before any is stored.  At most 64 KB a CTA, bound by its
// dependent loads (lengths, path, page table, row): 6.0 us alone with cold
// caches for 8 sequences, 4 layers, 4 KV heads.
__global__ void __launch_bounds__(256)
kv_accept_kernel(const __grid_constant__ LayerPools pools, int num_blocks, int Hkv, int vecs,
                 const int32_t* __restrict__ block_table, int max_blocks, SeqLens lens, int n_vis, int n_text, int T,
                 const int32_t* __restrict__ path, int P, const int32_t* __restrict__ n_path, int* status) {
  grid_dep_sync();
  const int b = blockIdx.x, g = blockIdx.y, layer = blockIdx.z;
  const bool report = threadIdx.x == 0 && g == 0 && layer == 0;
  SeqLens l = lens;
  l.k = nullptr;
  int nv, nt, kb;
  const bool ok = seq_lengths(l, b, n_vis, n_text, 0, nv, nt, kb);
  const int n = n_path ? __ldg(n_path + b) : P;
  if (!ok || n < 0 || n > P) {
    if (report) flag_status(status, kStatusBadLength);
    return;
  }
  const int32_t* row = path + (size_t)b * P;
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int v = __ldg(row + i);
    bad |= v < 0 || v >= T || (i > 0 && __ldg(row + i - 1) >= v);
  }
  if (__syncthreads_or(bad)) {
    if (report) flag_status(status, kStatusBadIndex);
    return;
  }
  const int32_t* bt = block_table + (size_t)b * max_blocks;
  const int base = nv + nt;
  uint4* kp = static_cast<uint4*>(pools.k[layer]);
  uint4* vp = static_cast<uint4*>(pools.v[layer]);
  // at most 64 rows x 16 vectors x (K, V) = 8 vectors a thread
  uint4 buf[8];
  long long to[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int x = threadIdx.x + 256 * i;
    to[i] = -1;
    const int r = x / (2 * vecs), v = x % (2 * vecs);
    if (r >= n) continue;
    const int from = __ldg(row + r);
    if (from == r) continue;
    const int sp = __ldg(bt + ((base + from) >> 4)), dp = __ldg(bt + ((base + r) >> 4));
    if (sp < 0 || sp >= num_blocks || dp < 0 || dp >= num_blocks) {
      flag_status(status, kStatusBadBlock);
      continue;
    }
    const bool is_v = v >= vecs;
    const int c = is_v ? v - vecs : v;
    buf[i] = (is_v ? vp : kp)[((((long long)sp * Hkv + g) << 4) + ((base + from) & 15)) * vecs + c];
    to[i] = (((((long long)dp * Hkv + g) << 4) + ((base + r) & 15)) * vecs + c) | ((long long)is_v << 62);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (to[i] >= 0) ((to[i] >> 62) ? vp : kp)[to[i] & ((1LL << 62) - 1)] = buf[i];
}

cudaError_t launch_pages_release(const PagesArgs& a, const int32_t* keep, cudaStream_t stream) {
  if (a.batch == 0) return cudaSuccess;
  return launch_dependent(pages_release_kernel, dim3(a.batch), dim3(256), 0, stream, a, keep);
}

cudaError_t launch_pages_fork(const PagesArgs& a, const int32_t* parent, const int32_t* child, int n,
                              const int32_t* n_tok, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  return launch_dependent(pages_fork_kernel, dim3(n), dim3(256), 0, stream, a, parent, child, n, n_tok);
}

size_t pages_workspace_bytes(long long batch, long long max_blocks, long long num_pages) {
  const long long entries = batch * max_blocks < num_pages ? batch * max_blocks : num_pages;
  // plan | counts [batch] | free ids
  return (size_t)(1 + entries) * sizeof(int4) + ((size_t)batch + 3) / 4 * 16 + (size_t)entries * sizeof(int32_t);
}

cudaError_t launch_pages_reserve(const PagesArgs& a, const SeqLens& lens, int n_vis, int n_text, int T,
                                 const int32_t* n_new, const LayerPools* pools, int n_pools, const int* layers,
                                 int page_bytes, void* ws, int num_sms, cudaStream_t stream) {
  if (a.batch == 0 || T == 0) return cudaSuccess;
  const long long all = (long long)a.batch * a.max_blocks;
  const long long entries = all < a.num_pages ? all : a.num_pages;
  int4* plan = static_cast<int4*>(ws);
  int32_t* counts = reinterpret_cast<int32_t*>(plan + 1 + entries);
  int32_t* free_ids = counts + ((size_t)a.batch + 3) / 4 * 4;
  cudaError_t e = launch_dependent(pages_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a, lens, n_vis, n_text,
                                   T, n_new, plan, counts, free_ids);
  for (int i = 0; i < n_pools && e == cudaSuccess; ++i) {
    const int chunks = page_bytes / 2048;
    // at most one shared page per written column; four CTAs an SM fill it
    const long long most = (long long)a.batch * ((T + 14) / 16 + 1) * layers[i] * 2 * chunks;
    const long long ctas = (most + 7) / 8;
    const int grid = (int)(ctas < 4LL * num_sms ? ctas : 4LL * num_sms);
    e = launch_dependent(pages_copy_kernel, dim3(grid), dim3(256), 0, stream, (const int4*)plan, pools[i], layers[i],
                         chunks);
  }
  return e;
}

cudaError_t launch_kv_accept(const LayerPools& pools, int layers, int num_blocks, int Hkv, int D,
                             const int32_t* block_table, int max_blocks, int batch, const SeqLens& lens, int n_vis,
                             int n_text, int T, const int32_t* path, int P, const int32_t* n_path, int* status,
                             cudaStream_t stream) {
  if (batch == 0 || layers == 0 || P == 0) return cudaSuccess;
  return launch_dependent(kv_accept_kernel, dim3(batch, Hkv, layers), dim3(256), 0, stream, pools, num_blocks, Hkv,
                          D / 8, block_table, max_blocks, lens, n_vis, n_text, T, path, P, n_path, status);
}

}  // namespace sv
