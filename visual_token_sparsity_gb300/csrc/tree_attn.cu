// Attention of T drafted (or question) tokens per sequence over the paged
// cache: the selected visual tokens, the text, and of the T tokens' own keys
// (already appended behind the text) those that the tree mask lets each see.
//
//   tok(i) = vis_idx[i] (i < k), then n_vis + (i - k): text, then drafted
//   z_i = scale q . K[tok(i)], seen(i) = i < k + n_text or bit (i - k - n_text)
//   out = sum_seen exp(z_i - m) V[tok(i)] / sum_seen exp(z_i - m)
//
// The R = T * G rows of a KV head (G query heads of each token) share its
// keys and values, so both products are matrix products on the tcgen05
// tensor cores: S = Q K^T (128 rows x 128 tokens), then O += P V with P as
// the bf16 A operand in tensor memory and V read token-major from shared
// memory.  One pass: running maximum and sum per row in fp32 registers, the
// accumulator rescaled only when a row's maximum grows far beyond it.
//
// A CTA runs two streams, each with its own S, P, O in tensor memory and four
// softmax warps, so that one's products run while the other's weights are
// formed.  Up to 128 rows: the streams take alternate token tiles of the same
// rows and their (m, l, O) are joined at the end (bound by the cache's bytes:
// padding to 128 rows costs 1024 tensor cycles a tile against the 2800 that
// its 64 KB take to arrive).  More rows: the streams take 128 rows each of
// the same token tile, which halves the bytes per product.
//
// Within a tile of rows the work is cut evenly: the token tiles of all
// (sequence, KV head) units form one line, cut into equal pieces, one per CTA
// column; a unit that lies in several pieces leaves fp32 partials that a second
// kernel joins in a fixed order.  CTAs of one piece and different row tiles are
// neighbours, so they meet in L2.  Every row tile gets the same whole number of
// columns, so with many row tiles SMs are left over, half of them from 77 on
// (28 / 4 heads, 50176 + T tokens: T 2770, 76 row tiles of 2 columns, 1.34
// PFLOP/s; T 2800, 77 of one, 0.69).
//
// Warps: 0-7 softmax and epilogue (one row per thread), 8-9 MMA issue (one per
// stream), 10-13 cache rows: cp.async gathers of 16 bytes into a ring of
// 128-row K and V tiles in the 128-byte-swizzled layout the MMA reads,
// page-table and index loads running two tiles ahead, 14-15 query rows.  Rows
// that are not there (behind the end, a bad page) are zero-filled and masked.
//
// The weights enter the value product as bf16, the type of V that the tensor
// core asks for, while the sum l takes them unrounded, which lse needs: at most
// 2^-8 of sum p |v| beside the output's own 2^-8.  (Measured against 64 bits,
// relative: 2.3e-3, where fp32 weights give 1.7e-3.)
//
// Measured (d 128): 16 sequences x 32 heads x 1584 tokens, 16 rows, 78 us =
// 5.4 TB/s of cache rows; 8 x 4 KV heads of up to 12827 tokens, 189 rows, 51.6 us =
// 3.1 TB/s; 1351 rows x 4 KV heads x 50392 tokens 133 us = 1.05 PFLOP/s, where a
// tile takes a CTA 3800 cycles, 2048 of them in the products: each stream's
// chain of S, weights and O is longer than what the other's hides.
#include "common.cuh"
#include "fastmath.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace sv {

namespace {

using ptx::mma_ts;
using ptx::tmem_ld16;
using ptx::tmem_st16;
using ptx::tmem_wait_st;

constexpr int kTile = 128;                  // tokens of a tile, rows of a stream
constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = 8;                 // and 9: one per stream
constexpr int kLoadWarp = 10, kLoadWarps = 4;
constexpr int kQueryWarp = 14, kQueryWarps = 2;
constexpr int kThreads = 512;
// Registers: 512 threads at 128 at launch; the softmax warps, which hold a
// whole row of S (128 columns), take some of the others'.  The cache-row warps
// need 80: with 64 they spill, and the LLaVA-NeXT batch took 81 us, not 77 (160 /
// 96, where the softmax warps spill: 79).
constexpr int kSoftRegs = 176, kOtherRegs = 80;
static_assert(256 * kSoftRegs + 256 * kOtherRegs <= 65536 && 32 * (kQueryWarp + kQueryWarps) == kThreads,
              "register split");
constexpr int kTmemCols = 512;              // S0 | S1 | O0 | O1, 128 columns each
constexpr int kCtas = 152;                  // one per SM (fewer than 2^15)
constexpr int kMaxSlots = 12;
constexpr int kValidRing = 16;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr size_t kMaxSmem = 232448;         // 227 KB
// A row's weights are taken relative to a reference that is raised, and O
// rescaled, only when the maximum outgrows it by 2^32: bf16 and fp32 have the
// exponents for it (as long as the values stay below 2^70 in magnitude, and the
// tokens below 2^25), and no rounding depends on it.
constexpr float kRescale = 32.f;
static_assert(kLoadWarps * 32 == kTile, "one loader thread per token");

// Ring slots (128 tokens of K or V) beside the query rows.  The next segment's
// queries are loaded while the last one runs where two sets fit (128 rows: many
// short segments; a load takes the time of two tiles when HBM is busy).
template <int D, int QT>
struct Smem {
  static constexpr int kSlotBytes = kTile * D * 2;
  static constexpr int kQBufs = QT == 128 ? 2 : 1;
  static constexpr int kQBytes = QT * D * 2;            // one set
  static constexpr int kSlots = D == 128 ? 5 : (QT == 128 ? 12 : 10);
  static constexpr int kRing = kQBufs * kQBytes;        // where the ring begins
  static constexpr int kBytes = kRing + kSlots * kSlotBytes;
  static_assert(kSlots <= kMaxSlots && kSlots / 2 + 1 < kValidRing, "ring sizes");
};

struct Shared {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full, done, turn[2];
  uint64_t valid_full[kValidRing];
  uint32_t tmem;
  int abort;
  int odd_values;                 // some drafted V held an infinity or NaN
  int b0;                         // this CTA's piece: first sequence,
  int off0, count, total;         // first tile inside it, tiles; the whole line
  alignas(16) uint32_t valid[kValidRing][4];  // tokens of a tile that are there
  float ml[2][kTile][2];          // the streams' maxima and sums
};
// the static part lies before the ring, which begins at a multiple of 1 KB
constexpr int kStaticSmem = 3 * 1024;
static_assert(sizeof(Shared) <= kStaticSmem && Smem<128, 128>::kBytes + kStaticSmem <= kMaxSmem &&
                  Smem<128, 256>::kBytes + kStaticSmem <= kMaxSmem &&
                  Smem<64, 128>::kBytes + kStaticSmem <= kMaxSmem &&
                  Smem<64, 256>::kBytes + kStaticSmem <= kMaxSmem,
              "shared memory");

__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t parity, Shared& sh) {
  if (ptx::mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = ptx::global_timer();
  for (;;) {
    if (ptx::mbar_try_wait_sleep(bar, parity, 100000)) return;
    if (*(volatile int*)&sh.abort) return;
    if (ptx::global_timer() - t0 > kWaitLimitNs) {
      *(volatile int*)&sh.abort = 1;
      return;
    }
  }
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void soft_bar() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory"); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Replaces the infinities and NaN among 8 bf16 values by 0.
__device__ __forceinline__ bool zero_odd(uint4* p) {
  uint4 v = *p;
  uint32_t* u = reinterpret_cast<uint32_t*>(&v);
  bool odd = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((u[e] & 0x7f80u) == 0x7f80u) { u[e] &= 0xffff0000u; odd = true; }
    if ((u[e] & 0x7f800000u) == 0x7f800000u) { u[e] &= 0xffffu; odd = true; }
  }
  if (odd) *p = v;
  return odd;
}

// 8 bf16 values times 0: infinities and NaN give NaN.
__device__ __forceinline__ void times_zero(uint4* p) {
  uint4 v = *p;
  uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    u[e] = ((u[e] & 0x7f80u) == 0x7f80u ? 0x7fc0u : 0u) | ((u[e] & 0x7f800000u) == 0x7f800000u ? 0x7fc00000u : 0u);
  *p = v;
}

// Tensor memory columns of a stream's S (and P) and O: the CTA holds all 512,
// so its allocation begins at column 0 (checked at the start).
__host__ __device__ constexpr uint32_t tmem_s(int s) { return s * 128; }
__host__ __device__ constexpr uint32_t tmem_o(int s) { return 256 + s * 128; }

// Ring positions of a CTA's K and V tiles: K0 K1 V0 K2 V1 K3 V2 ..., the order
// in which they are used (V a softmax later than K; requested together, V
// would hold its slot that much longer).
__device__ __forceinline__ uint32_t ring_k(uint32_t tile) { return tile > 0 ? 2 * tile - 1 : 0; }
__device__ __forceinline__ uint32_t ring_v(uint32_t tile) { return 2 * tile + 2; }

// ---- the line of tiles and its pieces

struct Seq {
  int nv, nt, kb, tn;   // visual, text, selected (or all visual), drafted tokens
};

// Sequence b's counts; a sequence with a count out of range has none.
__device__ __forceinline__ bool seq_of(const TreeArgs& a, int b, Seq& s) {
  bool ok = attn_lengths(a.lens, a.vis_idx != nullptr, b, a.n_vis, a.n_text, a.k_vis, false, a.status, s.nv, s.nt,
                         s.kb);
  s.tn = a.n_new ? __ldg(a.n_new + b) : a.T;
  ok = ok && s.tn >= 0 && s.tn <= a.T;
  if (!ok) s.nv = s.nt = s.kb = s.tn = 0;
  return ok;
}

// Tokens that rows [row0, row0 + QT) of a sequence can see (0: no such rows).
__device__ __forceinline__ int tokens_of(const TreeArgs& a, const Seq& s, int row0, int QT) {
  const int rows = s.tn * a.G;
  if (row0 >= rows) return 0;
  const int last = min(row0 + QT, rows) - 1;
  return s.kb + s.nt + (a.tree_mask ? s.tn : last / a.G + 1);
}
__device__ __forceinline__ int tiles_of(const TreeArgs& a, int b, int row0, int QT) {
  Seq s;
  seq_of(a, b, s);
  return (tokens_of(a, s, row0, QT) + kTile - 1) / kTile;
}

// First tile of piece c of C: floor(total * c / C).  (32 bits throughout: a 64-bit
// division is a hundred instructions, and code that runs once is mostly fetching.)
__device__ __forceinline__ int piece_begin(int total, int c, int C) {
  const int q = total / C;
  return q * c + (total - q * C) * c / C;
}

// Consecutive tiles [t0, t1) of one (sequence, KV head) unit.
struct Segment {
  Seq s;
  int b, g, t0, t1, tiles, tokens, rows;
  __device__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// Walks a CTA's piece; every warp has its own and sees the same segments.
struct Walk {
  int b, row0, QT, off, left;
  Segment x;
  __device__ void start(const Shared& sh, int top, int QT_) {
    row0 = top;
    QT = QT_;
    b = sh.b0;
    off = sh.off0;
    left = sh.count;
  }
  __device__ bool next(const TreeArgs& a) {
    while (left > 0 && b < a.batch) {
      seq_of(a, b, x.s);
      x.tokens = tokens_of(a, x.s, row0, QT);
      x.tiles = (x.tokens + kTile - 1) / kTile;
      if (off < x.tiles * a.Hkv) {
        x.b = b;
        x.g = off / x.tiles;
        x.t0 = off - x.g * x.tiles;
        x.t1 = min(x.tiles, x.t0 + left);
        x.rows = min(QT, x.s.tn * a.G - row0);
        off += x.t1 - x.t0;
        left -= x.t1 - x.t0;
        return true;
      }
      ++b;
      off = 0;
    }
    return false;
  }
};

// Partial results of a unit cut into pieces: slot 0 of a CTA continues a unit
// that an earlier piece began, slot 1 begins one that goes on.  (m, l) are
// [slot][row], O is [slot][dim / 4][row][4]: consecutive rows, which
// neighbouring lanes hold, lie side by side.
__device__ __forceinline__ size_t part_slot(int cta, bool begins) { return (size_t)cta * 2 + (begins ? 1 : 0); }

}  // namespace

template <int D, int QT>
__global__ void __launch_bounds__(kThreads, 1)
tree_attn_kernel(const __grid_constant__ TreeArgs a) {
  using M = Smem<D, QT>;
  constexpr int CPR = D / 8;                       // 16-byte chunks of a row
  constexpr int S = M::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];   // swizzle atoms are 1 KB
  __shared__ Shared sh;
  const uint32_t q_base = smem_u32(smem), ring = q_base + M::kRing;
  constexpr uint32_t QB = M::kQBufs;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x / a.row_tiles, row0 = (int)(blockIdx.x % a.row_tiles) * QT;

  if (warp == 0) ptx::tmem_alloc(&sh.tmem, kTmemCols);
  if (warp == 1) {
    // barriers: a lane each
    if (lane < S) {
      ptx::mbar_init(&sh.full[lane], kLoadWarps * 32);
      ptx::mbar_init(&sh.empty[lane], 2);            // both streams' products
    } else if (lane < S + 2) {
      ptx::mbar_init(&sh.s_full[lane - S], 1);
      ptx::mbar_init(&sh.p_full[lane - S], 4);
      ptx::mbar_init(&sh.turn[lane - S], 1);
      ptx::mbar_init(&sh.q_full[lane - S], kQueryWarps);
      ptx::mbar_init(&sh.q_empty[lane - S], 2);
    } else if (lane == S + 2) {
      ptx::mbar_init(&sh.o_full, 2);
      ptx::mbar_init(&sh.done, 2);
      sh.abort = 0;
      sh.odd_values = 0;
    }
    if (lane < kValidRing) ptx::mbar_init(&sh.valid_full[lane], kLoadWarps);
    ptx::mbar_fence_init();
  }
  grid_dep_sync();                                    // (nothing before it touches global memory)
  if (warp == 2) {
    // this CTA's piece of the line
    int b = 0, before = 0, begin, end, total;
    if (!a.lens.any() && a.n_new == nullptr) {
      const int per = a.Hkv * tiles_of(a, 0, row0, QT);
      total = per * a.batch;
      begin = piece_begin(total, col, a.columns);
      end = piece_begin(total, col + 1, a.columns);
      b = per > 0 ? begin / per : 0;
      before = b * per;
    } else {
      // tiles of sequences [b0, b0 + 32) up to this lane's
      auto scan = [&](int b0, int& n) {
        n = b0 + lane < a.batch ? a.Hkv * tiles_of(a, b0 + lane, row0, QT) : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        return inc;
      };
      int n, inc = scan(0, n);
      total = __shfl_sync(0xffffffffu, inc, 31);
      for (int b0 = 32; b0 < a.batch; b0 += 32) {
        int n2;
        total += __shfl_sync(0xffffffffu, scan(b0, n2), 31);
      }
      begin = piece_begin(total, col, a.columns);
      end = piece_begin(total, col + 1, a.columns);
      // the first sequence whose tiles reach past `begin`
      for (; begin < end && b < a.batch; b += 32) {
        if (b > 0) inc = scan(b, n);
        const uint32_t past = __ballot_sync(0xffffffffu, before + inc > begin);
        if (past) {
          const int f = __ffs(past) - 1;
          before += __shfl_sync(0xffffffffu, inc - n, f);
          b += f;
          break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    if (lane == 0) {
      sh.b0 = b;
      sh.off0 = begin - before;
      sh.count = end - begin;
      sh.total = total;
    }
  }
  // sequences whose counts are out of range: reported, their rows read 0 and -inf
  if (a.lens.any() || a.n_new != nullptr) {
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
      Seq s;
      if (seq_of(a, b, s)) continue;
      if (threadIdx.x == 0) flag_status(a.status, kStatusBadLength);
      const size_t n = (size_t)a.T * a.H;
      for (size_t i = threadIdx.x; i < n * CPR; i += kThreads)
        reinterpret_cast<uint4*>(a.out)[b * n * CPR + i] = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse != nullptr)
        for (size_t i = threadIdx.x; i < n; i += kThreads) a.lse[b * n + i] = -INFINITY;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  Walk w;
  w.start(sh, row0, QT);
  const bool misplaced = sh.tmem != 0 || (smem_u32(smem) & 1023u) != 0;   // (cannot be)
  if (misplaced) w.left = 0;

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp >= kLoadWarp && warp < kLoadWarp + kLoadWarps) {
    // ------------------------------------------------ cache rows
    const int me = threadIdx.x - kLoadWarp * 32;   // this thread's token of every tile
    // A warp instruction copies RPI rows of its 32: this lane's chunk of row
    // first + i * RPI, at a swizzle that repeats every 8 rows.
    constexpr int RPI = 32 / CPR, VAR = 8 / RPI;
    const uint32_t c = lane % CPR, first = lane / CPR;
    uint32_t to[VAR];
#pragma unroll
    for (int i = 0; i < VAR; ++i)
      to[i] = ring + (c >> 3) * kTile * 128 + ((warp - kLoadWarp) * 32 + first) * 128 +
              (((c & 7) ^ ((first + i * RPI) & 7)) * 16);
    auto copy = [&](const uint16_t* pool, uint32_t group, uint32_t rid, uint32_t there) {
      const uint32_t slot = group % S;
      uint32_t r[CPR];               // every row id first: no copy waits for a shuffle
#pragma unroll
      for (int i = 0; i < CPR; ++i) r[i] = __shfl_sync(0xffffffffu, rid, first + i * RPI);
      if (group >= (uint32_t)S) wait_bar(&sh.empty[slot], (group / S - 1) & 1, sh);
      __syncwarp();
      const uint8_t* src = reinterpret_cast<const uint8_t*>(pool + c * 8);
      const uint32_t dst = slot * M::kSlotBytes;
      if (there == 0xffffffffu) {
#pragma unroll
        for (int i = 0; i < CPR; ++i)
          cp_async16(dst + to[i % VAR] + i * RPI * 128, src + (size_t)r[i] * (D * 2), 16u);
      } else {
#pragma unroll
        for (int i = 0; i < CPR; ++i)
          cp_async16(dst + to[i % VAR] + i * RPI * 128, src + (size_t)r[i] * (D * 2),
                     (there >> (first + i * RPI)) & 1 ? 16u : 0u);
      }
      // the barrier counts this thread once its copies have landed; the
      // threads that read them fence the proxies
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh.full[slot])) : "memory");
    };

    // Tiles pass three steps: their indices are loaded (two tiles ahead),
    // their pages (one ahead), then their rows.
    struct Ahead {
      int index, pos, page, nv, g;
      const int32_t* bt;
      bool exists, visual, listed, there;
    };
    Ahead A = {}, B = {};
    int t = 0, t_end = 0;
    auto load_index = [&](Ahead& n) {
      n.exists = false;
      if (t >= t_end) {
        if (!w.next(a)) return;
        t = w.x.t0;
        t_end = w.x.t1;
      }
      const Segment& x = w.x;
      const int i = t * kTile + me;
      n.exists = true;
      n.there = i < x.tokens;
      n.visual = i < x.s.kb;
      n.nv = x.s.nv;
      n.g = x.g;
      n.bt = a.block_table + (size_t)x.b * a.max_blocks;
      n.pos = n.visual ? i : x.s.nv + i - x.s.kb;
      n.listed = n.visual && a.vis_idx != nullptr;
      if (n.listed) {
        const size_t at = ((size_t)x.b * a.Hkv + x.g) * a.k_vis + i;
        n.index = __ldg(a.vis_idx + at);
        // the list's lines reach L1 eight tiles ahead (the next unit's rows follow)
        if (at + 8 * kTile < (size_t)a.batch * a.Hkv * a.k_vis)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(a.vis_idx + at + 8 * kTile));
      }
      ++t;
    };
    auto load_page = [&](Ahead& n) {
      if (!n.exists || !n.there) return;
      if (n.listed) n.pos = n.index;
      if (n.visual && (n.pos < 0 || n.pos >= n.nv)) {
        flag_status(a.status, kStatusBadIndex);
        n.there = false;
        return;
      }
      n.page = __ldg(n.bt + (n.pos >> 4));
    };
    const uint16_t* k_pool = static_cast<const uint16_t*>(a.k_pool);
    const uint16_t* v_pool = static_cast<const uint16_t*>(a.v_pool);
    load_index(A);
    load_page(A);
    load_index(B);
    uint32_t tile = 0, rid = 0, there = 0;    // this tile's row (0: not there) and the warp's rows
    for (; A.exists; ++tile) {
      const uint32_t last_rid = rid, last_there = there;
      bool ok = A.there;
      if (ok && (A.page < 0 || A.page >= a.num_blocks)) {
        flag_status(a.status, kStatusBadBlock);
        ok = false;
      }
      rid = ok ? (((uint32_t)A.page * (uint32_t)a.Hkv + (uint32_t)A.g) << 4) | (uint32_t)(A.pos & 15) : 0u;
      A = B;
      load_page(A);
      load_index(B);
      there = __ballot_sync(0xffffffffu, ok);
      // (a barrier of their own: the one that the copies arrive at orders no
      // ordinary store)
      if (lane == 0) {
        sh.valid[tile % kValidRing][warp - kLoadWarp] = there;
        ptx::mbar_arrive(&sh.valid_full[tile % kValidRing]);
      }
      copy(k_pool, ring_k(tile), rid, there);
      if (tile > 0) copy(v_pool, ring_v(tile - 1), last_rid, last_there);
    }
    if (tile > 0) copy(v_pool, ring_v(tile - 1), rid, there);
    cp_async_wait_all();
  } else if (warp >= kQueryWarp) {
    // ------------------------------------------------ query rows: 32 at a time
    constexpr int RPI = 32 / CPR;
    const uint32_t c = lane % CPR, first = lane / CPR;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + c * 8;
    uint32_t n = 0;
    for (; w.next(a); ++n) {
      if (n >= QB) wait_bar(&sh.q_empty[n % QB], (n / QB - 1) & 1, sh);
      __syncwarp();
      const Segment& x = w.x;
      const uint32_t base = q_base + (n % QB) * M::kQBytes;
      for (int r0 = 32 * (warp - kQueryWarp); r0 < x.rows; r0 += 32 * kQueryWarps) {
        const int row = row0 + r0 + lane, tk = row / a.G;
        // (a row past the last one reads the sequence's first: its results go nowhere)
        const uint32_t mine = r0 + lane < x.rows ? (uint32_t)tk * a.H + (uint32_t)(x.g * a.G + row - tk * a.G) : 0u;
        const uint16_t* src = q + (size_t)x.b * a.T * a.H * D;
        const uint32_t dst = base + (r0 >> 7) * kTile * D * 2 + (c >> 3) * kTile * 128 + ((r0 & 127) + first) * 128;
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
          const uint32_t r = __shfl_sync(0xffffffffu, mine, first + i * RPI);
          cp_async16(dst + i * RPI * 128 + (((c & 7) ^ ((first + i * RPI) & 7)) * 16), src + (size_t)r * D, 16u);
        }
      }
      cp_async_wait_all();
      if (a.zero_scale) {
        // (each lane on the chunks that it copied itself)
#pragma unroll 1
        for (int r0 = 32 * (warp - kQueryWarp); r0 < x.rows; r0 += 32 * kQueryWarps)
#pragma unroll 1
          for (int i = 0; i < CPR; ++i) {
            const uint32_t r = first + i * RPI;
            times_zero(reinterpret_cast<uint4*>(smem + (n % QB) * M::kQBytes + (r0 >> 7) * kTile * D * 2 +
                                                (c >> 3) * kTile * 128 + ((r0 & 127) + r) * 128 + (((c & 7) ^ (r & 7)) * 16)));
          }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.q_full[n % QB]);
    }
  } else if (warp < kMmaWarp + 2) {
    // ------------------------------------------------ products
    // One warp per stream, so that neither waits for the other's weights.  The
    // whole warp walks the schedule and one elected lane issues: with the
    // operands uniform over the warp an instruction takes 25 cycles to issue,
    // in a single lane's own branch it took 110.
    constexpr uint32_t id_qk = ptx::idesc_bf16_f32(kTile, kTile);
    constexpr uint32_t id_pv = ptx::idesc_bf16_f32(kTile, D) | (1u << 16);   // B token-major
    constexpr uint32_t hi = ptx::smem_desc_hi_sw128(1024);
    const uint32_t s = __shfl_sync(0xffffffffu, warp - kMmaWarp, 0);         // (uniform)
    const uint32_t t_s = tmem_s(s), t_o = tmem_o(s);
    const uint32_t q_lo = ptx::smem_desc_lo_sw128(q_base), k_lo = ptx::smem_desc_lo_sw128(ring);
    // V: 64-dim column groups lie a whole tile apart
    const uint32_t v_lo = ((ring & 0x3FFFFu) >> 4) | ((uint32_t)(kTile * 128 / 16) << 16);
    uint32_t seg = 0, tile0 = 0, np = 0;       // segments, tiles, weights so far
    // In pairs the streams issue in turns, half a period apart: started
    // together they would form their weights, and then queue for the tensor
    // core, at the same time.
    uint32_t turns = 0;
    auto take_turn = [&]() {
      if (s == 1) wait_bar(&sh.turn[1], turns & 1, sh);
      else if (turns > 0) wait_bar(&sh.turn[0], (turns - 1) & 1, sh);
      ++turns;
    };
    auto pass_turn = [&]() {
      if (lane == 0) ptx::mbar_arrive(&sh.turn[s ^ 1]);
    };
    for (; w.next(a); ++seg) {
      const bool split = w.x.rows <= kTile;
      const int nt = w.x.t1 - w.x.t0;
      // this stream's tiles: every second one from s on, or all
      const int step = split ? 2 : 1, begin = split ? (int)s : 0;
      const uint32_t qb = __shfl_sync(0xffffffffu, seg % QB, 0);
      const uint32_t qa = q_lo + (qb * M::kQBytes + (split ? 0u : s) * kTile * D * 2) / 16;
      wait_bar(&sh.q_full[qb], (seg / QB) & 1, sh);
      auto qk = [&](int i) {
        const uint32_t grp = __shfl_sync(0xffffffffu, ring_k(tile0 + i), 0), slot = grp % S;
        wait_bar(&sh.full[slot], (grp / S) & 1, sh);
        __syncwarp();
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          ptx::fence_proxy_async_smem();          // the rows came through cp.async
          const uint32_t kb = k_lo + slot * (M::kSlotBytes / 16);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            constexpr uint32_t kBlock = kTile * 128 / 16;
            const uint32_t o = (uint32_t)(k / 4) * kBlock + (k % 4) * 2;
            ptx::mma_bf16_split(t_s, qa + o, kb + o, hi, id_qk, k > 0);
          }
          ptx::mma_commit(&sh.s_full[s]);
          ptx::mma_commit(&sh.empty[slot]);
          if (split) ptx::mma_commit(&sh.empty[slot]);    // (for the stream that does not use it)
          if (i + step >= nt) ptx::mma_commit(&sh.q_empty[qb]);
        }
      };
      auto pv = [&](int i) {
        const uint32_t grp = __shfl_sync(0xffffffffu, ring_v(tile0 + i), 0), slot = grp % S;
        wait_bar(&sh.full[slot], (grp / S) & 1, sh);
        wait_bar(&sh.p_full[s], np++ & 1, sh);
        __syncwarp();
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          ptx::fence_proxy_async_smem();
          const uint32_t vb = v_lo + slot * (M::kSlotBytes / 16);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)    // 16 tokens a step
            mma_ts(t_o, t_s + k * 8, vb + k * (2048 / 16), hi, id_pv, i > begin || k > 0);
          ptx::mma_commit(&sh.empty[slot]);
          if (split) ptx::mma_commit(&sh.empty[slot]);
          if (i + step >= nt) ptx::mma_commit(&sh.o_full);
        }
      };
      if (begin < nt) {
        if (!split) take_turn();
        qk(begin);
        if (!split) pass_turn();
        for (int i = begin; i < nt; i += step) {
          if (!split) take_turn();
          pv(i);
          if (i + step < nt) qk(i + step);
          __syncwarp();
          if (!split) pass_turn();
        }
      } else {
        // A stream without a tile has nothing that holds it back: it must not
        // count for this unit's O while the last unit's still misses the
        // other stream's count.
        if (seg > 0) wait_bar(&sh.o_full, (seg - 1) & 1, sh);
        __syncwarp();
        if (ptx::elect_one()) {
          ptx::mma_commit(&sh.q_empty[qb]);
          ptx::mma_commit(&sh.o_full);
        }
      }
      __syncwarp();
      tile0 += nt;
    }
    // every product has landed before the CTA gives its tensor memory back
    if (ptx::elect_one()) ptx::mma_commit(&sh.done);
    __syncwarp();
    const uint64_t t0 = ptx::global_timer();
    while (!ptx::mbar_try_wait_sleep(&sh.done, 0, 100000) && ptx::global_timer() - t0 < kWaitLimitNs) {}
  }
  } else {
    // ------------------------------------------------ softmax and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int s = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;    // TMEM lane 32 * (warp % 4)
    const uint32_t t_s = tmem_s(s) + lanes;
    uint32_t seg = 0, tile0 = 0, ns = 0;
    bool cut = false;                  // the last unit goes on in the next piece
    const float sl2 = a.scale_log2;
    for (; w.next(a); ++seg) {
      const Segment& x = w.x;
      const bool split = x.rows <= kTile;
      const int nt = x.t1 - x.t0, steps = split ? nt : 2 * nt;
      const int row = split ? r : s * kTile + r;          // of this tile of rows
      const bool active = row - lane < x.rows;            // this warp has rows at all
      const int tk = (row0 + row) / a.G;
      const int ctx = x.s.kb + x.s.nt;
      uint64_t tree = 0;
      if (a.tree_mask != nullptr && row < x.rows) tree = a.tree_mask[(size_t)x.b * a.T + tk];
      float m = -INFINITY, l = 0.f;
      for (int j = s; j < steps; j += 2, ++ns) {
        const int i = split ? j : j >> 1;
        uint32_t see[4];
        if (active) {
          // (written before the tile's copies began, and rewritten only when
          // its slots have long been given back)
          const uint32_t v = (tile0 + i) % kValidRing;
          wait_bar(&sh.valid_full[v], ((tile0 + i) / kValidRing) & 1, sh);
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(see[0]), "=r"(see[1]), "=r"(see[2]), "=r"(see[3])
                       : "r"(smem_u32(sh.valid[v]))
                       : "memory");
        }
        wait_bar(&sh.s_full[s], ns & 1, sh);
        __syncwarp();
        ptx::tc_fence_after();
        if (active) {
          const int base = (x.t0 + i) * kTile;
          if (base + kTile > ctx) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int in = ctx - (base + 32 * q);       // context tokens of this word
              if (in >= 32) continue;
              if (a.tree_mask != nullptr) {
                uint32_t bits = in > 0 ? (1u << in) - 1 : 0u;
                bits |= in >= 0 ? (uint32_t)(tree << in) : in > -64 ? (uint32_t)(tree >> -in) : 0u;
                see[q] &= bits;
              } else {
                const int vis = in + tk + 1;              // tokens of this word that the row sees
                see[q] &= vis >= 32 ? 0xffffffffu : vis > 0 ? (1u << vis) - 1 : 0u;
              }
            }
          }
          uint32_t u[kTile];
#pragma unroll
          for (int q = 0; q < 4; ++q) ptx::tmem_ld32(t_s + 32 * q, u + 32 * q);
#pragma unroll
          for (int q = 0; q < 4; ++q) ptx::tmem_wait_ld(u + 32 * q);
          if (__any_sync(0xffffffffu, (see[0] & see[1] & see[2] & see[3]) != 0xffffffffu)) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((see[q] >> e) & 1)) u[32 * q + e] = 0xff800000u;    // -inf: weight 0
          }
          // the tile's maximum
          float mx[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            mx[q] = __uint_as_float(u[32 * q]);
#pragma unroll
            for (int e = 1; e < 31; e += 2)
              mx[q] = fm::max3(mx[q], __uint_as_float(u[32 * q + e]), __uint_as_float(u[32 * q + e + 1]));
            mx[q] = fmaxf(mx[q], __uint_as_float(u[32 * q + 31]));
          }
          const float mz = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
          float alpha = 1.f;
          if (mz > m + kRescale || (m == -INFINITY && mz > m)) {
            if (m != -INFINITY) alpha = fast_exp2(m - mz);
            m = mz;
            l *= alpha;
          }
          const uint64_t sl2x2 = fm::splat2(sl2), off = fm::splat2(m == -INFINITY ? 0.f : -m);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint64_t z =
                  fm::fma2(fm::pack2(__uint_as_float(u[32 * q + 2 * e]), __uint_as_float(u[32 * q + 2 * e + 1])), sl2x2, off);
              const uint64_t pp = fm::exp2_mufu2(z);
              sum[e & 1] = fm::add2(sum[e & 1], pp);
              float p0, p1;
              fm::unpack2(pp, p0, p1);
              p[e] = bf16x2(p0, p1);
            }
            tmem_st16(t_s + 16 * q, p);                   // P lies over S
          }
          float s0, s1;
          fm::unpack2(fm::add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          if (j >= 2 && __any_sync(0xffffffffu, alpha != 1.f)) {
            const uint32_t t_o = tmem_o(s) + lanes;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(t_o + c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(t_o + c, o);
            }
          }
          tmem_wait_st();
        }
        if ((x.t0 + i + 1) * kTile > ctx) {
          // Drafted tokens: a row that does not see one multiplies its V by 0,
          // so an infinity or NaN there is taken out of the product (0
          // instead) and added by the epilogue to the rows that see it.
          const uint32_t grp = ring_v(tile0 + i), slot = grp % S;
          wait_bar(&sh.full[slot], (grp / S) & 1, sh);
          uint8_t* v = smem + M::kRing + slot * M::kSlotBytes;
          const int base = (x.t0 + i) * kTile, from = max(0, ctx - base);
          const int chunks = (min(kTile, ctx + x.s.tn - base) - from) * CPR;
          bool odd = false;
#pragma unroll 1
          for (int k = r; k < chunks; k += kTile) {
            const int tok = from + k / CPR, ch = k % CPR;
            odd |= zero_odd(reinterpret_cast<uint4*>(v + (ch >> 3) * kTile * 128 + tok * 128 + ((ch & 7) ^ (tok & 7)) * 16));
          }
          if (odd) *(volatile int*)&sh.odd_values = 1;
          ptx::fence_proxy_async_smem();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.p_full[s]);
      }
      tile0 += nt;

      // ---- this segment's rows
      wait_bar(&sh.o_full, seg & 1, sh);
      __syncwarp();
      ptx::tc_fence_after();
      float w0 = 1.f, w1 = 0.f;
      int c0 = 0, c1 = D;
      if (split) {
        // join the streams: both warps of a row's lane quarter, half the columns each
        sh.ml[s][r][0] = m;
        sh.ml[s][r][1] = l;
        soft_bar();
        const float ma = sh.ml[0][r][0], la = sh.ml[0][r][1], mb = sh.ml[1][r][0], lb = sh.ml[1][r][1];
        m = fmaxf(ma, mb);
        w0 = ma == -INFINITY ? 0.f : fast_exp2(ma - m);
        w1 = mb == -INFINITY ? 0.f : fast_exp2(mb - m);
        l = la * w0 + lb * w1;
        if (la != la || lb != lb) l = la + lb;            // NaN stays
        c0 = s * (D / 2);
        c1 = c0 + D / 2;
      }
      if (active) {
        const bool live = row < x.rows, whole = x.whole();
        const int h = x.g * a.G + (row0 + row) - tk * a.G;
        const size_t orow = ((size_t)x.b * a.T + tk) * a.H + h;
        const size_t slot = part_slot(blockIdx.x, x.t0 == 0);
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        // 16 columns at a time, rolled: this code runs once a segment, and
        // fetching it unrolled took longer than the work
#pragma unroll 1
        for (int c = c0; c < c1; c += 16) {
          uint32_t u[16];
          float o[16];
          tmem_ld16(tmem_o(split ? 0 : s) + lanes + c, u);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(u[e]);
          if (split) {
            tmem_ld16(tmem_o(1) + lanes + c, u);
            // (an empty stream's columns hold nothing that may be read)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              o[e] = (w0 == 0.f ? 0.f : o[e] * w0) + (w1 == 0.f ? 0.f : __uint_as_float(u[e]) * w1);
          }
          if (live && whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * D + c);
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              dst[e / 8] = make_uint4(bf16x2(o[e] * inv, o[e + 1] * inv), bf16x2(o[e + 2] * inv, o[e + 3] * inv),
                                      bf16x2(o[e + 4] * inv, o[e + 5] * inv), bf16x2(o[e + 6] * inv, o[e + 7] * inv));
          } else if (live) {
            float4* dst = reinterpret_cast<float4*>(a.part_o) + (slot * (D / 4) + c / 4) * QT + row;
#pragma unroll
            for (int e = 0; e < 16; e += 4) dst[(e / 4) * QT] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        if (*(volatile int*)&sh.odd_values != 0 && live) {
          // infinities and NaN of the drafted tokens that this row sees, added
          // to what this thread has just written
          const int d0 = max(0, x.t0 * kTile - ctx), d1 = min(x.s.tn, x.t1 * kTile - ctx);
#pragma unroll 1
          for (int dt = d0; dt < d1; ++dt) {
            if (a.tree_mask != nullptr ? !((tree >> dt) & 1) : dt > tk) continue;
            const int pos = x.s.nv + x.s.nt + dt;
            const int page = __ldg(a.block_table + (size_t)x.b * a.max_blocks + (pos >> 4));
            if (page < 0 || page >= a.num_blocks) continue;
            const uint16_t* v =
                static_cast<const uint16_t*>(a.v_pool) + ((((size_t)page * a.Hkv + x.g) << 4) + (pos & 15)) * D;
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
              const uint32_t bits = __ldg(v + c);
              if ((bits & 0x7f80u) != 0x7f80u) continue;
              uint16_t* out = static_cast<uint16_t*>(a.out) + orow * D + c;
              float* part = a.part_o + ((slot * (D / 4) + c / 4) * QT + row) * 4 + (c & 3);
              const float sum = __uint_as_float(bits << 16) + (whole ? __uint_as_float((uint32_t)*out << 16) : *part);
              if (whole) *out = (uint16_t)f32_to_bf16_bits(sum);
              else *part = sum;
            }
          }
        }
        if (live && c0 == 0) {
          if (!whole) reinterpret_cast<float2*>(a.part_ml)[slot * QT + row] = make_float2(m, l);
          else if (a.lse != nullptr) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
      }
      if (threadIdx.x == 0 && x.t0 == 0 && a.columns > 1) {
        // for the merge: the unit that begins here, its last piece (-1: it is
        // whole), its rows and the line's length; kept by unit (with this
        // CTA) where there are fewer units than CTAs, else by CTA (with the
        // sequence)
        int last = -1;
        if (x.t1 < x.tiles) {
          const int end = piece_begin(sh.total, col + 1, a.columns) + x.tiles - x.t1;
          for (last = col + 1; last + 1 < a.columns && piece_begin(sh.total, last + 1, a.columns) < end; ++last) {}
          cut = true;
        }
        const int at = a.by_unit ? (x.b * a.Hkv + x.g) * a.row_tiles + (int)(blockIdx.x % a.row_tiles) : (int)blockIdx.x;
        if (a.by_unit || last >= 0)
          reinterpret_cast<int4*>(a.part_unit)[at] =
              make_int4(a.by_unit ? (int)blockIdx.x : x.b, x.g, last, x.rows | min(sh.total, 0x7fff) << 16);
      }
      // the next segment's products overwrite what the other stream's warps read
      ptx::tc_fence_before();
      soft_bar();
      ptx::tc_fence_after();
    }
    if (threadIdx.x == 0 && a.columns > 1 && !a.by_unit && !cut)
      reinterpret_cast<int4*>(a.part_unit)[blockIdx.x] = make_int4(0, 0, -1, 0);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && (sh.abort || misplaced)) flag_status(a.status, kStatusTimeout);
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(sh.tmem, kTmemCols);
  }
}

// (M, L, O) of two parts of a row, the second given by (m, l): the factors
// that M's side and m's side take.
__device__ __forceinline__ void join(float& M, float& L, float m, float l, float& w0, float& w1) {
  const float x = fmaxf(M, m);
  w0 = M == -INFINITY ? 0.f : fast_exp2(M - x);
  w1 = m == -INFINITY ? 0.f : fast_exp2(m - x);
  L = (L == 0.f ? 0.f : L * w0) + (l == 0.f ? 0.f : l * w1);
  M = x;
}
__device__ __forceinline__ float4 join4(float4 a, float w0, float4 b, float w1) {
  return make_float4(a.x * w0 + b.x * w1, a.y * w0 + b.y * w1, a.z * w0 + b.z * w1, a.w * w0 + b.w * w1);
}

// Joins the partials of the units that were cut: a block has 32 rows x 32 dims
// of one that a CTA of the kernel above began.  Its warps take
// every eighth piece each (a unit may lie in two or in a hundred; one after the
// other they took 14 us for 38), then the eight results are joined, always in
// the same order.  Bound by latency (ncu, alone and with cold caches: 11.4 us
// for 152 pieces of 189 rows, 32 MB of L2 traffic, 15 MB of them from memory).
template <int D, int QT>
__global__ void __launch_bounds__(256)
tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ float4 part[8][8][32];    // [warp][dim / 4][row]
  __shared__ float2 part_ml[8][32];
  grid_dep_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y * 32 + lane;
  const int4 unit = __ldcg(reinterpret_cast<const int4*>(a.part_unit) + blockIdx.x);
  int b = unit.x, g = unit.y, cta = blockIdx.x;
  if (a.by_unit) {
    cta = unit.x;
    // (a unit without tiles, which no CTA has entered, has no rows either)
    const int u = blockIdx.x / a.row_tiles;
    b = u / a.Hkv;
    g = u - b * a.Hkv;
    Seq s;
    seq_of(a, b, s);
    if ((int)(blockIdx.x % a.row_tiles) * QT >= s.tn * a.G) return;
  }
  const int rows = unit.w & 0xffff, total = unit.w >> 16;   // total: exact where it is less than the pieces
  if (unit.z < 0 || (int)blockIdx.y * 32 >= rows) return;
  const int rt = cta % a.row_tiles, p0 = cta / a.row_tiles;
  float M = -INFINITY, L = 0.f;
  float4 acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = p0 + warp; p <= unit.z && row < rows; p += 8) {
    if (total < a.columns && piece_begin(total, p, a.columns) == piece_begin(total, p + 1, a.columns)) continue;
    const size_t slot = part_slot(p * a.row_tiles + rt, p == p0);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot * QT + row);
    const float4* src = reinterpret_cast<const float4*>(a.part_o) + (slot * (D / 4) + blockIdx.z * 8) * QT + row;
    float4 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __ldcg(src + i * QT);
    float w0, w1;
    join(M, L, ml.x, ml.y, w0, w1);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = join4(acc[i], w0, o[i], w1);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[warp][i][lane] = acc[i];
  part_ml[warp][lane] = make_float2(M, L);
  __syncthreads();
  if (row >= rows) return;
  // this thread: four dims of its row
  const int n = min(8, unit.z - p0 + 1);
  float4 o = part[0][warp][lane];
  M = part_ml[0][lane].x;
  L = part_ml[0][lane].y;
  for (int i = 1; i < n; ++i) {
    float w0, w1;
    join(M, L, part_ml[i][lane].x, part_ml[i][lane].y, w0, w1);
    o = join4(o, w0, part[i][warp][lane], w1);
  }
  const int c4 = blockIdx.z * 8 + warp;
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
  const int r = rt * QT + row, t = r / a.G, h = g * a.G + r - t * a.G;
  const size_t orow = ((size_t)b * a.T + t) * a.H + h;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + 4 * c4) =
      make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
  if (a.lse != nullptr && c4 == 0) a.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

namespace {

// Row tiles of 128 rows, or of 256 when there are more rows than that and at
// least eight tiles of 256 rows x 128 tokens for each CTA: the paired streams
// read the cache half as often, but a piece of theirs starts and ends with
// twice the rows.  128 against 256, 8 sequences of 4 KV heads, d 128: 224 rows
// 23.2 / 26.3 us at 2 such tiles a CTA, 28.3 / 30.5 at 4, 37.7 / 38.2 at 8, 72.3 /
// 67.7 at 24; 448 rows 32.5 / 35.1 at 4, 41.7 / 42.6 at 8, 59.8 / 57.1 at 16: at
// eight the two are within 2 % of one another, and 256 win somewhere between
// there and 16.  As many pieces of each row tile as SMs divided by the row
// tiles, rounded down, of two token tiles at least (one for each stream; pieces
// of one measured 2 % faster to 9 % slower).
struct Plan {
  int QT, row_tiles, columns;
  bool cut() const { return columns > 1; }
  size_t ctas() const { return (size_t)columns * row_tiles; }
};
Plan plan_of(int B, int T, int G, int Hkv, int n_tokens) {
  Plan p;
  const long long rows = (long long)T * G;
  const long long tiles = (long long)B * Hkv * (((long long)n_tokens + kTile - 1) / kTile);
  const long long pairs = (rows + 2 * kTile - 1) / (2 * kTile);
  p.QT = rows <= kTile || tiles < (8 * kCtas + pairs - 1) / (pairs > 0 ? pairs : 1) ? kTile : 2 * kTile;
  p.row_tiles = (int)((rows + p.QT - 1) / p.QT);
  long long c = p.row_tiles > 0 ? kCtas / p.row_tiles : 1;
  if (c > tiles / 2) c = tiles / 2;
  p.columns = (int)(c < 1 ? 1 : c);
  return p;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

template <int D, int QT>
cudaError_t launch_qt(const TreeArgs& a, cudaStream_t stream) {
  auto kernel = tree_attn_kernel<D, QT>;
  const size_t smem = Smem<D, QT>::kBytes;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  return launch_dependent(kernel, dim3((unsigned)(a.columns * a.row_tiles)), dim3(kThreads), smem, stream, a);
}

}  // namespace

// Workspace: the cut units | (m, l) of every partial row | their O.
// The rows of partials are those of the plan, or for the size that a caller
// asks for a bound that no call with fewer sequences, tokens or rows exceeds: a
// plan has at most one CTA per SM and at most one per two token tiles of each
// row tile, and 256-row tiles come only with more rows and tokens than 128-row
// ones.  (The plan itself is no such bound: 74 rows take less than 73, and with
// more row tiles than half the SMs nothing is cut.)
struct Layout {
  size_t ml, o, total;
};
static Layout layout_of(size_t ctas, int QT, int D) {
  const size_t rows = ctas * 2 * QT;
  Layout l;
  l.ml = round256(ctas * sizeof(int4));
  l.o = l.ml + round256(rows * sizeof(float2));
  l.total = l.o + rows * D * sizeof(float);
  return l;
}

size_t tree_attn_workspace_bytes(int B, int T, int H, int Hkv, int D, int n_tokens) {
  const Plan p = plan_of(B, T, H / Hkv, Hkv, n_tokens);
  const long long tiles = (long long)B * Hkv * (((long long)n_tokens + kTile - 1) / kTile);
  const long long most = tiles / 2 > 1 ? p.row_tiles * (tiles / 2) : 0;
  return layout_of((size_t)(most < kCtas ? most : kCtas), p.QT, D).total;
}

cudaError_t launch_tree_attn(const TreeArgs& args, cudaStream_t stream) {
  TreeArgs a = args;
  a.G = a.H / a.Hkv;
  const Plan p = plan_of(a.batch, a.T, a.G, a.Hkv, a.k_vis + a.n_text + a.T);
  const Layout l = layout_of(p.cut() ? p.ctas() : 0, p.QT, a.D);
  char* ws = static_cast<char*>(a.ws);
  a.row_tiles = p.row_tiles;
  a.columns = p.columns;
  a.by_unit = (long long)a.batch * a.Hkv * p.row_tiles <= (long long)p.ctas();
  a.part_unit = reinterpret_cast<int*>(ws);
  a.part_ml = reinterpret_cast<float*>(ws + l.ml);
  a.part_o = reinterpret_cast<float*>(ws + l.o);
  cudaError_t e;
  if (a.D == 128) e = p.QT == 128 ? launch_qt<128, 128>(a, stream) : launch_qt<128, 256>(a, stream);
  else e = p.QT == 128 ? launch_qt<64, 128>(a, stream) : launch_qt<64, 256>(a, stream);
  if (e != cudaSuccess || !p.cut()) return e;
  if (!a.lens.any() && a.n_new == nullptr && (a.tree_mask != nullptr || p.row_tiles == 1)) {
    // equal lengths: nothing to join when every piece ends with a unit
    const int tiles = (a.k_vis + a.n_text + a.T + kTile - 1) / kTile, total = tiles * a.batch * a.Hkv;
    bool whole = true;
    for (int c = 1; c < p.columns; ++c) whole = whole && (long long)total * c / p.columns % tiles == 0;
    if (whole) return e;
  }
  const long long rows = (long long)a.T * a.G;
  const dim3 grid((unsigned)(a.by_unit ? a.batch * a.Hkv * p.row_tiles : (int)p.ctas()), (unsigned)(((rows < p.QT ? rows : p.QT) + 31) / 32), (unsigned)(a.D / 32));
  auto merge = a.D == 128 ? (p.QT == 128 ? tree_merge_kernel<128, 128> : tree_merge_kernel<128, 256>)
                          : (p.QT == 128 ? tree_merge_kernel<64, 128> : tree_merge_kernel<64, 256>);
  return launch_dependent(merge, grid, dim3(256), 0, stream, a);
}

}  // namespace sv
