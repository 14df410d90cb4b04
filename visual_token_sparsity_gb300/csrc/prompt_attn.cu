// Causal attention of whole prompts: packed sequences, grouped heads, read from
// the token-major projections (slices of a fused one, for instance).
//
//   out_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j,  i and j in one sequence
//
// Both products are matrix products on the tcgen05 tensor cores: S = Q K^T (128
// rows x 128 tokens), then O += P V with P as the bf16 A operand in tensor
// memory and V read token-major from shared memory; one pass with a running
// maximum and sum per row in fp32 registers, the accumulator rescaled only when
// a row's maximum grows far beyond it.  The G query heads of a KV head share its
// keys and values, so a tile of rows is floor(128 / G) tokens times G heads.
//
// A CTA runs two streams, tiles of neighbouring tokens, each with its own S, P
// and O in tensor memory and four softmax warps: the products of one run while
// the other's weights are formed, and a tile of keys and values serves both.
// Units (sequence, KV head, pair of row tiles) are handed out by a counter, a
// sequence's longest first, to one CTA per SM; a stream goes on to its next
// unit's products while its softmax warps still write the last one's rows.
//
// Warps: 0-7 softmax and epilogue (one row per thread), 8-9 MMA issue (one per
// stream), 10 the units and the TMA loads (11 makes the group of four whole that
// gives registers up).
//
// Measured, inputs out of L2: 12800 tokens of 28 heads over 4, d 128 730 us, 1.61
// PFLOP/s (82 % of what the device reaches on a plain matrix product in a short burst),
// and 790 us, 1.49 PFLOP/s, in seconds of calls at the power limit (85 % of a matrix
// product there; SM clock 1.85 to 1.90 GHz against 2.07); 4 x 3008 tokens of 32 heads 228
// and 245 us; 48 questions of up to 97 tokens 18.1 us; one of 176 tokens, 4 heads over 2,
// d 64 6.6 us.  What bounds the long ones: a tile takes a stream some
// 3100 cycles against 2048 in the products, as load and maximum of S (600) and the
// weights (850) of a stream stand between its own two products; and some 3000 a unit
// for its rows.  With sixteen softmax warps 880 / 264 us (registers spill), the
// maximum taken over chunks while others load 832 / 250, streams in turns 831 / 247,
// rows written through shared memory 770 / 256.
//
// A token that a row does not see has weight 0, which an infinity or NaN of its
// V (or a row of the next sequence's) turns into NaN.  Such rows show in the
// output, where a row that is not finite is formed again by one warp over
// exactly its own tokens.
#include "common.cuh"
#include "fastmath.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"
#include "tensor_map.h"

namespace sv {

namespace {

constexpr int kTile = 128;                 // rows of a stream, tokens of a tile
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 10;
constexpr int kThreads = 384;              // at 168 registers at launch
// A softmax thread holds a row of S (128 columns).
constexpr int kSoftRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftRegs + 128 * kOtherRegs <= kThreads * 168, "register split");
constexpr int kTmemCols = 512;             // S0 | S1 | O0 | O1, 128 columns each
constexpr int kUnits = 4;                  // units on their way
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kRescale = 32.f;           // a row's reference is raised when its maximum outgrows it by 2^32
constexpr size_t kMaxSmem = 232448;

template <int D>
struct Smem {
  static constexpr int kTileBytes = kTile * D * 2;       // Q, K or V
  static constexpr int kSlots = D == 128 ? 5 : 10;       // K and V tiles beside two of Q
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kBytes = kRing + kSlots * kTileBytes;
};

// Tokens [first, first + n) of sequence [begin, begin + len) are a stream's rows
// times the G heads of KV head g; len < 0: no more units.
struct Unit {
  int begin, len, tok0, g;
};

struct Shared {
  uint64_t kv_full[10], kv_empty[10];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2];
  uint64_t unit_full[kUnits], unit_empty[kUnits], done;
  uint32_t tmem;
  int abort, progress;
  Unit unit[kUnits];
};
constexpr int kStaticSmem = 2 * 1024;
static_assert(sizeof(Shared) <= kStaticSmem && Smem<128>::kBytes + kStaticSmem <= kMaxSmem &&
                  Smem<64>::kBytes + kStaticSmem <= kMaxSmem, "shared memory");

// Waits for a phase, up to 2 s without progress.
__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t parity, Shared& sh) {
  if (ptx::mbar_try_wait(bar, parity)) return;
  uint64_t t0 = ptx::global_timer();
  int seen = *(volatile int*)&sh.progress;
  for (;;) {
    if (ptx::mbar_try_wait_sleep(bar, parity, 100000)) return;
    if (*(volatile int*)&sh.abort) return;
    if (ptx::global_timer() - t0 > kWaitLimitNs) {
      const int now = *(volatile int*)&sh.progress;
      if (now == seen) {
        *(volatile int*)&sh.abort = 1;
        return;
      }
      seen = now;
      t0 = ptx::global_timer();
    }
  }
}

// Whether a wait gave up, the same for the whole warp.
__device__ __forceinline__ bool aborted(Shared& sh) { return __any_sync(0xffffffffu, *(volatile int*)&sh.abort); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 32 bytes, in one store where the address is a multiple of 32: a lane's rows lie
// in lines of their own, and each store visits all of them.
__device__ __forceinline__ void store32(uint16_t* dst, const uint32_t* w, bool aligned) {
  if (aligned) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

__host__ __device__ constexpr uint32_t tmem_s(int s) { return s * 128; }
__host__ __device__ constexpr uint32_t tmem_o(int s) { return 256 + s * 128; }

// Tiles of keys that the rows of stream s of a unit see (0: it has no rows).
__device__ __forceinline__ int tiles_of(const Unit& u, int s, int tpt) {
  const int first = u.tok0 + s * tpt;
  return first < u.len ? (min(first + tpt, u.len) + kTile - 1) / kTile : 0;
}

// One query row by one warp: a lane per key for the products with K, then the
// lanes over the dims of V.
template <int D>
__device__ __noinline__ void attend_row(const PromptArgs& a, int begin, int tk, int g, int h, Shared& sh) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + (size_t)(begin + tk) * a.q_stride + (size_t)h * D;
  const uint16_t* k = static_cast<const uint16_t*>(a.k) + (size_t)begin * a.k_stride + (size_t)g * D;
  const uint16_t* v = static_cast<const uint16_t*>(a.v) + (size_t)begin * a.v_stride + (size_t)g * D;
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int j0 = 0; j0 <= tk; j0 += 32) {
    const int j = j0 + lane, cnt = min(32, tk + 1 - j0);
    float z = -INFINITY;
    if (j <= tk) {
      float dot = 0.f;
      const uint4* src = reinterpret_cast<const uint4*>(k + (size_t)j * a.k_stride);
#pragma unroll 1
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = __ldg(src + c), y = __ldg(reinterpret_cast<const uint4*>(q) + c);
        const uint32_t* xs = reinterpret_cast<const uint32_t*>(&x);
        const uint32_t* ys = reinterpret_cast<const uint32_t*>(&y);
#pragma unroll
        for (int e = 0; e < 4; ++e) dot = fmaf(bf16_hi(ys[e]), bf16_hi(xs[e]), fmaf(bf16_lo(ys[e]), bf16_lo(xs[e]), dot));
      }
      z = dot * a.scale_log2;
    }
    const float mx = fmaxf(m, warp_max(z)), off = mx == -INFINITY ? 0.f : mx;
    const float alpha = m == -INFINITY ? 0.f : fast_exp2(m - off), p = j <= tk ? fast_exp2(z - off) : 0.f;
    m = mx;
    l = l * alpha + warp_sum(p);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= alpha;
#pragma unroll 1
    for (int i = 0; i < cnt; ++i) {
      const float w = __shfl_sync(0xffffffffu, p, i);
      const uint16_t* src = v + (size_t)(j0 + i) * a.v_stride + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(src + e));
        o[e] = fmaf(w, bf16_lo(x), o[e]);
        o[e + 1] = fmaf(w, bf16_hi(x), o[e + 1]);
      }
    }
    if (lane == 0) atomicAdd(&sh.progress, 1);
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  const size_t row = (size_t)(begin + tk) * a.H + h;
#pragma unroll
  for (int e = 0; e < E; ++e)
    static_cast<uint16_t*>(a.out)[row * D + lane * E + e] = (uint16_t)f32_to_bf16_bits(o[e] * inv);
  if (lane == 0 && a.lse != nullptr) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_attn_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using M = Smem<D>;
  constexpr int S = M::kSlots, TB = M::kTileBytes;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Shared sh;
  const uint32_t q_base = smem_u32(smem), ring = q_base + M::kRing;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.Hkv, tpt = kTile / G;           // tokens of a row tile

  if (warp == 0) ptx::tmem_alloc(&sh.tmem, kTmemCols);
  if (warp == 1) {
    if (lane < S) {
      ptx::mbar_init(&sh.kv_full[lane], 1);
      ptx::mbar_init(&sh.kv_empty[lane], 2);            // both streams
    } else if (lane < S + 2) {
      const int s = lane - S;
      ptx::mbar_init(&sh.q_full[s], 1);
      ptx::mbar_init(&sh.q_empty[s], 1);
      ptx::mbar_init(&sh.s_full[s], 1);
      ptx::mbar_init(&sh.p_full[s][0], 4);
      ptx::mbar_init(&sh.p_full[s][1], 4);
      ptx::mbar_init(&sh.o_full[s], 1);
    } else if (lane < S + 2 + kUnits) {
      ptx::mbar_init(&sh.unit_full[lane - S - 2], 1);
      ptx::mbar_init(&sh.unit_empty[lane - S - 2], kSoftWarps + 2);
    } else if (lane == S + 2 + kUnits) {
      ptx::mbar_init(&sh.done, 2);
      sh.abort = sh.progress = 0;
    }
    ptx::mbar_fence_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    ptx::prefetch_tensormap(&map_q);
    ptx::prefetch_tensormap(&map_k);
    ptx::prefetch_tensormap(&map_v);
  }
  grid_dep_sync();                                      // (nothing before it touches global memory)
  // the starts have to ascend within the tokens; otherwise nothing is computed
  bool bad = false;
  for (int b = threadIdx.x; b <= a.batch; b += kThreads) {
    const int s = __ldg(a.seq_start + b);
    bad = bad || s < 0 || s > a.N || (b > 0 && __ldg(a.seq_start + b - 1) > s);
  }
  ptx::tc_fence_before();
  bad = __syncthreads_or(bad);
  ptx::tc_fence_after();
  const bool misplaced = sh.tmem != 0 || (q_base & 1023u) != 0;     // (cannot be)
  const bool idle = bad || misplaced;

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kLoadWarp) {
    // ------------------------------------------------ units and loads
    uint32_t u = blockIdx.x, n_unit = 0, kv = 0, nq[2] = {0, 0};
    uint32_t before = 0;                                // units of the sequences before b0
    int b0 = 0;
    for (;; ++n_unit) {
      Unit x = {0, -1, 0, 0};
      while (!idle && b0 < a.batch) {
        // 32 sequences at a time
        const int b = b0 + lane;
        int s0 = 0, s1 = 0;
        if (b < a.batch) {
          s0 = __ldg(a.seq_start + b);
          s1 = __ldg(a.seq_start + b + 1);
        }
        const uint32_t pairs = (uint32_t)(s1 - s0 + 2 * tpt - 1) / (uint32_t)(2 * tpt), mine = pairs * (uint32_t)a.Hkv;
        uint32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, before + inc > u);
        if (hit) {
          const int f = __ffs(hit) - 1;
          const uint32_t local = u - before - __shfl_sync(0xffffffffu, inc - mine, f);
          const uint32_t pf = __shfl_sync(0xffffffffu, pairs, f), nth = local / (uint32_t)a.Hkv;
          x.begin = __shfl_sync(0xffffffffu, s0, f);
          x.len = __shfl_sync(0xffffffffu, s1, f) - x.begin;
          x.g = (int)(local - nth * (uint32_t)a.Hkv);
          x.tok0 = (int)(pf - 1 - nth) * 2 * tpt;       // a sequence's longest first
          break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
        b0 += 32;
      }
      const uint32_t us = n_unit % kUnits;
      if (n_unit >= kUnits) wait_bar(&sh.unit_empty[us], (n_unit / kUnits - 1) & 1, sh);
      if (lane == 0) {
        sh.unit[us] = x;
        ptx::mbar_arrive(&sh.unit_full[us]);
      }
      if (x.len < 0 || aborted(sh)) break;
      if (lane == 0) {
        const int n0 = tiles_of(x, 0, tpt), n1 = tiles_of(x, 1, tpt), n = max(n0, n1);
        auto load_q = [&](int s) {
          if (nq[s] > 0) wait_bar(&sh.q_empty[s], (nq[s] - 1) & 1, sh);
          ++nq[s];
          ptx::mbar_arrive_expect_tx(&sh.q_full[s], (D / 64) * 128 * G * tpt);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            ptx::tma_load_3d(smem + s * TB + c * kTile * 128, &map_q, c * 64, x.g * G, x.begin + x.tok0 + s * tpt,
                             &sh.q_full[s]);
        };
        auto load_kv = [&](const CUtensorMap* map, int j) {
          const uint32_t slot = kv % S;
          if (kv >= (uint32_t)S) wait_bar(&sh.kv_empty[slot], (kv / S - 1) & 1, sh);
          ++kv;
          ptx::mbar_arrive_expect_tx(&sh.kv_full[slot], TB);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            ptx::tma_load_3d(smem + M::kRing + slot * TB + c * kTile * 128, map, c * 64, x.g, x.begin + j * kTile,
                             &sh.kv_full[slot]);
        };
        load_q(0);
        for (int j = 0; j < n; ++j) {
          load_kv(&map_k, j);
          if (j == 0 && n1 > 0) load_q(1);
          load_kv(&map_v, j);
        }
        u = gridDim.x + (uint32_t)atomicAdd(a.counters, 1);
      }
      u = __shfl_sync(0xffffffffu, u, 0);
    }
    // no copy is on its way when the CTA leaves (after a wait that gave up it might be)
    if (lane == 0) {
      const uint64_t t0 = ptx::global_timer();
      auto landed = [&](uint64_t* bar, uint32_t parity) {
        while (!ptx::mbar_try_wait_sleep(bar, parity, 100000) && ptx::global_timer() - t0 < kWaitLimitNs) {}
      };
      for (uint32_t i = kv > (uint32_t)S ? kv - S : 0; i < kv; ++i) landed(&sh.kv_full[i % S], (i / S) & 1);
      for (int s = 0; s < 2; ++s)
        if (nq[s] > 0) landed(&sh.q_full[s], (nq[s] - 1) & 1);
    }
    // the counters are zero again when the last CTA leaves
    if (lane == 0) {
      __threadfence();
      if (atomicAdd(a.counters + 1, 1) == (int)gridDim.x - 1) {
        a.counters[0] = 0;
        a.counters[1] = 0;
      }
    }
  } else if (warp < kMmaWarp + 2) {
    // ------------------------------------------------ products
    // One warp per stream: waits, issue and commits of a tile take a warp 1400
    // cycles, so that one for both streams was the bound.  The whole warp walks
    // the schedule and one elected lane issues (operands uniform over the warp).
    constexpr uint32_t id_qk = ptx::idesc_bf16_f32(kTile, kTile);
    constexpr uint32_t id_pv = ptx::idesc_bf16_f32(kTile, D) | (1u << 16);   // B token-major
    constexpr uint32_t hi = ptx::smem_desc_hi_sw128(1024);
    const int s = __shfl_sync(0xffffffffu, warp - kMmaWarp, 0);              // (uniform)
    const uint32_t t_s = tmem_s(s), t_o = tmem_o(s);
    const uint32_t qa = ptx::smem_desc_lo_sw128(q_base) + s * (TB / 16), k_lo = ptx::smem_desc_lo_sw128(ring);
    // V: 64-dim column groups lie a whole tile apart
    const uint32_t v_lo = ((ring & 0x3FFFFu) >> 4) | ((uint32_t)(kTile * 128 / 16) << 16);
    uint32_t slot = 0, phase = 0;      // of the next tile in the ring
    auto advance = [&]() {
      if (++slot == (uint32_t)S) {
        slot = 0;
        phase ^= 1;
      }
    };
    uint32_t vslot = 0, vphase = 0;    // of the V tile that a pending value product reads
    uint32_t units = 0, items = 0;     // with rows, products of weights so far
    bool pending = false, first = false, last = false;
    auto value_product = [&]() {
      wait_bar(&sh.kv_full[vslot], vphase, sh);
      const uint32_t vb = v_lo + vslot * (TB / 16);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        wait_bar(&sh.p_full[s][half], items & 1, sh);
        __syncwarp();
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
#pragma unroll
          for (int k = 4 * half; k < 4 * half + 4; ++k)                      // 16 tokens a step
            ptx::mma_ts(t_o, t_s + k * 8, vb + k * (2048 / 16), hi, id_pv, !first || k > 0);
          if (half == 1) {
            ptx::mma_commit(&sh.kv_empty[vslot]);
            if (last) ptx::mma_commit(&sh.o_full[s]);
          }
        }
        __syncwarp();
      }
      ++items;
      pending = false;
    };
    for (uint32_t unit = 0;; ++unit) {
      const uint32_t us = unit % kUnits;
      wait_bar(&sh.unit_full[us], (unit / kUnits) & 1, sh);
      const Unit x = sh.unit[us];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.unit_empty[us]);
      if (x.len < 0 || aborted(sh)) break;
      const int n = tiles_of(x, s, tpt), most = max(tiles_of(x, 0, tpt), tiles_of(x, 1, tpt));
      for (int j = 0; j < n; ++j) {
        // the value product of the tile before (the last unit's, too), then the
        // logits of this one, which take the place of its weights
        if (pending) value_product();
        if (j == 0) wait_bar(&sh.q_full[s], units++ & 1, sh);
        wait_bar(&sh.kv_full[slot], phase, sh);
        __syncwarp();
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint32_t kb = k_lo + slot * (TB / 16);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            constexpr uint32_t kBlock = kTile * 128 / 16;
            const uint32_t o = (uint32_t)(k / 4) * kBlock + (k % 4) * 2;
            ptx::mma_bf16_split(t_s, qa + o, kb + o, hi, id_qk, k > 0);
          }
          ptx::mma_commit(&sh.s_full[s]);
          ptx::mma_commit(&sh.kv_empty[slot]);
          if (j == n - 1) ptx::mma_commit(&sh.q_empty[s]);
        }
        __syncwarp();
        advance();
        vslot = slot;
        vphase = phase;
        advance();
        first = j == 0;
        last = j == n - 1;
        pending = true;
      }
      // Tiles that this stream's rows do not see: given back when they are there
      // (the pending product first, so that nothing waits for a slot that it holds).
      if (n < most && pending) value_product();
      for (int j = 2 * n; j < 2 * most; ++j) {
        wait_bar(&sh.kv_full[slot], phase, sh);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.kv_empty[slot]);
        advance();
      }
    }
    if (pending && !aborted(sh)) value_product();
    // every product has landed before the CTA gives its tensor memory back
    if (ptx::elect_one()) ptx::mma_commit(&sh.done);
    __syncwarp();
    const uint64_t t0 = ptx::global_timer();
    while (!ptx::mbar_try_wait_sleep(&sh.done, 0, 100000) && ptx::global_timer() - t0 < kWaitLimitNs) {}
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ------------------------------------------------ softmax and epilogue
    const int s = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;    // TMEM lane 32 * (warp % 4)
    const uint32_t t_s = tmem_s(s) + lanes, t_o = tmem_o(s) + lanes;
    const float sl2 = a.scale_log2;
    const int rt = r / G, rh = r - rt * G;                // this row's token and head of the tile
    const bool whole_sectors = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    uint32_t unit = 0, ns = 0, units = 0;
    for (;; ++unit) {
      const uint32_t us = unit % kUnits;
      wait_bar(&sh.unit_full[us], (unit / kUnits) & 1, sh);
      const Unit x = sh.unit[us];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.unit_empty[us]);
      if (x.len < 0 || aborted(sh)) break;
      const int n = tiles_of(x, s, tpt), first = x.tok0 + s * tpt, tk = first + rt;
      if (n == 0) continue;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++ns) {
        wait_bar(&sh.s_full[s], ns & 1, sh);
        __syncwarp();
        ptx::tc_fence_after();
        if (j * kTile + kTile - 1 > first) {
          // Some row does not see all columns: those are set to -inf (weight 0) in
          // tensor memory, 16 at a time from the first that any row of the warp does
          // not see (rolled: code beside the loop's costs the loop its fetches).
          const int vis = tk - j * kTile;                 // columns 0 .. vis are seen
          const int from = max(0, __reduce_min_sync(0xffffffffu, vis) + 1) & ~15;
#pragma unroll 1
          for (int c = from; c < kTile; c += 16) {
            uint32_t o[16];
            ptx::tmem_ld16(t_s + c, o);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (c + e > vis) o[e] = 0xff800000u;
            ptx::tmem_st16(t_s + c, o);
          }
          ptx::tmem_wait_st();
        }
        uint32_t u[kTile];
#pragma unroll
        for (int q = 0; q < 4; ++q) ptx::tmem_ld32(t_s + 32 * q, u + 32 * q);
#pragma unroll
        for (int q = 0; q < 4; ++q) ptx::tmem_wait_ld(u + 32 * q);
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
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // (the last product of weights has landed: S came behind it)
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            ptx::tmem_ld16(t_o + c, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            ptx::tmem_st16(t_o + c, o);
          }
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
          ptx::tmem_st16(t_s + 16 * q, p);                // P lies over S
          if (q & 1) {
            // half of the weights: their product may begin
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sh.p_full[s][q >> 1]);
          }
        }
        float s0, s1;
        fm::unpack2(fm::add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }

      // ---- this unit's rows
      wait_bar(&sh.o_full[s], units++ & 1, sh);
      __syncwarp();
      ptx::tc_fence_after();
      const bool live = rt < tpt && tk < x.len;
      const int h = x.g * G + rh;
      const size_t orow = (size_t)(x.begin + tk) * a.H + h;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      bool odd = false;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        ptx::tmem_ld32(t_o + c, o);
        ptx::tmem_wait_ld(o);
        uint16_t* dst = static_cast<uint16_t*>(a.out) + orow * D + c;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            w[e] = bf16x2(__uint_as_float(o[16 * q + 2 * e]) * inv, __uint_as_float(o[16 * q + 2 * e + 1]) * inv);
            odd = odd || (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
          }
          if (live) store32(dst + 16 * q, w, whole_sectors);
        }
      }
      if (live && a.lse != nullptr) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      // rows that are not finite, over exactly the tokens that they see
      uint32_t again = __ballot_sync(0xffffffffu, odd && live);
      if (again) __syncwarp();                            // (their lanes have stored what is written again)
      while (again) {
        const int f = __ffs(again) - 1;
        again &= again - 1;
        attend_row<D>(a, x.begin, __shfl_sync(0xffffffffu, tk, f), x.g, __shfl_sync(0xffffffffu, h, f), sh);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (sh.abort || misplaced) flag_status(a.status, kStatusTimeout);
    if (bad && blockIdx.x == 0) flag_status(a.status, kStatusBadLength);
  }
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(sh.tmem, kTmemCols);
  }
}

namespace {

// bf16 [tokens][heads][d] rows, `stride` elements between tokens; boxes of 64
// columns, `box_heads` heads and `box_tokens` tokens, 128-byte swizzled.
bool make_map(CUtensorMap* map, const void* base, int d, int heads, int tokens, long long stride, int box_heads,
              int box_tokens) {
  EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_d(const PromptArgs& a, int num_sms, cudaStream_t stream) {
  const int G = a.H / a.Hkv, tpt = kTile / G;
  CUtensorMap q, k, v;
  if (!make_map(&q, a.q, D, a.H, a.N, a.q_stride, G, tpt) || !make_map(&k, a.k, D, a.Hkv, a.N, a.k_stride, 1, kTile) ||
      !make_map(&v, a.v, D, a.Hkv, a.N, a.v_stride, 1, kTile))
    return cudaErrorInvalidValue;
  auto kernel = prompt_attn_kernel<D>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  // at most one pair of row tiles more per sequence than the tokens fill
  const long long units = ((long long)a.N / (2 * tpt) + a.batch) * a.Hkv;
  const unsigned grid = (unsigned)(units < num_sms ? units : num_sms);
  return launch_dependent(kernel, dim3(grid), dim3(kThreads), Smem<D>::kBytes, stream, a, q, k, v);
}

}  // namespace

cudaError_t launch_prompt_attn(const PromptArgs& a, int D, int num_sms, cudaStream_t stream) {
  return D == 128 ? launch_d<128>(a, num_sms, stream) : launch_d<64>(a, num_sms, stream);
}

}  // namespace sv
