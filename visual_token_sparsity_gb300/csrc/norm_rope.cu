// Per-head RMS norm and position rotation of queries and keys in one pass,
// into the salience operands (head-major) or straight into the paged cache.
//
//   x' = x * rsqrt(mean(x^2) + eps) * w          (each head of each token)
//   (a, c) -> (a cos - c sin, a sin + c cos)     (each of its rot / 2 pairs)
//
// Pair p turns by cos_sin[pos[axis(p)]][p]: one position per token, or up to
// three (time, row, column) that own consecutive sections of the pairs.
// Everything is fp32 between the bf16 load and the one rounding at the end.
// Rows on their way into the cache are rounded more closely: a query element
// that falls on the other side of a bf16 rounding boundary moves its row's
// log-sum-exp by some 1e-4, so results next to a boundary are formed again with
// twice the bits (the step's lse is then within 2e-7 of 64 bits, relative; with
// fp32 alone up to 9e-6).  "Next to" is measured in last bits of the result: a
// pair's larger member is then rounded as the 64-bit result, a smaller one
// whose fp32 error is many of its own last bits may still fall on the other side.
//
// Bound by memory: every row is read once and written once, a dozen
// operations per element.  16384 tokens of 16 + 16 heads, d 80: 28 us, 6.0 TB/s; a
// prefill of 9808 tokens of 36 heads with a norm 40 us, 4.5 TB/s, where issue
// slots are 60 % used and half of the warps resident: chains of shuffles, root
// and turns per row (34 us without the second forming of results in doubt).  A row is d / 8 lanes of 8 elements, 32 / (d / 8)
// rows side by side in a warp; a lane's elements are the two halves of four
// pairs (rotate-half: 4 at 4j and 4 at rot/2 + 4j; interleaved or not
// rotated: 8 in a row), so no pair crosses lanes and the four (cos, sin) it
// needs are loaded once per token and reused for the warp's rows.
#include "common.cuh"
#include "fastmath.cuh"
#include "kernels.h"
#include "norm_rope.cuh"

namespace sv {

using namespace nr;

namespace {

constexpr int kWarps = 4;
// Row groups in flight per warp (and as many more on their way) and the CTAs per
// SM that the registers leave: of 1 to 4 groups and 3 to 5 CTAs of 8 warps, 5 to
// 10 of 4, these were the fastest (16384 vision tokens 28 us, 28 to 43; the
// prefill 40 us, 40 to 49).
template <bool APPEND>
struct Shape {
  static constexpr int kUnroll = APPEND ? 2 : 3, kCtas = APPEND ? 7 : 8;
};
constexpr int kWarpsPerSm = 64;  // warps that a launch spreads over before they take more rows each

}  // namespace

// A warp takes `per_warp` consecutive rows of one token, where a token's rows
// are its H queries, Hk keys and (append) Hk values.  PARTLY: rot_dim
// ends inside the row, and the elements behind it are not turned (by a sine of
// 0 an infinity would reach its partner; told apart in the one kernel, the
// encoder's 16384 tokens took 29 us, not 28).
template <int L, bool APPEND, bool INTER, bool NORM, bool PARTLY>
__global__ void __launch_bounds__(kWarps * 32, Shape<APPEND>::kCtas)
norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int per_warp, uint32_t warps_per_token) {
  constexpr int D = 8 * L;
  constexpr int RPG = 32 / L;                 // rows side by side
  constexpr int kUnroll = Shape<APPEND>::kUnroll, RPC = RPG * kUnroll;
  grid_dep_sync();
  const int lane = threadIdx.x & 31;
  const int sub = lane / L, j = lane - sub * L;
  const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t tok = w / warps_per_token;
  if (tok >= (uint32_t)a.B * a.T) return;
  const int b = (int)(tok / (uint32_t)a.T), t = (int)(tok - (uint32_t)b * a.T);
  const int r0 = (int)(w - tok * warps_per_token) * per_warp, r1 = r0 + per_warp;
  const bool first = r0 == 0 && lane == 0;    // reports for the token
  RowLanes<L> next_lane;
  if (NORM) next_lane.set(sub, j, lane);

  // this lane's elements: off0.. and off1..
  const int half = a.rot >> 1;
  const bool turned = 4 * j < half, split = !INTER && turned;
  const int off0 = split ? 4 * j : 8 * j;
  const int off1 = split ? half + 4 * j : 8 * j + 4;
  // one chunk, of which this lane has the rows i * RPG < left
  Lane8<INTER> x[kUnroll];
  auto load = [&](Lane8<INTER>* to, const uint16_t* from, int left) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      to[i].u = make_uint4(0u, 0u, 0u, 0u);
      if (i * RPG < left) to[i].load(from + i * RPG * D, off0, off1);
    }
  };
  const uint16_t* q = a.q + tok * (size_t)a.q_stride;
  const uint16_t* k = a.k + tok * (size_t)a.k_stride;
  // (the first rows are on their way before anything waits for a length or a position)
  const bool has_q = r0 < a.H;
  const int k0 = max(0, r0 - a.H), k1 = min(a.Hk, r1 - a.H);
  if (has_q) load(x, q + (size_t)(r0 + sub) * D, sub < RPG ? min(r1, a.H) - r0 - sub : 0);
  else if (k0 < k1) load(x, k + (size_t)(k0 + sub) * D, sub < RPG ? k1 - k0 - sub : 0);

  // where the token goes in the cache, and whether it is there at all
  int page = 0, slot = 0;
  if (APPEND) {
    SeqLens l = a.lens;
    l.k = nullptr;
    int nv, nt, kb;
    const bool ok = seq_lengths(l, b, a.n_vis, a.n_text, 0, nv, nt, kb);
    const int tn = a.n_new ? __ldg(a.n_new + b) : a.T;
    if (!ok || tn < 0 || tn > a.T) {
      if (first && t == 0) flag_status(a.status, kStatusBadLength);
      return;
    }
    if (t >= tn) return;
    const int pos = nv + nt + t;
    page = __ldg(a.block_table + (size_t)b * a.max_blocks + (pos >> 4));
    slot = pos & 15;
    if (page < 0 || page >= a.num_blocks) {
      if (first) flag_status(a.status, kStatusBadBlock);
      page = -1;                              // the queries are still written
    }
  }

  // the four turns between this lane's elements, two to a register pair
  uint64_t cs[2] = {fm::splat2(1.f), fm::splat2(1.f)}, sn[2] = {0, 0};
  if (half > 0) {
    int p[3] = {0, 0, 0};
    bool bad = false;
#pragma unroll
    for (int x = 0; x < 3; ++x)
      if (x < a.n_axes && a.sec_end[x] > (x ? a.sec_end[x - 1] : 0)) {
        p[x] = __ldg(a.pos + ((size_t)x * a.B + b) * a.T + t);
        bad |= p[x] < 0 || p[x] >= a.n_pos;
      }
    if (bad) {
      if (first) flag_status(a.status, kStatusBadPosition);
      return;
    }
    if (turned) {
      float2 f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int pr = 4 * j + i;
        const int px = pr < a.sec_end[0] ? p[0] : pr < a.sec_end[1] ? p[1] : p[2];
        f[i] = __ldg(reinterpret_cast<const float2*>(a.cos_sin) + (size_t)px * half + pr);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        cs[i] = fm::pack2(f[2 * i].x, f[2 * i + 1].x);
        sn[i] = fm::pack2(f[2 * i].y, f[2 * i + 1].y);
      }
    }
  }
  const uint64_t ns[2] = {sn[0] ^ 0x8000000080000000ull, sn[1] ^ 0x8000000080000000ull};

  // rows [n0, n1) of one kind: at src + row * D (the first chunk is in x
  // already), to dst + row * stride
  auto rows = [&](const uint16_t* src, int n0, int n1, const uint16_t* weight, uint16_t* dst, size_t stride) {
    uint64_t gp[2], gy[2];
    if (NORM && weight != nullptr) {
      Lane8<INTER> g;
      g.load(weight, off0, off1);
      g.unpack(gp, gy);
    }
    const int mine = n0 + sub;
    const uint16_t* from = src + (size_t)mine * D;
    uint16_t* to = dst + (size_t)mine * stride;
    const int left = sub < RPG ? n1 - mine : 0;       // of this lane's rows, RPG apart
    for (int done = 0; done < n1 - n0; done += RPC, from += RPC * D, to += RPC * stride) {
      Lane8<INTER> next[kUnroll];
      if (done + RPC < n1 - n0) load(next, from + RPC * D, left - done - RPC);
      Lane8<INTER> y8[kUnroll];               // the results
      uint32_t near[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        uint64_t p[2], y[2];
        x[i].unpack(p, y);
        if (NORM && weight != nullptr) {
          uint64_t s2 = fm::mul2(p[0], p[0]);
          s2 = fm::fma2(p[1], p[1], s2);
          s2 = fm::fma2(y[0], y[0], s2);
          s2 = fm::fma2(y[1], y[1], s2);
          float s, s_hi;
          fm::unpack2(s2, s, s_hi);
          s += s_hi;
          s = row_sum<L>(s, next_lane);
          // x * w is exact (8 bits times 8), so x' carries the error of the
          // root, which one step of Newton's method makes small, and one rounding
          const float mean = s * (1.f / D) + a.eps, r0 = rsqrtf(mean);
          const float step = fmaf(-mean * r0, r0, 1.f);
          const uint64_t inv = fm::splat2(isfinite(step) ? fmaf(0.5f * r0, step, r0) : r0);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            p[e] = fm::mul2(fm::mul2(p[e], gp[e]), inv);
            y[e] = fm::mul2(fm::mul2(y[e], gy[e]), inv);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (PARTLY && !turned) break;
          const uint64_t re = fm::fma2(p[e], cs[e], fm::mul2(y[e], ns[e]));
          y[e] = fm::fma2(p[e], sn[e], fm::mul2(y[e], cs[e]));
          p[e] = re;
        }
        if constexpr (!APPEND) {
          if (!PARTLY || turned || (NORM && weight != nullptr)) x[i].pack(p, y);
          if (done + i * RPG < left) x[i].store(to + (size_t)(i * RPG) * stride, off0, off1);
          x[i] = next[i];
        } else {
          near[i] = 0xffffffffu;
          y8[i] = x[i];
          if (!PARTLY || turned || (NORM && weight != nullptr)) {
            y8[i].pack(p, y);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              constexpr uint32_t kOff = (0x8000u + kDoubt) * 0x10001u;
              near[i] = __viaddmin_u16x2(__byte_perm((uint32_t)p[e], (uint32_t)(p[e] >> 32), 0x5410), kOff, near[i]);
              near[i] = __viaddmin_u16x2(__byte_perm((uint32_t)y[e], (uint32_t)(y[e] >> 32), 0x5410), kOff, near[i]);
            }
          }
        }
      }
      if constexpr (APPEND) {
        // What goes on to the cache is rounded as from 64 bits: where fp32's
        // last bits could decide the rounding to bf16 (a result within kDoubt of
        // them of a tie), the warp forms the row again with twice the bits.
        auto doubt = [](uint32_t n) { return min(n & 0xffffu, n >> 16) <= 2 * kDoubt; };
        bool any = false;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) any = any || doubt(near[i]);
        if (__any_sync(0xffffffffu, any)) {
          const bool keep = PARTLY && !turned && !(NORM && weight != nullptr);
#pragma unroll
          for (int i = 0; i < kUnroll; ++i)
            if (__any_sync(0xffffffffu, doubt(near[i]))) {
              const uint4 u = exact_row<L, INTER>(x[i].u, y8[i].u, NORM ? weight : nullptr, off0, off1, a.eps, cs[0], cs[1], sn[0], sn[1]);
              if (!keep) y8[i].u = u;
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          if (done + i * RPG < left) y8[i].store(to + (size_t)(i * RPG) * stride, off0, off1);
          x[i] = next[i];
        }
      }
    }
  };
  if (has_q) {
    if (APPEND) rows(q, r0, min(r1, a.H), a.q_weight, a.q_out + (size_t)tok * a.H * D, D);
    else rows(q, r0, min(r1, a.H), a.q_weight, a.q_out + ((size_t)b * a.H * a.T + t) * D, (size_t)a.T * D);
  }
  if (page < 0) return;
  if (k0 < k1) {
    if (has_q) load(x, k + (size_t)(k0 + sub) * D, sub < RPG ? k1 - k0 - sub : 0);
    if (APPEND) rows(k, k0, k1, a.k_weight, a.k_out + ((size_t)page * a.Hk * 16 + slot) * D, 16 * D);
    else rows(k, k0, k1, a.k_weight, a.k_out + ((size_t)b * a.Hk * a.T + t) * D, (size_t)a.T * D);
  }
  if (APPEND && r1 > a.H + a.Hk) {
    // values: 16 bytes a lane, L lanes a row
    const uint16_t* v = a.v + tok * (size_t)a.v_stride;
    uint16_t* to = a.v_out + ((size_t)page * a.Hk * 16 + slot) * D;
    const int n0 = max(0, r0 - a.H - a.Hk), n1 = min(a.Hk, r1 - a.H - a.Hk);
    if (sub < RPG)
      for (int g = n0 + sub; g < n1; g += RPG)
        *reinterpret_cast<uint4*>(to + (size_t)g * 16 * D + 8 * j) = *reinterpret_cast<const uint4*>(v + (size_t)g * D + 8 * j);
  }
}

template <int L, bool APPEND, bool INTER>
static auto pick(bool norm, int rot) {
  if (rot < 8 * L)
    return norm ? norm_rope_kernel<L, APPEND, INTER, true, true> : norm_rope_kernel<L, APPEND, INTER, false, true>;
  return norm ? norm_rope_kernel<L, APPEND, INTER, true, false> : norm_rope_kernel<L, APPEND, INTER, false, false>;
}

// Rows per warp: one group side by side when there are few tokens (latency), up
// to a whole token's when there are enough to fill the SMs several times over.
template <int L>
static cudaError_t launch_l(const NormRopeArgs& a, bool append, int num_sms, cudaStream_t stream) {
  constexpr int RPG = 32 / L;
  const int rows = a.H + (append ? 2 : 1) * a.Hk, all = (rows + RPG - 1) / RPG;
  const long long tokens = (long long)a.B * a.T;
  long long groups = tokens * all / ((long long)num_sms * kWarpsPerSm);
  groups = groups < 1 ? 1 : groups > all ? all : groups;
  const long long per_token = (all + groups - 1) / groups;
  const long long blocks = (tokens * per_token + kWarps - 1) / kWarps;
  if (blocks * kWarps > 0xffffffffLL || blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const bool norm = a.q_weight != nullptr || a.k_weight != nullptr;
  auto kernel = a.interleaved ? pick<L, false, true>(norm, a.rot) : pick<L, false, false>(norm, a.rot);
  if constexpr (L == 8 || L == 16) {         // head dims of the cache
    if (append) kernel = a.interleaved ? pick<L, true, true>(norm, a.rot) : pick<L, true, false>(norm, a.rot);
  } else if (append) {
    return cudaErrorInvalidValue;
  }
  return launch_dependent(kernel, dim3((unsigned)blocks), dim3(kWarps * 32), 0, stream, a,
                          (int)groups * RPG, (uint32_t)per_token);
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, int d, bool append, int num_sms, cudaStream_t stream) {
  if ((long long)a.B * a.T == 0) return cudaSuccess;
  switch (d) {
    case 64: return launch_l<8>(a, append, num_sms, stream);
    case 72: return launch_l<9>(a, append, num_sms, stream);
    case 80: return launch_l<10>(a, append, num_sms, stream);
    case 128: return launch_l<16>(a, append, num_sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace sv
