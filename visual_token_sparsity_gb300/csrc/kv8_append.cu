// New tokens on their way into the 8-bit paged cache: per-head norm and rotation
// of queries and keys, and the rounding of keys and values to e4m3 with one
// power of two per page and KV head.
//
//   x -> x', rotated pairs, bf16                       (as norm_rope.cu)
//   s = 2^e, e the smallest >= -126 with max |row| <= 448 * 2^e over the page's
//   new rows; a page that holds rows already keeps max(s, its old one), and
//   where it grows the old rows are rounded again
//   byte = e4m3(x / s)
//
// A power of two costs e4m3 nothing (its precision is the same at every
// magnitude but the smallest), makes x / s exact, and makes the old rows of a
// growing page exact too, but for those that fall below e4m3's 2^-6.
//
// Measured: prompts of some 15,000 tokens in all, 28 query heads over 4, d 128, normed,
// with three axes and the keys' bf16 rows 72.2 us, 4.0 TB/s.  Neither issue (65 % of the
// slots) nor memory (45 %) is full: 24.5 warps an SM, with 1.6 of a scheduler's 6.2 ready,
// wait for one another's arithmetic, and at 64 registers the normed forms spill (rotate-half
// 80 bytes stored and 148 loaded, interleaved 84 and 160, partly turned 96 and 180).  16
// single tokens of 32 heads 3.6 us, a launch; two questions of 193 tokens, 4 heads over 2
// 4.7 us, the 16 rows that a warp forms one after the other.
#include "kernels.h"
#include "kv8.cuh"
#include "norm_rope.cuh"

namespace sv {

using namespace nr;

namespace {

constexpr int kWarps = 4;
// Groups of query rows at a time, and CTAs per SM that the registers leave: of 1 to 3
// groups and 6 to 8 CTAs within 2 % of one another (a prompt of some 15,000 tokens of 36
// heads, before keys were checked, 67 to 69 us; one group 74), eight the fastest for
// single tokens.
constexpr int kAhead = 2, kCtas = 8;
constexpr int kWarpsPerSm = 64;   // warps that the queries spread over before a warp takes more rows

// Token range of sequence b: [begin, end) of the packed rows.  False where the
// two entries do not ascend or lie outside them.
__device__ __forceinline__ bool tokens_of(const Kv8AppendArgs& a, int b, int& begin, int& end) {
  if (a.seq_start == nullptr) {
    begin = b * a.per_seq;
    end = begin + a.per_seq;
    return true;
  }
  begin = __ldg(a.seq_start + b);
  end = __ldg(a.seq_start + b + 1);
  if (begin >= 0 && begin <= end && end <= a.N) return true;
  begin = end = 0;
  return false;
}

// Where sequence b's pages begin in the line of all (sequence, page) units: n
// tokens touch at most ceil(n / 16) + 1 pages, and from one sequence to the next
// floor(start / 16) + 2 b grows by at least that.
__device__ __forceinline__ long long first_unit(const Kv8AppendArgs& a, int b) {
  int s = a.seq_start == nullptr ? b * a.per_seq : __ldg(a.seq_start + b);
  s = max(0, min(s, a.N));
  return (s >> 4) + 2ll * b;
}

// The last sequence whose units begin at or before u, by the whole warp.
__device__ __forceinline__ int sequence_of(const Kv8AppendArgs& a, long long u, int lane) {
  int lo = 0, n = a.batch;
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lane * step;
    const uint32_t in = __ballot_sync(0xffffffffu, at < n && first_unit(a, lo + at) <= u);
    if (in == 0) return 0;
    const int f = 31 - __clz(in);
    lo += f * step;
    n = min(step, n - f * step);
  }
  return lo;
}

// The positions of token `tok` on its axes; false when one is outside the table.
__device__ __forceinline__ bool positions(const Kv8AppendArgs& a, int tok, int* p) {
  bool ok = true;
  if (a.rot > 0) {
#pragma unroll
    for (int x = 0; x < 3; ++x)
      if (x < a.n_axes && a.sec_end[x] > (x ? a.sec_end[x - 1] : 0)) {
        p[x] = __ldg(a.pos + (size_t)x * a.N + tok);
        ok = ok && p[x] >= 0 && p[x] < a.n_pos;
      }
  }
  return ok;
}

// The four turns between a lane's elements, two to a register pair.
struct Turns {
  uint64_t cs[2], sn[2];
  __device__ __forceinline__ void none() {
    cs[0] = cs[1] = fm::splat2(1.f);
    sn[0] = sn[1] = 0;
  }
  __device__ __forceinline__ void set(const float2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      cs[i] = fm::pack2(f[2 * i].x, f[2 * i + 1].x);
      sn[i] = fm::pack2(f[2 * i].y, f[2 * i + 1].y);
    }
  }
};
__device__ __forceinline__ void load_turns(const Kv8AppendArgs& a, const int* p, int j, float2 (&f)[4]) {
  const int half = a.rot >> 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pr = 4 * j + i;
    const int px = pr < a.sec_end[0] ? p[0] : pr < a.sec_end[1] ? p[1] : p[2];
    f[i] = __ldg(reinterpret_cast<const float2*>(a.cos_sin) + (size_t)px * half + pr);
  }
}

// This lane's part of a row.
template <int L, bool INTER>
struct Place {
  int sub, j, off0, off1;
  bool turned;
  __device__ __forceinline__ Place(int rot, int lane) {
    const int half = rot >> 1;
    sub = lane / L;
    j = lane - sub * L;
    turned = 4 * j < half;
    const bool split = !INTER && turned;
    off0 = split ? 4 * j : 8 * j;
    off1 = split ? half + 4 * j : 8 * j + 4;
  }
};

// One group of rows side by side: normalised, rotated and rounded to bf16, with
// twice the bits where fp32's last ones could decide the rounding.  The whole
// warp takes part.  KEYS: wherever they could, as a key's 8 bits follow from its
// bf16 ones and one bit less there may be half a step of e4m3.  Counted in 2^-24: the
// sum of squares is off by 9 at most, its root by half of that and 1.5, which is 6 of
// the result; the element by one more (weight times bf16 is exact) and the product by
// one, which is 2 of t = |x cos| + |y sin|, however small their difference; the sum by
// one of the result and the interval's edges by another: 8 of the result and 2 of t;
// without a norm 2 and 1.  (Queries, which stay bf16, are looked at in terms of the
// result: where a pair cancels, one may be off by its last bit.)
template <int L, bool INTER, bool NORM, bool PARTLY, bool KEYS>
__device__ __forceinline__ Lane8<INTER> turn_rows(const Lane8<INTER>& x, const uint64_t* gp, const uint64_t* gy,
                                                  const uint16_t* weight, const Turns& t, const Place<L, INTER>& at,
                                                  float eps) {
  constexpr int D = 8 * L;
  uint64_t p[2], y[2];
  x.unpack(p, y);
  const bool normed = NORM && weight != nullptr;
  if (normed) {
    uint64_t s2 = fm::mul2(p[0], p[0]);
    s2 = fm::fma2(p[1], p[1], s2);
    s2 = fm::fma2(y[0], y[0], s2);
    s2 = fm::fma2(y[1], y[1], s2);
    float s, s_hi;
    fm::unpack2(s2, s, s_hi);
    s = row_sum<L>(s + s_hi, RowLanes<L>{});
    const float mean = s * (1.f / D) + eps, r0 = rsqrtf(mean);
    const float step = fmaf(-mean * r0, r0, 1.f);
    const uint64_t inv = fm::splat2(isfinite(step) ? fmaf(0.5f * r0, step, r0) : r0);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      p[e] = fm::mul2(fm::mul2(p[e], gp[e]), inv);
      y[e] = fm::mul2(fm::mul2(y[e], gy[e]), inv);
    }
  }
  bool doubt = false;
  uint64_t tp[2], ty[2];           // t of both members
  constexpr uint64_t kAbs = 0x7fffffff7fffffffull;
  if constexpr (KEYS) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint64_t ap = p[e] & kAbs, ay = y[e] & kAbs, ac = t.cs[e] & kAbs, as = t.sn[e] & kAbs;
      tp[e] = fm::fma2(ap, ac, fm::mul2(ay, as));
      ty[e] = fm::fma2(ap, as, fm::mul2(ay, ac));
    }
  }
  if (!PARTLY || at.turned) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint64_t ns = t.sn[e] ^ 0x8000000080000000ull;
      const uint64_t re = fm::fma2(p[e], t.cs[e], fm::mul2(y[e], ns));
      y[e] = fm::fma2(p[e], t.sn[e], fm::mul2(y[e], t.cs[e]));
      p[e] = re;
    }
  }
  const bool changed = !PARTLY || at.turned || normed;
  Lane8<INTER> out = x;
  if (changed) {
    out.pack(p, y);
    if constexpr (KEYS) {
      constexpr float kUnit = 1.f / 16777216.f;
      const uint64_t of_it = fm::splat2((normed ? 8.f : 2.f) * kUnit), of_t = fm::splat2((normed ? 2.f : 1.f) * kUnit);
      auto differ = [&](uint64_t v, uint64_t terms) {
        const uint64_t off = fm::fma2(v & kAbs, of_it, fm::mul2(terms, of_t));
        return bf16x2(fm::add2(v, off)) != bf16x2(fm::add2(v, off ^ 0x8000000080000000ull));
      };
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        doubt = doubt || differ(p[e], tp[e]);
        doubt = doubt || differ(y[e], ty[e]);
      }
    } else {
      constexpr uint32_t kOff = (0x8000u + kDoubt) * 0x10001u;
      uint32_t near = 0xffffffffu;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        near = __viaddmin_u16x2(__byte_perm((uint32_t)p[e], (uint32_t)(p[e] >> 32), 0x5410), kOff, near);
        near = __viaddmin_u16x2(__byte_perm((uint32_t)y[e], (uint32_t)(y[e] >> 32), 0x5410), kOff, near);
      }
      doubt = min(near & 0xffffu, near >> 16) <= 2 * kDoubt;
    }
  }
  if (__any_sync(0xffffffffu, doubt)) {
    const uint4 u = exact_row<L, INTER>(x.u, out.u, normed ? weight : nullptr, at.off0, at.off1, eps, t.cs[0], t.cs[1],
                                        t.sn[0], t.sn[1]);
    if (changed) out.u = u;
  }
  return out;
}

// The rows of one page and head that the call brings: slots [r0, r0 + n) of page
// `page` (negative: no cache to write), tokens t0, t0 + 1, ...
struct Unit {
  int b, page, r0, t0, n;
};

__device__ __forceinline__ bool unit_of(const Kv8AppendArgs& a, long long u, int lane, bool report, Unit& x) {
  x.b = sequence_of(a, u, lane);
  int begin, end;
  if (!tokens_of(a, x.b, begin, end)) return false;     // (reported by the first block)
  const long long nth = u - first_unit(a, x.b);
  if (nth < 0) return false;
  int nv, nt, kb;
  SeqLens l = a.lens;
  l.k = nullptr;
  bool ok = seq_lengths(l, x.b, a.n_vis, a.n_text, 0, nv, nt, kb);
  const int base = nv + nt;
  ok = ok && (long long)base + (end - begin) <= (long long)a.max_blocks * 16;
  const long long col = (base >> 4) + nth;               // of the block table
  const long long p0 = max((long long)base, col * 16), p1 = min((long long)base + (end - begin), (col + 1) * 16);
  if (p0 >= p1) return false;
  x.r0 = (int)(p0 & 15);
  x.n = (int)(p1 - p0);
  x.t0 = begin + (int)(p0 - base);
  x.page = -1;
  if (!ok) return true;                                  // (reported by the first block; keys still go out)
  x.page = __ldg(a.block_table + (size_t)x.b * a.max_blocks + col);
  if (x.page < 0 || x.page >= a.num_blocks) {
    if (report) flag_status(a.status, kStatusBadBlock);
    x.page = -1;
  }
  return true;
}

// The page's factor after rows of magnitude `top` joined it, and the rows that
// were there before rounded again where it grew.
template <int D>
__device__ __forceinline__ float settle_scale(const Kv8AppendArgs& a, uint8_t* rows, size_t unit, int which, int r0,
                                              uint32_t top, int lane) {
  const float need = kv8::scale_of(top);
  float* at = a.scales + unit * 2 + which;
  if (r0 == 0) {
    if (lane == 0) *at = need;
    return need;
  }
  float old = *at;
  if (!(old >= kv8::kLeastScale)) old = kv8::kLeastScale;
  const float s = fmaxf(old, need);
  __syncwarp();                                          // (every lane has read it)
  if (lane == 0) *at = s;
  if (s != old) {
    const float ratio = old / s;
    for (int c = lane; c < r0 * (D / 16); c += 32) {
      uint4 v = reinterpret_cast<const uint4*>(rows)[c];
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 lo = kv8::e4m3x2_to_float2((uint16_t)w[e]), hi = kv8::e4m3x2_to_float2((uint16_t)(w[e] >> 16));
        w[e] = kv8::f32x4_to_e4m3x4(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
      }
      reinterpret_cast<uint4*>(rows)[c] = v;
    }
  }
  return s;
}

// 16 bf16 values to e4m3.
__device__ __forceinline__ uint4 round16(uint4 lo, uint4 hi, float inv) {
  const uint32_t* a = reinterpret_cast<const uint32_t*>(&lo);
  const uint32_t* b = reinterpret_cast<const uint32_t*>(&hi);
  auto four = [&](uint32_t x, uint32_t y) {
    return kv8::f32x4_to_e4m3x4(bf16_lo(x) * inv, bf16_hi(x) * inv, bf16_lo(y) * inv, bf16_hi(y) * inv);
  };
  return make_uint4(four(a[0], a[1]), four(a[2], a[3]), four(b[0], b[1]), four(b[2], b[3]));
}

__device__ __forceinline__ uint32_t warp_top(uint32_t top) {
  return __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
}

}  // namespace

// Warps [0, kv_warps): one for the keys and one for the values of every (page, KV
// head); behind them query rows, `per_warp` of one token each (a page's keys are the
// longest work, which must not be the last).
template <int L, bool INTER, bool NORM, bool PARTLY>
__global__ void __launch_bounds__(kWarps * 32, kCtas)
kv8_append_kernel(const __grid_constant__ Kv8AppendArgs a, int per_warp, uint32_t warps_per_token, uint32_t q_warps,
                  uint32_t kv_warps) {
  constexpr int D = 8 * L, RPG = 32 / L;
  __shared__ __align__(16) uint16_t rows[kWarps][16 * D];
  grid_dep_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t w = blockIdx.x * kWarps + warp;
  if (blockIdx.x == 0) {
    // sequences that are skipped, reported once
    for (int b = threadIdx.x; b < a.batch; b += kWarps * 32) {
      int begin, end, nv, nt, kb;
      SeqLens l = a.lens;
      l.k = nullptr;
      if (!tokens_of(a, b, begin, end) || !seq_lengths(l, b, a.n_vis, a.n_text, 0, nv, nt, kb) ||
          (long long)nv + nt + (end - begin) > (long long)a.max_blocks * 16)
        flag_status(a.status, kStatusBadLength);
    }
  }
  const Place<L, INTER> at(a.rot, lane);
  Turns t;
  t.none();

  if (w >= kv_warps) {
    const uint32_t item = w - kv_warps;
    if (item >= q_warps) return;
    const int tok = (int)(item / warps_per_token);
    const int r0 = (int)(item - (uint32_t)tok * warps_per_token) * per_warp, r1 = min(r0 + per_warp, a.H);
    if (a.seq_start != nullptr && (tok < __ldg(a.seq_start) || tok >= __ldg(a.seq_start + a.batch))) return;
    const uint16_t* src = a.q + (size_t)tok * a.q_stride;
    uint16_t* dst = a.q_out + (size_t)tok * a.H * D;
    // kAhead groups of rows at a time, the next ones on their way
    Lane8<INTER> x[kAhead], next[kAhead];
    auto load = [&](Lane8<INTER>* to, int r) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int row = r + i * RPG + at.sub;
        to[i].u = make_uint4(0u, 0u, 0u, 0u);
        if (row < r1) to[i].load(src + (size_t)row * D, at.off0, at.off1);
      }
    };
    load(x, r0);
    int p[3] = {0, 0, 0};
    if (!positions(a, tok, p)) {
      if (r0 == 0 && lane == 0) flag_status(a.status, kStatusBadPosition);
      return;
    }
    if (at.turned) {
      float2 f[4];
      load_turns(a, p, at.j, f);
      t.set(f);
    }
    uint64_t gp[2], gy[2];
    if (NORM && a.q_weight != nullptr) {
      Lane8<INTER> g;
      g.load(a.q_weight, at.off0, at.off1);
      g.unpack(gp, gy);
    }
#pragma unroll 1
    for (int r = r0; r < r1; r += kAhead * RPG) {
      load(next, r + kAhead * RPG);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int row = r + i * RPG + at.sub;
        x[i] = turn_rows<L, INTER, NORM, PARTLY, false>(x[i], gp, gy, NORM ? a.q_weight : nullptr, t, at, a.eps);
        if (row < r1) x[i].store(dst + (size_t)row * D, at.off0, at.off1);
        x[i] = next[i];
      }
    }
    return;
  }
  const int which = (int)(w & 1u), g = (int)((w >> 1) % (uint32_t)a.Hkv);
  Unit x;
  if (!unit_of(a, (w >> 1) / (uint32_t)a.Hkv, lane, lane == 0 && g == 0 && which == 0, x)) return;
  uint16_t* sm = rows[warp];
  uint32_t top = 0;
  // the tokens' positions, a lane each; which of them are written
  int p[3] = {0, 0, 0};
  const bool fine = lane < x.n && positions(a, x.t0 + lane, p);
  const uint32_t there = __ballot_sync(0xffffffffu, fine);
  if (lane < x.n && !fine && g == 0 && which == 0) flag_status(a.status, kStatusBadPosition);

  if (which == 0) {
    uint64_t gp[2], gy[2];
    if (NORM && a.k_weight != nullptr) {
      Lane8<INTER> gw;
      gw.load(a.k_weight, at.off0, at.off1);
      gw.unpack(gp, gy);
    }
    // one group of rows with its turns, the next one on its way
    Lane8<INTER> v, next;
    float2 f[4], next_f[4];
    auto load = [&](int i0, Lane8<INTER>& to, float2 (&turns)[4]) {
      const int i = i0 + at.sub;
      int q[3];
#pragma unroll
      for (int e = 0; e < 3; ++e) q[e] = __shfl_sync(0xffffffffu, p[e], i & 31);
      to.u = make_uint4(0u, 0u, 0u, 0u);
      if (i < 16 && (there >> i) & 1) {
        to.load(a.k + (size_t)(x.t0 + i) * a.k_stride + (size_t)g * D, at.off0, at.off1);
        if (at.turned) load_turns(a, q, at.j, turns);
      }
    };
    load(0, v, f);
#pragma unroll 1
    for (int i0 = 0; i0 < x.n; i0 += RPG) {
      const int i = i0 + at.sub;
      const bool ok = (there >> i) & 1;
      load(i0 + RPG, next, next_f);
      t.none();
      if (ok && at.turned) t.set(f);
      v = turn_rows<L, INTER, NORM, PARTLY, true>(v, gp, gy, NORM ? a.k_weight : nullptr, t, at, a.eps);
      if (ok) {
        v.store(sm + i * D, at.off0, at.off1);
        if (a.k_out != nullptr) v.store(a.k_out + ((size_t)(x.t0 + i) * a.Hkv + g) * D, at.off0, at.off1);
        top = kv8::max_finite2(kv8::max_finite2(kv8::max_finite2(kv8::max_finite2(top, v.u.x), v.u.y), v.u.z), v.u.w);
      }
      v = next;
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = next_f[e];
    }
  } else {
    // 16 rows of L pieces of 16 bytes, all on their way at once
    uint4 v[L / 2];
#pragma unroll
    for (int c = 0; c < L / 2; ++c) {
      const int i = (c * 32 + lane) / L, j = (c * 32 + lane) % L;
      v[c] = make_uint4(0u, 0u, 0u, 0u);
      if ((there >> i) & 1)
        v[c] = *reinterpret_cast<const uint4*>(a.v + (size_t)(x.t0 + i) * a.v_stride + (size_t)g * D + 8 * j);
    }
#pragma unroll
    for (int c = 0; c < L / 2; ++c) {
      *reinterpret_cast<uint4*>(sm + (c * 32 + lane) * 8) = v[c];
      top = kv8::max_finite2(kv8::max_finite2(kv8::max_finite2(kv8::max_finite2(top, v[c].x), v[c].y), v[c].z), v[c].w);
    }
  }
  if (x.page < 0 || there == 0) return;
  top = warp_top(top);
  __syncwarp();
  const size_t unit = (size_t)x.page * a.Hkv + g;
  uint8_t* pool = (which ? a.v_pool : a.k_pool) + unit * 16 * D;
  const float inv = 1.f / settle_scale<D>(a, pool, unit, which, x.r0, top, lane);
  for (int c = lane; c < x.n * (D / 16); c += 32) {
    const int i = c / (D / 16), j = c - i * (D / 16);
    if (!((there >> i) & 1)) continue;
    const uint4* src = reinterpret_cast<const uint4*>(sm + i * D + 16 * j);
    *reinterpret_cast<uint4*>(pool + (size_t)(x.r0 + i) * D + 16 * j) = round16(src[0], src[1], inv);
  }
}

template <int L, bool INTER>
static auto pick(bool norm, int rot) {
  if (rot < 8 * L)
    return norm ? kv8_append_kernel<L, INTER, true, true> : kv8_append_kernel<L, INTER, false, true>;
  return norm ? kv8_append_kernel<L, INTER, true, false> : kv8_append_kernel<L, INTER, false, false>;
}

template <int L>
static cudaError_t launch_l(const Kv8AppendArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int RPG = 32 / L;
  const int all = (a.H + RPG - 1) / RPG;
  long long groups = (long long)a.N * all / ((long long)num_sms * kWarpsPerSm);
  groups = groups < 1 ? 1 : groups > all ? all : groups;
  const long long per_token = (all + groups - 1) / groups;
  const long long units = a.N / 16 + 2ll * a.batch;
  const long long q_warps = a.N * per_token, kv_warps = units * a.Hkv * 2;
  const long long blocks = (q_warps + kv_warps + kWarps - 1) / kWarps;
  if (blocks * kWarps > 0xffffffffLL || blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const bool norm = a.q_weight != nullptr || a.k_weight != nullptr;
  auto kernel = a.interleaved ? pick<L, true>(norm, a.rot) : pick<L, false>(norm, a.rot);
  return launch_dependent(kernel, dim3((unsigned)blocks), dim3(kWarps * 32), 0, stream, a, (int)groups * RPG,
                          (uint32_t)per_token, (uint32_t)q_warps, (uint32_t)kv_warps);
}

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, int d, int num_sms, cudaStream_t stream) {
  return d == 128 ? launch_l<16>(a, num_sms, stream) : launch_l<8>(a, num_sms, stream);
}

}  // namespace sv
