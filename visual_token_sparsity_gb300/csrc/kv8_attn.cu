// Sparse decode attention over the 8-bit cache: one query per head, the selected
// visual tokens and the text.
//
//   z_t = scale s_k[page(t)] q . K8[t],  out = sum softmax(z)_t s_v[page(t)] V8[t]
//
// Bound by the cache's bytes; what it takes beside them is turning e4m3 into
// something that multiplies.  e4m3 values are halves, and a query's bf16 elements
// are halves once its largest is brought to 2^14, so both products run on
// m16n8k16 tiles with fp32 accumulation and lose nothing but the weights' bits
// behind the eleventh:
//
//   S [16 tokens x 8 heads] = K (A) Q^T (B),   O [16 dims x 8 heads] += V^T (A) P^T (B)
//
// The order of the 16 elements that a tile sums over is free as long as both
// operands have it, and so are the tile's rows, so every lane takes 16 bytes in
// a row of its token and turns them in registers: as K, bytes (4i, 4i + 1 | 4i + 2,
// 4i + 3) are a tile's two pairs; as V, the bytes of two tokens are interleaved.
// S comes out token-major and goes back in as P^T by way of movmatrix.
//
// Rows are gathered by cp.async into a ring per warp, three steps of 16 tokens
// ahead (six of half the bytes at head dim 64); the indices, pages and factors
// that lead to them run two blocks of 32 tokens before that.
//
// The weights carry the factor s_v of their page relative to the largest so far
// (and 2^6), the scores a reference that is raised only when one outgrows it by
// 2^8, so that most steps need no maximum.  A weight keeps its eleven bits down to
// 2^-20 of the reference and vanishes below 2^-30.
//
// Work is cut evenly: the blocks of 32 tokens of all (sequence, KV head) units
// form one line, cut into equal pieces, one per warp.  A unit that lies in several
// pieces leaves fp32 partials, which the last of its warps joins (few pieces) or a
// second kernel (many), always in the order of the pieces.
#include "kernels.h"
#include "kv8.cuh"

namespace sv {

namespace {

constexpr int kWarps = 4, kCtas = 3;      // per CTA, and CTAs per SM (shared memory and 168 registers)
constexpr int kSms = 152;
constexpr int kBlock = 32;               // tokens whose rows a warp looks up at a time
constexpr int kStep = 16;                // tokens of a step
constexpr float kRaise = 8.f;            // log2: a reference is raised when a score outgrows it by more
constexpr int kMinBlocks = 1;            // of a piece (a call of 201 tokens 7.1 us; at 2, 4 and 8: 8.1, 9.9, 10.0)
constexpr int kFusedPieces = 16;         // of a unit of at most two heads that its last warp joins itself

// A warp's ring: per stage K and V rows of 16 tokens, the blocks' factors beside.
template <int D>
struct Ring {
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kPool = kStep * D, kStage = 2 * kPool;
  static constexpr int kFactors = kStages * kStage;             // a stage: 16 (s_k, s_v)
  static constexpr int kThere = kFactors + kStages * kStep * 8;  // a stage: which of the 16 tokens are there
  static constexpr int kBytes = kThere + kStages * 4 + (kStages * 4 % 128 ? 128 - kStages * 4 % 128 : 0);
};

// Where 16-byte unit `u` of row `t` of a stage's K or V lies.  Lanes that read
// together (as K: two neighbouring rows, four units; as V: four rows of one
// parity, two units) meet eight different units of a 128-byte line.
template <int D>
__device__ __forceinline__ uint32_t unit_at(uint32_t t, uint32_t u) {
  const uint32_t turn = ((t >> 1) & 3) << 1;
  if (D == 128) return t * 128 + ((u ^ turn ^ ((t & 1) << 2)) << 4);
  return (t >> 1) * 128 + (((((t & 1) << 2) | u) ^ turn) << 4);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The power of two 2^e, as fp32 bits, with 2^e <= max(|x|, |y|) < 2^(e + 1), within
// 2^-126 and 2^126.
__device__ __forceinline__ uint32_t exponent_of(float x, float y) {
  return min(max(__float_as_uint(fmaxf(fabsf(x), fabsf(y))) & 0x7f800000u, 0x00800000u), 253u << 23);
}

// First block of piece c of C: floor(total * c / C), in 32 bits.
__host__ __device__ __forceinline__ uint32_t piece_begin(uint32_t total, uint32_t c, uint32_t C) {
  const uint32_t q = total / C;
  return q * c + (total - q * C) * c / C;
}
// The piece that block s lies in.
__device__ __forceinline__ int piece_of(uint32_t total, uint32_t s, uint32_t C) {
  return (int)(((unsigned long long)(s + 1) * C - 1) / total);
}

struct Seq {
  int nv, nt, kb;       // visual, text, attended visual tokens
  __device__ int blocks() const { return (kb + nt + kBlock - 1) / kBlock; }
};
__device__ __forceinline__ bool seq_of(const Kv8AttnArgs& a, int b, Seq& s) {
  return attn_lengths(a.lens, a.vis_idx != nullptr, b, a.n_vis, a.n_text, a.k_vis, false, a.status, s.nv, s.nt, s.kb);
}

// Blocks of sequences [b0, b0 + 32) up to this lane's (and its own), by a whole warp.
__device__ __forceinline__ uint32_t scan_blocks(const Kv8AttnArgs& a, int b0, int lane, uint32_t& mine) {
  Seq s;
  mine = 0;
  if (b0 + lane < a.batch) {
    seq_of(a, b0 + lane, s);
    mine = (uint32_t)s.blocks() * (uint32_t)a.Hkv;
  }
  uint32_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  return inc;
}
// With equal counts the host has laid the line out (a.per_unit blocks a unit).
__device__ __forceinline__ uint32_t line_total(const Kv8AttnArgs& a, int lane) {
  uint32_t total = 0, mine;
  for (int b0 = 0; b0 < a.batch; b0 += 32) total += __shfl_sync(0xffffffffu, scan_blocks(a, b0, lane, mine), 31);
  return total;
}

// Piece `piece` of the line: its first block, its length, and the sequence that it
// begins in with the blocks before that one.
struct Piece {
  uint32_t total, C, from, before;
  int left, b;
  __device__ __forceinline__ void cut(int piece, int pieces) {
    C = min((uint32_t)pieces, total);
    left = 0;
    if (piece >= (int)C) return;
    from = piece_begin(total, piece, C);
    left = (int)(piece_begin(total, piece + 1, C) - from);
  }
};
__device__ __forceinline__ Piece equal_piece(const Kv8AttnArgs& a, int piece) {
  Piece p;
  const uint32_t in_seq = (uint32_t)a.per_unit * (uint32_t)a.Hkv;
  p.total = in_seq * (uint32_t)a.batch;
  p.cut(piece, a.pieces);
  p.b = p.left > 0 ? (int)(p.from / in_seq) : 0;
  p.before = (uint32_t)p.b * in_seq;
  return p;
}
__device__ __forceinline__ Piece ragged_piece(const Kv8AttnArgs& a, int piece, int lane) {
  Piece p;
  uint32_t mine, inc = scan_blocks(a, 0, lane, mine);
  p.total = __shfl_sync(0xffffffffu, inc, 31);
  for (int b0 = 32; b0 < a.batch; b0 += 32) {
    uint32_t other;
    p.total += __shfl_sync(0xffffffffu, scan_blocks(a, b0, lane, other), 31);
  }
  p.cut(piece, a.pieces);
  p.before = 0;
  for (p.b = 0; p.left > 0 && p.b < a.batch; p.b += 32) {
    if (p.b > 0) inc = scan_blocks(a, p.b, lane, mine);
    const uint32_t past = __ballot_sync(0xffffffffu, p.before + inc > p.from);
    if (past) {
      const int f = __ffs(past) - 1;
      p.before += __shfl_sync(0xffffffffu, inc - mine, f);
      p.b += f;
      break;
    }
    p.before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return p;
}

// (m, l) and O of a piece's part of a unit: slot 0 of a piece continues a unit,
// slot 1 begins one that goes on.
__device__ __forceinline__ size_t part_slot(int piece, bool begins) { return (size_t)piece * 2 + (begins ? 1 : 0); }

// (M, L, O) of head h of a unit over pieces p0 + w0, + step, ... < p0 + n, by a warp:
// D / 32 dims a lane, eight pieces in flight.
template <int D>
__device__ __forceinline__ void gather_pieces(const Kv8AttnArgs& a, int p0, int n, int w0, int step, int lane, int h,
                                              float& M, float& L, float (&acc)[D / 32]) {
  constexpr int E = D / 32, kBatch = 8;
  const int G = a.H / a.Hkv;
  M = -INFINITY;
  L = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int s0 = w0; s0 < n; s0 += kBatch * step) {
    float x[kBatch][E];
    float2 ml[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = s0 + i * step;
      const size_t at = part_slot(p0 + s, s == 0) * G + h;
      ml[i] = s < n ? __ldcg(reinterpret_cast<const float2*>(a.part_ml) + at) : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 y = s < n ? __ldcg(reinterpret_cast<const float2*>(a.part_o + at * D + lane * E + e)) : make_float2(0.f, 0.f);
        x[i][e] = y.x;
        x[i][e + 1] = y.y;
      }
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, ml[i].x);
    const float old = M == -INFINITY ? 0.f : fast_exp2(M - top);
    L *= old;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= old;
    M = top;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float w = ml[i].x == -INFINITY ? 0.f : fast_exp2(ml[i].x - top);
      L = fmaf(ml[i].y, w, L);                              // (a NaN stays)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, x[i][e], acc[e]);
    }
  }
}

}  // namespace

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, kCtas)
kv8_attn_kernel(const __grid_constant__ Kv8AttnArgs a) {
  using R = Ring<D>;
  constexpr int KS = D / 16, KC = D / 64, VB = D / 8, VW = VB / 4, S = R::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  const int G = a.H / a.Hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, q4 = lane & 3;
  uint8_t* ring = smem + warp * R::kBytes;
  const uint32_t ring_at = smem_u32(ring);
  const int piece = blockIdx.x * kWarps + warp;
  const bool ragged = a.lens.any();
  // (equal counts: nothing here waits for the kernel before)
  Piece line;
  if (!ragged) line = equal_piece(a, piece);
  grid_dep_sync();
  if (ragged) {
    // sequences without a token (or with a length out of range): 0 and -inf
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
      Seq s;
      const bool ok = seq_of(a, b, s);
      if (!ok && threadIdx.x == 0) flag_status(a.status, kStatusBadLength);
      if (s.kb + s.nt > 0) continue;
      for (int i = threadIdx.x; i < a.H * (D / 8); i += kWarps * 32)
        reinterpret_cast<uint4*>(a.out)[(size_t)b * a.H * (D / 8) + i] = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse != nullptr)
        for (int i = threadIdx.x; i < a.H; i += kWarps * 32) a.lse[(size_t)b * a.H + i] = -INFINITY;
    }
    line = ragged_piece(a, piece, lane);
  }
  const uint32_t total = line.total, C = line.C;
  uint32_t before = line.before, off = line.from - before;
  int left = line.left, b = line.b;

#pragma unroll 1
  for (; left > 0; ++b, off = 0) {
  Seq sq;
  seq_of(a, b, sq);
  const int nv = sq.nv, kb = sq.kb, total_tok = sq.kb + sq.nt, per_unit = sq.blocks();
  const uint32_t in_seq = (uint32_t)per_unit * (uint32_t)a.Hkv;
#pragma unroll 1
  while (left > 0 && off < in_seq) {
  const int g = (int)(off / (uint32_t)per_unit), blk0 = (int)off - g * per_unit, blk1 = min(per_unit, blk0 + left);
  off += blk1 - blk0;
  left -= blk1 - blk0;
  const int32_t* list = a.vis_idx != nullptr ? a.vis_idx + ((size_t)b * a.Hkv + g) * a.k_vis : nullptr;
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;
  const int first = blk0 * kBlock, end = min(total_tok, blk1 * kBlock);
  constexpr int stride = kBlock;

  // ---- a block's tokens, a lane each, in three steps: position (two blocks
  // ahead), page (one ahead), row and factors
  struct Ahead {
    int pos, page;
    bool there;
  };
  auto load_pos = [&](int t0, Ahead& n) {
    const int t = t0 + lane;
    n.there = t < end;
    n.pos = t < kb ? t : nv + t - kb;
    if (n.there && t < kb && list != nullptr) n.pos = __ldg(list + t);
  };
  auto load_page = [&](int t0, Ahead& n) {
    if (n.there && t0 + lane < kb && (n.pos < 0 || n.pos >= nv)) {
      flag_status(a.status, kStatusBadIndex);
      n.there = false;
    }
    n.page = n.there ? __ldg(bt + (n.pos >> 4)) : -1;
  };
  uint32_t rid, there;
  auto load_row = [&](const Ahead& n) {
    const bool ok = n.there && n.page >= 0 && n.page < a.num_blocks;
    if (n.there && !ok) flag_status(a.status, kStatusBadBlock);
    rid = ok ? ((uint32_t)n.page * (uint32_t)a.Hkv + (uint32_t)g) * 16u + (uint32_t)(n.pos & 15) : 0u;
    there = __ballot_sync(0xffffffffu, ok);
  };
  Ahead n1, n2;
  load_pos(first, n1);
  load_pos(first + stride, n2);
  uint2 raw[NT][KS];            // the queries, on their way with the positions
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint16_t* src = static_cast<const uint16_t*>(a.q) + ((size_t)b * a.H + (size_t)g * G + 8 * t + r) * D + q4 * 16;
#pragma unroll
    for (int k = 0; k < KS; ++k)
      raw[t][k] = 8 * t + r < G ? __ldg(reinterpret_cast<const uint2*>(src + (k >> 2) * 64 + (k & 3) * 4)) : make_uint2(0u, 0u);
  }
  load_page(first, n1);
  // Requests the rows and factors of step `i` (its tokens' ids are looked up with
  // the first of a block's two steps); tokens that are not there read as zeros.
  int t_ahead = first;
  auto request = [&](int i) {
    if ((i & 1) == 0) {
      load_row(n1);
      n1 = n2;
      load_page(t_ahead + stride, n1);
      load_pos(t_ahead + 2 * stride, n2);
      t_ahead += stride;
    }
    const int h = (i & 1) * 16;
    const uint32_t stage = (uint32_t)i % S;
    constexpr int U = D / 16, RPI = 32 / U;                 // 16-byte units of a row, rows of an instruction
    const uint32_t u = lane % U, t0 = lane / U;
#pragma unroll
    for (int c = 0; c < kStep / RPI; ++c) {
      const uint32_t t = t0 + c * RPI, row = __shfl_sync(0xffffffffu, rid, h + t), n = (there >> (h + t)) & 1 ? 16u : 0u;
      const uint32_t to = ring_at + stage * R::kStage + unit_at<D>(t, u);
      cp_async16(to, a.k_pool + (size_t)row * D + u * 16, n);
      cp_async16(to + R::kPool, a.v_pool + (size_t)row * D + u * 16, n);
    }
    const uint32_t mine = __shfl_sync(0xffffffffu, rid, h + (lane & 15));
    if (lane < 16)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(ring_at + R::kFactors + (stage * kStep + lane) * 8),
                   "l"(a.scales + (size_t)(mine >> 4) * 2), "r"((there >> (h + lane)) & 1 ? 8u : 0u)
                   : "memory");
    if (lane == 0) reinterpret_cast<uint32_t*>(ring + R::kThere)[stage] = there >> h;
    cp_async_commit();
  };

#pragma unroll
  for (int i = 0; i < S - 1; ++i) request(i);

  // ---- the queries: each head's elements over 2^e, so that the largest lies in
  // [2^14, 2^15); those that are not finite stay what they are
  uint32_t qf[NT][KS][2];
  float qs[NT][2];              // of heads 2 q4 and 2 q4 + 1: scale log2(e) 2^e
  {
    float mine[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint2* x = raw[t];
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < KS; ++k) top = kv8::max_finite2(kv8::max_finite2(top, x[k].x), x[k].y);
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^(14 - e) in two factors, as its exponent may be out of range
      const int e = (int)((top << 16) >> 23) - 127 - 14;              // (a head without a normal element: 2^-127 on)
      const float f0 = __uint_as_float((uint32_t)(127 - e / 2) << 23), f1 = __uint_as_float((uint32_t)(127 - (e - e / 2)) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[t][k][0] = half2_of(bf16_lo(x[k].x) * f0 * f1, bf16_hi(x[k].x) * f0 * f1);
        qf[t][k][1] = half2_of(bf16_lo(x[k].y) * f0 * f1, bf16_hi(x[k].y) * f0 * f1);
      }
      mine[t] = (float)e;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = (int)__shfl_sync(0xffffffffu, mine[t], (2 * q4 + i) * 4);
        qs[t][i] = a.scale_log2 * __uint_as_float((uint32_t)(127 + e / 2) << 23) * __uint_as_float((uint32_t)(127 + e - e / 2) << 23);
      }
  }

  float m[NT][2], l[NT][2], o[NT][KS][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[t][i] = -INFINITY;
      l[t][i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][j][e] = 0.f;
  }
  uint32_t vtop = 0x00800000u;      // the largest factor of V so far, rounded down to a power of two (bits)

  const int steps = (end - first + kStep - 1) / kStep;
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
      cp_async_wait<S - 2>();
      __syncwarp();
      request(i + S - 1);
      const uint32_t stage = (uint32_t)i % S;
      const uint8_t* at = ring + stage * R::kStage;
      const float2* fac = reinterpret_cast<const float2*>(ring + R::kFactors + stage * kStep * 8);
      const float2 f0 = fac[r], f1 = fac[r + 8];
      const float sk0 = f0.x, sv0 = f0.y, sk1 = f1.x, sv1 = f1.y;
      const uint32_t seen = reinterpret_cast<const uint32_t*>(ring + R::kThere)[stage];
      const bool ok0 = (seen >> r) & 1, ok1 = (seen >> (8 + r)) & 1;
      uint4 xk[2][KC];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int c = 0; c < KC; ++c) xk[n][c] = *reinterpret_cast<const uint4*>(at + unit_at<D>(r + 8 * n, 4 * c + q4));
      float z[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) z[t][e] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&xk[0][k >> 2]);
        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&xk[1][k >> 2]);
        const uint32_t y0 = w0[k & 3], y1 = w1[k & 3];
        const uint32_t a0 = kv8::e4m3x2_to_half2((uint16_t)y0), a1 = kv8::e4m3x2_to_half2((uint16_t)y1);
        const uint32_t a2 = kv8::e4m3x2_to_half2((uint16_t)(y0 >> 16)), a3 = kv8::e4m3x2_to_half2((uint16_t)(y1 >> 16));
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_f16(z[t], a0, a1, a2, a3, qf[t][k][0], qf[t][k][1]);
      }
      bool raise = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[t][e] = (e < 2 ? ok0 : ok1) ? z[t][e] * (e < 2 ? sk0 : sk1) * qs[t][e & 1] : -INFINITY;
          raise = raise || z[t][e] > m[t][e & 1] + kRaise || (m[t][e & 1] == -INFINITY && z[t][e] > -INFINITY);
        }
      raise = raise || exponent_of(sv0, sv1) > vtop;
      if (__any_sync(0xffffffffu, raise)) {
        // the factors' largest, and each head's
        const uint32_t top = __reduce_max_sync(0xffffffffu, max(vtop, exponent_of(sv0, sv1)));
        const float down = __uint_as_float(vtop) / __uint_as_float(top);
        vtop = top;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mx = fmaxf(m[t][i], fmaxf(z[t][i], z[t][i + 2]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float alpha = m[t][i] == -INFINITY ? 0.f : fast_exp2(m[t][i] - mx);
            m[t][i] = mx;
            l[t][i] *= alpha;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              o[t][j][i] *= alpha * down;
              o[t][j][i + 2] *= alpha * down;
            }
          }
      }
      // 2^6 s_v over the largest factor
      const float unit_v = __uint_as_float((254u - (vtop >> 23)) << 23);
      const float w0 = sv0 * unit_v * 64.f, w1 = sv1 * unit_v * 64.f;
      uint32_t p[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = m[t][e & 1];
          y[e] = fast_exp2(z[t][e] - (ref == -INFINITY ? 0.f : ref));
          l[t][e & 1] += y[e];
        }
        p[t][0] = transposed(half2_of(y[0] * w0, y[1] * w0));
        p[t][1] = transposed(half2_of(y[2] * w1, y[3] * w1));
      }
      uint32_t xv[4][VW];                         // tokens 2 q4, + 1, + 8, + 9
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const uint32_t t = 2 * q4 + (n & 1) + (n >> 1) * 8;
        if constexpr (D == 128) {
          const uint4 y = *reinterpret_cast<const uint4*>(at + R::kPool + unit_at<D>(t, r));
          xv[n][0] = y.x; xv[n][1] = y.y; xv[n][2] = y.z; xv[n][3] = y.w;
        } else {
          const uint2 y = *reinterpret_cast<const uint2*>(at + R::kPool + unit_at<D>(t, r >> 1) + (r & 1) * 8);
          xv[n][0] = y.x; xv[n][1] = y.y;
        }
      }
#pragma unroll
      for (int w = 0; w < VW; ++w)
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const uint32_t sel = i2 ? 0x7362u : 0x5140u;      // (token, next token) x two bytes
          const uint32_t lo = __byte_perm(xv[0][w], xv[1][w], sel), hi = __byte_perm(xv[2][w], xv[3][w], sel);
          const uint32_t a0 = kv8::e4m3x2_to_half2((uint16_t)lo), a1 = kv8::e4m3x2_to_half2((uint16_t)(lo >> 16));
          const uint32_t a2 = kv8::e4m3x2_to_half2((uint16_t)hi), a3 = kv8::e4m3x2_to_half2((uint16_t)(hi >> 16));
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_f16(o[t][2 * w + i2], a0, a1, a2, a3, p[t][0], p[t][1]);
        }
  }
  cp_async_wait<0>();
  __syncwarp();                                             // (the ring is free for the next unit)

  // ---- this part of the unit
  const float back = __uint_as_float(vtop) * (1.f / 64.f);
  const bool whole = blk0 == 0 && blk1 == per_unit;
  const size_t slot = part_slot(piece, blk0 == 0);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = 8 * t + 2 * q4 + i;
      float s = l[t][i];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      if (h >= G) continue;
      if (whole) {
        const float inv = s > 0.f ? 1.f / s : (s == 0.f ? 0.f : s);
        const size_t row = (size_t)b * a.H + (size_t)g * G + h;
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * D + r * VB);
#pragma unroll
        for (int j = 0; j < KS; ++j)
          dst[j] = f32_to_bf16_bits(o[t][j][i] * back * inv) | f32_to_bf16_bits(o[t][j][i + 2] * back * inv) << 16;
        if (r == 0 && a.lse != nullptr)
          a.lse[row] = s == 0.f ? -INFINITY : (m[t][i] + log2f(s)) * 0.6931471805599453f;
      } else {
        float* dst = a.part_o + (slot * G + h) * D + r * VB;
#pragma unroll
        for (int j = 0; j < KS; ++j)
          *reinterpret_cast<float2*>(dst + 2 * j) = make_float2(o[t][j][i] * back, o[t][j][i + 2] * back);
        if (r == 0) reinterpret_cast<float2*>(a.part_ml)[slot * G + h] = make_float2(m[t][i], s);
      }
    }
  if (whole || a.split_done == nullptr) continue;

  // ---- the last warp of a unit joins its pieces
  const uint32_t start = before + (uint32_t)g * (uint32_t)per_unit;
  const int p0 = piece_of(total, start, C), n = piece_of(total, start + per_unit - 1, C) - p0 + 1;
  const int unit = b * a.Hkv + g;
  __threadfence();
  __syncwarp();
  int last = 0;
  if (lane == 0) last = atomicAdd(a.split_done + unit, 1) == n - 1;
  if (!__shfl_sync(0xffffffffu, last, 0)) continue;
  __threadfence();
  if (lane == 0) a.split_done[unit] = 0;                  // ready for the next call
#pragma unroll 1
  for (int h = 0; h < G; ++h) {
    constexpr int E = D / 32;
    float M, L, acc[E];
    gather_pieces<D>(a, p0, n, 0, 1, lane, h, M, L, acc);
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    const size_t row = (size_t)b * a.H + (size_t)g * G + h;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = f32_to_bf16_bits(acc[e] * inv) | f32_to_bf16_bits(acc[e + 1] * inv) << 16;
    if (lane == 0 && a.lse != nullptr) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
  }
  before += in_seq;
  }
}

// Joins the units that were cut: a CTA per (unit, head), whose warps take every
// eighth piece each.
constexpr int kMergeWarps = 8;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
kv8_merge_kernel(const __grid_constant__ Kv8AttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float part[kMergeWarps][D];
  __shared__ float2 part_ml[kMergeWarps];
  grid_dep_sync();
  const int G = a.H / a.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / a.H, h = blockIdx.x - b * a.H, g = h / G;
  Seq s;
  seq_of(a, b, s);
  const int per_unit = s.blocks();
  if (per_unit == 0) return;
  uint32_t before = 0, total;
  if (!a.lens.any()) {
    before = (uint32_t)b * (uint32_t)per_unit * (uint32_t)a.Hkv;
    total = (uint32_t)a.batch * (uint32_t)per_unit * (uint32_t)a.Hkv;
  } else {
    total = line_total(a, lane);
    for (int b0 = 0; b0 <= b; b0 += 32) {
      uint32_t mine;
      const uint32_t inc = scan_blocks(a, b0, lane, mine);
      before += b - b0 < 32 ? __shfl_sync(0xffffffffu, inc - mine, b - b0) : __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  const uint32_t start = before + (uint32_t)g * (uint32_t)per_unit, C = min((uint32_t)a.pieces, total);
  const int p0 = piece_of(total, start, C), n = piece_of(total, start + per_unit - 1, C) - p0 + 1;
  if (n == 1) return;
  float M, L, acc[E];
  gather_pieces<D>(a, p0, n, warp, kMergeWarps, lane, h - g * G, M, L, acc);
#pragma unroll
  for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
  if (lane == 0) part_ml[warp] = make_float2(M, L);
  __syncthreads();
  if (threadIdx.x >= D) return;
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) M = fmaxf(M, part_ml[w].x);
  L = 0.f;
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    const float f = part_ml[w].x == -INFINITY ? 0.f : fast_exp2(part_ml[w].x - M);
    L += part_ml[w].y * f;
    v += part[w][threadIdx.x] * f;
  }
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
  const size_t row = (size_t)b * a.H + h;
  static_cast<uint16_t*>(a.out)[row * D + threadIdx.x] = (uint16_t)f32_to_bf16_bits(v * inv);
  if (threadIdx.x == 0 && a.lse != nullptr) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

namespace {

// Pieces of the line: one per resident warp, of kMinBlocks blocks at least.  Where
// that is four or more to a unit, the same number to each, so that none lies across
// two units (a warp's second unit begins with the whole chain of lookups).
int pieces_of(long long units, long long blocks) {
  const long long most = (long long)kSms * kCtas * kWarps;
  long long each = blocks / kMinBlocks;
  each = each > 1 ? each : 1;
  if (units * each <= most) return (int)(units * each > 1 ? units * each : 1);
  each = units > 0 ? most / units : 0;
  return (int)(each >= 4 ? units * each : most);
}
// No fewer pieces, for any smaller call.
long long pieces_bound(long long units, long long blocks) {
  const long long most = (long long)kSms * kCtas * kWarps, c = units * (blocks / kMinBlocks > 1 ? blocks / kMinBlocks : 1);
  return c < 1 ? 1 : c < most ? c : most;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// (m, l) | O of two parts of every piece: a bound that no smaller call exceeds
size_t kv8_attn_workspace_bytes(int B, int H, int Hkv, int D, int n_tokens) {
  const int G = H / Hkv;
  const size_t parts = 2 * (size_t)pieces_bound((long long)B * Hkv, ((long long)n_tokens + kBlock - 1) / kBlock);
  return up256(parts * G * 2 * sizeof(float)) + up256(parts * G * D * sizeof(float));
}

template <int D, int NT>
static cudaError_t launch_nt(const Kv8AttnArgs& a, cudaStream_t stream) {
  auto kernel = kv8_attn_kernel<D, NT>;
  const int smem = kWarps * Ring<D>::kBytes;
  static_assert(kCtas * (kWarps * Ring<D>::kBytes + 1024) <= 228 * 1024, "shared memory");
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  e = launch_dependent(kernel, dim3((unsigned)((a.pieces + kWarps - 1) / kWarps)), dim3(kWarps * 32), (size_t)smem, stream, a);
  if (e != cudaSuccess || a.split_done != nullptr) return e;
  return launch_dependent(kv8_merge_kernel<D>, dim3((unsigned)((long long)a.batch * a.H)), dim3(kMergeWarps * 32), 0,
                          stream, a);
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs& args, int D, cudaStream_t stream) {
  Kv8AttnArgs a = args;
  const int G = a.H / a.Hkv;
  const long long units = (long long)a.batch * a.Hkv, blocks = (a.k_vis + a.n_text + kBlock - 1) / kBlock;
  a.pieces = pieces_of(units, blocks);
  a.per_unit = (int)blocks;
  a.part_ml = static_cast<float*>(a.ws);
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(a.ws) + up256((size_t)a.pieces * 2 * G * 2 * sizeof(float)));
  // (the most pieces that a unit can lie in; with counts of its own per sequence
  // the line is shorter and a unit lies in more of them)
  const long long most = a.lens.any() ? (blocks < a.pieces ? blocks : a.pieces) : a.pieces / units + 2;
  a.split_done = units <= kWorkspaceCounters && G <= 2 && most <= kFusedPieces ? a.counters : nullptr;
  if (D == 128) return G <= 8 ? launch_nt<128, 1>(a, stream) : launch_nt<128, 2>(a, stream);
  return G <= 8 ? launch_nt<64, 1>(a, stream) : launch_nt<64, 2>(a, stream);
}

}  // namespace sv
