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
// A weight of the value product carries the factor s_v of its page, and has a
// reference of its own beside the sum's:
//
//   l += 2^(z - m),   p = 2^(z + log2 s_v - u) 2^6   in fp16,   O = 2^(u - m - 6) sum p V8
//
// m and u are raised only when a term outgrows them by 2^8, so that most steps need
// no maximum.  A weight keeps its eleven bits down to 2^-20 of the largest and vanishes
// below 2^-30: a page of large values that no row looks at takes none from the others.
// (One exponential more; with the factor relative to the largest so far, and one
// reference, such a page took all of them.)
//
// Work is cut evenly: the blocks of 32 tokens of all (sequence, KV head) units
// form one line, cut into equal pieces, one per CTA, whose four warps take every
// fourth block and are joined in shared memory.  A unit that lies in several pieces
// leaves fp32 partials, which the last of its CTAs joins (few rows) or a second
// kernel (many), always in the order of the pieces.
//
// Measured, inputs out of L2: 4 query heads over 2 KV heads, 201 tokens 5.0 us; 16
// sequences of 32 heads, 1440 + 128 tokens 42.2 us, 5.0 TB/s of cache rows; 8 ragged
// sequences of 28 heads over 4, up to 12544 + 256 tokens 25.2 us, 3 of them the join's
// kernel; 3001 sequences of 320 + 32 tokens, 28 heads over 4, 196, with lengths of their
// own 279.  Before the value product's reference of its own the first three took 5.3, 42.9
// and 25.4; with a piece per warp 7.2, 41.8 and 28.0; with the rows prefetched in registers
// instead of the ring the second took 45; with the next part's lookups ahead of this one's
// join 5.6, 42.9 and 25.4 (registers spill at 16 heads).
// Steps run at 6.5 TB/s in all; what is left is the chain lengths -> index -> page -> row
// before the first one (some 7000 cycles of 38,000 in the third call) and the joins.
#include "kernels.h"
#include "kv8.cuh"

namespace sv {

namespace {

constexpr int kWarps = 4, kCtas = 3;      // per CTA, and CTAs per SM (shared memory and 168 registers)
constexpr int kMostSms = 152;            // that a call is cut for (the workspace is sized without a device)
constexpr int kBlock = 32;               // tokens whose rows a warp looks up at a time
constexpr int kStep = 16;                // tokens of a step
constexpr float kRaise = 8.f;            // log2: a reference is raised when a score outgrows it by more
constexpr int kMinBlocks = 4;            // of a piece: a block for each warp
constexpr int kFusedRows = 32;           // pieces x heads of a unit that its last CTA joins itself (joining 7
                                         // heads of 14 and more pieces so takes 32.3 us against 27.7 for
                                         // LongVILA's call; 8 to 128 are equal)

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

// A factor s as 2^e times what is left, 2^e <= |s| < 2^(e + 1) within 2^-126 and
// 2^126; what is left times 2^6.
__device__ __forceinline__ void split_factor(float s, float& e, float& rest) {
  const uint32_t x = min(max(__float_as_uint(s) & 0x7f800000u, 0x00800000u), 253u << 23);
  e = __uint_as_float(0x4b000000u | x >> 23) - 8388735.f;                   // (2^23 + the exponent) - (2^23 + 127)
  rest = s * __uint_as_float((254u << 23) - x) * 64.f;
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
// Piece `piece` of the line: its first block, its length, and the sequence that it
// begins in with the blocks before that one.
struct Piece {
  uint32_t total, C, from, before;
  int left, b;
  __device__ __forceinline__ void cut(int piece, int pieces) {
    C = min((uint32_t)pieces, total);
    left = 0;
    if (piece >= (int)C) return;
    from = kv8::piece_begin(total, piece, C);
    left = (int)(kv8::piece_begin(total, piece + 1, C) - from);
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

// (M, L, O) of dims e and e + 1 of head h of a unit over pieces p0 + w0, + step, ...
// < p0 + n, eight in flight.
template <int D>
__device__ __forceinline__ void gather_pieces(const Kv8AttnArgs& a, int p0, int n, int w0, int step, int h, int e,
                                              float& M, float& L, float2& v) {
  constexpr int kBatch = 8;
  const int G = a.H / a.Hkv;
  M = -INFINITY;
  L = 0.f;
  v = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int s0 = w0; s0 < n; s0 += kBatch * step) {
    float2 x[kBatch], ml[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = s0 + i * step;
      const size_t at = part_slot(p0 + s, s == 0) * G + h;
      ml[i] = s < n ? __ldcg(reinterpret_cast<const float2*>(a.part_ml) + at) : make_float2(-INFINITY, 0.f);
      x[i] = s < n ? __ldcg(reinterpret_cast<const float2*>(a.part_o + at * D + e)) : make_float2(0.f, 0.f);
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, ml[i].x);
    const float old = M == -INFINITY ? 0.f : fast_exp2(M - top);
    L *= old;
    v.x *= old;
    v.y *= old;
    M = top;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float w = ml[i].x == -INFINITY ? 0.f : fast_exp2(ml[i].x - top);
      L = fmaf(ml[i].y, w, L);                              // (a NaN stays)
      v.x = fmaf(w, x[i].x, v.x);
      v.y = fmaf(w, x[i].y, v.y);
    }
  }
}

// Dims e and e + 1 of an output row, and its log-sum-exp with the first.
template <int D>
__device__ __forceinline__ void write_pair(const Kv8AttnArgs& a, size_t row, int e, float M, float L, float2 v) {
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
  *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * D + e) =
      f32_to_bf16_bits(v.x * inv) | f32_to_bf16_bits(v.y * inv) << 16;
  if (e == 0 && a.lse != nullptr) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
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
  const int piece = blockIdx.x;
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
      const int first = (blk0 + warp) * kBlock, end = min(total_tok, blk1 * kBlock);
      constexpr int stride = kWarps * kBlock;

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
        const size_t head = (size_t)b * a.H + (size_t)g * G + 8 * t + r;
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + head * D + q4 * 16;
#pragma unroll
        for (int k = 0; k < KS; ++k)
          raw[t][k] = 8 * t + r < G ? __ldg(reinterpret_cast<const uint2*>(src + (k >> 2) * 64 + (k & 3) * 4))
                                    : make_uint2(0u, 0u);
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
          const uint32_t t = t0 + c * RPI, row = __shfl_sync(0xffffffffu, rid, h + t);
          const uint32_t n = (there >> (h + t)) & 1 ? 16u : 0u;
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
          const float f0 = __uint_as_float((uint32_t)(127 - e / 2) << 23);
          const float f1 = __uint_as_float((uint32_t)(127 - (e - e / 2)) << 23);
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
            qs[t][i] = a.scale_log2 * __uint_as_float((uint32_t)(127 + e / 2) << 23) *
                       __uint_as_float((uint32_t)(127 + e - e / 2) << 23);
          }
      }

      float m[NT][2], u[NT][2], l[NT][2], o[NT][KS][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          m[t][i] = u[t][i] = -INFINITY;
          l[t][i] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][j][e] = 0.f;
      }

      // (two steps a block of this warp)
      const int steps = max(0, (end - first + stride - 1) / stride * 2);
#pragma unroll 1
      for (int i = 0; i < steps; ++i) {
        cp_async_wait<S - 2>();
        __syncwarp();
        request(i + S - 1);
        const uint32_t stage = (uint32_t)i % S;
        const uint8_t* at = ring + stage * R::kStage;
        const float2* fac = reinterpret_cast<const float2*>(ring + R::kFactors + stage * kStep * 8);
        const float2 f0 = fac[r], f1 = fac[r + 8];
        const float sk0 = f0.x, sk1 = f1.x;
        float ev[2], rest[2];
        split_factor(f0.y, ev[0], rest[0]);
        split_factor(f1.y, ev[1], rest[1]);
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
            // (of a row without a token so far both references are -inf)
            raise = raise || z[t][e] > m[t][e & 1] + kRaise || z[t][e] + ev[e >> 1] > u[t][e & 1] + kRaise;
          }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float mx = fmaxf(m[t][i], fmaxf(z[t][i], z[t][i + 2]));
              float ux = fmaxf(u[t][i], fmaxf(z[t][i] + ev[0], z[t][i + 2] + ev[1]));
#pragma unroll
              for (int x = 4; x <= 16; x *= 2) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                ux = fmaxf(ux, __shfl_xor_sync(0xffffffffu, ux, x));
              }
              l[t][i] *= m[t][i] == -INFINITY ? 0.f : fast_exp2(m[t][i] - mx);
              const float down = u[t][i] == -INFINITY ? 0.f : fast_exp2(u[t][i] - ux);
              m[t][i] = mx;
              u[t][i] = ux;
#pragma unroll
              for (int j = 0; j < KS; ++j) {
                o[t][j][i] *= down;
                o[t][j][i + 2] *= down;
              }
            }
        }
        uint32_t p[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float mr = m[t][e & 1], ur = u[t][e & 1];
            l[t][e & 1] += fast_exp2(z[t][e] - (mr == -INFINITY ? 0.f : mr));
            y[e] = fast_exp2(z[t][e] + ev[e >> 1] - (ur == -INFINITY ? 0.f : ur)) * rest[e >> 1];
          }
          p[t][0] = transposed(half2_of(y[0], y[1]));
          p[t][1] = transposed(half2_of(y[2], y[3]));
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

      // ---- this part of the unit: the warps' results joined in shared memory
      const bool whole = blk0 == 0 && blk1 == per_unit;
      const size_t slot = part_slot(piece, blk0 == 0), row0 = (size_t)b * a.H + (size_t)g * G;
      float* joined = reinterpret_cast<float*>(ring);          // [G][D], then (m, l)
      static_assert(16 * (D + 2) * 4 <= R::kFactors, "a warp's rows fit its ring");
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
          // O relative to m, by two factors as 2^(u - m) may be out of range
          const float back = m[t][i] == -INFINITY ? 0.f : fast_exp2(0.5f * (u[t][i] - m[t][i])), back64 = back * (1.f / 64.f);
          float* dst = joined + h * D + r * VB;
#pragma unroll
          for (int j = 0; j < KS; ++j)
            *reinterpret_cast<float2*>(dst + 2 * j) = make_float2(o[t][j][i] * back64 * back, o[t][j][i + 2] * back64 * back);
          if (r == 0) reinterpret_cast<float2*>(joined + G * D)[h] = make_float2(m[t][i], s);
        }
      __syncthreads();
      for (int i = threadIdx.x; i < G * D / 2; i += kWarps * 32) {
        const int h = i / (D / 2), e = 2 * i - h * D;
        float M = -INFINITY, L = 0.f;
        float2 v = make_float2(0.f, 0.f), ml[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          ml[w] = reinterpret_cast<const float2*>(smem + w * R::kBytes + G * D * 4)[h];
          M = fmaxf(M, ml[w].x);
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = ml[w].x == -INFINITY ? 0.f : fast_exp2(ml[w].x - M);
          const float2 y = reinterpret_cast<const float2*>(smem + w * R::kBytes)[i];
          L = fmaf(ml[w].y, f, L);                              // (a NaN stays)
          v.x = fmaf(f, y.x, v.x);
          v.y = fmaf(f, y.y, v.y);
        }
        if (whole) {
          write_pair<D>(a, row0 + h, e, M, L, v);
        } else {
          *reinterpret_cast<float2*>(a.part_o + (slot * G + h) * D + e) = v;
          if (e == 0) reinterpret_cast<float2*>(a.part_ml)[slot * G + h] = make_float2(M, L);
        }
      }
      // (and the rings are free for the next unit)
      const bool join = !whole && a.split_done != nullptr;
      if (join) __threadfence();
      __syncthreads();
      if (!join) continue;

      // ---- the last CTA of a unit joins its pieces
      const uint32_t start = before + (uint32_t)g * (uint32_t)per_unit;
      const int p0 = kv8::piece_of(total, start, C), n = kv8::piece_of(total, start + per_unit - 1, C) - p0 + 1;
      int* done = a.split_done + b * a.Hkv + g;
      __shared__ int last;
      if (threadIdx.x == 0) {
        last = atomicAdd(done, 1) == n - 1;
        if (last) *done = 0;                                    // ready for the next call
      }
      __syncthreads();
      if (last) {
        __threadfence();
        for (int i = threadIdx.x; i < G * D / 2; i += kWarps * 32) {
          const int h = i / (D / 2), e = 2 * i - h * D;
          float M, L;
          float2 v;
          gather_pieces<D>(a, p0, n, 0, 1, h, e, M, L, v);
          write_pair<D>(a, row0 + h, e, M, L, v);
        }
      }
      __syncthreads();                                          // (`last` is free)
    }
    before += in_seq;
  }
}

// Joins the units that were cut: a CTA per head of a unit, whose warps take every
// fourth (eighth) piece each.  BY_PIECE: of the unit that begins in a piece and goes on
// (with more units than pieces most are not cut, and looking each one's place up, which
// means looking at all sequences, would cost the square of the batch: 3001 sequences of
// their own lengths, 28 heads over 4, 4615 us).
constexpr int kMergeThreads = 256;
template <int D, bool BY_PIECE>
__global__ void __launch_bounds__(kMergeThreads)
kv8_merge_kernel(const __grid_constant__ Kv8AttnArgs a) {
  constexpr int kPer = D / 2, kParts = kMergeThreads / kPer, kMergeWarps = kMergeThreads / 32;
  __shared__ float2 part[kParts][kPer], part_ml[kParts];
  const int G = a.H / a.Hkv, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / G, h = blockIdx.x - unit * G;       // (a piece, BY_PIECE)
  // The lengths are read before the wait for the attention (it writes none, and let
  // this kernel begin only when those before it had completed).
  __shared__ int3 found;                                    // the first of the unit's pieces, their number, its first head
  if constexpr (BY_PIECE) {
    // a stretch of sequences to a warp
    __shared__ uint32_t sums[kMergeWarps];
    const int warp = threadIdx.x >> 5, each = ((a.batch + 31) / 32 + kMergeWarps - 1) / kMergeWarps * 32;
    const int b0 = warp * each, b1 = min(a.batch, b0 + each);
    uint32_t mine, sum = 0, before = 0, total = 0;
    for (int b = b0; b < b1; b += 32) sum += __shfl_sync(0xffffffffu, scan_blocks(a, b, lane, mine), 31);
    if (lane == 0) sums[warp] = sum;
    if (threadIdx.x == 0) found = make_int3(0, 0, 0);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      before += w < warp ? sums[w] : 0u;
      total += sums[w];
    }
    const uint32_t C = min((uint32_t)a.pieces, total);
    if ((uint32_t)unit + 1 < C) {
      const uint32_t end = kv8::piece_begin(total, unit + 1, C);
      if (end >= before && end < before + sum)
        for (int b = b0; b < b1; b += 32) {
          const uint32_t inc = scan_blocks(a, b, lane, mine), past = __ballot_sync(0xffffffffu, before + inc > end);
          if (past == 0) {
            before += __shfl_sync(0xffffffffu, inc, 31);
            continue;
          }
          // the unit that the next piece's first block lies in
          if (lane == __ffs(past) - 1) {
            before += inc - mine;
            const uint32_t per_unit = mine / (uint32_t)a.Hkv, g = (end - before) / per_unit, start = before + g * per_unit;
            if (start < end && kv8::piece_of(total, start, C) == unit)
              found = make_int3(unit, kv8::piece_of(total, start + per_unit - 1, C) - unit + 1, (b + lane) * a.H + (int)g * G);
          }
          break;
        }
    }
  } else if (threadIdx.x < 32) {                            // (by one warp, as it looks at all sequences)
    const int b = unit / a.Hkv, g = unit - b * a.Hkv;
    Seq s;
    seq_of(a, b, s);
    const int per_unit = s.blocks();
    uint32_t before = 0, total;
    if (!a.lens.any()) {
      before = (uint32_t)b * (uint32_t)per_unit * (uint32_t)a.Hkv;
      total = (uint32_t)a.batch * (uint32_t)per_unit * (uint32_t)a.Hkv;
    } else {
      total = 0;
      for (int b0 = 0; b0 < a.batch; b0 += 32) {
        uint32_t mine;
        const uint32_t inc = scan_blocks(a, b0, lane, mine);
        if (b >= b0 && b < b0 + 32) before = total + __shfl_sync(0xffffffffu, inc - mine, b - b0);
        total += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    const uint32_t start = before + (uint32_t)g * (uint32_t)per_unit, C = min((uint32_t)a.pieces, total);
    int3 p = make_int3(0, 0, unit * G);
    if (per_unit > 0) {
      p.x = kv8::piece_of(total, start, C);
      p.y = kv8::piece_of(total, start + per_unit - 1, C) - p.x + 1;
    }
    if (lane == 0) found = p;
  }
  __syncthreads();
  const int p0 = found.x, n = found.y;
  grid_dep_sync();
  if (n <= 1) return;                                       // (no token, or not cut)
  const int w = threadIdx.x / kPer, i = threadIdx.x - w * kPer;
  float M, L;
  float2 v;
  gather_pieces<D>(a, p0, n, w, kParts, h, 2 * i, M, L, v);
  part[w][i] = v;
  if (i == 0) part_ml[w] = make_float2(M, L);
  __syncthreads();
  if (w != 0) return;
  M = -INFINITY;
#pragma unroll
  for (int p = 0; p < kParts; ++p) M = fmaxf(M, part_ml[p].x);
  L = 0.f;
  v = make_float2(0.f, 0.f);
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    const float f = part_ml[p].x == -INFINITY ? 0.f : fast_exp2(part_ml[p].x - M);
    L = fmaf(part_ml[p].y, f, L);
    v.x = fmaf(f, part[p][i].x, v.x);
    v.y = fmaf(f, part[p][i].y, v.y);
  }
  write_pair<D>(a, (size_t)found.z + h, 2 * i, M, L, v);
}

namespace {

// Pieces of the line, one per resident CTA at most and of kMinBlocks blocks at
// least.  Where that is four or more to a unit, the same number to each, so that
// none lies across two units (a warp's second unit begins with the whole chain of
// lookups).
long long pieces_bound(long long units, long long blocks, int sms) {
  const long long most = (long long)(sms < kMostSms ? sms : kMostSms) * kCtas, each = blocks / kMinBlocks, c = units * (each > 1 ? each : 1);
  return c < 1 ? 1 : c < most ? c : most;
}
int pieces_of(long long units, long long blocks, int sms) {
  const long long c = pieces_bound(units, blocks, sms), each = units > 0 ? c / units : 0;
  return (int)(each >= 4 ? units * each : c);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// (m, l) | O of two parts of every piece: a bound that no smaller call exceeds
size_t kv8_attn_workspace_bytes(int B, int H, int Hkv, int D, int n_tokens) {
  const int G = H / Hkv;
  const size_t parts = 2 * (size_t)pieces_bound((long long)B * Hkv, ((long long)n_tokens + kBlock - 1) / kBlock, kMostSms);
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
  e = launch_dependent(kernel, dim3((unsigned)a.pieces), dim3(kWarps * 32), (size_t)smem, stream, a);
  if (e != cudaSuccess || !a.cut || a.split_done != nullptr) return e;
  const long long units = (long long)a.batch * a.Hkv;
  const bool by_piece = units > a.pieces;
  return launch_dependent(by_piece ? kv8_merge_kernel<D, true> : kv8_merge_kernel<D, false>,
                          dim3((unsigned)((by_piece ? a.pieces : units) * (a.H / a.Hkv))), dim3(kMergeThreads), 0, stream, a);
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs& args, int D, int num_sms, cudaStream_t stream) {
  Kv8AttnArgs a = args;
  const int G = a.H / a.Hkv;
  const long long units = (long long)a.batch * a.Hkv, blocks = (a.k_vis + a.n_text + kBlock - 1) / kBlock;
  a.pieces = pieces_of(units, blocks, num_sms);
  a.per_unit = (int)blocks;
  a.part_ml = static_cast<float*>(a.ws);
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(a.ws) + up256((size_t)a.pieces * 2 * G * 2 * sizeof(float)));
  // (the most pieces that a unit can lie in; with counts of its own per sequence
  // the line is shorter and a unit lies in more of them)
  const long long most = a.lens.any() ? (blocks < a.pieces ? blocks : a.pieces)
                                      : a.pieces % units == 0 ? a.pieces / units : a.pieces / units + 2;
  a.cut = a.lens.any() || units % a.pieces != 0;
  a.split_done = units <= kWorkspaceCounters && most * G <= kFusedRows ? a.counters : nullptr;
  if (D == 128) return G <= 8 ? launch_nt<128, 1>(a, stream) : launch_nt<128, 2>(a, stream);
  return G <= 8 ? launch_nt<64, 1>(a, stream) : launch_nt<64, 2>(a, stream);
}

}  // namespace sv
