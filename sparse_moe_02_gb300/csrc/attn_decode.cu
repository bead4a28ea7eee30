// Attention of few query rows over the paged 4-bit cache (include/attn.h): single tokens and
// short drafts, n_b G <= kDecodeRows rows per request and key/value head.
//
// Mathematics.  A key row of group g is k_c = s_g code_c + b_g, so a score is
//   q . k = sum_g s_g (sum_c q_c code_c) + b_g (sum_c q_c):
// the inner sums over codes run on the tensor cores (mma.sync, f16 with fp32 sums), the scales
// and biases enter in fp32.  The codes enter the MMA as they lie in memory: a nibble masked in
// place in the low mantissa bits of an f16 is the exact subnormal code * 2^-24 (second nibble of
// a byte: code * 2^-20, undone by an exact 2^-4 in q or at the end), so eight codes cost five
// integer instructions and no conversion.  q enters as f16 after a power-of-two scaling of its
// row (exact down to 2^-38 of the row's largest entry).  Likewise the output,
//   sum_t p_t v_tc = sum_t (p_t s_tg) code_tc + sum_t p_t b_tg,
// takes its codes as the MMA's A operand (channels by tokens) and w = p_t s_tg, rounded to f16
// (11 bits; the plain fp32 form's outputs are rounded to 8), as B; the bias sum stays in fp32.
// So that w fits f16 for any bf16 scale, the running softmax reference of a row is the maximum
// of score + exponent(largest |s_tg|), which bounds w, instead of the score alone (where all scales
// are 0 or nearly so, the biases' exponent less kBiasMore); it only moves (and the accumulators are
// only rescaled) when a token exceeds it by 2^6.
//
// What bounds it.  A tile of 16 tokens (4608 bytes with 256 channels) costs about 540 warp
// instructions for 8 rows; twelve warps an SM, each with 14 KB of copies in flight, read the cache at
// 5.9 TB/s in the main loop, 86% of a copy's rate.  Around it lie the launch, the cut of the work and
// the first copies, the join of a block's twelve warps (2200 clocks, bound by shared memory) and the
// launch that joins the blocks (3 us): these are most of the time of short and middling contexts.
// Four copies a tile (codes and parameters apart) took 55 us where one takes 50 (64 requests of 4096
// tokens, three blocks of four warps an SM); one block of twelve warps, the even cut and copies
// ahead into the next context made it 42, a block per context where lengths are alike 39.
// Measured, 16 query heads over 2 of 256 channels, one token: 256 cached tokens 7.4 us, 4096 10.7 us,
// 131072 23.8 us (3.2 TB/s with everything); 48 requests of up to 16248 23.9 us, 64 of 4096 38.2 us
// (3.9 TB/s); 8 requests of 2 to 5 tokens, 32 heads over 8 of 128 channels, contexts to 8000, 25.7 us.
//
// The form with masks (MASK) goes over the tiles of the first tokens and of the window only, and
// hides tokens by a word of drafted tokens and a window's start for each column.  Measured: 48
// requests of one token through a window of 2048, contexts to 32768 18.8 us (3882 tiles in all: a
// tenth of it; the rest as above, most of it for 96 contexts' fixed costs), 8 trees of 2 to 8
// tokens (32 heads over 8 of 128 channels), contexts to 8000 34 us (164 tiles an SM of 16 columns
// at 220 clocks each, 19 us).
//
// Layout of the work.  The rows of a key/value head (G query heads x new tokens) are the MMA's N
// side in tiles of 8, its 16 tokens the M side of the scores.  A cached row is read once for 8 of
// them (128 and 64 channels: 16, two tiles to a warp); a context with more rows is read again for
// each further tile, a unit of work of its own.  One block of twelve warps per SM; each warp takes
// every twelfth tile of 16 tokens of a context through a ring of its own (one bulk copy a tile, its
// cache record) and keeps its own softmax state and outputs; the block joins its warps through
// shared memory.  Contexts are cut evenly over the blocks: with W units of work in all (a tile is
// one, a context's fixed cost kPartCost more), block i takes [i W / n, (i + 1) W / n) whatever
// requests they belong to, so ragged batches balance; a second launch joins the partial results of
// contexts that several blocks share, in block order (the same inputs give the same bits).  Short
// contexts (max_kv small) take one block each and no second launch; longer ones of like lengths take
// one each too, and the second launch finds nothing to do.
#include <cfloat>
#include <climits>

#include "attn.cuh"
#include "attn_join.cuh"

namespace moe {
namespace {

constexpr int kWarps = 12;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;  // tokens per ring stage: the MMA's M side, and a whole number per page
// One block per context, no partial results and no second launch, up to 768 tokens and 8 more for
// each context, at most 1536: the cut costs 3 us and a block's fixed costs per part, a whole context
// the time of its tiles on one SM.  Whole against cut, 2 contexts of 768 tokens 10.5 and 10.8 us, of
// 1024 12.5 and 10.9; 16 of 1024 12.6 and 12.8; 96 of 1024 12.8 and 20.0, of 1500 16.1 and 22.7, of 1
// to 1500 15.7 and 15.4; 256 of 1 to 1500 20.5 and 22.7.  128 channels: 8 contexts of 768 7.8 and 9.2,
// of 1536 11.7 and 10.3, 128 of 1024 9.9 and 12.1, of 1500 12.3 and 14.4.  64 channels, where the cut
// pays later: 4 of 768 6.4 and 8.5, of 1536 9.2 and 9.5, 64 of 1500 9.2 and 12.9.
constexpr int kWholeKv = 768, kWholeMore = 8, kWholeMost = 1536;
constexpr float kSlack = 6.f;  // growth of the reference a tile may bring before a rescale
constexpr float kLift = 9.f;   // w <= 2^(kLift + kSlack) at the reference
// Biases may be this much larger than the bound of the scales (of groups that are nearly constant): p
// times a bias then stays below 2^(kLift + kSlack + 1 + kBiasMore), and its sum far within fp32.
constexpr int kBiasMore = 64;
constexpr int kJoinWarps = 4;  // warps whose outputs the join buffer holds at once
static_assert(kWarps % kJoinWarps == 0, "whole rounds of the join");

template <int D, int NT>
struct Cfg {
  static constexpr int NG = D / kGroup;
  static constexpr int kStage = Record<D>::kBytes;
  static constexpr int kStages = D == 256 ? 3 : D == 128 ? 5 : 8;
  static constexpr int kCols = 8 * NT;
  static constexpr int kPitch = D + 4;        // floats per column of the join buffer
  static constexpr int kQPitch = 2 * D + 64;  // bytes per staged query row
  // shared memory: ring, join buffer, staged queries (two parts), work before each request
  static constexpr int kJoin = kWarps * kStages * kStage;
  static constexpr int kQuery = kJoin + kJoinWarps * kCols * kPitch * 4;
  static constexpr int kFirst = kQuery + 2 * kCols * kQPitch;
  static constexpr int kSmem = kFirst;
  // threads that own outputs in the joins, and float4s of each
  static constexpr int kOwners = kCols * D / 4 < 256 ? kCols * D / 4 : 256;
  static constexpr int kVec = kCols * D / 4 / kOwners;
  static constexpr int kLanes = kOwners / kCols;  // owners of a column
};

// c += A B; mma_f16_first: c = A B.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                              uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// c = A B with tf32 operands (16 x 8 by 8 x 8).
__device__ __forceinline__ void mma_tf32_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// (a, b) += (x, y), one packed instruction
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%0, %1};\n\t"
      "mov.b64 q, {%2, %3};\n\t"
      "add.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}

template <int NG>
struct Words {
  uint32_t w[NG];
};

template <int NG>
__device__ __forceinline__ Words<NG> lds_words(uint32_t addr) {
  Words<NG> r;
  if constexpr (NG == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "r"(addr));
  else if constexpr (NG == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.w[0]) : "r"(addr));
  return r;
}

constexpr uint32_t kNib0 = 0x000f000fu, kNib1 = 0x00f000f0u;

// Token of MMA row r (0..7) inside its 8 tokens: the pairs of the transposed weights then are
// tokens c and c + 4, whose cached words lie in different shared-memory banks (row_swz).
__device__ __forceinline__ int row_token(int r) { return (r >> 1) | ((r & 1) << 2); }

__device__ __forceinline__ int row_tiles(const FwdArgs& a, int qn, int cols) {
  return (qn * a.d.G + cols - 1) / cols;
}

// Tiles left out of a request's context, and those that are gone over.
template <bool MASK>
__device__ __forceinline__ int skip_tiles(const FwdArgs& a, const Req& r) {
  return MASK ? skipped<kTile>(a, first_start(a, r)) : 0;
}

template <bool MASK>
__device__ __forceinline__ int kv_tiles(const FwdArgs& a, const Req& r) {
  return max(1, (r.kv + kTile - 1) / kTile - skip_tiles<MASK>(a, r));
}

// Work of a context: its tiles, and kPartCost tiles' worth for what a part costs besides (queries,
// page ids, first copies, joins), so that blocks of many short contexts get fewer tiles.  With 0, 20,
// 40 and 80: 48 requests to 16248 tokens (256 channels) 79.6, 29.2, 24.9 and 27.1 us, 8 drafts of 2
// to 5 tokens (128 channels) 37.3, 30.0, 27.2 and 29.7.
constexpr int kPartCost = 40;
// Longer contexts, seen to be of like lengths once their lengths are known, take a block each too, if
// none has this much more work than a block's share: a cut would cost a part and a join more (128
// contexts of 2500 tokens 27.4 and 33.3 us, of 4096 39.0 and 43.4).
constexpr int kEachMore = 64;
constexpr int kLeastWork = 12;  // of a block: a tile a warp (4096 tokens 10.5 us; with 32 12.5 us)

// What a column sees.  Without masks: tokens below lim.  With: tokens below c, the cached ones
// before the new ones, and those whose bit t - c is set (a request has at most kDecodeRows new
// tokens here); of all these the first ones and those from lo on.
template <bool MASK, int N, int M>
struct Seen {
  int lim[N][M];
};
template <int N, int M>
struct Seen<true, N, M> {
  uint32_t bits[N][M];
  int lo[N][M];
};
static_assert(kDecodeRows <= 32, "a word of bits");

// What a lane keeps of the query rows (columns) of one context; their MMA B fragments lie in
// shared memory, [column tile][group][word][lane] registers of two MMAs, for all warps.
template <int NT, bool MASK>
struct Query {
  uint32_t sum[NT][2];  // of column lane / 4: its scaled sum over group lane % 4 as two tf32 parts
  float scale[NT][2];   // of columns 2c, 2c + 1: turns the MMA's units into log2 units
  Seen<MASK, NT, 2> seen;
  int least;  // tokens below it the columns in use see all (those of the window at least)
  // with masks:
  int c, first;  // cached tokens before the new ones; first tokens
  int low;       // tokens from it on lie in every window
};

// The same for the block.
template <int D, int NT, bool MASK>
struct QueryShared {
  uint4 frags[NT * (D / kGroup) * 2 * 32];
  float sum[8 * NT][D / kGroup];
  float scale[8 * NT];
  Seen<MASK, 8 * NT, 1> seen;
};

// Starts copying the part's query rows [column][D] into shared memory, each followed by its mask.
template <int D, int NT, bool MASK>
__device__ __forceinline__ void fetch_query(const FwdArgs& a, const Part& p, uint8_t* raw) {
  constexpr int kPieces = D / 8;
  static_assert(8 * NT * kPieces + 8 * NT <= kThreads, "one piece a thread");
  if (MASK && a.masks) {
    const int col = threadIdx.x - 8 * NT * kPieces, row = p.rt * 8 * NT + col;
    if (col >= 0 && col < 8 * NT && row < p.r.qn * a.d.G) {
      const uint32_t* src = a.masks + (int64_t)(p.r.q0 + a.d.by_G(row)) * a.mask_words;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                       smem_u32(raw + col * Cfg<D, NT>::kQPitch + 2 * D)),
                   "l"(src)
                   : "memory");
    }
  }
  const int col = threadIdx.x / kPieces, piece = threadIdx.x % kPieces;
  if (col < 8 * NT) {
    const int row = p.rt * 8 * NT + col;
    uint8_t* dst = raw + col * Cfg<D, NT>::kQPitch + 16 * piece;
    if (row < p.r.qn * a.d.G) {
      const int tok = a.d.by_G(row);
      const __nv_bfloat16* src = a.q + (int64_t)(p.r.q0 + tok) * a.q_stride +
                                 (int64_t)(p.h * a.d.G + row - tok * a.d.G) * D + 8 * piece;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
                   : "memory");
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
    }
  }
}

__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// One warp prepares group g of column tile nt.
template <int D, int NT, bool MASK>
__device__ __forceinline__ void prepare_query(const FwdArgs& a, const Part& p, const uint8_t* raw,
                                              int nt, int g, QueryShared<D, NT, MASK>& S) {
  constexpr int NG = D / kGroup;
  const int lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
  const uint8_t* src = raw + (8 * nt + n) * Cfg<D, NT>::kQPitch + 16 * c;
  uint32_t top = 0;  // largest magnitude, as the order of bf16 bit patterns
#pragma unroll
  for (int k = 0; k < 2 * NG; ++k) {
    const uint4 w = *reinterpret_cast<const uint4*>(src + 64 * k);
    const uint32_t x = max_u16x2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
    top = max_u16x2(top, max_u16x2(x, max_u16x2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
  }
  top = max_u16x2(top, __shfl_xor_sync(~0u, top, 1));
  top = max_u16x2(top, __shfl_xor_sync(~0u, top, 2));
  top = max(top & 0xffffu, top >> 16);
  // 2^-e with the row's largest entry in [2^e, 2^(e+1)), kept a normal number
  const int e = min(max((int)(top >> 7) - 127, -100), 126);
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
  const float up = __uint_as_float((uint32_t)(e + 127) << 23);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = *reinterpret_cast<const uint4*>(src + 128 * g + 64 * i);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    float v[8];
    uint32_t f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = bf16_lo(x[k]) * down;
      v[2 * k + 1] = bf16_hi(x[k]) * down;
    }
    // the row in [2^13, 2^14) at its top; odd nibbles of a byte arrive 16 times as large
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float m = (k & 1) ? 512.f : 8192.f;
      f[k] = pack_f16(v[k] * m, v[k + 4] * m);
      sum += v[k] + v[k + 4];
    }
    S.frags[((nt * NG + g) * 2 + i) * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
  }
  sum += __shfl_xor_sync(~0u, sum, 1);
  sum += __shfl_xor_sync(~0u, sum, 2);
  if (c == 0) {
    const int col = 8 * nt + n, row = p.rt * 8 * NT + col;
    S.sum[col][g] = sum * (8192.f / 16777216.f);
    if (g == 0) {
      // code * 2^-24 * q * 2^13-e  ->  log2 units
      // (at most the largest fp32: 2^126 2^11 would be inf, and negative scores would read as masked)
      S.scale[col] = fminf(fmaxf(up * (16777216.f / 8192.f) * a.d.scale_log2, kLeastUnit), FLT_MAX);
      // columns beyond the rows see everything: nothing of them is written
      const int ctx = p.r.kv - p.r.qn, tok = a.d.by_G(row);
      const bool on = row < p.r.qn * a.d.G;
      if constexpr (MASK) {
        uint32_t bits = 0xffffffffu >> (32 - p.r.qn);
        int pos = ctx + tok;
        if (on && a.masks) {
          bits &= *reinterpret_cast<const uint32_t*>(raw + col * Cfg<D, NT>::kQPitch + 2 * D);
          pos = ctx + max(__popc(bits) - 1, 0);
        } else if (on) {
          bits = 0xffffffffu >> (31 - tok);
        }
        S.seen.bits[col][0] = bits;
        S.seen.lo[col][0] = on ? window_start(a, pos) : INT_MIN;
      } else {
        S.seen.lim[col][0] = on ? min(max(ctx + tok + 1, 0), p.r.kv) : p.r.kv;
      }
    }
  }
}

template <int D, int NT, bool MASK>
__device__ __forceinline__ void load_query(const FwdArgs& a, const Part& p,
                                           const QueryShared<D, NT, MASK>& S, Query<NT, MASK>& Q) {
  constexpr int NG = D / kGroup;
  const int lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
  Q.least = INT_MAX;
  if constexpr (MASK) {
    Q.c = Q.least = p.r.kv - p.r.qn;
    Q.first = a.sinks;
    Q.low = window_start(a, p.r.kv - 1);
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    // two tf32 parts of the sum: 22 bits of it
    const float sum = c < NG ? S.sum[8 * nt + n][c % NG] : 0.f;
    Q.sum[nt][0] = __float_as_uint(sum) & 0xffffe000u;
    Q.sum[nt][1] = __float_as_uint(sum - __uint_as_float(Q.sum[nt][0])) & 0xffffe000u;
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
      Q.scale[nt][cc] = S.scale[8 * nt + 2 * c + cc];
      if constexpr (MASK) {
        Q.seen.bits[nt][cc] = S.seen.bits[8 * nt + 2 * c + cc][0];
        Q.seen.lo[nt][cc] = S.seen.lo[8 * nt + 2 * c + cc][0];
      } else {
        Q.seen.lim[nt][cc] = S.seen.lim[8 * nt + 2 * c + cc][0];
      }
    }
    if constexpr (!MASK) {
#pragma unroll
      for (int k = 0; k < 8; ++k) Q.least = min(Q.least, S.seen.lim[8 * nt + k][0]);
    }
  }
}

// Softmax state and outputs of one warp: columns 2c, 2c + 1 of each column tile.
template <int D, int NT>
struct State {
  static constexpr int NG = D / kGroup;
  float o[NT][NG][4][4];  // code part: [group][nibble pair]{(nibble 2i: col 0, 1), (2i + 1: ...)}
  float ob[NT][2][NG];    // bias part, this lane's tokens
  float m[NT][2], l[NT][2];
};

template <int D, int NT>
__device__ __forceinline__ void clear(State<D, NT>& s) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int g = 0; g < D / kGroup; ++g) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s.o[nt][g][i][e] = 0.f;
      s.ob[nt][0][g] = s.ob[nt][1][g] = 0.f;
    }
    s.m[nt][0] = s.m[nt][1] = -INFINITY;
    s.l[nt][0] = s.l[nt][1] = 0.f;
  }
}

// One tile of 16 tokens at shared address `st`; tok0 is the first token's index in its context.
template <int D, int NT, bool MASK>
__device__ __forceinline__ void tile_step(uint32_t st, uint32_t frags, int tok0, int kv,
                                          const Query<NT, MASK>& Q, State<D, NT>& s) {
  using R = Record<D>;
  constexpr int NG = D / kGroup;
  const int lane = threadIdx.x & 31, j = lane >> 2, c = lane & 3;
  const int tr = row_token(j);  // the lane's score rows are tokens tr and tr + 8
  float x[NT][4];               // scores in MMA units, then weights
  {
    Words<NG> kw[2][2];  // [word][row]
    Words<NG> kp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t at = st + tr * R::kRow + (((c + 4 * i) ^ row_swz(tr)) * NG) * 4;
      kw[i][0] = lds_words<NG>(at);
      kw[i][1] = lds_words<NG>(at + 8 * R::kRow);
    }
    // the bias part: biases of group c (their upper halves are tf32 numbers) by the sums
    const uint32_t par = st + R::kKp + tr * R::kPar;
    const uint32_t ba = lds_words<1>(par + 4 * (c % NG)).w[0] & 0xffff0000u;
    const uint32_t bb = lds_words<1>(par + 8 * R::kPar + 4 * (c % NG)).w[0] & 0xffff0000u;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      mma_tf32_first(x[nt], ba, bb, ba, bb, Q.sum[nt][0], Q.sum[nt][1]);
    kp[0] = lds_words<NG>(par);
    kp[1] = lds_words<NG>(par + 8 * R::kPar);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float acc[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Words<4> f = lds_words<4>(frags + (((nt * NG + g) * 2 + i) * 32 + lane) * 16);
          const uint32_t a0 = kw[i][0].w[g], b0 = kw[i][1].w[g];
          const uint32_t a8 = a0 >> 8, b8 = b0 >> 8;
          if (i == 0)
            mma_f16_first(acc, a0 & kNib0, b0 & kNib0, a0 & kNib1, b0 & kNib1, f.w[0], f.w[1]);
          else
            mma_f16(acc, a0 & kNib0, b0 & kNib0, a0 & kNib1, b0 & kNib1, f.w[0], f.w[1]);
          mma_f16(acc, a8 & kNib0, b8 & kNib0, a8 & kNib1, b8 & kNib1, f.w[2], f.w[3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[nt][e] = fmaf(bf16_lo(kp[e >> 1].w[g]), acc[e], x[nt][e]);
      }
  }
  Words<NG> vp[2];  // value parameters of the lane's rows
#pragma unroll
  for (int r = 0; r < 2; ++r) vp[r] = lds_words<NG>(st + R::kVp + (8 * r + tr) * R::kPar);
  // what a row may not see, and what lies behind the context (never written: anything)
  if (tok0 + kTile > Q.least || (MASK && tok0 < Q.low && tok0 + kTile > Q.first)) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = tok0 + 8 * r + tr;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          if constexpr (MASK) {
            const int d = t - Q.c;  // a drafted token's index
            const bool off = d >= 0 && !(d < 32 && (Q.seen.bits[nt][cc] >> (d & 31) & 1));
            if (off || (t >= Q.first && t < Q.seen.lo[nt][cc])) x[nt][2 * r + cc] = -INFINITY;
          } else {
            if (t >= Q.seen.lim[nt][cc]) x[nt][2 * r + cc] = -INFINITY;
          }
        }
      if (t >= kv) {
#pragma unroll
        for (int g = 0; g < NG; ++g) vp[r].w[g] = 0;
      }
    }
  }
  // 2^ev bounds a token's scales (nonnegative bf16, the lower halves), 2^(ev + kBiasMore) its biases.  The
  // reference takes each token's bound with its own score: tokens that the row does not see (-inf) or
  // hardly weighs leave it alone, whatever they hold.
  float ev[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    uint32_t big = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) big = max_u16x2(big, vp[r].w[g] & 0x7fff7fffu);
    const int most =
        max(max((int)(big & 0xffffu), (int)(big >> 16) - (kBiasMore << 7)), (126 - 90) << 7);
    // (most >> 7) - 126 as a float: 2^23 + most / 128, less 2^23 + 126
    ev[r] = __uint_as_float(0x4b000000u | (uint32_t)most >> 7) - 8388734.f;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float top[2];
#pragma unroll
    for (int cc = 0; cc < 2; ++cc)  // of the lane's tokens
      top[cc] = fmaxf(fmaf(x[nt][cc], Q.scale[nt][cc], ev[0]),
                      fmaf(x[nt][2 + cc], Q.scale[nt][cc], ev[1]));
    if (__any_sync(~0u, top[0] > s.m[nt][0] + kSlack || top[1] > s.m[nt][1] + kSlack)) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc)
          top[cc] = fmaxf(top[cc], __shfl_xor_sync(~0u, top[cc], o));
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const float m = fmaxf(s.m[nt][cc], top[cc]);
        const float f = m == -INFINITY ? 1.f : exp2_fast(s.m[nt][cc] - m);
        const float root = m == -INFINITY ? 1.f : exp2_fast(0.5f * (s.m[nt][cc] - m));
        s.m[nt][cc] = m;
        s.l[nt][cc] = s.l[nt][cc] * root * root;  // (see part_root)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          s.ob[nt][cc][g] *= f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s.o[nt][g][i][cc] *= f;
            s.o[nt][g][i][2 + cc] *= f;
          }
        }
      }
    }
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
      const float m = s.m[nt][cc] == -INFINITY ? 0.f : kLift - s.m[nt][cc];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p = exp2_fast(fmaf(x[nt][2 * r + cc], Q.scale[nt][cc], m));
        x[nt][2 * r + cc] = p;
        s.l[nt][cc] += p;
#pragma unroll
        for (int g = 0; g < NG; ++g)
          s.ob[nt][cc][g] = fmaf(p, bf16_hi(vp[r].w[g]), s.ob[nt][cc][g]);
      }
    }
  }
  uint32_t wt[NT][NG][2];
  Words<NG> v[4];  // value words of the lane's tokens c, c + 4, c + 8, c + 12, unit j
#pragma unroll
  for (int q = 0; q < 4; ++q)
    v[q] = lds_words<NG>(st + R::kV + (c + 4 * q) * R::kRow +
                         ((j ^ row_swz(c + 4 * q)) * NG) * 4);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float sc = bf16_lo(vp[r].w[g]);
        wt[nt][g][r] = transpose8x8(pack_f16(x[nt][2 * r] * sc, x[nt][2 * r + 1] * sc));
      }
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const uint32_t sel = part ? 0x7632u : 0x5410u;
      uint32_t u0 = __byte_perm(v[0].w[g], v[1].w[g], sel);
      uint32_t u1 = __byte_perm(v[2].w[g], v[3].w[g], sel);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // The tile's sum joins the running one by a rounded addition: the MMA's own additions
          // truncate, and over thousands of tiles of nonnegative codes that would pull the code
          // part down against the bias part that it nearly cancels.
          float t[4];
          mma_f16_first(t, u0 & kNib0, u0 & kNib1, u1 & kNib0, u1 & kNib1, wt[nt][g][0],
                        wt[nt][g][1]);
          float(&o)[4] = s.o[nt][g][2 * part + k];
          add2(o[0], o[1], t[0], t[1]);
          add2(o[2], o[3], t[2], t[3]);
        }
        u0 >>= 8;
        u1 >>= 8;
      }
    }
}

// The part that holds work w of the block's [w, w1).
template <bool MASK>
__device__ __forceinline__ Part locate(const FwdArgs& a, const int64_t* first, int cols, int64_t w,
                                       int64_t w1) {
  Part p;
  p.some = false;
  while (w < w1) {
    p.b = find_request(first, a.B, w);
    p.r = load_req(a, p.b);
    p.tiles = kv_tiles<MASK>(a, p.r);
    if (MASK) p.skip = skip_tiles<MASK>(a, p.r);
    const int rts = row_tiles(a, p.r.qn, cols);
    const int k = (int)divide(w - first[p.b], p.tiles + kPartCost);
    p.h = k / rts;
    p.rt = k % rts;
    p.start = first[p.b] + (int64_t)k * (p.tiles + kPartCost) + kPartCost;
    p.t0 = (int)max(w - p.start, (int64_t)0);
    p.t1 = (int)min(w1 - p.start, (int64_t)p.tiles);
    w = p.next = min(p.start + p.tiles, w1);
    if (p.t1 > 0) {  // else the context's tiles begin in the next block
      p.some = true;
      break;
    }
  }
  return p;
}

// One block per SM.  While a part is worked on, the next part's queries and, as ring stages fall
// free, its first tiles are copied, so the joins between parts leave no gap in the stream.
template <int D, int NT, bool WHOLE, bool MASK>
__global__ void __launch_bounds__(kThreads, 1) attn_decode_kernel(FwdArgs a) {
  using C = Cfg<D, NT>;
  constexpr int NG = C::NG;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kWarps * C::kStages];
  __shared__ QueryShared<D, NT, MASK> S;
  __shared__ float2 join_ml[C::kCols][kWarps], join_sum[C::kCols];  // (m, l) of each warp, of all
  __shared__ float join_f[C::kCols][kWarps];                  // the warps' weights
  __shared__ float join_b[C::kCols][NG][kWarps], join_bias[C::kCols][NG];  // bias parts
  __shared__ Part parts[2];
  __shared__ int64_t sums[kWarps];
  __shared__ Cut cut_s;
  __shared__ int longest;  // work of the longest context
  __shared__ bool each;    // a block takes one context
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int j = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * C::kStages * C::kStage;
  uint64_t* full = bars + warp * C::kStages;
  float* join = reinterpret_cast<float*>(smem + C::kJoin);
  const uint64_t policy = policy_evict_first();
  if (lane == 0)
    for (int i = 0; i < C::kStages; ++i) mbar_init(full + i, 1);
  fence_mbar_init();
  if (!WHOLE) {
    if (tid == 0) longest = 0;
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();

  int64_t* first = reinterpret_cast<int64_t*>(smem + C::kFirst);  // [B + 1]
  if (!WHOLE) {
    const Cut cut = cut_work<kThreads>(a, first, sums, kLeastWork, [&](const Req& r) {
      if (r.qn == 0) return (int64_t)0;
      const int unit = kv_tiles<MASK>(a, r) + kPartCost;
      atomicMax(&longest, unit);
      return (int64_t)(a.d.Hkv * row_tiles(a, r.qn, C::kCols)) * unit;
    });
    if (tid == 0) cut_s = cut;
  }
  if (tid == 0) {
    Part p;
    p.some = false;
    const int rts_max = row_tiles(a, a.max_q, C::kCols);
    if (!WHOLE)
      each = (int64_t)a.B * a.d.Hkv * rts_max <= gridDim.x && longest <= cut_s.share + kEachMore;
    if (WHOLE || each) {
      const int k = blockIdx.x % (a.d.Hkv * rts_max);
      p.b = blockIdx.x / (a.d.Hkv * rts_max);
      p.h = k / rts_max;
      p.rt = k % rts_max;
      if (p.b < a.B) {
        p.r = load_req(a, p.b);
        p.t0 = 0;
        p.t1 = p.tiles = kv_tiles<MASK>(a, p.r);
        if (MASK) p.skip = skip_tiles<MASK>(a, p.r);
        p.some = p.rt < row_tiles(a, p.r.qn, C::kCols);
      }
      if (WHOLE && k == 0 && req_out_of_range(a, p.b)) record_error(a.err, kDevErrState);
    } else if ((int)blockIdx.x < cut_s.blocks) {
      p = locate<MASK>(a, first, C::kCols, cut_s.bound(blockIdx.x), cut_s.bound(blockIdx.x + 1));
    }
    parts[0] = p;
  }
  __syncthreads();
  if (!WHOLE && tid == 0) a.desc[2 * blockIdx.x].x = 0;
  if (!parts[0].some) return;
  fetch_query<D, NT, MASK>(a, parts[0], smem + C::kQuery);

  // the warp's tiles of a part: t0 + warp, + kWarps, ... below the end of the context
  auto lead_of = [&](const Part& p) { return p.t0 + warp; };
  auto tiles_of = [&](const Part& p) {
    const int held = (p.r.kv + kTile - 1) / kTile - (MASK ? p.skip : 0);
    const int n = min(p.t1, held) - lead_of(p);
    return n > 0 ? (n + kWarps - 1) / kWarps : 0;
  };
  int head = 0, used = 0;  // ring stages filled and emptied so far
  auto load = [&](uint32_t rec) {
    const int stage = head % C::kStages;
    if (lane == 0) {
      mbar_arrive_expect_tx(full + stage, C::kStage);
      bulk_load(ring + stage * C::kStage, a.cache + (uint64_t)rec * C::kStage, C::kStage,
                full + stage, policy);
    }
    ++head;
  };

  // record of the warp's tile i of a part
  auto record_of = [&](const Part& p, int i) {
    return cache_record(a, p.b, p.h, tile_at<MASK, kTile>(a, lead_of(p) + i * kWarps, p.skip));
  };

  int mine = tiles_of(parts[0]);
  uint32_t record = 0, record_more = 0;  // of 32 tiles ahead, one a lane
  if (lane < mine)
    record = record_of(parts[0], lane);
  int issued = min(mine, C::kStages);  // tiles of the part
  for (int i = 0; i < issued; ++i) load(__shfl_sync(~0u, record, i));

  bool ok = true;
  for (int cur = 0;; cur ^= 1) {
    const Part& p = parts[cur];
    Part& next = parts[cur ^ 1];
    wait_copies();
    __syncthreads();
    if (warp < NT * NG)
      prepare_query<D, NT, MASK>(a, p, smem + C::kQuery + cur * C::kCols * C::kQPitch, warp / NG,
                           warp % NG, S);
    if (tid == kThreads - 1) {
      if (WHOLE || each) next.some = false;
      else next = locate<MASK>(a, first, C::kCols, p.next, cut_s.bound(blockIdx.x + 1));
    }
    __syncthreads();
    Query<NT, MASK> Q;
    load_query<D, NT>(a, p, S, Q);
    int mine_next = 0, issued_next = 0;
    uint32_t record_next = 0;
    if (next.some) {
      fetch_query<D, NT, MASK>(a, next, smem + C::kQuery + (cur ^ 1) * C::kCols * C::kQPitch);
      mine_next = tiles_of(next);
      if (lane < mine_next)
        record_next = record_of(next, lane);
    }
    State<D, NT> s;
    clear(s);
    const int kv = p.r.kv;
    int tok0 = lead_of(p) * kTile;
    for (int i = 0; i < mine; ++i, tok0 += kWarps * kTile) {
      const int tok = MASK ? tile_at<MASK, kTile>(a, lead_of(p) + i * kWarps, p.skip) * kTile : tok0;
      const int stage = used % C::kStages;
      // after a wait that ran out nothing more is copied, but what is under way still lands
      if (used < head) ok = mbar_wait(full + stage, (used / C::kStages) & 1, a.err) && ok;
      ok = __all_sync(~0u, ok);
      if (!ok && used >= head) continue;
      if (ok)
        tile_step<D, NT>(smem_u32(ring + stage * C::kStage), smem_u32(S.frags), tok, kv, Q, s);
      ++used;
      __syncwarp();
      if (!ok) continue;
      if (issued < mine) {
        if ((issued & 31) == 0) record = record_more;
        if ((issued & 31) == 16) {  // the following 32 tiles, half a batch ahead
          const int f = issued + 16 + lane;
          if (f < mine) record_more = record_of(p, f);
        }
        load(__shfl_sync(~0u, record, issued & 31));
        ++issued;
      } else if (issued_next < min(mine_next, C::kStages)) {
        load(__shfl_sync(~0u, record_next, issued_next));
        ++issued_next;
      }
    }
    while (ok && head - used < C::kStages && issued_next < mine_next) {
      load(__shfl_sync(~0u, record_next, issued_next));
      ++issued_next;
    }

    // join the warps: a common reference for each column, then kJoinWarps warps at a time
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        float l = s.l[nt][cc];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(~0u, l, o);
        if (j == 0) join_ml[8 * nt + 2 * c + cc][warp] = make_float2(s.m[nt][cc], l);
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // bias parts, 2 NG values over 8 lanes: each exchange halves what a lane still sums
      float v[2 * NG];
#pragma unroll
      for (int i = 0; i < 2 * NG; ++i) v[i] = s.ob[nt][i / NG][i % NG];
      int at = 0;
#pragma unroll
      for (int o = 4, n = 2 * NG; o < 32; o <<= 1) {
        if (n > 1) {
          const bool up = lane & o;
#pragma unroll
          for (int i = 0; i < n / 2; ++i) {
            const float give = up ? v[i] : v[i + n / 2];
            const float keep = up ? v[i + n / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(~0u, give, o);
          }
          n >>= 1;
          at = at * 2 + up;
        } else {
          v[0] += __shfl_xor_sync(~0u, v[0], o);
        }
      }
      // lanes that share a value write the same one
      join_b[8 * nt + 2 * c + at / NG][at % NG][warp] = v[0];
    }
    __syncthreads();
    if (tid < C::kCols * NG) {
      const int col = tid / NG, g = tid % NG;
      float m = -INFINITY, l = 0.f, bias = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) m = fmaxf(m, join_ml[col][k].x);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 x = join_ml[col][k];
        const float root = part_root(x.x, x.y, m), f = root * root;
        l = fmaf(x.y * root, root, l);
        bias = fmaf(join_b[col][g][k], f, bias);
        if (g == 0) join_f[col][k] = f;
      }
      join_bias[col][g] = bias;
      if (g == 0) join_sum[col] = make_float2(m, l);
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const float f = join_f[8 * nt + 2 * c + cc][warp];
        const float f24 = f * 16777216.f, f20 = f * 1048576.f;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s.o[nt][g][i][cc] *= f24;
            s.o[nt][g][i][2 + cc] *= f20;
          }
      }
    const int own_col = tid / C::kLanes, own_ln = tid % C::kLanes;
    float4 own[C::kVec];
#pragma unroll
    for (int k = 0; k < C::kVec; ++k) {
      const float x = tid < C::kOwners ? join_bias[own_col][(own_ln + k * C::kLanes) / 16] : 0.f;
      own[k] = make_float4(x, x, x, x);
    }
#pragma unroll 1
    for (int round = 0; round < kWarps / kJoinWarps; ++round) {
      if (warp / kJoinWarps == round) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            float* dst = join + ((warp % kJoinWarps) * C::kCols + 8 * nt + 2 * c + cc) * C::kPitch +
                         4 * j;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float(&o0)[4] = s.o[nt][g][2 * k];
                const float(&o1)[4] = s.o[nt][g][2 * k + 1];
                *reinterpret_cast<float4*>(dst + 64 * g + 32 * k) =
                    make_float4(o0[cc], o0[2 + cc], o1[cc], o1[2 + cc]);
              }
          }
      }
      __syncthreads();
      if (tid < C::kOwners) {
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) {
          const float4* src = reinterpret_cast<const float4*>(
              join + (k * C::kCols + own_col) * C::kPitch);
#pragma unroll
          for (int v = 0; v < C::kVec; ++v) {
            const float4 x = src[own_ln + v * C::kLanes];
            own[v].x += x.x;
            own[v].y += x.y;
            own[v].z += x.z;
            own[v].w += x.w;
          }
        }
      }
      __syncthreads();
    }
    const bool whole = p.t1 - p.t0 == p.tiles;
    if (tid < C::kOwners) {
      const float2 ml = join_sum[own_col];
      if (whole) {
#pragma unroll
        for (int v = 0; v < C::kVec; ++v)
          store_out4(a, p, p.rt * C::kCols + own_col, D, own_ln + v * C::kLanes, own[v],
                     row_sum(ml.x, ml.y));
      } else {
        const int64_t at = (2 * blockIdx.x + (p.t0 == 0)) * C::kCols + own_col;
        float4* dst = reinterpret_cast<float4*>(a.part_o + at * D) + own_ln;
#pragma unroll
        for (int v = 0; v < C::kVec; ++v) dst[v * C::kLanes] = own[v];
        if (own_ln == 0) a.part_ml[at] = ml;
      }
    }
    if (WHOLE) return;
    if (!whole && p.t0 == 0 && tid == 0) {
      // the block of a shared context's first part names it for the joins
      const int n = cut_s.block_of(p.start + p.tiles - 1) - blockIdx.x + 1;
      a.desc[2 * blockIdx.x] = make_int4(n, p.h, p.rt, p.r.q0);
      a.desc[2 * blockIdx.x + 1].x = p.r.qn;
    }
    if (!next.some) return;
    mine = mine_next;
    issued = issued_next;
    record = record_next;
  }
}

template <int D, int NT, bool MASK>
cudaError_t prepare() {
  cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<D, NT, true, MASK>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D, NT>::kSmem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(attn_decode_kernel<D, NT, false, MASK>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<D, NT>::kSmem + (kMaxRequests + 1) * (int)sizeof(int64_t));
}

template <bool MASK>
cudaError_t prepare_all() {
  cudaError_t e;
  if ((e = prepare<64, 2, MASK>()) != cudaSuccess) return e;
  if ((e = prepare<64, 1, MASK>()) != cudaSuccess) return e;
  if ((e = prepare<128, 2, MASK>()) != cudaSuccess) return e;
  if ((e = prepare<128, 1, MASK>()) != cudaSuccess) return e;
  return prepare<256, 1, MASK>();
}

template <int D, int NT, bool MASK>
cudaError_t launch(const FwdArgs& a, int64_t max_kv, int sms, cudaStream_t s) {
  using C = Cfg<D, NT>;
  const int rts = (a.max_q * a.d.G + C::kCols - 1) / C::kCols;
  const int64_t grid = (int64_t)a.B * a.d.Hkv * rts;
  if (MASK && a.window) {  // what is gone over, at most
    const int64_t view = (int64_t)a.window + a.max_q + a.sinks + 2 * kTile;
    max_kv = max_kv < view ? max_kv : view;
  }
  if (max_kv <= kWholeKv || (max_kv <= kWholeMost && max_kv <= kWholeKv + kWholeMore * grid)) {
    if (grid <= 0x7fffffff)
      return launch_pdl(attn_decode_kernel<D, NT, true, MASK>, dim3((unsigned)grid), dim3(kThreads),
                        C::kSmem, s, a);
  }
  const int blocks = sms < kMaxBlocks ? sms : kMaxBlocks;
  const cudaError_t e =
      launch_pdl(attn_decode_kernel<D, NT, false, MASK>, dim3(blocks), dim3(kThreads),
                 C::kSmem + (a.B + 1) * sizeof(int64_t), s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_join_kernel<D, C::kCols>, dim3(2 * sms), dim3(kJoinThreads), 0, s, a, blocks);
}

template <bool MASK>
cudaError_t launch_any(const FwdArgs& a, int max_kv, int sms, cudaStream_t s) {
  // two column tiles per block where a context has more than 8 rows and the registers hold them
  // (D = 256 would need 128 accumulators a lane: its second 8 rows take a block of their own)
  const bool two = a.max_q * a.d.G > 8;
  if (a.d.D == 256) return launch<256, 1, MASK>(a, max_kv, sms, s);
  if (a.d.D == 128)
    return two ? launch<128, 2, MASK>(a, max_kv, sms, s) : launch<128, 1, MASK>(a, max_kv, sms, s);
  return two ? launch<64, 2, MASK>(a, max_kv, sms, s) : launch<64, 1, MASK>(a, max_kv, sms, s);
}

}  // namespace

// A block shares at most its first and its last context with others.
int attn_part_slots(int sms) { return 2 * sms; }

cudaError_t prepare_attn_decode_kernels() {
  const cudaError_t e = prepare_all<false>();
  return e != cudaSuccess ? e : prepare_all<true>();
}

cudaError_t launch_attn_decode(const FwdArgs& a, int max_kv, int sms, cudaStream_t s) {
  return a.window || a.masks ? launch_any<true>(a, max_kv, sms, s)
                             : launch_any<false>(a, max_kv, sms, s);
}

}  // namespace moe
