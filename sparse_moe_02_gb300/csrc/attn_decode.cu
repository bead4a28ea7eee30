// Attention of few query rows over the paged 4-bit cache (include/attn.h): single tokens and
// short drafts, n_b G <= 16 rows per request and key/value head.
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
// of score + exponent(largest |s_tg|), which bounds w, instead of the score alone; it only moves
// (and the accumulators are only rescaled) when a tile exceeds it by 2^6.
//
// Layout of the work.  The rows of a key/value head (G query heads x new tokens) are the MMA's N
// side in tiles of 8, its 16 tokens the M side of the scores; a cached row is read once for all
// of them.  A block of four warps, two blocks per SM; each warp takes every fourth tile of 32
// tokens of a context through a ring of its own (bulk copies: a tile of one head lies contiguous
// in its page) and keeps its own softmax state and outputs; the block joins its warps through
// shared memory.  Contexts are cut evenly over the blocks: with W tiles in all, block i takes
// tiles [i W / n, (i + 1) W / n) whatever requests they belong to, so ragged batches balance; a
// context that several blocks share leaves partial results that a second small launch joins in
// block order (the same inputs give the same bits).  Short contexts (max_kv small) take one block
// per context and no second launch.
#include "attn.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;  // tokens per ring stage
// One block per context, no second launch, up to this many tokens.
constexpr int kWholeKv = 512;
constexpr float kSlack = 6.f;     // growth of the reference a tile may bring before a rescale
constexpr float kLift = 9.f;      // w <= 2^(kLift + kSlack) at the reference

template <int D, int NT>
struct Cfg {
  static constexpr int NG = D / kGroup;
  static constexpr int kRow = D / 2;     // code bytes per row
  static constexpr int kPar = 4 * NG;    // parameter bytes per row
  static constexpr int kOffV = kTile * kRow;
  static constexpr int kOffKp = 2 * kTile * kRow;
  static constexpr int kOffVp = kOffKp + kTile * kPar;
  static constexpr int kStage = kOffVp + kTile * kPar;
  static constexpr int kStages = D == 256 ? 3 : D == 128 ? 6 : 8;
  static constexpr int kCols = 8 * NT;
  static constexpr int kPitch = D + 8;   // floats per column of the join buffer
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kJoin = kWarps * kCols * kPitch * 4;
  static constexpr int kSmem = (kRing > kJoin ? kRing : kJoin) + 128;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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

// One block's range of work: tiles [w0, w1) of all contexts in order.
struct Range {
  int64_t total, w0, w1;
  int blocks;  // that take part
  int b;       // request of w0
  int64_t before;  // tiles of the requests before it
};

__device__ __forceinline__ int row_tiles(const FwdArgs& a, int qn, int cols) {
  return (qn * a.d.G + cols - 1) / cols;
}

__device__ __forceinline__ int kv_tiles(int kv) { return max(1, (kv + kTile - 1) / kTile); }

__device__ __forceinline__ int64_t request_tiles(const FwdArgs& a, const Req& r, int cols) {
  return r.qn > 0 ? (int64_t)a.d.Hkv * row_tiles(a, r.qn, cols) * kv_tiles(r.kv) : 0;
}

__device__ __forceinline__ int64_t bound(int64_t total, int blocks, int i) {
  return total * i / blocks;
}

__device__ __forceinline__ int64_t scan64(int64_t v, int64_t* sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sums[w];
    all += sums[w];
  }
  __syncthreads();
  *total = all;
  return v + before;
}

// The block's range (every thread gets the same answer).
__device__ Range find_range(const FwdArgs& a, int cols, int64_t* sums, int64_t* found) {
  Range R;
  int64_t total = 0, sum, incl = 0, cnt = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    cnt = b < a.B ? request_tiles(a, load_req(a, b), cols) : 0;
    if (blockIdx.x == 0 && b < a.B && req_out_of_range(a, b)) record_error(a.err, kDevErrState);
    incl = total + scan64(cnt, sums, &sum);
    total += sum;
  }
  R.total = total;
  const int64_t most = (total + kWarps - 1) / kWarps;  // a tile for each warp at least
  R.blocks = (int)(most < (int64_t)gridDim.x ? most : (int64_t)gridDim.x);
  R.w0 = R.w1 = 0;
  R.b = 0;
  R.before = 0;
  if ((int)blockIdx.x >= R.blocks) return R;
  R.w0 = bound(total, R.blocks, blockIdx.x);
  R.w1 = bound(total, R.blocks, blockIdx.x + 1);
  int64_t run = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    if (a.B > kThreads) {
      cnt = b < a.B ? request_tiles(a, load_req(a, b), cols) : 0;
      incl = run + scan64(cnt, sums, &sum);
      run += sum;
    }
    if (incl - cnt <= R.w0 && R.w0 < incl) {
      found[0] = b;
      found[1] = incl - cnt;
    }
  }
  __syncthreads();
  R.b = (int)found[0];
  R.before = found[1];
  return R;
}

// Query rows of one context and tile of columns, as MMA B fragments, for the warp's lanes.
template <int D, int NT>
struct Query {
  static constexpr int NG = D / kGroup;
  uint32_t f[NT][NG][2][4];  // [column tile][group][word][registers of two MMAs]
  float sum[NT][2][NG];      // sum of the scaled row over a group, times 2^-24, columns 2c, 2c + 1
  float scale[NT][2];        // turns the MMA's units into log2 units
  int lim[NT][2];            // tokens the column sees
};

template <int D, int NT>
__device__ __forceinline__ void load_query(const FwdArgs& a, const Req& r, int h, int rt,
                                           Query<D, NT>& Q) {
  constexpr int NG = D / kGroup;
  const int lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = (rt * NT + nt) * 8 + n;
    const bool on = row < r.qn * a.d.G;
    const int tok = row / a.d.G;
    const __nv_bfloat16* p =
        a.q + (int64_t)(r.q0 + tok) * a.q_stride + (int64_t)(h * a.d.G + row % a.d.G) * D;
    uint4 raw[NG][2];
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        raw[g][i] = on ? *reinterpret_cast<const uint4*>(p + 64 * g + 8 * (c + 4 * i))
                       : make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {raw[g][i].x, raw[g][i].y, raw[g][i].z, raw[g][i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = fmaxf(top, fmaxf(fabsf(bf16_lo(x[e])), fabsf(bf16_hi(x[e]))));
      }
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
    // 2^-e with the row's largest entry in [2^e, 2^(e+1)), kept a normal number
    const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 126);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    const float up = __uint_as_float((uint32_t)(e + 127) << 23);
    float sums[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      sums[g] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x[4] = {raw[g][i].x, raw[g][i].y, raw[g][i].z, raw[g][i].w};
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[2 * k] = bf16_lo(x[k]) * down;
          v[2 * k + 1] = bf16_hi(x[k]) * down;
        }
        // the row in [2^13, 2^14) at its top; odd nibbles of a byte arrive 16 times as large
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float m = (k & 1) ? 512.f : 8192.f;
          Q.f[nt][g][i][k] = pack_f16(v[k] * m, v[k + 4] * m);
          sums[g] += v[k] + v[k + 4];
        }
      }
      sums[g] += __shfl_xor_sync(~0u, sums[g], 1);
      sums[g] += __shfl_xor_sync(~0u, sums[g], 2);
      sums[g] *= 8192.f / 16777216.f;
    }
    // code * 2^-24 * q * 2^13-e  ->  log2 units
    const float unit = up * (16777216.f / 8192.f) * a.d.scale_log2;
    const int seen = on ? min(max(r.kv - r.qn + tok + 1, 0), r.kv) : 0;
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
      const int from = (2 * c + cc) * 4;
#pragma unroll
      for (int g = 0; g < NG; ++g) Q.sum[nt][cc][g] = __shfl_sync(~0u, sums[g], from);
      Q.scale[nt][cc] = __shfl_sync(~0u, unit, from);
      Q.lim[nt][cc] = __shfl_sync(~0u, seen, from);
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

// One tile of 32 tokens (n of them valid from the first on, in `halves` halves of 16) at shared
// address `st`; tok0 is the first token's index in its context.
template <int D, int NT>
__device__ __forceinline__ void tile_step(uint32_t st, int tok0, int kv, const Query<D, NT>& Q,
                                          State<D, NT>& s) {
  using C = Cfg<D, NT>;
  constexpr int NG = C::NG;
  const int lane = threadIdx.x & 31, j = lane >> 2, c = lane & 3;
  const int tr = row_token(j);
  const int halves = kv - tok0 > 16 ? 2 : 1;
  float x[2][NT][4];    // scores, then weights
  Words<NG> vp[2][2];   // value parameters of the lane's rows
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    if (hf >= halves) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[hf][nt][e] = -INFINITY;
#pragma unroll
      for (int g = 0; g < NG; ++g) vp[hf][0].w[g] = vp[hf][1].w[g] = 0;
      continue;
    }
    const int row = 16 * hf + tr;
    float acc[NT][NG][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][g][e] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t at = st + row * C::kRow + (((c + 4 * i) ^ row_swz(tr)) * NG) * 4;
      const Words<NG> wa = lds_words<NG>(at), wb = lds_words<NG>(at + 8 * C::kRow);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t a8 = wa.w[g] >> 8, b8 = wb.w[g] >> 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(acc[nt][g], wa.w[g] & kNib0, wb.w[g] & kNib0, wa.w[g] & kNib1, wb.w[g] & kNib1,
                  Q.f[nt][g][i][0], Q.f[nt][g][i][1]);
          mma_f16(acc[nt][g], a8 & kNib0, b8 & kNib0, a8 & kNib1, b8 & kNib1, Q.f[nt][g][i][2],
                  Q.f[nt][g][i][3]);
        }
      }
    }
    const Words<NG> ka = lds_words<NG>(st + C::kOffKp + row * C::kPar);
    const Words<NG> kb = lds_words<NG>(st + C::kOffKp + (row + 8) * C::kPar);
    vp[hf][0] = lds_words<NG>(st + C::kOffVp + row * C::kPar);
    vp[hf][1] = lds_words<NG>(st + C::kOffVp + (row + 8) * C::kPar);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const Words<NG>& k = e < 2 ? ka : kb;
        float v = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          v = fmaf(bf16_lo(k.w[g]), acc[nt][g][e], v);
          v = fmaf(bf16_hi(k.w[g]), Q.sum[nt][e & 1][g], v);
        }
        x[hf][nt][e] = v * Q.scale[nt][e & 1];
      }
  }
  // what a row may not see, and what lies behind the context (never written: anything)
  int least = Q.lim[0][0];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) least = min(least, min(Q.lim[nt][0], Q.lim[nt][1]));
  if (__any_sync(~0u, tok0 + kTile > least)) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int t = tok0 + 16 * hf + 8 * r + tr;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int cc = 0; cc < 2; ++cc)
            if (t >= Q.lim[nt][cc]) x[hf][nt][2 * r + cc] = -INFINITY;
        if (t >= kv) {
#pragma unroll
          for (int g = 0; g < NG; ++g) vp[hf][r].w[g] = 0;
        }
      }
  }
  // exponent of the largest scale of each of the lane's four tokens
  float ev[2][2];
#pragma unroll
  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t top = 0;
#pragma unroll
      for (int g = 0; g < NG; ++g) top = max(top, (vp[hf][r].w[g] << 16) & 0x7fffffffu);
      ev[hf][r] = (float)max((int)(top >> 23) - 126, -60);
    }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float top[2];
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
      top[cc] = fmaxf(fmaxf(x[0][nt][cc] + ev[0][0], x[0][nt][2 + cc] + ev[0][1]),
                      fmaxf(x[1][nt][cc] + ev[1][0], x[1][nt][2 + cc] + ev[1][1]));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top[cc] = fmaxf(top[cc], __shfl_xor_sync(~0u, top[cc], o));
    }
    if (__any_sync(~0u, top[0] > s.m[nt][0] + kSlack || top[1] > s.m[nt][1] + kSlack)) {
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const float m = fmaxf(s.m[nt][cc], top[cc]);
        const float f = m == -INFINITY ? 1.f : exp2_fast(s.m[nt][cc] - m);
        s.m[nt][cc] = m;
        s.l[nt][cc] *= f;
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
      const float m = s.m[nt][cc] == -INFINITY ? 0.f : s.m[nt][cc] - kLift;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p = exp2_fast(x[hf][nt][2 * r + cc] - m);
          x[hf][nt][2 * r + cc] = p;
          s.l[nt][cc] += p;
#pragma unroll
          for (int g = 0; g < NG; ++g)
            s.ob[nt][cc][g] = fmaf(p, bf16_hi(vp[hf][r].w[g]), s.ob[nt][cc][g]);
        }
    }
  }
  uint32_t wt[2][NT][NG][2];
  Words<NG> v[2][4];  // value words of the lane's tokens c, c + 4, c + 8, c + 12, unit j
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    if (hf >= halves) continue;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float sc = bf16_lo(vp[hf][r].w[g]);
          wt[hf][nt][g][r] =
              transpose8x8(pack_f16(x[hf][nt][2 * r] * sc, x[hf][nt][2 * r + 1] * sc));
        }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[hf][q] = lds_words<NG>(st + C::kOffV + (16 * hf + c + 4 * q) * C::kRow +
                               ((j ^ row_swz(c + 4 * q)) * NG) * 4);
  }
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const uint32_t sel = part ? 0x7632u : 0x5410u;
      // The tile's sum starts from zero and joins the running one by a rounded addition: the
      // MMA's own additions truncate, and over thousands of tiles of nonnegative codes that
      // would pull the code part down against the bias part that it nearly cancels.
      float t[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[nt][0][e] = t[nt][1][e] = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (hf >= halves) continue;
        uint32_t u0 = __byte_perm(v[hf][0].w[g], v[hf][1].w[g], sel);
        uint32_t u1 = __byte_perm(v[hf][2].w[g], v[hf][3].w[g], sel);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(t[nt][k], u0 & kNib0, u0 & kNib1, u1 & kNib0, u1 & kNib1, wt[hf][nt][g][0],
                    wt[hf][nt][g][1]);
          u0 >>= 8;
          u1 >>= 8;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          add2(s.o[nt][g][2 * part + k][0], s.o[nt][g][2 * part + k][1], t[nt][k][0], t[nt][k][1]);
          add2(s.o[nt][g][2 * part + k][2], s.o[nt][g][2 * part + k][3], t[nt][k][2], t[nt][k][3]);
        }
    }
}

// Copies of a warp's tiles into its ring, by lane 0; `pages` holds the ids of 32 tiles ahead.
template <int D, int NT>
struct Feed {
  using C = Cfg<D, NT>;
  uint8_t* ring;
  uint64_t* bars;
  uint64_t policy;

  // pg0, pg1: pages of the tile's first and second 16 tokens
  __device__ __forceinline__ void issue(const FwdArgs& a, int h, int tile, int kv, int stage,
                                        int pg0, int pg1) {
    const int P = 1 << a.d.page_shift;
    const int tok0 = tile * kTile;
    const int rows = kv - tok0 > 16 ? 32 : 16;
    uint8_t* dst = ring + stage * C::kStage;
    uint64_t* bar = bars + stage;
    mbar_arrive_expect_tx(bar, rows * 2 * (C::kRow + C::kPar));
    const int step = P < kTile ? 16 : rows;
    for (int r = 0; r < rows; r += step) {
      const int pg = r ? pg1 : pg0;
      const int64_t at = ((int64_t)pg * a.d.Hkv + h) * P + ((tok0 + r) & (P - 1));
      bulk_load(dst + r * C::kRow, a.c.kc + at * C::kRow, step * C::kRow, bar, policy);
      bulk_load(dst + C::kOffKp + r * C::kPar, reinterpret_cast<uint8_t*>(a.c.kp) + at * C::kPar,
                step * C::kPar, bar, policy);
      bulk_load(dst + C::kOffV + r * C::kRow, a.c.vc + at * C::kRow, step * C::kRow, bar, policy);
      bulk_load(dst + C::kOffVp + r * C::kPar, reinterpret_cast<uint8_t*>(a.c.vp) + at * C::kPar,
                step * C::kPar, bar, policy);
    }
  }
};

// Page ids of the 16-token halves of `tile`; an id out of range reads page 0 and is recorded.
__device__ __forceinline__ int2 tile_pages(const FwdArgs& a, int b, int tile, int kv) {
  int id[2] = {0, 0};
  const int P = 1 << a.d.page_shift;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int tok = tile * kTile + 16 * i;
    if (tok < kv && (i == 0 || P < kTile)) {
      id[i] = a.table[(int64_t)b * a.table_width + (tok >> a.d.page_shift)];
      if (id[i] < 0 || id[i] >= a.d.n_pages) {
        record_error(a.err, kDevErrState);
        id[i] = 0;
      }
    }
  }
  return make_int2(id[0], id[1]);
}

template <int D, int NT, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 2) attn_decode_kernel(FwdArgs a) {
  using C = Cfg<D, NT>;
  constexpr int NG = C::NG;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kWarps * C::kStages];
  __shared__ int64_t sums[kWarps], found[2];
  __shared__ float join_m[kWarps][C::kCols], join_l[kWarps][C::kCols];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int j = lane >> 2, c = lane & 3;
  Feed<D, NT> feed;
  feed.ring = smem + warp * C::kStages * C::kStage;
  feed.bars = bars + warp * C::kStages;
  feed.policy = policy_evict_first();
  if (lane == 0)
    for (int i = 0; i < C::kStages; ++i) mbar_init(feed.bars + i, 1);
  fence_mbar_init();
  pdl_wait();
  pdl_trigger();

  Range R;
  int rts_max = 0;
  if (WHOLE) {
    rts_max = row_tiles(a, a.max_q, C::kCols);
    R.b = blockIdx.x / (a.d.Hkv * rts_max);
    R.w0 = 0;
    R.w1 = 1;
    R.before = 0;
    R.blocks = 0;
    if (tid == 0 && blockIdx.x % (a.d.Hkv * rts_max) == 0 && req_out_of_range(a, R.b))
      record_error(a.err, kDevErrState);
  } else {
    R = find_range(a, C::kCols, sums, found);
    if (tid == 0 && a.desc) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  __syncthreads();

  int used = 0;  // stages this warp has taken so far
  int64_t w = R.w0, before = R.before;
  bool ok = true;
  for (int b = R.b; w < R.w1; ) {
    const Req r = load_req(a, b);
    const int rts = row_tiles(a, r.qn, C::kCols);
    const int nt_kv = kv_tiles(r.kv);
    int h, rt, t0, t1;
    if (WHOLE) {
      const int k = blockIdx.x % (a.d.Hkv * rts_max);
      h = k / rts_max;
      rt = k % rts_max;
      t0 = 0;
      t1 = nt_kv;
      w = R.w1;
      if (rt >= rts) break;
    } else {
      const int64_t n = r.qn > 0 ? (int64_t)a.d.Hkv * rts * nt_kv : 0;
      if (w >= before + n) {
        before += n;
        ++b;
        continue;
      }
      const int64_t k = (w - before) / nt_kv;
      h = (int)(k / rts);
      rt = (int)(k % rts);
      t0 = (int)((w - before) % nt_kv);
      const int64_t left = R.w1 - w;
      t1 = (int)(left < nt_kv - t0 ? t0 + left : nt_kv);
    }
    // the warp's tiles: t0 + warp, + kWarps, ... below the end of the context
    const int last = min(t1, (r.kv + kTile - 1) / kTile);
    const int first = t0 + warp;
    const int mine = last > first ? (last - first + kWarps - 1) / kWarps : 0;
    int2 pages = make_int2(0, 0), pages_next = pages;
    if (lane < mine) pages = tile_pages(a, b, first + lane * kWarps, r.kv);
    const int start = min(mine, C::kStages);
    int issued = ok ? start : 0;
    for (int i = 0; i < issued; ++i) {
      const int pg0 = __shfl_sync(~0u, pages.x, i), pg1 = __shfl_sync(~0u, pages.y, i);
      if (lane == 0)
        feed.issue(a, h, first + i * kWarps, r.kv, (used + i) % C::kStages, pg0, pg1);
    }
    Query<D, NT> Q;
    load_query<D, NT>(a, r, h, rt, Q);
    State<D, NT> s;
    clear(s);
    for (int i = 0; i < mine; ++i) {
      const int stage = used % C::kStages;
      // after a wait that ran out nothing more is copied, but what is under way still lands
      if (i < issued) ok = mbar_wait(feed.bars + stage, (used / C::kStages) & 1, a.err) && ok;
      ok = __all_sync(~0u, ok);
      if (ok)
        tile_step<D, NT>(smem_u32(feed.ring + stage * C::kStage), (first + i * kWarps) * kTile,
                         r.kv, Q, s);
      ++used;
      __syncwarp();
      const int nx = i + C::kStages;
      if ((nx & 31) == 0) pages = pages_next;
      if ((nx & 31) == 16) {  // the ids of the following 32 tiles, half a batch ahead
        const int f = nx + 16 + lane;
        if (f < mine) pages_next = tile_pages(a, b, first + f * kWarps, r.kv);
      }
      if (nx < mine && ok) {
        issued = nx + 1;
        const int pg0 = __shfl_sync(~0u, pages.x, nx & 31);
        const int pg1 = __shfl_sync(~0u, pages.y, nx & 31);
        if (lane == 0) feed.issue(a, h, first + nx * kWarps, r.kv, stage, pg0, pg1);
      }
    }

    // join the warps
    __syncthreads();  // every warp is done with its ring
    float* join = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int col = 8 * nt + 2 * c + cc;
        float l = s.l[nt][cc];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(~0u, l, o);
        if (j == 0) {
          join_m[warp][col] = s.m[nt][cc];
          join_l[warp][col] = l;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float ob = s.ob[nt][cc][g];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) ob += __shfl_xor_sync(~0u, ob, o);
          float v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[2 * i] = fmaf(s.o[nt][g][i][cc], 16777216.f, ob);
            v[2 * i + 1] = fmaf(s.o[nt][g][i][2 + cc], 1048576.f, ob);
          }
          float4* dst = reinterpret_cast<float4*>(
              join + (warp * C::kCols + col) * C::kPitch + 64 * g + 8 * j);
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
    __syncthreads();
    const bool whole = WHOLE || (t0 == 0 && t1 == nt_kv);
    const int slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
    for (int i = tid; i < C::kCols * (D / 4); i += kThreads) {
      const int col = i / (D / 4), ch = 4 * (i % (D / 4));
      float m = join_m[0][col];
#pragma unroll
      for (int k = 1; k < kWarps; ++k) m = fmaxf(m, join_m[k][col]);
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float mk = join_m[k][col];
        const float f = mk == -INFINITY ? (join_l[k][col] == 0.f ? 0.f : 1.f) : exp2_fast(mk - m);
        const float4 v =
            *reinterpret_cast<const float4*>(join + (k * C::kCols + col) * C::kPitch + ch);
        l = fmaf(join_l[k][col], f, l);
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z);
        o.w = fmaf(v.w, f, o.w);
      }
      if (whole) {
        const int row = rt * C::kCols + col;
        if (row < r.qn * a.d.G) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          __nv_bfloat16* dst = a.out + (int64_t)(r.q0 + row / a.d.G) * a.out_stride +
                               (int64_t)(h * a.d.G + row % a.d.G) * D + ch;
          __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
          __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
          *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<uint32_t*>(&lo),
                                                      *reinterpret_cast<uint32_t*>(&hi));
        }
      } else {
        *reinterpret_cast<float4*>(a.part_o + ((int64_t)slot * C::kCols + col) * D + ch) = o;
        if (ch == 0) a.part_ml[slot * C::kCols + col] = make_float2(m, l);
      }
    }
    if (!WHOLE) {
      if (!whole && t0 == 0 && tid == 0) {
        // this block has the context's first part: it names the join
        const int64_t end = w + nt_kv;
        // the last block that starts before the end
        const int last_block = (int)((end * R.blocks + R.total - 1) / R.total) - 1;
        a.desc[blockIdx.x] = make_int4(last_block - blockIdx.x + 1, b, h, rt);
      }
      w += t1 - t0;
    }
    fence_proxy_async_smem();  // the ring is written by copies again
    __syncthreads();
  }
}

// Joins the parts of a context that several blocks share: block x names it (its own second part,
// then the first parts of the following blocks), y is the column.
template <int D, int NT>
__global__ void __launch_bounds__(128) attn_join_kernel(FwdArgs a) {
  constexpr int kCols = 8 * NT;
  constexpr int kLanes = D / 4;            // threads over the channels
  constexpr int kGroups = 128 / kLanes;    // over the parts
  __shared__ float4 acc[kGroups][kLanes];
  __shared__ float red[4], ls[kGroups];
  const int tid = threadIdx.x, col = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const int4 d = a.desc[blockIdx.x];
  if (d.x == 0) return;
  const Req r = load_req(a, d.y);
  const int row = d.w * kCols + col;
  if (row >= r.qn * a.d.G) return;
  const int base = 2 * blockIdx.x;
  float m = -INFINITY;
  for (int i = tid; i < d.x; i += 128)
    m = fmaxf(m, a.part_ml[(base + (i ? 2 * i : 1)) * kCols + col].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const int ln = tid % kLanes, grp = tid / kLanes;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int i = grp; i < d.x; i += kGroups) {
    const int slot = base + (i ? 2 * i : 1);
    const float2 ml = a.part_ml[slot * kCols + col];
    const float4 v =
        *reinterpret_cast<const float4*>(a.part_o + ((int64_t)slot * kCols + col) * D + 4 * ln);
    const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2_fast(ml.x - m);
    l = fmaf(ml.y, f, l);
    o.x = fmaf(v.x, f, o.x);
    o.y = fmaf(v.y, f, o.y);
    o.z = fmaf(v.z, f, o.z);
    o.w = fmaf(v.w, f, o.w);
  }
  acc[grp][ln] = o;
  if (ln == 0) ls[grp] = l;
  __syncthreads();
  if (grp == 0) {
    float sum = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      sum += ls[k];
      o.x += acc[k][ln].x;
      o.y += acc[k][ln].y;
      o.z += acc[k][ln].z;
      o.w += acc[k][ln].w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __nv_bfloat16* dst = a.out + (int64_t)(r.q0 + row / a.d.G) * a.out_stride +
                         (int64_t)(d.z * a.d.G + row % a.d.G) * D + 4 * ln;
    __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  }
}

template <int D, int NT>
cudaError_t prepare() {
  cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<D, NT, true>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D, NT>::kSmem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(attn_decode_kernel<D, NT, false>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, NT>::kSmem);
}

template <int D, int NT>
cudaError_t launch(const FwdArgs& a, int max_kv, int sms, cudaStream_t s) {
  using C = Cfg<D, NT>;
  const int rts = (a.max_q * a.d.G + C::kCols - 1) / C::kCols;
  if (max_kv <= kWholeKv) {
    const int64_t grid = (int64_t)a.B * a.d.Hkv * rts;
    if (grid <= 0x7fffffff)
      return launch_pdl(attn_decode_kernel<D, NT, true>, dim3((unsigned)grid), dim3(kThreads),
                        C::kSmem, s, a);
  }
  const int blocks = attn_decode_blocks(sms);
  cudaError_t e = launch_pdl(attn_decode_kernel<D, NT, false>, dim3(blocks), dim3(kThreads),
                             C::kSmem, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_join_kernel<D, NT>, dim3(blocks, C::kCols), dim3(128), 0, s, a);
}

}  // namespace

int attn_decode_blocks(int sms) { return 2 * sms; }

size_t attn_decode_part_floats(int D) { return (size_t)(D == 256 ? 8 : 16) * D; }

cudaError_t prepare_attn_decode_kernels() {
  cudaError_t e;
  if ((e = prepare<64, 2>()) != cudaSuccess) return e;
  if ((e = prepare<64, 1>()) != cudaSuccess) return e;
  if ((e = prepare<128, 2>()) != cudaSuccess) return e;
  if ((e = prepare<128, 1>()) != cudaSuccess) return e;
  return prepare<256, 1>();
}

cudaError_t launch_attn_decode(const FwdArgs& a, int max_kv, int sms, cudaStream_t s) {
  // two column tiles per block where a context has more than 8 rows and the registers hold them
  // (D = 256 would need 128 accumulators a lane: its second 8 rows take a block of their own)
  const bool two = a.max_q * a.d.G > 8;
  if (a.d.D == 256) return launch<256, 1>(a, max_kv, sms, s);
  if (a.d.D == 128)
    return two ? launch<128, 2>(a, max_kv, sms, s) : launch<128, 1>(a, max_kv, sms, s);
  return two ? launch<64, 2>(a, max_kv, sms, s) : launch<64, 1>(a, max_kv, sms, s);
}

}  // namespace moe
