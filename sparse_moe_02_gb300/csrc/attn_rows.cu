// The row kernels of the attention step (include/attn.h): norm and rotation of query and key
// heads, quantisation of keys and values into the paged 4-bit cache, both in one, accepted rows
// moved, and the way back.  Each is one pass over its rows, bound by launch latency for single
// tokens and for prompts as stated at each (by loads that wait for one another, append by
// instruction issue): a lane holds 8 channels (one 16-byte load), the D / 8 lanes of a row reduce
// by shuffles.
#include "attn.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMostHeads = 8;  // of a group of lanes, in the norm and rotation
constexpr int kMostQueries = 4;  // the same where rows are appended too: registers of five blocks an SM

struct Row8 {
  float x[8];
};

__device__ __forceinline__ Row8 widen(uint4 w) {
  Row8 r;
  r.x[0] = bf16_lo(w.x); r.x[1] = bf16_hi(w.x); r.x[2] = bf16_lo(w.y); r.x[3] = bf16_hi(w.y);
  r.x[4] = bf16_lo(w.z); r.x[5] = bf16_hi(w.z); r.x[6] = bf16_lo(w.w); r.x[7] = bf16_hi(w.w);
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 narrow(const Row8& r) {
  return make_uint4(pack_bf16(r.x[0], r.x[1]), pack_bf16(r.x[2], r.x[3]),
                    pack_bf16(r.x[4], r.x[5]), pack_bf16(r.x[6], r.x[7]));
}

// ------------------------------------------------------------------- norm and rotation

// A group of L = D / 8 lanes takes heads_per neighbouring heads of one token: the token's cosines
// and sines and the norm weights stay in registers for all of them.  Single tokens spread their
// heads over as many groups as there are; prompts take up to eight heads to a group, so that the
// rotation's table rows are read once for eight heads.
//
// Measured: one token, 16 query and 2 key heads of 256 channels, 2.1 us (a launch); a prompt of 16381
// tokens, 32 and 8 heads of 128, 73 us, 4.7 TB/s, 69% of a copy's rate.  There it issues on half of its
// slots and DRAM is busy for half of the time: the loads of a group are all in flight before its
// first use, and what is left is the latency of position, then table row, before the first store.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) attn_rope_kernel(RopeArgs a, int heads_per) {
  constexpr int L = D / 8;
  constexpr int kPerBlock = kThreads / L;
  const int li = threadIdx.x % L;
  const int ch = 8 * li;
  const int heads = a.Hq + a.Hkv;
  const uint32_t splits = (heads + heads_per - 1) / heads_per;
  const int half = a.rot / 2;
  const bool turn = ch < a.rot;
  pdl_wait();
  pdl_trigger();
  const Row8 wq = widen(*reinterpret_cast<const uint4*>(a.qw + ch));
  const Row8 wk = widen(*reinterpret_cast<const uint4*>(a.kw + ch));
  {
    const uint32_t item = blockIdx.x * kPerBlock + threadIdx.x / L;
    const bool live = item < (uint32_t)a.T * splits;
    const int t = live ? (int)(item / splits) : 0;
    const int h0 = live ? (int)(item % splits) * heads_per : heads;
    // all heads are requested before the position, which the table rows wait for
    uint4 raw[kMostHeads];
#pragma unroll
    for (int i = 0; i < kMostHeads; ++i) {
      const int h = h0 + i;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (i < heads_per && h < heads) {
        const __nv_bfloat16* src = h < a.Hq ? a.q + t * a.q_stride + (int64_t)h * D
                                            : a.k + t * a.k_stride + (int64_t)(h - a.Hq) * D;
        raw[i] = *reinterpret_cast<const uint4*>(src + ch);
      }
    }
    float cs[8], sn[8];
    if (turn && live) {
      int pos = a.positions[t];
      if (pos < 0 || pos >= a.n_positions) {
        if (li == 0) record_error(a.err, kDevErrState);
        pos = 0;
      }
      const float* row = a.cos_sin + (int64_t)pos * a.rot;
      if (INTER) {  // pairs ch / 2 .. ch / 2 + 3
        const float4 c = *reinterpret_cast<const float4*>(row + ch / 2);
        const float4 s = *reinterpret_cast<const float4*>(row + half + ch / 2);
        cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
        sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
      } else {
        const int i = ch < half ? ch : ch - half;
        // the upper half of a pair turns to b cos + a sin: its sine enters with the other sign
        const float sg = ch < half ? -1.f : 1.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 c = *reinterpret_cast<const float4*>(row + i + 4 * e);
          const float4 s = *reinterpret_cast<const float4*>(row + half + i + 4 * e);
          cs[4 * e] = c.x; cs[4 * e + 1] = c.y; cs[4 * e + 2] = c.z; cs[4 * e + 3] = c.w;
          sn[4 * e] = sg * s.x; sn[4 * e + 1] = sg * s.y;
          sn[4 * e + 2] = sg * s.z; sn[4 * e + 3] = sg * s.w;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kMostHeads; ++i) {
      if (i >= heads_per) break;
      const int h = h0 + i;
      const bool on = h < heads;
      const bool isq = h < a.Hq;
      Row8 r = widen(raw[i]);
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(r.x[e], r.x[e], sum);
#pragma unroll
      for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
      const float inv = rsqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) r.x[e] = r.x[e] * inv * (isq ? wq.x[e] : wk.x[e]);
      if (a.rot) {
        if (INTER) {
          if (turn) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = r.x[2 * e], y = r.x[2 * e + 1];
              r.x[2 * e] = x * cs[e] - y * sn[e];
              r.x[2 * e + 1] = y * cs[e] + x * sn[e];
            }
          }
        } else {
          // the pair's other half sits half / 8 lanes away
          const int base = (threadIdx.x & 31) - li;
          const int mate = turn ? base + (ch < half ? li + half / 8 : li - half / 8)
                                : (threadIdx.x & 31);
          Row8 m;
#pragma unroll
          for (int e = 0; e < 8; ++e) m.x[e] = __shfl_sync(~0u, r.x[e], mate);
          if (turn) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r.x[e] = r.x[e] * cs[e] + m.x[e] * sn[e];
          }
        }
      }
      if (on) {
        __nv_bfloat16* dst = isq ? a.q_out + t * a.q_out_stride + (int64_t)h * D
                                 : a.k_out + t * a.k_out_stride + (int64_t)(h - a.Hq) * D;
        *reinterpret_cast<uint4*>(dst + ch) = narrow(r);
      }
    }
  }
}

// ------------------------------------------------------------------- cached rows

// Larger and smaller of each bf16 pair, NaN if either is.
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Record of slot and head.
__device__ __forceinline__ int64_t record_of(const RowsArgs& a, int slot, int h) {
  const int64_t page = slot >> a.page_shift;
  return ((page * a.Hkv + h) << (a.page_shift - 4)) + ((slot & ((1 << a.page_shift) - 1)) >> 4);
}

struct Coded {
  uint32_t word;    // the lane's 8 codes
  uint32_t params;  // the group's scale and bias
  bool finite;
};

// A lane's 8 channels as the pairs (i, i + 4): what packed fp32 instructions work on.
struct Pairs8 {
  float2 p[4];
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Packed operations.  (ptxas fuses a packed product and sum, .rn or not: measured, sums that nearly
// cancel came out fused.  Where that would change a value, the product is formed by mul_each.)
#define MOE_PACKED2(name, op)                                                                  \
  __device__ __forceinline__ float2 name(float2 a, float2 b) {                                 \
    float2 r;                                                                                  \
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\t" op         \
        ".rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"                                      \
        : "=f"(r.x), "=f"(r.y)                                                                 \
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));                                             \
    return r;                                                                                  \
  }
MOE_PACKED2(add2, "add")
MOE_PACKED2(mul2, "mul")
#undef MOE_PACKED2

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 p, q, s;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\t"
      "mov.b64 s, {%6, %7};\n\tfma.rn.f32x2 p, p, q, s;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

__device__ __forceinline__ Pairs8 widen_pairs(uint4 w) {
  return Pairs8{{make_float2(bf16_lo(w.x), bf16_lo(w.z)), make_float2(bf16_hi(w.x), bf16_hi(w.z)),
                 make_float2(bf16_lo(w.y), bf16_lo(w.w)), make_float2(bf16_hi(w.y), bf16_hi(w.w))}};
}

__device__ __forceinline__ uint4 narrow(const Pairs8& r) {
  return make_uint4(pack_bf16(r.p[0].x, r.p[1].x), pack_bf16(r.p[2].x, r.p[3].x),
                    pack_bf16(r.p[0].y, r.p[1].y), pack_bf16(r.p[2].y, r.p[3].y));
}

// Largest magnitude of three.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// bf16(range / 15), the quotient rounded to fp32 before.  The product with 1 / 15 is within two
// units in the last place of that quotient, so both round to the same bf16 unless the product lies
// that near the middle between two: then, and for quotients that are no normal numbers, the
// division itself decides.
__device__ __forceinline__ __nv_bfloat16 step_of(float range) {
  float p = __fmul_rn(range, 1.f / 15.f);
  const uint32_t past = (__float_as_uint(p) & 0xffffu) - 0x7ffcu;
  if (past <= 8u || !(p > 1e-30f && p < 1e38f)) p = __fdiv_rn(range, 15.f);
  return __float2bfloat16_rn(p);
}

// Codes of the lane's 8 channels; the 8 lanes of a group share lo and step.  Every code equals the
// one that the definition's fp32 division and rounding give.
__device__ __forceinline__ Coded code_row(uint4 w) {
  const uint32_t lo2 = min_nan2(min_nan2(w.x, w.y), min_nan2(w.z, w.w));
  const uint32_t hi2 = max_nan2(max_nan2(w.x, w.y), max_nan2(w.z, w.w)) ^ 0x80008000u;
  // (smallest, largest negated): the smaller of each
  uint32_t ends = min_nan2(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) ends = min_nan2(ends, __shfl_xor_sync(~0u, ends, o));
  const float lo = bf16_lo(ends), hi = -bf16_hi(ends);
  const __nv_bfloat16 sb = step_of(__fsub_rn(hi, lo));
  const float step = __bfloat162float(sb);
  const Pairs8 r = widen_pairs(w);
  Coded c;
  c.finite = fabsf(lo) < kLargest && fabsf(hi) < kLargest;  // false for NaN
  float2 q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = both(0.f);
  if (step > 0.f) {
    // The product with the reciprocal (itself within a unit in the last place) is within 2^-18 of
    // the rounded quotient, so it rounds to the same code (at most 15) unless it lies near a half:
    // then, and for steps whose reciprocal is no normal number, the quotient itself decides.  2^23
    // is added and taken off to round.
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));
    float2 d[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = mul2(add2(r.p[e], both(-lo)), both(inv));
      q[e] = add2(add2(y, both(8388608.f)), both(-8388608.f));
      d[e] = fma2(q[e], both(-1.f), y);
    }
    const float far = fmaxf(max_abs3(max_abs3(d[0].x, d[0].y, d[1].x), d[1].y, d[2].x),
                            max_abs3(d[2].y, d[3].x, d[3].y));
    if (far > 0.49998f || step < 1e-35f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q[e].x = fminf(rintf(__fdiv_rn(__fsub_rn(r.p[e].x, lo), step)), 15.f);
        q[e].y = fminf(rintf(__fdiv_rn(__fsub_rn(r.p[e].y, lo), step)), 15.f);
      }
    }
  }
  // four codes as the low 16 bits of 2^23 + c0 + 16 c1 + 256 c2 + 4096 c3
  const float2 a = fma2(q[1], both(16.f), q[0]), b = fma2(q[3], both(16.f), q[2]);
  const float2 half = add2(fma2(b, both(256.f), a), both(8388608.f));
  c.word = __byte_perm(__float_as_uint(half.x), __float_as_uint(half.y), 0x5410);
  const __nv_bfloat16 lb = __float2bfloat16_rn(lo);
  c.params = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(lb) << 16);
  return c;
}

// Writes a token's coded key and value rows of head h to its slot, the lane's 8 channels of each.
template <int D>
__device__ __forceinline__ void write_rows(const RowsArgs& a, int slot, int h, int li,
                                           unsigned group_mask, Coded k, Coded v) {
  using R = Record<D>;
  constexpr int NG = D / kGroup;
  const bool good = (__ballot_sync(~0u, !(k.finite && v.finite)) & group_mask) == 0;
  if (!good) {  // queries that see the token read NaN, through its scores
    k.word = v.word = 0;
    k.params = 0x7fc00000u;
    v.params = 0;
  }
  if (slot >= a.n_slots) {
    if (li == 0) record_error(a.err, kDevErrState);
  } else if (slot >= 0) {
    uint8_t* rec = a.cache + record_of(a, slot, h) * R::kBytes;
    const int row = slot & 15, word = ((li & 7) ^ row_swz(slot)) * NG + (li >> 3);
    reinterpret_cast<uint32_t*>(rec + row * R::kRow)[word] = k.word;
    reinterpret_cast<uint32_t*>(rec + R::kV + row * R::kRow)[word] = v.word;
    if ((li & 7) == 0) {
      reinterpret_cast<uint32_t*>(rec + R::kKp + row * R::kPar)[li >> 3] = k.params;
      reinterpret_cast<uint32_t*>(rec + R::kVp + row * R::kPar)[li >> 3] = v.params;
    }
  }
}

// A group of L = D / 8 lanes per (token, head): key row and value row together, since a
// non-finite channel of either marks both.
//
// Bound by instruction issue for prompts (370 warp instructions a row and head, 72% of the slots): the
// fp32 quotient of the definition would be 16 divisions a lane, so the reciprocal decides where it
// provably rounds to the same code.  Measured: 32768 tokens, 2 heads of 256 channels, 27 us (3.1 TB/s),
// their reading 16 us (5.3 TB/s), both in turn 46 us; 48 tokens 4.0 us for both.
template <int D>
__global__ void __launch_bounds__(kThreads) attn_append_kernel(RowsArgs a) {
  constexpr int L = D / 8;
  constexpr int kPerBlock = kThreads / L;
  const int li = threadIdx.x % L;
  const unsigned group_mask = L == 32 ? ~0u : ((1u << L) - 1) << ((threadIdx.x & 31) - li);
  const uint32_t rows = (uint32_t)a.T * a.Hkv;  // below 2^27
  pdl_wait();
  pdl_trigger();
  {
    const uint32_t row = blockIdx.x * kPerBlock + threadIdx.x / L;
    const bool live = row < rows;
    const int t = live ? (int)(row / (uint32_t)a.Hkv) : 0, h = live ? (int)(row % (uint32_t)a.Hkv) : 0;
    const int slot = live ? a.slots[t] : -1;
    const uint4 kw = *reinterpret_cast<const uint4*>(a.k + t * a.k_stride + h * D + 8 * li);
    const uint4 vw = *reinterpret_cast<const uint4*>(a.v + t * a.v_stride + h * D + 8 * li);
    write_rows<D>(a, slot, h, li, group_mask, code_row(kw), code_row(vw));
  }
}

// ------------------------------------------------------------------- norm, rotation and append

// a times b, rounded by itself.
__device__ __forceinline__ float2 mul_each(float2 a, float2 b) {
  return make_float2(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y));
}

// a b + c d, the products rounded before they are added.
__device__ __forceinline__ float2 sum_of_products(float2 a, float2 b, float2 c, float2 d) {
  return add2(mul_each(a, b), mul_each(c, d));
}

// s + p, with what the sum rounds off (exactly, Knuth's two-sum) added to e.
__device__ __forceinline__ float add_exact(float s, float p, float& e) {
  const float t = __fadd_rn(s, p), u = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, u)), __fsub_rn(p, u)));
  return t;
}

__device__ __forceinline__ float2 add_exact(float2 s, float2 p, float2& e) {
  const float2 less = both(-1.f);
  const float2 t = add2(s, p), u = fma2(s, less, t);
  const float2 ds = fma2(fma2(u, less, t), less, s), dp = fma2(u, less, p);
  e = add2(e, add2(ds, dp));
  return t;
}

// Sum over L neighbouring lanes of the lanes' squares (fp32 numbers, those of bf16 values), rounded
// once: a second float carries what the first one's additions round off.
template <int L>
__device__ __forceinline__ float sum_squares_exact(const Pairs8& r) {
  float2 e2 = both(0.f), s2 = mul2(r.p[0], r.p[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s2 = add_exact(s2, mul2(r.p[i], r.p[i]), e2);
  float e = __fadd_rn(e2.x, e2.y), s = add_exact(s2.x, s2.y, e);
#pragma unroll
  for (int o = L / 2; o; o >>= 1) {
    const float p = __shfl_xor_sync(~0u, s, o);
    e = __fadd_rn(e, __shfl_xor_sync(~0u, e, o));
    s = add_exact(s, p, e);
  }
  return s < INFINITY ? __fadd_rn(s, e) : s;
}

// Cosines and sines of a lane's channels ch .. ch + 7 at a token's position (a position out of
// range at 0), in pairs as the channels': of the channels' angles, the sines of the lower half
// negated; INTER: of the angles of channels (2i, 2i + 1), the first two pairs.
struct Turn {
  float2 c[4], s[4];
};

// A token's row of the table; `first` lane records a position out of range.
__device__ __forceinline__ const float* turn_row_at(const RopeArgs& a, int t, bool first) {
  int pos = a.positions[t];
  if (pos < 0 || pos >= a.n_positions) {
    if (first) record_error(a.err, kDevErrState);
    pos = 0;
  }
  return a.cos_sin + (int64_t)pos * a.rot;
}

template <bool INTER>
__device__ __forceinline__ void load_turn(const RopeArgs& a, int t, int li, int ch, Turn& x) {
  const int half = a.rot / 2;
  const float* row = turn_row_at(a, t, li == 0);
  const int i = INTER ? ch / 2 : ch < half ? ch : ch - half;
  const float4 c0 = *reinterpret_cast<const float4*>(row + i);
  const float4 s0 = *reinterpret_cast<const float4*>(row + half + i);
  if (INTER) {
    x.c[0] = make_float2(c0.x, c0.z), x.c[1] = make_float2(c0.y, c0.w);
    x.s[0] = make_float2(s0.x, s0.z), x.s[1] = make_float2(s0.y, s0.w);
  } else {
    const float4 c1 = *reinterpret_cast<const float4*>(row + i + 4);
    const float4 s1 = *reinterpret_cast<const float4*>(row + half + i + 4);
    const float2 sg = both(ch < half ? -1.f : 1.f);
    x.c[0] = make_float2(c0.x, c1.x), x.c[1] = make_float2(c0.y, c1.y);
    x.c[2] = make_float2(c0.z, c1.z), x.c[3] = make_float2(c0.w, c1.w);
    x.s[0] = mul2(sg, make_float2(s0.x, s1.x)), x.s[1] = mul2(sg, make_float2(s0.y, s1.y));
    x.s[2] = mul2(sg, make_float2(s0.z, s1.z)), x.s[3] = mul2(sg, make_float2(s0.w, s1.w));
  }
}

// Norm (NORM) and rotation of a key row, in the single operations that include/attn.h states.
template <int D, bool INTER, bool NORM>
__device__ __forceinline__ uint4 turn_key(const RopeArgs& a, uint4 raw, const Pairs8& w, int li, int ch,
                                          const Turn& x) {
  constexpr int L = D / 8;
  Pairs8 r = widen_pairs(raw);
  if (NORM) {
    const float mean = __fmul_rn(sum_squares_exact<L>(r), 1.f / D);
    const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(mean, a.eps)));
#pragma unroll
    for (int e = 0; e < 4; ++e) r.p[e] = mul2(mul2(r.p[e], both(inv)), w.p[e]);
  }
  if (a.rot) {
    const bool turn = ch < a.rot;
    if (INTER) {
      if (turn) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 u = r.p[2 * e], v = r.p[2 * e + 1];
          const float2 minus = make_float2(-x.s[e].x, -x.s[e].y);
          r.p[2 * e] = sum_of_products(u, x.c[e], v, minus);
          r.p[2 * e + 1] = sum_of_products(v, x.c[e], u, x.s[e]);
        }
      }
    } else {
      // the pair's other half sits half / 8 lanes away
      const int half = a.rot / 2, lane = threadIdx.x & 31;
      const int mate = turn ? lane - li + (ch < half ? li + half / 8 : li - half / 8) : lane;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 m = make_float2(__shfl_sync(~0u, r.p[e].x, mate),
                                     __shfl_sync(~0u, r.p[e].y, mate));
        if (turn) r.p[e] = sum_of_products(r.p[e], x.c[e], m, x.s[e]);
      }
    }
  }
  return narrow(r);
}

// A lane's 8 channels of a query row, laid out so that a rotation's pairs (u, v) lie in one lane:
// neighbouring channels (INTER), or four channels and their mates half the rotated ones away;
// behind the rotated channels eight neighbouring ones.
template <bool INTER>
struct QueryPiece {
  int first, second;  // channels of the four lower and the four upper ones

  __device__ __forceinline__ QueryPiece(int rot, int li) {
    const bool split = !INTER && li < rot / 8;
    first = split ? 4 * li : 8 * li;
    second = split ? rot / 2 + 4 * li : 8 * li + 4;
  }
  __device__ __forceinline__ uint4 load(const __nv_bfloat16* row) const {
    if (INTER) return *reinterpret_cast<const uint4*>(row + first);
    const uint2 x = *reinterpret_cast<const uint2*>(row + first);
    const uint2 y = *reinterpret_cast<const uint2*>(row + second);
    return make_uint4(x.x, x.y, y.x, y.y);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* row, uint4 w) const {
    if (INTER) {
      *reinterpret_cast<uint4*>(row + first) = w;
    } else {
      *reinterpret_cast<uint2*>(row + first) = make_uint2(w.x, w.y);
      *reinterpret_cast<uint2*>(row + second) = make_uint2(w.z, w.w);
    }
  }
  // u0, u1, v0, v1
  static __device__ __forceinline__ Pairs8 pairs(uint4 w) {
    if (INTER)
      return Pairs8{{make_float2(bf16_lo(w.x), bf16_lo(w.y)), make_float2(bf16_lo(w.z), bf16_lo(w.w)),
                     make_float2(bf16_hi(w.x), bf16_hi(w.y)), make_float2(bf16_hi(w.z), bf16_hi(w.w))}};
    return Pairs8{{make_float2(bf16_lo(w.x), bf16_hi(w.x)), make_float2(bf16_lo(w.y), bf16_hi(w.y)),
                   make_float2(bf16_lo(w.z), bf16_hi(w.z)), make_float2(bf16_lo(w.w), bf16_hi(w.w))}};
  }
  static __device__ __forceinline__ uint4 words(const Pairs8& r) {
    if (INTER)
      return make_uint4(pack_bf16(r.p[0].x, r.p[2].x), pack_bf16(r.p[0].y, r.p[2].y),
                        pack_bf16(r.p[1].x, r.p[3].x), pack_bf16(r.p[1].y, r.p[3].y));
    return make_uint4(pack_bf16(r.p[0].x, r.p[0].y), pack_bf16(r.p[1].x, r.p[1].y),
                      pack_bf16(r.p[2].x, r.p[2].y), pack_bf16(r.p[3].x, r.p[3].y));
  }
};

// Norm (NORM) and rotation (by angles with cosines c and sines s) of a query row.
template <int D, bool INTER, bool NORM>
__device__ __forceinline__ uint4 turn_query(const RopeArgs& a, uint4 raw, const Pairs8& w, bool turn,
                                            const float2 (&c)[2], const float2 (&s)[2]) {
  Pairs8 r = QueryPiece<INTER>::pairs(raw);
  if (NORM) {
    float2 s2 = mul2(r.p[0], r.p[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s2 = fma2(r.p[i], r.p[i], s2);
    float sum = s2.x + s2.y;
#pragma unroll
    for (int o = D / 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const float inv = rsqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
    for (int e = 0; e < 4; ++e) r.p[e] = mul2(mul2(r.p[e], both(inv)), w.p[e]);
  }
  if (turn) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 u = r.p[e], v = r.p[2 + e];
      r.p[e] = fma2(u, c[e], mul2(v, make_float2(-s[e].x, -s[e].y)));
      r.p[2 + e] = fma2(v, c[e], mul2(u, s[e]));
    }
  }
  return QueryPiece<INTER>::words(r);
}

// How the blocks of attn_rope_append_kernel share the work.
struct Shares {
  int heads_per;     // neighbouring query heads of a token that a group of lanes takes
  uint32_t splits;   // groups for a token's
  uint32_t kv_rate;  // key and value blocks among all, over 2^32: block b is the (b kv_rate >> 32)-th
  Divide by_heads, by_splits;
};

// attn_qk_norm_rope_append: a group of L = D / 8 lanes per row.  kv_blocks of the blocks take a key
// and a value row each group, the others heads_per neighbouring query heads of a token, as in the
// norm and rotation alone; both kinds evenly mixed, since the first is bound by instruction issue
// and the second by memory.
//
// Bound by instruction issue for prompts (68% of the slots, DRAM at 4.4 TB/s): a warp takes 87
// instructions a query row of two (128 channels), 500 for two key and value rows, of which the
// exact sum and root are 110 and the codes 300.  Measured: 16381 tokens, 32 query and 8 key/value
// heads of 128 channels 75 us with neighbouring pairs, 80 with halves (the norm and rotation, then
// the append: 108 and 128), 16 and 2 of 256 64 and 68 us; 48 tokens 2.9 us.  Steps of the way
// there: key and value blocks first 115 us, four query heads a group and four blocks an SM instead
// of eight and three 96, products in place of divisions 86, five blocks an SM 77, a rotation's
// pairs of a query in one lane 75 (halves: 101 to 80).
template <int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads, 5) attn_rope_append_kernel(RopeArgs r, RowsArgs a,
                                                                    Shares n) {
  constexpr int L = D / 8;
  constexpr int kPerBlock = kThreads / L;
  const int li = threadIdx.x % L;
  const int ch = 8 * li;
  const unsigned group_mask = L == 32 ? ~0u : ((1u << L) - 1) << ((threadIdx.x & 31) - li);
  const bool turn = ch < r.rot;
  pdl_wait();
  pdl_trigger();
  // block b's place among the blocks of its kind
  const uint32_t kv_before = __umulhi(blockIdx.x, n.kv_rate);
  if (__umulhi(blockIdx.x + 1, n.kv_rate) > kv_before) {
    const uint32_t row = kv_before * kPerBlock + threadIdx.x / L;
    const bool live = row < (uint32_t)a.T * a.Hkv;  // below 2^27
    const int t = live ? (int)n.by_heads(row) : 0, h = live ? (int)row - t * a.Hkv : 0;
    const uint4 kw = *reinterpret_cast<const uint4*>(a.k + t * a.k_stride + h * D + ch);
    const uint4 vw = *reinterpret_cast<const uint4*>(a.v + t * a.v_stride + h * D + ch);
    const int slot = live ? a.slots[t] : -1;
    Turn x;
    if (turn && live) load_turn<INTER>(r, t, li, ch, x);
    Pairs8 w;
    if (NORM) w = widen_pairs(*reinterpret_cast<const uint4*>(r.kw + ch));
    const uint4 turned = turn_key<D, INTER, NORM>(r, kw, w, li, ch, x);
    write_rows<D>(a, slot, h, li, group_mask, code_row(turned), code_row(vw));
    return;
  }
  const uint32_t item = (blockIdx.x - kv_before) * kPerBlock + threadIdx.x / L;
  const bool live = item < (uint32_t)r.T * n.splits;
  const int t = live ? (int)n.by_splits(item) : 0;
  const int h0 = live ? (int)(item - t * n.splits) * n.heads_per : r.Hq;
  const int heads = min(n.heads_per, r.Hq - h0);
  const QueryPiece<INTER> piece(r.rot, li);
  const __nv_bfloat16* src = r.q + t * r.q_stride + h0 * D;
  __nv_bfloat16* dst = r.q_out + t * r.q_out_stride + h0 * D;
  uint4 raw[kMostQueries];
#pragma unroll
  for (int i = 0; i < kMostQueries; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (i < heads) raw[i] = piece.load(src + i * D);
  }
  float2 c[2], s[2];
  if (turn && live) {
    const float* row = turn_row_at(r, t, li == 0) + 4 * li;
    const float4 x = *reinterpret_cast<const float4*>(row);
    const float4 y = *reinterpret_cast<const float4*>(row + r.rot / 2);
    c[0] = make_float2(x.x, x.y), c[1] = make_float2(x.z, x.w);
    s[0] = make_float2(y.x, y.y), s[1] = make_float2(y.z, y.w);
  }
  Pairs8 w;
  if (NORM) w = piece.pairs(piece.load(r.qw));
#pragma unroll
  for (int i = 0; i < kMostQueries; ++i) {
    if (i >= n.heads_per) break;
    const uint4 y = turn_query<D, INTER, NORM>(r, raw[i], w, turn, c, s);
    if (i < heads) piece.store(dst + i * D, y);
  }
}

// ------------------------------------------------------------------- accepted rows

// Slot of a request's cached token; -1 if the table or the cache has none.
__device__ __forceinline__ int64_t slot_of(const AcceptArgs& p, const RowsArgs& a, int b,
                                           int64_t tok) {
  const int64_t page = tok >> a.page_shift;
  if (tok < 0 || page >= p.table_width) return -1;
  const int64_t slot = ((int64_t)p.table[(int64_t)b * p.table_width + page] << a.page_shift) +
                       (tok & ((1 << a.page_shift) - 1));
  return slot < a.n_slots ? slot : -1;
}

// A request's table entries whose pages hold no accepted token: none where its lengths make no sense.
__device__ __forceinline__ int2 rejected_pages(const AcceptArgs& p, const RowsArgs& a, int b) {
  const int len = p.path_lens[b], ctx = p.ctx[b], kv = p.kv_lens[b];
  if (len < 0 || len > p.path_width || ctx < 0 || kv < ctx) return make_int2(0, 0);
  auto pages = [&](int64_t tokens) { return (tokens + (1 << a.page_shift) - 1) >> a.page_shift; };
  const int64_t to = min(pages(kv), (int64_t)p.table_width);
  return make_int2((int)min(pages((int64_t)ctx + len), to), (int)to);
}

// Puts them back in front of the free list's cursor, requests in order, and moves the cursor; one block, a
// thread per request.  Page ids that the cache does not have are left out (and recorded).
__device__ __forceinline__ void put_back(const AcceptArgs& p, const RowsArgs& a) {
  __shared__ int sums[kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t n_pages = a.n_slots >> a.page_shift;
  auto there = [&](int b, int i) {
    const int page = p.table[(int64_t)b * p.table_width + i];
    return page >= 0 && page < n_pages;
  };
  int all = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    int n = 0;
    if (b0 + tid < p.B) {
      const int2 r = rejected_pages(p, a, b0 + tid);
      for (int i = r.x; i < r.y; ++i) n += there(b0 + tid, i);
      if (n < r.y - r.x) record_error(a.err, kDevErrState);
    }
    n = __reduce_add_sync(~0u, n);
    if (lane == 0) sums[warp] = n;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) all += sums[w];
    __syncthreads();
  }
  const int cursor = *p.cursor;
  if (cursor < all || cursor > p.n_free) {  // not a cursor of this list
    if (tid == 0) record_error(a.err, kDevErrState);
    return;
  }
  int32_t* dst = p.free_pages + (cursor - all);
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    int2 r = make_int2(0, 0);
    int n = 0;
    if (b0 + tid < p.B) {
      r = rejected_pages(p, a, b0 + tid);
      for (int i = r.x; i < r.y; ++i) n += there(b0 + tid, i);
    }
    int end = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(~0u, end, o);
      if (lane >= o) end += x;
    }
    if (lane == 31) sums[warp] = end;
    __syncthreads();
    int at = end - n, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += sums[w];
      total += sums[w];
    }
    for (int i = r.x; i < r.y; ++i)
      if (there(b0 + tid, i)) dst[at++] = p.table[(int64_t)(b0 + tid) * p.table_width + i];
    dst += total;
    __syncthreads();  // (the sums are free)
  }
  if (tid == 0) *p.cursor = cursor - all;
}

// A block per request and head, L = D / 8 lanes per accepted row, kThreads / L rows at a time: all
// are read before any is written.  Entry i of an ascending path is i at least, so no row is written
// before a later round reads it.  Bound by latency: lengths, path and table, rows, one after
// another (with its reading back, 64 requests of up to 12 accepted tokens, 2 heads of 256 channels:
// 4.4 us, two launches).
template <int D>
__global__ void __launch_bounds__(kThreads) attn_accept_kernel(AcceptArgs p, RowsArgs a) {
  using R = Record<D>;
  constexpr int L = D / 8, NG = D / kGroup;
  constexpr int kAtOnce = kThreads / L;
  const int li = threadIdx.x % L, row = threadIdx.x / L;
  const int b = blockIdx.x, h = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  if (b == p.B) {  // (there where pages are put back)
    if (h == 0) put_back(p, a);
    return;
  }
  int len = p.path_lens[b];
  const int ctx = p.ctx[b];
  if (len < 0 || len > p.path_width || ctx < 0) {
    if (threadIdx.x == 0) record_error(a.err, kDevErrState);
    len = 0;
  }
  const int32_t* path = p.paths + (int64_t)b * p.path_width;
  for (int i0 = 0; i0 < len; i0 += kAtOnce) {
    const int i = i0 + row;
    int64_t src = -1, dst = -1;
    if (i < len) {
      const int at = path[i], before = i ? path[i - 1] : -1;
      if (at > before) {
        src = slot_of(p, a, b, (int64_t)ctx + at);
        dst = slot_of(p, a, b, (int64_t)ctx + i);
      }
      if ((src < 0 || dst < 0) && li == 0) record_error(a.err, kDevErrState);
    }
    const bool moves = src >= 0 && dst >= 0 && src != dst;
    uint32_t kw, vw, kp, vp;
    if (moves) {
      const uint8_t* rec = a.cache + record_of(a, (int)src, h) * R::kBytes;
      const int r = (int)src & 15, word = ((li & 7) ^ row_swz((int)src)) * NG + (li >> 3);
      kw = reinterpret_cast<const uint32_t*>(rec + r * R::kRow)[word];
      vw = reinterpret_cast<const uint32_t*>(rec + R::kV + r * R::kRow)[word];
      kp = reinterpret_cast<const uint32_t*>(rec + R::kKp + r * R::kPar)[li >> 3];
      vp = reinterpret_cast<const uint32_t*>(rec + R::kVp + r * R::kPar)[li >> 3];
    }
    __syncthreads();
    if (moves) {
      uint8_t* rec = a.cache + record_of(a, (int)dst, h) * R::kBytes;
      const int r = (int)dst & 15, word = ((li & 7) ^ row_swz((int)dst)) * NG + (li >> 3);
      reinterpret_cast<uint32_t*>(rec + r * R::kRow)[word] = kw;
      reinterpret_cast<uint32_t*>(rec + R::kV + r * R::kRow)[word] = vw;
      if ((li & 7) == 0) {
        reinterpret_cast<uint32_t*>(rec + R::kKp + r * R::kPar)[li >> 3] = kp;
        reinterpret_cast<uint32_t*>(rec + R::kVp + r * R::kPar)[li >> 3] = vp;
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------- cached rows, read back

__device__ __forceinline__ uint4 decode_word(uint32_t w, uint32_t params) {
  const float step = bf16_lo(params), lo = bf16_hi(params);
  Row8 r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // the code as a float: 2^23 + code, less 2^23 (both exact)
    const float code = __fsub_rn(__uint_as_float(((w >> (4 * e)) & 15u) | 0x4b000000u), 8388608.f);
    r.x[e] = fmaf(step, code, lo);  // the product is exact: 8 bits by 4
  }
  return narrow(r);
}

// A group of lanes per (token, head).  A lane reads 4 bytes of codes and its group's parameter word,
// and writes 16, for keys and for values.  Bound by latency for prompts: the slot, then the record,
// then the stores, one row a group (4.2 TB/s, see above).
template <int D>
__global__ void __launch_bounds__(kThreads) attn_read_kernel(RowsArgs a) {
  using R = Record<D>;
  constexpr int L = D / 8, NG = D / kGroup;
  constexpr int kPerBlock = kThreads / L;
  const int li = threadIdx.x % L;
  pdl_wait();
  pdl_trigger();
  const uint32_t row = blockIdx.x * kPerBlock + threadIdx.x / L;
  if (row < (uint32_t)a.T * a.Hkv) {
    const int t = (int)(row / (uint32_t)a.Hkv), h = (int)(row % (uint32_t)a.Hkv);
    const int slot = a.slots[t];
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (slot >= 0 && slot < a.n_slots) {
      const uint8_t* rec = a.cache + record_of(a, slot, h) * R::kBytes;
      const int row = slot & 15, word = ((li & 7) ^ row_swz(slot)) * NG + (li >> 3);
      k = decode_word(reinterpret_cast<const uint32_t*>(rec + row * R::kRow)[word],
                      reinterpret_cast<const uint32_t*>(rec + R::kKp + row * R::kPar)[li >> 3]);
      v = decode_word(
          reinterpret_cast<const uint32_t*>(rec + R::kV + row * R::kRow)[word],
          reinterpret_cast<const uint32_t*>(rec + R::kVp + row * R::kPar)[li >> 3]);
    } else if (slot >= a.n_slots && li == 0) {
      record_error(a.err, kDevErrState);
    }
    *reinterpret_cast<uint4*>(a.ko + t * a.k_stride + h * D + 8 * li) = k;
    *reinterpret_cast<uint4*>(a.vo + t * a.v_stride + h * D + 8 * li) = v;
  }
}

int row_grid(const RowsArgs& a, int D) {
  const int per_block = kThreads / (D / 8);
  return (int)(((int64_t)a.T * a.Hkv + per_block - 1) / per_block);
}

// Items of neighbouring heads of a token: as few heads in each as still leave one item for every
// group of lanes that fits the GPU, up to `most`.
int heads_per_item(int T, int heads, int most, int D, int sms) {
  const int64_t groups = (int64_t)sms * (2048 / kThreads) * (kThreads / (D / 8));
  int64_t per = (T * (int64_t)heads + groups - 1) / groups;
  if (per > most) per = most;
  const int splits = (heads + (int)per - 1) / (int)per;
  return (heads + splits - 1) / splits;  // evenly
}

template <int D, bool INTER>
cudaError_t launch_rope_append(const RopeArgs& r, const RowsArgs& a, int sms, cudaStream_t s) {
  const int per_block = kThreads / (D / 8);
  const int heads_per = heads_per_item(r.T, r.Hq, kMostQueries, D, sms);
  const uint32_t splits = (r.Hq + heads_per - 1) / heads_per;
  const int64_t kv_blocks = row_grid(a, D);
  const int64_t blocks = kv_blocks + ((int64_t)r.T * splits + per_block - 1) / per_block;
  // rounded up by less than 1, so over all blocks (below 2^32) the count comes to kv_blocks exactly
  const uint32_t rate = (uint32_t)(((kv_blocks << 32) + blocks - 1) / blocks);
  const Shares n{heads_per, splits, rate, Divide(a.Hkv), Divide(splits)};
  const dim3 grid((unsigned)blocks);
  return r.qw ? launch_pdl(attn_rope_append_kernel<D, INTER, true>, grid, dim3(kThreads), 0, s, r, a, n)
              : launch_pdl(attn_rope_append_kernel<D, INTER, false>, grid, dim3(kThreads), 0, s, r, a,
                           n);
}

}  // namespace

cudaError_t launch_attn_qk_norm_rope(const RopeArgs& a, int D, bool inter, int sms,
                                     cudaStream_t s) {
  const int per_block = kThreads / (D / 8);
  const int heads = a.Hq + a.Hkv;
  const int heads_per = heads_per_item(a.T, heads, kMostHeads, D, sms);
  const int splits = (heads + heads_per - 1) / heads_per;
  const dim3 grid((unsigned)(((int64_t)a.T * splits + per_block - 1) / per_block)), block(kThreads);
  if (D == 64)
    return inter ? launch_pdl(attn_rope_kernel<64, true>, grid, block, 0, s, a, heads_per)
                 : launch_pdl(attn_rope_kernel<64, false>, grid, block, 0, s, a, heads_per);
  if (D == 128)
    return inter ? launch_pdl(attn_rope_kernel<128, true>, grid, block, 0, s, a, heads_per)
                 : launch_pdl(attn_rope_kernel<128, false>, grid, block, 0, s, a, heads_per);
  return inter ? launch_pdl(attn_rope_kernel<256, true>, grid, block, 0, s, a, heads_per)
               : launch_pdl(attn_rope_kernel<256, false>, grid, block, 0, s, a, heads_per);
}

cudaError_t launch_attn_rope_append(const RopeArgs& r, const RowsArgs& a, int D, bool inter, int sms,
                                    cudaStream_t s) {
  if (D == 64)
    return inter ? launch_rope_append<64, true>(r, a, sms, s)
                 : launch_rope_append<64, false>(r, a, sms, s);
  if (D == 128)
    return inter ? launch_rope_append<128, true>(r, a, sms, s)
                 : launch_rope_append<128, false>(r, a, sms, s);
  return inter ? launch_rope_append<256, true>(r, a, sms, s)
               : launch_rope_append<256, false>(r, a, sms, s);
}

cudaError_t launch_attn_accept(const AcceptArgs& p, const RowsArgs& a, int D, cudaStream_t s) {
  const dim3 grid(p.B + (p.kv_lens != nullptr), a.Hkv), block(kThreads);
  if (D == 64) return launch_pdl(attn_accept_kernel<64>, grid, block, 0, s, p, a);
  if (D == 128) return launch_pdl(attn_accept_kernel<128>, grid, block, 0, s, p, a);
  return launch_pdl(attn_accept_kernel<256>, grid, block, 0, s, p, a);
}

cudaError_t launch_attn_append(const RowsArgs& a, int D, cudaStream_t s) {
  const dim3 grid(row_grid(a, D)), block(kThreads);
  if (D == 64) return launch_pdl(attn_append_kernel<64>, grid, block, 0, s, a);
  if (D == 128) return launch_pdl(attn_append_kernel<128>, grid, block, 0, s, a);
  return launch_pdl(attn_append_kernel<256>, grid, block, 0, s, a);
}

cudaError_t launch_attn_read(const RowsArgs& a, int D, cudaStream_t s) {
  const dim3 grid(row_grid(a, D)), block(kThreads);
  if (D == 64) return launch_pdl(attn_read_kernel<64>, grid, block, 0, s, a);
  if (D == 128) return launch_pdl(attn_read_kernel<128>, grid, block, 0, s, a);
  return launch_pdl(attn_read_kernel<256>, grid, block, 0, s, a);
}

}  // namespace moe
