// The row kernels of the attention step (include/attn.h): norm and rotation of query and key
// heads, quantisation of keys and values into the paged 4-bit cache, and the way back.  Each is
// one pass over its rows, bound by launch latency for single tokens and for prompts as stated at each
// (by loads that wait for one another, append by instruction issue): a lane holds 8 channels (one
// 16-byte load), the D / 8 lanes of a row reduce by shuffles.
#include "attn.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMostHeads = 8;  // of a group of lanes, in the norm and rotation

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

// Codes of the lane's 8 channels; the 8 lanes of a group share lo and step.  Every code equals the
// one that the definition's fp32 division and rounding give.
__device__ __forceinline__ Coded code_row(uint4 w) {
  uint32_t lo2 = min_nan2(min_nan2(w.x, w.y), min_nan2(w.z, w.w));
  uint32_t hi2 = max_nan2(max_nan2(w.x, w.y), max_nan2(w.z, w.w));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo2 = min_nan2(lo2, __shfl_xor_sync(~0u, lo2, o));
    hi2 = max_nan2(hi2, __shfl_xor_sync(~0u, hi2, o));
  }
  const float lo = bf16_lo(min_nan2(lo2, lo2 >> 16)), hi = bf16_lo(max_nan2(hi2, hi2 >> 16));
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
  const float step = __bfloat162float(sb);
  const Row8 r = widen(w);
  Coded c;
  c.finite = fabsf(lo) < kLargest && fabsf(hi) < kLargest;  // false for NaN
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = 0.f;
  if (step > 0.f) {
    // The product with the reciprocal is within 2^-20 of the rounded quotient, so it rounds to the
    // same code (at most 15) unless it lies near a half: then, and for steps whose reciprocal is
    // no normal number, the quotient itself decides.  2^23 is added and taken off to round.
    const float inv = __frcp_rn(step);
    bool close = step < 1e-35f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = __fmul_rn(__fsub_rn(r.x[e], lo), inv);
      q[e] = __fsub_rn(__fadd_rn(y, 8388608.f), 8388608.f);
      close |= fabsf(__fsub_rn(y, q[e])) > 0.49998f;
    }
    if (close) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        q[e] = fminf(rintf(__fdiv_rn(__fsub_rn(r.x[e], lo), step)), 15.f);
    }
  }
  // four codes as the low 16 bits of 2^23 + c0 + 16 c1 + 256 c2 + 4096 c3
  uint32_t half[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float a = fmaf(q[4 * i + 1], 16.f, q[4 * i]);
    const float b = fmaf(q[4 * i + 3], 16.f, q[4 * i + 2]);
    half[i] = __float_as_uint(__fadd_rn(fmaf(b, 256.f, a), 8388608.f));
  }
  c.word = __byte_perm(half[0], half[1], 0x5410);
  const __nv_bfloat16 lb = __float2bfloat16_rn(lo);
  c.params = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(lb) << 16);
  return c;
}

// A group of L = D / 8 lanes per (token, head): key row and value row together, since a
// non-finite channel of either marks both.
//
// Bound by instruction issue for prompts (444 warp instructions a row and head, 80% of the slots): the
// fp32 quotient of the definition would be 16 divisions a lane, so the reciprocal decides where it
// provably rounds to the same code.  Measured: 32768 tokens, 2 heads of 256 channels, 34 us (2.5 TB/s)
// with cold caches, their reading 20 us (4.2 TB/s), both in turn 47 us; 48 tokens 3.9 us for both.
template <int D>
__global__ void __launch_bounds__(kThreads) attn_append_kernel(RowsArgs a) {
  using R = Record<D>;
  constexpr int L = D / 8, NG = D / kGroup;
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
    Coded k = code_row(kw), v = code_row(vw);
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
}

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

}  // namespace

cudaError_t launch_attn_qk_norm_rope(const RopeArgs& a, int D, bool inter, int sms,
                                     cudaStream_t s) {
  const int per_block = kThreads / (D / 8);
  const int heads = a.Hq + a.Hkv;
  // as few heads per group as still leave one item for every group that fits the GPU, up to eight
  const int64_t groups = (int64_t)sms * (2048 / kThreads) * per_block;
  int64_t heads_per64 = (a.T * (int64_t)heads + groups - 1) / groups;
  if (heads_per64 > kMostHeads) heads_per64 = kMostHeads;
  int splits = (heads + (int)heads_per64 - 1) / (int)heads_per64;
  const int heads_per = (heads + splits - 1) / splits;  // evenly
  splits = (heads + heads_per - 1) / heads_per;
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
