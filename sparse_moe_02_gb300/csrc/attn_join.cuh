// What the two attention kernels share: how the work of a step is cut over the blocks, partial
// results of contexts that several blocks share, and the launch that joins them.
#pragma once

#include "attn.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// a / b of nonnegative numbers, in 32 bits where they fit (a 64-bit division is a long routine)
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Inclusive prefix sum over the warp.
__device__ __forceinline__ int64_t warp_scan(int64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

struct Cut {
  int64_t share;  // work of a block, one more in the first `rest` blocks
  int rest;
  int blocks;
  __device__ __forceinline__ int64_t bound(int i) const { return share * i + min(i, rest); }
  // the block that does unit x
  __device__ __forceinline__ int block_of(int64_t x) const {
    const int64_t wide = (share + 1) * rest;
    return x < wide ? (int)divide(x, share + 1) : rest + (int)divide(x - wide, share);
  }
};

__device__ __forceinline__ Cut make_cut(int64_t total, int64_t least, int blocks) {
  const int64_t most = divide(total + least - 1, least);
  Cut c;
  c.blocks = (int)(most < (int64_t)blocks ? most : (int64_t)blocks);
  c.share = c.blocks ? divide(total, c.blocks) : 0;
  c.rest = (int)(total - c.share * c.blocks);
  return c;
}

// Fills first[b], b = 0 .. B, with the work before request b (work(b) of each) and returns the cut of
// all work into shares of `least` at least.  Whole block; `sums` holds a value per warp.
template <int kThreads, typename F>
__device__ __forceinline__ Cut cut_work(const FwdArgs& a, int64_t* first, int64_t* sums,
                                        int64_t least, F work) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t total = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int64_t n = 0;
    if (b0 + (int)(threadIdx.x & ~31u) < a.B) {  // warps behind the last request have nothing
      if (b < a.B) {
        const Req r = load_req(a, b);
        if (blockIdx.x == 0 && req_out_of_range(a, b)) record_error(a.err, kDevErrState);
        n = work(r);
      }
    }
    const int64_t end = warp_scan(n);
    if (lane == 31) sums[warp] = end;
    __syncthreads();
    int64_t before = total;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
      const int64_t x = sums[w];
      if (w < warp) before += x;
      total += x;
    }
    if (b < a.B) first[b] = before + end - n;
    if (b == a.B - 1) first[a.B] = total;
    __syncthreads();
  }
  return make_cut(total, least, gridDim.x);
}

// The request whose work holds unit w: first[b] <= w < first[b + 1].
__device__ __forceinline__ int find_request(const int64_t* first, int B, int64_t w) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= w) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The part of a context that a block works on.
struct Part {
  int b, h, rt;
  int t0, t1, tiles;  // its tiles, and the context's
  Req r;
  int64_t start;  // work before the context's first tile
  int unit;       // work of a tile
  int64_t next;   // the block's work after this part
  bool some;
};

// Record of `tile` of request b's context, head h; a page id out of range reads page 0 and is
// recorded.  (32 bits: 2^32 records are more than 5 TB.)
__device__ __forceinline__ uint32_t cache_record(const FwdArgs& a, int b, int h, int tile) {
  const int shift = a.d.page_shift - 4;  // tiles per page
  int id = a.table[(int64_t)b * a.table_width + (tile >> shift)];
  if (id < 0 || id >= a.d.n_pages) {
    record_error(a.err, kDevErrState);
    id = 0;
  }
  return (((uint32_t)id * a.d.Hkv + h) << shift) + (tile & ((1 << shift) - 1));
}

// Square root of a part's weight.  References hold the sizes of values as well as scores, so they may
// differ by more than fp32's exponents while the sums of weights, scaled by them, are alike: sums take
// the root twice, outputs its square, which may vanish as they do.
__device__ __forceinline__ float part_root(float m_part, float l_part, float m) {
  // a part that saw nothing has m = -inf and l = 0; one of NaN scores m = -inf and l = NaN
  return m_part == -INFINITY ? (l_part == 0.f ? 0.f : 1.f) : exp2_fast(0.5f * (m_part - m));
}

// The sum that a row's outputs are divided by.  References are rounded to fp32: from 2^23 on (in units
// of log 2) weights may leave f16 upwards (inf, and the row reads NaN), from 2^29 on downwards, which
// would read as zeros; such rows read NaN as well.
__device__ __forceinline__ float row_sum(float m, float l) {
  return m != -INFINITY && fabsf(m) >= 268435456.f ? NAN : l;  // 2^28
}

// Outputs are joined in the order in which the lanes hold them: float4 i of a column is channels
// out_channel(i) .. + 3.
__device__ __forceinline__ int out_channel(int i) {
  return (i >> 4) * 64 + (i & 7) * 8 + ((i >> 3) & 1) * 4;
}

__device__ __forceinline__ void store_out4(const FwdArgs& a, const Part& p, int row, int D, int i,
                                           float4 o, float l) {
  if (row >= p.r.qn * a.d.G) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* dst = a.out + (int64_t)(p.r.q0 + row / a.d.G) * a.out_stride +
                       (int64_t)(p.h * a.d.G + row % a.d.G) * D + out_channel(i);
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                              *reinterpret_cast<const uint32_t*>(&hi));
}

__device__ __forceinline__ void fma4(float4& o, const float4& v, float f) {
  o.x = fmaf(v.x, f, o.x);
  o.y = fmaf(v.y, f, o.y);
  o.z = fmaf(v.z, f, o.z);
  o.w = fmaf(v.w, f, o.w);
}

// Slot of part i of a context whose first part is block b0's: that block's second slot, then the
// first slots of the blocks behind it.
__device__ __forceinline__ int part_slot(int b0, int i) { return 2 * (b0 + i) + (i == 0); }

// Joins the parts of the contexts that several blocks share, in block order.  Contexts of few
// parts take one warp per column, as do all with many columns (row tiles); few columns of many
// parts take a block per column and 64 channels, with 16 groups of lanes over the parts, so that
// one long context (76 parts of 8 KB) is spread over 32 blocks and its parts are read in one round
// trip.  Bound by latency for tokens (3 us, most of it the launch; one warp per column took 11 us
// over a context of 1024 tokens), by the caches for row tiles (two parts of 128 KB a block, 40 MB
// in all; read eight at a time as for tokens, mostly the last one again, a prompt of 4096 took 156 us
// instead of 148).
constexpr int kJoinThreads = 256;
constexpr int kFewParts = 8;
constexpr int kMaxBlocks = 256;  // of the attention launch

template <int N>
__device__ __forceinline__ void add_scaled(float (&o)[N], const float* src, float f) {
  if constexpr (N == 2) {
    const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
    o[0] = fmaf(v.x, f, o[0]);
    o[1] = fmaf(v.y, f, o[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src + i));
      o[i] = fmaf(v.x, f, o[i]);
      o[i + 1] = fmaf(v.y, f, o[i + 1]);
      o[i + 2] = fmaf(v.z, f, o[i + 2]);
      o[i + 3] = fmaf(v.w, f, o[i + 3]);
    }
  }
}

template <int D, int kCols>
__global__ void __launch_bounds__(kJoinThreads, kCols > 16 ? 4 : 2)
    attn_join_kernel(FwdArgs a, int blocks) {
  constexpr int kWarpsJ = kJoinThreads / 32;
  __shared__ short few[kMaxBlocks], many[kMaxBlocks];
  __shared__ int2 counts[kWarpsJ];
  __shared__ float weight[kMaxBlocks];
  __shared__ float2 red[kWarpsJ];
  __shared__ float acc[16][64];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  // the lists of shared contexts, in the same order in every block
  const int n_mine = tid < blocks ? a.desc[2 * tid].x : 0;
  const bool is_few = n_mine <= kFewParts || kCols > 16;
  const unsigned f_mask = __ballot_sync(~0u, n_mine > 0 && is_few);
  const unsigned m_mask = __ballot_sync(~0u, n_mine > 0 && !is_few);
  if (lane == 0) counts[warp] = make_int2(__popc(f_mask), __popc(m_mask));
  __syncthreads();
  int nf = 0, nm = 0, f0 = 0, m0 = 0;
#pragma unroll
  for (int w = 0; w < kWarpsJ; ++w) {
    if (w == warp) f0 = nf, m0 = nm;
    nf += counts[w].x;
    nm += counts[w].y;
  }
  const unsigned below = (1u << lane) - 1;
  if (f_mask >> lane & 1) few[f0 + __popc(f_mask & below)] = (short)tid;
  if (m_mask >> lane & 1) many[m0 + __popc(m_mask & below)] = (short)tid;
  __syncthreads();

  Part p;
  if constexpr (kCols <= 16) {
    for (int u = blockIdx.x; u < nm * kCols * (D / 64); u += gridDim.x) {
      const int piece = u % (D / 64), col = u / (D / 64) % kCols;
      const int b0 = many[u / (D / 64) / kCols];
      const int4 d = a.desc[2 * b0];
      p.r.qn = a.desc[2 * b0 + 1].x;
      p.h = d.y;
      p.rt = d.z;
      p.r.q0 = d.w;
      const int n = d.x;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (tid < n) ml = __ldcg(a.part_ml + part_slot(b0, tid) * kCols + col);
      float m = ml.x;
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
      if (lane == 0) red[warp].x = m;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kWarpsJ; ++k) m = fmaxf(m, red[k].x);
      const float f = part_root(ml.x, ml.y, m);
      weight[tid] = f * f;
      float l = ml.y * f * f;
#pragma unroll
      for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
      if (lane == 0) red[warp].y = l;
      __syncthreads();
      const int ln = tid & 15, grp = tid >> 4;
      float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 5
      for (int i = grp; i < n; i += 16)
        add_scaled(o, a.part_o + ((int64_t)part_slot(b0, i) * kCols + col) * D + 64 * piece + 4 * ln,
                   weight[i]);
      *reinterpret_cast<float4*>(&acc[grp][4 * ln]) = make_float4(o[0], o[1], o[2], o[3]);
      __syncthreads();
      if (tid < 16) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kWarpsJ; ++k) sum += red[k].y;
#pragma unroll
        for (int k = 0; k < 16; ++k) fma4(x, *reinterpret_cast<const float4*>(&acc[k][4 * tid]), 1.f);
        store_out4(a, p, p.rt * kCols + col, D, 16 * piece + tid, x, row_sum(m, sum));
      }
      __syncthreads();
    }
  }

  constexpr int kCh = D / 32;  // channels of a lane
  // parts read at once: row tiles mostly have two, and their many columns keep enough in flight
  constexpr int kAtOnce = kCols > 16 ? 2 : kFewParts;
  for (int u = blockIdx.x * kWarpsJ + warp; u < nf * kCols; u += gridDim.x * kWarpsJ) {
    const int col = u % kCols, b0 = few[u / kCols];
    const int4 d = a.desc[2 * b0];
    p.r.qn = a.desc[2 * b0 + 1].x;
    p.h = d.y;
    p.rt = d.z;
    p.r.q0 = d.w;
    const int row = p.rt * kCols + col;
    if (row >= p.r.qn * a.d.G) continue;
    float m = -INFINITY;
    for (int i = lane; i < d.x; i += 32)
      m = fmaxf(m, __ldcg(a.part_ml + part_slot(b0, i) * kCols + col).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    float l = 0.f;
    float o[kCh];
#pragma unroll
    for (int e = 0; e < kCh; ++e) o[e] = 0.f;
    for (int i0 = 0; i0 < d.x; i0 += kAtOnce) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < kAtOnce && i0 + lane < d.x)
        ml = __ldcg(a.part_ml + part_slot(b0, i0 + lane) * kCols + col);
      const float root = part_root(ml.x, ml.y, m), f = root * root;
      l = fmaf(ml.y * root, root, l);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {  // beyond the last: it again, with weight 0
        const float fi = __shfl_sync(~0u, f, i);
        add_scaled(o,
                   a.part_o + ((int64_t)part_slot(b0, min(i0 + i, d.x - 1)) * kCols + col) * D +
                       lane * kCh,
                   i0 + i < d.x ? fi : 0.f);
      }
    }
#pragma unroll
    for (int i = kAtOnce / 2; i; i >>= 1) l += __shfl_xor_sync(~0u, l, i);
    l = row_sum(m, __shfl_sync(~0u, l, 0));
    if constexpr (kCh == 2) {
      // two lanes hold the four channels that are stored at once
      const float x = __shfl_down_sync(~0u, o[0], 1), y = __shfl_down_sync(~0u, o[1], 1);
      if ((lane & 1) == 0)
        store_out4(a, p, row, D, lane / 2, make_float4(o[0], o[1], x, y), l);
    } else {
#pragma unroll
      for (int e = 0; e < kCh; e += 4)
        store_out4(a, p, row, D, (lane * kCh + e) / 4,
                   make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]), l);
    }
  }
}

}  // namespace
}  // namespace moe
