// Attention through a window with first tokens, or of a drafted tree, over the paged 4-bit cache
// (include/attn.h).  A warp per new token and query head: the lanes hold the head's channels, go over
// the visible cached tokens one by one and keep a running softmax in fp32.
#include <cfloat>

#include "attn.cuh"
#include "attn_join.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <int D>
__device__ __forceinline__ void cached_channels(const uint8_t* rec, int row_at, int par_at, int slot,
                                                int lane, float (&x)[D / 32]) {
  using R = Record<D>;
  constexpr int N = D / 32, NG = D / kGroup;
  const int c0 = N * lane, g = c0 / kGroup, j = c0 % kGroup / 8, row = slot & 15;
  const uint32_t w = reinterpret_cast<const uint32_t*>(rec + row_at + row * R::kRow)
      [(j ^ row_swz(slot)) * NG + g];
  const uint32_t p = reinterpret_cast<const uint32_t*>(rec + par_at + row * R::kPar)[g];
#pragma unroll
  for (int i = 0; i < N; ++i)
    x[i] = fmaf(bf16_lo(p), (float)(w >> (4 * (c0 % 8 + i)) & 15u), bf16_hi(p));
}

template <int D>
__global__ void __launch_bounds__(kThreads) attn_masked_kernel(FwdArgs a) {
  using R = Record<D>;
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (unit >= (int64_t)a.T * a.d.Hq) return;
  const int t = (int)(unit / a.d.Hq), hq = (int)(unit % a.d.Hq);
  if (t >= a.q_off[a.B] || t < 0) return;
  int b = 0;
  while (b + 1 < a.B && a.q_off[b + 1] <= t) ++b;
  if (hq == 0 && req_out_of_range(a, b)) record_error(a.err, kDevErrState);
  const Req r = load_req(a, b);
  const int i = t - r.q0, h = hq / a.d.G;
  if (i < 0 || i >= r.qn) return;
  const int c = r.kv - r.qn;
  const uint32_t* mask = a.masks ? a.masks + (int64_t)t * a.mask_words : nullptr;
  int pos = c + i;
  if (mask) {
    pos = c - 1;
    for (int k = 0; k < r.qn; ++k) pos += mask[k >> 5] >> (k & 31) & 1;
  }
  const int end = mask ? r.kv : max(pos + 1, 0);
  const int lo = a.window ? pos - a.window + 1 : 0;
  float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    q[e] = __bfloat162float(a.q[(int64_t)t * a.q_stride + hq * D + N * lane + e]);
    o[e] = 0.f;
  }
  for (int k = 0; k < end; ++k) {
    if (k >= a.sinks && k < lo) {
      k = lo - 1;
      continue;
    }
    if (mask && k >= c && !(mask[(k - c) >> 5] >> ((k - c) & 31) & 1)) continue;
    const uint8_t* rec =
        a.cache + (uint64_t)cache_record(a, b, h, k >> 4) * R::kBytes;
    float x[N], s = 0.f;
    cached_channels<D>(rec, 0, R::kKp, k, lane, x);
#pragma unroll
    for (int e = 0; e < N; ++e) s = fmaf(q[e], x[e], s);
#pragma unroll
    for (int o2 = 16; o2; o2 >>= 1) s += __shfl_xor_sync(~0u, s, o2);
    s *= a.d.scale_log2;
    const float top = fmaxf(m, s);
    const float f = top == -INFINITY ? 1.f : exp2f(m - top), p = s != s ? s : exp2f(s - top);
    m = top;
    l = l * f + p;
    cached_channels<D>(rec, R::kV, R::kVp, k, lane, x);
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = fmaf(p, x[e], o[e] * f);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < N; ++e)
    a.out[(int64_t)t * a.out_stride + hq * D + N * lane + e] = __float2bfloat16_rn(o[e] * inv);
}

}  // namespace

cudaError_t launch_attn_masked(const FwdArgs& a, int max_kv, int sms, cudaStream_t s) {
  const dim3 grid((unsigned)(((int64_t)a.T * a.d.Hq + kThreads / 32 - 1) / (kThreads / 32)));
  if (a.d.D == 64) return launch_pdl(attn_masked_kernel<64>, grid, dim3(kThreads), 0, s, a);
  if (a.d.D == 128) return launch_pdl(attn_masked_kernel<128>, grid, dim3(kThreads), 0, s, a);
  return launch_pdl(attn_masked_kernel<256>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace moe
