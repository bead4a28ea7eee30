// Attention of many query rows over the paged 4-bit cache (include/attn.h): prompts, chunks of
// prompts, and batches that hold any of them, on the tcgen05 tensor cores.
//
// A block works on 128 query rows of one key/value head (row = new token * G + query head) in steps
// of 64 cached tokens.  Fourteen warps: four hold the softmax (a thread per row), eight turn cached
// rows into f16 MMA operands, one issues the MMAs, one copies cache records.
//   S [128 x 64] = Q K^T      A = Q in tensor memory, B = keys [64][D] in shared memory
//   O [128 x D] += P V        A = P in tensor memory (over S), B = values [D][64] (channels by
//                             tokens, so both operands are K-major)
// S has two buffers, so the scores of step n + 1 are formed while the softmax of step n runs.  Q lies
// in tensor memory because with 64 columns an MMA reads its A operand as often as B: from shared
// memory the reads alone would take longer than the arithmetic.
//
// Arithmetic.  Per record of 16 tokens, keys and values enter as f16(x 2^-(e + 6)), 2^e a bound of
// the record's magnitudes: one fused multiply-add per pair of codes, since a nibble masked in place
// is the exact f16 subnormal code * 2^-24 (or 2^-20) and step * 2^24 2^-(e + 6) fits f16.  f16 keeps
// 11 bits of the larger entries and 2^-18 of the record's largest for the smaller ones, against 8
// bits of a bf16 operand.  Queries are scaled by a power of two per row.  The exponents return in
// fp32 with the scores and, for the values, inside the weights: P = 2^(x + e - m), where the running
// reference m bounds x + e; the softmax sum takes 2^(x - m).  Scores, sums and outputs are fp32.
// The outputs are rescaled (in tensor memory) only when the reference grows by more than 2^6.
//
// Work.  Row tiles of all requests and heads, causally shortened, are cut evenly over the blocks as
// in the few-row kernel; shared row tiles are joined by its second launch.
#include "attn.cuh"
#include "attn_join.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;
constexpr int kStep = 64;            // tokens per step
constexpr int kRecs = kStep / 16;    // cache records per step
constexpr int kSoftWarps = 4, kDeqWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + kDeqWarps + 2);
constexpr int kRaw = 4;              // steps of cache records in flight
constexpr int kOps = 2;              // steps of MMA operands
constexpr float kSlack = 6.f, kLift = 9.f;  // as in the few-row kernel
constexpr int kExps = 8;             // steps of record exponents kept

template <int D>
struct Cfg {
  using R = Record<D>;
  static constexpr int NG = D / kGroup;
  static constexpr int kK = kStep * D * 2;  // bytes of a key (or value) operand
  static constexpr int kRawBytes = kRecs * R::kBytes;
  static constexpr int kOffV = kOps * kK;
  static constexpr int kOffRaw = 2 * kOps * kK;
  static constexpr int kFirst = kOffRaw + kRaw * kRawBytes;
  static constexpr int kSmem = kFirst + 1024;  // the operands start on a 1024-byte boundary
  // tensor memory columns: O, Q, two score buffers
  static constexpr int kColQ = D;
  static constexpr int kColS = D + D / 2;
  static constexpr int kCols = D == 64 ? 256 : 512;
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z,
                                       uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Bulk copy into shared memory with the default cache policy: the row tiles of a head read the
// same records one after another.
__device__ __forceinline__ void copy_record(void* dst, const void* src, uint32_t bytes,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Waits for this thread's tensor memory loads; the registers go through it, so that nothing
// reads them before.
__device__ __forceinline__ void wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31]));
}

// 32 lanes x 8 columns
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

// 32 lanes x 32 columns
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// tcgen05.mma kind::f16 with f16 operands, fp32 accumulation
__device__ __forceinline__ uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

constexpr uint32_t kNib0 = 0x000f000fu, kNib1 = 0x00f000f0u;

// ------------------------------------------------------------------- the work of a block

// Work is counted in (cached token x query head) units, 128 per row tile and token position: row
// tile rt of a request with `base` cached tokens before its new ones costs kPartCost G + base G +
// 128 (rt + 1) units, and its step t starts at unit (kPartCost + 64 t) G of them.
constexpr int kPartCost = 192;   // tokens: a row tile's fixed cost
constexpr int kLeastSteps = 4;   // of a block

struct Cost {
  int64_t fixed, base;  // per row tile, in units
  __device__ __forceinline__ int64_t before(int64_t rt) const {
    return rt * (fixed + base) + 64 * rt * (rt + 1);
  }
};

__device__ __forceinline__ Cost cost_of(const FwdArgs& a, const Req& r) {
  return Cost{(int64_t)kPartCost * a.d.G, (int64_t)max(r.kv - r.qn, 0) * a.d.G};
}

__device__ __forceinline__ int row_tiles(const FwdArgs& a, const Req& r) {
  return (r.qn * a.d.G + kRows - 1) / kRows;
}

// Cached tokens that new token `tok` of the request sees.
__device__ __forceinline__ int seen_by(const Req& r, int tok) {
  return min(max(r.kv - r.qn + tok + 1, 0), r.kv);
}

// Fills first[b], b = 0 .. B: the work before request b.  One warp.
__device__ __forceinline__ Cut cut_rows(const FwdArgs& a, int64_t* first) {
  const int lane = threadIdx.x & 31;
  int64_t total = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    int64_t n = 0;
    if (b < a.B) {
      const Req r = load_req(a, b);
      if (blockIdx.x == 0 && req_out_of_range(a, b)) record_error(a.err, kDevErrState);
      n = a.d.Hkv * cost_of(a, r).before(row_tiles(a, r));
    }
    const int64_t end = warp_scan(n);
    if (b < a.B) first[b] = total + end - n;
    total += __shfl_sync(~0u, end, 31);
  }
  if (lane == 0) first[a.B] = total;
  __syncwarp();
  return make_cut(total, (int64_t)kLeastSteps * kStep * a.d.G, gridDim.x);
}

// The part that holds work w of the block's [w, w1).
__device__ __forceinline__ Part locate(const FwdArgs& a, const int64_t* first, int64_t w,
                                       int64_t w1) {
  Part p;
  p.some = false;
  while (w < w1) {
    p.b = find_request(first, a.B, w);
    p.r = load_req(a, p.b);
    const Cost c = cost_of(a, p.r);
    const int rts = row_tiles(a, p.r);
    const int64_t head = c.before(rts);
    p.h = (int)divide(w - first[p.b], head);
    const int64_t at = first[p.b] + p.h * head;
    // 64 rt^2 + (fixed + base + 64) rt = w - at
    const double q = (double)(c.fixed + c.base + 64);
    int rt = (int)((sqrt(q * q + 256.0 * (double)(w - at)) - q) / 128.0);
    rt = min(max(rt, 0), rts - 1);
    while (rt > 0 && c.before(rt) > w - at) --rt;
    while (rt + 1 < rts && c.before(rt + 1) <= w - at) ++rt;
    p.rt = rt;
    const int last = min((rt + 1) * kRows, p.r.qn * a.d.G) - 1;
    p.tiles = max(1, (seen_by(p.r, last / a.d.G) + kStep - 1) / kStep);
    const int64_t end = at + c.before(rt + 1);
    p.unit = kStep * a.d.G;
    p.start = at + c.before(rt) + c.fixed;
    const int64_t stop = min(end, w1);
    // the steps that start in [w, stop)
    p.t0 = w <= p.start ? 0 : (int)min((int64_t)p.tiles, divide(w - p.start + p.unit - 1, p.unit));
    p.t1 = stop <= p.start
               ? 0
               : (int)min((int64_t)p.tiles, divide(stop - p.start + p.unit - 1, p.unit));
    w = p.next = stop;
    if (p.t1 > p.t0) {
      p.some = true;
      break;
    }
  }
  return p;
}

// ------------------------------------------------------------------- shared state

struct Bars {
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t k_full[kOps], k_empty[kOps], v_full[kOps], v_empty[kOps];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t q_full, o_free;
};

// Exponents of a record: keys were divided by 2^(ek + 6), values by 2^(ev + 6).
struct __align__(16) Exps {
  float up_k;    // 2^ek
  float ev;      // ev
  float down_v;  // 2^-ev
  float pad;
};

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Bound of |bias| + 15 |step| as bits of a nonnegative float, 0 if it is not finite.
__device__ __forceinline__ uint32_t magnitude(uint32_t params) {
  const float v = fmaf(15.f, fabsf(bf16_lo(params)), fabsf(bf16_hi(params)));
  return v < __int_as_float(0x7f800000) ? __float_as_uint(v) : 0u;
}

__device__ __forceinline__ int exponent_of(uint32_t bits) {
  return max((int)(bits >> 23) - 126, -90);  // at most 118: see kLargest
}

// One warp turns 8 cached tokens (half a record) of a step into operands: rows of the key operand
// [64 tokens][D] and columns of the value operand [D][64 tokens], both in the 128-byte swizzle.
template <int D>
struct Dequant {
  using C = Cfg<D>;
  using R = Record<D>;
  static constexpr int NG = C::NG;
  static constexpr int kWords = 2 * NG;  // a lane's words of a key row; nibbles of its value words

  // Parameters of token lane & 7, group (lane >> 3) % NG at offset `off` of the record (0 behind the
  // context), and the exponent of the record's 16 tokens.
  static __device__ __forceinline__ uint32_t params(uint32_t rec, int off, int oct, int tok, int kv,
                                                    int* e) {
    const int lane = threadIdx.x & 31, t = lane & 7, g = (lane >> 3) % NG;
    const uint32_t par = rec + off + (8 * (oct & 1) + t) * R::kPar + 4 * g;
    const int other = (oct & 1) ? -8 : 8;  // the record's other half
    uint32_t w = lds32(par), w2 = lds32(par + other * R::kPar);
    if (tok + t >= kv) w = 0;
    if (tok + t + other >= kv) w2 = 0;
    *e = exponent_of(__reduce_max_sync(~0u, max(magnitude(w), magnitude(w2))));
    return w;
  }

  // tok: the first token's index in the context.  Also leaves the record's exponents in *ex and
  // the value exponent and parameters for values().
  static __device__ __forceinline__ void keys(uint32_t raw, uint32_t dst, int oct, int tok, int kv,
                                              Exps* ex, uint32_t* v_params, int* v_exp) {
    const int lane = threadIdx.x & 31;
    const int t = lane & 7, g = (lane >> 3) % NG, sub = lane / (8 * NG);
    const uint32_t rec = raw + (oct >> 1) * R::kBytes;
    const int row = 8 * (oct & 1) + t;
    int e;
    const uint32_t w = params(rec, R::kKp, oct, tok, kv, &e);
    *v_params = params(rec, R::kVp, oct, tok, kv, v_exp);
    if (lane == 0 && (oct & 1) == 0)
      *ex = Exps{pow2(e), (float)*v_exp, pow2(-*v_exp), 0.f};
    const float down = pow2(-(e + 6));
    const float s = bf16_lo(w) * down, b = bf16_hi(w) * down;
    const uint32_t s24 = pack_f16(s * 16777216.f, s * 16777216.f);
    const uint32_t s20 = pack_f16(s * 1048576.f, s * 1048576.f);
    const uint32_t bb = pack_f16(b, b);
    const uint32_t src = rec + row * R::kRow + 4 * g;
    const uint32_t out = dst + g * (kStep * 128) + (8 * oct + t) * 128;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int j = (sub * kWords + i) ^ (t >> 2);
      const uint32_t c = lds32(src + ((j ^ row_swz(t)) * NG) * 4), c8 = c >> 8;
      sts128(out + ((j ^ t) << 4), fma_f16x2(c & kNib0, s24, bb), fma_f16x2(c & kNib1, s20, bb),
             fma_f16x2(c8 & kNib0, s24, bb), fma_f16x2(c8 & kNib1, s20, bb));
    }
  }

  // Row i * 32 + lane of the value operand is channel 64 g + 8 j + kWords sub + i (lane = (sub, g, j)),
  // so that the rows of a store differ in their last three bits, which the swizzle spreads over
  // the banks.  `table`: 16 bytes for each pair of tokens and group, of this warp.
  static __device__ __forceinline__ void values(uint32_t raw, uint32_t dst, uint4* table, int oct,
                                                uint32_t w, int e) {
    const int lane = threadIdx.x & 31;
    const uint32_t rec = raw + (oct >> 1) * R::kBytes;
    {
      const int t = lane & 7, g = (lane >> 3) % NG;
      const float down = pow2(-(e + 6));
      const uint32_t mate = __shfl_down_sync(~0u, w, 1);
      if ((t & 1) == 0 && lane < 8 * NG) {
        const float s0 = bf16_lo(w) * down, s1 = bf16_lo(mate) * down;
        table[(t >> 1) * NG + g] =
            make_uint4(pack_f16(s0 * 16777216.f, s1 * 16777216.f),
                       pack_f16(s0 * 1048576.f, s1 * 1048576.f),
                       pack_f16(bf16_hi(w) * down, bf16_hi(mate) * down), 0u);
      }
      __syncwarp();
    }
    const int j = lane & 7, g = (lane >> 3) % NG, sub = lane / (8 * NG);
    uint32_t out[kWords][4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int t = 2 * m;
      const uint32_t at = rec + R::kV + (8 * (oct & 1) + t) * R::kRow;
      const uint32_t w0 = lds32(at + ((j ^ row_swz(t)) * NG + g) * 4);
      const uint32_t w1 = lds32(at + R::kRow + ((j ^ row_swz(t + 1)) * NG + g) * 4);
      const uint4 p = table[m * NG + g];
      if constexpr (NG == 4) {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint32_t u = __byte_perm(w0, w1, part ? 0x7632u : 0x5410u), u8 = u >> 8;
          out[4 * part][m] = fma_f16x2(u & kNib0, p.x, p.z);
          out[4 * part + 1][m] = fma_f16x2(u & kNib1, p.y, p.z);
          out[4 * part + 2][m] = fma_f16x2(u8 & kNib0, p.x, p.z);
          out[4 * part + 3][m] = fma_f16x2(u8 & kNib1, p.y, p.z);
        }
      } else if constexpr (NG == 2) {
        const uint32_t u = __byte_perm(w0, w1, sub ? 0x7632u : 0x5410u), u8 = u >> 8;
        out[0][m] = fma_f16x2(u & kNib0, p.x, p.z);
        out[1][m] = fma_f16x2(u & kNib1, p.y, p.z);
        out[2][m] = fma_f16x2(u8 & kNib0, p.x, p.z);
        out[3][m] = fma_f16x2(u8 & kNib1, p.y, p.z);
      } else {
        const uint32_t u = __byte_perm(w0, w1, sub & 2 ? 0x7632u : 0x5410u) >> (8 * (sub & 1));
        out[0][m] = fma_f16x2(u & kNib0, p.x, p.z);
        out[1][m] = fma_f16x2(u & kNib1, p.y, p.z);
      }
    }
    __syncwarp();  // the table is free for the next step
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      sts128(dst + (32 * i + lane) * 128 + ((oct ^ j) << 4), out[i][0], out[i][1], out[i][2],
             out[i][3]);
  }
};

// Column of O that holds nibble k of word j of group g (see Dequant::values).
template <int NG>
__device__ __forceinline__ int out_column(int g, int k) {
  constexpr int kWords = 2 * NG;
  return 32 * (k % kWords) + (k / kWords) * 8 * NG + 8 * g;  // + j
}

// ------------------------------------------------------------------- the kernel

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(FwdArgs a) {
  using C = Cfg<D>;
  constexpr int NG = C::NG;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ Exps exps[kExps][kRecs];
  __shared__ uint4 tables[kDeqWarps][4 * NG];
  __shared__ uint32_t tmem_base;
  __shared__ Cut cut_s;
  uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  int64_t* first = reinterpret_cast<int64_t*>(smem + C::kFirst);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kRaw; ++i) mbar_init(&bars.raw_full[i], 1), mbar_init(&bars.raw_empty[i], kDeqWarps);
    for (int i = 0; i < kOps; ++i) {
      mbar_init(&bars.k_full[i], kDeqWarps);
      mbar_init(&bars.v_full[i], kDeqWarps);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 32 * kSoftWarps);
      mbar_init(&bars.pv_done[i], 1);
    }
    mbar_init(&bars.q_full, 32 * kSoftWarps);
    mbar_init(&bars.o_free, 32 * kSoftWarps);
    fence_mbar_init();
  }
  constexpr int kMmaWarp = kSoftWarps + kDeqWarps, kLoadWarp = kMmaWarp + 1;
  if (warp == kMmaWarp) tmem_alloc(&tmem_base, C::kCols);
  pdl_wait();
  pdl_trigger();
  if (warp == kLoadWarp) {
    const Cut cut = cut_rows(a, first);
    if (lane == 0) {
      cut_s = cut;
      a.desc[2 * blockIdx.x].x = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const Cut cut = cut_s;
  int64_t w0 = 0, w1 = 0;
  if ((int)blockIdx.x < cut.blocks) w0 = cut.bound(blockIdx.x), w1 = cut.bound(blockIdx.x + 1);
  const uint32_t ops = smem_u32(smem);
  bool ok = true;
  int n = 0;  // steps so far

  if (warp == kLoadWarp) {
    for (Part p = locate(a, first, w0, w1); p.some && ok; p = locate(a, first, p.next, w1)) {
      const int recs = (p.r.kv + 15) / 16;
      uint32_t record = 0;
      for (int t = p.t0; t < p.t1 && ok; ++t, ++n) {
        const int slot = (t - p.t0) & 7;
        if (slot == 0) {  // the records of eight steps, one a lane
          const int rec = t * kRecs + lane;
          if (rec < recs) record = cache_record(a, p.b, p.h, rec);
        }
        const int st = n % kRaw;
        ok = mbar_wait(&bars.raw_empty[st], ((n / kRaw) & 1) ^ 1, a.err);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        const int have = min(max(recs - t * kRecs, 0), kRecs);
        const uint32_t rec = __shfl_sync(~0u, record, slot * kRecs + (lane & 3));
        if (lane == 0) mbar_arrive_expect_tx(&bars.raw_full[st], have * C::R::kBytes);
        __syncwarp();
        if (lane < have)
          copy_record(smem + C::kOffRaw + st * C::kRawBytes + lane * C::R::kBytes,
                      a.cache + (uint64_t)rec * C::R::kBytes, C::R::kBytes, &bars.raw_full[st]);
      }
    }
    // nothing may be in flight when the block ends
    for (int k = max(0, n - kRaw); k < n; ++k) mbar_wait(&bars.raw_full[k % kRaw], (k / kRaw) & 1, a.err);
  } else if (warp >= kSoftWarps && warp < kMmaWarp) {
    const int oct = warp - kSoftWarps;
    for (Part p = locate(a, first, w0, w1); p.some && ok; p = locate(a, first, p.next, w1)) {
      for (int t = p.t0; t < p.t1 && ok; ++t, ++n) {
        const int st = n % kRaw, op = n % kOps;
        const uint32_t raw = ops + C::kOffRaw + st * C::kRawBytes;
        const int tok = t * kStep + 8 * oct;
        Exps* ex = &exps[n % kExps][oct >> 1];
        const uint32_t par = ((n / kOps) & 1) ^ 1;
        ok = mbar_wait(&bars.raw_full[st], (n / kRaw) & 1, a.err) &&
             mbar_wait(&bars.k_empty[op], par, a.err);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        uint32_t v_params;
        int v_exp;
        Dequant<D>::keys(raw, ops + op * C::kK, oct, tok, p.r.kv, ex, &v_params, &v_exp);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.k_full[op]);
        ok = __all_sync(~0u, mbar_wait(&bars.v_empty[op], par, a.err));
        if (!ok) break;
        Dequant<D>::values(raw, ops + C::kOffV + op * C::kK, tables[oct], oct, v_params, v_exp);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.v_full[op]);
          mbar_arrive(&bars.raw_empty[st]);
        }
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      const uint32_t id_s = idesc_f16(kRows, kStep), id_o = idesc_f16(kRows, D);
      // scores of step k
      auto scores = [&](int k) {
        if (!mbar_wait(&bars.k_full[k % kOps], (k / kOps) & 1, a.err)) return false;
        // the buffer's weights of step k - 2 have been used
        if (k >= 2 && !mbar_wait(&bars.pv_done[k & 1], ((k - 2) >> 1) & 1, a.err)) return false;
        tc_fence_after();
        const uint32_t kb = ops + (k % kOps) * C::kK;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_bf16_ts(tmem + C::kColS + (k & 1) * kStep, tmem + C::kColQ + 8 * i,
                      sdesc_k128(kb + (i / 4) * (kStep * 128) + (i % 4) * 32), id_s, i > 0);
        mma_commit(&bars.k_empty[k % kOps]);
        mma_commit(&bars.s_full[k & 1]);
        return true;
      };
      int part = 0;
      for (Part p = locate(a, first, w0, w1); p.some && ok;
           p = locate(a, first, p.next, w1), ++part) {
        ok = mbar_wait(&bars.q_full, part & 1, a.err);
        if (!ok) break;
        tc_fence_after();
        ok = scores(n);
        for (int t = p.t0; t < p.t1 && ok; ++t, ++n) {
          if (t + 1 < p.t1) ok = scores(n + 1);
          if (!ok) break;
          ok = mbar_wait(&bars.v_full[n % kOps], (n / kOps) & 1, a.err) &&
               mbar_wait(&bars.p_full[n & 1], (n >> 1) & 1, a.err) &&
               (t > p.t0 || part == 0 || mbar_wait(&bars.o_free, (part - 1) & 1, a.err));
          if (!ok) break;
          tc_fence_after();
          const uint32_t vb = ops + C::kOffV + (n % kOps) * C::kK;
#pragma unroll
          for (int i = 0; i < kStep / 16; ++i)
            mma_bf16_ts(tmem, tmem + C::kColS + (n & 1) * kStep + 8 * i, sdesc_k128(vb + i * 32),
                        id_o, t > p.t0 || i > 0);
          mma_commit(&bars.v_empty[n % kOps]);
          mma_commit(&bars.pv_done[n & 1]);
        }
      }
      // every MMA has ended before the tensor memory is given back
      if (n >= 1) mbar_wait(&bars.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, a.err);
    }
    __syncwarp();
  } else {
    // softmax: row `tid` of the row tile, tensor memory lane tid
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    for (Part p = locate(a, first, w0, w1); p.some && ok;) {
      const int row = p.rt * kRows + tid;
      const bool on = row < p.r.qn * a.d.G;
      const int tok = row / a.d.G;
      // the row as f16 in [2^13, 2^14) at its top, in the operands' channel order
      float unit;
      {
        const __nv_bfloat16* src =
            a.q + (int64_t)(p.r.q0 + (on ? tok : 0)) * a.q_stride +
            (int64_t)(p.h * a.d.G + (on ? row % a.d.G : 0)) * D;
        uint32_t top = 0;
#pragma unroll 8
        for (int i = 0; i < D / 8; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(src + 8 * i);
          const uint32_t x = __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
          top = __vmaxu2(top, __vmaxu2(x, __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
        }
        top = max(top & 0xffffu, top >> 16);
        const int e = min(max((int)(top >> 7) - 127, -100), 126);
        const float down = pow2(-e) * 8192.f;
        unit = pow2(e) * (64.f / 8192.f) * a.d.scale_log2;
#pragma unroll 1
        for (int g = 0; g < NG; ++g) {
          uint32_t q[32];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 w = on ? *reinterpret_cast<const uint4*>(src + 64 * g + 8 * j)
                               : make_uint4(0, 0, 0, 0);
            q[4 * j] = pack_f16(bf16_lo(w.x) * down, bf16_lo(w.z) * down);
            q[4 * j + 1] = pack_f16(bf16_hi(w.x) * down, bf16_hi(w.z) * down);
            q[4 * j + 2] = pack_f16(bf16_lo(w.y) * down, bf16_lo(w.w) * down);
            q[4 * j + 3] = pack_f16(bf16_hi(w.y) * down, bf16_hi(w.w) * down);
          }
          tmem_st32(lane_base + C::kColQ + 32 * g, q);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars.q_full);
      }
      const int lim = on ? seen_by(p.r, tok) : p.r.kv;
      const int least = seen_by(p.r, p.rt * kRows / a.d.G);
      float m = -INFINITY, l = 0.f;
      for (int t = p.t0; t < p.t1 && ok; ++t, ++n) {
        ok = __all_sync(~0u, mbar_wait(&bars.s_full[n & 1], (n >> 1) & 1, a.err));
        if (!ok) break;
        tc_fence_after();
        const uint32_t sb = lane_base + C::kColS + (n & 1) * kStep;
        uint32_t s[kStep];
        tmem_ld32(sb, s);
        tmem_ld32(sb + 32, s + 32);
        Exps ex[kRecs];
#pragma unroll
        for (int r = 0; r < kRecs; ++r) {
          const float4 v = *reinterpret_cast<const float4*>(&exps[n % kExps][r]);
          ex[r] = Exps{unit * v.x, v.y, v.z, 0.f};
        }
        wait_ld32(s);
        wait_ld32(s + 32);
        if ((t + 1) * kStep > least) {
#pragma unroll
          for (int i = 0; i < kStep; ++i)
            if (t * kStep + i >= lim) s[i] = 0xff800000u;  // -inf
        }
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < kRecs; ++r) {
          float x = __uint_as_float(s[16 * r]);
#pragma unroll
          for (int i = 1; i < 16; ++i) x = fmaxf(x, __uint_as_float(s[16 * r + i]));
          top = fmaxf(top, fmaf(x, ex[r].up_k, ex[r].ev));
        }
        if (__any_sync(~0u, top > m + kSlack)) {
          const float m_new = fmaxf(m, top);
          const float f = m_new == -INFINITY ? 1.f : exp2_fast(m - m_new);
          m = m_new;
          l *= f;
          if (t > p.t0) {
            // the outputs so far, once the last product has landed
            ok = __all_sync(~0u, mbar_wait(&bars.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, a.err));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(lane_base + c, o);
              wait_ld32(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st32(lane_base + c, o);
            }
            tmem_wait_st();
          }
        }
        const float ref = m == -INFINITY ? 0.f : kLift - m;
        uint32_t w[kStep / 2];
#pragma unroll
        for (int r = 0; r < kRecs; ++r) {
          const float add = ref + ex[r].ev;
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float p0 = exp2_fast(fmaf(__uint_as_float(s[16 * r + i]), ex[r].up_k, add));
            const float p1 = exp2_fast(fmaf(__uint_as_float(s[16 * r + i + 1]), ex[r].up_k, add));
            sum0 += p0;
            sum1 += p1;
            w[8 * r + i / 2] = pack_f16(p0, p1);
          }
          l = fmaf(sum0 + sum1, ex[r].down_v, l);
        }
        tmem_st32(sb, w);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars.p_full[n & 1]);
      }
      if (!ok) break;
      // outputs: after the last product
      ok = __all_sync(~0u, mbar_wait(&bars.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, a.err));
      if (!ok) break;
      tc_fence_after();
      const bool whole = p.t1 - p.t0 == p.tiles;
      const float inv = whole ? (l == 0.f ? 0.f : 64.f / l) : 64.f;
      const int64_t at = (int64_t)(2 * blockIdx.x + (p.t0 == 0)) * kRows + tid;
      __nv_bfloat16* dst = a.out + (int64_t)(p.r.q0 + tok) * a.out_stride +
                           (int64_t)(p.h * a.d.G + row % a.d.G) * D;
#pragma unroll 1
      for (int g = 0; g < NG; ++g) {
        uint32_t o[8][8];  // [nibble][word]
#pragma unroll
        for (int k = 0; k < 8; ++k) tmem_ld8(lane_base + out_column<NG>(g, k), o[k]);
        wait_ld32(&o[0][0]);
        wait_ld32(&o[4][0]);
        if (whole) {
          if (on) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 x =
                    __floats2bfloat162_rn(__uint_as_float(o[2 * k][j]) * inv,
                                          __uint_as_float(o[2 * k + 1][j]) * inv);
                v[k] = *reinterpret_cast<const uint32_t*>(&x);
              }
              *reinterpret_cast<uint4*>(dst + 64 * g + 8 * j) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
        } else {
          float4* part = reinterpret_cast<float4*>(a.part_o + at * D) + 16 * g;
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              part[8 * k + j] = make_float4(__uint_as_float(o[4 * k][j]) * inv,
                                            __uint_as_float(o[4 * k + 1][j]) * inv,
                                            __uint_as_float(o[4 * k + 2][j]) * inv,
                                            __uint_as_float(o[4 * k + 3][j]) * inv);
        }
      }
      tc_fence_before();
      mbar_arrive(&bars.o_free);
      if (!whole) {
        a.part_ml[at] = make_float2(m, l);
        if (p.t0 == 0 && tid == 0) {
          // the block of a shared row tile's first part names it for the joins
          const int parts =
              cut.block_of(p.start + (int64_t)(p.tiles - 1) * p.unit) - blockIdx.x + 1;
          a.desc[2 * blockIdx.x] = make_int4(parts, p.h, p.rt, p.r.q0);
          a.desc[2 * blockIdx.x + 1].x = p.r.qn;
        }
      }
      p = locate(a, first, p.next, w1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) {
    tmem_relinquish();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int D>
cudaError_t launch(const FwdArgs& a, int sms, cudaStream_t s) {
  const int blocks = sms < kMaxBlocks ? sms : kMaxBlocks;
  const cudaError_t e =
      launch_pdl(attn_prefill_kernel<D>, dim3(blocks), dim3(kThreads),
                 Cfg<D>::kSmem + (a.B + 1) * sizeof(int64_t), s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_join_kernel<D, kRows>, dim3(2 * sms), dim3(kJoinThreads), 0, s, a, blocks);
}

template <int D>
cudaError_t prepare(int max_requests) {
  return cudaFuncSetAttribute(attn_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<D>::kSmem + (max_requests + 1) * (int)sizeof(int64_t));
}

}  // namespace

size_t attn_prefill_part_floats(int D) { return (size_t)kRows * D; }

cudaError_t prepare_attn_prefill_kernels(int max_requests) {
  cudaError_t e;
  if ((e = prepare<64>(max_requests)) != cudaSuccess) return e;
  if ((e = prepare<128>(max_requests)) != cudaSuccess) return e;
  return prepare<256>(max_requests);
}

cudaError_t launch_attn_prefill(const FwdArgs& a, int sms, cudaStream_t s) {
  if (a.d.D == 256) return launch<256>(a, sms, s);
  if (a.d.D == 128) return launch<128>(a, sms, s);
  return launch<64>(a, sms, s);
}

}  // namespace moe
