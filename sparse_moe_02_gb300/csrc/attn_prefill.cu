// Attention of many query rows over the paged 4-bit cache (include/attn.h): prompts, chunks of
// prompts, and batches that hold any of them, on the tcgen05 tensor cores.
//
// A block works on 128 query rows of one key/value head (row = new token * G + query head) in steps
// of 64 cached tokens.  Four warps hold the softmax (a thread per row); eight turn cached keys and
// eight cached values into f16 MMA operands, and all sixteen stage queries and write outputs; one
// issues the MMAs, one finds the work, two copy.
//   S [128 x 64] = Q K^T      A = Q in tensor memory, B = keys [64][D] in shared memory
//   O [128 x D] += P V        A = P in tensor memory (over S), B = values [D][64] (channels by
//                             tokens, so both operands are K-major)
// Scores run ahead: those of step n + 2 are queued behind the product of step n.  With 256 channels
// a step of 64 tokens takes 1300 clocks of MMAs (64 columns: 49 clocks each, 256 columns: 129,
// measured alone).  The MMA warp runs its loop as a whole and one elected thread issues, from
// descriptors that are formed once and stepped by constants in uniform registers: issued from one
// thread's branch, the second case below took 957 us instead of 767.
//
// Every 128 rows of a head read the same context, and turning it into operands takes 2800 clocks a
// step (16 warps, two thirds of the block's issue slots), twice the MMAs.  So where contexts are read
// by many row tiles (kPrepTiles) a first launch, attn_prepare_kernel, forms the operands of every
// step once, in the handle's workspace, and this kernel copies them (64 KB a step from L2, 580 to 890
// clocks with all SMs at it) while its dequantising warps only stage queries and write outputs.  A
// step then takes 1600 clocks; what is left over the MMAs is the wait for the product whose weights
// lie where the next scores go (a third score buffer, with half of Q in shared memory, was no
// faster).
//
// Measured, 16 query heads over 2 of 256 channels: 4096 tokens from nothing 149 us (920 TFLOP/s,
// prepared; 209 us if not), 2048 over a context of 30000 755 us (1.37 PFLOP/s, 71% of a bf16 product's
// rate; 1100 us); 4096 tokens of 32 heads over 8 of 128 channels 186 us (281), over 4 of 64 channels
// 168 us (237); 7 ragged chunks and prompts of 28 heads over 4 of 128 85 us (106).  Of the 149 us the
// prepare launch takes 8, start and tail of the blocks and the joins 20.
//
// Arithmetic.  Per record of 16 tokens, keys and values enter as f16(x 2^-(e + 6)), 2^e a bound of
// the record's magnitudes: one fused multiply-add per pair of codes, since a nibble masked in place
// is the exact f16 subnormal code * 2^-24 (or 2^-20) and step * 2^24 2^-(e + 6) fits f16.  f16 keeps
// 11 bits of the larger entries and 2^-18 of the record's largest for the smaller ones, against 8
// bits of a bf16 operand.  Queries are scaled by a power of two per row.  The exponents return in
// fp32 with the scores and, for the values, inside the weights: P = 2^(x + e - m), where the running
// reference m bounds x + e; the softmax sum takes 2^(x - m), computed apart from P where e lies so far
// below others that P vanishes first (looking for that costs 128 channels 3%).  Scores, sums and
// outputs are fp32; 2^x is ex2.approx, within 2^-22.  The outputs are rescaled (in tensor memory)
// only when the reference grows by more than 2^6.  Entries 2^18 and more below the largest of their
// record lose bits, and weights 2^24 and more below the row's largest share of any value vanish: the
// values of a group or a token do beside others that are 2^20 times as large and count.
//
// Work.  Row tiles of all requests and heads, causally shortened, are cut evenly over the blocks as
// in the few-row kernel; shared row tiles are joined by its second launch.
#include <algorithm>
#include <climits>

#include "attn.cuh"
#include "attn_join.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;
constexpr int kStep = 64;            // tokens per step
constexpr int kRecs = kStep / 16;    // cache records per step
constexpr int kSoftWarps = 4;        // warps 0 .. 3
constexpr int kKeyWarp = 4, kValueWarp = 12, kDeqWarps = 8;  // the first of eight each
constexpr int kMmaWarp = 20, kLoadWarp = 21, kValueLoadWarp = 22, kFindWarp = 23;
constexpr int kThreads = 768;        // six warpgroups
// Registers of a thread by warpgroup (softmax, four of dequantising warps, the rest): together the
// 80 a thread that the launch grants.
constexpr int kRegsSoft = 168, kRegsDeq = 64, kRegsRest = 56;
static_assert(kRegsSoft + 4 * kRegsDeq + kRegsRest == 6 * 80, "the launch's registers");
constexpr int kParts = 4;            // parts announced ahead
constexpr float kSlack = 6.f, kLift = 9.f;  // as in the few-row kernel
// Values of a record this many binary orders below the largest so far: the reference may then lie so
// far above the record's weights that they leave fp32's range.
constexpr float kSpread = 64.f;
constexpr int kExps = 8;             // steps of record exponents kept
constexpr int kNotFinite = 127;      // in place of the exponent of a query row that is not finite

template <int D>
struct Cfg {
  using R = Record<D>;
  static constexpr int NG = D / kGroup;
  // a row tile's fixed cost in tokens (kPartCost) over prepared contexts, whose steps are shorter:
  // its queries and outputs
  static constexpr int kPartCostPrep = D == 64 ? 256 : D * 5 / 2;
  // steps of key operands, value operands, and the records' key and value sides held
  static constexpr int kOpsK = 2, kOpsV = 2, kRawK = D == 256 ? 3 : 4, kRawV = D == 256 ? 2 : 4;
  static constexpr int kS = D == 256 ? 2 : 4;  // score buffers: what tensor memory holds
  // A record's key side (with the parameters of its values: the softmax needs their exponents with
  // the scores) and its value side.
  static constexpr int kSideK = R::kV, kSideV = R::kBytes - R::kVp;
  static constexpr int kK = kStep * D * 2;  // bytes of a key (or value) operand
  // queries pass through shared memory two groups at a time
  static constexpr int kQGroups = NG < 2 ? NG : 2, kQPasses = NG / kQGroups;
  static constexpr int kOffK = kQGroups * kRows * 128;
  static constexpr int kOffV = kOffK + kOpsK * kK;
  static constexpr int kOffRaw = kOffV + kOpsV * kK;
  static constexpr int kOffRawV = kOffRaw + kRawK * kRecs * kSideK;
  static constexpr int kFirst = kOffRawV + kRawV * kRecs * kSideV;
  static constexpr int kSmem = kFirst + 1024;  // the operands start on a 1024-byte boundary
  // tensor memory columns: O, Q, the score buffers
  static constexpr int kColQ = D;
  static constexpr int kColS = D + D / 2;
  static constexpr int kCols = 512;
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

// 16 lanes x 8 columns: thread (n, c) = (i / 4, i % 4) of the warp gets columns 2c, 2c + 1 of lane n
// (r[0], r[1]) and of lane n + 8 (r[2], r[3]).
__device__ __forceinline__ void tmem_ld_16x8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
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

// Packed fp32 pairs: half the issue slots of the softmax's multiplications and additions.
__device__ __forceinline__ uint64_t pair(float x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void fma_pair(float& a, float& b, uint32_t x, uint32_t y, uint64_t mul,
                                         uint64_t add) {
  asm("{\n\t.reg .b64 p;\n\t"
      "mov.b64 p, {%2, %3};\n\t"
      "fma.rn.f32x2 p, p, %4, %5;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(a), "=f"(b)
      : "r"(x), "r"(y), "l"(mul), "l"(add));
}
__device__ __forceinline__ void add_pair(uint64_t& sum, float x, float y) {
  asm("{\n\t.reg .b64 p;\n\t"
      "mov.b64 p, {%1, %2};\n\t"
      "add.rn.f32x2 %0, %0, p;\n\t}"
      : "+l"(sum)
      : "f"(x), "f"(y));
}

constexpr uint32_t kNib0 = 0x000f000fu, kNib1 = 0x00f000f0u;

// ------------------------------------------------------------------- the work of a block

// Work is counted in (cached token x query head) units, 128 per row tile and token position: row
// tile rt of a request with `base` cached tokens before its new ones costs kPartCost G + base G +
// 128 (rt + 1) units, and its step t starts at unit (kPartCost + 64 t) G of them.  Row tiles of a
// request without cached tokens, whose rows are only zeroed, cost kZeroCost G each.
constexpr int kPartCost = 320;   // tokens: a row tile's fixed cost
constexpr int kZeroCost = 96;
constexpr int kLeastSteps = 4;   // of a block

struct Cost {
  int64_t fixed, base;  // per row tile, in units
  int grow;             // 64: the work of half a row tile more for each
  __device__ __forceinline__ int64_t before(int64_t rt) const {
    return rt * (fixed + base) + grow * rt * (rt + 1);
  }
};

__device__ __forceinline__ Cost cost_of(const FwdArgs& a, const Req& r, int part_cost) {
  if (r.kv == 0) return Cost{(int64_t)kZeroCost * a.d.G, 0, 0};
  return Cost{(int64_t)part_cost * a.d.G, (int64_t)max(r.kv - r.qn, 0) * a.d.G, 64};
}

__device__ __forceinline__ int row_tiles(const FwdArgs& a, const Req& r) {
  return (r.qn * a.d.G + kRows - 1) / kRows;
}

// Cached tokens that new token `tok` of the request sees.
__device__ __forceinline__ int seen_by(const Req& r, int tok) {
  return min(max(r.kv - r.qn + tok + 1, 0), r.kv);
}

// The part that holds work w of the block's [w, w1).
__device__ __forceinline__ Part locate(const FwdArgs& a, const int64_t* first, int part_cost,
                                       int64_t w, int64_t w1) {
  Part p;
  p.some = false;
  while (w < w1) {
    p.b = find_request(first, a.B, w);
    p.r = load_req(a, p.b);
    const Cost c = cost_of(a, p.r, part_cost);
    const int rts = row_tiles(a, p.r);
    const int64_t head = c.before(rts);
    p.h = (int)divide(w - first[p.b], head);
    const int64_t at = first[p.b] + p.h * head;
    int rt;
    if (c.grow) {
      // 64 rt^2 + (fixed + base + 64) rt = w - at, then the exact tile beside the rounded root
      const float q = (float)(c.fixed + c.base + 64), x = (float)(w - at);
      rt = (int)(2.f * x / (q + sqrtf(fmaf(q, q, 256.f * x))));
      rt = min(max(rt, 0), rts - 1);
      while (rt > 0 && c.before(rt) > w - at) --rt;
      while (rt + 1 < rts && c.before(rt + 1) <= w - at) ++rt;
    } else {
      rt = (int)divide(w - at, c.fixed);
    }
    p.rt = rt;
    const int last = min((rt + 1) * kRows, p.r.qn * a.d.G) - 1;
    p.tiles = (seen_by(p.r, last / a.d.G) + kStep - 1) / kStep;
    const int64_t end = at + c.before(rt + 1);
    p.unit = kStep * a.d.G;
    p.start = at + c.before(rt) + c.fixed;
    const int64_t stop = min(end, w1);
    // the steps that start in [w, stop)
    p.t0 = w <= p.start ? 0 : (int)min((int64_t)p.tiles, divide(w - p.start + p.unit - 1, p.unit));
    p.t1 = stop <= p.start
               ? 0
               : (int)min((int64_t)p.tiles, divide(stop - p.start + p.unit - 1, p.unit));
    // a row tile that sees nothing is one part without steps, where its work begins
    p.some = p.t1 > p.t0 || (p.tiles == 0 && w <= at + c.before(rt));
    w = p.next = stop;
    if (p.some) break;
  }
  return p;
}

// ------------------------------------------------------------------- shared state

template <int D>
struct Bars {
  using C = Cfg<D>;
  uint64_t part_full[kParts], part_empty[kParts];
  uint64_t raw_full[2][4], raw_empty[2][4];  // [keys, values]
  uint64_t k_full[C::kOpsK], k_empty[C::kOpsK], v_full[C::kOpsV], v_empty[C::kOpsV];
  uint64_t s_full[C::kS], p_full[C::kS], pv_done[C::kS];
  uint64_t x_full[kExps];  // exponents of prepared steps
  uint64_t q_staged, q_copied, q_full, q_free, o_done, o_free, ended;
  // Two in turn: the softmax of a part needs its queries, not the outputs of the part before, so it can
  // end while a warp has yet to look at the part before's; queries of the part after that are staged
  // behind those outputs by every warp.
  uint64_t o_scaled[2];
};

// True in one thread of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// Moves the warpgroup's threads to n registers.
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Exponents of a record: keys were divided by 2^(ek + 6), values by 2^(ev + 6).
struct __align__(16) Exps {
  float up_k;    // 2^ek
  float ev;      // ev
  float down_v;  // 2^-ev
  float pad;
};

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Magnitudes of a parameter word (step below, bias above) as packed bf16 bits; those of a token that
// is marked as not finite count as nothing.
__device__ __forceinline__ uint32_t magnitudes(uint32_t params) {
  return params == 0x7fc00000u ? 0u : params & 0x7fff7fffu;
}

// e with |bias| + 15 |step| < 2^e for the largest of either over the warp; at most 119: kLargest bounds
// the bias below 2^116 and the step below 2^117 / 15.
__device__ __forceinline__ int exponent_of(uint32_t packed) {
  const int s = (int)(__reduce_max_sync(~0u, packed & 0xffffu) >> 7);
  const int b = (int)(__reduce_max_sync(~0u, packed >> 16) >> 7);
  return max(max(s + 4, b) - 125, -90);  // 15 step < 2^(4 + its exponent + 1)
}

// One warp turns 8 cached tokens (half a record) of a step into operands: rows of the key operand
// [64 tokens][D] or columns of the value operand [D][64 tokens], both in the 128-byte swizzle.  The
// values are formed in registers first and stored once the operand's last readers are done, so
// only the stores lie between two MMAs on the same buffer.
template <int D>
struct Dequant {
  uint32_t out[2 * (D / kGroup)][4];

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
    *e = exponent_of(max_u16x2(magnitudes(w), magnitudes(w2)));
    return w;
  }

  // tok: the first token's index in the context.  Also leaves the record's exponents in *ex (those
  // of the values too: the softmax needs them with the scores).
  __device__ __forceinline__ void keys(uint32_t raw, int oct, int tok, int kv, Exps* ex) {
    const int lane = threadIdx.x & 31;
    const int t = lane & 7, g = (lane >> 3) % NG, sub = lane / (8 * NG);
    const uint32_t rec = raw + (oct >> 1) * C::kSideK;
    const int row = 8 * (oct & 1) + t;
    int e, ev;
    const uint32_t w = params(rec, R::kKp, oct, tok, kv, &e);
    params(rec, R::kVp, oct, tok, kv, &ev);
    if (lane == 0 && (oct & 1) == 0) *ex = Exps{pow2(e), (float)ev, pow2(-ev), 0.f};
    const float down = pow2(-(e + 6));
    const float s = bf16_lo(w) * down, b = bf16_hi(w) * down;
    const uint32_t s24 = pack_f16(s * 16777216.f, s * 16777216.f);
    const uint32_t s20 = pack_f16(s * 1048576.f, s * 1048576.f);
    const uint32_t bb = pack_f16(b, b);
    const uint32_t src = rec + row * R::kRow + 4 * g;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int j = (sub * kWords + i) ^ (t >> 2);
      const uint32_t c = lds32(src + ((j ^ row_swz(t)) * NG) * 4), c8 = c >> 8;
      out[i][0] = fma_f16x2(c & kNib0, s24, bb);
      out[i][1] = fma_f16x2(c & kNib1, s20, bb);
      out[i][2] = fma_f16x2(c8 & kNib0, s24, bb);
      out[i][3] = fma_f16x2(c8 & kNib1, s20, bb);
    }
  }

  __device__ __forceinline__ void store_keys(uint32_t dst, int oct) {
    const int lane = threadIdx.x & 31;
    const int t = lane & 7, g = (lane >> 3) % NG, sub = lane / (8 * NG);
    const uint32_t at = dst + g * (kStep * 128) + (8 * oct + t) * 128;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int j = (sub * kWords + i) ^ (t >> 2);
      sts128(at + ((j ^ t) << 4), out[i][0], out[i][1], out[i][2], out[i][3]);
    }
  }

  // Row i * 32 + lane of the value operand is channel 64 g + 8 j + kWords sub + i (lane = (sub, g, j)),
  // so that the rows of a store differ in their last three bits, which the swizzle spreads over
  // the banks.  `table`: 16 bytes for each pair of tokens and group, of this warp.
  __device__ __forceinline__ void values(uint32_t raw, uint4* table, int oct, int tok, int kv) {
    const int lane = threadIdx.x & 31;
    const uint32_t rec = raw + (oct >> 1) * C::kSideV;
    {
      int e;
      const uint32_t w = params(rec, R::kVp, oct, tok, kv, &e);
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
  }

  __device__ __forceinline__ void store_values(uint32_t dst, int oct) {
    const int lane = threadIdx.x & 31, j = lane & 7;
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

// Query rows row0 .. row0 + 7 of a part as f16 in [2^13, 2^14) at their top, in the operands' channel
// order: D / 8 lanes a row, 16-byte pieces, held by one warp.
template <int D>
struct QueryRows {
  static constexpr int kL = D / 8, kPer = 32 / kL;  // lanes a row, rows at a time
  uint4 w[8 / kPer];

  __device__ __forceinline__ void load(const FwdArgs& a, const Part& p, int row0, int8_t* exps) {
    const int lane = threadIdx.x & 31;
    // addresses of the eight rows, a lane each
    const int row = p.rt * kRows + row0 + (lane & 7);
    const uint64_t own =
        row < p.r.qn * a.d.G
            ? (uint64_t)(a.q + (int64_t)(p.r.q0 + row / a.d.G) * a.q_stride +
                         (int64_t)(p.h * a.d.G + row % a.d.G) * D)
            : 0;
#pragma unroll
    for (int i = 0; i < 8 / kPer; ++i) {
      const uint64_t src = __shfl_sync(~0u, own, i * kPer + lane / kL);
      w[i] = make_uint4(0, 0, 0, 0);
      if (src) w[i] = reinterpret_cast<const uint4*>(src)[lane % kL];
    }
#pragma unroll
    for (int i = 0; i < 8 / kPer; ++i) {
      uint32_t top = max_u16x2(max_u16x2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu),
                               max_u16x2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu));
#pragma unroll
      for (int o = kL / 2; o; o >>= 1) top = max_u16x2(top, __shfl_xor_sync(~0u, top, o));
      top = max(top & 0xffffu, top >> 16);
      const int e = min(max((int)(top >> 7) - 127, -100), 126);
      const float down = pow2(-e) * 8192.f;
      if (lane % kL == 0)
        exps[row0 + i * kPer + lane / kL] = (int8_t)(top >= 0x7f80u ? kNotFinite : e);
      w[i] = make_uint4(pack_f16(bf16_lo(w[i].x) * down, bf16_lo(w[i].z) * down),
                        pack_f16(bf16_hi(w[i].x) * down, bf16_hi(w[i].z) * down),
                        pack_f16(bf16_lo(w[i].y) * down, bf16_lo(w[i].w) * down),
                        pack_f16(bf16_hi(w[i].y) * down, bf16_hi(w[i].w) * down));
    }
  }

  // Groups g0 .. g0 + kQGroups - 1 into shared memory: [group][row] of 128 bytes, pieces swizzled.
  __device__ __forceinline__ void store(uint32_t dst, int row0, int g0) {
    const int lane = threadIdx.x & 31, g = ((lane % kL) >> 3) - g0, j = lane & 7;
    if (g < 0 || g >= Cfg<D>::kQGroups) return;
#pragma unroll
    for (int i = 0; i < 8 / kPer; ++i) {
      const int row = row0 + i * kPer + lane / kL;
      sts128(dst + g * (kRows * 128) + row * 128 + ((j ^ (row & 7)) << 4), w[i].x, w[i].y, w[i].z,
             w[i].w);
    }
  }
};

// The warp's 32 rows (tensor memory lanes 32 (warp % 4) ..) of those groups into tensor memory.
template <int D>
__device__ __forceinline__ void copy_queries(uint32_t src, uint32_t tmem, int g0) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, row = 32 * quarter + lane;
#pragma unroll 1
  for (int g = 0; g < C::kQGroups; ++g) {
    uint32_t q[32];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(q[4 * j]), "=r"(q[4 * j + 1]), "=r"(q[4 * j + 2]), "=r"(q[4 * j + 3])
                   : "r"(src + g * (kRows * 128) + row * 128 + ((j ^ (row & 7)) << 4)));
    tmem_st32(tmem + ((uint32_t)(32 * quarter) << 16) + C::kColQ + 32 * (g0 + g), q);
  }
  tmem_wait_st();
  tc_fence_before();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(FwdArgs a) {
  using C = Cfg<D>;
  constexpr int NG = C::NG;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars<D> bars;
  __shared__ Exps exps[kExps][kRecs];
  __shared__ uint4 tables[kDeqWarps][4 * NG];
  __shared__ Part parts[kParts];
  __shared__ int8_t row_exp[kExps][kRows];  // of the queries of the last parts
  __shared__ float out_scale[2][kRows];  // of the outputs of the last parts
  __shared__ uint32_t tmem_base;
  __shared__ int64_t sums[kThreads / 32];
  __shared__ Cut cut_s;
  uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&bars.part_full[i], 1);
      mbar_init(&bars.part_empty[i], kSoftWarps + 2 * kDeqWarps + 3);
    }
    for (int side = 0; side < 2; ++side)
      for (int i = 0; i < 4; ++i) {
        mbar_init(&bars.raw_full[side][i], 1);
        mbar_init(&bars.raw_empty[side][i], kDeqWarps);
      }
    for (int i = 0; i < C::kOpsK; ++i) {
      mbar_init(&bars.k_full[i], kDeqWarps);
      mbar_init(&bars.k_empty[i], 1);
    }
    for (int i = 0; i < C::kOpsV; ++i) {
      mbar_init(&bars.v_full[i], kDeqWarps);
      mbar_init(&bars.v_empty[i], 1);
    }
    for (int i = 0; i < C::kS; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 32 * kSoftWarps);
      mbar_init(&bars.pv_done[i], 1);
    }
    for (int i = 0; i < kExps; ++i) mbar_init(&bars.x_full[i], 1);
    mbar_init(&bars.q_staged, 2 * kDeqWarps);
    mbar_init(&bars.q_copied, 4);
    mbar_init(&bars.q_full, 4);
    mbar_init(&bars.q_free, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bars.o_scaled[i], kSoftWarps);
    mbar_init(&bars.o_done, 1);
    mbar_init(&bars.o_free, 2 * kDeqWarps);
    mbar_init(&bars.ended, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&tmem_base, C::kCols);
  pdl_wait();
  pdl_trigger();
  int64_t* first = reinterpret_cast<int64_t*>(smem + C::kFirst);
  const bool prepared = a.prep_cap > 0 && a.prep_at[0];
  const int part_cost = prepared ? C::kPartCostPrep : kPartCost;
  {
    const Cut cut =
        cut_work<kThreads>(a, first, sums, (int64_t)kLeastSteps * kStep * a.d.G, [&](const Req& r) {
          return a.d.Hkv * cost_of(a, r, part_cost).before(row_tiles(a, r));
        });
    if (tid == 0) {
      cut_s = cut;
      a.desc[2 * blockIdx.x].x = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const uint32_t ops = smem_u32(smem);
  bool ok = true;
  int n = 0;  // steps so far

  // The block's parts in order, as the load warp announces them: part k in parts[k % kParts].
  auto part_ready = [&](int k) {
    return mbar_wait(&bars.part_full[k % kParts], (k / kParts) & 1, a.err);
  };
  auto part_read = [&](int k) { mbar_arrive(&bars.part_empty[k % kParts]); };

  if (warp >= kMmaWarp) {
    registers_down<kRegsRest>();
    // copies the key (0) or value (1) sides of a part's records, a warp each
    auto copy_sides = [&](int which, int b, int h, int kv, int t0, int t1) {
      const int recs = (kv + 15) / 16, ring = which ? C::kRawV : C::kRawK;
      uint32_t record = 0;
      for (int t = t0; t < t1; ++t, ++n) {
        const int slot = (t - t0) & 7;
        if (slot == 0) {  // the records of eight steps, one a lane
          const int rec = t * kRecs + lane;
          if (rec < recs) record = cache_record(a, b, h, rec);
        }
        const int st = n % ring;
        uint64_t* full = &bars.raw_full[which][st];
        ok = mbar_wait(&bars.raw_empty[which][st], ((n / ring) & 1) ^ 1, a.err);
        ok = __all_sync(~0u, ok);
        if (!ok) return;
        const int have = min(max(recs - t * kRecs, 0), kRecs);
        const uint32_t rec = __shfl_sync(~0u, record, slot * kRecs + (lane & 3));
        const int side = which ? C::kSideV : C::kSideK;
        if (lane == 0) mbar_arrive_expect_tx(full, have * side);
        __syncwarp();
        if (lane < have)
          copy_record(smem + (which ? C::kOffRawV : C::kOffRaw) + (st * kRecs + lane) * side,
                      a.cache + (uint64_t)rec * C::R::kBytes + (which ? C::R::kVp : 0), side, full);
      }
    };
    // copies the prepared key (0) or value (1) operands of steps t0 .. t1 - 1 of a context whose
    // first is `at`, a warp each: eight arrivals a step, as from the dequantising warps
    auto copy_prepared = [&](int which, int at, int t0, int t1) {
      constexpr int kRing = C::kOpsK;
      static_assert(C::kOpsK == C::kOpsV && kDeqWarps == 8, "one rule for both");
      for (int t = t0; t < t1; ++t, ++n) {
        const int op = n % kRing;
        uint64_t* full = which ? &bars.v_full[op] : &bars.k_full[op];
        ok = mbar_wait(which ? &bars.v_empty[op] : &bars.k_empty[op], ((n / kRing) & 1) ^ 1, a.err);
        ok = __all_sync(~0u, ok);
        if (!ok) return;
        if (lane == 0) {
          mbar_arrive_expect_tx(full, C::kK);
          copy_record(smem + (which ? C::kOffV : C::kOffK) + op * C::kK,
                      a.prep + ((int64_t)(at + t) * 2 + which) * C::kK, C::kK, full);
        } else if (lane < kDeqWarps) {
          mbar_arrive(full);
        } else if (lane == kDeqWarps && which == 0) {
          mbar_arrive_expect_tx(&bars.x_full[n % kExps], sizeof(exps[0]));
          copy_record(exps[n % kExps], a.prep_exps + (int64_t)(at + t) * kRecs, sizeof(exps[0]),
                      &bars.x_full[n % kExps]);
        }
        __syncwarp();
      }
    };
    // first prepared step of a part's context
    auto prepared_at = [&](const Part& p) {
      return a.prep_at[1 + p.b] + p.h * ((p.r.kv + kStep - 1) / kStep);
    };
    // nothing may be in flight when the block ends
    auto drain = [&](int which) {
      if (prepared) {
        for (int k = max(0, n - C::kOpsK); k < n; ++k)
          mbar_wait(which ? &bars.v_full[k % C::kOpsK] : &bars.k_full[k % C::kOpsK],
                    (k / C::kOpsK) & 1, a.err);
        for (int k = max(0, n - kExps); which == 0 && k < n; ++k)
          mbar_wait(&bars.x_full[k % kExps], (k / kExps) & 1, a.err);
        return;
      }
      const int ring = which ? C::kRawV : C::kRawK;
      for (int k = max(0, n - ring); k < n; ++k)
        mbar_wait(&bars.raw_full[which][k % ring], (k / ring) & 1, a.err);
    };
    if (warp == kFindWarp) {
      int64_t w = 0, w1 = 0;
      if ((int)blockIdx.x < cut_s.blocks)
        w = cut_s.bound(blockIdx.x), w1 = cut_s.bound(blockIdx.x + 1);
      for (int k = 0; ok; ++k) {
        const Part p = locate(a, first, part_cost, w, w1);
        ok = mbar_wait(&bars.part_empty[k % kParts], ((k / kParts) & 1) ^ 1, a.err);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        if (lane == 0) {
          parts[k % kParts] = p;
          mbar_arrive(&bars.part_full[k % kParts]);
        }
        if (!p.some) break;
        w = p.next;
      }
    } else if (warp == kLoadWarp || warp == kValueLoadWarp) {
      const int which = warp == kValueLoadWarp;
      for (int k = 0; ok; ++k) {
        ok = __all_sync(~0u, part_ready(k));
        if (!ok) break;
        const Part p = parts[k % kParts];
        __syncwarp();
        if (lane == 0) part_read(k);
        if (!p.some) break;
        if (prepared) copy_prepared(which, prepared_at(p), p.t0, p.t1);
        else copy_sides(which, p.b, p.h, p.r.kv, p.t0, p.t1);
      }
      drain(which);
    } else if (warp == kMmaWarp) {
      // the whole warp walks through the steps, so that all that the MMAs take is uniform; one of
      // its threads issues them
      const bool lead = elect_one();
      const uint32_t id_s = idesc_f16(kRows, kStep), id_o = idesc_f16(kRows, D);
      const uint64_t k_desc = sdesc_k128(ops + C::kOffK), v_desc = sdesc_k128(ops + C::kOffV);
      // scores of step k; after a part's last ones its queries may be replaced
      auto scores = [&](int k, bool last) {
        const int op = k % C::kOpsK, sb = k % C::kS;
        // (the buffer's weights of step k - C::kS have been used)
        const bool go = mbar_wait(&bars.k_full[op], (k / C::kOpsK) & 1, a.err) &&
                        (k < C::kS ||
                         mbar_wait(&bars.pv_done[sb], ((k - C::kS) / C::kS) & 1, a.err));
        if (!__all_sync(~0u, go)) return false;
        tc_fence_after();
        if (lead) {
          const uint64_t kd = k_desc + op * (C::kK / 16);
          const uint32_t d = tmem + C::kColS + sb * kStep;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            mma_bf16_ts(d, tmem + C::kColQ + 8 * i, kd + ((i / 4) * (kStep * 8) + (i % 4) * 2), id_s,
                        i > 0);
          mma_commit(&bars.k_empty[op]);
          mma_commit(&bars.s_full[sb]);
          if (last) mma_commit(&bars.q_free);
        }
        __syncwarp();
        return true;
      };
      for (int k = 0, kq = 0; ok; ++k) {  // kq: parts with steps
        ok = __all_sync(~0u, part_ready(k));
        if (!ok) break;
        const bool some = __shfl_sync(~0u, parts[k % kParts].some, 0);
        const int steps = __shfl_sync(~0u, parts[k % kParts].t1 - parts[k % kParts].t0, 0);
        __syncwarp();
        if (lane == 0) part_read(k);
        if (!some) break;
        if (steps == 0) continue;
        ok = __all_sync(~0u, mbar_wait(&bars.q_full, kq & 1, a.err));
        if (!ok) break;
        // two steps of scores ahead of the products
        ok = scores(n, steps == 1) && (steps < 2 || scores(n + 1, steps == 2));
        for (int t = 0; t < steps && ok; ++t, ++n) {
          const int op = n % C::kOpsV, sb = n % C::kS;
          ok = mbar_wait(&bars.v_full[op], (n / C::kOpsV) & 1, a.err) &&
               mbar_wait(&bars.p_full[sb], (n / C::kS) & 1, a.err) &&
               (t > 0 || kq == 0 || mbar_wait(&bars.o_free, (kq - 1) & 1, a.err));
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          tc_fence_after();
          if (lead) {
            const uint64_t vd = v_desc + op * (C::kK / 16);
            const uint32_t w = tmem + C::kColS + sb * kStep;
            const uint32_t more = t > 0;
#pragma unroll
            for (int i = 0; i < kStep / 16; ++i)
              mma_bf16_ts(tmem, w + 8 * i, vd + 2 * i, id_o, i > 0 ? 1u : more);
            mma_commit(&bars.v_empty[op]);
            mma_commit(&bars.pv_done[sb]);
            if (t + 1 == steps) mma_commit(&bars.o_done);
          }
          __syncwarp();
          if (t + 2 < steps) ok = scores(n + 2, t + 3 == steps);
        }
        ++kq;
      }
      // every MMA, those of a run that a wait cut short too, has ended before the tensor memory is
      // given back
      if (lead) mma_commit(&bars.ended);
      __syncwarp();
      mbar_wait(&bars.ended, 0, a.err);
    }
    __syncwarp();
  } else if (warp >= kKeyWarp) {
    registers_down<kRegsDeq>();
    const bool is_key = warp < kValueWarp;
    const int oct = warp - (is_key ? kKeyWarp : kValueWarp);
    Dequant<D> d;
    // Outputs of part k, the kq-th with steps, from tensor memory: 16 rows of a group at a time, four
    // warps to the 32 lanes that each of them may read.
    auto outputs = [&](int k, int kq) {
      const int quarter = warp & 3;
      bool go = mbar_wait(&bars.o_done, kq & 1, a.err) &&
                mbar_wait(&bars.o_scaled[kq & 1], (kq >> 1) & 1, a.err);
      go = __all_sync(~0u, go);
      if (!go) return false;
      tc_fence_after();
      const Part& p = parts[k % kParts];
      const bool whole = p.t1 - p.t0 == p.tiles;
      const int64_t at = (int64_t)(2 * blockIdx.x + (p.t0 == 0)) * kRows;
      const int c = lane & 3;
#pragma unroll 1
      for (int u = (warp - kKeyWarp) >> 2; u < 2 * NG; u += 4) {
        const int hf = u & 1, g = u >> 1;
        const int ra = 32 * quarter + 16 * hf + (lane >> 2);
        // [nibble][row ra words 2c, 2c + 1; row ra + 8 words 2c, 2c + 1]
        uint32_t o[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          tmem_ld_16x8(tmem + ((uint32_t)(32 * quarter + 16 * hf) << 16) + out_column<NG>(g, i),
                       o[i]);
        wait_ld32(&o[0][0]);
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const int r = ra + 4 * q, row = p.rt * kRows + r;
          const float f = out_scale[kq & 1][r];
          uint8_t* d = nullptr;
          if (!whole)
            d = reinterpret_cast<uint8_t*>(a.part_o + (at + r) * D);
          else if (row < p.r.qn * a.d.G)
            d = reinterpret_cast<uint8_t*>(a.out + (int64_t)(p.r.q0 + row / a.d.G) * a.out_stride +
                                           (int64_t)(p.h * a.d.G + row % a.d.G) * D);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(o[i][q + w]) * f;
            if (whole) {
              uint32_t x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 y = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                x[i] = *reinterpret_cast<const uint32_t*>(&y);
              }
              if (d)
                *reinterpret_cast<uint4*>(d + 128 * g + 16 * (2 * c + w)) =
                    make_uint4(x[0], x[1], x[2], x[3]);
            } else {
              float4* part = reinterpret_cast<float4*>(d) + 16 * g + 2 * c + w;
              part[0] = make_float4(v[0], v[1], v[2], v[3]);
              part[8] = make_float4(v[4], v[5], v[6], v[7]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.o_free), part_read(k);
      return true;
    };
    int due = -1, kq = 0;  // the part whose outputs are to be written; parts with steps so far
    for (int k = 0; ok; ++k) {
      ok = __all_sync(~0u, part_ready(k));
      if (!ok) break;
      const Part p = parts[k % kParts];
      if (!p.some) break;
      if (p.t0 == p.t1) {
        // (a part's place is held until its outputs are written: not across parts without steps)
        if (due >= 0 && !(ok = outputs(due, kq - 1))) break;
        due = -1;
        __syncwarp();
        if (lane == 0) part_read(k);
        continue;
      }
      // queries: every warp scales eight rows, four warps (one for each 32 lanes) move them on once
      // the part before has used its own
      QueryRows<D> q;
      q.load(a, p, 8 * (warp - kKeyWarp), row_exp[kq % kExps]);
#pragma unroll
      for (int pass = 0; pass < C::kQPasses && ok; ++pass) {
        const int turn = kq * C::kQPasses + pass;
        if (turn > 0)
          ok = __all_sync(~0u, mbar_wait(&bars.q_copied, (turn - 1) & 1, a.err));
        if (!ok) break;
        q.store(ops, 8 * (warp - kKeyWarp), pass * C::kQGroups);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.q_staged);
        if (warp < kKeyWarp + 4) {
          ok = mbar_wait(&bars.q_staged, turn & 1, a.err) &&
               (pass > 0 || kq == 0 || mbar_wait(&bars.q_free, (kq - 1) & 1, a.err));
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          tc_fence_after();
          copy_queries<D>(ops, tmem, pass * C::kQGroups);
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars.q_copied);
            if (pass == C::kQPasses - 1) mbar_arrive(&bars.q_full);
          }
        }
      }
      if (!ok) break;
      if (due >= 0 && !(ok = outputs(due, kq - 1))) break;
      ++kq;
      due = k;
      if (prepared) continue;  // (steps are counted by those who use them)
      const int t0 = p.t0, t1 = p.t1, kv = p.r.kv;
      for (int t = t0; t < t1; ++t, ++n) {
        const int which = is_key ? 0 : 1, ring = is_key ? C::kRawK : C::kRawV;
        const int st = n % ring;
        const int tok = t * kStep + 8 * oct;
        ok = mbar_wait(&bars.raw_full[which][st], (n / ring) & 1, a.err);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        if (is_key)
          d.keys(ops + C::kOffRaw + st * kRecs * C::kSideK, oct, tok, kv,
                 &exps[n % kExps][oct >> 1]);
        else  // (a value side begins with its parameters: R::kVp from where the record would)
          d.values(ops + C::kOffRawV + st * kRecs * C::kSideV - C::R::kVp, tables[oct], oct, tok,
                   kv);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.raw_empty[which][st]);
        const int op = is_key ? n % C::kOpsK : n % C::kOpsV;
        const int turn = is_key ? n / C::kOpsK : n / C::kOpsV;
        ok = mbar_wait(is_key ? &bars.k_empty[op] : &bars.v_empty[op], (turn & 1) ^ 1, a.err);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        if (is_key) d.store_keys(ops + C::kOffK + op * C::kK, oct);
        else d.store_values(ops + C::kOffV + op * C::kK, oct);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(is_key ? &bars.k_full[op] : &bars.v_full[op]);
      }
    }
    if (ok && due >= 0) outputs(due, kq - 1);
  } else {
    registers_up<kRegsSoft>();
    // softmax: row `tid` of the row tile, tensor memory lane tid
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    for (int k = 0, kq = 0; ok; ++k) {  // kq: parts with steps
      ok = __all_sync(~0u, part_ready(k));
      if (!ok) break;
      const Part p = parts[k % kParts];
      __syncwarp();
      if (lane == 0) part_read(k);
      if (!p.some) break;
      const int row0 = p.rt * kRows + warp * 32;  // the warp's first row
      const int rows_left = p.r.qn * a.d.G;
      const int row = row0 + lane, tok = row / a.d.G;
      const bool on = row < rows_left;
      const int lim = on ? seen_by(p.r, tok) : p.r.kv;
      const int least = seen_by(p.r, p.rt * kRows / a.d.G);
      float m = -INFINITY, l = 0.f, unit = 0.f, most_ev = -INFINITY;
      for (int t = p.t0; t < p.t1 && ok; ++t, ++n) {
        ok = mbar_wait(&bars.s_full[n % C::kS], (n / C::kS) & 1, a.err) &&
             (!prepared || mbar_wait(&bars.x_full[n % kExps], (n / kExps) & 1, a.err));
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        tc_fence_after();
        if (t == p.t0)  // back from the scaled queries' units to log2 units
          unit = pow2(row_exp[kq % kExps][tid]) * (64.f / 8192.f) * a.d.scale_log2;
        const uint32_t sb = lane_base + C::kColS + (n % C::kS) * kStep;
        uint32_t s[kStep];
        tmem_ld32(sb, s);
        tmem_ld32(sb + 32, s + 32);
        Exps ex[kRecs];
#pragma unroll
        for (int r = 0; r < kRecs; ++r) {
          const float4 v = *reinterpret_cast<const float4*>(&exps[n % kExps][r]);
          ex[r] = Exps{fmaxf(unit * v.x, kLeastUnit), v.y, v.z, 0.f};
        }
        float least_ev = ex[0].ev;
        most_ev = fmaxf(most_ev, ex[0].ev);
#pragma unroll
        for (int r = 1; r < kRecs; ++r)
          least_ev = fminf(least_ev, ex[r].ev), most_ev = fmaxf(most_ev, ex[r].ev);
        const bool spread = least_ev < most_ev - kSpread;
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
          const float root = m_new == -INFINITY ? 1.f : exp2_fast(0.5f * (m - m_new));
          m = m_new;
          l = l * root * root;  // (see part_root)
          if (t > p.t0) {
            // the outputs so far, once the last product has landed
            ok = mbar_wait(&bars.pv_done[(n - 1) % C::kS], ((n - 1) / C::kS) & 1, a.err);
            ok = __all_sync(~0u, ok);
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
        if (__any_sync(~0u, spread)) {
          // with 2^ev weights may vanish that count in the sum: there they enter it without
#pragma unroll
          for (int r = 0; r < kRecs; ++r)
            if (ex[r].ev < most_ev - kSpread) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                l += exp2_fast(fmaf(__uint_as_float(s[16 * r + i]), ex[r].up_k, ref));
              ex[r].down_v = 0.f;
            }
        }
        uint32_t w[kStep / 2];
#pragma unroll
        for (int r = 0; r < kRecs; ++r) {
          const uint64_t add = pair(ref + ex[r].ev), mul = pair(ex[r].up_k);
          uint64_t sum = 0;  // two fp32 zeros
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float x0, x1;
            fma_pair(x0, x1, s[16 * r + i], s[16 * r + i + 1], mul, add);
            const float p0 = exp2_fast(x0), p1 = exp2_fast(x1);
            add_pair(sum, p0, p1);
            w[8 * r + i / 2] = pack_f16(p0, p1);
          }
          l = fmaf(__uint_as_float((uint32_t)sum) + __uint_as_float((uint32_t)(sum >> 32)),
                   ex[r].down_v, l);
        }
        tmem_st32(sb, w);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars.p_full[n % C::kS]);
      }
      if (!ok) break;
      if (p.tiles == 0) {  // rows that see nothing
        const uint64_t own =
            on ? reinterpret_cast<uint64_t>(a.out + (int64_t)(p.r.q0 + tok) * a.out_stride +
                                            (int64_t)(p.h * a.d.G + row % a.d.G) * D)
               : 0;
        for (int i = lane; i < 32 * (D / 8); i += 32) {
          const uint64_t dst = __shfl_sync(~0u, own, i / (D / 8));
          if (dst) reinterpret_cast<uint4*>(dst)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      // scores that are all -inf would read as a row that sees nothing
      if (lim > 0 && row_exp[kq % kExps][tid] == kNotFinite) l = NAN;
      const bool whole = p.t1 - p.t0 == p.tiles;
      out_scale[kq & 1][tid] = whole ? (l == 0.f ? 0.f : 64.f / row_sum(m, l)) : 64.f;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.o_scaled[kq & 1]);
      ++kq;
      const int64_t at = (int64_t)(2 * blockIdx.x + (p.t0 == 0)) * kRows + warp * 32;
      if (!whole) {
        a.part_ml[at + lane] = make_float2(m, l);
        if (p.t0 == 0 && tid == 0) {
          // the block of a shared row tile's first part names it for the joins
          const int count =
              cut_s.block_of(p.start + (int64_t)(p.tiles - 1) * p.unit) - blockIdx.x + 1;
          a.desc[2 * blockIdx.x] = make_int4(count, p.h, p.rt, p.r.q0);
          a.desc[2 * blockIdx.x + 1].x = p.r.qn;
        }
      }
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

// ------------------------------------------------------------------- contexts as operands

// Forms the MMA operands of every step of every context once, for calls whose contexts many row
// tiles read.
constexpr int kPrepThreads = 512;
// From this many row tiles per context, on average, it pays (256 channels, 16 contexts of 2000 to
// 4000 tokens, prepared against not: 4 row tiles 97 and 87 us, 6 114 and 113, 8 133 and 138, 16 (8
// contexts) 131 and 156; 128 channels: 4 206 and 181, 8 326 and 340).
constexpr int kPrepTiles = 8;
constexpr int64_t kMostPrep = 512ll << 20;  // bytes of operands held

template <int D>
struct PrepCfg {
  using C = Cfg<D>;
  static constexpr int kRaw = 2 * C::kK;
  static constexpr int kRawV = kRaw + kRecs * C::kSideK;
  static constexpr int kFirst = kRawV + kRecs * C::kSideV;
  static constexpr int kSmem = kFirst;
};

__device__ __forceinline__ void store_operands(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(kPrepThreads, 2) attn_prepare_kernel(FwdArgs a) {
  using C = Cfg<D>;
  using P = PrepCfg<D>;
  using R = Record<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint4 tables[kDeqWarps][4 * C::NG];
  __shared__ Exps exps[kRecs];
  __shared__ int64_t sums[kPrepThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5;
  int64_t* first = reinterpret_cast<int64_t*>(smem + P::kFirst);
  pdl_wait();
  pdl_trigger();
  // Steps of each context in the lower half, steps of its row tiles (a causal prompt's on average)
  // in the upper one; both capped far above what is ever taken.
  constexpr int64_t kCap = 1 << 20;
  cut_work<kPrepThreads>(a, first, sums, 1, [&](const Req& r) {
    if (r.qn == 0) return (int64_t)0;
    const int64_t steps = a.d.Hkv * (int64_t)((r.kv + kStep - 1) / kStep);
    const int64_t mean = a.d.Hkv * (int64_t)((max(r.kv - r.qn / 2, 0) + kStep - 1) / kStep);
    return min(steps, kCap) | min(mean * row_tiles(a, r), kCap) << 32;
  });
  const int64_t both = first[a.B];
  __syncthreads();  // every thread has it, and decides alike, before the sums lose their upper halves
  const int64_t steps = both & 0xffffffff;
  const bool prepared = steps <= a.prep_cap && (both >> 32) >= kPrepTiles * steps;
  for (int b = tid; b <= a.B; b += kPrepThreads) {
    first[b] &= 0xffffffff;
    if (blockIdx.x == 0 && b < a.B) a.prep_at[1 + b] = (int)min(first[b], (int64_t)INT_MAX);
  }
  if (blockIdx.x == 0 && tid == 0) a.prep_at[0] = prepared;
  if (!prepared) return;
  __syncthreads();

  const uint32_t ops = smem_u32(smem);
  for (int u = blockIdx.x; u < (int)steps; u += gridDim.x) {
    const int b = find_request(first, a.B, u);
    const int kv = load_req(a, b).kv, of = (kv + kStep - 1) / kStep;
    const int h = (u - (int)first[b]) / of, t = (u - (int)first[b]) % of;
    const int have = min((kv + 15) / 16 - t * kRecs, kRecs);
    constexpr int kPieces = R::kBytes / 16;
    for (int i = tid; i < have * kPieces; i += kPrepThreads) {
      const int rec = i / kPieces, at = i % kPieces * 16;
      const uint4 w = *reinterpret_cast<const uint4*>(
          a.cache + (uint64_t)cache_record(a, b, h, t * kRecs + rec) * R::kBytes + at);
      if (at < R::kV) *reinterpret_cast<uint4*>(smem + P::kRaw + rec * C::kSideK + at) = w;
      if (at >= R::kVp)
        *reinterpret_cast<uint4*>(smem + P::kRawV + rec * C::kSideV + at - R::kVp) = w;
    }
    __syncthreads();
    Dequant<D> d;
    const int oct = warp & 7, tok = t * kStep + 8 * oct;
    if (warp < kDeqWarps) {
      d.keys(ops + P::kRaw, oct, tok, kv, &exps[oct >> 1]);
      d.store_keys(ops, oct);
    } else {
      d.values(ops + P::kRawV - R::kVp, tables[oct], oct, tok, kv);
      d.store_values(ops + C::kK, oct);
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      store_operands(a.prep + (int64_t)u * 2 * C::kK, ops, 2 * C::kK);
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    } else if (tid >= 32 && tid < 32 + kRecs) {
      a.prep_exps[(int64_t)u * kRecs + tid - 32] = *reinterpret_cast<const uint4*>(&exps[tid - 32]);
    }
    __syncthreads();
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <int D>
cudaError_t launch(const FwdArgs& args, int sms, cudaStream_t s) {
  FwdArgs a = args;
  if ((int64_t)a.max_q * a.d.G > (kPrepTiles - 1) * kRows) {
    const cudaError_t e = launch_pdl(attn_prepare_kernel<D>, dim3(2 * sms), dim3(kPrepThreads),
                                     PrepCfg<D>::kSmem + (a.B + 1) * sizeof(int64_t), s, a);
    if (e != cudaSuccess) return e;
  } else {
    a.prep_cap = 0;
  }
  const int blocks = sms < kMaxBlocks ? sms : kMaxBlocks;
  const cudaError_t e =
      launch_pdl(attn_prefill_kernel<D>, dim3(blocks), dim3(kThreads),
                 Cfg<D>::kSmem + (a.B + 1) * sizeof(int64_t), s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_join_kernel<D, kRows>, dim3(8 * sms), dim3(kJoinThreads), 0, s, a, blocks);
}

template <int D>
cudaError_t prepare() {
  const cudaError_t e = cudaFuncSetAttribute(
      attn_prepare_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
      PrepCfg<D>::kSmem + (kMaxRequests + 1) * (int)sizeof(int64_t));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(attn_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<D>::kSmem + (kMaxRequests + 1) * (int)sizeof(int64_t));
}

}  // namespace

size_t attn_prefill_part_floats(int D) { return (size_t)kRows * D; }

size_t attn_prep_step_bytes(int D) { return (size_t)2 * kStep * D * 2; }

// As many as the cache's pages can make, up to kMostPrep bytes; calls with more of them (contexts
// that share pages) are not prepared.
int attn_prep_steps(const AttnDims& d, int max_requests) {
  const int64_t all =
      d.Hkv * ((((int64_t)d.n_pages << d.page_shift) + kStep - 1) / kStep + max_requests);
  return (int)std::min(all, kMostPrep / (int64_t)attn_prep_step_bytes(d.D));
}

cudaError_t prepare_attn_prefill_kernels() {
  cudaError_t e;
  if ((e = prepare<64>()) != cudaSuccess) return e;
  if ((e = prepare<128>()) != cudaSuccess) return e;
  return prepare<256>();
}

cudaError_t launch_attn_prefill(const FwdArgs& a, int sms, cudaStream_t s) {
  if (a.d.D == 256) return launch<256>(a, sms, s);
  if (a.d.D == 128) return launch<128>(a, sms, s);
  return launch<64>(a, sms, s);
}

}  // namespace moe
