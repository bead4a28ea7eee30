// Attention of many query rows over the paged 4-bit cache (include/attn.h): prompts, chunks of
// prompts, wide trees of drafted tokens, and batches that hold any of them, on the tcgen05 tensor
// cores.
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
// Every 128 rows of a head read the same context, and turning it into operands takes 2300 clocks a
// step (16 warps, two thirds of the block's issue slots), nearly twice the MMAs.  So where contexts
// are read by many row tiles (kPrepTiles) a first launch, attn_prepare_kernel, forms the operands
// of every step once, in the handle's workspace, and this kernel copies them (64 KB a step from L2,
// 580 to 890 clocks with all SMs at it) while its dequantising warps only stage queries and write
// outputs.  A step then takes 1600 clocks; what is left over the MMAs is the wait for the product
// whose weights lie where the next scores go (a third score buffer, with half of Q in shared
// memory, was no faster).
//
// Measured, 16 query heads over 2 of 256 channels: 4096 tokens from nothing 141 us (970 TFLOP/s,
// prepared; 209 us if not), 2048 over a context of 30000 757 us (1.36 PFLOP/s, 71% of a bf16 product's
// rate; 990 us); 4096 tokens of 32 heads over 8 of 128 channels 179 us, over 4 of 64 channels 165 us; 7
// ragged chunks and prompts of 28 heads over 4 of 128 80 us.  Of the 141 us the prepare launch takes 9,
// start and tail of the blocks and the joins 20.
//
// The form with masks (MASK) has the same steps over fewer of the context's tokens: the steps of
// the first tokens and those from a row tile's first window on.  A row's visible tokens of a step
// are 64 bits, formed only where a step holds a window's start, the first tokens' end or drafted
// tokens; of a wide tree all steps before the drafted ones need none.  Measured, 256 channels: a
// prompt of 8192 through a window of 1024 167 us (787 TFLOP/s of the visible pairs: a row tile's 18
// steps touch 1152 tokens for the 1040 that a row sees, and each of its 7 to a block costs some
// 5000 clocks besides, the change of queries and outputs), 16 trees of 20 to 60 tokens over
// contexts to 16384 59 us, 32 of 8 to 31 through a window of 1024 35 us: 5 steps a block, and
// around them the launch, the cut and the first row tile found (9000 clocks), its queries (8000),
// the first operands and scores (5000), outputs (5000) and the join.
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
// values of a group or a token do beside others that are 2^20 times as large and count, where a token
// counts as the one of its record with the largest weight.
//
// Uneven records.  What a row does not see must not cost it bits, so a record of which some rows see
// only a part is formed with an exponent for each token where the tokens' bounds differ by more than
// 2^kEven; the softmax then brings each score and weight to its token's.  Such records are looked for
// first: by the find warp, in a part's steps with edges, or by the prepare launch, whose findings the
// softmax warps read (where the find warp did, chunks through a window took 88 us instead of 85).  Parts
// without any run through loops that know nothing of them: checked for in every step (by the softmax,
// by the warps that form operands) they cost 3 to 20%, most of it instruction fetches.  As it is, prompts
// take 1 to 2% more than without, chunks 3%, trees 1 to 3%.
//
// Work.  Row tiles of all requests and heads, causally shortened, are cut evenly over the blocks as
// in the few-row kernel; shared row tiles are joined by its second launch.  Behind a window row
// tiles cost alike and blocks may take whole ones (kWholeMore).
#include <algorithm>
#include <climits>
#include <type_traits>

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
// Exponents by which the tokens of an even record differ at most.  An operand's rounding is half of
// f16's least spacing, 2^-25, so at most 2^(kEven + 6 - 25) of the bound of its own token, which is below
// 8 times the token's largest entry (|bias| and 15 |step|, rounded up to powers of two): 2^-11 of it.
constexpr int kEven = 5;
// Bounds of a score's unit where there are uneven records.  Scores times the least are nothing beside any
// that count, and what a token's exponent takes off, 209 at most, may be divided by it; the largest is far
// beyond the range of scores, but a number where the unit of keys that a row does not see is none.
constexpr float kLeastUp = 7.8886091e-31f, kMostUp = 1.2676506e30f;  // 2^-100, 2^100
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
  // A record's key side and its value side.
  static constexpr int kSideK = R::kVp, kSideV = R::kBytes - R::kVp;
  static constexpr int kK = kStep * D * 2;  // bytes of a key (or value) operand
  // queries pass through shared memory two groups at a time
  static constexpr int kQGroups = NG < 2 ? NG : 2, kQPasses = NG / kQGroups;
  static constexpr int kOffK = kQGroups * kRows * 128;
  static constexpr int kOffV = kOffK + kOpsK * kK;
  static constexpr int kOffRaw = kOffV + kOpsV * kK;
  static constexpr int kOffRawV = kOffRaw + kRawK * kRecs * kSideK;
  static constexpr int kFirst = kOffRawV + kRawV * kRecs * kSideV;
  static_assert(kQPasses <= 2 && (kQPasses == 1 || kFirst - kOffRaw >= kQGroups * kRows * 128),
                "room for the second half of the queries");
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
// Row tiles behind a window cost alike, so where a share is several of them blocks may take whole
// ones: no partial results and nothing to join, for up to this many steps more in the block that
// has most.  Cut against whole, 256 channels, a window of 1024: 7350 tokens (7.8 steps more) 151 and 145
// us, 6000 (11.3) 131 and 125, 8192 (17.0) 167 and 164.5, 2048 (18.5) 58.5 and 59.2, 4096 (27.7) 95
// and 100, 7700 (28.5) 158 and 160; a window of 300: 4096 (12.0) 68 and 63; of 3000: 8192 (21.2) 298 and
// 314; 128 channels: 4096 (0.8) 133 and 124, 2048 (9.7) 73 and 66, 6000 (21.0) 187 and 182; 64
// channels: 8192 (7.9) 235 and 218, 11000 (16.3) 305 and 287.  As a part of the share the border is no
// sharper: 0.24 gains 8% (2048 through 300), 0.06 loses 5% (8192 through 3000).
constexpr int kWholeMore = 18;

struct Cost {
  int64_t fixed, base;  // per row tile, in units
  int grow;             // 64: the work of half a row tile more for each
  // with masks: the row tiles from `bend` on cost `flat` each
  int64_t flat;
  int bend;
  template <bool MASK>
  __device__ __forceinline__ int64_t before(int64_t rt) const {
    if (MASK && rt > bend) return before<false>(bend) + (rt - bend) * flat;
    return rt * (fixed + base) + grow * rt * (rt + 1);
  }
};

// Steps that a row tile behind a window goes over at most: the first tokens, and a window of each
// of its tokens.
__device__ __forceinline__ int64_t window_steps(const FwdArgs& a, int tokens) {
  return ((int64_t)a.window + tokens + kStep - 1) / kStep + 1 + first_tiles<kStep>(a);
}

__device__ __forceinline__ int tile_tokens(const FwdArgs& a) { return (kRows - 1) / a.d.G + 1; }

template <bool MASK>
__device__ __forceinline__ Cost cost_of(const FwdArgs& a, const Req& r, int part_cost) {
  if (r.kv == 0) return Cost{(int64_t)kZeroCost * a.d.G, 0, 0, 0, INT_MAX};
  Cost c{(int64_t)part_cost * a.d.G, (int64_t)max(r.kv - r.qn, 0) * a.d.G, 64, 0, INT_MAX};
  if constexpr (MASK) {
    // the context at most (a tree's does), and what a window leaves of it
    int64_t most = a.masks ? r.kv : INT64_MAX;
    if (a.window) most = min(most, kStep * window_steps(a, a.masks ? r.qn : tile_tokens(a)));
    c.bend = 0;
    if (!a.masks)
      c.bend = (int)min(max(most * a.d.G - c.base, (int64_t)0) / kRows, (int64_t)INT_MAX);
    c.flat = c.fixed + most * a.d.G;
  }
  return c;
}

__device__ __forceinline__ int row_tiles(const FwdArgs& a, const Req& r) {
  return (r.qn * a.d.G + kRows - 1) / kRows;
}

// Cached tokens that new token `tok` of the request sees.
__device__ __forceinline__ int seen_by(const Req& r, int tok) {
  return min(max(r.kv - r.qn + tok + 1, 0), r.kv);
}

// A bound of the window starts of a row tile whose first token is `tok`.
__device__ __forceinline__ int tile_start(const FwdArgs& a, const Req& r, int tok) {
  return a.masks ? first_start(a, r) : window_start(a, r.kv - r.qn + tok);
}

// Where the queries of a row tile do not all see the same: tokens from `least` on, and, with masks, those
// between the first tokens and `low`, from which on tokens lie in every window.
template <bool MASK>
struct Edges {
  int least, low, first;
  __device__ __forceinline__ Edges(const FwdArgs& a, const Part& p) {
    least = seen_by(p.r, a.d.by_G(p.rt * kRows));
    low = INT_MIN;
    first = 0;
    if constexpr (MASK) {
      if (a.masks) least = p.r.kv - p.r.qn;
      // (or behind the row tile's last token)
      const int last = p.r.kv - p.r.qn + a.d.by_G((p.rt + 1) * kRows);
      low = window_start(a, a.masks ? p.r.kv - 1 : min(p.r.kv - 1, last));
      first = a.sinks;
    }
  }
  // whether the step from token t0 on holds such tokens
  __device__ __forceinline__ bool in(int t0) const {
    return t0 + kStep > least || (MASK && t0 < low && t0 + kStep > first);
  }
};

// The part that holds work w of the block's [w, w1).
template <bool MASK>
__device__ __forceinline__ Part locate(const FwdArgs& a, const int64_t* first, int part_cost,
                                       int64_t w, int64_t w1) {
  Part p;
  p.some = false;
  while (w < w1) {
    p.b = find_request(first, a.B, w);
    p.r = load_req(a, p.b);
    const Cost c = cost_of<MASK>(a, p.r, part_cost);
    const int rts = row_tiles(a, p.r);
    const int64_t head = c.template before<MASK>(rts);
    p.h = (int)divide(w - first[p.b], head);
    const int64_t at = first[p.b] + p.h * head;
    int rt;
    if (MASK && c.bend < rts && w - at >= c.template before<false>(c.bend)) {
      rt = c.bend + (int)divide(w - at - c.template before<false>(c.bend), c.flat);
    } else if (c.grow) {
      // 64 rt^2 + (fixed + base + 64) rt = w - at, then the exact tile beside the rounded root
      const float q = (float)(c.fixed + c.base + 64), x = (float)(w - at);
      rt = (int)(2.f * x / (q + sqrtf(fmaf(q, q, 256.f * x))));
      rt = min(max(rt, 0), rts - 1);
      while (rt > 0 && c.template before<MASK>(rt) > w - at) --rt;
      while (rt + 1 < rts && c.template before<MASK>(rt + 1) <= w - at) ++rt;
    } else {
      rt = (int)divide(w - at, c.fixed);
    }
    p.rt = rt;
    const int last = min((rt + 1) * kRows, p.r.qn * a.d.G) - 1;
    const int seen = MASK && a.masks ? p.r.kv : seen_by(p.r, a.d.by_G(last));
    p.tiles = (seen + kStep - 1) / kStep;
    if (MASK) {
      p.skip = skipped<kStep>(a, tile_start(a, p.r, a.d.by_G(rt * kRows)));
      p.tiles -= p.skip;
    }
    const int64_t end = at + c.template before<MASK>(rt + 1);
    p.unit = kStep * a.d.G;
    p.start = at + c.template before<MASK>(rt) + c.fixed;
    const int64_t stop = min(end, w1);
    // the steps that start in [w, stop)
    p.t0 = w <= p.start ? 0 : (int)min((int64_t)p.tiles, divide(w - p.start + p.unit - 1, p.unit));
    p.t1 = stop <= p.start
               ? 0
               : (int)min((int64_t)p.tiles, divide(stop - p.start + p.unit - 1, p.unit));
    // a row tile that sees nothing is one part without steps, where its work begins
    p.some = p.t1 > p.t0 || (p.tiles == 0 && w <= at + c.template before<MASK>(rt));
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
  uint64_t looked[kParts];  // whether a part has uneven records is known
  uint64_t raw_full[2][4], raw_empty[2][4];  // [keys, values]
  uint64_t k_full[C::kOpsK], k_empty[C::kOpsK], v_full[C::kOpsV], v_empty[C::kOpsV];
  uint64_t s_full[C::kS], p_full[C::kS], pv_done[C::kS];
  uint64_t x_full[kExps], ev_full[kExps];  // exponents of prepared steps; of the values of others
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

// Tokens of a context that its queries do not read: those behind it, and, with masks, those between the
// first tokens and every window, whose pages may have been given back.
template <bool MASK>
struct Unread {
  int kv;
  int first, start;
  __device__ __forceinline__ Unread(const FwdArgs& a, const Req& r) : kv(r.kv) {
    if constexpr (MASK) first = a.sinks, start = first_start(a, r);
  }
  __device__ __forceinline__ bool token(int t) const {
    return t >= kv || (MASK && t >= first && t < start);
  }
  // whether no token of a record is read
  __device__ __forceinline__ bool record(int rec) const {
    const int64_t t = 16 * (int64_t)rec;
    return t >= kv || (MASK && t >= first && t + 16 <= start);
  }
};

// Exponents of a record: keys were divided by 2^(ek + 6), values by 2^(ev + 6).  Of uneven ones (marked
// by the last bit of up_k or down_v) by those of their tokens.
struct __align__(16) Exps {
  float up_k;    // 2^ek
  float ev;      // ev
  float down_v;  // 2^-ev
  uint32_t some;  // of a prepared step's first record: whether any is uneven
};
struct StepExps {
  Exps rec[kRecs];
  int8_t tok[2][kStep];  // [keys, values], of uneven records
};
static_assert(sizeof(StepExps) == kPrepExps * sizeof(uint4), "as many words a prepared step");

__device__ __forceinline__ bool marked(float x) { return __float_as_uint(x) & 1; }

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

// e + 125 of a word's magnitudes alone, 0 where both are.
__device__ __forceinline__ uint32_t bound_of(uint32_t packed) {
  return packed ? max(((packed & 0xffffu) >> 7) + 4, packed >> 23) : 0u;
}

// A token's exponent from its bound, in a record whose largest is `all`.  Tokens that are not read fit
// any; those of zeros are formed with 1 at most, lest a row's unit times a larger one is no number.
__device__ __forceinline__ int exponent_of_bound(uint32_t bound, bool read, int all) {
  return bound ? max((int)bound - 125, -90) : read ? min(all, 0) : all;
}

// Exponents of a record, `all` that of the largest, from the bounds of a lane's tokens (own half, other
// half; whether they are read) in one of kGroups groups, 8 lanes apart: returns what to form the own
// token with.  Of uneven ones the warp of the first half leaves the tokens' in `left` and marks *scale.
template <int kGroups>
__device__ __forceinline__ int token_exponent(uint32_t own, bool read, uint32_t other,
                                              bool read_other, int all, int oct, int8_t* left,
                                              float* scale) {
  const int lane = threadIdx.x & 31;
  uint32_t both = own << 16 | other;
#pragma unroll
  for (int o = 8; o < 8 * kGroups; o <<= 1) both = max_u16x2(both, __shfl_xor_sync(~0u, both, o));
  const int e = exponent_of_bound(both >> 16, read, all);
  const int e2 = exponent_of_bound(both & 0xffffu, read_other, all);
  if (!__any_sync(~0u, min(e, e2) < all - kEven)) return all;
  if ((oct & 1) == 0) {
    if (lane < 8) {
      left[8 * oct + lane] = (int8_t)e;
      left[8 * oct + 8 + lane] = (int8_t)e2;
    }
    if (lane == 0) *scale = __uint_as_float(__float_as_uint(*scale) | 1u);
    __syncwarp();
  }
  return e;
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

  // Parameters of token lane & 7, group (lane >> 3) % NG of the record (0 behind the context) and *e, the
  // exponent of the record's 16 tokens, which the warp of its first half leaves in *ex; with LOOK, of
  // uneven records the token's own.
  template <bool kKeys, bool LOOK, bool MASK>
  static __device__ __forceinline__ uint32_t params(uint32_t rec, int oct, int tok,
                                                    const Unread<MASK>& un, StepExps* ex, int* e) {
    constexpr int off = kKeys ? R::kKp : R::kVp;
    const int lane = threadIdx.x & 31, t = lane & 7, g = (lane >> 3) % NG;
    const uint32_t par = rec + off + (8 * (oct & 1) + t) * R::kPar + 4 * g;
    const int other = (oct & 1) ? -8 : 8;  // the record's other half
    uint32_t w = lds32(par), w2 = lds32(par + other * R::kPar);
    if (un.token(tok + t)) w = 0;
    if (un.token(tok + t + other)) w2 = 0;
    *e = exponent_of(max_u16x2(magnitudes(w), magnitudes(w2)));
    Exps* own = &ex->rec[oct >> 1];
    if (lane == 0 && (oct & 1) == 0) {
      if (kKeys) {
        own->up_k = pow2(*e);
      } else {
        own->ev = (float)*e;
        own->down_v = pow2(-*e);
      }
    }
    if constexpr (LOOK) {
      // (groups of a token may be as small; seldom are all)
      const uint32_t b = bound_of(magnitudes(w)), b2 = bound_of(magnitudes(w2));
      const bool read = !un.token(tok + t), read2 = !un.token(tok + t + other);
      if (__any_sync(~0u, min(exponent_of_bound(b, read, *e), exponent_of_bound(b2, read2, *e)) <
                              *e - kEven))
        *e = token_exponent<NG>(b, read, b2, read2, *e, oct, ex->tok[!kKeys],
                                kKeys ? &own->up_k : &own->down_v);
    }
    return w;
  }

  // tok: the first token's index in the context.  Also leaves the exponents of the record's keys in *ex.
  template <bool LOOK, bool MASK>
  __device__ __forceinline__ void keys(uint32_t raw, int oct, int tok, const Unread<MASK>& un,
                                       StepExps* ex) {
    const int lane = threadIdx.x & 31;
    const int t = lane & 7, g = (lane >> 3) % NG, sub = lane / (8 * NG);
    const uint32_t rec = raw + (oct >> 1) * C::kSideK;
    const int row = 8 * (oct & 1) + t;
    int e;
    const uint32_t w = params<true, LOOK>(rec, oct, tok, un, ex, &e);
    const float down = pow2(-(e + 6));
    const float s = bf16_lo(w) * down, b = bf16_hi(w) * down;
    const uint32_t s24 = pack_f16(s * 16777216.f, s * 16777216.f);
    const uint32_t s20 = pack_f16(s * 1048576.f, s * 1048576.f);
    const uint32_t bb = pack_f16(b, b);
    // (rows start on multiples of their length: words are taken by an exclusive or with the address)
    const uint32_t src =
        rec + row * R::kRow + 4 * g + ((sub * kWords) ^ (t >> 2) ^ row_swz(t)) * (4 * NG);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t c = lds32(src ^ (i * 4 * NG)), c8 = c >> 8;
      out[i][0] = fma_f16x2(c & kNib0, s24, bb);
      out[i][1] = fma_f16x2(c & kNib1, s20, bb);
      out[i][2] = fma_f16x2(c8 & kNib0, s24, bb);
      out[i][3] = fma_f16x2(c8 & kNib1, s20, bb);
    }
  }

  __device__ __forceinline__ void store_keys(uint32_t dst, int oct) {
    const int lane = threadIdx.x & 31;
    const int t = lane & 7, g = (lane >> 3) % NG, sub = lane / (8 * NG);
    const uint32_t at = dst + g * (kStep * 128) + (8 * oct + t) * 128 +
                        (((sub * kWords) ^ (t >> 2) ^ t) << 4);
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      sts128(at ^ (i << 4), out[i][0], out[i][1], out[i][2], out[i][3]);
  }

  // Row i * 32 + lane of the value operand is channel 64 g + 8 j + kWords sub + i (lane = (sub, g,
  // j)), so that the rows of a store differ in their last three bits, which the swizzle spreads
  // over the banks.  `table`: 16 bytes for each pair of tokens and group, of this warp.  Leaves the
  // exponents of the record's values in *ex, and counts that on `left` if there is one (the softmax
  // needs them with the scores).
  template <bool LOOK, bool MASK>
  __device__ __forceinline__ void values(uint32_t raw, uint4* table, int oct, int tok,
                                         const Unread<MASK>& un, StepExps* ex, uint64_t* left) {
    const int lane = threadIdx.x & 31;
    const uint32_t rec = raw + (oct >> 1) * C::kSideV;
    {
      int e;
      const uint32_t w = params<false, LOOK>(rec, oct, tok, un, ex, &e);
      if (lane == 0 && (oct & 1) == 0 && left) mbar_arrive(left);
      const int t = lane & 7, g = (lane >> 3) % NG;
      const float down = pow2(-(e + 6));
      const uint32_t mate = __shfl_down_sync(~0u, w, 1);
      const float down1 = LOOK ? __shfl_down_sync(~0u, down, 1) : down;  // the next token's
      if ((t & 1) == 0 && lane < 8 * NG) {
        const float s0 = bf16_lo(w) * down, s1 = bf16_lo(mate) * down1;
        table[(t >> 1) * NG + g] =
            make_uint4(pack_f16(s0 * 16777216.f, s1 * 16777216.f),
                       pack_f16(s0 * 1048576.f, s1 * 1048576.f),
                       pack_f16(bf16_hi(w) * down, bf16_hi(mate) * down1), 0u);
      }
      __syncwarp();
    }
    const int j = lane & 7, g = (lane >> 3) % NG, sub = lane / (8 * NG);
    const uint32_t at = rec + R::kV + 8 * (oct & 1) * R::kRow + (j * NG + g) * 4;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int t = 2 * m;
      const uint32_t w0 = lds32((at ^ (row_swz(t) * (4 * NG))) + t * R::kRow);
      const uint32_t w1 = lds32((at ^ (row_swz(t + 1) * (4 * NG))) + (t + 1) * R::kRow);
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

// The exponents of 16 tokens.
struct TokenBytes {
  uint4 w;
  __device__ __forceinline__ int operator[](int i) const {
    const uint32_t x = i < 4 ? w.x : i < 8 ? w.y : i < 12 ? w.z : w.w;
    return (int8_t)(x >> (8 * (i & 3)));
  }
};

__device__ __forceinline__ TokenBytes token_bytes(const int8_t* p) {
  return TokenBytes{*reinterpret_cast<const uint4*>(p)};
}

// Turns a row's scores of a step, 64 columns of tensor memory from `at` on, of uneven records into those
// of even ones: each as if its key had the record's exponent, and with what its value's exponent lies
// below the record's taken off.  Whether there are any.
__device__ __forceinline__ bool scores_of_tokens(uint32_t at, const StepExps& ex, float unit) {
  uint32_t marks = 0;
#pragma unroll
  for (int r = 0; r < kRecs; ++r)
    marks |= __float_as_uint(ex.rec[r].up_k) | __float_as_uint(ex.rec[r].down_v);
  if (!(marks & 1)) return false;
#pragma unroll 1
  for (int r = 0; r < kRecs; r += 2) {
    uint32_t s[32];
    tmem_ld32(at + 16 * r, s);
    wait_ld32(s);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Exps rec = ex.rec[r + k];
      const TokenBytes ek = token_bytes(ex.tok[0] + 16 * (r + k));
      const TokenBytes ev = token_bytes(ex.tok[1] + 16 * (r + k));
      const float up = fminf(fmaxf(unit * rec.up_k, kLeastUp), kMostUp), down = 1.f / up;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = __uint_as_float(s[16 * k + i]);
        if (marked(rec.up_k)) x *= fmaxf(unit * pow2(ek[i]), kLeastUp) * down;
        if (marked(rec.down_v)) x = fmaf((float)ev[i] - rec.ev, down, x);
        s[16 * k + i] = __float_as_uint(x);
      }
    }
    tmem_st32(at + 16 * r, s);
  }
  tmem_wait_st();
  return true;
}

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
    const int row = p.rt * kRows + row0 + (lane & 7), tok = a.d.by_G(row);
    const uint64_t own =
        row < p.r.qn * a.d.G
            ? (uint64_t)(a.q + (int64_t)(p.r.q0 + tok) * a.q_stride +
                         (int64_t)(p.h * a.d.G + row - tok * a.d.G) * D)
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
      if constexpr (kL < 32) {
#pragma unroll
        for (int o = kL / 2; o; o >>= 1) top = max_u16x2(top, __shfl_xor_sync(~0u, top, o));
      }
      top = max(top & 0xffffu, top >> 16);
      if constexpr (kL == 32) top = __reduce_max_sync(~0u, top);
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

  // kQGroups groups from g0 on into shared memory: [group][row] of 128 bytes, pieces swizzled.
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

// A quarter of those groups' columns of the 32 rows (tensor memory lanes) that the warp may write
// into tensor memory.
template <int D>
__device__ __forceinline__ void copy_queries(uint32_t src, uint32_t tmem, int g0, int part) {
  using C = Cfg<D>;
  constexpr int kPieces = 2 * C::kQGroups;  // 16 bytes each: 4 columns
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, row = 32 * quarter + lane;
  uint32_t q[4 * kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int at = part * kPieces + i, g = at >> 3, j = at & 7;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q[4 * i]), "=r"(q[4 * i + 1]), "=r"(q[4 * i + 2]), "=r"(q[4 * i + 3])
                 : "r"(src + g * (kRows * 128) + row * 128 + ((j ^ (row & 7)) << 4)));
  }
  const uint32_t dst =
      tmem + ((uint32_t)(32 * quarter) << 16) + C::kColQ + 32 * g0 + 4 * kPieces * part;
  if constexpr (kPieces == 4) tmem_st16(dst, q);
  else tmem_st8(dst, q);
}

// Tokens t0 .. t0 + 63 of its context that a row sees, a bit each.
struct RowView {
  int lim;               // tokens below it: seen ones (causal), or cached before the new ones (a tree)
  int start;             // first token of its window
  const uint32_t* mask;  // of its drafted tokens, n of them; or none
  int n;

  static __device__ __forceinline__ uint64_t below(int k) {
    return k <= 0 ? 0 : k >= 64 ? ~0ull : (1ull << k) - 1;
  }

  __device__ __forceinline__ RowView(const FwdArgs& a, const Part& p, int tok, bool on)
      : lim(p.r.kv), start(INT_MIN), mask(nullptr), n(0) {
    if (!on) return;  // sees everything: nothing of it is written
    const int c = p.r.kv - p.r.qn;
    if (a.masks) {
      lim = c;
      n = p.r.qn;
      mask = a.masks + (int64_t)(p.r.q0 + tok) * a.mask_words;
      int seen = 0;
      if (a.window)
        for (int k = 0; 32 * k < n; ++k) seen += __popc(mask[k] & (uint32_t)below(n - 32 * k));
      start = window_start(a, c + max(seen - 1, 0));
    } else {
      lim = seen_by(p.r, tok);
      start = window_start(a, c + tok);
    }
  }

  __device__ __forceinline__ uint64_t seen(const FwdArgs& a, int t0) const {
    uint64_t v = below(lim - t0);
    if (mask) {
      const int k = t0 - lim, w0 = k >> 5;  // first drafted token of the step, its word
      uint32_t w[3];
#pragma unroll
      for (int i = 0; i < 3; ++i)
        w[i] = w0 + i >= 0 && 32 * (w0 + i) < n ? mask[w0 + i] : 0;
      const uint64_t bits = (uint64_t)__funnelshift_r(w[1], w[2], k & 31) << 32 |
                            __funnelshift_r(w[0], w[1], k & 31);
      v |= bits & below(n - k);
    }
    return start > t0 ? v & (below(a.sinks - t0) | ~below(start - t0)) : v;
  }
};

// First prepared step of a part's context and head.
template <bool MASK>
__device__ __forceinline__ int first_prepared(const FwdArgs& a, const Part& p) {
  const int left_out = MASK ? skipped<kStep>(a, first_start(a, p.r)) : 0;
  return a.prep_at[1 + p.b] + p.h * ((p.r.kv + kStep - 1) / kStep - left_out);
}

// The one of the part's step t.  (Where a row tile leaves steps out, its context does as many or fewer.)
template <bool MASK>
__device__ __forceinline__ int prepared_step(const FwdArgs& a, const Part& p, int first, int t) {
  if (MASK && t >= first_tiles<kStep>(a))
    return first + t + p.skip - skipped<kStep>(a, first_start(a, p.r));
  return first + t;
}

// Whether any of a part's prepared steps has uneven records.  One warp.
template <bool MASK>
__device__ __forceinline__ bool prepared_uneven(const FwdArgs& a, const Part& p) {
  const int at = first_prepared<MASK>(a, p);
  bool some = false;
#pragma unroll 1
  for (int t = p.t0 + (threadIdx.x & 31); t < p.t1; t += 32)
    some |= a.prep_exps[(int64_t)prepared_step<MASK>(a, p, at, t) * kPrepExps].w != 0;
  return __any_sync(~0u, some);
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const void* p) {
  if constexpr (N == 4) {
    const uint4 x = __ldg(static_cast<const uint4*>(p));
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = __ldg(static_cast<const uint2*>(p));
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = __ldg(static_cast<const uint32_t*>(p));
  }
}

// Whether a part has uneven records in steps with edges.  One warp: page ids of eight steps, a lane a
// record, then the parameters of four records at a time, those of a token's keys or values to a lane.
template <int D, bool MASK>
__device__ __forceinline__ bool look_for_uneven(const FwdArgs& a, const Part& p) {
  using R = Record<D>;
  constexpr int NG = D / kGroup, kAtOnce = 4;
  static_assert(R::kVp == R::kKp + 16 * R::kPar, "keys' and values' parameters lie together");
  const int lane = threadIdx.x & 31;
  bool some = false;
  if (p.t0 >= p.t1) return false;
  const Edges<MASK> edges(a, p);
  const Unread<MASK> un(a, p.r);
#pragma unroll 1
  for (int t0 = p.t0; t0 < p.t1; t0 += 32) {
    const int mine = t0 + lane;
    unsigned with = __ballot_sync(
        ~0u, mine < p.t1 && edges.in(tile_at<MASK, kStep>(a, mine, p.skip) * kStep));
#pragma unroll 1
    while (with) {
      int tile = 0, taken = 0;
#pragma unroll 1
      for (; with && taken < 8; ++taken, with &= with - 1) {
        const int t = tile_at<MASK, kStep>(a, t0 + __ffs(with) - 1, p.skip);
        if (lane / kRecs == taken) tile = t;
      }
      const int rec = tile * kRecs + lane % kRecs;
      const bool held = lane < taken * kRecs && !un.record(rec);
      uint32_t record = 0;
      if (held) record = cache_record(a, p.b, p.h, rec);
      const unsigned have = __ballot_sync(~0u, held);
#pragma unroll 1
      for (int k0 = 0; k0 < taken * kRecs; k0 += kAtOnce) {
        uint32_t w[kAtOnce][NG], read = 0;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const uint8_t* at = a.cache + (uint64_t)__shfl_sync(~0u, record, k0 + i) * R::kBytes +
                              R::kKp + lane * R::kPar;
          const int tok = 16 * __shfl_sync(~0u, rec, k0 + i) + (lane & 15);
#pragma unroll
          for (int g = 0; g < NG; ++g) w[i][g] = 0;
          if ((have >> (k0 + i) & 1) && !un.token(tok)) {
            load_words<NG>(w[i], at);
            read |= 1u << i;
          }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          uint32_t m = 0;
#pragma unroll
          for (int g = 0; g < NG; ++g) m = max_u16x2(m, magnitudes(w[i][g]));
          const uint32_t b = bound_of(m);
          const uint32_t of_keys = __reduce_max_sync(~0u, lane < 16 ? b : 0u);
          const uint32_t of_values = __reduce_max_sync(~0u, lane < 16 ? 0u : b);
          const int all = max((int)(lane < 16 ? of_keys : of_values) - 125, -90);
          some |= exponent_of_bound(b, read >> i & 1, all) < all - kEven;
        }
      }
    }
  }
  return __any_sync(~0u, some);
}

template <int D, bool MASK, bool PREP>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(FwdArgs a) {
  using C = Cfg<D>;
  constexpr int NG = C::NG;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars<D> bars;
  __shared__ __align__(16) StepExps exps[kExps];
  __shared__ uint4 tables[kDeqWarps][4 * NG];
  __shared__ Part parts[kParts];
  __shared__ bool uneven[kParts];  // whether they have uneven records
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
      mbar_init(&bars.looked[i], 1);
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
    for (int i = 0; i < kExps; ++i) mbar_init(&bars.x_full[i], 1), mbar_init(&bars.ev_full[i], kRecs);
    mbar_init(&bars.q_staged, 2 * kDeqWarps);
    mbar_init(&bars.q_copied, 2 * kDeqWarps);
    mbar_init(&bars.q_full, 2 * kDeqWarps);
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
  const bool prepared = PREP && a.prep_cap > 0 && a.prep_at[0];
  const int part_cost = prepared ? C::kPartCostPrep : kPartCost;
  {
    const Cut cut =
        cut_work<kThreads>(a, first, sums, (int64_t)kLeastSteps * kStep * a.d.G, [&](const Req& r) {
          return a.d.Hkv * cost_of<MASK>(a, r, part_cost).template before<MASK>(row_tiles(a, r));
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
  auto part_looked = [&](int k) {
    return mbar_wait(&bars.looked[k % kParts], (k / kParts) & 1, a.err);
  };
  auto part_read = [&](int k) { mbar_arrive(&bars.part_empty[k % kParts]); };

  if (warp >= kMmaWarp) {
    registers_down<kRegsRest>();
    // copies the key (0) or value (1) sides of a part's records, a warp each
    auto copy_sides = [&](int which, const Part& p) {
      const Unread<MASK> un(a, p.r);
      const int ring = which ? C::kRawV : C::kRawK;
      uint32_t record = 0, have = 0;
      for (int t = p.t0; t < p.t1; ++t, ++n) {
        const int slot = (t - p.t0) & 7;
        if (slot == 0) {  // the records of eight steps, one a lane
          const int rec = tile_at<MASK, kStep>(a, t + lane / kRecs, p.skip) * kRecs + lane % kRecs;
          const bool some = !un.record(rec);
          if (some) record = cache_record(a, p.b, p.h, rec);
          have = __ballot_sync(~0u, some);
        }
        const int st = n % ring;
        uint64_t* full = &bars.raw_full[which][st];
        ok = mbar_wait(&bars.raw_empty[which][st], ((n / ring) & 1) ^ 1, a.err);
        ok = __all_sync(~0u, ok);
        if (!ok) return;
        const uint32_t mine = have >> (slot * kRecs) & ((1u << kRecs) - 1);
        const uint32_t rec = __shfl_sync(~0u, record, slot * kRecs + (lane & 3));
        const int side = which ? C::kSideV : C::kSideK;
        if (lane == 0) mbar_arrive_expect_tx(full, __popc(mine) * side);
        __syncwarp();
        if (lane < kRecs && (mine >> lane & 1))
          copy_record(smem + (which ? C::kOffRawV : C::kOffRaw) + (st * kRecs + lane) * side,
                      a.cache + (uint64_t)rec * C::R::kBytes + (which ? C::R::kVp : 0), side, full);
      }
    };
    // copies the prepared key (0) or value (1) operands of a part's steps, a warp each: eight arrivals
    // a step, as from the dequantising warps
    auto copy_prepared = [&](int which, const Part& p) {
      const int at = first_prepared<MASK>(a, p);
      constexpr int kRing = C::kOpsK;
      static_assert(C::kOpsK == C::kOpsV && kDeqWarps == 8, "one rule for both");
      for (int t = p.t0; t < p.t1; ++t, ++n) {
        const int step = prepared_step<MASK>(a, p, at, t);
        const int op = n % kRing;
        uint64_t* full = which ? &bars.v_full[op] : &bars.k_full[op];
        ok = mbar_wait(which ? &bars.v_empty[op] : &bars.k_empty[op], ((n / kRing) & 1) ^ 1, a.err);
        ok = __all_sync(~0u, ok);
        if (!ok) return;
        if (lane == 0) {
          mbar_arrive_expect_tx(full, C::kK);
          copy_record(smem + (which ? C::kOffV : C::kOffK) + op * C::kK,
                      a.prep + ((int64_t)step * 2 + which) * C::kK, C::kK, full);
        } else if (lane < kDeqWarps) {
          mbar_arrive(full);
        } else if (lane == kDeqWarps && which == 0) {
          mbar_arrive_expect_tx(&bars.x_full[n % kExps], sizeof(exps[0]));
          copy_record(&exps[n % kExps], a.prep_exps + (int64_t)step * kPrepExps, sizeof(exps[0]),
                      &bars.x_full[n % kExps]);
        }
        __syncwarp();
      }
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
      bool whole = false;  // the row tiles that begin in the share, and nothing of others
      if constexpr (MASK) {
        if (a.window && !a.masks) {
          const int64_t unit = kStep * a.d.G;
          const int64_t tile = (int64_t)part_cost * a.d.G + window_steps(a, tile_tokens(a)) * unit;
          const int64_t more = divide(cut_s.share + tile - 1, tile) * tile - cut_s.share;
          whole = cut_s.share > tile && more <= kWholeMore * unit;
        }
        if (whole && w < w1) {
          const Part p = locate<MASK>(a, first, part_cost, w, INT64_MAX);
          // (a request without cached tokens has row tiles of one cost, without steps)
          const int64_t begin = p.start - (int64_t)(p.r.kv ? part_cost : kZeroCost) * a.d.G;
          if (begin < w) w = p.next;
        }
      }
      for (int k = 0; ok; ++k) {
        // (behind the share's end nothing begins in it)
        const Part p = locate<MASK>(a, first, part_cost, w, MASK && whole && w < w1 ? INT64_MAX : w1);
        ok = mbar_wait(&bars.part_empty[k % kParts], ((k / kParts) & 1) ^ 1, a.err);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        if (lane == 0) {
          parts[k % kParts] = p;
          mbar_arrive(&bars.part_full[k % kParts]);
        }
        if (!p.some) break;
        if (!prepared) {
          const bool look = look_for_uneven<D, MASK>(a, p);
          if (lane == 0) {
            uneven[k % kParts] = look;
            mbar_arrive(&bars.looked[k % kParts]);
          }
        }
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
        if (prepared) copy_prepared(which, p);
        else copy_sides(which, p);
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
      // (rows of outputs are only known to start on 16 bytes)
      const bool sectors =
          ((reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)(2 * a.out_stride)) & 31) == 0;
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
          if (!whole) {
            d = reinterpret_cast<uint8_t*>(a.part_o + (at + r) * D);
          } else if (row < p.r.qn * a.d.G) {
            const int tok = a.d.by_G(row);
            d = reinterpret_cast<uint8_t*>(a.out + (int64_t)(p.r.q0 + tok) * a.out_stride +
                                           (int64_t)(p.h * a.d.G + row - tok * a.d.G) * D);
          }
          if (whole) {
            uint32_t x[8];  // words 2c and 2c + 1, eight channels each
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int w = i / 4, m = 2 * (i % 4);
              const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(o[m][q + w]) * f,
                                                             __uint_as_float(o[m + 1][q + w]) * f);
              x[i] = *reinterpret_cast<const uint32_t*>(&y);
            }
            if (d) {
              d += 128 * g + 32 * c;
              if (sectors) {
                st_global_v8(d, x);
              } else {
                reinterpret_cast<uint4*>(d)[0] = make_uint4(x[0], x[1], x[2], x[3]);
                reinterpret_cast<uint4*>(d)[1] = make_uint4(x[4], x[5], x[6], x[7]);
              }
            }
          } else {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint32_t v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(__uint_as_float(o[i][q + w]) * f);
              st_global_v8(d + 256 * g + 64 * c + 32 * w, v);
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
      const Part& p = parts[k % kParts];  // (there until part_read)
      const bool some = p.some && p.t1 > p.t0;
      if (some) {
        // queries: every warp scales eight rows and moves a quarter of 32 on once the part before has
        // used its own
        QueryRows<D> q;
        q.load(a, p, 8 * (warp - kKeyWarp), row_exp[kq % kExps]);
        // prepared steps leave the room of the records free: all groups at once, the others there
        const int passes = prepared ? 1 : C::kQPasses;
#pragma unroll 1
        for (int pass = 0; pass < passes && ok; ++pass) {
          const int turn = kq * passes + pass;
          if (turn > 0)
            ok = __all_sync(~0u, mbar_wait(&bars.q_copied, (turn - 1) & 1, a.err));
          if (!ok) break;
          const bool all = C::kQPasses > 1 && prepared;
          q.store(ops, 8 * (warp - kKeyWarp), pass * C::kQGroups);
          if (all) q.store(ops + C::kOffRaw, 8 * (warp - kKeyWarp), C::kQGroups);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.q_staged);
          ok = mbar_wait(&bars.q_staged, turn & 1, a.err) &&
               (pass > 0 || kq == 0 || mbar_wait(&bars.q_free, (kq - 1) & 1, a.err));
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          tc_fence_after();
          copy_queries<D>(ops, tmem, pass * C::kQGroups, (warp - kKeyWarp) >> 2);
          if (all) copy_queries<D>(ops + C::kOffRaw, tmem, C::kQGroups, (warp - kKeyWarp) >> 2);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars.q_copied);
            if (pass == passes - 1) mbar_arrive(&bars.q_full);
          }
        }
        if (!ok) break;
      }
      if (due >= 0 && !(ok = outputs(due, kq - 1))) break;
      due = -1;
      if (!p.some) break;
      if (!some) {
        __syncwarp();
        if (lane == 0) part_read(k);
        continue;
      }
      due = k;
      ++kq;
      if (prepared) continue;  // (steps are counted by those who use them)
      const int t0 = p.t0, t1 = p.t1, skip = MASK ? p.skip : 0;
      const Unread<MASK> un(a, p.r);
      // loops for the keys' warps and for the values', of parts without uneven records and with them
      auto steps = [&](auto keys, auto look) {
        constexpr bool kKeys = decltype(keys)::value, kLook = decltype(look)::value;
        constexpr int kRing = kKeys ? C::kRawK : C::kRawV, kOps = kKeys ? C::kOpsK : C::kOpsV;
        for (int t = t0; t < t1; ++t, ++n) {
          const int st = n % kRing, op = n % kOps;
          const int tok = tile_at<MASK, kStep>(a, t, skip) * kStep + 8 * oct;
          ok = mbar_wait(&bars.raw_full[!kKeys][st], (n / kRing) & 1, a.err);
          ok = __all_sync(~0u, ok);
          if (!ok) return;
          StepExps* ex = &exps[n % kExps];
          if constexpr (kKeys)
            d.template keys<kLook>(ops + C::kOffRaw + st * kRecs * C::kSideK, oct, tok, un, ex);
          else  // (a value side begins with its parameters: R::kVp from where the record would)
            d.template values<kLook>(ops + C::kOffRawV + st * kRecs * C::kSideV - C::R::kVp, tables[oct],
                                     oct, tok, un, ex, &bars.ev_full[n % kExps]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.raw_empty[!kKeys][st]);
          ok = mbar_wait(kKeys ? &bars.k_empty[op] : &bars.v_empty[op], ((n / kOps) & 1) ^ 1, a.err);
          ok = __all_sync(~0u, ok);
          if (!ok) return;
          if constexpr (kKeys) d.store_keys(ops + C::kOffK + op * C::kK, oct);
          else d.store_values(ops + C::kOffV + op * C::kK, oct);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(kKeys ? &bars.k_full[op] : &bars.v_full[op]);
        }
      };
      ok = __all_sync(~0u, part_looked(k));
      if (!ok) break;
      const bool look = uneven[k % kParts];
      if (__builtin_expect(look, 0)) {
        if (is_key) steps(std::true_type(), std::true_type());
        else steps(std::false_type(), std::true_type());
      } else if (is_key) {
        steps(std::true_type(), std::false_type());
      } else {
        steps(std::false_type(), std::false_type());
      }
    }
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
      const int row = row0 + lane, tok = a.d.by_G(row);
      const bool on = row < rows_left;
      int lim = on ? seen_by(p.r, tok) : p.r.kv;
      const Edges<MASK> edges(a, p);
      RowView view(a, p, tok, MASK && on);
      if constexpr (MASK) {
        lim = 0;  // (tokens seen so far, of this part: whether there are any)
      }
      float m = -INFINITY, l = 0.f, unit = 0.f, most_ev = -INFINITY;
      // the steps of a part without uneven records, or with them
      auto steps = [&](auto has_uneven) {
        constexpr bool kLook = decltype(has_uneven)::value;
        for (int t = p.t0; t < p.t1 && ok; ++t, ++n) {
          ok = mbar_wait(&bars.s_full[n % C::kS], (n / C::kS) & 1, a.err) &&
               mbar_wait(prepared ? &bars.x_full[n % kExps] : &bars.ev_full[n % kExps], (n / kExps) & 1,
                         a.err);
          ok = __all_sync(~0u, ok);
          if (!ok) return;
          tc_fence_after();
          if (t == p.t0)  // back from the scaled queries' units to log2 units
            unit = pow2(row_exp[kq % kExps][tid]) * (64.f / 8192.f) * a.d.scale_log2;
          const uint32_t sb = lane_base + C::kColS + (n % C::kS) * kStep;
          bool apart = false;  // some weights enter the sum without their values' exponents
          if constexpr (kLook) apart = scores_of_tokens(sb, exps[n % kExps], unit);
          uint32_t s[kStep];
          tmem_ld32(sb, s);
          tmem_ld32(sb + 32, s + 32);
          Exps ex[kRecs];
#pragma unroll
          for (int r = 0; r < kRecs; ++r) {
            const float4 v = *reinterpret_cast<const float4*>(&exps[n % kExps].rec[r]);
            ex[r] = Exps{fmaxf(unit * v.x, kLook ? kLeastUp : kLeastUnit), v.y, v.z, 0u};
            if (kLook) ex[r].up_k = fminf(ex[r].up_k, kMostUp);
          }
          float least_ev = ex[0].ev;
          most_ev = fmaxf(most_ev, ex[0].ev);
#pragma unroll
          for (int r = 1; r < kRecs; ++r)
            least_ev = fminf(least_ev, ex[r].ev), most_ev = fmaxf(most_ev, ex[r].ev);
          const bool spread = least_ev < most_ev - kSpread;
          wait_ld32(s);
          wait_ld32(s + 32);
          if constexpr (MASK) {
            const int t0 = tile_at<MASK, kStep>(a, t, p.skip) * kStep;
            if (edges.in(t0)) {
              const uint64_t seen = view.seen(a, t0);
              const uint32_t half[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
#pragma unroll
              for (int i = 0; i < kStep; ++i)
                if (!(half[i / 32] >> (i % 32) & 1)) s[i] = 0xff800000u;  // -inf
              lim |= seen != 0;
            } else {
              lim = 1;
            }
          } else if (edges.in(t * kStep)) {
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
              if (!ok) return;
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
          if (__any_sync(~0u, spread || (kLook && apart))) {
            // with 2^ev weights may vanish that count in the sum: there they enter it without
#pragma unroll
            for (int r = 0; r < kRecs; ++r)
              if (kLook && marked(ex[r].down_v)) {
                const TokenBytes ev = token_bytes(exps[n % kExps].tok[1] + 16 * r);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  l += exp2_fast(fmaf(__uint_as_float(s[16 * r + i]), ex[r].up_k,
                                      ref + (ex[r].ev - (float)ev[i])));
                ex[r].down_v = 0.f;
              } else if (ex[r].ev < most_ev - kSpread) {
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
      };
      if (p.t1 > p.t0) {
        bool look;
        if (prepared) {
          look = prepared_uneven<MASK>(a, p);
        } else {
          ok = __all_sync(~0u, part_looked(k));
          if (!ok) break;
          // (written again for part k + kParts, once the outputs of this one are on their way)
          look = uneven[k % kParts];
        }
        if (__builtin_expect(look, 0)) steps(std::true_type());
        else steps(std::false_type());
      }
      if (!ok) break;
      if (p.tiles == 0) {  // rows that see nothing
        const uint64_t own =
            on ? reinterpret_cast<uint64_t>(a.out + (int64_t)(p.r.q0 + tok) * a.out_stride +
                                            (int64_t)(p.h * a.d.G + row - tok * a.d.G) * D)
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
// From this many row tiles per context, on average, it pays.  Row tiles of chunks, 8 contexts of 8000
// tokens, then 16 of 3000, prepared against not: 256 channels 8 row tiles 183 and 159, 141 and 134 us, 9 177
// and 176, 141 and 148, 10 187 and 192, 150 and 161; 128 channels 9 463 and 444, 380 and 368, 10 521 and 490,
// 408 and 410, 12 514 and 579, 449 and 478; 64 channels 4 115 and 110, 93 and 95, 5 131 and 133, 106 and
// 113, 6 147 and 156, 118 and 133.
template <int D>
constexpr int kPrepTiles = D == 64 ? 5 : D == 128 ? 11 : 9;
// The same behind a window, by a bound of the steps that its row tiles go over (for narrow windows twice
// what they do).  Prompts of 1200 over 3000, 4 of them, 256, 128 and 64 channels: a window of 16 51 and 58,
// 76 and 80, 68 and 79 us, of 600 78 and 104, 118 and 146, 97 and 131.
constexpr int kPrepTilesWindow = 7;
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

template <int D, bool MASK>
__global__ void __launch_bounds__(kPrepThreads, 2) attn_prepare_kernel(FwdArgs a) {
  using C = Cfg<D>;
  using P = PrepCfg<D>;
  using R = Record<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint4 tables[kDeqWarps][4 * C::NG];
  __shared__ __align__(16) StepExps exps;
  __shared__ int64_t sums[kPrepThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5;
  int64_t* first = reinterpret_cast<int64_t*>(smem + P::kFirst);
  pdl_wait();
  pdl_trigger();
  // (those that are gone over)
  auto steps_of = [&](const Req& r) {
    return (r.kv + kStep - 1) / kStep - (MASK ? skipped<kStep>(a, first_start(a, r)) : 0);
  };
  // Steps of each context in the lower half, steps of its row tiles (a causal prompt's on average)
  // in the upper one; both capped far above what is ever taken.
  constexpr int64_t kCap = 1 << 20;
  cut_work<kPrepThreads>(a, first, sums, 1, [&](const Req& r) {
    if (r.qn == 0) return (int64_t)0;
    const int64_t steps = a.d.Hkv * (int64_t)steps_of(r);
    int64_t all;
    if constexpr (MASK) {
      all = cost_of<MASK>(a, r, 0).template before<MASK>(row_tiles(a, r)) * a.d.Hkv / (kStep * a.d.G);
    } else {
      all = a.d.Hkv * (int64_t)((max(r.kv - r.qn / 2, 0) + kStep - 1) / kStep) * row_tiles(a, r);
    }
    return min(steps, kCap) | min(all, kCap) << 32;
  });
  const int64_t both = first[a.B];
  __syncthreads();  // every thread has it, and decides alike, before the sums lose their upper halves
  const int64_t steps = both & 0xffffffff;
  const int tiles = MASK && a.window ? kPrepTilesWindow : kPrepTiles<D>;
  const bool prepared = steps <= a.prep_cap && (both >> 32) >= tiles * steps;
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
    const Req r = load_req(a, b);
    const Unread<MASK> un(a, r);
    const int of = steps_of(r), h = (u - (int)first[b]) / of;
    const int t = tile_at<MASK, kStep>(a, (u - (int)first[b]) % of,
                                       MASK ? skipped<kStep>(a, first_start(a, r)) : 0);
    constexpr int kPieces = R::kBytes / 16;
    for (int i = tid; i < kRecs * kPieces; i += kPrepThreads) {
      const int rec = i / kPieces, at = i % kPieces * 16;
      if (un.record(t * kRecs + rec)) continue;
      const uint4 w = *reinterpret_cast<const uint4*>(
          a.cache + (uint64_t)cache_record(a, b, h, t * kRecs + rec) * R::kBytes + at);
      if (at < R::kVp)
        *reinterpret_cast<uint4*>(smem + P::kRaw + rec * C::kSideK + at) = w;
      if (at >= R::kVp)
        *reinterpret_cast<uint4*>(smem + P::kRawV + rec * C::kSideV + at - R::kVp) = w;
    }
    __syncthreads();
    Dequant<D> d;
    const int oct = warp & 7, tok = t * kStep + 8 * oct;
    if (warp < kDeqWarps) {
      d.template keys<true>(ops + P::kRaw, oct, tok, un, &exps);
      d.store_keys(ops, oct);
    } else {
      d.template values<true>(ops + P::kRawV - R::kVp, tables[oct], oct, tok, un, &exps, nullptr);
      d.store_values(ops + C::kK, oct);
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      store_operands(a.prep + (int64_t)u * 2 * C::kK, ops, 2 * C::kK);
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    } else if (tid >= 32 && tid < 32 + kPrepExps) {
      uint4 w = reinterpret_cast<const uint4*>(&exps)[tid - 32];
      if (tid == 32) {
        w.w = 0;
        for (int r = 0; r < kRecs; ++r) w.w |= marked(exps.rec[r].up_k) || marked(exps.rec[r].down_v);
      }
      a.prep_exps[(int64_t)u * kPrepExps + tid - 32] = w;
    }
    __syncthreads();
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <int D, bool MASK>
cudaError_t launch(const FwdArgs& a, int sms, cudaStream_t s) {
  // Calls that never form contexts first have a kernel without that: what it leaves out saves instruction
  // fetches (16 trees of 20 to 60 tokens 65 and 63 us, 8 requests of 64 tokens over 8000, 64 channels, 109
  // and 104).
  const int blocks = sms < kMaxBlocks ? sms : kMaxBlocks;
  const size_t smem = Cfg<D>::kSmem + (a.B + 1) * sizeof(int64_t);
  cudaError_t e;
  const int tiles = MASK && a.window ? kPrepTilesWindow : kPrepTiles<D>;
  if ((int64_t)a.max_q * a.d.G > (tiles - 1) * kRows) {
    e = launch_pdl(attn_prepare_kernel<D, MASK>, dim3(2 * sms), dim3(kPrepThreads),
                   PrepCfg<D>::kSmem + (a.B + 1) * sizeof(int64_t), s, a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(attn_prefill_kernel<D, MASK, true>, dim3(blocks), dim3(kThreads), smem, s, a);
  } else {
    e = launch_pdl(attn_prefill_kernel<D, MASK, false>, dim3(blocks), dim3(kThreads), smem, s, a);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_join_kernel<D, kRows>, dim3(8 * sms), dim3(kJoinThreads), 0, s, a, blocks);
}

template <bool MASK>
cudaError_t launch_any(const FwdArgs& a, int sms, cudaStream_t s) {
  if (a.d.D == 256) return launch<256, MASK>(a, sms, s);
  if (a.d.D == 128) return launch<128, MASK>(a, sms, s);
  return launch<64, MASK>(a, sms, s);
}

template <int D, bool MASK>
cudaError_t prepare() {
  constexpr cudaFuncAttribute kMost = cudaFuncAttributeMaxDynamicSharedMemorySize;
  constexpr int kFirsts = (kMaxRequests + 1) * (int)sizeof(int64_t), kSmem = Cfg<D>::kSmem + kFirsts;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(attn_prepare_kernel<D, MASK>, kMost, PrepCfg<D>::kSmem + kFirsts)) !=
          cudaSuccess ||
      (e = cudaFuncSetAttribute(attn_prefill_kernel<D, MASK, true>, kMost, kSmem)) != cudaSuccess)
    return e;
  return cudaFuncSetAttribute(attn_prefill_kernel<D, MASK, false>, kMost, kSmem);
}

template <bool MASK>
cudaError_t prepare_all() {
  cudaError_t e;
  if ((e = prepare<64, MASK>()) != cudaSuccess) return e;
  if ((e = prepare<128, MASK>()) != cudaSuccess) return e;
  return prepare<256, MASK>();
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
  const cudaError_t e = prepare_all<false>();
  return e != cudaSuccess ? e : prepare_all<true>();
}

cudaError_t launch_attn_prefill(const FwdArgs& a, int sms, cudaStream_t s) {
  return a.window || a.masks ? launch_any<true>(a, sms, s) : launch_any<false>(a, sms, s);
}

}  // namespace moe
