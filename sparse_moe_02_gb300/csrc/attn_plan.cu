// attn_plan: block tables and slot maps of one step from the requests' lengths (include/attn.h
// states the rule).
//
// Two prefix sums over the requests give each its first token and its first entry of the free
// list; every token then finds its request by binary search over the first tokens.  The work is
// a few bytes per token, so the launch is bound by latency: every block repeats the sums (B
// lengths, from L2) instead of waiting for one block to publish them, takes its share of the
// tokens and requests, and computes a new page's id from the free list itself rather than from a
// table entry that another block writes.  The last block to finish (a ticket) writes the cursor,
// which the others read: cursor_out may therefore be the cursor.
//
// Measured (inside a CUDA graph): 64 requests of one token 4.3 us, 301 requests of up to 400 tokens with
// pages of 16 5.4 us.  A block takes 1024 tokens, so one block serves token steps without the ticket.
#include "attn.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTokensPerBlock = 1024;
constexpr int kMaxLen = 1 << 30;

// Inclusive prefix sum over the block's threads; *total gets the block's sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int64_t x = warp_sums[w];
    if (w < warp) before += x;
    all += x;
  }
  __syncthreads();
  *total = all;
  return v + before;
}

__global__ void __launch_bounds__(kThreads) attn_plan_kernel(PlanArgs a) {
  // per request: first token, cached tokens, first free-list entry (-1: refused)
  extern __shared__ int smem[];
  int* first = smem;              // [B + 1]
  int* ctx = first + a.B + 1;     // [B]
  int* entry = ctx + a.B;         // [B]
  int* need = entry + a.B;        // [B]
  __shared__ int64_t warp_sums[kWarps];
  __shared__ int taken, code, last;
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if (tid == 0) taken = 0, code = 0;
  __syncthreads();
  const int cursor = *a.cursor;
  // nothing can be taken behind a cursor that is not an index of the list
  const int64_t avail = cursor < 0 ? 0 : (int64_t)a.n_free - cursor;
  const int page = 1 << a.page_shift;

  int64_t tokens = 0, pages = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int c = 0, n = 0;
    bool bad = false;
    if (b < a.B) {
      c = a.ctx[b];
      n = a.news[b];
      bad = c < 0 || n < 0 || c > kMaxLen || n > kMaxLen;
      if (c < 0 || c > kMaxLen) c = 0;
      n = min(max(n, 0), kMaxLen);
    }
    int64_t sum;
    const int64_t end = tokens + block_scan(n, warp_sums, &sum);
    tokens += sum;
    const int before = (c + page - 1) >> a.page_shift;
    const int after = (int)(((int64_t)c + n + page - 1) >> a.page_shift);
    bad = bad || end > a.T || after > a.table_width;
    const int want = (b < a.B && !bad) ? after - before : 0;
    const int64_t pend = pages + block_scan(want, warp_sums, &sum);
    pages += sum;
    if (b < a.B) {
      const bool lack = want > 0 && pend > avail;
      first[b] = (int)min(end - n, (int64_t)a.T);
      ctx[b] = c;
      need[b] = lack ? 0 : want;
      // a request that needs no page is served whatever the list holds
      entry[b] = bad || lack ? -1 : want > 0 ? (int)(cursor + pend - want) : 0;
      if (want > 0 && !lack) atomicMax(&taken, (int)pend);
      if (lack) atomicMax(&code, kDevErrNoMemory);
      if (bad) atomicMax(&code, kDevErrArg);
    }
  }
  if (tid == 0) first[a.B] = (int)min(tokens, (int64_t)a.T);
  __syncthreads();

  if (blockIdx.x == 0) {
    for (int b = tid; b <= a.B; b += kThreads) {
      a.q_offsets[b] = first[b];
      if (b < a.B) {
        const int n = a.news[b];
        a.kv_lens[b] = entry[b] < 0 ? 0 : ctx[b] + n;
      }
    }
    if (tid == 0 && code) record_error(a.err, code);
  }
  // the new table entries, a warp per request
  for (int b = blockIdx.x * kWarps + (tid >> 5); b < a.B; b += gridDim.x * kWarps) {
    const int before = (ctx[b] + page - 1) >> a.page_shift;
    int32_t* row = a.table + (int64_t)b * a.table_width + before;
    for (int j = tid & 31; j < need[b]; j += 32) row[j] = a.free_pages[entry[b] + j];
  }
  // positions and slots of the block's tokens
  for (int t = blockIdx.x * kThreads + tid; t < a.T; t += gridDim.x * kThreads) {
    int pos = 0, slot = -1;
    if (t < first[a.B]) {
      int lo = 0, hi = a.B;  // first[lo] <= t < first[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= t) lo = mid;
        else hi = mid;
      }
      pos = ctx[lo] + t - first[lo];
      if (entry[lo] >= 0) {
        const int before = (ctx[lo] + page - 1) >> a.page_shift;
        const int k = pos >> a.page_shift;
        const int id = k >= before ? a.free_pages[entry[lo] + k - before]
                                   : a.table[(int64_t)lo * a.table_width + k];
        const int64_t s = ((int64_t)id << a.page_shift) + (pos & (page - 1));
        slot = id < 0 || s > 0x7fffffff ? -1 : (int)s;
      }
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
  // every thread of the block has read the cursor: the last block may write it
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    last = gridDim.x == 1 || atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
    if (last) {
      if (gridDim.x > 1) *a.ticket = 0;
      *a.cursor_out = cursor + taken;
    }
  }
}

constexpr size_t plan_smem(int B) { return (size_t)(4 * B + 1) * sizeof(int); }
static_assert(plan_smem(kMaxRequests) + 1024 <= 48 << 10, "what a kernel may have without asking");

}  // namespace

cudaError_t launch_attn_plan(const PlanArgs& a, int sms, cudaStream_t s) {
  int grid = (a.T + kTokensPerBlock - 1) / kTokensPerBlock;
  grid = grid < 1 ? 1 : grid > sms ? sms : grid;
  return launch_pdl(attn_plan_kernel, dim3(grid), dim3(kThreads), plan_smem(a.B), s, a);
}

}  // namespace moe
