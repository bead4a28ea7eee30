// Internal interface of the attention step (include/attn.h): argument blocks, launchers, and the
// arithmetic of a cached row that the kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "layer.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kGroup = 64;        // channels per scale and bias
// Requests of a call at most.  The kernels' shared-memory limits are set for as many whatever a handle
// asks for: they belong to the functions, which the handles of a process share.
constexpr int kMaxRequests = 1024;
// Cached rows hold magnitudes below this only (larger ones count as not finite): the kernels'
// powers of two of a record's bound, 2^119 at most, and their inverses stay normal fp32 numbers.
constexpr float kLargest = 8.307675e34f;  // 2^116
// Least unit of a score (the smallest normal fp32): masked scores are -inf times it, which a unit that
// vanished, of a zero query row over empty or zero keys, would make NaN.
constexpr float kLeastUnit = 1.17549435e-38f;  // 2^-126
constexpr int kDevErrNoMemory = 7;
constexpr int kDevErrArg = 1;

struct AttnDims {
  int Hq, Hkv, G, D;
  int page_shift;  // log2 of the page size
  int n_pages;
  float scale_log2;  // softmax scale * log2(e)
};

// A cache record: 16 tokens of one head.
template <int D>
struct Record {
  static constexpr int kRow = D / 2;            // code bytes of a row
  static constexpr int kPar = 4 * (D / kGroup);  // parameter bytes of a row
  static constexpr int kKp = 16 * kRow;
  static constexpr int kVp = kKp + 16 * kPar;
  static constexpr int kV = kVp + 16 * kPar;
  static constexpr int kBytes = kV + 16 * kRow;
};

// Position (in units of D/64 words) of word j of every group in the row of slot s.
__host__ __device__ __forceinline__ int row_swz(int s) { return ((s & 3) << 1) ^ (s & 4); }

// Larger of each 16-bit half, unsigned: on the magnitudes of bf16 pairs their order.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A device-side error: of several the largest value stays.
__device__ __forceinline__ void record_error(int* err, int code) { atomicMax(err, code); }

// One request of a step as the kernels see it: its rows, and its lengths moved into range.
struct Req {
  int q0, qn, kv;
};

struct FwdArgs {
  const __nv_bfloat16* q;
  int64_t q_stride;
  __nv_bfloat16* out;
  int64_t out_stride;
  const uint8_t* cache;
  const int32_t* table;
  int table_width;
  const int32_t* q_off;
  const int32_t* kv_lens;
  int B, T, max_q;
  AttnDims d;
  float* part_o;     // partial outputs: [slots][columns][D] fp32
  float2* part_ml;   // their softmax reference and sum: [slots][columns]
  int4* desc;        // [2 * blocks]: (parts, head, row tile, first row), (rows) of shared contexts
  // Contexts as MMA operands (attn_prefill.cu): whether they are there and, from [1] on, each
  // request's first step; room for prep_cap steps, 0 where a call does not form them.
  int* prep_at;
  int prep_cap;
  uint8_t* prep;      // [steps]: a step's key operand, then its value operand
  uint4* prep_exps;   // [steps][4]: exponents of the records
  int* err;
};

__device__ __forceinline__ Req load_req(const FwdArgs& a, int b) {
  const int lo = a.q_off[b], hi = a.q_off[b + 1], kv = a.kv_lens[b];
  Req r;
  r.q0 = min(max(lo, 0), a.T);
  r.qn = min(max(hi, r.q0), a.T) - r.q0;
  if (r.qn > a.max_q) r.qn = a.max_q;
  const int64_t cap = (int64_t)a.table_width << a.d.page_shift;
  r.kv = (int)min((int64_t)max(kv, 0), cap);
  return r;
}

// Whether load_req had to move something into range.
__device__ __forceinline__ bool req_out_of_range(const FwdArgs& a, int b) {
  const int lo = a.q_off[b], hi = a.q_off[b + 1], kv = a.kv_lens[b];
  return lo < 0 || hi < lo || hi > a.T || hi - lo > a.max_q || kv < 0 ||
         kv > ((int64_t)a.table_width << a.d.page_shift);
}

// Records the cudaError_t for moe_last_cuda_error and returns the status.
int record_cuda_status(cudaError_t e);

struct PlanArgs {
  int32_t* table;
  int table_width;
  const int32_t* ctx;
  const int32_t* news;
  int B;
  const int32_t* free_pages;
  int n_free;
  const int32_t* cursor;
  int T;
  int32_t *q_offsets, *kv_lens, *positions, *slots, *cursor_out;
  int page_shift;
  int* ticket;  // blocks that are done; back to 0 when the launch ends
  int* err;
};

cudaError_t launch_attn_plan(const PlanArgs& a, int sms, cudaStream_t s);

struct RopeArgs {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *q_out, *k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  const int32_t* positions;
  const __nv_bfloat16 *qw, *kw;
  float eps;
  const float* cos_sin;
  int n_positions, rot, T, Hq, Hkv;
  int* err;
};

cudaError_t launch_attn_qk_norm_rope(const RopeArgs& a, int D, bool interleaved, int sms,
                                     cudaStream_t s);

struct RowsArgs {
  const __nv_bfloat16 *k, *v;  // append: inputs
  __nv_bfloat16 *ko, *vo;      // read: outputs
  int64_t k_stride, v_stride;
  const int32_t* slots;
  int T, Hkv, page_shift;
  int64_t n_slots;
  uint8_t* cache;
  int* err;
};

cudaError_t launch_attn_append(const RowsArgs& a, int D, cudaStream_t s);
cudaError_t launch_attn_read(const RowsArgs& a, int D, cudaStream_t s);

// Attention of few query rows per key/value head and request (n_b G <= 32): attn_decode.cu.  Its time
// grows with every 8 (128 and 64 channels: 16) rows, the other kernel's with every 128: 8 requests of
// 5 tokens, G = 4, took 27 us here and 44 there, of 8 tokens 49 and 59.
constexpr int kDecodeRows = 32;
cudaError_t prepare_attn_decode_kernels();
int attn_part_slots(int sms);  // partial results of a launch, of either kernel
cudaError_t launch_attn_decode(const FwdArgs& a, int max_kv, int sms, cudaStream_t s);

// Attention of more rows, and of batches that hold any such request: attn_prefill.cu.
cudaError_t prepare_attn_prefill_kernels();
size_t attn_prefill_part_floats(int D);  // fp32 of a partial result, the larger of the kernels'
int attn_prep_steps(const AttnDims& d, int max_requests);  // of contexts held as operands
size_t attn_prep_step_bytes(int D);                        // of one, without its exponents
cudaError_t launch_attn_prefill(const FwdArgs& a, int sms, cudaStream_t s);

}  // namespace moe
