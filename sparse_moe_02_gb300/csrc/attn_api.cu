// The C ABI of the attention step (declared and documented in include/attn.h): argument checks,
// the handle's workspace, and the launches.  Nothing here synchronises with the host except
// attn_create, attn_destroy and attn_get_device_error.
#include <cmath>
#include <new>

#include "attn.cuh"
#include "attn.h"

using moe::record_cuda_status;

struct attn_handle_s {
  attn_config cfg;
  moe::AttnDims d;
  int sms = 0;
  void* ws = nullptr;
  float* part_o = nullptr;
  float2* part_ml = nullptr;
  int4* desc = nullptr;
  uint8_t* prep = nullptr;
  uint4* prep_exps = nullptr;
  int* prep_at = nullptr;
  int prep_cap = 0;
  int* ticket = nullptr;
  int* err = nullptr;
};

namespace {

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

constexpr int kMaxTokens = 1 << 20;

int check_config(const attn_config* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->n_q_heads < 1 || c->n_kv_heads < 1 || c->head_dim < 1 || c->page_size < 1 ||
      c->n_pages < 1 || c->max_requests < 1)
    return MOE_ERR_INVALID_ARG;
  if (!(c->scale >= 0.f) || std::isinf(c->scale)) return MOE_ERR_INVALID_ARG;
  if (c->n_q_heads % c->n_kv_heads || c->n_q_heads / c->n_kv_heads > 16 || c->n_kv_heads > 128)
    return MOE_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 &&
      c->page_size != 256)
    return MOE_ERR_UNSUPPORTED;
  if ((int64_t)c->n_pages * c->page_size > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  if (c->max_requests > moe::kMaxRequests) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Rows of `width` channels a token, `stride` apart.
int check_rows(const void* p, int64_t stride, int64_t width) {
  if (!p || stride < width) return MOE_ERR_INVALID_ARG;
  if (off16(p) || stride % 8) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

int check_tokens(int T) {
  return T < 0 ? MOE_ERR_INVALID_ARG : T > kMaxTokens ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int check_cache(const void* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  return (reinterpret_cast<uintptr_t>(c) & 127u) ? MOE_ERR_ALIGNMENT : MOE_OK;
}

moe::RowsArgs rows_args(attn_handle h, const void* cache, const int32_t* slots, int T) {
  moe::RowsArgs a{};
  a.slots = slots;
  a.T = T;
  a.Hkv = h->d.Hkv;
  a.page_shift = h->d.page_shift;
  a.n_slots = (int64_t)h->d.n_pages << h->d.page_shift;
  a.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  a.err = h->err;
  return a;
}

moe::RopeArgs rope_args(attn_handle h, const void* q, int64_t q_stride, const void* k,
                        int64_t k_stride, const int32_t* positions, const void* q_weight,
                        const void* k_weight, float eps, const float* cos_sin, int n_positions,
                        int rotary_dim, int T, void* q_out, int64_t q_out_stride) {
  moe::RopeArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.positions = positions;
  a.qw = static_cast<const __nv_bfloat16*>(q_weight);
  a.kw = static_cast<const __nv_bfloat16*>(k_weight);
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.n_positions = n_positions;
  a.rot = rotary_dim;
  a.T = T;
  a.Hq = h->d.Hq;
  a.Hkv = h->d.Hkv;
  a.err = h->err;
  return a;
}

// Masks of drafted tokens (NULL: none to check but the sizes).
int check_masks(int max_q_len, const uint32_t* masks, int mask_words) {
  if (max_q_len < 1 || mask_words < 1) return MOE_ERR_INVALID_ARG;
  if (max_q_len > moe::kMaxDrafts || mask_words > moe::kMaxDrafts / 32 ||
      max_q_len > 32 * mask_words)
    return MOE_ERR_UNSUPPORTED;
  return off4(masks) ? MOE_ERR_ALIGNMENT : MOE_OK;
}

constexpr int kMostTokens = 1 << 30;  // of a window: its bounds stay in 32 bits

// The checks and arguments that both forms of the forward call share; *none: nothing to do.
int forward_args(attn_handle h, const void* q, int64_t q_stride, const void* cache,
                 const int32_t* block_table, int table_width, const int32_t* q_offsets,
                 const int32_t* kv_lens, int B, int T, int max_q_len, int max_kv_len, void* out,
                 int64_t out_stride, moe::FwdArgs* args, bool* none) {
  *none = false;
  if (!h || B < 0 || table_width < 0 || max_q_len < 1 || max_kv_len < 0)
    return MOE_ERR_INVALID_ARG;
  int st = check_tokens(T);
  if (st) return st;
  if (B > h->cfg.max_requests) return MOE_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) {
    *none = true;
    return MOE_OK;
  }
  const int64_t w = (int64_t)h->d.Hq * h->d.D;
  if ((st = check_rows(q, q_stride, w)) || (st = check_rows(out, out_stride, w)) ||
      (st = check_cache(cache)))
    return st;
  if (!q_offsets || !kv_lens || (table_width > 0 && !block_table)) return MOE_ERR_INVALID_ARG;
  if (off4(q_offsets) || off4(kv_lens) || off4(block_table)) return MOE_ERR_ALIGNMENT;
  moe::FwdArgs& a = *args;
  a = moe::FwdArgs{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_stride;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.out_stride = out_stride;
  a.cache = static_cast<const uint8_t*>(cache);
  a.table = block_table;
  a.table_width = table_width;
  a.q_off = q_offsets;
  a.kv_lens = kv_lens;
  a.B = B;
  a.T = T;
  a.max_q = max_q_len < T ? max_q_len : T;
  a.d = h->d;
  a.part_o = h->part_o;
  a.part_ml = h->part_ml;
  a.desc = h->desc;
  a.prep_at = h->prep_at;
  a.prep_cap = h->prep_cap;
  a.prep = h->prep;
  a.prep_exps = h->prep_exps;
  a.err = h->err;
  return MOE_OK;
}

int launch_forward(attn_handle h, const moe::FwdArgs& a, int max_kv_len, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return record_cuda_status(
      a.max_q * h->d.G <= moe::kDecodeRows ? moe::launch_attn_decode(a, max_kv_len, h->sms, s)
                                           : moe::launch_attn_prefill(a, h->sms, s));
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

extern "C" {

int attn_create(const attn_config* cfg, attn_handle* out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  int st = check_config(cfg);
  if (st) return st;
  int dev = 0, sms = 0;
  if ((st = record_cuda_status(cudaGetDevice(&dev)))) return st;
  if ((st = record_cuda_status(
           cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev))))
    return st;
  if ((st = record_cuda_status(moe::prepare_attn_decode_kernels()))) return st;
  if ((st = record_cuda_status(moe::prepare_attn_prefill_kernels()))) return st;

  attn_handle h = new (std::nothrow) attn_handle_s;
  if (!h) return MOE_ERR_NO_MEMORY;
  h->cfg = *cfg;
  h->sms = sms;
  h->d.Hq = cfg->n_q_heads;
  h->d.Hkv = cfg->n_kv_heads;
  h->d.G = cfg->n_q_heads / cfg->n_kv_heads;
  h->d.D = cfg->head_dim;
  h->d.by_G = moe::Divide(h->d.G);
  h->d.page_shift = 0;
  while ((1 << h->d.page_shift) < cfg->page_size) ++h->d.page_shift;
  h->d.n_pages = cfg->n_pages;
  const double scale = cfg->scale > 0.f ? cfg->scale : 1.0 / std::sqrt((double)cfg->head_dim);
  h->d.scale_log2 = (float)(scale * 1.4426950408889634);

  const size_t slots = moe::attn_part_slots(sms);
  const size_t o_bytes =
      round256(slots * moe::attn_prefill_part_floats(cfg->head_dim) * sizeof(float));
  const size_t ml_bytes = round256(slots * 128 * sizeof(float2));
  const size_t desc_bytes = round256(slots * sizeof(int4));
  h->prep_cap = moe::attn_prep_steps(h->d, cfg->max_requests);
  const size_t prep_bytes = round256(h->prep_cap * moe::attn_prep_step_bytes(cfg->head_dim));
  const size_t exps_bytes = round256((size_t)h->prep_cap * moe::kPrepExps * sizeof(uint4));
  const size_t at_bytes = round256((1 + (size_t)cfg->max_requests) * sizeof(int));
  const size_t zeroed = 2 * sizeof(int);  // the plan's ticket, the error word
  const size_t bytes =
      o_bytes + ml_bytes + desc_bytes + prep_bytes + exps_bytes + at_bytes + zeroed;
  cudaError_t e = cudaMalloc(&h->ws, bytes);
  if (e == cudaErrorMemoryAllocation) {
    cudaGetLastError();
    delete h;
    return MOE_ERR_NO_MEMORY;
  }
  if (e == cudaSuccess) {
    char* p = static_cast<char*>(h->ws);
    h->part_o = reinterpret_cast<float*>(p);
    h->part_ml = reinterpret_cast<float2*>(p += o_bytes);
    h->desc = reinterpret_cast<int4*>(p += ml_bytes);
    h->prep = reinterpret_cast<uint8_t*>(p += desc_bytes);
    h->prep_exps = reinterpret_cast<uint4*>(p += prep_bytes);
    h->prep_at = reinterpret_cast<int*>(p += exps_bytes);
    h->ticket = reinterpret_cast<int*>(p += at_bytes);
    h->err = h->ticket + 1;
    e = cudaMemset(h->ticket, 0, zeroed);
    // the handle may be used on a stream that does not order itself behind the default one
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
  if (e != cudaSuccess) {
    st = record_cuda_status(e);
    if (h->ws) cudaFree(h->ws);
    delete h;
    return st;
  }
  *out = h;
  return MOE_OK;
}

int attn_destroy(attn_handle h) {
  if (!h) return MOE_OK;
  int st = record_cuda_status(cudaDeviceSynchronize());
  const int st2 = record_cuda_status(cudaFree(h->ws));
  delete h;
  return st ? st : st2;
}

int attn_get_device_error(attn_handle h, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int v = 0, st;
  if ((st = record_cuda_status(cudaMemcpyAsync(&v, h->err, sizeof(int), cudaMemcpyDeviceToHost, s))))
    return st;
  if ((st = record_cuda_status(cudaStreamSynchronize(s)))) return st;
  if (v != 0) {
    if ((st = record_cuda_status(cudaMemsetAsync(h->err, 0, sizeof(int), s)))) return st;
    if ((st = record_cuda_status(cudaStreamSynchronize(s)))) return st;
  }
  return v;
}

int attn_plan(attn_handle h, int32_t* block_table, int table_width, const int32_t* ctx_lens,
              const int32_t* new_lens, int B, const int32_t* free_pages, int n_free,
              const int32_t* cursor, int T, int32_t* q_offsets, int32_t* kv_lens,
              int32_t* positions, int32_t* slots, int32_t* cursor_out, void* stream) {
  if (!h || B < 0 || table_width < 0 || n_free < 0) return MOE_ERR_INVALID_ARG;
  int st = check_tokens(T);
  if (st) return st;
  if (B > h->cfg.max_requests) return MOE_ERR_UNSUPPORTED;
  if (!q_offsets || !cursor || !cursor_out) return MOE_ERR_INVALID_ARG;
  if (B > 0 && (!ctx_lens || !new_lens || !kv_lens)) return MOE_ERR_INVALID_ARG;
  if (B > 0 && table_width > 0 && !block_table) return MOE_ERR_INVALID_ARG;
  if (n_free > 0 && !free_pages) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!positions || !slots)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)block_table, (const void*)ctx_lens, (const void*)new_lens,
                        (const void*)free_pages, (const void*)cursor, (const void*)q_offsets,
                        (const void*)kv_lens, (const void*)positions, (const void*)slots,
                        (const void*)cursor_out})
    if (off4(p)) return MOE_ERR_ALIGNMENT;
  moe::PlanArgs a{block_table, table_width, ctx_lens, new_lens, B, free_pages, n_free, cursor, T,
                  q_offsets, kv_lens, positions, slots, cursor_out, h->d.page_shift, h->ticket,
                  h->err};
  return record_cuda_status(moe::launch_attn_plan(a, h->sms, static_cast<cudaStream_t>(stream)));
}

int attn_qk_norm_rope(attn_handle h, const void* q, int64_t q_stride, const void* k,
                      int64_t k_stride, const int32_t* positions, const void* q_weight,
                      const void* k_weight, float eps, const float* cos_sin, int n_positions,
                      int rotary_dim, int interleaved, int T, void* q_out, int64_t q_out_stride,
                      void* k_out, int64_t k_out_stride, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  int st = check_tokens(T);
  if (st) return st;
  if (rotary_dim < 0 || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (rotary_dim % 16 || rotary_dim > h->d.D) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!q_weight || !k_weight) return MOE_ERR_INVALID_ARG;
  if (rotary_dim > 0 && (!positions || !cos_sin || n_positions < 1)) return MOE_ERR_INVALID_ARG;
  const int64_t qw = (int64_t)h->d.Hq * h->d.D, kw = (int64_t)h->d.Hkv * h->d.D;
  if ((st = check_rows(q, q_stride, qw)) || (st = check_rows(k, k_stride, kw)) ||
      (st = check_rows(q_out, q_out_stride, qw)) || (st = check_rows(k_out, k_out_stride, kw)))
    return st;
  if (off16(q_weight) || off16(k_weight) || (rotary_dim > 0 && (off16(cos_sin) || off4(positions))))
    return MOE_ERR_ALIGNMENT;
  moe::RopeArgs a = rope_args(h, q, q_stride, k, k_stride, positions, q_weight, k_weight, eps,
                              cos_sin, n_positions, rotary_dim, T, q_out, q_out_stride);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.k_out_stride = k_out_stride;
  return record_cuda_status(moe::launch_attn_qk_norm_rope(
      a, h->d.D, interleaved != 0, h->sms, static_cast<cudaStream_t>(stream)));
}

int attn_qk_norm_rope_append(attn_handle h, const void* q, int64_t q_stride, const void* k,
                             int64_t k_stride, const void* v, int64_t v_stride,
                             const int32_t* positions, const int32_t* slots, const void* q_weight,
                             const void* k_weight, float eps, const float* cos_sin,
                             int n_positions, int rotary_dim, int interleaved, int T, void* q_out,
                             int64_t q_out_stride, void* cache, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  int st = check_tokens(T);
  if (st) return st;
  if (rotary_dim < 0 || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (rotary_dim % 16 || rotary_dim > h->d.D) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!slots || !q_weight != !k_weight) return MOE_ERR_INVALID_ARG;
  if (rotary_dim > 0 && (!positions || !cos_sin || n_positions < 1)) return MOE_ERR_INVALID_ARG;
  const int64_t qw = (int64_t)h->d.Hq * h->d.D, kw = (int64_t)h->d.Hkv * h->d.D;
  if ((st = check_rows(q, q_stride, qw)) || (st = check_rows(k, k_stride, kw)) ||
      (st = check_rows(v, v_stride, kw)) || (st = check_rows(q_out, q_out_stride, qw)) ||
      (st = check_cache(cache)))
    return st;
  if (off16(q_weight) || off16(k_weight) || off4(slots) ||
      (rotary_dim > 0 && (off16(cos_sin) || off4(positions))))
    return MOE_ERR_ALIGNMENT;
  moe::RopeArgs r = rope_args(h, q, q_stride, k, k_stride, positions, q_weight, k_weight, eps,
                              cos_sin, n_positions, rotary_dim, T, q_out, q_out_stride);
  moe::RowsArgs a = rows_args(h, cache, slots, T);
  a.k = r.k;
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  return record_cuda_status(moe::launch_attn_rope_append(
      r, a, h->d.D, interleaved != 0, h->sms, static_cast<cudaStream_t>(stream)));
}

int attn_kv4_append(attn_handle h, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, const int32_t* slots, int T, void* cache, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  int st = check_tokens(T);
  if (st) return st;
  if (T == 0) return MOE_OK;
  const int64_t w = (int64_t)h->d.Hkv * h->d.D;
  if ((st = check_rows(k, k_stride, w)) || (st = check_rows(v, v_stride, w)) ||
      (st = check_cache(cache)))
    return st;
  if (!slots) return MOE_ERR_INVALID_ARG;
  if (off4(slots)) return MOE_ERR_ALIGNMENT;
  moe::RowsArgs a = rows_args(h, cache, slots, T);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  return record_cuda_status(
      moe::launch_attn_append(a, h->d.D, static_cast<cudaStream_t>(stream)));
}

int attn_kv4_read(attn_handle h, const void* cache, const int32_t* slots, int T, void* k,
                  int64_t k_stride, void* v, int64_t v_stride, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  int st = check_tokens(T);
  if (st) return st;
  if (T == 0) return MOE_OK;
  const int64_t w = (int64_t)h->d.Hkv * h->d.D;
  if ((st = check_rows(k, k_stride, w)) || (st = check_rows(v, v_stride, w)) ||
      (st = check_cache(cache)))
    return st;
  if (!slots) return MOE_ERR_INVALID_ARG;
  if (off4(slots)) return MOE_ERR_ALIGNMENT;
  moe::RowsArgs a = rows_args(h, cache, slots, T);
  a.ko = static_cast<__nv_bfloat16*>(k);
  a.vo = static_cast<__nv_bfloat16*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  return record_cuda_status(
      moe::launch_attn_read(a, h->d.D, static_cast<cudaStream_t>(stream)));
}

int attn_kv4_forward(attn_handle h, const void* q, int64_t q_stride, const void* cache,
                     const int32_t* block_table, int table_width, const int32_t* q_offsets,
                     const int32_t* kv_lens, int B, int T, int max_q_len, int max_kv_len,
                     void* out, int64_t out_stride, void* stream) {
  moe::FwdArgs a;
  bool none;
  const int st = forward_args(h, q, q_stride, cache, block_table, table_width, q_offsets, kv_lens, B,
                              T, max_q_len, max_kv_len, out, out_stride, &a, &none);
  if (st || none) return st;
  return launch_forward(h, a, max_kv_len, stream);
}

int attn_kv4_forward_masked(attn_handle h, const void* q, int64_t q_stride, const void* cache,
                            const int32_t* block_table, int table_width, const int32_t* q_offsets,
                            const int32_t* kv_lens, int B, int T, int max_q_len, int max_kv_len,
                            int window, int sinks, const uint32_t* masks, int mask_words,
                            void* out, int64_t out_stride, void* stream) {
  if (window < 0 || sinks < 0) return MOE_ERR_INVALID_ARG;
  if (window > kMostTokens || sinks > kMostTokens) return MOE_ERR_UNSUPPORTED;
  if (masks) {
    int st = check_masks(max_q_len, masks, mask_words);
    if (st) return st;
    if (window > 0 && max_q_len > window) return MOE_ERR_UNSUPPORTED;
  }
  moe::FwdArgs a;
  bool none;
  const int st = forward_args(h, q, q_stride, cache, block_table, table_width, q_offsets, kv_lens, B,
                              T, max_q_len, max_kv_len, out, out_stride, &a, &none);
  if (st || none) return st;
  a.window = window;
  a.sinks = sinks;
  a.masks = masks;
  a.mask_words = mask_words;
  return launch_forward(h, a, max_kv_len, stream);
}

int attn_tree_plan(attn_handle h, const int32_t* parents, const int32_t* q_offsets,
                   const int32_t* kv_lens, int B, int T, int max_q_len, int32_t* positions,
                   uint32_t* masks, int mask_words, void* stream) {
  if (!h || B < 0) return MOE_ERR_INVALID_ARG;
  int st = check_tokens(T);
  if (st) return st;
  if (!masks && T > 0) return MOE_ERR_INVALID_ARG;
  if ((st = check_masks(max_q_len, masks, mask_words))) return st;
  if (B > h->cfg.max_requests) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!positions || (B > 0 && (!parents || !q_offsets || !kv_lens))) return MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)parents, (const void*)q_offsets, (const void*)kv_lens,
                        (const void*)positions})
    if (off4(p)) return MOE_ERR_ALIGNMENT;
  moe::TreeArgs a{parents, q_offsets, kv_lens, B, T, max_q_len, positions, masks, mask_words,
                  h->err};
  return record_cuda_status(moe::launch_attn_tree_plan(a, static_cast<cudaStream_t>(stream)));
}

int attn_kv4_accept_pages(attn_handle h, void* cache, const int32_t* block_table, int table_width,
                          const int32_t* ctx_lens, const int32_t* paths, int path_width,
                          const int32_t* path_lens, int B, const int32_t* kv_lens,
                          int32_t* free_pages, int n_free, int32_t* cursor, void* stream) {
  if (!h || B < 0 || table_width < 0 || path_width < 0 || n_free < 0) return MOE_ERR_INVALID_ARG;
  if (B > h->cfg.max_requests || path_width > kMaxTokens) return MOE_ERR_UNSUPPORTED;
  if (B == 0) return MOE_OK;
  const int st = check_cache(cache);
  if (st) return st;
  if (!ctx_lens || !path_lens || !kv_lens || !cursor || (path_width > 0 && !paths) ||
      (table_width > 0 && !block_table) || (n_free > 0 && !free_pages))
    return MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)block_table, (const void*)ctx_lens, (const void*)paths,
                        (const void*)path_lens, (const void*)kv_lens, (const void*)free_pages,
                        (const void*)cursor})
    if (off4(p)) return MOE_ERR_ALIGNMENT;
  const moe::RowsArgs a = rows_args(h, cache, nullptr, 0);
  const moe::AcceptArgs p{block_table, table_width, ctx_lens, paths,      path_lens, path_width,
                          B,           kv_lens,     free_pages, n_free, cursor};
  return record_cuda_status(
      moe::launch_attn_accept(p, a, h->d.D, static_cast<cudaStream_t>(stream)));
}

int attn_kv4_accept(attn_handle h, void* cache, const int32_t* block_table, int table_width,
                    const int32_t* ctx_lens, const int32_t* paths, int path_width,
                    const int32_t* path_lens, int B, void* stream) {
  if (!h || B < 0 || table_width < 0 || path_width < 0) return MOE_ERR_INVALID_ARG;
  if (B > h->cfg.max_requests || path_width > kMaxTokens) return MOE_ERR_UNSUPPORTED;
  if (B == 0 || path_width == 0) return MOE_OK;
  const int st = check_cache(cache);
  if (st) return st;
  if (!ctx_lens || !paths || !path_lens || (table_width > 0 && !block_table))
    return MOE_ERR_INVALID_ARG;
  if (off4(block_table) || off4(ctx_lens) || off4(paths) || off4(path_lens))
    return MOE_ERR_ALIGNMENT;
  const moe::RowsArgs a = rows_args(h, cache, nullptr, 0);
  const moe::AcceptArgs p{block_table, table_width, ctx_lens, paths, path_lens, path_width, B,
                          nullptr,     nullptr,     0,        nullptr};
  return record_cuda_status(
      moe::launch_attn_accept(p, a, h->d.D, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
