// C ABI of the paged-cache operators: argument checks and launches.  The
// contract of every entry point is in include/csa2.h.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>

#include "common.cuh"
#include "launch.cuh"

namespace csa2 {

static bool on(const void *p, size_t a) { return p != nullptr && ((uintptr_t)p % a) == 0; }
static bool off_or_on(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

static bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

}  // namespace csa2

using namespace csa2;

extern "C" {

csa2_status csa2_page_plan_at(const int32_t *seq_len, const int32_t *new_len, const int32_t *gone, int n_seq,
                              int page_size, int n_pages, const int32_t *free_pages, int n_free,
                              const int32_t *free_head, int32_t *block_table, int64_t table_stride, int swa_cap,
                              int32_t *desc, int max_tokens, int32_t *first, int32_t *totals, csa2_stream_t stream) {
  if (n_seq < 0 || page_size < 1 || n_pages < 1 || n_free < 0 || table_stride < 1 || swa_cap < 0 || max_tokens < 0)
    return CSA2_ERR_INVALID_ARG;
  if ((int64_t)n_pages * page_size > INT_MAX || (int64_t)n_seq * swa_cap > INT_MAX) return CSA2_ERR_UNSUPPORTED;
  if (n_seq > kPlanMaxSeq || table_stride > INT_MAX) return CSA2_ERR_UNSUPPORTED;
  if (!on(first, 4) || !on(totals, 4) || (max_tokens > 0 && !on(desc, 4))) return CSA2_ERR_INVALID_ARG;
  if (n_seq > 0 && (!on(seq_len, 4) || !on(new_len, 4) || !on(block_table, 4))) return CSA2_ERR_INVALID_ARG;
  if ((n_free > 0 && !on(free_pages, 4)) || !off_or_on(free_head, 4) || !off_or_on(gone, 4)) return CSA2_ERR_INVALID_ARG;
  PlanArgs P;
  P.seq_len = seq_len;
  P.new_len = new_len;
  P.gone = gone;
  P.n_seq = n_seq;
  P.page = page_size;
  P.n_pages = n_pages;
  P.free_pages = free_pages;
  P.n_free = n_free;
  P.free_head = free_head;
  P.block_table = block_table;
  P.table_stride = table_stride;
  const int64_t row = table_stride * page_size;
  P.row_cap = row < INT_MAX ? row : INT_MAX;
  P.swa_cap = swa_cap;
  P.desc = desc;
  P.max_tokens = max_tokens;
  P.first = first;
  P.totals = totals;
  P.status = status_word_ptr();
  if (P.status == nullptr) return CSA2_ERR_CUDA;
  return launch_page_plan(P, (cudaStream_t)stream) == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

csa2_status csa2_page_plan(const int32_t *seq_len, const int32_t *new_len, int n_seq, int page_size, int n_pages,
                           const int32_t *free_pages, int n_free, const int32_t *free_head, int32_t *block_table,
                           int64_t table_stride, int swa_cap, int32_t *desc, int max_tokens, int32_t *first,
                           int32_t *totals, csa2_stream_t stream) {
  return csa2_page_plan_at(seq_len, new_len, nullptr, n_seq, page_size, n_pages, free_pages, n_free, free_head,
                           block_table, table_stride, swa_cap, desc, max_tokens, first, totals, stream);
}

csa2_status csa2_qk_norm_rope(const void *q, int64_t q_stride, const float *q_gain, void *q_out, const void *latent,
                              int64_t latent_stride, const float *latent_gain, void *latent_out, const int32_t *pos,
                              const int32_t *slot, const int32_t *swa_slot, int n, double eps, void *kv_cache,
                              int64_t kv_slots, void *swa_cache, int64_t swa_slots, const csa2_params *params,
                              csa2_stream_t stream) {
  if (!params_ok(params)) return CSA2_ERR_UNSUPPORTED;
  if (n < 0 || kv_slots < 0 || swa_slots < 0 || !(eps > 0.0) || !isfinite(eps)) return CSA2_ERR_INVALID_ARG;
  if (n > (1 << 27) || kv_slots > INT_MAX || swa_slots > INT_MAX) return CSA2_ERR_UNSUPPORTED;
  if ((q != nullptr) != (q_out != nullptr)) return CSA2_ERR_INVALID_ARG;
  if (q == nullptr && latent == nullptr && n > 0) return CSA2_ERR_INVALID_ARG;
  if (latent == nullptr && (latent_out != nullptr || kv_cache != nullptr || swa_cache != nullptr))
    return CSA2_ERR_INVALID_ARG;
  if ((kv_cache != nullptr && slot == nullptr) || (swa_cache != nullptr && swa_slot == nullptr))
    return CSA2_ERR_INVALID_ARG;
  // rows start on 16-B boundaries; strides may skip elements but not overlap rows
  if (q != nullptr && (q_stride < kHeads * kDim || q_stride % 8 != 0)) return CSA2_ERR_INVALID_ARG;
  if (latent != nullptr && (latent_stride < kDim || latent_stride % 8 != 0)) return CSA2_ERR_INVALID_ARG;
  if (n == 0) return CSA2_OK;
  if (!on(pos, 4) || !off_or_on(slot, 4) || !off_or_on(swa_slot, 4)) return CSA2_ERR_INVALID_ARG;
  if (!off_or_on(q, 16) || !off_or_on(q_out, 16) || !off_or_on(latent, 16) || !off_or_on(latent_out, 16) ||
      !off_or_on(q_gain, 16) || !off_or_on(latent_gain, 16) || !off_or_on(kv_cache, 16) || !off_or_on(swa_cache, 16))
    return CSA2_ERR_INVALID_ARG;
  // in place, or apart: a shifted overlap would read rows that another row's result has replaced
  const size_t q_in = ((size_t)(n - 1) * (size_t)q_stride + kHeads * kDim) * 2, q_to = (size_t)n * kHeads * kDim * 2;
  if (q != nullptr && !(q == q_out && q_stride == kHeads * kDim) && overlap(q, q_in, q_out, q_to))
    return CSA2_ERR_INVALID_ARG;
  const size_t l_in = ((size_t)(n - 1) * (size_t)latent_stride + kDim) * 2, l_to = (size_t)n * kDim * 2;
  if (latent_out != nullptr && !(latent == latent_out && latent_stride == kDim) &&
      overlap(latent, l_in, latent_out, l_to))
    return CSA2_ERR_INVALID_ARG;
  NormArgs A;
  A.q = static_cast<const uint16_t *>(q);
  A.q_stride = q_stride;
  A.q_gain = q_gain;
  A.q_out = static_cast<uint16_t *>(q_out);
  A.lat = static_cast<const uint16_t *>(latent);
  A.lat_stride = latent_stride;
  A.lat_gain = latent_gain;
  A.lat_out = static_cast<uint16_t *>(latent_out);
  A.pos = pos;
  A.slot = slot;
  A.swa_slot = swa_slot;
  A.n = n;
  A.kv = static_cast<uint8_t *>(kv_cache);
  A.kv_slots = kv_slots;
  A.swa = static_cast<uint8_t *>(swa_cache);
  A.swa_slots = swa_slots;
  A.status = status_word_ptr();
  if (A.status == nullptr) return CSA2_ERR_CUDA;
  const double rope_base = params ? params->rope_base : 10000.0;
  return launch_qk_norm_rope(A, eps, rope_base, (cudaStream_t)stream) == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

csa2_status csa2_cache_read(int kind, const void *cache, int64_t n_slots, const int32_t *slots, int64_t n, void *out,
                            int out_dtype, csa2_stream_t stream) {
  if (kind != CSA2_KV_NVFP4 && kind != CSA2_SWA_MXFP8)
    return kind == CSA2_IDX_MXFP4 ? CSA2_ERR_UNSUPPORTED : CSA2_ERR_INVALID_ARG;
  if (n_slots < 0 || n < 0 || (out_dtype != CSA2_OUT_BF16 && out_dtype != CSA2_OUT_F32)) return CSA2_ERR_INVALID_ARG;
  if (n > ((int64_t)1 << 40)) return CSA2_ERR_UNSUPPORTED;
  if (n == 0) return CSA2_OK;
  if (!on(cache, 16) || !on(slots, 4) || !on(out, 16)) return CSA2_ERR_INVALID_ARG;
  int *st = status_word_ptr();
  if (st == nullptr) return CSA2_ERR_CUDA;
  return launch_cache_read(kind, cache, n_slots, slots, n, out, out_dtype, st, (cudaStream_t)stream) == cudaSuccess
             ? CSA2_OK
             : CSA2_ERR_CUDA;
}

csa2_status csa2_paged_attn(const void *q, const void *pages, int n_pages, int page_size, const int32_t *block_table,
                            int64_t table_stride, int n_seq, const int32_t *sel, int sel_stride, const void *swa_cache,
                            int swa_cap, const int32_t *q_seq, const int32_t *n_vis, const int32_t *pos,
                            const int32_t *swa_first, const int32_t *swa_cnt, int n_q, void *out, int out_dtype,
                            float *lse, const csa2_params *params, void *workspace, size_t workspace_bytes,
                            csa2_stream_t stream) {
  if (!params_ok(params)) return CSA2_ERR_UNSUPPORTED;
  if (n_q < 0 || n_seq < 1 || n_pages < 1 || page_size < 1 || table_stride < 1 || swa_cap < 0)
    return CSA2_ERR_INVALID_ARG;
  if (out_dtype != CSA2_OUT_BF16 && out_dtype != CSA2_OUT_F32) return CSA2_ERR_INVALID_ARG;
  if (sel != nullptr && (sel_stride < 1 || sel_stride > kTopK)) return CSA2_ERR_INVALID_ARG;
  if (n_q > 65535 || table_stride > INT_MAX || (int64_t)n_pages * page_size > INT_MAX) return CSA2_ERR_UNSUPPORTED;
  // chunks of 128 entries are counted in 32 bits (a row of n_vis entries never has more)
  const int64_t row = sel != nullptr ? sel_stride : table_stride * page_size < INT_MAX ? table_stride * page_size : INT_MAX;
  if (n_q * ((row + 127) / 128 + 1) > (1 << 30)) return CSA2_ERR_UNSUPPORTED;
  if (n_q == 0) return CSA2_OK;
  if (!on(q, 16) || !on(pages, 32) || !on(block_table, 4) || !off_or_on(sel, 4) || !on(q_seq, 4) || !on(n_vis, 4) ||
      !on(pos, 4) || !on(swa_first, 4) || !on(swa_cnt, 4) || !on(out, 16) || !off_or_on(lse, 4))
    return CSA2_ERR_INVALID_ARG;
  if (swa_cap > 0 ? !on(swa_cache, 16) : !off_or_on(swa_cache, 16)) return CSA2_ERR_INVALID_ARG;
  if (workspace == nullptr || ((uintptr_t)workspace % 256) != 0 || workspace_bytes < paged_attn_workspace_bytes())
    return CSA2_ERR_WORKSPACE;
  PagedArgs A;
  A.q = static_cast<const uint16_t *>(q);
  A.pages = static_cast<const uint8_t *>(pages);
  A.n_pages = n_pages;
  A.page = page_size;
  A.table = block_table;
  A.table_stride = table_stride;
  A.n_seq = n_seq;
  A.sel = sel;
  A.sel_stride = sel != nullptr ? sel_stride : 0;
  A.swa = static_cast<const uint8_t *>(swa_cache);
  A.swa_cap = swa_cap;
  A.q_seq = q_seq;
  A.n_vis = n_vis;
  A.pos = pos;
  A.swa_first = swa_first;
  A.swa_cnt = swa_cnt;
  A.n_q = n_q;
  A.out = out;
  A.out_f32 = out_dtype == CSA2_OUT_F32;
  A.lse = lse;
  A.status = status_word_ptr();
  if (A.status == nullptr) return CSA2_ERR_CUDA;
  A.scale = params ? params->sm_scale : 1.0f / sqrtf((float)kDim);
  const double rope_base = params ? params->rope_base : 10000.0;
  return launch_paged_attn(A, rope_base, workspace, (cudaStream_t)stream) == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

}  // extern "C"
