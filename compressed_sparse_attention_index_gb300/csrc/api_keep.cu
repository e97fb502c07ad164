// C ABI of the operators that decide what a paged cache keeps: argument checks and
// launches.  The contract of every entry point is in include/csa2.h.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>

#include "common.cuh"
#include "launch.cuh"

namespace csa2 {

static bool on(const void *p, size_t a) { return p != nullptr && ((uintptr_t)p % a) == 0; }
static bool off_or_on(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Entries of a row: the end of the last tile of 128 is counted in 32 bits.
constexpr int64_t kRowMax = INT_MAX - 255;

}  // namespace csa2

using namespace csa2;

extern "C" {

csa2_status csa2_attn_weight(const void *q, const void *pages, int n_pages, int page_size, const int32_t *block_table,
                             int64_t table_stride, const int32_t *first, int n_seq, const int32_t *sel, int sel_stride,
                             const int32_t *n_vis, const float *lse, int n_q, float decay, const float *prior,
                             float *weight, const csa2_params *params, void *workspace, size_t workspace_bytes,
                             csa2_stream_t stream) {
  if (!params_ok(params)) return CSA2_ERR_UNSUPPORTED;
  if (n_q < 0 || n_seq < 0 || n_pages < 1 || page_size < 1 || table_stride < 1 || !isfinite(decay))
    return CSA2_ERR_INVALID_ARG;
  if (sel != nullptr && (sel_stride < 1 || sel_stride > kTopK)) return CSA2_ERR_INVALID_ARG;
  if (n_q > 65535 || n_seq > kPlanMaxSeq || table_stride > INT_MAX || (int64_t)n_pages * page_size > INT_MAX ||
      table_stride * page_size > kRowMax)
    return CSA2_ERR_UNSUPPORTED;
  // work is counted in chunks of 128 entries and queries, in 32 bits
  const int64_t row = sel != nullptr ? sel_stride : table_stride * page_size;
  if (n_q * ((row + 127) / 128 + 1) > (1 << 30)) return CSA2_ERR_UNSUPPORTED;
  if (n_q == 0 || n_seq == 0) return CSA2_OK;
  if (!on(q, 16) || !on(pages, 32) || !on(block_table, 4) || !on(first, 4) || !off_or_on(sel, 4) || !on(n_vis, 4) ||
      !on(lse, 4) || !off_or_on(prior, 4) || !on(weight, 4))
    return CSA2_ERR_INVALID_ARG;
  if (workspace == nullptr || ((uintptr_t)workspace % 256) != 0 ||
      workspace_bytes < weigh_workspace_bytes(n_q, n_seq, sel != nullptr ? sel_stride : 0))
    return CSA2_ERR_WORKSPACE;
  WeighArgs A = {};
  A.q = static_cast<const uint16_t *>(q);
  A.pages = static_cast<const uint8_t *>(pages);
  A.n_pages = n_pages;
  A.page = page_size;
  A.table = block_table;
  A.table_stride = table_stride;
  A.first = first;
  A.n_seq = n_seq;
  A.sel = sel;
  A.sel_stride = sel != nullptr ? sel_stride : 0;
  A.n_vis = n_vis;
  A.lse = lse;
  A.n_q = n_q;
  A.decay = decay;
  A.prior = prior;
  A.weight = weight;
  A.status = status_word_ptr();
  if (A.status == nullptr) return CSA2_ERR_CUDA;
  A.scale = params ? params->sm_scale : 1.0f / sqrtf((float)kDim);
  return launch_weigh(A, workspace, (cudaStream_t)stream) == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

csa2_status csa2_evict(const void *pages, const float *weight, int n_pages, int page_size, const int32_t *block_table,
                       int64_t table_stride, const int32_t *seq_len, const int32_t *keep, int n_seq, int recent,
                       void *dst_pages, float *dst_weight, int n_dst_pages, const int32_t *dst_table,
                       int64_t dst_stride, int32_t *new_len, int32_t *from, int64_t from_stride, void *workspace,
                       size_t workspace_bytes, csa2_stream_t stream) {
  if (n_seq < 0 || n_pages < 1 || page_size < 1 || table_stride < 1 || recent < 0 || n_dst_pages < 1 || dst_stride < 1)
    return CSA2_ERR_INVALID_ARG;
  if (from != nullptr && from_stride < 1) return CSA2_ERR_INVALID_ARG;
  // the source's table in the source's pages: in place (other pages of the same cache are another destination)
  const bool in_place = dst_pages == pages && dst_table == block_table;
  if (in_place && (dst_weight != weight || n_dst_pages != n_pages || dst_stride != table_stride)) return CSA2_ERR_INVALID_ARG;
  if (n_seq > kPlanMaxSeq || table_stride > INT_MAX || dst_stride > INT_MAX ||
      (int64_t)n_pages * page_size > INT_MAX || (int64_t)n_dst_pages * page_size > INT_MAX ||
      table_stride * page_size > kRowMax || dst_stride * page_size > kRowMax)
    return CSA2_ERR_UNSUPPORTED;
  if (n_seq == 0) return CSA2_OK;
  if (!on(pages, 32) || !on(weight, 16) || !on(block_table, 4) || !on(seq_len, 4) || !on(keep, 4) ||
      !on(dst_pages, 32) || !on(dst_weight, 4) || !on(dst_table, 4) || !on(new_len, 4) || !off_or_on(from, 4))
    return CSA2_ERR_INVALID_ARG;
  if (workspace == nullptr || ((uintptr_t)workspace % 256) != 0 ||
      workspace_bytes < evict_workspace_bytes(n_seq, table_stride * page_size))
    return CSA2_ERR_WORKSPACE;
  EvictArgs A = {};
  A.pages = static_cast<const uint8_t *>(pages);
  A.weight = weight;
  A.n_pages = n_pages;
  A.page = page_size;
  A.table = block_table;
  A.table_stride = table_stride;
  A.seq_len = seq_len;
  A.keep = keep;
  A.n_seq = n_seq;
  A.recent = recent;
  A.dst_pages = static_cast<uint8_t *>(dst_pages);
  A.dst_weight = dst_weight;
  A.n_dst = n_dst_pages;
  A.dst_table = dst_table;
  A.dst_stride = dst_stride;
  A.in_place = in_place;
  A.new_len = new_len;
  A.from = from;
  A.from_stride = from_stride;
  A.status = status_word_ptr();
  if (A.status == nullptr) return CSA2_ERR_CUDA;
  return launch_evict(A, workspace, (cudaStream_t)stream) == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

csa2_status csa2_page_trim(const int32_t *len, const int32_t *new_len, int n_seq, int page_size, int n_pages,
                           int32_t *free_pages, int n_free, int32_t *free_head, int32_t *block_table,
                           int64_t table_stride, csa2_stream_t stream) {
  if (n_seq < 0 || page_size < 1 || n_pages < 1 || n_free < 0 || table_stride < 1) return CSA2_ERR_INVALID_ARG;
  if (n_seq > kPlanMaxSeq || table_stride > INT_MAX || (int64_t)n_pages * page_size > INT_MAX) return CSA2_ERR_UNSUPPORTED;
  if (n_seq == 0) return CSA2_OK;
  if (!on(len, 4) || !on(new_len, 4) || (n_free > 0 && !on(free_pages, 4)) || !on(free_head, 4) || !on(block_table, 4))
    return CSA2_ERR_INVALID_ARG;
  TrimArgs A = {};
  A.len = len;
  A.new_len = new_len;
  A.n_seq = n_seq;
  A.page = page_size;
  A.n_pages = n_pages;
  A.free_pages = free_pages;
  A.n_free = n_free;
  A.free_head = free_head;
  A.table = block_table;
  A.table_stride = table_stride;
  const int64_t row = table_stride * page_size;
  A.row_cap = row < INT_MAX ? row : INT_MAX;
  A.status = status_word_ptr();
  if (A.status == nullptr) return CSA2_ERR_CUDA;
  return launch_page_trim(A, (cudaStream_t)stream) == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

csa2_status csa2_verify_drafts(int mode, const void *target, int64_t target_stride, const void *draft,
                               int64_t draft_stride, int dtype, int vocab, const int32_t *tokens, const int32_t *first,
                               int n_seq, int n_rows, const float *u, const float *v, int32_t *kept, int32_t *next,
                               void *workspace, size_t workspace_bytes, csa2_stream_t stream) {
  if (mode != CSA2_VERIFY_SAMPLE && mode != CSA2_VERIFY_GREEDY) return CSA2_ERR_INVALID_ARG;
  if (dtype != CSA2_PROB_BF16 && dtype != CSA2_PROB_F32 && dtype != CSA2_PROB_F16) return CSA2_ERR_INVALID_ARG;
  if (n_seq < 0 || n_rows < 0 || vocab < 1 || target_stride < vocab) return CSA2_ERR_INVALID_ARG;
  const bool greedy = mode == CSA2_VERIFY_GREEDY;
  if (greedy ? draft != nullptr : draft != nullptr && draft_stride < vocab) return CSA2_ERR_INVALID_ARG;
  if (n_seq > kPlanMaxSeq || n_rows > 65535 || vocab > (1 << 28)) return CSA2_ERR_UNSUPPORTED;
  if (n_seq == 0) return CSA2_OK;
  const size_t size = dtype == CSA2_PROB_F32 ? 4 : 2;
  if (!on(first, 4) || !on(kept, 4) || !on(next, 4) || !off_or_on(draft, size)) return CSA2_ERR_INVALID_ARG;
  if (n_rows > 0 && (!on(target, size) || !on(tokens, 4))) return CSA2_ERR_INVALID_ARG;
  if (!greedy && (!on(v, 4) || (n_rows > 0 && !on(u, 4)))) return CSA2_ERR_INVALID_ARG;
  if (greedy && (workspace == nullptr || ((uintptr_t)workspace % 256) != 0 || workspace_bytes < verify_workspace_bytes(n_rows)))
    return CSA2_ERR_WORKSPACE;
  VerifyArgs A = {};
  A.target = target;
  A.target_stride = target_stride;
  A.draft = draft;
  A.draft_stride = draft_stride;
  A.vocab = vocab;
  A.tokens = tokens;
  A.first = first;
  A.n_seq = n_seq;
  A.n_rows = n_rows;
  A.u = u;
  A.v = v;
  A.kept = kept;
  A.next = next;
  A.best = static_cast<unsigned long long *>(workspace);
  A.status = status_word_ptr();
  if (A.status == nullptr) return CSA2_ERR_CUDA;
  return launch_verify(A, dtype, greedy, (cudaStream_t)stream) == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

}  // extern "C"
