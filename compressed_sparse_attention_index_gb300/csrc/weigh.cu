// The attention weight that cache entries get from a step's queries (csa2_attn_weight):
//
//     w_j = decay prior_j + sum over the queries that see j, and their heads, of
//           exp(scale q_h . k_j - lse_h)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "attn.cuh"
#include "common.cuh"
#include "launch.cuh"

namespace csa2 {

constexpr int kWgTile = 32, kWgThreads = 256, kWgDims = 64;

// A sequence's queries, or none where that is out of range.
__device__ __forceinline__ bool weigh_queries(const WeighArgs &A, int b, int &c0, int &c1) {
  c0 = __ldg(A.first + b);
  c1 = __ldg(A.first + b + 1);
  if (c0 >= 0 && c1 >= c0 && c1 <= A.n_q) return true;
  c0 = c1 = 0;
  return false;
}
// Entries that query q sees, -1 where that is out of range.
__device__ __forceinline__ int weigh_vis(const WeighArgs &A, int q) {
  const int v = __ldg(A.n_vis + q);
  return v < 0 || (int64_t)v > A.table_stride * A.page ? -1 : v;
}
__device__ __forceinline__ int64_t weigh_slot(const WeighArgs &A, int b, int j) {
  const int c = (int)(((uint64_t)(unsigned)j * A.page_mul) >> A.page_shift);
  const int id = __ldg(A.table + (int64_t)b * A.table_stride + c);
  return id >= 0 && id < A.n_pages ? (int64_t)id * A.page + (j - c * A.page) : -1;
}

// 32 entries of a sequence (SEL: of a query's selection) against its queries, 64 dims at a time.
template <bool SEL>
__global__ void __launch_bounds__(kWgThreads) weigh_kernel(const __grid_constant__ WeighArgs A, float *part) {
  __shared__ float ks[kWgTile][kWgDims + 1], qs[kHeads][kWgDims + 1];
  __shared__ int64_t slot_sh[kWgTile];
  const int t = threadIdx.x, e = t >> 3, hg = t & 7;
  griddep_wait();
  griddep_launch();
  int b = blockIdx.y, c0, c1;
  if (SEL) {                                         // the sequence that has this query
    const int q = blockIdx.y;
    int lo = 0, hi = A.n_seq;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(A.first + mid) <= q) lo = mid;
      else hi = mid;
    }
    b = lo;
    if (!weigh_queries(A, b, c0, c1) || q < c0 || q >= c1) return;
    c0 = q;
    c1 = q + 1;
  } else if (!weigh_queries(A, b, c0, c1) && t == 0) {
    record_error(A.status, CSA2_ERR_BOUNDS);
  }
  int most = 0;
  for (int q = c0 + t; q < c1; q += kWgThreads) {
    const int v = weigh_vis(A, q);
    if (v < 0) record_error(A.status, CSA2_ERR_BOUNDS);
    most = max(most, v);
  }
  __shared__ int most_sh;
  if (t == 0) most_sh = 0;
  __syncthreads();
  atomicMax(&most_sh, most);
  __syncthreads();
  most = most_sh;
  const int n = SEL ? A.sel_stride : most;
  for (int j0 = blockIdx.x * kWgTile; j0 < n; j0 += gridDim.x * kWgTile) {
    int j = j0 + e;
    if (j >= n) j = -1;
    if (SEL && j >= 0) {
      j = __ldg(A.sel + (int64_t)c0 * A.sel_stride + j);
      if (j >= most) {
        if (hg == 0) record_error(A.status, CSA2_ERR_BOUNDS);
        j = -1;
      }
    }
    int64_t slot = -1;
    if (j >= 0) {
      slot = weigh_slot(A, b, j);
      if (slot < 0 && hg == 0) record_error(A.status, CSA2_ERR_BOUNDS);
    }
    if (hg == 0) slot_sh[e] = slot;
    float sum = 0.f;
    for (int q = c0; q < c1; q++) {
      const int vis = weigh_vis(A, q);
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int d0 = 0; d0 < kDim; d0 += kWgDims) {
        __syncthreads();
        for (int i = t; i < kWgTile * kWgDims; i += kWgThreads) {
          const int r = i / kWgDims, d = d0 + i % kWgDims;
          float x = 0.f;
          if (slot_sh[r] >= 0) {
            const uint8_t *rec = A.pages + slot_sh[r] * kKvBytes;
            x = 0.5f * (float)e2m1_x2((rec[d >> 1] >> (4 * (d & 1))) & 15u) * e4m3_to_float(rec[256 + (d >> 4)]);
          }
          ks[r][i % kWgDims] = x;
        }
        for (int i = t; i < kHeads * kWgDims; i += kWgThreads)
          qs[i / kWgDims][i % kWgDims] = __uint_as_float((uint32_t)A.q[((int64_t)q * kHeads + i / kWgDims) * kDim + d0 + i % kWgDims] << 16);
        __syncthreads();
        for (int d = 0; d < kWgDims; d++)
#pragma unroll
          for (int h = 0; h < 8; h++) acc[h] = fmaf(ks[e][d], qs[hg * 8 + h][d], acc[h]);
      }
      float p = 0.f;
#pragma unroll
      for (int h = 0; h < 8; h++) {
        const float l = __ldg(A.lse + (int64_t)q * kHeads + hg * 8 + h);
        if (fabsf(l) < INFINITY && fabsf(acc[h]) < INFINITY) p += exp2f((acc[h] * A.scale - l) * 1.4426950408889634f);
      }
      if (j < vis) sum += p;
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (hg == 0) {
      if (SEL) {
        if (j0 + e < n) part[(int64_t)c0 * A.sel_stride + j0 + e] = slot >= 0 ? sum : 0.f;
      } else if (slot >= 0) {
        A.weight[slot] = (A.prior != nullptr ? A.decay * A.prior[slot] : 0.f) + sum;
      }
    }
    __syncthreads();
  }
}

// What selections start from: decay prior, of every entry that a query of the sequence sees.
__global__ void __launch_bounds__(kWgThreads) weigh_decay_kernel(const __grid_constant__ WeighArgs A) {
  const int t = threadIdx.x, b = blockIdx.y;
  griddep_wait();
  griddep_launch();
  int c0, c1, most = 0;
  weigh_queries(A, b, c0, c1);
  for (int q = c0 + t; q < c1; q += kWgThreads) most = max(most, weigh_vis(A, q));
  __shared__ int most_sh;
  if (t == 0) most_sh = 0;
  __syncthreads();
  atomicMax(&most_sh, most);
  __syncthreads();
  most = most_sh;
  for (int64_t j = (int64_t)blockIdx.x * kWgThreads + t; j < most; j += (int64_t)gridDim.x * kWgThreads) {
    const int64_t s = weigh_slot(A, b, (int)j);
    if (s >= 0) A.weight[s] = A.prior != nullptr ? A.decay * A.prior[s] : 0.f;
  }
}

// Adds the selections' weights, a CTA per sequence, query by query: entries that several queries
// selected get their parts in the queries' order, so the sums are the same on every call.  (Within
// a query an entry named twice gets the same part twice: their order does not matter.)
__global__ void __launch_bounds__(kTopK) weigh_add_kernel(const __grid_constant__ WeighArgs A, const float *part) {
  const int t = threadIdx.x, b = blockIdx.x;
  griddep_wait();
  griddep_launch();
  int c0, c1;
  if (!weigh_queries(A, b, c0, c1) && t == 0) record_error(A.status, CSA2_ERR_BOUNDS);
  for (int q = c0; q < c1; q++) {
    if (t < A.sel_stride) {
      const int j = __ldg(A.sel + (int64_t)q * A.sel_stride + t);
      if (j >= 0 && j < weigh_vis(A, q)) {
        const int64_t s = weigh_slot(A, b, j);
        if (s >= 0) atomicAdd(A.weight + s, __ldg(part + (int64_t)q * A.sel_stride + t));
      }
    }
    __syncthreads();
  }
}

static void weigh_magic(unsigned n, uint64_t &mul, int &shift) {      // j / n, exact for j below 2^31
  int s = 0;
  while (((int64_t)1 << s) < (int64_t)n) s++;
  shift = 31 + s;
  mul = (uint64_t)((((unsigned __int128)1 << shift) + n - 1) / n);
}

size_t weigh_workspace_bytes(int n_q, int64_t n_seq, int sel_stride) {
  (void)n_seq;
  return (size_t)n_q * (size_t)sel_stride * sizeof(float) + 256;
}

cudaError_t launch_weigh(WeighArgs A, void *ws, cudaStream_t st) {
  weigh_magic((unsigned)A.page, A.page_mul, A.page_shift);
  float *part = static_cast<float *>(ws);
  const int64_t row = A.table_stride * A.page;
  if (A.sel == nullptr) {
    const int64_t tiles = (row + kWgTile - 1) / kWgTile;
    return launch_pdl(weigh_kernel<false>, dim3((unsigned)(tiles < 8192 ? tiles : 8192), (unsigned)A.n_seq), dim3(kWgThreads), 0, st, 1u, A, part);
  }
  cudaError_t e = cudaSuccess;
  if (A.prior != A.weight || A.decay != 1.f) {
    const int64_t tiles = (row + 4 * kWgThreads - 1) / (4 * kWgThreads);
    e = launch_pdl(weigh_decay_kernel, dim3((unsigned)(tiles < 512 ? tiles : 512), (unsigned)A.n_seq), dim3(kWgThreads), 0, st, 1u, A);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(weigh_kernel<true>, dim3((unsigned)(A.sel_stride + kWgTile - 1) / kWgTile, (unsigned)A.n_q), dim3(kWgThreads), 0, st, 1u, A, part);
  if (e != cudaSuccess) return e;
  return launch_pdl(weigh_add_kernel, dim3((unsigned)A.n_seq), dim3(kTopK), 0, st, 1u, A, (const float *)part);
}

}  // namespace csa2
