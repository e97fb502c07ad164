// Paged caches: the plan of a step from the sequences' lengths
// (csa2_page_plan) and reading records back (csa2_cache_read).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>

#include "attn.cuh"
#include "common.cuh"
#include "launch.cuh"

namespace csa2 {

// ------------------------------------------------------------------ plan
// Sequence b holds len_b entries and gets new_b tokens; its pages grow from
// have_b = ceil(len_b / p) to need_b = ceil((len_b + new_b) / p) columns.  With
// the exclusive prefix sums of new and of need - have over the sequences, every
// new page and every token finds its own values by one binary search, so the
// work spreads over any number of CTAs; each CTA makes the two prefix sums for
// itself in shared memory (8 B a sequence from L2, cheaper than a grid-wide
// barrier or a second launch).  Latency-bound for a decode step; for a prompt
// the 28 B written per token.
struct PlanSeq {
  int len, add, have, need;
};

__device__ __forceinline__ int sat_add(int a, int b) {       // non-negative, saturating
  return (int)min((unsigned)a + (unsigned)b, (unsigned)INT_MAX);
}

__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs &P, int b, bool &bad) {
  PlanSeq s;
  s.len = __ldg(P.seq_len + b);
  s.add = __ldg(P.new_len + b);
  // a sequence that cannot be: it takes no part in the step
  bad = s.len < 0 || s.add < 0 || (int64_t)s.len + s.add > P.row_cap;
  if (bad) s.len = s.add = 0;
  s.have = (int)(((unsigned)s.len + (unsigned)P.page - 1u) / (unsigned)P.page);
  s.need = (int)(((unsigned)(s.len + s.add) + (unsigned)P.page - 1u) / (unsigned)P.page);
  return s;
}

// largest b in [0, n) with first[b] <= x (first ascending, first[0] = 0)
__device__ __forceinline__ int seq_of(const int *first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ PlanArgs P) {
  extern __shared__ int plan_sh[];                             // tok[n_seq + 1], pg[n_seq + 1]
  __shared__ int wt[kPlanThreads / 32], wp[kPlanThreads / 32];
  int *tok = plan_sh, *pg = plan_sh + P.n_seq + 1;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, nt = blockDim.x;
  griddep_wait();
  griddep_launch();
  // prefix sums: thread t has sequences [b0, b1)
  const int per = (P.n_seq + nt - 1) / nt, b0 = min(t * per, P.n_seq), b1 = min(b0 + per, P.n_seq);
  int st = 0, sp = 0;
  bool any_bad = false;
  for (int b = b0; b < b1; b++) {
    bool bad;
    const PlanSeq s = plan_seq(P, b, bad);
    any_bad |= bad;
    st = sat_add(st, s.add);
    sp = sat_add(sp, s.need - s.have);
  }
  int it = st, ip = sp;                                        // inclusive over the warp, then the block
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, it, o), c = __shfl_up_sync(0xFFFFFFFFu, ip, o);
    if (lane >= o) { it = sat_add(it, a); ip = sat_add(ip, c); }
  }
  if (lane == 31) { wt[warp] = it; wp[warp] = ip; }
  int et = __shfl_up_sync(0xFFFFFFFFu, it, 1), ep = __shfl_up_sync(0xFFFFFFFFu, ip, 1);
  if (lane == 0) et = ep = 0;
  __syncthreads();
  for (int w = 0; w < warp; w++) { et = sat_add(et, wt[w]); ep = sat_add(ep, wp[w]); }
  for (int b = b0; b < b1; b++) {
    bool bad;
    const PlanSeq s = plan_seq(P, b, bad);
    tok[b] = et;
    pg[b] = ep;
    et = sat_add(et, s.add);
    ep = sat_add(ep, s.need - s.have);
  }
  if (t == nt - 1) { tok[P.n_seq] = et; pg[P.n_seq] = ep; }
  __syncthreads();
  const int n_tok = tok[P.n_seq], n_new = pg[P.n_seq];
  const int head = P.free_head != nullptr ? __ldg(P.free_head) : 0;
  // new page j of the step: the free list's entry, or -1 where the list ends or names no page
  auto free_page = [&](int j) -> int {
    const int64_t i = (int64_t)head + j;
    if (head < 0 || i >= P.n_free) return -1;
    const int id = __ldg(P.free_pages + i);
    return id >= 0 && id < P.n_pages ? id : -1;
  };
  bool err = any_bad && blockIdx.x == 0;
  const int64_t me = (int64_t)blockIdx.x * nt + t, all = (int64_t)gridDim.x * nt;
  for (int64_t j = me; j < n_new; j += all) {
    const int b = seq_of(pg, P.n_seq, (int)j);
    bool bad;
    const PlanSeq s = plan_seq(P, b, bad);
    const int id = free_page((int)j);
    err |= id < 0;
    P.block_table[(int64_t)b * P.table_stride + s.have + ((int)j - pg[b])] = id;
  }
  for (int64_t i = me; i < P.max_tokens; i += all) {
    int v[7] = {0, 0, 0, 0, 0, -1, -1};                        // a row without a token
    if (i < n_tok) {
      const int b = seq_of(tok, P.n_seq, (int)i);              // (has tokens, so its lengths are sound)
      const int len = __ldg(P.seq_len + b), add = __ldg(P.new_len + b);
      const int have = (int)(((unsigned)len + (unsigned)P.page - 1u) / (unsigned)P.page);
      const int pos = len + ((int)i - tok[b]), col = (int)((unsigned)pos / (unsigned)P.page);
      int id;
      if (col < have) {                                      // (columns that this step does not write)
        id = P.block_table[(int64_t)b * P.table_stride + col];
        if (id >= P.n_pages) id = -1;
      } else {
        id = free_page(pg[b] + (col - have));
      }
      err |= id < 0;
      const int cnt = min(min(kSwa, P.swa_cap), pos + 1);
      v[0] = b;
      v[1] = pos + 1;
      v[2] = pos;
      v[3] = P.swa_cap > 0 ? (int)((unsigned)(pos + 1 - cnt) % (unsigned)P.swa_cap) : 0;
      v[4] = cnt;
      v[5] = id < 0 ? -1 : id * P.page + (pos - col * P.page);
      // a ring slot that a later token of this step takes again is not written (a token
      // without a descriptor takes none)
      const int kept = min(add, P.max_tokens - tok[b]);
      v[6] = P.swa_cap > 0 && (int64_t)pos + P.swa_cap >= (int64_t)len + kept
                 ? b * P.swa_cap + (int)((unsigned)pos % (unsigned)P.swa_cap)
                 : -1;
    }
#pragma unroll
    for (int k = 0; k < 7; k++) P.desc[k * (int64_t)P.max_tokens + i] = v[k];
  }
  if (blockIdx.x == 0) {
    for (int b = t; b <= P.n_seq; b += nt) P.first[b] = tok[b];
    if (t == 0) {
      P.totals[0] = n_tok;
      P.totals[1] = n_new;
      err |= n_tok > P.max_tokens;
    }
  }
  if (err) record_error(P.status, CSA2_ERR_BOUNDS);
}

cudaError_t launch_page_plan(const PlanArgs &P, cudaStream_t st) {
  const int dev = current_device();
  static std::atomic<int> attr_done[kMaxDevices];
  cudaError_t e = once_per_device(attr_done, dev, [&] {
    return cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                2 * (kPlanMaxSeq + 1) * (int)sizeof(int));
  });
  if (e != cudaSuccess) return e;
  const size_t smem = 2 * (size_t)(P.n_seq + 1) * sizeof(int);
  // a warp's worth of sequences or tokens needs no 1,024 threads; a token a thread up to a CTA per SM (its
  // search and loads are a chain: 1,000 sequences and 131,072 tokens take 5.7 us, 9.8 with four a thread)
  const int most = P.n_seq > P.max_tokens ? P.n_seq : P.max_tokens;
  const int threads = most <= 128 ? 128 : most <= 512 ? 512 : kPlanThreads;
  const int64_t ctas = ((int64_t)P.max_tokens + threads - 1) / threads;
  const int64_t cap = device_sm_count(dev);
  return launch_pdl(page_plan_kernel, dim3((unsigned)(ctas < 1 ? 1 : ctas < cap ? ctas : cap)), dim3(threads), smem, st,
                    1u, P);
}

// ------------------------------------------------------------------ read
// One warp per record, kReadRows records in flight; a lane has channels
// [8 lane, 8 lane + 8) and 256 + that, so loads are 128 (256) and stores 512
// contiguous bytes a warp.  Bound by HBM: 288 (528) B in, 1 (2) KB out.
// E2M1 x E4M3 and E4M3 x 2^e are exact in fp32, the former also in bf16.  500,001
// records of NVFP4: 105 us (6.2 TB/s); with eight CTAs an SM that go around, and stores
// that stay in L2, 119.
constexpr int kReadThreads = 256, kReadRows = 4;

template <bool KV, bool F32>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const uint8_t *__restrict__ cache, int64_t n_slots,
                                                                  const int32_t *__restrict__ slots, int64_t n,
                                                                  void *__restrict__ out, int *status) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kReadThreads / 32);
  griddep_wait();
  griddep_launch();
  for (int64_t i0 = ((int64_t)blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5)) * kReadRows; i0 < n;
       i0 += warps * kReadRows) {
    int slot[kReadRows];
#pragma unroll
    for (int r = 0; r < kReadRows; r++) slot[r] = i0 + r < n ? __ldg(slots + i0 + r) : -1;
    uint2 raw[kReadRows][2];
    uint32_t sc[kReadRows][2];
#pragma unroll
    for (int r = 0; r < kReadRows; r++) {
      const bool ok = slot[r] >= 0 && slot[r] < n_slots;
      if (slot[r] >= n_slots && lane == 0) record_error(status, CSA2_ERR_BOUNDS);
      const uint8_t *rec = cache + (int64_t)(ok ? slot[r] : 0) * (KV ? kKvBytes : kSwaBytes);
#pragma unroll
      for (int f = 0; f < 2; f++) {
        raw[r][f] = make_uint2(0u, 0u);
        sc[r][f] = 0u;
        if (ok) {
          if (KV) raw[r][f].x = __ldg(reinterpret_cast<const uint32_t *>(rec + f * 128 + lane * 4));
          else raw[r][f] = __ldg(reinterpret_cast<const uint2 *>(rec + f * 256 + lane * 8));
          sc[r][f] = KV ? rec[256 + f * 16 + (lane >> 1)] : rec[512 + f * 8 + (lane >> 2)];
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kReadRows; r++) {
      if (i0 + r >= n) break;
#pragma unroll
      for (int f = 0; f < 2; f++) {
        uint32_t h2[4];
        if (KV) {
          e2m1x8_to_f16(raw[r][f].x, h2);
        } else {
#pragma unroll
          for (int k = 0; k < 4; k++) h2[k] = e4m3x2_to_f16x2((k < 2 ? raw[r][f].x : raw[r][f].y) >> (16 * (k & 1)));
        }
        const float s = KV ? e4m3_to_float(sc[r][f]) : e8m0_to_float(sc[r][f]);
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&h2[k]));
          v[2 * k] = p.x * s;
          v[2 * k + 1] = p.y * s;
        }
        const int64_t o = (i0 + r) * kDim + f * 256 + lane * 8;
        if (F32) {
          float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(out) + o);
          __stcs(d, make_float4(v[0], v[1], v[2], v[3]));
          __stcs(d + 1, make_float4(v[4], v[5], v[6], v[7]));
        } else {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; k++) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t *>(&b);
          }
          __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + o), make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
    }
  }
}

cudaError_t launch_cache_read(int kind, const void *cache, int64_t n_slots, const int32_t *slots, int64_t n, void *out,
                              int out_dtype, int *status, cudaStream_t st) {
  const int64_t per = (kReadThreads / 32) * kReadRows;
  const int64_t ctas = (n + per - 1) / per, cap = 1 << 20;
  const dim3 grid((unsigned)(ctas < cap ? ctas : cap)), block(kReadThreads);
  const uint8_t *c = static_cast<const uint8_t *>(cache);
  const bool f32 = out_dtype == CSA2_OUT_F32;
  if (kind == CSA2_KV_NVFP4)
    return f32 ? launch_pdl(cache_read_kernel<true, true>, grid, block, 0, st, 1u, c, n_slots, slots, n, out, status)
               : launch_pdl(cache_read_kernel<true, false>, grid, block, 0, st, 1u, c, n_slots, slots, n, out, status);
  return f32 ? launch_pdl(cache_read_kernel<false, true>, grid, block, 0, st, 1u, c, n_slots, slots, n, out, status)
             : launch_pdl(cache_read_kernel<false, false>, grid, block, 0, st, 1u, c, n_slots, slots, n, out, status);
}

}  // namespace csa2
