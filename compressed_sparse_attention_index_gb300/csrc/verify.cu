// Which drafted tokens the target's probabilities accept, and the token that comes
// after them (csa2_verify_drafts).
//
// Speculative sampling with given random numbers: token x_{t+1}, drawn from q_t, stays while
// u_t q_t(x) < p_t(x); at the first refusal the next token is drawn from max(p_t - q_t, 0), without
// one from the last row's p, by inverting the running sum at v times its total.  Greedy: x_{t+1}
// stays while it is the largest entry of row t.
//
// A token is a whole number, so which side of a border a sum falls on has to be that of the exact
// one: u q is a product of two fp32 in fp64 (exact), p - q and the running sums are pairs of fp32
// (an fp32 sum of 131,072 probabilities picks another token in a call of a few hundred; fp64 has a
// sixtieth of fp32's rate here, and 64 rows would take 55 us of it), and the last few sums are fp64.
//
// What bounds it: one row of p, and of q where a draft was refused, for each sequence (HBM; a few
// sequences: a chain of loads).  A sequence's row is dealt to the CTAs of a cluster, whose sums meet
// in each of them through distributed shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace csa2 {

constexpr int kVfThreads = 512, kVfWarps = kVfThreads / 32, kVfMaxParts = 8;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// What is no probability (negative, NaN, above 2^96) counts as none.
__device__ __forceinline__ float probability(float x) { return x >= 0.f && x <= 0x1p96f ? x : 0.f; }

// A row of `n` elements in groups that start on 16-byte boundaries: group k has elements
// [k VEC - skew, .. + VEC), the first and the last one's may lie outside the row.
template <class T>
struct ProbRow {
  static constexpr int kVec = 16 / sizeof(T);
  const T *row;
  int n, skew;
  __device__ __forceinline__ ProbRow(const T *r, int n_) : row(r), n(n_), skew((int)(((uintptr_t)r / sizeof(T)) % kVec)) {}
  __device__ __forceinline__ int groups() const { return (n + skew + kVec - 1) / kVec; }
};
// Elements e0 .. e0 + VEC of a row, as they are; `none` outside.  wide: e0 is on a 16-byte boundary.
template <class T>
__device__ __forceinline__ void load_group(const T *row, int n, int e0, bool wide, float none, float (&x)[16 / sizeof(T)]) {
  constexpr int V = 16 / sizeof(T);
  if (wide && e0 >= 0 && e0 + V <= n) {
    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(row + e0));
    const T *y = reinterpret_cast<const T *>(&w);
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = to_f32(y[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = e0 + i >= 0 && e0 + i < n ? to_f32(row[e0 + i]) : none;
  }
}

// h + l: a sum of fp32 numbers to twice fp32's precision
struct Pair32 {
  float h, l;
  __device__ __forceinline__ void add(float x, float rest) {
    const float s = h + x, b = s - h;
    l += (h - (s - b)) + (x - b) + rest;
    h = s;
  }
  __device__ __forceinline__ double f64() const { return (double)h + (double)l; }
};

// What the sampled token is drawn from: weights w_e of a row's elements.
template <class T>
struct Weights {
  const T *p, *q;               // q: null, none
  int n, skew, out;             // out: an element of weight 0, or -1
  bool q_wide;
  // the group's weights, as value and what its rounding left
  __device__ __forceinline__ void get(int k, float (&w)[16 / sizeof(T)], float (&rest)[16 / sizeof(T)]) const {
    constexpr int V = 16 / sizeof(T);
    const int e0 = k * V - skew;
    load_group(p, n, e0, true, 0.f, w);
    float y[V];
    if (q != nullptr) load_group(q, n, e0, q_wide, 0.f, y);
#pragma unroll
    for (int i = 0; i < V; i++) {
      const float a = probability(w[i]), b = q != nullptr ? probability(y[i]) : 0.f;
      const float d = a - b;
      const bool some = d > 0.f && e0 + i != out;
      w[i] = some ? d : 0.f;
      rest[i] = some ? (a - d) - b : 0.f;          // exact, as a >= b >= 0
    }
  }
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Stores v at the place of p (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ void put_f64(const double *p, uint32_t rank, double v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(a), "d"(v) : "memory");
}

template <class T>
__global__ void __launch_bounds__(kVfThreads) verify_sample_kernel(const __grid_constant__ VerifyArgs A) {
  constexpr int V = 16 / sizeof(T);
  __shared__ double sums[2][kVfMaxParts * kVfWarps];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, parts = gridDim.x;
  const int b = blockIdx.y;
  const uint32_t rank = cluster_rank();
  griddep_wait();
  griddep_launch();
  const int c0 = __ldg(A.first + b), c1 = __ldg(A.first + b + 1);
  const bool bad = c0 < 0 || c1 < c0 || c1 > A.n_rows;
  if (bad || c1 == c0) {                             // (the whole cluster alike)
    if (t == 0 && rank == 0) {
      A.kept[b] = 0;
      A.next[b] = -1;
      if (bad) record_error(A.status, CSA2_ERR_BOUNDS);
    }
    return;
  }
  const T *target = static_cast<const T *>(A.target), *draft = static_cast<const T *>(A.draft);
  // the first refused draft: every warp for itself, a lane to a draft
  const int drafts = c1 - c0 - 1;
  int accepted = drafts, refused_token = -1;
  for (int i0 = 0; i0 < drafts; i0 += 32) {
    const int i = i0 + lane;
    bool ok = true;
    int x = -1;
    if (i < drafts) {
      const int64_t r = c0 + i;
      x = __ldg(A.tokens + r + 1);
      ok = x >= 0 && x < A.vocab;
      if (ok) {
        const float p = probability(to_f32(target[r * A.target_stride + x]));
        const float q = draft != nullptr ? probability(to_f32(draft[r * A.draft_stride + x])) : 1.f;
        ok = (double)__ldg(A.u + r) * (double)q < (double)p;
      } else {
        x = -1;
      }
    }
    const uint32_t no = __ballot_sync(0xFFFFFFFFu, !ok);
    if (no != 0u) {
      const int from = __ffs((int)no) - 1;
      accepted = i0 + from;
      refused_token = __shfl_sync(0xFFFFFFFFu, x, from);
      if (refused_token < 0 && t == 0 && rank == 0) record_error(A.status, CSA2_ERR_BOUNDS);
      break;
    }
  }
  const int64_t row = c0 + accepted;
  Weights<T> W;
  const ProbRow<T> P(target + row * A.target_stride, A.vocab);
  W.p = P.row;
  W.n = A.vocab;
  W.skew = P.skew;
  const bool refused = accepted < drafts;
  W.q = refused && draft != nullptr ? draft + row * A.draft_stride : nullptr;
  W.q_wide = W.q != nullptr && ProbRow<T>(W.q, A.vocab).skew == W.skew;
  W.out = refused && draft == nullptr ? refused_token : -1;
  const int groups = P.groups(), segs = parts * kVfWarps;
  // this warp's segment of the row
  const int per = (groups + segs - 1) / segs, seg = (int)rank * kVfWarps + warp;
  const int g0 = min(seg * per, groups), g1 = min(g0 + per, groups);
  const double v = (double)__ldg(A.v + b);
  int next = -1;
#pragma unroll 1
  for (int pass = 0; pass < 2; pass++) {
    Pair32 s = {0.f, 0.f};
#pragma unroll 2
    for (int k = g0 + lane; k < g1; k += 32) {
      float w[V], rest[V];
      W.get(k, w, rest);
#pragma unroll
      for (int i = 0; i < V; i++) s.add(w[i], rest[i]);
    }
    double sum = s.f64();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane < parts) put_f64(&sums[pass][seg], (uint32_t)lane, sum);
    __syncwarp();
    cluster_sync();
    // every warp: the segment in which the running sum passes v times the total
    double run = 0.0, at[kVfMaxParts * kVfWarps / 32];
#pragma unroll
    for (int c = 0; c < kVfMaxParts * kVfWarps / 32; c++) {
      double x = c * 32 + lane < segs ? sums[pass][c * 32 + lane] : 0.0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
      }
      at[c] = run + x;
      run = __shfl_sync(0xFFFFFFFFu, at[c], 31);
    }
    if (!(run > 0.0)) {                              // nothing is left of p - q: p itself, else no token
      W.q = nullptr;
      W.out = -1;
      continue;
    }
    const double goal = v * run;
    int hit = -1, some = 0;
    double before = 0.0, carry = 0.0;                // (carry: of the 32 segments before)
#pragma unroll
    for (int c = 0; c < kVfMaxParts * kVfWarps / 32; c++) {
      const double left = __shfl_up_sync(0xFFFFFFFFu, at[c], 1);
      const double ahead = lane > 0 ? left : carry;
      carry = __shfl_sync(0xFFFFFFFFu, at[c], 31);
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, at[c] > goal);
      const uint32_t any = __ballot_sync(0xFFFFFFFFu, at[c] > ahead);
      if (any != 0u) some = c * 32 + 31 - __clz((int)any);
      if (hit < 0 && past != 0u) {
        hit = c * 32 + __ffs((int)past) - 1;
        before = __shfl_sync(0xFFFFFFFFu, ahead, hit & 31);
      }
    }
    const bool end = hit < 0;                        // (v is not below 1: the last element that weighs anything)
    if (end) hit = some;
    if (hit == seg) {
      // ------------------------------------------------ inside the segment, 32 groups at a time
      int last = -1;
      for (int k0 = g0; k0 < g1 && next < 0; k0 += 32) {
        float w[V], rest[V];
        const bool in = k0 + lane < g1;
        Pair32 y = {0.f, 0.f};
        int mine = -1;
        if (in) {
          W.get(k0 + lane, w, rest);
#pragma unroll
          for (int i = 0; i < V; i++) {
            y.add(w[i], rest[i]);
            if (w[i] > 0.f) mine = (k0 + lane) * V - W.skew + i;
          }
        }
        double x = y.f64();
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double z = __shfl_up_sync(0xFFFFFFFFu, x, o);
          if (lane >= o) x += z;
        }
        last = max(last, __reduce_max_sync(0xFFFFFFFFu, mine));
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, !end && in && before + x > goal);
        if (past != 0u) {
          const int from = __ffs((int)past) - 1;
          const double left = __shfl_up_sync(0xFFFFFFFFu, x, 1);
          const double z = lane > 0 ? before + left : before;
          int e = mine;
          if (lane == from) {
#pragma unroll
            for (int i = V - 1; i >= 0; i--) {       // (backwards: the first that passes stays)
              double zi = z;
              for (int j = 0; j <= i; j++) zi += (double)w[j] + (double)rest[j];
              if (w[i] > 0.f && zi > goal) e = (k0 + lane) * V - W.skew + i;
            }
          }
          next = __shfl_sync(0xFFFFFFFFu, e, from);
        }
        before += __shfl_sync(0xFFFFFFFFu, x, 31);
      }
      if (next < 0) next = last;
      if (lane == 0) A.next[b] = next;
    }
    if (t == 0 && rank == 0) A.kept[b] = 1 + accepted;
    return;                                          // (the whole cluster: run is the same in all of it)
  }
  if (t == 0 && rank == 0) {
    A.kept[b] = 1 + accepted;
    A.next[b] = -1;
    record_error(A.status, CSA2_ERR_BOUNDS);
  }
}

// ------------------------------------------------------------------ greedy
// The largest element of a part of a row: its order key above the complement of its index, so that
// the largest word is the largest element, the lowest index among equals (0: nothing but NaN).
template <class T>
__global__ void __launch_bounds__(kVfThreads) verify_best_kernel(const __grid_constant__ VerifyArgs A) {
  constexpr int V = 16 / sizeof(T);
  __shared__ unsigned long long best_sh[kVfWarps];
  const int t = threadIdx.x, parts = gridDim.x;
  const int64_t row = blockIdx.y;
  griddep_wait();
  griddep_launch();
  if (row >= __ldg(A.first + A.n_seq)) return;       // (a row of no sequence)
  const ProbRow<T> P(static_cast<const T *>(A.target) + row * A.target_stride, A.vocab);
  const int groups = P.groups(), per = (groups + parts - 1) / parts;
  const int g0 = min((int)blockIdx.x * per, groups), g1 = min(g0 + per, groups);
  unsigned long long best = 0ull;
#pragma unroll 4
  for (int k = g0 + t; k < g1; k += kVfThreads) {
    float x[V];
    const int e0 = k * V - P.skew;
    load_group(P.row, P.n, e0, true, __int_as_float(0x7FC00000), x);
#pragma unroll
    for (int i = 0; i < V; i++)
      if (x[i] == x[i]) {
        const unsigned long long w = (unsigned long long)order_key(x[i]) << 32 | (uint32_t) ~(uint32_t)(e0 + i);
        best = w > best ? w : best;
      }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long w = __shfl_xor_sync(0xFFFFFFFFu, best, o);
    best = w > best ? w : best;
  }
  if ((t & 31) == 0) best_sh[t >> 5] = best;
  __syncthreads();
  if (t == 0) {
    for (int w = 1; w < kVfWarps; w++) best = best_sh[w] > best ? best_sh[w] : best;
    A.best[row * kVfMaxParts + blockIdx.x] = best;
  }
}

// A warp per sequence, a lane to a row.
__global__ void __launch_bounds__(128) verify_greedy_kernel(const __grid_constant__ VerifyArgs A, int parts) {
  const int b = (int)blockIdx.x * 4 + (int)(threadIdx.x >> 5), lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch();
  if (b >= A.n_seq) return;
  const int c0 = __ldg(A.first + b), c1 = __ldg(A.first + b + 1);
  const bool bad = c0 < 0 || c1 < c0 || c1 > A.n_rows || c1 > __ldg(A.first + A.n_seq);
  int kept = 0, next = -1;
  if (!bad && c1 > c0) {
    for (int r0 = c0; r0 < c1; r0 += 32) {
      const int r = r0 + lane;
      int pick = -1, x = -1;
      if (r < c1) {
        unsigned long long best = 0ull;
        for (int p = 0; p < parts; p++) {
          const unsigned long long w = __ldcg(A.best + (int64_t)r * kVfMaxParts + p);
          best = w > best ? w : best;
        }
        pick = best == 0ull ? -1 : (int)~(uint32_t)best;
        if (r + 1 < c1) x = __ldg(A.tokens + r + 1);
      }
      const uint32_t no = __ballot_sync(0xFFFFFFFFu, r + 1 >= c1 || pick != x || pick < 0);
      if (no != 0u) {
        const int from = __ffs((int)no) - 1;
        kept = r0 + from - c0 + 1;
        next = __shfl_sync(0xFFFFFFFFu, pick, from);
        x = __shfl_sync(0xFFFFFFFFu, x, from);
        if (lane == 0 && (next < 0 || (r0 + from + 1 < c1 && (x < 0 || x >= A.vocab)))) record_error(A.status, CSA2_ERR_BOUNDS);
        break;
      }
    }
  }
  if (lane == 0) {
    A.kept[b] = kept;
    A.next[b] = next;
    if (bad) record_error(A.status, CSA2_ERR_BOUNDS);
  }
}

size_t verify_workspace_bytes(int n_rows) { return (size_t)n_rows * kVfMaxParts * sizeof(unsigned long long); }

template <class T>
static cudaError_t launch_verify_as(VerifyArgs A, bool greedy, cudaStream_t st) {
  const int64_t sms = device_sm_count(current_device());
  // parts of a row: about two CTAs an SM in all, and at least 16 KB of the row each
  const int64_t rows = greedy ? A.n_rows : A.n_seq, most = (int64_t)A.vocab * (int64_t)sizeof(T) / 16384;
  int parts = 1;
  while (parts < kVfMaxParts && 2 * parts <= most && parts * rows < 2 * sms) parts *= 2;
  if (!greedy) return launch_pdl(verify_sample_kernel<T>, dim3((unsigned)parts, (unsigned)A.n_seq), dim3(kVfThreads), 0, st, (unsigned)parts, A);
  if (A.n_rows > 0) {
    const cudaError_t e = launch_pdl(verify_best_kernel<T>, dim3((unsigned)parts, (unsigned)A.n_rows), dim3(kVfThreads), 0, st, 1u, A);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(verify_greedy_kernel, dim3((unsigned)(A.n_seq + 3) / 4), dim3(128), 0, st, 1u, A, parts);
}

cudaError_t launch_verify(const VerifyArgs &A, int dtype, bool greedy, cudaStream_t st) {
  switch (dtype) {
    case CSA2_PROB_F32: return launch_verify_as<float>(A, greedy, st);
    case CSA2_PROB_BF16: return launch_verify_as<__nv_bfloat16>(A, greedy, st);
    default: return launch_verify_as<__half>(A, greedy, st);
  }
}

}  // namespace csa2
