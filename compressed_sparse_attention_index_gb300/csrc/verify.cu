// Which drafted tokens the target's probabilities accept, and the token that comes
// after them (csa2_verify_drafts).
//
// Speculative sampling with given random numbers: token x_{t+1}, drawn from q_t, stays while
// u_t q_t(x) < p_t(x); at the first refusal the next token is drawn from max(p_t - q_t, 0), without
// one from the last row's p, by inverting the running sum at v times its total.  Greedy: x_{t+1}
// stays while it is the largest entry of row t.
//
// A token is a whole number, so which side of a border a sum falls on has to be that of the exact
// one: u q is a product of two fp32 in fp64 (exact), and p - q and the running sums are pairs of fp32
// (an fp32 sum of 131,072 probabilities picks another token in a call of a few hundred; fp64 has a
// sixtieth of fp32's rate here, and a few sums of it in every warp took half of the kernel's time).  Pairs are good
// to 2^-46 of the total in rows of up to 2^20, and to 2^-42 in the longest, where the lower halves add up many roundings.
//
// What bounds it: one row of p, and of q where a draft was refused, for each sequence (HBM; a few
// sequences: a chain of loads).  A sequence's row is dealt to the warps of a cluster in
// contiguous segments, whose sums meet in each CTA through distributed shared memory; the CTA that has the
// segment where the running sum passes looks through it with all its threads (one warp, 32 groups at a
// time, took 25 us of a 4,096-entry segment).  With rows that are not in L2 yet: 256 of 131,072 fp32 probabilities 34 us, 4.0 TB/s; 64 pairs of
// 100,003 in bf16 15; one row 6.7, a chain of seven loads or barriers.  Greedy, 384 rows of 131,072 in bf16: 20, 5.0 TB/s of all rows, in two
// launches, the first of 768 CTAs (five or six an SM).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace csa2 {

constexpr int kVfThreads = 256, kVfWarps = kVfThreads / 32, kVfMaxParts = 16;
constexpr int kVfCtas = 4, kVfBestCtas = 6;         // of an SM at a time (sampled, greedy)

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// What is no probability (negative, NaN, above 2^96) counts as none.
__device__ __forceinline__ float probability(float x) { return __float_as_uint(x) <= 0x6F800000u ? x : 0.f; }

// Four words of a row: 16 / sizeof(T) elements as fp32.
__device__ __forceinline__ void widen(const uint4 &w, float (&x)[4], float) {
  x[0] = __uint_as_float(w.x);
  x[1] = __uint_as_float(w.y);
  x[2] = __uint_as_float(w.z);
  x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void widen(const uint4 &w, float (&x)[8], __nv_bfloat16) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    x[2 * i] = bf16_lo(v[i]);
    x[2 * i + 1] = bf16_hi(v[i]);
  }
}
__device__ __forceinline__ void widen(const uint4 &w, float (&x)[8], __half) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// A row of n elements in groups of VEC that start on 16-byte boundaries: group k has elements
// k VEC - skew .. + VEC; the first and the last one's may lie outside the row (`none` there).
template <class T>
struct ProbRow {
  static constexpr int kVec = 16 / sizeof(T);
  const T *row;
  int n, skew;
  __device__ __forceinline__ ProbRow(const T *r, int n_) : row(r), n(n_), skew((int)(((uintptr_t)r / sizeof(T)) % kVec)) {}
  __device__ __forceinline__ int groups() const { return (n + skew + kVec - 1) / kVec; }
  __device__ __forceinline__ int first(int k) const { return k * kVec - skew; }
  __device__ __forceinline__ bool inside(int k) const { return first(k) >= 0 && first(k) + kVec <= n; }
  __device__ __forceinline__ uint4 wide(int k) const { return __ldg(reinterpret_cast<const uint4 *>(row + first(k))); }
  // element by element
  __device__ __forceinline__ void edge(int k, float none, float (&x)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; i++) {
      const int e = first(k) + i;
      x[i] = e >= 0 && e < n ? to_f32(row[e]) : none;
    }
  }
  __device__ __forceinline__ void get(int k, float none, float (&x)[kVec]) const {
    if (inside(k)) widen(wide(k), x, T());
    else edge(k, none, x);
  }
};

// h + l: a sum to twice fp32's precision
struct Pair32 {
  float h, l;
  __device__ __forceinline__ void add(float x) {
    const float s = h + x, b = s - h;
    l += (h - (s - b)) + (x - b);
    h = s;
  }
  __device__ __forceinline__ void add(const Pair32 &y) {
    add(y.h);
    l += y.l;
  }
  __device__ __forceinline__ Pair32 up(int o) const { return {__shfl_up_sync(0xFFFFFFFFu, h, o), __shfl_up_sync(0xFFFFFFFFu, l, o)}; }
  __device__ __forceinline__ Pair32 from(int lane) const { return {__shfl_sync(0xFFFFFFFFu, h, lane), __shfl_sync(0xFFFFFFFFu, l, lane)}; }
};
__device__ __forceinline__ bool above(const Pair32 &a, const Pair32 &b) { return (a.h - b.h) + (a.l - b.l) > 0.f; }
// sum over the warp's lanes up to this one
__device__ __forceinline__ Pair32 warp_scan(Pair32 x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair32 y = x.up(o);
    if (lane >= o) x.add(y);
  }
  return x;
}

// What the sampled token is drawn from: the weights max(p - q, 0) of a row's elements.
template <class T>
struct Weights {
  static constexpr int V = 16 / sizeof(T);
  ProbRow<T> p, q;              // q.row null: none
  int out;                      // an element of weight 0, or -1
  bool wide;                    // q's groups are p's
  // a group's weights, as value and what its rounding left
  __device__ __forceinline__ void weigh(int k, float (&w)[V], const float (&y)[V], float (&rest)[V]) const {
#pragma unroll
    for (int i = 0; i < V; i++) {
      const float a = probability(w[i]), b = probability(y[i]), d = a - b;
      w[i] = fmaxf(d, 0.f);
      rest[i] = d > 0.f ? (a - d) - b : 0.f;         // exact, as a >= b >= 0
    }
  }
  __device__ __forceinline__ void plain(int k, float (&w)[V]) const {
#pragma unroll
    for (int i = 0; i < V; i++) w[i] = probability(w[i]);
    const int x = out - p.first(k);
    if ((unsigned)x < (unsigned)V && out >= 0) {
#pragma unroll
      for (int i = 0; i < V; i++)
        if (i == x) w[i] = 0.f;
    }
  }
  __device__ __forceinline__ void get_q(int k, float (&y)[V]) const {
    if (wide && p.inside(k)) {
      widen(__ldg(reinterpret_cast<const uint4 *>(q.row + p.first(k))), y, T());
    } else {
#pragma unroll
      for (int i = 0; i < V; i++) {
        const int e = p.first(k) + i;
        y[i] = e >= 0 && e < p.n ? to_f32(q.row[e]) : 0.f;
      }
    }
  }
  __device__ __forceinline__ void get(int k, float (&w)[V], float (&rest)[V]) const {
    p.get(k, 0.f, w);
    if (q.row != nullptr) {
      float y[V];
      get_q(k, y);
      weigh(k, w, y, rest);
    } else {
      plain(k, w);
#pragma unroll
      for (int i = 0; i < V; i++) rest[i] = 0.f;
    }
  }
  __device__ __forceinline__ void take(Pair32 &s, float (&w)[V], const float (&y)[V], int k) const {
    float rest[V];
    weigh(k, w, y, rest);
#pragma unroll
    for (int i = 0; i < V; i++) {
      s.add(w[i]);
      s.l += rest[i];
    }
  }
  // this lane's part of groups [g0, g1): every 32nd, four of them in flight (the row's first and last group, which may
  // not be whole, on their own)
  __device__ __forceinline__ Pair32 sum(int g0, int g1, int lane) const {
    Pair32 s = {0.f, 0.f};
    for (int side = 0; side < 2 && g0 < g1; side++) {
      const int k = side == 0 ? g0 : g1 - 1;
      if (p.inside(k)) continue;
      if (side == 0) g0++;
      else g1--;
      if (lane > 0) continue;
      float w[V], rest[V];
      get(k, w, rest);
#pragma unroll
      for (int i = 0; i < V; i++) {
        s.add(w[i]);
        s.l += rest[i];
      }
    }
    int k = g0 + lane;
    if (q.row == nullptr) {
      for (; k < g1; k += 128) {
        uint4 a[4];
#pragma unroll
        for (int u = 0; u < 4; u++) a[u] = k + 32 * u < g1 ? p.wide(k + 32 * u) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < 4; u++) {
          float w[V];
          widen(a[u], w, T());
          plain(k + 32 * u, w);
#pragma unroll
          for (int i = 0; i < V; i++) s.add(w[i]);
        }
      }
    } else if (wide) {
      for (; k < g1; k += 128) {
        uint4 a[4], b[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
          const bool in = k + 32 * u < g1;
          a[u] = in ? p.wide(k + 32 * u) : make_uint4(0u, 0u, 0u, 0u);
          b[u] = in ? __ldg(reinterpret_cast<const uint4 *>(q.row + p.first(k + 32 * u))) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < 4; u++) {
          float w[V], y[V];
          widen(a[u], w, T());
          widen(b[u], y, T());
          take(s, w, y, k + 32 * u);
        }
      }
    } else {
      for (; k < g1; k += 32) {
        float w[V], y[V];
        widen(p.wide(k), w, T());
        get_q(k, y);
        take(s, w, y, k);
      }
    }
    return s;
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
__device__ __forceinline__ void put_pair(const float2 *p, uint32_t rank, const Pair32 &v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.h), "f"(v.l) : "memory");
}

// The place in an ascending list of sums (32 SLOTS of them, lane and slot c: number 32 c + lane, x[c] the sum
// of its own) where the running sum first passes goal: its number, -1 where none does, the sum ahead of it, and
// the last number that adds anything.
template <int SLOTS>
__device__ __forceinline__ int find_pass(const Pair32 (&x)[SLOTS], const Pair32 &goal, int lane, Pair32 &ahead, int &some) {
  Pair32 in[SLOTS];
#pragma unroll
  for (int c = 0; c < SLOTS; c++) in[c] = x[c];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Pair32 y[SLOTS];                                 // (the slots' scans beside one another)
#pragma unroll
    for (int c = 0; c < SLOTS; c++) y[c] = in[c].up(o);
#pragma unroll
    for (int c = 0; c < SLOTS; c++)
      if (lane >= o) in[c].add(y[c]);
  }
  int hit = -1;
  Pair32 run = {0.f, 0.f};
  some = -1;
#pragma unroll
  for (int c = 0; c < SLOTS; c++) {
    Pair32 at = run, before = in[c].up(1);
    at.add(in[c]);
    if (lane == 0) before = {0.f, 0.f};
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, above(at, goal) && x[c].h > 0.f);
    const uint32_t any = __ballot_sync(0xFFFFFFFFu, x[c].h > 0.f);
    if (any != 0u) some = c * 32 + 31 - __clz((int)any);
    if (hit < 0 && past != 0u) {
      const int from = __ffs((int)past) - 1;
      hit = c * 32 + from;
      ahead = run;
      ahead.add(before.from(from));
    }
    run.add(in[c].from(31));
  }
  return hit;
}

template <class T>
__global__ void __launch_bounds__(kVfThreads, kVfCtas) verify_sample_kernel(const __grid_constant__ VerifyArgs A) {
  constexpr int V = 16 / sizeof(T), kSlots = kVfMaxParts * kVfWarps / 32;
  __shared__ float2 sums[2][kVfMaxParts * kVfWarps], inner[kVfWarps];
  __shared__ int accepted_sh, refused_sh;
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
  if (parts > 1) ptx::cluster_begin();
  const T *target = static_cast<const T *>(A.target), *draft = static_cast<const T *>(A.draft);
  // the first refused draft, a lane to a draft
  const int drafts = c1 - c0 - 1;
  if (warp == 0) {
    int accepted = drafts, refused = -1;
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
        refused = __shfl_sync(0xFFFFFFFFu, x, from);
        if (refused < 0 && lane == 0 && rank == 0) record_error(A.status, CSA2_ERR_BOUNDS);
        break;
      }
    }
    if (lane == 0) {
      accepted_sh = accepted;
      refused_sh = refused;
    }
  }
  __syncthreads();
  const int accepted = accepted_sh;
  const bool refused = accepted < drafts;
  const int64_t row = c0 + accepted;
  const ProbRow<T> P(target + row * A.target_stride, A.vocab);
  const ProbRow<T> Q(refused && draft != nullptr ? draft + row * A.draft_stride : nullptr, A.vocab);
  Weights<T> W = {P, Q, refused && draft == nullptr ? refused_sh : -1, Q.skew == P.skew};
  const int groups = P.groups(), segs = parts * kVfWarps;
  // this warp's segment of the row
  const int per = (groups + segs - 1) / segs, seg = (int)rank * kVfWarps + warp;
  const int g0 = min(seg * per, groups), g1 = min(g0 + per, groups);
  const float v = __ldg(A.v + b);
#pragma unroll 1
  for (int pass = 0; pass < 2; pass++) {
    Pair32 s = warp_scan(W.sum(g0, g1, lane), lane).from(31);
    if (parts > 1 && pass == 0) ptx::cluster_begun();          // (the others' sums may be written)
    if (lane < parts) put_pair(&sums[pass][seg], (uint32_t)lane, s);
    __syncwarp();
    cluster_sync();
    Pair32 x[kSlots], total = {0.f, 0.f}, ahead = {0.f, 0.f}, none = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kSlots; c++) {
      const float2 y = c * 32 + lane < segs ? sums[pass][c * 32 + lane] : make_float2(0.f, 0.f);
      x[c] = {y.x, y.y};
      total.add(x[c]);
    }
    total = warp_scan(total, lane).from(31);
    if (!(total.h > 0.f)) {                          // nothing is left of p - q: p itself, else no token
      W.q.row = nullptr;
      W.out = -1;
      continue;
    }
    // the segment in which the running sum passes v times the total
    Pair32 goal = {v * total.h, 0.f};
    goal.l = fmaf(v, total.h, -goal.h) + v * total.l;
    int some;
    int hit = find_pass<kSlots>(x, goal, lane, ahead, some);
    const bool end = hit < 0;                        // (v is not below 1: the last element that weighs anything)
    if (end) hit = some;
    if (t == 0 && rank == 0) A.kept[b] = 1 + accepted;
    if (hit / kVfWarps != (int)rank) return;         // (another CTA of the cluster has it)
    // ---------------------------------------------------- inside the segment: contiguous groups to every thread
    const int h0 = min(hit * per, groups), h1 = min(h0 + per, groups), each = (h1 - h0 + kVfThreads - 1) / kVfThreads;
    const int k0 = min(h0 + t * each, h1), k1 = min(k0 + each, h1);
    Pair32 own = none;
    for (int k = k0; k < k1; k++) {
      float w[V], rest[V];
      W.get(k, w, rest);
#pragma unroll
      for (int i = 0; i < V; i++) {
        own.add(w[i]);
        own.l += rest[i];
      }
    }
    const Pair32 in = warp_scan(own, lane);
    if (lane == 31) inner[warp] = make_float2(in.h, in.l);
    __syncthreads();
    const float2 y = lane < kVfWarps ? inner[lane] : make_float2(0.f, 0.f);
    const Pair32 z[1] = {{y.x, y.y}};
    // (rounding may leave the goal behind the last one: then the last that weighs anything)
    Pair32 to = goal;
    to.add(-ahead.h);
    to.l -= ahead.l;
    Pair32 ahead2 = none;
    int warp_hit = end ? -1 : find_pass<1>(z, to, lane, ahead2, some);
    const uint32_t any_warp = __ballot_sync(0xFFFFFFFFu, z[0].h > 0.f);
    const bool last_warp = warp_hit < 0;
    if (last_warp) warp_hit = 31 - __clz((int)any_warp);
    if (warp != warp_hit) return;
    const Pair32 o[1] = {own};
    Pair32 to2 = to;
    to2.add(-ahead2.h);
    to2.l -= ahead2.l;
    Pair32 ahead3 = none;
    int lane_hit = last_warp ? -1 : find_pass<1>(o, to2, lane, ahead3, some);
    const uint32_t any_lane = __ballot_sync(0xFFFFFFFFu, own.h > 0.f);
    const bool last_lane = lane_hit < 0;
    if (last_lane) lane_hit = 31 - __clz((int)any_lane);
    if (lane != lane_hit) return;
    Pair32 at = ahead3;
    int next = -1;
    bool passed = false;
    for (int k = k0; k < k1 && !passed; k++) {
      float w[V], rest[V];
      W.get(k, w, rest);
#pragma unroll
      for (int i = 0; i < V; i++) {
        at.add(w[i]);
        at.l += rest[i];
        if (w[i] > 0.f && !passed) {
          next = W.p.first(k) + i;
          passed = !last_lane && above(at, to2);
        }
      }
    }
    A.next[b] = next;
    return;
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
// A lane's elements come in ascending order, so a comparison and two selections keep its largest.
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
  float top = -INFINITY;
  int at = -1;
  auto take = [&](int k, const float (&x)[V]) {
    const int e0 = P.first(k);
#pragma unroll
    for (int i = 0; i < V; i++)
      if (x[i] > top) {
        top = x[i];
        at = e0 + i;
      }
  };
  // (the row's first and last group, which may not be whole, on their own; a lane's elements still ascend)
  int a0 = g0, a1 = g1;
  if (a0 < a1 && !P.inside(a0)) {
    if (t == 0) {
      float x[V];
      P.edge(a0, -INFINITY, x);
      take(a0, x);
    }
    a0++;
  }
  if (a0 < a1 && !P.inside(a1 - 1)) a1--;
  int k = a0 + t;
  for (; k + 3 * kVfThreads < a1; k += 4 * kVfThreads) {
    uint4 w[4];
#pragma unroll
    for (int u = 0; u < 4; u++) w[u] = P.wide(k + u * kVfThreads);
#pragma unroll
    for (int u = 0; u < 4; u++) {
      float x[V];
      widen(w[u], x, T());
      take(k + u * kVfThreads, x);
    }
  }
  for (; k < a1; k += kVfThreads) {
    float x[V];
    widen(P.wide(k), x, T());
    take(k, x);
  }
  if (a1 < g1 && a1 >= a0 && t == 0) {
    float x[V];
    P.edge(a1, -INFINITY, x);
    take(a1, x);
  }
  // nothing above -inf: the first -inf, if any
  if (__syncthreads_or(at >= 0) == 0) {
    for (int k = g0 + t; k < g1 && at < 0; k += kVfThreads) {
      float x[V];
      P.get(k, __int_as_float(0x7FC00000), x);
#pragma unroll
      for (int i = V - 1; i >= 0; i--)
        if (x[i] == -INFINITY) at = P.first(k) + i;
    }
  }
  unsigned long long best = at >= 0 ? (unsigned long long)order_key(top) << 32 | (uint32_t) ~(uint32_t)at : 0ull;
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
  // parts of a row: as many as run at a time (256 rows of 131,072 in two waves took twice as long), of at
  // least 16 KB of the row each; clusters of more than eight CTAs for a few rows only (32 rows: 9.4 us with eight, 13
  // with sixteen; one row: 7.6, 6.6)
  const int64_t rows = greedy ? A.n_rows : A.n_seq, most = (int64_t)A.vocab * (int64_t)sizeof(T) / 16384;
  int parts = 1;
  while (parts < kVfMaxParts && 2 * parts <= most && 2 * parts * rows <= (greedy ? kVfBestCtas : kVfCtas) * sms &&
         (greedy || parts < 8 || rows * 32 <= sms))
    parts *= 2;
  static std::atomic<int> attr_done[kMaxDevices];
  const cudaError_t attr = once_per_device(attr_done, current_device(), [&] {
    return cudaFuncSetAttribute(verify_sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (attr != cudaSuccess) return attr;
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
