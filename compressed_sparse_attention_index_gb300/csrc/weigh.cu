// The attention weight that cache entries get from a step's queries (csa2_attn_weight):
//
//     w_j = decay prior_j + sum over the queries that see j, and their heads, of
//           exp(scale q_h . k_j - lse_h)
//
// Work: the entries that a sequence's queries see form chunks of 128, its queries groups
// of NQ.  All sequences' (chunk, group) products are dealt to the CTAs (one an SM) in contiguous runs of equal
// numbers, cut between chunks, so that one CTA has all of an entry's queries and sums them in a fixed order.
// With several groups a CTA takes up to 24 chunks at a time (one query a group: 8), group by group: Q stays in shared memory
// for them, their records in L2 for the groups, and their sums in shared memory.  A selection is a
// sequence of its own: its chunks' weights go to scratch, and are added query by query.
//
// Per chunk and group, on the 5th-generation tensor cores:
//   S^T[entry][head] = K . Q^T     tcgen05 kind::f16, M = 128, N = 64 NQ, K = 512
//   w[entry] += sum over heads of 2^(f_h S - lse_h log2 e)
// An entry's heads lie in one row of tensor memory, so the sum is a thread's own.  K (E2M1 x E4M3) is exact
// in f16; every head of Q goes to f16 under a power of two that brings its largest value into [2^14, 2^15),
// so a bf16 value 2^-29 of that and above is exact; f_h = scale log2(e) over that power.  (A first launch does
// that, and lays Q out as the tensor cores read it.)
//
// Warps, with their own barriers between them: two fetch records and one Q by bulk copies; sixteen dequantise,
// a row per thread and 128 dims a team, into tensor memory, where the MMAs read K as their A operand;
// two threads issue the MMAs; eight sum S.
//
// What bounds it.  One query a sequence: a chunk's records take 1,600 cycles of HBM and its MMAs 1,060; it takes 2,200, as the 6,000 instructions
// of its roles (2,600 of them conversions) leave little room for their latencies: 8 x 1,048,576 entries 452 us, 5.5 TB/s, in short runs, and 488 in long ones, where the power
// limit lowers the clock.  Two queries: the MMAs' 2,050 cycles a chunk; 8 x 262,144 entries x 16 queries 1,304 us, 1.69 PFLOP/s; 32 x 65,536 x 5: 470 us
// (505; its fifth query costs nearly as much as two).  One short row is a chain of latencies: 1 x 4,096 entries 9 us, the preparation's 4 among them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
#include <math.h>

#include "attn.cuh"
#include "common.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace csa2 {

constexpr int kWgChunk = 128;                      // entries
constexpr int kWgSumWarps = 8, kWgKWarps = 16, kWgWarps = 32;
constexpr int kWgThreads = kWgWarps * 32;
// Registers: 1,024 threads are launched with 64 each; the summing warps, which read tensor memory ahead of
// their arithmetic, take what the others give up.
constexpr int kWgRegsSum = 88, kWgRegsK = 56, kWgRegsRest = 56;
static_assert(kWgSumWarps * kWgRegsSum + kWgKWarps * kWgRegsK + 8 * kWgRegsRest <= 64 * kWgWarps, "register split");
constexpr int kWgRaw = kWgChunk * kKvBytes;        // one chunk's records
constexpr int kWgQBlock = 64 * 128;                // 64 heads x 64 dims f16: [h/8][h%8][128 B]
constexpr int kWgImage = 8 * kWgQBlock;            // a query as the tensor cores read it
constexpr int kWgMeta = 2 * kHeads * 4;            // its heads' f, then their -lse log2(e)
constexpr int kWgMetas = 8;                        // groups whose f and lse are in shared memory
constexpr int kWgScatter = 8;                      // pages of fewer entries are fetched as scattered records

template <int NQ>
struct WgSmem {
  static constexpr int kStages = NQ == 1 ? 4 : 2;  // records of as many chunks
  static constexpr int kBlock = NQ == 1 ? 8 : 24;  // chunks that take turns at several groups
  static constexpr int kSums = NQ == 1 ? 4 : 2;    // accumulators of S in tensor memory
  static constexpr int kSlots = NQ == 1 ? 16 : 8;  // chunks whose slots are in shared memory
  static constexpr int kQ = 0;                     // [dims / 64][query][heads]
  static constexpr int kRaw = kQ + NQ * kWgImage;
  static constexpr int kAcc = kRaw + kStages * kWgRaw;         // [kBlock chunks][128]
  static constexpr int kMeta = kAcc + kBlock * kWgChunk * 4;
  static constexpr int kSlot = kMeta + kWgMetas * NQ * kWgMeta;
  static constexpr int kPart = kSlot + kSlots * kWgChunk * 4;  // [2][128]: the second query's sums (NQ = 2)
  static constexpr int kEnd = kPart + (NQ == 2 ? 2 * kWgChunk * 4 : 0);
  static constexpr int kAlloc = kEnd + 1024;
  static_assert(kAlloc + 512 <= 227 * 1024, "shared memory");
};
constexpr uint32_t kWgColK = 0, kWgColS = 256, kWgTmemCols = 512;

// What a sequence (a query, for selections) takes: entries, groups, its first query, its queries.
struct WgWs {
  int4 *item;
  int32_t *off;                 // products ahead of it; [items] all of them
  int32_t *q_seq;               // of each query (selections), -1: none
  unsigned char *image;         // [n_q][kWgImage]
  unsigned char *meta;          // [n_q][kWgMeta]
  float *part;                  // [n_q][sel_stride]
};
static size_t wg_up(size_t x) { return (x + 255) / 256 * 256; }
static size_t wg_layout(WgWs *W, void *ws, int n_q, int64_t n_seq, int sel_stride) {
  const size_t items = (size_t)(n_q > n_seq ? n_q : n_seq);
  char *p = static_cast<char *>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char *r = p == nullptr ? nullptr : p + at;
    at += wg_up(bytes);
    return r;
  };
  char *item = take(items * sizeof(int4)), *off = take((items + 1) * 4), *q_seq = take((size_t)n_q * 4);
  char *image = take((size_t)n_q * kWgImage), *meta = take((size_t)n_q * kWgMeta), *part = take((size_t)n_q * (size_t)sel_stride * 4);
  if (W != nullptr) {
    W->item = reinterpret_cast<int4 *>(item);
    W->off = reinterpret_cast<int32_t *>(off);
    W->q_seq = reinterpret_cast<int32_t *>(q_seq);
    W->image = reinterpret_cast<unsigned char *>(image);
    W->meta = reinterpret_cast<unsigned char *>(meta);
    W->part = reinterpret_cast<float *>(part);
  }
  return at;
}
size_t weigh_workspace_bytes(int n_q, int64_t n_seq, int sel_stride) { return wg_layout(nullptr, nullptr, n_q, n_seq, sel_stride); }

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
__device__ __forceinline__ int weigh_col(const WeighArgs &A, int j) { return (int)(((uint64_t)(unsigned)j * A.page_mul) >> A.page_shift); }
__device__ __forceinline__ int64_t weigh_slot(const WeighArgs &A, int b, int j) {
  const int c = weigh_col(A, j);
  const int id = __ldg(A.table + (int64_t)b * A.table_stride + c);
  return id >= 0 && id < A.n_pages ? (int64_t)id * A.page + (j - c * A.page) : -1;
}

// Shared memory by its own addresses (behind the base's alignment the compiler takes pointers for any memory's, and
// loads through them cost half as many instructions again).
__device__ __forceinline__ uint4 wg_lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 wg_lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ ulonglong2 wg_lds2x64(uint32_t a) {
  ulonglong2 v;
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t wg_lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float wg_ldsf(uint32_t a) { return __uint_as_float(wg_lds4(a)); }
__device__ __forceinline__ void wg_sts4(uint32_t a, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }

// ------------------------------------------------------------------ what the products need
constexpr int kPrepThreads = 256, kPrepCtas = 8;     // CTAs of a query
__device__ __forceinline__ float wg_power(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// What selections start from: decay prior, of every entry that a query of the sequence sees.
__device__ __forceinline__ void weigh_decay(const WeighArgs &A, int b, int part, int parts) {
  __shared__ int most_sh;
  const int t = threadIdx.x;
  int c0, c1, most = 0;
  weigh_queries(A, b, c0, c1);
  for (int q = c0 + t; q < c1; q += kPrepThreads) most = max(most, weigh_vis(A, q));
  if (t == 0) most_sh = 0;
  __syncthreads();
  atomicMax(&most_sh, most);
  __syncthreads();
  most = most_sh;
  for (int64_t j = (int64_t)part * kPrepThreads + t; j < most; j += (int64_t)parts * kPrepThreads) {
    const int64_t s = weigh_slot(A, b, (int)j);
    if (s >= 0) A.weight[s] = A.prior != nullptr ? A.decay * A.prior[s] : 0.f;
  }
}

// The first CTA: the items and the products ahead of each.  Eight for each query behind it: its
// heads' powers of two, f16 image and constants.  For selections, where the weights change by more than what is added:
// decay_parts for each sequence behind those.
__global__ void __launch_bounds__(kPrepThreads) weigh_prep_kernel(const __grid_constant__ WeighArgs A, WgWs W, int nq, int decay_parts) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  griddep_wait();
  griddep_launch();
  const int64_t behind = (int64_t)blockIdx.x - 1 - (int64_t)A.n_q * kPrepCtas;
  if (behind >= 0) {
    weigh_decay(A, (int)(behind / decay_parts), (int)(behind % decay_parts), decay_parts);
    return;
  }
  if (blockIdx.x > 0) {
    const int q = ((int)blockIdx.x - 1) / kPrepCtas, part = ((int)blockIdx.x - 1) % kPrepCtas;
    if (A.sel != nullptr && part == 0 && warp == 0) {
      int seq = 0, hi = A.n_seq;                     // the last sequence with first <= q
      while (hi - seq > 1) {
        const int mid = (seq + hi) >> 1;
        if (__ldg(A.first + mid) <= q) seq = mid;
        else hi = mid;
      }
      int c0, c1;
      if (!(weigh_queries(A, seq, c0, c1) && q >= c0 && q < c1)) {
        // a query of no sequence, or ranges that do not ascend: the first one that has it
        seq = INT_MAX;
        for (int b = lane; b < A.n_seq && seq == INT_MAX; b += 32)
          if (weigh_queries(A, b, c0, c1) && q >= c0 && q < c1) seq = b;
        seq = __reduce_min_sync(0xFFFFFFFFu, seq);
      }
      if (lane == 0) W.q_seq[q] = seq < INT_MAX ? seq : -1;
    }
    // a head a warp, 16 dims a lane
    {
      const int h = part * (kPrepThreads / 32) + warp;
      const uint4 *src = reinterpret_cast<const uint4 *>(A.q + ((int64_t)q * kHeads + h) * kDim) + lane * 2;
      const uint4 x = __ldg(src), y = __ldg(src + 1);
      const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      uint32_t m = 0u;
#pragma unroll
      for (int u = 0; u < 8; u++) m = __vmaxu2(m, w[u] & 0x7FFF7FFFu);
      m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
      const float lse = __ldg(A.lse + (int64_t)q * kHeads + h);
      const bool none = m >= 0x7F80u || !(fabsf(lse) < INFINITY);      // not finite: adds nothing
      // max |q| in [2^e, 2^(e + 1)) (below 2^-126 its place among the subnormals)
      const int e = m == 0u ? 14 : m < 0x80u ? -134 + 31 - __clz((int)m) + 1 : (int)(m >> 7) - 127;
      const int by = none ? 0 : 14 - e, b0 = by / 2, b1 = by - b0;      // (2^by itself may be beyond fp32)
      const float s0 = none ? 0.f : wg_power(b0), s1 = wg_power(b1);
      uint32_t o[8];
#pragma unroll
      for (int u = 0; u < 8; u++) {
        const float a = none ? 0.f : bf16_lo(w[u]) * s0 * s1, c = none ? 0.f : bf16_hi(w[u]) * s0 * s1;
        const __half2 p = __floats2half2_rn(a, c);
        o[u] = *reinterpret_cast<const uint32_t *>(&p);
      }
      // dims 16 lane ..: block of 64 dims lane / 4, 16-byte chunks 2 (lane % 4) and the next
      unsigned char *dst = W.image + (int64_t)q * kWgImage + (lane >> 2) * kWgQBlock + (h >> 3) * 1024;
      *reinterpret_cast<uint4 *>(dst + sw128(h & 7, (lane & 3) * 2)) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4 *>(dst + sw128(h & 7, (lane & 3) * 2 + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
      if (lane == 0) {
        float *meta = reinterpret_cast<float *>(W.meta + (int64_t)q * kWgMeta);
        meta[h] = none ? 0.f : A.scale * 1.4426950408889634f * wg_power(-b0) * wg_power(-b1);
        meta[kHeads + h] = none ? -INFINITY : -lse * 1.4426950408889634f;
      }
    }
    return;
  }
  // ---------------------------------------------------- items
  const bool sel = A.sel != nullptr;
  const int items = sel ? A.n_q : A.n_seq;
  __shared__ int wt[kPrepThreads / 32], base_sh;
  // (ranges that cross may have more products than 31 bits hold: sums stay at INT_MAX then)
  auto sum = [](int a, int b) { return (int)min((unsigned)a + (unsigned)b, (unsigned)INT_MAX); };
  if (t == 0) base_sh = 0;
  for (int i0 = 0; i0 < items; i0 += kPrepThreads) {
    const int i = i0 + t;
    int groups = 0, c0 = i, cnt = 0, most = 0;
    if (sel) {
      if (i < items) {
        if (weigh_vis(A, i) < 0) record_error(A.status, CSA2_ERR_BOUNDS);
        most = A.sel_stride;
        cnt = 1;
      }
    } else {
      int c1 = 0;
      if (i < items && !weigh_queries(A, i, c0, c1)) record_error(A.status, CSA2_ERR_BOUNDS);
      if (i < items) cnt = c1 - c0;
      if (cnt <= 16)
#pragma unroll 4
        for (int q = c0; q < c0 + cnt; q++) {
          const int v = weigh_vis(A, q);
          if (v < 0) record_error(A.status, CSA2_ERR_BOUNDS);
          most = max(most, v);
        }
      // sequences of many queries, one after another, by the whole warp
      uint32_t many = __ballot_sync(0xFFFFFFFFu, cnt > 16);
      while (many != 0u) {
        const int from = __ffs((int)many) - 1;
        many &= many - 1u;
        const int a = __shfl_sync(0xFFFFFFFFu, c0, from), n = __shfl_sync(0xFFFFFFFFu, cnt, from);
        int m = 0;
        bool out = false;
        for (int q = a + lane; q < a + n; q += 32) {
          const int v = weigh_vis(A, q);
          out |= v < 0;
          m = max(m, v);
        }
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (__any_sync(0xFFFFFFFFu, out) && lane == 0) record_error(A.status, CSA2_ERR_BOUNDS);
        if (lane == from) most = m;
      }
    }
    groups = most > 0 ? (cnt + nq - 1) / nq : 0;
    const int own = (int)(((unsigned)most + kWgChunk - 1u) / kWgChunk) * groups;
    int inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc = sum(inc, y);
    }
    if (lane == 31) wt[warp] = inc;
    __syncthreads();
    int ahead = sum(base_sh, inc - own);
    for (int w = 0; w < warp; w++) ahead = sum(ahead, wt[w]);
    if (i < items) {
      W.item[i] = make_int4(most, groups, c0, cnt);
      W.off[i] = ahead;
    }
    __syncthreads();
    if (t == kPrepThreads - 1) base_sh = sum(ahead, own);
    __syncthreads();
  }
  // more products than ranges that do not cross can have: none (nothing else of the items is read then)
  if (t == 0) {
    const bool fits = base_sh < INT_MAX;
    if (!fits) record_error(A.status, CSA2_ERR_BOUNDS);
    W.off[items] = fits ? base_sh : 0;
  }
}

// ------------------------------------------------------------------ a CTA's run
// Its products in order: item by item, block of chunks by block, group by group, chunk by chunk.
__device__ __forceinline__ int wg_chunks(int n) { return (int)(((unsigned)n + kWgChunk - 1u) / kWgChunk); }
template <int NQ>
struct WgWalk {
  int b, end_b, end_c;          // the item; the run's end: chunk end_c of item end_b
  int4 I;
  int lo, hi, seq_hi;           // the block's chunks; the item's end in this run
  int g, c;
  int group;                    // groups of the run that have begun, less one
  __device__ __forceinline__ void block() {
    hi = seq_hi;
    if (I.y > 1) {                                   // (what is left in equal parts: a short one fetches Q for a few chunks)
      const int left = seq_hi - lo, parts = (left + WgSmem<NQ>::kBlock - 1) / WgSmem<NQ>::kBlock;
      hi = lo + (left + parts - 1) / parts;
    }
    g = 0;
    c = lo;
    group++;
  }
  // the next item that has a chunk in the run (false: the run is over)
  __device__ __forceinline__ bool settle(const WgWs &W, int from) {
    lo = from;
    for (;; b++, lo = 0) {
      if (b > end_b || (b == end_b && lo >= end_c)) return false;
      I = __ldg(W.item + b);
      seq_hi = b == end_b ? end_c : wg_chunks(I.x);
      if (I.y > 0 && lo < seq_hi) break;
    }
    block();
    return true;
  }
  __device__ __forceinline__ bool next(const WgWs &W) {
    if (++c < hi) return true;
    if (++g < I.y) {
      c = lo;
      group++;
      return true;
    }
    lo = hi;
    if (lo < seq_hi) {
      block();
      return true;
    }
    b++;
    return settle(W, 0);
  }
  __device__ __forceinline__ bool group_ends() const { return c + 1 == hi; }
  __device__ __forceinline__ bool last_group() const { return g + 1 == I.y; }
};

struct WgShared {
  uint64_t raw_full[4], raw_free[4], k_full[2][4], k_free[4], q_full[4], q_free[4], s_full[4], s_free[4], m_full[kWgMetas], drain;
  uint32_t tmem;
  int begin_b, begin_c, end_b, end_c, steps;
  volatile int bad;
};

// A wait that runs out marks the CTA bad; from then on no role waits, so that all of them run out
// of products in bounded time.
__device__ __forceinline__ void wg_wait_long(int *status, volatile int *bad, uint64_t *bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (int i = 0; !ptx::mbar_try_wait_sleep(bar, parity, 1000000u); i++) {
    if (*bad) return;
    if (i < 64) {
      t0 = ptx::globaltimer();
    } else if (ptx::globaltimer() - t0 > 2000000000ull) {
      record_error(status, CSA2_ERR_TIMEOUT);
      *bad = 1;
      return;
    }
  }
}
__device__ __forceinline__ void wg_wait(const WeighArgs &A, WgShared &S, uint64_t *bar, uint32_t parity) {
  if (!ptx::mbar_try_wait(bar, parity)) wg_wait_long(A.status, &S.bad, bar, parity);
}
__device__ __forceinline__ bool wg_bad(const WgShared &S) { return __any_sync(0xFFFFFFFFu, S.bad); }

// ------------------------------------------------------------------ records and Q
// Two warps take turns at the chunks (one took longer over a chunk than the MMAs).
//
// Where pages hold at least kWgScatter entries a lane has one of the (at most 17) pages that a chunk touches, asks
// for its number a chunk ahead, and copies what the chunk has of it in one piece.
template <int NQ>
__device__ __forceinline__ void wg_fetch_runs(const WeighArgs &A, const WgWs &W, WgShared &S, unsigned char *sm, WgWalk<NQ> C, bool more, int turn) {
  using M = WgSmem<NQ>;
  static_assert((kWgChunk + kWgScatter - 2) / kWgScatter + 1 <= 32, "a lane a page");
  const int lane = threadIdx.x & 31;
  const uint32_t smu = ptx::smem_u32(sm);
  int id = -1, first = 0, rows = 0, off = 0;           // of this lane's page: its first row of the chunk, rows, place of the first
  int j0 = 0, col0 = 0, end = 0;                       // the chunk: its first entry, that one's page, the end of its entries
  bool out = false;
  auto ask = [&]() {
    j0 = C.c * kWgChunk;
    end = min(j0 + kWgChunk, C.I.x);
    col0 = weigh_col(A, j0);
    const int64_t at = (int64_t)(col0 + lane) * A.page;        // the page's first entry
    const int from = (int)(at > j0 ? (at < end ? at : end) : j0), to = (int)(at + A.page < end ? at + A.page : end);
    rows = max(to - from, 0);
    first = from - j0;
    off = (int)(from - at);
    if (rows > 0) id = __ldg(A.table + (int64_t)C.b * A.table_stride + col0 + lane);
  };
  if (more && turn > 0) more = C.next(W);
  if (more) ask();
  int k = turn;
#pragma unroll 1
  for (; more; k += 2) {
    const int stage = k % M::kStages;
    const bool ok = rows > 0 && id >= 0 && id < A.n_pages, last = C.last_group();
    out |= rows > 0 && !ok;
    const int copied = (int)__reduce_add_sync(0xFFFFFFFFu, ok ? (uint32_t)rows : 0u);
    const int page = ok ? id : -1, to = first, n = rows, at = off, j = j0, c0 = col0, j_end = end;
    more = C.next(W);
    if (more) more = C.next(W);
    if (more) ask();
    if (k >= M::kStages) wg_wait(A, S, &S.raw_free[stage], (uint32_t)(k / M::kStages - 1) & 1u);
    if (wg_bad(S)) break;                            // no copy is started any more
    if (last) {
      // (its place was used kSlots products ago.  The buffer was freed by the rows of product k - kStages, which came after the
      // MMAs of k - kStages - 2, which came after the sums of k - kStages - 2 - kSums had read theirs)
      static_assert(M::kSlots >= M::kStages + 2 + M::kSums, "slots");
      const uint32_t slot = smu + M::kSlot + (uint32_t)((k % M::kSlots) * kWgChunk + lane) * 4u;
#pragma unroll
      for (int g = 0; g < 4; g++) {
        const int e = j + 32 * g + lane, c = e < j_end ? weigh_col(A, e) : c0;
        const int has = __shfl_sync(0xFFFFFFFFu, page, c - c0);
        const int rec = e < j_end && has >= 0 ? has * A.page + (e - c * A.page) : -1;
        wg_sts4(slot + 128u * g, (uint32_t)rec);
        if (A.prior != nullptr && rec >= 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(A.prior + rec));
      }
    }
    uint64_t *full = &S.raw_full[stage];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive_expect_tx(full, (uint32_t)(copied * kKvBytes));
    __syncwarp();
    if (page >= 0)
      ptx::bulk_load(sm + M::kRaw + stage * kWgRaw + to * kKvBytes, A.pages + ((int64_t)page * A.page + at) * kKvBytes, (uint32_t)(n * kKvBytes), full);
  }
  if (out) record_error(A.status, CSA2_ERR_BOUNDS);
  // its last copies have landed before the CTA may leave (bounded)
  for (int i = k - 2; i >= 0 && i >= k - M::kStages; i -= 2) ptx::mbar_wait(&S.raw_full[i % M::kStages], (uint32_t)(i / M::kStages) & 1u);
}

// A selection, and pages of a few entries: a lane finds the records of four rows, and two lanes copy a record by 16 B.
template <int NQ, bool SEL>
__device__ __forceinline__ void wg_fetch_rows(const WeighArgs &A, const WgWs &W, WgShared &S, unsigned char *sm, WgWalk<NQ> C, bool more, int turn) {
  using M = WgSmem<NQ>;
  const int lane = threadIdx.x & 31;
  const uint32_t smu = ptx::smem_u32(sm);
  int id[4], off[4];                                 // rows 32 g + lane: the page (-1: none), the place in it
  bool out = false;
  auto ask = [&]() {
    int j[4], seq = C.b;
    if (SEL) {
      seq = __ldg(W.q_seq + C.b);
      const int vis = seq >= 0 ? weigh_vis(A, C.b) : 0;
#pragma unroll
      for (int g = 0; g < 4; g++) {
        const int i = C.c * kWgChunk + 32 * g + lane;
        j[g] = i < A.sel_stride && seq >= 0 ? __ldg(A.sel + (int64_t)C.b * A.sel_stride + i) : -1;
        if (j[g] >= vis) {
          out |= vis > 0;                            // (one that sees nothing has no selection; one out of range is recorded already)
          j[g] = -1;
        }
      }
    } else {
#pragma unroll
      for (int g = 0; g < 4; g++) {
        const int i = C.c * kWgChunk + 32 * g + lane;
        j[g] = i < C.I.x ? i : -1;
      }
    }
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const int col = j[g] >= 0 ? weigh_col(A, j[g]) : 0;
      off[g] = j[g] - col * A.page;
      id[g] = -1;
      if (j[g] >= 0) {
        id[g] = __ldg(A.table + (int64_t)seq * A.table_stride + col);
        if (id[g] < 0) id[g] = INT_MIN;              // (an entry without a page)
      }
    }
  };
  if (more && turn > 0) more = C.next(W);
  if (more) ask();
  int k = turn;
#pragma unroll 1
  for (; more; k += 2) {
    const int stage = k % M::kStages;
    int rec[4];                                      // the record, -1: none
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const bool ok = id[g] >= 0 && id[g] < A.n_pages;
      out |= !ok && id[g] != -1;
      rec[g] = ok ? id[g] * A.page + off[g] : -1;
    }
    const bool last = C.last_group();
    more = C.next(W);
    if (more) more = C.next(W);
    if (more) ask();
    if (k >= M::kStages) wg_wait(A, S, &S.raw_free[stage], (uint32_t)(k / M::kStages - 1) & 1u);
    if (wg_bad(S)) break;                            // no copy is started any more
    if (!SEL && last) {                              // (as in wg_fetch_runs)
      const uint32_t slot = smu + M::kSlot + (uint32_t)((k % M::kSlots) * kWgChunk + lane) * 4u;
#pragma unroll
      for (int g = 0; g < 4; g++) wg_sts4(slot + 128u * g, (uint32_t)rec[g]);
    }
    uint64_t *full = &S.raw_full[stage];
    unsigned char *to = sm + M::kRaw + stage * kWgRaw;
#pragma unroll
    for (int g = 0; g < 8; g++) {                    // 16 records at a time
      const int from = (g & 1) * 16 + (lane >> 1);
      const int r = __shfl_sync(0xFFFFFFFFu, rec[g >> 1], from);
      const uint8_t *src = A.pages + (int64_t)r * kKvBytes + (lane & 1) * 16;
      unsigned char *dst = to + ((g >> 1) * 32 + from) * kKvBytes + (lane & 1) * 16;
      if (r >= 0)
#pragma unroll
        for (int i = 0; i < kKvBytes; i += 32) ptx::cp_async16(dst + i, src + i);
    }
    ptx::cp_async_arrive(full);                      // (each lane's copies, pending from here on)
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(full);
    __syncwarp();
  }
  if (out) record_error(A.status, CSA2_ERR_BOUNDS);
  // its last copies have landed before the CTA may leave (bounded)
  for (int i = k - 2; i >= 0 && i >= k - M::kStages; i -= 2) ptx::mbar_wait(&S.raw_full[i % M::kStages], (uint32_t)(i / M::kStages) & 1u);
}

// Q of a group slab by slab, as the group before lets go of it, and beside the first of them f and lse
// (their place was used eight groups ago: the sums have left it once the group before is at its last product).
template <int NQ>
__device__ __forceinline__ void wg_fetch_q(const WeighArgs &A, const WgWs &W, WgShared &S, unsigned char *sm, WgWalk<NQ> C, bool more) {
  using M = WgSmem<NQ>;
  int slabs = 0;
#pragma unroll 1
  for (int group = 0; more; group++) {
    const int q0 = C.I.z + C.g * NQ, n = min(NQ, C.I.w - C.g * NQ), place = group % kWgMetas;
#pragma unroll 1
    for (int s = 0; s < 4; s++) {
      if (group > 0) wg_wait(A, S, &S.q_free[s], (uint32_t)(group - 1) & 1u);
      if (S.bad) break;
      if (s == 0) {
        ptx::mbar_arrive_expect_tx(&S.m_full[place], (uint32_t)(n * kWgMeta));
        ptx::bulk_load(sm + M::kMeta + place * NQ * kWgMeta, W.meta + (int64_t)q0 * kWgMeta, (uint32_t)(n * kWgMeta), &S.m_full[place]);
      }
      ptx::mbar_arrive_expect_tx(&S.q_full[s], (uint32_t)(n * 2 * kWgQBlock));
      for (int i = 0; i < 2; i++)
        for (int x = 0; x < n; x++)
          ptx::bulk_load(sm + M::kQ + ((2 * s + i) * NQ + x) * kWgQBlock, W.image + (int64_t)(q0 + x) * kWgImage + (2 * s + i) * kWgQBlock, kWgQBlock, &S.q_full[s]);
      slabs++;
    }
    C.c = C.hi - 1;
    more = C.next(W) && !S.bad;
  }
  // its last copies have landed before the CTA may leave (bounded)
  for (int i = max(0, slabs - 4); i < slabs; i++) ptx::mbar_wait(&S.q_full[i & 3], (uint32_t)(i >> 2) & 1u);
  const int metas = (slabs + 3) / 4;
  for (int i = max(0, metas - kWgMetas); i < metas; i++) ptx::mbar_wait(&S.m_full[i % kWgMetas], (uint32_t)(i / kWgMetas) & 1u);
}

// ------------------------------------------------------------------ dequantisation
// Sixteen warps in four teams, a team a slab of 128 dims of every chunk, a row per thread.
template <int NQ>
__device__ __forceinline__ void wg_load(const WeighArgs &A, WgShared &S, const unsigned char *sm, int steps, uint32_t tmem) {
  using M = WgSmem<NQ>;
  const int lt = (int)threadIdx.x - kWgSumWarps * 32, lane = lt & 31;
  const int e = lt & 127, team = lt >> 7;            // row
  const uint32_t kcol = tmem + ((uint32_t)(e & 96) << 16) + kWgColK + (uint32_t)team * 64u;
  // Records are 18 16-B units apart, so rows r and r + 4 of a unit share their banks: every
  // other four rows read the units of a pair the other way round.
  const bool flip = (e & 4) != 0;
  const uint32_t rows = ptx::smem_u32(sm) + M::kRaw + (uint32_t)(e * kKvBytes), own = (uint32_t)(team * 64) + (flip ? 16u : 0u), other = flip ? 0u - 16u : 16u;
  int stage = 0;
  uint32_t turn = 0u;
#pragma unroll 1
  for (int k = 0; k < steps; k++) {
    wg_wait(A, S, &S.raw_full[stage], turn);
    const uint32_t row = rows + (uint32_t)(stage * kWgRaw), raw = row + own;
    const uint2 sc = wg_lds8(row + 256u + (uint32_t)team * 8u);
    uint4 code[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const uint4 x = wg_lds16(raw + j * 16u), y = wg_lds16(raw + j * 16u + other);
      code[j] = flip ? y : x;
      code[j + 1] = flip ? x : y;
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.raw_free[stage]);
    if (++stage == M::kStages) {
      stage = 0;
      turn ^= 1u;
    }
    // half of the slab is converted before the wait for its place, beside the MMAs of the chunk before
#pragma unroll
    for (int hf = 0; hf < 2; hf++) {
      uint32_t o[2][16];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int j = 2 * hf + i;
        const uint32_t w[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
        const uint32_t two = e4m3x2_to_f16x2((hf == 0 ? sc.x : sc.y) >> (16 * i));
        const __half2 sh = *reinterpret_cast<const __half2 *>(&two), s2[2] = {__low2half2(sh), __high2half2(sh)};
#pragma unroll
        for (int u = 0; u < 4; u++) {
          uint32_t x[4];
          e2m1x8_to_f16(w[u], x);
#pragma unroll
          for (int q = 0; q < 4; q++) {
            const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x[q]), s2[u >> 1]);
            o[i][4 * u + q] = *reinterpret_cast<const uint32_t *>(&y);
          }
        }
      }
      if (hf == 0) {
        if (k > 0) wg_wait(A, S, &S.k_free[team], (uint32_t)(k - 1) & 1u);
        ptx::tc_fence_after();
      }
#pragma unroll
      for (int i = 0; i < 2; i++) ptx::tmem_st_32x32b_x16(kcol + (2 * hf + i) * 16, o[i]);
    }
    ptx::tmem_wait_st();
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.k_full[k & 1][team]);
  }
}

// ------------------------------------------------------------------ MMAs
// Two threads take turns at the chunks (one took longer to issue a chunk's than they take to run).  A slab of K is
// written again only when the MMAs that read it are complete, so a chunk's MMAs on a slab follow the chunk's before.
// (A wait by parity holds only for who has seen the phase before, or knows of it: each thread has K's barriers of its own,
// and once a slab of K is there the group before has had its Q.)
template <int NQ>
__device__ __forceinline__ void wg_issue(const WeighArgs &A, const WgWs &W, WgShared &S, unsigned char *sm, WgWalk<NQ> C, bool more, int turn, uint32_t tmem) {
  const uint64_t d_q = ptx::smem_desc(ptx::smem_u32(sm + WgSmem<NQ>::kQ), 16, 1024, 2);
  using M = WgSmem<NQ>;
  int seen = -1;                                     // the group whose Q this thread has waited for
  if (more && turn > 0) more = C.next(W);
#pragma unroll 1
  for (int k = turn; more && !S.bad; k += 2) {
    const bool fresh = C.group != seen, ends = C.group_ends();
    const uint32_t q_parity = (uint32_t)C.group & 1u;
    seen = C.group;
    const uint32_t id = NQ == 2 && C.I.w - C.g * NQ >= 2 ? idesc_m128(0, true, 2 * kHeads) : idesc_m128(0, true, kHeads);
    const int place = k % M::kSums;
    const uint32_t d = tmem + kWgColS + (uint32_t)place * (64u * NQ);
    if (k >= M::kSums) wg_wait(A, S, &S.s_free[place], (uint32_t)(k / M::kSums - 1) & 1u);
#pragma unroll 1
    for (int s = 0; s < 4; s++) {
      wg_wait(A, S, &S.k_full[turn][s], (uint32_t)(k >> 1) & 1u);
      if (fresh) wg_wait(A, S, &S.q_full[s], q_parity);
      ptx::tc_fence_after();
      const uint32_t ka = tmem + kWgColK + (uint32_t)s * 64u;
      const uint64_t qa = d_q + (uint64_t)(s * 2 * NQ * (kWgQBlock >> 4));
#pragma unroll
      for (int kk = 0; kk < 8; kk++)
        ptx::tc_mma_f16_ts(d, ka + kk * 8, qa + (kk >> 2) * (NQ * (kWgQBlock >> 4)) + (kk & 3) * 2, id, kk > 0 ? 1u : (uint32_t)(s > 0));
      ptx::tc_commit(&S.k_free[s]);
      if (ends) ptx::tc_commit(&S.q_free[s]);
    }
    ptx::tc_commit(&S.s_full[place]);
    more = C.next(W);
    if (more) more = C.next(W);
  }
  ptx::tc_commit(&S.drain);
}

// ------------------------------------------------------------------ sums
__device__ __forceinline__ uint64_t wg_pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t wg_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t wg_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2 wg_unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float wg_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Adds 32 heads' numerators of this lane's entry to sum.
__device__ __forceinline__ void wg_add_heads(const uint32_t (&a)[32], uint32_t f, uint64_t (&sum)[4]) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const ulonglong2 x = wg_lds2x64(f + 4u * i), y = wg_lds2x64(f + 4u * (kHeads + i));
    const float2 u = wg_unpair(wg_fma2(wg_pair(__uint_as_float(a[i]), __uint_as_float(a[i + 1])), x.x, y.x));
    const float2 v = wg_unpair(wg_fma2(wg_pair(__uint_as_float(a[i + 2]), __uint_as_float(a[i + 3])), x.y, y.y));
    sum[(i >> 1) & 2] = wg_add2(sum[(i >> 1) & 2], wg_pair(wg_ex2(u.x), wg_ex2(u.y)));
    sum[((i >> 1) & 2) + 1] = wg_add2(sum[((i >> 1) & 2) + 1], wg_pair(wg_ex2(v.x), wg_ex2(v.y)));
  }
}
__device__ __forceinline__ float wg_total(const uint64_t (&sum)[4]) {
  const float2 all = wg_unpair(wg_add2(wg_add2(sum[0], sum[1]), wg_add2(sum[2], sum[3])));
  return all.x + all.y;
}

// Each warp has 32 of a chunk's entries and 64 heads: a query at a time, warps 0 .. 3 and 4 .. 7 take turns at the
// chunks; of two queries the former have the first and the latter the second, whose sums go to the former
// through shared memory.  Tensor memory is read 32 heads ahead of the arithmetic.
template <int NQ, bool SEL>
__device__ __forceinline__ void wg_sum(const WeighArgs &A, const WgWs &W, WgShared &S, unsigned char *sm, WgWalk<NQ> C, bool more, uint32_t tmem) {
  using M = WgSmem<NQ>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, side = warp >> 2, row = quarter * 32 + lane;
  const uint32_t ts = tmem + ((uint32_t)(quarter * 32) << 16) + kWgColS + (NQ == 2 ? (uint32_t)side * 64u : 0u);
  const uint32_t smu = ptx::smem_u32(sm), acc = smu + M::kAcc + row * 4u, part = smu + M::kPart + row * 4u;
  int seen = -1, vis = 0;
  bool two = false;
#pragma unroll 1
  for (int k = 0; more; k++, more = C.next(W)) {
    if (C.group != seen) {
      seen = C.group;
      // (a chunk's sums of the group before may be the other four warps', or not be read yet)
      if (!SEL) asm volatile("bar.sync %0, 64;" ::"r"(quarter + 1) : "memory");
      two = NQ == 2 && C.I.w - C.g * NQ >= 2;
      if (!SEL) vis = weigh_vis(A, C.I.z + C.g * NQ + (two ? side : 0));
    }
    if (NQ == 1 && (k & 1) != side) continue;
    const bool last = C.last_group(), works = NQ == 1 || side == 0 || two;
    const int place = k % M::kSums;
    wg_wait(A, S, &S.s_full[place], (uint32_t)(k / M::kSums) & 1u);
    // (f and lse: as the group's products, or later; those of the groups before are there)
    wg_wait(A, S, &S.m_full[seen % kWgMetas], (uint32_t)(seen / kWgMetas) & 1u);
    ptx::tc_fence_after();
    int slot = -1;
    float before = 0.f, w = 0.f;
    if (!SEL && last && (NQ == 1 || side == 0)) {    // where the entry's weight is, asked for ahead of the sum
      slot = (int)wg_lds4(smu + M::kSlot + (uint32_t)((k % M::kSlots) * kWgChunk + row) * 4u);
      if (S.bad) slot = -1;                          // (a place left from before, once a wait has run out)
      if (slot >= 0 && A.prior != nullptr) before = A.prior[slot];
    }
    const int j = C.c * kWgChunk + row;
    const uint32_t f = smu + M::kMeta + (uint32_t)((seen % kWgMetas) * NQ * kWgMeta + (NQ == 2 ? side * kWgMeta : 0));
    uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
    uint32_t a1[32];
    if (works) {
      uint32_t a0[32];
      ptx::tmem_ld_32x32b_x32(ts + place * (64 * NQ), a0);
      ptx::tmem_wait_ld();
      ptx::tmem_ld_32x32b_x32(ts + place * (64 * NQ) + 32, a1);
      wg_add_heads(a0, f, sum);
      ptx::tmem_wait_ld();
    }
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.s_free[place]);
    if (works) {
      wg_add_heads(a1, f + 128u, sum);
      if (SEL || j < vis) w = wg_total(sum);
    }
    if (NQ == 2 && two) {
      const uint32_t at = part + (uint32_t)(k & 1) * (kWgChunk * 4u);
      if (side == 1) wg_sts4(at, __float_as_uint(w));
      asm volatile("bar.sync %0, 64;" ::"r"(quarter + 1) : "memory");
      if (side == 0) w += wg_ldsf(at);
    }
    if (NQ == 2 && side == 1) continue;
    const uint32_t mine = acc + (uint32_t)(C.c - C.lo) * (kWgChunk * 4u);        // (of several groups)
    if (C.g > 0) w += wg_ldsf(mine);
    if (!last) {
      wg_sts4(mine, __float_as_uint(w));
    } else if (SEL) {
      if (j < A.sel_stride) W.part[(int64_t)C.b * A.sel_stride + j] = w;
    } else if (slot >= 0) {
      A.weight[slot] = A.decay * before + w;
    }
  }
}

// The last b with off[b] <= x, by the whole warp (off ascending, off[0] = 0; x < off[items]).
__device__ __forceinline__ int wg_find(const int32_t *off, int items, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = items;                             // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool ok = at < lo + n && __ldg(off + at) <= x;
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, ok);       // lanes 0 .. some lane
    const int last = 31 - __clz((int)hit);
    const int end = lo + n;
    lo += last * step;
    n = min(step, end - lo);
  }
  return lo;
}

template <int NQ, bool SEL>
__global__ void __launch_bounds__(kWgThreads, 1) weigh_kernel(const __grid_constant__ WeighArgs A, WgWs W) {
  using M = WgSmem<NQ>;
  extern __shared__ __align__(1024) unsigned char wg_smem_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(wg_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(16) WgShared S;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (t == 0) {
    for (int i = 0; i < 4; i++) {
      ptx::mbar_init(&S.raw_full[i], 1);
      ptx::mbar_init(&S.raw_free[i], kWgKWarps);
      ptx::mbar_init(&S.k_full[0][i], kWgKWarps / 4);
      ptx::mbar_init(&S.k_full[1][i], kWgKWarps / 4);
      ptx::mbar_init(&S.k_free[i], 1);
      ptx::mbar_init(&S.q_full[i], 1);
      ptx::mbar_init(&S.q_free[i], 1);
    }
    for (int i = 0; i < 4; i++) {
      ptx::mbar_init(&S.s_full[i], 1);
      ptx::mbar_init(&S.s_free[i], NQ == 1 ? kWgSumWarps / 2 : kWgSumWarps);
    }
    for (int i = 0; i < kWgMetas; i++) ptx::mbar_init(&S.m_full[i], 1);
    ptx::mbar_init(&S.drain, 2);
    S.bad = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0) ptx::tmem_alloc(&S.tmem, kWgTmemCols);
  griddep_wait();
  griddep_launch();
  // ---------------------------------------------------------- this CTA's run
  const int items = SEL ? A.n_q : A.n_seq;
  if (warp == 1 || warp == 2) {
    const int T = __ldg(W.off + items), G = min((int)gridDim.x, max(T, 1));
    const int i = min((int)blockIdx.x + warp - 1, G);
    const int x = (int)((int64_t)T * i / G);
    int b = items, c = 0;
    if (x < T) {
      b = wg_find(W.off, items, x);
      // (items without products share their place with the one behind them: the last of them has it)
      c = (x - __ldg(W.off + b)) / __ldg(&W.item[b].y);
    }
    if (lane == 0) {
      if (warp == 1) {
        S.begin_b = b;
        S.begin_c = c;
      } else {
        S.end_b = b;
        S.end_c = c;
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = S.tmem;
  WgWalk<NQ> C;
  C.b = S.begin_b;
  C.end_b = min(S.end_b, items - 1);
  C.end_c = S.end_c;
  if (S.end_b >= items) C.end_c = wg_chunks(__ldg(&W.item[items - 1].x));
  C.group = -1;
  const bool more = C.b < items && C.settle(W, S.begin_c);
  if (warp >= kWgSumWarps && warp < kWgSumWarps + kWgKWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWgRegsK));
    // products of the run (the team needs no more of it)
    int steps = 0;
    WgWalk<NQ> D = C;
    for (bool m = more; m; m = D.settle(W, 0)) {
      steps += (D.seq_hi - D.lo) * D.I.y;
      D.b++;
    }
    wg_load<NQ>(A, S, sm, steps, tmem);
  } else if (warp < kWgSumWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWgRegsSum));
    wg_sum<NQ, SEL>(A, W, S, sm, C, more, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWgRegsRest));
    const int role = warp - kWgSumWarps - kWgKWarps;
    if (role < 2) {
      if (SEL || A.page < kWgScatter) wg_fetch_rows<NQ, SEL>(A, W, S, sm, C, more, role);
      else wg_fetch_runs<NQ>(A, W, S, sm, C, more, role);
    } else if (role < 4) {
      if (ptx::elect_one()) wg_issue<NQ>(A, W, S, sm, C, more, role - 2, tmem);
    } else if (role == 4) {
      if (ptx::elect_one()) wg_fetch_q<NQ>(A, W, S, sm, C, more);
    }
  }
  __syncwarp();
  __syncthreads();
  if (S.bad) {
    // a wait ran out: every MMA issued here finishes before the tensor memory goes back (bounded)
    ptx::mbar_wait(&S.drain, 0);
    ptx::tc_fence_after();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kWgTmemCols);
  }
}

// ------------------------------------------------------------------ selections
// Adds the selections' weights, a CTA per sequence, query by query: entries that several queries
// selected get their parts in the queries' order, so the sums are the same on every call.  (Within
// a query an entry named twice gets the same part twice: their order does not matter.)
// Slots and parts of kAddAhead queries are read at a time.  (Ranges that cross: a query's part is that of one of its sequences.)
constexpr int kAddAhead = 8;
__global__ void __launch_bounds__(kTopK) weigh_add_kernel(const __grid_constant__ WeighArgs A, const float *part, const int32_t *q_seq) {
  const int t = threadIdx.x, b = blockIdx.x;
  griddep_wait();
  griddep_launch();
  int c0, c1;
  if (!weigh_queries(A, b, c0, c1) && t == 0) record_error(A.status, CSA2_ERR_BOUNDS);
  for (int q0 = c0; q0 < c1; q0 += kAddAhead) {
    int j[kAddAhead];
    int64_t s[kAddAhead];
    float w[kAddAhead];
#pragma unroll
    for (int i = 0; i < kAddAhead; i++) j[i] = q0 + i < c1 && t < A.sel_stride ? __ldg(A.sel + (int64_t)(q0 + i) * A.sel_stride + t) : -1;
#pragma unroll
    for (int i = 0; i < kAddAhead; i++) {
      const bool in = j[i] >= 0 && j[i] < weigh_vis(A, q0 + i) && __ldg(q_seq + q0 + i) == b;
      s[i] = in ? weigh_slot(A, b, j[i]) : -1;
      w[i] = in ? __ldg(part + (int64_t)(q0 + i) * A.sel_stride + t) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAddAhead; i++) {
      if (q0 + i >= c1) break;
      if (s[i] >= 0) atomicAdd(A.weight + s[i], w[i]);
      __syncthreads();
    }
  }
}

static void weigh_magic(unsigned n, uint64_t &mul, int &shift) {      // j / n, exact for j below 2^31
  int s = 0;
  while (((int64_t)1 << s) < (int64_t)n) s++;
  shift = 31 + s;
  mul = (uint64_t)((((unsigned __int128)1 << shift) + n - 1) / n);
}

template <int NQ, bool SEL>
static cudaError_t launch_products(const WeighArgs &A, const WgWs &W, int decay_parts, int dev, cudaStream_t st) {
  static std::atomic<int> attr_done[kMaxDevices];
  cudaError_t e = once_per_device(attr_done, dev, [&] {
    return cudaFuncSetAttribute(weigh_kernel<NQ, SEL>, cudaFuncAttributeMaxDynamicSharedMemorySize, WgSmem<NQ>::kAlloc);
  });
  if (e != cudaSuccess) return e;
  const unsigned ctas = 1u + (unsigned)A.n_q * kPrepCtas + (unsigned)A.n_seq * (unsigned)decay_parts;
  e = launch_pdl(weigh_prep_kernel, dim3(ctas), dim3(kPrepThreads), 0, st, 1u, A, W, NQ, decay_parts);
  if (e != cudaSuccess) return e;
  // no more CTAs than there can be chunks
  const int64_t sms = device_sm_count(dev), row = SEL ? A.sel_stride : A.table_stride * A.page;
  const int64_t chunks = (SEL ? A.n_q : A.n_seq) * ((row + kWgChunk - 1) / kWgChunk);
  return launch_pdl(weigh_kernel<NQ, SEL>, dim3((unsigned)(chunks < sms ? chunks : sms)), dim3(kWgThreads), (size_t)WgSmem<NQ>::kAlloc, st, 1u, A, W);
}

cudaError_t launch_weigh(WeighArgs A, void *ws, cudaStream_t st) {
  const int dev = current_device();
  weigh_magic((unsigned)A.page, A.page_mul, A.page_shift);
  WgWs W;
  wg_layout(&W, ws, A.n_q, A.n_seq, A.sel_stride);
  // Two queries at a time where there are more queries than sequences, so that some sequence has two for sure (how many each has
  // is on the device).  Else one at a time: right for any, slower where few sequences have all of the queries.
  if (A.sel == nullptr)
    return A.n_q > A.n_seq ? launch_products<2, false>(A, W, 0, dev, st) : launch_products<1, false>(A, W, 0, dev, st);
  // a CTA for each 1,024 places of a row, up to 512
  const int64_t tiles = (A.table_stride * A.page + 4 * kPrepThreads - 1) / (4 * kPrepThreads);
  const int decay_parts = A.prior == A.weight && A.decay == 1.f ? 0 : (int)(tiles < 512 ? tiles : 512);
  const cudaError_t e = launch_products<1, true>(A, W, decay_parts, dev, st);
  if (e != cudaSuccess) return e;
  return launch_pdl(weigh_add_kernel, dim3((unsigned)A.n_seq), dim3(kTopK), 0, st, 1u, A, (const float *)W.part, (const int32_t *)W.q_seq);
}

}  // namespace csa2
