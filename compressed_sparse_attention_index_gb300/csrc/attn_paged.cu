// Attention over paged latents on the 5th-generation tensor cores
// (csa2_paged_attn): 64 query heads over one 512-wide latent per entry (k = v),
// every visible entry of a sequence or a selection of them, and the window.
//
//     l_i = scale q_h . k_i,   o_h = sum_i exp(l_i) k_i / sum_i exp(l_i)
//
// with the RoPE dims of o_h rotated by -pos, and lse_h = log sum_i exp(l_i)
// ("An infra-oriented diagram of the DeepSeek-V4.1-Flash architecture", reading
// notes on the k = v latent, the window and the un-rotated output).
//
// Work: the entries of a query form chunks of 128, its window one more chunk
// ahead of them.  The chunks of all queries, in query order, are dealt to the
// CTAs (one per SM) in contiguous, equal runs, whatever the queries' lengths;
// a query cut by a run's border leaves unnormalised partials with their maximum
// and denominator, which paged_join_kernel combines.  A CTA has at most two cut
// queries, so the partials take a fixed workspace.
//
// Per chunk: the 128 records are dequantised to f16 (an E2M1 x E4M3 product has <= 6
// significant bits in [2^-10, 2688]: exact), then
//   S^T[entry][head] = K . Q^T        tcgen05 kind::f16, M = 128, N = 64, K = 512
//   P[entry][head] = 2^(S - m + 7)    rounded to f16 (11 bits)
//   O^T[dim][head] += K^T . P         M = 128 dims (4 blocks), N = 64, K = 128
// m is a head's reference in log2 units: the maximum of the first chunk, raised only
// when a later logit exceeds it by more than 8, so numerators stay within 2^15 and most
// chunks need no maximum, no exchange between warps and no rescaling of O.  The factor
// 2^7 keeps the tail of a long row (2^-21 of the largest weight) in f16's normal range.
// The denominator sums the unrounded fp32 numerators.
//
// Window records (E4M3 x 2^e) are exact in f16 where -15 <= e <= 7; otherwise
// the window is scaled by 2^kx, kx = 7 - (the largest e): exact but for values
// below 2^-31 of the window's largest, and undone on its logits and, being the
// first chunk, on O before the next one.  A head of Q out of f16's range goes to f16
// under a power of two of its own, undone on its logits.
//
// Warps, with their own barriers between them: two fetch records into shared memory;
// eight (K) dequantise them, a row per thread, into slabs of 128 dims in tensor memory,
// where QK reads them as its A operand; eight (V) copy the slabs from there into shared
// memory, where PV reads them MN-major; eight (softmax) turn S into P and read O out; one
// thread each issues QK and PV.
//
// What bounds it: the heads fill half of an MMA's width, so the tensor cores' 2,600
// cycles a chunk are far from the peak rate by themselves, and shared memory moves more:
// V's slabs 1,024 cycles to write and as much for PV to read, Q 512, P 128 to write and
// 512 to read, the records 288 in and 320 out, and (counted) 1,330 of barriers, waits,
// descriptions, the softmax's exchanges, global accesses and conflicts: 5,140 of the 5,100
// to 5,400 cycles that a chunk takes.  That is why K goes through tensor memory (both
// operands in shared memory took 512 cycles more), and why its rows are dequantised once (a
// second time for V cost more arithmetic than everything else together).  8 x 1,048,576
// entries: 1,220 us, 0.90 PFLOP/s; 32 x 65,536: 334 us; 33 sequences of up to 40,001: 147 us;
// 40 queries x 512 selected: 35 us.
// A few short rows are a chain of latencies: 18 us for one chunk each, the join included.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "attn.cuh"
#include "common.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace csa2 {

constexpr int kPgChunk = 128;
constexpr int kPgSoft = 256, kPgLoad = 256;        // threads of the softmax group and of each loading group
constexpr int kPgThreads = kPgSoft + 2 * kPgLoad + 128;
// Registers: 896 threads are launched with 72 each; the softmax and V groups take what
// the K group and the other warps give up.
constexpr int kPgRegsSoft = 88, kPgRegsK = 56, kPgRegsV = 80, kPgRegsRest = 56;
static_assert(kPgSoft * kPgRegsSoft + kPgLoad * (kPgRegsK + kPgRegsV) + 128 * kPgRegsRest <= 72 * kPgThreads, "register split");
constexpr int kPgSlab = 128 * 128 * 2;             // one slab: 128 entries x 128 dims f16
constexpr int kPgRaw = kPgChunk * kKvBytes;        // one chunk's records
constexpr unsigned kPgKRing = 3, kPgVRing = 3;     // slabs of K in tensor memory, of V in shared memory
constexpr int kPgSmV = 0;                          // slabs: [e/8][dim/64][e%8][128 B]
constexpr int kPgSmQ = kPgSmV + (int)kPgVRing * kPgSlab;       // 64 heads x 512 dims f16: [h/8][dim/64][h%8][128 B]
constexpr int kPgSmP = kPgSmQ + 64 * 1024;         // 128 entries x 64 heads f16: [e/8][e%8][128 B]
constexpr int kPgSmRaw = kPgSmP + 16 * 1024;       // a chunk's records
constexpr int kPgSmEnd = kPgSmRaw + kPgRaw;
constexpr int kPgSmAlloc = kPgSmEnd + 1024;
static_assert(kPgSmAlloc + 5120 <= 227 * 1024, "shared memory");
// tensor memory: S^T, O^T, the ring of K
constexpr uint32_t kPgColS = 0, kPgColO = 64, kPgColK = 320, kPgTmemCols = 512;
constexpr float kPgRaise = 8.f, kPgShift = 7.f, kPgNoRef = 3e38f;   // (kPgNoRef: no entry met yet)
constexpr int kPgScatter = 8;                      // pages of fewer entries are fetched as scattered records
constexpr int kPgSnap = 2, kPgSnapRun = 2, kPgSnapFew = 5;
constexpr int kPgInfo = 8;                         // chunks described in shared memory at a time

// Votes of the softmax group, at places that each of its warps reaches once a chunk.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool soft_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p)
      : "memory");
  return r != 0u;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// j / n by a multiplication: exact for j below 2^31 (mul = ceil(2^(31 + s) / n) with
// 2^s >= n is at most 2^32 and off by less than one in 2^s)
__device__ __forceinline__ unsigned magic_div(unsigned j, uint64_t mul, int shift) { return (unsigned)(((uint64_t)j * mul) >> shift); }
static void magic_of(unsigned n, uint64_t &mul, int &shift) {
  int s = 0;
  while (((int64_t)1 << s) < (int64_t)n) s++;
  shift = 31 + s;
  mul = (uint64_t)((((unsigned __int128)1 << shift) + n - 1) / n);
}

struct PagedQuery {
  int seq, n, chunks, win, first;      // entries (or selection slots), chunks in all, the window's
  bool bad;
};

__device__ __forceinline__ PagedQuery paged_query(const PagedArgs &A, int q) {
  PagedQuery r;
  r.seq = __ldg(A.q_seq + q);
  const int vis = __ldg(A.n_vis + q);
  r.win = __ldg(A.swa_cnt + q);
  r.first = __ldg(A.swa_first + q);
  r.bad = r.seq < 0 || r.seq >= A.n_seq || vis < 0 || (int64_t)vis > A.table_stride * A.page || r.win < 0 ||
          r.win > kSwa || r.win > A.swa_cap || (r.win > 0 && (r.first < 0 || r.first >= A.swa_cap));
  r.n = r.bad ? 0 : A.sel != nullptr ? (vis > 0 ? A.sel_stride : 0) : vis;
  if (r.bad) r.win = 0;
  r.chunks = (int)(((unsigned)r.n + kPgChunk - 1) / kPgChunk) + (r.win > 0 ? 1 : 0);
  return r;
}

// The CTAs that share T chunks (a launch may have more)
__device__ __forceinline__ int run_ctas(int T, int grid) { return min(grid, max(1, T)); }
// Chunks are dealt to G CTAs in runs of T / G (T below 2^31), but a border that falls
// within `snap` chunks of an end of a query is moved there: a piece of a query costs a
// CTA its Q, a window or a read-out and a partial of 128 KB for the join, about as much
// as two chunks.  Up to half a run, and no more than two chunks (256 x 512 entries: 79 us,
// 98 with none; 100 x 2,000: 83, three 89); one at least where a query's chunks are a
// few runs only (40 x 512 selected, four runs a query: 33 us, none 36; but 24 x 1,000, six runs
// a query: 31 instead of 28, and 8 x 4,096: 32 instead of 28).
__device__ __forceinline__ int run_snap(int T, int G, int n_q) {
  return T <= G ? 0 : min(kPgSnap, max(T / (kPgSnapRun * G), kPgSnapFew * n_q > G ? 1 : 0));
}
// The first border that stays inside a query of n chunks from off, and the last one.
__device__ __forceinline__ int run_first_cut(int off, int T, int G, int n_q) {
  return (int)((((int64_t)off + run_snap(T, G, n_q) + 1) * G + T - 1) / T);
}
__device__ __forceinline__ int run_last_cut(int off, int n, int T, int G, int n_q) {
  return (int)((((int64_t)off + n - run_snap(T, G, n_q)) * G + T - 1) / T) - 1;
}

// A position in a CTA's run of chunks.
struct PagedCursor {
  int c, end, off;              // the chunk, the run's end, the query's first chunk
  int qi;
  PagedQuery Q;
  // moves to the query that holds chunk c (false: the run is over)
  __device__ __forceinline__ bool settle(const PagedArgs &A) {
    while (c < end) {
      if (c < off + Q.chunks) return true;
      off += Q.chunks;
      Q = paged_query(A, ++qi);
    }
    return false;
  }
  __device__ __forceinline__ int local() const { return c - off; }
  __device__ __forceinline__ bool window() const { return Q.win > 0 && c == off; }
};

// j / page
__device__ __forceinline__ unsigned paged_col(unsigned j, const PagedArgs &A) { return magic_div(j, A.page_mul, A.page_shift); }

// What the roles need to know of a chunk (kPgInfo of them, by chunk number).
struct PagedInfo {
  int4 at;                      // query, place in it, its chunks, its first chunk
  uint32_t valid[4];            // rows that hold an entry
  int seq, win, first;          // sequence; window entries (0: entries of the cache), the oldest one's place
  float f;                      // of a query's first chunk here: logits in log2 units per unit of S, negative where
  int units;                    // its heads have units, which stand there
  int kx;                       // a window's scale (its tile holds 2^kx times its values)
};

struct PagedShared {
  // of slab n: number n % 6 (each team passes every phase of what it waits on)
  uint64_t k_full[6], k_free[6], v_full[6], v_free[6];
  uint64_t raw_full[2], raw_free[2];   // one buffer; by the parity of the chunk, so that each fetching warp
                                       // passes every phase of what it waits on
  uint64_t q_full, q_done, s_full, s_free, p_full, o_done, drain;
  uint64_t meet[3];             // of the softmax, K and V groups' warps
  PagedInfo info[kPgInfo];
  __align__(16) float less[kHeads];    // minus a head's reference, which is kPgShift below a maximum
  float alpha[kHeads];
  float l[4][kHeads], red[4][kHeads];
  float unit[2][kHeads];               // minus the heads' powers of two, for queries that have others than 1, by turns
  uint32_t tmem, hmax[8][16], v_met[8];   // a V warp's largest |q| of its heads; its parities (see stage_q)
  int emin, emax, units;               // (units: of the softmax's query)
  int scan[kPgThreads / 32], end[2], start, off, T, G;      // the run's ends; its first query, that one's first chunk; all chunks, their CTAs
  PagedQuery Q;
  volatile int bad;
};

// A wait that runs out marks the CTA bad; from then on no role waits, so that all
// of them run out of chunks (and meet their groups' barriers) in bounded time.
__device__ __forceinline__ void paged_wait(const PagedArgs &A, PagedShared &S, uint64_t *bar, uint32_t parity) {
  // (asleep in hardware until the phase ends; the timer is read only after many tries)
  uint64_t t0 = 0;
  for (int i = 0; !ptx::mbar_try_wait_sleep(bar, parity, 1000000u); i++) {
    if (S.bad) return;
    if (i < 64) {
      t0 = ptx::globaltimer();
    } else if (ptx::globaltimer() - t0 > 2000000000ull) {
      record_error(A.status, CSA2_ERR_TIMEOUT);
      S.bad = 1;
      return;
    }
  }
}

// The warps of a group meet, where a chunk's description says so.  (Not a barrier of the
// hardware's: once a wait has run out the warps may read different descriptions.)
__device__ __forceinline__ void paged_meet(const PagedArgs &A, PagedShared &S, int group, uint32_t &met) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&S.meet[group]);
  paged_wait(A, S, &S.meet[group], met & 1);
  met ^= 1;
}
__device__ __forceinline__ bool paged_bad(const PagedShared &S) { return __any_sync(0xFFFFFFFFu, S.bad); }

// Where slab n of the run stands, for a role that takes slabs n, n + STEP, ..: its
// slot in a ring of three and its barriers' number and phase.  Two teams take turns
// at the slabs, so a slot passes from one to the other; the six barriers do not, and
// a wait for the slab three before (the slot's last) is on a barrier of the other
// parity, every phase of which that team waits for in turn.
template <unsigned STEP>
struct PagedSlab {
  unsigned bar, phase, slot;
  bool reuse;                   // the slot was used before (by slab n - 3)
  __device__ __forceinline__ explicit PagedSlab(unsigned n) : bar(n), phase(0), slot(n), reuse(false) {}
  __device__ __forceinline__ unsigned last_bar() const { return bar >= 3 ? bar - 3 : bar + 3; }
  __device__ __forceinline__ unsigned last_phase() const { return bar >= 3 ? phase : phase ^ 1; }
  __device__ __forceinline__ void next() {
    bar += STEP;
    if (bar >= 6) {
      bar -= 6;
      phase ^= 1;
      reuse = true;
    }
    slot = bar >= 3 ? bar - 3 : bar;
  }
  __device__ __forceinline__ bool used() const { return reuse || bar >= 3; }
};

// ------------------------------------------------------------------ records
// Two warps take turns at the chunks: a lane finds the records of four rows.  The first
// lane of every run of rows that are neighbours in the cache copies the run into shared
// memory by one bulk copy, and a warp's next chunk is looked up, and asked into L2, before
// the wait for the buffer (one warp for both took longer over a chunk than the MMAs).
// Bulk copies of single records take 65 cycles each, 8,300 a chunk: a selection, and
// pages of a few entries, go by 16-B copies, two lanes to a record, in 1,700 (40 queries x
// 512 selected: 45 -> 41 us).  A window chunk is read by the K group itself (its records
// do not fit the buffer).
__device__ __forceinline__ void paged_fetch(const PagedArgs &A, PagedShared &S, unsigned char *sm, int c_begin, int c_end, int first) {
  const int lane = threadIdx.x & 31;
  const bool scattered = A.sel != nullptr || A.page < kPgScatter;
  PagedCursor C;
  C.c = c_begin + first;
  C.end = c_end;
  C.qi = S.start;
  C.off = S.off;
  C.Q = S.Q;
  unsigned rec[4];                                   // rows 32 g + lane: the record
  uint32_t valid[4];
  int rows[4], all_rows = 0;               // of the run this lane leads, 0: none; of the chunk
  int4 at;
  int seq, win;
  auto look_up = [&]() {
    at = make_int4(C.qi, C.local(), C.Q.chunks, C.off);
    seq = C.Q.seq;
    win = C.window() ? C.Q.win : 0;
    const int i0 = (C.local() - (C.Q.win > 0 ? 1 : 0)) * kPgChunk + lane;
    int j[4];
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const int i = i0 + 32 * g;
      j[g] = win == 0 && i < C.Q.n ? i : -1;
      if (j[g] >= 0 && A.sel != nullptr) j[g] = __ldg(A.sel + (int64_t)C.qi * A.sel_stride + i);
    }
    const int vis = A.sel != nullptr ? __ldg(A.n_vis + C.qi) : C.Q.n;
    int id[4], off[4];
    bool out = false;
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const int col = (int)paged_col((unsigned)j[g], A);
      off[g] = j[g] - col * A.page;
      id[g] = j[g] >= 0 && j[g] < vis ? __ldg(A.table + (int64_t)C.Q.seq * A.table_stride + col) : -1;
    }
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const bool ok = id[g] >= 0 && id[g] < A.n_pages;
      out |= j[g] >= 0 && !ok;
      if (!ok) id[g] = -1;
      rec[g] = (unsigned)id[g] * (unsigned)A.page + (unsigned)off[g];
      const int pid = __shfl_up_sync(0xFFFFFFFFu, id[g], 1), poff = __shfl_up_sync(0xFFFFFFFFu, off[g], 1);
      const bool leads = ok && (lane == 0 || pid != id[g] || poff + 1 != off[g]);
      valid[g] = __ballot_sync(0xFFFFFFFFu, ok);
      // its run ends before the next leader or the next row without an entry
      const uint32_t lead = __ballot_sync(0xFFFFFFFFu, leads);
      const uint32_t stop = (lead | ~valid[g]) & ~((2u << lane) - 1u);     // (lane 31: 2 << 31 is 0)
      rows[g] = leads ? (stop != 0u ? __ffs(stop) - 1 : 32) - lane : 0;
    }
    all_rows = __popc(valid[0]) + __popc(valid[1]) + __popc(valid[2]) + __popc(valid[3]);
    if (out) record_error(A.status, CSA2_ERR_BOUNDS);
  };
  bool more = C.settle(A);
  if (more) look_up();
  int k = first;
  for (; more; k += 2) {
    PagedInfo &I = S.info[k & (kPgInfo - 1)];
    if (lane == 0) {
      I.at = at;
      I.seq = seq;
      I.win = win;
      I.first = C.Q.first;
#pragma unroll
      for (int g = 0; g < 4; g++)
        I.valid[g] = win == 0 ? valid[g] : win > 32 * g ? (win >= 32 * g + 32 ? 0xFFFFFFFFu : (1u << (win - 32 * g)) - 1u) : 0u;
    }
    if (k >= 1) paged_wait(A, S, &S.raw_free[first ^ 1], ((k - 1) >> 1) & 1);
    if (paged_bad(S)) break;                         // no copy is started any more
    uint64_t *full = &S.raw_full[first];
    if (scattered) {
#pragma unroll
      for (int g = 0; g < 8; g++) {                  // two lanes to a row of 16
        const int from = (g & 1) * 16 + (lane >> 1);
        const uint8_t *src = A.pages + (int64_t)__shfl_sync(0xFFFFFFFFu, rec[g >> 1], from) * kKvBytes + (lane & 1) * 16;
        unsigned char *dst = sm + kPgSmRaw + ((g >> 1) * 32 + from) * kKvBytes + (lane & 1) * 16;
        if ((valid[g >> 1] >> from) & 1u)
#pragma unroll
          for (int i = 0; i < kKvBytes; i += 32) ptx::cp_async16(dst + i, src + i);
      }
      ptx::cp_async_arrive(full);                    // (each lane's copies, pending from here on)
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive_expect_tx(full, scattered ? 0u : (uint32_t)(all_rows * kKvBytes));
    __syncwarp();
#pragma unroll
    for (int g = 0; g < 4; g++)
      if (!scattered && rows[g] > 0) ptx::bulk_load(sm + kPgSmRaw + (32 * g + lane) * kKvBytes, A.pages + (int64_t)rec[g] * kKvBytes, (uint32_t)(rows[g] * kKvBytes), full);
    C.c += 2;
    more = C.settle(A);
    if (more) {
      look_up();
#pragma unroll
      for (int g = 0; g < 4; g++)
        if (!scattered && rows[g] > 0) ptx::bulk_prefetch_l2(A.pages + (int64_t)rec[g] * kKvBytes, (uint32_t)(rows[g] * kKvBytes));
    }
  }
  // its last copies have landed before the CTA may leave (bounded)
  if (k >= 2) ptx::mbar_wait(&S.raw_full[first], ((k >> 1) - 1) & 1);
}

// The K group dequantises the chunks into a ring of slabs in tensor memory, in two
// teams of four warps, a row per thread: team g has slabs g and g + 2 of every chunk.
// QK reads them there, 32 cycles an MMA (48 from shared memory, whose bandwidth PV
// needs), and the V group copies them from there.
__device__ __forceinline__ void paged_load(const PagedArgs &A, PagedShared &S, unsigned char *sm, int n_run, uint32_t tmem) {
  const int lt = (int)threadIdx.x - kPgSoft, lane = lt & 31;
  const int e = lt & 127, team = lt >> 7;            // row
  const uint32_t kcol0 = tmem + ((uint32_t)(e & 96) << 16) + kPgColK;
  PagedSlab<2> n((unsigned)team);                    // the next slab
  uint32_t met = 0;
  for (int k = 0; k < n_run; k++) {
    // (a run's first chunk, if a window, needs no records: its own description will do)
    const bool ahead = k == 0 && S.Q.win > 0 && S.off == S.end[0];
    if (!ahead) paged_wait(A, S, &S.raw_full[k & 1], (k >> 1) & 1);
    PagedInfo &I = S.info[k & (kPgInfo - 1)];
    const int win = __shfl_sync(0xFFFFFFFFu, ahead ? S.Q.win : I.win, 0);
    if (win > 0 && paged_bad(S)) break;
    int kx = 0;
    uint4 ws = make_uint4(0u, 0u, 0u, 0u);           // a window record's 16 scales
    const uint8_t *wrec = nullptr;
    uint4 x[2];                                      // 32 of its dims
    auto window_dims = [&](int i) {
#pragma unroll
      for (int u = 0; u < 2; u++)
        x[u] = wrec != nullptr ? __ldg(reinterpret_cast<const uint4 *>(wrec + (team + 2 * (i >> 2)) * 128 + (i & 3) * 32 + u * 16))
                               : make_uint4(0u, 0u, 0u, 0u);
    };
    if (win > 0) {
      // ---------------------------------------------------- a window's rows and scale
      if (e < win) {
        const int ring = (int)(((unsigned)(ahead ? S.Q.first : I.first) + (unsigned)e) % (unsigned)A.swa_cap);
        wrec = A.swa + ((int64_t)(ahead ? S.Q.seq : I.seq) * A.swa_cap + ring) * kSwaBytes;
        ws = __ldg(reinterpret_cast<const uint4 *>(wrec + 512));
      }
      window_dims(0);
      // the range of the scales' exponents (0 marks a group of zeros)
      const uint32_t w4[4] = {ws.x, ws.y, ws.z, ws.w};
      int lo = 255, hi = 0;
#pragma unroll
      for (int i = 0; i < 16; i++) {
        const int x = (int)((w4[i >> 2] >> (8 * (i & 3))) & 0xFFu);
        if (x != 0) { lo = min(lo, x); hi = max(hi, x); }
      }
      lo = __reduce_min_sync(0xFFFFFFFFu, lo);
      hi = __reduce_max_sync(0xFFFFFFFFu, hi);
      if (lt == 0) { S.emin = 255; S.emax = 0; }
      paged_meet(A, S, 1, met);
      if (lane == 0) { atomicMin(&S.emin, lo); atomicMax(&S.emax, hi); }
      paged_meet(A, S, 1, met);
      const int emax = S.emax - 127, emin = S.emin - 127;
      if (emax > -127 && (emax > 7 || emin < -15)) kx = 7 - emax;
    }
    if (lt == 0) I.kx = kx;
    // 32 dims (16 words of two f16) at a time.  (One slab's code, not the chunk's: six
    // roles share the instruction caches, and with everything unrolled the warps waited
    // for instructions four times as long as they issued them.)
    uint32_t kcol = kcol0;
    auto begin = [&]() {
      kcol = kcol0 + n.slot * 64;
      if (n.used()) paged_wait(A, S, &S.k_free[n.last_bar()], n.last_phase());
      ptx::tc_fence_after();
    };
    auto end = [&]() {
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.k_full[n.bar]);
      n.next();
    };
    auto release = [&]() {                           // the buffer is read
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.raw_free[k & 1]);
    };
    if (win > 0) {
      if (ahead) paged_wait(A, S, &S.raw_full[0], 0);
      release();
#pragma unroll 1
      for (int i = 0; i < 8; i++) {
        const int b = team + 2 * (i >> 2);
        const uint32_t wb = b == 0 ? ws.x : b == 1 ? ws.y : b == 2 ? ws.z : ws.w;
        if ((i & 3) == 0) begin();
        const int eb = (int)((wb >> (8 * (i & 3))) & 0xFFu);
        const __half2 fac = __float2half2_rn(eb == 0 ? 0.f : ldexpf(1.f, eb - 127 + kx));
        uint32_t o[16];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t w[4] = {x[h].x, x[h].y, x[h].z, x[h].w};
#pragma unroll
          for (int q = 0; q < 8; q++) {
            const uint32_t hv = e4m3x2_to_f16x2(w[q >> 1] >> (16 * (q & 1)));
            const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&hv), fac);
            o[8 * h + q] = *reinterpret_cast<const uint32_t *>(&y);
          }
        }
        ptx::tmem_st_32x32b_x16(kcol + (i & 3) * 16, o);
        if (i < 7) window_dims(i + 1);
        if ((i & 3) == 3) end();
      }
    } else {
      const bool ok = ((I.valid[e >> 5] >> lane) & 1u) != 0u;
      // Records are 18 16-B units apart, so rows r and r + 4 of a unit share their banks:
      // every other four rows read the units of a pair the other way round (shared memory
      // is what bounds the kernel; the selects are cheap).  Rows without an entry read
      // what is there: any code is finite, and their scales are zeroed.
      const bool flip = (e & 4) != 0;
      const unsigned char *raw = sm + kPgSmRaw + e * kKvBytes + (flip ? 16 : 0);
      const int other = flip ? -16 : 16;
      uint32_t sc[4];                                // two slabs' eight scales
      {
        const uint4 x = *reinterpret_cast<const uint4 *>(raw + 256), y = *reinterpret_cast<const uint4 *>(raw + 256 + other);
        const uint32_t x0 = team ? x.z : x.x, x1 = team ? x.w : x.y, y0 = team ? y.z : y.x, y1 = team ? y.w : y.y;
        sc[0] = ok ? (flip ? y0 : x0) : 0u;
        sc[1] = ok ? (flip ? y1 : x1) : 0u;
        sc[2] = ok ? (flip ? x0 : y0) : 0u;
        sc[3] = ok ? (flip ? x1 : y1) : 0u;
      }
      raw += team * 64;
#pragma unroll 1
      for (int t = 0; t < 2; t++) {
        uint4 code[4];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const uint4 x = *reinterpret_cast<const uint4 *>(raw + j * 16), y = *reinterpret_cast<const uint4 *>(raw + j * 16 + other);
          code[j] = flip ? y : x;
          code[j + 1] = flip ? x : y;
        }
        raw += 128;
        if (t == 1) release();
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const uint32_t w[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
          const uint32_t two = e4m3x2_to_f16x2(sc[j >> 1] >> (16 * (j & 1)));
          const uint32_t s2[2] = {__byte_perm(two, two, 0x1010), __byte_perm(two, two, 0x3232)};
          uint32_t o[16];
#pragma unroll
          for (int u = 0; u < 4; u++) {
            uint32_t x[4];
            e2m1x8_to_f16(w[u], x);
#pragma unroll
            for (int q = 0; q < 4; q++) {
              const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x[q]), *reinterpret_cast<const __half2 *>(&s2[u >> 1]));
              o[4 * u + q] = *reinterpret_cast<const uint32_t *>(&y);
            }
          }
          if (j == 0) begin();
          ptx::tmem_st_32x32b_x16(kcol + j * 16, o);
        }
        sc[0] = sc[2];
        sc[1] = sc[3];
        end();
      }
    }
  }
}

// 16-B chunk lt % 64 of head lt / 64 + 4 i of Q, times `by`, into shared memory as f16,
// K-major, 128B swizzle; returns the warp's largest |q|.
__device__ __forceinline__ uint32_t put_q(unsigned char *sm, int lt, const uint4 &x, int i, float by) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w}, m = 0u;
#pragma unroll
  for (int u = 0; u < 4; u++) {
    m = __vmaxu2(m, w[u] & 0x7FFF7FFFu);
    const __half2 h2 = __floats2half2_rn(bf16_lo(w[u]) * by, bf16_hi(w[u]) * by);
    w[u] = *reinterpret_cast<const uint32_t *>(&h2);
  }
  const int h = (lt >> 6) + 4 * i;
  unsigned char *dst = sm + kPgSmQ + ((lt & 63) >> 3) * 1024 + (h >> 3) * 8192;
  *reinterpret_cast<uint4 *>(dst + sw128(h & 7, lt & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
  return __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
}
__device__ __forceinline__ uint32_t head_max(const PagedShared &S, int g, int i) {       // of head g + 4 i
  return max(S.hmax[2 * g][i], S.hmax[2 * g + 1][i]);
}
__device__ __forceinline__ int head_power(uint32_t m) {
  const int ex = (int)(m >> 7) - 127;                // max |q| in [2^ex, 2^(ex + 1)) if normal
  return m == 0u || m >= 0x7F80u || (ex >= -4 && ex < 15) ? 0 : max(ex - 14, -126);
}
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// The V group brings Q of a query into shared memory.  One pass as it is where every head's
// max |q| lies in [2^-4, 2^15), or is zero or not finite: f16 holds a bf16 value exactly down
// to 2^-17 and to 2^-25 below; else a second one.  Heads of about one size (2^18) that are too
// small, or all too large, go under one power of two that brings the largest into [2^14, 2^15)
// and counts as part of the scale.  Else each head that needs it has its own, a unit, as one of
// them may be 2^40 times another, and under one power the smaller would become zero: that is
// slower (see paged_units), so it is not for queries that are small as a whole.  (The parities, 1 of the group's
// meetings, 2 of q_done, 4 of the queries, rest in shared memory between queries: the copying
// loop has no register for them.)
__device__ __forceinline__ void stage_q(const PagedArgs &A, PagedShared &S, unsigned char *sm, int qi, int k) {
  const int lt = (int)threadIdx.x - kPgSoft - kPgLoad, lane = lt & 31;
  uint32_t met = S.v_met[lt >> 5];
  const uint4 *src = reinterpret_cast<const uint4 *>(A.q + (int64_t)qi * kHeads * kDim) + lt;
#pragma unroll 1
  for (int i0 = 0; i0 < 16; i0 += 8) {
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = __ldg(src + (i0 + i) * kPgLoad);
    if (i0 == 0 && k > 0) {                          // (the query before is multiplied)
      paged_wait(A, S, &S.q_done, (met >> 1) & 1);
      met ^= 2;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t m = put_q(sm, lt, x[i], i0 + i, 1.f);
      if (lane == 0) S.hmax[lt >> 5][i0 + i] = m;
    }
  }
  // (the maxima are read before q_full, and written again after the next q_done)
  paged_meet(A, S, 2, met);
  const uint32_t m0 = head_max(S, lane >> 4, lane & 15), m1 = head_max(S, 2 + (lane >> 4), lane & 15);
  const bool scaled = __any_sync(0xFFFFFFFFu, head_power(m0) != 0 || head_power(m1) != 0);
  // (of the two places for units, the softmax may still read the other for the query before)
  const int place = (int)(met >> 2) & 1;
  met ^= 4;
  float f = A.scale * 1.4426950408889634f;
  if (__builtin_expect(scaled, 0)) {
    const bool h0 = m0 != 0u && m0 < 0x7F80u, h1 = m1 != 0u && m1 < 0x7F80u;
    const int hi = (int)__reduce_max_sync(0xFFFFFFFFu, max(h0 ? m0 : 0u, h1 ? m1 : 0u) >> 7) - 127;
    const int lo = (int)__reduce_min_sync(0xFFFFFFFFu, min(h0 ? m0 : 0x7F80u, h1 ? m1 : 0x7F80u) >> 7) - 127;
    const bool units = hi - lo > 18 || (hi >= 15 && lo < 15) || hi < -86;
#pragma unroll 1
    for (int i0 = 0; i0 < 16; i0 += 4) {
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; i++) x[i] = __ldg(src + (i0 + i) * kPgLoad);
#pragma unroll
      for (int i = 0; i < 4; i++)
        put_q(sm, lt, x[i], i0 + i, power_of_2(-(units ? head_power(head_max(S, lt >> 6, i0 + i)) : hi - 14)));
    }
    if (units && lt < kHeads) S.unit[place][lt] = -power_of_2(head_power(head_max(S, lt & 3, lt >> 2)));
    f *= units ? -1.f : power_of_2(hi - 14);
  }
  if (lt == 0) {
    PagedInfo &I = S.info[k & (kPgInfo - 1)];
    I.f = f;
    I.units = place;
  }
  ptx::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    S.v_met[lt >> 5] = met;
    ptx::mbar_arrive(&S.q_full);
  }
  __syncwarp();
}

// The V group copies the slabs from tensor memory into a ring in shared memory, where
// PV reads them MN-major, in two teams as the K group: a thread per row, holding a slab
// in registers until PV has freed its slot.  (Dequantising them a second time cost more
// arithmetic than everything else together.)
__device__ __forceinline__ void paged_copy(const PagedArgs &A, PagedShared &S, unsigned char *sm, int n_run, uint32_t tmem) {
  const int lt = (int)threadIdx.x - kPgSoft - kPgLoad, lane = lt & 31;
  const int e = lt & 127, team = lt >> 7;
  const uint32_t kcol = tmem + ((uint32_t)(e & 96) << 16) + kPgColK;
  // the row's 128 B of the first 64 dims in slot 0, chunk c at `tile` ^ 16 c
  const uintptr_t tile = reinterpret_cast<uintptr_t>(sm + kPgSmV + (e >> 3) * 2048 + (e & 7) * 128 + (e & 7) * 16);
  static_assert(kPgVRing == kPgKRing, "one slot number for both rings");
  PagedSlab<2> n((unsigned)team);
  bool last = true;                                  // the chunk before was its query's last
#pragma unroll 1
  for (int i = 0; i < 2 * n_run; i++, n.next()) {
    if (last && (i & 1) == 0) {                      // the next query's, before its first slab
      int qi = S.start;                              // (the first one's while its records are looked up)
      if (i > 0) {
        paged_wait(A, S, &S.raw_full[(i >> 1) & 1], (i >> 2) & 1);
        if (paged_bad(S)) break;
        qi = S.info[(i >> 1) & (kPgInfo - 1)].at.x;
      }
      stage_q(A, S, sm, qi, i >> 1);
    }
    uint32_t r[2][32];
    paged_wait(A, S, &S.k_full[n.bar], n.phase);
    ptx::tc_fence_after();
    ptx::tmem_ld_32x32b_x32(kcol + n.slot * 64, r[0]);
    ptx::tmem_ld_32x32b_x32(kcol + n.slot * 64 + 32, r[1]);
    ptx::tmem_wait_ld();
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.k_free[n.bar]);
    if (n.used()) paged_wait(A, S, &S.v_free[n.last_bar()], n.last_phase());
    const uintptr_t at = tile + n.slot * kPgSlab;
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int c = 0; c < 8; c++)
        *reinterpret_cast<uint4 *>((at ^ (uintptr_t)(c << 4)) + h * 1024) =
            make_uint4(r[h][4 * c], r[h][4 * c + 1], r[h][4 * c + 2], r[h][4 * c + 3]);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.v_full[n.bar]);
    if ((i & 1) == 0) {
      const PagedInfo &I = S.info[(i >> 1) & (kPgInfo - 1)];
      last = __shfl_sync(0xFFFFFFFFu, I.at.y + 1 == I.at.z, 0);
    }
  }
}

// ------------------------------------------------------------------ softmax, read-out
// Two fp32 at a time.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// This lane's entry: 32 heads' logits in log2 units (-inf for a row without an
// entry: `none` = -inf, else 0), plus the heads' `less`.  (The product is rounded before
// the sum, as the maximum's was: in one step, the difference of two huge logits would be
// off by that rounding.)
__device__ __forceinline__ void paged_logits(uint32_t ta, float f, float none, const float *less, uint64_t (&s)[16]) {
  const uint64_t f2 = pair(f, f), n2 = pair(none, none);
#pragma unroll
  for (int h = 0; h < 32; h += 16) {
    uint32_t a[16];
    ptx::tmem_ld_32x32b_x16(ta + h, a);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(less + h + i);
      s[(h + i) / 2] = add2(fma2(pair(__uint_as_float(a[i]), __uint_as_float(a[i + 1])), f2, n2), m.x);
      s[(h + i) / 2 + 1] = add2(fma2(pair(__uint_as_float(a[i + 2]), __uint_as_float(a[i + 3])), f2, n2), m.y);
    }
  }
}
// Their numerators 2^s; true where one is out of the range that f16 should hold.
__device__ __forceinline__ bool paged_numerators(uint64_t (&s)[16]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const float2 x = unpair(s[i]);
    const float p0 = ex2(x.x), p1 = ex2(x.y);
    s[i] = pair(p0, p1);
    top = fmaxf(top, fmaxf(p0, p1));
  }
  return top > 32768.f;
}

// This lane's entry: S of 32 heads times their units, in place (and for the whole query, so
// that nothing else has to know of them; a factor in the logits took 8 % of every row's time).
__device__ __noinline__ void paged_units(uint32_t ta, const float *unit) {
#pragma unroll 1
  for (int h = 0; h < 32; h += 16) {
    uint32_t a[16];
    ptx::tmem_ld_32x32b_x16(ta + h, a);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; i++) a[i] = __float_as_uint(__uint_as_float(a[i]) * unit[h + i]);
    ptx::tmem_st_32x32b_x16(ta + h, a);
  }
  ptx::tmem_wait_st();
}

// Warp w has TMEM lane quarter w % 4 (S: entries, O: dims) and heads 32 (w / 4) ..
__device__ __forceinline__ void paged_softmax(const PagedArgs &A, PagedShared &S, unsigned char *sm, int n_run,
                                              uint32_t tmem) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int quarter = warp & 3, hb = (warp >> 2) * 32, e_row = quarter * 32 + lane;
  const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16);
  uint64_t l_acc[16];                                // 32 heads' denominators
  float q_f = 0.f;                                   // logits in log2 units per unit of S; negative: S still lacks its units
  uint32_t met = 0;
  float o_scale = 1.f;                               // what O still has to be multiplied by
  bool acc = false;                                  // O holds something of this query
  int lc0 = 0;
  for (int k = 0; k < n_run; k++) {
    paged_wait(A, S, &S.s_full, k & 1);
    ptx::tc_fence_after();
    const PagedInfo &info = S.info[k & (kPgInfo - 1)];
    if (k == 0 || info.at.y == 0) {                  // a query begins
      lc0 = info.at.y;
      acc = false;
      o_scale = 1.f;
#pragma unroll
      for (int i = 0; i < 16; i++) l_acc[i] = 0ull;
      if (t < kHeads) S.less[t] = kPgNoRef;
      q_f = info.f;
      if (t == 0) S.units = info.units;
      paged_meet(A, S, 0, met);
    }
    const int kx = info.kx;
    const float f = kx == 0 ? q_f : ldexpf(q_f, -kx);
    const float none = ((info.valid[quarter] >> lane) & 1u) != 0u ? 0.f : -INFINITY;
    const uint32_t ta = tq + kPgColS + hb;
    uint64_t s[16];
    paged_logits(ta, f, none, &S.less[hb], s);
    const bool over = paged_numerators(s);
    // (a window's 2^-kx is undone before the next chunk; heads with units are always dealt with here)
    if (__builtin_expect(soft_any(over || q_f < 0.f || (acc && o_scale != 1.f)), 0)) {
      if (__builtin_expect(q_f < 0.f, 0)) paged_units(ta, &S.unit[S.units & 1][hb]);
      // the chunk's maximum of every head, 16 at a time: lanes L and L + 16 end with head L
#pragma unroll 1
      for (int h = 0; h < 32; h += 16) {
        uint32_t a[16];
        float v[16];
        ptx::tmem_ld_32x32b_x16(ta + h, a);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] = __fmul_rn(__uint_as_float(a[i]), f) + none;
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1) {
          const bool upper = (lane & w) != 0;
#pragma unroll
          for (int i = 0; i < 8; i++) {
            if (i < w) {
              const float keep = upper ? v[i + w] : v[i], send = upper ? v[i] : v[i + w];
              v[i] = fmaxf(keep, __shfl_xor_sync(0xFFFFFFFFu, send, w));
            }
          }
        }
        v[0] = fmaxf(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 16));
        if (lane < 16) S.red[quarter][hb + h + lane] = v[0];
      }
      soft_sync();
      if (t < kHeads) {
        const float cm = fmaxf(fmaxf(S.red[0][t], S.red[1][t]), fmaxf(S.red[2][t], S.red[3][t])) - kPgShift;
        const float mo = -S.less[t];
        float al = 1.f;
        if (cm > mo + kPgRaise) {
          al = mo == -kPgNoRef ? 0.f : exp2f(mo - cm);
          S.less[t] = -cm;
        }
        S.alpha[t] = al;
      }
      soft_sync();
      if (acc) {
        // O *= alpha (and the window's factor), once PV of the chunk before is complete
        paged_wait(A, S, &S.o_done, (k - 1) & 1);
        ptx::tc_fence_after();
        for (int blk = warp >> 2; blk < 4; blk += 2)
#pragma unroll 1
          for (int h = 0; h < kHeads; h += 16) {
            uint32_t x[16];
            const uint32_t to = tq + kPgColO + blk * kHeads + h;
            ptx::tmem_ld_32x32b_x16(to, x);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; i++) x[i] = __float_as_uint(__uint_as_float(x[i]) * S.alpha[h + i] * o_scale);
            ptx::tmem_st_32x32b_x16(to, x);
          }
        ptx::tmem_wait_st();
        o_scale = 1.f;
      }
#pragma unroll
      for (int i = 0; i < 16; i++) {
        const float2 l = unpair(l_acc[i]);
        l_acc[i] = pair(l.x * S.alpha[hb + 2 * i], l.y * S.alpha[hb + 2 * i + 1]);
      }
      paged_logits(ta, f, none, &S.less[hb], s);
      paged_numerators(s);
    }
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.s_free);
#pragma unroll
    for (int i = 0; i < 16; i++) l_acc[i] = add2(l_acc[i], s[i]);
    // P is free once PV of the chunk before is complete
    if (k > 0) paged_wait(A, S, &S.o_done, (k - 1) & 1);
    unsigned char *row = sm + kPgSmP + (e_row >> 3) * 1024;
#pragma unroll
    for (int q = 0; q < 4; q++) {
      uint32_t o[4];
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const float2 x = unpair(s[4 * q + u]);
        const __half2 h2 = __floats2half2_rn(x.x, x.y);
        o[u] = *reinterpret_cast<const uint32_t *>(&h2);
      }
      *reinterpret_cast<uint4 *>(row + sw128(e_row & 7, (hb >> 3) + q)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    ptx::tc_fence_before();
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.p_full);
    acc = true;
    if (kx != 0) o_scale = ldexpf(1.f, -kx);
    const int4 I = info.at;
    const int lc = I.y;
    if (lc + 1 != I.z && k + 1 != n_run) continue;
    if ((unsigned)I.x >= (unsigned)A.n_q) continue;  // (a description left from before, once a wait has run out)

    // -------------------------------------------------------- the query's last chunk here: read-out
#pragma unroll
    for (int h = 0; h < 32; h += 16) {               // (as the maxima)
      float v[16];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float2 l = unpair(l_acc[h / 2 + i]);
        v[2 * i] = l.x;
        v[2 * i + 1] = l.y;
      }
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1) {
        const bool upper = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          if (i < w) {
            const float keep = upper ? v[i + w] : v[i], send = upper ? v[i] : v[i + w];
            v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, w);
          }
        }
      }
      v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], 16);
      if (lane < 16) S.l[quarter][hb + h + lane] = v[0];
    }
    paged_meet(A, S, 0, met);
    const bool whole = lc0 == 0 && lc + 1 == I.z;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (lc0 > 0 ? 0 : 1);
    if (t < kHeads) {
      const float l = S.l[0][t] + S.l[1][t] + S.l[2][t] + S.l[3][t];
      if (whole) {
        if (A.lse != nullptr)
          A.lse[(int64_t)I.x * kHeads + t] =
              l > 0.f || l != l ? (log2f(l) - S.less[t]) * 0.6931471805599453f : -INFINITY;
        S.alpha[t] = l != 0.f ? o_scale / l : 0.f;
      } else {
        A.part_ml[slot * 2 * kHeads + t] = -S.less[t];
        A.part_ml[slot * 2 * kHeads + kHeads + t] = l;
        S.alpha[t] = o_scale;
      }
    }
    const int pos = __ldg(A.pos + I.x);
    paged_meet(A, S, 0, met);
    paged_wait(A, S, &S.o_done, k & 1);              // PV is complete
    ptx::tc_fence_after();
    for (int blk = warp >> 2; blk < 4; blk += 2) {
      const int d = blk * 128 + quarter * 32 + lane;
      float cs = 1.f, sn = 0.f;
      if (whole && d >= kRopeOff) {
        turn_cs((uint64_t)(int64_t)pos * A.turn[(d - kRopeOff) >> 1], cs, sn);
        if (d & 1) sn = -sn;                         // (a, b) -> (a c + b s, b c - a s)
      }
#pragma unroll 1
      for (int h = 0; h < kHeads; h += 16) {
        uint32_t r[16];
        ptx::tmem_ld_32x32b_x16(tq + kPgColO + blk * kHeads + h, r);
        ptx::tmem_wait_ld();
        if (!whole) {
          float *P = A.part + (slot * kHeads + h) * kDim + d;
#pragma unroll
          for (int i = 0; i < 16; i++) P[i * kDim] = __uint_as_float(r[i]) * S.alpha[h + i];
          continue;
        }
        const int64_t at = ((int64_t)I.x * kHeads + h) * kDim + d;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          // the lane's dim and its neighbour's, of two heads: the rotation by -pos needs
          // both, and an even lane then stores the pair of one head, an odd lane of the other
          float x0 = __uint_as_float(r[i]) * S.alpha[h + i], x1 = __uint_as_float(r[i + 1]) * S.alpha[h + i + 1];
          float y0 = __shfl_xor_sync(0xFFFFFFFFu, x0, 1), y1 = __shfl_xor_sync(0xFFFFFFFFu, x1, 1);
          if (blk == 3 && quarter >= 2) {
            const float w0 = x0 * cs + y0 * sn, w1 = x1 * cs + y1 * sn;
            y0 = y0 * cs - x0 * sn;
            y1 = y1 * cs - x1 * sn;
            x0 = w0;
            x1 = w1;
          }
          if (A.out_f32) {
            static_cast<float *>(A.out)[at + (int64_t)i * kDim] = x0;
            static_cast<float *>(A.out)[at + (int64_t)(i + 1) * kDim] = x1;
          } else {
            const bool odd = (lane & 1) != 0;
            const __nv_bfloat162 v = odd ? __floats2bfloat162_rn(y1, x1) : __floats2bfloat162_rn(x0, y0);
            *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(A.out) + at + (int64_t)(i + (odd ? 1 : 0)) * kDim - (odd ? 1 : 0)) = v;
          }
        }
      }
    }
    ptx::tc_fence_before();                          // (before the next query's PV, behind p_full)
    // the first CTA after the one that begins a cut query names it for the join (not by a
    // description that may be none)
    if (t == 0 && !S.bad && lc0 > 0 && (int)blockIdx.x == run_first_cut(I.w, S.T, S.G, A.n_q))
      A.joins[blockIdx.x] = make_int4(I.x, I.z, I.w, S.T);
  }
}

// ------------------------------------------------------------------ MMAs
// One thread each for QK and PV, chosen by elect.sync, with operands addressed by
// a base plus constants: it issues an MMA every 48 cycles, what N = 64 takes with
// both operands in shared memory (6 KB).  With the descriptors built at each MMA
// a thread issued one in 81 to 118 cycles.
__device__ __forceinline__ void paged_issue_qk(const PagedArgs &A, PagedShared &S, unsigned char *sm, int n_run,
                                               uint32_t tmem) {
  constexpr uint32_t id = idesc_m128(0, true, kHeads);
  const uint64_t d_q = ptx::smem_desc(ptx::smem_u32(sm + kPgSmQ), 16, 8192, 2);
  uint32_t q_parity = 0;
  bool fresh = true;                                 // the next chunk is a query's first here
  PagedSlab<1> n(0u);
  for (int k = 0; k < n_run && !S.bad; k++) {
    if (k >= 1) paged_wait(A, S, &S.s_free, (k - 1) & 1);
#pragma unroll 1
    for (int b = 0; b < 4; b++) {                    // S^T += K Q^T over slab 4 k + b
      paged_wait(A, S, &S.k_full[n.bar], n.phase);
      if (b == 0 && fresh) {
        paged_wait(A, S, &S.q_full, q_parity);
        q_parity ^= 1;
      }
      ptx::tc_fence_after();
      const uint64_t qa = d_q + b * 128;
      const uint32_t ka = tmem + kPgColK + n.slot * 64;
#pragma unroll
      for (int kk = 0; kk < 8; kk++)
        ptx::tc_mma_f16_ts(tmem + kPgColS, ka + kk * 8, qa + (kk >> 2) * 64 + (kk & 3) * 2, id,
                           kk > 0 ? 1u : (uint32_t)(b > 0));
      ptx::tc_commit(&S.k_free[n.bar]);
      n.next();
    }
    ptx::tc_commit(&S.s_full);
    const int4 at = S.info[k & (kPgInfo - 1)].at;
    fresh = at.y + 1 == at.z;
    if (fresh) ptx::tc_commit(&S.q_done);
  }
  ptx::tc_commit(&S.drain);
}
__device__ __forceinline__ void paged_issue_pv(const PagedArgs &A, PagedShared &S, unsigned char *sm, int n_run,
                                               uint32_t tmem) {
  constexpr uint32_t id = idesc_m128(1, true, kHeads) | (1u << 16);   // both operands MN-major
  const uint64_t d_v = ptx::smem_desc(ptx::smem_u32(sm + kPgSmV), 1024, 2048, 2);
  const uint64_t d_p = ptx::smem_desc(ptx::smem_u32(sm + kPgSmP), 1024, 1024, 2);
  PagedSlab<1> n(0u);
  for (int k = 0; k < n_run && !S.bad; k++) {
    paged_wait(A, S, &S.p_full, k & 1);
    const uint32_t acc = k == 0 || S.info[k & (kPgInfo - 1)].at.y == 0 ? 0u : 1u;
#pragma unroll 1
    for (int b = 0; b < 4; b++) {                    // O^T block b += V^T P over slab 4 k + b
      paged_wait(A, S, &S.v_full[n.bar], n.phase);
      ptx::tc_fence_after();
      const uint64_t va = d_v + n.slot * (kPgSlab >> 4);
#pragma unroll
      for (int ks = 0; ks < kPgChunk / 16; ks++)
        ptx::tc_mma_bf16(tmem + kPgColO + b * kHeads, va + ks * 256, d_p + ks * 128, id, ks > 0 ? 1u : acc);
      ptx::tc_commit(&S.v_free[n.bar]);
      n.next();
    }
    ptx::tc_commit(&S.o_done);
  }
  ptx::tc_commit(&S.drain);
}

__global__ void __launch_bounds__(kPgThreads, 1) paged_attn_kernel(const __grid_constant__ PagedArgs A) {
  extern __shared__ __align__(1024) unsigned char pg_smem_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(pg_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(16) PagedShared S;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (t == 0) {
    for (int i = 0; i < 6; i++) {
      ptx::mbar_init(&S.k_full[i], kPgLoad / 64);
      ptx::mbar_init(&S.k_free[i], 1 + kPgLoad / 64);
      ptx::mbar_init(&S.v_full[i], kPgLoad / 64);
      ptx::mbar_init(&S.v_free[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      ptx::mbar_init(&S.raw_full[i], 1);
      ptx::mbar_init(&S.raw_free[i], kPgLoad / 32);
    }
    ptx::mbar_init(&S.q_full, kPgLoad / 32);
    ptx::mbar_init(&S.q_done, 1);
    for (int i = 0; i < 3; i++) ptx::mbar_init(&S.meet[i], 8);
    ptx::mbar_init(&S.s_full, 1);
    ptx::mbar_init(&S.s_free, kPgSoft / 32);
    ptx::mbar_init(&S.p_full, kPgSoft / 32);
    ptx::mbar_init(&S.o_done, 1);
    ptx::mbar_init(&S.drain, 2);
    S.bad = 0;
    for (int i = 0; i < 8; i++) S.v_met[i] = 0u;
    S.start = S.off = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0) ptx::tmem_alloc(&S.tmem, kPgTmemCols);
  griddep_wait();
  griddep_launch();

  // ---------------------------------------------------------- this CTA's run
  // prefix sums of the queries' chunks: thread t has queries [u0, u1)
  const int per = (A.n_q + kPgThreads - 1) / kPgThreads, u0 = min(t * per, A.n_q), u1 = min(u0 + per, A.n_q);
  int mine = 0;
  bool any_bad = false, none = false;
  PagedQuery own = {};                               // the last of them
  for (int q = u0; q < u1; q++) {
    own = paged_query(A, q);
    mine += own.chunks;
    any_bad |= own.bad;
    none |= own.chunks == 0;
  }
  if (any_bad && blockIdx.x == 0) record_error(A.status, CSA2_ERR_BOUNDS);
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) S.scan[warp] = inc;
  none = __syncthreads_or(none) != 0;
  int before = 0, total = 0;
  for (int w = 0; w < kPgThreads / 32; w++) {
    if (w < warp) before += S.scan[w];
    total += S.scan[w];
  }
  before += inc - mine;
  const int T = total, G = run_ctas(T, gridDim.x);
  // g T / G, by the launch's reciprocal of its grid (T <= grid: G = T)
  const int each = T > (int)gridDim.x ? (int)magic_div((unsigned)T, A.grid_mul, A.grid_shift) : min(T, 1);
  const int over = T - each * G;
  const int snap = T <= G ? 0 : min(kPgSnap, max(each / kPgSnapRun, kPgSnapFew * A.n_q > G ? 1 : 0));      // (run_snap)
  auto border = [&](int g) { return g * each + (over > 0 ? (int)magic_div((unsigned)(g * over), A.grid_mul, A.grid_shift) : 0); };
#pragma unroll
  for (int i = 0; i < 2; i++) {
    // the run's two ends
    const int g = min((int)blockIdx.x + i, G), raw = border(g);
    if (raw < T && before <= raw && raw < before + mine) {
      int o = before, q = u0;
      PagedQuery R = per == 1 ? own : paged_query(A, q);
      while (raw >= o + R.chunks) {
        o += R.chunks;
        R = paged_query(A, ++q);
      }
      const int head = raw - o, tail = o + R.chunks - raw;
      int c = raw;
      if (head <= snap && head <= tail) {
        c = o;
      } else if (tail <= snap) {                     // the next query that has any
        o += R.chunks;
        c = o;
        for (R.chunks = 0; R.chunks == 0 && ++q < A.n_q;) R = paged_query(A, q);
      }
      S.end[i] = c;
      if (i == 0) {
        S.start = q;
        S.off = o;
        S.Q = R;
      }
    } else if (raw >= T && t == 0) {
      S.end[i] = T;
    }
  }
  if (t == 0) {
    S.T = T;
    S.G = G;
    A.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  // queries with nothing to attend to: zeros
  for (int q = none ? blockIdx.x : A.n_q; q < A.n_q; q += gridDim.x) {
    if (paged_query(A, q).chunks > 0) continue;
    for (int i = t * 4; i < kHeads * kDim; i += kPgThreads * 4) {
      const int64_t o = (int64_t)q * kHeads * kDim + i;
      if (A.out_f32) *reinterpret_cast<float4 *>(static_cast<float *>(A.out) + o) = make_float4(0.f, 0.f, 0.f, 0.f);
      else *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(A.out) + o) = make_uint2(0u, 0u);
    }
    if (A.lse != nullptr && t < kHeads) A.lse[(int64_t)q * kHeads + t] = -INFINITY;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = S.tmem;
  const int c_begin = S.end[0], c_end = S.end[1], n_run = c_end - c_begin;

  if (warp < kPgSoft / 32) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPgRegsSoft));
    paged_softmax(A, S, sm, n_run, tmem);
  } else if (warp < (kPgSoft + kPgLoad) / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPgRegsK));
    paged_load(A, S, sm, n_run, tmem);
  } else if (warp < (kPgSoft + 2 * kPgLoad) / 32) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPgRegsV));
    paged_copy(A, S, sm, n_run, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPgRegsRest));
    if (warp == (kPgSoft + 2 * kPgLoad) / 32) {
      if (ptx::elect_one()) paged_issue_qk(A, S, sm, n_run, tmem);
    } else if (warp == (kPgSoft + 2 * kPgLoad) / 32 + 1) {
      if (ptx::elect_one()) paged_issue_pv(A, S, sm, n_run, tmem);
    } else {
      paged_fetch(A, S, sm, c_begin, c_end, warp - (kPgSoft + 2 * kPgLoad) / 32 - 2);
    }
    __syncwarp();
  }
  __syncthreads();
  if (S.bad) {
    // a wait ran out: every MMA issued here finishes before the tensor memory goes
    // back (bounded; each issuer commits to the drain barrier when it leaves)
    ptx::mbar_wait(&S.drain, 0);
    ptx::tc_fence_after();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kPgTmemCols);
  }
}

// Joins a cut query's partials: grid (kHeads, as many as queries can be cut), 128 NG
// threads.  A thread has four of its head's 512 dims, so a partial's row is read as 2 KB
// in one piece; NG groups of 128 threads each take every NG-th partial, with four loads in
// flight, the first of them beside the weights', and meet in shared memory.  Each warp
// finds its head's weights 2^(m_s - max m) by itself, a lane to a partial.  All sums have a
// fixed order, so the same inputs give the same bits.  A chain of L2 trips and a matter of
// waves: 40 registers hold 12 groups on an SM (at 50, 128 x 1,000 entries took 81 us
// instead of 75).  NG = 1 ends its waves evenly (32 x 4,096: 50 us; NG = 2: 57, NG = 4: 76;
// 8 x 4,096: 28, NG = 4: 31); a query or two, which do not fill the SMs, take NG = 4
// (1 x 4,096, 33 partials: 20.3 us, NG = 1: 21.0).
template <int NG>
__global__ void __launch_bounds__(128 * NG, 12 / NG) paged_join_kernel(const __grid_constant__ PagedArgs A, int n_ctas) {
  __shared__ float4 sum_sh[NG > 1 ? NG : 1][128];
  const int t = threadIdx.x, lane = t & 31, grp = t >> 7;
  const int h = blockIdx.x, d = (t & 127) * 4;
  griddep_wait();
  griddep_launch();
  // what the blockIdx.y-th CTA that names a cut query says: query, its chunks, its first chunk, all chunks
  int4 J = make_int4(-1, 0, 0, 0);
  int left = (int)blockIdx.y;
  for (int c0 = 0; c0 < n_ctas && J.x < 0; c0 += 160) {
    int4 x[5];
#pragma unroll
    for (int i = 0; i < 5; i++) x[i] = c0 + i * 32 + lane < n_ctas ? __ldcg(A.joins + c0 + i * 32 + lane) : make_int4(-1, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 5; i++) {
      const uint32_t named = __ballot_sync(0xFFFFFFFFu, x[i].x >= 0);
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, x[i].x >= 0 && __popc(named & ((1u << lane) - 1u)) == left);
      if (J.x < 0 && hit != 0u) {
        const int from = __ffs((int)hit) - 1;
        J.x = __shfl_sync(0xFFFFFFFFu, x[i].x, from);
        J.y = __shfl_sync(0xFFFFFFFFu, x[i].y, from);
        J.z = __shfl_sync(0xFFFFFFFFu, x[i].z, from);
        J.w = __shfl_sync(0xFFFFFFFFu, x[i].w, from);
      }
      left -= __popc(named);
    }
  }
  if (J.x < 0) return;
  const int qi = J.x, off = J.z, T = J.w, G = run_ctas(T, n_ctas);
  const int g0 = run_first_cut(off, T, G, A.n_q) - 1, g1 = run_last_cut(off, J.y, T, G, A.n_q);
  auto slot_of = [&](int g) { return 2 * (int64_t)g + (g == g0 ? 1 : 0); };
  // four of the group's partials, from the i0-th of a batch on
  auto rows = [&](int b0, int i0, float4 (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int i = i0 + j * NG;
      v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < 32 && b0 + i <= g1)
        v[j] = __ldcg(reinterpret_cast<const float4 *>(A.part + (slot_of(b0 + i) * kHeads + h) * kDim + d));
    }
  };
  float4 v[4];
  rows(g0, grp, v);                                  // (the first ones beside the weights)
  bool ahead = true;
  float M = -kPgNoRef, m = -kPgNoRef;
  int b0 = g0;
  for (int b = g0; b <= g1; b += 32) {
    m = b + lane <= g1 ? __ldcg(A.part_ml + slot_of(b + lane) * 2 * kHeads + h) : -kPgNoRef;
    M = fmaxf(M, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = 0.f;
  for (; b0 <= g1; b0 += 32) {
    float w = 0.f;                                   // of partial b0 + lane
    if (b0 + lane <= g1) {
      const float *ml = A.part_ml + slot_of(b0 + lane) * 2 * kHeads + h;
      if (g1 - g0 >= 32) m = __ldcg(ml);
      w = exp2f(m - M);
      L += w * __ldcg(ml + kHeads);
    }
    for (int i0 = grp; i0 < 32 && b0 + i0 <= g1; i0 += 4 * NG) {
      if (!ahead) rows(b0, i0, v);
      ahead = false;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int i = i0 + j * NG;
        const float u = __shfl_sync(0xFFFFFFFFu, w, i & 31);
        if (i < 32 && u != 0.f) {                    // (a partial that met no entry weighs nothing)
          y.x = fmaf(u, v[j].x, y.x);
          y.y = fmaf(u, v[j].y, y.y);
          y.z = fmaf(u, v[j].z, y.z);
          y.w = fmaf(u, v[j].w, y.w);
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
  if (NG > 1) {
    sum_sh[grp][t & 127] = y;
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int g = 1; g < NG; g++) {
      const float4 z = sum_sh[g][t];
      y.x += z.x;
      y.y += z.y;
      y.z += z.z;
      y.w += z.w;
    }
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;
  y.x *= inv;
  y.y *= inv;
  y.z *= inv;
  y.w *= inv;
  if (d >= kRopeOff) {
    const uint64_t pos = (uint64_t)(int64_t)__ldg(A.pos + qi);
    float c, s;
    turn_cs(pos * A.turn[(d - kRopeOff) >> 1], c, s);
    const float a = y.x, b = y.z;
    y.x = a * c + y.y * s;
    y.y = y.y * c - a * s;
    turn_cs(pos * A.turn[(d + 2 - kRopeOff) >> 1], c, s);
    y.z = b * c + y.w * s;
    y.w = y.w * c - b * s;
  }
  const int64_t o = ((int64_t)qi * kHeads + h) * kDim + d;
  if (A.out_f32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(A.out) + o) = y;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(y.x, y.y), b = __floats2bfloat162_rn(y.z, y.w);
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(A.out) + o) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  }
  if (A.lse != nullptr && d == 0)
    A.lse[(int64_t)qi * kHeads + h] = L > 0.f || L != L ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

// The workspace: two partials per CTA, their maxima and denominators, and the joins.
size_t paged_attn_workspace_bytes() {
  const size_t g = (size_t)device_sm_count(current_device());
  return 2 * g * (kHeads * kDim + 2 * kHeads) * sizeof(float) + (g * sizeof(int4) + 255) / 256 * 256;
}

cudaError_t launch_paged_attn(PagedArgs A, double rope_base, void *ws, cudaStream_t st) {
  const int dev = current_device();
  static std::atomic<int> attr_done[kMaxDevices];
  cudaError_t e = once_per_device(attr_done, dev, [&] {
    return cudaFuncSetAttribute(paged_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPgSmAlloc);
  });
  if (e != cudaSuccess) return e;
  const int64_t sms = device_sm_count(dev);
  rope_turns(rope_base, A.turn);
  magic_of((unsigned)A.page, A.page_mul, A.page_shift);
  A.part = static_cast<float *>(ws);
  A.part_ml = A.part + 2 * (size_t)sms * kHeads * kDim;
  A.joins = reinterpret_cast<int4 *>(A.part_ml + 2 * (size_t)sms * 2 * kHeads);
  // no more CTAs than there can be chunks
  const int64_t longest = A.sel != nullptr ? A.sel_stride : A.table_stride * A.page;
  const int64_t chunks = (int64_t)A.n_q * ((longest + kPgChunk - 1) / kPgChunk + (A.swa_cap > 0 ? 1 : 0));
  const unsigned grid = (unsigned)(chunks < sms ? (chunks < 1 ? 1 : chunks) : sms);
  magic_of(grid, A.grid_mul, A.grid_shift);
  e = launch_pdl(paged_attn_kernel, dim3(grid), dim3(kPgThreads), (size_t)kPgSmAlloc, st, 1u, A);
  if (e != cudaSuccess || grid == 1) return e;
  // a query is cut at a border between two CTAs' runs
  const unsigned cut = (unsigned)A.n_q < grid ? (unsigned)A.n_q : grid;
  if (cut * kHeads <= sms) return launch_pdl(paged_join_kernel<4>, dim3(kHeads, cut), dim3(512), 0, st, 1u, A, (int)grid);
  return launch_pdl(paged_join_kernel<1>, dim3(kHeads, cut), dim3(128), 0, st, 1u, A, (int)grid);
}

}  // namespace csa2
