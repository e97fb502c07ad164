// Eviction from paged caches by accumulated attention weight (csa2_evict), and giving pages
// behind a new length back (csa2_page_trim).
//
// Of a sequence's n entries the last min(recent, k) stay, and of the others the heaviest, k in
// all; they move together, in order, to places 0 .. k - 1.  Two launches:
//
// evict_select_kernel: a cluster per sequence finds the smallest weight that stays, as an order key,
// by histograms of 11, 11 and 10 of its bits, one pass over the keys each (they stay in shared memory, up to 49,152 of a CTA's
// part of the row; those behind in the workspace, 8 x 1M 490 -> 475 us against reading the weights again).  Each warp has a
// contiguous part of the row, so that one count of every part gives every kept entry its rank, and writes which entry each
// new place comes from.
//
// evict_move_kernel: tiles of kMvTile new places, read whole and then written.  In place, a tile's
// places may hold entries that are still to be moved, but only those of its own and of earlier tiles
// (an entry never moves behind its place, so ranks are not above places): tiles are handed out in order, each
// raises a flag when it has read, and before it writes waits for the at most two tiles that its places'
// entries belong to.  A tile that is waited for has been handed out, and reads without waiting for any.  One whose wait runs out
// writes nothing.
// The places behind the kept entries are tiles too, behind a sequence's others: their weights are cleared in the same way.
//
// What bounds it: 288 B read and written for each entry that stays (HBM; a record is in 5 granules of 64 B, so 1.1 times its
// bytes are read), and for the selection the instructions of its five passes.  8 x 1,048,576 entries cut to half: 464 us, 80 of
// them the selection (in place 520); 33 x 40,001 to 9,999: 49 (60); 1 x 4,096: 12 (13), a chain of latencies and cold code.
#include <limits.h>

#include <algorithm>

#include "common.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace csa2 {

constexpr int kEvThreads = 1024, kEvWarps = kEvThreads / 32, kEvBits = 11, kEvBins = 1 << kEvBits;
constexpr int kEvMaxCtas = 16, kEvWhole = 4;
constexpr int kEvKeyTiles = 12;                     // tiles of a warp's part whose keys fit shared memory (192 KB)
constexpr int kEvRowKeys = kEvKeyTiles * kEvWarps * 128;             // entries of a row that one CTA holds
constexpr int kMvTile = 128, kMvThreads = 288, kMvUnits = 8;     // a record is 18 units of 16 B
constexpr int kMvClear = 16;                        // tiles of places that are cleared at a time
static_assert(kMvThreads / 18 * kMvUnits == kMvTile, "a tile's units");

// ------------------------------------------------------------------ workspace
// per sequence: {n, k, entries of the row it reads, -}; the ticket; then from, before, flags
struct EvictWs {
  int4 *meta;
  uint32_t *ticket;
  int32_t *from;
  int64_t from_stride;
  int32_t *before;            // kept entries ahead of every kMvTile-th place
  uint32_t *flag;             // of each tile: read
  int64_t tile_stride;
  uint32_t *keys;             // of entries that shared memory does not hold, by place (rows that may have some)
};
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
size_t evict_workspace_bytes(int n_seq, int64_t row) {
  const size_t tiles = (size_t)(row / kMvTile + 2);
  const size_t keys = row > kEvRowKeys ? (size_t)n_seq * tiles * kMvTile * 4 : 0;
  return 256 + up256((size_t)n_seq * sizeof(int4)) + up256((size_t)n_seq * (size_t)row * 4) + 2 * up256((size_t)n_seq * tiles * 4) + keys;
}
static EvictWs evict_ws(void *ws, int n_seq, int64_t row) {
  char *p = static_cast<char *>(ws);
  EvictWs W;
  W.ticket = reinterpret_cast<uint32_t *>(p);
  p += 256;
  W.meta = reinterpret_cast<int4 *>(p);
  p += up256((size_t)n_seq * sizeof(int4));
  W.from = reinterpret_cast<int32_t *>(p);
  W.from_stride = row;
  p += up256((size_t)n_seq * (size_t)row * 4);
  W.tile_stride = row / kMvTile + 2;
  W.before = reinterpret_cast<int32_t *>(p);
  p += up256((size_t)n_seq * (size_t)W.tile_stride * 4);
  W.flag = reinterpret_cast<uint32_t *>(p);
  p += up256((size_t)n_seq * (size_t)W.tile_stride * 4);
  W.keys = row > kEvRowKeys ? reinterpret_cast<uint32_t *>(p) : nullptr;
  return W;
}

// ------------------------------------------------------------------ select
__device__ __forceinline__ void ev_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t ev_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Two words at the place of p (this CTA's shared memory) in CTA `rank` of the cluster, read and written.
__device__ __forceinline__ uint2 ev_get2(const uint32_t *p, uint32_t rank) {
  uint32_t a;
  uint2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void ev_put2(const uint32_t *p, uint32_t rank, uint32_t x, uint32_t y) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

struct __align__(16) EvictShared {
  uint32_t hist[2][kEvBins];                         // of the phases by turns
  uint32_t slice[kEvMaxCtas][2], found[2], count[kEvMaxCtas][2];       // by CTA of the cluster
  uint32_t above[kEvWarps], gt[kEvWarps], eq[kEvWarps];
  int32_t stage[kEvWarps][kMvTile];
};

// Order key of entry j's weight, larger is heavier (NaN: 1, below everything).  The last entries, which stay in any case,
// have the largest key of all and those behind the row 0, so that no pass over the keys asks where an entry stands.
constexpr uint32_t kEvLeast = 1u;
struct EvictRow {
  const float *weight;
  const int32_t *table;
  int page, n_pages;
  uint64_t mul;
  int shift;
  int *status;
  __device__ __forceinline__ int col(int j) const { return (int)(((uint64_t)(unsigned)j * mul) >> shift); }
  __device__ __forceinline__ int64_t slot(int j, int c) const {
    const int id = __ldg(table + c);
    return id >= 0 && id < n_pages ? (int64_t)id * page + (j - c * page) : -1;
  }
  __device__ __forceinline__ uint32_t key(float w) const { return w == w ? order_key(w) : kEvLeast; }
  // keys of two tiles from `tile` on, four entries from j on of each for this lane: those below n, of which those from m on stay
  __device__ __forceinline__ void keys(int tile, int lane, int m, int n, uint32_t (&x)[2][4]) const {
    const int j0 = tile * kMvTile + lane * 4;
    bool out = false;
    if ((page & 3) == 0) {                           // (one page holds the lane's four, on a 16-byte boundary)
      int64_t s[2];
      float4 w[2];
#pragma unroll
      for (int u = 0; u < 2; u++) s[u] = j0 + u * kMvTile < n ? slot(j0 + u * kMvTile, col(j0 + u * kMvTile)) : -1;
#pragma unroll
      for (int u = 0; u < 2; u++) {
        out |= s[u] < 0 && j0 + u * kMvTile < n;
        w[u] = s[u] >= 0 ? __ldg(reinterpret_cast<const float4 *>(weight + s[u])) : make_float4(NAN, NAN, NAN, NAN);
      }
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const int left = n - (j0 + u * kMvTile);
        x[u][0] = left > 0 ? key(w[u].x) : 0u;
        x[u][1] = left > 1 ? key(w[u].y) : 0u;
        x[u][2] = left > 2 ? key(w[u].z) : 0u;
        x[u][3] = left > 3 ? key(w[u].w) : 0u;
      }
    } else {
#pragma unroll
      for (int u = 0; u < 2; u++) {
        int64_t s[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int j = j0 + u * kMvTile + i;
          s[i] = j < n ? slot(j, col(j)) : -1;
          out |= s[i] < 0 && j < n;
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float w = s[i] >= 0 ? __ldg(weight + s[i]) : NAN;
          x[u][i] = j0 + u * kMvTile + i < n ? key(w) : 0u;
        }
      }
    }
    if ((tile + 2) * kMvTile > m) {
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int j = j0 + u * kMvTile + i;
          if (j >= m && j < n) x[u][i] = 0xFFFFFFFFu;
        }
    }
    if (out) record_error(status, CSA2_ERR_BOUNDS);
  }
};

__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const __grid_constant__ EvictArgs A, EvictWs W, int cache_tiles) {
  extern __shared__ __align__(16) uint32_t ev_keys[];          // the CTA's keys, if they fit
  __shared__ EvictShared S;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, ctas = gridDim.x, b = blockIdx.y;
  const uint32_t rank = ev_rank();
  griddep_wait();
  griddep_launch();
  const int64_t row = A.table_stride * A.page, dst_row = A.dst_stride * A.page;
  int n = __ldg(A.seq_len + b), k = __ldg(A.keep + b);
  const bool bad = n < 0 || k < 0 || n > row || min(n, k) > dst_row || (A.from != nullptr && min(n, k) > A.from_stride);
  // (a sequence that is out of range keeps its length and moves nothing: from here on it has no entries)
  const int stays = !bad ? min(n, k) : A.in_place ? n : 0;
  if (bad) n = k = 0;
  k = min(n, k);
  if (t == 0 && rank == 0) {
    if (bad) record_error(A.status, CSA2_ERR_BOUNDS);
    W.meta[b] = make_int4(n, k, stays, 0);
    if (b == 0) *W.ticket = 0u;
  }
  const int last = min(A.recent, k), m = n - last, kk = k - last;        // candidates, those of them that stay
  const int tiles = (n + kMvTile - 1) / kMvTile;
  // contiguous parts of whole tiles: of the CTAs, of their warps
  const int per_cta = (tiles + ctas - 1) / ctas, t0 = min((int)rank * per_cta, tiles), t1 = min(t0 + per_cta, tiles);
  const int per_warp = (t1 - t0 + kEvWarps - 1) / kEvWarps;
  const int w0 = min(t0 + warp * per_warp, t1), w1 = min(w0 + per_warp, t1);
  for (int i = t0 + t; i < t1; i += kEvThreads) W.flag[(int64_t)b * W.tile_stride + i] = 0u;
  if (k == 0) return;                                // (the whole cluster)
  EvictRow R;
  R.weight = A.weight;
  R.table = A.table + (int64_t)b * A.table_stride;
  R.page = A.page;
  R.n_pages = A.n_pages;
  R.mul = A.page_mul;
  R.shift = A.page_shift;
  R.status = A.status;
  // (without a histogram the counts are the first that one CTA writes into another: all have to have begun by then)
  const bool counts_first = ctas > 1 && !(kk > 0 && kk < m);
  if (counts_first) ptx::cluster_begin();
  // Keys in shared memory: of this warp's first kept_tiles tiles, and behind them two tiles at a time of the others.
  uint32_t *mine = ev_keys + (size_t)warp * cache_tiles * kMvTile + lane * 4;
  uint4 *far_keys = reinterpret_cast<uint4 *>(W.keys + (int64_t)b * W.tile_stride * kMvTile) + lane;
  const int kept_tiles = per_warp <= cache_tiles ? per_warp : cache_tiles - 2;
  auto meet = [&]() {                                // all threads of the cluster
    if (ctas > 1) ev_cluster_sync();
    else __syncthreads();
  };
  // stay: keys above T, and the first `ties` of those at T (all entries: those above 0; no candidate: those of the largest key)
  uint32_t T = kk == m ? 0u : 0xFFFFFFFEu, ties = 0u;
  uint32_t gt = 0u, eq = 0u;                         // entries that stay for sure, that tie: of the warp's part; then that stay, that tie ahead
  int low = 32;                                      // bits of T that are not known yet
  uint32_t known = 0u, top = 0u, need = (uint32_t)k;  // T's known bits, at the low end and in their places
  // bins 2 t and 2 t + 1 of this CTA's slice of a histogram
  // (of a few CTAs each sums all of the histograms: no exchange of its sums, one barrier of the cluster instead of three; 33 rows of
  // four CTAs each 52 -> 51 us, but eight rows of twelve 471 -> 476)
  const bool whole = ctas <= kEvWhole;
  const int pairs = whole ? kEvBins / 2 : (kEvBins / 2 + ctas - 1) / ctas;
  const int bin = 2 * ((whole ? 0 : (int)rank * pairs) + t), warps = (pairs + 31) / 32;
  const bool has_bins = t < pairs && bin < kEvBins;
  int32_t *from = W.from + (int64_t)b * W.from_stride, *before = W.before + (int64_t)b * W.tile_stride;
  bool first = true;
  // 0 .. 2: a histogram of the next bits; 3: counts; 4: the places.  (One loop over the tiles for all of them: in a short row
  // each instruction runs once, and fetching them is most of the time.)
#pragma unroll 1
  for (int phase = kk > 0 && kk < m ? 0 : 3; phase < 5; phase++) {
    const int w = min(kEvBits, low);
    uint32_t *hist = S.hist[phase & 1];
    if (phase < 3) {
      for (int i = t; i < kEvBins; i += kEvThreads) hist[i] = 0u;
      __syncthreads();
    }
#pragma unroll 1
    for (int tile0 = w0; tile0 < w1; tile0 += 2) {
      const bool kept = tile0 - w0 < kept_tiles;
      uint32_t *at = mine + (kept ? tile0 - w0 : kept_tiles) * kMvTile;
      uint4 *far = far_keys + (int64_t)tile0 * (kMvTile / 4);
      if (first) {
        uint32_t x[2][4];
        R.keys(tile0, lane, m, min(n, w1 * kMvTile), x);
#pragma unroll
        for (int u = 0; u < 2; u++)
          if (tile0 + u < w1) {
            const uint4 y = make_uint4(x[u][0], x[u][1], x[u][2], x[u][3]);
            *reinterpret_cast<uint4 *>(at + u * kMvTile) = y;
            if (!kept) __stcg(far + u * (kMvTile / 4), y);
          }
      } else if (!kept) {                            // (what this lane has written)
        uint4 y[2];
#pragma unroll
        for (int u = 0; u < 2; u++) y[u] = tile0 + u < w1 ? __ldcg(far + u * (kMvTile / 4)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < 2; u++)
          if (tile0 + u < w1) *reinterpret_cast<uint4 *>(at + u * kMvTile) = y[u];
      }
#pragma unroll 1
      for (int tile = tile0; tile < min(tile0 + 2, w1); tile++, at += kMvTile) {
        const uint4 v = *reinterpret_cast<const uint4 *>(at);          // (the lane's own)
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
        if (phase < 3) {
          // the next w bits of the keys that begin as T does; of others the result is above them
          uint32_t d[4];
#pragma unroll
          for (int i = 0; i < 4; i++) d[i] = (x[i] ^ top) >> (low - w);
          // (many equal weights: one lane counts for all)
          const uint32_t one = __shfl_sync(0xFFFFFFFFu, d[0], 0);
          if (__all_sync(0xFFFFFFFFu, d[0] == one && d[1] == one && d[2] == one && d[3] == one)) {
            if (lane == 0 && one >> w == 0u) atomicAdd(&hist[one], (uint32_t)kMvTile);
          } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
              if (d[i] >> w == 0u) atomicAdd(&hist[d[i]], 1u);
          }
          continue;
        }
        uint32_t g = 0u, e = 0u;                     // bits of the lane's entries that stay for sure, that tie
#pragma unroll
        for (int i = 0; i < 4; i++) {
          if (x[i] > T) g |= 1u << i;
          if (x[i] == T) e |= 1u << i;
        }
        if (phase == 3) {
          gt += (uint32_t)__popc(g);
          eq += (uint32_t)__popc(e);
          continue;
        }
        auto scan = [&](uint32_t v) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t z = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += z;
          }
          return v;
        };
        if (__any_sync(0xFFFFFFFFu, e != 0u) && eq < ties) {           // (eq: the whole warp's)
          const uint32_t sum = scan((uint32_t)__popc(e));
          uint32_t c = eq + sum - (uint32_t)__popc(e);
#pragma unroll
          for (int i = 0; i < 4; i++)
            if ((e >> i) & 1u) {
              if (c < ties) g |= 1u << i;
              c++;
            }
          eq += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        const uint32_t sum = scan((uint32_t)__popc(g)), count = __shfl_sync(0xFFFFFFFFu, sum, 31);
        // (through shared memory: the places of a tile's kept entries are neighbours)
        int32_t *to = &S.stage[warp][sum - (uint32_t)__popc(g)];
#pragma unroll
        for (int i = 0; i < 4; i++)
          if ((g >> i) & 1u) *to++ = tile * kMvTile + lane * 4 + i;
        __syncwarp();
        for (uint32_t i = lane; i < count; i += 32) from[gt + i] = S.stage[warp][i];
        if (lane == 0) before[tile] = (int32_t)gt;
        gt += count;
        __syncwarp();
      }
    }
    first = false;
    if (phase < 3) {
      // the digit at which the count from the top passes `need`: each CTA sums a slice of the histograms
      meet();
      uint32_t h0 = 0u, h1 = 0u, above = 0u;
      if (has_bins) {
        if (ctas == 1) {
          h0 = hist[bin];
          h1 = hist[bin + 1];
        } else {
#pragma unroll 1
          for (int c = 0; c < ctas; c += 8) {        // (eight loads in flight)
            uint2 y[8];
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] = c + i < ctas ? ev_get2(&hist[bin], (uint32_t)(c + i)) : make_uint2(0u, 0u);
#pragma unroll
            for (int i = 0; i < 8; i++) {
              h0 += y[i].x;
              h1 += y[i].y;
            }
          }
        }
      }
      above = h0 + h1;                               // of this thread's bins and those above them
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_down_sync(0xFFFFFFFFu, above, o);
        if (lane + o < 32) above += y;
      }
      if (lane == 0) S.above[warp] = above;
      __syncthreads();
      const uint32_t part = lane < warps ? S.above[lane] : 0u;
      above += __reduce_add_sync(0xFFFFFFFFu, lane > warp ? part : 0u);
      if (!whole) {
        const uint32_t sum = __reduce_add_sync(0xFFFFFFFFu, part);
        if (t < ctas) ev_put2(S.slice[rank], (uint32_t)t, sum, 0u);
        __syncwarp();
        ev_cluster_sync();
        const uint32_t other = lane > (int)rank && lane < ctas ? S.slice[lane & (kEvMaxCtas - 1)][0] : 0u;
        above += __reduce_add_sync(0xFFFFFFFFu, other);
      }
      if (has_bins) {
        const uint32_t top1 = above - h0 - h1, top0 = above - h0;        // above bin + 1, above bin
        const bool hit1 = top1 < need && need <= top1 + h1, hit0 = top0 < need && need <= above;
        if (hit0 || hit1) {                          // (one thread of the cluster, or of each CTA)
          const uint32_t digit = (uint32_t)bin + (hit1 ? 1u : 0u), rest = need - (hit1 ? top1 : top0);
          if (whole) {
            S.found[0] = digit;
            S.found[1] = rest;
          } else {
            for (int c = 0; c < ctas; c++) ev_put2(S.found, (uint32_t)c, digit, rest);
          }
        }
      }
      __syncwarp();
      if (whole) __syncthreads();
      else ev_cluster_sync();
      known = known << w | S.found[0];
      need = S.found[1];
      low -= w;
      top = known << low;
      if (low == 0) {
        T = known;
        ties = need;
      }
    } else if (phase == 3) {
      gt = __reduce_add_sync(0xFFFFFFFFu, gt);
      eq = __reduce_add_sync(0xFFFFFFFFu, eq);
      if (lane == 0) {
        S.gt[warp] = gt;
        S.eq[warp] = eq;
      }
      __syncthreads();
      if (counts_first) ptx::cluster_begun();
      gt = lane < warp ? S.gt[lane] : 0u;
      eq = lane < warp ? S.eq[lane] : 0u;
      if (ctas > 1) {
        if (warp == 0) {
          const uint32_t a = __reduce_add_sync(0xFFFFFFFFu, S.gt[lane]), c = __reduce_add_sync(0xFFFFFFFFu, S.eq[lane]);
          if (lane < ctas) ev_put2(S.count[rank], (uint32_t)lane, a, c);
          __syncwarp();
        }
        ev_cluster_sync();                           // (nothing of another CTA is read or written from here on)
        gt += lane < (int)rank ? S.count[lane & (kEvMaxCtas - 1)][0] : 0u;
        eq += lane < (int)rank ? S.count[lane & (kEvMaxCtas - 1)][1] : 0u;
      }
      gt = __reduce_add_sync(0xFFFFFFFFu, gt);
      eq = __reduce_add_sync(0xFFFFFFFFu, eq);
      gt += min(eq, ties);                           // the rank of the warp's first
    }
  }
  if (w1 == tiles && w0 < w1 && lane == 0) before[tiles] = k;
}

// ------------------------------------------------------------------ move
// Loads that stay where they stand between barriers (what they read is written by other CTAs of the
// same launch once this one has said that it has read it).  Records come by 64 B of L2's lines of 128: neighbours
// are often not kept (8 x 1M cut to half 560 -> 544 us).
__device__ __forceinline__ uint4 mv_load16(const uint8_t *p) {
  uint4 v;
  asm volatile("ld.relaxed.gpu.global.L1::no_allocate.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ float mv_load4(const float *p) {
  float v;
  asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

__global__ void __launch_bounds__(kMvThreads, 4) evict_move_kernel(const __grid_constant__ EvictArgs A, EvictWs W) {
  __shared__ int64_t src_sh[kMvTile], dst_sh[kMvTile];
  __shared__ uint32_t next_sh;
  const int t = threadIdx.x, lane = t & 31;
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0)
    for (int b = t; b < A.n_seq; b += kMvThreads) A.new_len[b] = W.meta[b].z;
  // tiles of all sequences are numbered in order; the cursor moves on with the tile number
  int b0 = 0;                                        // 32 sequences from b0 on have tiles from base on
  int64_t base = 0;
  uint32_t tile = blockIdx.x;
  if (A.in_place && t == 0) next_sh = atomicAdd(W.ticket, 1u);
  for (;; tile += gridDim.x) {
    __syncthreads();                                 // (the last tile's slots are read)
    if (A.in_place) {
      tile = next_sh;
      __syncthreads();
      // the next ticket is on its way during this tile (33 x 40,001 to 9,999: 105 us with one at a time, 88 so).  A CTA's tickets
      // ascend and are done in turn, so the least tile that is not done is always one that some CTA is at, and waits for none.
      if (t == 0) next_sh = atomicAdd(W.ticket, 1u);
    }
    // (every warp finds the sequence for itself)
    int b = -1, i = 0, k = 0, n = 0;
    // tiles of k kept entries, and kMvClear at a time of the places behind them
    auto moved = [](int k) { return (k + kMvTile - 1) / kMvTile; };
    auto cleared = [&](int n, int k) { return A.in_place && k < n ? ((n - 1) / kMvTile - k / kMvTile + kMvClear) / kMvClear : 0; };
    while (b0 < A.n_seq) {
      const int4 M = b0 + lane < A.n_seq ? W.meta[b0 + lane] : make_int4(0, 0, 0, 0);
      const int own = moved(M.y) + cleared(M.x, M.y);
      int64_t inc = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += y;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, (int64_t)tile < base + inc);
      if (past != 0u) {
        const int from = __ffs((int)past) - 1;
        b = b0 + from;
        i = (int)((int64_t)tile - (base + __shfl_sync(0xFFFFFFFFu, inc - own, from)));
        n = __shfl_sync(0xFFFFFFFFu, M.x, from);
        k = __shfl_sync(0xFFFFFFFFu, M.y, from);
        break;
      }
      base += __shfl_sync(0xFFFFFFFFu, inc, 31);
      b0 += 32;
    }
    if (b < 0) return;                               // (no tile is left: the whole CTA)
    const int32_t *table = A.table + (int64_t)b * A.table_stride, *dst_table = A.dst_table + (int64_t)b * A.dst_stride;
    uint32_t *flag = W.flag + (int64_t)b * W.tile_stride;
    const int32_t *before = W.before + (int64_t)b * W.tile_stride;
    // waits, the x-th tile for x = t, t + step, .., until the entries at the places of ranks [lo, hi) are read, and none is of
    // a tile behind this one (`self`); false: a wait ran out
    auto wait_read = [&](int lo, int hi, int self, int from, int step) {
      for (int x = lo / kMvTile + from; lo < hi && x <= (hi - 1) / kMvTile; x += step)
        if (x != self && !ptx::poll_at_least_u32(flag + x, 1u)) {
          record_error(A.status, CSA2_ERR_TIMEOUT);
          return false;
        }
      return true;
    };
    if (i >= moved(k)) {                             // places that nothing is at any more
      const int p0 = k / kMvTile + (i - moved(k)) * kMvClear, p1 = min(p0 + kMvClear, (n - 1) / kMvTile + 1);
      if (k > 0) {
        const bool read = wait_read(__ldcg(before + p0), __ldcg(before + p1), -1, t, kMvThreads);
        if (!__syncthreads_and(read)) return;        // (as below)
      }
      for (int j = max(k, p0 * kMvTile) + t; j < min(n, p1 * kMvTile); j += kMvThreads) {
        const int c = (int)(((uint64_t)(unsigned)j * A.page_mul) >> A.page_shift), id = __ldg(table + c);
        if (id >= 0 && id < A.n_pages) A.dst_weight[(int64_t)id * A.page + (j - c * A.page)] = 0.f;
      }
      continue;
    }
    const int r0 = i * kMvTile, rows = min(kMvTile, k - r0);
    bool there = true;                               // the entry is where it goes
    if (t < rows) {
      const int j = __ldg(W.from + (int64_t)b * W.from_stride + r0 + t), r = r0 + t;
      const int cs = (int)(((uint64_t)(unsigned)j * A.page_mul) >> A.page_shift), cd = (int)(((uint64_t)(unsigned)r * A.page_mul) >> A.page_shift);
      const int ps = __ldg(table + cs), pd = __ldg(dst_table + cd);
      there = A.in_place && j == r;
      const bool ok = ps >= 0 && ps < A.n_pages && pd >= 0 && pd < A.n_dst;
      if (!ok) record_error(A.status, CSA2_ERR_BOUNDS);
      src_sh[t] = ok ? (int64_t)ps * A.page + (j - cs * A.page) : -1;
      dst_sh[t] = ok ? (int64_t)pd * A.page + (r - cd * A.page) : -1;
    }
    const bool still = __syncthreads_and(there) != 0;
    if (still) {
      if (A.in_place && t == 0) ptx::st_release_u32(flag + i, 1u);
      continue;
    }
    // kept entries ahead of this tile's places and of the next one's: they are read by the tiles that hold those ranks
    const int lo = A.in_place && t < 2 ? __ldcg(before + i) : 0, hi = A.in_place && t < 2 ? __ldcg(before + i + 1) : 0;
    uint4 x[kMvUnits];
    float w = 0.f;
    const int unit = t % 18, sub = t / 18;
#pragma unroll
    for (int u = 0; u < kMvUnits; u++) {
      const int r = u * (kMvThreads / 18) + sub;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && src_sh[r] >= 0) x[u] = mv_load16(A.pages + src_sh[r] * kKvBytes + unit * 16);
    }
    if (t < rows && src_sh[t] >= 0) w = mv_load4(A.weight + src_sh[t]);
    if (A.in_place) {
      // All of the tile is read once every thread has used what it loaded.  The barriers and one thread's release and acquire
      // order these reads ahead of the other CTAs' stores; a fence of every thread would wait for its stores of the tile before
      // as well (8 x 1M: 549 us, 530 so).
      uint32_t used = __float_as_uint(w);
#pragma unroll
      for (int u = 0; u < kMvUnits; u++) used |= x[u].x | x[u].w;
      __syncthreads_or((int)used);
      if (t == 0) ptx::st_release_u32(flag + i, 1u);
      // Nothing is written where something may not have been read.  The CTA ends, and the waits for its next tile run out too, so
      // that all end in bounded time.
      const bool read = t >= 2 || wait_read(lo, hi, i, t, 2);
      if (!__syncthreads_and(read)) return;
    }
#pragma unroll
    for (int u = 0; u < kMvUnits; u++) {
      const int r = u * (kMvThreads / 18) + sub;
      if (r < rows && dst_sh[r] >= 0) *reinterpret_cast<uint4 *>(A.dst_pages + dst_sh[r] * kKvBytes + unit * 16) = x[u];
    }
    if (t < rows && dst_sh[t] >= 0) A.dst_weight[dst_sh[t]] = w;
  }
}

// j / n by a multiplication, exact for j below 2^31
static void evict_magic(unsigned n, uint64_t &mul, int &shift) {
  int s = 0;
  while (((int64_t)1 << s) < (int64_t)n) s++;
  shift = 31 + s;
  mul = (uint64_t)((((unsigned __int128)1 << shift) + n - 1) / n);
}

cudaError_t launch_evict(EvictArgs A, void *ws, cudaStream_t st) {
  const int dev = current_device();
  constexpr size_t kTileBytes = (size_t)kEvWarps * kMvTile * 4;
  static std::atomic<int> attr_done[kMaxDevices], fit[kMaxDevices][kEvMaxCtas + 1];     // clusters that run at a time (0: unknown)
  cudaError_t e = once_per_device(attr_done, dev, [&] {
    cudaError_t f = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kEvKeyTiles * kTileBytes));
    if (f == cudaSuccess) f = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    // The move's loads in flight stand in L1 (147 KB an SM), which the selection's CTAs leave small: 8 % of it for shared memory
    // hold four CTAs' 3 KB (8 x 1M cut to half, the move: 388 us, 445 as the selection leaves it, 505 with all for shared memory)
    if (f == cudaSuccess) f = cudaFuncSetAttribute(evict_move_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 8);
    for (int c = 1; f == cudaSuccess && dev >= 0 && dev < kMaxDevices && c <= kEvMaxCtas; c++) {
      cudaLaunchAttribute a;
      a.id = cudaLaunchAttributeClusterDimension;
      a.val.clusterDim.x = (unsigned)c;
      a.val.clusterDim.y = a.val.clusterDim.z = 1;
      cudaLaunchConfig_t config = {};
      config.gridDim = dim3((unsigned)c, 64);
      config.blockDim = dim3(kEvThreads);
      config.dynamicSmemBytes = kEvKeyTiles * kTileBytes;
      config.attrs = &a;
      config.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, evict_select_kernel, &config) == cudaSuccess) fit[dev][c].store(n, std::memory_order_relaxed);
      else cudaGetLastError();
    }
    return f;
  });
  if (e != cudaSuccess) return e;
  const int64_t sms = device_sm_count(dev), row = A.table_stride * A.page;
  evict_magic((unsigned)A.page, A.page_mul, A.page_shift);
  EvictWs W = evict_ws(ws, A.n_seq, row);
  if (A.from != nullptr) {
    W.from = A.from;
    W.from_stride = A.from_stride;
  }
  // CTAs of a row: up to one for each 8,192 entries, as many as give the least time when a CTA takes that of 6,500 entries beside
  // its own and only so many clusters run at a time (an SM holds one CTA and a cluster has to fit one of the chip's groups of SMs:
  // of 16 CTAs seven fit, of 12 eight; 8 x 1M entries: 139 us of selection with 16, 100 with 12)
  int ctas = 1;
  int64_t least = LLONG_MAX;
  for (int c = 1; c <= kEvMaxCtas && (c == 1 || (int64_t)(c - 1) * 8192 < row); c++) {
    const int fits = dev >= 0 && dev < kMaxDevices ? fit[dev][c].load(std::memory_order_relaxed) : 0;
    const int64_t at_once = fits > 0 ? fits : std::max<int64_t>(1, sms / c);
    const int64_t cost = (A.n_seq + at_once - 1) / at_once * (6500 + row / c);
    if (cost < least) {
      least = cost;
      ctas = c;
    }
  }
  const int64_t share = ((row + kMvTile - 1) / kMvTile + ctas - 1) / ctas, warp_share = (share + kEvWarps - 1) / kEvWarps;
  const int cache = (int)(warp_share < kEvKeyTiles ? warp_share : kEvKeyTiles);
  e = launch_pdl(evict_select_kernel, dim3((unsigned)ctas, (unsigned)A.n_seq), dim3(kEvThreads), cache * kTileBytes, st, (unsigned)ctas, A, W, cache);
  if (e != cudaSuccess) return e;
  // Into other pages: no more CTAs than there can be tiles, and many more than run at a time, as SMs differ in speed (8 x 1M
  // entries cut to half: 720 us with four CTAs an SM that take equal shares).  In place: as many as run, which take tickets.
  const int64_t dst_row = A.dst_stride * A.page, most = dst_row < row ? dst_row : row;
  const int64_t tiles = A.n_seq * ((most + kMvTile - 1) / kMvTile + (A.in_place ? 1 : 0)), waves = A.in_place ? 4 : 64;
  const int64_t grid = tiles < waves * sms ? tiles : waves * sms;
  return launch_pdl(evict_move_kernel, dim3((unsigned)grid), dim3(kMvThreads), 0, st, 1u, A, W);
}

// ------------------------------------------------------------------ trim
// One CTA: pages behind the new lengths, counted by a prefix sum over the sequences, found by a
// binary search each.  (One, because the list's head is read by all and written at the end.)
__global__ void __launch_bounds__(kPlanThreads) page_trim_kernel(const __grid_constant__ TrimArgs A) {
  extern __shared__ int trim_sh[];                   // pages given back ahead of each sequence, [n_seq + 1]
  __shared__ int wt[kPlanThreads / 32];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  griddep_wait();
  griddep_launch();
  const int per = (A.n_seq + kPlanThreads - 1) / kPlanThreads, b0 = min(t * per, A.n_seq), b1 = min(b0 + per, A.n_seq);
  auto columns = [&](int b, int &c0) -> int {        // -1: out of range
    const int len = __ldg(A.len + b), to = __ldg(A.new_len + b);
    if (len < 0 || to < 0 || to > len || len > A.row_cap) return -1;
    c0 = (int)(((unsigned)to + (unsigned)A.page - 1u) / (unsigned)A.page);
    return (int)(((unsigned)len + (unsigned)A.page - 1u) / (unsigned)A.page) - c0;
  };
  int sum = 0, c0 = 0;
  bool err = false;
  for (int b = b0; b < b1; b++) {
    const int c = columns(b, c0);
    err |= c < 0;
    sum = (int)min((unsigned)sum + (unsigned)max(c, 0), (unsigned)INT_MAX);
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc = (int)min((unsigned)inc + (unsigned)y, (unsigned)INT_MAX);
  }
  if (lane == 31) wt[warp] = inc;
  int ahead = __shfl_up_sync(0xFFFFFFFFu, inc, 1);
  if (lane == 0) ahead = 0;
  __syncthreads();
  for (int w = 0; w < warp; w++) ahead = (int)min((unsigned)ahead + (unsigned)wt[w], (unsigned)INT_MAX);
  for (int b = b0; b < b1; b++) {
    trim_sh[b] = ahead;
    ahead = (int)min((unsigned)ahead + (unsigned)max(columns(b, c0), 0), (unsigned)INT_MAX);
  }
  if (t == kPlanThreads - 1) trim_sh[A.n_seq] = ahead;
  const int head = *A.free_head;
  __syncthreads();
  const int total = trim_sh[A.n_seq];
  // more pages than were taken from the list, or a head outside it: nothing is given back
  const bool fits = head >= 0 && head <= A.n_free && total <= head;
  err |= !fits;
  if (fits) {
    for (int i = t; i < total; i += kPlanThreads) {
      int lo = 0, hi = A.n_seq;                      // the last sequence with trim_sh <= i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (trim_sh[mid] <= i) lo = mid;
        else hi = mid;
      }
      columns(lo, c0);
      int32_t *at = A.table + (int64_t)lo * A.table_stride + c0 + (i - trim_sh[lo]);
      const int id = *at;
      err |= id < 0 || id >= A.n_pages;
      A.free_pages[head - total + i] = id;
      *at = -1;
    }
    if (t == 0) *A.free_head = head - total;
  }
  if (err) record_error(A.status, CSA2_ERR_BOUNDS);
}

cudaError_t launch_page_trim(const TrimArgs &A, cudaStream_t st) {
  const int dev = current_device();
  static std::atomic<int> attr_done[kMaxDevices];
  const cudaError_t e = once_per_device(attr_done, dev, [&] {
    return cudaFuncSetAttribute(page_trim_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kPlanMaxSeq + 1) * (int)sizeof(int));
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(page_trim_kernel, dim3(1), dim3(kPlanThreads), (size_t)(A.n_seq + 1) * sizeof(int), st, 1u, A);
}

}  // namespace csa2
