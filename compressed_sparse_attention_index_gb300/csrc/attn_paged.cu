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
// Per chunk: the 128 records are dequantised to f16 in shared memory (an
// E2M1 x E4M3 product has <= 6 significant bits in [2^-10, 2688]: exact), then
//   S^T[entry][head] = K . Q^T        tcgen05 kind::f16, M = 128, N = 64, K = 512
//   P[entry][head] = 2^(S - m + 7)    rounded to f16 (11 bits)
//   O^T[dim][head] += K^T . P         M = 128 dims (4 blocks), N = 64, K = 128
// with K^T read from the same tile MN-major.  m is a head's reference in log2
// units: the maximum of the first chunk, raised only when a later logit exceeds
// it by more than 8, so numerators stay within 2^15 and most chunks need no
// maximum, no exchange between warps and no rescaling of O.  The factor 2^7
// keeps the tail of a long row (2^-21 of the largest weight) in f16's normal
// range.  The denominator sums the unrounded fp32 numerators.
//
// Window records (E4M3 x 2^e) are exact in f16 where -15 <= e <= 7; otherwise
// the window is scaled by 2^kx, kx = 7 - (the largest e): exact but for values
// below 2^-31 of the window's largest, and undone on its logits and, being the
// first chunk, on O before the next one.  Q goes to f16 under the power of two
// that brings max |q| into [2^14, 2^15), undone on the logits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "attn.cuh"
#include "common.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace csa2 {

constexpr int kPgChunk = 128;
constexpr int kPgSoftWarps = 8, kPgLoadWarps = 16;
constexpr int kPgSoft = kPgSoftWarps * 32, kPgLoad = kPgLoadWarps * 32;
constexpr int kPgThreads = kPgSoft + kPgLoad + 128;
// Registers: 896 threads are launched with 72 each; the softmax groups take what
// the others give up.
constexpr int kPgRegsSoft = 104, kPgRegsLoad = 64, kPgRegsIssue = 40;
static_assert(kPgSoft * kPgRegsSoft + kPgLoad * kPgRegsLoad + 128 * kPgRegsIssue <= 72 * kPgThreads, "register split");
constexpr int kPgSmK = 0;                          // 128 entries x 512 dims f16: [e/8][dim/64][e%8][128 B]
constexpr int kPgSmQ = kPgSmK + 128 * 1024;        // 64 heads x 512 dims f16, the same order
constexpr int kPgSmP = kPgSmQ + 64 * 1024;         // 128 entries x 64 heads f16: [e/8][e%8][128 B]
constexpr int kPgSmEnd = kPgSmP + 16 * 1024;
constexpr int kPgSmAlloc = kPgSmEnd + 1024;
constexpr uint32_t kPgColS = 0, kPgColO = 64, kPgTmemCols = 512;
constexpr float kPgRaise = 8.f, kPgShift = 7.f;

// Barriers among the softmax warps (1) and among the loading warps (2); every
// warp of a group reaches each of them, whatever its waits returned.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kPgSoft) : "memory"); }
__device__ __forceinline__ void load_sync() { asm volatile("bar.sync 2, %0;" ::"n"(kPgLoad) : "memory"); }
__device__ __forceinline__ bool soft_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "n"(kPgSoft)
      : "memory");
  return r != 0u;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct PagedQuery {
  int seq, n, chunks, win;      // entries (or selection slots), chunks in all, window entries
  bool bad;
};

__device__ __forceinline__ PagedQuery paged_query(const PagedArgs &A, int q) {
  PagedQuery r;
  r.seq = __ldg(A.q_seq + q);
  const int vis = __ldg(A.n_vis + q);
  r.win = __ldg(A.swa_cnt + q);
  const int first = __ldg(A.swa_first + q);
  r.bad = r.seq < 0 || r.seq >= A.n_seq || vis < 0 || (int64_t)vis > A.table_stride * A.page || r.win < 0 ||
          r.win > kSwa || r.win > A.swa_cap || (r.win > 0 && (first < 0 || first >= A.swa_cap));
  r.n = r.bad ? 0 : A.sel != nullptr ? (vis > 0 ? A.sel_stride : 0) : vis;
  if (r.bad) r.win = 0;
  r.chunks = (int)(((unsigned)r.n + kPgChunk - 1) / kPgChunk) + (r.win > 0 ? 1 : 0);
  return r;
}

// CTA g of G has chunks [g T / G, (g + 1) T / G) of T (T below 2^31)
__device__ __forceinline__ int run_start(int g, int T, int G) { return (int)((int64_t)g * T / G); }
__device__ __forceinline__ int run_owner(int c, int T, int G) { return (int)((((int64_t)c + 1) * G - 1) / T); }

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

// The record of row e of an entry chunk, or null (none, or out of range: recorded).
__device__ __forceinline__ const uint8_t *paged_record(const PagedArgs &A, const PagedCursor &C, int e, bool report) {
  const int i = (C.local() - (C.Q.win > 0 ? 1 : 0)) * kPgChunk + e;
  if (i >= C.Q.n) return nullptr;
  int j = i;
  if (A.sel != nullptr) {
    j = __ldg(A.sel + (int64_t)C.qi * A.sel_stride + i);
    if (j < 0) return nullptr;
    if (j >= __ldg(A.n_vis + C.qi)) {
      if (report) record_error(A.status, CSA2_ERR_BOUNDS);
      return nullptr;
    }
  }
  const int col = (int)((unsigned)j / (unsigned)A.page);
  const int id = __ldg(A.table + (int64_t)C.Q.seq * A.table_stride + col);
  if (id < 0 || id >= A.n_pages) {
    if (report) record_error(A.status, CSA2_ERR_BOUNDS);
    return nullptr;
  }
  return A.pages + ((int64_t)id * A.page + (j - col * A.page)) * kKvBytes;
}

// 32 heads' dot products of this lane's entry.
__device__ __forceinline__ void paged_scores(uint32_t ta, float (&r)[32]) {
  uint32_t a[32];
  ptx::tmem_ld_32x32b_x32(ta + kPgColS, a);
  ptx::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; i++) r[i] = __uint_as_float(a[i]);
}

// Roles: warps 0-7 softmax, rescaling and read-out (warp w: TMEM lane quarter
// w % 4, heads 32 (w / 4) ..); warps 8-23 load and dequantise (32 dims of each
// slab of a row per thread) and stage Q; one lane of warp
// 24 issues the MMAs.
// A chunk's tile is four slabs of 128 dims, each with its own barriers: PV's
// block b reads slab b only, so slab b of the next chunk is written, and its
// part of the next QK runs, while the blocks behind b still run.  The records of
// the next chunk are in registers by then.
__global__ void __launch_bounds__(kPgThreads, 1) paged_attn_kernel(const __grid_constant__ PagedArgs A) {
  extern __shared__ __align__(1024) unsigned char pg_smem_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(pg_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t bar_full[4], bar_free[4], bar_s, bar_p, bar_drain;
  __shared__ uint32_t tmem_sh, qmax_sh[kPgLoadWarps];
  __shared__ __align__(16) float m_ref[kHeads], alpha_sh[kHeads];    // m_ref: the reference less kPgShift
  __shared__ float l_sh[4][kHeads], red_sh[4][kHeads];
  __shared__ uint8_t valid_sh[kPgChunk];
  __shared__ int scan_sh[kPgThreads / 32], off_sh;
  __shared__ int start_sh, emin_sh, emax_sh, kx_sh;
  __shared__ float qscale_sh;
  __shared__ int4 info_sh[2];                        // of chunk k: query, place in it, its chunks, its first chunk
  __shared__ volatile int bad_sh;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (t == 0) {
    for (int b = 0; b < 4; b++) {
      ptx::mbar_init(&bar_full[b], kPgLoadWarps);
      ptx::mbar_init(&bar_free[b], 1);
    }
    ptx::mbar_init(&bar_s, 1);
    ptx::mbar_init(&bar_p, kPgSoftWarps);
    ptx::mbar_init(&bar_drain, 1);
    bad_sh = 0;
    start_sh = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0) ptx::tmem_alloc(&tmem_sh, kPgTmemCols);
  griddep_wait();
  griddep_launch();

  // ---------------------------------------------------------- this CTA's run
  // prefix sums of the queries' chunks: thread t has queries [u0, u1)
  const int per = (A.n_q + kPgThreads - 1) / kPgThreads, u0 = min(t * per, A.n_q), u1 = min(u0 + per, A.n_q);
  int mine = 0;
  bool any_bad = false;
  for (int q = u0; q < u1; q++) {
    const PagedQuery r = paged_query(A, q);
    mine += r.chunks;
    any_bad |= r.bad;
  }
  if (any_bad && blockIdx.x == 0) record_error(A.status, CSA2_ERR_BOUNDS);
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) scan_sh[warp] = inc;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < kPgThreads / 32; w++) {
    if (w < warp) before += scan_sh[w];
    total += scan_sh[w];
  }
  before += inc - mine;
  const int G = gridDim.x, T = total;
  const int c_begin = run_start(blockIdx.x, T, G), c_end = run_start(blockIdx.x + 1, T, G);
  if (c_begin < c_end && before <= c_begin && c_begin < before + mine) {
    int o = before, q = u0;
    for (; q < u1; q++) {
      const int n = paged_query(A, q).chunks;
      if (c_begin < o + n) break;
      o += n;
    }
    start_sh = q;
    off_sh = o;
  }
  if (t == 0) A.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);
  // queries with nothing to attend to: zeros
  for (int q = blockIdx.x; q < A.n_q; q += gridDim.x) {
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
  const uint32_t tmem = tmem_sh;
  // A wait that runs out marks the CTA bad; from then on no role waits, so that
  // all of them run out of chunks (and meet their groups' barriers) in bounded time.
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (bad_sh) return;
    for (int i = 0; i < 64; i++)                     // (each try waits a while in hardware; no timer is read)
      if (ptx::mbar_try_wait(bar, parity)) return;
    if (ptx::mbar_wait(bar, parity)) return;
    record_error(A.status, CSA2_ERR_TIMEOUT);
    bad_sh = 1;
  };
  const int n_run = c_end - c_begin;

  if (warp < kPgSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPgRegsSoft));
    // ======================================================== softmax, read-out
    const int quarter = warp & 3, hb = (warp >> 2) * 32, e_row = quarter * 32 + lane;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16);
    float l_acc[32];
    float o_scale = 1.f;                             // what O still has to be multiplied by
    bool acc = false;                                // O holds something of this query
    int lc0 = 0;
    for (int k = 0; k < n_run; k++) {
      wait(&bar_s, k & 1);
      ptx::tc_fence_after();
      const int4 I = info_sh[k & 1];
      const int lc = I.y;
      if (k == 0 || lc == 0) {                       // a query begins
        lc0 = lc;
        acc = false;
        o_scale = 1.f;
#pragma unroll
        for (int i = 0; i < 32; i++) l_acc[i] = 0.f;
        if (t < kHeads) m_ref[t] = -INFINITY;
        soft_sync();
      }
      const float f = A.scale * 1.4426950408889634f * ldexpf(qscale_sh, -kx_sh);
      const int kx = kx_sh;
      const bool ev = valid_sh[e_row] != 0;
      float s[32];
      {
        float r[32];
        paged_scores(tq + hb, r);
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 m = *reinterpret_cast<const float4 *>(&m_ref[hb + i]);
          // (the product rounded first, as the maximum's was: fused, the difference
          // of two huge logits would be off by that rounding)
          s[i] = __fmul_rn(r[i], f) - m.x;
          s[i + 1] = __fmul_rn(r[i + 1], f) - m.y;
          s[i + 2] = __fmul_rn(r[i + 2], f) - m.z;
          s[i + 3] = __fmul_rn(r[i + 3], f) - m.w;
          top = fmaxf(fmaxf(top, fmaxf(s[i], s[i + 1])), fmaxf(s[i + 2], s[i + 3]));
        }
        const bool rescale = acc && o_scale != 1.f;  // a window's 2^-kx, undone before the next chunk
        if (soft_any((ev && top > kPgRaise + kPgShift) || rescale)) {
          // the chunk's maximum of every head: lane L ends with head hb + L
          // (S is read again rather than kept in registers)
          float v[32];
          paged_scores(tq + hb, r);
#pragma unroll
          for (int i = 0; i < 32; i++) v[i] = ev ? __fmul_rn(r[i], f) : -INFINITY;
#pragma unroll
          for (int w = 16; w >= 1; w >>= 1) {
            const bool upper = (lane & w) != 0;
#pragma unroll
            for (int i = 0; i < 16; i++) {
              if (i < w) {
                const float keep = upper ? v[i + w] : v[i], send = upper ? v[i] : v[i + w];
                v[i] = fmaxf(keep, __shfl_xor_sync(0xFFFFFFFFu, send, w));
              }
            }
          }
          red_sh[quarter][hb + lane] = v[0];
          soft_sync();
          if (t < kHeads) {
            const float cm = fmaxf(fmaxf(red_sh[0][t], red_sh[1][t]), fmaxf(red_sh[2][t], red_sh[3][t])) - kPgShift;
            const float mo = m_ref[t];
            float al = 1.f;
            if (cm > mo + kPgRaise) {
              al = mo == -INFINITY ? 0.f : exp2f(mo - cm);
              m_ref[t] = cm;
            }
            alpha_sh[t] = al;
          }
          soft_sync();
          if (acc) {
            // O *= alpha (and the window's factor); PV of the chunk before is complete (S is)
            for (int blk = warp >> 2; blk < 4; blk += 2)
#pragma unroll 1
              for (int hh = 0; hh < 2; hh++) {
                uint32_t o[32];
                const uint32_t ta = tq + kPgColO + blk * kHeads + hh * 32;
                ptx::tmem_ld_32x32b_x32(ta, o);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i++)
                  o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha_sh[hh * 32 + i] * o_scale);
                ptx::tmem_st_32x32b_x32(ta, o);
              }
            ptx::tmem_wait_st();
            o_scale = 1.f;
          }
          paged_scores(tq + hb, r);
#pragma unroll
          for (int i = 0; i < 32; i++) {
            l_acc[i] *= alpha_sh[hb + i];
            s[i] = __fmul_rn(r[i], f) - m_ref[hb + i];
          }
        }
      }
      unsigned char *row = sm + kPgSmP + (e_row >> 3) * 1024;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        uint32_t o[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
          const int i = 8 * j + 2 * u;
          const float p0 = ev ? ex2(s[i]) : 0.f, p1 = ev ? ex2(s[i + 1]) : 0.f;
          l_acc[i] += p0;
          l_acc[i + 1] += p1;
          const __half2 h2 = __floats2half2_rn(p0, p1);
          o[u] = *reinterpret_cast<const uint32_t *>(&h2);
        }
        *reinterpret_cast<uint4 *>(row + sw128(e_row & 7, (hb >> 3) + j)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      ptx::tc_fence_before();
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bar_p);
      acc = true;
      if (kx != 0) o_scale = ldexpf(1.f, -kx);
      if (lc + 1 != I.z && k + 1 != n_run) continue;

      // ------------------------------------------------------ the query's last chunk here: read-out
#pragma unroll
      for (int w = 16; w >= 1; w >>= 1) {
        const bool upper = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < 16; i++) {
          if (i < w) {
            const float keep = upper ? l_acc[i + w] : l_acc[i], send = upper ? l_acc[i] : l_acc[i + w];
            l_acc[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, w);
          }
        }
      }
      l_sh[quarter][hb + lane] = l_acc[0];
      soft_sync();
      const bool whole = lc0 == 0 && lc + 1 == I.z;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (lc0 > 0 ? 0 : 1);
      if (t < kHeads) {
        const float l = l_sh[0][t] + l_sh[1][t] + l_sh[2][t] + l_sh[3][t];
        if (whole) {
          if (A.lse != nullptr)
            A.lse[(int64_t)I.x * kHeads + t] =
                l > 0.f || l != l ? (m_ref[t] + log2f(l)) * 0.6931471805599453f : -INFINITY;
          alpha_sh[t] = l != 0.f ? o_scale / l : 0.f;
        } else {
          A.part_ml[slot * 2 * kHeads + t] = m_ref[t];
          A.part_ml[slot * 2 * kHeads + kHeads + t] = l;
          alpha_sh[t] = o_scale;
        }
      }
      const int pos = __ldg(A.pos + I.x);
      soft_sync();
      wait(&bar_free[3], k & 1);                     // PV is complete
      ptx::tc_fence_after();
      for (int blk = warp >> 2; blk < 4; blk += 2) {
        const int d = blk * 128 + quarter * 32 + lane;
        float cs = 1.f, sn = 0.f;
        if (whole && d >= kRopeOff) turn_cs((uint64_t)(int64_t)pos * A.turn[(d - kRopeOff) >> 1], cs, sn);
#pragma unroll 1
        for (int hh = 0; hh < 2; hh++) {
          uint32_t r[32];
          ptx::tmem_ld_32x32b_x32(tq + kPgColO + blk * kHeads + hh * 32, r);
          ptx::tmem_wait_ld();
          if (!whole) {
            float *P = A.part + (slot * kHeads + hh * 32) * kDim + d;
#pragma unroll
            for (int i = 0; i < 32; i++) P[i * kDim] = __uint_as_float(r[i]) * alpha_sh[hh * 32 + i];
            continue;
          }
#pragma unroll
          for (int i = 0; i < 32; i++) {
            float x = __uint_as_float(r[i]) * alpha_sh[hh * 32 + i];
            if (blk == 3 && quarter >= 2) {          // (a, b) by -pos; the partner is in the next lane
              const float y = __shfl_xor_sync(0xFFFFFFFFu, x, 1);
              x = (d & 1) ? x * cs - y * sn : x * cs + y * sn;
            }
            const int64_t o = ((int64_t)I.x * kHeads + hh * 32 + i) * kDim + d;
            if (A.out_f32) static_cast<float *>(A.out)[o] = x;
            else static_cast<__nv_bfloat16 *>(A.out)[o] = __float2bfloat16_rn(x);
          }
        }
      }
      ptx::tc_fence_before();                        // (before the next query's PV, behind bar_p)
      // the first CTA after the one that begins a cut query names it for the join
      if (t == 0 && lc0 > 0 && I.w + lc0 == run_start(run_owner(I.w, T, G) + 1, T, G))
        A.joins[blockIdx.x] = make_int4(I.x, I.z, I.w, T);
    }
  } else if (warp < kPgSoftWarps + kPgLoadWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPgRegsLoad));
    // ======================================================== records to f16, Q
    const int lt = t - kPgSoft, lw = warp - kPgSoftWarps;
    const int e = lt >> 2, part = lt & 3;            // row, 32-dim part of each slab
    unsigned char *tile = sm + kPgSmK + (e >> 3) * 8192 + (part >> 1) * 1024;
    const int ch0 = (part & 1) * 4;                  // the part's first 16-B chunk within its 128 B
    // the chunk's records: this part's codes of each slab, and slab `part`'s
    // eight scales (the row's four threads pass them around)
    uint4 v[4];
    uint2 sc = make_uint2(0u, 0u);
    bool ok = false;
    auto load = [&](const uint8_t *rec, int b) {
      v[b] = rec != nullptr ? __ldg(reinterpret_cast<const uint4 *>(rec + b * 64 + part * 16)) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto load_scales = [&](const uint8_t *rec) {
      sc = rec != nullptr ? __ldg(reinterpret_cast<const uint2 *>(rec + 256 + part * 8)) : make_uint2(0u, 0u);
    };
    PagedCursor C;
    C.c = c_begin;
    C.end = c_end;
    C.qi = start_sh;
    C.off = n_run > 0 ? off_sh : 0;
    if (n_run > 0) C.Q = paged_query(A, C.qi);
    bool more = C.settle(A);
    if (more && !C.window()) {
      const uint8_t *rec = paged_record(A, C, e, part == 0);
      ok = rec != nullptr;
      load_scales(rec);
#pragma unroll
      for (int b = 0; b < 4; b++) load(rec, b);
    }
    uint32_t k = 0;
    for (; more; k++) {
      const int qi = C.qi;
      const int4 info = make_int4(qi, C.local(), C.Q.chunks, C.off);
      const bool win = C.window(), begins = k == 0 || C.local() == 0;
      const uint8_t *wrec = nullptr;
      if (win) {
        ok = e < C.Q.win;
        if (ok) {
          const int ring = (int)(((unsigned)__ldg(A.swa_first + qi) + (unsigned)e) % (unsigned)A.swa_cap);
          wrec = A.swa + ((int64_t)C.Q.seq * A.swa_cap + ring) * kSwaBytes;
        }
      }
      // the next chunk's row
      C.c++;
      more = C.settle(A);
      const uint8_t *next = more && !C.window() ? paged_record(A, C, e, part == 0) : nullptr;
      // the chunk before is through with slab 0, the row marks, Q and the scales
      if (k > 0) wait(&bar_free[0], (k - 1) & 1);
      if (begins) {
        // Q to f16, K-major, 128B swizzle
        const uint4 *src = reinterpret_cast<const uint4 *>(A.q + (int64_t)qi * kHeads * kDim);
        uint32_t m = 0u;
#pragma unroll 2
        for (int j = 0; j < 8; j++) {
          const uint4 x = __ldg(src + lt + j * kPgLoad);
          m = __vmaxu2(m, x.x & 0x7FFF7FFFu);
          m = __vmaxu2(m, x.y & 0x7FFF7FFFu);
          m = __vmaxu2(m, x.z & 0x7FFF7FFFu);
          m = __vmaxu2(m, x.w & 0x7FFF7FFFu);
        }
        m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
        if (lane == 0) qmax_sh[lw] = m;
        load_sync();
#pragma unroll
        for (int w = 0; w < kPgLoadWarps; w++) m = max(m, qmax_sh[w]);
        const int qs = m == 0u ? 0 : max((int)(m >> 7) - 127 - 14, -100);
        const float inv = ldexpf(1.f, -qs);
        if (lt == 0) qscale_sh = ldexpf(1.f, qs);
#pragma unroll 2
        for (int j = 0; j < 8; j++) {
          const uint4 x = __ldg(src + lt + j * kPgLoad);
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int u = 0; u < 4; u++) {
            const __half2 h2 = __floats2half2_rn(bf16_lo(w[u]) * inv, bf16_hi(w[u]) * inv);
            w[u] = *reinterpret_cast<const uint32_t *>(&h2);
          }
          const int i = lt + j * kPgLoad, h = i >> 6, ch = i & 63;
          *reinterpret_cast<uint4 *>(sm + kPgSmQ + (h >> 3) * 8192 + (ch >> 3) * 1024 + sw128(h & 7, ch & 7)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (part == 0) valid_sh[e] = ok ? 1 : 0;
      int kx = 0;
      uint32_t ws[4] = {0u, 0u, 0u, 0u};             // a window record's 16 scales
      if (win) {
        if (ok) {
          const uint4 s4 = __ldg(reinterpret_cast<const uint4 *>(wrec + 512));
          ws[0] = s4.x; ws[1] = s4.y; ws[2] = s4.z; ws[3] = s4.w;
        }
        // the range of the scales' exponents (0 marks a group of zeros)
        int lo = 255, hi = 0;
#pragma unroll
        for (int i = 0; i < 16; i++) {
          const int x = (int)((ws[i >> 2] >> (8 * (i & 3))) & 0xFFu);
          if (x != 0) { lo = min(lo, x); hi = max(hi, x); }
        }
        lo = __reduce_min_sync(0xFFFFFFFFu, lo);
        hi = __reduce_max_sync(0xFFFFFFFFu, hi);
        if (lt == 0) { emin_sh = 255; emax_sh = 0; }
        load_sync();
        if (lane == 0) { atomicMin(&emin_sh, lo); atomicMax(&emax_sh, hi); }
        load_sync();
        if (emax_sh > 0 && (emax_sh - 127 > 7 || emin_sh - 127 < -15)) kx = 7 - (emax_sh - 127);
      }
      if (lt == 0) {
        kx_sh = kx;
        info_sh[k & 1] = info;
      }
      if (win) {
#pragma unroll 1
        for (int b = 0; b < 4; b++) {
          if (b > 0 && k > 0) wait(&bar_free[b], (k - 1) & 1);
          unsigned char *row = tile + 2 * b * 1024;
          // 32 dims, one scale group
          const uint32_t wsb = b == 0 ? ws[0] : b == 1 ? ws[1] : b == 2 ? ws[2] : ws[3];
          const int eb = (int)((wsb >> (8 * part)) & 0xFFu);
          const __half2 fac = __float2half2_rn(eb == 0 ? 0.f : ldexpf(1.f, eb - 127 + kx));
#pragma unroll
          for (int q = 0; q < 2; q++) {
            const uint4 x = ok ? __ldg(reinterpret_cast<const uint4 *>(wrec + b * 128 + part * 32 + q * 16))
                               : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t o[8];
#pragma unroll
            for (int u = 0; u < 8; u++) {
              const uint32_t hv = e4m3x2_to_f16x2(w[u >> 1] >> (16 * (u & 1)));
              const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&hv), fac);
              o[u] = *reinterpret_cast<const uint32_t *>(&y);
            }
            *reinterpret_cast<uint4 *>(row + sw128(e & 7, ch0 + 2 * q)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(row + sw128(e & 7, ch0 + 2 * q + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bar_full[b]);
        }
#pragma unroll
        for (int b = 0; b < 4; b++) load(next, b);
      } else {
#pragma unroll
        for (int b = 0; b < 4; b++) {
          if (b > 0 && k > 0) wait(&bar_free[b], (k - 1) & 1);
          unsigned char *row = tile + 2 * b * 1024;
          // 32 dims, two scale groups
          const uint32_t sx = __shfl_sync(0xFFFFFFFFu, sc.x, b, 4), sy = __shfl_sync(0xFFFFFFFFu, sc.y, b, 4);
          const uint32_t two = e4m3x2_to_f16x2(((part & 2) ? sy : sx) >> (16 * (part & 1)));
          const uint32_t sg[2] = {__byte_perm(two, two, 0x1010), __byte_perm(two, two, 0x3232)};
          const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
          for (int u = 0; u < 4; u++) {              // 8 dims, half a scale group
            uint32_t o[4];
            e2m1x8_to_f16(w[u], o);
#pragma unroll
            for (int q = 0; q < 4; q++) {
              const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&o[q]),
                                        *reinterpret_cast<const __half2 *>(&sg[u >> 1]));
              o[q] = *reinterpret_cast<const uint32_t *>(&y);
            }
            *reinterpret_cast<uint4 *>(row + sw128(e & 7, ch0 + u)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bar_full[b]);
          load(next, b);
        }
      }
      load_scales(next);
      ok = next != nullptr;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPgRegsIssue));
    // ======================================================== MMAs
    // One thread, chosen by elect.sync, and descriptors that are a base plus a
    // constant: 48 cycles an MMA, what N = 64 takes (6 KB of operands).  With the
    // descriptors built at each MMA a thread issued one in 81 to 118 cycles.
    if (warp == kPgSoftWarps + kPgLoadWarps && ptx::elect_one()) {
      constexpr uint32_t id_qk = idesc_m128(0, true, kHeads);
      constexpr uint32_t id_pv = idesc_m128(1, true, kHeads) | (1u << 16);   // both operands MN-major
      const uint32_t base = ptx::smem_u32(sm);
      const uint64_t d_k = ptx::smem_desc(base + kPgSmK, 16, 8192, 2), d_q = ptx::smem_desc(base + kPgSmQ, 16, 8192, 2);
      const uint64_t d_v = ptx::smem_desc(base + kPgSmK, 1024, 8192, 2), d_p = ptx::smem_desc(base + kPgSmP, 1024, 1024, 2);
      for (int k = 0; k < n_run && !bad_sh; k++) {
#pragma unroll 1
        for (int b = 0; b < 4; b++) {                // S^T += K Q^T over slab b
          wait(&bar_full[b], k & 1);
          ptx::tc_fence_after();
          const uint64_t ka = d_k + b * 128, qa = d_q + b * 128;
#pragma unroll
          for (int kk = 0; kk < 8; kk++)
            ptx::tc_mma_bf16(tmem + kPgColS, ka + (kk >> 2) * 64 + (kk & 3) * 2, qa + (kk >> 2) * 64 + (kk & 3) * 2,
                             id_qk, kk > 0 ? 1u : (uint32_t)(b > 0));
        }
        ptx::tc_commit(&bar_s);
        const uint32_t acc = k == 0 || info_sh[k & 1].y == 0 ? 0u : 1u;
        wait(&bar_p, k & 1);
        ptx::tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < 4; b++) {                // O^T block b += K^T P
          const uint64_t va = d_v + b * 128;
#pragma unroll
          for (int ks = 0; ks < kPgChunk / 16; ks++)
            ptx::tc_mma_bf16(tmem + kPgColO + b * kHeads, va + ks * 1024, d_p + ks * 128, id_pv, ks > 0 ? 1u : acc);
          ptx::tc_commit(&bar_free[b]);
        }
      }
      ptx::tc_commit(&bar_drain);
    }
    __syncwarp();
  }
  __syncthreads();
  if (bad_sh) {
    // a wait ran out: every MMA issued here finishes before the tensor memory goes back (bounded;
    // the issuer commits to the drain barrier when it leaves)
    ptx::mbar_wait(&bar_drain, 0);
    ptx::tc_fence_after();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kPgTmemCols);
  }
}

// Joins a cut query's partials over 32 output dims: grid (kDim / 32, CTAs of the
// attention), thread = (head, 8 dims).  Weights 2^(m_s - max m) per head; the
// sums run over the partials in CTA order, so the same inputs give the same bits.
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedArgs A) {
  const int t = threadIdx.x, h = t >> 2, d = blockIdx.x * 32 + (t & 3) * 8;
  griddep_wait();
  griddep_launch();
  const int4 J = __ldcg(A.joins + blockIdx.y);
  if (J.x < 0) return;
  const int qi = J.x;
  const int off = J.z, T = J.w, G = gridDim.y;
  const int g0 = run_owner(off, T, G), g1 = run_owner(off + J.y - 1, T, G);
  auto slot_of = [&](int g) { return 2 * (int64_t)g + (g == g0 ? 1 : 0); };
  auto empty = [&](int g) { return run_start(g, T, G) == run_start(g + 1, T, G); };
  float M = -INFINITY;
  for (int g = g0; g <= g1; g++)
    if (!empty(g)) M = fmaxf(M, __ldcg(A.part_ml + slot_of(g) * 2 * kHeads + h));
  float L = 0.f, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int g = g0; g <= g1; g++) {
    if (empty(g)) continue;
    const int64_t s = slot_of(g);
    const float m = __ldcg(A.part_ml + s * 2 * kHeads + h), l = __ldcg(A.part_ml + s * 2 * kHeads + kHeads + h);
    const float4 *src = reinterpret_cast<const float4 *>(A.part + (s * kHeads + h) * kDim + d);
    const float4 a = __ldcg(src), b = __ldcg(src + 1);
    if (m == -INFINITY) continue;                    // nothing there to attend to
    const float w = exp2f(m - M);
    L += w * l;
    const float e[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] += w * e[j];
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;
#pragma unroll
  for (int j = 0; j < 8; j++) y[j] *= inv;
  if (d >= kRopeOff) {
    const uint64_t pos = (uint64_t)(int64_t)__ldg(A.pos + qi);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float c, s;
      turn_cs(pos * A.turn[(d + j - kRopeOff) >> 1], c, s);
      const float a = y[j], b = y[j + 1];
      y[j] = a * c + b * s;
      y[j + 1] = b * c - a * s;
    }
  }
  const int64_t o = ((int64_t)qi * kHeads + h) * kDim + d;
  if (A.out_f32) {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(A.out) + o);
    p[0] = make_float4(y[0], y[1], y[2], y[3]);
    p[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t *>(&b2);
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(A.out) + o) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (A.lse != nullptr && blockIdx.x == 0 && (t & 3) == 0)
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
  A.part = static_cast<float *>(ws);
  A.part_ml = A.part + 2 * (size_t)sms * kHeads * kDim;
  A.joins = reinterpret_cast<int4 *>(A.part_ml + 2 * (size_t)sms * 2 * kHeads);
  // no more CTAs than there can be chunks
  const int64_t longest = A.sel != nullptr ? A.sel_stride : A.table_stride * A.page;
  const int64_t chunks = (int64_t)A.n_q * ((longest + kPgChunk - 1) / kPgChunk + (A.swa_cap > 0 ? 1 : 0));
  const unsigned grid = (unsigned)(chunks < sms ? (chunks < 1 ? 1 : chunks) : sms);
  e = launch_pdl(paged_attn_kernel, dim3(grid), dim3(kPgThreads), (size_t)kPgSmAlloc, st, 1u, A);
  if (e != cudaSuccess || grid == 1) return e;
  return launch_pdl(paged_join_kernel, dim3(kDim / 32, grid), dim3(256), 0, st, 1u, A);
}

}  // namespace csa2
