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
constexpr int kPgThreads = 256;
constexpr int kPgSmK = 0;                          // 128 entries x 512 dims f16: [e/8][dim/64][e%8][128 B]
constexpr int kPgSmQ = kPgSmK + 128 * 1024;        // 64 heads x 512 dims f16, the same order
constexpr int kPgSmP = kPgSmQ + 64 * 1024;         // 128 entries x 64 heads f16: [e/8][e%8][128 B]
constexpr int kPgSmEnd = kPgSmP + 16 * 1024;
constexpr int kPgSmAlloc = kPgSmEnd + 1024;
constexpr uint32_t kPgColS = 0, kPgColO = 64, kPgTmemCols = 512;
constexpr float kPgRaise = 8.f, kPgShift = 7.f;

// 32 B, 32-byte aligned, in one load
__device__ __forceinline__ void ldg32(const void *p, uint32_t (&r)[8]) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
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

// CTA g of G has chunks [g T / G, (g + 1) T / G) of T
__device__ __forceinline__ int64_t run_start(int64_t g, int64_t T, int64_t G) { return g * T / G; }
__device__ __forceinline__ int64_t run_owner(int64_t c, int64_t T, int64_t G) { return ((c + 1) * G - 1) / T; }

__global__ void __launch_bounds__(kPgThreads, 1) paged_attn_kernel(const __grid_constant__ PagedArgs A) {
  extern __shared__ __align__(1024) unsigned char pg_smem_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(pg_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t bar_s, bar_o, bar_drain;
  __shared__ uint32_t tmem_sh, qmax_sh[kPgThreads / 32];
  __shared__ float m_ref[kHeads], alpha_sh[kHeads], l_sh[4][kHeads], red_sh[4][kHeads];
  __shared__ uint8_t valid_sh[kPgChunk];
  __shared__ long long scan_sh[kPgThreads / 32], off_sh;
  __shared__ int start_sh, emin_sh, emax_sh;
  __shared__ volatile int bad_sh;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (t == 0) {
    ptx::mbar_init(&bar_s, 1);
    ptx::mbar_init(&bar_o, 4);
    ptx::mbar_init(&bar_drain, 4);
    bad_sh = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0) ptx::tmem_alloc(&tmem_sh, kPgTmemCols);
  griddep_wait();
  griddep_launch();

  // ---------------------------------------------------------- this CTA's run
  // prefix sums of the queries' chunks: thread t has queries [u0, u1)
  const int per = (A.n_q + kPgThreads - 1) / kPgThreads, u0 = min(t * per, A.n_q), u1 = min(u0 + per, A.n_q);
  long long mine = 0;
  bool any_bad = false;
  for (int q = u0; q < u1; q++) {
    const PagedQuery r = paged_query(A, q);
    mine += r.chunks;
    any_bad |= r.bad;
  }
  if (any_bad && blockIdx.x == 0) record_error(A.status, CSA2_ERR_BOUNDS);
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) scan_sh[warp] = inc;
  if (t == 0) start_sh = A.n_q;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kPgThreads / 32; w++) {
    if (w < warp) before += scan_sh[w];
    total += scan_sh[w];
  }
  before += inc - mine;
  const int64_t G = gridDim.x, T = total;
  const int64_t c_begin = run_start(blockIdx.x, T, G), c_end = run_start((int64_t)blockIdx.x + 1, T, G);
  if (c_begin < c_end && before <= c_begin && c_begin < before + mine) {
    long long o = before;
    int q = u0;
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
  const uint32_t sK = ptx::smem_u32(sm + kPgSmK), sQ = ptx::smem_u32(sm + kPgSmQ), sP = ptx::smem_u32(sm + kPgSmP);
  constexpr uint32_t id_qk = idesc_m128(0, true, kHeads);
  constexpr uint32_t id_pv = idesc_m128(1, true, kHeads) | (1u << 16);   // both operands MN-major
  int qi = start_sh;
  int64_t off = qi < A.n_q ? off_sh : 0;
  uint32_t phase = 0;
  const int quarter = warp & 3, hb = (warp >> 2) * 32, e_row = quarter * 32 + lane;   // softmax: TMEM lane, heads

  for (int64_t c = c_begin; c < c_end && !bad_sh;) {
    const PagedQuery Q = paged_query(A, qi);
    const int lc0 = (int)(c - off), lc1 = (int)min((int64_t)Q.chunks, c_end - off);
    if (lc1 <= lc0) {                                // (a query without chunks)
      off += Q.chunks;
      qi++;
      continue;
    }
    // ------------------------------------------------------ Q to f16, K-major, 128B swizzle
    float q_scale;                                   // 2^qs
    {
      const uint4 *src = reinterpret_cast<const uint4 *>(A.q + (int64_t)qi * kHeads * kDim);
      uint4 v[16];
#pragma unroll
      for (int j = 0; j < 16; j++) v[j] = __ldg(src + t + j * kPgThreads);
      uint32_t m = 0u;
#pragma unroll
      for (int j = 0; j < 16; j++) {
        m = __vmaxu2(m, v[j].x & 0x7FFF7FFFu);
        m = __vmaxu2(m, v[j].y & 0x7FFF7FFFu);
        m = __vmaxu2(m, v[j].z & 0x7FFF7FFFu);
        m = __vmaxu2(m, v[j].w & 0x7FFF7FFFu);
      }
      m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
      if (lane == 0) qmax_sh[warp] = m;
      if (t < kHeads) m_ref[t] = -INFINITY;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kPgThreads / 32; w++) m = max(m, qmax_sh[w]);
      const int qs = m == 0u ? 0 : max((int)(m >> 7) - 127 - 14, -100);
      q_scale = ldexpf(1.f, qs);
      const float inv = ldexpf(1.f, -qs);
#pragma unroll
      for (int j = 0; j < 16; j++) {
        uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const __half2 h2 = __floats2half2_rn(bf16_lo(w[k]) * inv, bf16_hi(w[k]) * inv);
          w[k] = *reinterpret_cast<const uint32_t *>(&h2);
        }
        const int i = t + j * kPgThreads, h = i >> 6, ch = i & 63;
        *reinterpret_cast<uint4 *>(sm + kPgSmQ + (h >> 3) * 8192 + (ch >> 3) * 1024 + sw128(h & 7, ch & 7)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    float l_acc[32];
#pragma unroll
    for (int i = 0; i < 32; i++) l_acc[i] = 0.f;
    bool acc = false;                                // O holds something
    float o_scale = 1.f;                             // what O still has to be multiplied by
    for (int lc = lc0; lc < lc1; lc++) {
      const bool win = Q.win > 0 && lc == 0;
      const int e = t >> 1, half = t & 1;            // row, 64-dim half of each 128-dim slab
      // ---------------------------------------------------- dequantise
      bool ok = false;
      int kx = 0;
      if (win) {
        const uint8_t *rec = nullptr;
        if (e < Q.win) {
          ok = true;
          const int ring = (int)(((unsigned)__ldg(A.swa_first + qi) + (unsigned)e) % (unsigned)A.swa_cap);
          rec = A.swa + ((int64_t)Q.seq * A.swa_cap + ring) * kSwaBytes;
        }
        uint32_t sc[4] = {0u, 0u, 0u, 0u};
        if (ok) {
          const uint4 s4 = __ldg(reinterpret_cast<const uint4 *>(rec + 512));
          sc[0] = s4.x; sc[1] = s4.y; sc[2] = s4.z; sc[3] = s4.w;
        }
        // the range of the scales' exponents (0 marks a group of zeros)
        int lo = 255, hi = 0;
#pragma unroll
        for (int k = 0; k < 16; k++) {
          const int b = (int)((sc[k >> 2] >> (8 * (k & 3))) & 0xFFu);
          if (b != 0) { lo = min(lo, b); hi = max(hi, b); }
        }
        lo = __reduce_min_sync(0xFFFFFFFFu, lo);
        hi = __reduce_max_sync(0xFFFFFFFFu, hi);
        if (t == 0) { emin_sh = 255; emax_sh = 0; }
        __syncthreads();
        if (lane == 0) { atomicMin(&emin_sh, lo); atomicMax(&emax_sh, hi); }
        __syncthreads();
        if (emax_sh > 0 && (emax_sh - 127 > 7 || emin_sh - 127 < -15)) kx = 7 - (emax_sh - 127);
#pragma unroll
        for (int b = 0; b < 4; b++) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; k++)
            v[k] = ok ? __ldg(reinterpret_cast<const uint4 *>(rec + b * 128 + half * 64 + k * 16)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int k = 0; k < 4; k++) {              // 16 dims, half a scale group
            const int gidx = b * 4 + half * 2 + (k >> 1);
            const int eb = (int)((sc[gidx >> 2] >> (8 * (gidx & 3))) & 0xFFu);
            const __half2 f = __float2half2_rn(eb == 0 ? 0.f : ldexpf(1.f, eb - 127 + kx));
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            uint32_t o[8];
#pragma unroll
            for (int u = 0; u < 8; u++) {
              const uint32_t hv = e4m3x2_to_f16x2(w[u >> 1] >> (16 * (u & 1)));
              const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&hv), f);
              o[u] = *reinterpret_cast<const uint32_t *>(&x);
            }
            unsigned char *row = sm + kPgSmK + (e >> 3) * 8192 + (2 * b + half) * 1024;
            *reinterpret_cast<uint4 *>(row + sw128(e & 7, 2 * k)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(row + sw128(e & 7, 2 * k + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      } else {
        const int i = (lc - (Q.win > 0 ? 1 : 0)) * kPgChunk + e;
        const uint8_t *rec = nullptr;
        int j = -1;
        if (i < Q.n) j = A.sel != nullptr ? __ldg(A.sel + (int64_t)qi * A.sel_stride + i) : i;
        if (j >= 0) {
          const int vis = A.sel != nullptr ? __ldg(A.n_vis + qi) : Q.n;
          const int col = (int)((unsigned)j / (unsigned)A.page);
          const int id = j < vis ? __ldg(A.table + (int64_t)Q.seq * A.table_stride + col) : -1;
          if (id >= 0 && id < A.n_pages) {
            rec = A.pages + ((int64_t)id * A.page + (j - col * A.page)) * kKvBytes;
            ok = true;
          } else if (half == 0) {
            record_error(A.status, CSA2_ERR_BOUNDS);
          }
        }
#pragma unroll
        for (int b = 0; b < 4; b++) {
          uint32_t v[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, sc = 0u;
          if (ok) {
            ldg32(rec + b * 64 + half * 32, v);
            sc = __ldg(reinterpret_cast<const uint32_t *>(rec + 256 + b * 8 + half * 4));
          }
          const uint32_t s01 = e4m3x2_to_f16x2(sc), s23 = e4m3x2_to_f16x2(sc >> 16);
          unsigned char *row = sm + kPgSmK + (e >> 3) * 8192 + (2 * b + half) * 1024;
#pragma unroll
          for (int u = 0; u < 8; u++) {              // 8 dims, half a scale group
            const uint32_t two = u < 4 ? s01 : s23;
            const uint32_t s2 = (u & 2) ? __byte_perm(two, two, 0x3232) : __byte_perm(two, two, 0x1010);
            uint32_t o[4];
            e2m1x8_to_f16(v[u], o);
#pragma unroll
            for (int k = 0; k < 4; k++) {
              const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&o[k]), *reinterpret_cast<const __half2 *>(&s2));
              o[k] = *reinterpret_cast<const uint32_t *>(&x);
            }
            *reinterpret_cast<uint4 *>(row + sw128(e & 7, u)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      if (half == 0) valid_sh[e] = ok ? 1 : 0;
      ptx::fence_proxy_async_smem();
      __syncthreads();
      // ---------------------------------------------------- S^T = K Q^T
      if (t == 0) {
        ptx::tc_fence_after();
#pragma unroll 1
        for (int kk = 0; kk < kDim / 16; kk++) {
          const uint32_t ko = (kk >> 2) * 1024 + (kk & 3) * 32;
          ptx::tc_mma_bf16(tmem + kPgColS, ptx::smem_desc(sK + ko, 16, 8192, 2), ptx::smem_desc(sQ + ko, 16, 8192, 2),
                           id_qk, kk > 0 ? 1u : 0u);
        }
        ptx::tc_commit(&bar_s);
      }
      __syncwarp();
      if (!ptx::mbar_wait(&bar_s, phase)) { record_error(A.status, CSA2_ERR_TIMEOUT); bad_sh = 1; }
      ptx::tc_fence_after();
      // ---------------------------------------------------- softmax
      float s[32];
      {
        uint32_t r[32];
        ptx::tmem_ld_32x32b_x32(tmem + ((uint32_t)(quarter * 32) << 16) + kPgColS + hb, r);
        ptx::tmem_wait_ld();
        const float f = A.scale * 1.4426950408889634f * ldexpf(q_scale, -kx);
#pragma unroll
        for (int i = 0; i < 32; i++) s[i] = __uint_as_float(r[i]) * f;
      }
      const bool ev = valid_sh[e_row] != 0;
      bool over = false;
#pragma unroll
      for (int i = 0; i < 32; i++) over |= s[i] > m_ref[hb + i] + kPgRaise;
      float fac = o_scale;                           // (a window's 2^-kx, undone before the next chunk)
      bool rescale = acc && fac != 1.f;
      if (__syncthreads_or(ev && over)) {
        // the chunk's maximum of every head: lane L ends with head hb + L
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; i++) v[i] = ev ? s[i] : -INFINITY;
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
        __syncthreads();
        if (t < kHeads) {
          const float cm = fmaxf(fmaxf(red_sh[0][t], red_sh[1][t]), fmaxf(red_sh[2][t], red_sh[3][t]));
          const float mo = m_ref[t];
          float al = 1.f;
          if (cm > mo + kPgRaise) {
            al = mo == -INFINITY ? 0.f : exp2f(mo - cm);
            m_ref[t] = cm;
          }
          alpha_sh[t] = al;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 32; i++) l_acc[i] *= alpha_sh[hb + i];
        rescale = acc;
      } else if (rescale) {
        if (t < kHeads) alpha_sh[t] = 1.f;
        __syncthreads();
      }
      if (rescale) {
        // O *= alpha (x fac): warp w has lane quarter w % 4 of blocks w / 4 and w / 4 + 2
        for (int blk = warp >> 2; blk < 4; blk += 2)
          for (int hh = 0; hh < 2; hh++) {
            uint32_t r[32];
            const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + kPgColO + blk * kHeads + hh * 32;
            ptx::tmem_ld_32x32b_x32(ta, r);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i++) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha_sh[hh * 32 + i] * fac);
            ptx::tmem_st_32x32b_x32(ta, r);
          }
        ptx::tmem_wait_st();
        o_scale = 1.f;
      }
      {
        unsigned char *row = sm + kPgSmP + (e_row >> 3) * 1024;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; k++) {
            const int i = 8 * j + 2 * k;
            const float p0 = ev ? exp2f(s[i] - (m_ref[hb + i] - kPgShift)) : 0.f;
            const float p1 = ev ? exp2f(s[i + 1] - (m_ref[hb + i + 1] - kPgShift)) : 0.f;
            l_acc[i] += p0;
            l_acc[i + 1] += p1;
            const __half2 h2 = __floats2half2_rn(p0, p1);
            o[k] = *reinterpret_cast<const uint32_t *>(&h2);
          }
          *reinterpret_cast<uint4 *>(row + sw128(e_row & 7, (hb >> 3) + j)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      ptx::tc_fence_before();
      ptx::fence_proxy_async_smem();
      __syncthreads();
      // ---------------------------------------------------- O^T += K^T P
      if (lane == 0 && warp < 4) {
        ptx::tc_fence_after();
#pragma unroll 1
        for (int ks = 0; ks < kPgChunk / 16; ks++)
          ptx::tc_mma_bf16(tmem + kPgColO + warp * kHeads,
                           ptx::smem_desc(sK + (2 * ks) * 8192 + (2 * warp) * 1024, 1024, 8192, 2),
                           ptx::smem_desc(sP + (2 * ks) * 1024, 1024, 1024, 2), id_pv, (acc || ks > 0) ? 1u : 0u);
        ptx::tc_commit(&bar_o);
      }
      __syncwarp();
      if (!ptx::mbar_wait(&bar_o, phase)) { record_error(A.status, CSA2_ERR_TIMEOUT); bad_sh = 1; }
      ptx::tc_fence_after();
      phase ^= 1;
      acc = true;
      if (win) o_scale = ldexpf(1.f, -kx);
      __syncthreads();
      if (bad_sh) break;
    }
    if (bad_sh) break;
    // ------------------------------------------------------ denominators
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
    __syncthreads();
    // ------------------------------------------------------ read-out
    const bool whole = lc0 == 0 && lc1 == Q.chunks;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (lc0 > 0 ? 0 : 1);
    if (t < kHeads) {
      const float l = l_sh[0][t] + l_sh[1][t] + l_sh[2][t] + l_sh[3][t];
      if (whole) {
        if (A.lse != nullptr)
          A.lse[(int64_t)qi * kHeads + t] = l > 0.f || l != l ? (m_ref[t] - kPgShift + log2f(l)) * 0.6931471805599453f : -INFINITY;
        alpha_sh[t] = l != 0.f ? o_scale / l : 0.f;
      } else {
        A.part_ml[slot * 2 * kHeads + t] = m_ref[t];
        A.part_ml[slot * 2 * kHeads + kHeads + t] = l;
        alpha_sh[t] = o_scale;
      }
    }
    __syncthreads();
    const int pos = __ldg(A.pos + qi);
    for (int blk = warp >> 2; blk < 4; blk += 2) {
      const int d = blk * 128 + quarter * 32 + lane;
      float cs = 1.f, sn = 0.f;
      if (whole && d >= kRopeOff) turn_cs((uint64_t)(int64_t)pos * A.turn[(d - kRopeOff) >> 1], cs, sn);
#pragma unroll
      for (int hh = 0; hh < 2; hh++) {
        uint32_t r[32];
        ptx::tmem_ld_32x32b_x32(tmem + ((uint32_t)(quarter * 32) << 16) + kPgColO + blk * kHeads + hh * 32, r);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i++) {
          const int h = hh * 32 + i;
          float x = __uint_as_float(r[i]) * alpha_sh[h];
          if (!whole) {
            A.part[(slot * kHeads + h) * kDim + d] = x;
            continue;
          }
          if (d >= kRopeOff) {                       // (a, b) by -pos; the partner is in the next lane
            const float y = __shfl_xor_sync(0xFFFFFFFFu, x, 1);
            x = (d & 1) ? x * cs - y * sn : x * cs + y * sn;
          }
          const int64_t o = ((int64_t)qi * kHeads + h) * kDim + d;
          if (A.out_f32) static_cast<float *>(A.out)[o] = x;
          else static_cast<__nv_bfloat16 *>(A.out)[o] = __float2bfloat16_rn(x);
        }
      }
    }
    // the first CTA after the one that begins a cut query names it for the join
    if (t == 0 && lc0 > 0 && c == run_start(run_owner(off, T, G) + 1, T, G))
      A.joins[blockIdx.x] = make_int4(qi, (int)Q.chunks, (int)(off & 0xFFFFFFFF), (int)(off >> 32));
    ptx::tc_fence_before();
    __syncthreads();
    c = off + lc1;
    off += Q.chunks;
    qi++;
  }
  if (bad_sh) {
    // a wait ran out: every MMA issued here finishes before the tensor memory goes back (bounded)
    if (lane == 0 && warp < 4) ptx::tc_commit(&bar_drain);
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
  __shared__ long long total_sh;
  const int t = threadIdx.x, h = t >> 2, d = blockIdx.x * 32 + (t & 3) * 8;
  griddep_wait();
  griddep_launch();
  const int4 J = __ldcg(A.joins + blockIdx.y);
  if (J.x < 0) return;
  const int qi = J.x;
  // T again, from the queries' chunks
  if (t == 0) total_sh = 0;
  __syncthreads();
  long long mine = 0;
  for (int q = t; q < A.n_q; q += 256) mine += paged_query(A, q).chunks;
  atomicAdd(reinterpret_cast<unsigned long long *>(&total_sh), (unsigned long long)mine);
  __syncthreads();
  const int64_t T = total_sh, G = gridDim.y;
  const int64_t off = (int64_t)(((uint64_t)(uint32_t)J.w << 32) | (uint32_t)J.z);
  const int64_t g0 = run_owner(off, T, G), g1 = run_owner(off + J.y - 1, T, G);
  auto slot_of = [&](int64_t g) { return 2 * g + (g == g0 ? 1 : 0); };
  auto empty = [&](int64_t g) { return run_start(g, T, G) == run_start(g + 1, T, G); };
  float M = -INFINITY;
  for (int64_t g = g0; g <= g1; g++)
    if (!empty(g)) M = fmaxf(M, __ldcg(A.part_ml + slot_of(g) * 2 * kHeads + h));
  float L = 0.f, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t g = g0; g <= g1; g++) {
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
    A.lse[(int64_t)qi * kHeads + h] = L > 0.f || L != L ? (M - kPgShift + log2f(L)) * 0.6931471805599453f : -INFINITY;
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
