// Norm of the query heads and of the latent, rotation of their last 64 dims
// and cache write, in one pass (csa2_qk_norm_rope).
//
// Per 512-wide row x with gain g:  y_c = x_c g_c / sqrt(mean(x^2) + eps), then
// the pairs (a, b) = (y[448 + 2i], y[449 + 2i]) become (a cos t - b sin t,
// a sin t + b cos t), t = pos * rope_base^(-2i/64): the rotation that
// csa2_sparse_attn and csa2_paged_attn undo on their output ("An infra-oriented
// diagram of the DeepSeek-V4.1-Flash architecture", reading notes: RoPE acts on
// 64 of the 512 dims).
//
// Angles: pos * t is kept in turns, as a 64-bit fixed-point fraction (the
// integer product drops whole turns exactly), so a position of 2^20 loses
// nothing; the fraction goes to fp32 for the sine and cosine.
//
// Query rows, 1 KB in and 1 KB out each, are bound by HBM: one warp per row, a
// lane holds channels [8 lane, 8 lane + 8) and 256 + that, so every access of a
// warp is 512 contiguous bytes; a CTA's 8 warps take the heads of one token and
// share its 32 angles.  Sums are fp32 (32 terms of a lane's row at most, then a
// shuffle tree), the result is rounded once; a row whose mean square is out of
// [2^-100, 2^100], or not a number, goes to fp64.
//
// Latent rows, one warp per token, feed cache records, whose codes hang on
// which side of a rounding border a value falls.  So that the records do not
// depend on the order of fp32 sums, the latent is the exact value rounded once
// to bf16: the sum of squares (each square exact in fp32) and the normalised
// values are carried as unevaluated sums of two fp32 (about 2^-44 relative),
// the rotated channels in fp32 with an error bound; a pair whose bound straddles a
// bf16 border (about one row in forty has one) is rotated again in fp64, and a row
// whose range leaves fp32 is recomputed in fp64 (fp64 is slow here: with the
// whole row recomputed for such a pair, 8,192 latents took 38 us instead of 23).
#include <cuda_bf16.h>
#include <math.h>

#include "attn.cuh"
#include "common.cuh"
#include "convert.cuh"
#include "launch.cuh"

namespace csa2 {

constexpr int kNormThreads = 256;

__device__ __forceinline__ void unpack8(const uint4 &v, float *x) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x);
  x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z);
  x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}

// a lane's 16 gains (channels 8 lane .. and 256 + 8 lane ..)
__device__ __forceinline__ void load_gain(const float *gain, int lane, float *g) {
  if (gain == nullptr) {
#pragma unroll
    for (int i = 0; i < 16; i++) g[i] = 1.f;
    return;
  }
#pragma unroll
  for (int v = 0; v < 4; v++) {
    const float4 f = __ldg(reinterpret_cast<const float4 *>(gain + (v >> 1) * 256 + lane * 8) + (v & 1));
    g[4 * v] = f.x; g[4 * v + 1] = f.y; g[4 * v + 2] = f.z; g[4 * v + 3] = f.w;
  }
}

// fp64 to bf16, any value
__device__ __forceinline__ uint32_t bf16_of_f64(double v) {
  if (isnan(v)) return 0x7FFFu;
  if (fabs(v) >= 0x1.FFp127) return v > 0 ? 0x7F80u : 0xFF80u;      // half a step above the largest: infinity
  return bf16_from_f64(v);
}

// A row in fp64 (warp-wide): y[i] = bf16 bits of the lane's 16 channels.
__device__ __noinline__ void row_f64(const float *x, const float *g, double eps, uint64_t turn, int lane,
                                            uint32_t *y) {
  double ss = 0.0;
  for (int i = 0; i < 16; i++) ss = fma((double)x[i], (double)x[i], ss);
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  const double inv = 1.0 / sqrt(ss / kDim + eps);
  double c, s;
  sincospi((double)(int64_t)turn * 0x1p-63, &s, &c);                 // pair `lane`
  for (int i = 0; i < 8; i++) y[i] = bf16_of_f64((double)x[i] * (double)g[i] * inv);
  for (int k = 0; k < 4; k++) {
    const double ck = __shfl_sync(0xFFFFFFFFu, c, (lane & 7) * 4 + k);
    const double sk = __shfl_sync(0xFFFFFFFFu, s, (lane & 7) * 4 + k);
    double a = (double)x[8 + 2 * k] * (double)g[8 + 2 * k] * inv;
    double b = (double)x[9 + 2 * k] * (double)g[9 + 2 * k] * inv;
    if (lane >= (kRopeOff - 256) / 8) {
      const double a0 = a;
      a = a0 * ck - b * sk;
      b = a0 * sk + b * ck;
    }
    y[8 + 2 * k] = bf16_of_f64(a);
    y[9 + 2 * k] = bf16_of_f64(b);
  }
}

// ------------------------------------------------------------------ queries
// A query row whose mean square (plus eps) fp32 does not hold well: in fp64.
__device__ __noinline__ void query_row_f64(const NormArgs &A, int64_t tok, const uint16_t *row, int lane, uint4 *out) {
  float x[16], g[16];
  uint32_t y[16];
  unpack8(*reinterpret_cast<const uint4 *>(row), x);
  unpack8(*reinterpret_cast<const uint4 *>(row + 256), x + 8);
  load_gain(A.q_gain, lane, g);
  row_f64(x, g, A.eps, (uint64_t)(int64_t)__ldg(A.pos + tok) * A.turn[lane], lane, y);
  out[0] = make_uint4(y[0] | y[1] << 16, y[2] | y[3] << 16, y[4] | y[5] << 16, y[6] | y[7] << 16);
  out[32] = make_uint4(y[8] | y[9] << 16, y[10] | y[11] << 16, y[12] | y[13] << 16, y[14] | y[15] << 16);
}

template <int HPW>
__device__ __forceinline__ void query_rows(const NormArgs &A, int idx, float2 *cs_sh) {
  constexpr int B = HPW < 2 ? HPW : 2;              // rows of a warp in flight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = 8 / HPW;                        // CTAs per token
  const int64_t tok = idx / parts;
  const int h0 = (idx % parts) * 8 * HPW + warp;    // heads h0 + 8 j
  const uint16_t *src = A.q + tok * A.q_stride + lane * 8;
  uint16_t *dst = A.q_out + tok * (kHeads * kDim) + lane * 8;
  uint4 r[B][2];
  uint32_t again = 0u;                              // rows left to fp64
  auto load = [&](int j0) {
#pragma unroll
    for (int j = 0; j < B; j++) {
      const uint4 *p = reinterpret_cast<const uint4 *>(src + (h0 + 8 * (j0 + j)) * kDim);
      r[j][0] = __ldcs(p);
      r[j][1] = __ldcs(p + 32);
    }
  };
  load(0);
  if (warp == 0) {
    float c, s;
    turn_cs((uint64_t)(int64_t)__ldg(A.pos + tok) * A.turn[lane], c, s);
    cs_sh[lane] = make_float2(c, s);
  }
  float g[16];
  load_gain(A.q_gain, lane, g);
  __syncthreads();
  float2 cs[4];
#pragma unroll
  for (int k = 0; k < 4; k++) cs[k] = cs_sh[(lane & 7) * 4 + k];
#pragma unroll
  for (int j0 = 0; j0 < HPW; j0 += B) {
    if (j0 > 0) load(j0);
    float ss[B];
#pragma unroll
    for (int j = 0; j < B; j++) {
      float x[16];
      unpack8(r[j][0], x);
      unpack8(r[j][1], x + 8);
      ss[j] = 0.f;
#pragma unroll
      for (int i = 0; i < 16; i++) ss[j] = fmaf(x[i], x[i], ss[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < B; j++) ss[j] += __shfl_xor_sync(0xFFFFFFFFu, ss[j], o);
#pragma unroll
    for (int j = 0; j < B; j++) {
      const float ms = fmaf(ss[j], 1.f / kDim, A.eps_hi), inv = rsqrtf(ms);
      uint4 *p = reinterpret_cast<uint4 *>(dst + (h0 + 8 * (j0 + j)) * kDim);
      const bool held = ms > 0x1p-100f && ms < 0x1p100f;      // (the same for all lanes; false for NaN)
      if (!held) again |= 1u << (j0 + j);
      float x[16];
      unpack8(r[j][0], x);
      unpack8(r[j][1], x + 8);
#pragma unroll
      for (int i = 0; i < 16; i++) x[i] = x[i] * inv * g[i];
      if (lane >= (kRopeOff - 256) / 8) {           // channels 448 .. 511
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const float a = x[8 + 2 * k], b = x[9 + 2 * k];
          x[8 + 2 * k] = a * cs[k].x - b * cs[k].y;
          x[9 + 2 * k] = a * cs[k].y + b * cs[k].x;
        }
      }
      const uint4 lo = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                  pack_bf16x2(x[6], x[7]));
      const uint4 hi = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]),
                                  pack_bf16x2(x[14], x[15]));
      if (held) {
        p[0] = lo;
        p[32] = hi;
      }
    }
  }
  // (read again, behind all others: a call among them costs the loop 33 us of 8,192 tokens' 184 in spills)
  while (__builtin_expect(again != 0u, 0)) {
    const int h = h0 + 8 * (__ffs((int)again) - 1);
    query_row_f64(A, tok, src + h * kDim, lane, reinterpret_cast<uint4 *>(dst + h * kDim));
    again &= again - 1u;
  }
}

// ------------------------------------------------------------------ latents
// s + e = a + b exactly
__device__ __forceinline__ float two_sum(float a, float b, float &e) {
  const float s = a + b, bb = s - a;
  e = (a - (s - bb)) + (b - bb);
  return s;
}

// h + l rounded once to bf16 (|l| at most a rounding of h)
__device__ __forceinline__ uint32_t bf16_of_pair(float h, float l) {
  const float s = h + l, t = l - (s - h);
  const uint32_t u = __float_as_uint(s);
  // a tie of the rounded sum is decided by what it left out
  if ((u & 0xFFFFu) == 0x8000u && t != 0.f) return (u >> 16) + ((t > 0.f) == (s > 0.f) ? 1u : 0u);
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// A rotated pair in fp64: its bf16 bits, the first channel's in the lower half.
__device__ __noinline__ uint32_t rotated_pair_f64(double a, double b, uint64_t turn) {
  double c, s;
  sincospi((double)(int64_t)turn * 0x1p-63, &s, &c);
  return bf16_of_f64(a * c - b * s) | bf16_of_f64(a * s + b * c) << 16;
}

__device__ __forceinline__ void latent_row(const NormArgs &A, int tok, int lane) {
  const uint4 *p = reinterpret_cast<const uint4 *>(A.lat + (int64_t)tok * A.lat_stride + lane * 8);
  const uint4 v0 = __ldcs(p), v1 = __ldcs(p + 32);
  const int slot = A.kv != nullptr ? __ldg(A.slot + tok) : -1;
  const int wslot = A.swa != nullptr ? __ldg(A.swa_slot + tok) : -1;
  const uint64_t turn = (uint64_t)(int64_t)__ldg(A.pos + tok) * A.turn[lane];
  float g[16], x[16];
  load_gain(A.lat_gain, lane, g);
  unpack8(v0, x);
  unpack8(v1, x + 8);
  // the sum of squares as hi + lo
  float hi = 0.f, lo = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i++) {
    float e;
    hi = two_sum(hi, x[i] * x[i], e);
    lo += e;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float oh = __shfl_xor_sync(0xFFFFFFFFu, hi, o), ol = __shfl_xor_sync(0xFFFFFFFFu, lo, o);
    float e;
    hi = two_sum(hi, oh, e);
    lo = lo + ol + e;
  }
  // m = mean + eps as a pair, then r0 + rl = 1 / sqrt(m): with the seed r0 and
  // e = 1 - m r0^2, 1 / sqrt(m) = r0 (1 + e / 2 + 3 e^2 / 8 + ..)
  float e0;
  const float s0 = two_sum(hi * (1.f / kDim), A.eps_hi, e0);
  e0 += lo * (1.f / kDim) + A.eps_lo;
  const float mh = s0 + e0, ml = e0 - (mh - s0);
  const float r0 = rsqrtf(mh);
  const float q = r0 * r0, qe = fmaf(r0, r0, -q), mq = mh * q, mqe = fmaf(mh, q, -mq);
  const float e = (1.f - mq) - mqe - mh * qe - ml * q;
  const float rl = r0 * fmaf(0.375f * e, e, 0.5f * e);
  const bool plain = mh > 0x1p-100f && mh < 0x1p100f;                // (false for NaN)
  bool again = !plain;
  uint32_t y[16];
  float c, s;
  turn_cs(turn, c, s);                                               // pair `lane`
  float ck[4], sk[4];
#pragma unroll
  for (int k = 0; k < 4; k++) {
    ck[k] = __shfl_sync(0xFFFFFFFFu, c, (lane & 7) * 4 + k);
    sk[k] = __shfl_sync(0xFFFFFFFFu, s, (lane & 7) * 4 + k);
  }
  float h[16], l[16];
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const float pr = x[i] * g[i], pe = fmaf(x[i], g[i], -pr);
    h[i] = pr * r0;
    l[i] = fmaf(pe, r0, fmaf(pr, rl, fmaf(pr, r0, -h[i])));
    // the low parts hold only while nothing under- or overflows
    const bool zero = x[i] == 0.f || g[i] == 0.f;
    again |= !zero && !(fabsf(pr) > 0x1p-90f && fabsf(pr) < 0x1p100f && fabsf(h[i]) > 0x1p-90f &&
                        fabsf(h[i]) < 0x1p100f);
    y[i] = bf16_of_pair(h[i], l[i]);
  }
  uint32_t close = 0u;                                               // pairs whose bound straddles a border
  if (lane >= (kRopeOff - 256) / 8) {
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float a = h[8 + 2 * k] + l[8 + 2 * k], b = h[9 + 2 * k] + l[9 + 2 * k];
      const float ra = a * ck[k] - b * sk[k], rb = a * sk[k] + b * ck[k];
      // cos and sin to 2^-22 (2 ulps and the angle's rounding), a, b and the
      // products to 2^-24 each: below (|a| + |b|) 2^-21
      const float d = (fabsf(a) + fabsf(b)) * 0x1p-21f;
      const uint32_t al = __bfloat16_as_ushort(__float2bfloat16_rn(ra - d));
      const uint32_t ah = __bfloat16_as_ushort(__float2bfloat16_rn(ra + d));
      const uint32_t bl = __bfloat16_as_ushort(__float2bfloat16_rn(rb - d));
      const uint32_t bh = __bfloat16_as_ushort(__float2bfloat16_rn(rb + d));
      close |= (uint32_t)(al != ah || bl != bh) << k;
      y[8 + 2 * k] = al;
      y[9 + 2 * k] = bl;
    }
  }
  if (__any_sync(0xFFFFFFFFu, again)) {
    row_f64(x, g, A.eps, turn, lane, y);
  } else if (__any_sync(0xFFFFFFFFu, close != 0u)) {
#pragma unroll
    for (int k = 0; k < 4; k++) {
      if (!__any_sync(0xFFFFFFFFu, (close >> k) & 1u)) continue;
      const uint64_t t = __shfl_sync(0xFFFFFFFFu, turn, (lane & 7) * 4 + k);
      if ((close >> k) & 1u) {
        const uint32_t two = rotated_pair_f64((double)h[8 + 2 * k] + l[8 + 2 * k], (double)h[9 + 2 * k] + l[9 + 2 * k], t);
        y[8 + 2 * k] = two & 0xFFFFu;
        y[9 + 2 * k] = two >> 16;
      }
    }
  }
  if (A.lat_out != nullptr) {
    uint4 *o = reinterpret_cast<uint4 *>(A.lat_out + (int64_t)tok * kDim + lane * 8);
    o[0] = make_uint4(y[0] | y[1] << 16, y[2] | y[3] << 16, y[4] | y[5] << 16, y[6] | y[7] << 16);
    o[32] = make_uint4(y[8] | y[9] << 16, y[10] | y[11] << 16, y[12] | y[13] << 16, y[14] | y[15] << 16);
  }
#pragma unroll
  for (int i = 0; i < 16; i++) x[i] = __uint_as_float(y[i] << 16);
  float amax[2];                                                     // of this lane's 8 channels, each half
#pragma unroll
  for (int f = 0; f < 2; f++) {
    amax[f] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) amax[f] = fmaxf(amax[f], fabsf(x[8 * f + i]));
    amax[f] = fmaxf(amax[f], __shfl_xor_sync(0xFFFFFFFFu, amax[f], 1));   // groups of 16: lane pairs
  }
  if (slot >= 0) {                                                   // (the same for all lanes)
    if (slot < A.kv_slots) {
      uint8_t *rec = A.kv + (int64_t)slot * kKvBytes;
#pragma unroll
      for (int f = 0; f < 2; f++) {
        const uint32_t sc = cvt_e4m3x2(0.f, __fdiv_rn(amax[f], 6.0f)) & 0xFFu;
        const float sv = e4m3_to_float(sc);
        uint32_t nib = 0u;
        if (sv != 0.f) {
          float w[8];
#pragma unroll
          for (int i = 0; i < 8; i++) w[i] = __fdiv_rn(x[8 * f + i], sv);
          nib = cvt_e2m1x8(w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
        }
        *reinterpret_cast<uint32_t *>(rec + f * 128 + lane * 4) = nib;
        if ((lane & 1) == 0) rec[256 + f * 16 + (lane >> 1)] = (uint8_t)sc;
      }
    } else if (lane == 0) {
      record_error(A.status, CSA2_ERR_BOUNDS);
    }
  }
  if (wslot >= 0) {
    if (wslot < A.swa_slots) {
      uint8_t *rec = A.swa + (int64_t)wslot * kSwaBytes;
#pragma unroll
      for (int f = 0; f < 2; f++) {
        const float am = fmaxf(amax[f], __shfl_xor_sync(0xFFFFFFFFu, amax[f], 2));   // groups of 32: four lanes
        uint32_t sb = 0u, w[2] = {0u, 0u};
        if (am > 0.f) {
          const int ex = pow2_exp_fp8(am);
          sb = (uint32_t)(ex + 127);
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const uint32_t two = cvt_e4m3x2(ldexpf(x[8 * f + 2 * i + 1], -ex), ldexpf(x[8 * f + 2 * i], -ex));
            w[i >> 1] |= two << (16 * (i & 1));
          }
        }
        *reinterpret_cast<uint2 *>(rec + f * 256 + lane * 8) = make_uint2(w[0], w[1]);
        if ((lane & 3) == 0) rec[512 + f * 8 + (lane >> 2)] = (uint8_t)sb;
      }
    } else if (lane == 0) {
      record_error(A.status, CSA2_ERR_BOUNDS);
    }
  }
}

// Grid: lat_ctas CTAs of eight latent rows (first: their rare fp64 rows take
// longest), then 8 / HPW CTAs per token of 8 HPW query heads each.  Two rows of a warp
// in flight and four CTAs an SM: of 8,192 tokens the queries take 158 us (a copy of
// their bytes 163), the latents alone 19 (their arithmetic), both together 171; four
// rows in flight, or what registers the compiler likes, took 14 and 4 us more.
template <int HPW>
__global__ void __launch_bounds__(kNormThreads, 4) qk_norm_rope_kernel(const __grid_constant__ NormArgs A) {
  __shared__ float2 cs_sh[kRopeDim / 2];
  griddep_wait();
  griddep_launch();
  if ((int)blockIdx.x >= A.lat_ctas) {
    query_rows<HPW>(A, (int)blockIdx.x - A.lat_ctas, cs_sh);
    return;
  }
  const int tok = (int)blockIdx.x * (kNormThreads / 32) + (int)(threadIdx.x >> 5);
  if (tok < A.n) latent_row(A, tok, threadIdx.x & 31);
}

cudaError_t launch_qk_norm_rope(NormArgs A, double eps, double rope_base, cudaStream_t st) {
  A.eps = eps;
  A.eps_hi = (float)eps;
  A.eps_lo = (float)(eps - (double)A.eps_hi);
  rope_turns(rope_base, A.turn);
  A.lat_ctas = A.lat != nullptr ? (A.n + kNormThreads / 32 - 1) / (kNormThreads / 32) : 0;
  // heads per warp: one CTA per token once that fills the SMs four times over
  // (a warp then has eight rows, two in flight); fewer heads per warp below that
  const int64_t want = 4 * (int64_t)device_sm_count(current_device());
  const int hpw = A.q == nullptr || A.n >= want ? 8 : 2 * (int64_t)A.n >= want ? 4 : 4 * (int64_t)A.n >= want ? 2 : 1;
  const unsigned grid = (unsigned)A.lat_ctas + (A.q != nullptr ? (unsigned)A.n * (8 / hpw) : 0u);
  const dim3 g(grid), b(kNormThreads);
  switch (hpw) {
    case 8: return launch_pdl(qk_norm_rope_kernel<8>, g, b, 0, st, 1u, A);
    case 4: return launch_pdl(qk_norm_rope_kernel<4>, g, b, 0, st, 1u, A);
    case 2: return launch_pdl(qk_norm_rope_kernel<2>, g, b, 0, st, 1u, A);
    default: return launch_pdl(qk_norm_rope_kernel<1>, g, b, 0, st, 1u, A);
  }
}

}  // namespace csa2
