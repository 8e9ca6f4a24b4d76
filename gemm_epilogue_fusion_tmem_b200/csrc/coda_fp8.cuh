// The 8-bit passes around the 8-bit GEMMs: quantisation of an activation, a
// gradient or a weight; RMSNorm with the residual and an 8-bit output, and its
// backward; the SwiGLU backward from an 8-bit checkpoint of [a | b].
//
// Numbers: a block of up to 128 values shares one fp32 scale.  With amax the
// largest magnitude in the block and c = max(amax, 2^-100),
//   S = c / fmax,   q = round_to_8_bits(x * (fmax / c)),   x ~ q * S,
// fmax = 448 (e4m3) or 57344 (e5m2): the block's largest value lands on the
// type's largest.  The floor 2^-100 keeps fmax / c finite, so an all-zero
// block has q = 0 and a positive scale.  NaNs are left out of amax and stay
// NaN in q; a block that holds an infinity has S = inf and comes back as NaN.
//
// Blocks of a stored matrix [R, C]: rows (1 x 128, S [ceil(C/128), R]),
// columns (128 x 1, S [ceil(R/128), C]) or 128 x 128 (S [ceil(R/128),
// ceil(C/128)]).  Row and column scales keep the blocked axis first: a product
// reduces over that axis, and its tile reads one contiguous line of scales per
// 128 of the reduction.
#pragma once

#include "coda_ptx.cuh"

namespace coda {

enum Fp8 : int { FP8_E4M3 = 0, FP8_E5M2 = 1 };

template <int FMT>
__host__ __device__ constexpr float fp8_max() {
  return FMT == FP8_E4M3 ? 448.f : 57344.f;
}
template <int V>
struct IntC {
  static constexpr int value = V;
};
constexpr float kFp8Tiny = 7.888609052210118e-31f;  // 2^-100

// Scale of a block and the factor its values are multiplied by, each the nearest
// fp32 number to its quotient.  The scale's divisor is a constant, so one step on
// the remainder does (P. W. Markstein, IBM J. Res. Dev. 34, 1990): with q = c times
// the rounded 1 / fmax, the remainder c - fmax q is exact and q + (c - fmax q) / fmax
// rounds to c / fmax.  All 1.9e9 fp32 numbers c from 2^-100 to infinity were compared
// with the division, for both types; q alone is another number for 55 % of them.
template <int FMT>
__device__ __forceinline__ float fp8_scale(float amax) {
  constexpr float kInv = 1.0f / fp8_max<FMT>();
  const float c = fmaxf(amax, kFp8Tiny), q = __fmul_rn(c, kInv);
  const float s = __fmaf_rn(__fmaf_rn(-fp8_max<FMT>(), q, c), kInv, q);
  return c <= 3.4028234663852886e38f ? s : q;  // infinity stays
}
template <int FMT>
__device__ __forceinline__ float fp8_factor(float amax) {
  return __fdiv_rn(fp8_max<FMT>(), fmaxf(amax, kFp8Tiny));
}

// Two floats to two 8-bit values (lo in the low byte), nearest even, saturating.
template <int FMT>
__device__ __forceinline__ uint32_t fp8_pack2(float lo, float hi) {
  uint16_t r;
  if constexpr (FMT == FP8_E4M3)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int FMT>
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  return fp8_pack2<FMT>(a, b) | (fp8_pack2<FMT>(c, d) << 16);
}
template <int FMT>
__device__ __forceinline__ uint2 fp8_pack8(const float* f, float factor) {
  return make_uint2(fp8_pack4<FMT>(f[0] * factor, f[1] * factor, f[2] * factor, f[3] * factor),
                    fp8_pack4<FMT>(f[4] * factor, f[5] * factor, f[6] * factor, f[7] * factor));
}

__device__ __forceinline__ uint2 ldg_nc_v2(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ldg_nc_u32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void stg_u32(void* p, uint32_t v) {
  asm volatile("st.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void stg_v2(void* p, const uint2& v) {
  asm volatile("st.global.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}

__device__ __forceinline__ void sts8(float* p, const float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void lds8(const float* p, float* f) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Largest of the warp's values, which are not negative (and then ordered as their bits are).
__device__ __forceinline__ float warp_max(float v) {
  uint32_t r;
  asm("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(r) : "r"(__float_as_uint(v)));
  return __uint_as_float(r);
}

// Largest of three, magnitudes of the last two.
__device__ __forceinline__ float max3_abs(float m, float a, float b) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// Two floats in one register pair: the packed operations issue once for both.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// The two e4m3 values in a word's low half (exact: e4m3 is a subset of fp16).
__device__ __forceinline__ F2 e4m3_pair(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  const float2 v = __half22float2(*reinterpret_cast<__half2*>(&h));
  return f2(v.x, v.y);
}

// Sigmoids of a pair: 1 / (1 + 2^(-x log2 e)), with the approximate exponential and
// reciprocal, since the pass is bound by its instructions: off by at most 6 + 1.2 |x|
// ulp, the latter from the rounded product x log2 e, four orders below an 8-bit step.
__device__ __forceinline__ F2 sigmoid2(F2 x) {
  float e0, e1, s0, s1;
  split(x * f2(-1.4426950408889634f, -1.4426950408889634f), e0, e1);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s0) : "f"(e0));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s1) : "f"(e1));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(1.f + s0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(1.f + s1));
  return f2(e0, e1);
}

// Makes the compiler forget what it knows of a word, so that values formed from
// it again are formed again instead of being kept.
__device__ __forceinline__ void forget(uint32_t& w) { asm volatile("" : "+r"(w)); }
__device__ __forceinline__ void forget(uint4& q) { forget(q.x), forget(q.y), forget(q.z), forget(q.w); }
__device__ __forceinline__ void forget(uint2& q) { forget(q.x), forget(q.y); }

// Largest of the 16 lanes that hold one row's 128 columns.
__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Larger of two pairs of bf16 (a NaN beside a number is left out).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 8 values times their factors, as 8-bit values.
template <int FMT>
__device__ __forceinline__ uint2 fp8_pack8(const F2 (&v)[4], const F2 (&f)[4]) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    split(v[i] * f[i], lo, hi);
    r[i] = fp8_pack2<FMT>(lo, hi);
  }
  return make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
}
template <int FMT>
__device__ __forceinline__ uint2 fp8_pack8(const uint4& q, const F2 (&f)[4]) {
  const F2 v[4] = {f2(bf16lo(q.x), bf16hi(q.x)), f2(bf16lo(q.y), bf16hi(q.y)), f2(bf16lo(q.z), bf16hi(q.z)),
                   f2(bf16lo(q.w), bf16hi(q.w))};
  return fp8_pack8<FMT>(v, f);
}

// ------------------------------------------------------------------ quantiser

// One CTA per 128 x 128 tile, read once: a thread holds 8 columns of 8 rows
// (16 threads to a row).  The pass is bound by memory as long as the warps need
// few instructions per byte: maxima are taken of the bf16 values two to a word,
// the 16 lanes of a row halve what they hold at each step, so that each lane
// ends with one row and divides once, and products are packed.  Column maxima
// meet in shared memory over the 8 warps.  With VEC the matrix is X scaled by
// rowvec (fp32, rows) and colvec (bf16, columns), which gives the column form of
// RMSNorm's output from H, r and g without storing it; its maxima are of fp32
// values, and it takes three CTAs per SM (at four the columns form spills, 24.2 us
// for 19.4 with a warm L2; rows and columns together spill 76 bytes at three).
// Measured at 8192 x 4096 with a cold L2: rows 18.6 us (5.4 TB/s), rows and columns
// 24.8 (5.4), columns of H r g 23.2 (4.3), both of H r g 38.5; blocks of 22016 x
// 4096 42.5 us (6.4).
constexpr int kQuantThreads = 256;
constexpr int kQuantRows = 128 * 16 / kQuantThreads;  // rows per thread

struct QuantParams {
  const __nv_bfloat16* x;
  const float* rowvec;
  const __nv_bfloat16* colvec;
  uint8_t *qr, *qc;
  float *sr, *sc;
  int R, C, tiles_c;
};

template <int FMT, bool ROWS, bool COLS, bool BLOCKS, bool VEC>
__global__ void __launch_bounds__(kQuantThreads, VEC ? 3 : 4) quant_fp8_kernel(const QuantParams p) {
  __shared__ __align__(16) float smax[kQuantThreads / 32][128];
  __shared__ __align__(16) float sfac[128];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int tr = blockIdx.x / p.tiles_c, tc = blockIdx.x - tr * p.tiles_c;
  const int c0 = tc * 128 + (lane % 16) * 8;
  const int r0 = tr * 128 + warp * 2 + lane / 16;  // then + 16 per step
  const bool cv = c0 < p.C;
  // The tile's first row, and this thread's 32-bit offset from it.
  const size_t t0 = (size_t)tr * 128 * p.C;
  const uint32_t o0 = (uint32_t)(r0 - tr * 128) * p.C + c0;
  uint4 x[kQuantRows];
#pragma unroll
  for (int i = 0; i < kQuantRows; ++i) {
    const int row = r0 + 16 * i;
    x[i] = (cv && row < p.R) ? ldg_nc_v4(p.x + t0 + (o0 + (uint32_t)(16 * i) * p.C)) : make_uint4(0u, 0u, 0u, 0u);
  }
  // Without VEC the maxima are taken of the bf16 values, two to a word.
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  uint32_t cm[4] = {0u, 0u, 0u, 0u};  // columns, then the tile
  if constexpr (!VEC) {
    uint32_t rm[kQuantRows];
#pragma unroll
    for (int i = 0; i < kQuantRows; ++i) {
      const uint32_t w[4] = {x[i].x & kAbs, x[i].y & kAbs, x[i].z & kAbs, x[i].w & kAbs};
      if constexpr (COLS || BLOCKS) {
#pragma unroll
        for (int j = 0; j < 4; ++j) cm[j] = max_bf16x2(cm[j], w[j]);
      }
      if constexpr (ROWS) rm[i] = max_bf16x2(max_bf16x2(max_bf16x2(0u, w[0]), w[1]), max_bf16x2(max_bf16x2(0u, w[2]), w[3]));
    }
    if constexpr (ROWS) {
      // Rows 2 t and 2 t + 1 to word t; then the 16 lanes halve what they hold:
      // lane l ends with word l / 4, and takes the row l % 2 of it.
      static_assert(kQuantRows == 8, "8 rows over 16 lanes");
      uint32_t m[4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
        m[t] = max_bf16x2(__byte_perm(rm[2 * t], rm[2 * t + 1], 0x5410), __byte_perm(rm[2 * t], rm[2 * t + 1], 0x7632));
      const bool up8 = lane & 8, up4 = lane & 4;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up8 ? m[t] : m[t + 2], 8);
        m[t] = max_bf16x2(up8 ? m[t + 2] : m[t], got);
      }
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up4 ? m[0] : m[1], 4);
      uint32_t w = max_bf16x2(up4 ? m[1] : m[0], got);
      w = max_bf16x2(w, __shfl_xor_sync(0xffffffffu, w, 2));
      w = max_bf16x2(w, __shfl_xor_sync(0xffffffffu, w, 1));
      const float amax = lane & 1 ? bf16hi(w) : bf16lo(w);
      const int mine = r0 + 16 * (lane % 16 / 4 * 2 + (lane & 1));
      if (!(lane & 2) && mine < p.R) p.sr[(size_t)tc * p.R + mine] = fp8_scale<FMT>(amax);
      const float factor = fp8_factor<FMT>(amax);
#pragma unroll
      for (int i = 0; i < kQuantRows; ++i) {
        const float fr = __shfl_sync(0xffffffffu, factor, (lane & 16) | (i / 2 * 4) | (i & 1));
        const F2 f[4] = {f2(fr, fr), f2(fr, fr), f2(fr, fr), f2(fr, fr)};
        if (cv && r0 + 16 * i < p.R) stg_v2(p.qr + t0 + (o0 + (uint32_t)(16 * i) * p.C), fp8_pack8<FMT>(x[i], f));
      }
    }
  }
  F2 cvec[4];
  float rvec[kQuantRows];
  if constexpr (VEC) {
    float c[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (p.colvec != nullptr && cv) unpack8(ldg_nc_v4_l1(p.colvec + c0), c);
#pragma unroll
    for (int j = 0; j < 4; ++j) cvec[j] = f2(c[2 * j], c[2 * j + 1]);
#pragma unroll
    for (int i = 0; i < kQuantRows; ++i) {
      const int row = r0 + 16 * i;
      rvec[i] = (p.rowvec != nullptr && row < p.R) ? p.rowvec[row] : 1.f;
    }
  }
  auto values = [&](int i, F2 (&f)[4]) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = f2(bf16lo(w[j]), bf16hi(w[j])) * f2(rvec[i], rvec[i]) * cvec[j];
  };
  float cmax[8];
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[j] = 0.f;
#pragma unroll
    for (int i = 0; i < kQuantRows; i += 2) {
      F2 f[2][4];
      float v[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        values(i + k, f[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) split(f[k][j], v[k][2 * j], v[k][2 * j + 1]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) cmax[j] = max3_abs(cmax[j], v[0][j], v[1][j]);
      if constexpr (ROWS) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float rmax = 0.f;
#pragma unroll
          for (int j = 0; j < 8; j += 2) rmax = max3_abs(rmax, v[k][j], v[k][j + 1]);
          rmax = max16(rmax);
          const int row = r0 + 16 * (i + k);
          if (row < p.R) {
            const float fr = fp8_factor<FMT>(rmax);
            const F2 factor[4] = {f2(fr, fr), f2(fr, fr), f2(fr, fr), f2(fr, fr)};
            if (cv) stg_v2(p.qr + t0 + (o0 + (uint32_t)(16 * (i + k)) * p.C), fp8_pack8<FMT>(f[k], factor));
            if (lane % 16 == 0) p.sr[(size_t)tc * p.R + row] = fp8_scale<FMT>(rmax);
          }
        }
      }
    }
  }
  if constexpr (COLS || BLOCKS) {
    F2 fac[4];
    if constexpr (BLOCKS) {
      uint32_t w = max_bf16x2(max_bf16x2(cm[0], cm[1]), max_bf16x2(cm[2], cm[3]));
      float m = warp_max(fmaxf(bf16lo(w), bf16hi(w)));
      if (lane == 0) smax[warp][0] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kQuantThreads / 32; ++w) m = fmaxf(m, smax[w][0]);
      if (threadIdx.x == 0) p.sc[(size_t)tr * p.tiles_c + tc] = fp8_scale<FMT>(m);
      m = fp8_factor<FMT>(m);
#pragma unroll
      for (int j = 0; j < 4; ++j) fac[j] = f2(m, m);
    } else {
      if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          cm[j] = max_bf16x2(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
          cmax[2 * j] = bf16lo(cm[j]);
          cmax[2 * j + 1] = bf16hi(cm[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) cmax[j] = fmaxf(cmax[j], __shfl_xor_sync(0xffffffffu, cmax[j], 16));
      }
      if (lane < 16) sts8(&smax[warp][lane * 8], cmax);
      __syncthreads();
      if (threadIdx.x < 128) {  // one column each: maximum, scale, factor
        float m = smax[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kQuantThreads / 32; ++w) m = fmaxf(m, smax[w][threadIdx.x]);
        sfac[threadIdx.x] = fp8_factor<FMT>(m);
        const int c = tc * 128 + threadIdx.x;
        if (c < p.C) p.sc[(size_t)tr * p.C + c] = fp8_scale<FMT>(m);
      }
      __syncthreads();
      lds8(&sfac[(lane % 16) * 8], cmax);
#pragma unroll
      for (int j = 0; j < 4; ++j) fac[j] = f2(cmax[2 * j], cmax[2 * j + 1]);
    }
#pragma unroll
    for (int i = 0; i < kQuantRows; ++i) {
      if (!cv || r0 + 16 * i >= p.R) continue;
      forget(x[i]);
      uint8_t* dst = p.qc + t0 + (o0 + (uint32_t)(16 * i) * p.C);
      if constexpr (VEC) {
        F2 f[4];
        values(i, f);
        stg_v2(dst, fp8_pack8<FMT>(f, fac));
      } else {
        stg_v2(dst, fp8_pack8<FMT>(x[i], fac));
      }
    }
  }
}

// ------------------------------------------------------------------ RMSNorm

// Sum over the block's THREADS threads, in every thread.  `scratch` holds
// THREADS / 32 floats and is free again after the next block-wide barrier.
template <int THREADS>
__device__ __forceinline__ float block_sum_all(float v, float* scratch) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x / 32] = v;
  __syncthreads();
  float t = (threadIdx.x & 31) < THREADS / 32 ? scratch[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

struct RmsParams {
  const __nv_bfloat16 *x, *res, *g;
  __nv_bfloat16* h;
  float* r;
  uint8_t* q;
  float* s;
  int M, d;
  float inv_d, eps;
};

// H = bf16(X + R); r = rsqrt(mean_j H_j^2 + eps) from the stored H;
// (Q, S) = row blocks of H r g.  One CTA per row, the row in registers (CH
// chunks of 8 columns per thread), so X and R are read once and nothing is
// read back; 16 neighbouring threads hold one scale block.  Bound by memory:
// 7 bytes per value, at 8192 x 4096 40.0 us (5.9 TB/s), at 8192 x 8192 76.5 us
// (6.1).
template <int THREADS, int CH>
__global__ void __launch_bounds__(THREADS) rmsnorm_fp8_fwd_kernel(const RmsParams p) {
  __shared__ float scratch[32];
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x;
  const size_t base = (size_t)row * p.d;
  uint4 hq[CH];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (k * THREADS + threadIdx.x) * 8;
    hq[k] = c < p.d ? ldg_nc_v4(p.x + base + c) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (p.res != nullptr) {
    uint4 rq[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * THREADS + threadIdx.x) * 8;
      rq[k] = c < p.d ? ldg_nc_v4(p.res + base + c) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * THREADS + threadIdx.x) * 8;
      float a[8], b[8];
      unpack8(hq[k], a);
      unpack8(rq[k], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] += b[i];
      hq[k] = pack8(a);
      if (c < p.d) stg_v4(p.h + base + c, hq[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    float a[8];
    unpack8(hq[k], a);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], ss);
  }
  const float r = rsqrtf(fmaf(block_sum_all<THREADS>(ss, scratch), p.inv_d, p.eps));
  if (threadIdx.x == 0) p.r[row] = r;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (k * THREADS + threadIdx.x) * 8;
    const bool v = c < p.d;
    float a[8], g[8];
    unpack8(hq[k], a);
    unpack8(v ? ldg_nc_v4_l1(p.g + c) : make_uint4(0u, 0u, 0u, 0u), g);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = a[i] * r * g[i];
      m = fmaxf(m, fabsf(a[i]));
    }
    m = max16(m);
    if (v) {
      stg_v2(p.q + base + c, fp8_pack8<FP8_E4M3>(a, fp8_factor<FP8_E4M3>(m)));
      if (threadIdx.x % 16 == 0) p.s[(size_t)(c / 128) * p.M + row] = fp8_scale<FP8_E4M3>(m);
    }
  }
}

struct RmsBwdParams {
  const __nv_bfloat16 *dn, *h, *g, *dh_in;
  const float* r;
  __nv_bfloat16* dh;
  float* part;  // [gridDim.x][d] partial sums of dg
  int M, d;
  float inv_d;
};

// u = dN g;  dH = r u - H r^3 mean_j(u_j H_j) (+ dH_in);  dg partials: each CTA
// takes every gridDim.x-th row and keeps sum_i dN_i H_i r_i of its columns in
// registers, so one pass reads everything once; rmsnorm_fp8_dg_kernel adds the
// CTAs' partials in a fixed order.  8 bytes per value: 8192 x 4096 with dH_in
// 51 us (5.2 TB/s) with the reduce (a cold L2); each row's block-wide sum, during which only
// the next row's loads are in flight, is what keeps it from the copy rate.
template <int THREADS, int CH>
__global__ void __launch_bounds__(THREADS) rmsnorm_fp8_bwd_kernel(const RmsBwdParams p) {
  __shared__ float scratch[2][32];
  griddep_wait();
  griddep_launch_dependents();
  float dg[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[k][i] = 0.f;
  // The next row's loads are issued before this row's reduction, where registers allow.
  constexpr bool AHEAD = CH == 1;
  uint4 nq[CH], hq[CH], eq[CH];
  float r = 0.f;
  auto load = [&](int row) {
    const size_t base = (size_t)row * p.d;
    r = p.r[row];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * THREADS + threadIdx.x) * 8;
      const bool v = c < p.d;
      nq[k] = v ? ldg_nc_v4(p.dn + base + c) : make_uint4(0u, 0u, 0u, 0u);
      hq[k] = v ? ldg_nc_v4(p.h + base + c) : make_uint4(0u, 0u, 0u, 0u);
      eq[k] = v && p.dh_in != nullptr ? ldg_nc_v4(p.dh_in + base + c) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  int row = blockIdx.x, parity = 0;
  if (AHEAD && row < p.M) load(row);
  for (; row < p.M; parity ^= 1) {
    float s = 0.f;
    if (!AHEAD) load(row);
    uint4 n0[CH], h0[CH], e0[CH];
    const float r0 = r;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      n0[k] = nq[k];
      h0[k] = hq[k];
      e0[k] = eq[k];
    }
    const size_t base = (size_t)row * p.d;
    row += gridDim.x;
    if (AHEAD && row < p.M) load(row);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * THREADS + threadIdx.x) * 8;
      float n[8], h[8], g[8];
      unpack8(n0[k], n);
      unpack8(h0[k], h);
      unpack8(c < p.d ? ldg_nc_v4_l1(p.g + c) : make_uint4(0u, 0u, 0u, 0u), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float nh = n[i] * h[i];
        s = fmaf(nh, g[i], s);
        dg[k][i] = fmaf(nh, r0, dg[k][i]);
      }
    }
    // Two scratch rows in turn: a thread may still read one while another starts the next row.
    const float coef = block_sum_all<THREADS>(s, scratch[parity]) * p.inv_d * r0 * r0 * r0;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * THREADS + threadIdx.x) * 8;
      if (c >= p.d) continue;
      float n[8], h[8], g[8], e[8];
      unpack8(n0[k], n);
      unpack8(h0[k], h);
      unpack8(e0[k], e);
      unpack8(ldg_nc_v4_l1(p.g + c), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = fmaf(n[i] * g[i], r0, fmaf(-coef, h[i], e[i]));
      stg_v4(p.dh + base + c, pack8(n));
    }
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (k * THREADS + threadIdx.x) * 8;
    if (c >= p.d) continue;
    float* o = p.part + (size_t)blockIdx.x * p.d + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = dg[k][i];
  }
}

// dg_j = sum of the CTAs' partials, 32 columns to a block: warp w adds rows w,
// w + 32, ..., all in flight together, and the 32 sums are added in warp order.
constexpr int kRmsDgThreads = 1024;
__global__ void __launch_bounds__(kRmsDgThreads)
    rmsnorm_fp8_dg_kernel(const float* __restrict__ part, int rows, int d, float* __restrict__ dg) {
  __shared__ float sums[32][33];
  griddep_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int j = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (j < d) {
#pragma unroll 8
    for (int t = warp; t < rows; t += 32) s += part[(size_t)t * d + j];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && j < d) {
    float tot = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) tot += sums[w][lane];
    dg[j] = tot;
  }
}

// ------------------------------------------------------------------ SwiGLU backward from the 8-bit checkpoint

// With s = sigmoid(a), u = a s: da = dY b (s + u (1 - s)), db = dY u, y = u b.
// One CTA per 128 tokens x 128 columns.  A warp holds 8 whole rows, a lane 4
// columns of each (dY bf16; a, b e4m3 with one scale per row and 128 columns),
// so row maxima are one warp reduction and column
// maxima stay in the lane until the warps meet in shared memory.  The gradients
// are formed twice, once for the maxima and once to be rounded: keeping them
// would take 96 registers and half the warps.  Outputs: dA = [da | db] in row
// blocks (operand of dgrad) and, with COLS, dA and y in column blocks (operands
// of the two weight gradients).  Measured at 8190 x 11008: with COLS 200 us (4.1
// TB/s; 64 registers, 44 to 52 bytes spilled), e5m2 alike, without 143 us (3.8).
// It is bound by its instructions, some 57 per element of which two
// exponentials and two reciprocals: the schedulers issue in 73% of the clocks,
// the special-function unit is 43% busy, DRAM 48%.
constexpr int kSwBwdThreads = 512;
constexpr int kSwBwdWarps = kSwBwdThreads / 32;
constexpr int kSwBwdRows = 128 / kSwBwdWarps;  // rows per warp

struct SwigluBwd8Params {
  const __nv_bfloat16* dy;
  const uint8_t* ab;
  const float* sab;
  uint8_t *da, *dac, *yc;
  float *sda, *sdac, *syc;
  int M, F;
};

template <int FMT, bool COLS>
__global__ void __launch_bounds__(kSwBwdThreads, 1024 / kSwBwdThreads) swiglu_fp8_bwd_kernel(const SwigluBwd8Params p) {
  __shared__ __align__(16) float smax[COLS ? kSwBwdWarps : 1][3][128];
  __shared__ __align__(16) float sfac[3][128];
  __shared__ __align__(16) float srow[128][4];  // per row: scales of a and b, factors of da and db
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int fb = p.F / 128;
  const int tr = blockIdx.x / fb, tc = blockIdx.x - tr * fb;
  const int r0 = tr * 128 + warp * kSwBwdRows;
  // The tile's origin in [M, F] (of 2-byte dY and 1-byte y) and in [M, 2F], and
  // this lane's 32-bit offsets in it.
  const size_t t1 = (size_t)tr * 128 * p.F + tc * 128, t2 = (size_t)tr * 256 * p.F + tc * 128;
  const uint32_t o1 = (uint32_t)(warp * kSwBwdRows) * p.F + lane * 4, o2 = (uint32_t)(warp * kSwBwdRows) * 2 * p.F + lane * 4;
  uint2 dyq[kSwBwdRows];
  uint32_t aq[kSwBwdRows], bq[kSwBwdRows];
#pragma unroll
  for (int i = 0; i < kSwBwdRows; ++i) {
    const int row = r0 + i;
    dyq[i] = make_uint2(0u, 0u);
    aq[i] = bq[i] = 0u;
    if (row < p.M) {
      dyq[i] = ldg_nc_v2(p.dy + t1 + (o1 + (uint32_t)i * p.F));
      aq[i] = ldg_nc_u32(p.ab + t2 + (o2 + (uint32_t)i * 2 * p.F));
      bq[i] = ldg_nc_u32(p.ab + t2 + p.F + (o2 + (uint32_t)i * 2 * p.F));
    }
  }
  // Lanes 0-7 fetch the rows' scales of a, lanes 8-15 those of b.
  const int sr = r0 + lane % kSwBwdRows, half = lane / kSwBwdRows;
  if (half < 2) srow[warp * kSwBwdRows + lane % kSwBwdRows][half] = sr < p.M ? p.sab[(size_t)(half * fb + tc) * p.M + sr] : 0.f;
  __syncwarp();
  // da, db, y of two columns (pair k) of the warp's row i.
  auto grads = [&](int i, int k, F2& da, F2& db, F2& y) {
    const float2 sc = *reinterpret_cast<const float2*>(srow[warp * kSwBwdRows + i]);
    const uint32_t w = k ? dyq[i].y : dyq[i].x;
    const F2 dy = f2(bf16lo(w), bf16hi(w));
    const F2 a = e4m3_pair(aq[i] >> (16 * k)) * f2(sc.x, sc.x), b = e4m3_pair(bq[i] >> (16 * k)) * f2(sc.y, sc.y);
    const F2 sg = sigmoid2(a);
    const F2 u = a * sg;
    da = dy * b * fma2(u, fma2(sg, f2(-1.f, -1.f), f2(1.f, 1.f)), sg);
    db = dy * u;
    y = u * b;
  };
  float cmax[3][4];
#pragma unroll
  for (int t = 0; t < 3; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) cmax[t][j] = 0.f;
  float mine = 0.f;  // lane i: row i's maximum of da, lane kSwBwdRows + i: of db
#pragma unroll
  for (int i = 0; i < kSwBwdRows; ++i) {
    float ma = 0.f, mb = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      F2 g[3];
      grads(i, k, g[0], g[1], g[2]);
      float x0, x1;
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        split(g[t], x0, x1);
        if (t == 0) ma = max3_abs(ma, x0, x1);
        if (t == 1) mb = max3_abs(mb, x0, x1);
        if constexpr (COLS) {
          cmax[t][2 * k] = fmaxf(cmax[t][2 * k], fabsf(x0));
          cmax[t][2 * k + 1] = fmaxf(cmax[t][2 * k + 1], fabsf(x1));
        }
      }
    }
    ma = warp_max(ma);
    mb = warp_max(mb);
    if (lane == i) mine = ma;
    if (lane == kSwBwdRows + i) mine = mb;
  }
  if (half < 2) {
    srow[warp * kSwBwdRows + lane % kSwBwdRows][2 + half] = fp8_factor<FMT>(mine);
    if (sr < p.M) p.sda[(size_t)(half * fb + tc) * p.M + sr] = fp8_scale<FMT>(mine);
  }
  __syncwarp();
  if constexpr (COLS) {
#pragma unroll
    for (int t = 0; t < 3; ++t)
      *reinterpret_cast<float4*>(&smax[warp][t][lane * 4]) = make_float4(cmax[t][0], cmax[t][1], cmax[t][2], cmax[t][3]);
    __syncthreads();
    if (threadIdx.x < 3 * 128) {
      const int t = threadIdx.x / 128, c = threadIdx.x % 128;
      float m = smax[0][t][c];
#pragma unroll
      for (int w = 1; w < kSwBwdWarps; ++w) m = fmaxf(m, smax[w][t][c]);
      if (t == 2) {
        sfac[t][c] = fp8_factor<FP8_E4M3>(m);
        p.syc[(size_t)tr * p.F + tc * 128 + c] = fp8_scale<FP8_E4M3>(m);
      } else {
        sfac[t][c] = fp8_factor<FMT>(m);
        p.sdac[(size_t)tr * 2 * p.F + (size_t)t * p.F + tc * 128 + c] = fp8_scale<FMT>(m);
      }
    }
    __syncthreads();
  }
  {
#pragma unroll
    for (int i = 0; i < kSwBwdRows; ++i) {
      const int row = r0 + i;
      if (row >= p.M) break;
      forget(dyq[i]);
      forget(aq[i]);
      forget(bq[i]);
      const float2 fr = *reinterpret_cast<const float2*>(&srow[warp * kSwBwdRows + i][2]);
      uint32_t q[5] = {0u, 0u, 0u, 0u, 0u};  // da and db by rows; da, db and y by columns
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        F2 da, db, y;
        grads(i, k, da, db, y);
        auto put = [&](uint32_t& w, F2 x, auto fmt) {
          float lo, hi;
          split(x, lo, hi);
          w |= fp8_pack2<decltype(fmt)::value>(lo, hi) << (16 * k);
        };
        put(q[0], da * f2(fr.x, fr.x), IntC<FMT>());
        put(q[1], db * f2(fr.y, fr.y), IntC<FMT>());
        if constexpr (COLS) {
          put(q[2], da * F2{*reinterpret_cast<const uint64_t*>(&sfac[0][lane * 4 + 2 * k])}, IntC<FMT>());
          put(q[3], db * F2{*reinterpret_cast<const uint64_t*>(&sfac[1][lane * 4 + 2 * k])}, IntC<FMT>());
          put(q[4], y * F2{*reinterpret_cast<const uint64_t*>(&sfac[2][lane * 4 + 2 * k])}, IntC<FP8_E4M3>());
        }
      }
      const uint32_t o = o2 + (uint32_t)i * 2 * p.F;
      stg_u32(p.da + t2 + o, q[0]);
      stg_u32(p.da + t2 + p.F + o, q[1]);
      if constexpr (COLS) {
        stg_u32(p.dac + t2 + o, q[2]);
        stg_u32(p.dac + t2 + p.F + o, q[3]);
        stg_u32(p.yc + t1 + (o1 + (uint32_t)i * p.F), q[4]);
      }
    }
  }
}

}  // namespace coda
