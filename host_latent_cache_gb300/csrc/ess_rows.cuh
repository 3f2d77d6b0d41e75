// Row formats of the device row cache: sizes, scales, codes, and the sums
// behind the norms.
#pragma once

#include "ess_device.cuh"

namespace ess {

// exponents of a q4 block scale: with these every value is exact in fp16
// (0.5 * 2^-23 is its smallest subnormal, 6 * 2^13 is below its largest value)
constexpr int kQ4MinExp = -23;
constexpr int kQ4MaxExp = 13;
constexpr int kQ4RowBytes = 400;

__host__ __device__ constexpr int row_bytes_of(int format) {
  return format == ESS_ROW_BF16 ? kRowBytes : format == ESS_ROW_COMPACT ? 656 : kQ4RowBytes;
}

__device__ __forceinline__ float bf16_lo(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t bits) {
  return __uint_as_float(bits & 0xffff0000u);
}
__device__ __forceinline__ uint32_t bf16_bits(float f) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(f)));
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  f[0] = bf16_lo(u.x);
  f[1] = bf16_hi(u.x);
  f[2] = bf16_lo(u.y);
  f[3] = bf16_hi(u.y);
  f[4] = bf16_lo(u.z);
  f[5] = bf16_hi(u.z);
  f[6] = bf16_lo(u.w);
  f[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint4 pack8_bf16(const float* f) {
  return make_uint4(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]), bf16x2_bits(f[4], f[5]),
                    bf16x2_bits(f[6], f[7]));
}

__device__ __forceinline__ float amax8(const float* f) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
  return m;
}
// maximum over aligned groups of N lanes (all 32 lanes call it)
template <int N>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = 1; o < N; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float exp2i(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// Exponent of the smallest power of two at or above fl32(amax / top), kept
// within -126..126; 0 for amax = 0 (and for an infinite or NaN one, whose
// codes saturate).
__device__ __forceinline__ int scale_exp(float amax, float top) {
  if (!(amax > 0.0f) || amax > 3.402823466e38f) return 0;
  const uint32_t q = __float_as_uint(__fdiv_rn(amax, top));
  const int e = static_cast<int>(q >> 23) - 127 + ((q & 0x7fffffu) ? 1 : 0);
  return min(max(e, -126), 126);
}

// e4m3(f * inv), nearest even, saturating at +-448
__device__ __forceinline__ uint2 pack8_e4m3(const float* f, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    w[q] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * q] * inv, f[2 * q + 1] * inv),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}
// e2m1(f * inv), nearest even, saturating at +-6; value 2i in the low half of byte i
__device__ __forceinline__ uint32_t pack8_e2m1(const float* f, float inv) {
  uint32_t out;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
      : "=r"(out)
      : "f"(f[0] * inv), "f"(f[1] * inv), "f"(f[2] * inv), "f"(f[3] * inv), "f"(f[4] * inv),
        "f"(f[5] * inv), "f"(f[6] * inv), "f"(f[7] * inv));
  return out;
}

// eight e2m1 codes as four pairs of fp16 values (exact)
__device__ __forceinline__ void e2m1_to_f16x2(uint32_t codes, uint32_t* h) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

// The exponent byte of a q4 block, within the format's range.
__device__ __forceinline__ int q4_exp_byte(int byte) {
  return min(max(byte, kQ4MinExp + 127), kQ4MaxExp + 127);
}

// fp16 pairs that hold e2m1 values times 2^(byte - 127), as bf16 pairs.  An
// fp16 pattern shifted right by three is the bf16 pattern of 2^-112 times its
// value (neither format's exponent is zero here but for the value zero); the
// product with 2^(112 + e) is exact.
__device__ __forceinline__ uint32_t q4_bf16x2(uint32_t h, uint32_t scale2) {
  const uint32_t t = (h & 0x80008000u) | ((h >> 3) & 0x0fff0fffu);
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&t),
                                   *reinterpret_cast<const __nv_bfloat162*>(&scale2));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// scale2 of q4_bf16x2 for a clamped exponent byte
__device__ __forceinline__ uint32_t q4_bf16_scale(int byte) {
  return static_cast<uint32_t>(byte + 112) * 0x00800080u;
}

__device__ __forceinline__ uint4 widen8_e2m1(uint32_t codes, int byte) {
  uint32_t h[4];
  e2m1_to_f16x2(codes, h);
  const uint32_t s2 = q4_bf16_scale(q4_exp_byte(byte));
  return make_uint4(q4_bf16x2(h[0], s2), q4_bf16x2(h[1], s2), q4_bf16x2(h[2], s2),
                    q4_bf16x2(h[3], s2));
}
// eight e4m3 codes times a power of two as bf16 (exact)
__device__ __forceinline__ uint4 widen8_e4m3(const uint2& c, float scale) {
  const uint32_t w[2] = {c.x, c.y};
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __nv_fp8x2_storage_t p =
        static_cast<__nv_fp8x2_storage_t>((w[q >> 1] >> (16 * (q & 1))) & 0xffffu);
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(p, __NV_E4M3);
    const float2 f = __half22float2(__half2(hr));
    o[q] = bf16x2_bits(f.x * scale, f.y * scale);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A sum of squares as an unevaluated pair hi + lo (about 48 bits): the codes
// of values next to a rounding border, and a scale next to a power of two,
// hang on the last bit of r, so the sum must not depend on its order.
struct SumSq {
  float hi = 0.0f, lo = 0.0f;

  __device__ __forceinline__ void add(float x) {
    const float p = __fmul_rn(x, x);
    merge(p, __fmaf_rn(x, x, -p));
  }
  // (hi, lo) += (p, e): the exact sum of hi and p, its error into lo
  __device__ __forceinline__ void merge(float p, float e) {
    const float t = __fadd_rn(hi, p);
    const float b = __fsub_rn(t, hi);
    const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(p, b));
    hi = t;
    lo = __fadd_rn(lo, __fadd_rn(err, e));
  }
  // over aligned groups of N lanes (all 32 lanes call it)
  template <int N>
  __device__ __forceinline__ void warp_reduce() {
#pragma unroll
    for (int o = 1; o < N; o <<= 1) {
      const float p = __shfl_xor_sync(0xffffffffu, hi, o);
      const float e = __shfl_xor_sync(0xffffffffu, lo, o);
      merge(p, e);
    }
  }
  // 1 / sqrt((hi + lo) / n + eps): the hardware's reciprocal root, then one
  // Newton step whose residual 1 - m r^2 is formed from exact products, so
  // the result is the rounded root up to a few in 2^20 cases.
  __device__ __forceinline__ float rsqrt_mean(int n, float eps) const {
    const float d = static_cast<float>(n);
    const float q = __fdiv_rn(hi, d);
    const float rem = __fadd_rn(__fmaf_rn(-q, d, hi), lo);
    float ml = __fdiv_rn(rem, d);
    const float mh = __fadd_rn(q, eps);
    const float b = __fsub_rn(mh, q);
    ml = __fadd_rn(ml, __fadd_rn(__fsub_rn(q, __fsub_rn(mh, b)), __fsub_rn(eps, b)));
    const float r0 = rsqrtf(mh);
    const float r2 = __fmul_rn(r0, r0);
    const float r2e = __fmaf_rn(r0, r0, -r2);
    const float t = __fmul_rn(mh, r2);
    const float te = __fmaf_rn(mh, r2, -t);
    const float res = __fsub_rn(__fsub_rn(__fsub_rn(__fsub_rn(1.0f, t), te), __fmul_rn(mh, r2e)),
                                __fmul_rn(ml, r2));
    const float r = __fmaf_rn(__fmul_rn(0.5f, r0), res, r0);
    // a mean of zero (or one past fp32's range) has no residual: 1 / 0 and 1 / inf as they are
    return (mh > 0.0f && mh < 3.0e38f) ? r : r0;
  }
};

}  // namespace ess
