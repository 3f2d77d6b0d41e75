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

inline bool aligned_to(const void* p, uintptr_t n) {
  return reinterpret_cast<uintptr_t>(p) % n == 0;
}
inline bool aligned16(const void* p) { return aligned_to(p, 16); }

// i / d = umulhi(i, mul) >> shift for i < 2^31: mul = ceil(2^(32 + shift) / d) with
// 2^shift < d <= 2^(shift + 1); d = 1 gives shift -1, and i itself.
inline void fast_divisor(int d, uint32_t* mul, int* shift) {
  *mul = 0;
  *shift = -1;
  if (d == 1) return;
  int s = 0;
  while ((2LL << s) < d) ++s;
  *shift = s;
  *mul = static_cast<uint32_t>(((1ull << (32 + s)) + d - 1) / d);
}

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
// Exponent e of the smallest power of two at or above fl32(amax / TOP), TOP = 6
// or 448; 0 for amax = 0 (and for an infinite or NaN one, whose codes
// saturate).  With TOP = c 2^t and amax = m 2^k, 1 <= c, m < 2, that is k - t
// for m <= c and one more above it: the next float after c 2^k is far enough
// away (a third of its ulp at least) for fl32 not to round it down to 2^(k - t).
template <int TOP>
__device__ __forceinline__ int scale_exp(float amax) {
  static_assert(TOP == 6 || TOP == 448, "1.5 * 2^2 or 1.75 * 2^8");
  constexpr uint32_t kMant = TOP == 6 ? 0x400000u : 0x600000u;
  constexpr int kExp = TOP == 6 ? 2 : 8;
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>((b + (0x7fffffu - kMant)) >> 23) - 127 - kExp;
  return b - 1u < 0x7f7fffffu ? max(e, -126) : 0;   // 0 < amax < infinity
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

// ---------------------------------------------------------------- pairs
// Two fp32 operations in one instruction.
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 fma2(const F2& a, const F2& b, const F2& c) {
  F2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ F2 add2(const F2& a, const F2& b) {
  F2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 mul2(const F2& a, const F2& b) {
  F2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 both(float v) { return F2{v, v}; }

// e4m3(f * inv), nearest even, saturating at +-448
__device__ __forceinline__ uint2 pack8_e4m3(const float* f, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const F2 v = mul2(F2{f[2 * q], f[2 * q + 1]}, both(inv));
    w[q] = __nv_cvt_float2_to_fp8x2(make_float2(v.x, v.y), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}
// e2m1(f * inv), nearest even, saturating at +-6; value 2i in the low half of byte i
__device__ __forceinline__ uint32_t pack8_e2m1(const float* f, float inv) {
  F2 v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = mul2(F2{f[2 * q], f[2 * q + 1]}, both(inv));
  uint32_t out;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
      : "=r"(out)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x),
        "f"(v[3].y));
  return out;
}

// ---------------------------------------------------------------- norms
// A sum of squares as an unevaluated pair hi + lo: the codes of values next to
// a rounding border, and a scale next to a power of two, hang on the last bit
// of r, so the sum must not depend on its order.
struct SumSq {
  float hi = 0.0f, lo = 0.0f;

  // (hi, lo) += (p, e): the exact sum of hi and p, its error into lo
  __device__ __forceinline__ void merge(float p, float e) {
    const float t = __fadd_rn(hi, p);
    const float b = __fsub_rn(t, hi);
    const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(p, b));
    hi = t;
    lo = __fadd_rn(lo, __fadd_rn(err, e));
  }

  // The squares of N values in each of G neighbouring lanes (all 32 lanes call
  // it).  A power of two C above their sum, known from the largest value, is
  // put under the running sum s: then every s + x^2 is rounded at one place,
  // the rounding is t = (s + x^2) - s exactly, and x^2 - t, from one fma, is
  // what was rounded off.  The parts kept are multiples of that place below C
  // and add up exactly in any order; those rounded off are 2^-24 of C or less
  // and are summed apart.  (Four operations a value, in pairs, where an exact
  // addition without C takes eight.)
  template <int N, int G>
  __device__ __forceinline__ void sum(const float* x) {
    sum_below<N, G>(x, largest<N, G>(x), 1.0f);
  }
  // the largest magnitude of them
  template <int N, int G>
  __device__ static __forceinline__ float largest(const float* x) {
    float m[4] = {fabsf(x[0]), fabsf(x[1]), fabsf(x[2]), fabsf(x[3])};
#pragma unroll
    for (int i = 4; i < N; ++i) m[i & 3] = fmaxf(m[i & 3], fabsf(x[i]));
    const float mx = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    if (G == 32) return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
    return group_max<G>(mx);
  }
  // sum() of the values times f, none of whose products is above mx
  template <int N, int G>
  __device__ __forceinline__ void sum_below(const float* x, float mx, float f) {
    constexpr int kLog = N * G <= 64 ? 6 : N * G <= 128 ? 7 : N * G <= 256 ? 8 : N * G <= 512 ? 9 : 10;
    static_assert(N * G <= 1024 && N % 2 == 0 && N >= 4, "values of one sum");
    const int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;   // mx < 2^(e + 1)
    const float c = exp2i(min(max(2 * e + 2 + kLog, -100), 126));
    F2 s = both(0.5f * c), l = both(0.0f);   // two running sums, each below half of it
    const F2 neg = both(-1.0f);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const F2 v{x[i] * f, x[i + 1] * f};
      const F2 u = fma2(v, v, s);
      const F2 t = fma2(s, neg, u);
      const F2 r = fma2(v, v, mul2(t, neg));
      l = add2(l, r);
      s = u;
    }
    hi = __fadd_rn(__fsub_rn(s.x, 0.5f * c), __fsub_rn(s.y, 0.5f * c));
    lo = __fadd_rn(l.x, l.y);
#pragma unroll
    for (int o = 1; o < G; o <<= 1) {
      hi = __fadd_rn(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = __fadd_rn(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
  }
  // 1 / sqrt((hi + lo) / n + eps), 1 / n given as a pair too: the hardware's
  // reciprocal root, then one Newton step whose residual 1 - m r^2 is formed
  // from exact products, so the result is the rounded root but for a few of
  // 2^20 cases.  m is mean + eps: between 2^-60 and 2^100 (near) that holds for
  // sum()'s result, as no square came near fp32's end and none that counts was
  // rounded as a subnormal.  Other rows take far_root.
  __device__ __forceinline__ float rsqrt_mean(float2 inv_n, float eps, float* m) const {
    const float q = __fmul_rn(hi, inv_n.x);
    float ml = __fmaf_rn(lo, inv_n.x, __fmaf_rn(hi, inv_n.y, __fmaf_rn(hi, inv_n.x, -q)));
    const float mh = __fadd_rn(q, eps);
    const float b = __fsub_rn(mh, q);
    ml = __fadd_rn(ml, __fadd_rn(__fsub_rn(q, __fsub_rn(mh, b)), __fsub_rn(eps, b)));
    float r0;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(mh));
    const float r2 = __fmul_rn(r0, r0);
    const float r2e = __fmaf_rn(r0, r0, -r2);
    const float t = __fmul_rn(mh, r2);
    const float te = __fmaf_rn(mh, r2, -t);
    const float res = __fsub_rn(__fsub_rn(__fsub_rn(__fsub_rn(1.0f, t), te), __fmul_rn(mh, r2e)),
                                __fmul_rn(ml, r2));
    *m = mh;
    return __fmaf_rn(__fmul_rn(0.5f, r0), res, r0);
  }
  __device__ static __forceinline__ bool near(float m) { return m >= 0x1p-60f && m < 0x1p100f; }
};

// r of rows whose mean of squares is far from 1 (or of a warp with such a row), the
// long way: the sum is of 2^-80 or 2^80 times the values where the row's largest is
// outside 2^+-40, so it stays below 2^111, and its mean above 2^-121.  Values of a
// small row are multiplied themselves, as their r may be past fp32's range.  A row
// with an infinity has r = 0, one with a NaN r = NaN.  TPR threads share a row; above
// a warp they all come here, or none, and part is one place a warp of the block.
template <int N, int TPR>
__device__ __forceinline__ float far_root(float* x, float2 inv_n, float eps, float2* part) {
  constexpr int kWarps = TPR / 32;
  const int w = threadIdx.x >> 5, row = threadIdx.x / TPR;
  // (barriers by number: one named by a register takes all sixteen of a CTA, and
  // 32768 x 1024 then 28.8 us instead of 26.6)
  auto meet = [&] {
    if (TPR > 128 || (TPR > 32 && row == 0)) asm volatile("bar.sync 1, %0;" ::"n"(TPR) : "memory");
    else if (TPR > 64 || (TPR > 32 && row == 1)) asm volatile("bar.sync 2, %0;" ::"n"(TPR) : "memory");
    else if (TPR > 32 && row == 2) asm volatile("bar.sync 3, %0;" ::"n"(TPR) : "memory");
    else if (TPR > 32) asm volatile("bar.sync 4, %0;" ::"n"(TPR) : "memory");
  };
  float mx = SumSq::largest<N, (TPR < 32 ? TPR : 32)>(x);
  if (TPR > 32) {
    meet();
    part[w].x = mx;
    meet();
    for (int q = 0; q < kWarps; ++q) mx = fmaxf(mx, part[row * kWarps + q].x);
    meet();
  }
  const int pow2 = mx >= 0x1p41f ? -80 : mx < 0x1p-40f && eps < 0x1p-60f ? 80 : 0;
  const float f = exp2i(pow2);
  if (pow2 > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= f;
  }
  SumSq s;
  s.sum_below<N, (TPR < 32 ? TPR : 32)>(x, mx * f, pow2 > 0 ? 1.0f : f);
  if (TPR > 32) {
    part[w] = make_float2(s.hi, s.lo);
    meet();
    s = SumSq();
    for (int q = 0; q < kWarps; ++q) s.merge(part[row * kWarps + q].x, part[row * kWarps + q].y);
  }
  float m;
  float r = s.rsqrt_mean(inv_n, eps * f * f, &m);
  if (m == 0.0f || m == INFINITY) r = rsqrtf(m);   // 1 / 0 and 1 / inf have no residual
  return pow2 < 0 ? r * f : r;
}

}  // namespace ess
