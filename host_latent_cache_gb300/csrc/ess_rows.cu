// Device row cache: writing raw token rows into a paged cache (norm, rotation,
// encoding), reading cache rows back as bf16, and the 8-bit norm that makes
// indexer keys.  All three stream rows once, so HBM is their floor; the writes
// and short norms are bound by their arithmetic.
//
// One warp per cache row.  Lane l holds the 16-byte units l and 32 + l of the
// 512 latents (dims 8l .. 8l + 7 and 256 + 8l ..), so every load and store
// instruction of a warp covers consecutive bytes whatever the format: 16, 8 or
// 4 bytes a lane for bf16, e4m3 and e2m1.
//
// Measured (bytes that the call cannot do without / time): 131072 q4 rows read
// 33.7 us (6.07 TB/s, 89 % of the measured copy rate); 65536 q4 rows written
// 27.0 us (3.80 TB/s), without norm and rotation 21.3, as compact rows 28.1, as
// bf16 rows 29.0 (a plain copy of the same bytes takes 23.9); the norm of
// 16384 x 4096 with a residual 87.3 us (5.38 TB/s), of 131072 keys 12.6 us
// (4.04 TB/s).
#include <algorithm>
#include <cmath>

#include "ess_rows.cuh"

namespace ess {
namespace {

constexpr int kRowWarps = 8;          // rows in flight per CTA
constexpr int kWriteCtas = 152 * 3;   // writing CTAs at most: one wave

struct RopeFreq {
  // turns per position as a binary fraction of 2^64: position * fraction
  // modulo 2^64 is the angle, off by the fraction's own error times the
  // position (2^-33 of a turn at 2^31), with no range reduction
  unsigned long long f[32];
};

// x modulo 1 as a binary fraction of 2^64
unsigned long long binary_fraction(double x) {
  const double a = std::fabs(x);
  const unsigned long long u =
      static_cast<unsigned long long>(std::rint((a - std::floor(a)) * 18446744073709551616.0));
  return x < 0 ? 0 - u : u;
}
// The turns of an angle in radians, modulo 1, to 2^-64 (up to 2^40 radians): 1 / (2 pi)
// and the product are sums of two doubles.
unsigned long long turns_of(double radians) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  const double p = radians * kHi;
  return binary_fraction(p) + binary_fraction(std::fma(radians, kHi, -p) + radians * kLo);
}

struct WriteArgs {
  const uint16_t* kv;
  long long stride;
  long long n;
  const uint16_t* gamma;
  float eps;
  const int32_t* pos;      // null: no rotation
  int halves;
  const int64_t* slots;
  uint8_t* rows;
  long long n_rows;
  int* status;
};

// A warp's raw row: the two units of its lane, its pair of k^R, where it goes.
struct RawRow {
  uint4 u0, u1;
  uint32_t ra, rb;
  int32_t pos;
  long long slot;

  __device__ __forceinline__ void load(const WriteArgs& a, long long i, int lane) {
    const uint16_t* x = a.kv + i * a.stride;
    slot = a.slots[i];
    u0 = reinterpret_cast<const uint4*>(x)[lane];
    u1 = reinterpret_cast<const uint4*>(x)[32 + lane];
    if (a.halves) {
      ra = x[kLatent + lane];
      rb = x[kLatent + 32 + lane];
    } else {
      ra = *reinterpret_cast<const uint32_t*>(x + kLatent + 2 * lane);
      rb = 0u;
    }
    pos = a.pos ? a.pos[i] : 0;
  }
};

// Warps walk over the rows, the next row's loads in flight while one is
// worked on, with gamma in registers.  It takes about 300 instructions a row and
// warp, and two thirds of the issue slots.  65536 q4 rows written and read back
// took 41.8 us this way, 42.4 with two rows a warp of sixteen lanes each (fewer
// instructions, but 122 registers), 46.2 with two rows in flight a warp; 42.2
// now, with the long way round for far rows beside the usual one.
template <int FMT>
__global__ void __launch_bounds__(kRowWarps * 32) cache_write_kernel(
    const WriteArgs a, const __grid_constant__ RopeFreq fr) {
  pdl_wait_previous();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long step = static_cast<long long>(gridDim.x) * kRowWarps;
  long long i = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (i >= a.n) return;
  RawRow next;
  next.load(a, i, lane);
  float gm[16];
  if (a.gamma) {
    const uint4* gv = reinterpret_cast<const uint4*>(a.gamma);
    unpack8(gv[lane], gm);
    unpack8(gv[32 + lane], gm + 8);
  }
  // kept in a register: an indexed constant is read lane by lane
  unsigned long long freq = fr.f[lane];
  asm volatile("" : "+l"(freq));
  for (; i < a.n; i += step) {
    const RawRow row = next;
    if (i + step < a.n) next.load(a, i + step, lane);
    if (row.slot < 0) continue;
    if (row.slot >= a.n_rows) {
      if (lane == 0) set_status(a.status, ESS_ERR_DEVICE_CHECK);
      continue;
    }
    float y[16];
    unpack8(row.u0, y);
    unpack8(row.u1, y + 8);
    if (a.gamma) {
      SumSq s;
      s.sum<16, 32>(y);
      float m;
      float root = s.rsqrt_mean(make_float2(1.0f / kLatent, 0.0f), a.eps, &m);
      if (__builtin_expect(!__all_sync(0xffffffffu, SumSq::near(m)), 0))
        root = far_root<16, 32>(y, make_float2(1.0f / kLatent, 0.0f), a.eps, nullptr);
      const F2 r = both(root);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const F2 v = mul2(mul2(F2{y[e], y[e + 1]}, r), F2{gm[e], gm[e + 1]});
        y[e] = v.x;
        y[e + 1] = v.y;
      }
    }
    // k^R: lane l turns pair l
    uint32_t ra = row.ra, rb = row.rb;
    if (!a.halves) {
      rb = ra >> 16;
      ra &= 0xffffu;
    }
    if (a.pos) {
      const unsigned long long turn =
          static_cast<unsigned long long>(static_cast<long long>(row.pos)) * freq;
      // the top 32 bits as a signed fraction of a turn, in radians within
      // +-pi, where the hardware's sine and cosine are off by at most 2^-21: far
      // below half a bf16 step of the pair's larger value (and of the result,
      // unless the two products cancel)
      const float h = static_cast<float>(static_cast<int32_t>(turn >> 32)) * (3.14159265358979f * 0x1p-31f);
      const float sn = __sinf(h), cs = __cosf(h);
      const float xa = bf16_lo(ra), xb = bf16_lo(rb);
      ra = bf16_bits(xa * cs - xb * sn);
      rb = bf16_bits(xa * sn + xb * cs);
    }
    uint8_t* out = a.rows + row.slot * row_bytes_of(FMT);
    uint16_t* rope;
    if (FMT == ESS_ROW_BF16) {
      uint4* o = reinterpret_cast<uint4*>(out);
      o[lane] = pack8_bf16(y);
      o[32 + lane] = pack8_bf16(y + 8);
      rope = reinterpret_cast<uint16_t*>(out + 1024);
    } else if (FMT == ESS_ROW_COMPACT) {
      // a tile of 128 dims is 16 lanes of one unit
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float m = group_max<16>(amax8(y + 8 * h));
        const int e = scale_exp<448>(m);
        const float inv = exp2i(-e);
        reinterpret_cast<uint2*>(out)[32 * h + lane] = pack8_e4m3(y + 8 * h, inv);
        if ((lane & 15) == 0)
          reinterpret_cast<float*>(out + 512)[2 * h + (lane >> 4)] = exp2i(e);
      }
      rope = reinterpret_cast<uint16_t*>(out + 528);
    } else {
      // a block of 32 dims is 4 lanes of one unit
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float m = group_max<4>(amax8(y + 8 * h));
        const int e = min(max(scale_exp<6>(m), kQ4MinExp), kQ4MaxExp);
        const float inv = exp2i(-e);
        reinterpret_cast<uint32_t*>(out)[32 * h + lane] = pack8_e2m1(y + 8 * h, inv);
        if ((lane & 3) == 0) out[256 + 8 * h + (lane >> 2)] = static_cast<uint8_t>(e + 127);
      }
      rope = reinterpret_cast<uint16_t*>(out + 272);
    }
    if (a.halves) {
      rope[lane] = static_cast<uint16_t>(ra);
      rope[32 + lane] = static_cast<uint16_t>(rb);
    } else {
      reinterpret_cast<uint32_t*>(rope)[lane] = ra | (rb << 16);
    }
  }
}

// rows and slots are plain pointers: the kernel may be launched while the one that
// writes them still runs, so they are not read-only for its whole life, which is
// what loads through __restrict__ pointers may take for granted.
template <int FMT>
__global__ void __launch_bounds__(kRowWarps * 32) cache_read_kernel(
    const uint8_t* rows, long long n_rows, const int64_t* slots, long long n, uint16_t* out,
    int* status) {
  pdl_wait_previous();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long i = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (i >= n) return;
  const long long slot = slots[i];
  uint4* o = reinterpret_cast<uint4*>(out + i * kRowDim);
  if (slot < 0 || slot >= n_rows) {
    if (slot >= n_rows && lane == 0) set_status(status, ESS_ERR_DEVICE_CHECK);
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    o[lane] = z;
    o[32 + lane] = z;
    if (lane < 8) o[64 + lane] = z;
    return;
  }
  const uint8_t* row = rows + slot * row_bytes_of(FMT);
  constexpr int kRopeOff = row_bytes_of(FMT) - 128;
  uint4 rope = make_uint4(0u, 0u, 0u, 0u);
  if (lane < 8) rope = reinterpret_cast<const uint4*>(row + kRopeOff)[lane];
  if (FMT == ESS_ROW_BF16) {
    const uint4* s = reinterpret_cast<const uint4*>(row);
    const uint4 u0 = s[lane], u1 = s[32 + lane];
    o[lane] = u0;
    o[32 + lane] = u1;
  } else if (FMT == ESS_ROW_COMPACT) {
    const uint2* s = reinterpret_cast<const uint2*>(row);
    const uint2 c0 = s[lane], c1 = s[32 + lane];
    const float* sc = reinterpret_cast<const float*>(row + 512);
    const float s0 = sc[lane >> 4], s1 = sc[2 + (lane >> 4)];
    o[lane] = widen8_e4m3(c0, s0);
    o[32 + lane] = widen8_e4m3(c1, s1);
  } else {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(row);
    const uint32_t c0 = s[lane], c1 = s[32 + lane];
    const int b0 = row[256 + (lane >> 2)], b1 = row[264 + (lane >> 2)];
    o[lane] = widen8_e2m1(c0, b0);
    o[32 + lane] = widen8_e2m1(c1, b1);
  }
  if (lane < 8) o[64 + lane] = rope;
}

__global__ void status_take_kernel(int* status, int* taken) {
  pdl_wait_previous();
  *taken = atomicExch(status, ESS_OK);
}

struct NormArgs {
  const uint16_t* x;
  long long x_stride;
  const uint16_t* res;
  long long res_stride;
  const uint16_t* gamma;
  float eps;
  long long n;
  int dim;
  float2 inv_dim;      // 1 / dim as a sum of two floats
  uint16_t* res_out;
  uint8_t* codes;
  float* scales;
};

// TPR threads hold one row, UNITS 16-byte units (8 values) each: unit u of the
// row sits in thread u % TPR, so 16 neighbouring lanes hold one group of 128;
// with TPR = 8 (an indexer key) both units of eight lanes do.  A warp so takes
// four keys at once, and what is done once a row (the root, the joining of
// sums), which weighs most in rows this short, is shared by them: 131072 keys in
// 11.6 us, where sixteen lanes a key took 16.0 (12.1 since nothing starts ahead
// of a key norm's end, 12.6 with far_root beside it).  Two units a thread is the
// best for long rows too (16384 x 4096 with a residual: 87 us, four units 90).  The
// resident CTAs asked for are those that fit without far_root, which is off the
// usual path and must not cost them registers.
template <int TPR, int UNITS, bool RES>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256, TPR <= 32 ? 6 : TPR <= 256 ? 5 : 2)
    norm_quant_kernel(const NormArgs a) {
  constexpr int kThreads = TPR > 256 ? TPR : 256;
  constexpr int kRows = kThreads / TPR;
  pdl_wait_previous();
  // Rows of up to 128 values may be bound indexer keys, and an indexer loads its
  // first keys ahead of its own wait: nothing is launched before they are written.
  if (TPR > 8) pdl_launch_dependents();
  const int t = threadIdx.x % TPR;
  const long long i = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / TPR;
  const bool live = i < a.n;
  const int units = a.dim >> 3;
  float h[UNITS * 8];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int c = u * TPR + t;
    uint4 v = make_uint4(0u, 0u, 0u, 0u), w = v;
    if (live && c < units) {
      v = reinterpret_cast<const uint4*>(a.x + i * a.x_stride)[c];
      if (RES) w = reinterpret_cast<const uint4*>(a.res + i * a.res_stride)[c];
    }
    unpack8(v, h + 8 * u);
    if (RES) {
      float r[8];
      unpack8(w, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[8 * u + e] += r[e];
    }
  }
  uint4 gm[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int c = u * TPR + t;
    gm[u] = c < units ? reinterpret_cast<const uint4*>(a.gamma)[c] : make_uint4(0u, 0u, 0u, 0u);
    if (RES && a.res_out && live && c < units)
      reinterpret_cast<uint4*>(a.res_out + i * a.res_stride)[c] = pack8_bf16(h + 8 * u);
  }
  SumSq s;
  s.template sum<UNITS * 8, (TPR < 32 ? TPR : 32)>(h);
  __shared__ float2 part[kThreads / 32];
  if (TPR > 32) {
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) part[w] = make_float2(s.hi, s.lo);
    __syncthreads();
    const int w0 = (threadIdx.x / TPR) * (TPR / 32);
    s = SumSq();
#pragma unroll
    for (int q = 0; q < TPR / 32; ++q) s.merge(part[w0 + q].x, part[w0 + q].y);
  }
  float m;
  float root = s.rsqrt_mean(a.inv_dim, a.eps, &m);
  if (__builtin_expect(!__all_sync(0xffffffffu, SumSq::near(m)), 0))
    root = far_root<UNITS * 8, TPR>(h, a.inv_dim, a.eps, part);
  const F2 r = both(root);
  const int groups = (a.dim + 127) >> 7;
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    float g[8];
    unpack8(gm[u], g);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const F2 v = mul2(mul2(F2{h[8 * u + e], h[8 * u + e + 1]}, r), F2{g[e], g[e + 1]});
      h[8 * u + e] = v.x;
      h[8 * u + e + 1] = v.y;
    }
  }
  constexpr int kPer = TPR < 16 ? UNITS : 1;   // units of a thread in one group
#pragma unroll
  for (int u0 = 0; u0 < UNITS; u0 += kPer) {
    float m = 0.0f;
#pragma unroll
    for (int u = u0; u < u0 + kPer; ++u) m = fmaxf(m, amax8(h + 8 * u));
    m = group_max<(TPR < 16 ? TPR : 16)>(m);
    const int e = scale_exp<448>(m);
    const float inv = exp2i(-e);
#pragma unroll
    for (int u = u0; u < u0 + kPer; ++u) {
      const int c = u * TPR + t;
      if (live && c < units) {
        reinterpret_cast<uint2*>(a.codes + i * a.dim)[c] = pack8_e4m3(h + 8 * u, inv);
        if ((c & 15) == 0) a.scales[i * groups + (c >> 4)] = exp2i(e);
      }
    }
  }
}

template <int TPR, int UNITS>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  constexpr int kThreads = TPR > 256 ? TPR : 256;
  constexpr int kRows = kThreads / TPR;
  const dim3 grid(static_cast<unsigned>((a.n + kRows - 1) / kRows));
  return a.res ? launch_pdl_once(norm_quant_kernel<TPR, UNITS, true>, grid, dim3(kThreads), 0, st, a)
               : launch_pdl_once(norm_quant_kernel<TPR, UNITS, false>, grid, dim3(kThreads), 0, st, a);
}

// rows of one launch: the grid's x extent is a 31-bit number of CTAs
constexpr long long kMaxRows = 1LL << 33;

}  // namespace
}  // namespace ess

using namespace ess;

extern "C" {

ess_status ess_row_bytes(int32_t format, int32_t* bytes) {
  if (!bytes || format < ESS_ROW_BF16 || format > ESS_ROW_Q4) return ESS_ERR_INVALID_ARG;
  *bytes = row_bytes_of(format);
  return ESS_OK;
}

ess_status ess_status_take(int32_t* status, int32_t* taken, ess_stream_t stream) {
  if (!status || !taken || !aligned_to(status, 4) || !aligned_to(taken, 4))
    return ESS_ERR_INVALID_ARG;
  return launch_pdl_once(status_take_kernel, dim3(1), dim3(1), 0,
                         static_cast<cudaStream_t>(stream), status, taken) == cudaSuccess
             ? ESS_OK
             : ESS_ERR_CUDA;
}

ess_status ess_cache_write(const void* kv, int64_t kv_stride, int64_t n, const void* gamma,
                           float eps, const double* inv_freq, const int32_t* pos, int32_t pairs,
                           const int64_t* slots, void* rows, int64_t n_rows, int32_t format,
                           int32_t* status, ess_stream_t stream) {
  if (format < ESS_ROW_BF16 || format > ESS_ROW_Q4 || n < 0 || n > kMaxRows || n_rows < 0)
    return ESS_ERR_INVALID_ARG;
  if (kv_stride < kRowDim || kv_stride % 8 != 0 || !(eps >= 0.0f)) return ESS_ERR_INVALID_ARG;
  if (pairs != ESS_ROPE_ADJACENT && pairs != ESS_ROPE_HALVES) return ESS_ERR_INVALID_ARG;
  RopeFreq fr = {};
  if (inv_freq) {
    for (int i = 0; i < 32; ++i) {
      if (!std::isfinite(inv_freq[i])) return ESS_ERR_INVALID_ARG;
      fr.f[i] = turns_of(inv_freq[i]);
    }
  }
  if (n == 0) return ESS_OK;
  if (!kv || !slots || !rows || (inv_freq && !pos) || !aligned16(kv) || !aligned16(rows) ||
      (gamma && !aligned16(gamma)) || !aligned_to(slots, 8) || !aligned_to(status, 4) ||
      (inv_freq && !aligned_to(pos, 4)))
    return ESS_ERR_INVALID_ARG;
  WriteArgs a;
  a.kv = static_cast<const uint16_t*>(kv);
  a.stride = kv_stride;
  a.n = n;
  a.gamma = static_cast<const uint16_t*>(gamma);
  a.eps = eps;
  a.pos = inv_freq ? pos : nullptr;
  a.halves = pairs == ESS_ROPE_HALVES;
  a.slots = slots;
  a.rows = static_cast<uint8_t*>(rows);
  a.n_rows = n_rows;
  a.status = status;
  const dim3 grid(static_cast<unsigned>(
      std::min<long long>((n + kRowWarps - 1) / kRowWarps, kWriteCtas)));
  const dim3 block(kRowWarps * 32);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (format == ESS_ROW_BF16)
    e = launch_pdl_once(cache_write_kernel<ESS_ROW_BF16>, grid, block, 0, st, a, fr);
  else if (format == ESS_ROW_COMPACT)
    e = launch_pdl_once(cache_write_kernel<ESS_ROW_COMPACT>, grid, block, 0, st, a, fr);
  else
    e = launch_pdl_once(cache_write_kernel<ESS_ROW_Q4>, grid, block, 0, st, a, fr);
  return e == cudaSuccess ? ESS_OK : ESS_ERR_CUDA;
}

ess_status ess_cache_read(const void* rows, int64_t n_rows, int32_t format, const int64_t* slots,
                          int64_t n, void* out, int32_t* status, ess_stream_t stream) {
  if (format < ESS_ROW_BF16 || format > ESS_ROW_Q4 || n < 0 || n > kMaxRows || n_rows < 0)
    return ESS_ERR_INVALID_ARG;
  if (n == 0) return ESS_OK;
  if (!rows || !slots || !out || !aligned16(rows) || !aligned16(out) || !aligned_to(slots, 8) ||
      !aligned_to(status, 4))
    return ESS_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned>((n + kRowWarps - 1) / kRowWarps));
  const dim3 block(kRowWarps * 32);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint8_t* r = static_cast<const uint8_t*>(rows);
  uint16_t* o = static_cast<uint16_t*>(out);
  cudaError_t e;
  if (format == ESS_ROW_BF16)
    e = launch_pdl_once(cache_read_kernel<ESS_ROW_BF16>, grid, block, 0, st, r, n_rows, slots, n, o,
                   status);
  else if (format == ESS_ROW_COMPACT)
    e = launch_pdl_once(cache_read_kernel<ESS_ROW_COMPACT>, grid, block, 0, st, r, n_rows, slots, n, o,
                   status);
  else
    e = launch_pdl_once(cache_read_kernel<ESS_ROW_Q4>, grid, block, 0, st, r, n_rows, slots, n, o,
                   status);
  return e == cudaSuccess ? ESS_OK : ESS_ERR_CUDA;
}

ess_status ess_norm_quant(const void* x, int64_t x_stride, const void* residual,
                          int64_t residual_stride, const void* gamma, float eps, int64_t n,
                          int32_t dim, void* residual_out, void* codes, float* scales,
                          ess_stream_t stream) {
  if (n < 0 || n > kMaxRows || dim < 1 || !(eps >= 0.0f) || x_stride < dim ||
      (residual && residual_stride < dim) || (residual_out && !residual) ||
      (residual_out && residual_out == x && x_stride != residual_stride))
    return ESS_ERR_INVALID_ARG;
  if (dim % 8 != 0 || dim > 16384) return ESS_ERR_UNSUPPORTED;
  if (x_stride % 8 != 0 || (residual && residual_stride % 8 != 0)) return ESS_ERR_INVALID_ARG;
  if (n == 0) return ESS_OK;
  if (!x || !gamma || !codes || !scales || !aligned16(x) || !aligned16(gamma) ||
      !aligned16(codes) || !aligned_to(scales, 4) ||
      (residual && !aligned16(residual)) || (residual_out && !aligned16(residual_out)))
    return ESS_ERR_INVALID_ARG;
  NormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.x_stride = x_stride;
  a.res = static_cast<const uint16_t*>(residual);
  a.res_stride = residual_stride;
  a.gamma = static_cast<const uint16_t*>(gamma);
  a.eps = eps;
  a.n = n;
  a.dim = dim;
  a.inv_dim.x = static_cast<float>(1.0 / dim);
  a.inv_dim.y = static_cast<float>(1.0 / dim - a.inv_dim.x);
  a.res_out = static_cast<uint16_t*>(residual_out);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dim <= 128) ++key_norms();   // the next indexer of each layer waits
  if (dim <= 128) e = launch_norm<8, 2>(a, st);
  else if (dim <= 256) e = launch_norm<16, 2>(a, st);
  else if (dim <= 512) e = launch_norm<32, 2>(a, st);
  else if (dim <= 1024) e = launch_norm<64, 2>(a, st);
  else if (dim <= 2048) e = launch_norm<128, 2>(a, st);
  else if (dim <= 4096) e = launch_norm<256, 2>(a, st);
  else if (dim <= 8192) e = launch_norm<512, 2>(a, st);
  else e = launch_norm<512, 4>(a, st);
  return e == cudaSuccess ? ESS_OK : ESS_ERR_CUDA;
}

}  // extern "C"
