// Absorbed-MLA attention over a device row cache held in 4 bits.
//
// For every query row (b, m, h): softmax_t(sm_scale * q . row_t) @ row_t[:512]
// over the tokens of request b that way m sees, in one pass with the running
// maximum and sum.
//
// One warp per query row, eight heads of one (request, way) per CTA: a tile of
// 32 tokens is widened to fp32 in shared memory and shared by the eight warps.
#include <cmath>

#include "ess_rows.cuh"

namespace ess {
namespace {

constexpr int kTile = 32;
constexpr int kHeadsPerCta = 8;
constexpr int kMaxCacheWays = 4;
constexpr int kMaxCacheHeads = 128;

struct MlaArgs {
  const uint16_t* q;
  const uint8_t* rows;
  long long n_rows;
  const int32_t* page_table;
  int max_pages, page;
  const int32_t* T;
  int batch, ways, heads;
  const int32_t* tokens;
  int k;
  float c2;                // sm_scale * log2(e)
  uint16_t* out;
  float* lse;
  int* status;
};

__global__ void __launch_bounds__(kHeadsPerCta * 32) cache_mla_kernel(const MlaArgs a) {
  extern __shared__ float tile[];   // [kTile][576]
  __shared__ int live[kTile];
  pdl_wait_previous();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int m = blockIdx.y, b = blockIdx.z;
  const int h = blockIdx.x * kHeadsPerCta + warp;
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  int Tb = a.T[b];
  if (Tb < 0 || Tb > cap) {
    if (threadIdx.x == 0) set_status(a.status, ESS_ERR_DEVICE_CHECK);
    Tb = Tb < 0 ? 0 : static_cast<int>(cap);
  }
  const int32_t* list =
      a.tokens ? a.tokens + (static_cast<size_t>(b) * a.ways + m) * a.k : nullptr;
  const int n = list ? min(a.k, Tb) : max(0, Tb - (a.ways - 1) + m);
  const size_t qrow = (static_cast<size_t>(b) * a.ways + m) * a.heads + min(h, a.heads - 1);
  float q[18], o[16];
#pragma unroll
  for (int j = 0; j < 18; ++j) q[j] = bf16_lo(a.q[qrow * kRowDim + 32 * j + lane]);
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = 0.0f;
  float mx = -INFINITY, l = 0.0f;
  for (int t0 = 0; t0 < n; t0 += kTile) {
    __syncthreads();
    for (int r = warp; r < kTile; r += kHeadsPerCta) {
      const int e = t0 + r;
      long long row = -1;
      if (e < n) {
        const int t = list ? list[e] : e;
        if (t >= 0) {
          if (t < Tb) {
            const int pg = a.page_table[static_cast<size_t>(b) * a.max_pages + t / a.page];
            row = static_cast<long long>(pg) * a.page + t % a.page;
          }
          if (row < 0 || row >= a.n_rows) {
            if (lane == 0) set_status(a.status, ESS_ERR_DEVICE_CHECK);
            row = -1;
          }
        }
      }
      if (lane == 0) live[r] = row >= 0;
      float* d = tile + r * kRowDim;
      if (row >= 0) {
        const uint8_t* s = a.rows + row * kQ4RowBytes;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint4 w = widen8_e2m1(reinterpret_cast<const uint32_t*>(s)[32 * half + lane],
                                      s[256 + 8 * half + (lane >> 2)]);
          unpack8(w, d + 256 * half + 8 * lane);
        }
        const uint32_t w = reinterpret_cast<const uint32_t*>(s + 272)[lane];
        d[512 + 2 * lane] = bf16_lo(w);
        d[513 + 2 * lane] = bf16_hi(w);
      }
    }
    __syncthreads();
    for (int r = 0; r < kTile; ++r) {
      if (!live[r]) continue;
      const float* d = tile + r * kRowDim;
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 18; ++j) s = fmaf(q[j], d[32 * j + lane], s);
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= a.c2;
      const float m2 = fmaxf(mx, s);
      const float base = m2 == -INFINITY ? 0.0f : m2;
      const float f = exp2f(mx - base), p = exp2f(s - base);
      mx = m2;
      l = fmaf(l, f, p);
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = fmaf(o[j], f, p * d[32 * j + lane]);
    }
  }
  if (h >= a.heads) return;
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    a.out[qrow * kLatent + 32 * j + lane] = static_cast<uint16_t>(bf16_bits(o[j] * inv));
  if (a.lse && lane == 0)
    a.lse[qrow] = l > 0.0f || l != l ? (mx + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

ess_status check_shape(int batch, int ways, int heads) {
  if (batch < 1 || ways < 1 || heads < 1) return ESS_ERR_INVALID_ARG;
  if (ways > kMaxCacheWays || heads > kMaxCacheHeads || batch > 65535) return ESS_ERR_UNSUPPORTED;
  return ESS_OK;
}

}  // namespace
}  // namespace ess

using namespace ess;

extern "C" {

ess_status ess_cache_mla_bytes(int32_t batch, int32_t ways, int32_t heads, size_t* bytes) {
  if (!bytes) return ESS_ERR_INVALID_ARG;
  const ess_status s = check_shape(batch, ways, heads);
  if (s != ESS_OK) return s;
  *bytes = 256;
  return ESS_OK;
}

ess_status ess_cache_mla(const void* q, const void* rows, int64_t n_rows, int32_t format,
                         const int32_t* page_table, int32_t max_pages, int32_t page,
                         const int32_t* T, int32_t batch, int32_t ways, int32_t heads,
                         const int32_t* tokens, int32_t k, float sm_scale, void* out, float* lse,
                         void* workspace, size_t ws_bytes, int32_t* status, ess_stream_t stream) {
  size_t need = 0;
  const ess_status s = ess_cache_mla_bytes(batch, ways, heads, &need);
  if (s != ESS_OK) return s;
  if (format < ESS_ROW_BF16 || format > ESS_ROW_Q4 || n_rows < 1 || max_pages < 1 || page < 1 ||
      (tokens && k < 1) || !(sm_scale > 0.0f) || !std::isfinite(sm_scale))
    return ESS_ERR_INVALID_ARG;
  if (format != ESS_ROW_Q4 || n_rows > 0x7fffffffLL ||
      static_cast<long long>(max_pages) * page > 0x7fffffffLL)
    return ESS_ERR_UNSUPPORTED;
  if (!q || !rows || !page_table || !T || !out || !workspace || !aligned16(q) ||
      !aligned16(rows) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return ESS_ERR_INVALID_ARG;
  if (ws_bytes < need) return ESS_ERR_OOM;
  MlaArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.rows = static_cast<const uint8_t*>(rows);
  a.n_rows = n_rows;
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.page = page;
  a.T = T;
  a.batch = batch;
  a.ways = ways;
  a.heads = heads;
  a.tokens = tokens;
  a.k = k;
  a.c2 = sm_scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = status;
  const size_t smem = kTile * kRowDim * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(cache_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return ESS_ERR_CUDA;
  const dim3 grid((heads + kHeadsPerCta - 1) / kHeadsPerCta, ways, batch);
  e = launch_pdl(cache_mla_kernel, grid, dim3(kHeadsPerCta * 32), smem,
                 static_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? ESS_OK : ESS_ERR_CUDA;
}

}  // extern "C"
