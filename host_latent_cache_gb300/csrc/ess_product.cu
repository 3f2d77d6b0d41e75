// 8-bit products: bf16 values quantised to e4m3 with a power-of-two scale for
// 128 values of a row (activations) or for 128 x 128 values (weights), and
//
//   out[t][f] = sum_j xs[t][j] ws[f / 128][j] sum_{k in group j} x[t][k] w[f][k]
//
// over the groups j of 128 along K.  All scales are powers of two, so the tensor
// core multiplies them in itself: kind::mxf8f6f4 takes one 8-bit exponent per
// row and 32 values of K, from TMEM, at the full 8-bit rate, and no accumulator
// is read before its sum is complete.
//
//   warps 0-3  epilogue: accumulators out of TMEM, converted and stored
//   warps 4-7  scales: fp32 scales -> exponent bytes -> TMEM.  The four bytes of a
//              32-bit cell are four groups of K; row 32 c + l sits in column c of
//              lane l, once for each quarter of the lanes
//   warp 8     TMA: 128 bytes of K of both operands a stage, 128B swizzle
//   warp 9     MMA
//
// Few tokens: tiles of 128 weight rows (the MMA's M) x 16 to 64 tokens, one a CTA and
// two CTAs an SM, so that reading the weight, which bounds them, wastes no tensor width
// and a warp of the epilogue writes runs of neighbouring columns.  The CTAs of a cluster
// share a tile, each with a part of K; each adds up the sums of its part of the tokens,
// which come to it by bulk copies between the CTAs' shared memories, in the order of the
// parts.  Many tokens: pairs of CTAs (cta_group::2) compute tiles of 256 tokens x 256
// columns, walking over them, the epilogue of one beside the MMAs of the next: two
// accumulators of 256 columns and the scales need 536 of 512, so they share 32, which are
// read first.  Few such tiles, and fp32 results, take 128 columns.
//
// Measured, back to back on one set of inputs for a few milliseconds, so that L2 holds
// weights and codes (time; flops): 8192 x 4096 x 8192 (tokens x ins x outs) 148 to 153 us, 3.6
// PFLOP/s or 93 % of twice the measured bf16 rate (a library's product with the same form of
// scales takes 151); in fp32 208 to 225; 8192 x 1024 x 24576 131 to 138, 2048 x 4096 x 8192 44,
// 512 x 4096 x 8192 15.9, 128 x 4096 x 8192 11.8, 333 x 4112 x 1601 12.9, 64 x 4096 x 8192 9.5, 32 x
// 1024 x 24576 6.4 to 6.8, 4 x 4096 x 1600 4.1; a launch that multiplies 16 x 128 x 128 2.9.  The
// first one on end, at the power limit: 174 to 186 us, 86 to 92 % of twice the sustained rate.
// What bounds them: a large product the tensor pipe, busy for 78 % of an SM's cycles under
// ncu at 2048 tokens (L2 35 %, its crossbar 41 %, shared memory's banks 17 %), with some
// 1000 cycles between two tiles; seconds on end the power limit.  Rows of K that are not
// multiples of 128 bytes straddle L2's lines: 2048 x 4112 x 8192 57 us.  With one tile a
// pair the chain of its stages, 0.2 us each, and with few tokens launch, first loads and
// the exchange of sums beside the weight's stream.
#include <algorithm>
#include <atomic>
#include <cstddef>

#include "ess_rows.cuh"

namespace ess {
namespace {

// ---------------------------------------------------------------- quantisation
struct QuantArgs {
  const uint16_t* x;
  long long stride;
  int n;
  int dim;
  int groups;              // ceil(dim / 128)
  uint32_t mul;            // i / groups = umulhi(i, mul) >> shift for i < 2^31
  int shift;
  uint8_t* codes;
  float* scales;
};

constexpr int kQuantThreads = 256;

// Sixteen neighbouring values (c and on) of a row, zeros behind its end.
__device__ __forceinline__ void quant_load(const QuantArgs& a, bool live, int row, int c,
                                           uint4* v) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    v[h] = make_uint4(0u, 0u, 0u, 0u);
    if (live && c + 8 * h < a.dim)
      v[h] = *reinterpret_cast<const uint4*>(a.x + row * a.stride + c + 8 * h);
  }
}
// Their codes; wide: rows are multiples of 16 bytes.
__device__ __forceinline__ void quant_store(const QuantArgs& a, int row, int c, const float* f,
                                            int e, bool wide) {
  uint8_t* o = a.codes + static_cast<size_t>(row) * a.dim + c;
  const uint2 lo = pack8_e4m3(f, exp2i(-e)), hi = pack8_e4m3(f + 8, exp2i(-e));
  if (wide) {
    if (c < a.dim) *reinterpret_cast<uint4*>(o) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  } else {
    if (c < a.dim) *reinterpret_cast<uint2*>(o) = lo;
    if (c + 8 < a.dim) *reinterpret_cast<uint2*>(o + 8) = hi;
  }
}

// Eight lanes a group of 128 values, sixteen values a lane, so that codes leave 16 bytes
// a store: 16384 x 4096 take 32.6 us (6.2 TB/s, 92 % of the measured copy rate); sixteen
// lanes, 8 bytes a store, 38.5 with one, two or four groups in flight.
__global__ void __launch_bounds__(kQuantThreads) quant_rows_kernel(const QuantArgs a) {
  pdl_wait_previous();
  // rows of 128 values may be bound indexer keys: nothing starts before they are written
  if (a.dim > 128) pdl_launch_dependents();
  const int lane = threadIdx.x & 7;
  const uint32_t total = static_cast<uint32_t>(a.n) * static_cast<uint32_t>(a.groups);
  const uint32_t i = blockIdx.x * (kQuantThreads / 8) + (threadIdx.x >> 3);
  const uint32_t r = a.shift < 0 ? i : __umulhi(i, a.mul) >> a.shift;
  const int row = static_cast<int>(r), g = static_cast<int>(i - r * static_cast<uint32_t>(a.groups));
  const int c = g * 128 + lane * 16;
  uint4 v[2];
  quant_load(a, i < total, row, c, v);
  float f[16];
  unpack8(v[0], f);
  unpack8(v[1], f + 8);
  const int e = scale_exp<448>(group_max<8>(fmaxf(amax8(f), amax8(f + 8))));
  if (i >= total) return;
  quant_store(a, row, c, f, e, a.dim % 16 == 0);
  if (lane == 0) a.scales[static_cast<size_t>(row) * a.groups + g] = exp2i(e);
}

// One CTA a block of 128 x 128: eight lanes a row, 32 rows at a time.  16384 x 4096 take
// 36.7 us (5.5 TB/s), 1600 x 4096 (from L2) 2.9; with 512 threads 39.7, with 1024 45.9: all of a
// block is loaded before any of it leaves, so several small CTAs an SM do better.
__global__ void __launch_bounds__(kQuantThreads) quant_square_kernel(const QuantArgs a) {
  __shared__ float part[kQuantThreads / 32];
  constexpr int kRows = kQuantThreads / 8, kTimes = 128 / kRows;
  pdl_wait_previous();
  pdl_launch_dependents();
  const int r0 = blockIdx.y * 128 + (threadIdx.x >> 3);
  const int c = blockIdx.x * 128 + (threadIdx.x & 7) * 16;
  uint4 v[kTimes][2];
#pragma unroll
  for (int q = 0; q < kTimes; ++q) quant_load(a, r0 + kRows * q < a.n, r0 + kRows * q, c, v[q]);
  float m = 0.0f;
#pragma unroll
  for (int q = 0; q < kTimes; ++q) {
    float f[16];
    unpack8(v[q][0], f);
    unpack8(v[q][1], f + 8);
    m = fmaxf(m, fmaxf(amax8(f), amax8(f + 8)));
  }
  m = group_max<32>(m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) m = fmaxf(m, part[w]);
  const int e = scale_exp<448>(m);
  const bool wide = a.dim % 16 == 0;
#pragma unroll
  for (int q = 0; q < kTimes; ++q) {
    float f[16];
    unpack8(v[q][0], f);
    unpack8(v[q][1], f + 8);
    if (r0 + kRows * q < a.n) quant_store(a, r0 + kRows * q, c, f, e, wide);
  }
  if (threadIdx.x == 0)
    a.scales[static_cast<size_t>(blockIdx.y) * a.groups + blockIdx.x] = exp2i(e);
}

// ---------------------------------------------------------------- product
constexpr int kEpiWarps = 4, kScaleWarps = 4;
constexpr int kTmaWarp = kEpiWarps + kScaleWarps, kProdMmaWarp = kTmaWarp + 1;
constexpr int kProdThreads = (kProdMmaWarp + 1) * 32;
constexpr uint32_t kATile = 128 * 128;   // bytes of the first operand's part of a stage
constexpr int kMaxStages = 8;
constexpr uint32_t kOutBlock = 32 * 128;  // results on their way out: 32 tokens, 128 bytes each
constexpr int kOverlap = 32;             // columns that two accumulators of 256 share

// Groups of K that one accumulator adds up when sums are short.  The tensor core
// cuts off what an addition shifts out, so a sum drifts towards zero with each of
// its additions.  Of values of one sign, in parts of their sum: 2e-6 over 1024 of them,
// 1e-5 over 4096, 4e-5 over 16384, 1.8e-4 over 65536; of both signs, products of 4096
// values were off by 2e-6 of their norm (2^-24 is 6e-8).  For fp32 results sums of 1024 are
// added up in registers, rounded, instead: 2e-6 of one sign for any K.  A bf16 result (half
// a step is 4e-3 of it) is one sum of up to kOneSum values, and short sums above that: eight
// sums of 2^19 were 1.8e-3 short, eight of 2^23 1.6e-2.
constexpr int kSumGroups = 8;
constexpr int kOneSum = 1 << 16;

constexpr int prod_stages(int bn, bool pair) {
  return pair ? (bn == 256 ? 6 : 8) : bn <= 16 ? 5 : bn <= 32 ? 4 : 3;
}
constexpr int prod_b_rows(int bn, bool pair) { return pair ? bn / 2 : bn; }   // a CTA's part of B
constexpr uint32_t prod_stage_bytes(int bn, bool pair) {
  return kATile + prod_b_rows(bn, pair) * 128;
}

struct ProdMisc {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t sf_full[2], sf_empty[2];
  uint64_t acc_full[2], acc_free[2];
  uint64_t sums_here;
  uint32_t tmem;
  int abort;
};
// Scales on their way to TMEM.  A piece is the 16 bytes of four groups of K (a round); a
// fetch brings prod_run neighbouring pieces of each of the CTA's tokens and of its one
// or two blocks of the weight, as L2 serves a whole line for the price of a piece (with
// single pieces 8192 x 4096 x 8192 took 212 us).
constexpr int prod_run(bool pair) { return pair ? 4 : 2; }
constexpr int prod_fetches(bool pair) { return pair ? 2 : 3; }   // in flight or in use
constexpr int prod_blocks(int bn, bool pair) { return pair ? bn / 128 : 1; }   // of the weight
constexpr int prod_tokens(int bn, bool pair) { return pair ? 128 : bn; }   // of one CTA
constexpr uint32_t prod_fetch_bytes(int bn, bool pair) {
  return (prod_tokens(bn, pair) + prod_blocks(bn, pair)) * prod_run(pair) * 16;
}
// Parts of K meet in places for BN tokens and these more: p parts of a tile leave
// p ceil(BN / p) tokens' sums in a CTA at most.  (For 64 tokens no more than two fit beside
// a second CTA on the SM, which leaves out seven parts.)
constexpr int kMaxParts = 8;
static_assert(kMaxParts <= 8, "portable clusters");
constexpr int prod_places(int bn) { return bn + (bn <= 32 ? 7 : 2); }
constexpr bool parts_fit(int bn, int parts) {
  return parts * ((bn + parts - 1) / parts) <= prod_places(bn);
}
static_assert(parts_fit(16, 7) && parts_fit(32, 7) && parts_fit(64, 6) && !parts_fit(64, 7) &&
                  parts_fit(64, 8),
              "parts of K");
constexpr uint32_t prod_smem(int bn, bool pair) {
  return prod_stages(bn, pair) * prod_stage_bytes(bn, pair) +
         prod_fetches(pair) * prod_fetch_bytes(bn, pair) + (pair ? kEpiWarps * kOutBlock : prod_places(bn) * 512) +
         sizeof(ProdMisc);
}

struct ProdArgs {
  const float* xs;        // [n][groups]
  const float* ws;        // [ceil(outs / 128)][groups]
  int n, outs, groups;
  int m_tiles, n_tiles;
  void* out;
  long long stride;
  bool blocks;            // a pair's results leave through omap
  bool keys;              // the results may be indexer keys: nothing starts early
  bool wide;              // rows of scales are multiples of 16 bytes, 16-byte aligned
  int* status;
};

// a block of shared memory to global memory; what lies outside the tensor is left out
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t src, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(m)),
      "r"(src), "r"(x), "r"(y)
      : "memory");
}
// a load into this CTA that counts its bytes on the even CTA's barrier
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* m,
                                                 uint32_t cluster_bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(cluster_bar), "r"(x), "r"(y)
      : "memory");
}
// D (+)= (A * scales) (B * scales)^T, e4m3, one exponent byte per row and 32 values
template <bool PAIR>
__device__ __forceinline__ void umma_mx8(uint32_t d, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// Instruction descriptor of the scaled kinds: bits 4-5 which byte of B's scale cells,
// 17-22 N>>3, 23 scales are exponents, 27-28 M>>7, 29-30 which byte of A's.
__device__ __forceinline__ uint32_t mx_idesc(uint32_t M, uint32_t N, uint32_t byte) {
  return (byte << 4) | ((N >> 3) << 17) | (1u << 23) | ((M >> 7) << 27) | (byte << 29);
}
template <bool PAIR>
__device__ __forceinline__ void prod_commit(uint32_t bar) {   // in both CTAs of a pair
  if (PAIR) umma_commit_pair(bar);
  else umma_commit(bar);
}
template <bool PAIR>
__device__ __forceinline__ void prod_alloc(uint32_t dst, uint32_t cols) {
  if (PAIR) {
    tmem_alloc_pair(dst, cols);
    tmem_relinquish_pair();
  } else {
    tmem_alloc(dst, cols);
    tmem_relinquish();
  }
}
template <bool PAIR>
__device__ __forceinline__ void prod_dealloc(uint32_t taddr, uint32_t cols) {
  if (PAIR) tmem_dealloc_pair(taddr, cols);
  else tmem_dealloc(taddr, cols);
}
// N consecutive columns of this lane
template <int N>
__device__ __forceinline__ void tmem_put(uint32_t t, const uint32_t* r) {
  static_assert(N == 1 || N == 2 || N == 4 || N == 8, "columns");
  if (N == 1)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(t), "r"(r[0]) : "memory");
  else if (N == 2)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(t), "r"(r[0]),
                 "r"(r[N > 1 ? 1 : 0])
                 : "memory");
  else
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(t + i),
                   "r"(r[i]), "r"(r[N > 2 ? i + 1 : 0]), "r"(r[N > 2 ? i + 2 : 0]),
                   "r"(r[N > 2 ? i + 3 : 0])
                   : "memory");
}
// 16 consecutive fp32 columns of this lane
__device__ __forceinline__ void tmem_ld16(uint32_t t, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// shared memory of this CTA -> of another one of the cluster, counted on its barrier
__device__ __forceinline__ void bulk_to_cta(uint32_t cluster_dst, uint32_t src, uint32_t bytes,
                                            uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, "
      "[%3];" ::"r"(cluster_dst),
      "r"(src), "r"(bytes), "r"(cluster_bar)
      : "memory");
}

// Four scales from global to shared memory; groups past the last count as 1.  wide:
// rows of scales are 16-byte aligned (then there are four).
__device__ __forceinline__ void fetch_scales(uint8_t* to, const float* s, int left, bool wide) {
  if (wide) {
    cp_async16(smem_u32(to), s);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j < left)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to) + 4 * j),
                   "l"(s + j)
                   : "memory");
    else
      reinterpret_cast<float*>(to)[j] = 1.0f;
  }
}
// Their exponent bytes.
__device__ __forceinline__ uint32_t scale_word(const uint4& s, bool* bad) {
  const uint32_t v[4] = {s.x, s.y, s.z, s.w};
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = v[j];
    const uint32_t e = (b >> 23) & 0xffu;
    *bad |= (b & 0x807fffffu) != 0u || e == 0u || e == 255u;
    w |= min(max(e, 1u), 254u) << (8 * j);
  }
  return w;
}

// What a CTA works on: tiles first, first + step, ..., groups [g0, g1) of K.
struct ProdShare {
  int first, step, tiles, g0, g1;
};

template <int BN, bool PAIR, typename Out, bool SUMS>
__global__ void __launch_bounds__(kProdThreads, PAIR ? 1 : 2)
    product_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                   const __grid_constant__ CUtensorMap omap, const ProdArgs a) {
  constexpr bool kSums = SUMS;               // short sums, added up in registers
  static_assert(!kSums || BN <= 128, "sums in registers");
  static_assert(kSums || sizeof(Out) == 2, "fp32 results");
  constexpr int kStages = prod_stages(BN, PAIR);
  constexpr uint32_t kStage = prod_stage_bytes(BN, PAIR);
  constexpr int kBRows = prod_b_rows(BN, PAIR);
  constexpr int kAcc = BN < 32 ? 32 : BN;                   // columns of an accumulator
  constexpr bool kShared = BN == 256;        // two that share columns
  constexpr bool kTwo = !kShared && (PAIR || kSums);   // two of their own
  constexpr uint32_t kAcc2 = kShared ? kAcc - kOverlap : kTwo ? kAcc : 0;   // the second one
  constexpr uint32_t kColSf = kAcc2 + kAcc;
  constexpr uint32_t kSfBuf = 4 + (BN <= 128 ? 4 : 8);      // columns of scales: A's, B's
  constexpr uint32_t kNeed = kColSf + 2 * kSfBuf;
  constexpr uint32_t kCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
  static_assert(kNeed <= kCols, "TMEM columns");
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring;            // of scales
  constexpr uint32_t kFetch = prod_fetch_bytes(BN, PAIR);
  // a pair's results on their way out (at multiples of 1024), or the sums of a tile's
  // tokens [part][token of this CTA's share][128] from the cluster's CTAs
  uint8_t* blocks = smem + kStages * kStage;
  ring = blocks + (PAIR ? kEpiWarps * kOutBlock : prod_places(BN) * 512);
  ProdMisc* mi = reinterpret_cast<ProdMisc*>(ring + prod_fetches(PAIR) * kFetch);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t rank = cluster_ctarank();
  uint32_t parts;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(parts));
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&mi->full[i]), 1);
      mbar_init(smem_u32(&mi->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&mi->sf_full[i]), kScaleWarps * (PAIR ? 2 : 1));
      mbar_init(smem_u32(&mi->sf_empty[i]), 1);
      mbar_init(smem_u32(&mi->acc_full[i]), 1);
      mbar_init(smem_u32(&mi->acc_free[i]), kEpiWarps * (PAIR ? 2 : 1));
    }
    mbar_init(smem_u32(&mi->sums_here), 1);
    mi->abort = 0;
    fence_mbar_init();
    if (!PAIR && parts > 1)
      mbar_arrive_expect_tx(smem_u32(&mi->sums_here),
                            parts * 512 * (BN * (rank + 1) / parts - BN * rank / parts));
    tma_prefetch_desc(&amap);
    tma_prefetch_desc(&bmap);
    if (PAIR && a.blocks) tma_prefetch_desc(&omap);
  }
  if (warp == kProdMmaWarp) prod_alloc<PAIR>(smem_u32(&mi->tmem), kCols);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (parts > 1) cluster_sync();   // the peers' barriers exist
  tc_fence_after();
  const uint32_t tmem = mi->tmem;
  pdl_wait_previous();
  if (!a.keys) pdl_launch_dependents();

  ProdShare sh;
  sh.tiles = a.m_tiles * a.n_tiles;
  sh.first = static_cast<int>(blockIdx.x / parts);
  sh.step = static_cast<int>(gridDim.x / parts);
  sh.g0 = PAIR ? 0 : static_cast<int>(static_cast<long long>(a.groups) * rank / parts);
  sh.g1 = PAIR ? a.groups : static_cast<int>(static_cast<long long>(a.groups) * (rank + 1) / parts);
  // tile -> first row of this CTA's A, first row of B
  auto m_of = [&](int t) {
    return PAIR ? (t / a.n_tiles) * 256 + static_cast<int>(rank) * 128
                : (t % a.m_tiles) * 128;
  };
  auto n_of = [&](int t) { return (PAIR ? t % a.n_tiles : t / a.m_tiles) * BN; };

  if (warp == kTmaWarp) {
    if (elect_one()) {
      int stage = 0, turn = 0;
      bool ok = true;   // after a wait that gave up nothing more is loaded
      for (int t = sh.first; ok && t < sh.tiles; t += sh.step) {
        const int m0 = m_of(t), n0 = n_of(t) + (PAIR ? static_cast<int>(rank) * kBRows : 0);
        for (int g = sh.g0; g < sh.g1; ++g) {
          if (turn > 0) ok = wait_or_abort(&mi->empty[stage], (turn - 1) & 1, mi, a.status);
          if (!ok) break;
          const uint32_t dst = smem_u32(smem + stage * kStage), bar = smem_u32(&mi->full[stage]);
          if (PAIR) {
            if (rank == 0) mbar_arrive_expect_tx(bar, 2 * kStage);
            const uint32_t lead = dsmem_addr(bar, 0);
            tma_load_2d_pair(dst, &amap, lead, g * 128, m0);
            tma_load_2d_pair(dst + kATile, &bmap, lead, g * 128, n0);
          } else {
            mbar_arrive_expect_tx(bar, kStage);
            tma_load_2d(dst, &amap, bar, g * 128, m0);
            tma_load_2d(dst + kATile, &bmap, bar, g * 128, n0);
          }
          if (++stage == kStages) {
            stage = 0;
            ++turn;
          }
        }
      }
      // The last arrivals of every stage are waited for, so that none is on its way
      // when the CTA ends.  After a wait that gave up, copies may be: the stages'
      // last ones are waited for with a limit of their own.  (The odd CTA's bytes
      // are counted by the even one, which stays until the cluster's last barrier.)
      for (int i = 0; i < kStages; ++i) {
        const int last = i < stage ? turn : turn - 1;   // the stage's last use
        if (last < 0 || wait_or_abort(&mi->empty[i], last & 1, mi, a.status)) continue;
        const long long t0 = clock64();
        while ((!PAIR || rank == 0) && !mbar_try_wait(smem_u32(&mi->full[i]), last & 1) &&
               clock64() - t0 < kWaitLimitCycles) {
        }
      }
    }
    __syncwarp();
  } else if (warp == kProdMmaWarp) {
    if (!PAIR || rank == 0) {
      const bool lead = elect_one();
      int stage = 0, turn = 0, sb = 0, sturn = 0, i = 0;   // i counts sums
      bool ok = true;
      for (int t = sh.first; t < sh.tiles; t += sh.step) {
        for (int g = sh.g0; g < sh.g1; ++g) {
          const bool first = g == sh.g0 || (kSums && (g - sh.g0) % kSumGroups == 0);
          const bool last = g + 1 == sh.g1 || (kSums && (g + 1 - sh.g0) % kSumGroups == 0);
          if (first) {
            // the accumulator is read out: where two share columns, the part that the sum
            // before shares with it, and so all of the one before that
            if (kShared && i > 0) ok = wait_or_abort(&mi->acc_free[0], (i - 1) & 1, mi, a.status) && ok;
            if (kTwo && i > 1)
              ok = wait_or_abort(&mi->acc_free[i & 1], ((i >> 1) - 1) & 1, mi, a.status) && ok;
          }
          if (g == sh.g0 || (g & 3) == 0)
            ok = wait_or_abort(&mi->sf_full[sb], sturn & 1, mi, a.status) && ok;
          ok = wait_or_abort(&mi->full[stage], turn & 1, mi, a.status) && ok;
          tc_fence_after();
          const bool cells = (g & 3) == 3 || g + 1 == sh.g1;   // done with a buffer of scales
          if (ok && lead) {
            const uint32_t at = smem_u32(smem + stage * kStage);
            const uint64_t dw = make_sdesc_sw128(at, 16, 1024);
            const uint64_t dx = make_sdesc_sw128(at + kATile, 16, 1024);
            const uint32_t idesc = mx_idesc(PAIR ? 256 : 128, BN, g & 3);
            const uint32_t sf = tmem + kColSf + sb * kSfBuf, acc = tmem + (i & 1) * kAcc2;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_mx8<PAIR>(acc, dw + 2 * k, dx + 2 * k, idesc, sf, sf + 4, !first || k > 0);
            prod_commit<PAIR>(smem_u32(&mi->empty[stage]));
            if (cells) prod_commit<PAIR>(smem_u32(&mi->sf_empty[sb]));
            if (last) prod_commit<PAIR>(smem_u32(&mi->acc_full[i & 1]));
          }
          __syncwarp();
          if (last) ++i;
          if (++stage == kStages) {
            stage = 0;
            ++turn;
          }
          if (cells && ++sb == 2) {
            sb = 0;
            ++sturn;
          }
        }
      }
    }
  } else if (warp >= kEpiWarps) {
    // scales
    const int q = warp & 3;
    const uint32_t ts = tmem + (static_cast<uint32_t>(q * 32) << 16) + kColSf;
    int sb = 0, sturn = 0;
    bool bad = false;
    constexpr int kTok = prod_tokens(BN, PAIR), kRun = prod_run(PAIR), kFetches = prod_fetches(PAIR);
    constexpr int kBlocks = prod_blocks(BN, PAIR), kTokCols = kTok < 32 ? 1 : kTok / 32;
    const int s0 = sh.g0 >> 2, s1 = ((sh.g1 - 1) >> 2) + 1;   // rounds
    const int me = q * 32 + lane;
    int lt = sh.first, ls = s0, lslot = 0;   // what is fetched next
    // piece p of row r lies at place p ^ (r % kRun): a warp's reads then meet all banks
    auto fetch = [&] {
      if (lt < sh.tiles) {
        uint8_t* to = ring + lslot * kFetch;
        const int f0 = PAIR ? n_of(lt) : m_of(lt), x0 = PAIR ? m_of(lt) : n_of(lt);
#pragma unroll 1
        for (int i = me; i < (kTok + kBlocks) * kRun; i += kScaleWarps * 32) {
          const int r = i / kRun, p = i % kRun, s = ls / kRun * kRun + p;
          if (s >= s1) continue;
          uint8_t* at = to + (r * kRun + (p ^ (r & (kRun - 1)))) * 16;
          const bool token = r < kTok;
          if (token && x0 + r >= a.n) {
            *reinterpret_cast<float4*>(at) = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
          } else {
            const int row = token ? x0 + r : min(f0 + 128 * (r - kTok), a.outs - 1) >> 7;
            fetch_scales(at, (token ? a.xs : a.ws) + static_cast<size_t>(row) * a.groups + 4 * s,
                         a.groups - 4 * s, a.wide);
          }
        }
        ls = ls / kRun * kRun + kRun;
        if (ls >= s1) {
          ls = s0;
          lt += sh.step;
        }
      }
      cp_async_commit();
      if (++lslot == kFetches) lslot = 0;
    };
    int slot = kFetches - 1;
#pragma unroll
    for (int i = 0; i < kFetches - 1; ++i) fetch();
    for (int t = sh.first; t < sh.tiles; t += sh.step) {
      for (int s = s0; s < s1; ++s) {
        if (s == s0 || s % kRun == 0) {
          cp_async_wait<kFetches - 2>();
          asm volatile("bar.sync 1, %0;" ::"n"(kScaleWarps * 32) : "memory");
          fetch();   // into the place that every warp had read before the barrier
          if (++slot == kFetches) slot = 0;
        }
        const uint4* in = reinterpret_cast<const uint4*>(ring + slot * kFetch);
        auto piece = [&](int r) { return in[r * kRun + ((s % kRun) ^ (r & (kRun - 1)))]; };
        uint32_t w[8], x[kTokCols];
        w[0] = w[1] = w[2] = w[3] = scale_word(piece(kTok), &bad);
        if (kBlocks == 2) w[4] = w[5] = w[6] = w[7] = scale_word(piece(kTok + kBlocks - 1), &bad);
#pragma unroll
        for (int c = 0; c < kTokCols; ++c)
          x[c] = scale_word(piece(kTok < 32 ? lane % kTok : 32 * c + lane), &bad);
        if (sturn > 0) wait_or_abort(&mi->sf_empty[sb], (sturn - 1) & 1, mi, a.status);
        tc_fence_after();
        if (PAIR) {
          tmem_put<kTokCols>(ts + sb * kSfBuf, x);
          tmem_put<4 * kBlocks>(ts + sb * kSfBuf + 4, w);
        } else {
          tmem_put<4>(ts + sb * kSfBuf, w);
          tmem_put<kTokCols>(ts + sb * kSfBuf + 4, x);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_remote(dsmem_addr(smem_u32(&mi->sf_full[sb]), 0));
          else mbar_arrive(smem_u32(&mi->sf_full[sb]));
        }
        if (++sb == 2) {
          sb = 0;
          ++sturn;
        }
      }
    }
    for (int i = 0; i < 2; ++i) {   // the last arrivals, which nothing else waits for
      const int last = i < sb ? sturn : sturn - 1;
      if (last >= 0) wait_or_abort(&mi->sf_empty[i], last & 1, mi, a.status);
    }
    cp_async_wait<0>();
    if (q == 0 && bad) set_status(a.status, ESS_ERR_DEVICE_CHECK);
  } else {
    // epilogue: lane l of warp q holds output column 32 q + l (a pair's: token 32 q + l)
    constexpr int kBlocks = kAcc / 32, kLive = BN < 32 ? BN : 32;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    auto store = [&](int t, int b, const float* v) {
      const int f = m_of(t) + warp * 32 + lane, x0 = n_of(t) + 32 * b;
      const int left = min(a.n - x0, kLive);
      if (f >= a.outs) return;
      Out* o = static_cast<Out*>(a.out) + x0 * a.stride + f;
#pragma unroll
      for (int c = 0; c < kLive; ++c)
        if (c < left) o[c * a.stride] = static_cast<Out>(v[c]);
    };
    // This part's sums of a block of tokens, into the stages, which nothing uses any
    // more, and from there to the CTAs that add them up, [token][128] floats.
    auto keep = [&](int b, const float* v) {
      float* o = reinterpret_cast<float*>(smem) + 32 * b * 128 + warp * 32 + lane;
#pragma unroll
      for (int c = 0; c < kLive; ++c) o[c * 128] = v[c];
    };
    auto send = [&] {
      fence_proxy_async_smem();
      asm volatile("bar.sync 2, %0;" ::"n"(kEpiWarps * 32) : "memory");
      if (tid < static_cast<int>(parts)) {
        const uint32_t t0 = BN * tid / parts, some = BN * (tid + 1) / parts - t0;
        bulk_to_cta(dsmem_addr(smem_u32(blocks) + rank * some * 512, tid), smem_u32(smem) + t0 * 512,
                    some * 512, dsmem_addr(smem_u32(&mi->sums_here), tid));
      }
    };
    // A pair's results: lane l of warp q holds a token.  Its columns go through shared
    // memory, 128 bytes at a time, so that they leave in whole lines: L2 serves a line for
    // the price of a sector.  j: the j-th block of 32 columns that is written of a tile.
    auto leave = [&](int t, int j, int b, const float* v) {
      constexpr int kPer = 4 / sizeof(Out);   // blocks of 32 columns in 128 bytes
      uint8_t* o = blocks + warp * kOutBlock;
      if (j % kPer == 0) {   // the ones before have left
        if (a.blocks && lane == 0) bulk_wait_read<0>();
        __syncwarp();
      }
      if (sizeof(Out) == 2) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(o + sw128_off(lane, 4 * (b & 1) + c)) = pack8_bf16(v + 8 * c);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<float4*>(o + sw128_off(lane, c)) =
              make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
      }
      if (j % kPer != kPer - 1) return;
      const int f0 = n_of(t) + 32 * (b - b % kPer), t0 = m_of(t) + warp * 32;
      if (a.blocks) fence_proxy_async_smem();
      __syncwarp();
      if (a.blocks) {
        if (lane == 0) {
          if (f0 < a.outs && t0 < a.n) tma_store_2d(&omap, smem_u32(o), f0, t0);
          bulk_commit();
        }
        return;
      }
      // rows that TMA does not take (not multiples of 16 bytes)
      constexpr int kUnit = 16 / sizeof(Out);
      for (int r = 0; r < min(32, a.n - t0); ++r) {
        Out* row = static_cast<Out*>(a.out) + (t0 + r) * a.stride + f0;
#pragma unroll
        for (int c = lane; c < 32 * kPer; c += 32)
          if (f0 + c < a.outs)
            row[c] = *reinterpret_cast<Out*>(o + sw128_off(r, c / kUnit) + c % kUnit * sizeof(Out));
      }
    };
    auto read_out = [&](int i) {   // the i-th sum's accumulator may be used again
      tc_fence_before();
      __syncwarp();
      if (lane != 0) return;
      if (PAIR) mbar_arrive_remote(dsmem_addr(smem_u32(&mi->acc_free[kShared ? 0 : i & 1]), 0));
      else mbar_arrive(smem_u32(&mi->acc_free[i & 1]));
    };
    int i = 0;   // counts sums
    for (int t = sh.first; t < sh.tiles; t += sh.step) {
      if (kSums) {
        float sum[kAcc];
#pragma unroll
        for (int c = 0; c < kAcc; ++c) sum[c] = 0.0f;
        for (int g = sh.g0; g < sh.g1; g += kSumGroups, ++i) {
          wait_or_abort(&mi->acc_full[i & 1], (i >> 1) & 1, mi, a.status);
          tc_fence_after();
#pragma unroll
          for (int b = 0; b < kAcc; b += 16) {
            float v[16];
            tmem_ld16(tmem + lanes + (i & 1) * kAcc2 + b, v);
#pragma unroll
            for (int c = 0; c < 16; ++c) sum[b + c] += v[c];
          }
          read_out(i);
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          if (PAIR) leave(t, b, b, sum + 32 * b);
          else if (parts > 1) keep(b, sum + 32 * b);
          else store(t, b, sum + 32 * b);
        }
      } else {
        wait_or_abort(&mi->acc_full[i & 1], (i >> 1) & 1, mi, a.status);
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < kBlocks; ++j) {
          // the columns that the next tile's accumulator shares come first
          const int b = kShared && (i & 1) == 0 ? kBlocks - 1 - j : j;
          float v[32];
          tmem_ld32(tmem + lanes + (i & 1) * kAcc2 + 32 * b, v);
          if (PAIR && j == (kShared ? 0 : kBlocks - 1)) read_out(i);
          if (PAIR) leave(t, j, b, v);
          else if (parts > 1) keep(b, v);
          else store(t, b, v);
        }
        ++i;
      }
      if (!PAIR && parts > 1) send();
    }
    if (PAIR && a.blocks && lane == 0) bulk_wait_all();
  }

  if (!PAIR && parts > 1) {
    // The cluster's CTAs held the same tile's sums over their parts of K: each adds up
    // the tokens [BN rank / parts, BN (rank + 1) / parts), in the order of the parts.
    wait_or_abort(&mi->sums_here, 0, mi, a.status);
    const int t0 = static_cast<int>(BN * rank / parts);
    const int share = static_cast<int>(BN * (rank + 1) / parts) - t0;
    const int f = m_of(sh.first) + (tid & 127);
    const int x0 = n_of(sh.first) + t0;
    if (tid < 256 && f < a.outs) {
      const float* in = reinterpret_cast<const float*>(blocks) + (tid & 127);
      for (int c = tid >> 7; c < share && x0 + c < a.n; c += 2) {
        float s = in[c * 128];
        for (uint32_t p = 1; p < parts; ++p) s += in[(p * share + c) * 128];
        static_cast<Out*>(a.out)[(x0 + c) * a.stride + f] = static_cast<Out>(s);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (parts > 1) cluster_sync();
  tc_fence_after();
  if (warp == kProdMmaWarp) prod_dealloc<PAIR>(tmem, kCols);
}

// A launch of the kernel as a programmatic dependent, in clusters of `cluster` CTAs.
struct ProdLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[3];
  ProdLaunch(int ctas, int cluster, uint32_t smem, cudaStream_t st) {
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
    at[1].val.sharedMemCarveout = static_cast<int>(cudaSharedmemCarveoutMaxShared);
    at[2].id = cudaLaunchAttributeClusterDimension;
    at[2].val.clusterDim.x = cluster;
    at[2].val.clusterDim.y = at[2].val.clusterDim.z = 1;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kProdThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 3;
  }
};

template <int BN, bool PAIR, typename Out, bool SUMS>
cudaError_t launch_product(const CUtensorMap& am, const CUtensorMap& bm, const CUtensorMap& om,
                           const ProdArgs& a, int ctas, int cluster, int dev, cudaStream_t st) {
  const cudaError_t e = allow_smem<product_kernel<BN, PAIR, Out, SUMS>>(dev, prod_smem(BN, PAIR));
  if (e != cudaSuccess) return e;
  ProdLaunch l(ctas, cluster, prod_smem(BN, PAIR), st);
  return cudaLaunchKernelEx(&l.cfg, product_kernel<BN, PAIR, Out, SUMS>, am, bm, om, a);
}

// Clusters of `parts` CTAs, two an SM, that run at once, which depends on how SMs are
// grouped (of 152: 97 of three, 74 of four, 36 of eight); 0 when the runtime does not say.
// It is asked about a kernel of the same threads and shared memory, as of one that uses
// TMEM it counts a single CTA an SM.
__global__ void __launch_bounds__(kProdThreads, 2) place_kernel() {}

int clusters_at_once(int parts, int dev) {
  constexpr uint32_t kSmem = prod_smem(64, false);   // the largest of them
  static std::atomic<int> known[64][kMaxParts + 1];   // the number and 1
  if (dev < 64) {
    const int k = known[dev][parts].load(std::memory_order_relaxed);
    if (k > 0) return k - 1;
  }
  int n = 0;
  ProdLaunch l(parts, parts, kSmem, nullptr);
  if (cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmem)) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, place_kernel, &l.cfg) != cudaSuccess)
    n = 0;
  if (dev < 64) known[dev][parts].store(n + 1, std::memory_order_relaxed);
  return n;
}

// K is cut into as many parts as still run at once, with two stages each (us): 4 x 4096 x
// 1600, 13 tiles, takes 10.5 uncut, 7.2 in two parts, 5.1 in four, 4.1 in eight; 16 x 4096 x
// 4736, 37 tiles, 9.0 in eight parts, of which 36 clusters run at once.
template <int BN, typename Out, bool SUMS>
cudaError_t launch_single(const CUtensorMap& w, const CUtensorMap& x, const ProdArgs& a, int tiles,
                          int dev, cudaStream_t st) {
  int parts = kMaxParts;
  while (parts > 1 && (a.groups < 2 * parts || !parts_fit(BN, parts) ||
                       tiles > clusters_at_once(parts, dev)))
    --parts;
  return launch_product<BN, false, Out, SUMS>(w, x, w, a, tiles * parts, parts, dev, st);
}

template <int BN>
cudaError_t launch_single(bool fp32, bool sums, const CUtensorMap& w, const CUtensorMap& x,
                          const ProdArgs& a, int tiles, int dev, cudaStream_t st) {
  return fp32   ? launch_single<BN, float, true>(w, x, a, tiles, dev, st)
         : sums ? launch_single<BN, __nv_bfloat16, true>(w, x, a, tiles, dev, st)
                : launch_single<BN, __nv_bfloat16, false>(w, x, a, tiles, dev, st);
}

int sms_of(int dev) {
  static std::atomic<int> known[64];
  if (dev >= 0 && dev < 64) {
    const int k = known[dev].load(std::memory_order_relaxed);
    if (k > 0) return k;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace
}  // namespace ess

using namespace ess;

extern "C" {

ess_status ess_quant(const void* x, int64_t x_stride, int64_t n, int32_t dim, int32_t square,
                     void* codes, float* scales, ess_stream_t stream) {
  if (n < 0 || n > 0x7fffffffLL || dim < 1 || x_stride < dim || x_stride % 8 != 0 ||
      (square != 0 && square != 1))
    return ESS_ERR_INVALID_ARG;
  if (dim % 8 != 0) return ESS_ERR_UNSUPPORTED;
  if (n == 0) return ESS_OK;
  if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned_to(scales, 4))
    return ESS_ERR_INVALID_ARG;
  QuantArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.stride = x_stride;
  a.n = static_cast<int>(n);
  a.dim = dim;
  a.groups = (dim - 1) / 128 + 1;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  fast_divisor(a.groups, &a.mul, &a.shift);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (square) {
    const long long high = (n + 127) / 128;
    if (high > 65535) return ESS_ERR_UNSUPPORTED;
    return launch_pdl_once(quant_square_kernel, dim3(a.groups, static_cast<unsigned>(high)),
                           dim3(kQuantThreads), 0, st, a) == cudaSuccess
               ? ESS_OK
               : ESS_ERR_CUDA;
  }
  if (dim <= 128) ++key_norms();   // the next indexer of each layer waits
  // rows of one launch: below 2^30 groups
  const int most = static_cast<int>(std::max(1LL, (1LL << 30) / a.groups));
  for (long long r = 0; r < n; r += most) {
    QuantArgs b = a;
    b.n = static_cast<int>(std::min<long long>(most, n - r));
    b.x += r * x_stride;
    b.codes += r * dim;
    b.scales += r * a.groups;
    const long long items = static_cast<long long>(b.n) * a.groups;
    constexpr int kPer = kQuantThreads / 8;
    if (launch_pdl_once(quant_rows_kernel, dim3(static_cast<unsigned>((items + kPer - 1) / kPer)),
                        dim3(kQuantThreads), 0, st, b) != cudaSuccess)
      return ESS_ERR_CUDA;
  }
  return ESS_OK;
}

ess_status ess_product(const void* x, const float* x_scales, int64_t n, const void* w,
                       const float* w_scales, int32_t outs, int32_t ins, void* out,
                       int64_t out_stride, int32_t fp32, int32_t* status, ess_stream_t stream) {
  if (n < 0 || outs < 1 || ins < 1 || out_stride < outs || (fp32 != 0 && fp32 != 1))
    return ESS_ERR_INVALID_ARG;
  // (a tile's sums are waited for, for about a second: 2^26 values of K take a fifth)
  if (ins % 16 != 0 || ins > 1 << 26 || outs > 0x7fffff00 || n > 0x7fffff00LL)
    return ESS_ERR_UNSUPPORTED;
  if (n == 0) return ESS_OK;
  if (!x || !x_scales || !w || !w_scales || !out || !aligned16(x) || !aligned16(w) ||
      !aligned_to(x_scales, 4) || !aligned_to(w_scales, 4) || !aligned_to(out, fp32 ? 4 : 2) ||
      !aligned_to(status, 4))
    return ESS_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ESS_ERR_CUDA;
  const int sms = sms_of(dev);
  if (sms < 2) return ESS_ERR_CUDA;
  ProdArgs a;
  a.xs = x_scales;
  a.ws = w_scales;
  a.n = static_cast<int>(n);
  a.outs = outs;
  a.groups = (ins - 1) / 128 + 1;
  a.out = out;
  a.stride = out_stride;
  a.wide = a.groups % 4 == 0 && aligned16(x_scales) && aligned16(w_scales);
  a.status = status;
  auto cover = [](long long v, int by) { return static_cast<int>((v + by - 1) / by); };
  // Pairs (256 tokens x 128 columns) where a fifth of the SMs gets a tile (us): 200 x 4096
  // x 4096, 32 tiles, 11.2 against 12.6 in tiles of 128 x 64, 128 x 4096 x 8192, 64 tiles,
  // 11.7 against 12.6, 333 x 4096 x 1600, 26 tiles, 11.1 against 10.7; up to 64 tokens the
  // others: 64 x 4096 x 8192 9.6 against 11.5.  256 columns once tiles of 128 would take
  // more than one wave: 1024 x 4096 x 1600, 52 of 128, 11.8 against 14.4; 512 x 4096 x
  // 8192, 128 of 128, 18.8 against 15.8.  Short sums have registers for 128.
  const long long pair_tiles = static_cast<long long>(cover(outs, 128)) * cover(n, 256);
  const bool pair = n > 64 && pair_tiles >= sms / 5;
  const bool f = fp32 != 0, sums = f || ins > kOneSum;
  const bool wide = !sums && pair_tiles > sms / 2;
  const int bn = pair ? (wide ? 256 : 128) : n <= 16 ? 16 : n <= 32 ? 32 : 64;
  a.m_tiles = pair ? cover(n, 256) : cover(outs, 128);
  a.n_tiles = pair ? cover(outs, bn) : cover(n, bn);
  const long long tiles = static_cast<long long>(a.m_tiles) * a.n_tiles;
  if (tiles > 0x3fffffffLL) return ESS_ERR_UNSUPPORTED;
  const int ctas = 2 * static_cast<int>(std::min<long long>(tiles, sms / 2));   // of pairs
  const int some = static_cast<int>(tiles);
  CUtensorMap wm, xm, om;
  if (!encode_map_2d(&wm, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, ins, outs, ins, 128,
                     pair ? bn / 2 : 128) ||
      !encode_map_2d(&xm, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, ins, n, ins, 128, pair ? 128 : bn))
    return ESS_ERR_CUDA;
  // (a row's end has to be one of 16 bytes too: TMA cuts a block off there, not within)
  const int size = fp32 ? 4 : 2;
  a.blocks = pair && aligned16(out) && out_stride * size % 16 == 0 &&
             static_cast<long long>(outs) * size % 16 == 0;
  if (!a.blocks) om = wm;   // not used
  else if (!encode_map_2d(&om, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                          out, outs, n, static_cast<uint64_t>(out_stride) * size, 128 / size, 32))
    return ESS_ERR_CUDA;
  // rows of 64 bf16 values may be indexer keys, which an indexer loads ahead of its wait
  a.keys = !fp32 && outs <= 64;
  if (a.keys) ++key_norms();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (pair && f) e = launch_product<128, true, float, true>(xm, wm, om, a, ctas, 2, dev, st);
  else if (pair && sums) e = launch_product<128, true, __nv_bfloat16, true>(xm, wm, om, a, ctas, 2, dev, st);
  else if (pair && !wide) e = launch_product<128, true, __nv_bfloat16, false>(xm, wm, om, a, ctas, 2, dev, st);
  else if (pair) e = launch_product<256, true, __nv_bfloat16, false>(xm, wm, om, a, ctas, 2, dev, st);
  else if (bn == 16) e = launch_single<16>(f, sums, wm, xm, a, some, dev, st);
  else if (bn == 32) e = launch_single<32>(f, sums, wm, xm, a, some, dev, st);
  else e = launch_single<64>(f, sums, wm, xm, a, some, dev, st);
  return e == cudaSuccess ? ESS_OK : ESS_ERR_CUDA;
}

}  // extern "C"
