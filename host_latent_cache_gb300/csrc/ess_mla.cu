// Absorbed-MLA attention over a device row cache held in 4 bits.
//
// For every query row (b, m, h): softmax_t(sm_scale * q . row_t) @ row_t[:512]
// over the tokens of request b that way m sees, in one pass with a running
// maximum and sum.
//
// With 128 heads a cached token costs 278 kflop and 400 bytes, so the tensor
// cores are the floor (0.149 ns a token at 1868 TFLOP/s against 0.059 ns at
// 6.78 TB/s).  A pair of CTAs (cta_group::2) shares one tile of 128 tokens and
// 128 query rows, 64 rows a CTA: the pair form with M = 128 runs at the full
// rate (32 cycles for N = 128, 64 for N = 256, as measured) and keeps each
// CTA's O[64][512] in 256 TMEM columns, lanes 64..127 holding the second half
// of the columns.  That leaves room for two score buffers, where one CTA with
// 128 rows would fill TMEM with O alone.
//
//   S[128 rows][128 tokens] = Q K^T   each CTA widens its 64 tokens of K
//   O[128 rows][512]       += P V     each CTA widens its 256 dims of V
//
// The rows' 4-bit codes are widened to fp16, exactly, by one conversion and one
// multiplication a pair.  Queries become fp16 under a power of two of their
// row, P keeps 11 bits, and the 64 RoPE dims stay bf16 in MMAs of their own.
// Sixteen warps gather and widen (and bring in a segment's queries), eight run the
// softmax, one resolves the tokens' rows, one of the even CTA issues the MMAs: QK
// of tile i + 1, then PV of tile i, so the softmax of a tile and the widening of
// the next run beside them.  O is rescaled only when a row's maximum grows by
// more than 2^8: 76 requests of 800 tokens take 28.7 us where it grows at every
// tile, 27.1 where it does not.
//
// What it spends its time on: no unit is saturated.  The data path of shared
// memory and L1 is the busiest (63 % over a ragged launch, the tensor pipe 46 %,
// DRAM 12 %, 0.45 issues a cycle and scheduler), and between its bursts the roles
// wait for loads and for one another.  A tile writes 147 KB of widened operands
// and P, reads 34 KB of raw rows through L1, in pieces of 128 bytes that straddle
// its lines, and the MMAs read 245 KB of operands, beside 2200 cycles of tensor
// work.  All tokens of eight 128K contexts with 128 heads: 188 us, 1.23 PFLOP/s or
// 65 % of the measured tensor rate, 3900 cycles a tile.  Fewer heads cost as much,
// as a tile has 128 query rows whether they are there or not: 182 us with 16 heads,
// 3.7 times what their bytes take.  A segment costs about 5 us beside its tiles: its
// queries (1.2 us of conversions and stores), O's way out (2.2 us) and the
// pipeline's start.
// Measured on the way there (same case): one thread issuing in divergent code
// 526 us (110 cycles an MMA); V before K of the next tile 447; four softmax
// warps, rows resolved by the widening warps 346; lanes across rows (32 lines a
// load) 300; cluster-scope arrivals, which wait for loads in flight, 235; whole
// tiles handed over instead of halves, eight widening warps 211; queries by the
// softmax warps, V loaded whole 197; K's loads after V's first half 190; L2
// prefetches of rows by the row warp +7 %; loads that skip L1 +14 %; warps of
// their own for K and for V +1 %, and for even and odd tiles +17 %; V's loads a
// step earlier, or K's in two halves, +9 to 11 % (more loads in flight than the
// data path takes); any spill of registers in the tile loop 10 to 25 %.
//
// All tiles of all requests are dealt evenly to the pairs, a segment's queries and
// output counted too (lengths are read on the device, so captured calls follow
// them); a request cut by a boundary leaves fp32 partials, which a second kernel
// joins.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstddef>

#include "ess_rows.cuh"

namespace ess {
namespace {

constexpr int kMaxCacheWays = 4;
constexpr int kMaxCacheHeads = 128;
constexpr int kMt = 128;              // tokens per tile
constexpr int kPairRows = 128;        // query rows per pair
constexpr int kCtaRows = 64;          // of them per CTA
constexpr int kMaxPairs = 76;         // one pair per two of the 152 SMs (any number is right)

constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = 8;
constexpr int kWidenWarp0 = 9;
constexpr int kWidenWarps = 16;
constexpr int kRowWarp = kWidenWarp0 + kWidenWarps;
constexpr int kMlaThreads = (kRowWarp + 1) * 32;
// What a segment costs beside its tiles, in tiles, when they are dealt: ragged
// requests to 8192 took 97.3 us with 0, 94.1 with 1, 91.9 with 2, 92.3 with 3.  A chunk's
// segments may be short, and long ones among them: thirteen ragged requests, three of them
// prompts without a prefix, take 1485 us with 3, 1492 with 2; prompts alone 557 and 547.
constexpr int kSegmentCost = 2;
constexpr int kChunkSegmentCost = 3;
constexpr int kRing = 3;              // tiles whose rows are known ahead of their use

constexpr uint32_t kKBlk = 8192;      // [64 rows][64 dims], 128-byte swizzled
constexpr uint32_t kVBlk = 16384;     // [128 tokens][64 dims]
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = 9 * kKBlk;
constexpr uint32_t kOffV = kOffK + 9 * kKBlk;
constexpr uint32_t kOffP = kOffV + 4 * kVBlk;
constexpr uint32_t kOffMisc = kOffP + 2 * kKBlk;

constexpr uint32_t kColO = 0;         // TMEM columns: O, then two score buffers
constexpr uint32_t kColS = 256;
// P is 2^((s - m) c2 + kLift) for a reference m that follows the row's maximum
// score once that is 2^kGrow past it: at most 2^15, inside fp16's range, with
// all 11 bits down to 2^-21 of the largest and steps of 2^-31 of it below that.
// m stays in the scores' own units, where differences are exact, and the
// rounding of m c2 is put back, so scores of any size keep their weights.
constexpr float kGrow = 8.0f;
constexpr float kLift = 7.0f;

struct Misc {
  uint64_t q_ready, q_here[2], q_free, k_full[2], vp_full[2], qk_half, qk_done[2], pv_half, pv_done;
  uint64_t row_full[kRing], row_free[kRing];
  uint32_t tmem;
  int abort;
  int start_v, start_rt, start_tile;
  long long first_tile, end_tile;     // of all tiles of all requests
  uint32_t mask[kRing][4];            // tokens of a tile that exist
  int32_t row[kRing][kMt];            // cache rows of a tile's tokens (0 for one that is not)
  float xch[4][kCtaRows];             // a row's statistics from the four threads that share it
  int2 seg[kRing];                    // entry and row tile of a segment that a tile begins, or -1
  int8_t qexp[2][kCtaRows];           // log2 of what a query row was divided by, of two segments
  int fell;                           // chunks: some offset is below the one before it
};
constexpr uint32_t kMlaSmem = 232448;
static_assert(kOffMisc + sizeof(Misc) <= kMlaSmem, "shared memory of one CTA");
static_assert(offsetof(Misc, xch) % 8 == 0 && kMlaThreads / 32 * 8 <= sizeof(Misc::xch) &&
                  kRing * kMt <= kMlaThreads,
              "the scan's scratch, and the rows' first values");

struct MlaArgs {
  const uint16_t* q;
  const uint8_t* rows;
  int n_rows;
  const int32_t* page_table;
  int max_pages, page;
  int page_shift;          // log2(page), or -1
  const int32_t* T;
  int batch, ways, heads;
  const int32_t* tokens;
  int k;
  int entries;             // dense: requests; listed: (request, way)
  int row_tiles;           // pairs' row tiles per entry
  int entry_rows;          // query rows per entry
  float c2;                // sm_scale * log2(e)
  uint16_t* out;
  float* lse;
  const int32_t* cu;       // chunks: [batch + 1] first query token of each request
  int total;               // chunks: query tokens
  int unit_rows;           // chunks: query rows that share tiles: 128, or a token's heads
  bool wide_out;           // chunks: out is 32-byte aligned
  int pairs;               // chunks: pairs of the launch
  int4* rec;               // chunks: [pairs] which units the pairs cut
  int2* span;              // [entries][row_tiles]: first pair * 2 + slot, last pair
  float* part_o;           // [pairs][2][512 / 8][128][8]: a lane's 32 bytes beside its neighbours'
  float4* part_ml;         // [pairs][2][128]: reference, sum, c2 of the row
  int* status;
  volatile int* unit0;     // chunks whose offsets fall: [batch + 1] units of the requests before
};

__device__ __forceinline__ int request_len(const MlaArgs& a, int b) {
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  const int T = a.T[b];
  return T < 0 ? 0 : (T > cap ? static_cast<int>(cap) : T);
}
__device__ __forceinline__ int entry_len(const MlaArgs& a, int v) {
  return a.tokens ? min(a.k, request_len(a, v / a.ways)) : request_len(a, v);
}

// ---------------------------------------------------------------- chunks
// (See the head of the file for the tiles.  Measured: 512 new tokens of 32768 x 128 heads
// 3.34 ms, 1.39 PFLOP/s or 81 % of the measured sustained rate; seven ragged requests with
// 556 new tokens to 8192 528 us, 1.23 PFLOP/s; lists of 2048 for 320 tokens 187 us, with 16
// heads 167; twelve prompts of 20 to 700 tokens 557 us; 16 new tokens of 4096 x 16 heads
// 19.8 us; 1000 requests of 3 new tokens of 70 x 16 heads 98 us.  A tile takes 1.95 us and a
// segment 4 beside its tiles: the last softmax and P V, O's way out, the next queries,
// during which the tensor cores wait.  Under ncu, 128 new tokens of 8192: the data path of
// shared memory and L1 72 %, the tensor pipe 53 %, DRAM 1 %.)
//
// Requests with any number of new tokens each (CHUNK).  Request b's queries are the rows
// [start, start + n) x heads of q, its newest tokens.  What a segment belongs to is a
// unit: unit_rows neighbouring query rows of a request, dense 128 of them, listed one
// token's heads.  A unit's tokens end with those that its last row sees; rows that see
// fewer are masked.  Every unit has a tile, though none of its tokens may exist, so that
// every row is written.  The join finds the units that were cut from what each pair
// leaves in rec: x the first query row of the unit that the pair starts inside of (-1:
// none), y that unit's rows, w the slot of the partial that the pair ends with.
struct Chunk {
  int start, n;   // n = 0 for offsets that are out of order or range
  bool ok;
};
__device__ __forceinline__ Chunk chunk_of(const MlaArgs& a, int b) {
  const int lo = a.cu[b], hi = a.cu[b + 1];
  const bool ok = lo >= 0 && lo <= hi && hi <= a.total;
  return Chunk{ok ? lo : 0, ok ? hi - lo : 0, ok};
}
__device__ __forceinline__ int units_of(const MlaArgs& a, int n) {
  return (n * a.heads + a.unit_rows - 1) / a.unit_rows;
}
// Where offsets fall, and then rise again, a request that starts ahead of the end of one
// before it has no units: so a query row belongs to one unit at most, and there are no more
// units than the host counts.  The units that are left are kept in the workspace then, the
// same numbers from every CTA, as each walks over them.
__device__ __forceinline__ int end_before(const MlaArgs& a, int b) {
  int end = 0;
  for (int i = 0; i < b; ++i) {
    const Chunk c = chunk_of(a, i);
    end = max(end, c.n > 0 ? c.start + c.n : 0);
  }
  return end;
}
// Units of request b behind those that leave off at `end`, which becomes its own end.
__device__ __forceinline__ int units_behind(const MlaArgs& a, int b, int* end) {
  const Chunk c = chunk_of(a, b);
  const int units = c.start < *end ? 0 : units_of(a, c.n);
  *end = max(*end, c.n > 0 ? c.start + c.n : 0);
  return units;
}
__device__ __forceinline__ int request_units(const MlaArgs& a, int b, bool fell) {
  return fell ? a.unit0[b + 1] - a.unit0[b] : units_of(a, chunk_of(a, b).n);
}
// Tokens that the last row of unit u of a request sees.
__device__ __forceinline__ int unit_sees(const MlaArgs& a, int T, int n, int u) {
  const int last = min(n * a.heads, (u + 1) * a.unit_rows) - 1;
  return max(T - n + last / a.heads + 1, 0);
}
// Listed: entries of a unit's list; dense: its tokens.
__device__ __forceinline__ int unit_len(const MlaArgs& a, int T, int n, int u) {
  const int sees = unit_sees(a, T, n, u);
  return a.tokens ? min(a.k, sees) : sees;
}
__device__ __forceinline__ int unit_tiles(int len) { return max((len + kMt - 1) / kMt, 1); }

// A walk over the units of all requests.
struct UnitWalk {
  const int* unit0;   // [batch + 1]: units of the requests before each
  int b, u, n, T;
  __device__ __forceinline__ void load(const MlaArgs& a) {
    n = chunk_of(a, b).n;
    T = request_len(a, b);
  }
  __device__ __forceinline__ void start(const MlaArgs& a, const int* first, int v, bool live) {
    unit0 = first;
    int lo = 0, hi = live ? a.batch - 1 : 0;   // the last request that starts at v or before
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (unit0[mid] <= v) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    load(a);
    u = live ? v - unit0[b] : 0;
  }
  __device__ __forceinline__ int tiles(const MlaArgs& a) const {
    return unit_tiles(unit_len(a, T, n, u));
  }
  __device__ __forceinline__ void next(const MlaArgs& a) {
    for (++u; u >= unit0[b + 1] - unit0[b] && b + 1 < a.batch; u = 0) {
      ++b;
      load(a);
    }
  }
};
constexpr int kMaxChunkBatch = 32768;
static_assert((kMaxChunkBatch + 1) * sizeof(int) <= kOffMisc,
              "the first units, in the operands' place");

// The deal counts tiles and segments in one 64-bit sum, tiles below this bit and segments
// above it.  Entries are at most 65535 requests x 4 segments, of 2^24 tiles each.  Chunks
// may have a unit for each query token: calls whose units or tiles could reach these
// limits are refused, which keeps a pair's tiles within an int as well.
constexpr int kSegShift = 43;
constexpr int kChunkSegShift = 37;
constexpr long long kMaxChunkTiles = 1LL << kChunkSegShift;
constexpr long long kMaxChunkUnits = 1LL << (63 - kChunkSegShift);
static_assert(kMaxChunkTiles / kMaxPairs < 0x7fffffffLL, "a pair's tiles");

// Units of all requests; unit0[b], those before request b.  All threads call it.
__device__ __forceinline__ int chunk_units(const MlaArgs& a, int* unit0, int* sums, int* fell_out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.batch + kMlaThreads - 1) / kMlaThreads;
  const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  int mine = 0, before;
  bool bad = false, falls = false, fell = false;
  for (int b = b0; b < b1; ++b) {
    const Chunk c = chunk_of(a, b);
    const int T = a.T[b];
    bad |= !c.ok || T < 0 || T > static_cast<long long>(a.max_pages) * a.page;
    falls |= a.cu[b + 1] < a.cu[b];
    mine += units_of(a, c.n);
  }
  if (bad && blockIdx.x == 0) set_status(a.status, ESS_ERR_DEVICE_CHECK);
  for (;;) {
    before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += x;
    }
    if (lane == 31) sums[warp] = before;
    if (!__syncthreads_or(falls)) break;
    fell = true;   // counted again, without the requests that start inside another
    falls = false;
    mine = 0;
    for (int b = b0, end = end_before(a, b0); b < b1; ++b) mine += units_behind(a, b, &end);
  }
  int all = lane < kMlaThreads / 32 ? sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += x;
  }
  const int total = __shfl_sync(0xffffffffu, all, 31);
  const int earlier = __shfl_sync(0xffffffffu, all, max(warp - 1, 0));
  before += (warp > 0 ? earlier : 0) - mine;
  int end = fell ? end_before(a, b0) : 0;
  for (int b = b0; b < b1; ++b) {
    unit0[b] = before;
    if (fell) a.unit0[b] = before;
    before += fell ? units_behind(a, b, &end) : units_of(a, chunk_of(a, b).n);
  }
  if (tid == 0) {
    unit0[a.batch] = total;
    if (fell) a.unit0[a.batch] = total;
    *fell_out = fell;
  }
  __syncthreads();
  return total;
}

// ---------------------------------------------------------------- pair PTX
// REUSE: 0 reads A from shared memory, 1 does and keeps it in the collector
// buffer, 2 takes it from there (the MMA before had the same A).
template <int REUSE>
__device__ __forceinline__ void umma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
#define ESS_UMMA_PAIR(collector)                                                              \
  asm volatile(                                                                               \
      "{\n\t.reg .pred p;\n\t"                                                                \
      "setp.ne.b32 p, %4, 0;\n\t"                                                             \
      "tcgen05.mma.cta_group::2.kind::f16" collector " [%0], %1, %2, %3, p;\n\t}\n" ::"r"(     \
          d_tmem),                                                                            \
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)                                   \
      : "memory")
  if (REUSE == 1) ESS_UMMA_PAIR(".collector::a::fill");
  else if (REUSE == 2) ESS_UMMA_PAIR(".collector::a::lastuse");
  else ESS_UMMA_PAIR("");
#undef ESS_UMMA_PAIR
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// four runs of 8 consecutive columns of this lane, 64 columns apart
__device__ __forceinline__ void tmem_ld8x4(uint32_t t, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%33];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%34];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%24,%25,%26,%27,%28,%29,%30,%31}, [%35];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t), "r"(t + 64), "r"(t + 128), "r"(t + 192)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// two runs of 8 consecutive columns of this lane, 64 columns apart
__device__ __forceinline__ void tmem_ld8x2(uint32_t t, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(t), "r"(t + 64)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// 32 bytes, 32-byte aligned, in one store
__device__ __forceinline__ void st_global_32(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// this lane's 4 consecutive columns times f, in place
__device__ __forceinline__ void tmem_scale4(uint32_t taddr, float f) {
  uint32_t r[4];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// Barrier over `threads` threads that says whether any of them has x.
__device__ __forceinline__ bool named_any(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Natural logarithm of a row's softmax sum from its reference and scaled sum.
__device__ __forceinline__ float row_lse(float m, float c2, float l) {
  return l > 0.0f || l != l ? (fmaf(m, c2, -kLift) + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// The tiles of one pair, in order: entry v, row tile rt, token tile (chunks: request v,
// unit rt of it).
template <bool CHUNK>
struct Tiles {
  int left;   // tiles from this one on
  int v, rt, tile, nt, len;
  bool begins;   // the pair's first tile

  __device__ __forceinline__ Tiles(const MlaArgs& a, const Misc* mi) {
    left = static_cast<int>(mi->end_tile - mi->first_tile);
    v = mi->start_v;
    if (CHUNK) rt = mi->start_rt;
    load(a);
    rt = mi->start_rt;
    tile = mi->start_tile;
    begins = true;
  }
  __device__ __forceinline__ void load(const MlaArgs& a) {
    if (CHUNK) {
      len = unit_len(a, request_len(a, v), chunk_of(a, v).n, rt);
      nt = unit_tiles(len);
    } else {
      len = entry_len(a, v);
      nt = (len + kMt - 1) / kMt;
    }
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  // of a segment: a run of tiles of one entry and row tile
  __device__ __forceinline__ bool first() const { return begins || tile == 0; }
  __device__ __forceinline__ bool last() const { return left == 1 || tile + 1 == nt; }
  __device__ __forceinline__ void next(const MlaArgs& a, const Misc* mi) {
    begins = false;
    --left;
    if (++tile == nt && left > 0) {
      tile = 0;
      if (CHUNK) {
        ++rt;
        while (v + 1 < a.batch && rt >= request_units(a, v, mi->fell)) {
          rt = 0;
          ++v;
        }
        load(a);
      } else if (++rt == a.row_tiles) {
        rt = 0;
        do {   // a tile is left, so an entry that has one follows
          ++v;
          load(a);
        } while (nt == 0);
      }
    }
  }
};

// Where a unit's query rows lie: row r of the pair is row first + r of q and out, for
// r < rows.
struct QueryRows {
  size_t first;
  int rows;
};
__device__ __forceinline__ QueryRows query_rows(const MlaArgs& a, int v, int rt) {
  const Chunk c = chunk_of(a, v);
  return QueryRows{static_cast<size_t>(c.start) * a.heads + static_cast<size_t>(rt) * a.unit_rows,
                   min(c.n * a.heads - rt * a.unit_rows, a.unit_rows)};
}

// The cache rows of a lane's four tokens e, e + 32, .. of an entry, -1 for one
// that is not.  The four list entries are loaded together, then the four page
// table entries, so that a tile costs one latency of each.
template <bool CHUNK>
__device__ __forceinline__ void token_rows(const MlaArgs& a, int v, int rt, int len, int e,
                                           int* row) {
  int t[4], pg[4];
  const int b = !CHUNK && a.tokens ? v / a.ways : v;
  int T, list = v;   // tokens that may be named, and by which list
  if constexpr (CHUNK) {
    T = len;
    if (a.tokens) {
      const Chunk c = chunk_of(a, b);
      T = unit_sees(a, request_len(a, b), c.n, rt);
      list = c.start + rt;
    }
  } else {
    T = a.tokens ? request_len(a, b) : len;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int x = e + 32 * j;
    t[j] = x;
    if (a.tokens) t[j] = x < len ? a.tokens[static_cast<size_t>(list) * a.k + x] : -1;
    else if (x >= len) t[j] = -1;
  }
  const int32_t* table = a.page_table + static_cast<size_t>(b) * a.max_pages;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int u = t[j] >= 0 && t[j] < T ? t[j] : 0;
    pg[j] = a.page_shift >= 0 ? u >> a.page_shift : u / a.page;
    row[j] = u - pg[j] * a.page;
    pg[j] = t[j] >= 0 && t[j] < T ? table[pg[j]] : -1;
  }
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long long r = static_cast<long long>(pg[j]) * a.page + row[j];
    const bool ok = pg[j] >= 0 && r < a.n_rows;
    bad |= !ok && t[j] >= 0;
    row[j] = ok ? static_cast<int>(r) : -1;
  }
  if (bad) set_status(a.status, ESS_ERR_DEVICE_CHECK);
}

// 32 codes (one block) -> four 16-byte units of fp16
__device__ __forceinline__ void widen_block(const uint4& codes, int byte, uint4* unit) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  const __half2 s2 =
      __float2half2_rn(__uint_as_float(static_cast<uint32_t>(q4_exp_byte(byte)) << 23));
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t h[4];
    e2m1_to_f16x2(w[q], h);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&h[e]), s2);
      h[e] = *reinterpret_cast<const uint32_t*>(&r);
    }
    unit[q] = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

__device__ __forceinline__ uint4 pick4(bool p, const uint4& a, const uint4& b) {
  return make_uint4(p ? a.x : b.x, p ? a.y : b.y, p ? a.z : b.z, p ? a.w : b.w);
}

// ---------------------------------------------------------------- roles
// One warp resolves the cache rows of the tiles to come, four tokens a lane,
// up to kRing tiles ahead, so that the page table's latency meets nobody.
template <bool CHUNK>
__device__ __forceinline__ void row_role(const MlaArgs& a, Misc* mi) {
  const int lane = threadIdx.x & 31;
  Tiles<CHUNK> it(a, mi);
  int slot = 0, turn = 0;
  for (int g = 0; it.more(); ++g) {
    int row[4];
    token_rows<CHUNK>(a, it.v, it.rt, it.len, it.tile * kMt + lane, row);
    if (turn > 0) wait_or_abort(&mi->row_free[slot], (turn - 1) & 1, mi, a.status);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      mi->row[slot][32 * j + lane] = max(row[j], 0);
      const uint32_t m = __ballot_sync(0xffffffffu, row[j] >= 0);
      if (lane == 0) mi->mask[slot][j] = m;
    }
    if (it.first() && g > 0) {   // the segment's queries into L2
      const int row0 = (CHUNK ? 0 : it.rt * kPairRows) +
                       static_cast<int>(cluster_ctarank()) * kCtaRows;
      QueryRows unit{static_cast<size_t>(it.v) * a.entry_rows, a.entry_rows};
      if constexpr (CHUNK) unit = query_rows(a, it.v, it.rt);
      const char* q = reinterpret_cast<const char*>(a.q + (unit.first + row0) * kRowDim);
      const int bytes = min(kCtaRows, unit.rows - row0) * kRowDim * 2;
      for (int x = lane * 128; x < bytes; x += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + x));
    }
    if (lane == 0) mi->seg[slot] = make_int2(it.first() ? it.v : -1, it.rt);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&mi->row_full[slot]));
    if (++slot == kRing) {
      slot = 0;
      ++turn;
    }
    it.next(a, mi);
  }
}

// Four rows of queries per widening warp into shared memory, all in flight: the latent
// part as fp16, beside the fp16 latents, each row divided by the power of two that brings
// its largest value to [2^14, 2^15) (exact down to 2^-31 of that value, with an error below
// 2^-39 of it under that); the RoPE part, divided alike, as bf16.  A lane takes unit
// 32 h + 4 (lane % 8) + lane / 8: chunk 8 h + lane % 8, its unit lane / 8; eight lanes then
// fill the places of one swizzled row.
template <bool CHUNK>
__device__ __forceinline__ void load_queries(const MlaArgs& a, uint8_t* smem, Misc* mi, int v,
                                             int rt, int q0, int warp, int lane, int seg) {
  constexpr int kRows = kCtaRows / kWidenWarps;
  uint8_t* sq = smem + kOffQ;
  int row0 = rt * kPairRows + q0;
  int rows = 0;
  size_t first = 0;
  if constexpr (CHUNK) {
    const Chunk c = chunk_of(a, v);
    row0 = rt * a.unit_rows + q0;
    rows = min(c.n * a.heads, (rt + 1) * a.unit_rows);
    first = static_cast<size_t>(c.start) * a.heads;
  }
  const int un = 4 * (lane & 7) + (lane >> 3);
  uint4 u[kRows][2];
  uint32_t rope[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + warp * kRows + i;
    u[i][0] = u[i][1] = make_uint4(0u, 0u, 0u, 0u);
    rope[i] = 0u;
    if (row < (CHUNK ? rows : a.entry_rows)) {
      const uint16_t* q =
          a.q + ((CHUNK ? first : static_cast<size_t>(v) * a.entry_rows) + row) * kRowDim;
      u[i][0] = reinterpret_cast<const uint4*>(q)[un];
      u[i][1] = reinterpret_cast<const uint4*>(q)[32 + un];
      rope[i] = reinterpret_cast<const uint32_t*>(q + kLatent)[lane];
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp * kRows + i;
    float x[16];
    unpack8(u[i][0], x);
    unpack8(u[i][1], x + 8);
    const float ra = bf16_lo(rope[i]), rb = bf16_hi(rope[i]);
    const float mx = __uint_as_float(__reduce_max_sync(
        0xffffffffu, __float_as_uint(fmaxf(fmaxf(amax8(x), amax8(x + 8)),
                                           fmaxf(fabsf(ra), fabsf(rb))))));
    // 2^e <= mx < 2^(e + 1); rows of zeros, infinities and NaN as they are
    const int e = mx > 0.0f && mx < INFINITY
                      ? static_cast<int>(__float_as_uint(mx) >> 23) - 127 - 14
                      : 0;
    const int ec = min(max(e, -126), 126);
    const float inv = exp2i(-ec);
    if (lane == 0) mi->qexp[seg & 1][r] = static_cast<int8_t>(ec);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* y = x + 8 * h;
      *reinterpret_cast<uint4*>(sq + (4 * h + (lane >> 3)) * kKBlk + sw128_off(r, lane & 7)) =
          make_uint4(half2_bits(y[0] * inv, y[1] * inv), half2_bits(y[2] * inv, y[3] * inv),
                     half2_bits(y[4] * inv, y[5] * inv), half2_bits(y[6] * inv, y[7] * inv));
    }
    *reinterpret_cast<uint32_t*>(sq + 8 * kKBlk + sw128_off(r, lane >> 2) + (lane & 3) * 4) =
        bf16x2_bits(ra * inv, rb * inv);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(smem_u32(&mi->q_here[seg & 1]));   // this CTA's softmax reads the powers
    mbar_arrive_remote(dsmem_addr(smem_u32(&mi->q_ready), 0));
  }
}

// Sixteen warps: gather the rows of a tile and widen them, K of this CTA's 64
// tokens, and V of its 256 dims of all 128 tokens.  Eight neighbouring lanes
// read 128 neighbouring bytes of one row, eight chunks of 32 codes; each chunk
// makes four 16-byte units of 8 dims.  Unit q of chunk c goes to 64-dim block
// q (of four), place c: at every store the eight lanes then fill all eight
// bank groups of one swizzled row.  So the dims lie in the order
// (half, q, c, 8 dims) for (half, c, q, 8 dims); Q is stored in the same
// order, and O comes out in it.  A token that does not exist reads row 0: its
// scores are masked, and its V, finite like all codes, meets P = 0.
//
// K is written in two halves of its dims and V in two halves of the tokens,
// each as soon as the MMAs that read the half before it are done.
template <bool CHUNK>
__device__ __forceinline__ void widen_role(const MlaArgs& a, uint8_t* smem, Misc* mi,
                                           uint32_t rank) {
  const int wt = threadIdx.x - kWidenWarp0 * 32;
  const int w = wt >> 5, lane = wt & 31;
  const int n = static_cast<int>(mi->end_tile - mi->first_tile);
  const int c8 = lane & 7, r4 = 4 * w + (lane >> 3);   // K's row; V's tokens r4 and 64 + r4
  const uint8_t* code = a.rows + 16 * c8;
  const uint32_t place = static_cast<uint32_t>(r4 * 128 + ((c8 ^ (r4 & 7)) << 4));
  uint8_t* sk = smem + kOffK + place;
  uint8_t* sv = smem + kOffV + place;

  // Raw codes and exponent bytes: K's two halves of the dims and its RoPE unit,
  // and this CTA's dims of two tokens of V: one that is K's row too, kept from K
  // (loaded again it cost 1.6 % of the long attention), and one of the other CTA's.
  uint4 kc[2], kr, own, other;
  int ke[2], own_e, other_e;
  auto at = [](int row) { return static_cast<size_t>(static_cast<uint32_t>(row)) * kQ4RowBytes; };
  auto load_k = [&](int slot) {
    const uint8_t* s = code + at(mi->row[slot][rank * kCtaRows + r4]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      kc[h] = *reinterpret_cast<const uint4*>(s + 128 * h);
      ke[h] = s[256 + 8 * h - 15 * c8];
    }
    kr = *reinterpret_cast<const uint4*>(s + 272);
  };
  auto load_v = [&](int slot) {
    const uint8_t* s = code + 128 * rank + at(mi->row[slot][64 * (rank ^ 1) + r4]);
    other = *reinterpret_cast<const uint4*>(s);
    other_e = s[256 - 120 * static_cast<int>(rank) - 15 * c8];
  };
  auto put = [&](uint8_t* d, uint32_t block_bytes, const uint4& codes, int byte) {
    uint4 unit[4];
    widen_block(codes, byte, unit);
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(d + q * block_bytes) = unit[q];
  };
  auto told = [&](uint64_t* bar) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_remote(dsmem_addr(smem_u32(bar), 0));
  };
  auto store_k = [&](int h) {
    put(sk + h * 4 * kKBlk, kKBlk, kc[h], ke[h]);
    if (h == 1) *reinterpret_cast<uint4*>(sk + 8 * kKBlk) = kr;
    told(&mi->k_full[h]);
  };
  auto store_v = [&](int h, const uint4& codes, int byte) {
    put(sv + h * 64 * 128, kVBlk, codes, byte);
    told(&mi->vp_full[h]);
  };
  // K runs one tile ahead of V: K of tile g + 1 is written beside PV of tile
  // g - 1, V of tile g beside QK of tile g + 1.  Slot s of the rows holds tile
  // g for the (g / kRing)th time.
  const int q0 = static_cast<int>(rank) * kCtaRows;
  load_queries<CHUNK>(a, smem, mi, mi->start_v, mi->start_rt, q0, w, lane, 0);
  int seg = 0;
  wait_or_abort(&mi->row_full[0], 0, mi, a.status);
  load_k(0);
  load_v(0);
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&mi->row_free[0]));
  store_k(0);
  store_k(1);
  own = pick4(rank, kc[1], kc[0]);
  own_e = rank ? ke[1] : ke[0];
  if (n > 1) {
    wait_or_abort(&mi->row_full[1], 0, mi, a.status);
    load_k(1);
  }
  int slot2 = 2, turn2 = 0;   // of tile g + 2
  int slot1 = 1;              // of tile g + 1
  for (int g = 0; g < n; ++g) {
    if (g + 1 < n) {
      wait_or_abort(&mi->qk_half, g & 1, mi, a.status);
      store_k(0);
      wait_or_abort(&mi->qk_done[g & 1], (g >> 1) & 1, mi, a.status);
      store_k(1);
    }
    if (g + 2 < n) wait_or_abort(&mi->row_full[slot2], turn2 & 1, mi, a.status);
    const uint4 c0 = pick4(rank, other, own), c1 = pick4(rank, own, other);
    const int e0 = rank ? other_e : own_e, e1 = rank ? own_e : other_e;
    own = pick4(rank, kc[1], kc[0]);   // of tile g + 1
    own_e = rank ? ke[1] : ke[0];
    if (g + 2 < n) load_k(slot2);
    if (g > 0) wait_or_abort(&mi->pv_half, (g - 1) & 1, mi, a.status);
    store_v(0, c0, e0);
    if (g > 0) wait_or_abort(&mi->pv_done, (g - 1) & 1, mi, a.status);
    store_v(1, c1, e1);
    if (g + 1 < n) {
      const int2 next = mi->seg[slot1];
      // The next tile begins a segment: its queries, beside this one's softmax and
      // output.  (Before V they would be there sooner, but with V's codes in
      // registers too the tile loop spills, or with two rows in flight costs 2 %.  Here
      // four rows in flight are 0.35 us a segment faster than two.)
      if (next.x >= 0) {
        wait_or_abort(&mi->q_free, seg & 1, mi, a.status);
        load_queries<CHUNK>(a, smem, mi, next.x, next.y, q0, w, lane, ++seg);
      }
      load_v(slot1);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&mi->row_free[slot1]));
    }
    slot1 = slot2;
    if (++slot2 == kRing) {
      slot2 = 0;
      ++turn2;
    }
  }
  // the last arrivals on these two, which nothing else waits for
  wait_or_abort(&mi->qk_half, (n - 1) & 1, mi, a.status);
  wait_or_abort(&mi->pv_half, (n - 1) & 1, mi, a.status);
}

// One warp of the even CTA issues the MMAs.  The whole warp walks the tiles and
// one elected lane issues: with uniform control flow the descriptors stay in
// uniform registers, and an MMA is issued every 32 cycles (N = 128).  The two
// MMAs of PV that share a slice of P read it from shared memory once.
template <bool CHUNK>
__device__ __forceinline__ void mma_role(const MlaArgs& a, uint8_t* smem, Misc* mi,
                                         uint32_t tmem) {
  const uint64_t dq = make_sdesc_sw128(smem_u32(smem + kOffQ), 16, 1024);
  const uint64_t dk = make_sdesc_sw128(smem_u32(smem + kOffK), 16, 1024);
  const uint64_t dv = make_sdesc_sw128(smem_u32(smem + kOffV), kVBlk, 1024);
  const uint64_t dp = make_sdesc_sw128(smem_u32(smem + kOffP), 16, 1024);
  const uint32_t idesc_qk = make_idesc(kFmtF16, kFmtF16, 0, kMt, kPairRows);
  const uint32_t idesc_rope = make_idesc(kFmtBF16, kFmtBF16, 0, kMt, kPairRows);
  const uint32_t idesc_pv = make_idesc(kFmtF16, kFmtF16, 1, 256, kPairRows);
  const bool lead = elect_one();
  bool ok = true;
  auto pv = [&](int g, bool accumulate) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // 64 tokens each
      ok = wait_or_abort(&mi->vp_full[h], g & 1, mi, a.status) && ok;
      tc_fence_after();
      if (ok && lead) {
#pragma unroll
        for (int kt = 4 * h; kt < 4 * h + 4; ++kt) {
          const uint64_t ad = dp + (h * kKBlk + (kt & 3) * 32) / 16, bd = dv + kt * 2048 / 16;
          const uint32_t more = accumulate || kt > 0;
          umma_f16_pair<1>(tmem + kColO, ad, bd, idesc_pv, more);
          umma_f16_pair<2>(tmem + kColO + 128, ad, bd + 2 * kVBlk / 16, idesc_pv, more);
        }
        umma_commit_pair(smem_u32(h == 0 ? &mi->pv_half : &mi->pv_done));
      }
      __syncwarp();
    }
  };
  int seg = 0;
  bool acc = false;   // the tile before was not the first of its segment
  Tiles<CHUNK> it(a, mi);
  for (int g = 0; it.more(); ++g) {
    const bool first = it.first(), last = it.last();
    if (first) {
      if (g > 0) pv(g - 1, acc);
      ok = wait_or_abort(&mi->q_ready, seg & 1, mi, a.status) && ok;
      ++seg;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // 256 dims each, the RoPE dims with the second
      ok = wait_or_abort(&mi->k_full[h], g & 1, mi, a.status) && ok;
      tc_fence_after();
      if (ok && lead) {
#pragma unroll
        for (int k = 16 * h; k < 16 + 20 * h; ++k)
          umma_f16_pair<0>(tmem + kColS + (g & 1) * 64, dq + ((k >> 2) * kKBlk + (k & 3) * 32) / 16,
                        dk + ((k >> 2) * kKBlk + (k & 3) * 32) / 16,
                        k < 32 ? idesc_qk : idesc_rope, k != 0);
        umma_commit_pair(smem_u32(h == 0 ? &mi->qk_half : &mi->qk_done[g & 1]));
        if (h == 1 && last) umma_commit_pair(smem_u32(&mi->q_free));
      }
      __syncwarp();
    }
    if (!first) pv(g - 1, acc);
    acc = !first;
    it.next(a, mi);
    if (!it.more()) pv(g, acc);
  }
}

// Eight warps.  Four threads share a query row: (half, sub) names 32 of a
// tile's tokens, and 128 of the row's output dims.
template <bool CHUNK>
__device__ __forceinline__ void softmax_role(const MlaArgs& a, uint8_t* smem, Misc* mi,
                                             uint32_t rank, uint32_t tmem, int pair) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = (warp & 1) * 32 + lane, half = (warp >> 1) & 1, sub = warp >> 2;
  const int part = 2 * half + sub;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t to = tmem + lanes + kColO + sub * 128;
  uint8_t* sp = smem + kOffP + half * kKBlk;
  const int bar_id = 1 + (warp & 1);   // the four warps that hold the same rows
  float m = -INFINITY, l = 0.0f, c2 = 0.0f;
  int limit = 0, seg_first_tile = 0, seg = 0;
  Tiles<CHUNK> it(a, mi);
  for (int g = 0; it.more(); ++g) {
    const bool first = it.first(), last = it.last();
    if (first) {
      if (CHUNK) {
        const int row = it.rt * a.unit_rows + static_cast<int>(rank) * kCtaRows + r;
        const int n = chunk_of(a, it.v).n;
        limit = row - it.rt * a.unit_rows >= a.unit_rows || row >= n * a.heads ? 0 : it.len;
        if (!a.tokens && limit) limit = request_len(a, it.v) - n + row / a.heads + 1;
      } else {
        const int row = it.rt * kPairRows + static_cast<int>(rank) * kCtaRows + r;
        limit = row >= a.entry_rows ? 0 : it.len;
        if (!a.tokens && limit) limit = it.len - (a.ways - 1) + row / a.heads;
      }
      // The rows' powers of two.  Those of the segment after the next wait for
      // this one's P, so two places and two barriers are enough.
      wait_or_abort(&mi->q_here[seg & 1], (seg >> 1) & 1, mi, a.status);
      // at least 2^-126: |s| < 2^41 then still weighs less than half a step of
      // 1 apart, and 0 * infinity does not arise; finite, for the same reason
      c2 = fminf(fmaxf(a.c2 * exp2i(mi->qexp[seg & 1][r]), 0x1p-126f), FLT_MAX);
      m = -INFINITY;
      l = 0.0f;
      seg_first_tile = it.tile;
    }
    bool ok = wait_or_abort(&mi->qk_done[g & 1], (g >> 1) & 1, mi, a.status);
    tc_fence_after();
    uint32_t live = mi->mask[g % kRing][part];
    const int nv = limit - it.tile * kMt - part * 32;   // tokens of these 32 before the limit
    if (nv < 32) live = nv <= 0 ? 0u : live & ((1u << nv) - 1u);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&mi->row_free[g % kRing]));
    float s[32];
    tmem_ld32(tmem + lanes + kColS + (g & 1) * 64 + sub * 32, s);
    if (live != 0xffffffffu) {
#pragma unroll
      for (int c = 0; c < 32; ++c) s[c] = (live >> c) & 1u ? s[c] : -INFINITY;
    }
    float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int c = 4; c < 28; c += 8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) m4[e] = fmaxf(fmaxf(m4[e], s[c + e]), s[c + 4 + e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], s[28 + e]);
    float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
    // The row's maximum is only looked up when one of its parts outgrew the
    // one in use (or there is none yet: a difference of infinity).
    float f = 1.0f;
    const bool grown = named_any(bar_id, kSoftWarps * 16, (mt - m) * c2 > kGrow);
    if (grown) {
      mi->xch[part][r] = mt;
      named_sync(bar_id, kSoftWarps * 16);
      mt = fmaxf(fmaxf(mi->xch[0][r], mi->xch[1][r]), fmaxf(mi->xch[2][r], mi->xch[3][r]));
      named_sync(bar_id, kSoftWarps * 16);
      if (m == -INFINITY) {
        m = mt;   // nothing summed yet: O's row is zero
      } else if ((mt - m) * c2 > kGrow) {
        f = ex2_approx((m - mt) * c2);
        m = mt;
      }
    }
    const float hi = m == -INFINITY ? 0.0f : m * c2;
    const float lo = m == -INFINITY ? 0.0f : fmaf(m, c2, -hi);
    const F2 c2v = both(c2), hv = both(-hi), lv = both(kLift - lo);
    F2 sum2[2] = {both(0.0f), both(0.0f)};
    uint32_t p[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      F2 z = add2(fma2(F2{s[2 * c], s[2 * c + 1]}, c2v, hv), lv);
      z.x = ex2_approx(z.x);
      z.y = ex2_approx(z.y);
      sum2[c & 1] = add2(sum2[c & 1], z);
      p[c] = half2_bits(z.x, z.y);
    }
    sum2[0] = add2(sum2[0], sum2[1]);
    l = fmaf(l, f, sum2[0].x + sum2[0].y);
    // P and O are free once PV of the tile before is done
    if (g > 0) ok = wait_or_abort(&mi->pv_done, (g - 1) & 1, mi, a.status) && ok;
    if (!first && grown) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 32; ++c) tmem_scale4(to + 4 * c, f);
      tmem_wait_st();
      // Each half of PV adds to all of O's columns, so these rows are scaled in both
      // halves before any of the four warps lets its own half start.  (grown is the
      // barrier's answer: all four come here or none.)
      tc_fence_before();
      named_sync(bar_id, kSoftWarps * 16);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<uint4*>(sp + sw128_off(r, 4 * sub + u)) =
          make_uint4(p[4 * u], p[4 * u + 1], p[4 * u + 2], p[4 * u + 3]);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_remote(dsmem_addr(smem_u32(&mi->vp_full[half]), 0));

    if (!last) {
      it.next(a, mi);
    } else {
      const int v = it.v;
      const int row0 = (CHUNK ? 0 : it.rt * kPairRows) + static_cast<int>(rank) * kCtaRows;
      const int span = it.v * a.row_tiles + it.rt;
      QueryRows unit{0, 0};
      if constexpr (CHUNK) unit = query_rows(a, it.v, it.rt);
      const bool ends = it.tile + 1 == it.nt;
      const bool whole = seg_first_tile == 0 && ends;
      const int slot = pair * 2 + (seg == 0 ? 0 : 1);
      it.next(a, mi);
      ++seg;
      // the whole row's sum, then O out of TMEM: final, or a partial
      mi->xch[part][r] = l;
      named_sync(bar_id, kSoftWarps * 16);
      const float lt = (mi->xch[0][r] + mi->xch[1][r]) + (mi->xch[2][r] + mi->xch[3][r]);
      named_sync(bar_id, kSoftWarps * 16);
      ok = wait_or_abort(&mi->pv_done, g & 1, mi, a.status) && ok;
      tc_fence_after();
      const bool mine = row0 + r < (CHUNK ? unit.rows : a.entry_rows);
      const size_t orow =
          (CHUNK ? unit.first : static_cast<size_t>(v) * a.entry_rows) + row0 + r;
      const float inv = !whole ? 1.0f : (lt > 0.0f || lt != lt ? 1.0f / lt : 0.0f);
      const int prow = static_cast<int>(rank) * kCtaRows + r;
      // column 64 q + 8 c + e holds dim 256 half + 32 c + 8 q + e: a thread
      // takes four c, so it has 32 neighbouring dims at a time
      const uint32_t tq = tmem + lanes + kColO + sub * 32;
      const int d0 = half * 256 + sub * 128;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        if (CHUNK && whole && a.wide_out) {
          // Two lanes write 64 bytes of one's row, then of the other's, 32 each, so that a
          // store meets 16 lines: with 64 bytes a lane, 32 lines a store, a segment took
          // 0.6 us more, in stores of 16 bytes 0.75 more still.
          const bool odd = lane & 1;
          uint32_t keep[8], give[8];   // this lane's half of its own 64 bytes, and the other
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float o[16];
            tmem_ld8x2(tq + 8 * c + 128 * h, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t w = bf16x2_bits(o[2 * e] * inv, o[2 * e + 1] * inv);
              if (h == 0) keep[e] = give[e] = w;
              else if (odd) keep[e] = w;
              else give[e] = w;
            }
          }
          float to_even[8], to_odd[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, give[e], 1);
            to_even[e] = __uint_as_float(odd ? got : keep[e]);
            to_odd[e] = __uint_as_float(odd ? keep[e] : got);
          }
          uint16_t* at = a.out + (orow - odd) * kLatent + d0 + 32 * c + 16 * odd;
          const int first = row0 + r - odd;
          if (first < unit.rows) st_global_32(reinterpret_cast<float*>(at), to_even);
          if (first + 1 < unit.rows) st_global_32(reinterpret_cast<float*>(at + kLatent), to_odd);
          continue;
        }
        float o[32];
        tmem_ld8x4(tq + 8 * c, o);
        if (!mine) {
          continue;
        } else if (whole) {
          uint16_t* dst = a.out + orow * kLatent + d0 + 32 * c;
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= inv;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            reinterpret_cast<uint4*>(dst)[x] = pack8_bf16(o + 8 * x);
        } else {
          float* dst = a.part_o + static_cast<size_t>(slot) * kPairRows * kLatent +
                       ((d0 + 32 * c) / 8 * kPairRows + prow) * 8;
#pragma unroll
          for (int x = 0; x < 4; ++x) st_global_32(dst + x * kPairRows * 8, o + 8 * x);
        }
      }
      if (part == 0) {
        if (whole) {
          if (mine && a.lse)
            a.lse[orow] = row_lse(m, c2, lt);
        } else {
          if (mine) a.part_ml[static_cast<size_t>(slot) * kPairRows + prow] = make_float4(m, lt, c2, 0.0f);
        }
      }
      if (tid == 0 && rank == 0) {
        if (CHUNK) {
          if (!ends) a.rec[pair].w = slot;   // of the pair's last partial
        } else {
          if (seg_first_tile == 0) a.span[span].x = slot;
          if (ends) a.span[span].y = pair;
        }
      }
      tc_fence_before();
    }
  }
  // the last arrival on this CTA's q_free, which nothing else waits for
  wait_or_abort(&mi->q_free, (seg - 1) & 1, mi, a.status);
}

template <bool CHUNK>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMlaThreads, 1)
    cache_mla_kernel(const MlaArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc* mi = reinterpret_cast<Misc*>(smem + kOffMisc);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (tid == 0) {
    mbar_init(smem_u32(&mi->q_ready), 2 * kWidenWarps);
    mbar_init(smem_u32(&mi->q_here[0]), kWidenWarps);
    mbar_init(smem_u32(&mi->q_here[1]), kWidenWarps);
    mbar_init(smem_u32(&mi->q_free), 1);
    // those of the even CTA count both CTAs' warps
    for (int h = 0; h < 2; ++h) {
      mbar_init(smem_u32(&mi->k_full[h]), 2 * kWidenWarps);
      mbar_init(smem_u32(&mi->vp_full[h]), 2 * kWidenWarps + kSoftWarps);
    }
    mbar_init(smem_u32(&mi->qk_half), 1);
    mbar_init(smem_u32(&mi->pv_half), 1);
    mbar_init(smem_u32(&mi->qk_done[0]), 1);
    mbar_init(smem_u32(&mi->qk_done[1]), 1);
    mbar_init(smem_u32(&mi->pv_done), 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_u32(&mi->row_full[i]), 1);
      mbar_init(smem_u32(&mi->row_free[i]), kWidenWarps + kSoftWarps);
    }
    mi->abort = 0;
    fence_mbar_init();
  }
  // a role that gives up a wait goes on with what it finds: always rows that exist
  if (tid < kRing * kMt) mi->row[tid / kMt][tid % kMt] = 0;
  if (tid < kRing) mi->seg[tid] = make_int2(-1, 0);
  if (warp == kMmaWarp) {
    tmem_alloc_pair(smem_u32(&mi->tmem), 512);
    tmem_relinquish_pair();
  }
  __syncwarp();
  cluster_arrive();   // the peer may arrive on this CTA's barriers once it has waited
  pdl_wait_previous();
  // This pair's share.  A segment (one entry and row tile) costs its tiles and
  // kSegmentCost more (its queries, its output), so positions are dealt in which
  // each segment has that many in front of its tiles: a scan of the entries'
  // tiles and segments, a run of neighbouring entries per thread.  With few
  // tiles those positions are left out, as a pair with none but them would lie
  // between two that share a request.  (Few entries are scanned by every warp,
  // without the block: 0.3 us of a small call.)
  constexpr int kShift = CHUNK ? kChunkSegShift : kSegShift;
  // Chunks scan units, whose requests are found among the requests' first units, kept
  // where the operands will be.
  int* unit0 = reinterpret_cast<int*>(smem);
  const int entries = CHUNK ? chunk_units(a, unit0, reinterpret_cast<int*>(mi->xch), &mi->fell) : a.entries;
  const int per = (entries + kMlaThreads - 1) / kMlaThreads;
  const bool few = !CHUNK && entries <= 32;   // then each warp scans them
  const int v0 = min(entries, few ? lane : tid * per), v1 = min(entries, v0 + per);
  long long mine = 0;
  int nt0 = 0;
  UnitWalk walk0;   // at unit v0
  if (CHUNK) {
    walk0.start(a, unit0, v0, v0 < v1);
    UnitWalk w = walk0;
    for (int v = v0; v < v1; ++v, w.next(a)) mine += w.tiles(a) + (1LL << kShift);
  } else {
    for (int v = v0; v < v1; ++v) {
      const int nt = (entry_len(a, v) + kMt - 1) / kMt;
      if (v == v0) nt0 = nt;
      if (nt > 0) mine += (static_cast<long long>(nt) + (1LL << kShift)) * a.row_tiles;
    }
  }
  long long before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  long long* scan = reinterpret_cast<long long*>(mi->xch);   // free until the roles start
  long long total = __shfl_sync(0xffffffffu, before, 31);
  before -= mine;
  if (!few) {
    if (lane == 31) scan[warp] = total;
    __syncthreads();
    long long sums = lane < kMlaThreads / 32 ? scan[lane] : 0;   // of the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, sums, o);
      if (lane >= o) sums += x;
    }
    total = __shfl_sync(0xffffffffu, sums, 31);
    before += warp > 0 ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0;
  }
  constexpr long long kTileMask = (1LL << kShift) - 1;
  const long long tiles = total & kTileMask;
  constexpr int kCost = CHUNK ? kChunkSegmentCost : kSegmentCost;
  const int cost = tiles >= static_cast<long long>(kCost + 1) * pairs ? kCost : 0;
  const long long tiles_before = before & kTileMask;
  const long long pos0 = tiles_before + cost * (before >> kShift);
  const long long pos1 = pos0 + (mine & kTileMask) + cost * (mine >> kShift);
  const long long all = tiles + cost * (total >> kShift);
  // the first all % busy pairs take one position more
  const int busy = tiles < pairs ? max(static_cast<int>(tiles), 1) : pairs;
  const long long share = all < 0x7fffffffLL
                              ? static_cast<unsigned>(all) / static_cast<unsigned>(busy)
                              : all / busy;
  const int extra = static_cast<int>(all - share * busy);
  const bool deals = !few || warp == 0;
#pragma unroll 1
  for (int end = 0; deals && end < 2; ++end) {
    const long long at = share * (pair + end) + min(pair + end, extra);
    if (at == all && tid == 0) mi->end_tile = tiles;   // of the last pair (and idle ones)
    if (at < pos0 || at >= pos1) continue;
    long long off = at - pos0, t = tiles_before;
    if (CHUNK) {
      UnitWalk w = walk0;
      int nt = w.tiles(a);
      for (; off >= nt + cost; w.next(a), nt = w.tiles(a)) {
        off -= nt + cost;
        t += nt;
      }
      const int tile = max(static_cast<int>(off) - cost, 0);
      if (end) {
        mi->end_tile = t + tile;
      } else {
        mi->start_v = w.b;
        mi->start_rt = w.u;
        mi->start_tile = tile;
        mi->first_tile = t + tile;
      }
      continue;
    }
    int v = v0, nt, rt = 0;
    for (;; ++v) {
      nt = v == v0 ? nt0 : (entry_len(a, v) + kMt - 1) / kMt;
      const long long w = nt > 0 ? static_cast<long long>(nt + cost) * a.row_tiles : 0;
      if (off < w) break;
      off -= w;
      t += static_cast<long long>(nt) * a.row_tiles;
    }
    for (; off >= nt + cost; off -= nt + cost) ++rt;   // at most kMaxCacheWays row tiles
    const int tile = max(static_cast<int>(off) - cost, 0);
    t += static_cast<long long>(rt) * nt + tile;
    if (end) {
      mi->end_tile = t;
    } else {
      mi->start_v = v;
      mi->start_rt = rt;
      mi->start_tile = tile;
      mi->first_tile = t;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = mi->tmem;

  if (CHUNK && rank == 0 && tid == kMmaWarp * 32) {   // see the join
    const bool inside = pair < tiles && mi->start_tile > 0;
    QueryRows q{0, 0};
    if (inside) q = query_rows(a, mi->start_v, mi->start_rt);
    a.rec[pair].x = inside ? static_cast<int>(q.first) : -1;
    a.rec[pair].y = q.rows;
  }
  __syncwarp();
  if (pair >= tiles) {
    // nothing to do: both CTAs of the pair
  } else if (warp < kSoftWarps) {
    softmax_role<CHUNK>(a, smem, mi, rank, tmem, pair);
  } else if (warp == kMmaWarp) {
    if (rank == 0) mma_role<CHUNK>(a, smem, mi, tmem);
  } else if (warp == kRowWarp) {
    row_role<CHUNK>(a, mi);
  } else {
    widen_role<CHUNK>(a, smem, mi, rank);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // no barrier of the peer is arrived on after this
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc_pair(tmem, 512);
}

// Joins the partials of a query row that several pairs share, and writes the
// rows of requests without a token.  A CTA takes SLICE of the 64 parts (8 dims) of
// ROWS neighbouring rows, one thread a part, in GROUPS groups; a group takes
// every GROUPS-th partial of its rows, FLY of them in flight.  Partials lie with
// 8 dims of all 128 rows side by side, so that a warp of the attention, a row a
// lane, writes 1 KB at a time (with rows of 2 KB its stores met 32 lines each
// and O took 4.0 us to leave a CTA; 2.2 now), and four rows here fill a line.
constexpr int kJoinThreads = 64;

// CHUNK: of the rows of the units that pairs cut, 128 a unit.
template <bool CHUNK, int ROWS, int SLICE, int GROUPS, int FLY>
__global__ void __launch_bounds__(SLICE* ROWS* GROUPS) cache_mla_join_kernel(
    const MlaArgs a, int all_rows) {
  constexpr int kSlices = kJoinThreads / SLICE;
  constexpr int kSpan = SLICE * ROWS;   // threads of one group
  __shared__ float shared[GROUPS > 1 ? (GROUPS - 1) * kSpan * 10 : 1];
  pdl_wait_previous();
  // neighbouring threads: the halves of 32 bytes of one row, then the next row
  const int at = threadIdx.x % kSpan, g = threadIdx.x / kSpan;
  const int t = static_cast<int>(blockIdx.x % kSlices) * SLICE + 2 * (at / (2 * ROWS)) +
                (at & 1);                               // dims 4t .. and 256 + 4t ..
  const int x = static_cast<int>(blockIdx.x / kSlices) * ROWS + (at >> 1) % ROWS;   // (b, m, h)
  const bool real = x < all_rows;
  bool join;                 // else one pair wrote the row
  int p0 = 0, first = 0, last = -1, pr;   // its first pair, that one's slot, its last pair
  size_t orow = x;
  if (CHUNK) {
    // The x / 128th unit that is cut: the pair that is the first to start inside of it,
    // found by one warp from all records at once (one after another takes a latency each).
    __shared__ int4 cut_unit;   // first pair, its slot, last pair, first row; and the rows
    __shared__ int cut_rows;
    if (threadIdx.x < 32) {
      constexpr int kPer = (kMaxPairs + 31) / 32;
      const int lane = threadIdx.x;
      int4 rec[kPer];
      int before[kPer];
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const int i = 32 * c + lane;
        rec[c] = i < a.pairs ? a.rec[i] : make_int4(-1, 0, 0, 0);
        before[c] = i > 0 && i < a.pairs ? a.rec[i - 1].x : -1;
      }
      int left = x / kPairRows, p = 0, unit = -1, rows = 0, inside = 0, slot = 0;
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const uint32_t cut = __ballot_sync(0xffffffffu, rec[c].x >= 0 && rec[c].x != before[c] &&
                                                            32 * c + lane > 0);
        int here = -1;
        if (left < __popc(cut) && p == 0) {
          uint32_t bits = cut;
          for (int i = 0; i < left; ++i) bits &= bits - 1;
          here = __ffs(bits) - 1;
        }
        left -= __popc(cut);
        const int u = __shfl_sync(0xffffffffu, rec[c].x, max(here, 0));
        const int n = __shfl_sync(0xffffffffu, rec[c].y, max(here, 0));
        if (here >= 0) {
          p = 32 * c + here;
          unit = u;
          rows = n;
        }
      }
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        // pairs that start inside of it, side by side, behind the one that begins it
        inside += __popc(__ballot_sync(0xffffffffu, rec[c].x >= 0 && rec[c].x == unit));
        const int w = __shfl_sync(0xffffffffu, rec[c].w, (p - 1) & 31);
        if ((p - 1) >> 5 == c) slot = w;
      }
      if (lane == 0) {
        cut_unit = make_int4(p - 1, slot, p - 1 + inside, unit);
        cut_rows = p > 0 ? rows : 0;
      }
    }
    __syncthreads();
    pr = x % kPairRows;
    join = real && pr < cut_rows;
    if (join) {
      p0 = cut_unit.x;
      first = cut_unit.y;
      last = cut_unit.z;
      orow = static_cast<size_t>(cut_unit.w) + pr;
    }
  } else {
    const int xr = real ? x : 0;
    const int h = xr % a.heads, bm = xr / a.heads, b = bm / a.ways, m = bm % a.ways;
    const int v = a.tokens ? bm : b;
    const int row = a.tokens ? h : m * a.heads + h;
    const int T = a.T[b];
    const int2 sp = a.span[static_cast<size_t>(v) * a.row_tiles + row / kPairRows];
    if (real && h == 0 && m == 0 && t == 0 &&
        (T < 0 || T > static_cast<long long>(a.max_pages) * a.page))
      set_status(a.status, ESS_ERR_DEVICE_CHECK);
    const bool empty = entry_len(a, v) == 0;   // then nothing wrote its span
    join = real && !empty && sp.x >> 1 != sp.y;
    p0 = join ? sp.x >> 1 : 0;
    first = sp.x;
    last = join ? sp.y : -1;
    pr = row % kPairRows;
    if (real && empty && g == 0) {
      uint2* out = reinterpret_cast<uint2*>(a.out + static_cast<size_t>(x) * kLatent) + t;
      out[0] = out[kJoinThreads] = make_uint2(0u, 0u);
      if (t == 0 && a.lse) a.lse[x] = -INFINITY;
    }
  }
  uint2* out = reinterpret_cast<uint2*>(a.out + orow * kLatent) + t;
  if (GROUPS == 1 && !join) return;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  // of every part
  const float c2 = join ? a.part_ml[static_cast<size_t>(first) * kPairRows + pr].z : 0.0f;
  float mx = -INFINITY, l = 0.0f;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int pb = p0 + g; pb <= last; pb += FLY * GROUPS) {
    float2 ml[FLY];
    float4 o[FLY][2];
#pragma unroll
    for (int q = 0; q < FLY; ++q) {
      const int p = pb + q * GROUPS;
      const size_t i = p == p0 ? first : 2 * p;
      const float4* po = reinterpret_cast<const float4*>(a.part_o + i * kPairRows * kLatent) +
                         ((t >> 1) * kPairRows + pr) * 2 + (t & 1);
      const bool in = p <= last;
      ml[q] = in ? *reinterpret_cast<const float2*>(a.part_ml + i * kPairRows + pr)
                 : make_float2(-INFINITY, 0.0f);
      o[q][0] = in ? po[0] : zero;
      o[q][1] = in ? po[256 / 8 * kPairRows * 2] : zero;
    }
    float m2 = mx;
#pragma unroll
    for (int q = 0; q < FLY; ++q) m2 = fmaxf(m2, ml[q].x);
    const float base = m2 == -INFINITY ? 0.0f : m2;
    const float f = exp2f((mx - base) * c2);
    l *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= f;
#pragma unroll
    for (int q = 0; q < FLY; ++q) {
      // a part without a token has l = 0 and O = 0; its weight is 0 beside others
      const float w = exp2f((ml[q].x - base) * c2);
      l = fmaf(w, ml[q].y, l);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        acc[4 * e] = fmaf(w, o[q][e].x, acc[4 * e]);
        acc[4 * e + 1] = fmaf(w, o[q][e].y, acc[4 * e + 1]);
        acc[4 * e + 2] = fmaf(w, o[q][e].z, acc[4 * e + 2]);
        acc[4 * e + 3] = fmaf(w, o[q][e].w, acc[4 * e + 3]);
      }
    }
    mx = m2;
  }
  if (GROUPS > 1) {   // the groups' sums to the first one
    if (g > 0) {
      float* to = shared + (g - 1) * kSpan * 10 + at;
      to[0] = mx;
      to[kSpan] = l;
#pragma unroll
      for (int e = 0; e < 8; ++e) to[(2 + e) * kSpan] = acc[e];
    }
    __syncthreads();
    if (g > 0 || !join) return;
    float m2 = mx;
#pragma unroll
    for (int q = 0; q < GROUPS - 1; ++q) m2 = fmaxf(m2, shared[q * kSpan * 10 + at]);
    const float base = m2 == -INFINITY ? 0.0f : m2;
    const float f = exp2f((mx - base) * c2);
    l *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= f;
#pragma unroll
    for (int q = 0; q < GROUPS - 1; ++q) {
      const float* from = shared + q * kSpan * 10 + at;
      const float w = exp2f((from[0] - base) * c2);
      l = fmaf(w, from[kSpan], l);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, from[(2 + e) * kSpan], acc[e]);
    }
    mx = m2;
  }
  const bool some = l > 0.0f || l != l;
  const float inv = some ? 1.0f / l : 0.0f;
#pragma unroll
  for (int e = 0; e < 2; ++e)
    out[e * kJoinThreads] =
        make_uint2(bf16x2_bits(acc[4 * e] * inv, acc[4 * e + 1] * inv),
                   bf16x2_bits(acc[4 * e + 2] * inv, acc[4 * e + 3] * inv));
  if (t == 0 && a.lse)
    a.lse[orow] = row_lse(mx, c2, l);
}

template <bool CHUNK, int ROWS, int SLICE, int GROUPS, int FLY>
cudaError_t launch_join(const MlaArgs& a, long long all_rows, cudaStream_t st) {
  const long long ctas = (all_rows + ROWS - 1) / ROWS * (kJoinThreads / SLICE);
  return launch_pdl_once(cache_mla_join_kernel<CHUNK, ROWS, SLICE, GROUPS, FLY>,
                         dim3(static_cast<unsigned>(ctas)), dim3(SLICE * ROWS * GROUPS), 0, st, a,
                         static_cast<int>(all_rows));
}

ess_status check_shape(int batch, int ways, int heads) {
  if (batch < 1 || ways < 1 || heads < 1) return ESS_ERR_INVALID_ARG;
  if (ways > kMaxCacheWays || heads > kMaxCacheHeads || batch > 65535) return ESS_ERR_UNSUPPORTED;
  return ESS_OK;
}

struct MlaLayout {
  size_t span, part_o, part_ml, total;
};
MlaLayout mla_layout(int batch, int ways) {
  MlaLayout L;
  size_t o = 0;
  // at most one row tile per (request, way), listed or not
  L.span = o;
  o += (static_cast<size_t>(batch) * ways * sizeof(int2) + 255) & ~static_cast<size_t>(255);
  L.part_ml = o;
  o += static_cast<size_t>(kMaxPairs) * 2 * kPairRows * sizeof(float4);
  L.part_o = o;
  o += static_cast<size_t>(kMaxPairs) * 2 * kPairRows * kLatent * sizeof(float);
  L.total = o;
  return L;
}

struct ChunkLayout {
  size_t rec, unit0, part_o, part_ml, total;
};
ChunkLayout chunk_layout() {
  ChunkLayout L;
  L.rec = 0;
  L.unit0 = (kMaxPairs * sizeof(int4) + 255) & ~static_cast<size_t>(255);
  L.part_ml = L.unit0 + (((kMaxChunkBatch + 1) * sizeof(int) + 255) & ~static_cast<size_t>(255));
  L.part_o = L.part_ml + static_cast<size_t>(kMaxPairs) * 2 * kPairRows * sizeof(float4);
  L.total = L.part_o + static_cast<size_t>(kMaxPairs) * 2 * kPairRows * kLatent * sizeof(float);
  return L;
}

int page_shift(int page) {   // log2, or -1
  for (int i = 0; i < 31; ++i)
    if (page == 1 << i) return i;
  return -1;
}

}  // namespace
}  // namespace ess

using namespace ess;

extern "C" {

ess_status ess_cache_mla_bytes(int32_t batch, int32_t ways, int32_t heads, size_t* bytes) {
  if (!bytes) return ESS_ERR_INVALID_ARG;
  const ess_status s = check_shape(batch, ways, heads);
  if (s != ESS_OK) return s;
  *bytes = mla_layout(batch, ways).total;
  return ESS_OK;
}

ess_status ess_cache_mla(const void* q, const void* rows, int64_t n_rows, int32_t format,
                         const int32_t* page_table, int32_t max_pages, int32_t page,
                         const int32_t* T, int32_t batch, int32_t ways, int32_t heads,
                         const int32_t* tokens, int32_t k, float sm_scale, void* out, float* lse,
                         void* workspace, size_t ws_bytes, int32_t* status, ess_stream_t stream) {
  const ess_status s = check_shape(batch, ways, heads);
  if (s != ESS_OK) return s;
  if (format < ESS_ROW_BF16 || format > ESS_ROW_Q4 || n_rows < 1 || max_pages < 1 || page < 1 ||
      (tokens && k < 1) || !(sm_scale > 0.0f) || !std::isfinite(sm_scale))
    return ESS_ERR_INVALID_ARG;
  if (format != ESS_ROW_Q4 || n_rows > 0x7fffffffLL ||
      static_cast<long long>(max_pages) * page > 0x7fffff00LL || k > 0x7fffff00)
    return ESS_ERR_UNSUPPORTED;
  if (!q || !rows || !page_table || !T || !out || !workspace || !aligned16(q) ||
      !aligned16(rows) || !aligned16(out) || !aligned_to(workspace, 256) ||
      !aligned_to(page_table, 4) || !aligned_to(T, 4) || !aligned_to(tokens, 4) ||
      !aligned_to(lse, 4) || !aligned_to(status, 4))
    return ESS_ERR_INVALID_ARG;
  const MlaLayout L = mla_layout(batch, ways);
  if (ws_bytes < L.total) return ESS_ERR_OOM;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ESS_ERR_CUDA;
  const long long all_rows = static_cast<long long>(batch) * ways * heads;
  MlaArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.rows = static_cast<const uint8_t*>(rows);
  a.n_rows = static_cast<int>(n_rows);
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.page = page;
  a.page_shift = page_shift(page);
  a.T = T;
  a.batch = batch;
  a.ways = ways;
  a.heads = heads;
  a.tokens = tokens;
  a.k = k;
  a.entries = tokens ? batch * ways : batch;
  a.entry_rows = tokens ? heads : ways * heads;
  a.row_tiles = (a.entry_rows + kPairRows - 1) / kPairRows;
  a.c2 = std::min(sm_scale * 1.4426950408889634f, FLT_MAX);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  char* ws = static_cast<char*>(workspace);
  a.span = reinterpret_cast<int2*>(ws + L.span);
  a.part_o = reinterpret_cast<float*>(ws + L.part_o);
  a.part_ml = reinterpret_cast<float4*>(ws + L.part_ml);
  a.status = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // no more pairs than tiles there can be
  const long long most = static_cast<long long>(a.entries) * a.row_tiles *
                         (((tokens ? std::min<long long>(k, static_cast<long long>(max_pages) * page)
                                   : static_cast<long long>(max_pages) * page) +
                           kMt - 1) /
                          kMt);
  const int pairs = static_cast<int>(std::min<long long>(most, kMaxPairs));
  cudaError_t e = allow_smem<cache_mla_kernel<false>>(dev, kMlaSmem);
  if (e != cudaSuccess) return ESS_ERR_CUDA;
  e = launch_pdl_once(cache_mla_kernel<false>, dim3(2 * pairs), dim3(kMlaThreads), kMlaSmem, st, a);
  if (e != cudaSuccess) return ESS_ERR_CUDA;
  // Few rows with many parts (a 4096-token request: 32) are cut into many small
  // slices: 12.1 us a call, where whole rows took 14.4.  Many rows (2048 and more
  // fill the GPU) have two or three parts each where requests are alike: one group is
  // enough, and four parts in flight cost 1.5 us of 97 more than two.  Between, two
  // groups: 2048 listed tokens of eight requests 19.3 us, four groups 21.7, slices of 16
  // 19.7.  Only rows are counted, as the parts of a row are known on the device: one
  // 128K request among 31 of 512 tokens, with some 70 parts a row in one group, takes
  // 69 us where it takes 42 alone.
  if (all_rows <= 608) e = launch_join<false, 4, 8, 16, 2>(a, all_rows, st);
  else if (all_rows < 2048) e = launch_join<false, 4, 64, 2, 4>(a, all_rows, st);
  else e = launch_join<false, 4, 64, 1, 2>(a, all_rows, st);
  return e == cudaSuccess ? ESS_OK : ESS_ERR_CUDA;
}

ess_status ess_cache_chunk_bytes(size_t* bytes) {
  if (!bytes) return ESS_ERR_INVALID_ARG;
  *bytes = chunk_layout().total;
  return ESS_OK;
}

ess_status ess_cache_chunk(const void* q, int64_t total, const int32_t* cu, const void* rows,
                           int64_t n_rows, int32_t format, const int32_t* page_table,
                           int32_t max_pages, int32_t page, const int32_t* T, int32_t batch,
                           int32_t heads, const int32_t* tokens, int32_t k, float sm_scale,
                           void* out, float* lse, void* workspace, size_t ws_bytes,
                           int32_t* status, ess_stream_t stream) {
  if (batch < 1 || heads < 1 || total < 0) return ESS_ERR_INVALID_ARG;
  if (heads > kMaxCacheHeads || batch > kMaxChunkBatch || total > (0x7fffff00LL - 128) / heads)
    return ESS_ERR_UNSUPPORTED;
  if (format < ESS_ROW_BF16 || format > ESS_ROW_Q4 || n_rows < 1 || max_pages < 1 || page < 1 ||
      (tokens && k < 1) || !(sm_scale > 0.0f) || !std::isfinite(sm_scale))
    return ESS_ERR_INVALID_ARG;
  if (format != ESS_ROW_Q4 || n_rows > 0x7fffffffLL ||
      static_cast<long long>(max_pages) * page > 0x7fffff00LL || k > 0x7fffff00)
    return ESS_ERR_UNSUPPORTED;
  if (total == 0) return ESS_OK;
  if (!q || !cu || !rows || !page_table || !T || !out || !workspace || !aligned16(q) ||
      !aligned16(rows) || !aligned16(out) || !aligned_to(workspace, 256) || !aligned_to(cu, 4) ||
      !aligned_to(page_table, 4) || !aligned_to(T, 4) || !aligned_to(tokens, 4) ||
      !aligned_to(lse, 4) || !aligned_to(status, 4))
    return ESS_ERR_INVALID_ARG;
  // units and tiles there can be
  const long long context = static_cast<long long>(max_pages) * page;
  const long long units = tokens ? total : total * heads / kPairRows + std::min<long long>(total, batch);
  const long long most = units * (((tokens ? std::min<long long>(k, context) : context) + kMt - 1) / kMt);
  if (units >= kMaxChunkUnits || most >= kMaxChunkTiles) return ESS_ERR_UNSUPPORTED;
  const ChunkLayout L = chunk_layout();
  if (ws_bytes < L.total) return ESS_ERR_OOM;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ESS_ERR_CUDA;
  MlaArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.rows = static_cast<const uint8_t*>(rows);
  a.n_rows = static_cast<int>(n_rows);
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.page = page;
  a.page_shift = page_shift(page);
  a.T = T;
  a.batch = batch;
  a.heads = heads;
  a.tokens = tokens;
  a.k = k;
  a.cu = cu;
  a.total = static_cast<int>(total);
  a.wide_out = aligned_to(out, 32);
  a.unit_rows = tokens ? heads : kPairRows;
  a.c2 = std::min(sm_scale * 1.4426950408889634f, FLT_MAX);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  char* ws = static_cast<char*>(workspace);
  a.rec = reinterpret_cast<int4*>(ws + L.rec);
  a.unit0 = reinterpret_cast<int*>(ws + L.unit0);
  a.part_o = reinterpret_cast<float*>(ws + L.part_o);
  a.part_ml = reinterpret_cast<float4*>(ws + L.part_ml);
  a.status = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // no more pairs than tiles there can be
  a.pairs = static_cast<int>(std::max(1LL, std::min<long long>(most, kMaxPairs)));
  cudaError_t e = allow_smem<cache_mla_kernel<true>>(dev, kMlaSmem);
  if (e != cudaSuccess) return ESS_ERR_CUDA;
  e = launch_pdl_once(cache_mla_kernel<true>, dim3(2 * a.pairs), dim3(kMlaThreads), kMlaSmem, st, a);
  if (e == cudaSuccess && a.pairs > 1) {
    const long long cut = std::min<long long>(units, a.pairs - 1) * kPairRows;
    // Few units have many parts each; with more units than pairs a cut one has two or
    // three: one group a row, two parts in flight (two chunks of 160 tokens with lists of
    // 2048, 75 cut units: 189.8 us, with two groups and every warp reading the records 198.6).
    if (units > a.pairs) e = launch_join<true, 4, 64, 1, 2>(a, cut, st);
    else if (units <= 8) e = launch_join<true, 4, 8, 16, 2>(a, cut, st);
    else e = launch_join<true, 4, 64, 2, 4>(a, cut, st);
  }
  return e == cudaSuccess ? ESS_OK : ESS_ERR_CUDA;
}

}  // extern "C"
