// Attention of ragged chunks of new tokens over a paged latent cache: q of 576
// dims for every token and head, one latent key row of 576 for all heads, its
// first 512 dims the value; request b's queries see its keys up to their own
// position (causal, aligned at the end) or all of them.
//
//   s_ij = scale q_i . k_j,  out_i = sum_j e^(s_ij - r_i) k_j[:512] / l_i,
//   l_i = sum_j e^(s_ij - r_i),  lse_i = r_i + ln l_i
//
// Units.  A request's queries are rows, token-major; 128 rows and the keys that
// the last of them sees are a unit.  The plan cuts the units' 128-key tiles into
// one run for each pair of CTAs, all of the same cost; a unit that a cut divides
// leaves partial sums, which the combine merges, every other one its output.
//
// The pair splits the rows, not the values: CTA c has rows 64 c .. 64 c + 63, and
// every product is a cta_group::2 MMA of M = 128, whose accumulator holds a CTA's
// 64 rows in 128 lanes: columns [0, N/2) in lanes 0 .. 63, [N/2, N) in lanes 64
// .. 127 (and which runs at the full rate, 4090 multiply-adds a cycle and SM, at
// N = 128 and 256).  A row's scores, weights and output never leave its CTA, so
// nothing is exchanged between the two but barrier arrivals:
//   * Q K^T: N = 128 keys, two pages; CTA c loads page 2 j + c, all 576 dims.
//   * P V: N = 256 dims, twice; CTA c loads dims 256 c .. 256 c + 255 of both
//     pages.  (The half of them that are in its key page too cannot serve: an MMA
//     reads both CTAs' operands at one offset, and they lie at different ones.)
//   * TMEM: O 64 x 512 as 256 columns, two score buffers of 64.
//   * Shared memory: Q 72 KB, K in three stages of three 64-dim slices, V in two
//     stages of a page, P 16 KB.
//   * One warp issues  Q K^T (t+1)  P V (t):  the softmax of tile t+1 runs under
//     P V (t) and Q K^T (t+2), that of t under Q K^T (t+1).
//   * Four threads hold a row's 128 scores, 32 each, and share their maxima in
//     shared memory.  The reference r (2^7 below the maximum where weights are
//     fp16) is raised only when the maximum grows by more than 2^8 (then O is
//     rescaled, rarely).  Weights are rounded to the cache's type for P V and divided
//     by the sum of the unrounded ones.
//   * Rows of a page behind the unit's last key may hold anything: their scores
//     are masked, and their values zeroed in shared memory (0 x NaN is not 0).
//
// Bound by the tensor pipe over 16-bit caches: busy 92% of the cycles of 3 chunks of
// up to 300 tokens x 128 heads over 8000 keys (580 us, 1930 TFLOP/s), 80% of 64
// requests' up to 6 drafts over up to 4096 keys (148 us; a unit's output, 2 us, and
// the first scores, 6 us, are not under anything).  Both products feed it from shared
// memory, whose 128 bytes a cycle Q K^T takes to the full (4 KB an MMA of 32 cycles),
// so that loads and weights stored at the same time cost it cycles: 1.35 us a tile
// where the MMAs alone are 1.15.
//
// FP8 records: below.  1.8 us a tile, bound by the softmax threads' chain (five sums
// of a score from TMEM and their scales from shared memory, 0.2 us each); tiles whose
// values no other unit shares, 2.4 us among others and 2.8 where all are such, by
// their conversion.  43 requests, 3 chunks of up to 400 tokens among single ones, 16
// heads over up to 3400 keys: 112 us, of which the slowest pair has 100 (first scores
// 5, 41 tiles a pair 74, changes of units 9, the last output 4, pairs that end 7
// apart) and the kernels before and behind it the rest.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>

#include "mla_serving.h"
#include "common.cuh"
#include "ptx.cuh"
#include "serving.cuh"

// Timeline hooks: empty in the library; an instrumented build defines
// MLA_TRACE(event, index) to record timestamps.
#ifndef MLA_TRACE
#define MLA_TRACE(ev, i) \
  do {                   \
  } while (0)
#endif

namespace mla {
namespace ck {

constexpr int kCtaRows = 64;               // query rows of one CTA
constexpr int kBN = 128;                   // keys of a tile: two pages
constexpr int kSlices = kDqk / 64;
constexpr int kSliceBytes = 64 * 128;      // 64 rows or keys x 64 dims
constexpr int kKSlices = 3;                // slices of a K stage
// FP8 records.  Keys are multiplied as the codes they are: a bf16 query has eight
// significant bits, which two E4M3 numbers hold (four bits, and the remainder's
// four), so that Q K^T is two kind::f8f6f4 MMAs a group, at twice the rate, and K
// needs no conversion.  Each 128-dim group has a sum of its own, which the softmax
// threads multiply by the key's scale in fp32; the RoPE part (bf16) has the fifth.
// A query is scaled by a power of two that brings its largest element to 128 .. 256:
// elements down to 2^-9 of that one are exact, smaller ones are off by 2^-17 of it.
// Values are code x (scale / 2^E) in fp16, E a key's own multiple of 8 that leaves its
// largest scale at 1/2 .. 128, and weights are those of the products times 2^E, fp16
// too: with values and weights in bf16 the output was off by half as much again as
// its own rounding.  A tile whose keys all have the same E, as a normalised cache's
// do, takes it as one term of the exponent.
constexpr int kParts = 5;                         // sums of a score: four groups, RoPE
constexpr int kQueryRow = MLA_CHUNK_QUERY_BYTES;  // 512 codes, the remainders', 2^f and 2^-f as fp32, 8 bytes of nothing
constexpr int kFp8Stages = 8;                     // of K: one 64-key x 128-byte part of a page each
constexpr int kOffScales = kSlices * kSliceBytes + kFp8Stages * kSliceBytes;  // [2][4 groups, E][128 keys]
static_assert(MLA_CHUNK_PAGE_BYTES == 2 * MLA_D_V * MLA_PAGE_SIZE && kQueryRow % 16 == 0 && kQueryRow >= 2 * MLA_D_V + 8,
              "a page's values and a query in the workspace");
constexpr int kKBytes = kKSlices * kSliceBytes;
constexpr int kKStages = 3;
constexpr int kVBytes = 4 * kSliceBytes;   // a page's 64 keys x this CTA's 256 dims
constexpr int kVStages = 2;
constexpr int kPBytes = 2 * kSliceBytes;   // 64 rows x 128 keys
constexpr int kOffK = kSlices * kSliceBytes;
constexpr int kOffV = kOffK + kKStages * kKBytes;
constexpr int kOffP = kOffV + kVStages * kVBytes;
constexpr int kOffBar = kOffP + kPBytes;
constexpr int kOffTileE = kOffScales + 2 * 5 * kBN * 4;  // [2]: E of a tile's keys, or kMixed; 2^-E
static_assert(kOffTileE + 16 <= kOffV, "the scales lie behind the K stages");
constexpr float kMixed = 1000.f;

enum : int {
  Q_FULL = 0,
  Q_EMPTY,                        // the unit's last Q K^T is done
  K_FULL,                         // +stage
  K_EMPTY = K_FULL + kFp8Stages,    // +stage
  V_FULL = K_EMPTY + kFp8Stages,    // +stage
  V_EMPTY = V_FULL + kVStages,    // +stage
  S_FULL = V_EMPTY + kVStages,    // +buffer
  // FP8 records: the tile's first sum, and all five, read by all softmax warps of both CTAs; then a tile's scales
  // written (+ tile & 1), and read by this CTA's softmax warps
  S_FIRST = S_FULL + 4,
  S_ALL,
  SCALE_FULL,
  SCALE_EMPTY = SCALE_FULL + 2,
  P_FULL = SCALE_EMPTY + 2,       // weights written, O rescaled (one arrival per softmax warp of both CTAs)
  PV_DONE,                        // one completion a tile: P may be overwritten, O rescaled or read
  TAIL,                           // a V page whose last rows are to be zeroed has landed
  DRAIN,
  kNumBars
};
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kOffRow = (kOffMisc + 16 + 15) / 16 * 16;  // [2][4 parts][64 rows]: maxima of a tile, or sums
constexpr int kSmemBytes = kOffRow + 2 * 4 * kCtaRows * 4;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kKSlices * 3 == kSlices, "three K stages a tile");

// Warps: 0 .. 7 softmax (with 16 and 16 keys a thread FP8 records took 5% longer),
// then one each for MMAs, Q (FP8 records: and scales) and K.  16-bit caches: one for
// V; FP8 records: kConverters convert it (eight of them instead of four leave the
// softmax threads 96 registers: 4% longer).
constexpr int kSoftmax = 8, kWarpMma = 8, kWarpQ = 9, kWarpK = 10, kWarpV = 11;
constexpr int kConverters = 4;
constexpr int kLaneKeys = 8 / kConverters;  // keys of a page that a converting lane has, 8 kConverters apart
constexpr int threads_of(bool fp8) { return 32 * (kWarpV + (fp8 ? kConverters : 1)); }
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 256;  // two buffers of 64 columns; four for the sums over FP8 records
constexpr float kTau = 8.0f;  // the reference is raised when the maximum is 2^kTau above the one it was last set by
// Weights in fp16 are held 2^7 as large, 2^15 at most: what lies 2^21 below a row's
// largest is still a normal number, and lost are those below 2^-32 of it.  (With the
// largest near 1 they were lost below 2^-25, while the sum l kept them: the output of
// 131072 keys that lie 2^25 below one of values near 0 was 0.  Raising the reference at
// 2^4 would leave room for 2^11: scores with a deviation of 4, 64 requests x 4 tokens x
// 128 heads, 155 us instead of 152, FP8 records 255 instead of 250.)
template <bool kF16>
constexpr float kLift = kF16 ? 7.0f : 0.0f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (kHalf) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// tcgen05.ld of 32 columns that also returns the maximum of this thread's 32 values.
__device__ __forceinline__ void tmem_ld32_max(uint32_t taddr, float* f, float& mx) {
  uint32_t(&r)[32] = *reinterpret_cast<uint32_t(*)[32]>(f);
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
        "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31]), "=f"(mx)
      : "r"(taddr));
}

// Arrive on a barrier of either CTA of the pair (address from mapa) after writes
// to this CTA's own shared memory that fence.proxy.async has handed to its async
// proxy, where an MMA issued by the other CTA reads them.
__device__ __forceinline__ void arrive_pair(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// ------------------------------------------------------------------ units

struct Unit {
  int row0;    // first query row in the packed q, of total_q * h_q
  int rows;    // at most 128
  int rel;     // row0's place among its request's rows
  int req;
  int len;     // keys that its last row sees
  int limit0;  // causal: keys that a row of the request's token 0 sees (may be below 1)
  int pages0;  // its request's first page among those converted once for all of its units, or -1
  // of one of the plan's two schedules (16-bit caches, FP8 records)
  int slot;    // first partial slot
  int parts;   // pieces it is cut into (1: none; 0: no keys)
  bool whole;  // one pair's as a whole (pair u % pairs); else in the list that is cut
};
constexpr int kPages0 = 6, kSchedule = 8, kWhole = 1 << 16;  // ints of a unit; a schedule's: slot, parts (+ kWhole)
static_assert(kSchedule + 4 == kChunkUnitInts && kMaxChunkParts < kWhole, "three int4");

__device__ __forceinline__ Unit load_unit(const ChunkParams& p, int u) {
  const int32_t* at = p.units + static_cast<long long>(u) * kChunkUnitInts;
  const int4 a = reinterpret_cast<const int4*>(at)[0], b = reinterpret_cast<const int4*>(at)[1];
  const int2 c = reinterpret_cast<const int2*>(at + kSchedule)[p.schedule];
  return Unit{a.x, a.y, a.z, a.w, b.x, b.y, b.z, c.x, c.y & (kWhole - 1), c.y >= kWhole};
}

__device__ __forceinline__ int pages_of(int len) { return (len + kTile - 1) / kTile; }
__device__ __forceinline__ int tiles_of(int len) { return (len + kBN - 1) / kBN; }

// A pair's work: the whole units among u = pair, pair + pairs, .. (in waves: the
// pairs are then at neighbouring units at a time, which are the same requests' and
// read the same keys), then its run of the units that are cut, from tile t0 of
// entry u0 of their list to tile t1 of entry u1 (not included).
struct Run {
  int u0, t0, u1, t1, piece;  // piece: of entry u0, among those it is cut into
  int pair, pairs, units;
};

__device__ __forceinline__ Run load_run(const ChunkParams& p) {
  const int pair = blockIdx.x >> 1;
  const int32_t* e = p.sched + pair * MLA_SCHED_INTS;
  return Run{e[0], e[1], e[2], e[3], e[4], pair, static_cast<int>(gridDim.x >> 1), p.head[kHeadWhole]};
}

// The units of a run one after another, and each one's tiles lo .. hi - 1.
struct Walk {
  Unit unit;
  int lo, hi;
  int u;         // next unit to look at, then
  int at;        // next entry of the list
  bool first;    // the unit is the run's first entry: its pieces are counted from `piece`
};

__device__ __forceinline__ Walk walk_begin(const Run& r) { return Walk{Unit{}, 0, 0, r.pair, r.u0, false}; }

__device__ __forceinline__ bool walk_next(const ChunkParams& p, const Run& r, Walk& w) {
  while (w.u < r.units) {
    w.unit = load_unit(p, w.u);
    w.u += r.pairs;
    if (!w.unit.whole) continue;
    w.lo = 0;
    w.hi = tiles_of(w.unit.len);
    return true;
  }
  while (w.at < r.u1 || (w.at == r.u1 && r.t1 > 0)) {
    w.unit = load_unit(p, p.rest[w.at]);
    w.first = w.at == r.u0;
    w.lo = w.first ? r.t0 : 0;
    w.hi = w.at == r.u1 ? r.t1 : tiles_of(w.unit.len);
    ++w.at;
    if (w.hi > w.lo) return true;
  }
  return false;
}

// Page ids of a request's pages base .. base + 31, one a lane: -1 for one outside
// the pool (reported; its keys are masked and page 0 is read in its place) or past
// the unit's last key.
__device__ __forceinline__ int page_window(const ChunkParams& p, const Unit& unit, int base, int lane) {
  const int k = base + lane;
  if (k >= pages_of(unit.len)) return -1;
  const int page = k < p.max_pages ? p.block_table[static_cast<long long>(unit.req) * p.max_pages + k] : -1;
  if (page >= 0 && page < p.num_pages) return page;
  report(p.status, MLA_ERR_BAD_INDEX);
  return -1;
}

// Whether the plan is that of the caller's offsets and lengths, and these are in
// range; the call's results are those of the plan either way.
__device__ __forceinline__ void check_plan(const ChunkParams& p) {
  if ((p.cu != nullptr || p.lens != nullptr) && blockIdx.x == 0 && (threadIdx.x & 31) == 0 && p.head[kHeadBroken] != 0)
    report(p.status, MLA_ERR_BAD_INDEX);
  for (int i = blockIdx.x * 32 + (threadIdx.x & 31); i <= p.batch; i += gridDim.x * 32)
    if ((p.cu != nullptr && p.made[i] != p.cu[i]) ||
        (p.lens != nullptr && i < p.batch && p.made[p.batch + 1 + i] != p.lens[i]))
      report(p.status, MLA_ERR_STALE_PLAN);
}

__device__ __forceinline__ void fail(volatile int* abort_flag, int32_t* status) {
  *abort_flag = 1;
  report(status, MLA_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ FP8 records

// E of a key: 8 k - 10, its largest scale being in 2^(8 k - 11) .. 2^(8 k - 3).  Within
// -66 .. 62, so that weights of keys that far apart stay floats: scales below 2^-61
// keep fewer bits, from 2^69 on values overflow.
__device__ __forceinline__ int key_exponent(const float4& scale) {
  const float most = fmaxf(fmaxf(fabsf(scale.x), fabsf(scale.y)), fmaxf(fabsf(scale.z), fabsf(scale.w)));
  const int e = static_cast<int>(__float_as_uint(most) >> 23) - 127;
  return ((min(max(e, -61), 61) + 11) >> 3) * 8 - 10;
}

__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// 16 codes times their key's scale / 2^E, as fp16, into the two 16-byte chunks from
// `chunk` on of a swizzled 128-byte row.
__device__ __forceinline__ uint32_t scaled2(uint32_t two, __half2 scale) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h), scale);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 scaled8(uint32_t a, uint32_t b, __half2 scale) {
  return make_uint4(scaled2(a & 0xffffu, scale), scaled2(a >> 16, scale), scaled2(b & 0xffffu, scale),
                    scaled2(b >> 16, scale));
}

__device__ __forceinline__ void store_codes(uint8_t* row, uint32_t chunk, uint32_t swz, const uint4& codes,
                                            __half2 scale) {
  *reinterpret_cast<uint4*>(row + ((chunk ^ swz) << 4)) = scaled8(codes.x, codes.y, scale);
  *reinterpret_cast<uint4*>(row + (((chunk + 1) ^ swz) << 4)) = scaled8(codes.z, codes.w, scale);
}

// What a converting lane has of a page: kLaneKeys keys (8 a warp at a time) and every
// fourth 16-byte piece of their records: the same quarter of every 64-dim slice.  The four
// lanes of a key read 64 bytes in a row, and the stores of eight lanes (two keys of
// different parity) go to eight different bank groups.
struct RecordLane {
  int key;      // of the page, the first
  int quarter;  // of a slice
  uint32_t swz;
};
__device__ __forceinline__ RecordLane record_lane(int warp, int lane) {
  const int key = 8 * warp + (lane >> 2);
  return RecordLane{key, lane & 3, static_cast<uint32_t>(key & 7)};
}

__device__ __forceinline__ const uint8_t* record_at(const ChunkParams& p, int page, int key) {
  return p.records + (static_cast<long long>(max(page, 0)) * kTile + key) * MLA_RECORD_BYTES;
}

// Whether the unit's request has been converted as a whole (chunk_convert_kernel).
__device__ __forceinline__ bool converted(const ChunkParams& p, const Unit& unit) {
  return unit.pages0 >= 0 && p.conv[unit.req + 1] <= p.room;
}

// Converts V pages: this CTA's 256 dims of both pages of a tile; keys behind the
// unit's last one (and pages outside the pool) as zeros.  Two pages' loads in
// flight.
__device__ __forceinline__ bool convert_v(const ChunkParams& p, const Run& run, uint32_t rank, int warp, int lane,
                                          uint8_t* sV, const CUtensorMap* map, uint64_t* bars, uint32_t bar0,
                                          volatile int* abort_flag, uint64_t wait_ns) {
  const RecordLane me = record_lane(warp, lane);
  Walk w = walk_begin(run);
  uint32_t n = 0;
  bool ok = true;
  const uint64_t pol = policy_evict_last();
  uint4 raw[2][kLaneKeys][4];
  float4 key_scale[2][kLaneKeys];
  int left[2];  // keys of the page that count, less the lane's first one
  while (ok && walk_next(p, run, w)) {
    const int pages = min(pages_of(w.unit.len), 2 * w.hi);
    if (converted(p, w.unit)) {  // (rows behind the last key are zeros there)
      for (int k = 2 * w.lo; k < pages && ok; ++k, ++n) {
        const int s = static_cast<int>(n % kVStages), r = static_cast<int>(n / kVStages);
        if (r >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&bars[V_EMPTY + s], (r - 1) & 1, abort_flag, wait_ns));
        if (ok && warp == 0)
          tma_load_4d_pair_warp(sV + s * kVBytes, map, bar0 + 8 * (V_FULL + s), kVBytes, 0, 0, 4 * static_cast<int>(rank),
                                w.unit.pages0 + k, pol);
        else if (ok && lane == 0)
          mbar_arrive_remote_relaxed(bar0 + 8 * (V_FULL + s));
      }
      continue;
    }
    int ids = 0, base = -32;
    const uint8_t* from;
    auto find = [&](int k, int h) {  // page k: where this lane's first key is, and how many count
      if (k - base >= 32) {
        base = k;
        ids = page_window(p, w.unit, base, lane);
      }
      const int id = __shfl_sync(0xffffffffu, ids, k - base);
      left[h] = id < 0 ? 0 : w.unit.len - k * kTile - me.key;
      from = record_at(p, id, me.key);
    };
    auto load = [&](int h, int y, int i) {  // the lane's key y: a quarter of slice i
      const uint8_t* rec = from + y * (8 * kConverters * MLA_RECORD_BYTES);
      if (i == 0) key_scale[h][y] = __ldcg(reinterpret_cast<const float4*>(rec + kDv));
      raw[h][y][i] = __ldcg(reinterpret_cast<const uint4*>(rec + 256 * rank + 16 * me.quarter + 64 * i));
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * w.lo + h >= pages) continue;
      find(2 * w.lo + h, h);
#pragma unroll
      for (int y = 0; y < kLaneKeys; ++y)
#pragma unroll
        for (int i = 0; i < 4; ++i) load(h, y, i);
    }
    for (int k0 = 2 * w.lo; k0 < pages && ok; k0 += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (k0 + h >= pages) continue;
        const int s = static_cast<int>(n % kVStages), r = static_cast<int>(n / kVStages);
        ++n;
        const int mine = left[h];
        const bool more = k0 + h + 2 < pages;
        if (more) find(k0 + h + 2, h);
        if (ok && r >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&bars[V_EMPTY + s], (r - 1) & 1, abort_flag, wait_ns));
        const uint32_t chunk = static_cast<uint32_t>(2 * me.quarter);
#pragma unroll
        for (int y = 0; y < kLaneKeys; ++y) {
          const float4 sc = key_scale[h][y];
          const float down = two_to(-key_exponent(sc));
          const __half2 scale[2] = {__float2half2_rn((rank == 0 ? sc.x : sc.z) * down),
                                    __float2half2_rn((rank == 0 ? sc.y : sc.w) * down)};
          uint8_t* row = sV + s * kVBytes + (me.key + 8 * kConverters * y) * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i, row += kSliceBytes) {
            if (mine > 8 * kConverters * y) {
              store_codes(row, chunk, me.swz, raw[h][y][i], scale[i >> 1]);
            } else {
              *reinterpret_cast<uint4*>(row + ((chunk ^ me.swz) << 4)) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(row + (((chunk + 1) ^ me.swz) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            if (more) load(h, y, i);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && ok) arrive_pair(bar0 + 8 * (V_FULL + s));
      }
    }
  }
  return ok;
}

// The scales of a unit's tiles, in turn in two buffers of [4 groups][128 keys]:
// lane i has keys 4 i .. of a tile, the next tile's loads in flight.  (Pages outside
// the pool or past the last one: page 0's, whose scores are masked.)  With them each
// key's E and the tile's.
__device__ __forceinline__ bool stage_scales(const ChunkParams& p, const Walk& w, int lane, uint8_t* smem,
                                             uint64_t* bars, volatile int* abort_flag, uint64_t wait_ns,
                                             uint32_t& n) {
  float4 key[4];
  int ids = 0, base = -32, live = 0;  // live: this lane's keys that are any
  auto load = [&](int j) {
    if (2 * j - base >= 32) {
      base = 2 * j;
      ids = page_window(p, w.unit, base, lane);
    }
    const int page = __shfl_sync(0xffffffffu, ids, 2 * j + (lane >> 4) - base);
    live = page < 0 ? 0 : w.unit.len - j * kBN - 4 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      key[i] = __ldcg(reinterpret_cast<const float4*>(record_at(p, page, 4 * (lane & 15) + i) + kDv));
  };
  bool ok = true;
  load(w.lo);
  for (int j = w.lo; j < w.hi && ok; ++j, ++n) {
    if (n >= 2)
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[SCALE_EMPTY + (n & 1)], ((n >> 1) - 1) & 1, abort_flag, wait_ns));
    int e[4], least = INT_MAX, most = INT_MIN;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[i] = key_exponent(key[i]);
      if (i < live) {
        least = min(least, e[i]);
        most = max(most, e[i]);
      }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    float4* to = reinterpret_cast<float4*>(smem + kOffScales) + (n & 1) * (5 * kBN / 4) + lane;
    to[4 * kBN / 4] = make_float4(static_cast<float>(e[0]), static_cast<float>(e[1]), static_cast<float>(e[2]),
                                  static_cast<float>(e[3]));
    const int all = least == most ? least : 0;  // (no key at all: whatever)
    if (lane == 0)
      reinterpret_cast<float2*>(smem + kOffTileE)[n & 1] =
          make_float2(least < most ? kMixed : static_cast<float>(all), two_to(-all));
    to[0] = make_float4(key[0].x, key[1].x, key[2].x, key[3].x);
    to[kBN / 4] = make_float4(key[0].y, key[1].y, key[2].y, key[3].y);
    to[2 * kBN / 4] = make_float4(key[0].z, key[1].z, key[2].z, key[3].z);
    to[3 * kBN / 4] = make_float4(key[0].w, key[1].w, key[2].w, key[3].w);
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(&bars[SCALE_FULL + (n & 1)]);
    if (j + 1 < w.hi) load(j + 1);
  }
  return ok;
}

constexpr uint64_t kStallWaitNs = 200000;  // wait budget of the stall-test instance, whose first K stage is never loaded

template <bool kHalf, bool kFp8, bool kStall = false>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of(kFp8), 1)
    chunk_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap rope_map,
                 const ChunkParams p) {
  constexpr uint64_t kWaitNs = kStall ? kStallWaitNs : MLA_WAIT_LIMIT_NS;
  const uint32_t rank = cluster_ctarank();
  extern __shared__ __align__(1024) uint8_t smem[];  // swizzle atoms need 1024-byte alignment
  uint8_t* sQ = smem;
  uint8_t* sK = smem + kOffK;
  uint8_t* sV = smem + kOffV;
  uint8_t* sP = smem + kOffP;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  float* sRow = reinterpret_cast<float*>(smem + kOffRow);

  const int tid = threadIdx.x;
  if (tid == 0) MLA_TRACE(0, 0);
  // by a shuffle: the compiler then knows that a warp takes one role, and keeps
  // MMA operands in uniform registers
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if ((smem_u32(smem) & 1023u) != 0u) {  // not what was asked for (all CTAs alike)
    if (tid == 0) report(p.status, MLA_ERR_UNSUPPORTED);
    return;
  }
  if (tid == 0) {
    *abort_flag = 0;
    // the barriers that MMAs wait for are the even CTA's and count both CTAs' parts
    mbar_init(&bars[Q_FULL], 2);
    mbar_init(&bars[Q_EMPTY], 1);
    for (int i = 0; i < (kFp8 ? kFp8Stages : kKStages); ++i) {
      mbar_init(&bars[K_FULL + i], 2);
      mbar_init(&bars[K_EMPTY + i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&bars[V_FULL + i], 2 * (kFp8 ? kConverters : 1));
      mbar_init(&bars[V_EMPTY + i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&bars[S_FULL + i], 1);
    mbar_init(&bars[S_FIRST], 2 * kSoftmax);
    mbar_init(&bars[S_ALL], 2 * kSoftmax);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[SCALE_FULL + i], 1);
      mbar_init(&bars[SCALE_EMPTY + i], kSoftmax);
    }
    mbar_init(&bars[P_FULL], 2 * kSoftmax);
    mbar_init(&bars[PV_DONE], 1);
    mbar_init(&bars[TAIL], 1);
    mbar_init(&bars[DRAIN], 1);
    fence_mbar_init_cluster();
  }
  if (warp == kWarpMma) {
    tmem2_alloc(tmem_slot, kTmemCols);
    tmem2_relinquish();
  }
  if (warp == kWarpQ && lane == 0) {
    prefetch_tmap(&q_map);
    prefetch_tmap(&k_map);
    prefetch_tmap(&v_map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();  // the other CTA's barriers are ready before anything arrives there
  cluster_wait();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_prior_grid();  // the kernel before is done from here on
  pdl_launch_dependents();
  const Run run = load_run(p);
  const int causal = p.head[kHeadCausal];
  if (tid == 0) MLA_TRACE(0, 1);
  Walk w = walk_begin(run);

  if (kFp8 && warp >= kWarpV) {
    // ------------------------------------------------------------ FP8 records: V converted
    const uint32_t bar0 = mapa_shared(smem_u32(bars), 0);
    const bool ok = convert_v(p, run, rank, warp - kWarpV, lane, sV, &v_map, bars, bar0, abort_flag, kWaitNs);
    if (!ok && lane == 0) {
      fail(abort_flag, p.status);
      // copies in flight land (bounded) before this CTA may end
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) {
      }
    }
    __syncwarp();
  } else if (warp > kWarpMma) {
    // ------------------------------------------------------------ loads: Q, K or V
    bool ok = true;
    const uint64_t pol_q = policy_evict_first(), pol_kv = policy_evict_last();
    const uint32_t bar0 = mapa_shared(smem_u32(bars), 0);
    auto expect = [&](int bar, uint32_t bytes) { mbar_arrive_expect_tx_remote_relaxed(bar0 + 8 * bar, bytes); };
    uint32_t n = 0, tails = 0;  // stages (or units of Q) and tail pages so far
    uint32_t scaled = 0;        // FP8 records: tiles whose scales are written
    while (ok && walk_next(p, run, w)) {
      if (warp == kWarpQ) {
        if (n >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&bars[Q_EMPTY], (n - 1) & 1, abort_flag, kWaitNs));
        if (ok && lane == 0) {
          expect(Q_FULL, kOffK);
          const int row0 = w.unit.row0 + kCtaRows * static_cast<int>(rank);
          tma_load_4d_pair(sQ, &q_map, bar0 + 8 * Q_FULL, 0, row0, 0, 0, pol_q);
          if (kFp8)
            tma_load_4d_pair(sQ + (kSlices - 1) * kSliceBytes, &rope_map, bar0 + 8 * Q_FULL, 0, row0, kSlices - 1, 0,
                             pol_q);
        }
        ++n;
        if (kFp8 && ok) ok = stage_scales(p, w, lane, smem, bars, abort_flag, kWaitNs, scaled);
        continue;
      }
      const int pages = pages_of(w.unit.len);
      int ids = 0, base = -32;
      for (int j = w.lo; j < w.hi && ok; ++j) {
        if (2 * j - base >= 32) {
          base = 2 * j;
          ids = page_window(p, w.unit, base, lane);
        }
        if (warp == kWarpK) {
          const int k = 2 * j + static_cast<int>(rank);
          const int page = max(__shfl_sync(0xffffffffu, ids, k - base), 0);
          constexpr int kStages = kFp8 ? kFp8Stages : kKStages, kLoads = kFp8 ? kParts : 3;
          constexpr int kBytes = kFp8 ? kSliceBytes : kKBytes;
          // (the whole warp, of which one lane issues)
          for (int c = 0; c < kLoads && ok; ++c, ++n) {
            const int s = static_cast<int>(n % kStages), r = static_cast<int>(n / kStages);
            if (r >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&bars[K_EMPTY + s], (r - 1) & 1, abort_flag, kWaitNs));
            if (!ok || (kStall && rank == 0 && n == 0)) continue;
            if (k < pages) {
              // FP8 records, in 16-bit units: 128 codes, the last time the 64 RoPE dims (from byte 528 on)
              const int x = !kFp8 ? 0 : c < 4 ? 64 * c : 264, slice = kFp8 ? 0 : kKSlices * c;
              tma_load_4d_pair_warp(sK + s * kBytes, &k_map, bar0 + 8 * (K_FULL + s), kBytes, x, 0, slice, page, pol_kv);
            } else if (lane == 0) {  // no such page: whatever the stage holds is masked
              mbar_arrive_remote_relaxed(bar0 + 8 * (K_FULL + s));
            }
          }
          continue;
        }
        for (int half = 0; half < 2 && ok; ++half) {
          const int k = 2 * j + half;
          if (k >= pages) break;  // its P V is left out
          const int id = __shfl_sync(0xffffffffu, ids, k - base), page = max(id, 0);
          const int keep = id < 0 ? 0 : w.unit.len - k * kTile;  // rows of the page that are keys
          const int s = static_cast<int>(n % kVStages), r = static_cast<int>(n / kVStages);
          uint8_t* dst = sV + s * kVBytes;
          if (r >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&bars[V_EMPTY + s], (r - 1) & 1, abort_flag, kWaitNs));
          if (ok && keep >= kTile) {
            tma_load_4d_pair_warp(dst, &v_map, bar0 + 8 * (V_FULL + s), kVBytes, 0, 0, 4 * static_cast<int>(rank), page,
                                  pol_kv);
          } else if (ok && lane == 0) {  // onto this CTA's own barrier
            mbar_arrive_expect_tx(&bars[TAIL], kVBytes);
            tma_load_4d(dst, &v_map, &bars[TAIL], 0, 0, 4 * static_cast<int>(rank), page, pol_kv);
          }
          ++n;
          if (!ok || keep >= kTile) continue;
          ok = __all_sync(0xffffffffu, mbar_wait(&bars[TAIL], tails & 1, abort_flag, kWaitNs));
          ++tails;
          if (!ok) continue;
          for (int b = 0; b < 4; ++b) {
            uint4* z = reinterpret_cast<uint4*>(dst + b * kSliceBytes + keep * 128);
            for (int i = lane; i < (kTile - keep) * 8; i += 32) z[i] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive_pair(bar0 + 8 * (V_FULL + s));
        }
      }
    }
    if (warp == kWarpQ) check_plan(p);
    if (!ok && lane == 0) {
      fail(abort_flag, p.status);
      // copies in flight land (bounded) before this CTA may end
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) {
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMAs
    // The even CTA's warp issues for the pair, converged: its control flow and
    // operands are the same in all lanes.
    if (rank == 0) {
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      constexpr uint32_t idesc_qk = idesc_16bit_f32(128, kBN, false, kHalf);
      constexpr uint32_t idesc_codes = idesc_e4m3_f32(128, kBN);
      constexpr uint32_t idesc_pv = idesc_16bit_f32(128, 256, true, kHalf || kFp8);
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(sV), kSliceBytes, 1024);  // MN-major
      const uint64_t p_desc = sdesc_sw128(smem_u32(sP), 16, 1024);
      auto wait = [&](int bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(&bars[bar], parity, abort_flag, kWaitNs));
      };
      bool ok = true;
      uint32_t kn = 0, vn = 0, tn = 0, qn = 0;  // K and V stages, tiles and units so far
      int before = 0;                           // pages of the tile whose P V is due
      bool fresh = false;                       // that tile is its unit's first here
      auto issue_pv = [&]() {
        ok = ok && wait(P_FULL, (tn - 1) & 1);
        MLA_TRACE(3, tn - 1);
        for (int half = 0; half < before && ok; ++half, ++vn) {
          const int vs = static_cast<int>(vn % kVStages);
          ok = wait(V_FULL + vs, (vn / kVStages) & 1);
          if (!ok) break;
          MLA_TRACE(4 + half, tn - 1);
          tc_fence_after();
          const uint64_t vd = v_desc + static_cast<uint64_t>((vs * kVBytes) >> 4);
          const uint64_t pd = p_desc + static_cast<uint64_t>((half * kSliceBytes) >> 4);
          const bool first = fresh && half == 0;
#pragma unroll
          for (int d = 0; d < 2; ++d)
            umma2_f16_warp4<2, 128>(tm + 128u * d, pd, vd + static_cast<uint64_t>((2 * d * kSliceBytes) >> 4), idesc_pv,
                                    first ? 0u : 1u);
          umma2_commit_warp(&bars[V_EMPTY + vs]);
        }
        if (ok) umma2_commit_warp(&bars[PV_DONE]);
      };
      while (ok && walk_next(p, run, w)) {
        const int pages = __shfl_sync(0xffffffffu, pages_of(w.unit.len), 0);
        const int lo = __shfl_sync(0xffffffffu, w.lo, 0), hi = __shfl_sync(0xffffffffu, w.hi, 0);
        // between units the last P V goes first: the output waits for it, and Q K^T for the new Q
        if (before > 0) issue_pv();
        before = 0;
        if (ok) ok = wait(Q_FULL, qn & 1);
        MLA_TRACE(1, qn);
        ++qn;
        for (int j = lo; j < hi && ok; ++j) {
          if constexpr (kFp8) {
#pragma unroll
            for (int c = 0; c < kParts; ++c, ++kn) {  // a sum each, in four buffers
              // the fifth waits until the softmax warps have begun with this tile: the P V that they wait for goes first
              if (c == 4 && before > 0) issue_pv();
              if (ok && c == 0 && tn >= 1) ok = wait(S_ALL, (tn - 1) & 1);
              if (ok && c == 4) ok = wait(S_FIRST, tn & 1);
              const int ks = static_cast<int>(kn % kFp8Stages);
              if (ok) ok = wait(K_FULL + ks, (kn / kFp8Stages) & 1);
              if (!ok) break;
              if (c == 0) MLA_TRACE(2, tn);
              if (c == kParts - 1) MLA_TRACE(6, tn);
              tc_fence_after();
              const uint32_t s_col = tm + kTmemS + 64u * (kn & 3);
              const uint64_t kd = k_desc + static_cast<uint64_t>((ks * kSliceBytes) >> 4);
#pragma unroll
              for (int h = 0; h < (c < 4 ? 2 : 1); ++h) {  // codes, remainders
                const int slice = c < 4 ? c + 4 * h : kSlices - 1;
                const uint64_t qd = q_desc + static_cast<uint64_t>((slice * kSliceBytes) >> 4);
                if (c < 4)
                  umma2_f8_warp4<2, 2>(s_col, qd, kd, idesc_codes, h);
                else
                  umma2_f16_warp4<2, 2>(s_col, qd, kd, idesc_qk, 0u);
              }
              umma2_commit_warp(&bars[S_FULL + (kn & 3)]);
              umma2_commit_warp(&bars[K_EMPTY + ks]);
            }
          } else {
            const uint32_t s_col = tm + kTmemS + 64u * (tn & 1);
#pragma unroll
            for (int c = 0; c < 3; ++c, ++kn) {
              const int ks = static_cast<int>(kn % kKStages);
              if (ok) ok = wait(K_FULL + ks, (kn / kKStages) & 1);
              if (!ok) break;
              if (c == 0) MLA_TRACE(2, tn);
              if (c == 2) MLA_TRACE(6, tn);
              tc_fence_after();
              const uint64_t kd = k_desc + static_cast<uint64_t>((ks * kKBytes) >> 4);
              const uint64_t qd = q_desc + static_cast<uint64_t>((c * kKBytes) >> 4);
#pragma unroll
              for (int s = 0; s < kKSlices; ++s)
                umma2_f16_warp4<2, 2>(s_col, qd + static_cast<uint64_t>((s * kSliceBytes) >> 4),
                                      kd + static_cast<uint64_t>((s * kSliceBytes) >> 4), idesc_qk,
                                      (c == 0 && s == 0) ? 0u : 1u);
              umma2_commit_warp(&bars[K_EMPTY + ks]);
            }
          }
          if (!ok) break;
          if (!kFp8) umma2_commit_warp(&bars[S_FULL + (tn & 1)]);
          if (j == hi - 1) umma2_commit_warp(&bars[Q_EMPTY]);
          if (!kFp8 && before > 0) issue_pv();
          ++tn;
          before = min(pages - 2 * j, 2);
          fresh = j == lo;
        }
      }
      if (ok && before > 0) issue_pv();
      if (!ok && lane == 0) fail(abort_flag, p.status);
      // every MMA is done with shared memory and TMEM before this CTA ends
      umma2_commit_warp(&bars[DRAIN]);
      mbar_wait(&bars[DRAIN], 0, nullptr, kWaitNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    // Warp quarter q (TMEM lanes 32 q ..): rows 32 (q & 1) .. of this CTA and page
    // q >> 1 of the tile (or 256-dim half of the output); warps 4 .. 7 the second
    // 32 keys (128 dims) of those.
    const int q = warp & 3, kh = q >> 1, ch = warp >> 2, part = 2 * kh + ch;
    const int r = 32 * (q & 1) + lane, row = kCtaRows * static_cast<int>(rank) + r;  // row: of the unit
    const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
    const uint32_t s_addr = tmem + lane_base + kTmemS + 32u * ch;
    const uint32_t o_addr = tmem + lane_base + 128u * ch;
    const uint32_t row_bar = 1 + (q & 1);  // the four warps of these 32 rows
    const uint32_t p_full = mapa_shared(smem_u32(&bars[P_FULL]), 0), s_first = mapa_shared(smem_u32(&bars[S_FIRST]), 0);
    uint8_t* prow = sP + kh * kSliceBytes + r * 128;
    const uint32_t swz = static_cast<uint32_t>(r & 7);
    // What this thread has for its row, to be shared with the other three.  (Two
    // buffers in turn, a barrier each time: a warp may be one turn ahead of one
    // that still reads, not two.)
    uint32_t turn = 0;
    auto shared_row = [&](float v) {
      float* buf = sRow + (turn & 1) * 4 * kCtaRows + r;
      buf[part * kCtaRows] = v;
      ++turn;
      return buf;
    };
    bool ok = true;
    uint32_t tn = 0, sn = 0;
    // what the tile loop keeps of a unit: the keys this row sees (rows past the unit's last one: unmasked, not
    // stored), the block table's row, and its pages outside the pool within the window from page `base` on
    int limit, base;
    uint32_t bad;
    float c_log2 = p.scale_log2;  // FP8 records: times 2^-f, the scores being 2^f as large
    float up = 1.f;               // 2^f of this row's query
    float2 factor;                // of the unit that is entered: 2^f and 2^-f
    const float* const sScale = reinterpret_cast<const float*>(smem + kOffScales) + kTile * kh + 32 * ch;
    auto look = [&](int page) {
      base = page;
      const int k = base + lane;
      bool out = false;
      if (k < pages_of(w.unit.len)) {
        const int id = k < p.max_pages ? p.block_table[static_cast<long long>(w.unit.req) * p.max_pages + k] : -1;
        out = id < 0 || id >= p.num_pages;
      }
      bad = __ballot_sync(0xffffffffu, out);
    };
    auto enter = [&]() {
      if (!walk_next(p, run, w)) return false;
      limit = row >= w.unit.rows ? 1 << 30
              : causal           ? min(w.unit.len, w.unit.limit0 + (w.unit.rel + row) / p.h_q)
                                 : w.unit.len;
      look(2 * w.lo);
      if constexpr (kFp8) {
        // (the row after the unit's last one is another unit's, or none)
        const int at = w.unit.row0 + min(row, w.unit.rows - 1);
        factor = *reinterpret_cast<const float2*>(p.queries + static_cast<long long>(at) * kQueryRow + 2 * kDv);
      }
      return true;
    };
    const int dim0 = 256 * kh + 128 * ch;
    // 8 words of a row (of 16 it + 8 up + lane / 4): word n of lane q4 -> word q4 of
    // lane n, within four lanes and four words: each then holds whole 16-byte pieces,
    // and a store of the warp covers 64 bytes of 8 rows
    auto store16 = [&](uint32_t (&x)[8], int it, int up, long long first, int rows) {
      const int q4 = lane & 3, orow = row - lane + 16 * (it & 1) + 8 * up + (lane >> 2);
      uint16_t* dst = static_cast<uint16_t*>(p.out) + (first + orow) * kDv + dim0 + 64 * (it >> 1) + 8 * q4;
#pragma unroll
      for (int g = 0; g < 8; g += 4) {
        uint32_t* y = x + g;
        {
          const bool odd = q4 & 1;
          const uint32_t s0 = odd ? y[0] : y[1], s1 = odd ? y[2] : y[3];
          const uint32_t r0 = __shfl_xor_sync(0xffffffffu, s0, 1), r1 = __shfl_xor_sync(0xffffffffu, s1, 1);
          if (odd) {
            y[0] = r0;
            y[2] = r1;
          } else {
            y[1] = r0;
            y[3] = r1;
          }
        }
        {
          const bool odd = q4 & 2;
          const uint32_t s0 = odd ? y[0] : y[2], s1 = odd ? y[1] : y[3];
          const uint32_t r0 = __shfl_xor_sync(0xffffffffu, s0, 2), r1 = __shfl_xor_sync(0xffffffffu, s1, 2);
          if (odd) {
            y[0] = r0;
            y[1] = r1;
          } else {
            y[2] = r0;
            y[3] = r1;
          }
        }
        if (orow < rows) *reinterpret_cast<uint4*>(dst + 8 * g) = make_uint4(y[0], y[1], y[2], y[3]);
      }
    };
    constexpr float lift = kLift<kHalf || kFp8>;
    bool more = enter();
    while (more) {
      float ref = -INFINITY, l = 0.f;
      if constexpr (kFp8) {
        up = factor.x;
        c_log2 = p.scale_log2 * factor.y;
      }
      for (int j = w.lo; j < w.hi; ++j, ++tn) {
        int seen = limit - j * kBN - kTile * kh - 32 * ch;
        if (2 * j - base >= 32) look(2 * j);
        if ((bad >> (2 * j + kh - base)) & 1u) seen = 0;
        // (pages past the unit's last one have keys past every valid row's limit; rows past its last row are masked
        // there too, for what the stage holds may be no number)
        if (row >= w.unit.rows && (2 * j + kh) * kTile >= w.unit.len) seen = 0;
        float s[32], top;
        float2 tile_e = make_float2(0.f, 1.f);
        if constexpr (kFp8) {
          const float* scales = sScale + (tn & 1) * 5 * kBN;
          ok = ok && mbar_wait(&bars[SCALE_FULL + (tn & 1)], (tn >> 1) & 1, abort_flag, kWaitNs);
#pragma unroll
          for (int n = 0; n < kParts; ++n, ++sn) {
            if (n == kParts - 1) tile_e = reinterpret_cast<const float2*>(smem + kOffTileE)[tn & 1];
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&bars[S_FULL + (sn & 3)], (sn >> 2) & 1, abort_flag, kWaitNs));
            if (tid == 0 && n == 0) MLA_TRACE(7, tn);
            tc_fence_after();
            uint32_t v[32];
            tmem_ld32(s_addr + 64u * (sn & 3), v);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && n == 0) mbar_arrive_remote_relaxed(s_first);
            if (lane == 0 && n == kParts - 1) {
              mbar_arrive_remote_relaxed(s_first + 8 * (S_ALL - S_FIRST));
            }
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 f = n == kParts - 1 ? make_float4(up, up, up, up)
                                               : *reinterpret_cast<const float4*>(scales + kBN * n + i);
              const float2 f2[2] = {make_float2(f.x, f.y), make_float2(f.z, f.w)};
#pragma unroll
              for (int k = i; k < i + 4; k += 2) {
                const float2 y = make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                const float2 z = n == 0 ? __fmul2_rn(y, f2[(k - i) >> 1])
                                        : __ffma2_rn(y, f2[(k - i) >> 1], make_float2(s[k], s[k + 1]));
                s[k] = z.x;
                s[k + 1] = z.y;
              }
            }
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; ++i) m4[i & 3] = fmaxf(m4[i & 3], s[i]);
          top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        } else {
          ok = __all_sync(0xffffffffu, ok && mbar_wait(&bars[S_FULL + (tn & 1)], (tn >> 1) & 1, abort_flag, kWaitNs));
          if (tid == 0) MLA_TRACE(7, tn);
          tc_fence_after();
          tmem_ld32_max(s_addr + 64u * (tn & 1), s, top);
          tmem_wait_ld();
        }
        if (__any_sync(0xffffffffu, seen < 32)) {
          const uint32_t keep = seen >= 32 ? ~0u : (seen <= 0 ? 0u : (1u << seen) - 1u);
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (!((keep >> i) & 1u)) s[i] = -INFINITY;
            m4[i & 3] = fmaxf(m4[i & 3], s[i]);
          }
          top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
        // (FP8 records: of scores to which the keys' E are added, one by one or as one for all)
        float c = c_log2, add = 0.f, down = 1.f;  // down: 2^-add
        bool mixed = false;
        const float* key_e = sScale + (tn & 1) * 5 * kBN + 4 * kBN;
        if constexpr (kFp8) {
          add = tile_e.x;
          down = tile_e.y;
          mixed = add == kMixed;
          if (mixed) {
            top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              s[i] = fmaf(s[i], c, key_e[i]);
              top = fmaxf(top, s[i]);
            }
            c = down = 1.f;
            add = 0.f;
          }
        }
        // the row's maximum over its four threads
        const float* buf = shared_row(top);
        ok = !named_bar_or(row_bar, 128, !ok);  // (a warp that gave up waiting takes the others along)
        if (!ok) break;
        const float mt = fmaf(fmaxf(fmaxf(buf[0], buf[kCtaRows]), fmaxf(buf[2 * kCtaRows], buf[3 * kCtaRows])), c, add);
        const float r_new = mt > ref + (kTau + lift) ? mt - lift : ref;
        const float alpha = r_new == ref ? 1.f : ex2(ref - r_new);
        ref = r_new;
        const float mref = ref == -INFINITY ? 0.f : ref;
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 cl = make_float2(c, c), nr = make_float2(add - mref, add - mref);
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), cl, nr);
          const float p0 = ex2(x.x), p1 = ex2(x.y);
          pk[i] = pack2<kHalf || kFp8>(p0, p1);
          ls[i & 1] = __fadd2_rn(ls[i & 1], make_float2(p0, p1));
        }
        float sum_p = (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
        if constexpr (kFp8) {  // without the 2^E
          sum_p *= down;
          if (mixed) {
            sum_p = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) sum_p = fmaf(ex2(s[i] - mref), two_to(-static_cast<int>(key_e[i])), sum_p);
          }
          __syncwarp();  // every lane has read the scales
          if (lane == 0) mbar_arrive(&bars[SCALE_EMPTY + (tn & 1)]);
        }
        l = l * alpha + sum_p;
        // P V of the tile before is done: P may be overwritten and O rescaled
        if (tn >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&bars[PV_DONE], (tn - 1) & 1, abort_flag, kWaitNs));
        if (j > w.lo && ok && __any_sync(0xffffffffu, alpha != 1.f)) {
          tc_fence_after();
#pragma unroll 1
          for (uint32_t c0 = 0; c0 < 128; c0 += 16) {
            uint32_t v[16];
            tmem_ld16(o_addr + c0, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
            tmem_st16(o_addr + c0, v);
          }
          tmem_wait_st();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(prow + ((static_cast<uint32_t>(4 * ch + c) ^ swz) << 4)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_pair(p_full);
        if (tid == 0) MLA_TRACE(8, tn);
      }
      // the next unit is looked at while the last P V runs
      const bool direct = w.unit.parts == 1;
      const int rows = w.unit.rows, slot = w.unit.slot + (w.first ? run.piece : 0);
      const long long first = direct ? w.unit.row0 : static_cast<long long>(slot) * kRowsPerBlock;
      if (ok) more = enter();
      // the row's sum, in an order that all four share.  (A warp that gave up takes the others along.)
      const float* sum = shared_row(l);
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars[PV_DONE], (tn - 1) & 1, abort_flag, kWaitNs));
      ok = !named_bar_or(row_bar, 128, !ok);
      if (!ok) break;
      if (tid == 0) MLA_TRACE(10, tn);
      tc_fence_after();
      l = (sum[0] + sum[kCtaRows]) + (sum[2 * kCtaRows] + sum[3 * kCtaRows]);
      const float inv = l == 0.f ? 0.f : 1.f / l;  // 0: the row sees none of these keys
      // 16 rows x 64 dims at a time.  The load leaves a row's values with four
      // lanes, two of every eight each.
      const bool wide = !direct || p.out_type == MLA_DTYPE_FP32, half_out = p.out_type == MLA_DTYPE_FP16;
      auto load = [&](int it, uint32_t (&v)[32]) {
        tmem_ld_16x64(o_addr + 64 * (it >> 1) + (static_cast<uint32_t>(16 * (it & 1)) << 16), v);
        tmem_wait_ld();
      };
      if (wide) {
#pragma unroll 1
        for (int it = 0; it < 4; ++it) {
          uint32_t v[32];
          load(it, v);
#pragma unroll
          for (int up = 0; up < 2; ++up) {
            const int from = 16 * (it & 1) + 8 * up + (lane >> 2);  // lane that has this row's sum
            const float iv = __shfl_sync(0xffffffffu, inv, from);
            const int orow = row - lane + from;
            float* dst = (direct ? static_cast<float*>(p.out) : p.o_accum) + (first + orow) * kDv + dim0 +
                         64 * (it >> 1) + 2 * (lane & 3);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const float a = __uint_as_float(v[4 * n + 2 * up]), b = __uint_as_float(v[4 * n + 2 * up + 1]);
              if (orow < rows)
                *reinterpret_cast<float2*>(dst + 8 * n) =
                    iv == 0.f ? make_float2(0.f, 0.f) : make_float2(a * iv, b * iv);
            }
          }
        }
      } else {
#pragma unroll 1
        for (int it = 0; it < 4; ++it) {
          uint32_t v[32];
          load(it, v);
#pragma unroll
          for (int up = 0; up < 2; ++up) {
            const float iv = __shfl_sync(0xffffffffu, inv, 16 * (it & 1) + 8 * up + (lane >> 2));  // of that row's lane
            uint32_t x[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const float a = __uint_as_float(v[4 * n + 2 * up]) * iv, b = __uint_as_float(v[4 * n + 2 * up + 1]) * iv;
              x[n] = iv == 0.f ? 0u : half_out ? pack2<true>(a, b) : pack2<false>(a, b);
            }
            store16(x, it, up, first, rows);
          }
        }
      }
      if (part == 0 && row < rows)
        (direct ? p.lse : p.lse_accum)[first + row] =
            l == 0.f ? -INFINITY : (ref + lift + __log2f(l * two_to(-static_cast<int>(lift)))) * kLn2;
      if (tid == 0) MLA_TRACE(9, tn);
      // O has been read: the next unit's first P V waits for this warp's P
      tc_fence_before();
    }
    if (!ok && lane == 0) fail(abort_flag, p.status);
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // the other CTA loads, arrives and multiplies here no more
  cluster_wait();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem2_dealloc(tmem, kTmemCols);
  }
  cluster_arrive();  // neither CTA ends while the other gives TMEM back
  cluster_wait();
}

// ------------------------------------------------------------------ convert

// What a call over FP8 records prepares in the workspace.  Queries: 512 dims as E4M3
// codes of q 2^f and of what they leave of it, 2^f bringing the row's largest element
// to 128 .. 256 (f at most 40: a row of nothing but numbers below 2^-33 keeps fewer
// bits).  A row that holds an infinity or a NaN is codes of NaN.  Pages: the values
// of requests of kConvertUnits units and more that fit, rows behind the last key, and
// of pages outside the pool (reported), as zeros.  A warp a query, a block a page at
// a time.  Every unit that reads a page would convert it again, for 2.4 us a tile
// instead of 1.8: with no room for pages the mixed batch above takes 142 us, 3 chunks
// x 128 heads over 8000 keys 1080 instead of 740.  Why from three units on: 64 requests
// x 2 tokens x 128 heads (two units) over 4096 keys take 148 us, 166 with their pages
// converted before; x 3 tokens 199, and 213 without; 200 x 2 over 1000 keys 145 and 162.
__global__ void __launch_bounds__(256)
    chunk_convert_kernel(const ChunkParams p, const uint16_t* __restrict__ q, uint16_t* __restrict__ pages) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (long long i = blockIdx.x * 8ll + warp; i < p.rows; i += gridDim.x * 8ll) {
    const uint4* from = reinterpret_cast<const uint4*>(q + i * MLA_D_QK) + 2 * lane;
    const uint4 a = __ldcs(from), b = __ldcs(from + 1);
    const uint32_t two[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t most = 0;  // of the bits without the sign: infinities above numbers, NaN above those
#pragma unroll
    for (int k = 0; k < 8; ++k) most = max(most, max(two[k] & 0x7fffu, two[k] >> 16 & 0x7fffu));
    most = __reduce_max_sync(0xffffffffu, most);
    const bool finite = most < 0x7f80u;
    // (a subnormal's exponent field is 0: f is 40 there too)
    const int f = finite ? min(134 - static_cast<int>(most >> 7), 40) : 0;
    const float up = __uint_as_float(static_cast<uint32_t>(127 + f) << 23);
    uint32_t code[4], rest[4];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      uint32_t c[2], r[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 x = make_float2(__uint_as_float(two[k + h] << 16) * up,
                                     __uint_as_float(two[k + h] & 0xffff0000u) * up);
        c[h] = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
        const __half2_raw raw = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c[h]), __NV_E4M3);
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&raw));
        r[h] = __nv_cvt_float2_to_fp8x2(make_float2(x.x - y.x, x.y - y.y), __NV_SATFINITE, __NV_E4M3);
      }
      code[k >> 1] = finite ? c[0] | c[1] << 16 : 0x7f7f7f7fu;
      rest[k >> 1] = finite ? r[0] | r[1] << 16 : 0u;
    }
    uint8_t* to = p.queries + i * kQueryRow;
    reinterpret_cast<uint4*>(to)[lane] = make_uint4(code[0], code[1], code[2], code[3]);
    reinterpret_cast<uint4*>(to + kDv)[lane] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
    if (lane == 0)
      *reinterpret_cast<float2*>(to + 2 * kDv) = make_float2(up, __uint_as_float(static_cast<uint32_t>(127 - f) << 23));
  }
  const int total = min(p.conv[p.batch], p.room);
  for (int i = blockIdx.x; i < total; i += gridDim.x) {
    int lo = 0, hi = p.batch;  // conv[lo] <= i < conv[hi]
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
      const int n = __popc(__ballot_sync(0xffffffffu, at < hi && p.conv[at] <= i));
      lo += n * step;
      hi = min(lo + step, hi);
    }
    if (p.conv[lo + 1] > p.room) return;  // only whole requests, and this is the last one
    const int k = i - p.conv[lo], keys = p.made[p.batch + 1 + lo] - k * kTile;
    const int page = k < p.max_pages ? p.block_table[static_cast<long long>(lo) * p.max_pages + k] : -1;
    const bool good = page >= 0 && page < p.num_pages;
    if (!good && threadIdx.x == 0) report(p.status, MLA_ERR_BAD_INDEX);
    const int row0 = 8 * warp;
    const uint8_t* rec = p.records + (static_cast<long long>(good ? page : 0) * kTile + row0) * MLA_RECORD_BYTES;
    uint16_t* out = pages + (static_cast<long long>(i) * kTile + row0) * kDv;
    uint2 code[8][2];
    float4 scale[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const uint8_t* r = rec + n * MLA_RECORD_BYTES;
#pragma unroll
      for (int h = 0; h < 2; ++h) code[n][h] = __ldcs(reinterpret_cast<const uint2*>(r + 256 * h) + lane);
      scale[n] = __ldcs(reinterpret_cast<const float4*>(r + kDv));
    }
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float down = two_to(-key_exponent(scale[n]));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float mine = h == 0 ? (lane < 16 ? scale[n].x : scale[n].y) : (lane < 16 ? scale[n].z : scale[n].w);
        reinterpret_cast<uint4*>(out + n * kDv)[32 * h + lane] =
            good && row0 + n < keys ? scaled8(code[n][h].x, code[n][h].y, __float2half2_rn(mine * down))
                                    : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
}

// ------------------------------------------------------------------ combine

// Rows of the units that were cut (their pieces merged) and of those without
// keys (zeros):  out = sum_s e^(lse_s - m) O_s / Z, lse = m + ln Z.
// A warp a row, 16 columns a lane; four pieces in flight, their lse beside them.
// Bound by latency, the rows being at most 128 for each pair: about 5 us behind the
// attention of 64 requests x up to 6 drafts x 128 heads (6.5 with pieces loaded after
// the maximum of their lse, and units found after the wait).
__global__ void __launch_bounds__(128) chunk_combine_kernel(const ChunkParams p) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31;
  // what the plan says does not wait for the kernel before, which has waited for the plan
  const long long rows = static_cast<long long>(p.head[kHeadFix + p.schedule]) * kRowsPerBlock;
  const long long first = blockIdx.x * 4ll + (threadIdx.x >> 5);
  Unit unit{};
  if (first < rows) unit = load_unit(p, p.fix[first / kRowsPerBlock]);
  pdl_wait_prior_grid();  // (also by blocks without work: a plan made next must not meet the kernel before)
  pdl_launch_dependents();  // the next call's kernel sets up under this one (the same case, calls in a row: 148 -> 145 us)
  for (long long i = first; i < rows; i += gridDim.x * 4ll) {
    if (i != first) unit = load_unit(p, p.fix[i / kRowsPerBlock]);
    const int r = static_cast<int>(i % kRowsPerBlock);
    if (r >= unit.rows) continue;
    const long long at = static_cast<long long>(unit.slot) * kRowsPerBlock + r;
    float4 v[kAhead][4];
    float e[kAhead];
    auto load = [&](int s0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const bool in = s0 + k < unit.parts;
        const long long a = at + (s0 + k) * kRowsPerBlock;
        e[k] = in ? p.lse_accum[a] : -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          v[k][c] = in ? *reinterpret_cast<const float4*>(p.o_accum + a * kDv + 128 * c + 4 * lane)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    load(0);
    float m = -INFINITY;
    if (unit.parts > kAhead) {
      for (int s = lane; s < unit.parts; s += 32) m = fmaxf(m, p.lse_accum[at + s * kRowsPerBlock]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    } else {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) m = fmaxf(m, e[k]);
    }
    float4 acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    float z = 0.f;
    for (int s0 = 0; s0 < unit.parts; s0 += kAhead) {
      if (s0 > 0) load(s0);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float w = e[k] == -INFINITY ? 0.f : expf(e[k] - m);
        z += w;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[c].x = fmaf(w, v[k][c].x, acc[c].x);
          acc[c].y = fmaf(w, v[k][c].y, acc[c].y);
          acc[c].z = fmaf(w, v[k][c].z, acc[c].z);
          acc[c].w = fmaf(w, v[k][c].w, acc[c].w);
        }
      }
    }
    const float inv = z == 0.f ? 0.f : 1.f / z;
    const long long row = (static_cast<long long>(unit.row0) + r) * kDv + 4 * lane;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 o = make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv);
      const long long at_out = row + 128 * c;
      if (p.out_type == MLA_DTYPE_FP32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at_out) = o;
      else if (p.out_type == MLA_DTYPE_FP16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at_out) =
            make_uint2(pack2<true>(o.x, o.y), pack2<true>(o.z, o.w));
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at_out) =
            make_uint2(pack2<false>(o.x, o.y), pack2<false>(o.z, o.w));
    }
    if (lane == 0) p.lse[unit.row0 + r] = z == 0.f ? -INFINITY : m + logf(z);
  }
}

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 1024;

// Sum over the block of one value a thread, exclusive; *total gets all of it.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* s_warp, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T y = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    s_warp[lane] = y;
  }
  __syncthreads();
  const T base = warp > 0 ? s_warp[warp - 1] : T(0);
  *total = s_warp[31];
  __syncthreads();
  return base + x - v;
}

// What each pair does of the units, for schedule v.  A unit costs its tiles (half
// as much again over FP8 records that are not converted before: mixed batch 115 us,
// 120 with the same, 121 with twice as much) and kFixedCost more (its
// Q, its epilogue), in half tiles.  Pair i takes units i, i + pairs, .. as a whole
// while they fit its share of the whole cost; the others are cut so that every pair's
// share is filled: the pair whose room is reached at x of their sum begins there.  A
// cut within a unit's fixed part moves to its border.
__device__ __forceinline__ int tile_cost(int pages0, int v) { return v == 1 && pages0 < 0 ? 3 : 2; }

__device__ void plan_schedule(const ChunkPlanParams& p, int v, int units, int* cut_u, int* cut_t, int* s_warp,
                              long long* s_warp64) {
  const int tid = threadIdx.x;
  const ChunkSchedule& out = p.schedule[v];
  auto unit_int = [&](int u, int i) -> int32_t& { return p.units[static_cast<long long>(u) * kChunkUnitInts + i]; };
  long long cost = 0;
  for (int u0 = 0; u0 < units; u0 += kPlanThreads) {
    const int u = u0 + tid;
    int mine = 0;
    if (u < units) {
      const int tiles = tiles_of(unit_int(u, 4));
      mine = tiles > 0 ? tiles * tile_cost(unit_int(u, kPages0), v) + kFixedCost : 0;
      out.cost[u] = mine;
    }
    long long all;
    block_scan(static_cast<long long>(mine), s_warp64, &all);
    cost += all;
  }
  __syncthreads();
  // whole units: thread i for pair i
  const long long share = (cost + p.parts - 1) / p.parts;
  long long room = 0;
  if (tid < p.parts) {
    room = share;
    constexpr int kAhead = 8;  // costs in flight: the loop is their latency
    for (int u0 = tid; u0 < units; u0 += kAhead * p.parts) {
      int c[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) c[k] = u0 + k * p.parts < units ? out.cost[u0 + k * p.parts] : 0;
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (c[k] > 0 && c[k] <= room) {
          room -= c[k];
          out.cost[u0 + k * p.parts] = 0;
          unit_int(u0 + k * p.parts, kSchedule + 2 * v + 1) = 1 + kWhole;
        }
    }
  }
  __syncthreads();
  // the others, one after another, with the sum of the costs before each
  int rest = 0;
  long long sum = 0;
  for (int u0 = 0; u0 < units; u0 += kPlanThreads) {
    const int u = u0 + tid;
    const long long mine = u < units ? out.cost[u] : 0;
    int all;
    long long all_cost;
    const int at = block_scan(mine > 0 ? 1 : 0, s_warp, &all);
    const long long before = block_scan(mine, s_warp64, &all_cost);
    if (mine > 0) {
      out.rest[rest + at] = u;
      out.prefix[rest + at] = sum + before;
    }
    rest += all;
    sum += all_cost;
  }
  __syncthreads();
  {
    long long all;
    const long long x = block_scan(room, s_warp64, &all);
    if (tid < p.parts) {
      int e = rest, t = 0;
      if (x < sum) {
        int lo = 0, hi = rest;  // the last entry that begins at or before x
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (out.prefix[mid] <= x)
            lo = mid;
          else
            hi = mid;
        }
        e = lo;
        const int u = out.rest[e], tiles = tiles_of(unit_int(u, 4)), per = tile_cost(unit_int(u, kPages0), v);
        t = static_cast<int>(min(max(x - out.prefix[e] - kFixedCost, 0ll) / per, static_cast<long long>(tiles)));
        if (t == tiles) {
          ++e;
          t = 0;
        }
      }
      cut_u[tid] = e;
      cut_t[tid] = t;
    }
    if (tid == 0) {
      cut_u[p.parts] = rest;
      cut_t[p.parts] = 0;
    }
  }
  __syncthreads();
  // Cuts inside a unit, each counted once; the first of a unit opens its slots.
  const bool in = tid < p.parts;
  const bool inside = in && cut_t[tid] > 0 && (tid == 0 || cut_u[tid] != cut_u[tid - 1] || cut_t[tid] != cut_t[tid - 1]);
  const bool opens = inside && (tid == 0 || cut_u[tid] != cut_u[tid - 1] || cut_t[tid - 1] == 0);
  int all;
  const int at = block_scan((inside ? 1 : 0) + (opens ? 1 : 0), s_warp, &all);
  if (opens) {
    int cuts = 1;
    for (int i = tid + 1; i < p.parts && cut_u[i] == cut_u[tid]; ++i) cuts += cut_t[i] != cut_t[i - 1];
    const int u = out.rest[cut_u[tid]];
    unit_int(u, kSchedule + 2 * v) = at;
    unit_int(u, kSchedule + 2 * v + 1) = cuts + 1;
    out.fix[atomicAdd(&p.head[kHeadFix + v], 1)] = u;
  }
  if (in) {
    int piece = 0;
    if (cut_t[tid] > 0)
      for (int i = tid; i >= 0 && cut_u[i] == cut_u[tid] && cut_t[i] > 0; --i)
        piece += i == 0 || cut_u[i - 1] != cut_u[i] || cut_t[i - 1] != cut_t[i];
    int4* e = reinterpret_cast<int4*>(out.sched + tid * MLA_SCHED_INTS);
    e[0] = make_int4(cut_u[tid], cut_t[tid], cut_u[tid + 1], cut_t[tid + 1]);
    e[1] = make_int4(piece, 0, 0, 0);
  }
}

// The plan: units of all requests, in order, and both schedules, a block each (what
// they have in common both find and write alike).  Made once for a batch: 64 requests
// x up to 6 tokens x 128 heads 11 us, the latency of a few passes over the units.
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkPlanParams p) {
  __shared__ long long s_warp64[32];
  __shared__ int s_warp[32];
  __shared__ int broken;
  __shared__ int cut_u[kMaxChunkParts + 1], cut_t[kMaxChunkParts + 1];
  const int tid = threadIdx.x, v = blockIdx.x;
  if (tid == 0) broken = 0;
  __syncthreads();
  for (int b = tid; b < p.batch; b += kPlanThreads) {
    const int a = p.cu[b], e = p.cu[b + 1], n = p.lens[b];
    p.made[b] = a;
    if (b == p.batch - 1) p.made[p.batch] = e;
    p.made[p.batch + 1 + b] = n;
    if (a < 0 || e < a || e > p.total_q || n > kMaxChunkKeys) broken = 1;
  }
  __syncthreads();
  if (broken) {  // offsets out of order could make requests overlap: nothing is done then
    if (tid == 0) {
      report(p.status, MLA_ERR_BAD_INDEX);
      p.head[kHeadWhole] = 0;
      p.head[kHeadCausal] = p.causal;
      p.head[kHeadFix + v] = 0;
      p.head[kHeadBroken] = 1;
    }
    for (int b = tid; b <= p.batch; b += kPlanThreads) p.conv[b] = 0;
    for (int i = tid; i < p.parts * MLA_SCHED_INTS; i += kPlanThreads) p.schedule[v].sched[i] = 0;
    return;
  }
  // first unit of each request, and its first page among those of requests that are
  // converted as a whole
  int units = 0;
  long long pages = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < p.batch) n = ((p.cu[b + 1] - p.cu[b]) * p.h_q + kRowsPerBlock - 1) / kRowsPerBlock;
    int all;
    const int at = block_scan(n, s_warp, &all);
    long long all_pages;
    const long long page = block_scan(n >= kConvertUnits ? static_cast<long long>(pages_of(max(p.lens[b], 0))) : 0ll,
                                      s_warp64, &all_pages);
    if (b < p.batch) {
      p.first[b] = units + at;
      p.conv[b] = static_cast<int>(min(pages + page, static_cast<long long>(INT32_MAX)));
    }
    units += all;
    pages += all_pages;
  }
  if (tid == 0) p.conv[p.batch] = static_cast<int>(min(pages, static_cast<long long>(INT32_MAX)));
  if (tid == 0) {
    p.head[kHeadWhole] = units;
    p.head[kHeadCausal] = p.causal;
    p.head[kHeadFix + v] = 0;
    p.head[kHeadBroken] = 0;
  }
  __syncthreads();
  for (int u = tid; u < units; u += kPlanThreads) {
    int lo = 0, hi = p.batch;  // first[lo] <= u: the last such request (those before it with none have the same first)
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (p.first[mid] <= u)
        lo = mid;
      else
        hi = mid;
    }
    const int tok0 = p.cu[lo], n = p.cu[lo + 1] - tok0, keys = max(p.lens[lo], 0);
    const int rel = (u - p.first[lo]) * kRowsPerBlock, rows = min(n * p.h_q - rel, kRowsPerBlock);
    const int limit0 = keys - n + 1;
    const int len = p.causal ? max(limit0 + (rel + rows - 1) / p.h_q, 0) : keys;
    int4* e = reinterpret_cast<int4*>(p.units + static_cast<long long>(u) * kChunkUnitInts);
    e[0] = make_int4(tok0 * p.h_q + rel, rows, rel, lo);
    e[1] = make_int4(len, limit0, p.conv[lo + 1] > p.conv[lo] ? p.conv[lo] : -1, 0);
    reinterpret_cast<int2*>(e + 2)[v] = make_int2(0, len > 0 ? 1 : 0);
    if (len == 0) p.schedule[v].fix[atomicAdd(&p.head[kHeadFix + v], 1)] = u;  // (in any order: no result depends on it)
  }
  __syncthreads();
  plan_schedule(p, v, units, cut_u, cut_t, s_warp, s_warp64);
}
static_assert(kMaxChunkParts <= kPlanThreads, "a thread a cut");

}  // namespace ck

ChunkPlanLayout chunk_plan_layout(int batch, int total_q, int h_q, int parts) {
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  ChunkPlanLayout z;
  z.max_units = static_cast<int>(static_cast<long long>(total_q) * h_q / kRowsPerBlock) + batch;
  const size_t units = static_cast<size_t>(z.max_units);
  z.units = 256;
  size_t at = z.units + up(units * kChunkUnitInts * 4);
  for (auto& c : z.schedule) {
    c.sched = at;
    c.fix = c.sched + up(static_cast<size_t>(parts) * MLA_SCHED_INTS * 4);
    c.rest = c.fix + up(units * 4);
    c.cost = c.rest + up(units * 4);
    c.prefix = c.cost + up(units * 4);
    at = c.prefix + up(units * 8);
  }
  z.first = at;
  z.conv = z.first + up(static_cast<size_t>(batch) * 4);
  z.made = z.conv + up((static_cast<size_t>(batch) + 1) * 4);
  z.bytes = z.made + up((2 * static_cast<size_t>(batch) + 1) * 4);
  return z;
}

cudaError_t launch_chunk_plan(const ChunkPlanParams& p, cudaStream_t st) {
  ck::chunk_plan_kernel<<<2, ck::kPlanThreads, 0, st>>>(p);
  return cudaGetLastError();
}

namespace {

using ChunkKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, ChunkParams);
ChunkKernel chunk_kernel_of(bool half, bool fp8, bool stall) {
  if (fp8) return stall ? ck::chunk_kernel<false, true, true> : ck::chunk_kernel<false, true>;
  return stall ? ck::chunk_kernel<false, false, true> : half ? ck::chunk_kernel<true, false> : ck::chunk_kernel<false, false>;
}

}  // namespace

cudaError_t chunk_setup() {
  for (int v = 0; v < 5; ++v) {
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(chunk_kernel_of(v == 4, v & 1, v == 2 || v == 3)),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, ck::kSmemBytes);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// A launch that may begin while the kernel before ends: each kernel waits for that
// one (griddepcontrol.wait) before it reads or writes memory.
template <typename... Params, typename... Args>
static cudaError_t launch_early(void (*kernel)(Params...), int blocks, int threads, size_t smem, cudaStream_t st,
                                const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_chunk(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& rope,
                         const ChunkParams& p, bool half, bool stall, int parts, cudaStream_t st) {
  const bool fp8 = p.records != nullptr;
  return launch_early(chunk_kernel_of(half, fp8, stall), 2 * parts, ck::threads_of(fp8), ck::kSmemBytes, st, q, k, v,
                      rope, p);
}

cudaError_t launch_chunk_convert(const ChunkParams& p, const uint16_t* q, uint16_t* pages, int sms, cudaStream_t st) {
  const long long blocks = std::max((p.rows + 7) / 8, static_cast<long long>(p.room));
  return launch_early(ck::chunk_convert_kernel, static_cast<int>(std::min(blocks, 8ll * sms)), 256, 0, st, p, q, pages);
}

cudaError_t launch_chunk_combine(const ChunkParams& p, int parts, int sms, cudaStream_t st) {
  return launch_early(ck::chunk_combine_kernel, std::min(parts * (kRowsPerBlock / 4), 16 * sms), 128, 0, st, p);
}

}  // namespace mla
