// Attention over whole prompts, packed one after another, causal or not, with
// grouped heads: q, k of 192 (or 128) dims, v of 128.
//
//   s_ij = scale q_i . k_j,  out_i = sum_j e^(s_ij - r_i) v_j / l_i,
//   l_i = sum_j e^(s_ij - r_i),  lse_i = r_i + ln l_i,  j <= i + Lk - Lq
//
// A worker takes (query head, query tile) items from the plan's list, longest
// first.  A tile has two halves, each with its own scores, softmax warps and
// accumulator, that take turns on the tensor cores: one half's exponentials
// run while the other half's products do.  128 keys at a time:
//   * TMEM (512 columns): scores of both halves (2 x 128), outputs (2 x 128).
//     A half's weights P overwrite its scores as packed 16-bit pairs and are the
//     A operand of P V from there, so P never touches shared memory.
//   * Shared memory: Q of both halves, and a ring of K and of V stages.
//   * One warp issues every MMA in the order
//       PV0(j-1) QK0(j)  PV1(j-1) QK1(j)
//     The tensor pipe runs them in order, so S(j) being ready means PV(j-1) of
//     that half is done: its P may be overwritten, and its O rescaled, without a
//     wait of their own.  Two barriers a half remain: scores ready, weights ready.
//     The same order lets the next item's first products follow the last ones of
//     this item while its output is still being written.
//   * The softmax reference r is raised only when a row's maximum grows by more
//     than 2^8 (then O is rescaled in TMEM, rarely); weights stay below 2^8, so
//     sums stay far from overflow.  Statistics are fp32; P is rounded to the
//     inputs' type, which is what the tensor cores take and keeps each weight
//     within half a step of it.
//   * Keys past the sequence's end in its last tile belong to another sequence
//     (or to nothing): their scores are masked and their V rows are zeroed in
//     shared memory, since 0 x NaN would not be 0.
//   * A softmax warp has 32 rows and 64 of the 128 keys, so that the chain from
//     scores to weights is half as long; the two warps of a row exchange their
//     maxima through one word each.
// A worker is a pair of CTAs for long prompts (kPair): cta_group::2 MMAs over
// 256 rows a half, 128 in each CTA, with K and V split between the two shared
// memories (K by keys, V by dims).  One CTA alone has room for 1.6 key tiles
// beside its 96 KB of Q, too few to cover the latency of the loads; half a tile
// each gives the pair three.  Shorter prompts would leave half a pair idle: those
// run on single CTAs with two 128-row halves (see prompt_pairs).
//
// Bound: the tensor pipe.  128 x 128 x (192 + 128) multiply-adds a half and key
// tile are 1280 cycles at 4096 a cycle, 2560 a step of both halves, 1.24 us at
// 2.06 GHz.  Measured (bf16, 192 dims): 1.52 us a step where all pairs have one
// item (1.98 PFLOP/s), 688 us for a causal prompt of 16384 tokens x 16 heads (2.0
// PFLOP/s; 780 us back to back, under the power limit), 102 us for 8192 x 8,
// 168 us for 32 prompts of 1024 x 16 (their 670 MB are 100 us of HBM).  An item's
// change costs about 1.3 us a worker.
// Steps that made it (16384 x 16): one thread issuing MMAs from divergent code
// 1137 us, a converged warp 953 (an MMA's operand moves cost a lone thread 110
// cycles), pairs 912, weights announced by relaxed cluster arrivals 779 (a release
// waits for earlier stores to reach the cluster: 1700 cycles), stores exchanged
// among lanes 770, the roles' dispatch made warp-uniform 688.  (Ragged batches: deal.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "ptx.cuh"
#include "serving.cuh"

namespace mla {
namespace pr {

constexpr int kBM = 128;              // query rows of a half in one CTA
constexpr int kBN = 128;              // keys of a tile
constexpr int kBoxBytes = 128 * 128;  // 128 rows x 64 16-bit values

// 16 softmax warps: two for each 32 rows of a half, 64 of the 128 keys each;
// then the MMA warp, and the warps that load K, V and Q.
constexpr int kThreads = 640;
constexpr int kWarpMma = 16, kWarpK = 17, kWarpV = 18, kWarpQ = 19;
constexpr int kMaxStages = 5;

enum : int {
  Q_FULL = 0,                     // +half
  Q_EMPTY = Q_FULL + 2,           // +half: the item's last Q K^T is done: Q may be loaded over
  K_FULL = Q_EMPTY + 2,           // +stage
  K_EMPTY = K_FULL + kMaxStages,  // +stage: its MMAs are done
  V_FULL = K_EMPTY + kMaxStages,
  V_EMPTY = V_FULL + kMaxStages,
  S_FULL = V_EMPTY + kMaxStages,  // +half: scores ready, and P V of the tile before done
  P_FULL = S_FULL + 2,            // +half: weights written (one arrival per softmax warp)
  O_FULL = P_FULL + 2,            // +half: the item's last P V is done
  TAIL = O_FULL + 2,              // the last V tile, before its rows past the end are zeroed
  DRAIN,                          // every MMA issued is done
  kNumBars
};

// Shared memory of one CTA: Q (2 halves x kQBoxes boxes), then K stages (the
// CTA's keys x kQBoxes 64-dim slices), then V stages (128 keys x the CTA's dims).
// Dealing out the last kRanked rounds of items (deal); in Q's place before the
// first loads.
constexpr int kRanked = 3;
constexpr int kMaxWorkers = 80;
constexpr int kLongTiles = 12;  // key tiles of an item of 20 us
struct Deal {
  uint32_t keys[2][kMaxWorkers];
  uint32_t times[kRanked][kMaxWorkers];
  uint8_t dealt[kRanked];
};
static_assert(kRanked == 3 && kMaxWorkers <= 255, "three bytes of a word");

template <int kQBoxes, bool kPair>
struct Layout {
  static constexpr int kHalfRows = kPair ? 256 : 128;          // query rows of a half
  static constexpr int kKeys = kPair ? 64 : 128;               // keys of a tile in this CTA's K stage
  static constexpr int kVBoxes = kPair ? 1 : 2;                // 64-dim boxes of its V stage
  static constexpr int kKBoxBytes = kKeys * 128;
  static constexpr int kKBytes = kQBoxes * kKBoxBytes;
  static constexpr int kVBytes = kVBoxes * kBoxBytes;
  static constexpr int kKStages = kPair ? (kQBoxes == 3 ? 3 : 5) : (kQBoxes == 3 ? 2 : 3);
  static constexpr int kVStages = kPair ? (kQBoxes == 3 ? 3 : 5) : (kQBoxes == 3 ? 1 : 2);
  static constexpr int kOffK = 2 * kQBoxes * kBoxBytes;
  static constexpr int kOffV = kOffK + kKStages * kKBytes;
  static constexpr int kOffBar = kOffV + kVStages * kVBytes;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffRow = kOffMisc + 16;                // one float per half, key half and row
  static constexpr int kBytes = kOffRow + 2 * 2 * kBM * 4;
  static_assert(kBytes <= 232448, "shared memory budget");
  static_assert(kKStages <= kMaxStages && kVStages <= kMaxStages, "barriers");
};

constexpr uint32_t kTmemCols = 512;
constexpr float kTau = 8.0f;
constexpr float kLn2 = 0.69314718055994530942f;

// Plan: a header {tiles, causal, deal by sums}, then the tiles, kTileInts int32
// each, then the offsets it was made for: batch + 1 of the queries, as many of
// the keys.
struct Tile {
  int q0;    // first query row of the tile in the packed q
  int rows;  // queries of the sequence from q0 on (the first two halves' worth matter)
  int k0;    // first key row of the sequence
  int lk;    // keys of the sequence
  int vis;   // keys that the tile's first query sees
};
constexpr int kTileInts = 8;

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

// 128-key tiles that half h of a tile has to visit: keys its last valid row
// sees, at most the sequence's; 0 for a half without rows.
__device__ __forceinline__ int half_tiles(const Tile& t, int h, int half_rows, int causal) {
  const int rows = min(t.rows - h * half_rows, half_rows);
  if (rows <= 0) return 0;
  const int keys = causal ? min(t.lk, t.vis + h * half_rows + rows - 1) : t.lk;
  return keys > 0 ? (keys + kBN - 1) / kBN : 0;
}

// The items of one worker, the same in every role.  An item is one tile of the
// plan and one query head, all heads of a tile in a row in the list.  In round r
// a worker gets one of the list's numbers r * workers .. (r + 1) * workers - 1:
// counted backwards in every other round, and in the last rounds the longest of
// them goes to the worker whose sum is smallest (deal).  It runs them 32 rounds
// at a time in the order of their heads: the workers then read the keys of few
// heads at a time, which stay in L2.  (In the list's order a ragged batch read
// its keys 2.3 times from HBM.)
struct Items {
  int at, total;    // the current item's number; `total`: no more
  int base;         // first of the 32 rounds
  uint32_t key;     // head and round of the current one, + 1
  int ranked;       // first round whose place is a byte of `dealt`
  uint32_t dealt;
};

__device__ __forceinline__ int place_in_round(int round, int worker, int workers) {
  return (round & 1) ? workers - 1 - worker : worker;
}

__device__ __forceinline__ int item_of_round(const Items& it, int round, int worker, int workers) {
  const int k = round - it.ranked;
  const int place = k < 0 ? place_in_round(round, worker, workers) : static_cast<int>(it.dealt >> (8 * k & 31) & 255u);
  return round * workers + place;
}

// By a whole warp: lane i looks at round base + i.
__device__ __forceinline__ void next_item(Items& it, int worker, int workers, int heads) {
  const int lane = threadIdx.x & 31;
  while (true) {
    const int at = item_of_round(it, it.base + lane, worker, workers);
    const uint32_t key = (static_cast<uint32_t>(at % heads) << 5 | static_cast<uint32_t>(lane)) + 1u;
    const uint32_t mine = at < it.total && key > it.key ? key : ~0u;
    if (__any_sync(0xffffffffu, mine != ~0u)) {
      it.key = __shfl_sync(0xffffffffu, __reduce_min_sync(0xffffffffu, mine), 0);
      it.at = item_of_round(it, it.base + static_cast<int>((it.key - 1u) & 31u), worker, workers);
      return;
    }
    it.base += 32;
    it.key = 0;
    if (it.base * workers >= it.total) {
      it.at = it.total;
      return;
    }
  }
}

__device__ __forceinline__ Tile load_tile(const PromptParams& p, const Items& it) {
  if (it.at >= it.total) return Tile{0, 0, 0, 0, 0};
  const int4* e = reinterpret_cast<const int4*>(p.plan + kTileInts * (it.at / p.h_q + 1));
  const int4 a = e[0];
  return Tile{a.x, a.y, a.z, a.w, e[1].x};
}

// Time of an item in tenths of a microsecond, near enough to compare sums:
// steps of both halves, of one, and the change of items.
__device__ __forceinline__ uint32_t item_time(const int32_t* plan, int heads, int at, int total, int half_rows,
                                              int causal) {
  if (at >= total) return 0;
  const int4* e = reinterpret_cast<const int4*>(plan + kTileInts * (at / heads + 1));
  const int4 a = e[0];
  const Tile t{a.x, a.y, a.z, a.w, e[1].x};
  const int n0 = half_tiles(t, 0, half_rows, causal), n1 = half_tiles(t, 1, half_rows, causal);
  return 15u * min(n0, n1) + 12u * abs(n0 - n1) + 13u;
}

// The worker's places in the last kRanked of at least as many rounds, a byte
// each, worked out by every CTA alike (kG threads keep a worker's sum): within a
// round the list descends, so the rank among the sums, smallest first, is the
// place to take.  Going back and forth alone leaves the longest worker 2 to 12%
// over the mean for ragged batches, this 1 to 4%, and it takes 2 to 3 us: 8 ragged
// prompts up to 4000 tokens x 16 heads 242 -> 233 us, 8 others 128.5 -> 125, 3 x 128
// heads 247 -> 242; but 32 of 1024 tokens 169 -> 172, 16 ragged ones up to 700 39 ->
// 41.  So the plan asks for it where lengths differ and an item takes 20 us, and
// pairs of CTAs alone do it (152 single workers rank in 6 us).  By all threads of
// the CTA; a call, so that its registers cost the roles none.
template <int kG>
__device__ __noinline__ uint32_t deal(const int32_t* plan, int heads, int total, int rounds, int worker, int workers,
                                      int half_rows, int causal, Deal* s) {
  constexpr uint32_t kMost = (1u << 23) - 1;  // sums beyond 0.8 s count as equal
  const int w = threadIdx.x / kG, sub = threadIdx.x % kG, from = rounds - kRanked;
  const bool mine = w < workers;
  uint32_t sum = 0;
  if (mine) {
    for (int k = sub; k < kRanked; k += kG)
      s->times[k][w] = item_time(plan, heads, (from + k) * workers + w, total, half_rows, causal);
#pragma unroll 2
    for (int r = sub; r < from; r += kG)
      sum = min(sum + item_time(plan, heads, r * workers + place_in_round(r, w, workers), total, half_rows, causal),
                kMost);
  }
#pragma unroll
  for (int o = 1; o < kG; o <<= 1) sum = min(sum + __shfl_xor_sync(0xffffffffu, sum, o), kMost);
  for (int k = 0; k < kRanked; ++k) {
    const uint32_t key = sum << 8 | static_cast<uint32_t>(w);
    if (sub == 0) s->keys[k & 1][w] = mine ? key : ~0u;
    __syncthreads();
    int place = 0;
#pragma unroll 10
    for (int i = sub; i < kThreads / kG; i += kG) place += s->keys[k & 1][i] < key;
#pragma unroll
    for (int o = 1; o < kG; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
    if (mine) {
      sum = min(sum + s->times[k][place], kMost);
      if (w == worker && sub == 0) s->dealt[k] = static_cast<uint8_t>(place);
    }
  }
  __syncthreads();
  const uint32_t dealt = s->dealt[0] | s->dealt[1] << 8 | s->dealt[2] << 16;
  fence_proxy_async_smem();  // the loads may write there next
  __syncthreads();
  return dealt;
}

// Whether the plan is that of the caller's offsets, by warps that have loaded
// their last tile; the call's results are those of the plan either way.
__device__ __forceinline__ void check_plan(const PromptParams& p) {
  if (p.cu_q == nullptr) return;
  const int32_t* made = p.plan + kTileInts * (p.max_tiles + 1);
  for (int i = blockIdx.x * 32 + (threadIdx.x & 31); i <= p.batch; i += gridDim.x * 32)
    if (made[i] != p.cu_q[i] || made[p.batch + 1 + i] != p.cu_k[i]) report(p.status, MLA_ERR_STALE_PLAN);
}

__device__ __forceinline__ void fail(volatile int* abort_flag, int32_t* status) {
  *abort_flag = 1;
  report(status, MLA_ERR_TIMEOUT);
}

// Wait budget of the stall-test instances (kStall), whose first K stage is never
// loaded; the others keep the 2 s budget of every wait.
constexpr uint64_t kStallWaitNs = 200000;  // 200 us

template <bool kHalf, int kQBoxes, bool kPair, bool kStall = false>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, const PromptParams p) {
  using L = Layout<kQBoxes, kPair>;
  constexpr uint64_t kWaitNs = kStall ? kStallWaitNs : MLA_WAIT_LIMIT_NS;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const int worker = kPair ? blockIdx.x >> 1 : blockIdx.x;
  const int workers = kPair ? gridDim.x >> 1 : gridDim.x;

  extern __shared__ __align__(1024) uint8_t smem[];  // swizzle atoms need 1024-byte alignment
  uint8_t* sQ = smem;
  uint8_t* sK = smem + L::kOffK;
  uint8_t* sV = smem + L::kOffV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  float* sRow = reinterpret_cast<float*>(smem + L::kOffRow);

  const int tid = threadIdx.x;
  // The warp's number by a shuffle: the compiler then knows that a warp takes one
  // role, keeps that role's code convergent and its MMA operands in uniform
  // registers (16384-token prompt: 771 us without, 704 with).
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if ((smem_u32(smem) & 1023u) != 0u) {  // not what was asked for (all CTAs alike)
    if (tid == 0) report(p.status, MLA_ERR_UNSUPPORTED);
    return;
  }
  if (tid == 0) {
    *abort_flag = 0;
    constexpr uint32_t kCtas = kPair ? 2 : 1;  // loaders that fill a stage, each its part
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&bars[K_FULL + i], kCtas);
      mbar_init(&bars[K_EMPTY + i], 1);
      mbar_init(&bars[V_FULL + i], kCtas);
      mbar_init(&bars[V_EMPTY + i], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&bars[Q_FULL + h], kCtas);
      mbar_init(&bars[Q_EMPTY + h], 1);
      mbar_init(&bars[S_FULL + h], 1);
      mbar_init(&bars[P_FULL + h], 8 * kCtas);
      mbar_init(&bars[O_FULL + h], 1);
    }
    mbar_init(&bars[TAIL], 1);
    mbar_init(&bars[DRAIN], 1);
    fence_mbar_init_cluster();
  }
  if (warp == kWarpMma) {
    if constexpr (kPair) {
      tmem2_alloc(tmem_slot, kTmemCols);
      tmem2_relinquish();
    } else {
      tmem_alloc(tmem_slot, kTmemCols);
      tmem_relinquish();
    }
  }
  if (warp == kWarpK && lane == 0) {
    prefetch_tmap(&q_map);
    prefetch_tmap(&k_map);
    prefetch_tmap(&v_map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (kPair) {  // the other CTA's barriers are ready before anything arrives there
    cluster_arrive();
    cluster_wait();
  }
  const uint32_t tmem = *tmem_slot;
  const int causal = p.plan[1];
  Items it{0, p.plan[0] * p.h_q, 0, 0, 1 << 30, 0};
  if constexpr (kPair) {
    const int rounds = (it.total + workers - 1) / workers;
    if (p.plan[2] && rounds >= kRanked) {  // (two rounds back and forth are the same)
      it.dealt = deal<kThreads / kMaxWorkers>(p.plan, p.h_q, it.total, rounds, worker, workers, L::kHalfRows, causal,
                                              reinterpret_cast<Deal*>(sQ));
      it.ranked = rounds - kRanked;
    }
  }
  next_item(it, worker, workers, p.h_q);

  if (warp > kWarpMma) {
    // ------------------------------------------------------------ loads: K, V or Q
    bool ok = true;
    uint32_t n_loaded = 0, q0n = 0, q1n = 0, tails = 0;  // stages, Q halves and tail tiles loaded so far
    const uint64_t pol_q = policy_evict_first(), pol_kv = policy_evict_last();
    // The barriers that count loads are the even CTA's: its MMA warp waits for
    // both CTAs' parts there.
    const uint32_t bar0 = kPair ? mapa_shared(smem_u32(bars), 0) : smem_u32(bars);
    auto expect = [&](int bar, uint32_t bytes) {
      if constexpr (kPair)
        mbar_arrive_expect_tx_remote_relaxed(bar0 + 8 * bar, bytes);
      else
        mbar_arrive_expect_tx(&bars[bar], bytes);
    };
    // rows from `row` on of slices from `slice` on of one head
    auto load = [&](uint8_t* dst, const CUtensorMap* map, int bar, int row, int slice, int hd, uint64_t pol) {
      if constexpr (kPair)
        tma_load_4d_pair(dst, map, bar0 + 8 * bar, 0, row, slice, hd, pol);
      else
        tma_load_4d(dst, map, &bars[bar], 0, row, slice, hd, pol);
    };
    for (; it.at < it.total && ok; next_item(it, worker, workers, p.h_q)) {
      const Tile t = load_tile(p, it);
      const int head = it.at % p.h_q, kvh = head / p.group;
      const int n0 = half_tiles(t, 0, L::kHalfRows, causal), n1 = half_tiles(t, 1, L::kHalfRows, causal);
      const int n = max(n0, n1);
      if (warp == kWarpQ) {
        // a half's rows as soon as its last Q K^T of the item before is done
        // (rows past the sequence's last query come along and are not stored)
        if (lane == 0)
          for (int h = 0; h < 2 && ok; ++h) {
            if ((h ? n1 : n0) == 0) continue;
            const uint32_t before = h ? q1n++ : q0n++;
            if (before >= 1) ok = mbar_wait(&bars[Q_EMPTY + h], (before - 1) & 1, abort_flag, kWaitNs);
            if (!ok) break;
            expect(Q_FULL + h, kQBoxes * kBoxBytes);
            load(sQ + h * kQBoxes * kBoxBytes, &q_map, Q_FULL + h,
                 t.q0 + h * L::kHalfRows + static_cast<int>(rank) * kBM, 0, head, pol_q);
          }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      } else if (warp == kWarpK) {
        if (lane == 0)
          for (int j = 0; j < n && ok; ++j, ++n_loaded) {
            const int s = static_cast<int>(n_loaded % L::kKStages), r = static_cast<int>(n_loaded / L::kKStages);
            if (r >= 1) ok = mbar_wait(&bars[K_EMPTY + s], (r - 1) & 1, abort_flag, kWaitNs);
            if (ok && !(kStall && rank == 0 && n_loaded == 0)) {
              expect(K_FULL + s, L::kKBytes);
              load(sK + s * L::kKBytes, &k_map, K_FULL + s, t.k0 + j * kBN + static_cast<int>(rank) * L::kKeys, 0, kvh,
                   pol_kv);
            }
          }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      } else {
        for (int j = 0; j < n && ok; ++j, ++n_loaded) {
          const bool tail = (j + 1) * kBN > t.lk;  // the sequence ends inside this tile
          const int s = static_cast<int>(n_loaded % L::kVStages), r = static_cast<int>(n_loaded / L::kVStages);
          uint8_t* dst = sV + s * L::kVBytes;
          if (lane == 0) {
            if (r >= 1) ok = mbar_wait(&bars[V_EMPTY + s], (r - 1) & 1, abort_flag, kWaitNs);
            if (ok && tail) {  // onto this CTA's own barrier
              mbar_arrive_expect_tx(&bars[TAIL], L::kVBytes);
              tma_load_4d(dst, &v_map, &bars[TAIL], 0, t.k0 + j * kBN, kPair ? static_cast<int>(rank) : 0, kvh, pol_kv);
            } else if (ok) {
              expect(V_FULL + s, L::kVBytes);
              load(dst, &v_map, V_FULL + s, t.k0 + j * kBN, kPair ? static_cast<int>(rank) : 0, kvh, pol_kv);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok || !tail) continue;
          ok = __all_sync(0xffffffffu, mbar_wait(&bars[TAIL], tails & 1, abort_flag, kWaitNs));
          ++tails;
          if (!ok) continue;
          const int keep = t.lk - j * kBN;  // rows of this tile that are the sequence's
          for (int b = 0; b < L::kVBoxes; ++b) {
            uint4* z = reinterpret_cast<uint4*>(dst + b * kBoxBytes + keep * 128);
            for (int i = lane; i < (kBN - keep) * 8; i += 32) z[i] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if constexpr (kPair)
              mbar_arrive_remote(bar0 + 8 * (V_FULL + s));
            else
              mbar_arrive(&bars[V_FULL + s]);
          }
        }
      }
    }
    if (warp == kWarpV) check_plan(p);
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
    // The even CTA's warp issues for the pair.  The whole warp runs this loop
    // (see umma_f16_warp); its control flow and operands are the same in all lanes.
    if (rank == 0) {
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      constexpr uint32_t kM = kPair ? 256 : 128;
      constexpr uint32_t idesc_qk = idesc_16bit_f32(kM, kBN, false, kHalf);
      constexpr uint32_t idesc_pv = idesc_16bit_f32(kM, 128, true, kHalf);
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(sV), kBoxBytes, 1024);  // MN-major
      auto wait = [&](int bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(&bars[bar], parity, abort_flag, kWaitNs));
      };
      // a stage of V may hold rows that threads of the other CTA zeroed
      auto wait_v = [&](int bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait<kPair>(&bars[bar], parity, abort_flag, kWaitNs));
      };
      auto commit = [&](int bar) {
        if constexpr (kPair)
          umma2_commit_warp(&bars[bar]);
        else
          umma_commit_warp(&bars[bar]);
      };
      // One step a key tile, through all items: P V of the tile before, then
      // Q K^T of this one, half by half.  At an item's end the tile before is
      // its last one and this one the next item's first.
      bool ok = true;
      uint32_t kn = 0, vn = 0, q0n = 0, q1n = 0, tiles0 = 0, tiles1 = 0;  // stages, Q halves, tiles of each half so far
      int n0 = 0, n1 = 0, j = 0;        // this item's key tiles, and this one
      int pn0 = 0, pn1 = 0, pj = 0;     // the same of the tile before
      Tile next = load_tile(p, it);
      // on to the next item with keys; n0 = n1 = 0 past the last one
      auto enter = [&]() {
        n0 = n1 = j = 0;
        while (it.at < it.total && max(n0, n1) == 0) {
          n0 = __shfl_sync(0xffffffffu, half_tiles(next, 0, L::kHalfRows, causal), 0);
          n1 = __shfl_sync(0xffffffffu, half_tiles(next, 1, L::kHalfRows, causal), 0);
          next_item(it, worker, workers, p.h_q);
          next = load_tile(p, it);  // not needed before this item's end
        }
      };
      enter();
      while (ok && (max(n0, n1) > 0 || max(pn0, pn1) > 0)) {
        bool have_v = false, have_k = false;
        const int ks = static_cast<int>(kn % L::kKStages);
        const int vs = static_cast<int>(vn % L::kVStages);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int nh = h ? n1 : n0, pnh = h ? pn1 : pn0;
          const uint32_t s_col = tm + 128u * h, o_col = tm + 256u + 128u * h;
          if (ok && pj < pnh) {
            if (!have_v) ok = wait_v(V_FULL + vs, (vn / L::kVStages) & 1);
            have_v = true;
            if (ok) ok = wait(P_FULL + h, ((h ? tiles1 : tiles0) - 1) & 1);
            if (ok) {
              tc_fence_after();
              const uint64_t vd = v_desc + static_cast<uint64_t>((vs * L::kVBytes) >> 4);
#pragma unroll
              for (int kk = 0; kk < kBN / 16; ++kk) {
                const uint32_t acc = (pj == 0 && kk == 0) ? 0u : 1u;
                if constexpr (kPair)
                  umma2_f16_ts_warp(o_col, s_col + 8u * kk, vd + static_cast<uint64_t>((kk * 2048) >> 4), idesc_pv, acc);
                else
                  umma_f16_ts_warp(o_col, s_col + 8u * kk, vd + static_cast<uint64_t>((kk * 2048) >> 4), idesc_pv, acc);
              }
              if (pj == pnh - 1) commit(O_FULL + h);
              if (h == 1 || pj >= pn1) commit(V_EMPTY + vs);  // read for the last time
            }
          }
          if (ok && j < nh) {
            if (j == 0) ok = wait(Q_FULL + h, (h ? q1n++ : q0n++) & 1);
            if (ok && !have_k) ok = wait(K_FULL + ks, (kn / L::kKStages) & 1);
            have_k = true;
            if (ok) {
              tc_fence_after();
              const uint64_t kd0 = k_desc + static_cast<uint64_t>((ks * L::kKBytes) >> 4);
#pragma unroll
              for (int s = 0; s < kQBoxes; ++s) {
                const uint64_t kd = kd0 + static_cast<uint64_t>((s * L::kKBoxBytes) >> 4);
                const uint64_t qd = q_desc + static_cast<uint64_t>(((h * kQBoxes + s) * kBoxBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  const uint32_t acc = (s == 0 && kk == 0) ? 0u : 1u;
                  if constexpr (kPair)
                    umma2_f16_warp(s_col, qd + static_cast<uint64_t>((kk * 32) >> 4),
                                   kd + static_cast<uint64_t>((kk * 32) >> 4), idesc_qk, acc);
                  else
                    umma_f16_warp(s_col, qd + static_cast<uint64_t>((kk * 32) >> 4),
                                  kd + static_cast<uint64_t>((kk * 32) >> 4), idesc_qk, acc);
                }
              }
              commit(S_FULL + h);
              if (h)
                ++tiles1;
              else
                ++tiles0;
              if (j == nh - 1) commit(Q_EMPTY + h);
              if (h == 1 || j >= n1) commit(K_EMPTY + ks);
            }
          }
        }
        if (max(pn0, pn1) > 0) ++vn;
        pn0 = n0;
        pn1 = n1;
        pj = j;
        if (max(n0, n1) > 0) {
          ++kn;
          if (++j == max(n0, n1)) enter();
        }
      }
      if (!ok && lane == 0) fail(abort_flag, p.status);
      // every MMA is done with shared memory and TMEM before this CTA ends
      commit(DRAIN);
      mbar_wait(&bars[DRAIN], 0, nullptr, kWaitNs);
    }
    __syncwarp();
  } else if (warp < kWarpMma) {
    // ------------------------------------------------------------ softmax + epilogue
    const int h = warp >> 3, part = (warp >> 2) & 1;  // half, and which 64 of the 128 keys (and output dims)
    const int r = tid & 127;                          // row of the half in this CTA == TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_addr = tmem + lane_base + 128u * h + 64u * part;
    const uint32_t p_addr = tmem + lane_base + 128u * h + 32u * part;
    const uint32_t o_addr = tmem + lane_base + 256u + 128u * h + 64u * part;
    const int row = h * L::kHalfRows + static_cast<int>(rank) * kBM + r;  // of a tile
    // the other warp of these 32 rows: one float each way, behind a barrier of the two
    float* mine = sRow + (2 * h + part) * kBM + r;
    const float* other = sRow + (2 * h + (part ^ 1)) * kBM + r;
    const uint32_t row_bar = 1 + 4 * h + (warp & 3);
    const uint32_t p_full = kPair ? mapa_shared(smem_u32(&bars[P_FULL + h]), 0) : smem_u32(&bars[P_FULL + h]);
    const float c_log2 = p.scale_log2;
    bool ok = true;
    uint32_t tiles = 0, items = 0;
    // key tiles of this half, and keys this row sees.  (All that the loop below
    // keeps of the tile: the rest is read again after it, which costs nothing
    // beside the wait for the last P V, and the registers do not go round.)
    int nh, limit;
    auto enter = [&](const Tile& t) {
      nh = half_tiles(t, h, L::kHalfRows, causal);
      limit = causal ? min(t.lk, t.vis + row) : t.lk;
    };
    enter(load_tile(p, it));
    while (it.at < it.total) {
      float ref = -INFINITY, l = 0.f;
      for (int j = 0; j < nh; ++j, ++tiles) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[S_FULL + h], tiles & 1, abort_flag, kWaitNs));
        tc_fence_after();
        float s[64];
        float m0, m1;
        tmem_ld32_max(s_addr, s, m0);
        tmem_ld32_max(s_addr + 32u, s + 32, m1);
        tmem_wait_ld();
        float top = fmaxf(m0, m1);
        const int seen = limit - j * kBN - 64 * part;
        if (__any_sync(0xffffffffu, seen < 64)) {
          // (bit tests of two masks: cheaper than a comparison an element)
          const uint32_t lo = seen >= 32 ? ~0u : (seen <= 0 ? 0u : (1u << seen) - 1u);
          const uint32_t hi = seen >= 64 ? ~0u : (seen <= 32 ? 0u : (1u << (seen - 32)) - 1u);
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (!((lo >> i) & 1u)) s[i] = -INFINITY;
            if (!((hi >> i) & 1u)) s[i + 32] = -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < 64; ++i) m4[i & 3] = fmaxf(m4[i & 3], s[i]);
          top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
        // the row's maximum over both warps.  (The other warp's word is read
        // before its next write: that needs S(j+1), which needs this warp's P.)
        *mine = top;
        // (a warp that gave up waiting takes the other one along)
        ok = !named_bar_or(row_bar, 64, !ok);
        if (!ok) break;
        const float mt = fmaxf(top, *other) * c_log2;
        const float r_new = mt > ref + kTau ? mt : ref;
        const float alpha = r_new == ref ? 1.f : ex2(ref - r_new);
        ref = r_new;
        const float mref = ref == -INFINITY ? 0.f : ref;
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 cl = make_float2(c_log2, c_log2), nr = make_float2(-mref, -mref);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 x = __ffma2_rn(make_float2(s[16 * c + 2 * i], s[16 * c + 2 * i + 1]), cl, nr);
            const float p0 = ex2(x.x), p1 = ex2(x.y);
            pk[i] = pack2<kHalf>(p0, p1);
            ls[i & 1] = __fadd2_rn(ls[i & 1], make_float2(p0, p1));
          }
          tmem_st8(p_addr + 8u * c, pk);
        }
        // P V of the tile before is done (see above): O may be rescaled here (after the
        // scores have been used up: fewer registers)
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (uint32_t c0 = 0; c0 < 64; c0 += 16) {
            uint32_t v[16];
            tmem_ld16(o_addr + c0, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
            tmem_st16(o_addr + c0, v);
          }
        }
        l = l * alpha + ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair)
            mbar_arrive_remote_relaxed(p_full);
          else
            mbar_arrive(&bars[P_FULL + h]);
        }
      }
      if (!ok) break;
      const Tile t = load_tile(p, it);
      const int head = it.at % p.h_q;
      next_item(it, worker, workers, p.h_q);
      const Tile t_next = load_tile(p, it);
      if (nh > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[O_FULL + h], items & 1, abort_flag, kWaitNs));
        ++items;
        tc_fence_after();
        // the row's sum over both warps, in an order that both share
        *mine = l;
        ok = !named_bar_or(row_bar, 64, !ok);
        if (!ok) break;
        const float l2 = *other;
        l = part == 0 ? l + l2 : l2 + l;
        named_bar_sync(row_bar, 64);  // read before the next item's first maximum is written
      }
      // 0 marks a row that sees no key: its output is 0 whatever the accumulator holds
      const float inv = limit > 0 ? 1.f / l : 0.f;
      // 16 rows at a time.  The load leaves a row's 64 values with four lanes, two
      // of every eight each; exchanged among the four, each holds whole 16-byte
      // pieces, and a store of the warp covers 64 bytes of 8 rows.  (With a row a
      // thread, every 16 bytes of a store went to a line of their own: the
      // stores took 14 us of 274 on a ragged batch, 29 of 157 on 512-token ones.)
      const int q4 = lane & 3;
      const size_t row_bytes = static_cast<size_t>(p.h_q) * 256;
      uint8_t* out0 = static_cast<uint8_t*>(p.out) + (static_cast<size_t>(t.q0) * p.h_q + head) * 256 + 128 * part;
#pragma unroll 1
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t v[32];
        tmem_ld_16x64(o_addr + (static_cast<uint32_t>(16 * hh) << 16), v);
        tmem_wait_ld();
#pragma unroll
        for (int up = 0; up < 2; ++up) {
          const int from = 16 * hh + 8 * up + (lane >> 2);  // lane that has this row's sum
          const float iv = __shfl_sync(0xffffffffu, inv, from);
          const int orow = row - lane + from;  // of the tile
          uint32_t w[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const float a = __uint_as_float(v[4 * n + 2 * up]) * iv, b = __uint_as_float(v[4 * n + 2 * up + 1]) * iv;
            w[n] = iv != 0.f ? pack2<kHalf>(a, b) : 0u;
          }
          // word n of lane q4 -> word q4 of lane n, within four lanes and four words
#pragma unroll
          for (int g = 0; g < 8; g += 4) {
            uint32_t* x = w + g;
            {
              const bool odd = q4 & 1;
              const uint32_t s0 = odd ? x[0] : x[1], s1 = odd ? x[2] : x[3];
              const uint32_t r0 = __shfl_xor_sync(0xffffffffu, s0, 1), r1 = __shfl_xor_sync(0xffffffffu, s1, 1);
              if (odd) {
                x[0] = r0;
                x[2] = r1;
              } else {
                x[1] = r0;
                x[3] = r1;
              }
            }
            {
              const bool odd = q4 & 2;
              const uint32_t s0 = odd ? x[0] : x[2], s1 = odd ? x[1] : x[3];
              const uint32_t r0 = __shfl_xor_sync(0xffffffffu, s0, 2), r1 = __shfl_xor_sync(0xffffffffu, s1, 2);
              if (odd) {
                x[0] = r0;
                x[1] = r1;
              } else {
                x[2] = r0;
                x[3] = r1;
              }
            }
            if (orow < t.rows)
              *reinterpret_cast<uint4*>(out0 + orow * row_bytes + 16 * (g + q4)) = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      }
      if (row < t.rows && part == 0)
        p.lse[static_cast<size_t>(t.q0 + row) * p.h_q + head] = limit > 0 ? (ref + __log2f(l)) * kLn2 : -INFINITY;
      // O has been read: the next item's first P V waits for this warp's P
      tc_fence_before();
      enter(t_next);
    }
    if (!ok && lane == 0) fail(abort_flag, p.status);
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) {  // the other CTA loads, arrives and multiplies here no more
    cluster_arrive();
    cluster_wait();
  }
  if (warp == kWarpMma) {
    tc_fence_after();
    if constexpr (kPair)
      tmem2_dealloc(tmem, kTmemCols);
    else
      tmem_dealloc(tmem, kTmemCols);
  }
  if constexpr (kPair) {  // neither CTA ends while the other gives TMEM back
    cluster_arrive();
    cluster_wait();
  }
}

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 1024;
constexpr int kBins = 1024;  // tiles sorted by their key tiles, in this many steps

// Bounds of sequence b; false for an offset outside [0, total] or below the
// one before it.
__device__ __forceinline__ bool seq_bounds(const int32_t* cu, int b, int total, int& first, int& len) {
  first = cu[b];
  const int end = cu[b + 1];
  if (first < 0 || end < first || end > total) {
    first = 0;
    len = 0;
    return false;
  }
  len = end - first;
  return true;
}

// One block: a counting sort of the tiles by the keys they visit, longest
// first.  The order within a bin is by chance; no result depends on it.
__global__ void __launch_bounds__(kPlanThreads)
    prompt_plan_kernel(const int32_t* cu_q, const int32_t* cu_k, int batch, int total_q, int total_k, int causal,
                       int tile_q, int max_tiles, int32_t* plan, int32_t* status) {
  __shared__ int bin[kBins];
  __shared__ int warp_sum[32];
  __shared__ int longest, broken, ragged;
  for (int i = threadIdx.x; i < kBins; i += kPlanThreads) bin[i] = 0;
  if (threadIdx.x == 0) {
    longest = 1;
    broken = 0;
    ragged = 0;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* made = plan + kTileInts * (max_tiles + 1);
  for (int i = threadIdx.x; i <= batch; i += kPlanThreads) {
    made[i] = cu_q[i];
    made[batch + 1 + i] = cu_k[i];
  }
  const int len_q = cu_q[1] - cu_q[0], len_k = cu_k[1] - cu_k[0];
  // warp per sequence, lanes over its tiles
  auto each = [&](auto f) {
    for (int b = warp; b < batch; b += kPlanThreads / 32) {
      int q0, lq, k0, lk;
      bool good = seq_bounds(cu_q, b, total_q, q0, lq);
      good = seq_bounds(cu_k, b, total_k, k0, lk) && good;
      if (!good) {
        lq = 0;
        broken = 1;
      }
      if (lq != len_q || lk != len_k) ragged = 1;
      for (int m = lane; m * tile_q < lq; m += 32) {
        const int row0 = m * tile_q;
        const Tile t{q0 + row0, lq - row0, k0, lk, lk - lq + row0 + 1};
        f(t, max(half_tiles(t, 0, tile_q / 2, causal), half_tiles(t, 1, tile_q / 2, causal)));
      }
    }
  };
  each([&](const Tile&, int n) { atomicMax(&longest, n); });
  __syncthreads();
  const int step = (longest + kBins - 1) / kBins;  // key tiles per bin
  auto bin_of = [&](int n) { return kBins - 1 - min(n / step, kBins - 1); };
  each([&](const Tile&, int n) { atomicAdd(&bin[bin_of(n)], 1); });
  __syncthreads();
  const int mine = bin[threadIdx.x];
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  bin[threadIdx.x] = base + inc - mine;
  if (threadIdx.x == kPlanThreads - 1) {
    // offsets out of order could make sequences overlap: no tiles at all then
    plan[0] = broken ? 0 : base + inc;
    plan[1] = causal;
    plan[2] = ragged && longest >= kLongTiles;
    if (broken) report(status, MLA_ERR_BAD_INDEX);
  }
  __syncthreads();
  each([&](const Tile& t, int n) {
    const int at = atomicAdd(&bin[bin_of(n)], 1);
    if (at >= max_tiles) return;  // a broken plan only
    int4* e = reinterpret_cast<int4*>(plan + kTileInts * (at + 1));
    e[0] = make_int4(t.q0, t.rows, t.k0, t.lk);
    e[1] = make_int4(t.vis, 0, 0, 0);
  });
}
static_assert(kBins == kPlanThreads, "one bin a thread");

}  // namespace pr

// Pairs of CTAs on 512-query tiles where prompts are longer than one CTA's 256
// queries on average, else CTAs on 256.  Causal batches x 16 heads, pairs against
// single CTAs: 128 x 200 tokens 136 and 98 us, 128 x 256 137 and 110, 128 x 300 173
// and 194, 128 x 384 187 and 211, 64 x 512 123 and 139; 64 x 700, whose second tile
// is a third full, 250 and 238.
bool prompt_pairs(int batch, int total_q) { return total_q / batch > 256; }
namespace {
int prompt_tile_q(int batch, int total_q) { return prompt_pairs(batch, total_q) ? 512 : 256; }
}  // namespace
int prompt_plan_tiles(int batch, int total_q) { return total_q / prompt_tile_q(batch, total_q) + batch; }
size_t prompt_plan_bytes(int batch, int total_q) {
  return static_cast<size_t>(prompt_plan_tiles(batch, total_q) + 1) * pr::kTileInts * 4 +
         2 * (static_cast<size_t>(batch) + 1) * 4;
}

cudaError_t launch_prompt_plan(const int32_t* cu_q, const int32_t* cu_k, int batch, int total_q, int total_k,
                               int causal, void* plan, int32_t* status, cudaStream_t st) {
  pr::prompt_plan_kernel<<<1, pr::kPlanThreads, 0, st>>>(cu_q, cu_k, batch, total_q, total_k, causal,
                                                         prompt_tile_q(batch, total_q),
                                                         prompt_plan_tiles(batch, total_q),
                                                         static_cast<int32_t*>(plan), status);
  return cudaGetLastError();
}

namespace {

using PromptKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, PromptParams);

PromptKernel prompt_kernel_of(bool half, int d_qk, bool pair, bool stall = false) {
  if (stall) return pair ? pr::prompt_kernel<false, 3, true, true> : pr::prompt_kernel<false, 3, false, true>;
  if (d_qk == 192) {
    if (half) return pair ? pr::prompt_kernel<true, 3, true> : pr::prompt_kernel<true, 3, false>;
    return pair ? pr::prompt_kernel<false, 3, true> : pr::prompt_kernel<false, 3, false>;
  }
  if (half) return pair ? pr::prompt_kernel<true, 2, true> : pr::prompt_kernel<true, 2, false>;
  return pair ? pr::prompt_kernel<false, 2, true> : pr::prompt_kernel<false, 2, false>;
}

int prompt_smem(int d_qk, bool pair) {
  return d_qk == 192 ? (pair ? pr::Layout<3, true>::kBytes : pr::Layout<3, false>::kBytes)
                     : (pair ? pr::Layout<2, true>::kBytes : pr::Layout<2, false>::kBytes);
}

}  // namespace

cudaError_t prompt_setup() {
  for (int v = 0; v < 10; ++v) {
    const bool stall = v >= 8, pair = stall ? v & 1 : v & 4;
    const int d_qk = stall || (v & 1) ? 192 : 128;
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(prompt_kernel_of(v & 2, d_qk, pair, stall)),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, prompt_smem(d_qk, pair));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_prompt(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PromptParams& p,
                          bool half, int d_qk, bool pair, bool stall, int sms, cudaStream_t st) {
  const int ctas = pair ? 2 : 1;
  const long long items = static_cast<long long>(p.max_tiles) * p.h_q;
  const int most = pair ? std::min(sms / 2, pr::kMaxWorkers) : sms;
  const int workers = static_cast<int>(items < most ? items : most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(workers * ctas), 1, 1);
  cfg.blockDim = dim3(pr::kThreads, 1, 1);
  cfg.dynamicSmemBytes = prompt_smem(d_qk, pair);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_kernel_of(half, d_qk, pair, stall), q, k, v, p);
}

}  // namespace mla
