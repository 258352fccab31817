// Attention over whole prompts, packed one after another, causal or not, with
// grouped heads: q, k of 192 (or 128) dims, v of 128.
//
//   s_ij = scale q_i . k_j,  out_i = sum_j e^(s_ij - r_i) v_j / l_i,
//   l_i = sum_j e^(s_ij - r_i),  lse_i = r_i + ln l_i,  j <= i + Lk - Lq
//
// One CTA per (query head, 256-query tile): two 128-row halves, each with its
// own scores, softmax warps and accumulator, take turns on the tensor cores, so
// that one half's exponentials run while the other half's products do.  128
// keys at a time:
//   * TMEM (512 columns): scores of both halves (2 x 128), outputs (2 x 128).
//     A half's weights P overwrite its scores as packed 16-bit pairs and are the
//     A operand of P V from there, so P never touches shared memory.
//   * Shared memory: Q of both halves (6 boxes of 128 rows x 64 dims, 96 KB) and
//     a ring of eight 16 KB boxes through which K (3 boxes) and V (2) stream in
//     the order they are used, K0 V0 K1 V1 ...
//   * One thread issues every MMA in the order
//       PV0(j-1) QK0(j)  PV1(j-1) QK1(j)
//     The tensor pipe runs them in order, so S(j) being ready means PV(j-1) of
//     that half is done: its P may be overwritten, and its O rescaled, without a
//     wait of their own.  Two barriers a half remain: scores ready, weights ready.
//   * The softmax reference r is raised only when a row's maximum grows by more
//     than 2^8 (then O is rescaled in TMEM, rarely); weights stay below 2^8, so
//     sums stay far from overflow.  Statistics are fp32; P is rounded to the
//     inputs' type, which is what the tensor cores take and keeps each weight
//     within half a step of it.
//   * Keys past the sequence's end in its last tile belong to another sequence
//     (or to nothing): their scores are masked and their V rows are zeroed in
//     shared memory, since 0 x NaN would not be 0.
// The tensor work a tile of 128 keys costs one half is 128 x 128 x (192 + 128)
// multiply-adds = 640 cycles at 8192 a cycle; its 16384 exponentials take about
// 512 at 32 a cycle.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "ptx.cuh"
#include "serving.cuh"

namespace mla {
namespace pr {

constexpr int kBM = 128;                  // query rows of a half
constexpr int kBN = 128;                  // keys of a tile
constexpr int kTileQ = 2 * kBM;
constexpr int kBoxBytes = 128 * 128;      // 128 rows x 64 16-bit values
constexpr int kRing = 8;
constexpr int kVBoxes = 2;

constexpr int kThreads = 320;
constexpr int kWarpMma = 8, kWarpLoad = 9;

enum : int {
  Q_FULL = 0,
  R_FULL = 1,               // +slot: a ring box has landed
  R_EMPTY = R_FULL + kRing,  // +slot: its MMAs are done
  S_FULL = R_EMPTY + kRing,  // +half: scores ready, and P V of the tile before done
  P_FULL = S_FULL + 2,       // +half: weights written (128 arrivals)
  O_FULL = P_FULL + 2,       // +half: the last P V is done
  TAIL = O_FULL + 2,         // the last V tile, before its rows past the end are zeroed
  DRAIN,                     // every MMA issued is done
  kNumBars
};

template <int kQBoxes>
struct Layout {
  static constexpr int kOffRing = 2 * kQBoxes * kBoxBytes;
  static constexpr int kOffBar = kOffRing + kRing * kBoxBytes;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 16 + 1024;  // slack to align the base to 1024 B
};
static_assert(Layout<3>::kBytes <= 232448, "shared memory budget");

constexpr uint32_t kTmemCols = 512;
constexpr float kTau = 8.0f;
constexpr float kLn2 = 0.69314718055994530942f;

// Plan: a header {tiles, causal}, then the tiles, kTileInts int32 each.
struct Tile {
  int q0;    // first query row of the tile in the packed q
  int rows;  // queries of the sequence from q0 on (at most 256 matter)
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
__device__ __forceinline__ int half_tiles(const Tile& t, int h, int causal) {
  const int rows = min(t.rows - h * kBM, kBM);
  if (rows <= 0) return 0;
  const int keys = causal ? min(t.lk, t.vis + h * kBM + rows - 1) : t.lk;
  return keys > 0 ? (keys + kBN - 1) / kBN : 0;
}

__device__ __forceinline__ void fail(volatile int* abort_flag, int32_t* status) {
  *abort_flag = 1;
  report(status, MLA_ERR_TIMEOUT);
}

template <bool kHalf, int kQBoxes>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, const PromptParams p) {
  using L = Layout<kQBoxes>;
  // tiles longest first, every head of a tile before the next one: the last CTAs
  // to start are the short ones of all heads
  const int item = blockIdx.x / p.h_q;
  const int head = blockIdx.x - item * p.h_q;
  if (item >= p.plan[0]) return;
  const int causal = p.plan[1];
  const int4* e = reinterpret_cast<const int4*>(p.plan + kTileInts * (item + 1));
  const int4 e0 = e[0];
  const Tile t{e0.x, e0.y, e0.z, e0.w, e[1].x};

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + L::kOffRing;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);

  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int n0 = half_tiles(t, 0, causal), n1 = half_tiles(t, 1, causal);
  const int n = max(n0, n1);

  if (tid == 0) {
    *abort_flag = 0;
    mbar_init(&bars[Q_FULL], 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bars[R_FULL + i], 1);
      mbar_init(&bars[R_EMPTY + i], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&bars[S_FULL + h], 1);
      mbar_init(&bars[P_FULL + h], 128);
      mbar_init(&bars[O_FULL + h], 1);
    }
    mbar_init(&bars[TAIL], 1);
    mbar_init(&bars[DRAIN], 1);
    fence_mbar_init_cluster();
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kWarpLoad && lane == 0) {
    prefetch_tmap(&q_map);
    prefetch_tmap(&k_map);
    prefetch_tmap(&v_map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kWarpLoad) {
    // ------------------------------------------------------------ loads
    const int kvh = head / p.group;
    bool ok = true;
    uint32_t fill = 0;  // ring boxes issued
    const int halves = t.rows > kBM ? 2 : 1;
    bool q_issued = false;
    if (lane == 0 && n > 0) {
      const uint64_t pol = policy_evict_first();
      mbar_arrive_expect_tx(&bars[Q_FULL], halves * kQBoxes * kBoxBytes);
      for (int h = 0; h < halves; ++h)
        for (int s = 0; s < kQBoxes; ++s)
          tma_load_3d(sQ + (h * kQBoxes + s) * kBoxBytes, &q_map, &bars[Q_FULL], 64 * s, head, t.q0 + h * kBM, pol);
      q_issued = true;
    }
    const uint64_t pol_kv = policy_evict_last();
    // one box into the next slot; the tail's boxes complete on their own barrier
    auto box = [&](const CUtensorMap* map, int col, int row, bool tail) {
      const int s = static_cast<int>(fill % kRing);
      const uint32_t round = fill / kRing;
      if (round >= 1) ok = mbar_wait(&bars[R_EMPTY + s], (round - 1) & 1, abort_flag);
      if (!ok) return;
      uint64_t* bar = tail ? &bars[TAIL] : &bars[R_FULL + s];
      if (!tail) mbar_arrive_expect_tx(bar, kBoxBytes);
      tma_load_3d(sRing + s * kBoxBytes, map, bar, col, kvh, row, pol_kv);
      ++fill;
    };
    bool tail_issued = false;
    for (int j = 0; j < n && ok; ++j) {
      const bool tail = (j + 1) * kBN > t.lk;  // the sequence ends inside this tile
      if (lane == 0) {
        for (int s = 0; s < kQBoxes && ok; ++s) box(&k_map, 64 * s, t.k0 + j * kBN, false);
        if (tail && ok) {
          mbar_arrive_expect_tx(&bars[TAIL], kVBoxes * kBoxBytes);
          tail_issued = true;
        }
        // where the two V boxes wrap around the ring, dims 0-63 take slot 0, so
        // that they come first in shared memory too
        const int swap = fill % kRing == kRing - 1 ? 1 : 0;
        for (int s = 0; s < kVBoxes && ok; ++s) box(&v_map, 64 * (s ^ swap), t.k0 + j * kBN, tail);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      fill = __shfl_sync(0xffffffffu, fill, 0);
      if (tail && ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[TAIL], 0, abort_flag));
        if (ok) {
          const int keep = t.lk - j * kBN;  // rows of this tile that are the sequence's
          for (int b = 0; b < kVBoxes; ++b) {
            const int s = static_cast<int>((fill - kVBoxes + b) % kRing);
            uint4* dst = reinterpret_cast<uint4*>(sRing + s * kBoxBytes + keep * 128);
            for (int i = lane; i < (kBN - keep) * 8; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0)
            for (int b = 0; b < kVBoxes; ++b)
              mbar_arrive(&bars[R_FULL + static_cast<int>((fill - kVBoxes + b) % kRing)]);
        }
      }
    }
    if (lane == 0) {
      if (!ok) fail(abort_flag, p.status);
      // no TMA write may land after this CTA exits
      if (q_issued) mbar_wait(&bars[Q_FULL], 0, nullptr);
      if (!ok) {
        if (tail_issued) mbar_wait(&bars[TAIL], 0, nullptr);
        for (uint32_t s = 0; s < kRing && s < fill; ++s) {
          const uint32_t last = (fill - 1 - s) / kRing;  // the slot's last round
          mbar_wait(&bars[R_FULL + s], last & 1, nullptr, 1000000);
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMAs
    // the whole warp runs this loop (see umma_f16_warp); its control flow and
    // every operand are the same in all lanes
    if (n > 0) {
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      constexpr uint32_t idesc_qk = idesc_16bit_f32(128, kBN, false, kHalf);
      constexpr uint32_t idesc_pv = idesc_16bit_f32(128, 128, true, kHalf);
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(sRing), 16, 1024);
      auto wait = [&](int bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(&bars[bar], parity, abort_flag));
      };
      bool ok = wait(Q_FULL, 0);
      uint32_t use = 0;  // ring boxes waited for
      uint32_t k_at = 0, v_at = 0;
      auto wait_boxes = [&](int count) {
        const uint32_t at = use;
        for (int i = 0; i < count && ok; ++i, ++use)
          ok = wait(R_FULL + use % kRing, (use / kRing) & 1);
        return at;
      };
      for (int j = 0; j <= n && ok; ++j) {
        // boxes in load order: V(j-1) before K(j)
        bool have_v = false, have_k = false;
#pragma unroll 1
        for (int h = 0; h < 2 && ok; ++h) {
          const int nh = h ? n1 : n0;
          const uint32_t s_col = tm + 128u * h, o_col = tm + 256u + 128u * h;
          if (j >= 1 && j - 1 < nh) {
            if (!have_v) {
              v_at = wait_boxes(kVBoxes);
              have_v = true;
            }
            if (ok) ok = wait(P_FULL + h, (j - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            // V as the MN-major B operand: dims 0-63 in one box, 64-127 in the
            // next, or (where the ring wraps) seven boxes further on
            const uint32_t s0 = v_at % kRing;
            const bool wrap = s0 == kRing - 1;
            const uint64_t vd = sdesc_sw128(smem_u32(sRing + (wrap ? 0u : s0) * kBoxBytes),
                                            (wrap ? kRing - 1 : 1) * kBoxBytes, 1024);
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk)
              umma_f16_ts_warp(o_col, s_col + 8u * kk, vd + static_cast<uint64_t>((kk * 2048) >> 4), idesc_pv,
                          (j == 1 && kk == 0) ? 0u : 1u);
            if (j == nh) umma_commit_warp(&bars[O_FULL + h]);
          }
          if (j < nh) {
            if (!have_k) {
              k_at = wait_boxes(kQBoxes);
              have_k = true;
            }
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < kQBoxes; ++s) {
              const uint64_t kd = k_desc + static_cast<uint64_t>((((k_at + s) % kRing) * kBoxBytes) >> 4);
              const uint64_t qd = q_desc + static_cast<uint64_t>(((h * kQBoxes + s) * kBoxBytes) >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_f16_warp(s_col, qd + static_cast<uint64_t>((kk * 32) >> 4), kd + static_cast<uint64_t>((kk * 32) >> 4),
                         idesc_qk, (s == 0 && kk == 0) ? 0u : 1u);
            }
            umma_commit_warp(&bars[S_FULL + h]);
          }
        }
        if (!ok) break;
        if (have_v)
          for (int b = 0; b < kVBoxes; ++b) umma_commit_warp(&bars[R_EMPTY + (v_at + b) % kRing]);
        if (have_k)
          for (int s = 0; s < kQBoxes; ++s) umma_commit_warp(&bars[R_EMPTY + (k_at + s) % kRing]);
      }
      if (!ok && lane == 0) fail(abort_flag, p.status);
      // every MMA is done with shared memory and TMEM before this CTA ends
      umma_commit_warp(&bars[DRAIN]);
      mbar_wait(&bars[DRAIN], 0, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int h = warp >> 2;
    const int r = tid & 127;  // row of the half == TMEM lane
    const int row = h * kBM + r;
    const int nh = h ? n1 : n0;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_addr = tmem + lane_base + 128u * h;
    const uint32_t o_addr = tmem + lane_base + 256u + 128u * h;
    const bool row_ok = row < t.rows;
    const int limit = causal ? min(t.lk, t.vis + row) : t.lk;  // keys this row sees
    const float c_log2 = p.scale_log2;
    float ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nh; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[S_FULL + h], j & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      float s[kBN];
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32_max(s_addr + 32u * c, s + 32 * c, mx[c]);
      tmem_wait_ld();
      float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      const int seen = limit - j * kBN;
      if (__any_sync(0xffffffffu, seen < kBN)) {
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kBN; ++i) {
          s[i] = i < seen ? s[i] : -INFINITY;
          m4[i & 3] = fmaxf(m4[i & 3], s[i]);
        }
        top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      }
      const float mt = top * c_log2;
      const float r_new = mt > ref + kTau ? mt : ref;
      const float alpha = r_new == ref ? 1.f : ex2(ref - r_new);
      // P V of the tile before is done (see above): O may be rescaled here
      if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
        for (uint32_t c0 = 0; c0 < 128; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(o_addr + c0, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
          tmem_st16(o_addr + c0, v);
        }
      }
      ref = r_new;
      const float mref = ref == -INFINITY ? 0.f : ref;
      float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      const float2 cl = make_float2(c_log2, c_log2), nr = make_float2(-mref, -mref);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x = __ffma2_rn(make_float2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), cl, nr);
          const float p0 = ex2(x.x), p1 = ex2(x.y);
          pk[i] = pack2<kHalf>(p0, p1);
          ls[i & 1] = __fadd2_rn(ls[i & 1], make_float2(p0, p1));
        }
        tmem_st16(s_addr + 16u * c, pk);
      }
      l = l * alpha + ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y));
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars[P_FULL + h]);
    }
    if (ok && nh > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[O_FULL + h], 0, abort_flag));
      tc_fence_after();
    }
    if (ok) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const size_t orow = static_cast<size_t>(t.q0 + row) * p.h_q + head;
      uint16_t* out = static_cast<uint16_t*>(p.out) + orow * 128;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t v[32];
        if (nh > 0) {
          tmem_ld32(o_addr + 32u * c, v);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
        if (row_ok) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // a row without keys has l = 0 and an untouched or zero sum: 0 by selection
              const float a = __uint_as_float(v[8 * q + 2 * i]) * inv, b = __uint_as_float(v[8 * q + 2 * i + 1]) * inv;
              w[i] = limit > 0 ? pack2<kHalf>(a, b) : 0u;
            }
            *reinterpret_cast<uint4*>(out + 32 * c + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (row_ok) p.lse[orow] = limit > 0 ? (ref + __log2f(l)) * kLn2 : -INFINITY;
    } else if (lane == 0) {
      fail(abort_flag, p.status);
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
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
                       int max_tiles, int32_t* plan, int32_t* status) {
  __shared__ int bin[kBins];
  __shared__ int warp_sum[32];
  __shared__ int longest, broken;
  for (int i = threadIdx.x; i < kBins; i += kPlanThreads) bin[i] = 0;
  if (threadIdx.x == 0) {
    longest = 1;
    broken = 0;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
      for (int m = lane; m * kTileQ < lq; m += 32) {
        const int row0 = m * kTileQ;
        const Tile t{q0 + row0, lq - row0, k0, lk, lk - lq + row0 + 1};
        f(t, max(half_tiles(t, 0, causal), half_tiles(t, 1, causal)));
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

int prompt_plan_tiles(int batch, int total_q) { return total_q / pr::kTileQ + batch; }
size_t prompt_plan_bytes(int batch, int total_q) {
  return static_cast<size_t>(prompt_plan_tiles(batch, total_q) + 1) * pr::kTileInts * 4;
}

cudaError_t launch_prompt_plan(const int32_t* cu_q, const int32_t* cu_k, int batch, int total_q, int total_k,
                               int causal, void* plan, int32_t* status, cudaStream_t st) {
  pr::prompt_plan_kernel<<<1, pr::kPlanThreads, 0, st>>>(cu_q, cu_k, batch, total_q, total_k, causal,
                                                         prompt_plan_tiles(batch, total_q),
                                                         static_cast<int32_t*>(plan), status);
  return cudaGetLastError();
}

cudaError_t prompt_setup() {
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(pr::prompt_kernel<false, 3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                pr::Layout<3>::kBytes)) != cudaSuccess)
    return e;
  if ((e = cudaFuncSetAttribute(pr::prompt_kernel<true, 3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                pr::Layout<3>::kBytes)) != cudaSuccess)
    return e;
  if ((e = cudaFuncSetAttribute(pr::prompt_kernel<false, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                pr::Layout<2>::kBytes)) != cudaSuccess)
    return e;
  return cudaFuncSetAttribute(pr::prompt_kernel<true, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              pr::Layout<2>::kBytes);
}

cudaError_t launch_prompt(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PromptParams& p,
                          bool half, int d_qk, cudaStream_t st) {
  const int grid = p.max_tiles * p.h_q;
  if (d_qk == 192) {
    if (half)
      pr::prompt_kernel<true, 3><<<grid, pr::kThreads, pr::Layout<3>::kBytes, st>>>(q, k, v, p);
    else
      pr::prompt_kernel<false, 3><<<grid, pr::kThreads, pr::Layout<3>::kBytes, st>>>(q, k, v, p);
  } else {
    if (half)
      pr::prompt_kernel<true, 2><<<grid, pr::kThreads, pr::Layout<2>::kBytes, st>>>(q, k, v, p);
    else
      pr::prompt_kernel<false, 2><<<grid, pr::kThreads, pr::Layout<2>::kBytes, st>>>(q, k, v, p);
  }
  return cudaGetLastError();
}

}  // namespace mla
