// Shared definitions of the MLA decode kernels (device side).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mla_paged_kv.h"

namespace mla {

constexpr int kTile = MLA_PAGE_SIZE;        // keys per pipeline tile = one page
constexpr int kRowsPerBlock = MLA_ROWS_PER_BLOCK;
constexpr int kDqk = MLA_D_QK;
constexpr int kDv = MLA_D_V;

// First error wins; later ones are dropped so the caller sees the root cause.
__device__ __forceinline__ void report(int32_t* status, int code) {
  if (status != nullptr) atomicCAS(reinterpret_cast<int*>(status), 0, code);
}

__host__ __device__ __forceinline__ int ceil_div_i(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ int num_tiles(int len) { return len > 0 ? ceil_div_i(len, kTile) : 0; }

// One unit of a shared-prefix plan: up to 128 consecutive query rows and the
// run of keys they all read (a 128-row block over the shared pages, or a
// block of one request's rows over the pages behind them).
struct SharedUnit {
  int row0;       // first query row, of batch * s_q * h_q
  int rows;       // query rows
  int rel;        // row0's place among its request's rows (causal), or -1: every key is visible
  int table_off;  // its first page's entry, from the block table's start
  int avail;      // entries of the block-table row from there on
};
constexpr int kUnitInts = 8;

// Everything the split-KV attention kernels read besides the tensor maps.
struct DecodeParams {
  // keys per unit (dense: cache_seqlens, sparse: topk_length or NULL)
  const int32_t* lengths;
  int default_length;       // used when lengths == NULL
  int n_units;              // dense: batch; sparse: batch * s_q
  int rows;                 // query rows per unit (dense s_q*h_q, sparse h_q)
  int row_blocks;           // CTA pairs per partition: h_kv * blocks_per_group
  int h_q;
  // dense: latent KV heads.  Query head h reads KV head h / group_heads.  With
  // h_kv = 1 a row block is 128 consecutive rows (token-major) of the unit;
  // with h_kv > 1 it is block_tokens whole tokens of one head group.
  int h_kv;
  int group_heads;          // h_q / h_kv
  int block_tokens;         // h_kv > 1: tokens per row block (group_heads * block_tokens <= 128)
  int blocks_per_group;     // row blocks per head group
  int s_q;                  // query tokens per request (causal alignment)
  int causal;
  float scale_log2;         // softmax_scale * log2(e)
  // dense
  int q_vring;              // host: 1 selects the kernel instance that stages the first unit's Q in the V ring
  const int32_t* block_table;
  int max_pages;
  int num_pages;
  // sparse
  const int32_t* indices;   // [n_units, topk] (native selection), or NULL when packed
  int topk;
  const uint8_t* kv8;       // [num_pages, 64, 656]; packed: the packed records
  const uint64_t* packed_mask;  // packed: [n_units, ceil(topk/64)] valid-slot bits, else NULL
  // sparse kernel over a dense FP8 cache (block_table set): unit b reads
  // block-table row b / unit_request_div (s_q when a unit is one query token
  // of a request, 1 when it is the whole request)
  int unit_request_div;
  // shared-prefix plan (kShared instances): what each unit is, kUnitInts int32
  // each (SharedUnit); rows = 128, a unit's rows being its own count
  const int32_t* units;
  // schedule
  const int32_t* sched;
  const int32_t* split_offset;
  int num_parts;
  // outputs
  float* o_accum;           // [slots, rows, 512]
  float* lse_accum;         // [slots, rows]
  void* out;                // [n_units, rows, 512]
  int out_type;             // MLA_DTYPE_BF16, MLA_DTYPE_FP32 or MLA_DTYPE_FP16
  float* lse;               // [n_units, rows]
  int32_t* status;
};

// The kWarp instances' further parameters: the caller's lengths [n], to be
// compared with those of the plan (check_plan), or NULL; under a shared-prefix
// plan request b's first own unit is first + b * per.
struct LiveLengths {
  const int32_t* lengths = nullptr;
  int n = 0, first = 0, per = 0;
};
struct WarpParams : DecodeParams {
  LiveLengths live;
};
template <bool kWarp>
struct KernelParams {
  using type = DecodeParams;
};
template <>
struct KernelParams<true> {
  using type = WarpParams;
};

__device__ __forceinline__ SharedUnit load_unit(const DecodeParams& p, int u) {
  const int32_t* e = p.units + u * kUnitInts;
  return SharedUnit{e[0], e[1], e[2], e[3], e[4]};
}

// Whether the plan is that of the caller's lengths (and, under a shared prefix,
// each request that takes part still ends it on the page that they share), by
// warps that have loaded their last tile; the call's results are those of the
// plan either way.  (In the softmax warps, before their first tile, it took 3% of
// the kernel.)
template <bool kShared>
__device__ __forceinline__ void check_plan(const WarpParams& p, int thread, int threads) {
  const LiveLengths& live = p.live;
  if (live.lengths == nullptr) return;
  for (int b = thread; b < live.n; b += threads) {
    bool same;
    if constexpr (kShared) {
      const int u = live.first + b * live.per;
      const SharedUnit su = load_unit(p, u), front = load_unit(p, 0);
      const int skip = su.table_off - b * p.max_pages;  // shared pages
      same = p.lengths[u] + skip * kTile == max(live.lengths[b], 0) &&
             (skip == 0 || p.block_table[su.table_off - 1] == p.block_table[front.table_off + skip - 1]);
    } else {
      same = p.lengths[b] == live.lengths[b];
    }
    if (!same) report(p.status, MLA_ERR_STALE_PLAN);
  }
}

}  // namespace mla
