// Parameter blocks and launch functions of the serving operators (append,
// pages, prompt attention), shared by their kernels and the C ABI layer.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mla {

// From the C ABI layer of the decode: MLA_OK and the SM count if the current
// device is one this library runs on, else a status; and a tiled tensor map
// over 16-bit elements, dims innermost first, 128-byte swizzle.
int device_ready(int* sms);
int encode_map16(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box);

// The decode kernels over the units of a shared-prefix plan, and the scheduler
// over unit lengths (both with the decode's own code).
struct SharedLaunch {
  const void* q;
  const void* kv;
  long long total_rows;  // batch * s_q * h_q
  const int32_t* live;   // the caller's lengths, to be compared with the plan's, or NULL
  int batch, num_pages, max_pages, n_units, s_q, h_q, num_parts;
  int dtype;  // MLA_DTYPE_BF16, _FP16 or _FP8_RECORD
  float scale_log2;
  const int32_t *block_table, *units, *lengths, *sched, *split_offset;
  float *o_accum, *lse_accum;  // [slots][128][512], [slots][128]
  int32_t* status;
  int stall;  // 1: the stall-test instances
};
int launch_shared(const SharedLaunch& c, cudaStream_t stream);
int decode_full_blocks(const void* q, const void* kv, const int32_t* block_table, int max_pages, int num_pages,
                       const int32_t* lengths, const int32_t* live, int batch, int s_q, int h_q, int dtype,
                       int causal, float scale, const int32_t* sched, const int32_t* split_offset, int num_parts,
                       void* ws, size_t ws_bytes, void* out, int out_type, float* lse, int32_t* status, int stall,
                       cudaStream_t stream);
cudaError_t launch_plan(const int32_t* lengths, int n_units, int num_parts, int32_t* sched, int32_t* split_offset,
                        cudaStream_t stream);

cudaError_t launch_shared_units(const int32_t* block_table, int max_pages, const int32_t* seqlens, int batch,
                                int s_q, int h_q, int causal, int32_t* units, int32_t* lengths,
                                cudaStream_t st);
cudaError_t launch_shared_lengths(const int32_t* seqlens, int batch, int32_t* lengths, cudaStream_t st);
cudaError_t launch_shared_combine(const float* o_accum, const float* lse_accum, const int32_t* units,
                                  const int32_t* split_offset, int batch, int rows, void* out, int out_type,
                                  float* lse, int sms, cudaStream_t st);
constexpr int kMaxSharedParts = 1024;  // partitions of a shared-prefix plan

struct AppendParams {
  const uint16_t* c;
  long long c_stride;
  const uint16_t* r;
  long long r_stride;
  int total, batch;
  const int32_t* cu;  // NULL: total / batch tokens each
  const int32_t* seqlens;
  const int32_t* table;
  int max_pages, num_pages;
  void* cache;
  const uint16_t* weight;
  float eps;
  const float* cos_sin;
  int max_pos, interleaved;
  const int32_t* refcount;
  int32_t* status;
};
cudaError_t launch_append(const AppendParams& p, bool half, bool fp8, int sms, cudaStream_t stream);

// A rotary table: each pair's step a position, in 2^-64 turns.
constexpr int kMaxRopeDim = 256;
struct RopeSteps {
  unsigned long long step[kMaxRopeDim / 2];
};
cudaError_t launch_rope_table(const RopeSteps& f, int dim, float magnitude, long long first, int positions, float* out,
                              int sms, cudaStream_t st);

// Rotation (and norm) of heads: queries, and keys or none (heads = 0).
struct RopeSide {
  const uint16_t* x;
  uint16_t* out;  // may be x
  const uint16_t* weight;
  long long x_token_stride, x_head_stride, out_token_stride, out_head_stride;
  int heads;
};
struct RopeHeadsParams {
  RopeSide side[2];
  int total, batch, dim, rope, offset, interleaved;
  int pairs, items, lane_bits, units;  // rope_heads_layout; units: warps a token
  float eps, inv_dim;
  const int32_t *positions, *cu, *seqlens;
  const float* cos_sin;  // NULL: no rotation
  int max_pos;
  int32_t* status;
};
constexpr int kMaxHeadDim = 1024;
// The kernel's layout; passes: dims outside the rotary part are read and
// written too.  False where the grid would be too large.
bool rope_heads_layout(RopeHeadsParams* p, bool passes, int* per_lane, long long* blocks);
cudaError_t launch_rope_heads(const RopeHeadsParams& p, bool half, int per_lane, long long blocks, cudaStream_t st);

struct GatherParams {
  const void* cache;
  const int32_t *table, *cu, *starts;  // starts: NULL: 0
  int max_pages, num_pages, batch, total;
  uint16_t* out;
  long long out_stride;
  int32_t* status;
};
cudaError_t launch_gather(const GatherParams& p, bool fp8, cudaStream_t st);

// The bookkeeping of a page pool.
struct PageState {
  int32_t* refcount;
  int num_pages;
  int32_t* table;
  int rows, max_pages;
  int32_t* seqlens;
  int32_t* status;
};
constexpr int kMaxPageRows = 65536;  // rows of a block table
constexpr int kMaxPageList = 4096;   // list entries a call
cudaError_t launch_grow(const PageState& s, const int32_t* rows, const int32_t* new_tokens, int n, cudaStream_t st);
cudaError_t launch_fork(const PageState& s, const int32_t* parents, const int32_t* children, int n, int32_t* pairs,
                        cudaStream_t st);
cudaError_t launch_free(const PageState& s, const int32_t* rows, int n, cudaStream_t st);
size_t compact_workspace_bytes(int num_pages);
cudaError_t launch_compact(const PageState& s, int32_t* pairs, int32_t* count, void* ws, cudaStream_t st);
cudaError_t copy_pages_setup();  // once per device: shared-memory opt-in
cudaError_t launch_copy_pages(void* pool, int layers, long long layer_stride, int num_pages, long long page_bytes,
                              const int32_t* pairs, const int32_t* count, int n, int32_t* status, int sms,
                              cudaStream_t st);

struct PromptParams {
  const int32_t* plan;  // header and tiles
  int max_tiles;        // tiles the plan has room for
  int h_q, group;       // query heads, query heads per key head
  int total_q;
  int batch;
  const int32_t *cu_q, *cu_k;  // the caller's offsets, to be compared with the plan's, or NULL
  float scale_log2;
  void* out;            // [total_q, h_q, 128]
  float* lse;           // [total_q, h_q]
  int32_t* status;
};
size_t prompt_plan_bytes(int batch, int total_q);
bool prompt_pairs(int batch, int total_q);  // CTA pairs on 512 queries (else CTAs on 256)
int prompt_plan_tiles(int batch, int total_q);
cudaError_t launch_prompt_plan(const int32_t* cu_q, const int32_t* cu_k, int batch, int total_q, int total_k,
                               int causal, void* plan, int32_t* status, cudaStream_t st);
cudaError_t prompt_setup();  // once per device: shared-memory opt-in
cudaError_t launch_prompt(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PromptParams& p,
                          bool half, int d_qk, bool pair, bool stall, int sms, cudaStream_t st);

// Attention of ragged chunks over a paged cache: the plan's parts, from its start.
constexpr int kMaxChunkParts = 1024;
constexpr int kMaxChunkKeys = 1 << 24;  // keys of a request
constexpr int kFixedCost = 6;            // a unit's Q load and epilogue, in half tiles of 128 keys
constexpr int kChunkUnitInts = 12;
constexpr int kConvertUnits = 3;         // units from which a request's FP8 pages are converted once for all
// header: units, causal, units for the combine (2), whether an offset or length was out of range (no units then)
enum : int { kHeadWhole = 0, kHeadCausal = 1, kHeadFix = 2, kHeadBroken = 4 };
struct ChunkPlanLayout {
  int max_units;
  size_t units, first, conv, made, bytes;
  struct {
    size_t sched, fix, rest, cost, prefix;
  } schedule[2];  // for 16-bit caches, and FP8 records
};
ChunkPlanLayout chunk_plan_layout(int batch, int total_q, int h_q, int parts);
struct ChunkSchedule {
  int32_t *sched, *fix, *rest, *cost;
  long long* prefix;
};
struct ChunkPlanParams {
  const int32_t *cu, *lens;
  int batch, total_q, h_q, causal, parts;
  int32_t *head, *units, *first, *conv, *made;
  ChunkSchedule schedule[2];
  int32_t* status;
};
struct ChunkParams {
  const int32_t *head, *units, *sched, *fix, *rest, *conv, *made;  // of the plan
  int schedule;                                                    // 0, or 1: FP8 records
  const int32_t *cu, *lens;                          // the caller's, to be compared with the plan's, or NULL
  const uint8_t* records;  // a cache of FP8 records, or NULL
  int room;                // pages that the workspace holds converted
  uint8_t* queries;        // [total_q * h_q][MLA_CHUNK_QUERY_BYTES], behind them
  long long rows;          // total_q * h_q
  const int32_t* block_table;
  int max_pages, num_pages, batch, h_q;
  float scale_log2;
  void* out;  // [total_q * h_q, 512]
  int out_type;
  float* lse;
  float *o_accum, *lse_accum;  // [2 parts][128][512], [2 parts][128]
  int32_t* status;
};
cudaError_t chunk_setup();  // once per device: shared-memory opt-in
cudaError_t launch_chunk_plan(const ChunkPlanParams& p, cudaStream_t st);
cudaError_t launch_chunk(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& rope,
                         const ChunkParams& p, bool half, bool stall, int parts, cudaStream_t st);
cudaError_t launch_chunk_convert(const ChunkParams& p, const uint16_t* q, uint16_t* pages, int sms, cudaStream_t st);
cudaError_t launch_chunk_combine(const ChunkParams& p, int parts, int sms, cudaStream_t st);

}  // namespace mla
