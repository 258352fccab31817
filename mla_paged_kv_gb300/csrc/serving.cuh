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

}  // namespace mla
