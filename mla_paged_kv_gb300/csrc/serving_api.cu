// C ABI of the serving operators (mla_serving.h): argument checks, tensor
// maps and launches.  No device memory is allocated here.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "mla_serving.h"
#include "common.cuh"
#include "serving.cuh"

using namespace mla;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
cudaStream_t to_stream(mla_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
int launched(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

constexpr long long kMaxInt = (1LL << 31) - 1;
constexpr int kMaxRowPages = 1 << 18;  // pages of one block-table row: positions and sums stay in 32 bits

// Checks common to the calls that take a page pool's bookkeeping.
int page_state(int32_t* refcount, int num_pages, int32_t* table, int rows, int max_pages, int32_t* seqlens,
               int32_t* status, PageState* s) {
  if (!refcount || !table || !seqlens || !status) return MLA_ERR_INVALID_ARG;
  if (num_pages < 1 || rows < 1 || max_pages < 1) return MLA_ERR_INVALID_ARG;
  if (!aligned(refcount, 4) || !aligned(table, 4) || !aligned(seqlens, 4) || !aligned(status, 4))
    return MLA_ERR_INVALID_ARG;
  if (rows > kMaxPageRows || max_pages > kMaxRowPages) return MLA_ERR_UNSUPPORTED;
  if (num_pages > (1 << 30)) return MLA_ERR_UNSUPPORTED;
  *s = PageState{refcount, num_pages, table, rows, max_pages, seqlens, status};
  return MLA_OK;
}

int check_list(const int32_t* a, const int32_t* b, int n) {
  if (n < 0 || (n > 0 && (!a || !b)) || !aligned(a, 4) || !aligned(b, 4)) return MLA_ERR_INVALID_ARG;
  return n > kMaxPageList ? MLA_ERR_UNSUPPORTED : MLA_OK;
}

// device_ready, and this file's kernels set up for the current device (once).
int serving_device(int* sms) {
  constexpr int kMaxDevices = 64;
  static bool done[kMaxDevices] = {};
  static std::mutex mu;
  int dev = -1;
  const int rc = device_ready(sms);
  if (rc != MLA_OK) return rc;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MLA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    if (prompt_setup() != cudaSuccess || copy_pages_setup() != cudaSuccess) {
      cudaGetLastError();
      return MLA_ERR_CUDA;
    }
    done[dev] = true;
  }
  return MLA_OK;
}

// [total, heads, dim] of 16-bit elements, viewed as (64 dims of a slice, total,
// slices, heads), innermost first; one box = `slices` consecutive 64-dim slices
// of `rows` rows of one head, which lands slice after slice, each `rows` rows of
// 128 swizzled bytes, by one TMA instruction.
int head_map(CUtensorMap* m, const void* base, long long total, int heads, int dim, long long token_stride,
             long long head_stride, unsigned rows, unsigned slices) {
  // a stride that no second index uses may be anything: take a legal one
  if (heads == 1) head_stride = dim;
  if (total == 1) token_stride = static_cast<long long>(heads) * head_stride;
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(total), static_cast<cuuint64_t>(dim / 64),
                              static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(token_stride) * 2, 128,
                                 static_cast<cuuint64_t>(head_stride) * 2};
  const cuuint32_t box[4] = {64, rows, slices, 1};
  return encode_map16(m, base, 4, dims, strides, box);
}

// Strides of a [total, heads, dim] tensor: multiples of 8 elements, no
// smaller than a row, within what a tensor map takes.
bool good_strides(long long total, int heads, int dim, long long ts, long long hs) {
  const long long most = 1LL << 38;
  if (heads > 1 && (hs < dim || hs % 8 != 0 || hs > most)) return false;
  return total <= 1 || (ts >= dim && ts % 8 == 0 && ts <= most);
}

// Sizes of a shared-prefix batch, and where its plan's and workspace's parts
// lie (each from a 256-byte boundary).
struct SharedSizes {
  int share;      // 1: a prefix is attended together
  int units;      // at most: prefix blocks, then the requests' own
  long long rows;  // batch * s_q * h_q
  size_t lengths_off, offset_off, sched_off, plan_bytes;
  size_t lse_off, ws_bytes;
};

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int shared_sizes(int batch, int s_q, int h_q, int num_parts, SharedSizes* z) {
  if (batch < 1 || s_q < 1 || h_q < 1 || num_parts < 1) return MLA_ERR_INVALID_ARG;
  const long long per_request = static_cast<long long>(s_q) * h_q;
  z->rows = per_request * batch;
  if (per_request > (1 << 20) || batch > 65535 || z->rows > kMaxInt || num_parts > kMaxSharedParts)
    return MLA_ERR_UNSUPPORTED;
  const long long own = batch * ((per_request + MLA_ROWS_PER_BLOCK - 1) / MLA_ROWS_PER_BLOCK);
  const long long front = (z->rows + MLA_ROWS_PER_BLOCK - 1) / MLA_ROWS_PER_BLOCK;
  // Attended together where that takes at most 7/8 of the row blocks: the prefix's
  // partials and their merge have to be won back.  Together and request by request
  // (64 requests unless said, 8192 shared and 500 own keys, bf16): 96 heads 111 and
  // 125 us, 104 116 and 128, 112 126 and 127, 120 136 and 131; 32 requests x 2 x 100
  // heads, 4096 keys 72 and 75, 2 x 112 80 and 76.  (A prefix of 1024 keys and 96
  // heads loses: 42 and 39; 64 heads 33.5 and 36.)  FP8 records: 96 heads 290 and
  // 358 us, 112 334 and 358, 120 355 and 360.
  z->share = front * 8 <= own * 7;
  const long long units = z->share ? own + front : batch;
  z->units = static_cast<int>(units);
  z->lengths_off = up256(static_cast<size_t>(units) * kUnitInts * 4);
  z->offset_off = z->lengths_off + up256(static_cast<size_t>(units) * 4);
  z->sched_off = z->offset_off + up256(static_cast<size_t>(units + 1) * 4);
  z->plan_bytes = z->sched_off + up256(static_cast<size_t>(num_parts) * MLA_SCHED_INTS * 4);
  if (!z->share) {  // the plan and the workspace of the plain decode
    z->ws_bytes = mla_workspace_bytes(batch, static_cast<int>(per_request), num_parts);
    return MLA_OK;
  }
  const size_t slots = static_cast<size_t>(units) + num_parts;
  z->lse_off = slots * MLA_ROWS_PER_BLOCK * MLA_D_V * 4;
  z->ws_bytes = z->lse_off + slots * MLA_ROWS_PER_BLOCK * 4;
  return MLA_OK;
}

// mla_prompt_attention_fwd, with offsets to be compared with the plan's or NULL.
int prompt_attention(const void* d_q, long long q_token_stride, long long q_head_stride, const void* d_k,
                     long long k_token_stride, long long k_head_stride, const void* d_v, long long v_token_stride,
                     long long v_head_stride, int dtype, int total_q, int total_k, int batch, int h_q, int h_kv,
                     int d_qk, float softmax_scale, const int32_t* cu_q, const int32_t* cu_k, const void* d_plan,
                     size_t plan_bytes, void* d_out, float* d_lse, int32_t* d_status, bool stall,
                     mla_stream_t stream) {
  if (!d_plan || !d_status || batch < 1 || total_q < 0 || total_k < 0 || h_q < 1 || h_kv < 1 || h_q % h_kv != 0)
    return MLA_ERR_INVALID_ARG;
  if (total_q > 0 && (!d_q || !d_out || !d_lse)) return MLA_ERR_INVALID_ARG;
  if (total_k > 0 && (!d_k || !d_v)) return MLA_ERR_INVALID_ARG;
  if (dtype != MLA_DTYPE_BF16 && dtype != MLA_DTYPE_FP16) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  if (!aligned(d_q, 16) || !aligned(d_k, 16) || !aligned(d_v, 16) || !aligned(d_plan, 16) || !aligned(d_out, 16) ||
      !aligned(d_lse, 4) || !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(d_status, 4))
    return MLA_ERR_INVALID_ARG;
  if (!good_strides(total_q, h_q, d_qk, q_token_stride, q_head_stride) ||
      !good_strides(total_k, h_kv, d_qk, k_token_stride, k_head_stride) ||
      !good_strides(total_k, h_kv, 128, v_token_stride, v_head_stride))
    return MLA_ERR_INVALID_ARG;
  if (d_qk != 192 && d_qk != 128) return MLA_ERR_UNSUPPORTED;
  if (total_q > (1 << 30) || total_k > (1 << 30) || batch > (1 << 20)) return MLA_ERR_UNSUPPORTED;
  if (plan_bytes < prompt_plan_bytes(batch, total_q)) return MLA_ERR_INVALID_ARG;
  const int tiles = prompt_plan_tiles(batch, total_q);
  if (static_cast<long long>(tiles) * h_q > (1 << 30)) return MLA_ERR_UNSUPPORTED;
  int sms = 0;
  const int rc0 = serving_device(&sms);
  if (rc0 != MLA_OK || total_q == 0) return rc0;
  PromptParams p{};
  p.plan = static_cast<const int32_t*>(d_plan);
  p.max_tiles = tiles;
  p.h_q = h_q;
  p.group = h_q / h_kv;
  p.total_q = total_q;
  p.batch = batch;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  p.out = d_out;
  p.lse = d_lse;
  p.status = d_status;
  const bool pair = prompt_pairs(batch, total_q);
  CUtensorMap qm, km, vm;
  int rc = head_map(&qm, d_q, total_q, h_q, d_qk, q_token_stride, q_head_stride, 128, d_qk / 64);
  if (total_k == 0) {  // no CTA loads K or V: any valid map serves
    km = vm = qm;
  } else {
    // a pair's CTAs load 64 keys each, and all 128 for their half of V's dims
    if (rc == MLA_OK)
      rc = head_map(&km, d_k, total_k, h_kv, d_qk, k_token_stride, k_head_stride, pair ? 64 : 128, d_qk / 64);
    if (rc == MLA_OK)
      rc = head_map(&vm, d_v, total_k, h_kv, 128, v_token_stride, v_head_stride, 128, pair ? 1 : 2);
  }
  if (rc != MLA_OK) return rc;
  return launched(launch_prompt(qm, km, vm, p, dtype == MLA_DTYPE_FP16, d_qk, pair, stall, sms, to_stream(stream)));
}

// mla_shared_prefix_decode_fwd, with lengths to be compared with the plan's or NULL.
int shared_decode(const void* d_q, const void* d_kv, const int32_t* d_block_table, int max_pages, int num_pages,
                  int batch, int s_q, int h_q, int dtype, int causal, float softmax_scale, const int32_t* live,
                  const void* d_plan, size_t plan_bytes, int num_parts, void* d_workspace, size_t workspace_bytes,
                  void* d_out, int out_type, float* d_lse, int32_t* d_status, int stall, mla_stream_t stream) {
  if (!d_q || !d_kv || !d_block_table || !d_plan || !d_workspace || !d_out || !d_lse || !d_status)
    return MLA_ERR_INVALID_ARG;
  if (max_pages < 1 || num_pages < 1) return MLA_ERR_INVALID_ARG;
  if (dtype != MLA_DTYPE_BF16 && dtype != MLA_DTYPE_FP16 && dtype != MLA_DTYPE_FP8_RECORD)
    return MLA_ERR_INVALID_ARG;
  if (out_type != MLA_DTYPE_BF16 && out_type != MLA_DTYPE_FP32 && out_type != MLA_DTYPE_FP16)
    return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  if (!aligned(d_q, 16) || !aligned(d_kv, 16) || !aligned(d_plan, 16) || !aligned(d_workspace, 16) ||
      !aligned(d_out, 16) || !aligned(d_block_table, 4) || !aligned(d_lse, 4) || !aligned(live, 4) || !aligned(d_status, 4))
    return MLA_ERR_INVALID_ARG;
  SharedSizes z;
  int rc = shared_sizes(batch, s_q, h_q, num_parts, &z);
  if (rc != MLA_OK) return rc;
  if (max_pages > kMaxRowPages || static_cast<long long>(batch) * max_pages > kMaxInt ||
      static_cast<long long>(num_pages) * MLA_PAGE_SIZE > kMaxInt)
    return MLA_ERR_UNSUPPORTED;
  if (plan_bytes < z.plan_bytes || workspace_bytes < z.ws_bytes) return MLA_ERR_INVALID_ARG;
  int sms = 0;
  rc = device_ready(&sms);
  if (rc != MLA_OK) return rc;
  const char* plan = static_cast<const char*>(d_plan);
  if (!z.share)
    return decode_full_blocks(d_q, d_kv, d_block_table, max_pages, num_pages,
                              reinterpret_cast<const int32_t*>(plan + z.lengths_off), live, batch, s_q, h_q, dtype, causal,
                              softmax_scale, reinterpret_cast<const int32_t*>(plan + z.sched_off),
                              reinterpret_cast<const int32_t*>(plan + z.offset_off), num_parts, d_workspace,
                              workspace_bytes, d_out, out_type, d_lse, d_status, stall, to_stream(stream));
  SharedLaunch c{};
  c.q = d_q;
  c.kv = d_kv;
  c.total_rows = z.rows;
  c.live = live;
  c.batch = batch;
  c.num_pages = num_pages;
  c.n_units = z.units;
  c.s_q = s_q;
  c.h_q = h_q;
  c.num_parts = num_parts;
  c.max_pages = max_pages;
  c.dtype = dtype;
  c.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  c.block_table = d_block_table;
  c.units = reinterpret_cast<const int32_t*>(plan);
  c.lengths = reinterpret_cast<const int32_t*>(plan + z.lengths_off);
  c.split_offset = reinterpret_cast<const int32_t*>(plan + z.offset_off);
  c.sched = reinterpret_cast<const int32_t*>(plan + z.sched_off);
  c.o_accum = static_cast<float*>(d_workspace);
  c.lse_accum = reinterpret_cast<float*>(static_cast<char*>(d_workspace) + z.lse_off);
  c.status = d_status;
  c.stall = stall;
  const cudaStream_t st = to_stream(stream);
  rc = launch_shared(c, st);
  if (rc != MLA_OK) return rc;
  return launched(launch_shared_combine(c.o_accum, c.lse_accum, c.units, c.split_offset, batch, s_q * h_q, d_out,
                                        out_type, d_lse, sms, st));
}

}  // namespace

extern "C" {

int mla_cache_append(const void* d_c, long long c_stride, const void* d_r, long long r_stride, int in_dtype,
                     int total_tokens, const int32_t* d_cu_seqlens, const int32_t* d_cache_seqlens, int batch,
                     const int32_t* d_block_table, int max_pages, void* d_cache, int cache_dtype, int num_pages,
                     const void* d_norm_weight, float norm_eps, const float* d_cos_sin, int max_pos,
                     int rope_interleaved, const int32_t* d_refcount, int32_t* d_status, mla_stream_t stream) {
  if (!d_cache_seqlens || !d_block_table || !d_cache || !d_status) return MLA_ERR_INVALID_ARG;
  if (total_tokens < 0 || batch < 1 || max_pages < 1 || num_pages < 1) return MLA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!d_c || !d_r)) return MLA_ERR_INVALID_ARG;
  if (in_dtype != MLA_DTYPE_BF16 && in_dtype != MLA_DTYPE_FP16) return MLA_ERR_INVALID_ARG;
  if (cache_dtype != in_dtype && cache_dtype != MLA_DTYPE_FP8_RECORD) return MLA_ERR_INVALID_ARG;
  if (!d_cu_seqlens && total_tokens % batch != 0) return MLA_ERR_INVALID_ARG;
  if (c_stride < 0 || r_stride < 0 || c_stride % 8 != 0 || r_stride % 8 != 0) return MLA_ERR_INVALID_ARG;
  if (d_norm_weight && !(std::isfinite(norm_eps) && norm_eps >= 0.f)) return MLA_ERR_INVALID_ARG;
  if (d_cos_sin && max_pos < 1) return MLA_ERR_INVALID_ARG;
  if (!aligned(d_c, 16) || !aligned(d_r, 16) || !aligned(d_cache, 16) || !aligned(d_norm_weight, 16) ||
      !aligned(d_cos_sin, 16) || !aligned(d_cu_seqlens, 4) || !aligned(d_cache_seqlens, 4) ||
      !aligned(d_block_table, 4) || !aligned(d_refcount, 4) || !aligned(d_status, 4))
    return MLA_ERR_INVALID_ARG;
  if (max_pages > kMaxRowPages || num_pages > (1 << 30) || total_tokens > (1 << 30)) return MLA_ERR_UNSUPPORTED;
  int sms = 0;
  const int rc = device_ready(&sms);
  if (rc != MLA_OK) return rc;
  if (total_tokens == 0) return MLA_OK;
  AppendParams p{};
  p.c = static_cast<const uint16_t*>(d_c);
  p.c_stride = c_stride;
  p.r = static_cast<const uint16_t*>(d_r);
  p.r_stride = r_stride;
  p.total = total_tokens;
  p.batch = batch;
  p.cu = d_cu_seqlens;
  p.seqlens = d_cache_seqlens;
  p.table = d_block_table;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.cache = d_cache;
  p.weight = static_cast<const uint16_t*>(d_norm_weight);
  p.eps = norm_eps;
  p.cos_sin = d_cos_sin;
  p.max_pos = max_pos;
  p.interleaved = rope_interleaved ? 1 : 0;
  p.refcount = d_refcount;
  p.status = d_status;
  return launched(
      launch_append(p, in_dtype == MLA_DTYPE_FP16, cache_dtype == MLA_DTYPE_FP8_RECORD, sms, to_stream(stream)));
}

int mla_cache_grow(int32_t* d_refcount, int num_pages, int32_t* d_block_table, int rows, int max_pages,
                   int32_t* d_seqlens, const int32_t* d_rows, const int32_t* d_new_tokens, int n, int32_t* d_status,
                   mla_stream_t stream) {
  PageState s;
  int sms = 0, rc = page_state(d_refcount, num_pages, d_block_table, rows, max_pages, d_seqlens, d_status, &s);
  if (rc == MLA_OK) rc = check_list(d_rows, d_new_tokens, n);
  if (rc == MLA_OK) rc = device_ready(&sms);
  if (rc != MLA_OK || n == 0) return rc;
  return launched(launch_grow(s, d_rows, d_new_tokens, n, to_stream(stream)));
}

int mla_cache_fork(int32_t* d_refcount, int num_pages, int32_t* d_block_table, int rows, int max_pages,
                   int32_t* d_seqlens, const int32_t* d_parents, const int32_t* d_children, int n, int32_t* d_pairs,
                   int32_t* d_status, mla_stream_t stream) {
  PageState s;
  int sms = 0, rc = page_state(d_refcount, num_pages, d_block_table, rows, max_pages, d_seqlens, d_status, &s);
  if (rc == MLA_OK) rc = check_list(d_parents, d_children, n);
  if (rc == MLA_OK && ((n > 0 && !d_pairs) || !aligned(d_pairs, 8))) rc = MLA_ERR_INVALID_ARG;
  if (rc == MLA_OK) rc = device_ready(&sms);
  if (rc != MLA_OK || n == 0) return rc;
  return launched(launch_fork(s, d_parents, d_children, n, d_pairs, to_stream(stream)));
}

int mla_cache_free(int32_t* d_refcount, int num_pages, int32_t* d_block_table, int rows, int max_pages,
                   int32_t* d_seqlens, const int32_t* d_rows, int n, int32_t* d_status, mla_stream_t stream) {
  PageState s;
  int sms = 0, rc = page_state(d_refcount, num_pages, d_block_table, rows, max_pages, d_seqlens, d_status, &s);
  if (rc == MLA_OK) rc = check_list(d_rows, d_rows, n);
  if (rc == MLA_OK) rc = device_ready(&sms);
  if (rc != MLA_OK || n == 0) return rc;
  return launched(launch_free(s, d_rows, n, to_stream(stream)));
}

size_t mla_cache_compact_workspace_bytes(int num_pages) {
  return num_pages < 1 || num_pages > (1 << 30) ? 0 : compact_workspace_bytes(num_pages);
}

int mla_cache_compact(int32_t* d_refcount, int num_pages, int32_t* d_block_table, int rows, int max_pages,
                      const int32_t* d_seqlens, int32_t* d_pairs, int32_t* d_count, void* d_workspace,
                      size_t workspace_bytes, int32_t* d_status, mla_stream_t stream) {
  PageState s;
  int sms = 0, rc = page_state(d_refcount, num_pages, d_block_table, rows, max_pages,
                               const_cast<int32_t*>(d_seqlens), d_status, &s);
  if (rc != MLA_OK) return rc;
  if (!d_count || !d_workspace || (num_pages > 1 && !d_pairs)) return MLA_ERR_INVALID_ARG;
  if (!aligned(d_pairs, 8) || !aligned(d_count, 4) || !aligned(d_workspace, 16)) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < compact_workspace_bytes(num_pages)) return MLA_ERR_INVALID_ARG;
  rc = device_ready(&sms);
  if (rc != MLA_OK) return rc;
  return launched(launch_compact(s, d_pairs, d_count, d_workspace, to_stream(stream)));
}

int mla_cache_copy_pages(void* d_pool, int layers, long long layer_stride, int num_pages, long long page_bytes,
                         const int32_t* d_pairs, const int32_t* d_count, int n, int32_t* d_status,
                         mla_stream_t stream) {
  if (!d_pool || !d_status || n < 0 || (n > 0 && !d_pairs)) return MLA_ERR_INVALID_ARG;
  if (layers < 1 || num_pages < 1 || page_bytes < 16 || page_bytes % 16 != 0 || layer_stride % 16 != 0)
    return MLA_ERR_INVALID_ARG;
  if (!aligned(d_pool, 16) || !aligned(d_pairs, 8) || !aligned(d_count, 4) || !aligned(d_status, 4))
    return MLA_ERR_INVALID_ARG;
  if (page_bytes > (1LL << 24) || num_pages > (1 << 30) || layers > (1 << 12) || n > (1 << 24))
    return MLA_ERR_UNSUPPORTED;
  if (layers > 1 && layer_stride < page_bytes * num_pages) return MLA_ERR_INVALID_ARG;
  int sms = 0;
  const int rc = serving_device(&sms);
  if (rc != MLA_OK || n == 0) return rc;
  return launched(launch_copy_pages(d_pool, layers, layer_stride, num_pages, page_bytes, d_pairs, d_count, n,
                                    d_status, sms, to_stream(stream)));
}

size_t mla_prompt_plan_bytes(int batch, int total_q) {
  return batch < 1 || total_q < 0 ? 0 : prompt_plan_bytes(batch, total_q);
}

int mla_prompt_get_plan(const int32_t* d_cu_seqlens_q, const int32_t* d_cu_seqlens_k, int batch, int total_q,
                        int total_k, int causal, void* d_plan, size_t plan_bytes, int32_t* d_status,
                        mla_stream_t stream) {
  if (!d_cu_seqlens_q || !d_plan || !d_status || batch < 1 || total_q < 0 || total_k < 0) return MLA_ERR_INVALID_ARG;
  if (!d_cu_seqlens_k && total_k != total_q) return MLA_ERR_INVALID_ARG;
  if (!aligned(d_cu_seqlens_q, 4) || !aligned(d_cu_seqlens_k, 4) || !aligned(d_plan, 16) || !aligned(d_status, 4))
    return MLA_ERR_INVALID_ARG;
  if (total_q > (1 << 30) || total_k > (1 << 30) || batch > (1 << 20)) return MLA_ERR_UNSUPPORTED;
  if (plan_bytes < prompt_plan_bytes(batch, total_q)) return MLA_ERR_INVALID_ARG;
  int sms = 0;
  const int rc = device_ready(&sms);
  if (rc != MLA_OK) return rc;
  return launched(launch_prompt_plan(d_cu_seqlens_q, d_cu_seqlens_k ? d_cu_seqlens_k : d_cu_seqlens_q, batch, total_q,
                                     total_k, causal ? 1 : 0, d_plan, d_status, to_stream(stream)));
}

int mla_prompt_attention_fwd(const void* d_q, long long q_token_stride, long long q_head_stride, const void* d_k,
                             long long k_token_stride, long long k_head_stride, const void* d_v,
                             long long v_token_stride, long long v_head_stride, int dtype, int total_q, int total_k,
                             int batch, int h_q, int h_kv, int d_qk, float softmax_scale, const void* d_plan,
                             size_t plan_bytes, void* d_out, float* d_lse, int32_t* d_status, mla_stream_t stream) {
  return prompt_attention(d_q, q_token_stride, q_head_stride, d_k, k_token_stride, k_head_stride, d_v, v_token_stride,
                          v_head_stride, dtype, total_q, total_k, batch, h_q, h_kv, d_qk, softmax_scale, nullptr,
                          nullptr, d_plan, plan_bytes, d_out, d_lse, d_status, false, stream);
}

int mla_prompt_attention_checked_fwd(const void* d_q, long long q_token_stride, long long q_head_stride,
                                     const void* d_k, long long k_token_stride, long long k_head_stride,
                                     const void* d_v, long long v_token_stride, long long v_head_stride, int dtype,
                                     int total_q, int total_k, int batch, int h_q, int h_kv, int d_qk,
                                     float softmax_scale, const int32_t* d_cu_seqlens_q,
                                     const int32_t* d_cu_seqlens_k, const void* d_plan, size_t plan_bytes,
                                     void* d_out, float* d_lse, int32_t* d_status, mla_stream_t stream) {
  if (!d_cu_seqlens_q || (!d_cu_seqlens_k && total_k != total_q)) return MLA_ERR_INVALID_ARG;
  return prompt_attention(d_q, q_token_stride, q_head_stride, d_k, k_token_stride, k_head_stride, d_v, v_token_stride,
                          v_head_stride, dtype, total_q, total_k, batch, h_q, h_kv, d_qk, softmax_scale,
                          d_cu_seqlens_q, d_cu_seqlens_k ? d_cu_seqlens_k : d_cu_seqlens_q, d_plan, plan_bytes, d_out,
                          d_lse, d_status, false, stream);
}

int mla_test_prompt_timeout(const void* d_q, long long q_token_stride, long long q_head_stride, const void* d_k,
                            long long k_token_stride, long long k_head_stride, const void* d_v,
                            long long v_token_stride, long long v_head_stride, int dtype, int total_q, int total_k,
                            int batch, int h_q, int h_kv, int d_qk, float softmax_scale, const void* d_plan,
                            size_t plan_bytes, void* d_out, float* d_lse, int32_t* d_status, mla_stream_t stream) {
  if (dtype != MLA_DTYPE_BF16 || d_qk != 192) return MLA_ERR_UNSUPPORTED;
  return prompt_attention(d_q, q_token_stride, q_head_stride, d_k, k_token_stride, k_head_stride, d_v, v_token_stride,
                          v_head_stride, dtype, total_q, total_k, batch, h_q, h_kv, d_qk, softmax_scale, nullptr,
                          nullptr, d_plan, plan_bytes, d_out, d_lse, d_status, true, stream);
}

int mla_shared_prefix_num_parts(int batch, int s_q, int h_q) {
  SharedSizes z;
  const int rc = shared_sizes(batch, s_q, h_q, 1, &z);
  if (rc != MLA_OK) return -rc;
  const int parts = mla_num_parts(z.share ? MLA_ROWS_PER_BLOCK : s_q * h_q, 0);
  return parts > kMaxSharedParts ? kMaxSharedParts : parts;
}

size_t mla_shared_prefix_plan_bytes(int batch, int s_q, int h_q, int num_parts) {
  SharedSizes z;
  return shared_sizes(batch, s_q, h_q, num_parts, &z) == MLA_OK ? z.plan_bytes : 0;
}

size_t mla_shared_prefix_workspace_bytes(int batch, int s_q, int h_q, int num_parts) {
  SharedSizes z;
  return shared_sizes(batch, s_q, h_q, num_parts, &z) == MLA_OK ? z.ws_bytes : 0;
}

int mla_shared_prefix_get_plan(const int32_t* d_block_table, int max_pages, const int32_t* d_cache_seqlens, int batch,
                               int s_q, int h_q, int causal, int num_parts, void* d_plan, size_t plan_bytes,
                               mla_stream_t stream) {
  if (!d_block_table || !d_cache_seqlens || !d_plan || max_pages < 1) return MLA_ERR_INVALID_ARG;
  if (!aligned(d_block_table, 4) || !aligned(d_cache_seqlens, 4) || !aligned(d_plan, 16)) return MLA_ERR_INVALID_ARG;
  SharedSizes z;
  int rc = shared_sizes(batch, s_q, h_q, num_parts, &z);
  if (rc != MLA_OK) return rc;
  if (max_pages > kMaxRowPages || static_cast<long long>(batch) * max_pages > kMaxInt) return MLA_ERR_UNSUPPORTED;
  if (plan_bytes < z.plan_bytes) return MLA_ERR_INVALID_ARG;
  int sms = 0;
  rc = device_ready(&sms);
  if (rc != MLA_OK) return rc;
  char* plan = static_cast<char*>(d_plan);
  int32_t* lengths = reinterpret_cast<int32_t*>(plan + z.lengths_off);
  const cudaStream_t st = to_stream(stream);
  rc = z.share ? launched(launch_shared_units(d_block_table, max_pages, d_cache_seqlens, batch, s_q, h_q,
                                              causal ? 1 : 0, reinterpret_cast<int32_t*>(plan), lengths, st))
               : launched(launch_shared_lengths(d_cache_seqlens, batch, lengths, st));
  if (rc != MLA_OK) return rc;
  return launched(launch_plan(lengths, z.units, num_parts, reinterpret_cast<int32_t*>(plan + z.sched_off),
                              reinterpret_cast<int32_t*>(plan + z.offset_off), st));
}

int mla_shared_prefix_decode_fwd(const void* d_q, const void* d_kv, const int32_t* d_block_table, int max_pages,
                                 int num_pages, int batch, int s_q, int h_q, int dtype, int causal,
                                 float softmax_scale, const void* d_plan, size_t plan_bytes, int num_parts,
                                 void* d_workspace, size_t workspace_bytes, void* d_out, int out_type, float* d_lse,
                                 int32_t* d_status, mla_stream_t stream) {
  return shared_decode(d_q, d_kv, d_block_table, max_pages, num_pages, batch, s_q, h_q, dtype, causal, softmax_scale,
                       nullptr, d_plan, plan_bytes, num_parts, d_workspace, workspace_bytes, d_out, out_type, d_lse,
                       d_status, 0, stream);
}

int mla_shared_prefix_decode_checked_fwd(const void* d_q, const void* d_kv, const int32_t* d_block_table,
                                         int max_pages, int num_pages, int batch, int s_q, int h_q, int dtype,
                                         int causal, float softmax_scale, const int32_t* d_cache_seqlens,
                                         const void* d_plan, size_t plan_bytes, int num_parts, void* d_workspace,
                                         size_t workspace_bytes, void* d_out, int out_type, float* d_lse,
                                         int32_t* d_status, mla_stream_t stream) {
  if (!d_cache_seqlens) return MLA_ERR_INVALID_ARG;
  return shared_decode(d_q, d_kv, d_block_table, max_pages, num_pages, batch, s_q, h_q, dtype, causal, softmax_scale,
                       d_cache_seqlens, d_plan, plan_bytes, num_parts, d_workspace, workspace_bytes, d_out, out_type,
                       d_lse, d_status, 0, stream);
}

int mla_test_shared_prefix_timeout(const void* d_q, const void* d_kv, const int32_t* d_block_table, int max_pages,
                                   int num_pages, int batch, int s_q, int h_q, int dtype, int causal,
                                   float softmax_scale, const void* d_plan, size_t plan_bytes, int num_parts,
                                   void* d_workspace, size_t workspace_bytes, void* d_out, int out_type, float* d_lse,
                                   int32_t* d_status, mla_stream_t stream) {
  if (dtype == MLA_DTYPE_FP16) return MLA_ERR_UNSUPPORTED;
  return shared_decode(d_q, d_kv, d_block_table, max_pages, num_pages, batch, s_q, h_q, dtype, causal, softmax_scale,
                       nullptr, d_plan, plan_bytes, num_parts, d_workspace, workspace_bytes, d_out, out_type, d_lse,
                       d_status, 1, stream);
}

int mla_serving_call(int op, const void* args, size_t bytes) {
  constexpr size_t kWords[] = {22, 11, 12, 10, 12, 10, 23, 21, 22, 25};  // by mla_call_t
  if (!args || op < 0 || op > MLA_CALL_PROMPT_CHECKED || bytes != 8 * kWords[op]) return MLA_ERR_INVALID_ARG;
  const char* a = static_cast<const char*>(args);
  auto word = [&](int i) {
    int64_t v;
    std::memcpy(&v, a + 8 * i, 8);
    return v;
  };
  auto I = [&](int i) {  // beyond 32 bits: a number that every size and type refuses
    const int64_t v = word(i);
    return v == static_cast<int>(v) ? static_cast<int>(v) : INT32_MIN;
  };
  auto F = [&](int i) {
    double v;
    std::memcpy(&v, a + 8 * i, 8);
    return static_cast<float>(v);
  };
  auto P = [&](int i) { return reinterpret_cast<void*>(word(i)); };
  auto N = [&](int i) { return static_cast<int32_t*>(P(i)); };
  auto R = [&](int i) { return static_cast<float*>(P(i)); };
  auto S = [&](int i) { return static_cast<mla_stream_t>(P(i)); };
  switch (op) {
    case MLA_CALL_APPEND:
      return mla_cache_append(P(0), word(1), P(2), word(3), I(4), I(5), N(6), N(7), I(8), N(9), I(10), P(11), I(12),
                              I(13), P(14), F(15), R(16), I(17), I(18), N(19), N(20), S(21));
    case MLA_CALL_GROW:
      return mla_cache_grow(N(0), I(1), N(2), I(3), I(4), N(5), N(6), N(7), I(8), N(9), S(10));
    case MLA_CALL_FORK:
      return mla_cache_fork(N(0), I(1), N(2), I(3), I(4), N(5), N(6), N(7), I(8), N(9), N(10), S(11));
    case MLA_CALL_FREE:
      return mla_cache_free(N(0), I(1), N(2), I(3), I(4), N(5), N(6), I(7), N(8), S(9));
    case MLA_CALL_COMPACT:
      return mla_cache_compact(N(0), I(1), N(2), I(3), I(4), N(5), N(6), N(7), P(8), static_cast<size_t>(word(9)),
                               N(10), S(11));
    case MLA_CALL_COPY_PAGES:
      return mla_cache_copy_pages(P(0), I(1), word(2), I(3), word(4), N(5), N(6), I(7), N(8), S(9));
    case MLA_CALL_PROMPT:
      return mla_prompt_attention_fwd(P(0), word(1), word(2), P(3), word(4), word(5), P(6), word(7), word(8), I(9),
                                      I(10), I(11), I(12), I(13), I(14), I(15), F(16), P(17),
                                      static_cast<size_t>(word(18)), P(19), R(20), N(21), S(22));
    case MLA_CALL_SHARED_PREFIX:
      return mla_shared_prefix_decode_fwd(P(0), P(1), N(2), I(3), I(4), I(5), I(6), I(7), I(8), I(9), F(10), P(11),
                                          static_cast<size_t>(word(12)), I(13), P(14), static_cast<size_t>(word(15)),
                                          P(16), I(17), R(18), N(19), S(20));
    case MLA_CALL_SHARED_PREFIX_CHECKED:
      return mla_shared_prefix_decode_checked_fwd(P(0), P(1), N(2), I(3), I(4), I(5), I(6), I(7), I(8), I(9), F(10),
                                                  N(11), P(12), static_cast<size_t>(word(13)), I(14), P(15),
                                                  static_cast<size_t>(word(16)), P(17), I(18), R(19), N(20), S(21));
    case MLA_CALL_PROMPT_CHECKED:
      return mla_prompt_attention_checked_fwd(P(0), word(1), word(2), P(3), word(4), word(5), P(6), word(7), word(8),
                                              I(9), I(10), I(11), I(12), I(13), I(14), I(15), F(16), N(17), N(18),
                                              P(19), static_cast<size_t>(word(20)), P(21), R(22), N(23), S(24));
    default: return MLA_ERR_INVALID_ARG;
  }
}

}  // extern "C"
