// Decode for a batch that shares its first pages: the plan's units and the
// combine (the attention itself is the dense decode kernel over those units).
//
//   out = sum over prefix keys and own keys of softmax(s) v, in two kinds of
//   units: all requests' query rows, 128 at a time, over the shared pages, and
//   each request's rows over its own.  Every (unit, split) leaves O / l and its
//   LSE; a row merges the splits of its prefix unit and of its own unit:
//   out = sum_s e^(lse_s - m) O_s / Z, lse = m + ln Z, Z = sum_s e^(lse_s - m).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "ptx.cuh"
#include "serving.cuh"

namespace mla {
namespace {

constexpr int kRB = kRowsPerBlock;

// Ints of a unit's entry behind SharedUnit's: an own unit's, 1 where it holds
// all of the request's keys.
constexpr int kAlone = 5;

// Keys that the first of a request's queries sees.  Less than a page shares
// nothing: such a request (an empty slot of a padded batch, say) stands apart
// and the others share without it.
__device__ __forceinline__ int keys_seen(const int32_t* seqlens, int b, int s_q, int causal) {
  return max(seqlens[b], 0) - (causal ? s_q - 1 : 0);
}

// The pages every request that sees one starts with (the longest common run of
// block-table entries, whole pages that every query sees), and the units over
// them and over the rest.  A single request shares with none, and a row block
// whose requests all stand apart (the empty slots at the end of a padded batch)
// has no keys.  One block, made once for a batch; its time is the
// latency of reading the tables (64 requests that share 2048 pages 9.8 us, with
// one entry a lane in flight 29).
__global__ void __launch_bounds__(1024)
    shared_units_kernel(const int32_t* table, int max_pages, const int32_t* seqlens, int batch, int s_q, int h_q,
                        int causal, int32_t* units, int32_t* lengths) {
  __shared__ int common, first, last;  // pages in common; the first and the last request that take part
  if (threadIdx.x == 0) common = max_pages, first = batch, last = -1;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kAhead = 8;  // entries a lane has in flight: the loop is their latency
  for (int b = threadIdx.x; b < batch; b += 1024) {
    const int seen = keys_seen(seqlens, b, s_q, causal);
    if (seen >= kTile) {
      atomicMin(&common, seen / kTile);
      atomicMin(&first, b);
      atomicMax(&last, b);
    }
  }
  __syncthreads();
  const bool none = first == batch;
  const int ref = none ? 0 : first;
  const int32_t* head = table + static_cast<long long>(ref) * max_pages;
  for (int b = ref + 1 + warp; b < batch; b += 32) {
    if (keys_seen(seqlens, b, s_q, causal) < kTile) continue;
    const int32_t* row = table + static_cast<long long>(b) * max_pages;
    const int most = *reinterpret_cast<volatile int*>(&common);
    int at = max_pages;  // the lane's first entry that differs
    for (int c0 = 0; c0 < most && at == max_pages; c0 += 32 * kAhead) {
      int a[kAhead], h[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int c = c0 + 32 * i + lane;
        a[i] = c < most ? row[c] : 0;
        h[i] = c < most ? head[c] : 0;
      }
#pragma unroll
      for (int i = kAhead - 1; i >= 0; --i)
        if (a[i] != h[i]) at = c0 + 32 * i + lane;
      at = __reduce_min_sync(0xffffffffu, at);
    }
    if (lane == 0 && at < max_pages) atomicMin(&common, at);
  }
  __syncthreads();
  const int shared = first < last ? common : 0;
  const int rows = s_q * h_q;
  const long long total = static_cast<long long>(batch) * rows;
  const int front = static_cast<int>((total + kRB - 1) / kRB), per = ceil_div_i(rows, kRB);
  for (int u = threadIdx.x; u < front + batch * per; u += 1024) {
    int4* e = reinterpret_cast<int4*>(units + u * kUnitInts);
    if (u < front) {
      const int row0 = u * kRB;
      e[0] = make_int4(row0, static_cast<int>(min(total - row0, static_cast<long long>(kRB))), -1,
                       ref * max_pages);
      e[1] = make_int4(max_pages, 0, 0, 0);
      int b = row0 / rows;
      const int end = static_cast<int>((min(total, static_cast<long long>(row0) + kRB) - 1) / rows);
      while (b < end && keys_seen(seqlens, b, s_q, causal) < kTile) ++b;
      lengths[u] = keys_seen(seqlens, b, s_q, causal) < kTile ? 0 : shared * kTile;
    } else {
      const int b = (u - front) / per, blk = (u - front) - b * per;
      const int rel = blk * kRB;
      const bool alone = keys_seen(seqlens, b, s_q, causal) < kTile;
      const int skip = alone ? 0 : shared;
      e[0] = make_int4(b * rows + rel, min(rows - rel, kRB), causal ? rel : -1, b * max_pages + skip);
      e[1] = make_int4(max_pages - skip, alone ? 1 : 0, 0, 0);
      lengths[u] = max(seqlens[b], 0) - skip * kTile;
    }
  }
}

// Where nothing is attended together the plan keeps the lengths as they are.
__global__ void __launch_bounds__(256) shared_lengths_kernel(const int32_t* seqlens, int batch, int32_t* lengths) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b < batch) lengths[b] = seqlens[b];
}

__device__ __forceinline__ void store4(void* out, int out_type, size_t elem, float4 v) {
  if (out_type == MLA_DTYPE_FP32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + elem) = v;
    return;
  }
  uint2 w;
  if (out_type == MLA_DTYPE_FP16) {
    const __half2 lo = __floats2half2_rn(v.x, v.y), hi = __floats2half2_rn(v.z, v.w);
    w.x = *reinterpret_cast<const uint32_t*>(&lo);
    w.y = *reinterpret_cast<const uint32_t*>(&hi);
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    w.x = *reinterpret_cast<const uint32_t*>(&lo);
    w.y = *reinterpret_cast<const uint32_t*>(&hi);
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + elem) = w;
}

// What a row merges: the splits of its prefix unit (if the request takes part in
// it), then those of its own unit.
struct RowSplits {
  int p0, np, o0, n;  // prefix: slots p0 .. p0 + np - 1; own: o0 .. o0 + n - np - 1
  int pr, orow;       // the row within either unit

  // Row of split i among all slots' 128 rows.
  __device__ __forceinline__ size_t at(int i) const {
    return i < np ? static_cast<size_t>(p0 + i) * kRB + pr : static_cast<size_t>(o0 + i - np) * kRB + orow;
  }
};

__device__ __forceinline__ RowSplits row_splits(const int32_t* units, const int32_t* split_offset, int batch,
                                                int rows, long long g) {
  const int b = static_cast<int>(g / rows), r = static_cast<int>(g - static_cast<long long>(b) * rows);
  const int front = static_cast<int>((static_cast<long long>(batch) * rows + kRB - 1) / kRB);
  const int own = front + b * ceil_div_i(rows, kRB) + r / kRB;
  const int pre = static_cast<int>(g / kRB);
  RowSplits s;
  s.p0 = split_offset[pre];
  s.np = units[own * kUnitInts + kAlone] ? 0 : split_offset[pre + 1] - s.p0;
  s.o0 = split_offset[own];
  s.n = s.np + split_offset[own + 1] - s.o0;
  s.pr = static_cast<int>(g % kRB);
  s.orow = r % kRB;
  return s;
}

__device__ __forceinline__ void add4(float4& acc, float w, const float4& v) {
  if (w != 0.f) {  // an empty split weighs 0 whatever its partial holds
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
}

// Many rows: a warp merges 128 columns of a row (four a lane).  The lanes hold
// the splits' LSEs, 32 at a time; the partials of eight splits are in flight at
// once.  No shared memory, so the blocks are resident beside the attention
// kernel's CTAs and start as it ends.  Bound by the partials' bytes.
__global__ void __launch_bounds__(128)
    shared_combine_rows_kernel(const float* __restrict__ o_accum, const float* __restrict__ lse_accum,
                               const int32_t* __restrict__ units, const int32_t* __restrict__ split_offset, int batch,
                               int rows, void* __restrict__ out, int out_type, float* __restrict__ lse) {
  constexpr int kBatch = 8;
  const long long g = blockIdx.x;
  const int lane = threadIdx.x & 31, col = 4 * threadIdx.x;
  const RowSplits s = row_splits(units, split_offset, batch, rows, g);  // the plan's: read before the wait
  pdl_wait_prior_grid();
  const float l0 = lane < s.n ? lse_accum[s.at(lane)] : -INFINITY;
  float m = l0;
  for (int i = 32 + lane; i < s.n; i += 32) m = fmaxf(m, lse_accum[s.at(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float z = 0.f;
  for (int c0 = 0; c0 < s.n; c0 += 32) {
    const int cnt = min(32, s.n - c0);
    float l = l0;
    if (c0 > 0) l = lane < cnt ? lse_accum[s.at(c0 + lane)] : -INFINITY;
    const float w = l == -INFINITY ? 0.f : expf(l - m);
    z += w;
    for (int j = 0; j < cnt; j += kBatch) {
      float4 v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        v[k] = j + k < cnt ? __ldg(reinterpret_cast<const float4*>(o_accum + s.at(c0 + j + k) * kDv + col))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) add4(acc, __shfl_sync(0xffffffffu, w, (j + k) & 31), v[k]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  const float inv = z > 0.f ? 1.f / z : 0.f;
  acc.x *= inv;
  acc.y *= inv;
  acc.z *= inv;
  acc.w *= inv;
  store4(out, out_type, static_cast<size_t>(g) * kDv + col, acc);
  if (threadIdx.x == 0) lse[g] = z > 0.f ? m + logf(z) : -INFINITY;
}

// Few rows: a block per row, eight warps to each 128 columns, every eighth
// split each; merged through shared memory.  Bound by the latency of dozens of
// splits.
constexpr int kGroups = 8;
__global__ void __launch_bounds__(128 * kGroups)
    shared_combine_splits_kernel(const float* __restrict__ o_accum, const float* __restrict__ lse_accum,
                                 const int32_t* __restrict__ units, const int32_t* __restrict__ split_offset,
                                 int batch, int rows, void* __restrict__ out, int out_type,
                                 float* __restrict__ lse) {
  constexpr int kBatch = 4;
  __shared__ float part_m[kGroups][4], part_z[kGroups][4];
  __shared__ float4 part[kGroups][128];
  const long long g = blockIdx.x;
  const int grp = threadIdx.x >> 7, tid = threadIdx.x & 127, quarter = tid >> 5;
  const int col = 4 * tid;
  const RowSplits s = row_splits(units, split_offset, batch, rows, g);
  pdl_wait_prior_grid();
  float m = -INFINITY, z = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = grp; i < s.n; i += kBatch * kGroups) {
    float4 v[kBatch];
    float l[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int si = i + k * kGroups;
      l[k] = si < s.n ? lse_accum[s.at(si)] : -INFINITY;
      v[k] = si < s.n ? __ldg(reinterpret_cast<const float4*>(o_accum + s.at(si) * kDv + col))
                      : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mb = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) mb = fmaxf(mb, l[k]);
    if (mb == -INFINITY) continue;  // nothing but empty splits so far
    const float r = m == -INFINITY ? 0.f : expf(m - mb);
    z *= r;
    acc.x *= r;
    acc.y *= r;
    acc.z *= r;
    acc.w *= r;
    m = mb;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float w = l[k] == -INFINITY ? 0.f : expf(l[k] - m);
      z += w;
      add4(acc, w, v[k]);
    }
  }
  part[grp][tid] = acc;
  if ((tid & 31) == 0) {
    part_m[grp][quarter] = m;
    part_z[grp][quarter] = z;
  }
  __syncthreads();
  if (grp > 0) return;
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) top = fmaxf(top, part_m[k][quarter]);
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = 0.f;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const float mk = part_m[k][quarter];
    const float r = mk == -INFINITY ? 0.f : expf(mk - top);
    total = fmaf(part_z[k][quarter], r, total);
    add4(t, r, part[k][tid]);
  }
  const float inv = total > 0.f ? 1.f / total : 0.f;
  store4(out, out_type, static_cast<size_t>(g) * kDv + col, make_float4(t.x * inv, t.y * inv, t.z * inv, t.w * inv));
  if (tid == 0) lse[g] = total > 0.f ? top + logf(total) : -INFINITY;
}

}  // namespace

cudaError_t launch_shared_units(const int32_t* block_table, int max_pages, const int32_t* seqlens, int batch,
                                int s_q, int h_q, int causal, int32_t* units, int32_t* lengths,
                                cudaStream_t st) {
  shared_units_kernel<<<1, 1024, 0, st>>>(block_table, max_pages, seqlens, batch, s_q, h_q, causal, units, lengths);
  return cudaGetLastError();
}

cudaError_t launch_shared_lengths(const int32_t* seqlens, int batch, int32_t* lengths, cudaStream_t st) {
  shared_lengths_kernel<<<ceil_div_i(batch, 256), 256, 0, st>>>(seqlens, batch, lengths);
  return cudaGetLastError();
}

cudaError_t launch_shared_combine(const float* o_accum, const float* lse_accum, const int32_t* units,
                                  const int32_t* split_offset, int batch, int rows, void* out, int out_type,
                                  float* lse, int sms, cudaStream_t st) {
  const long long total = static_cast<long long>(batch) * rows;
  // A block of eight groups hides the latency of its splits, 128 threads a row
  // leave more rows resident.  Whole calls with 16 heads, groups and rows, over
  // 1024 / 16384 shared keys: 128 rows 14.3 and 18.9 / 20.6 and 36.3 us, 256 17.2
  // and 18.0 / 26.1 and 30.1, 384 20.5 and 18.3 / 32.3 and 31.9, 1024 32.6 and
  // 23.2 / 60.2 and 49.0.
  const bool few = total <= 2ll * sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(total), 1, 1);
  cfg.blockDim = dim3(few ? 128 * kGroups : 128, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (few)
    return cudaLaunchKernelEx(&cfg, shared_combine_splits_kernel, o_accum, lse_accum, units, split_offset, batch, rows,
                              out, out_type, lse);
  return cudaLaunchKernelEx(&cfg, shared_combine_rows_kernel, o_accum, lse_accum, units, split_offset, batch, rows,
                            out, out_type, lse);
}

}  // namespace mla
