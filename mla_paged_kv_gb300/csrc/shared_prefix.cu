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

// The pages every request starts with (the longest common run of block-table
// entries, whole pages that every query sees), and the units over them and
// over the rest.  One block; made once for a batch.
__global__ void __launch_bounds__(1024)
    shared_units_kernel(const int32_t* table, int max_pages, const int32_t* seqlens, int batch, int s_q, int h_q,
                        int causal, int share, int32_t* units, int32_t* lengths) {
  __shared__ int common;
  if (threadIdx.x == 0) common = share ? max_pages : 0;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (share) {
    for (int b = threadIdx.x; b < batch; b += 1024) {
      const int seen = max(seqlens[b], 0) - (causal ? s_q - 1 : 0);  // keys the first query sees
      atomicMin(&common, max(seen, 0) / kTile);
    }
    __syncthreads();
    for (int b = 1 + warp; b < batch; b += 32) {
      const int32_t* row = table + static_cast<long long>(b) * max_pages;
      const int most = *reinterpret_cast<volatile int*>(&common);
      for (int c0 = 0; c0 < most; c0 += 32) {
        const int c = c0 + lane;
        const unsigned diff = __ballot_sync(0xffffffffu, c < most && row[c] != table[c]);
        if (diff) {
          if (lane == 0) atomicMin(&common, c0 + __ffs(diff) - 1);
          break;
        }
      }
    }
  }
  __syncthreads();
  const int shared = common;
  const int rows = s_q * h_q;
  const long long total = static_cast<long long>(batch) * rows;
  const int front = share ? static_cast<int>((total + kRB - 1) / kRB) : 0, per = ceil_div_i(rows, kRB);
  for (int u = threadIdx.x; u < front + batch * per; u += 1024) {
    int4* e = reinterpret_cast<int4*>(units + u * kUnitInts);
    if (u < front) {
      const int row0 = u * kRB;
      e[0] = make_int4(row0, static_cast<int>(min(total - row0, static_cast<long long>(kRB))), -1, 0);
      e[1] = make_int4(max_pages, 0, 0, 0);
      lengths[u] = shared * kTile;
    } else {
      const int b = (u - front) / per, blk = (u - front) - b * per;
      const int rel = blk * kRB;
      e[0] = make_int4(b * rows + rel, min(rows - rel, kRB), causal ? rel : -1, b * max_pages + shared);
      e[1] = make_int4(max_pages - shared, 0, 0, 0);
      lengths[u] = max(seqlens[b], 0) - shared * kTile;
    }
  }
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

// One block per query row; kGroups groups of 128 threads take every kGroups-th
// split (four columns a thread), merged through shared memory.  Bound by the
// partials' bytes where there are many rows (kGroups = 1), by the latency of
// dozens of splits where there are few (kGroups = 8).
template <int kGroups>
__global__ void __launch_bounds__(128 * kGroups)
    shared_combine_kernel(const float* __restrict__ o_accum, const float* __restrict__ lse_accum,
                          const int32_t* __restrict__ split_offset, int batch, int rows, int share,
                          void* __restrict__ out, int out_type, float* __restrict__ lse) {
  constexpr int kBatch = 4;
  __shared__ float weight[2 * kMaxSharedParts];
  __shared__ float red[kGroups * 4 + 1];
  __shared__ float4 part[kGroups > 1 ? kGroups - 1 : 1][128];
  const long long g = blockIdx.x;  // query row of batch * rows
  const int b = static_cast<int>(g / rows), r = static_cast<int>(g - static_cast<long long>(b) * rows);
  const int front = share ? static_cast<int>((static_cast<long long>(batch) * rows + kRB - 1) / kRB) : 0;
  const int own = front + b * ceil_div_i(rows, kRB) + r / kRB;
  const int pre = static_cast<int>(g / kRB);
  // the plan is complete long before: its offsets are read before the wait
  const int p0 = share ? split_offset[pre] : 0;
  const int np = share ? split_offset[pre + 1] - p0 : 0;
  const int o0 = split_offset[own];
  const int n = np + split_offset[own + 1] - o0;
  const int pr = static_cast<int>(g % kRB), orow = r % kRB;
  // row of split i: its slot's 128 rows, then the unit's row
  auto slot_row = [&](int i) {
    return i < np ? static_cast<size_t>(p0 + i) * kRB + pr : static_cast<size_t>(o0 + i - np) * kRB + orow;
  };
  pdl_wait_prior_grid();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float m = -INFINITY;
  for (int i = tid; i < n; i += 128 * kGroups) {
    const float l = lse_accum[slot_row(i)];
    weight[i] = l;
    m = fmaxf(m, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int w = 1; w < 4 * kGroups; ++w) m = fmaxf(m, red[w]);
  // the sum in split order, the same in every thread
  float z = 0.f;
  for (int i = 0; i < n; ++i) {
    const float l = weight[i];
    z += l == -INFINITY ? 0.f : expf(l - m);
  }
  const float inv_z = z > 0.f ? 1.f / z : 0.f;
  const int col = 4 * (tid & 127), grp = tid >> 7;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int i, const float4& v) {
    const float l = weight[i];
    const float w = l == -INFINITY ? 0.f : expf(l - m) * inv_z;
    if (w != 0.f) {  // an empty split weighs 0 whatever its partial holds
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
  };
  int i = grp;
  for (; i + (kBatch - 1) * kGroups < n; i += kBatch * kGroups) {
    float4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      v[k] = __ldg(reinterpret_cast<const float4*>(o_accum + slot_row(i + k * kGroups) * kDv + col));
#pragma unroll
    for (int k = 0; k < kBatch; ++k) add(i + k * kGroups, v[k]);
  }
  for (; i < n; i += kGroups) add(i, __ldg(reinterpret_cast<const float4*>(o_accum + slot_row(i) * kDv + col)));
  if constexpr (kGroups > 1) {
    if (grp > 0) part[grp - 1][tid & 127] = acc;
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int k = 0; k < kGroups - 1; ++k) {
      const float4 v = part[k][tid];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
  }
  store4(out, out_type, static_cast<size_t>(g) * kDv + col, acc);
  if (tid == 0) lse[g] = z > 0.f ? m + logf(z) : -INFINITY;
}

}  // namespace

cudaError_t launch_shared_units(const int32_t* block_table, int max_pages, const int32_t* seqlens, int batch,
                                int s_q, int h_q, int causal, int share, int32_t* units, int32_t* lengths,
                                cudaStream_t st) {
  shared_units_kernel<<<1, 1024, 0, st>>>(block_table, max_pages, seqlens, batch, s_q, h_q, causal, share, units,
                                          lengths);
  return cudaGetLastError();
}

cudaError_t launch_shared_combine(const float* o_accum, const float* lse_accum, const int32_t* split_offset,
                                  int batch, int rows, int share, void* out, int out_type, float* lse, int sms,
                                  cudaStream_t st) {
  const long long total = static_cast<long long>(batch) * rows;
  const bool few = total < 4ll * sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(total), 1, 1);
  cfg.blockDim = dim3(few ? 1024 : 128, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (few)
    return cudaLaunchKernelEx(&cfg, shared_combine_kernel<8>, o_accum, lse_accum, split_offset, batch, rows, share,
                              out, out_type, lse);
  return cudaLaunchKernelEx(&cfg, shared_combine_kernel<1>, o_accum, lse_accum, split_offset, batch, rows, share, out,
                            out_type, lse);
}

}  // namespace mla
