// Rows of a paged latent cache as packed rows: what cache_append wrote, read
// back.  16-bit rows are copied, FP8 records become bf16 rows (code x scale in
// fp32, rounded once; the RoPE part as it is).
//
// Memory bound: a row reads 1152 bytes (a record 656) and writes 1152.  A warp
// takes kRows consecutive rows, whose targets lanes 0 .. kRows - 1 find together,
// so that the chain of small loads (offsets, start, block table) runs once for
// them, and all loads of the rows are in flight before the first store.  24577 rows of
// records 8.4 us (5.3 TB/s; with a row a warp 10.3), 49153 of bf16 16.7 (6.7 TB/s, what
// a copy reaches here), up to 2400 of either 4.2 (a launch).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "serving.cuh"

namespace mla {
namespace {

constexpr int kGatherWarps = 4, kRows = 4;

// Slot of packed row t, or -1: of no sequence, or refused and reported.
__device__ __forceinline__ long long row_slot(const GatherParams& p, int t, int b) {
  const long long pos = static_cast<long long>(p.starts != nullptr ? p.starts[b] : 0) + t - p.cu[b];
  int page = -1;
  if (pos >= 0 && pos < static_cast<long long>(p.max_pages) * kTile)
    page = p.table[static_cast<long long>(b) * p.max_pages + pos / kTile];
  if (page < 0 || page >= p.num_pages) {
    report(p.status, MLA_ERR_BAD_INDEX);
    return -1;
  }
  return static_cast<long long>(page) * kTile + pos % kTile;
}

// Two E4M3 codes times a scale, as a pair of bf16.
__device__ __forceinline__ uint32_t codes2(uint32_t two, float scale) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));  // (every E4M3 value is an fp16 value)
  const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * scale, f.y * scale);
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <bool kFp8>
__global__ void __launch_bounds__(32 * kGatherWarps) gather_kernel(const GatherParams p) {
  const int lane = threadIdx.x & 31;
  const int t0 = (blockIdx.x * kGatherWarps + (threadIdx.x >> 5)) * kRows;
  if (t0 >= p.total) return;  // uniform over the warp
  const int first = p.cu[0], last = p.cu[p.batch];
  if (t0 + kRows - 1 < first || t0 >= last) return;
  long long mine = -1;
  {
    // the request of the first row that has one, by a 32-way search, then on from there
    const int from = max(t0, first);
    int lo = 0, hi = p.batch;  // cu[lo] <= from < cu[hi]
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
      const int n = __popc(__ballot_sync(0xffffffffu, at < hi && p.cu[at] <= from));
      lo += n * step;
      hi = min(lo + step, hi);
    }
    const int t = t0 + lane;
    if (lane < kRows && t >= first && t < min(last, p.total)) {
      int b = lo;
      while (p.cu[b + 1] <= t) ++b;
      mine = row_slot(p, t, b);
    }
  }
  long long slot[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) slot[i] = __shfl_sync(0xffffffffu, mine, i);
  uint16_t* out = p.out + t0 * p.out_stride;
  if constexpr (kFp8) {
    uint2 code[kRows][2];
    float scale[kRows][2];
    uint4 rope[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (slot[i] < 0) continue;
      const uint8_t* rec = static_cast<const uint8_t*>(p.cache) + slot[i] * MLA_RECORD_BYTES;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        code[i][h] = __ldcs(reinterpret_cast<const uint2*>(rec + 256 * h) + lane);
        scale[i][h] = __ldcs(reinterpret_cast<const float*>(rec + 512) + 2 * h + (lane >> 4));
      }
      if (lane < 8) rope[i] = __ldcs(reinterpret_cast<const uint4*>(rec + 528) + lane);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (slot[i] < 0) continue;
      uint4* row = reinterpret_cast<uint4*>(out + i * p.out_stride);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 c = code[i][h];
        const float s = scale[i][h];
        row[32 * h + lane] = make_uint4(codes2(c.x & 0xffffu, s), codes2(c.x >> 16, s), codes2(c.y & 0xffffu, s),
                                        codes2(c.y >> 16, s));
      }
      if (lane < 8) row[64 + lane] = rope[i];
    }
  } else {
    uint4 v[kRows][3];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (slot[i] < 0) continue;
      const uint4* row = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.cache) + slot[i] * kDqk);
      v[i][0] = __ldcs(row + lane);
      v[i][1] = __ldcs(row + 32 + lane);
      if (lane < 8) v[i][2] = __ldcs(row + 64 + lane);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (slot[i] < 0) continue;
      uint4* row = reinterpret_cast<uint4*>(out + i * p.out_stride);
      row[lane] = v[i][0];
      row[32 + lane] = v[i][1];
      if (lane < 8) row[64 + lane] = v[i][2];
    }
  }
}

}  // namespace

cudaError_t launch_gather(const GatherParams& p, bool fp8, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>((p.total + kGatherWarps * kRows - 1ll) / (kGatherWarps * kRows));
  if (fp8)
    gather_kernel<true><<<grid, 32 * kGatherWarps, 0, st>>>(p);
  else
    gather_kernel<false><<<grid, 32 * kGatherWarps, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
