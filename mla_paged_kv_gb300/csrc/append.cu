// New tokens' latent rows into the paged cache: RMS norm of the latent part,
// RoPE of the rotary part, and either 16-bit rows or 656-byte FP8 records,
// in one pass.
//
//   c' = c * rsqrt(mean(c^2) + eps) * w,   r' = r rotated by the angle of pos
//   record: scale_g = max|c'_g| / 448, code = e4m3(c' / scale_g), bf16 r'
//
// Memory bound: a token reads 1152 bytes (and 256 of its angles) and writes
// 1152 or 656.  One warp per token: lane l holds columns 8l .. 8l+7 of each
// half of the latent row, so that every load and store of the row is one
// contiguous run over the warp (16 bytes a lane; 8 for codes) and a 128-column
// group is 16 lanes of one half, whose maximum takes four shuffles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "serving.cuh"

namespace mla {
namespace {

constexpr int kAppendWarps = 4;

template <bool kHalf>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (kHalf)
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  else
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

template <bool kHalf>
__device__ __forceinline__ uint32_t pack2f(float a, float b) {
  if constexpr (kHalf) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <bool kHalf>
__device__ __forceinline__ float load1(const uint16_t* p) {
  const uint16_t v = *p;
  if constexpr (kHalf)
    return __half2float(*reinterpret_cast<const __half*>(&v));
  else
    return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(&v));
}

template <bool kHalf>
__device__ __forceinline__ uint16_t round1(float a) {
  return static_cast<uint16_t>(pack2f<kHalf>(a, 0.f) & 0xffffu);
}

// The last request b with cu[b] <= t, by a 32-way search (cu[0] <= t < cu[batch]).
__device__ __forceinline__ int find_request(const int32_t* cu, int batch, int t, int lane) {
  int lo = 0, hi = batch;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;
    const bool below = at < hi && cu[at] <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, below));
    lo += n * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

template <bool kHalf, bool kFp8>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (t >= p.total) return;  // uniform over the warp
  // the token's row does not depend on where it goes: in flight during the search
  const uint16_t* crow = p.c + static_cast<long long>(t) * p.c_stride;
  const uint16_t* rrow = p.r + static_cast<long long>(t) * p.r_stride;
  uint4 raw[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) raw[h] = __ldg(reinterpret_cast<const uint4*>(crow + 256 * h) + lane);
  float rx, ry;
  if (p.interleaved) {
    const float2 v = unpack2<kHalf>(__ldg(reinterpret_cast<const uint32_t*>(rrow) + lane));
    rx = v.x;
    ry = v.y;
  } else {
    rx = load1<kHalf>(rrow + lane);
    ry = load1<kHalf>(rrow + 32 + lane);
  }

  int b, left;  // request, and its new tokens from t on
  if (p.cu == nullptr) {
    const int each = p.total / p.batch;
    b = t / each;
    left = (b + 1) * each - t;
  } else {
    if (t < p.cu[0] || t >= p.cu[p.batch]) return;
    b = find_request(p.cu, p.batch, t, lane);
    left = p.cu[b + 1] - t;
  }
  const int pos = p.seqlens[b] - left;
  int page = -1;
  if (pos >= 0 && pos < p.max_pages * kTile && (p.cos_sin == nullptr || pos < p.max_pos))
    page = p.table[static_cast<long long>(b) * p.max_pages + pos / kTile];
  bool bad = page < 0 || page >= p.num_pages;
  if (!bad && p.refcount != nullptr) bad = p.refcount[page] != 1;
  if (bad) {
    if (lane == 0) report(p.status, MLA_ERR_BAD_INDEX);
    return;
  }
  const long long slot = static_cast<long long>(page) * kTile + pos % kTile;

  float x[2][8];
  float ss = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {raw[h].x, raw[h].y, raw[h].z, raw[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2<kHalf>(w[i]);
      x[h][2 * i] = v.x;
      x[h][2 * i + 1] = v.y;
      ss = fmaf(v.x, v.x, ss);
      ss = fmaf(v.y, v.y, ss);
    }
  }
  if (p.weight != nullptr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float rstd = 1.f / sqrtf(ss * (1.f / kDv) + p.eps);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 wv = __ldg(reinterpret_cast<const uint4*>(p.weight + 256 * h) + lane);
      const uint32_t w[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 g = unpack2<kHalf>(w[i]);
        x[h][2 * i] = x[h][2 * i] * rstd * g.x;
        x[h][2 * i + 1] = x[h][2 * i + 1] * rstd * g.y;
      }
    }
  }
  if (p.cos_sin != nullptr) {
    const float c = __ldg(p.cos_sin + static_cast<long long>(pos) * 64 + lane);
    const float s = __ldg(p.cos_sin + static_cast<long long>(pos) * 64 + 32 + lane);
    const float a = rx * c - ry * s, e = ry * c + rx * s;
    rx = a;
    ry = e;
  }

  uint16_t* rope_out;
  if constexpr (kFp8) {
    uint8_t* rec = static_cast<uint8_t*>(p.cache) + slot * MLA_RECORD_BYTES;
    float* scales = reinterpret_cast<float*>(rec + 512);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[h][i]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float scale = top > 0.f ? top / 448.f : 1.f;
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[h][4 * i] / scale, x[h][4 * i + 1] / scale),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[h][4 * i + 2] / scale, x[h][4 * i + 3] / scale),
                                                     __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
      }
      *reinterpret_cast<uint2*>(rec + 256 * h + 8 * lane) = make_uint2(w[0], w[1]);
      if ((lane & 15) == 0) scales[2 * h + (lane >> 4)] = scale;
    }
    rope_out = reinterpret_cast<uint16_t*>(rec + 528);
  } else {
    uint16_t* row = static_cast<uint16_t*>(p.cache) + slot * kDqk;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *(reinterpret_cast<uint4*>(row + 256 * h) + lane) =
          make_uint4(pack2f<kHalf>(x[h][0], x[h][1]), pack2f<kHalf>(x[h][2], x[h][3]),
                     pack2f<kHalf>(x[h][4], x[h][5]), pack2f<kHalf>(x[h][6], x[h][7]));
    rope_out = row + kDv;
  }
  constexpr bool kRopeHalf = kHalf && !kFp8;  // a record's RoPE part is bf16
  if (p.interleaved) {
    reinterpret_cast<uint32_t*>(rope_out)[lane] = pack2f<kRopeHalf>(rx, ry);
  } else {
    rope_out[lane] = round1<kRopeHalf>(rx);
    rope_out[32 + lane] = round1<kRopeHalf>(ry);
  }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, bool half, bool fp8, cudaStream_t stream) {
  const int grid = ceil_div_i(p.total, kAppendWarps);
  if (half) {
    if (fp8)
      append_kernel<true, true><<<grid, 32 * kAppendWarps, 0, stream>>>(p);
    else
      append_kernel<true, false><<<grid, 32 * kAppendWarps, 0, stream>>>(p);
  } else {
    if (fp8)
      append_kernel<false, true><<<grid, 32 * kAppendWarps, 0, stream>>>(p);
    else
      append_kernel<false, false><<<grid, 32 * kAppendWarps, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace mla
