// New tokens' latent rows into the paged cache: RMS norm of the latent part,
// RoPE of the rotary part, and either 16-bit rows or 656-byte FP8 records,
// in one pass.
//
//   c' = c * rsqrt(mean(c^2) + eps) * w,   r' = r rotated by the angle of pos
//   record: scale_g = max|c'_g| / 448, code = e4m3(c' / scale_g), bf16 r'
//
// Memory bound: a token reads 1152 bytes (and 256 of its angles) and writes
// 1152 or 656.  A warp holds a token (two, one after the other, in larger
// calls): lane l has columns 8l .. 8l+7 of each half of the latent row, so that
// every load and store of the row is one contiguous run over the warp (16 bytes
// a lane; 8 for codes) and a 128-column group is 16 lanes of one half, whose
// maximum takes four shuffles.
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

// Where token t goes: its slot and position, or slot -1 (outside every
// sequence, or refused and reported).
struct Target {
  long long slot;
  int pos;
};

__device__ __forceinline__ Target find_target(const AppendParams& p, int t, int b, int left) {
  const int pos = p.seqlens[b] - left;
  int page = -1;
  if (pos >= 0 && pos < p.max_pages * kTile && (p.cos_sin == nullptr || pos < p.max_pos))
    page = p.table[static_cast<long long>(b) * p.max_pages + pos / kTile];
  bool bad = page < 0 || page >= p.num_pages;
  if (!bad && p.refcount != nullptr) bad = p.refcount[page] != 1;
  if (bad) {
    report(p.status, MLA_ERR_BAD_INDEX);
    return Target{-1, 0};
  }
  return Target{static_cast<long long>(page) * kTile + pos % kTile, pos};
}

// A warp takes kTokens consecutive tokens: their rows are all in flight before
// the first is needed, and the chain of small loads that finds the targets
// (offsets, length, block table) runs once, lane i for token i.
template <bool kHalf, bool kFp8, int kTokens>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int t0 = (blockIdx.x * kAppendWarps + (threadIdx.x >> 5)) * kTokens;
  if (t0 >= p.total) return;  // uniform over the warp
  uint4 raw[kTokens][2];
  uint32_t rope[kTokens];  // this lane's pair
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int t = min(t0 + i, p.total - 1);
    const uint16_t* crow = p.c + static_cast<long long>(t) * p.c_stride;
    const uint16_t* rrow = p.r + static_cast<long long>(t) * p.r_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h) raw[i][h] = __ldcs(reinterpret_cast<const uint4*>(crow + 256 * h) + lane);
    if (p.interleaved)
      rope[i] = __ldcs(reinterpret_cast<const uint32_t*>(rrow) + lane);
    else
      rope[i] = __ldcs(rrow + lane) | (static_cast<uint32_t>(__ldcs(rrow + 32 + lane)) << 16);
  }
  uint4 gain[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    gain[h] = p.weight != nullptr ? __ldg(reinterpret_cast<const uint4*>(p.weight + 256 * h) + lane)
                                  : make_uint4(0u, 0u, 0u, 0u);

  // lane i: token t0 + i
  Target mine{-1, 0};
  {
    const int t = t0 + lane;
    const bool is_mine = lane < kTokens && t < p.total;
    if (p.cu == nullptr) {
      const int each = p.total / p.batch;
      if (is_mine) {
        const int b = t / each;
        mine = find_target(p, t, b, (b + 1) * each - t);
      }
    } else if (t0 + kTokens - 1 >= p.cu[0] && t0 < p.cu[p.batch]) {
      // the request of the first token that has one, then on from there
      const int first = p.cu[0], last = p.cu[p.batch];
      int b = find_request(p.cu, p.batch, max(t0, first), lane);
      if (is_mine && t >= first && t < last) {
        while (p.cu[b + 1] <= t) ++b;
        mine = find_target(p, t, b, p.cu[b + 1] - t);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const long long slot = __shfl_sync(0xffffffffu, mine.slot, i);
    const int pos = __shfl_sync(0xffffffffu, mine.pos, i);
    if (slot < 0) continue;
    float x[2][8];
    float ss = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w[4] = {raw[i][h].x, raw[i][h].y, raw[i][h].z, raw[i][h].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = unpack2<kHalf>(w[k]);
        x[h][2 * k] = v.x;
        x[h][2 * k + 1] = v.y;
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
        const uint32_t w[4] = {gain[h].x, gain[h].y, gain[h].z, gain[h].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 g = unpack2<kHalf>(w[k]);
          x[h][2 * k] = x[h][2 * k] * rstd * g.x;
          x[h][2 * k + 1] = x[h][2 * k + 1] * rstd * g.y;
        }
      }
    }
    const float2 pair = unpack2<kHalf>(rope[i]);
    float rx = pair.x, ry = pair.y;
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
        for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[h][k]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float scale = top / 448.f;
        if (!(scale > 0.f)) scale = 1.f;  // (all zero, or below the smallest number times 448)
        // c' / scale, with one division a group: q = c' * (1 / scale) is off by at
        // most 2 units of its 24 bits, and q + (c' - q scale) (1 / scale), the
        // difference exact in an FMA (P. Markstein, IBM J. Res. Dev. 34, 1990), by
        // 2^-46 of the quotient before its rounding: at the ties of E4M3, where q alone
        // takes the other neighbour now and then, it is the quotient.  (24577
        // tokens back to back in L2: 12.7 us, with q alone 11.9, with sixteen
        // divisions a lane 15.1; from HBM 13.1 either of the first two.)  Tiny groups and
        // their scale both by 2^64 before it, where 1 / scale would be infinite; a
        // scale of infinity divides to zeros.
        float den = scale;
        if (scale < 0x1p-64f) {
          den = scale * 0x1p64f;
#pragma unroll
          for (int k = 0; k < 8; ++k) x[h][k] *= 0x1p64f;
        }
        const float inv = 1.f / den;
        if (inv == 0.f) den = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float q = x[h][k] * inv;
          x[h][k] = fmaf(fmaf(-q, den, x[h][k]), inv, q);
        }
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[h][4 * k], x[h][4 * k + 1]), __NV_SATFINITE,
                                                       __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[h][4 * k + 2], x[h][4 * k + 3]), __NV_SATFINITE,
                                                       __NV_E4M3);
          w[k] = lo | (hi << 16);
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
}

template <int kTokens>
void launch_tokens(const AppendParams& p, bool half, bool fp8, cudaStream_t stream) {
  const int grid = static_cast<int>((static_cast<long long>(p.total) + kAppendWarps * kTokens - 1) / (kAppendWarps * kTokens));
  const int threads = 32 * kAppendWarps;
  if (half) {
    if (fp8)
      append_kernel<true, true, kTokens><<<grid, threads, 0, stream>>>(p);
    else
      append_kernel<true, false, kTokens><<<grid, threads, 0, stream>>>(p);
  } else {
    if (fp8)
      append_kernel<false, true, kTokens><<<grid, threads, 0, stream>>>(p);
    else
      append_kernel<false, false, kTokens><<<grid, threads, 0, stream>>>(p);
  }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, bool half, bool fp8, int sms, cudaStream_t stream) {
  // one token a warp until that fills the GPU.  (Two against one and four tokens
  // a warp: 13.2, 13.3 and 14.5 us for 24577 tokens into FP8 records, 23.2, 24.6
  // and 24.4 us for 49153 into bf16 rows.)
  if (p.total <= 16 * sms)
    launch_tokens<1>(p, half, fp8, stream);
  else
    launch_tokens<2>(p, half, fp8, stream);
  return cudaGetLastError();
}

}  // namespace mla
