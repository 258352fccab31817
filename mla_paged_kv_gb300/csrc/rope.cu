// Rotary positions: the table of cosines and sines that the cache append and
// the rotation below read, and the rotation of part of each query and key head,
// after an optional RMS norm of the head, in one pass.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "serving.cuh"

namespace mla {
namespace {

// ------------------------------------------------------------------ table

// cos_sin[p] = magnitude * (cos(p f_0) .. , sin(p f_0) ..).
//
// Angles in whole turns of 2^64 steps: step_i = round(f_i / 2 pi * 2^64), and
// p * step_i modulo 2^64 is the angle modulo a turn with no rounding at all: what
// is left of the frequency's own rounding (2^-53 of it) is below 2^-31 turns at
// position 2^24, where an fp32 angle would be off by a radian.  The nearest
// quarter turn comes off in integers too, so that sincospif sees at most a
// quarter of a half turn, and values next to zero keep their leading bits.
// Bound by the writes for many positions (163840 x 64: 42 MB), by the launch for
// few; a thread takes four pairs, whose cosines and sines are a 16-byte store each.
__global__ void __launch_bounds__(256)
    rope_table_kernel(const RopeSteps f, int dim, float magnitude, unsigned long long first, long long threads,
                      float* __restrict__ out) {
  const int quads = dim / 8;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < threads; i += gridDim.x * 256ll) {
    const long long p = i / quads;
    const int q = static_cast<int>(i - p * quads);
    float c[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned long long angle = (first + static_cast<unsigned long long>(p)) * f.step[4 * q + k];
      const unsigned long long quarter = (angle + (1ull << 61)) >> 62;  // nearest, modulo 4
      const float x = static_cast<float>(static_cast<long long>(angle - (quarter << 62))) * 0x1p-63f;  // half turns
      float sn, cs;
      sincospif(x, &sn, &cs);
      const bool swap = quarter & 1;
      const float a = swap ? sn : cs, b = swap ? cs : sn;
      c[k] = ((quarter + 1) & 2) ? -a * magnitude : a * magnitude;  // quarters 1 and 2
      s[k] = (quarter & 2) ? -b * magnitude : b * magnitude;        // quarters 2 and 3
    }
    float* row = out + p * dim + 4 * q;
    *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(row + dim / 2) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

// ------------------------------------------------------------------ heads

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
__device__ __forceinline__ void widen(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = unpack2<kHalf>(w[k]);
    f[2 * k] = a.x;
    f[2 * k + 1] = a.y;
  }
}

template <bool kHalf>
__device__ __forceinline__ uint4 narrow(const float* f) {
  return make_uint4(pack2f<kHalf>(f[0], f[1]), pack2f<kHalf>(f[2], f[3]), pack2f<kHalf>(f[4], f[5]),
                    pack2f<kHalf>(f[6], f[7]));
}

// y = x * rsqrt(mean(x^2) + eps) * w over a head's dims (with weights), then the
// pairs of its rotary part turned by the angle of the token's position.
//
// Memory bound: each head is read and written once, in 16-byte pieces of 8
// elements.  A lane's unit of work (an item) is two pieces: those that a rotation
// pairs with each other (in the half layout they lie rope / 2 apart, interleaved
// side by side), or two that only pass.  `lanes` lanes hold a head, kItems items
// each, and a warp takes one token and as many heads as it has lanes for, kIter
// times over: the position, found by a chain of small loads while the heads'
// own are in flight, and the angles are read once for all of them.
template <bool kHalf, int kItems, int kIter, bool kNorm>
__global__ void __launch_bounds__(128) rope_heads_kernel(const RopeHeadsParams p) {
  const int lane = threadIdx.x & 31;
  const long long unit = blockIdx.x * 4ll + (threadIdx.x >> 5);
  const int per_token = p.side[0].units + p.side[1].units;
  const long long t64 = unit / per_token;
  if (t64 >= p.total) return;  // uniform over the warp
  const int t = static_cast<int>(t64);
  int u = static_cast<int>(unit - t64 * per_token);
  const bool second = u >= p.side[0].units;
  const RopeSide& s = p.side[second];
  if (second) u -= p.side[0].units;
  const int slots = 32 / p.lanes, mine = lane & (p.lanes - 1);
  const int head0 = u * slots * kIter + lane / p.lanes;

  // Elements of an item's two pieces; -1: none.
  int at[kItems][2];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int item = mine + i * p.lanes;
    if (item < p.pairs) {
      at[i][0] = p.offset + (p.interleaved ? 16 * item : 8 * item);
      at[i][1] = at[i][0] + (p.interleaved ? 8 : p.rope / 2);
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int e = 8 * (2 * (item - p.pairs) + k);
        if (e >= p.offset) e += p.rope;
        at[i][k] = item < p.items && e < p.dim ? e : -1;
      }
    }
  }
  uint4 raw[kIter][kItems][2];
  const uint16_t* x = s.x + t64 * s.x_token_stride;
#pragma unroll
  for (int n = 0; n < kIter; ++n) {
    const int head = head0 + n * slots;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        raw[n][i][k] = head < s.heads && at[i][k] >= 0
                           ? *reinterpret_cast<const uint4*>(x + head * s.x_head_stride + at[i][k])
                           : make_uint4(0u, 0u, 0u, 0u);
  }

  int pos = 0;
  if (p.cos_sin != nullptr) {
    if (p.positions != nullptr) {
      pos = p.positions[t];
    } else {
      int b, left;
      if (p.cu == nullptr) {
        const int each = p.total / p.batch;
        b = t / each;
        left = (b + 1) * each - t;
      } else {
        if (t < p.cu[0] || t >= p.cu[p.batch]) return;  // of no sequence
        int lo = 0, hi = p.batch;                       // cu[lo] <= t < cu[hi], 32 ways at a time
        while (hi - lo > 1) {
          const int step = (hi - lo + 31) / 32, probe = lo + (lane + 1) * step;
          const int n = __popc(__ballot_sync(0xffffffffu, probe < hi && p.cu[probe] <= t));
          lo += n * step;
          hi = min(lo + step, hi);
        }
        b = lo;
        left = p.cu[b + 1] - t;
      }
      pos = p.seqlens[b] - left;
    }
    if (pos < 0 || pos >= p.max_pos) {
      report(p.status, MLA_ERR_BAD_INDEX);
      return;
    }
  }
  float cs[kItems][8], sn[kItems][8];
  if (p.cos_sin != nullptr) {
    const float* row = p.cos_sin + static_cast<long long>(pos) * p.rope;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int item = mine + i * p.lanes;
      if (item >= p.pairs) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        *reinterpret_cast<float4*>(cs[i] + 4 * k) = __ldg(reinterpret_cast<const float4*>(row + 8 * item) + k);
        *reinterpret_cast<float4*>(sn[i] + 4 * k) =
            __ldg(reinterpret_cast<const float4*>(row + p.rope / 2 + 8 * item) + k);
      }
    }
  }
  uint16_t* out = s.out + t64 * s.out_token_stride;
#pragma unroll
  for (int n = 0; n < kIter; ++n) {
    const int head = head0 + n * slots;
    float rstd = 1.f;
    if constexpr (kNorm) {
      if (s.weight != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kItems; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float f[8];
            widen<kHalf>(raw[n][i][k], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
          }
        for (int o = p.lanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rstd = 1.f / sqrtf(ss / static_cast<float>(p.dim) + p.eps);
      }
    }
    if (head >= s.heads) continue;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      float f[2][8];
      widen<kHalf>(raw[n][i][0], f[0]);
      widen<kHalf>(raw[n][i][1], f[1]);
      if constexpr (kNorm) {
        if (s.weight != nullptr) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (at[i][k] < 0) continue;
            float w[8];
            widen<kHalf>(__ldg(reinterpret_cast<const uint4*>(s.weight + at[i][k])), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[k][e] = f[k][e] * rstd * w[e];
          }
        }
      }
      if (mine + i * p.lanes < p.pairs) {
        // pair j of the item: elements j of both pieces, or (interleaved) 2j and 2j + 1 of the 16
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float& a = p.interleaved ? f[j >> 2][2 * (j & 3)] : f[0][j];
          float& b = p.interleaved ? f[j >> 2][2 * (j & 3) + 1] : f[1][j];
          const float y = a * cs[i][j] - b * sn[i][j], z = b * cs[i][j] + a * sn[i][j];
          a = y;
          b = z;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (at[i][k] >= 0)
          *reinterpret_cast<uint4*>(out + head * s.out_head_stride + at[i][k]) = narrow<kHalf>(f[k]);
    }
  }
}

template <bool kHalf, int kItems, int kIter>
cudaError_t launch_heads(const RopeHeadsParams& p, bool norm, unsigned grid, cudaStream_t st) {
  if (norm)
    rope_heads_kernel<kHalf, kItems, kIter, true><<<grid, 128, 0, st>>>(p);
  else
    rope_heads_kernel<kHalf, kItems, kIter, false><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool kHalf>
cudaError_t launch_items(const RopeHeadsParams& p, int per_lane, bool norm, unsigned grid, cudaStream_t st) {
  switch (per_lane) {
    case 1: return launch_heads<kHalf, 1, 4>(p, norm, grid, st);
    case 2: return launch_heads<kHalf, 2, 2>(p, norm, grid, st);
    case 3: return launch_heads<kHalf, 3, 1>(p, norm, grid, st);
    default: return launch_heads<kHalf, 4, 1>(p, norm, grid, st);
  }
}

}  // namespace

cudaError_t launch_rope_table(const RopeSteps& f, int dim, float magnitude, long long first, int positions, float* out,
                              int sms, cudaStream_t st) {
  const long long threads = static_cast<long long>(positions) * (dim / 8);
  const long long blocks = std::min<long long>((threads + 255) / 256, 8ll * sms);
  rope_table_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(f, dim, magnitude,
                                                                   static_cast<unsigned long long>(first), threads, out);
  return cudaGetLastError();
}

bool rope_heads_layout(RopeHeadsParams* p, bool passes, int* per_lane, long long* blocks) {
  p->pairs = p->rope / 16;
  const int plain = (p->dim - p->rope) / 8;
  p->items = p->pairs + (passes ? (plain + 1) / 2 : 0);
  // lanes and items a lane that leave the fewest lanes idle (heads of 192 dims: 4 lanes of 3 items, not 16 of which
  // 4 idle); among equals the fewest items a lane
  int best = 1 << 30;
  for (int n = 1; n <= 4; ++n) {
    int lanes = 1;
    while (lanes * n < p->items) lanes *= 2;
    if (lanes <= 32 && lanes * n - p->items < best) {
      best = lanes * n - p->items;
      p->lanes = lanes;
      *per_lane = n;
    }
  }
  const int iter = *per_lane == 1 ? 4 : *per_lane == 2 ? 2 : 1;
  for (RopeSide& s : p->side) s.units = (s.heads + 32 / p->lanes * iter - 1) / (32 / p->lanes * iter);
  *blocks = (static_cast<long long>(p->total) * (p->side[0].units + p->side[1].units) + 3) / 4;
  return best < (1 << 30) && *blocks < (1ll << 31);
}

cudaError_t launch_rope_heads(const RopeHeadsParams& p, bool half, int per_lane, long long blocks, cudaStream_t st) {
  const bool norm = p.side[0].weight != nullptr || p.side[1].weight != nullptr;
  const unsigned grid = static_cast<unsigned>(blocks);
  return half ? launch_items<true>(p, per_lane, norm, grid, st) : launch_items<false>(p, per_lane, norm, grid, st);
}

}  // namespace mla
