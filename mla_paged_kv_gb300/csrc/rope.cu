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

constexpr double kPi = 3.14159265358979323846;
__host__ __device__ constexpr double pi_to(int n) { return n == 0 ? 1.0 : kPi * pi_to(n - 1); }
__host__ __device__ constexpr double factorial(int n) { return n < 2 ? 1.0 : n * factorial(n - 1); }
// The coefficient of x^n in the series of sin(pi x) (n odd) or cos(pi x) (n even), twice.
template <int n>
__device__ __forceinline__ float2 series() {
  constexpr float c = static_cast<float>(((n >> 1) & 1 ? -1.0 : 1.0) * pi_to(n) / factorial(n));
  return make_float2(c, c);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// For |x| <= 1/4.
__device__ __forceinline__ float2 sin_pi(float2 x) {
  constexpr float kHigh = static_cast<float>(kPi), kLow = static_cast<float>(kPi - static_cast<double>(kHigh));
  const float2 t = __fmul2_rn(x, x);
  float2 y = __ffma2_rn(t, series<9>(), series<7>());
  y = __ffma2_rn(t, y, series<5>());
  y = __ffma2_rn(t, y, series<3>());
  y = __ffma2_rn(t, y, both(kLow));
  return __ffma2_rn(x, both(kHigh), __fmul2_rn(x, y));
}
__device__ __forceinline__ float2 cos_pi(float2 x) {
  const float2 t = __fmul2_rn(x, x);
  float2 y = __ffma2_rn(t, series<10>(), series<8>());
  y = __ffma2_rn(t, y, series<6>());
  y = __ffma2_rn(t, y, series<4>());
  y = __ffma2_rn(t, y, series<2>());
  return __ffma2_rn(t, y, both(1.f));
}

// cos_sin[p] = magnitude * (cos(p f_0) .. , sin(p f_0) ..).
//
// Angles in whole turns of 2^64 steps: step_i is the fraction of f_i / 2 pi, in 64-bit
// arithmetic (off by 2^-52 of it) and cut behind 2^-64, and p * step_i modulo 2^64 is
// the angle modulo a turn with no rounding.  It is off by 2^-52 of the whole angle and
// 2^-64 turns a position: below 2^-30 turns at position 2^24 for f = 1, where an fp32
// angle would be off by a radian, and below 2^-23 at the last position, 2^31.  The
// nearest quarter turn comes off in integers too; what is left, at most an eighth of a
// turn to either side, is converted high and low word apart, so that values next to
// zero keep their leading bits (to 2^-52), and the Taylor series of sin(pi x) and
// cos(pi x) to x^9 and x^10 leave 2^-28 of it there.
// A thread keeps four pairs, two at a time in packed arithmetic, and steps through
// positions, so that an angle is one addition.  Bound by the launch for few positions
// (4096 x 64: 4.2 us), for many by issue, with half of it left to the writes (163840 x
// 64: 41 MB in 10.4 us; 14.5 with the library's sincospif).
__global__ void __launch_bounds__(256)
    rope_table_kernel(const RopeSteps f, int dim, float magnitude, unsigned long long first, int positions,
                      float* __restrict__ out) {
  const int quads = dim / 8, rows = 256 / quads;  // threads of a position, positions of a block at a time
  const int q = threadIdx.x % quads, r = threadIdx.x / quads;
  if (r >= rows) return;
  const int step = gridDim.x * rows;
  long long p = static_cast<long long>(blockIdx.x) * rows + r;
  unsigned long long angle[4], turn[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    angle[k] = (first + static_cast<unsigned long long>(p)) * f.step[4 * q + k];
    turn[k] = static_cast<unsigned long long>(step) * f.step[4 * q + k];
  }
  for (; p < positions; p += step) {
    float c[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      uint32_t quarter[2];  // nearest, modulo 4
      float2 x;             // half turns past it
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t high = static_cast<uint32_t>(angle[k + h] >> 32), low = static_cast<uint32_t>(angle[k + h]);
        quarter[h] = (high + (1u << 29)) >> 30;
        const int rest = static_cast<int>(high - (quarter[h] << 30));
        (h ? x.y : x.x) = fmaf(static_cast<float>(low), 0x1p-63f, static_cast<float>(rest) * 0x1p-31f);
        angle[k + h] += turn[k + h];
      }
      const float2 sn = sin_pi(x), cs = cos_pi(x);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a = h ? cs.y : cs.x, b = h ? sn.y : sn.x;
        const bool swap = quarter[h] & 1;
        // quarters 1 and 2, and 2 and 3, are negative
        c[k + h] = __uint_as_float(__float_as_uint(swap ? b : a) ^ ((quarter[h] + 1) & 2) << 30) * magnitude;
        s[k + h] = __uint_as_float(__float_as_uint(swap ? a : b) ^ (quarter[h] & 2) << 30) * magnitude;
      }
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

// 8 elements as four pairs of fp32: the arithmetic runs on packed pairs.
template <bool kHalf>
__device__ __forceinline__ void widen(const uint4& v, float2 (&f)[4]) {
  f[0] = unpack2<kHalf>(v.x);
  f[1] = unpack2<kHalf>(v.y);
  f[2] = unpack2<kHalf>(v.z);
  f[3] = unpack2<kHalf>(v.w);
}

template <bool kHalf>
__device__ __forceinline__ uint4 narrow(const float2 (&f)[4]) {
  return make_uint4(pack2f<kHalf>(f[0].x, f[0].y), pack2f<kHalf>(f[1].x, f[1].y), pack2f<kHalf>(f[2].x, f[2].y),
                    pack2f<kHalf>(f[3].x, f[3].y));
}

// y = x * rsqrt(mean(x^2) + eps) * w over a head's dims (with weights), then the
// pairs of its rotary part turned by the angle of the token's position.
//
// Memory bound: each head is read and written once, in 16-byte pieces of 8
// elements.  A lane's unit of work (an item) is two pieces: two of the rotary part,
// rope / 2 apart (in the half layout a rotation pairs them with each other), or two
// that only pass, half of those apart: neighbouring lanes have neighbouring pieces
// (side by side in a lane, 32 bytes, 8193 tokens x 128 heads x 64 took 51.6 us, not
// 49.9).  `lanes` lanes hold a head, kItems items
// each, and a warp takes one token and as many heads as it has lanes for, kIter
// times over: the position, found by a chain of small loads while the heads'
// own are in flight, and the angles are read once for all of them.  Issue comes
// next after memory: layout and norm are template arguments, the arithmetic is
// packed, and few registers leave many warps resident (24577 tokens x 40 heads x 128
// dims with norm 94 us, 5.5 TB/s; 138 with one code for all and the items' values kept).
// kTurn: items of a lane that may turn, its first ones.
template <bool kHalf, int kItems, int kTurn, int kIter, bool kNorm, bool kInter>
__global__ void __launch_bounds__(128) rope_heads_kernel(const RopeHeadsParams p) {
  const int lane = threadIdx.x & 31;
  const long long unit = blockIdx.x * 4ll + (threadIdx.x >> 5);
  const int t = static_cast<int>(unit / p.units);
  if (t >= p.total) return;  // uniform over the warp
  const int slots = 32 >> p.lane_bits, mine = lane & ((1 << p.lane_bits) - 1);
  // this lane's first head, of queries and then keys
  const int head0 = static_cast<int>(unit - static_cast<long long>(t) * p.units) * slots * kIter + (lane >> p.lane_bits);
  const int heads = p.side[0].heads + p.side[1].heads;

  // Where an item's two pieces lie in a head, and whether they are any of it.
  int at[kItems][2];
  bool is[kItems][2], turns[kTurn];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int item = mine + (i << p.lane_bits);
    if (i < kTurn) turns[i] = item < p.pairs;
    if (i < kTurn && turns[i]) {
      at[i][0] = p.offset + 8 * item;
      at[i][1] = at[i][0] + p.rope / 2;
      is[i][0] = is[i][1] = true;
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int e = 8 * (item - p.pairs + k * (p.items - p.pairs));
        if (e >= p.offset) e += p.rope;
        is[i][k] = item < p.items && e < p.dim;
        at[i][k] = is[i][k] ? e : 0;
      }
    }
  }
  uint4 raw[kIter][kItems][2];
#pragma unroll
  for (int n = 0; n < kIter; ++n) {
    const int head = head0 + n * slots;
    const bool second = head >= p.side[0].heads;
    const RopeSide& s = p.side[second];
    const uint16_t* x = s.x + static_cast<long long>(t) * s.x_token_stride +
                        (head - (second ? p.side[0].heads : 0)) * s.x_head_stride;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        raw[n][i][k] = head < heads && is[i][k] ? *reinterpret_cast<const uint4*>(x + at[i][k]) : make_uint4(0u, 0u, 0u, 0u);
  }

  const bool rotate = p.cos_sin != nullptr;
  int pos = 0;
  if (rotate) {
    if (p.positions != nullptr) {
      pos = p.positions[t];
    } else {
      int b, left;
      if (p.cu == nullptr) {
        const int each = p.total / p.batch;
        b = t / each;
        left = (b + 1) * each - t;
        pos = p.seqlens[b] - left;
      } else if (p.batch <= 32) {  // all requests at once: one trip to memory
        const int b0 = min(lane, p.batch - 1);
        const int first = p.cu[b0], last = p.cu[b0 + 1], len = p.seqlens[b0];
        const uint32_t in = __ballot_sync(0xffffffffu, lane < p.batch && first <= t && t < last);
        if (in == 0) return;  // of no sequence
        pos = __shfl_sync(0xffffffffu, len - (last - t), 31 - __clz(in));
      } else {
        if (t < p.cu[0] || t >= p.cu[p.batch]) return;
        int lo = 0, hi = p.batch;  // cu[lo] <= t < cu[hi], 32 ways at a time
        while (hi - lo > 1) {
          const int step = (hi - lo + 31) / 32, probe = lo + (lane + 1) * step;
          const int n = __popc(__ballot_sync(0xffffffffu, probe < hi && p.cu[probe] <= t));
          lo += n * step;
          hi = min(lo + step, hi);
        }
        b = lo;
        left = p.cu[b + 1] - t;
        pos = p.seqlens[b] - left;
      }
    }
    if (pos < 0 || pos >= p.max_pos) {
      report(p.status, MLA_ERR_BAD_INDEX);
      return;
    }
  }
  // cosines and sines of an item's eight pairs, two at a time
  float2 cs[kTurn][4], sn[kTurn][4];
  if (rotate) {
    const float* row = p.cos_sin + static_cast<long long>(pos) * p.rope;
#pragma unroll
    for (int i = 0; i < kTurn; ++i) {
      if (!turns[i]) continue;
      const int item = mine + (i << p.lane_bits);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float* c = row + (kInter ? 4 * item + k * (p.rope / 4) : 8 * item + 4 * k);
        *reinterpret_cast<float4*>(cs[i] + 2 * k) = __ldg(reinterpret_cast<const float4*>(c));
        *reinterpret_cast<float4*>(sn[i] + 2 * k) = __ldg(reinterpret_cast<const float4*>(c + p.rope / 2));
      }
    }
  }
#pragma unroll
  for (int n = 0; n < kIter; ++n) {
    const int head = head0 + n * slots;
    const bool second = head >= p.side[0].heads;
    const RopeSide& s = p.side[second];
    uint16_t* out = s.out + static_cast<long long>(t) * s.out_token_stride +
                    (head - (second ? p.side[0].heads : 0)) * s.out_head_stride;
    const bool normed = kNorm && s.weight != nullptr;
    float2 r2 = make_float2(1.f, 1.f);
    if constexpr (kNorm) {
      float2 ss[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < kItems; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float2 f[4];
          widen<kHalf>(raw[n][i][k], f);
#pragma unroll
          for (int e = 0; e < 4; ++e) ss[e & 1] = __ffma2_rn(f[e], f[e], ss[e & 1]);
        }
      float sum = (ss[0].x + ss[0].y) + (ss[1].x + ss[1].y);
      for (int o = 1 << p.lane_bits >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float r = rsqrtf(fmaf(sum, p.inv_dim, p.eps));
      r2 = make_float2(r, r);
    }
    if (head >= heads) continue;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      float2 f[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        widen<kHalf>(raw[n][i][k], f[k]);
        if (normed) {
          float2 g[4];
          widen<kHalf>(__ldg(reinterpret_cast<const uint4*>(s.weight + at[i][k])), g);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[k][e] = __fmul2_rn(__fmul2_rn(f[k][e], r2), g[e]);
        }
      }
      // (products and sums in the order of cache_append's, so that a key turned there has the same bits)
      if (i < kTurn && turns[i]) {
        if constexpr (kInter) {  // pair j: element pair j of the item's eight
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float2& a = f[j >> 2][j & 3];
            const float c = (j & 1) ? cs[i][j >> 1].y : cs[i][j >> 1].x, w = (j & 1) ? sn[i][j >> 1].y : sn[i][j >> 1].x;
            a = __ffma2_rn(a, make_float2(c, c), __fmul2_rn(make_float2(a.y, a.x), make_float2(-w, w)));
          }
        } else {  // pair j: element j of both pieces
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 a = f[0][j], b = f[1][j], c = cs[i][j], w = sn[i][j];
            f[0][j] = __ffma2_rn(a, c, __fmul2_rn(make_float2(-b.x, -b.y), w));
            f[1][j] = __ffma2_rn(b, c, __fmul2_rn(a, w));
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (is[i][k]) *reinterpret_cast<uint4*>(out + at[i][k]) = narrow<kHalf>(f[k]);
    }
  }
}

template <bool kHalf, int kItems, int kTurn, int kIter>
cudaError_t launch_heads(const RopeHeadsParams& p, bool norm, unsigned grid, cudaStream_t st) {
  if (norm) {
    if (p.interleaved)
      rope_heads_kernel<kHalf, kItems, kTurn, kIter, true, true><<<grid, 128, 0, st>>>(p);
    else
      rope_heads_kernel<kHalf, kItems, kTurn, kIter, true, false><<<grid, 128, 0, st>>>(p);
  } else if (p.interleaved) {
    rope_heads_kernel<kHalf, kItems, kTurn, kIter, false, true><<<grid, 128, 0, st>>>(p);
  } else {
    rope_heads_kernel<kHalf, kItems, kTurn, kIter, false, false><<<grid, 128, 0, st>>>(p);
  }
  return cudaGetLastError();
}

template <bool kHalf>
cudaError_t launch_items(const RopeHeadsParams& p, int per_lane, bool norm, unsigned grid, cudaStream_t st) {
  const bool one = p.pairs <= 1 << p.lane_bits;  // a lane's first item alone may turn
  switch (per_lane) {
    case 1: return launch_heads<kHalf, 1, 1, 2>(p, norm, grid, st);
    case 2:
      return one ? launch_heads<kHalf, 2, 1, 2>(p, norm, grid, st) : launch_heads<kHalf, 2, 2, 2>(p, norm, grid, st);
    case 3:
      return one ? launch_heads<kHalf, 3, 1, 2>(p, norm, grid, st) : launch_heads<kHalf, 3, 3, 2>(p, norm, grid, st);
    default:
      return one ? launch_heads<kHalf, 4, 1, 1>(p, norm, grid, st) : launch_heads<kHalf, 4, 4, 1>(p, norm, grid, st);
  }
}

}  // namespace

cudaError_t launch_rope_table(const RopeSteps& f, int dim, float magnitude, long long first, int positions, float* out,
                              int sms, cudaStream_t st) {
  const int rows = 256 / (dim / 8);
  const long long blocks = std::min<long long>((positions + rows - 1ll) / rows, 8ll * sms);
  rope_table_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(
      f, dim, magnitude, static_cast<unsigned long long>(first), positions, out);
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
    int bits = 0;
    while ((n << bits) < p->items) ++bits;
    if (bits <= 5 && (n << bits) - p->items < best) {
      best = (n << bits) - p->items;
      p->lane_bits = bits;
      *per_lane = n;
    }
  }
  p->inv_dim = 1.f / static_cast<float>(p->dim);
  const int heads = (32 >> p->lane_bits) * (*per_lane < 4 ? 2 : 1);  // of a warp
  p->units = (p->side[0].heads + p->side[1].heads + heads - 1) / heads;
  *blocks = (static_cast<long long>(p->total) * p->units + 3) / 4;
  return best < (1 << 30) && *blocks < (1ll << 31);
}

cudaError_t launch_rope_heads(const RopeHeadsParams& p, bool half, int per_lane, long long blocks, cudaStream_t st) {
  const bool norm = p.side[0].weight != nullptr || p.side[1].weight != nullptr;
  const unsigned grid = static_cast<unsigned>(blocks);
  return half ? launch_items<true>(p, per_lane, norm, grid, st) : launch_items<false>(p, per_lane, norm, grid, st);
}

}  // namespace mla
