// Rotary positions of query (and output) heads, reading R20:
//   y1 = a (x1 cos f - x2 sin f),  y2 = a (x1 sin f + x2 cos f),  f = p theta_i,
// for the pairs (x1, x2) of the rotated channels; the other channels are copied.
//
// Angles: the table holds theta_i / 2 pi in 0.64 fixed point, p times that mod 2^64 is the angle's fraction of a
// turn (as in pack.cu, so that queries and cached keys agree), and the fraction is cut to a quarter turn and its
// rest in integers before it becomes fp32: the rest is below 1/8 of a turn, so its rounding is at most 2^-27
// turns and sinpi / cospi of it lose nothing to a large argument.
//
// Bound: bytes.  A block takes a few tokens: its threads compute the tokens' sines and cosines into shared memory
// once for all heads while the copied channels are on their way, then rotate 8 channels (two halves of 8) at a time
// with 16-byte loads and stores.  Shapes that 8 channels at a time do not divide go channel pair by channel pair.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "operands.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxAngles = 2048;    // (token, pair) angles of a block in shared memory
constexpr int kUnit = 8;            // channels of a load

// n / d and n % d for n < 2^31 by a multiplication (d >= 1): m = ceil(2^(31 + l) / d), l = ceil(log2 d), is below
// 2^32 and its excess over 2^(31 + l) / d below 2^l / 2^(31 + l), so that floor(n m / 2^(31 + l)) is exact there.
struct Divisor {
  uint32_t d, m, shift;
  static Divisor of(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return {d, (uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
  }
  __device__ __forceinline__ void split(uint32_t n, uint32_t* q, uint32_t* r) const {
    *q = (uint32_t)(((uint64_t)n * m) >> shift);
    *r = n - *q * d;
  }
};

struct RopePlan {
  RopeArgs a;
  int tokens, heads;                // of a block
  Divisor units, head_div;          // work units of a head, heads of a block
};

// cos and sin of p turns-per-position g, times the amplitude.
__device__ __forceinline__ float2 rotation(int32_t p, uint64_t g, float amplitude, int inverse) {
  const uint64_t turn = (uint64_t)(int64_t)p * g;
  const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);               // nearest quarter turn
  const int64_t rest = (int64_t)(turn - ((uint64_t)quarter << 62));               // in [-1/8, 1/8) turns
  float sn, cs;
  sincospif((float)rest * 0x1p-63f, &sn, &cs);
  const float c = quarter == 0 ? cs : quarter == 1 ? -sn : quarter == 2 ? -cs : sn;
  const float s = quarter == 0 ? sn : quarter == 1 ? cs : quarter == 2 ? -sn : -cs;
  return make_float2(amplitude * c, amplitude * (inverse ? -s : s));
}

// 8 channels as fp32 (plain loads: y may be x).
template <typename T> struct Eight;
template <> struct Eight<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = word_of(v, j);
      f[2 * j] = __uint_as_float(w << 16);
      f[2 * j + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
  }
};
template <> struct Eight<float> {
  float4 lo, hi;
  __device__ __forceinline__ void load(const float* p) {
    lo = reinterpret_cast<const float4*>(p)[0];
    hi = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = lo.x; f[1] = lo.y; f[2] = lo.z; f[3] = lo.w; f[4] = hi.x; f[5] = hi.y; f[6] = hi.z; f[7] = hi.w;
  }
};
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(f32x2_bf16x2(f[0], f[1]), f32x2_bf16x2(f[2], f[3]), f32x2_bf16x2(f[4], f[5]), f32x2_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ float to_f32(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = (uint16_t)(f32x2_bf16x2(x, 0.f) & 0xFFFFu); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

// The block's tokens' rotations into shared memory: cs[token][pair].
__device__ __forceinline__ void rotations(const RopeArgs& a, int64_t t0, int tokens, float2* cs) {
  const int pairs = a.r / 2;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = i / pairs, k = i - t * pairs;
    if (t0 + t < a.rows) cs[i] = rotation(a.positions[t0 + t], a.table[k], a.amplitude, a.inverse);
  }
}

// 8 channels at a time.  Units of a head: with half pairs r / 16 pairs of 8 + 8 channels, with interleaved ones
// r / 8 of 8; then, unless y is x, (d - r) / 8 copied ones.
template <typename In, typename Out, bool kHalf>
__global__ void __launch_bounds__(kThreads) k_rope(RopePlan pl) {
  __shared__ float2 cs[kMaxAngles];
  const RopeArgs& a = pl.a;
  pdl_wait();
  const int64_t t0 = (int64_t)blockIdx.x * pl.tokens;
  const int h0 = blockIdx.y * pl.heads;
  rotations(a, t0, pl.tokens, cs);
  __syncthreads();
  const In* x = static_cast<const In*>(a.x);
  Out* y = static_cast<Out*>(a.y);
  const int rot = kHalf ? a.r / 16 : a.r / 8;      // rotated units of a head come first
  const int total = pl.tokens * pl.heads * (int)pl.units.d;
  constexpr int kMany = sizeof(In) == 4 ? 2 : 4;   // units in flight
  for (int u0 = threadIdx.x; u0 < total; u0 += kMany * kThreads) {
    Eight<In> v[kMany], w[kMany];
    int64_t to[kMany];
    int at[kMany];                                  // first angle; -1: copied; -2: nothing
#pragma unroll
    for (int k = 0; k < kMany; ++k) {
      const uint32_t u = u0 + k * kThreads;
      at[k] = -2;
      to[k] = 0;
      if (u >= (uint32_t)total) continue;
      uint32_t th, unit, t, h;
      pl.units.split(u, &th, &unit);
      pl.head_div.split(th, &t, &h);
      if (t0 + t >= a.rows || h0 + (int)h >= a.heads) continue;
      int c;
      if ((int)unit < rot) {
        c = a.start + unit * kUnit;
        at[k] = t * (a.r / 2) + unit * (kHalf ? kUnit : kUnit / 2);
      } else {
        c = (unit - rot) * kUnit;
        if (c >= a.start) c += a.r;
        at[k] = -1;
      }
      const In* p = x + (t0 + t) * a.x_token + (int64_t)(h0 + h) * a.x_head + c;
      v[k].load(p);
      if (kHalf && at[k] >= 0) w[k].load(p + a.r / 2);
      to[k] = (t0 + t) * a.y_token + (int64_t)(h0 + h) * a.y_head + c;
    }
#pragma unroll
    for (int k = 0; k < kMany; ++k) {
      if (at[k] == -2) continue;
      float f[8];
      v[k].get(f);
      if (at[k] >= 0) {
        if (kHalf) {
          float g[8];
          w[k].get(g);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 q = cs[at[k] + j];
            const float f1 = f[j] * q.x - g[j] * q.y;
            g[j] = f[j] * q.y + g[j] * q.x;
            f[j] = f1;
          }
          store8(y + to[k] + a.r / 2, g);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 q = cs[at[k] + j];
            const float f1 = f[2 * j] * q.x - f[2 * j + 1] * q.y;
            f[2 * j + 1] = f[2 * j] * q.y + f[2 * j + 1] * q.x;
            f[2 * j] = f1;
          }
        }
      }
      store8(y + to[k], f);
    }
  }
}

// Any shape: a unit is a pair, or a copied channel.
template <typename In, typename Out>
__global__ void __launch_bounds__(kThreads) k_rope_any(RopePlan pl) {
  __shared__ float2 cs[kMaxAngles];
  const RopeArgs& a = pl.a;
  pdl_wait();
  const int64_t t0 = (int64_t)blockIdx.x * pl.tokens;
  const int h0 = blockIdx.y * pl.heads;
  rotations(a, t0, pl.tokens, cs);
  __syncthreads();
  const In* x = static_cast<const In*>(a.x);
  Out* y = static_cast<Out*>(a.y);
  const int total = pl.tokens * pl.heads * (int)pl.units.d, pairs = a.r / 2;
  for (int u = threadIdx.x; u < total; u += kThreads) {
    uint32_t th, unit, t, h;
    pl.units.split(u, &th, &unit);
    pl.head_div.split(th, &t, &h);
    if (t0 + t >= a.rows || h0 + (int)h >= a.heads) continue;
    const In* p = x + (t0 + t) * a.x_token + (int64_t)(h0 + h) * a.x_head;
    Out* q = y + (t0 + t) * a.y_token + (int64_t)(h0 + h) * a.y_head;
    if ((int)unit < pairs) {
      const int c1 = a.start + (a.layout == CSA2_ROPE_HALF ? (int)unit : 2 * (int)unit);
      const int c2 = a.layout == CSA2_ROPE_HALF ? c1 + pairs : c1 + 1;
      const float x1 = to_f32(p[c1]), x2 = to_f32(p[c2]);
      const float2 z = cs[t * pairs + unit];
      store1(q + c1, x1 * z.x - x2 * z.y);
      store1(q + c2, x1 * z.y + x2 * z.x);
    } else {
      int c = unit - pairs;
      if (c >= a.start) c += a.r;
      store1(q + c, to_f32(p[c]));
    }
  }
}

__global__ void k_rope_table(const __grid_constant__ RopeTable t, int n, uint64_t* out) {
  pdl_wait();
  for (int i = threadIdx.x; i < n; i += blockDim.x) out[i] = t.g[i];
}

template <typename In, typename Out>
cudaError_t launch_typed(const RopePlan& pl, dim3 grid, bool eight, cudaStream_t s) {
  if (!eight) return launch_step(k_rope_any<In, Out>, grid, dim3(kThreads), 0, s, pl);
  return pl.a.layout == CSA2_ROPE_HALF ? launch_step(k_rope<In, Out, true>, grid, dim3(kThreads), 0, s, pl)
                                       : launch_step(k_rope<In, Out, false>, grid, dim3(kThreads), 0, s, pl);
}

}  // namespace

cudaError_t launch_rope_table(const RopeTable& t, int pairs, uint64_t* out, cudaStream_t s) {
  return launch_step(k_rope_table, dim3(1), dim3(256), 0, s, t, pairs, out);
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  const bool in_place = a.x == a.y;
  const int in = a.x_dtype == CSA2_F32 ? 4 : 2, out = a.y_dtype == CSA2_F32 ? 4 : 2;
  auto whole = [](const void* p, int64_t token, int64_t head, int size) {   // rows start on 16 bytes
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && token * size % 16 == 0 && head * size % 16 == 0;
  };
  const bool eight = a.d % kUnit == 0 && a.start % kUnit == 0 && a.r % (a.layout == CSA2_ROPE_HALF ? 2 * kUnit : kUnit) == 0 &&
                     whole(a.x, a.x_token, a.x_head, in) && whole(a.y, a.y_token, a.y_head, out);
  const int copied = in_place ? 0 : a.d - a.r;
  RopePlan pl;
  pl.a = a;
  const int units = eight ? (a.layout == CSA2_ROPE_HALF ? a.r / 16 : a.r / 8) + copied / kUnit : a.r / 2 + copied;
  if (units == 0) return cudaSuccess;       // (in place, nothing rotated)
  // A block: about 2,048 units, whole tokens while their angles fit; fewer heads of one token where there are
  // few tokens, so that every SM has a block (one token of 64 heads x 512 channels in 32 blocks).
  const int64_t per_token = (int64_t)a.heads * units;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(2048, a.rows * per_token / (2 * 152) + 1));
  pl.heads = (int)std::min<int64_t>(a.heads, std::max<int64_t>(1, (want + units - 1) / units));
  pl.tokens = 1;
  if (pl.heads == a.heads) pl.tokens = (int)std::max<int64_t>(1, std::min<int64_t>(want / per_token, kMaxAngles / std::max(1, a.r / 2)));
  pl.units = Divisor::of(units);
  pl.head_div = Divisor::of(pl.heads);
  const int64_t gx = (a.rows + pl.tokens - 1) / pl.tokens;
  if (gx > INT_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)gx, (unsigned)((a.heads + pl.heads - 1) / pl.heads));
  if (a.x_dtype == CSA2_F32)
    return a.y_dtype == CSA2_F32 ? launch_typed<float, float>(pl, grid, eight, s) : launch_typed<float, uint16_t>(pl, grid, eight, s);
  return a.y_dtype == CSA2_F32 ? launch_typed<uint16_t, float>(pl, grid, eight, s) : launch_typed<uint16_t, uint16_t>(pl, grid, eight, s);
}

}  // namespace csa2
