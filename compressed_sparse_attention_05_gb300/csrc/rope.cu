// Rotary positions of query (and output) heads, reading R20:
//   y1 = a (x1 cos f - x2 sin f),  y2 = a (x1 sin f + x2 cos f),  f = p theta_i,
// for the pairs (x1, x2) of the rotated channels; the other channels are copied.
//
// Angles: the table holds theta_i / 2 pi in 0.64 fixed point, p times that mod 2^64 is the angle's fraction of a
// turn (as in pack.cu, so that queries and cached keys agree), and the fraction is cut to a quarter turn and its
// rest in integers before it becomes fp32: the rest is below 1/8 of a turn, so its rounding is at most 2^-27
// turns and sinpi / cospi of it lose nothing to a large argument.  The table's words come from fp64 and are off by a few
// 2^-53 of themselves, which p multiplies: an angle is known to p 2^-50 radians, 2^-19 at the last position, and the same
// angle for queries and keys.
//
// Bound: bytes.  A block takes about 2,048 units of work of 16-byte loads (8 channels; two halves of 8) that lie behind
// one another, over tokens and heads: its threads compute their tokens' sines and cosines into shared memory once for
// all heads, then rotate and copy with 2 or 4 units' loads in flight each.  4,096 tokens x 64 heads x 512 channels, 64
// rotated, bf16: 79 us, 6.8 TB/s (whole heads a block: 90; four blocks an SM: 85).  With one head, whose
// rotations serve no other, nothing lies under a block's start (positions, sines, barrier): 109,307 x 512 takes 42 us (5.3
// TB/s), 338,137 x 64 with 32 rotated 32.5 (2.7; half pairs 44).
// Half pairs that 8 channels do not divide, odd starts and unaligned rows go pair by pair (445 x 40 x 512, 62 rotated,
// half: 11 us, at 3.3 TB/s).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "operands.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxAngles = 2048;    // (token, pair) angles of a block in shared memory
constexpr int kUnit = 8;            // channels of a load

// The units of work in a row, token after token, head after head; a block takes `span` of them.
struct RopePlan {
  RopeArgs a;
  int64_t total;                    // units of all tokens
  int span, tokens;                 // of a block: units, tokens that they can touch
  int far;                          // total >= 2^31
  Divisor per_token, units;         // units of a token, of a head
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
// 8 channels on their way out.  Copied ones of the same type keep their bits: a NaN's payload would not come through a
// conversion.
template <typename T> struct Result;
template <> struct Result<uint16_t> {
  uint32_t w[4];
  __device__ __forceinline__ void copy(const Eight<uint16_t>& e) { w[0] = e.v.x; w[1] = e.v.y; w[2] = e.v.z; w[3] = e.v.w; }
  __device__ __forceinline__ void copy(const Eight<float>& e) {
    set(0, e.lo.x, e.lo.y); set(1, e.lo.z, e.lo.w); set(2, e.hi.x, e.hi.y); set(3, e.hi.z, e.hi.w);
  }
  __device__ __forceinline__ void set(int pair, float a, float b) { w[pair] = f32x2_bf16x2(a, b); }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]); }
  __device__ __forceinline__ void store_pair(uint16_t* p, int pair) const { *reinterpret_cast<uint32_t*>(p + 2 * pair) = w[pair]; }
};
template <> struct Result<float> {
  float f[8];
  template <typename In> __device__ __forceinline__ void copy(const Eight<In>& e) { e.get(f); }
  __device__ __forceinline__ void set(int pair, float a, float b) { f[2 * pair] = a; f[2 * pair + 1] = b; }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void store_pair(float* p, int pair) const { *reinterpret_cast<float2*>(p + 2 * pair) = make_float2(f[2 * pair], f[2 * pair + 1]); }
};
__device__ __forceinline__ float to_f32(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = (uint16_t)(f32x2_bf16x2(x, 0.f) & 0xFFFFu); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
// A copied channel, its bits too.
template <typename In>
__device__ __forceinline__ void copy1(uint16_t* p, float x) {
  if (sizeof(In) == 2) *p = (uint16_t)(__float_as_uint(x) >> 16);
  else store1(p, x);
}
template <typename In>
__device__ __forceinline__ void copy1(float* p, float x) { *p = x; }

// A block's first token and the units of it that lie before the block's.
__device__ __forceinline__ void first_unit(const RopePlan& pl, int64_t* t0, uint32_t* before) {
  const int64_t u = (int64_t)blockIdx.x * pl.span;
  if (pl.far) {
    *t0 = u / pl.per_token.d;
    *before = (uint32_t)(u - *t0 * pl.per_token.d);
  } else {
    uint32_t t;
    pl.per_token.split((uint32_t)u, &t, before);
    *t0 = t;
  }
}

// The block's tokens' rotations into shared memory: cs[token][pair].
__device__ __forceinline__ void rotations(const RopeArgs& a, int64_t t0, int tokens, float2* cs) {
  const int pairs = a.r / 2;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = i / pairs, k = i - t * pairs;
    if (t0 + t < a.rows) cs[i] = rotation(a.positions[t0 + t], a.table[k], a.amplitude, a.inverse);
  }
}

// 8 channels at a time.  Units of a head: with half pairs r / 16 pairs of 8 + 8 channels, with interleaved ones
// r / 8 of 8; then, unless y is x, (d - r) / 8 copied ones.  kRagged: interleaved pairs from any even channel on, so
// that the rotated units' first and last may have pairs that are copied; kRaggedInPlace: that are left alone (somebody else
// may be writing them).
enum Mode { kInterleaved, kHalves, kRagged, kRaggedInPlace, kOnes, kOnesWhole };
// 8-channel loads of a head that have a rotated channel.
__host__ __device__ inline int touched_units(const RopeArgs& a) { return a.r ? (a.start + a.r + kUnit - 1) / kUnit - a.start / kUnit : 0; }
__host__ __device__ inline int rotated_units(const RopeArgs& a, Mode mode) {
  return mode == kHalves ? a.r / 16 : mode == kInterleaved ? a.r / 8 : touched_units(a);
}

// Blocks of an SM: as many as take no spills (4,096 x 64 x 512 of bf16: interleaved 78.6 us with 5, 83.5 with 4; ragged 79.4
// with 6, 83.3 with 5); 0 leaves it to the compiler.
template <typename In, typename Out, Mode kMode>
constexpr int kBlocks = kMode == kHalves ? 3 : kMode == kRaggedInPlace ? 0 : kMode == kRagged && sizeof(In) + sizeof(Out) == 4 ? 6 : 5;

template <typename In, typename Out, Mode kMode>
__global__ void __launch_bounds__(kThreads, kBlocks<In, Out, kMode>) k_rope(RopePlan pl) {
  __shared__ float2 cs[kMaxAngles];
  constexpr bool kHalf = kMode == kHalves, kAnyPair = kMode == kRagged || kMode == kRaggedInPlace;
  const RopeArgs& a = pl.a;
  pdl_wait();
  int64_t t0;
  uint32_t before;
  first_unit(pl, &t0, &before);
  rotations(a, t0, pl.tokens, cs);
  __syncthreads();
  const In* x = static_cast<const In*>(a.x);
  Out* y = static_cast<Out*>(a.y);
  const int rot = rotated_units(a, kMode);         // of a head; they come first
  const int first = kAnyPair ? a.start & ~(kUnit - 1) : a.start, width = kAnyPair ? rot * kUnit : a.r;
  const int total = (int)min((int64_t)pl.span, pl.total - (int64_t)blockIdx.x * pl.span);
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
      uint32_t t, h, unit;
      pl.per_token.split(before + u, &t, &unit);
      pl.units.split(unit, &h, &unit);
      int c;
      if ((int)unit < rot) {
        c = first + unit * kUnit;
        at[k] = kAnyPair ? (int)(t << 16 | unit) : t * (a.r / 2) + unit * (kHalf ? kUnit : kUnit / 2);
      } else {
        c = (unit - rot) * kUnit;
        if (c >= first) c += width;
        at[k] = -1;
      }
      const In* p = x + (t0 + t) * a.x_token + (int64_t)h * a.x_head + c;
      v[k].load(p);
      if (kHalf && at[k] >= 0) w[k].load(p + a.r / 2);
      to[k] = (t0 + t) * a.y_token + (int64_t)h * a.y_head + c;
    }
#pragma unroll
    for (int k = 0; k < kMany; ++k) {
      if (at[k] == -2) continue;
      Result<Out> out;
      if (!kAnyPair && at[k] < 0) {
        out.copy(v[k]);
        out.store(y + to[k]);
        continue;
      }
      float f[8];
      v[k].get(f);
      if (kHalf) {
        float g[8];
        w[k].get(g);
        Result<Out> second;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float2 q = cs[at[k] + j], z = cs[at[k] + j + 1];
          out.set(j / 2, f[j] * q.x - g[j] * q.y, f[j + 1] * z.x - g[j + 1] * z.y);
          second.set(j / 2, f[j] * q.y + g[j] * q.x, f[j + 1] * z.y + g[j + 1] * z.x);
        }
        second.store(y + to[k] + a.r / 2);
        out.store(y + to[k]);
        continue;
      }
      // pair j of the unit, the i-th angle of its token on
      auto turn = [&](int j, int i) {
        const float2 q = cs[i + j];
        out.set(j, f[2 * j] * q.x - f[2 * j + 1] * q.y, f[2 * j] * q.y + f[2 * j + 1] * q.x);
      };
      if (kAnyPair) {
        out.copy(v[k]);
        if (at[k] >= 0) {
          const int pairs = a.r / 2, i0 = (first - a.start) / 2 + (at[k] & 0xFFFF) * (kUnit / 2);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((uint32_t)(i0 + j) < (uint32_t)pairs) turn(j, (at[k] >> 16) * pairs + i0);
          if (kMode == kRaggedInPlace && (i0 < 0 || i0 + 4 > pairs)) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if ((uint32_t)(i0 + j) < (uint32_t)pairs) out.store_pair(y + to[k], j);
            continue;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) turn(j, at[k]);
      }
      out.store(y + to[k]);
    }
  }
}

// Any shape.  Units of a head: r / 2 pairs; then, unless y is x, copied channels one by one and, kWhole, where rows are
// of whole 16 bytes, 8 by 8 those of loads without a rotated channel.
template <typename In, typename Out, bool kWhole>
__global__ void __launch_bounds__(kThreads) k_rope_any(RopePlan pl) {
  __shared__ float2 cs[kMaxAngles];
  const RopeArgs& a = pl.a;
  pdl_wait();
  int64_t t0;
  uint32_t before;
  first_unit(pl, &t0, &before);
  rotations(a, t0, pl.tokens, cs);
  __syncthreads();
  const In* x = static_cast<const In*>(a.x);
  Out* y = static_cast<Out*>(a.y);
  const int total = (int)min((int64_t)pl.span, pl.total - (int64_t)blockIdx.x * pl.span), pairs = a.r / 2;
  const int first = kWhole ? a.start & ~(kUnit - 1) : 0, width = kWhole ? touched_units(a) * kUnit : a.d;
  const int ones = pairs + width - a.r;             // units below: a pair or a channel
  constexpr int kMany = sizeof(In) == 4 ? 2 : 4;    // units in flight
  for (int u0 = threadIdx.x; u0 < total; u0 += kMany * kThreads) {
    Eight<In> v[kMany];
    float x1[kMany], x2[kMany];
    int64_t to[kMany];
    int c2[kMany], at[kMany];                       // second channel, angle; at -1: copied; -2: nothing; -3: copied 8
#pragma unroll
    for (int k = 0; k < kMany; ++k) {
      const uint32_t u = u0 + k * kThreads;
      at[k] = -2;
      to[k] = c2[k] = 0;
      if (u >= (uint32_t)total) continue;
      uint32_t t, h, unit;
      pl.per_token.split(before + u, &t, &unit);
      pl.units.split(unit, &h, &unit);
      int c;
      if ((int)unit < pairs) {
        c = a.start + (a.layout == CSA2_ROPE_HALF ? (int)unit : 2 * (int)unit);
        c2[k] = a.layout == CSA2_ROPE_HALF ? pairs : 1;
        at[k] = t * pairs + unit;
      } else if (!kWhole || (int)unit < ones) {
        c = first + unit - pairs;
        if (c >= a.start) c += a.r;
        at[k] = -1;
      } else {
        c = (unit - ones) * kUnit;
        if (c >= first) c += width;
        at[k] = -3;
      }
      const In* p = x + (t0 + t) * a.x_token + (int64_t)h * a.x_head + c;
      to[k] = (t0 + t) * a.y_token + (int64_t)h * a.y_head + c;
      if (kWhole && at[k] == -3) v[k].load(p);
      else x1[k] = to_f32(*p);
      if (at[k] >= 0) x2[k] = to_f32(p[c2[k]]);
    }
#pragma unroll
    for (int k = 0; k < kMany; ++k) {
      if (at[k] == -2) continue;
      if (kWhole && at[k] == -3) {
        Result<Out> out;
        out.copy(v[k]);
        out.store(y + to[k]);
        continue;
      }
      if (at[k] >= 0) {
        const float2 z = cs[at[k]];
        const float f1 = x1[k] * z.x - x2[k] * z.y;
        store1(y + to[k] + c2[k], x1[k] * z.y + x2[k] * z.x);
        store1(y + to[k], f1);
      } else {
        copy1<In>(y + to[k], x1[k]);
      }
    }
  }
}

// The table comes from the host with the launch, 256 pairs at a time.
struct RopeTable {
  uint64_t g[256];
};
__global__ void __launch_bounds__(256) k_rope_table(const __grid_constant__ RopeTable t, int n, uint64_t* out) {
  pdl_wait();
  if (threadIdx.x < n) out[threadIdx.x] = t.g[threadIdx.x];
}

template <typename In, typename Out>
cudaError_t launch_typed(const RopePlan& pl, int64_t grid, Mode mode, cudaStream_t s) {
  const auto kernel = mode == kHalves    ? k_rope<In, Out, kHalves>
                      : mode == kRagged  ? k_rope<In, Out, kRagged>
                      : mode == kRaggedInPlace ? k_rope<In, In, kRaggedInPlace>
                      : mode == kOnes    ? k_rope_any<In, Out, false>
                      : mode == kOnesWhole ? k_rope_any<In, Out, true>
                                         : k_rope<In, Out, kInterleaved>;
  return launch_step(kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, pl);
}

}  // namespace

cudaError_t launch_rope_table(const uint64_t* turns, int pairs, uint64_t* out, cudaStream_t s) {
  for (int i = 0; i < pairs; i += 256) {
    RopeTable t = {};
    const int n = std::min(256, pairs - i);
    std::copy(turns + i, turns + i + n, t.g);
    const cudaError_t e = launch_step(k_rope_table, dim3(1), dim3(256), 0, s, t, n, out + i);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  const bool in_place = a.x == a.y, half = a.layout == CSA2_ROPE_HALF;
  const int in = a.x_dtype == CSA2_F32 ? 4 : 2, out = a.y_dtype == CSA2_F32 ? 4 : 2;
  auto whole = [](const void* p, int64_t token, int64_t head, int size) {   // rows start on 16 bytes
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && token * size % 16 == 0 && head * size % 16 == 0;
  };
  const bool eight = a.d % kUnit == 0 && whole(a.x, a.x_token, a.x_head, in) && whole(a.y, a.y_token, a.y_head, out);
  const Mode mode = !eight ? kOnes
                    : half ? (a.start % kUnit == 0 && a.r % (2 * kUnit) == 0 ? kHalves : kOnesWhole)
                           : (a.start % 2 != 0 ? kOnesWhole : a.start % kUnit == 0 && a.r % kUnit == 0 ? kInterleaved : in_place ? kRaggedInPlace : kRagged);
  int units, copied;                        // of a head: in all, copied ones of them
  switch (mode) {
    case kOnes: units = a.d - a.r / 2, copied = a.d - a.r; break;
    case kOnesWhole: copied = 7 * touched_units(a) + a.d / kUnit - a.r, units = a.r / 2 + copied; break;
    default: units = a.d / kUnit - (half ? a.r / 16 : 0), copied = units - rotated_units(a, mode);
  }
  if (in_place) units -= copied;
  if (units == 0) return cudaSuccess;       // (nothing rotated)
  RopePlan pl;
  pl.a = a;
  // A block: 2,048 units (8 a thread), fewer where there are few, so
  // that every SM has work (one token of 64 heads x 512 channels goes to 64 blocks), and no more tokens than there is
  // shared memory for their angles.
  const int64_t per_token = (int64_t)a.heads * units;
  if (per_token > 1 << 30) {                // (positions in a token, with a block's units behind them, fit 31 bits)
    RopeArgs b = a;
    b.heads = a.heads / 2;
    const cudaError_t e = launch_rope(b, s);
    if (e != cudaSuccess) return e;
    b.heads = a.heads - b.heads;
    b.x = static_cast<const uint8_t*>(a.x) + (a.heads - b.heads) * a.x_head * in;
    b.y = static_cast<uint8_t*>(a.y) + (a.heads - b.heads) * a.y_head * out;
    return launch_rope(b, s);
  }
  const int pairs = std::max(1, a.r / 2);
  pl.total = a.rows * per_token;
  pl.far = pl.total > INT_MAX;
  pl.span = (int)std::min<int64_t>(std::max<int64_t>(64, std::min<int64_t>(2048, pl.total / (2 * 152))), (kMaxAngles / pairs - 1) * per_token);
  pl.tokens = (int)((pl.span - 2) / per_token) + 2;
  if (pl.span % per_token == 0) pl.tokens = (int)(pl.span / per_token);
  pl.per_token = Divisor::of((uint32_t)per_token);
  pl.units = Divisor::of(units);
  const int64_t grid = (pl.total + pl.span - 1) / pl.span;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  if (a.x_dtype == CSA2_F32)
    return a.y_dtype == CSA2_F32 ? launch_typed<float, float>(pl, grid, mode, s) : launch_typed<float, uint16_t>(pl, grid, mode, s);
  return a.y_dtype == CSA2_F32 ? launch_typed<uint16_t, float>(pl, grid, mode, s) : launch_typed<uint16_t, uint16_t>(pl, grid, mode, s);
}

}  // namespace csa2
