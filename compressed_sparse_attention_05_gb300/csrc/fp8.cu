// FP8 rows with one scale per block of 128 columns (reading R18) and their matrix product (R19):
//   C[m][n] = sum_kb sa[m][kb] sb[n/128][kb] sum_{k in block kb} a[m][k] b[n][k].
//
// A block's 128 products are summed by the tensor cores (tcgen05.mma, kind::f8f6f4, E4M3 x E4M3, fp32
// accumulation) into a tensor-memory accumulator of their own; the accumulator is then read back, multiplied by the
// block's two scales and added to the sum in registers, while the tensor cores work on the next block's.
//
// k_matmul_fp8_wide (many rows of A, or more rows of B than the SMs take 128 at a time): tiles of 128 rows of A x 256 rows
//   of B.  A row of A is a lane of the accumulator, so a thread has one scale per block: sa[its row] sb[its 128 columns].
//   4,096 x 32,768 x 4,096 takes 440 us (2.5 PFLOP/s) at first and 458 to 466 (2.4) in a row, at the card's 1,400 W, which
//   sets the clock (1.91 GHz, with zeros 1.96) but not the cycles: a block takes 963 of them, its MMAs 513 (the tensor pipe
//   is active for 52%).  The sums and their hand-over set the pace: a warp waits 200 cycles for an accumulator, releases it 400 after that (four
//   loads of 32 columns with their additions) and adds the rest, while the MMA warp waits 430 for a free one of the two (all
//   of tensor memory); operands are always ahead (the copy warp waits 720 for a free stage).
//   Tried: a pair of CTAs with one MMA for both (cta_group::2; its arrivals from SM to SM are too slow for this way:
//   480 us), 16 sum warps (570, registers), halves of the accumulator on their own (478), named barriers in the place of
//   shared-memory ones, loads and looks ahead in the sums (no difference).
// k_matmul_fp8_thin (few rows of A, or few tiles): the rows of B, the weights, are the MMA's M side, 128 at a time, and
//   16 to 128 rows of A its N side, so that no part of the tensor cores' work and of shared memory goes to rows that are
//   not there, and 128 B-rows x 128 columns (16 KB) per block stream through a deep ring.  A thread has a weight row and
//   up to 32 rows of A; their scales go through shared memory.  32 x 32,768 x 4,096: 24.8 us, 5.5 TB/s.
//   Where its tiles do not fill the SMs, the blocks of K are split over several CTAs, which leave fp32 partial sums that
//   k_matmul_fp8_sum adds in order.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "operands.cuh"
#include "tc.cuh"
#include "tma.cuh"

namespace csa2 {
namespace {

constexpr int kBlock = 128;                // columns that share a scale (and rows of B)

// ---- packing --------------------------------------------------------------------------------------
// amax of a block's 128 values, a = max(amax, 2^-100); scale a / 448, codes E4M3_rne_satfinite(x * (448 / a)).
// Bytes bound it, and instructions not far behind (a block of bf16 leaves 66 issue slots per SM): a lane loads 16 bytes,
// so a block is 16 lanes of bf16 or 32 of fp32, and 2, 4 .. lanes where rows are shorter than half a block; every group
// of lanes takes two blocks, both loads in flight, and divides for both at once, in an even and an odd lane.
// 16,411 x 4,240 of fp32 in a wider tensor: 53 us, 6.6 TB/s.  460,166 x 96 of bf16: 26.5 us (a warp a block, 8-byte
// loads: 44); 2,368,205 x 16 of fp32: 33 us (204).
constexpr int kPackThreads = 256, kPackMany = 2;
constexpr float kFloor = 0x1p-100f;

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{ .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n mov.b32 %0, {lo, hi}; }"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// The larger of each half (bf16); a NaN only where both are.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// kLanes = 2^lanes_log: lanes of a block; kLanes 0: fewer than a whole block has, at least 2.  many: blocks of a group of lanes (at most
// kPackMany).
template <bool kF32, int kLanes>
__global__ void __launch_bounds__(kPackThreads, 8) k_pack_fp8_blocks(const void* x, int64_t stride, int K, Divisor per_row, uint32_t blocks,
                                                                     int many, int lanes_log, uint8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int kCols = kF32 ? 4 : 8;               // of a lane: 16 bytes
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, n_lanes = kLanes ? kLanes : 1 << lanes_log, groups = 32 >> lanes_log;
  const uint32_t b0 = (blockIdx.x * (kPackThreads / 32) + (threadIdx.x >> 5)) * (uint32_t)(many * groups);
  if (b0 >= blocks) return;
  const int col0 = (lane & (n_lanes - 1)) * kCols;
  uint32_t b[kPackMany];
  int64_t at[kPackMany];                            // in codes; -1: nothing
  uint4 v[kPackMany];
#pragma unroll
  for (int i = 0; i < kPackMany; ++i) {
    b[i] = b0 + i * groups + (kLanes == 32 ? 0 : lane >> lanes_log);
    v[i] = make_uint4(0, 0, 0, 0);
    at[i] = -1;
    if (i >= many || b[i] >= blocks) {
      b[i] = blocks;
      continue;
    }
    uint32_t row, kb;
    per_row.split(b[i], &row, &kb);
    const int col = (int)kb * kBlock + col0;
    if (col >= K) continue;
    const int64_t from = row * stride + col;
    v[i] = __ldg(reinterpret_cast<const uint4*>(kF32 ? static_cast<const void*>(static_cast<const float*>(x) + from)
                                                     : static_cast<const void*>(static_cast<const uint16_t*>(x) + from)));
    at[i] = (int64_t)row * K + col;
  }
  // The blocks' largest magnitudes, in every lane of the group.  (The maxima drop a NaN.)
  float amax[kPackMany];
  if (kF32) {
#pragma unroll
    for (int i = 0; i < kPackMany; ++i) {
      const float m = fmaxf(fmaxf(fmaxf(0.f, fabsf(__uint_as_float(v[i].x))), fabsf(__uint_as_float(v[i].y))),
                            fmaxf(fmaxf(0.f, fabsf(__uint_as_float(v[i].z))), fabsf(__uint_as_float(v[i].w))));
      uint32_t w = __float_as_uint(m);              // (orders like the values)
      if (kLanes == 32) {
        w = __reduce_max_sync(0xffffffffu, w);
      } else {
#pragma unroll 1
        for (int o = n_lanes / 2; o > 0; o >>= 1) w = max(w, __shfl_xor_sync(0xffffffffu, w, o));
      }
      amax[i] = __uint_as_float(w);
    }
  } else {
    uint32_t m[kPackMany];
#pragma unroll
    for (int i = 0; i < kPackMany; ++i)
      m[i] = max_bf16x2(max_bf16x2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu), max_bf16x2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
    static_assert(kPackMany == 2, "a half-word for each");
    uint32_t w = max_bf16x2(prmt(m[0], m[1], 0x5410), prmt(m[0], m[1], 0x7632));
#pragma unroll
    for (int o = kLanes ? kLanes / 2 : 8; o > 0; o >>= 1)
      if (kLanes || o < n_lanes) w = max_bf16x2(w, __shfl_xor_sync(0xffffffffu, w, o));
    amax[0] = __uint_as_float(w << 16);
    amax[1] = __uint_as_float(w & 0xFFFF0000u);
  }
  // The divisions: an even lane block 0's, an odd lane block 1's.
  const int mine = lane & 1;
  const float a = fmaxf(mine ? amax[1] : amax[0], kFloor), inv = 448.f / a;
  const uint32_t b_mine = mine ? b[1] : b[0];
  if ((lane & (n_lanes - 1)) < kPackMany && b_mine < blocks) scales[b_mine] = a / 448.f;
#pragma unroll
  for (int i = 0; i < kPackMany; ++i) {
    const float q = __shfl_sync(0xffffffffu, inv, (lane & ~1) | i);
    if (at[i] < 0) continue;
    if (kF32) {
      *reinterpret_cast<uint32_t*>(codes + at[i]) = e4m3x4(__uint_as_float(v[i].x) * q, __uint_as_float(v[i].y) * q, __uint_as_float(v[i].z) * q,
                                                           __uint_as_float(v[i].w) * q);
    } else {
      auto lo = [&](uint32_t w) { return __uint_as_float(w << 16) * q; };
      auto hi = [&](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u) * q; };
      *reinterpret_cast<uint2*>(codes + at[i]) =
          make_uint2(e4m3x4(lo(v[i].x), hi(v[i].x), lo(v[i].y), hi(v[i].y)), e4m3x4(lo(v[i].z), hi(v[i].z), lo(v[i].w), hi(v[i].w)));
    }
  }
}

// ---- the product ------------------------------------------------------------------------------------
struct MatmulPlan {
  const float* sa;          // [M][kb]
  const float* sb;          // [ceil(N / 128)][kb]
  void* C;                  // [M][N], or null: partial sums
  float* partial;           // [n_split][M][ld]
  int64_t ld;
  int M, N, kb, n_split, f32;
  int c_map;                // C's rows start on 16 bytes: it is written by tensor-map copies
  int m_tiles, n_tiles;
};

constexpr uint32_t kIdFp8 = 1u << 4;   // instruction descriptor: fp32 accumulation, E4M3 x E4M3, both K-major
__host__ __device__ constexpr uint32_t idesc_fp8(int M, int N) { return kIdFp8 | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }

// D[tmem] (+)= A . B^T of E4M3, issued by one lane of a warp that runs as a whole (tc::elect_lane): from a single thread's
// branch a block's four MMAs with their two commits took longer to issue than the 513 cycles that they run.
__device__ __forceinline__ void mma_fp8(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 e, %5, 0;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// The MMA warp's wait for two barriers with one look at a time: lane i looks at its own (bar, parity); `need`
// has the bits of the lanes that count.  Never suspends; bounded.
__device__ __forceinline__ bool wait_lanes(uint32_t bar, uint32_t parity, uint32_t need, volatile int* abort) {
#pragma unroll 1
  for (uint32_t i = 0; i < (1u << 25); ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if ((__ballot_sync(0xffffffffu, ok != 0) & need) == need) return true;
    if ((i & 255) == 255 && __any_sync(0xffffffffu, *abort != 0)) return false;
  }
  *abort = 1;
  return false;
}
// K-major operand rows of 128 bytes as a tensor map writes them with the 128-byte swizzle.
__device__ __forceinline__ uint64_t desc128(uint32_t saddr) { return tc::smem_desc(saddr, 16, 1024) | ((uint64_t)2 << 61); }

// Bounded wait; on time-out the CTA's abort flag is raised.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (uint32_t i = 0; i < (1u << 21); ++i) {   // <= 2^21 suspensions of <= 1 us
    if (tc::mbar_try_wait_sleep(bar, parity, 1000)) return true;
    if ((i & 63) == 63 && *abort) return false;
  }
  *abort = 1;
  return false;
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// The loads of this warp have arrived (r is named, so that nothing that uses it moves ahead of the wait).
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// (a.x b.x + c.x, a.y b.y + c.y)
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{ .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// The blocks [k0, k1) of split s.
__device__ __forceinline__ void split_range(const MatmulPlan& p, int s, int* k0, int* k1) {
  *k0 = (int)((int64_t)s * p.kb / p.n_split);
  *k1 = (int)((int64_t)(s + 1) * p.kb / p.n_split);
}

// The barriers of a ring of operand stages and of the accumulators.
template <typename Smem>
__device__ __forceinline__ void ring_init(Smem& sm, int stages, int bufs, uint32_t readers) {
  for (int i = 0; i < stages; ++i) {
    tc::mbar_init(&sm.full[i], 1);
    tc::mbar_init(&sm.empty[i], 1);
  }
  for (int i = 0; i < bufs; ++i) {
    tc::mbar_init(&sm.acc_full[i], 1);
    tc::mbar_init(&sm.acc_empty[i], readers);
  }
  sm.abort = 0;
  tc::mbar_fence_init();
}

// ---- many rows of A ----
constexpr int kWM = 128, kWN = 256, kWStages = 4, kWBufs = 2;
constexpr int kWStageBytes = (kWM + kWN) * kBlock;       // 48 KB
constexpr int kWSumWarps = 8;
constexpr int kWThreads = kWSumWarps * 32 + 128;
// Registers: 2 x 216 + 72 = 3 x 168, without spills.  (Splits that make the compiler spill in one role's loop take up to
// twice as long.)
constexpr int kWRegs = 168;
constexpr int kWRegsSum = 216, kWRegsMisc = 72;
struct WideSmem {
  unsigned char stage[kWStages][kWStageBytes];   // 1024-aligned
  unsigned char out[kWSumWarps][4096];           // of each sum warp: 32 rows x 128 bytes of C on their way out
  uint64_t full[kWStages], empty[kWStages], acc_full[kWBufs], acc_empty[kWBufs];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(WideSmem) + 1024 <= 232448, "shared memory");

// 32 rows x 128 bytes of C (lane = row, piece j of 16 bytes: get(j)) from row y, column x on, through the warp's staging
// rows: by a tensor-map copy where C's rows start on 16 bytes, else row by row with a lane to an element.  (Written by the
// threads themselves, each along its own row, C took 75 of 520 us of a product of 4,096 x 32,768 x 4,096 with 16 bytes
// at a time, and 119 us for 351 x 27,102 element by element.)
template <typename T, typename Get>
__device__ __forceinline__ void store_box(unsigned char* stage, const CUtensorMap* map, const MatmulPlan& p, int x, int y, int lane, Get get) {
  constexpr int kCols = 128 / (int)sizeof(T);
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the box before has left
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = get(j);   // 128-byte swizzle
  if (p.c_map) {
    tc::fence_async_smem();
    __syncwarp();
    if (lane == 0 && y < p.M && x < p.N)     // (the copy leaves out what lies outside of C)
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\tcp.async.bulk.commit_group;" ::"l"(
                       reinterpret_cast<uint64_t>(map)),
                   "r"(x), "r"(y), "r"(tc::smem_addr(stage))
                   : "memory");
    return;
  }
  __syncwarp();
  T* out = static_cast<T*>(p.C) + (int64_t)y * p.N + x;
  const int rows = min(32, p.M - y), cols = min(kCols, p.N - x);
#pragma unroll 2
  for (int r = 0; r < rows; ++r)
#pragma unroll
    for (int c = lane; c < kCols; c += 32)
      if (c < cols) {
        const int at = c * (int)sizeof(T);
        out[(int64_t)r * p.N + c] = *reinterpret_cast<const T*>(stage + r * 128 + (((at >> 4) ^ (r & 7)) << 4) + (at & 15));
      }
  __syncwarp();
}

__global__ void __launch_bounds__(kWThreads, 1)
k_matmul_fp8_wide(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, const __grid_constant__ CUtensorMap cmap,
                  const __grid_constant__ MatmulPlan p, uint32_t* status) {
  extern __shared__ unsigned char smem_raw[];
  WideSmem& sm = *reinterpret_cast<WideSmem*>(smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) ring_init(sm, kWStages, kWBufs, kWSumWarps);
  if (warp == kWSumWarps) tc::tmem_alloc(&sm.tmem, kWBufs * kWN);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tm = sm.tmem;
  volatile int* abort = &sm.abort;
  pdl_wait();
  // the tiles of a column after one another
  const int items = p.m_tiles * p.n_tiles;   // (below 2^31)
  struct Item {
    int m0, n0;   // first row and column
  };
  auto item = [&](int it) {
    const int n = it / p.m_tiles;
    return Item{(it - n * p.m_tiles) * kWM, n * kWN};
  };

  if (warp >= kWSumWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWRegsMisc));
    if (warp == kWSumWarps && lane == 0) {
      // ================= operand copies =================
      uint32_t n = 0;
      bool ok = true;
      for (int it = blockIdx.x; ok && it < items; it += gridDim.x) {
        const Item w = item(it);
        for (int k = 0; k < p.kb; ++k, ++n) {
          const uint32_t st = n % kWStages, use = n / kWStages;
          if (use > 0 && !wait_bar(&sm.empty[st], (use - 1) & 1, abort)) {
            ok = false;
            break;
          }
          tc::mbar_arrive_expect_tx(&sm.full[st], kWStageBytes);
          tma::load_2d(sm.stage[st], &amap, k * kBlock, w.m0, &sm.full[st]);
          tma::load_2d(sm.stage[st] + kWM * kBlock, &bmap, k * kBlock, w.n0, &sm.full[st]);
        }
      }
      for (uint32_t i = n > kWStages ? n - kWStages : 0; i < n; ++i)   // every issued copy lands before exit
        for (uint32_t t = 0; t < (1u << 22); ++t)
          if (tc::mbar_try_wait(&sm.full[i % kWStages], (i / kWStages) & 1)) break;
    } else if (warp == kWSumWarps + 1) {
      // ================= MMA issue =================
      constexpr uint32_t idesc = idesc_fp8(kWM, kWN);
      const uint32_t leader = tc::elect_lane();
      uint32_t n = 0;
      bool ok = true;
      for (int it = blockIdx.x; ok && it < items; it += gridDim.x) {
        const Item w = item(it);
        for (int k = 0; k < p.kb; ++k, ++n) {
          const uint32_t st = n % kWStages, buf = n % kWBufs, use = n / kWBufs;
          ok = wait_lanes(tc::smem_addr(lane == 1 ? &sm.acc_empty[buf] : &sm.full[st]), lane == 1 ? (use - 1) & 1 : (n / kWStages) & 1,
                          use > 0 ? 3u : 1u, abort);
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t sa = tc::smem_addr(sm.stage[st]), sb = sa + kWM * kBlock;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_fp8(leader, tm + buf * kWN, desc128(sa + 32 * ks), desc128(sb + 32 * ks), idesc, ks > 0);
          tc::mma_commit_by(leader, &sm.acc_full[buf]);
          tc::mma_commit_by(leader, &sm.empty[st]);
        }
      }
    }
    __syncwarp();
  } else {
    // ================= scales and sums: thread = row of A, 128 columns =================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWRegsSum));
    const int lq = warp & 3, half = warp >> 2;
    const uint32_t t0 = tm + ((uint32_t)(32 * lq) << 16) + 128 * half;
    const bool vec = p.kb % 4 == 0;   // (the scales' rows start on 16 bytes)
    uint32_t n = 0;
    bool ok = true;
    for (int it = blockIdx.x; ok && it < items; it += gridDim.x) {
      const Item w = item(it);
      const int y = w.m0 + 32 * lq, n0 = w.n0 + 128 * half;
      const int m = y + lane < p.M ? y + lane : 0, nb = n0 < p.N ? n0 / kBlock : 0;   // rows of the scales
      float2 acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
      // Scales four blocks at a time: a row's lie behind one another, so that a warp's load touches 32 lines whether it
      // takes 4 bytes of each or 16.
      float4 sc;
      auto block = [&](float both) {
        const uint32_t buf = n % kWBufs;
        ok = __all_sync(0xffffffffu, wait_bar(&sm.acc_full[buf], (n / kWBufs) & 1, abort));
        if (!ok) return;
        tc::tc_fence_after();
        ++n;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(t0 + buf * kWN + 32 * c, r);
          tmem_wait32(r);
          if (c == 3) {       // the accumulator has been read
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm.acc_empty[buf]);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[16 * c + j] = fma2(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), make_float2(both, both), acc[16 * c + j]);
        }
      };
#pragma unroll 1
      for (int k = 0; ok && k < p.kb; ++k) {
        const int i = k & 3;
        if (i == 0) {
          const float* sa = p.sa + (int64_t)m * p.kb + k;
          const float* sb = p.sb + (int64_t)nb * p.kb + k;
          if (vec) {
            const float4 fa = __ldg(reinterpret_cast<const float4*>(sa)), fb = __ldg(reinterpret_cast<const float4*>(sb));
            sc = make_float4(fa.x * fb.x, fa.y * fb.y, fa.z * fb.z, fa.w * fb.w);
          } else {
            auto at = [&](int j) { return k + j < p.kb ? __ldg(sa + j) * __ldg(sb + j) : 0.f; };
            sc = make_float4(at(0), at(1), at(2), at(3));
          }
        }
        block(i == 0 ? sc.x : i == 1 ? sc.y : i == 2 ? sc.z : sc.w);
      }
      if (!ok) break;
      unsigned char* stage = sm.out[warp];
      if (p.f32) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          store_box<float>(stage, &cmap, p, n0 + 32 * b, y, lane, [&](int j) {
            const float2 u = acc[16 * b + 2 * j], v = acc[16 * b + 2 * j + 1];
            return make_uint4(__float_as_uint(u.x), __float_as_uint(u.y), __float_as_uint(v.x), __float_as_uint(v.y));
          });
      } else {
#pragma unroll
        for (int b = 0; b < 2; ++b)
          store_box<uint16_t>(stage, &cmap, p, n0 + 64 * b, y, lane, [&](int j) {
            const float2* u = acc + 32 * b + 4 * j;
            return make_uint4(f32x2_bf16x2(u[0].x, u[0].y), f32x2_bf16x2(u[1].x, u[1].y), f32x2_bf16x2(u[2].x, u[2].y), f32x2_bf16x2(u[3].x, u[3].y));
          });
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kWSumWarps) tc::tmem_dealloc(tm, kWBufs * kWN);
  if (tid == 0 && *abort) raise_status(status, CSA2_STATUS_TIMEOUT);
}

// ---- few rows of A, or few tiles ----
// A tile is 128 rows of B x kRows (16 to 128) rows of A.
constexpr int kTN = 128, kTBufs = 4;                // rows of B; accumulators
template <int kRows> constexpr int kTSumWarps = kRows > 64 ? 16 : kRows > 16 ? 8 : 4;   // groups of four share the rows of A
template <int kRows> constexpr int kTThreads = (kTSumWarps<kRows> + 2) * 32;
template <int kRows> constexpr int kTOwn = kRows / (kTSumWarps<kRows> / 4);   // rows of A of a sum warp: 16, 16, 32, 32
template <int kRows> constexpr int kTStageBytes = (kTN + kRows) * kBlock;
// CTAs that an SM can hold.  With more tiles than SMs two of them, with half the ring each, read at the same time, and
// no second wave of tiles leaves SMs idle: 32 x 32,768 x 4,096 takes 25.1 us instead of 27.5.
template <int kRows> constexpr int kTCtas = kRows <= 64 ? 2 : 1;
constexpr int kTRingBytes = 200 * 1024, kTMaxStages = kTRingBytes / kTStageBytes<16>;
template <int kRows>
struct ThinSmem {              // the ring's stages follow, 1024-aligned
  uint64_t full[kTMaxStages], empty[kTMaxStages], acc_full[kTBufs], acc_empty[kTBufs];
  alignas(16) float scale[kTSumWarps<kRows>][2][kTOwn<kRows>];   // of a block, for all lanes of a warp
  uint32_t tmem;
  int abort;
};
template <int kRows> constexpr size_t kTSmemBytes(int stages) { return 1024 + (sizeof(ThinSmem<kRows>) + 1023) / 1024 * 1024 + (size_t)stages * kTStageBytes<kRows>; }

template <int kRows>
__global__ void __launch_bounds__(kTThreads<kRows>, kTCtas<kRows>)
k_matmul_fp8_thin(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, const __grid_constant__ MatmulPlan p,
                  int n_stages, uint32_t* status) {
  extern __shared__ unsigned char smem_raw[];
  using Smem = ThinSmem<kRows>;
  constexpr int kBytes = kTStageBytes<kRows>, kSumWarps = kTSumWarps<kRows>, kOwn = kTOwn<kRows>;
  unsigned char* base = smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u);
  Smem& sm = *reinterpret_cast<Smem*>(base);
  unsigned char* ring = base + (sizeof(Smem) + 1023) / 1024 * 1024;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (p.partial) pdl_trigger();
  constexpr uint32_t kCols = kTBufs * kRows;        // 64 to 512 columns
  if (tid == 0) ring_init(sm, n_stages, kTBufs, kSumWarps);
  if (warp == kSumWarps) tc::tmem_alloc(&sm.tmem, kCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tm = sm.tmem;
  volatile int* abort = &sm.abort;
  pdl_wait();
  const int items = p.m_tiles * p.n_tiles * p.n_split;   // (below 2^31)
  struct Item {
    int s, m0, n0, k0, k1;   // split, first rows of A and of B, blocks of K
  };
  auto item = [&](int it) {
    Item w;
    const int tile = it / p.n_split;
    w.s = it - tile * p.n_split;
    w.n0 = tile / p.m_tiles;
    w.m0 = (tile - w.n0 * p.m_tiles) * kRows;
    w.n0 *= kTN;
    split_range(p, w.s, &w.k0, &w.k1);
    return w;
  };

  if (warp == kSumWarps) {
    // ================= operand copies =================
    if (lane == 0) {
      int st = 0;
      uint32_t round = 0;                 // uses of the stage before this one
      bool ok = true;
      for (int it = blockIdx.x; ok && it < items; it += gridDim.x) {
        const Item w = item(it);
        for (int k = w.k0; k < w.k1; ++k) {
          if (round > 0 && !wait_bar(&sm.empty[st], (round - 1) & 1, abort)) {
            ok = false;
            break;
          }
          unsigned char* stage = ring + st * kBytes;
          tc::mbar_arrive_expect_tx(&sm.full[st], kBytes);
          tma::load_2d(stage, &bmap, k * kBlock, w.n0, &sm.full[st]);
          tma::load_2d(stage + kTN * kBlock, &amap, k * kBlock, w.m0, &sm.full[st]);
          if (++st == n_stages) {
            st = 0;
            ++round;
          }
        }
      }
      // every issued copy lands before exit: the last use of stage i is `round` where i < st, else the one before
      for (int i = 0; i < n_stages; ++i) {
        if (i >= st && round == 0) break;
        for (uint32_t w = 0; w < (1u << 22); ++w)
          if (tc::mbar_try_wait(&sm.full[i], (i < st ? round : round - 1) & 1)) break;
      }
    }
    __syncwarp();
  } else if (warp == kSumWarps + 1) {
    // ================= MMA issue =================
    constexpr uint32_t idesc = idesc_fp8(kTN, kRows);
    const uint32_t leader = tc::elect_lane();
    uint32_t n = 0, phase = 0;
    int st = 0;
    bool ok = true;
    for (int it = blockIdx.x; ok && it < items; it += gridDim.x) {
      const Item w = item(it);
      for (int k = w.k0; k < w.k1; ++k, ++n) {
        const uint32_t buf = n % kTBufs, use = n / kTBufs;
        ok = wait_lanes(tc::smem_addr(lane == 1 ? &sm.acc_empty[buf] : &sm.full[st]), lane == 1 ? (use - 1) & 1 : phase,
                        use > 0 ? 3u : 1u, abort);
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t sw = tc::smem_addr(ring) + st * kBytes, sx = sw + kTN * kBlock;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_fp8(leader, tm + buf * kRows, desc128(sw + 32 * ks), desc128(sx + 32 * ks), idesc, ks > 0);
        tc::mma_commit_by(leader, &sm.empty[st]);
        tc::mma_commit_by(leader, &sm.acc_full[buf]);
        if (++st == n_stages) {
          st = 0;
          phase ^= 1;
        }
      }
    }
    __syncwarp();
  } else {
    // ================= scales and sums: thread = row of B, kOwn rows of A =================
    constexpr int kHeld = (kOwn + 31) / 32;          // rows of A whose scales a lane reads
    const int lq = warp & 3, own0 = (warp >> 2) * kOwn;
    const bool vec = p.kb % 4 == 0;                  // (the scales' rows start on 16 bytes)
    uint32_t n = 0;
    bool ok = true;
    for (int it = blockIdx.x; ok && it < items; it += gridDim.x) {
      const Item w = item(it);
      const int m0 = w.m0 + own0;
      const float* sb = p.sb + (int64_t)(w.n0 / kBlock) * p.kb;
      float2 acc[kOwn / 2];
#pragma unroll
      for (int j = 0; j < kOwn / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      float4 sc[kHeld];
#pragma unroll 1
      for (int k = w.k0; k < w.k1; ++k, ++n) {
        const int i = k & 3, q = k & ~3;
        if (k == w.k0 || i == 0) {                   // the scales of four blocks
#pragma unroll
          for (int h = 0; h < kHeld; ++h) {
            const int m = m0 + lane + 32 * h;
            const float* sa = p.sa + (int64_t)(m < p.M ? m : 0) * p.kb;
            if (vec) {
              const float4 a = __ldg(reinterpret_cast<const float4*>(sa + q)), b = __ldg(reinterpret_cast<const float4*>(sb + q));
              sc[h] = make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
            } else {
              auto at = [&](int j) { return q + j < p.kb ? __ldg(sa + q + j) * __ldg(sb + q + j) : 0.f; };
              sc[h] = make_float4(at(0), at(1), at(2), at(3));
            }
          }
        }
        float* shared = sm.scale[warp][n & 1];
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
          if (lane + 32 * h < kOwn) shared[lane + 32 * h] = i == 0 ? sc[h].x : i == 1 ? sc[h].y : i == 2 ? sc[h].z : sc[h].w;
        __syncwarp();
        const uint32_t buf = n % kTBufs;
        ok = __all_sync(0xffffffffu, wait_bar(&sm.acc_full[buf], (n / kTBufs) & 1, abort));
        if (!ok) break;
        tc::tc_fence_after();
#pragma unroll
        for (int c = 0; c < kOwn; c += 16) {
          uint32_t r[16];
          tmem_ld16(tm + ((uint32_t)(32 * lq) << 16) + buf * kRows + own0 + c, r);
          tmem_wait16(r);
          if (c + 16 == kOwn) {   // the accumulator has been read
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm.acc_empty[buf]);
          }
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(shared + c + j);
            acc[(c + j) / 2] = fma2(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), make_float2(f.x, f.y), acc[(c + j) / 2]);
            acc[(c + j) / 2 + 1] = fma2(make_float2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])), make_float2(f.z, f.w), acc[(c + j) / 2 + 1]);
          }
        }
      }
      const int col = w.n0 + 32 * lq + lane;
      if (!ok || col >= p.N) continue;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        if (m0 + j >= p.M) break;
        const float v = j & 1 ? acc[j / 2].y : acc[j / 2].x;
        if (p.partial) p.partial[((int64_t)w.s * p.M + m0 + j) * p.ld + col] = v;
        else if (p.f32) static_cast<float*>(p.C)[(int64_t)(m0 + j) * p.N + col] = v;
        else static_cast<uint16_t*>(p.C)[(int64_t)(m0 + j) * p.N + col] = (uint16_t)(f32x2_bf16x2(v, 0.f) & 0xFFFFu);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kSumWarps) tc::tmem_dealloc(tm, kCols);
  if (tid == 0 && *abort) raise_status(status, CSA2_STATUS_TIMEOUT);
}

// The splits' partial sums, in order.
__global__ void __launch_bounds__(256) k_matmul_fp8_sum(const __grid_constant__ MatmulPlan p) {
  pdl_wait();
  const int64_t m = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (m >= p.M || n >= p.N) return;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < p.n_split; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(p.partial + ((int64_t)s * p.M + m) * p.ld + n);
    acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
  }
  const float f[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (n + j >= p.N) break;
    if (p.f32) static_cast<float*>(p.C)[m * p.N + n + j] = f[j];
    else static_cast<uint16_t*>(p.C)[m * p.N + n + j] = (uint16_t)(f32x2_bf16x2(f[j], 0.f) & 0xFFFFu);
  }
}
constexpr int kSms = 152;
// How a product is cut: the rows of A and of B of a tile, and the splits of K.
struct Cut {
  int m, n, n_split;
  bool thin;
};
// Estimated times in us without the launch, fitted to measurements of shapes around the borders.  A block of K takes 0.42
// us in the wide kernel, 0.45 where there is more than one tile for an SM, 0.47 where the weights come from memory for one
// row of tiles; the end of a tile 1.2.  In the thin kernel a block takes 0.45 (128 rows of A) or 0.3, the end of a tile 1 or
// 0.5, a launch that adds the partial sums 2.5, and these go to L2 and back at 5 TB/s.
// 128 x 32,768 x 4,096: thin 34.6 us, wide 26.8; 128 x 8,192 x 8,192: 20.6 (split) and 30.4; 200 x 16,384 x 4,096: 33 and
// 17.3; 161 x 1,001 x 1,552: 7.6 (split) and 18.
struct Estimate {
  int n_split;
  double us;
};
Estimate thin_time(int64_t tiles, int64_t kb, double block, double end, double bytes) {
  Estimate best{1, (double)((tiles + kSms - 1) / kSms) * (kb * block + end)};
  for (int n = 2; n <= std::min<int64_t>(kb, kSms / tiles); ++n) {
    const double us = (double)((kb + n - 1) / n) * block + end + 2.5 + n * 2 * bytes / 5e6;
    if (us < best.us) best = Estimate{n, us};
  }
  return best;
}
Cut cut_of(int M, int N, int K) {
  const int64_t kb = (K + kBlock - 1) / kBlock;
  auto tiles = [&](int m, int n) { return (int64_t)((M + m - 1) / m) * ((N + n - 1) / n); };
  const int rows = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const Estimate thin = thin_time(std::max<int64_t>(1, tiles(rows, kTN)), kb, rows == 128 ? 0.45 : 0.3, rows == 128 ? 1. : 0.5, 4. * M * N);
  const int64_t wide_tiles = tiles(kWM, kWN);
  const double wide = (double)((wide_tiles + kSms - 1) / kSms) * (kb * (M <= kWM ? 0.47 : wide_tiles <= kSms ? 0.42 : 0.45) + 1.2);
  if (M <= 64 || thin.us <= wide) return Cut{rows, kTN, thin.n_split, true};
  return Cut{kWM, kWN, 1, false};
}
int64_t partial_ld(int N) { return ((int64_t)N + 127) / 128 * 128; }

bool row_map(CUtensorMap* map, const uint8_t* p, int rows, int K, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)K};
  const cuuint32_t box[2] = {(cuuint32_t)kBlock, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return tensor_map_encoder() &&
         tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Kernel, typename... Rest>
cudaError_t launch_matmul(Kernel kernel, size_t smem, int threads, int64_t items, int ctas, cudaStream_t s, const CUtensorMap& am,
                          const CUtensorMap& bm, const Rest&... rest) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_step(kernel, dim3((unsigned)std::min<int64_t>(items, ctas)), dim3(threads), smem, s, am, bm, rest..., status_word());
}
cudaError_t launch_wide(int64_t items, int sms, const CUtensorMap& am, const CUtensorMap& bm, MatmulPlan p, cudaStream_t s) {
  cudaFuncAttributes at;
  const cudaError_t e = cudaFuncGetAttributes(&at, k_matmul_fp8_wide);
  if (e != cudaSuccess) return e;
  if (at.numRegs < kWRegs) return cudaErrorInvalidConfiguration;   // the register split would wait forever
  CUtensorMap cm = am;
  const int size = p.f32 ? 4 : 2;
  p.c_map = (int64_t)p.N * size % 16 == 0;
  if (p.c_map) {
    const cuuint64_t dims[2] = {(cuuint64_t)p.N, (cuuint64_t)p.M};
    const cuuint64_t strides[1] = {(cuuint64_t)p.N * size};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), 32}, estr[2] = {1, 1};
    if (tensor_map_encoder()(&cm, p.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.C, dims, strides, box, estr,
                             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  return launch_matmul(k_matmul_fp8_wide, sizeof(WideSmem) + 1024, kWThreads, items, sms, s, am, bm, cm, p);
}

template <int kRows>
cudaError_t launch_thin(int64_t items, int sms, const CUtensorMap& am, const CUtensorMap& bm, const MatmulPlan& p, cudaStream_t s) {
  const int ctas = items > sms ? kTCtas<kRows> : 1, stages = kTRingBytes / ctas / kTStageBytes<kRows>;
  static_assert(kTSmemBytes<kRows>(kTRingBytes / kTStageBytes<kRows>) <= 232448, "shared memory of a block");
  static_assert(kTCtas<kRows> * (kTSmemBytes<kRows>(kTRingBytes / kTCtas<kRows> / kTStageBytes<kRows>) + 1024) <= 233472, "shared memory of an SM");
  return launch_matmul(k_matmul_fp8_thin<kRows>, kTSmemBytes<kRows>(stages), kTThreads<kRows>, items, ctas * sms, s, am, bm, p, stages);
}

}  // namespace

cudaError_t launch_pack_fp8_blocks(const void* x, int dtype, int64_t stride, int64_t rows, int K, uint8_t* codes, float* scales, cudaStream_t s) {
  const bool f32 = dtype == CSA2_F32;
  const int kb = (K + kBlock - 1) / kBlock, whole = f32 ? 32 : 16;
  const int64_t blocks = rows * kb;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  int lanes_log = f32 ? 5 : 4;                       // short rows leave no lane without work
  while (K <= kBlock / 2 && (kBlock / whole << (lanes_log - 1)) >= K) --lanes_log;
  const int groups = 32 >> lanes_log;
  // one block a group of lanes where there are not enough of them for two blocks of threads on every SM
  const int many = (int)std::max<int64_t>(1, std::min<int64_t>(kPackMany, blocks / (152 * 2 * (kPackThreads / 32) * groups)));
  const int64_t per = (int64_t)many * groups * (kPackThreads / 32), grid = (blocks + per - 1) / per;
  const auto kernel = f32 ? (K > kBlock / 2 ? k_pack_fp8_blocks<true, 32> : k_pack_fp8_blocks<true, 0>)
                          : (K > kBlock / 2 ? k_pack_fp8_blocks<false, 16> : k_pack_fp8_blocks<false, 0>);
  return launch_step(kernel, dim3((unsigned)grid), dim3(kPackThreads), 0, s, x, stride, K, Divisor::of(kb), (uint32_t)blocks, many, lanes_log, codes,
                     scales);
}

// Tiles times splits are at most kSms where K is split, and a tile's partial sums at most 128 x 128.
static_assert((size_t)kSms * 128 * kTN * sizeof(float) == CSA2_MATMUL_FP8_WORKSPACE_MAX, "workspace of any product");
size_t matmul_fp8_workspace_bytes(int M, int N, int K) {
  const int n = cut_of(M, N, K).n_split;
  return n > 1 ? (size_t)n * M * partial_ld(N) * sizeof(float) : 0;
}

cudaError_t launch_matmul_fp8(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb, int M, int N, int K, void* C, int f32, void* ws,
                              cudaStream_t s) {
  const Cut cut = cut_of(M, N, K);
  MatmulPlan p = {};
  p.sa = sa; p.sb = sb; p.C = C; p.M = M; p.N = N; p.kb = (K + kBlock - 1) / kBlock; p.f32 = f32;
  p.n_split = cut.n_split;
  p.ld = partial_ld(N);
  p.partial = p.n_split > 1 ? static_cast<float*>(ws) : nullptr;
  p.m_tiles = (M + cut.m - 1) / cut.m;
  p.n_tiles = (N + cut.n - 1) / cut.n;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  CUtensorMap am, bm;
  if (!row_map(&am, a, M, K, cut.m) || !row_map(&bm, b, N, K, cut.n)) return cudaErrorInvalidValue;
  const int64_t items = (int64_t)p.m_tiles * p.n_tiles * p.n_split;
  if (items > INT_MAX) return cudaErrorInvalidConfiguration;
  if (!cut.thin) e = launch_wide(items, sms, am, bm, p, s);
  else if (cut.m == 16) e = launch_thin<16>(items, sms, am, bm, p, s);
  else if (cut.m == 32) e = launch_thin<32>(items, sms, am, bm, p, s);
  else if (cut.m == 64) e = launch_thin<64>(items, sms, am, bm, p, s);
  else e = launch_thin<128>(items, sms, am, bm, p, s);
  if (e != cudaSuccess || p.n_split == 1) return e;
  const unsigned gy = (unsigned)std::min(M, 32768);
  return launch_step(k_matmul_fp8_sum, dim3((unsigned)((N + 1023) / 1024), gy, (unsigned)((M + gy - 1) / gy)), dim3(256), 0, s, p);
}

}  // namespace csa2
