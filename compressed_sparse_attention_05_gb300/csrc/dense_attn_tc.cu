// Attention over every visible entry of the compressed cache (reading R14) and the
// entries' attention weights (reading R15) on the fifth-generation tensor cores,
// d = 512.
//
//   l_rj = cap tanh(tau q_r . k_j / cap) - slope_h |t_r - p_j|
//   O_r  = sum_j exp(l_rj - m) k_j / sum_j exp(l_rj - m),  lse_r = m + log(sum)
//   w_j  = decay w_j + sum_r exp(l_rj - lse_r)
//
// One shared KV head, so the (token, head) pairs of a sequence are the rows of one
// matrix whatever the number of heads: a tile is 64 consecutive rows (one token of
// 64 heads, half a token of 128, several tokens of fewer heads; 128 rows for the weights
// of more than 64), each row with its own masks.  A tile's keys come in chunks of 128,
// nearest first (window rows, then entries from the newest to the oldest), so that a
// distance bias only lowers later chunks and the reference maxima hardly move.  Per chunk
//   S^T [128 keys x 64 rows]  = K [128 x 512] . Q^T        (32 MMAs, k = 16 channels)
//   O^T [512 dims x 64 rows] += V^T [512 x 128] . P^T      (4 M-tiles x 8 MMAs, k = 16 keys)
//
// The score product reads K as an A operand in tensor memory, where three 128-channel
// quarters of the dequantised chunk fit at a time; the value product reads V from shared
// memory, in three quarters too.  (Shared memory holds one dequantised chunk (128 KB) beside
// Q (64 KB) and P, so with both products reading it the softmax would stand between them.  And
// at N = 64 an MMA with both operands in shared memory reads 6 KB in 48 cycles, all that the
// memory gives, while the dequantising warps' stores and every barrier wait: with the scores
// of every second chunk from shared memory a batch of 32 x 32,768 entries took 281 us.)  In
// a probe of 32 MMAs back to back one takes 87 cycles with A in tensor memory and 52 with
// both operands in shared memory, which would make 32 x 87 + 32 x 52 = 4,450 cycles per 128
// keys x 64 rows; in the kernel they take somewhat less (next paragraph).  S(c+1) is issued
// before PV(c), so that the softmax of a chunk has a whole chunk's products to hide behind.
//
// What bounds it: a chunk takes 3.6 us, 6,800 cycles at the 1.9 GHz of these runs.  In a copy
// with clock stamps the MMA warp waits for 2,700 of them, for the last quarters of K and V,
// and the products take the other 4,100.  A fill warp's step (64 channels of 32 keys) takes
// 1,400 cycles, of which 400 are conversion and stores; the others are trips through a shared
// memory that the products keep busy (a barrier looked at: 180) and instruction issue (half of
// all slots are taken, by 24 warps; no pipe is over 40%).  The products of a chunk interleaved with
// the next scores, so that the last quarters have more time, changed nothing.  A batch of
// 32 x 32,768 entries takes 214 us (643 TFLOP/s, 1.4 TB/s of packed entries), the weights of
// the same batch 92 us, of which the products are 82 at the probe's rate.
//
// Work is split over the SMs by chunks, not by tiles: every CTA computes the chunk
// count of all tiles (lengths live on the device), takes an equal contiguous share,
// and walks the tiles in it.  A tile counts kTileUnits chunks more than it has.  A
// tile that falls to several CTAs leaves partial (m, l, O) in the workspace and
// k_dense_merge joins them in order.
//
// Roles (896 threads): warps 0-7 dequantise V into shared memory, warps 8-15 K into tensor
// memory (with the weights all sixteen do K); before a tile's products the same warps bring in
// Q, after them they write O.  Warps 16-23 do the softmax (thread = one key x 32 rows), warp 24
// issues the MMAs, warps 25 and 26 copy the packed codes of K and V into staging slots (tensor
// map copies: read by the dequantising warps themselves, lane = key, they throttled the L1),
// warp 27 requests pages into L2 ahead.  Operand ranges as in attention_tc.cu (R11's powers of
// two for Q rows and window rows); P is rounded to fp16 (kTopLog2), the normaliser sums the
// unrounded fp32 P, everything else is fp32.
#include <cuda_fp16.h>

#include <algorithm>

#include "dense.cuh"
#include "operands.cuh"
#include "tc.cuh"
#include "tma.cuh"

namespace csa2 {
namespace {

constexpr int kD = 512;
// What a kernel does: 0 attention; else the weights, with tiles of that many rows (64 or 128).  Attention's
// O^T takes tensor memory for 64 rows only.  An MMA with A in tensor memory takes 87 cycles for 64 rows as
// for 128, so the weights take 128 where a sequence has more than 64: 2 x 257 tokens x 64 heads over 16,384
// entries took 649 us instead of 861 when this was changed, and take 651.
template <int kMode> constexpr bool kWeights = kMode != 0;
template <int kMode> constexpr int kRowsOf = kMode ? kMode : 64;
constexpr int kRows = 64;                 // rows of an attention tile (N of both products)
constexpr int kChunk = 128;               // keys of a chunk
constexpr int kValWarps = 8, kKeyWarps = 8, kSoftWarps = 8;
constexpr int kSoftFirst = (kValWarps + kKeyWarps) * 32;   // first softmax thread
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kThreads = 896;             // + MMA warp, two staging warps, L2 warp
constexpr int kMmaWarp = kValWarps + kKeyWarps + kSoftWarps;
constexpr int kMaxCtas = 256;             // bound of the grid (workspace slots)
// registers per thread after the split of the seven warpgroups: 4 x 56 + 2 x 120 + 40 = 4 x 64 + 2 x 104 + 40 = 7 x 72
constexpr int kRegsLaunch = 72, kRegsMisc = 40;
template <int kMode> constexpr int kRegsFill = kMode ? 64 : 56;
template <int kMode> constexpr int kRegsSoft = kMode ? 104 : 120;
constexpr uint32_t kTmemCols = 512;
// Tensor memory.  Attention: O^T (four M-tiles of 64 columns), S^T, and a ring of three
// quarters of K (64 columns each: 128 channels of fp16).  Weights: two S^T, a ring of four.
constexpr uint32_t kColO = 0;
template <int kMode> struct Cols { static constexpr uint32_t S = 0, K = 2 * kMode; static constexpr int ring = 4; };
template <> struct Cols<0> { static constexpr uint32_t S = 256, K = 320; static constexpr int ring = 3; };
// P = 2^(l - m_ref + kTopLog2): fp16 then holds a weight down to 2^-(24 + kTopLog2) of the reference, so that what
// a long tail loses, at most 2^-32 of the reference per key, is far below O's bf16 step (2^-25 per key, without
// the factor, took 0.6% of the mass of 262,144 keys at 2^-25.3 beside a peak).  O and l carry the same factor.
constexpr float kTopLog2 = 7.f, kBottom = 1.f / 128;   // and 2^-kTopLog2
constexpr float kRescaleLog2 = 8.f;       // a reference maximum moves only beyond this growth: P <= 2^15
constexpr float kUnset = 3e38f;           // kTopLog2 - m_ref of a row without keys: any finite logit outgrows it, -inf stays -inf
constexpr int kPartFloats = kRows * kD + 2 * kRows;   // O, then m and l

constexpr int kQuarter = 128;                         // channels of a quarter
constexpr int kVSlots = 3;                            // quarters of V in shared memory
constexpr int kStageBytes = kChunk * kQuarter / 2;    // packed codes of a chunk's quarter
template <int kMode> struct Stages { static constexpr int K = 8, V = 1; };   // staging slots of the K and V streams
template <> struct Stages<0> { static constexpr int K = 3, V = 3; };

// Operand tiles (no-swizzle canonical layout, core matrices of 8 rows x 16 bytes):
//   Q [row][dim]:         (r/8)*8192 + (d/8)*128 + (r%8)*16 + (d%8)*2
//   V slot [key][dim]:    (k/8)*2048 + (d/8)*128 + (k%8)*16 + (d%8)*2   (128 channels)
//   P [key][row]:         (k/8)*1024 + (r/8)*128 + (k%8)*16 + (r%8)*2
// Staging slots hold the codes of one quarter of 128 keys as tensor-map copies with the
// 64-byte swizzle write them: 16-byte piece p of key k at 64 k + 16 (p ^ (k/2)%4), so that
// the 8 lanes of a phase (lane = key) read all banks.
struct Segment {            // what the roles need to know of the current tile
  int b, nw, c_hi;          // window chunks; entry chunks end at c_hi
  int n_chunks;
  int e_lo, e_hi;           // entries any row of the tile may see
  int w_lo, w_hi;           // window rows any row sees (raw positions, inclusive)
  int all_lim, all_doc;     // every row sees the entries that these would let through (as lim and doc of a row)
  int one_t;                // all rows belong to one token
  int one_tok;              // bit k: rows 32 k .. +31 do (weights: 0 if a row of the tile has an infinite lse)
  int next_t;               // first row of the tile's second token
  int pos0;
};
template <int kMode>
struct Smem {
  unsigned char kst[Stages<kMode>::K][kStageBytes];   // (1024-aligned)
  unsigned char vst[kWeights<kMode> ? 1 : Stages<kMode>::V][kWeights<kMode> ? 16 : kStageBytes];
  uint16_t q[kRowsOf<kMode> * kD];
  uint16_t v[kWeights<kMode> ? 8 : kVSlots * kChunk * kQuarter];
  uint16_t p[kWeights<kMode> ? 8 : kChunk * kRowsOf<kMode>];
  float mult[kRowsOf<kMode>];        // logit multiplier: softmax scale * log2(e) * 2^e_r
  float nref[kRowsOf<kMode>];        // attention: kTopLog2 - m_ref (kUnset before the row's first key); weights: -lse * log2(e)
  float slope2[kRowsOf<kMode>];      // slope * log2(e)
  // a row sees an entry if its last token is at or before lim and its first at or after doc, and
  // the window row at position p if 0 <= t - p < W and p >= doc
  int lim[kRowsOf<kMode>], doc[kRowsOf<kMode>], t[kRowsOf<kMode>];
  union {
    float red[4][kRowsOf<kMode>];            // per-lane-quarter maxima / sums of a row over the keys; [0] also: see below
    int qexp[4][kRowsOf<kMode>];             // [1]: largest exponent field of each row of Q, before the products
    struct {                        // before the first tile
      int scan[kThreads / 32];
      int found_start, found_tile, found_end;
    };
  };
  uint64_t kst_full[Stages<kMode>::K], kst_free[Stages<kMode>::K];   // staging slots
  uint64_t vst_full[Stages<kMode>::V], vst_free[Stages<kMode>::V];
  uint64_t kq_full[4], kq_free[4];  // quarters of a chunk's K in tensor memory
  uint64_t v_full[4], v_free[4];    // quarters of a chunk's V in shared memory
  uint64_t s_full[2], s_free[2], p_full, p_free;
  Segment seg;
  uint32_t tmem;
  int abort;
  int progress;             // chunks whose softmax has begun (paces the L2 requests)
};
// red[0][r] holds the factor of a row's rescaling and, at the end of a tile, its sum l:
// each is computed by the one thread that reads the column, from the column.
static_assert(sizeof(Smem<0>) <= 232448 && sizeof(Smem<64>) <= 232448 && sizeof(Smem<128>) <= 232448, "shared memory");

struct Plan {
  int rows;                 // rows of a tile
  int tile0, tiles;         // tiles [tile0, tile0 + tiles) of every sequence are this launch's
  int n_ctas;
  float* parts;             // attention: partial results, kPartFloats per slot, two slots per CTA
  int32_t* cont;            // attention: [n_ctas] tile that the CTA's share starts in the middle of, or -1
  float* sums;              // weights: [B * tiles][sum_stride] when a sequence has several tiles, else null
  int2* ranges;             // weights: [B * tiles] entry chunks written to sums
  int64_t sum_stride;
};

__device__ __forceinline__ void block_sync() { asm volatile("bar.sync 0, %0;" ::"n"(kThreads) : "memory"); }
constexpr int kFillThreads = (kValWarps + kKeyWarps) * 32;
__device__ __forceinline__ void fill_sync() { asm volatile("bar.sync 2, %0;" ::"n"(kFillThreads) : "memory"); }
// The softmax warps announce a tile's chunks (seg) to the last warpgroup.
__device__ __forceinline__ void seg_arrive() { asm volatile("bar.arrive 5, %0;" ::"n"(kSoftThreads + 128) : "memory"); }
__device__ __forceinline__ void seg_sync() { asm volatile("bar.sync 5, %0;" ::"n"(kSoftThreads + 128) : "memory"); }
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory"); }
// The 128 threads of one half of the softmax warps (32 rows).
__device__ __forceinline__ void half_sync(int half) { asm volatile("bar.sync %0, 128;" ::"r"(3 + half) : "memory"); }
__device__ __forceinline__ bool half_or(int half, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(3 + half)
      : "memory");
  return r != 0;
}
// Maximum over the warp.
__device__ __forceinline__ float warp_max_f32(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// 32 lanes x 32 columns: thread i of the warp gets lane (base + i).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ bool mbar_try_wait_at(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000u)
      : "memory");
  return ok != 0;
}
// Bounded wait of a whole warp; on time-out the CTA's abort flag is raised.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  bool ok = false;
#pragma unroll 1
  for (uint32_t i = 0; i < (1u << 21); ++i) {   // <= 2^21 suspensions of <= 1 us
    if (mbar_try_wait_at(bar, parity)) {
      ok = true;
      break;
    }
    if ((i & 63) == 63 && *abort) break;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) *abort = 1;
  return ok;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return warp_wait(tc::smem_addr(bar), parity, abort);
}

// Shared-memory descriptors as their low words (address and leading offset; an operand's
// steps only move the address); the high word (stride offset, version) is a constant.  The
// issuing thread has few registers and a spilled descriptor costs it more than an MMA takes.
__device__ __forceinline__ uint32_t desc_lo(const void* p, uint32_t lbo) {
  return ((tc::smem_addr(p) & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14); }

// D[tmem] (+)= A . B^T, kind::f16, fp32 accumulation; A in shared memory or (K-major, two fp16
// per column) in tensor memory.  The whole warp runs the issuing code, so that its operands are
// uniform registers from the start, and the elected lane (leader != 0) issues.
template <uint32_t kAHi, uint32_t kBHi, uint32_t kIdesc>
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 da, db;\n setp.ne.b32 e, %7, 0;\n setp.ne.b32 p, %3, 0;\n"
      " mov.b64 da, {%1, %4};\n mov.b64 db, {%2, %5};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %6, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(accumulate), "n"(kAHi), "n"(kBHi), "n"(kIdesc), "r"(leader)
      : "memory");
}
template <uint32_t kBHi, uint32_t kIdesc>
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 db;\n setp.ne.b32 e, %6, 0;\n setp.ne.b32 p, %3, 0;\n"
      " mov.b64 db, {%2, %4};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %5, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(accumulate), "n"(kBHi), "n"(kIdesc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_commit_by(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(tc::smem_addr(bar)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Whether the phase of the given parity is complete (never suspends).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]));
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// tanh up to 1/2: an odd polynomial (least-squares fit of (tanh x / x - 1) / x^2 in x^2, weighted to the
// relative error, which is 1.1 x 2^-24).
__device__ __forceinline__ float small_tanh(float x) {
  const float z = x * x;
  float r = -0.00666007306f;
  r = fmaf(r, z, 0.02130601f);
  r = fmaf(r, z, -0.0539009757f);
  r = fmaf(r, z, 0.133329809f);
  r = fmaf(r, z, -0.333333284f);
  return fmaf(x * z, r, x);
}
// min(a, b), NaN where one is NaN (fminf gives the other one).
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Any x: above 1/2, 1 - 2 / (e^2x + 1) (relative error < 2^-21); a NaN stays one.
__device__ __forceinline__ float fast_tanh(float x) {
  const float a = fabsf(x);
  const float e = ex2(min_nan(a, 10.f) * (2.f * kLog2e));   // tanh(10) rounds to 1
  const float big = copysignf(1.f - 2.f * rcp_approx(e + 1.f), x);
  return a < 0.5f ? small_tanh(x) : big;
}

// ---- tiles and their chunks ----------------------------------------------------------
struct Range {
  int e_lo, e_hi, w_lo, w_hi;
};
__device__ __forceinline__ int range_chunks(const Range& r, bool weights) {
  const int ne = r.e_hi > r.e_lo ? (r.e_hi + kChunk - 1) / kChunk - r.e_lo / kChunk : 0;
  const int nw = !weights && r.w_hi >= r.w_lo ? (int)(((int64_t)r.w_hi - r.w_lo) / kChunk) + 1 : 0;
  return ne + nw;
}
// Units of work of a tile (tile = index among this launch's tiles): its chunks, and what beginning and
// ending a tile takes (17 us, a chunk 3.6 us; without it an SM with 50 tiles of two chunks was still at
// work when the SMs with tiles of 17 chunks had long finished: 1,181 us for a prompt of 1,024 tokens with
// documents; with 2, 3, 4, 5, 6 units 743, 649, 602, 573, 574).  The figure is the attention kernel's; the
// weights kernels, which have no O to write, use it too: from 4 to 5 units 257 tokens over 16,384 entries went
// from 649 us to 658.  A share never begins or ends in the first kTileUnits units: such a bound moves to the
// tile's start.
constexpr int kTileUnits = 5;
template <int kMode>
__device__ int tile_units(const DenseArgs& a, const Plan& pl, int tile) {
  const int b = tile / pl.tiles;
  const int r0 = (pl.tile0 + tile % pl.tiles) * kRowsOf<kMode>;
  const int64_t rows = (int64_t)a.Tq * a.Hq;
  if (r0 >= rows) return kTileUnits;
  const int n_ent = dense_entries(a, b);
  Range g{INT_MAX, 0, INT_MAX, INT_MIN};
  if (kWeights<kMode> && !pl.sums) {
    g.e_lo = 0;
    g.e_hi = n_ent;
  } else {
    const int64_t shift = dense_shift(a, b);
    const int pos0 = a.swa_cap > 0 ? a.swa_pos0[b] : 0;
    const int i1 = (int)(min((int64_t)r0 + kRowsOf<kMode>, rows) - 1) / a.Hq;
#pragma unroll 1
    for (int i = r0 / a.Hq; i <= i1; ++i) {
      const DenseRow r = dense_row(a, b, i, n_ent, shift, pos0);
      const int lo = dense_first(a, r.doc, shift);
      if (r.nv > lo) {
        g.e_lo = min(g.e_lo, lo);
        g.e_hi = max(g.e_hi, r.nv);
      }
      if (r.w_n > 0) {
        g.w_lo = min(g.w_lo, r.w_lo);
        g.w_hi = max(g.w_hi, r.w_lo + r.w_n - 1);
      }
    }
  }
  return kTileUnits + range_chunks(g, kWeights<kMode>);
}

// Inclusive block-wide prefix sum (all threads), and the total.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}
__device__ __forceinline__ int block_scan(int v, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v, lane);
  __syncthreads();
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  const int w = warp_scan(lane < kThreads / 32 ? sums[lane] : 0, lane);   // every warp: the warps' prefix sums
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return v + (warp ? before : 0);
}

// ---- dequantisation --------------------------------------------------------------------
// min(a, b); the other one where one is NaN.  V takes NaN and infinity as some finite value: a row that sees
// the key gets them through K and the weight, and a row that does not must not get 0 x NaN.
__device__ __forceinline__ uint32_t min_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Half h (16 channels) of a piece with its two E4M3 scales (at most 448): 8 fp16 pairs.
template <bool kV>
__device__ __forceinline__ void dequant16(const uint4& c, uint32_t scales, int h, uint32_t (&o)[8]) {
  uint32_t s = e4m3x2_f16x2(scales & 0xFFFFu);
  if (kV) s = min_f16x2(s, 0x5F005F00u);
  const uint32_t g = prmt(s, s, h ? 0x3232u : 0x1010u);
  e2m1x8_f16x8(h ? c.z : c.x, o[0], o[1], o[2], o[3]);
  e2m1x8_f16x8(h ? c.w : c.y, o[4], o[5], o[6], o[7]);
#pragma unroll
  for (int x = 0; x < 8; ++x) o[x] = hmul2(o[x], g);   // exact: <= 6 significant bits
}

template <int kMode>
struct Ctx {
  const DenseArgs& a;
  const Plan& pl;
  Smem<kMode>& sm;
  uint32_t tm;
  int u0, u1;              // this CTA's units (a launch has fewer than 2^31)
  int tile;                // first tile and its first unit
  int tstart;
  uint32_t* status;
  const CUtensorMap* map;  // codes: [n_pages * 64][256] bytes in boxes of 64 x 64
};

// A window row as its dequantising thread needs it (null: no key, zeros).
struct KeyRef {
  const uint8_t* codes;    // the row's first code byte
  float wsc;               // scale * 2^-f
};

template <int kMode>
__device__ __forceinline__ KeyRef window_ref(const Ctx<kMode>& cx, int k, int key) {
  const Segment& sg = cx.sm.seg;
  KeyRef r{nullptr, 0.f};
  const int64_t p = (int64_t)sg.w_lo + (int64_t)k * kChunk + key;
  if (p > sg.w_hi) return r;
  bool seen = sg.one_t != 0;      // one token: the tile's rows all see its whole window
  if (!seen)                      // else: the first row of each token, and the tile's first
#pragma unroll 1
    for (int i = 0; i < kRowsOf<kMode>; i = i ? i + cx.a.Hq : sg.next_t)
      seen |= (uint32_t)(cx.sm.t[i] - (int)p) < (uint32_t)cx.a.W && p >= cx.sm.doc[i];
  if (!seen) return r;
  const int64_t w = (int64_t)sg.b * cx.a.swa_cap + (p - sg.pos0);
  const float s = __ldg(cx.a.swa_scales + w);
  r.wsc = s * pow2i(-window_exp(s));
  r.codes = cx.a.swa_codes + w * kD;
  return r;
}

// Page-table entry of entry j, or -1 if no row of the tile sees it.
template <int kMode>
__device__ __forceinline__ int page_of(const Ctx<kMode>& cx, int j, bool exists) {
  const Segment& sg = cx.sm.seg;
  if (!exists || j < sg.e_lo || j >= sg.e_hi) return -1;
  return __ldg(cx.a.page_table + (int64_t)sg.b * cx.a.max_pages + (j >> 6));
}

// 16 channels of a window row.
template <bool kV>
__device__ __forceinline__ void window_piece(const uint4& c, float wsc, uint32_t (&o)[8]) {
  if (kV && !isfinite(wsc)) wsc = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = word_of(c, j);
    o[2 * j] = win2_f16x2<kV>(x & 0xFFFFu, wsc);   // V: finite, but for NaN (scales past 2^107 leave fp16's range)
    o[2 * j + 1] = win2_f16x2<kV>(x >> 16, wsc);
    if (kV) {
      o[2 * j] = min_f16x2(o[2 * j], 0x7BFF7BFFu);
      o[2 * j + 1] = min_f16x2(o[2 * j + 1], 0x7BFF7BFFu);
    }
  }
}

// ---- roles ------------------------------------------------------------------------------

// This CTA's part of the current tile.
struct Span {
  int k0, n;        // chunks k0 .. k0 + n - 1
  bool first, last; // holds the tile's first / last unit
};
__device__ __forceinline__ Span span_of(const Segment& sg, int u, int u1, int tstart) {
  Span s;
  const int units = sg.n_chunks + kTileUnits;
  const int end = min(u1, tstart + units);
  s.k0 = max(0, u - tstart - kTileUnits);
  s.n = end - tstart - kTileUnits - s.k0;
  s.first = u == tstart;
  s.last = end == tstart + units;
  return s;
}

// Counters that run through all tiles of a CTA: chunks, and those at even and odd places
// of their tile (double buffers).  Phase k of a barrier is its k-th use.
struct Count {
  uint32_t all = 0, even = 0, odd = 0;
  __device__ __forceinline__ void add(int n) {
    all += n;
    even += (n + 1) / 2;
    odd += n / 2;
  }
  __device__ __forceinline__ uint32_t phase(int i) const { return ((i & 1) ? odd : even) + i / 2; }
};

// O^T of the finished tile from tensor memory: M-tile mt, this warp's lanes (dims), all rows.
template <int kMode>
__device__ __forceinline__ void drain_o(const Ctx<kMode>& cx, const Span& sp, int tile, int mt, int lq, int lane) {
  const DenseArgs& a = cx.a;
  const int b = tile / cx.pl.tiles;
  const int r0 = (cx.pl.tile0 + tile % cx.pl.tiles) * kRowsOf<kMode>;
  const int64_t rows = (int64_t)a.Tq * a.Hq;
  const int dim = 128 * mt + 32 * lq + lane;
  const bool whole = sp.first && sp.last;
  float* part = cx.pl.parts + (int64_t)(2 * blockIdx.x + (sp.first ? 1 : 0)) * kPartFloats;
#pragma unroll 1
  for (int c0 = 0; c0 < kRowsOf<kMode>; c0 += 16) {
    float o[16];
    tc::tmem_ld16(cx.tm + kColO + 64 * mt + c0 + ((uint32_t)(32 * lq) << 16), o);
    tc::tmem_wait_ld();
    if (sp.n == 0) {   // (a tile without keys has no products)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = 0.f;
    }
    if (!whole) {
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c0 + j) * kD + dim] = o[j];
    } else {
      uint16_t* out = a.O + ((int64_t)b * rows + r0 + c0) * kD + dim;
      const int live = (int)min(rows - r0 - c0, (int64_t)16);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < live) out[j * kD] = (uint16_t)(f32x2_bf16x2(o[j] * cx.sm.red[0][c0 + j], 0.f) & 0xFFFFu);
    }
  }
  tc::tc_fence_before();
}

// Dequantises the chunks of a tile, quarter by quarter, lane = key.  kV: into the shared-memory
// slots that the value product reads; else K, into the tensor-memory slots that the score product
// reads.  Attention: the operand's eight warps share every quarter, half of its channels to four of
// them (a quarter to four warps took so long, 1,900 cycles, that the tensor pipe stood waiting for
// the last one of every chunk: 228 us instead of 221 for 32 x 32,768 entries).  Weights: no V, so
// that sixteen warps do K, four a quarter (a ring of four: 93 us, shared quarters 108).
// Quarter number n = 4 chunk + q goes where number n - ring was; barriers belong to quarters (and
// staging slots to the same warps), so that a warp waits for consecutive phases.
template <int kMode> constexpr int kSplit = kMode ? 1 : 2;   // warps that share a quarter's keys
template <int kMode, bool kV>
__device__ __forceinline__ void fill_tile(const Ctx<kMode>& cx, int k0, int n_chunks, uint32_t chunks, uint32_t entries, int group,
                                          int lq, int lane) {
  Smem<kMode>& sm = cx.sm;
  const DenseArgs& a = cx.a;
  constexpr int kRing = kV ? kVSlots : Cols<kMode>::ring, kStage = kV ? Stages<kMode>::V : Stages<kMode>::K;
  constexpr int kStep = kWeights<kMode> ? 4 : 1;    // quarters from one step to the next
  constexpr int kPieces = 8 / kSplit<kMode>;   // of 16 channels, in a step
  const int key = 32 * lq + lane, first = kWeights<kMode> ? group : 0, half = kWeights<kMode> ? 0 : group;
  volatile int* abort = &sm.abort;
  constexpr uint32_t kSlot = kV ? kChunk * kQuarter * 2 : 64;   // a ring slot: bytes, or tensor-memory columns
  const uint32_t dst0 = kV ? tc::smem_addr(sm.v) + (key >> 3) * 2048 + (key & 7) * 16 + half * 1024
                           : cx.tm + Cols<kMode>::K + 32 * half + ((uint32_t)(32 * lq) << 16);
  auto put = [&](uint32_t dst, int p, const uint32_t (&o)[8]) {   // the step's channels 16 p .. +15
    if (kV) {
      sts16(dst + 256 * p, o[0], o[1], o[2], o[3]);
      sts16(dst + 256 * p + 128, o[4], o[5], o[6], o[7]);
    } else {
      tmem_st8u(dst + 8 * p, o);
    }
  };
  // Barriers of quarter q's data, and of the quarter that was in its slot before (a slot's first use: a
  // phase that is over); cp: the chunk's running number.
  const uint32_t full_bar = tc::smem_addr(kV ? sm.v_full : sm.kq_full), free_bar = tc::smem_addr(kV ? sm.v_free : sm.kq_free);
  auto ring_bar = [&](int q) { return free_bar + 8 * ((q - kRing) & 3); };
  auto ring_parity = [&](uint32_t cp, int q) { return (kRing == 3 && q == 3 ? cp : cp + 1) & 1; };
  auto ring_full = [&](int q) {
    if (kV) {
      tc::fence_async_smem();
    } else {
      tc::tmem_wait_st();
      tc::tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) arrive_at(full_bar + 8 * q);
  };
  const int i0 = min(max(sm.seg.nw - k0, 0), n_chunks);   // first entry chunk of the span
  uint32_t ring = (4 * chunks + first) % kRing;   // slot of the step's quarter
  if (!kWeights<kMode>) {
    KeyRef w{nullptr, 0.f};
#pragma unroll 1
    for (int n = 0; n < 4 * i0; ++n) {
      const int q = n & 3;
      if (q == 0) w = window_ref<kMode>(cx, k0 + (n >> 2), key);
      uint4 c[4];                         // in flight over the wait
#pragma unroll
      for (int p = 0; p < 4; ++p)
        c[p] = w.codes ? __ldg(reinterpret_cast<const uint4*>(w.codes) + 8 * q + 4 * half + p) : make_uint4(0, 0, 0, 0);
      if (!warp_wait(ring_bar(q), ring_parity(chunks, q), abort)) return;
      if (!kV) tc::tc_fence_after();
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t o[8];
        window_piece<kV>(c[p], w.wsc, o);
        put(dst0 + ring * kSlot, p, o);
      }
      ring_full(q);
      ring = ring + 1 == kRing ? 0 : ring + 1;
      chunks += q == 3;
    }
  }
  if (i0 >= n_chunks) return;
  // A step's scales are read two steps ahead, the key's page a chunk ahead of that.  The offset is
  // the key's place in the pool (32 bits: 2^32 entries would be 1 TB of codes); none if there is no
  // such key, or behind a bad page: then the scales are zero, and whatever the staging slot holds
  // becomes zeros.
  constexpr uint32_t kNone = 0xFFFFFFFFu;
  const int e_lo = sm.seg.e_lo, e_hi = sm.seg.e_hi;
  const int32_t* table = a.page_table + (int64_t)sm.seg.b * a.max_pages;
  int j = (sm.seg.c_hi - 1 - (k0 + i0 - sm.seg.nw)) * kChunk + key;   // the key's entry
  auto page_at = [&](int j) { return j >= e_lo && j < e_hi ? __ldg(table + (j >> 6)) : -1; };
  auto place = [&](int j, int page) -> uint32_t {
    if (page >= 0 && page < a.n_pages) return (uint32_t)page * kPage + (j & (kPage - 1));
    if (!kV && group == 0 && j >= e_lo && j < e_hi) raise_status(cx.status, CSA2_STATUS_BAD_PAGE);
    return kNone;
  };
  const uint8_t* scales = a.kv_scales + 8 * first + 4 * half;
  auto scales_of = [&](uint32_t at, int q) -> uint2 {
    if (at == kNone) return make_uint2(0, 0);
    const uint8_t* s = scales + (size_t)at * (kD / 16) + 8 * q;
    return kPieces == 8 ? __ldg(reinterpret_cast<const uint2*>(s)) : make_uint2(__ldg(reinterpret_cast<const uint32_t*>(s)), 0);
  };
  int left = n_chunks - i0;               // chunks of which scales are still to be read
  uint32_t at = place(j, page_at(j));
  int page1 = left > 1 ? page_at(j - kChunk) : -1;
  int qs = 0;
  auto next_scales = [&]() -> uint2 {     // of the steps in order
    const uint2 v = scales_of(at, qs);
    qs += kStep;
    if (qs >= 4) {
      qs = 0;
      j -= kChunk;
      --left;
      at = left > 0 ? place(j, page1) : kNone;
      page1 = left > 1 ? page_at(j - kChunk) : -1;
    }
    return v;
  };
  int steps = (n_chunks - i0) * (4 / kStep);
  uint2 s = next_scales(), next = next_scales();
  // the staging slot of the step's codes and its phase
  uint32_t slot = (4 * entries + first) % kStage, phase = ((4 * entries + first) / kStage) & 1;
  const uint32_t st_full = tc::smem_addr(kV ? sm.vst_full : sm.kst_full), st_free = tc::smem_addr(kV ? sm.vst_free : sm.kst_free);
  const uint32_t codes = tc::smem_addr(kV ? sm.vst[0] : sm.kst[0]) + 64 * key + 16 * ((2 * half) ^ ((key >> 1) & 3));
  uint4 t[kPieces / 2];
  auto load_staged = [&] {
#pragma unroll
    for (int p = 0; p < kPieces / 2; ++p) t[p] = lds16((codes + slot * kStageBytes) ^ (16 * p));
  };
  // The slot may be written again once the loads have arrived, not when they are issued: the vote reads
  // a word of each (lane 0 always votes yes).
  auto free_staged = [&] {
    uint32_t any = 0;
#pragma unroll
    for (int p = 0; p < kPieces / 2; ++p) any ^= t[p].x;
    if (__ballot_sync(0xffffffffu, lane == 0 || any == 0x5A5A5A5Au) & (lane == 0)) arrive_at(st_free + 8 * slot);
  };
  if (!warp_wait(st_full + 8 * slot, phase, abort)) return;
  load_staged();
  free_staged();
#pragma unroll 1
  for (int q = first;;) {
    const bool more = --steps > 0;
    slot += kStep;                        // the next step's
    if (slot >= kStage) {
      slot -= kStage;
      phase ^= 1;
    }
    // One look at two barriers (a look is a trip through the busy shared-memory pipe, 180 cycles): lane
    // 0 at this step's ring slot, lane 1 at the next step's codes.
    const uint32_t parity = ring_parity(chunks, q);
    const uint32_t look = __ballot_sync(
        0xffffffffu, mbar_test(lane == 1 ? st_full + 8 * slot : ring_bar(q), lane == 1 ? phase : parity));
    __syncwarp();
    if (!(look & 1) && !warp_wait(ring_bar(q), parity, abort)) return;
    if (!kV) tc::tc_fence_after();
    const uint32_t dst = dst0 + ring * kSlot;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      uint32_t o[8];
      dequant16<kV>(t[p >> 1], (p & 4 ? s.y : s.x) >> (16 * ((p >> 1) & 1)), p & 1, o);
      put(dst, p, o);
    }
    if (more) {
      if (!(look & 2) && !warp_wait(st_full + 8 * slot, phase, abort)) return;
      load_staged();
    }
    s = next;
    next = next_scales();
    ring_full(q);
    if (more) free_staged();
    ring += kStep;
    if (ring >= kRing) ring -= kRing;
    if (!more) break;
    q += kStep;
    if (q >= 4) {
      q -= 4;
      ++chunks;
    }
  }
}
// Entry chunks of a span (the others are window chunks).
__device__ __forceinline__ int entry_chunks(const Segment& sg, const Span& sp) {
  return sp.n - min(max(sg.nw - sp.k0, 0), sp.n);
}

// Warps 0-7 fill V, warps 8-15 K; before that they bring in the tile's Q, after it they write O.
template <int kMode>
__device__ __forceinline__ void role_fill(const Ctx<kMode>& cx) {
  Smem<kMode>& sm = cx.sm;
  const DenseArgs& a = cx.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const bool values = tid < kValWarps * 32;
  const int warp = (tid >> 5) - (values ? 0 : kValWarps);
  volatile int* abort = &sm.abort;
  uint32_t chunks = 0, entries = 0;
  int tile = cx.tile;
  int u = cx.u0, tstart = cx.tstart;
  while (u < cx.u1) {
    // ---- Q rows -> fp16 B operand, row r scaled by 2^-e_r (exact)
    const int b = tile / cx.pl.tiles;
    const int r0 = (cx.pl.tile0 + tile % cx.pl.tiles) * kRowsOf<kMode>;
    const int64_t rows = (int64_t)a.Tq * a.Hq;
    {
      // row 8 g + tid % 8, channels 8 (tid / 8) .. +7; four rows at a time, and once more for the conversion
      // (from L2: eight of them in registers would have the other roles' code spill)
      const uint16_t* src = a.Q + ((int64_t)b * rows + r0 + (tid & 7)) * kD + (tid >> 3) * 8;
      const int live = (int)min(rows - r0 - (tid & 7), (int64_t)kRowsOf<kMode>);
      auto load4 = [&](int g0, uint4 (&qv)[4]) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
          qv[g] = 8 * (g0 + g) < live ? __ldg(reinterpret_cast<const uint4*>(src + 8 * (g0 + g) * kD)) : make_uint4(0, 0, 0, 0);
      };
      constexpr int kLast = kRowsOf<kMode> / 8 - 4;
      uint4 qv[4];
      load4(0, qv);
      if (tid < kRowsOf<kMode>) sm.qexp[1][tid] = 0;
      fill_sync();
#pragma unroll 1
      for (int g0 = 0; g0 < kLast + 4; g0 += 4) {
        if (g0) load4(g0, qv);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t e = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) e = max(e, max(word_of(qv[g], j) & 0x7F80u, (word_of(qv[g], j) >> 16) & 0x7F80u));
          e = max(e, __shfl_xor_sync(0xffffffffu, e, 8));
          e = max(e, __shfl_xor_sync(0xffffffffu, e, 16));
          if (lane < 8 && e) atomicMax(&sm.qexp[1][8 * (g0 + g) + lane], (int)(e >> 7));
        }
      }
      fill_sync();
#pragma unroll 1
      for (int g0 = kLast; g0 >= 0; g0 -= 4) {
        if (g0 != kLast) load4(g0, qv);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float qs = pow2i(-q_head_exp(sm.qexp[1][8 * (g0 + g) + (tid & 7)]));
          uint32_t ov[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w = word_of(qv[g], j);
            ov[j] = f32x2_f16x2(__uint_as_float(w << 16) * qs, __uint_as_float(w & 0xFFFF0000u) * qs);
          }
          *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(sm.q) + (g0 + g) * 8192 + (tid >> 3) * 128 + (tid & 7) * 16) =
              make_uint4(ov[0], ov[1], ov[2], ov[3]);
        }
      }
    }
    if (tid < kRowsOf<kMode>) sm.mult[tid] = a.scale * kLog2e * pow2i(q_head_exp(sm.qexp[1][tid]));
    tc::fence_async_smem();
    tc::tc_fence_before();
    block_sync();                       // Q, row constants and the tile's chunks are there, O of the last tile is not
    tc::tc_fence_after();
    const Span sp = span_of(sm.seg, u, cx.u1, tstart);
    const int units = sm.seg.n_chunks + kTileUnits, more = entry_chunks(sm.seg, sp);
    if (kWeights<kMode> || !values)
      fill_tile<kMode, false>(cx, sp.k0, sp.n, chunks, entries, (warp >> 2) + (kWeights<kMode> && values ? 2 : 0), warp & 3, lane);
    else
      fill_tile<kMode, true>(cx, sp.k0, sp.n, chunks, entries, warp >> 2, warp & 3, lane);
    block_sync();                       // the tile's products are complete, l is known
    tc::tc_fence_after();
    if (*abort) break;
    if (!kWeights<kMode>) drain_o<kMode>(cx, sp, tile, (values ? 0 : 2) + (warp >> 2), warp & 3, lane);
    chunks += sp.n;
    entries += more;
    u = min(cx.u1, tstart + units);
    tstart += units;
    ++tile;
  }
}

// One warp each for K and V: the codes of every entry chunk's quarters into the staging slots,
// two tensor-map copies (one per page) a quarter.
template <int kMode, bool kV>
__device__ __forceinline__ void role_stage(const Ctx<kMode>& cx) {
  Smem<kMode>& sm = cx.sm;
  const DenseArgs& a = cx.a;
  constexpr int kStage = kV ? Stages<kMode>::V : Stages<kMode>::K;
  const int lane = threadIdx.x & 31;
  volatile int* abort = &sm.abort;
  uint32_t entries = 0, issued = 0;     // quarters given to the copy engine
  int u = cx.u0, tstart = cx.tstart;
  while (u < cx.u1) {
    seg_sync();                         // the tile's chunks are known (the copies need no more than that)
    const Span sp = span_of(sm.seg, u, cx.u1, tstart);
    const int units = sm.seg.n_chunks + kTileUnits, more = entry_chunks(sm.seg, sp);
    const int nw = sm.seg.nw, i0 = sp.n - more, steps = kV && kWeights<kMode> ? 0 : 4 * more;
    // lane l: page l % 2 of chunk i + l / 2, for 16 chunks; the next 16 are on their way
    auto pages_at = [&](int i) -> int {
      i += lane >> 1;
      const int lp = (sm.seg.c_hi - 1 - (sp.k0 + i - nw)) * (kChunk / kPage) + (lane & 1);
      if (i >= sp.n || (lp + 1) * kPage <= sm.seg.e_lo || lp * kPage >= sm.seg.e_hi) return -1;
      const int p = __ldg(a.page_table + (int64_t)sm.seg.b * a.max_pages + lp);
      return p < a.n_pages ? p : -1;
    };
    int pages = -1, ahead = pages_at(i0);
    bool synced = false;
#pragma unroll 1
    for (int n = 0; n < steps; ++n) {
      if (n == kStage) {                // the slots are full: only now wait for the other roles
        block_sync();
        synced = true;
      }
      const int i = i0 + (n >> 2), q = n & 3;
      const uint32_t st = 4 * entries + n, slot = st % kStage, use = st / kStage;
      if ((n & 63) == 0) {
        pages = ahead;
        ahead = pages_at(i + 16);
      }
      const int page = __shfl_sync(0xffffffffu, pages, 2 * ((n >> 2) & 15) + (lane & 1));
      if (use > 0 && !warp_wait(kV ? &sm.vst_free[slot] : &sm.kst_free[slot], (use - 1) & 1, abort)) break;
      const uint32_t have = __ballot_sync(0xffffffffu, lane < 2 && page >= 0);
      uint64_t* full = kV ? &sm.vst_full[slot] : &sm.kst_full[slot];
      if (lane == 0) tc::mbar_arrive_expect_tx(full, __popc(have) * (kStageBytes / 2));
      __syncwarp();
      if (lane < 2 && page >= 0)
        tma::load_2d((kV ? sm.vst[slot] : sm.kst[slot]) + lane * (kStageBytes / 2), cx.map, 64 * q, page * kPage, full);
      issued = st + 1;
    }
    if (!synced) block_sync();
    block_sync();
    if (*abort) break;
    entries += more;
    u = min(cx.u1, tstart + units);
    tstart += units;
  }
  // an abandoned tile may leave copies in flight: they land before the block ends
  if (*abort)
    for (uint32_t st = issued > (uint32_t)kStage ? issued - kStage : 0; st < issued; ++st)
      for (uint32_t n = 0; n < (1u << 22); ++n)
        if (tc::mbar_try_wait(kV ? &sm.vst_full[st % kStage] : &sm.kst_full[st % kStage], (st / kStage) & 1)) break;
}

// One key of a chunk as its softmax thread sees it.
struct KeyView {
  bool masked;         // some row may not see the key, or its window row is rescaled (uniform over the warp)
  bool seen;           // a key that some row may see
  int win;             // 1: window row
  int p;               // raw position (an entry's: of its last token)
  float kf, ff;        // window row: 2^f and f
};

// |t - p| in fp32 (exact below 2^24).
__device__ __forceinline__ float distance(int t, int p) {
  return (float)(t > p ? (uint32_t)t - (uint32_t)p : (uint32_t)p - (uint32_t)t);
}
template <int kMode>
__device__ __forceinline__ bool row_sees(const Ctx<kMode>& cx, const KeyView& kv, int r) {
  const Smem<kMode>& sm = cx.sm;
  if (kv.win) return (uint32_t)(sm.t[r] - kv.p) < (uint32_t)cx.a.W && kv.p >= sm.doc[r];
  return kv.p <= sm.lim[r] && kv.p - 3 >= sm.doc[r];
}

// Columns c0 .. c0+31 of this thread's key: the logits in the log2 domain as the value
// product carries them, -inf where the row does not see the key.
template <int kMode>
__device__ __forceinline__ void load_logits(const Ctx<kMode>& cx, const KeyView& kv, uint32_t taddr, int c0, uint64_t* done,
                                            float (&x)[32]) {
  const Smem<kMode>& sm = cx.sm;
  tmem_ld32(taddr, x);
  tc::tmem_wait_ld();
  if (done) {   // the buffer's last columns
    tc::tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(done);
  }
#pragma unroll
  for (int j4 = 0; j4 < 8; ++j4) {
    const float4 m = *reinterpret_cast<const float4*>(&sm.mult[c0 + 4 * j4]);
    x[4 * j4] *= m.x; x[4 * j4 + 1] *= m.y; x[4 * j4 + 2] *= m.z; x[4 * j4 + 3] *= m.w;
  }
  if (kv.kf != 1.f) {
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] *= kv.kf;
  }
  if (cx.a.cap > 0.f) {
    const float cap2 = cx.a.cap * kLog2e, inv = 1.f / cap2;
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) top = fmaxf(top, fabsf(x[j]));
    if (__all_sync(0xffffffffu, top * inv < 0.5f)) {
      // the usual case: every logit of the warp is well below the cap
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = cap2 * small_tanh(x[j] * inv);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = cap2 * fast_tanh(x[j] * inv);
    }
  }
  auto one = [&] { return (sm.seg.one_tok >> (c0 / 32) & 1) != 0; };   // the columns belong to one token
  if (cx.a.slopes) {
    if (one()) {
      const float dist = distance(sm.t[c0], kv.p);
#pragma unroll
      for (int j4 = 0; j4 < 8; ++j4) {
        const float4 m = *reinterpret_cast<const float4*>(&sm.slope2[c0 + 4 * j4]);
        x[4 * j4] = fmaf(-m.x, dist, x[4 * j4]); x[4 * j4 + 1] = fmaf(-m.y, dist, x[4 * j4 + 1]);
        x[4 * j4 + 2] = fmaf(-m.z, dist, x[4 * j4 + 2]); x[4 * j4 + 3] = fmaf(-m.w, dist, x[4 * j4 + 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = fmaf(-sm.slope2[c0 + j], distance(sm.t[c0 + j], kv.p), x[j]);
    }
  }
  if (!kv.masked) return;
  if (one()) {
    const bool seen = kv.seen && row_sees<kMode>(cx, kv, c0);
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = seen ? x[j] + kv.ff : -INFINITY;
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = kv.seen && row_sees<kMode>(cx, kv, c0 + j) ? x[j] + kv.ff : -INFINITY;
  }
}

template <int kMode>
__device__ __forceinline__ void role_softmax(const Ctx<kMode>& cx) {
  Smem<kMode>& sm = cx.sm;
  const DenseArgs& a = cx.a;
  const int st = threadIdx.x - kSoftFirst, warp = st >> 5, lane = st & 31;
  const int lq = warp & 3, half = warp >> 2;   // lane quarter; attention: rows 32 half .. +31, weights: chunks of that parity
  const int key = 32 * lq + lane;              // thread = key of the chunk = tensor-memory lane
  const uint32_t lane_q = (uint32_t)(32 * lq) << 16;
  volatile int* abort = &sm.abort;
  Count c;
  int tile = cx.tile;
  int u = cx.u0, tstart = cx.tstart;
  const int64_t rows = (int64_t)a.Tq * a.Hq;
  while (u < cx.u1) {
    // ---- rows of the tile
    const int b = tile / cx.pl.tiles;
    const int r0 = (cx.pl.tile0 + tile % cx.pl.tiles) * kRowsOf<kMode>;
    const int n_ent = dense_entries(a, b);
    const int64_t shift = dense_shift(a, b);
    if (st == 0) {
      sm.seg.b = b;
      sm.seg.pos0 = a.swa_cap > 0 ? a.swa_pos0[b] : 0;
      sm.seg.e_lo = INT_MAX; sm.seg.e_hi = 0; sm.seg.w_lo = INT_MAX; sm.seg.w_hi = INT_MIN;
      sm.seg.all_lim = INT_MAX; sm.seg.all_doc = 0;
      sm.seg.next_t = a.Hq - r0 % a.Hq;
      sm.seg.one_tok = 0;
      for (int k = 0; k < kRowsOf<kMode> / 32; ++k)
        sm.seg.one_tok |= (r0 + 32 * k) / a.Hq == (r0 + 32 * k + 31) / a.Hq ? 1 << k : 0;
      sm.seg.one_t = r0 / a.Hq == (int)(min((int64_t)r0 + kRowsOf<kMode>, rows) - 1) / a.Hq;
      if (tile % cx.pl.tiles == 0 && tstart == u && dense_count_bad(a, b)) raise_status(cx.status, CSA2_STATUS_BAD_COUNT);
    }
    soft_sync();
    if (st < kRowsOf<kMode>) {
      const bool live = r0 + st < rows;
      DenseRow r{-1, 0, INT_MIN, INT_MAX, 0, 0};        // no row: it sees nothing
      int lim = INT_MIN;
      float slope = 0.f, nref = kUnset;
      if (live) {
        const int i = (r0 + st) / a.Hq, h = (r0 + st) % a.Hq;
        r = dense_row(a, b, i, n_ent, shift, sm.seg.pos0);
        const int lo = dense_first(a, r.doc, shift);
        if (r.nv > lo) {
          atomicMin(&sm.seg.e_lo, lo);
          atomicMax(&sm.seg.e_hi, r.nv);
        }
        if (r.w_n > 0) {
          atomicMin(&sm.seg.w_lo, r.w_lo);
          atomicMax(&sm.seg.w_hi, r.w_lo + r.w_n - 1);
        }
        lim = r.last;
        if (kWeights<kMode>) {
          const float lse = a.lse_in[(int64_t)b * rows + r0 + st];
          nref = -lse * kLog2e;
          if (isinf(lse)) {       // the row adds nothing: masks of its own, since a NaN key must not reach it either
            nref = -INFINITY;
            lim = INT_MIN;
            sm.seg.one_tok = 0;
          }
        }
        atomicMin(&sm.seg.all_lim, lim);
        atomicMax(&sm.seg.all_doc, r.doc);
        if (a.slopes) slope = a.slopes[h];
      } else if (kWeights<kMode>) {
        nref = -INFINITY;
      }
      sm.lim[st] = lim;
      sm.doc[st] = r.doc;
      sm.t[st] = max(r.t, -1);   // any t below 0 sees nothing, and from -1 no t - p wraps around into a window
      sm.slope2[st] = slope * kLog2e;
      sm.nref[st] = nref;
    }
    soft_sync();
    if (st == 0) {
      Range g{sm.seg.e_lo, sm.seg.e_hi, sm.seg.w_lo, sm.seg.w_hi};
      if (kWeights<kMode> && !cx.pl.sums) {
        g.e_lo = sm.seg.e_lo = 0;
        g.e_hi = sm.seg.e_hi = n_ent;
      }
      sm.seg.n_chunks = range_chunks(g, kWeights<kMode>);
      sm.seg.c_hi = (g.e_hi + kChunk - 1) / kChunk;
      sm.seg.nw = !kWeights<kMode> && g.w_hi >= g.w_lo ? (int)(((int64_t)g.w_hi - g.w_lo) / kChunk) + 1 : 0;
    }
    soft_sync();
    seg_arrive();
    block_sync();
    const Span sp = span_of(sm.seg, u, cx.u1, tstart);
    const Segment& sg = sm.seg;   // (read where needed: registers are what this role is short of)

    const int shift32 = (int)min(shift, (int64_t)1 << 29);
    // The key of a chunk; its page is read one chunk ahead.
    auto entry_of = [&](int i) -> int { return (sg.c_hi - 1 - (sp.k0 + i - sg.nw)) * kChunk + key; };
    constexpr int kStep = kWeights<kMode> ? 2 : 1;
    const int first = kWeights<kMode> ? half : 0;
    auto page_ahead = [&](int i) -> int { return page_of<kMode>(cx, entry_of(i), i < sp.n && sp.k0 + i >= sg.nw); };
    int page = page_ahead(first);
    auto view = [&](int i, int64_t* slot) -> KeyView {
      KeyView kv;
      const int k = sp.k0 + i;
      kv.win = k < sg.nw;
      kv.kf = 1.f;
      kv.ff = 0.f;
      *slot = -1;
      if (kv.win) {
        const int64_t p = (int64_t)sm.seg.w_lo + (int64_t)k * kChunk + key;
        kv.seen = p <= sm.seg.w_hi;
        kv.p = kv.seen ? (int)p : 0;
        kv.masked = true;
        if (kv.seen) {
          const int f = window_exp(__ldg(a.swa_scales + (int64_t)b * a.swa_cap + (kv.p - sm.seg.pos0)));
          if (f != 0) {
            kv.kf = pow2i(f);
            kv.ff = (float)f;
          }
        }
      } else {
        const int j = entry_of(i);
        const bool there = j >= sg.e_lo && j < sg.e_hi && page >= 0 && page < a.n_pages;
        if (there) *slot = (int64_t)page * kPage + (j & (kPage - 1));
        kv.seen = there && (a.entry_pos || j + shift32 < (1 << 29));   // no token is past 2^31 - 1
        kv.p = a.entry_pos && there ? max(__ldg(a.entry_pos + *slot), INT_MIN + 3) : 4 * min(j + shift32, (1 << 29) - 1) + 3;
        kv.masked = __any_sync(0xffffffffu, !kv.seen || kv.p > sm.seg.all_lim || kv.p - 3 < sm.seg.all_doc);
      }
      page = page_ahead(i + kStep);
      return kv;
    };

    if (kWeights<kMode>) {
      for (int i = first; i < sp.n; i += 2) {
        if (st == 0) *reinterpret_cast<volatile int*>(&sm.progress) = (int)(c.all + i);
        int64_t slot;
        const KeyView kv = view(i, &slot);
        const float before = slot >= 0 && !cx.pl.sums && a.weight_in ? a.weight_in[slot] : 0.f;
        if (!warp_wait(&sm.s_full[i & 1], c.phase(i) & 1, abort)) break;
        tc::tc_fence_after();
        float sum = 0.f;
#pragma unroll 1
        for (int c0 = 0; c0 < kRowsOf<kMode>; c0 += 32) {
          float x[32];
          load_logits<kMode>(cx, kv, cx.tm + Cols<kMode>::S + kRowsOf<kMode> * (i & 1) + c0 + lane_q, c0,
                                c0 + 32 == kRowsOf<kMode> ? &sm.s_free[i & 1] : nullptr, x);
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j4 = 0; j4 < 8; ++j4) {
            const float4 z = *reinterpret_cast<const float4*>(&sm.nref[c0 + 4 * j4]);
            s4[0] += ex2(x[4 * j4] + z.x);
            s4[1] += ex2(x[4 * j4 + 1] + z.y);
            s4[2] += ex2(x[4 * j4 + 2] + z.z);
            s4[3] += ex2(x[4 * j4 + 3] + z.w);
          }
          sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
        }
        if (cx.pl.sums)
          cx.pl.sums[(int64_t)tile * cx.pl.sum_stride + entry_of(i)] = slot >= 0 ? sum : 0.f;
        else if (slot >= 0)
          a.weight_out[slot] = (a.weight_in ? a.decay * before : 0.f) + sum;
      }
      if (st == 0) *reinterpret_cast<volatile int*>(&sm.progress) = (int)(c.all + sp.n);
    } else {
      float lsum[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) lsum[j] = 0.f;
      const int c0 = 32 * half;
      for (int i = 0; i < sp.n; ++i) {
        const uint32_t ph = c.all + i, ts = cx.tm + Cols<0>::S + c0 + lane_q;
        if (st == 0) *reinterpret_cast<volatile int*>(&sm.progress) = (int)(c.all + i);
        int64_t slot;
        const KeyView kv = view(i, &slot);
        const bool ok = warp_wait(&sm.s_full[0], ph & 1, abort);
        tc::tc_fence_after();
        // ---- logits over the reference, and whether one outgrows it
        float x[32];
        float top = -INFINITY;
        load_logits<kMode>(cx, kv, ts, c0, &sm.s_free[0], x);
#pragma unroll
        for (int j4 = 0; j4 < 8; ++j4) {
          const float4 z = *reinterpret_cast<const float4*>(&sm.nref[c0 + 4 * j4]);
          top = fmaxf(top, fmaxf(fmaxf(x[4 * j4] + z.x, x[4 * j4 + 1] + z.y), fmaxf(x[4 * j4 + 2] + z.z, x[4 * j4 + 3] + z.w)));
        }
        const bool seen_abort = !ok || *abort != 0;
        if (half_or(half, top > kTopLog2 + kRescaleLog2 || seen_abort)) {
          if (half_or(half, seen_abort)) break;   // (a wait that fails below is met by the next vote)
          // maxima of the half's 32 rows over the 128 keys
          float mine = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float mx = warp_max_f32(x[j]);
            if (lane == j) mine = mx;
          }
          sm.red[lq][c0 + lane] = mine;
          half_sync(half);
          bool need = false;
          if (lq == 0) {
            const int r = c0 + lane;
            const float m = fmaxf(fmaxf(sm.red[0][r], sm.red[1][r]), fmaxf(sm.red[2][r], sm.red[3][r]));
            const float no = sm.nref[r];
            float al = 1.f;
            if (m + no > kTopLog2 + kRescaleLog2) {
              const float now = kTopLog2 - m;
              if (no != kUnset) {
                al = ex2(now - no);
                need = true;
              }
              sm.nref[r] = now;
            }
            sm.red[0][r] = al;
          }
          if (half_or(half, need)) {
            // O^T *= alpha (column = row of the tile): the value products so far must be done
            if (ph > 0) warp_wait(&sm.p_free, (ph - 1) & 1, abort);
            tc::tc_fence_after();
#pragma unroll 1
            for (int mt = 0; mt < 4; ++mt) {
#pragma unroll 1
              for (int q = 0; q < 32; q += 16) {
                const uint32_t ta = cx.tm + kColO + 64 * mt + c0 + q + lane_q;
                float o[16];
                tc::tmem_ld16(ta, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= sm.red[0][c0 + q + j];
                tc::tmem_st16(ta, o);
              }
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
#pragma unroll
            for (int j = 0; j < 32; ++j) lsum[j] *= sm.red[0][c0 + j];
          }
          half_sync(half);                     // red is read; the next vote may come
        }
        // ---- P, rounded to fp16 for the value product
        const float pf = pow2i(-(int)kv.ff);   // the normaliser adds p = 2^-f (2^f p)
        uint32_t pk[16];
#pragma unroll
        for (int j4 = 0; j4 < 8; ++j4) {
          const float4 z = *reinterpret_cast<const float4*>(&sm.nref[c0 + 4 * j4]);
          const float p0 = ex2(x[4 * j4] + z.x), p1 = ex2(x[4 * j4 + 1] + z.y);
          const float p2 = ex2(x[4 * j4 + 2] + z.z), p3 = ex2(x[4 * j4 + 3] + z.w);
          lsum[4 * j4] = fmaf(p0, pf, lsum[4 * j4]);
          lsum[4 * j4 + 1] = fmaf(p1, pf, lsum[4 * j4 + 1]);
          lsum[4 * j4 + 2] = fmaf(p2, pf, lsum[4 * j4 + 2]);
          lsum[4 * j4 + 3] = fmaf(p3, pf, lsum[4 * j4 + 3]);
          pk[2 * j4] = f32x2_f16x2(p0, p1);
          pk[2 * j4 + 1] = f32x2_f16x2(p2, p3);
        }
        if (ph > 0) warp_wait(&sm.p_free, (ph - 1) & 1, abort);
        unsigned char* pd = reinterpret_cast<unsigned char*>(sm.p) + (key >> 3) * 1024 + (c0 / 8) * 128 + (key & 7) * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(pd + j * 128) = make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.p_full);
      }
      if (st == 0) *reinterpret_cast<volatile int*>(&sm.progress) = (int)(c.all + sp.n);
      // all products of the tile, and the row sums over its keys
      if (sp.n > 0) warp_wait(&sm.p_free, (c.all + sp.n - 1) & 1, abort);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = lsum[16 * q + j];
        const float s = reduce16<false>(y, lane);
        if (lane < 16) sm.red[lq][c0 + 16 * q + lane] = s;
      }
      soft_sync();
      if (st < kRowsOf<kMode>) {
        const float l = (sm.red[0][st] + sm.red[1][st]) + (sm.red[2][st] + sm.red[3][st]);
        const float m = sm.nref[st] == kUnset ? -INFINITY : -sm.nref[st];   // log2 of the unit of l and O
        sm.red[0][st] = l == 0.f ? 0.f : 1.f / l;   // the factor of O
        if (sp.first && sp.last) {
          if (a.lse && r0 + st < rows)
            a.lse[(int64_t)b * rows + r0 + st] = l == 0.f ? -INFINITY : (m + kTopLog2 + log2f(l * kBottom)) * kLn2;
        } else {
          float* ml = cx.pl.parts + (int64_t)(2 * blockIdx.x + (sp.first ? 1 : 0)) * kPartFloats + kRowsOf<kMode> * kD;
          ml[st] = m;
          ml[kRowsOf<kMode> + st] = l;
        }
      }
    }
    const int units = sm.seg.n_chunks + kTileUnits;
    block_sync();
    if (*abort) break;
    c.add(sp.n);
    u = min(cx.u1, tstart + units);
    tstart += units;
    ++tile;
  }
}

// Order of the products: S(0) | S(1) PV(0) | S(2) PV(1) | ...
template <int kMode>
__device__ __forceinline__ void role_mma(const Ctx<kMode>& cx) {
  Smem<kMode>& sm = cx.sm;
  volatile int* abort = &sm.abort;
  constexpr uint32_t kIdS = tc::idesc_f16(128, kRowsOf<kMode>, 0, 0, 0);   // K-major A (tensor memory) and B
  constexpr uint32_t kIdO = tc::idesc_f16(128, kRowsOf<kMode>, 0, 1, 1);   // MN-major A and B
  constexpr uint32_t kHiS = desc_hi(8192), kHiO = desc_hi(128);
  constexpr int kRing = Cols<kMode>::ring;
  const uint32_t dq = desc_lo(sm.q, 128), dv = desc_lo(sm.v, 2048), dp = desc_lo(sm.p, 1024);
  const uint32_t leader = elect_lane();
  const int lane = threadIdx.x & 31;
  Count c;
  int u = cx.u0, tstart = cx.tstart;
  while (u < cx.u1) {
    seg_sync();
    block_sync();
    tc::tc_fence_after();
    const Span sp = span_of(sm.seg, u, cx.u1, tstart);
    const int units = sm.seg.n_chunks + kTileUnits;
    // Round i does S(i + 1), then PV(i), in steps
    //   0 S buffer free   1-4 a quarter of K there: its products   5 P there   6-9 a quarter of V there: its products
    // Lane n looks at the barrier of step n, so that one look (a trip through the busy shared
    // memory pipe) tells of all the round's steps.
    bool ok = true;
#pragma unroll 1
    for (int i = -1; ok && i < sp.n; ++i) {
      const bool more = i + 1 < sp.n;
      const uint32_t cs = c.all + i + 1, cv = c.all + i;      // running numbers of the two chunks
      const int es = kWeights<kMode> ? (i + 1) & 1 : 0;
      const uint32_t ps = kWeights<kMode> ? c.phase(i + 1) : cs;
      const int first = !more ? 5 : ps > 0 ? 0 : 1, last = kWeights<kMode> || i < 0 ? 4 : 9;
      const uint32_t bar = tc::smem_addr(lane == 0 ? &sm.s_free[es] : lane <= 4 ? &sm.kq_full[lane - 1]
                                                  : lane == 5 ? &sm.p_full : &sm.v_full[(lane - 6) & 3]);
      const uint32_t parity = (lane == 0 ? ps - 1 : lane <= 4 ? cs : cv) & 1;
      uint32_t ready = 0;
#pragma unroll 1
      for (int step = first; step <= last; ++step) {
        uint32_t n = 0;
#pragma unroll 1
        while (!(ready >> step & 1)) {
          ready = __ballot_sync(0xffffffffu, mbar_test(bar, parity));
          if ((++n & 255) == 0 && (n >> 24 || __any_sync(0xffffffffu, *abort != 0))) break;
        }
        ok = ready >> step & 1;
        if (!ok) {
          *abort = 1;
          break;
        }
        tc::tc_fence_after();
        if (step >= 1 && step <= 4) {
          const uint32_t q = step - 1, ka = cx.tm + Cols<kMode>::K + 64 * ((4 * cs + q) % kRing);
          const uint32_t d = cx.tm + Cols<kMode>::S + kRowsOf<kMode> * es;
#pragma unroll
          for (uint32_t ks = 0; ks < 8; ++ks) mma_ts<kHiS, kIdS>(leader, d, ka + 8 * ks, dq + (8 * q + ks) * 16, q | ks);
          mma_commit_by(leader, &sm.kq_free[q]);
          if (step == 4) mma_commit_by(leader, &sm.s_full[es]);
        } else if (!kWeights<kMode> && step >= 6) {
          const uint32_t mt = step - 6, va = dv + ((4 * cv + mt) % kVSlots) * (kChunk * kQuarter * 2 / 16);
#pragma unroll
          for (uint32_t kk = 0; kk < 8; ++kk)
            mma_ss<kHiO, kHiO, kIdO>(leader, cx.tm + kColO + 64 * mt, va + kk * 256,
                                     dp + kk * 128, (uint32_t)i | kk);
          mma_commit_by(leader, &sm.v_free[mt]);
          if (step == 9) mma_commit_by(leader, &sm.p_free);
        }
      }
    }
    __syncwarp();
    block_sync();
    if (*abort) break;
    c.add(sp.n);
    u = min(cx.u1, tstart + units);
    tstart += units;
  }
}

// The last warp: the packed pages of the chunks ahead into L2.
template <int kMode>
__device__ __forceinline__ void role_prefetch(const Ctx<kMode>& cx) {
  Smem<kMode>& sm = cx.sm;
  const DenseArgs& a = cx.a;
  volatile int* abort = &sm.abort;
  constexpr int kAhead = 5;
  const int lane = threadIdx.x & 31;
  uint32_t c = 0;
  int tile = cx.tile;
  int u = cx.u0, tstart = cx.tstart;
  while (u < cx.u1) {
    seg_sync();
    const Span sp = span_of(sm.seg, u, cx.u1, tstart);
    const int units = sm.seg.n_chunks + kTileUnits;
    {
      // the next tile's Q rows (contiguous)
      const int64_t rows = (int64_t)a.Tq * a.Hq;
      const int tn = tile + 1;
      if (tstart + units < cx.u1 && lane < kRowsOf<kMode> / 16) {
        const int64_t r0 = (int64_t)(cx.pl.tile0 + tn % cx.pl.tiles) * kRowsOf<kMode> + 16 * lane;
        const int64_t live = min(rows - r0, (int64_t)16);
        if (live > 0)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.Q + ((int64_t)(tn / cx.pl.tiles) * rows + r0) * kD),
                       "r"((uint32_t)(live * kD * 2))
                       : "memory");
      }
      auto request = [&](int i) {
        const int k = sp.k0 + i;
        if (i >= sp.n || k < sm.seg.nw || lane >= 4) return;
        const int lp = (sm.seg.c_hi - 1 - (k - sm.seg.nw)) * (kChunk / kPage) + (lane & 1);
        if (lp >= a.max_pages || (int64_t)lp * kPage >= sm.seg.e_hi) return;
        const int page = __ldg(a.page_table + (int64_t)sm.seg.b * a.max_pages + lp);
        if (page < 0 || page >= a.n_pages) return;
        const uint32_t bytes = (lane & 2) ? kPage * (kD / 16) : kPage * (kD / 2);
        const uint8_t* src = ((lane & 2) ? a.kv_scales : a.kv_codes) + (int64_t)page * bytes;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
      };
#pragma unroll 1
      for (int i = 1; i < kAhead; ++i) request(i);
      block_sync();
#pragma unroll 1
      for (int i = 0; i + kAhead < sp.n; ++i) {
        request(i + kAhead);
        // not a wait on s_full: this warp may fall behind by more than a phase
#pragma unroll 1
        for (uint32_t k = 0; k < (1u << 22); ++k) {
          if (*reinterpret_cast<volatile int*>(&sm.progress) >= (int)c + i + 1 || *abort) break;
          __nanosleep(100);
        }
        if (*abort) break;
      }
    }
    __syncwarp();
    block_sync();
    if (*abort) break;
    c += sp.n;
    u = min(cx.u1, tstart + units);
    tstart += units;
    ++tile;
  }
}

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1) k_dense_tc(DenseArgs a, Plan pl, const __grid_constant__ CUtensorMap map, uint32_t* status) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem<kMode>& sm = *reinterpret_cast<Smem<kMode>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5;
  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&sm.kq_full[i], 4 * kSplit<kMode>);
      tc::mbar_init(&sm.kq_free[i], 1);
      tc::mbar_init(&sm.v_full[i], 4 * kSplit<kMode>);
      tc::mbar_init(&sm.v_free[i], 1);
    }
    for (int i = 0; i < Stages<kMode>::K; ++i) {
      tc::mbar_init(&sm.kst_full[i], 1);
      tc::mbar_init(&sm.kst_free[i], 4 * kSplit<kMode>);
    }
    for (int i = 0; i < Stages<kMode>::V; ++i) {
      tc::mbar_init(&sm.vst_full[i], 1);
      tc::mbar_init(&sm.vst_free[i], 4 * kSplit<kMode>);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.s_free[i], kWeights<kMode> ? kSoftWarps / 2 : kSoftWarps);
    }
    tc::mbar_init(&sm.p_full, kSoftWarps);
    tc::mbar_init(&sm.p_free, 1);
    sm.abort = 0;
    sm.progress = 0;
    tc::mbar_fence_init();
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&sm.tmem, kTmemCols);
  pdl_wait();

  // ---- this CTA's share of the chunks of all tiles (their number is below 2^31)
  const int tiles = a.B * pl.tiles;
  int mine = 0, total = 0;
#pragma unroll 1
  for (int t = tid; t < tiles; t += kThreads) mine += tile_units<kMode>(a, pl, t);
  int inc = block_scan(mine, sm.scan, &total);
  const int ctas = min((int)gridDim.x, total), g = blockIdx.x;
  int u0 = g < ctas ? (int)((int64_t)total * g / ctas) : 0;
  int u1 = g < ctas ? (int)((int64_t)total * (g + 1) / ctas) : 0;
  if (tid == 0) sm.found_end = u1;
  __syncthreads();
  if (u1 > u0) {
    int base = 0, v = mine, all = total;
#pragma unroll 1
    for (int t0 = 0; t0 < tiles; t0 += kThreads) {
      if (tiles > kThreads) {          // (with one batch the first scan holds the answer)
        v = t0 + tid < tiles ? tile_units<kMode>(a, pl, t0 + tid) : 0;
        inc = block_scan(v, sm.scan, &all);
      }
      const int start = base + inc - v;
      if (t0 + tid < tiles && u0 >= start && u0 < start + v) {
        sm.found_tile = t0 + tid;
        sm.found_start = start;
      }
      if (t0 + tid < tiles && u1 >= start && u1 < start + v && u1 - start <= kTileUnits) sm.found_end = start;
      base += all;
      if (u1 < base) break;            // uniform
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tm = sm.tmem;
  if (u1 > u0) {
    if (u0 - sm.found_start <= kTileUnits) u0 = sm.found_start;
    u1 = sm.found_end;
  }
  Ctx<kMode> cx{a, pl, sm, tm, u0, u1, sm.found_tile, sm.found_start, status, &map};
  if (u1 <= u0) cx.tile = 0;
  if (!kWeights<kMode> && tid == 0) pl.cont[g] = (u1 > u0 && cx.tstart < u0) ? cx.tile : -1;

  // ---- roles, each with its own walk over the tiles (every walk meets the same barriers)
  if (warp < kValWarps + kKeyWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFill<kMode>));
    role_fill<kMode>(cx);
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft<kMode>));
    role_softmax<kMode>(cx);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMisc));
    if (warp == kMmaWarp)
      role_mma<kMode>(cx);
    else if (warp == kMmaWarp + 1)
      role_stage<kMode, false>(cx);
    else if (warp == kMmaWarp + 2)
      role_stage<kMode, true>(cx);
    else
      role_prefetch<kMode>(cx);
  }
  tc::tc_fence_before();
  block_sync();
  if (warp == kMmaWarp) tc::tmem_dealloc(tm, kTmemCols);
  if (tid == 0 && sm.abort) raise_status(status, CSA2_STATUS_TIMEOUT);
}

// Joins the partial results of tiles that several CTAs shared.  blockIdx.x = n-th such
// tile, blockIdx.y = row; 4 groups of 128 threads (4 channels each) take the partials
// in turn, and their sums are added in group order.
constexpr int kMergeGroups = 4;
__global__ void __launch_bounds__(128 * kMergeGroups) k_dense_merge(DenseArgs a, Plan pl) {
  __shared__ int s_first, s_count;
  __shared__ int s_cont[kMaxCtas];
  __shared__ float s_fac[kMaxCtas + 1];
  __shared__ float4 s_sum[kMergeGroups][128];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, r = blockIdx.y;
  for (int g = tid; g < pl.n_ctas; g += blockDim.x) s_cont[g] = pl.cont[g];
  if (tid == 0) s_first = -1;
  __syncthreads();
  if (tid < 32) {   // the n-th CTA that is the first to continue a tile
    int n = (int)blockIdx.x;
    for (int g0 = 0; g0 < pl.n_ctas; g0 += 32) {
      const int g = g0 + tid;
      const bool head = g > 0 && g < pl.n_ctas && s_cont[g] >= 0 && s_cont[g - 1] != s_cont[g];
      const uint32_t m = __ballot_sync(0xffffffffu, head);
      const int k = __popc(m);
      if (n < k) {
        if (head && __popc(m & ((1u << tid) - 1)) == n) s_first = g;
        break;
      }
      n -= k;
    }
  }
  __syncthreads();
  const int first = s_first;
  if (first < 0) return;
  const int tile = s_cont[first];
  const int b = tile / pl.tiles;
  const int64_t rows = (int64_t)a.Tq * a.Hq;
  const int64_t row = (int64_t)(pl.tile0 + tile % pl.tiles) * kRows + r;
  if (row >= rows) return;
  // partial 0: the CTA before (its last share), then every CTA that continues the tile
  if (tid < 32) {
    int count = 0;
    for (int g0 = first; g0 < pl.n_ctas; g0 += 32) {
      const bool in = g0 + tid < pl.n_ctas && s_cont[g0 + tid] == tile;
      const int k = __popc(__ballot_sync(0xffffffffu, in));
      count += k;
      if (k < 32) break;
    }
    if (tid == 0) s_count = count + 1;
    __syncwarp();
    float M = -INFINITY, L = 0.f;
    for (int q = tid; q <= count; q += 32) {
      const float* ml = pl.parts + (int64_t)(q == 0 ? 2 * (first - 1) + 1 : 2 * (first - 1 + q)) * kPartFloats + kRows * kD;
      M = fmaxf(M, ml[r]);
    }
    M = warp_max(M);
    for (int q = tid; q <= count; q += 32) {
      const float* ml = pl.parts + (int64_t)(q == 0 ? 2 * (first - 1) + 1 : 2 * (first - 1 + q)) * kPartFloats + kRows * kD;
      const float f = ml[r] == -INFINITY ? 0.f : ex2(ml[r] - M);
      s_fac[q] = f;
      L += f * ml[kRows + r];
    }
    L = warp_sum(L);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    for (int q = tid; q <= count; q += 32) s_fac[q] *= inv;
    if (a.lse && tid == 0)
      a.lse[(int64_t)b * rows + row] = L == 0.f ? -INFINITY : (M + kTopLog2 + log2f(L * kBottom)) * kLn2;
  }
  __syncthreads();
  const int n = s_count, grp = tid >> 7, c4 = tid & 127;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int q = grp; q < n; q += kMergeGroups) {
    const float* part = pl.parts + (int64_t)(q == 0 ? 2 * (first - 1) + 1 : 2 * (first - 1 + q)) * kPartFloats;
    const float4 v = *reinterpret_cast<const float4*>(part + r * kD + 4 * c4);
    const float f = s_fac[q];
    acc.x = fmaf(v.x, f, acc.x); acc.y = fmaf(v.y, f, acc.y); acc.z = fmaf(v.z, f, acc.z); acc.w = fmaf(v.w, f, acc.w);
  }
  s_sum[grp][c4] = acc;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int k = 1; k < kMergeGroups; ++k) {
      const float4 v = s_sum[k][c4];
      acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
    *reinterpret_cast<uint2*>(a.O + ((int64_t)b * rows + row) * kD + 4 * c4) =
        make_uint2(f32x2_bf16x2(acc.x, acc.y), f32x2_bf16x2(acc.z, acc.w));
  }
}

// weight_out[j] = (first slab: decay * weight_in[j], later ones: weight_out[j]) + the
// sums of the slab's tiles, in tile order.
__global__ void __launch_bounds__(256) k_weights_sum(DenseArgs a, Plan pl, int first_slab, uint32_t* status) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y;
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= dense_entries(a, b)) return;
  const int64_t slot = entry_slot(a.page_table, a.max_pages, a.n_pages, b, j, first_slab ? status : nullptr);
  if (slot < 0) return;
  const float w = first_slab ? (a.weight_in ? a.decay * a.weight_in[slot] : 0.f) : a.weight_out[slot];
  float sum = 0.f;                        // (by itself: the weight that was there may be much larger)
  for (int t = 0; t < pl.tiles; ++t) {
    const int64_t tile = (int64_t)b * pl.tiles + t;
    const int2 rg = pl.ranges[tile];
    if (j >= rg.x && j < rg.y) sum += pl.sums[tile * pl.sum_stride + j];
  }
  a.weight_out[slot] = w + sum;
}
// The entries whose sums a tile writes (whole chunks).
__global__ void __launch_bounds__(128) k_weights_ranges(DenseArgs a, Plan pl) {
  pdl_trigger();
  pdl_wait();
  const int tile = blockIdx.x * 128 + threadIdx.x;
  if (tile >= a.B * pl.tiles) return;
  const int b = tile / pl.tiles;
  const int r0 = (pl.tile0 + tile % pl.tiles) * pl.rows;
  const int64_t rows = (int64_t)a.Tq * a.Hq;
  int lo = INT_MAX, hi = 0;
  if (r0 < rows) {
    const int n_ent = dense_entries(a, b);
    const int64_t shift = dense_shift(a, b);
    const int i1 = (int)(min((int64_t)r0 + pl.rows, rows) - 1) / a.Hq;
#pragma unroll 1
    for (int i = r0 / a.Hq; i <= i1; ++i) {
      const DenseRow r = dense_row(a, b, i, n_ent, shift, 0);
      const int f = dense_first(a, r.doc, shift);
      if (r.nv > f) {
        lo = min(lo, f);
        hi = max(hi, r.nv);
      }
    }
  }
  pl.ranges[tile] = hi > lo ? make_int2(lo / kChunk * kChunk, (hi + kChunk - 1) / kChunk * kChunk) : make_int2(0, 0);
}

int tiles_of(const csa2_dims* dm, int rows) { return (int)(((int64_t)dm->Tq * dm->Hq + rows - 1) / rows); }
int weights_rows(const csa2_dims* dm) { return (int64_t)dm->Tq * dm->Hq > 64 ? 128 : 64; }

// Units that a sequence's tile can have.
int64_t max_chunks(int max_entries, int W, int64_t tq) {
  return ((int64_t)max_entries + kChunk - 1) / kChunk + ((int64_t)W + tq + kChunk - 1) / kChunk + 2 + kTileUnits;
}

cudaError_t device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e;
}

// The register split adds up to what the block is launched with; a build whose
// kernel has fewer registers per thread must not run it (its wait would not end).
template <int kMode>
cudaError_t prepare_kernel() {
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, k_dense_tc<kMode>);
  if (e != cudaSuccess) return e;
  static_assert(4 * kRegsFill<kMode> + 2 * kRegsSoft<kMode> + kRegsMisc <= 7 * kRegsLaunch, "register split");
  if (at.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(k_dense_tc<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sizeof(Smem<kMode>));
}

// Sums of the weights' tiles: at most this many bytes per slab of tiles.
constexpr size_t kSumBytes = (size_t)256 << 20;

int slab_tiles(const csa2_dims* dm, int max_entries, int64_t* stride) {
  *stride = ((int64_t)max_entries + kChunk - 1) / kChunk * kChunk;
  const int64_t per = std::max<int64_t>(1, dm->B) * *stride * 4;
  return (int)std::max<int64_t>(1, std::min<int64_t>(tiles_of(dm, weights_rows(dm)), (int64_t)kSumBytes / std::max<int64_t>(1, per)));
}

// Tiles of every sequence that one launch takes: its units of work stay below 2^31.
int launch_tiles(int64_t units_per_tile, int tiles) {
  return (int)std::min<int64_t>(tiles, ((int64_t)INT_MAX) / std::max<int64_t>(1, units_per_tile));
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

bool dense_tc_supported(const csa2_dims* dm) { return dm->d == kD; }

size_t dense_attn_workspace_bytes(const csa2_dims* dm, int max_entries) {
  // two slots per CTA, and never more CTAs than chunks
  const int64_t units = (int64_t)dm->B * tiles_of(dm, kRows) * max_chunks(max_entries, dm->W, dm->swa_cap);
  const int64_t ctas = std::min<int64_t>(kMaxCtas, std::max<int64_t>(1, units));
  return up((size_t)kMaxCtas * 4) + (size_t)ctas * 2 * kPartFloats * sizeof(float);
}

// The packed codes as rows of 256 bytes; a box is one quarter of a page's 64 entries.
static bool codes_map(const DenseArgs& a, CUtensorMap* map) {
  const cuuint64_t dims[2] = {(cuuint64_t)(kD / 2), (cuuint64_t)a.n_pages * kPage};
  const cuuint64_t strides[1] = {(cuuint64_t)(kD / 2)};
  const cuuint32_t box[2] = {(cuuint32_t)(kQuarter / 2), (cuuint32_t)kPage};
  const cuuint32_t estr[2] = {1, 1};
  return tensor_map_encoder() &&
         tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.kv_codes), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_dense_attn_tc(const csa2_dims* dm, const DenseArgs& a, void* ws, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e == cudaSuccess) e = prepare_kernel<0>();
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  if (!codes_map(a, &map)) return cudaErrorInvalidValue;
  Plan pl = {};
  pl.rows = kRows;
  const int all = tiles_of(dm, kRows);
  pl.cont = static_cast<int32_t*>(ws);
  pl.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + up((size_t)kMaxCtas * 4));
  const int64_t per_tile = (int64_t)a.B * max_chunks(a.max_entries, a.W, a.swa_cap);   // units of a tile of every sequence
  const int slab = launch_tiles(per_tile, all);
  if (slab == 0) return cudaErrorInvalidConfiguration;
  for (int t0 = 0; t0 < all; t0 += slab) {
    pl.tile0 = t0;
    pl.tiles = std::min(slab, all - t0);
    pl.n_ctas = (int)std::min<int64_t>(std::min(sms, kMaxCtas), per_tile * pl.tiles);
    e = launch_step(k_dense_tc<0>, dim3(pl.n_ctas), dim3(kThreads), sizeof(Smem<0>), s, a, pl, map, status_word());
    if (e != cudaSuccess) return e;
    if (pl.n_ctas == 1) continue;
    const unsigned shared = (unsigned)std::min<int64_t>((int64_t)a.B * pl.tiles, pl.n_ctas - 1);
    e = launch_step(k_dense_merge, dim3(shared, kRows), dim3(128 * kMergeGroups), 0, s, a, pl);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

size_t entry_weights_workspace_bytes(const csa2_dims* dm, int max_entries) {
  if (tiles_of(dm, weights_rows(dm)) <= 1) return 0;
  int64_t stride;
  const int tiles = slab_tiles(dm, max_entries, &stride);
  return up((size_t)dm->B * tiles * sizeof(int2)) + (size_t)dm->B * tiles * stride * sizeof(float);
}

template <int kMode>
static cudaError_t launch_weights(const csa2_dims* dm, const DenseArgs& a, void* ws, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e == cudaSuccess) e = prepare_kernel<kMode>();
  if (e != cudaSuccess) return e;
  const int all = tiles_of(dm, kMode);
  CUtensorMap map;
  if (!codes_map(a, &map)) return cudaErrorInvalidValue;
  Plan pl = {};
  pl.rows = kMode;
  const int64_t per_tile = (int64_t)a.B * max_chunks(a.max_entries, 0, 0);
  const int slab = std::min(launch_tiles(per_tile, all), all <= 1 ? 1 : slab_tiles(dm, a.max_entries, &pl.sum_stride));
  if (slab == 0) return cudaErrorInvalidConfiguration;
  for (int t0 = 0; t0 < all; t0 += slab) {
    pl.tile0 = t0;
    pl.tiles = std::min(slab, all - t0);
    pl.n_ctas = (int)std::min<int64_t>(std::min(sms, kMaxCtas), per_tile * pl.tiles);
    if (all > 1) {
      pl.ranges = static_cast<int2*>(ws);
      pl.sums = reinterpret_cast<float*>(static_cast<char*>(ws) + up((size_t)a.B * slab * sizeof(int2)));
      e = launch_step(k_weights_ranges, dim3((unsigned)(((int64_t)a.B * pl.tiles + 127) / 128)), dim3(128), 0, s, a, pl);
      if (e != cudaSuccess) return e;
    }
    e = launch_step(k_dense_tc<kMode>, dim3(pl.n_ctas), dim3(kThreads), sizeof(Smem<kMode>), s, a, pl, map, status_word());
    if (e != cudaSuccess) return e;
    if (all > 1) {
      e = launch_step(k_weights_sum, dim3((unsigned)((a.max_entries + 255) / 256), (unsigned)a.B), dim3(256), 0, s, a, pl,
                      (int)(t0 == 0), status_word());
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

cudaError_t launch_entry_weights_tc(const csa2_dims* dm, const DenseArgs& a, void* ws, cudaStream_t s) {
  return weights_rows(dm) == 64 ? launch_weights<64>(dm, a, ws, s) : launch_weights<128>(dm, a, ws, s);
}

}  // namespace csa2
