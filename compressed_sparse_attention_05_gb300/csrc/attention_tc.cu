// Gathered sparse MQA attention on the fifth-generation tensor cores
// (tcgen05, accumulators in tensor memory).  "DeepSeek-V4.1 架构解析" §02
// (one shared latent KV head, attention over the Top-K selection) and §03
// (FP4 main KV dequantised before the matmul; FP8 sliding window of the last
// 128 tokens).  Same result as the legacy kernels of attention.cu: head
// layout, key set and softmax follow reading R11 of include/csa2.h.
//
// Shapes: d = 512, up to 128 query heads (one CTA per group of 64), up to
// 3,072 keys per token (K <= 2,048 plus W <= 1,024).  The
// token's key list (selected entries, then window rows) is cut into chunks
// of 128 keys.  Swapped operands put the 128 keys of a chunk, not the 64
// heads, on the MMA's M side:
//   S^T [128 keys x 64 heads]  = K_chunk [128 x 512] . Q^T      (32 MMAs, k = 16 dims)
//   O^T [512 dims x 64 heads] += V_chunk^T [512 x 128] . P^T    (4 M-tiles x 8 MMAs, k = 16 keys)
// K = V, so one dequantised shared-memory tile serves as the K-major A
// operand of the first product and as the MN-major A operand of the second.
// S^T takes 64 tensor-memory columns and O^T four M-tiles of 64.  PV runs
// tile by tile with a commit per two tiles, so that the next chunk's half of
// the K tile is rewritten as soon as the tiles that read it are done.
//
// A CTA (16 worker warps and one MMA warp) owns one token (all heads) and a contiguous run of its
// chunks.  Per chunk: the threads dequantise the tile in two halves of 256 dims
// (thread = one key x 64 dims of each half, a warp = 8 whole keys); each
// warp announces a written half on an mbarrier and
// the MMA warp issues the half's sixteen S MMAs once all warps have, so
// dequantisation overlaps the tensor core.  (An MMA issue blocks the issuing
// thread while the tensor pipe is full, hence a warp of its own.)  The next
// chunk's bytes are requested together once the tile is written.  The load
// units bound a chunk as much as the tensor cores do: they take a request of
// a warp line by line, so a key's four threads read whole lines, 32 bytes each
// (256 tokens of 640 keys: 61 us; 16 bytes each, twice the requests, 69; four
// slices of 128 dims instead of two halves made no difference).  Softmax (thread = one key x 16 heads): the reference maximum of a
// head only moves when a score exceeds it by more than 2^8 (then O^T is
// rescaled in tensor memory), so P = exp2(s - m) <= 256 fits fp16 and most
// chunks need no maximum reduction at all; row sums stay per thread until
// the end of the token.
//
// Few tokens (decode): a token's keys are spread evenly over a cluster of up
// to 8 CTAs; each CTA finishes a partial (m, l, O) and the cluster merges
// them through distributed shared memory, without global scratch: every rank
// owns a slice of the heads and sums the ranks' scaled partials of those heads
// in rank order.
//
// Operands are fp16.  MXFP4 values (<= 6 significant bits, in [2^-10, 2688])
// are exact.  bf16 values outside fp16's range are brought into it by powers
// of two, which change no bit of a significand: each head of Q is scaled by
// 2^-e_h so that its largest magnitude lies in [2^14, 2^15) (and its logits
// are multiplied back by 2^e_h), and a window row whose per-token scale lies
// outside [2^-8, 2^7] is dequantised with the scale 2^-f s (s' in [1, 2)), its
// logits multiplied back by 2^f and its softmax weight carried as 2^f p in the
// PV product (the reference maximum then follows the largest 2^f p, and the
// normaliser adds p itself).  Main-KV entries in the FP8 format (the V4-style
// layout kept for the A/B against MXFP4: E4M3 row + fp32 scale, one 32-byte
// run of codes per thread and 128 dims) go through the window rows' path: code x
// scale rounded to bf16, the same power-of-two treatment; the kernel is
// instantiated once per format.  P is rounded to fp16 for the PV product; the
// normaliser sums the unrounded fp32 P (relative difference <= 2^-11).
// Accumulation is fp32.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "operands.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kD = 512;          // latent width (keys = values)
constexpr int kHeads = 64;       // N of both products; fewer heads are zero-padded
constexpr int kChunk = 128;      // keys per chunk (M of the score product)
constexpr int kMaxChunks = 24;   // keys per token <= 3,072 (K <= 2,048 plus W <= 1,024)
constexpr int kMaxSplit = 8;     // CTAs per token in the cluster path (largest portable cluster)
constexpr int kWorkers = 512;             // 16 warps: dequantisation and softmax
constexpr int kThreads = kWorkers + 32;   // + one warp that allocates tensor memory and issues the MMAs
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;     // S^T: 64 columns
constexpr uint32_t kColO = 256;   // O^T: four M-tiles of 64 columns
constexpr float kRescaleLog2 = 8.f;  // move a head's reference maximum only beyond this growth

// Byte offsets inside the operand tiles (no-swizzle canonical layout: core
// matrices of 8 rows x 16 bytes).
//   Q  [head][dim]: (h/8)*8192 + (d/8)*128 + (h%8)*16 + (d%8)*2
//   K  [key][dim]:  (k/8)*8192 + (d/8)*128 + (k%8)*16 + (d%8)*2
//   P  [key][head]: (k/8)*1024 + (h/8)*128 + (k%8)*16 + (h%8)*2
struct TcSmem {
  uint16_t q[kHeads * kD];
  uint16_t k[kChunk * kD];             // becomes the fp32 partial O [64][512] in the cluster merge
  uint16_t p[kChunk * kHeads];
  int32_t slot[kMaxChunks * kChunk];   // >= 0 main-KV slot; <= -2 window row (-2 - row); -1 none
  int8_t kexp[kMaxChunks * kChunk];    // window row: exponent f of its dequantisation scale (0: none)
  float red[4][kHeads];                // per lane-quarter partial max / sum
  float sl2h[kHeads];                  // logit multiplier of each head: softmax scale * log2(e) * 2^e_h
  int qexp[kHeads];                    // largest bf16 exponent field of each head of Q
  float m_ref[kHeads];                 // reference maximum (log2 domain) of each head
  float m_thr[kHeads];                 // m_ref + 2^8 growth allowance
  float m_exp[kHeads];                 // m_ref, or 0 while the head has seen no key
  float alpha[kHeads], l_run[kHeads], fac[kHeads];
  uint64_t k_ready[2];   // workers -> MMA warp: half of the K tile (256 dims) written (one arrival per warp)
  uint64_t p_ready;      // workers -> MMA warp: P written, O^T rescaled
  uint64_t bar_q;        // Q's rows have arrived in the K tile
  uint64_t bar_s;        // MMA commit: S^T complete
  uint64_t bar_pv[2];    // MMA commit: two PV M-tiles complete (their half of the K tile is free again)
  uint32_t tmem;
  int abort;
};

// ---- distributed shared memory (cluster merge) ------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Barrier / vote among the worker warps only (the MMA warp never joins).
__device__ __forceinline__ void workers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kWorkers) : "memory");
}
__device__ __forceinline__ bool workers_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(kWorkers)
      : "memory");
  return r != 0;
}

// Packed bytes of one key, held in registers from the moment they are requested until the
// half of the dims that they belong to is stored, so that the gather of the next chunk
// overlaps this chunk's products.
struct KeyBytes {
  uint4 v[4];
};
// Loads that the compiler keeps where they are written (volatile): a plain load
// may be moved down to its first use, which would turn the prefetch into a stall.
// 32 bytes (rows of 256 or 512 bytes: aligned as the tensor is, at least to 16).
__device__ __forceinline__ void ld_gather32(const uint8_t* p, uint4& lo, uint4& hi) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(lo.x), "=r"(lo.y), "=r"(lo.z), "=r"(lo.w), "=r"(hi.x), "=r"(hi.y), "=r"(hi.z), "=r"(hi.w)
                 : "l"(p));
  } else {
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(lo.x), "=r"(lo.y), "=r"(lo.z), "=r"(lo.w) : "l"(p));
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(hi.x), "=r"(hi.y), "=r"(hi.z), "=r"(hi.w) : "l"(p + 16));
  }
}
__device__ __forceinline__ uint2 ld_gather8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_gather4f(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
// MXFP4 scales of a key: quarter qd loads bytes 8*qd .. +7 (the groups of dims 128 qd ..)
__device__ __forceinline__ uint2 load_scales(const AttnArgs& a, int32_t src, int qd) {
  return src >= 0 ? ld_gather8(a.kv_scales + (int64_t)src * (kD / 16) + 8 * qd) : make_uint2(0, 0);
}
// Codes and scale of window row w: the rows of the window buffer, then (with a tree of drafted tokens) the nodes'.
template <bool kTree>
__device__ __forceinline__ const uint8_t* window_codes(const AttnArgs& a, int64_t w) {
  if (kTree && w >= (int64_t)a.B * a.swa_cap) return a.tree_codes + (w - (int64_t)a.B * a.swa_cap) * kD;
  return a.swa_codes + w * kD;
}
template <bool kTree>
__device__ __forceinline__ const float* window_scale(const AttnArgs& a, int64_t w) {
  if (kTree && w >= (int64_t)a.B * a.swa_cap) return a.tree_scales + (w - (int64_t)a.B * a.swa_cap);
  return a.swa_scales + w;
}
// A key stored as an FP8 row: a window row, or a main-KV entry in the FP8 format.
template <bool kFp8>
__device__ __forceinline__ bool fp8_row_key(int32_t src) {
  return src <= -2 || (kFp8 && src >= 0);
}

// Packed bytes of a key for the thread's 64 dims of half P (256 P ..).  MXFP4 entry: dims 64 qd .. +63, 32 bytes, in
// v[2 P] and the next (both halves are requested together).  FP8 row: dims 32 qd .. +31 and 128 + 32 qd .. +31, in all
// four (the second half reuses the registers once the first is stored).  Either way the quarters of a key read whole
// 128-byte lines, half as many requests as 16 bytes a lane.
template <int P, bool kFp8, bool kTree>
__device__ __forceinline__ void load_half(const AttnArgs& a, int32_t src, int qd, KeyBytes& kb) {
  if (src == -1) return;
  if (fp8_row_key<kFp8>(src)) {
    const uint8_t* p = (src <= -2 ? window_codes<kTree>(a, -2 - (int64_t)src) : a.kv_codes + (int64_t)src * kD) +
                       256 * P + 32 * qd;
    ld_gather32(p, kb.v[0], kb.v[1]);
    ld_gather32(p + 128, kb.v[2], kb.v[3]);
  } else {
    ld_gather32(a.kv_codes + (int64_t)src * (kD / 2) + 128 * P + 32 * qd, kb.v[2 * P], kb.v[2 * P + 1]);
  }
}
// Dequantisation scale of an FP8 row (a window row, or a main-KV entry in the FP8
// format), times 2^-f (see window_exp); 0 for an MXFP4 entry or no key.
template <bool kFp8, bool kTree>
__device__ __forceinline__ float load_wscale(const AttnArgs& a, int32_t src) {
  float sw;
  if (src <= -2) sw = ld_gather4f(window_scale<kTree>(a, -2 - (int64_t)src));
  else if (kFp8 && src >= 0) sw = ld_gather4f(reinterpret_cast<const float*>(a.kv_scales) + src);
  else return 0.f;
  return sw * pow2i(-window_exp(sw));
}
// Exponent f of a key's FP8 scale (0 for MXFP4 entries and missing keys).
template <bool kFp8, bool kTree>
__device__ __forceinline__ int key_exp(const AttnArgs& a, int32_t src) {
  if (src <= -2) return window_exp(__ldg(window_scale<kTree>(a, -2 - (int64_t)src)));
  if (kFp8 && src >= 0) return window_exp(__ldg(reinterpret_cast<const float*>(a.kv_scales) + src));
  return 0;
}

// 32 E4M3 codes (c0: dims 0-15, c1: 16-31) times the (2^-f scaled) row scale,
// rounded to bf16 as the operand rule says, into 4 core-matrix rows of fp16.
__device__ __forceinline__ void store_fp8_dims(uint4 c0, uint4 c1, float sc, unsigned char* dst) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 c = j < 2 ? c0 : c1;
    const uint32_t w0 = word_of(c, (j & 1) * 2), w1 = word_of(c, (j & 1) * 2 + 1);
    uint4 o;
    o.x = win2_f16x2(w0 & 0xFFFFu, sc);
    o.y = win2_f16x2(w0 >> 16, sc);
    o.z = win2_f16x2(w1 & 0xFFFFu, sc);
    o.w = win2_f16x2(w1 >> 16, sc);
    *reinterpret_cast<uint4*>(dst + j * 128) = o;
  }
}

// Dequantise the thread's 64 dims of half P into the K tile (8 core-matrix rows); scales: of its four groups of 16 dims.
template <int P, bool kFp8>
__device__ __forceinline__ void store_half(const KeyBytes& kb, uint32_t scales, int32_t src, float wsc, int key, int qd,
                                           unsigned char* ktile) {
  unsigned char* dst = ktile + (key >> 3) * 8192 + 32 * P * 128 + (key & 7) * 16;
  if (fp8_row_key<kFp8>(src)) {
    store_fp8_dims(kb.v[0], kb.v[1], wsc, dst + 4 * qd * 128);
    store_fp8_dims(kb.v[2], kb.v[3], wsc, dst + (16 + 4 * qd) * 128);
  } else {
    dst += 8 * qd * 128;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t s = e4m3x2_f16x2(scales >> (16 * i) & 0xFFFFu);
      const uint32_t g0 = prmt(s, s, 0x1010u), g1 = prmt(s, s, 0x3232u);   // (scale, scale) of each group
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 o = make_uint4(0, 0, 0, 0);
        if (src >= 0) {
          const uint32_t s2 = j < 2 ? g0 : g1;
          e2m1x8_f16x8(word_of(kb.v[2 * P + i], j), o.x, o.y, o.z, o.w);
          o.x = hmul2(o.x, s2);   // exact: <= 6 significant bits
          o.y = hmul2(o.y, s2);
          o.z = hmul2(o.z, s2);
          o.w = hmul2(o.w, s2);
        }
        *reinterpret_cast<uint4*>(dst + (4 * i + j) * 128) = o;
      }
    }
  }
}

// Resolves key kk of a CTA's key list -- sel_cap selection slots (slots sel_off ..
// of the token's Top-K, the first n_sel of which hold selected entries), then
// window rows from raw position w_first -- to a main-KV slot (page table) or a
// window row, or -1 past the list [.., kk_end) or in an unused selection slot.
// The index load does not wait for n_sel when sel_cap is fixed (the cluster path).
// With a tree, window row w_first + i is the token's ancestor of that position from
// position `ctx` on (and the window's rows end there).
template <bool kTree>
__device__ __forceinline__ int32_t key_source(const AttnArgs& a, int64_t row, int b, int kk, int n_sel, int sel_off,
                                              int sel_cap, int kk_end, int nv, int w_first, int pos0, int ctx,
                                              uint32_t* status) {
  if (kk >= kk_end) return -1;
  if (kk < sel_cap) {
    const int j = __ldg(a.idx + row * a.K + sel_off + kk);
    if (sel_off + kk >= n_sel) return -1;
    if (j < 0 || j >= nv || (j >> 6) >= a.max_pages) {
      raise_status(status, CSA2_STATUS_BAD_INDEX);
      return -1;
    }
    const int p = __ldg(a.page_table + (int64_t)b * a.max_pages + (j >> 6));
    if (p < 0 || p >= a.n_pages) {
      raise_status(status, CSA2_STATUS_BAD_PAGE);
      return -1;
    }
    return p * kPage + (j & (kPage - 1));
  }
  const int p = w_first + (kk - sel_cap);
  if (kTree && p >= ctx) {
    const int node = p - ctx < a.max_depth ? __ldg(a.path + row * a.max_depth + (p - ctx)) : -1;
    if (node < 0 || node >= a.Tq) {
      raise_status(status, CSA2_STATUS_BAD_INDEX);
      return -1;
    }
    return (int32_t)(-2 - ((int64_t)a.B * a.swa_cap + (int64_t)b * a.Tq + node));
  }
  if (kTree && (p < pos0 || (uint32_t)p - (uint32_t)pos0 >= (uint32_t)a.swa_cap)) return -1;   // not held by the buffer
  return (int32_t)(-2 - ((int64_t)b * a.swa_cap + (p - pos0)));
}

// Scores of the thread's key for heads 16*hg .. +15 in the log2 domain, as
// the PV product carries them: y = x + f with x = S^T * scale * log2(e) (the
// head's and the key's powers of two undone), or -inf for a missing key.
__device__ __forceinline__ void load_scores(uint32_t tm, int hg, uint32_t lane_q, bool valid, const float* sl2h,
                                            int fk, float (&x)[16]) {
  tc::tmem_ld16(tm + kColS + 16 * hg + lane_q, x);
  tc::tmem_wait_ld();
  const float4* m4 = reinterpret_cast<const float4*>(sl2h + 16 * hg);
#pragma unroll
  for (int j4 = 0; j4 < 4; ++j4) {
    const float4 m = m4[j4];
    x[4 * j4] *= m.x; x[4 * j4 + 1] *= m.y; x[4 * j4 + 2] *= m.z; x[4 * j4 + 3] *= m.w;
  }
  if (fk != 0) {   // a rescaled window row: logits times 2^f, weights carried as 2^f p
    const float kf = pow2i(fk), ff = (float)fk;
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = x[j] * kf + ff;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = valid ? x[j] : -INFINITY;
}

// Bounded wait of a whole warp; on time-out the CTA's abort flag is raised.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool ok = false;
  for (uint32_t i = 0; i < (1u << 21); ++i) {   // <= 2^21 suspensions of <= 1 us
    if (tc::mbar_try_wait_sleep(bar, parity, 1000)) {
      ok = true;
      break;
    }
    if ((i & 63) == 63 && *abort) break;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) *abort = 1;
  return ok;
}

template <bool kFp8, bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
k_sparse_attn_tc(AttnArgs a, uint32_t* status, int n_split) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  TcSmem& sm = *reinterpret_cast<TcSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool mma_warp = warp == kWorkers / 32;
  const int64_t row = blockIdx.x / n_split;
  const int rank = (int)(blockIdx.x % n_split);
  const int b = (int)(row / a.Tq);
  const int hb = kHeads * (int)blockIdx.y;   // first head of this CTA's group of 64
  // dequantisation: one key, 64 dims of each half.  A warp holds 8 whole keys
  // (coalesced loads); lanes 8q .. 8q+7 hold quarter q of the 8 keys, so each
  // 8-lane phase of a 16-byte store covers 8 distinct bank groups.
  const int key = ((warp & 15) << 3) | (lane & 7), qd = (lane >> 3) & 3;
  const int q4 = warp & 3, hg = (warp >> 2) & 3;             // softmax: key 32*q4 + lane (= key), heads 16*hg ..
  volatile int* abort = &sm.abort;

  pdl_trigger();
  if (kTree) pdl_wait();
  // ---- before the previous kernel of the step is done: the token's own inputs
  // (scalars, Q rows), barriers, tensor memory and the Q operand (a tree's positions come from its plan, which lets
  // nothing start before it is done)
  const int t = kTree ? max(a.q_pos[row], -1) : a.q_pos[row];   // (-1: no node of the tree)
  int n_sel = kTree ? a.cnt[row] : 0;
  const int n_ent = a.n_entries[b];
  const int pos0 = a.swa_cap > 0 ? a.swa_pos0[b] : 0;
  if (tid == 0) {
    tc::mbar_init(&sm.bar_q, 1);
    tc::mbar_init(&sm.bar_s, 1);
    tc::mbar_init(&sm.p_ready, kWorkers / 32);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.bar_pv[i], 1);
      tc::mbar_init(&sm.k_ready[i], kWorkers / 32);
    }
    sm.abort = 0;
    tc::mbar_fence_init();
    // Q's rows into the K tile, which is free until the first chunk is dequantised
    const uint32_t bytes = (uint32_t)min(kHeads, a.Hq - hb) * kD * sizeof(uint16_t);
    tc::mbar_arrive_expect_tx(&sm.bar_q, bytes);
    tc::bulk_g2s(sm.k, a.Q + (row * a.Hq + hb) * kD, bytes, &sm.bar_q);
  }
  if (mma_warp) tc::tmem_alloc(&sm.tmem, kTmemCols);
  if (tid < kHeads) {
    sm.m_ref[tid] = -INFINITY;
    sm.m_thr[tid] = -INFINITY;
    sm.m_exp[tid] = 0.f;
    sm.qexp[tid] = 0;
  }
  // the window rows of the token: raw positions max(0, t-W+1, pos0) .. min(t, last row held)
  // (t may lie before the first position, and the buffer's last row behind the last)
  const int first = max(0, max(t, 0) - max(a.W - 1, 0));
  int w_lo = max(first, pos0);
  int w_hi = pos0 <= t && (uint32_t)t - (uint32_t)pos0 >= (uint32_t)a.swa_cap ? pos0 + a.swa_cap - 1 : t;
  int ctx = 0;
  if (kTree) {   // from the first position that the buffer holds (or the first ancestor) to the token itself
    ctx = max(0, a.ctx_len[b]);
    w_lo = max(first, min(a.swa_cap > 0 ? pos0 : INT_MAX, ctx));
    w_hi = t;
  }
  const int n_win = a.W > 0 && w_hi >= w_lo ? w_hi - w_lo + 1 : 0;
  int n_mine = 0, n_my = 0;
  int32_t cur_src = -1;
  float cur_wsc = 0.f;
  uint2 cur_sc = make_uint2(0, 0);
  KeyBytes kb;
  auto load_first = [&] {   // the first chunk's packed bytes
    load_half<0, kFp8, kTree>(a, cur_src, qd, kb);
    if (!fp8_row_key<kFp8>(cur_src)) {
      load_half<1, kFp8, kTree>(a, cur_src, qd, kb);
      cur_sc = load_scales(a, cur_src, qd);
    }
    cur_wsc = load_wscale<kFp8, kTree>(a, cur_src);
  };
  auto resolve = [&] {
    // ---- the selection (and the window rows) come from earlier kernels of the step
    if (!kTree) {
      pdl_wait();
      n_sel = a.cnt[row];
    } else if (t < 0) {
      n_sel = 0;
    }
    const int nv = n_visible(n_ent, t);
    if (n_sel < 0 || n_sel > a.K) {
      if (tid == 0 && rank == 0) raise_status(status, CSA2_STATUS_BAD_COUNT);
      n_sel = n_sel < 0 ? 0 : a.K;
    }
    // the key list.  One CTA per token: its n_sel selected entries, then its window
    // rows.  A cluster: rank r takes an equal share of the K selection slots (unused
    // ones empty, so that the index loads need not wait for the count) and an equal
    // share of the window rows.  With a tree the count is there as early as the
    // position, and rank r takes an equal share of the keys that there are: none has a
    // chunk more than it must (640 keys over five ranks are 128 for each, where two
    // shares rounded by themselves are 129 for one), and short contexts no empty ones.
    int sel_off = 0, sel_cap = n_sel, w_first = w_lo;
    n_mine = n_sel + n_win;
    if (n_split > 1) {
      auto cut = [&](int r, int* win) {   // the first selected entry and window row of rank r
        const int sel = (int)((int64_t)(kTree ? n_sel : a.K) * r / n_split);
        *win = (int)((int64_t)n_win * r / n_split);
        if (!kTree) return sel;
        const int all = (int)((int64_t)(n_sel + n_win) * r / n_split);
        const int mine = n_win >= n_split ? sel : min(all, n_sel);   // (so that the rest never goes back)
        *win = all - mine;
        return mine;
      };
      int u0, u1;
      sel_off = cut(rank, &u0);
      sel_cap = cut(rank + 1, &u1) - sel_off;
      w_first = w_lo + u0;
      n_mine = sel_cap + (u1 - u0);
    }
    n_my = (n_mine + kChunk - 1) / kChunk;   // chunks of kChunk keys, <= kMaxChunks

    // ---- key sources: a key's chunks are shared out among its four threads, the first four chunks before the first
    // chunk's packed bytes are requested
    if (!mma_warp && n_my > 0) {
      auto resolve_chunk = [&](int c) {
        const int32_t src = key_source<kTree>(a, row, b, c * kChunk + key, n_sel, sel_off, sel_cap, n_mine, nv, w_first, pos0, ctx,
                                              status);
        sm.slot[c * kChunk + key] = src;
        sm.kexp[c * kChunk + key] = (int8_t)key_exp<kFp8, kTree>(a, src);
        return src;
      };
      const int32_t src = qd < n_my ? resolve_chunk(qd) : -1;
      cur_src = __shfl_sync(0xffffffffu, src, lane & 7);
      load_first();
      for (int c = qd + 4; c < n_my; c += 4) resolve_chunk(c);
    }
  };
  // The keys' chain of loads (index, page, bytes) runs while Q is on its way.  A cluster of the layer step does the
  // work on Q first, which needs none of the previous kernel's results and hides behind its end.
  const bool early = kTree || n_split == 1;
  if (early) resolve();
  __syncthreads();
  // units of (head 8 r + lane % 8, 8 dims): eight lanes have eight dim groups too, so that neither the reads of rows nor
  // the writes of core matrices meet in a bank
  uint4 qv[8];
  const int c8 = (tid >> 3 & ~7) | (((tid >> 3) + lane) & 7);
  if (!mma_warp) {
    const bool here = warp_wait(&sm.bar_q, 0, abort);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int h = 8 * r + (lane & 7);
      qv[r] = here && hb + h < a.Hq ? *reinterpret_cast<const uint4*>(sm.k + h * kD + c8 * 8) : make_uint4(0, 0, 0, 0);
    }
    // largest bf16 exponent field of each head (lanes L, L^8, L^16, L^24 share a head), of heads h and h + 32 at once
    uint32_t e[4];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max_u16x2(m, word_of(qv[r], j) & 0x7FFF7FFFu);
      m = max(m >> 23, (m >> 7) & 0xFFu);
      if (r < 4) e[r] = m;
      else e[r - 4] |= m << 16;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      e[r] = max_u16x2(e[r], __shfl_xor_sync(0xffffffffu, e[r], 8));
      e[r] = max_u16x2(e[r], __shfl_xor_sync(0xffffffffu, e[r], 16));
    }
    const uint32_t m = qd == 0 ? e[0] : qd == 1 ? e[1] : qd == 2 ? e[2] : e[3];
    atomicMax(&sm.qexp[lane], (int)(m & 0xFFFFu));
    atomicMax(&sm.qexp[32 + lane], (int)(m >> 16));
  }
  __syncthreads();
  // per head: 2^-e_h brings the largest magnitude into [2^14, 2^15) (e_h in [-110, 110])
  if (tid < kHeads) {
    const int eh = q_head_exp(sm.qexp[tid]);
    sm.qexp[tid] = eh;
    sm.sl2h[tid] = a.scale * 1.4426950408889634f * pow2i(eh);
  }
  __syncthreads();
  // Q (bf16) -> fp16 B operand, head h scaled by 2^-e_h (exact)
  if (!mma_warp) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int h = 8 * r + (lane & 7);
      const float qs = pow2i(-sm.qexp[h]);
      uint32_t ov[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = word_of(qv[r], j);
        ov[j] = f32x2_f16x2(__uint_as_float(w << 16) * qs, __uint_as_float(w & 0xFFFF0000u) * qs);
      }
      *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(sm.q) + (h >> 3) * 8192 + c8 * 128 + (h & 7) * 16) =
          make_uint4(ov[0], ov[1], ov[2], ov[3]);
    }
  }
  if (!early) resolve();
  tc::fence_async_smem();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tm = sm.tmem;

  if (mma_warp) {
    // ================= MMA issue (a warp of its own: an MMA issue blocks while the tensor pipe is busy) ====
    constexpr uint32_t kIdS = tc::idesc_f16(128, kHeads, 0, 0, 0);   // K-major A and B
    constexpr uint32_t kIdO = tc::idesc_f16(128, kHeads, 0, 1, 1);   // MN-major A and B
    const uint64_t dk_s = tc::smem_desc(tc::smem_addr(sm.k), 128, 8192);
    const uint64_t dq_s = tc::smem_desc(tc::smem_addr(sm.q), 128, 8192);
    const uint64_t dk_o = tc::smem_desc(tc::smem_addr(sm.k), 8192, 128);
    const uint64_t dp_o = tc::smem_desc(tc::smem_addr(sm.p), 1024, 128);
    const uint32_t leader = tc::elect_lane();
    for (int it = 0; it < n_my; ++it) {
      bool ok = true;
#pragma unroll
      for (int sl = 0; sl < 2; ++sl) {
        ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&sm.k_ready[sl], it & 1, 1u << 22));
        if (!ok) break;
        tc::tc_fence_after();
#pragma unroll
        for (int ks = 16 * sl; ks < 16 * sl + 16; ++ks)   // descriptor addresses advance in 16-byte units
          tc::mma_f16_by(leader, tm + kColS, dk_s + (uint64_t)(ks * 16), dq_s + (uint64_t)(ks * 16), kIdS, ks > 0);
      }
      if (!ok) { *abort = 1; break; }
      tc::mma_commit_by(leader, &sm.bar_s);
      if (!__all_sync(0xffffffffu, tc::mbar_wait(&sm.p_ready, it & 1, 1u << 22))) { *abort = 1; break; }
      tc::tc_fence_after();
      // PV over the chunk's keys only (a short last chunk skips its empty 16-key steps)
      const int ksteps = (min(kChunk, n_mine - kChunk * it) + 15) / 16;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {   // tile by tile: two finished ones free their half of the K tile for the next chunk
#pragma unroll
        for (int kk = 0; kk < kChunk / 16; ++kk)
          if (kk < ksteps)
            tc::mma_f16_by(leader, tm + kColO + 64 * mt, dk_o + (uint64_t)(mt * 128 + kk * 1024), dp_o + (uint64_t)(kk * 128),
                           kIdO, (it > 0 || kk > 0) ? 1u : 0u);
        if (mt & 1) tc::mma_commit_by(leader, &sm.bar_pv[mt >> 1]);
      }
    }
    __syncwarp();
  } else {
    // ================= workers: dequantisation and softmax =================
    unsigned char* ktile = reinterpret_cast<unsigned char*>(sm.k);
    const uint32_t lane_q = (uint32_t)(32 * q4) << 16;
    const int kc = 32 * q4 + lane;   // the softmax thread's key
    float lsum[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) lsum[j] = 0.f;

    for (int it = 0; it < n_my; ++it) {
      const int32_t nxt_src = it + 1 < n_my ? sm.slot[(it + 1) * kChunk + key] : -1;
      bool wok = true;
      // ---- dequantise in two halves of the dims
#define CSA2_HALF(P)                                                                     \
  {                                                                                      \
    if (it > 0) wok = wok && warp_wait(&sm.bar_pv[P], (it - 1) & 1, abort);              \
    /* the four group scales of the thread's 64 dims were loaded by quarter 2 P + qd / 2 of the key */ \
    const uint32_t w0 = __shfl_sync(0xffffffffu, cur_sc.x, (lane & 7) | ((2 * P + (qd >> 1)) << 3)); \
    const uint32_t w1 = __shfl_sync(0xffffffffu, cur_sc.y, (lane & 7) | ((2 * P + (qd >> 1)) << 3)); \
    if (wok) store_half<P, kFp8>(kb, (qd & 1) ? w1 : w0, cur_src, cur_wsc, key, qd, ktile); \
    /* FP8 rows: the second half reuses the registers of the first */                    \
    if (P == 0 && fp8_row_key<kFp8>(cur_src)) load_half<1, kFp8, kTree>(a, cur_src, qd, kb); \
    tc::fence_async_smem();                                                              \
    __syncwarp();                                                                        \
    if (lane == 0) tc::mbar_arrive(&sm.k_ready[P]);                                      \
  }
      CSA2_HALF(0)
      CSA2_HALF(1)
#undef CSA2_HALF
      // the next chunk's bytes, requested together once this chunk's tile is written
      if (it + 1 < n_my) {
        load_half<0, kFp8, kTree>(a, nxt_src, qd, kb);
        if (!fp8_row_key<kFp8>(nxt_src)) {
          load_half<1, kFp8, kTree>(a, nxt_src, qd, kb);
        }
      }
      const bool valid = sm.slot[it * kChunk + kc] != -1;   // the softmax thread's key
      const int fk = sm.kexp[it * kChunk + kc];
      cur_src = nxt_src;
      cur_wsc = load_wscale<kFp8, kTree>(a, nxt_src);
      if (!kFp8) cur_sc = load_scales(a, nxt_src, qd);

      // ---- softmax of the chunk: this thread's key, heads 16*hg .. +15
      wok = wok && warp_wait(&sm.bar_s, it & 1, abort);
      tc::tc_fence_after();
      float x[16];
      bool above = false;
      if (wok) {
        load_scores(tm, hg, lane_q, valid, sm.sl2h, fk, x);
        const float4* thr = reinterpret_cast<const float4*>(&sm.m_thr[16 * hg]);
#pragma unroll
        for (int j4 = 0; j4 < 4; ++j4) {
          const float4 th = thr[j4];
          above |= (x[4 * j4] > th.x) | (x[4 * j4 + 1] > th.y) | (x[4 * j4 + 2] > th.z) | (x[4 * j4 + 3] > th.w);
        }
      }
      // one vote per chunk: did a score outgrow its head's reference, or has a
      // wait failed?  (The flag is read before the vote, so all workers agree.)
      const bool seen_abort = *abort != 0;
      if (workers_or(above || seen_abort)) {
        if (workers_or(seen_abort)) break;
        // reduce the chunk's maxima (x is consumed, then summed again from tensor memory)
        const float mx = reduce16<true>(x, lane);
        if (lane < 16) sm.red[q4][16 * hg + lane] = mx;
        load_scores(tm, hg, lane_q, valid, sm.sl2h, fk, x);
        workers_sync();
        int need = 0;
        if (tid < kHeads) {
          const float mloc = fmaxf(fmaxf(sm.red[0][tid], sm.red[1][tid]), fmaxf(sm.red[2][tid], sm.red[3][tid]));
          const float mo = sm.m_ref[tid];
          float al = 1.f;
          if (mloc > mo + kRescaleLog2 || (mo == -INFINITY && mloc > -INFINITY)) {
            if (mo != -INFINITY) {   // the head holds keys already: rescale them
              al = ex2(mo - mloc);
              need = 1;
            }
            sm.m_ref[tid] = mloc;
            sm.m_thr[tid] = mloc + kRescaleLog2;
            sm.m_exp[tid] = mloc;
          }
          sm.alpha[tid] = al;
        }
        if (workers_or(need)) {
          // O^T *= alpha (per head = column): warp 4*mt + q4 takes M-tile mt, its lane quarter
          const int mt = warp >> 2;
#pragma unroll 1
          for (int c = 0; c < kHeads; c += 16) {
            const uint32_t ta = tm + kColO + 64 * mt + c + lane_q;
            float o[16];
            tc::tmem_ld16(ta, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= sm.alpha[c + j];
            tc::tmem_st16(ta, o);
          }
          tc::tmem_wait_st();
#pragma unroll
          for (int j = 0; j < 16; ++j) lsum[j] *= sm.alpha[16 * hg + j];
        }
      }
      // P = exp2(s - m_ref) in fp16 (the MN-major B operand of the PV product)
      {
        uint32_t pk[8];
        const float pf = pow2i(-fk);   // the normaliser adds p = 2^-f (2^f p)
        const float4* me = reinterpret_cast<const float4*>(&sm.m_exp[16 * hg]);
#pragma unroll
        for (int j4 = 0; j4 < 4; ++j4) {
          const float4 m4 = me[j4];
          const float p0 = ex2(x[4 * j4] - m4.x), p1 = ex2(x[4 * j4 + 1] - m4.y);
          const float p2 = ex2(x[4 * j4 + 2] - m4.z), p3 = ex2(x[4 * j4 + 3] - m4.w);
          lsum[4 * j4] += p0 * pf;
          lsum[4 * j4 + 1] += p1 * pf;
          lsum[4 * j4 + 2] += p2 * pf;
          lsum[4 * j4 + 3] += p3 * pf;
          pk[2 * j4] = f32x2_f16x2(p0, p1);
          pk[2 * j4 + 1] = f32x2_f16x2(p2, p3);
        }
        unsigned char* pdst =
            reinterpret_cast<unsigned char*>(sm.p) + (kc >> 3) * 1024 + (2 * hg) * 128 + (kc & 7) * 16;
        *reinterpret_cast<uint4*>(pdst) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        *reinterpret_cast<uint4*>(pdst + 128) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
      }
      tc::fence_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.p_ready);
    }
    // row sums over the 128 keys: warp, then lane quarters
    const float s = reduce16<false>(lsum, lane);
    if (lane < 16) sm.red[q4][16 * hg + lane] = s;
    // all PV products of the CTA are complete once the last commit has arrived
    if (!*abort && n_my > 0) warp_wait(&sm.bar_pv[1], (n_my - 1) & 1, abort);
    tc::tc_fence_after();
  }
  __syncthreads();
  const bool ok = *abort == 0;
  const bool have_o = ok && n_my > 0;
  if (tid < kHeads) {
    const float l = (sm.red[0][tid] + sm.red[1][tid]) + (sm.red[2][tid] + sm.red[3][tid]);
    sm.l_run[tid] = l;
    if (n_split > 1 && l != l) sm.m_ref[tid] = 0.f;   // (-inf where all logits were NaN: the merge would leave the rank out)
  }
  __syncthreads();
  const int mt = (warp >> 2) & 3;   // epilogue (workers): warp takes M-tile mt, dims 128*mt + 32*q4 + lane

  if (n_split == 1) {
    if (tid < kHeads) sm.fac[tid] = sm.l_run[tid] > 0.f ? 1.f / sm.l_run[tid] : 0.f;
    if (a.lse && tid < kHeads && hb + tid < a.Hq) {
      const float l = sm.l_run[tid];
      a.lse[row * a.Hq + hb + tid] = (sm.m_ref[tid] + log2f(l)) * 0.6931471805599453f;   // (no key: -inf twice)
    }
    __syncthreads();
    if (!mma_warp) {
      for (int c = 0; c < kHeads; c += 16) {
        float o[16];
        if (have_o) {
          tc::tmem_ld16(tm + kColO + 64 * mt + c + ((uint32_t)(32 * q4) << 16), o);
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int h = c + j;
          const float v = have_o ? o[j] * sm.fac[h] : 0.f;
          const int64_t at = (row * a.Hq + hb + h) * kD + 128 * mt + 32 * q4 + lane;
          if (hb + h < a.Hq) {
            if (kTree) a.O16[at] = (uint16_t)(f32x2_bf16x2(v, 0.f) & 0xFFFFu);
            else a.O[at] = v;
          }
        }
      }
    }
  } else {
    // ---- merge the cluster's partials with one exchange.  Every rank publishes its
    // (m, l) and its unscaled partial O in its own shared memory, [head][dim] (a
    // warp's remote reads below are then contiguous); after one cluster barrier
    // rank r sums heads [own(r), own(r+1)) over the ranks in rank order, each rank's
    // partial scaled by 2^(m_q - M) / L.
    const int crank = (int)cluster_rank();
    float* part = reinterpret_cast<float*>(sm.k);   // every MMA that read the K tile is complete
    if (!mma_warp) {
      const int dim = 128 * mt + 32 * q4 + lane;
      for (int c = 0; c < kHeads; c += 16) {
        float o[16];
        if (have_o) {
          tc::tmem_ld16(tm + kColO + 64 * mt + c + ((uint32_t)(32 * q4) << 16), o);
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * kD + dim] = have_o ? o[j] : 0.f;
      }
    }
    cluster_sync();   // every rank's (m, l) and partial O are published
    const int h0 = kHeads * crank / n_split, h1 = kHeads * (crank + 1) / n_split;
    // this rank's heads, 4 dims per element; every rank's value of two elements in flight, the first two while the
    // factors are computed
    const uint32_t pbase = tc::smem_addr(part);
    const int n4 = (h1 - h0) * (kD / 4);
    float4 r[2][kMaxSplit];
    auto request = [&](int e0) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int e = e0 + u * kThreads, at = h0 * (kD / 4) + e;
#pragma unroll
        for (int q = 0; q < kMaxSplit; ++q)
          r[u][q] = q >= n_split || e >= n4 ? make_float4(0.f, 0.f, 0.f, 0.f)
                    : q == crank            ? reinterpret_cast<const float4*>(part)[at]
                                            : ld_cluster4(map_to_rank(pbase + 16u * (uint32_t)at, q));
      }
    };
    request(tid);
    float* facq = reinterpret_cast<float*>(sm.q);    // [rank][head]: the Q tile is no longer read
    if (tid < kHeads) {
      // every rank's (m, l) of this head; the loads are independent (unrolled, predicated)
      const uint32_t am = tc::smem_addr(&sm.m_ref[tid]), al = tc::smem_addr(&sm.l_run[tid]);
      float mq[kMaxSplit], lq[kMaxSplit];
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q) {
        mq[q] = q < n_split ? ld_cluster(map_to_rank(am, q)) : -INFINITY;
        lq[q] = q < n_split ? ld_cluster(map_to_rank(al, q)) : 0.f;
      }
      float M = -INFINITY;
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q) M = fmaxf(M, mq[q]);
      float L = 0.f;
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q)
        if (mq[q] != -INFINITY) L += lq[q] * ex2(mq[q] - M);
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q)
        if (q < n_split) facq[q * kHeads + tid] = (mq[q] == -INFINITY || L <= 0.f) ? 0.f : ex2(mq[q] - M) / L;
      if (crank == 0 && a.lse && hb + tid < a.Hq)
        a.lse[row * a.Hq + hb + tid] = (M + log2f(L)) * 0.6931471805599453f;
    }
    __syncthreads();
    for (int e0 = tid; e0 < n4; e0 += 2 * kThreads) {
      if (e0 != tid) request(e0);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int e = e0 + u * kThreads;
        if (e >= n4) continue;
        const int h = h0 + e / (kD / 4);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < kMaxSplit; ++q) {
          if (q >= n_split) break;
          const float f = facq[q * kHeads + h];
          acc.x += r[u][q].x * f; acc.y += r[u][q].y * f; acc.z += r[u][q].z * f; acc.w += r[u][q].w * f;
        }
        const int64_t at = (row * a.Hq + hb + h) * kD + (e % (kD / 4)) * 4;
        if (hb + h < a.Hq) {
          if (kTree) *reinterpret_cast<uint2*>(a.O16 + at) = make_uint2(f32x2_bf16x2(acc.x, acc.y), f32x2_bf16x2(acc.z, acc.w));
          else *reinterpret_cast<float4*>(a.O + at) = acc;
        }
      }
    }
    cluster_sync();   // no CTA leaves while another still reads its shared memory
  }
  tc::tc_fence_before();
  __syncthreads();
  if (mma_warp) tc::tmem_dealloc(tm, kTmemCols);
  if (tid == 0 && !ok) raise_status(status, CSA2_STATUS_TIMEOUT);
}

}  // namespace

bool sparse_attn_tc_supported(const AttnArgs& a) {
  return a.d == kD && a.Hq >= 1 && a.Hq <= 2 * kHeads && a.K >= 0 && a.W >= 0 &&
         (int64_t)a.K + a.W <= (int64_t)kMaxChunks * kChunk && a.n_pages * kPage < ((int64_t)1 << 31) &&
         (int64_t)a.B * ((int64_t)a.swa_cap + (a.path ? a.Tq : 0)) < ((int64_t)1 << 31) - 2;
}

cudaError_t launch_sparse_attn_tc(const AttnArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.B * a.Tq;
  if (rows == 0) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int max_chunks = (int)((a.K + a.W + kChunk - 1) / kChunk);
  int n_split = 1;
  if (rows < sms && max_chunks > 1)
    n_split = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(max_chunks, kMaxSplit), sms / rows));
  const size_t smem = sizeof(TcSmem);
  auto kernel = a.path ? (a.kv_fp8 ? k_sparse_attn_tc<true, true> : k_sparse_attn_tc<false, true>)
                       : (a.kv_fp8 ? k_sparse_attn_tc<true, false> : k_sparse_attn_tc<false, false>);
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (rows * n_split >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * n_split), (unsigned)((a.Hq + kHeads - 1) / kHeads));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see pdl_trigger / pdl_wait
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)n_split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = n_split > 1 ? 2 : 1;
  return counted(cudaLaunchKernelEx(&cfg, kernel, a, status_word(), n_split));
}

}  // namespace csa2
