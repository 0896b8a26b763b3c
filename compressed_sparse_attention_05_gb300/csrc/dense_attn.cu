// Attention over every visible entry of the compressed cache (reading R14) and
// the entries' attention weights (reading R15), plain form: fp32 arithmetic on
// the CUDA cores, one softmax pass with a running maximum and sum.  These
// kernels take d = 64 (the tiny model); d = 512 runs on the tensor cores
// (dense_attn_tc.cu).
//
//   l_rj = cap tanh(tau q_r . k_j / cap) - slope_h |t_r - p_j|
//   O_r  = sum_j exp(l_rj - m) k_j / sum_j exp(l_rj - m),  lse_r = m + log(sum)
//   w_j  = decay w_j + sum_r exp(l_rj - lse_r)
//
// A tile of 32 keys is dequantised once into shared memory (rows padded by one
// float: lane = key reads a column of rows without bank conflicts).  A warp owns
// one head; lane k computes the dot product of key k, and the 32 weights are then
// broadcast one by one while every lane adds its d/32 channels.
#include "dense.cuh"
#include "operands.cuh"

namespace csa2 {
namespace {

constexpr int kTile = 32;
constexpr int kWarps = 8;
constexpr int D = 64, kLd = D + 1;   // tile row, padded
constexpr size_t kSmem = ((size_t)kTile * kLd + (size_t)kWarps * D) * sizeof(float);

// An E4M3 code, its NaN included.
__device__ __forceinline__ float fp8_to_f32(uint8_t c) { return (c & 0x7F) == 0x7F ? NAN : e4m3_to_f32(c); }
__device__ __forceinline__ float e2m1_to_f32(uint32_t c) { return bf16_bits_to_f32(e2m1_to_bf16_bits(c)); }

// |t - p| in fp32 (exact below 2^24)
__device__ __forceinline__ float dense_distance(int t, int64_t p) {
  const int64_t d = (int64_t)t - p;
  return (float)(d < 0 ? -d : d);
}
__device__ __forceinline__ float dense_logit(const DenseArgs& a, float dot, float slope, float dist) {
  float l = dot * a.scale;
  if (a.cap > 0.f) l = a.cap * tanhf(l / a.cap);
  return l - slope * dist;
}

// Dequantises entries e0 .. e0+31 of sequence b into the tile; pos[k] receives the
// raw position of each entry's last token, or INT64_MIN for none (a bad page too).
__device__ void load_entries(const DenseArgs& a, int b, int e0, int n_ent, int64_t shift, float* tile,
                             int64_t* pos, int64_t* slots, uint32_t* status) {
  const int tid = threadIdx.x;
  if (tid < kTile) {
    const int j = e0 + tid;
    int64_t slot = -1;
    if (j < n_ent) slot = entry_slot(a.page_table, a.max_pages, a.n_pages, b, j, status);
    slots[tid] = slot;
    pos[tid] = slot < 0 ? INT64_MIN : a.entry_pos ? (int64_t)a.entry_pos[slot] : 4 * ((int64_t)j + shift) + 3;
  }
  __syncthreads();
  constexpr int per = D / 2;   // code bytes of an entry
  for (int u = tid; u < kTile * per; u += blockDim.x) {
    const int k = u / per, c = u % per;
    const int64_t slot = slots[k];
    float x0 = 0.f, x1 = 0.f;
    if (slot >= 0) {
      const uint32_t byte = a.kv_codes[slot * per + c];
      const float s = fp8_to_f32(a.kv_scales[slot * (D / 16) + c / 8]);
      x0 = e2m1_to_f32(byte & 15u) * s;
      x1 = e2m1_to_f32(byte >> 4) * s;
    }
    tile[k * kLd + 2 * c] = x0;
    tile[k * kLd + 2 * c + 1] = x1;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kWarps * 32) k_dense_attn_plain(DenseArgs a, uint32_t* status) {
  constexpr int kPer = D / 32;
  extern __shared__ float smem[];
  float* tile = smem;                       // [32][D + 1]
  float* qs = tile + kTile * kLd;           // [8][D]
  __shared__ int64_t pos[kTile], slots[kTile];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const int b = (int)(row / a.Tq), i = (int)(row % a.Tq);
  const int h = (int)blockIdx.y * kWarps + warp;
  const bool live = h < a.Hq;
  const int n_ent = dense_entries(a, b);
  if (threadIdx.x == 0 && dense_count_bad(a, b)) raise_status(status, CSA2_STATUS_BAD_COUNT);
  const int64_t shift = dense_shift(a, b);
  const int pos0 = a.swa_cap > 0 ? a.swa_pos0[b] : 0;
  const DenseRow r = dense_row(a, b, i, n_ent, shift, pos0);
  float q[kPer], o[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    q[c] = live ? bf16_bits_to_f32(a.Q[(row * a.Hq + h) * D + 32 * c + lane]) : 0.f;
    qs[warp * D + 32 * c + lane] = q[c];
    o[c] = 0.f;
  }
  const float slope = (a.slopes && live) ? a.slopes[h] : 0.f;
  float m = -INFINITY, l = 0.f;
  // one tile: lane = key
  auto attend = [&](bool seen, float dist) {
    float dot = 0.f;
    for (int c = 0; c < D; ++c) dot += qs[warp * D + c] * tile[lane * kLd + c];
    if (!__any_sync(0xffffffffu, seen)) return;
    const float x = seen ? dense_logit(a, dot, slope, dist) : -INFINITY;
    const float mn = fmaxf(m, warp_max(x));             // -inf if all that was seen so far is NaN
    const float al = m == -INFINITY ? 0.f : expf(m - mn);
    const float p = seen ? expf(x - (mn == -INFINITY ? 0.f : mn)) : 0.f;
    m = mn;
    l = l * al + warp_sum(p);
#pragma unroll
    for (int c = 0; c < kPer; ++c) o[c] *= al;
    for (int k = 0; k < kTile; ++k) {
      const float pk = __shfl_sync(0xffffffffu, p, k);
      if (pk == 0.f) continue;   // uniform; a hidden key may hold NaN
#pragma unroll
      for (int c = 0; c < kPer; ++c) o[c] += pk * tile[k * kLd + 32 * c + lane];
    }
  };
  // Window rows (R5's operand: bf16 of code times scale).  The conversion instruction keeps a NaN; rounding
  // the bits as integers turns the one that arithmetic makes, 0x7FFFFFFF, into -0.
  for (int w0 = 0; w0 < r.w_n; w0 += kTile) {
    __syncthreads();
    for (int u = threadIdx.x; u < kTile * D; u += blockDim.x) {
      const int k = u / D, c = u % D;
      float x = 0.f;
      if (w0 + k < r.w_n) {
        const int64_t wr = (int64_t)b * a.swa_cap + ((int64_t)r.w_lo + w0 + k - pos0);
        x = __uint_as_float(f32x2_bf16x2(fp8_to_f32(a.swa_codes[wr * D + c]) * a.swa_scales[wr], 0.f) << 16);
      }
      tile[k * kLd + c] = x;
    }
    __syncthreads();
    attend(w0 + lane < r.w_n, dense_distance(r.t, (int64_t)r.w_lo + w0 + lane));
  }
  for (int e0 = dense_first(a, r.doc, shift) / kTile * kTile; e0 < r.nv; e0 += kTile) {
    __syncthreads();
    load_entries(a, b, e0, n_ent, shift, tile, pos, slots, status);
    const int64_t p = pos[lane];
    attend(e0 + lane < r.nv && p != INT64_MIN && p <= r.last && p - 3 >= r.doc, dense_distance(r.t, p));
  }
  if (!live) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int c = 0; c < kPer; ++c)
    a.O[(row * a.Hq + h) * D + 32 * c + lane] = (uint16_t)(f32x2_bf16x2(o[c] * inv, 0.f) & 0xFFFFu);
  if (a.lse && lane == 0) a.lse[row * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

// One CTA per 32 entries of a sequence; its warps share out the (token, head) rows
// and their sums are added in warp order.
__global__ void __launch_bounds__(kWarps * 32) k_entry_weights_plain(DenseArgs a, uint32_t* status) {
  extern __shared__ float smem[];
  float* tile = smem;
  float* qs = tile + kTile * kLd;
  __shared__ int64_t pos[kTile], slots[kTile];
  __shared__ float part[kWarps][kTile];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = (int)blockIdx.y;
  const int n_ent = dense_entries(a, b);
  if (threadIdx.x == 0 && blockIdx.x == 0 && dense_count_bad(a, b)) raise_status(status, CSA2_STATUS_BAD_COUNT);
  const int64_t shift = dense_shift(a, b);
  for (int64_t e0 = (int64_t)blockIdx.x * kTile; e0 < n_ent; e0 += (int64_t)gridDim.x * kTile) {
    __syncthreads();
    load_entries(a, b, (int)e0, n_ent, shift, tile, pos, slots, status);
    const int64_t p = pos[lane];
    float w = 0.f;
    for (int i = 0; i < a.Tq; ++i) {
      const DenseRow r = dense_row(a, b, i, n_ent, shift, 0);
      const bool seen = e0 + lane < r.nv && p != INT64_MIN && p <= r.last && p - 3 >= r.doc;
      for (int h = warp; h < a.Hq; h += kWarps) {
        const int64_t row = ((int64_t)b * a.Tq + i) * a.Hq + h;
        __syncwarp();
        for (int c = lane; c < D; c += 32) qs[warp * D + c] = bf16_bits_to_f32(a.Q[row * D + c]);
        __syncwarp();
        const float lse = a.lse_in[row];
        if (isinf(lse)) continue;   // a row that saw nothing
        float dot = 0.f;
        for (int c = 0; c < D; ++c) dot += qs[warp * D + c] * tile[lane * kLd + c];
        if (seen) w += expf(dense_logit(a, dot, a.slopes ? a.slopes[h] : 0.f, dense_distance(r.t, p)) - lse);
      }
    }
    part[warp][lane] = w;
    __syncthreads();
    if (warp == 0 && slots[lane] >= 0) {
      float s = 0.f;
      for (int k = 0; k < kWarps; ++k) s += part[k][lane];
      a.weight_out[slots[lane]] = (a.weight_in ? a.decay * a.weight_in[slots[lane]] : 0.f) + s;
    }
  }
}

}  // namespace

cudaError_t launch_dense_attn_plain(const DenseArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.B * a.Tq;
  if (rows == 0) return cudaSuccess;
  if (rows >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)rows, (unsigned)((a.Hq + kWarps - 1) / kWarps));
  return launch_step(k_dense_attn_plain, grid, dim3(kWarps * 32), kSmem, s, a, status_word());
}

cudaError_t launch_entry_weights_plain(const DenseArgs& a, cudaStream_t s) {
  if (a.B == 0 || a.max_entries == 0) return cudaSuccess;
  const dim3 grid((unsigned)((a.max_entries + kTile - 1) / kTile), (unsigned)a.B);
  return launch_step(k_entry_weights_plain, grid, dim3(kWarps * 32), kSmem, s, a, status_word());
}

}  // namespace csa2
