// Eviction from the compressed cache by accumulated attention weight (reading R16).
//
// Of a sequence's n entries the `keep` best stay: the first n_sink and the newest
// n_recent always, then by weight (equal weights -> lower index).  Nothing that can
// stay moves: the survivors at indices >= keep go, in order, into the holes that
// the evicted entries leave below keep, so the bytes moved are those of
// min(evicted below keep, survivors above keep) entries, not of the whole cache
// (a cache of 4,160 entries cut to 4,096 moves at most 64 rows of 552 B).
// Sources (>= keep) and destinations (< keep) are disjoint, so the moves need no
// order and no staging.
//
// k_evict_select: a cluster of up to 8 CTAs per sequence.  Every CTA holds its
// share of the order-preserving weight keys in shared memory (one read of the
// weights); three radix passes (11, 11, 10 bits) over cluster-wide histograms
// (distributed shared memory) find the keep-th largest key and how many of its
// equals stay; a prefix count over the cluster then numbers holes and movers in
// index order.  k_evict_move copies the rows, one warp per row, over all SMs.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace csa2 {
namespace {

constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxCached = 48 * 1024;    // keys of one CTA held in shared memory (192 KB)
constexpr int kMinPerCta = 2048;         // entries that make another CTA of the cluster worth its barriers

// Order-preserving key of a weight (larger key = larger weight; zeros are equal;
// a NaN with the sign bit clear counts as the largest), below the key of an entry
// that always stays.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  const uint32_t k = u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return min(k, 0xFFFFFFFEu);
}

__device__ __forceinline__ uint32_t cl_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cl_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cl_load(const uint32_t* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

struct EvictWs {
  int32_t* n_moves;   // [B]
  int32_t* holes;     // [B][cap]
  int32_t* movers;    // [B][cap]
  int64_t cap;
};

// Sum over the block of v, and the exclusive prefix of this thread (thread order).
__device__ __forceinline__ uint64_t block_prefix(uint64_t v, uint64_t* warp_sums, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  uint64_t before = 0, all = 0;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) {
    const uint64_t s = warp_sums[k];
    if (k < warp) before += s;
    all += s;
  }
  *total = all;
  return before + inc - v;
}

__global__ void __launch_bounds__(kThreads) k_evict_select(EvictArgs a, EvictWs ws, int n_cl, int cached,
                                                           uint32_t* status) {
  extern __shared__ uint32_t keys[];     // [cached] this CTA's keys (when its share fits)
  __shared__ uint32_t hist[kBins];
  __shared__ uint64_t warp_sums[kThreads / 32];
  __shared__ uint32_t pub[4];            // read by the cluster's other CTAs
  __shared__ uint32_t found[2];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int b = (int)blockIdx.x / n_cl;
  const int rank = n_cl > 1 ? (int)cl_rank() : 0;
  const int n = a.n_entries[b];
  const int64_t room = min((int64_t)a.max_entries, (int64_t)a.max_pages * kPage);
  const int64_t shift = a.shift[b];
  const bool bad = n < 0 || n > room || shift < 0;
  if (bad || n <= a.keep) {              // the same in every CTA of the cluster
    if (rank == 0 && tid == 0) {
      ws.n_moves[b] = 0;
      if (bad) raise_status(status, CSA2_STATUS_BAD_COUNT);
    }
    return;
  }
  // this CTA's entries [lo, hi), each thread's run of them [t0, t1)
  const int lo = (int)((int64_t)n * rank / n_cl), hi = (int)((int64_t)n * (rank + 1) / n_cl);
  const bool in_smem = hi - lo <= cached;
  const int64_t first_recent = 4 * ((int64_t)n + shift - a.n_recent) + 3;
  auto fetch = [&](int j, bool report) -> uint32_t {
    const int64_t slot = entry_slot(a.page_table, a.max_pages, a.n_pages, b, j, report ? status : nullptr);
    if (slot < 0) return 0u;
    const int64_t p = a.entry_pos[slot];
    return (p < 4ll * a.n_sink || p >= first_recent) ? 0xFFFFFFFFu : weight_key(a.weight[slot]);
  };
  if (in_smem) {
    for (int j = lo + tid; j < hi; j += kThreads) keys[j - lo] = fetch(j, true);
  }
  auto key_of = [&](int j) -> uint32_t { return in_smem ? keys[j - lo] : fetch(j, false); };

  // ---- the keep-th largest key, digit by digit from the top
  uint32_t prefix = 0, mask = 0;
  uint32_t need = (uint32_t)a.keep;      // entries still to be taken among those that match the prefix
  const int shifts[3] = {21, 10, 0}, widths[3] = {11, 11, 10};
  for (int pass = 0; pass < 3; ++pass) {
    const int sh = shifts[pass], nb = 1 << widths[pass];
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    for (int j = lo + tid; j < hi; j += kThreads) {
      const uint32_t k = key_of(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> sh) & (nb - 1)], 1u);
    }
    __syncthreads();
    if (n_cl > 1) cl_sync();
    // bins from the top: thread t holds bins nb-1-4t .. nb-4-4t
    uint32_t c[4] = {0, 0, 0, 0};
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int bin = nb - 1 - (4 * tid + i);
      if (bin >= 0) {
        if (n_cl > 1)
          for (int q = 0; q < n_cl; ++q) c[i] += cl_load(&hist[bin], q);
        else
          c[i] = hist[bin];
      }
      mine += c[i];
    }
    uint64_t total;
    const uint64_t before = block_prefix(mine, warp_sums, &total);
    if (before < need && before + mine >= need) {
      uint32_t above = (uint32_t)before;
      for (int i = 0; i < 4; ++i) {
        if (above + c[i] >= need) {
          found[0] = (uint32_t)(nb - 1 - (4 * tid + i));
          found[1] = need - above;
          break;
        }
        above += c[i];
      }
    }
    if (n_cl > 1) cl_sync(); else __syncthreads();   // also: every rank has read this pass's histograms
    prefix |= found[0] << sh;
    mask |= (uint32_t)(nb - 1) << sh;
    need = found[1];
    __syncthreads();
  }
  const uint32_t thr = prefix;           // keys above stay; of its equals the `need` lowest indices

  // ---- equals before each thread's run, over the cluster
  const int run = (hi - lo + kThreads - 1) / kThreads;
  const int t0 = min(hi, lo + tid * run), t1 = min(hi, t0 + run);
  uint32_t eq = 0;
  for (int j = t0; j < t1; ++j) eq += key_of(j) == thr;
  uint64_t total;
  uint32_t eq_before = (uint32_t)block_prefix(eq, warp_sums, &total);
  if (tid == 0) pub[0] = (uint32_t)total;
  if (n_cl > 1) {
    cl_sync();
    for (int q = 0; q < rank; ++q) eq_before += cl_load(&pub[0], q);
  }
  // ---- holes (evicted, below keep) and movers (kept, at or above keep)
  uint32_t holes = 0, movers = 0, e = eq_before;
  for (int j = t0; j < t1; ++j) {
    const uint32_t k = key_of(j);
    const bool kept = k > thr || (k == thr && e < need);
    e += k == thr;
    holes += !kept && j < a.keep;
    movers += kept && j >= a.keep;
  }
  uint64_t both = block_prefix(((uint64_t)holes << 32) | movers, warp_sums, &total);
  if (tid == 0) {
    pub[1] = (uint32_t)(total >> 32);
    pub[2] = (uint32_t)total;
  }
  uint32_t h = (uint32_t)(both >> 32), m = (uint32_t)both, all_holes = (uint32_t)(total >> 32);
  if (n_cl > 1) {
    cl_sync();
    all_holes = 0;
    for (int q = 0; q < n_cl; ++q) {
      const uint32_t hq = cl_load(&pub[1], q), mq = cl_load(&pub[2], q);
      if (q < rank) {
        h += hq;
        m += mq;
      }
      all_holes += hq;
    }
  }
  e = eq_before;
  int32_t* hl = ws.holes + (int64_t)b * ws.cap;
  int32_t* ml = ws.movers + (int64_t)b * ws.cap;
  for (int j = t0; j < t1; ++j) {
    const uint32_t k = key_of(j);
    const bool kept = k > thr || (k == thr && e < need);
    e += k == thr;
    if (!kept && j < a.keep) hl[h++] = j;
    if (kept && j >= a.keep) ml[m++] = j;
  }
  if (n_cl > 1) cl_sync();               // no CTA leaves while another still reads its shared memory,
  if (rank == 0 && tid == 0) {           // and every CTA has read the count before it changes
    ws.n_moves[b] = (int32_t)all_holes;
    a.n_entries[b] = a.keep;
    a.shift[b] = (int32_t)(shift + n - a.keep);
  }
}

// Copies `bytes` (a multiple of 4) of a row with a warp, 16 bytes at a time where both
// rows start on 16 bytes.
__device__ __forceinline__ void copy_row(uint8_t* base, int64_t to, int64_t from, int bytes, int lane) {
  if (bytes % 16 == 0) {
    const uint4* s = reinterpret_cast<const uint4*>(base + from * bytes);
    uint4* d = reinterpret_cast<uint4*>(base + to * bytes);
    for (int i = lane; i < bytes / 16; i += 32) d[i] = s[i];
  } else {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(base + from * bytes);
    uint32_t* d = reinterpret_cast<uint32_t*>(base + to * bytes);
    for (int i = lane; i < bytes / 4; i += 32) d[i] = s[i];
  }
}

__global__ void __launch_bounds__(256) k_evict_move(EvictArgs a, EvictWs ws, uint32_t* status) {
  pdl_trigger();
  pdl_wait();
  const int b = (int)blockIdx.y, lane = threadIdx.x & 31;
  const int n = ws.n_moves[b];
  for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += gridDim.x * 8) {
    const int to = ws.holes[(int64_t)b * ws.cap + i], from = ws.movers[(int64_t)b * ws.cap + i];
    const int64_t d = entry_slot(a.page_table, a.max_pages, a.n_pages, b, to, status);
    const int64_t s = entry_slot(a.page_table, a.max_pages, a.n_pages, b, from, status);
    if (d < 0 || s < 0) continue;
    copy_row(a.kv_codes, d, s, a.code_bytes, lane);
    copy_row(a.kv_scales, d, s, a.scale_bytes, lane);
    if (a.idx_k) copy_row(a.idx_k, d, s, a.idx_bytes, lane);
    if (lane == 0) {
      a.weight[d] = a.weight[s];
      a.entry_pos[d] = a.entry_pos[s];
    }
  }
}

int64_t list_cap(int max_entries) { return ((int64_t)max_entries + 3) / 4 * 4; }

}  // namespace

size_t evict_workspace_bytes(int B, int max_entries) {
  if (B <= 0 || max_entries <= 0) return 0;
  return (((size_t)B + 63) / 64 * 64 + 2 * (size_t)B * (size_t)list_cap(max_entries)) * sizeof(int32_t);
}

cudaError_t launch_evict(const EvictArgs& a, void* wsp, cudaStream_t s) {
  if (a.B == 0 || a.max_entries <= a.keep) return cudaSuccess;
  EvictWs ws;
  ws.cap = list_cap(a.max_entries);
  ws.n_moves = static_cast<int32_t*>(wsp);
  ws.holes = ws.n_moves + ((size_t)a.B + 63) / 64 * 64;
  ws.movers = ws.holes + (int64_t)a.B * ws.cap;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int n_cl = std::max(1, std::min(kMaxCluster, (a.max_entries + kMinPerCta - 1) / kMinPerCta));
  const int cached = std::min(kMaxCached, (a.max_entries + n_cl - 1) / n_cl + 1);
  const size_t smem = (size_t)cached * sizeof(uint32_t);
  e = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)(kMaxCached * sizeof(uint32_t)));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * n_cl));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)n_cl;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = n_cl > 1 ? 2 : 1;
  e = counted(cudaLaunchKernelEx(&cfg, k_evict_select, a, ws, n_cl, cached, status_word()));
  if (e != cudaSuccess) return e;
  const int64_t most = std::min<int64_t>(a.keep, (int64_t)a.max_entries - a.keep);
  const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>((most + 7) / 8, ((int64_t)sms * 8 + a.B - 1) / a.B));
  return launch_step(k_evict_move, dim3((unsigned)blocks, (unsigned)a.B), dim3(256), 0, s, a, ws, status_word());
}

}  // namespace csa2
