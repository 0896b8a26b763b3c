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
// weights; a share that does not fit lies in the workspace); three radix passes
// (11, 11, 10 bits), each over its own cluster-wide histogram (distributed shared
// memory), find the keep-th largest key and how many of its equals stay; counts
// by ballots, in index order, number holes and movers over the cluster.  A call on
// a cache of a few thousand entries is a chain of dependent trips (page, weight,
// five cluster barriers, lists, pages again, rows), so every step has all its
// loads in flight at once.  k_evict_move copies the rows, one warp per row and
// four rows of a warp in flight, over all SMs.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace csa2 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxCached = 48 * 1024;    // keys of one CTA held in shared memory (192 KB beside 24 KB of histograms)
constexpr uint32_t kNone = 0xFFFFFFFFu;    // no such entry (a pool of 2^32 entries would be 1 TB of codes)
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
  uint32_t* keys;     // [B][cap], or null while every share fits in shared memory
  int64_t cap;
};

__device__ __forceinline__ uint32_t warp_inclusive(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}
// v0 and v1 of each warp (uniform): the sums over the warps before it, and over all.
__device__ __forceinline__ void warps_prefix(uint32_t v0, uint32_t v1, uint32_t (*sums)[2], uint32_t (&before)[2],
                                             uint32_t (&all)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane < 2) sums[warp][lane] = lane ? v1 : v0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t inc = warp_inclusive(sums[lane][k], lane);
    all[k] = __shfl_sync(0xffffffffu, inc, 31);
    before[k] = __shfl_sync(0xffffffffu, inc, max(warp - 1, 0));
    if (warp == 0) before[k] = 0;
  }
}
static_assert(kWarps == 32, "a warp scans the warps' sums");

__global__ void __launch_bounds__(kThreads) k_evict_select(EvictArgs a, EvictWs ws, int n_cl, int cached,
                                                           uint32_t* status) {
  extern __shared__ uint32_t smem_keys[];   // [cached] this CTA's keys (when its share fits)
  __shared__ uint32_t hist[3][kBins];    // read by the cluster's other CTAs, as are pub
  __shared__ uint32_t group[3][kWarps];  // sums of 64 bins
  __shared__ uint32_t sums[kWarps][2];
  __shared__ uint32_t pub[3];
  __shared__ uint32_t found[3];
  __shared__ uint32_t no_page;           // an entry of this CTA's share lies behind a bad page (read by rank 0)
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 3 * kBins; i += kThreads) hist[0][i] = 0;
  if (tid == 0) no_page = 0;
  pdl_wait();
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
  // this CTA's entries [lo, lo + count)
  const int lo = (int)((int64_t)n * rank / n_cl), count = (int)((int64_t)n * (rank + 1) / n_cl) - lo;
  uint32_t* keys = count <= cached ? smem_keys : ws.keys + (int64_t)b * ws.cap + lo;
  const int64_t first_recent = 4 * ((int64_t)n + shift - a.n_recent) + 3;
  __syncthreads();
  // ---- keys, eight loads of each kind in flight, and the first digit's histogram
  constexpr int kAhead = 8;

  for (int j0 = tid; j0 < count; j0 += kAhead * kThreads) {
    uint32_t slot[kAhead];
    int pos[kAhead];
    float w[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = j0 + i * kThreads;
      slot[i] = j < count ? (uint32_t)entry_slot(a.page_table, a.max_pages, a.n_pages, b, lo + j, status) : kNone;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      pos[i] = slot[i] != kNone ? a.entry_pos[slot[i]] : 0;
      w[i] = slot[i] != kNone ? a.weight[slot[i]] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = j0 + i * kThreads;
      if (j >= count) break;
      if (slot[i] == kNone) no_page = 1;
      const uint32_t k = slot[i] == kNone ? 0u
                         : pos[i] < 4ll * a.n_sink || pos[i] >= first_recent ? 0xFFFFFFFFu
                                                                              : weight_key(w[i]);
      keys[j] = k;
      atomicAdd(&hist[0][k >> 21], 1u);
    }
  }

  // ---- the keep-th largest key, digit by digit from the top
  uint32_t prefix = 0, mask = 0;
  uint32_t need = (uint32_t)a.keep;      // entries still to be taken among those that match the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int sh = pass == 0 ? 21 : pass == 1 ? 10 : 0, nb = pass == 2 ? 1024 : 2048;
    if (pass > 0)
      for (int j = tid; j < count; j += kThreads) {
        const uint32_t k = keys[j];
        if ((k & mask) == prefix) atomicAdd(&hist[pass][(k >> sh) & (nb - 1)], 1u);
      }
    __syncthreads();
    // The keep-th key's bin in two looks: first the sums of 64 bins (warp w: bins 64 w ..), over the
    // cluster, then the 64 bins of the one group; a look is one round of remote loads, all in flight.
    // (Every CTA reading all 2,048 bins of all eight took 3.5 us a pass.)
    const uint32_t g = __reduce_add_sync(0xffffffffu, hist[pass][64 * warp + lane] + hist[pass][64 * warp + 32 + lane]);
    if (lane == 0) group[pass][warp] = g;
    if (n_cl > 1) cl_sync(); else __syncthreads();
    if (warp == 0) {
      auto over_cluster = [&](const uint32_t* p) {
        if (n_cl == 1) return *p;
        uint32_t v[kMaxCluster], sum = 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) v[q] = q < n_cl ? cl_load(p, q) : 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) sum += v[q];
        return sum;
      };
      // lane l: the l-th group from the top, then its l-th pair of bins from the top
      uint32_t c = over_cluster(&group[pass][31 - lane]);
      uint32_t inc = warp_inclusive(c, lane);
      const int gl = __ffs(__ballot_sync(0xffffffffu, inc >= need)) - 1;
      uint32_t left = need - (__shfl_sync(0xffffffffu, inc, gl) - __shfl_sync(0xffffffffu, c, gl));
      const int top = 64 * (31 - gl) + 63 - 2 * lane;
      const uint32_t c0 = over_cluster(&hist[pass][top]), c1 = over_cluster(&hist[pass][top - 1]);
      c = c0 + c1;
      inc = warp_inclusive(c, lane);
      const int bl = __ffs(__ballot_sync(0xffffffffu, inc >= left)) - 1;
      if (lane == bl) {
        left -= inc - c;
        const bool second = left > c0;
        found[0] = (uint32_t)(top - second);
        found[1] = left - (second ? c0 : 0);
        found[2] = second ? c1 : c0;
      }
    }
    __syncthreads();
    prefix |= found[0] << sh;
    mask |= (uint32_t)(nb - 1) << sh;
    need = found[1];
  }
  const uint32_t thr = prefix;           // keys above stay; of its equals the `need` lowest indices
  const bool all_equals = found[2] == need;

  // ---- each warp a run of the share, 32 entries at a time, in index order
  const int run = (count + kThreads - 1) / kThreads * 32;
  const int w0 = min(count, warp * run), w1 = min(count, w0 + run);
  uint32_t eq_before = 0;                // equals at lower indices than the warp's run
  uint32_t before[2], all[2];
  // Lane q: rank q's published number; the sums over the ranks before this one, and over all.
  auto ranks_prefix = [&](const uint32_t* p, uint32_t* sum) -> uint32_t {
    const uint32_t v = lane < n_cl ? cl_load(p, lane) : 0;
    *sum = __reduce_add_sync(0xffffffffu, v);
    return __reduce_add_sync(0xffffffffu, lane < rank ? v : 0);
  };
  if (!all_equals) {
    uint32_t eq = 0, sum;
    for (int j0 = w0; j0 < w1; j0 += 32) eq += __popc(__ballot_sync(0xffffffffu, j0 + lane < w1 && keys[j0 + lane] == thr));
    warps_prefix(eq, 0, sums, before, all);
    eq_before = before[0];
    if (n_cl > 1) {
      if (tid == 0) pub[0] = all[0];
      cl_sync();
      eq_before += ranks_prefix(&pub[0], &sum);
    }
  }
  // Lane's entry j0 + lane of the run: whether it stays; e counts the equals so far.
  const uint32_t below = (1u << lane) - 1;
  auto stays = [&](int j0, uint32_t& e) -> bool {
    const bool in = j0 + lane < w1;
    const uint32_t k = in ? keys[j0 + lane] : 0;
    if (all_equals) return in && k >= thr;
    const uint32_t m = __ballot_sync(0xffffffffu, in && k == thr);
    const bool kept = in && (k > thr || (k == thr && e + __popc(m & below) < need));
    e += __popc(m);
    return kept;
  };
  // ---- holes (evicted, below keep) and movers (kept, at or above keep)
  uint32_t holes = 0, movers = 0, e = eq_before;
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const bool kept = stays(j0, e);
    const int j = lo + j0 + lane;
    holes += __popc(__ballot_sync(0xffffffffu, !kept && j0 + lane < w1 && j < a.keep));
    movers += __popc(__ballot_sync(0xffffffffu, kept && j >= a.keep));
  }
  warps_prefix(holes, movers, sums, before, all);
  uint32_t h = before[0], m = before[1], all_holes = all[0];
  bool lost = no_page != 0;
  if (n_cl > 1) {
    if (tid == 0) {
      pub[1] = all[0];
      pub[2] = all[1];
    }
    cl_sync();
    uint32_t sum;
    h += ranks_prefix(&pub[1], &all_holes);
    m += ranks_prefix(&pub[2], &sum);
    if (rank == 0 && warp == 0) lost = __any_sync(0xffffffffu, lane < n_cl && cl_load(&no_page, lane) != 0);
    // no CTA leaves while another still reads its shared memory, and every CTA has read the count
    // before it changes (waited for at the end)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  e = eq_before;
  int32_t* hl = ws.holes + (int64_t)b * ws.cap;
  int32_t* ml = ws.movers + (int64_t)b * ws.cap;
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const bool kept = stays(j0, e);
    const int j = lo + j0 + lane;
    const bool hole = !kept && j0 + lane < w1 && j < a.keep, mover = kept && j >= a.keep;
    const uint32_t hm = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
    if (hole) hl[h + __popc(hm & below)] = j;
    if (mover) ml[m + __popc(mm & below)] = j;
    h += __popc(hm);
    m += __popc(mm);
  }
  if (n_cl > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  else __syncthreads();
  if (rank == 0 && tid == 0) {
    // a survivor cannot move to a hole without a page: a sequence with a bad one stays as it is
    ws.n_moves[b] = lost ? 0 : (int32_t)all_holes;
    if (!lost) {
      a.n_entries[b] = a.keep;
      a.shift[b] = (int32_t)(shift + n - a.keep);
    }
  }
}

// A row's bytes as a lane sees them: 16-byte pieces of the arrays whose rows are a multiple of 16
// bytes, 4-byte words of the others (4 bytes of scales) and of the weight and position.  The
// largest rows have 512 bytes of codes and 512 of keys: two pieces and one word for a lane.
struct Field {
  uint8_t* base;       // the piece of row 0 (null: none)
  uint32_t bytes;      // row stride
};
__device__ __forceinline__ Field piece16(const EvictArgs& a, int i) {
  const int nc = a.code_bytes / 16, ni = a.idx_k ? a.idx_bytes / 16 : 0, ns = a.scale_bytes / 16;
  if (i < nc) return {a.kv_codes + 16 * i, (uint32_t)a.code_bytes};
  i -= nc;
  if (i < ni) return {a.idx_k + 16 * i, (uint32_t)a.idx_bytes};
  i -= ni;
  if (i < ns) return {a.kv_scales + 16 * i, (uint32_t)a.scale_bytes};
  return {nullptr, 0};
}
__device__ __forceinline__ Field piece4(const EvictArgs& a, int i) {
  if (i == 0) return {reinterpret_cast<uint8_t*>(a.weight), 4};
  if (i == 1) return {reinterpret_cast<uint8_t*>(a.entry_pos), 4};
  if (i == 2 && a.scale_bytes == 4) return {a.kv_scales, 4};
  return {nullptr, 0};
}

constexpr int kRowsAhead = 4, kMoveBlocks = 4;   // rows of a warp in flight; blocks of an SM
__global__ void __launch_bounds__(256, kMoveBlocks) k_evict_move(EvictArgs a, EvictWs ws, uint32_t* status) {
  pdl_trigger();
  const int b = (int)blockIdx.y, lane = threadIdx.x & 31;
  const int warps = gridDim.x * 8, w = blockIdx.x * 8 + (threadIdx.x >> 5);
  const Field f0 = piece16(a, lane), f1 = piece16(a, lane + 32), g0 = piece4(a, lane);
  pdl_wait();
  const int n = ws.n_moves[b];
  // 32 of the warp's rows (w, w + warps, ...) at a time: lane l looks up row l of them
  for (int i0 = 0; (int64_t)i0 * warps + w < n; i0 += 32) {
    const int64_t at = (int64_t)(i0 + lane) * warps + w;
    uint32_t d = kNone, s = kNone;
    if (at < n) {
      d = (uint32_t)entry_slot(a.page_table, a.max_pages, a.n_pages, b, ws.holes[(int64_t)b * ws.cap + at], status);
      s = (uint32_t)entry_slot(a.page_table, a.max_pages, a.n_pages, b, ws.movers[(int64_t)b * ws.cap + at], status);
      if (s == kNone) d = kNone;
    }
    const int here = (int)min((int64_t)32, (n - w + (int64_t)warps - 1) / warps - i0);
    for (int r = 0; r < here; r += kRowsAhead) {
      uint32_t to[kRowsAhead], from[kRowsAhead];
      uint4 v0[kRowsAhead], v1[kRowsAhead];
      uint32_t v2[kRowsAhead];
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) {
        to[k] = __shfl_sync(0xffffffffu, d, r + k);
        from[k] = __shfl_sync(0xffffffffu, s, r + k);
        if (r + k >= here) to[k] = kNone;
        if (to[k] == kNone) continue;
        if (f0.base) v0[k] = *reinterpret_cast<const uint4*>(f0.base + (size_t)from[k] * f0.bytes);
        if (f1.base) v1[k] = *reinterpret_cast<const uint4*>(f1.base + (size_t)from[k] * f1.bytes);
        if (g0.base) v2[k] = *reinterpret_cast<const uint32_t*>(g0.base + (size_t)from[k] * g0.bytes);
      }
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) {
        if (to[k] == kNone) continue;
        if (f0.base) *reinterpret_cast<uint4*>(f0.base + (size_t)to[k] * f0.bytes) = v0[k];
        if (f1.base) *reinterpret_cast<uint4*>(f1.base + (size_t)to[k] * f1.bytes) = v1[k];
        if (g0.base) *reinterpret_cast<uint32_t*>(g0.base + (size_t)to[k] * g0.bytes) = v2[k];
      }
    }
  }
}

int64_t list_cap(int max_entries) { return ((int64_t)max_entries + 3) / 4 * 4; }
int cluster_size(int max_entries) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxCluster, ((int64_t)max_entries + kMinPerCta - 1) / kMinPerCta));
}
// Entries that a CTA's share can have.
int64_t share_cap(int max_entries) {
  const int n = cluster_size(max_entries);
  return ((int64_t)max_entries + n - 1) / n + 1;
}

}  // namespace

size_t evict_workspace_bytes(int B, int max_entries) {
  if (B <= 0 || max_entries <= 0) return 0;
  const size_t lists = share_cap(max_entries) > kMaxCached ? 3 : 2;   // holes, movers, and keys that do not fit
  return (((size_t)B + 63) / 64 * 64 + lists * (size_t)B * (size_t)list_cap(max_entries)) * sizeof(int32_t);
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
  const int n_cl = cluster_size(a.max_entries);
  const int cached = (int)std::min<int64_t>(kMaxCached, share_cap(a.max_entries));
  ws.keys = share_cap(a.max_entries) > kMaxCached ? reinterpret_cast<uint32_t*>(ws.movers + (int64_t)a.B * ws.cap) : nullptr;
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
  const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>((most + 7) / 8, ((int64_t)sms * kMoveBlocks + a.B - 1) / a.B));
  return launch_step(k_evict_move, dim3((unsigned)blocks, (unsigned)a.B), dim3(256), 0, s, a, ws, status_word());
}

}  // namespace csa2
