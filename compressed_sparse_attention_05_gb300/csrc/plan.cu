// Plans of a step, computed on the GPU from what the requests are: pages, positions and cache slots of the
// sequences' new tokens and entries (reading R17), and positions and paths of a tree of drafted tokens (R21).
//
// csa2_page_plan.  Per sequence the entries before and after the step,
//   e0 = len/4 - shift,  e1 = (len + n_new)/4 - shift,  need = ceil(e1 / 64),
// and two prefix sums over the sequences: of the pages given back (held - need where positive) and of the pages
// wanted (need - held where positive).  The free list with the released pages on top is a stack S of n_free + R
// pages; the k-th page handed out is S[n_free + R - 1 - k], so every page of the result follows from the sums alone
// and no thread waits for another's pop.  k_page_plan (one block) makes the sums; the columns (slots, positions,
// page-table entries) are written by the same block where they are few and by k_page_fill where they are many.
// Bound: latency of a chain of dependent loads in the small case, the bytes written in the large one.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace csa2 {
namespace {

// What the columns of a sequence follow from.
struct PageRow {
  int32_t len, n_new;     // tokens before the step, tokens it adds (granted, positive) or 0
  int32_t e0, e1;         // new entries [e0, e1)
  int32_t held, need;     // new pages [held, need), or released pages [need, held)
  int32_t take, back;     // prefix sums: pages handed out / released before this sequence's
};
struct PageHead {
  int32_t n_free, released, taken, pad;
};

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int64_t warp_scan64(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}
// Inclusive prefix sum over the block and its total (all threads call; two barriers).
__device__ __forceinline__ int64_t block_scan64(int64_t v, int64_t* sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  v = warp_scan64(v, lane);
  __syncthreads();
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  const int64_t w = warp_scan64(lane < warps ? sums[lane] : 0, lane);
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return v + (warp ? before : 0);
}

// The page at place i of the stack: the free list, then the released pages in the order of their sequences.
__device__ __forceinline__ int32_t stack_page(const PagePlanArgs& a, const PageHead& h, const PageRow* rows, int64_t i) {
  if (i < h.n_free) return a.free_pages[i];
  const int32_t j = (int32_t)(i - h.n_free);
  int lo = 0, hi = a.B - 1;                 // the last sequence whose released pages begin at or before j
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (rows[mid].back <= j) lo = mid;
    else hi = mid - 1;
  }
  const PageRow& r = rows[lo];
  return a.page_table[(int64_t)lo * a.max_pages + r.need + (j - r.back)];
}

// Columns first, first + step, ... of sequence b.
__device__ __forceinline__ void fill_row(const PagePlanArgs& a, const PageHead& h, const PageRow* rows, const PageRow& r, int b,
                                         int64_t first, int64_t step, uint32_t* status) {
  auto new_page = [&](int p) { return stack_page(a, h, rows, (int64_t)h.n_free + h.released - 1 - (r.take + (p - r.held))); };
  int32_t* table = a.page_table + (int64_t)b * a.max_pages;
  for (int64_t k = first; k < (int64_t)r.need - r.held; k += step) {
    const int32_t page = new_page(r.held + (int)k);
    if (page < 0 || page >= a.n_pages) raise_status(status, CSA2_STATUS_BAD_PAGE);
    table[r.held + k] = page;
  }
  if (a.q_pos)
    for (int64_t i = first; i < a.Tq; i += step) a.q_pos[(int64_t)b * a.Tq + i] = i < r.n_new ? r.len + (int32_t)i : -1;
  if (a.slots)
    for (int64_t i = first; i < a.max_new; i += step) {
      const int64_t e = r.e0 + i;
      int64_t slot = -1;
      if (e < r.e1) {
        const int p = (int)(e >> 6);
        // (a page behind `held` may not be in the table yet: another thread writes it)
        const int32_t page = p < r.held ? table[p] : new_page(p);
        if (page >= 0 && page < a.n_pages) slot = (int64_t)page * kPage + (e & (kPage - 1));
        else raise_status(status, CSA2_STATUS_BAD_PAGE);
      }
      a.slots[(int64_t)b * a.max_new + i] = slot;
    }
}

// Released pages that nobody took go back on the free list.
__device__ __forceinline__ void push_released(const PagePlanArgs& a, const PageHead& h, const PageRow* rows, int64_t first, int64_t step,
                                              uint32_t* status) {
  for (int64_t i = first; i < (int64_t)h.released - h.taken; i += step) {
    const int32_t page = stack_page(a, h, rows, h.n_free + i);
    if (page < 0 || page >= a.n_pages) raise_status(status, CSA2_STATUS_BAD_PAGE);
    a.free_pages[h.n_free + i] = page;
  }
}

__global__ void __launch_bounds__(kPlanThreads) k_page_plan(PagePlanArgs a, PageHead* head, PageRow* rows, int fill_here, uint32_t* status) {
  __shared__ int64_t s_sums[32];
  __shared__ PageHead s_head;
  if (!fill_here) pdl_trigger();   // k_page_fill waits for this kernel; what follows it must not start before both are done
  pdl_wait();
  const int tid = threadIdx.x, threads = blockDim.x;
  // one sequence's counts, or a change of nothing where its state is impossible
  auto read = [&](int b, bool report) {
    PageRow r;
    r.len = a.seq_len[b];
    r.n_new = a.n_new[b];
    r.held = a.held[b];
    const int32_t shift = a.shift ? a.shift[b] : 0;
    const int64_t len1 = (int64_t)r.len + r.n_new;
    const int64_t e0 = (r.len >> 2) - (int64_t)shift, e1 = (len1 >> 2) - shift;
    const int64_t need = (e1 + kPage - 1) >> 6;
    const bool ok = r.len >= 0 && len1 >= 0 && len1 <= INT_MAX && shift >= 0 && e0 >= 0 && e1 >= 0 && r.held >= 0 &&
                    r.held <= a.max_pages && ((e0 + kPage - 1) >> 6) <= r.held && need <= a.max_pages &&
                    (!a.q_pos || r.n_new <= a.Tq) && (!a.slots || e1 - e0 <= a.max_new);
    r.e0 = (int32_t)max((int64_t)0, e0);
    r.e1 = ok ? (int32_t)e1 : -1;          // -1: impossible
    r.need = ok ? (int32_t)need : r.held;
    r.take = r.back = 0;
    if (!ok && report) raise_status(status, CSA2_STATUS_BAD_COUNT);
    return r;
  };
  // pages given back by all sequences (they are there to be handed out to any)
  int64_t mine = 0, released = 0;
  for (int b = tid; b < a.B; b += threads) {
    const PageRow r = read(b, false);
    mine += max(0, r.held - r.need);
  }
  block_scan64(mine, s_sums, &released);
  const int32_t n_free = *a.n_free;
  const int64_t avail = (int64_t)n_free + released;
  const bool sane = n_free >= 0 && avail <= a.n_pages;
  if (!sane && tid == 0) raise_status(status, CSA2_STATUS_BAD_COUNT);
  int64_t back0 = 0, want0 = 0, taken = 0;
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    const int b = b0 + tid;
    const bool live = b < a.B;
    PageRow r = {};
    if (live) r = read(b, true);
    const int64_t back = live ? max(0, r.held - r.need) : 0, want = live ? max(0, r.need - r.held) : 0;
    int64_t back_all, want_all;
    const int64_t back_inc = block_scan64(back, s_sums, &back_all);
    const int64_t want_inc = block_scan64(want, s_sums, &want_all);
    // in order: a sequence gets its pages if they and all that was asked for before it are there
    const bool granted = live && r.e1 >= 0 && sane && (want == 0 || want0 + want_inc <= avail);
    if (live) {
      const int32_t len0 = r.len, e_last = granted ? r.e1 : r.e0;
      a.seq_len_out[b] = granted ? len0 + r.n_new : len0;
      a.n_entries[b] = e_last;
      a.first_entry[b] = min(r.e0, e_last);
      if (a.granted) a.granted[b] = granted ? 1 : 0;
      a.held[b] = granted ? r.need : r.held;
      if (!granted) r.need = r.held;
      r.n_new = granted ? max(0, r.n_new) : 0;
      r.e1 = granted ? r.e1 : r.e0;
      r.back = (int32_t)(back0 + back_inc - back);
      r.take = (int32_t)min((int64_t)INT_MAX, want0 + want_inc - want);
      rows[b] = r;
      if (granted && want > 0) taken = want0 + want_inc;   // (grows with b: the last one granted has the sum)
    }
    back0 += back_all;
    want0 += want_all;
  }
  // the largest sum that was granted
  __syncthreads();
  if (tid == 0) s_head = PageHead{n_free, sane ? (int32_t)released : 0, 0, 0};
  __syncthreads();
  if (taken > 0) atomicMax(&s_head.taken, (int32_t)taken);
  __syncthreads();
  if (tid == 0) {
    *head = s_head;
    if (sane) *a.n_free = s_head.n_free + s_head.released - s_head.taken;
  }
  if (!fill_here) return;
  // ---- few columns: written here (rows[] of this block are visible after the barrier)
  const PageHead h = s_head;
  const int64_t cols = max(max((int64_t)(a.q_pos ? a.Tq : 0), a.slots ? (int64_t)a.max_new : 0), (int64_t)32);
  const int per = cols >= threads ? threads : (int)((cols + 31) / 32) * 32;   // threads to a sequence
  const int lanes = threads / per * per;
  if (tid < lanes)
    for (int b = tid / per; b < a.B; b += threads / per) fill_row(a, h, rows, rows[b], b, tid % per, per, status);
  push_released(a, h, rows, tid, threads, status);
}

constexpr int kFillThreads = 256, kFillPer = 8;   // threads of a block, columns of a thread

__global__ void __launch_bounds__(kFillThreads) k_page_fill(PagePlanArgs a, const PageHead* head, const PageRow* rows, uint32_t* status) {
  pdl_wait();
  const PageHead h = *head;
  const int64_t first = (int64_t)blockIdx.x * kFillThreads + threadIdx.x, step = (int64_t)gridDim.x * kFillThreads;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) fill_row(a, h, rows, rows[b], b, first, step, status);
  push_released(a, h, rows, first + step * blockIdx.y, step * gridDim.y, status);
}

// ---- a tree of drafted tokens -----------------------------------------------------------------
// One block per sequence; the parents lie in shared memory and every thread walks from its nodes to the root.
constexpr int kTreeThreads = 128, kTreeMax = 1024;

__global__ void __launch_bounds__(kTreeThreads) k_tree_plan(int Tq, int max_depth, const int32_t* __restrict__ parent,
                                                            const int32_t* __restrict__ ctx_len, int32_t* __restrict__ q_pos,
                                                            int32_t* __restrict__ path, uint32_t* status) {
  __shared__ int16_t up[kTreeMax];     // parent; -1: child of the committed text; -2: no node
  pdl_wait();
  const int b = blockIdx.x;
  const int32_t ctx = ctx_len[b];
  if (ctx < 0 && threadIdx.x == 0) raise_status(status, CSA2_STATUS_BAD_COUNT);
  for (int i = threadIdx.x; i < Tq; i += kTreeThreads) {
    const int32_t p = parent[(int64_t)b * Tq + i];
    if (p >= i) raise_status(status, CSA2_STATUS_BAD_INDEX);
    up[i] = (int16_t)(p < -1 || p >= i ? -2 : p);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < Tq; i += kTreeThreads) {
    int depth = -1, at = i;             // (a parent's index is below its child's: the walk ends)
    while (at >= 0) {
      ++depth;
      at = up[at];
    }
    bool node = at == -1 && ctx >= 0;
    if (at == -2 && depth > 0) raise_status(status, CSA2_STATUS_BAD_INDEX);   // hangs on something that is no node
    if (node && (depth >= max_depth || ctx > INT_MAX - depth)) {
      raise_status(status, CSA2_STATUS_BAD_COUNT);
      node = false;
    }
    const int64_t row = (int64_t)b * Tq + i;
    q_pos[row] = node ? ctx + depth : -1;
    int32_t* out = path + row * max_depth;
    for (int k = node ? depth + 1 : 0; k < max_depth; ++k) out[k] = -1;
    if (node) {
      at = i;
      for (int k = depth; k >= 0; --k) {
        out[k] = at;
        at = up[at];
      }
    }
  }
}

size_t head_bytes() { return 256; }

}  // namespace

size_t page_plan_workspace_bytes(int B) { return head_bytes() + (size_t)B * sizeof(PageRow); }

// Columns that one block writes itself: the second launch costs about as long as they take.
constexpr int64_t kFillHere = 16384;

cudaError_t launch_page_plan(const PagePlanArgs& a, void* ws, cudaStream_t s) {
  PageHead* head = static_cast<PageHead*>(ws);
  PageRow* rows = reinterpret_cast<PageRow*>(static_cast<char*>(ws) + head_bytes());
  const int64_t cols = std::max<int64_t>(std::max<int64_t>(a.q_pos ? a.Tq : 0, a.slots ? a.max_new : 0), 1);
  const bool here = cols * a.B <= kFillHere;
  const int threads = here ? kPlanThreads : std::min(kPlanThreads, (a.B + 31) / 32 * 32);
  cudaError_t e = launch_step(k_page_plan, dim3(1), dim3(threads), 0, s, a, head, rows, (int)here, status_word());
  if (e != cudaSuccess || here) return e;
  const unsigned gx = (unsigned)std::min<int64_t>((cols + kFillThreads * kFillPer - 1) / (kFillThreads * kFillPer), 65535);
  return launch_step(k_page_fill, dim3(gx, (unsigned)std::min(a.B, 65535)), dim3(kFillThreads), 0, s, a, head, rows, status_word());
}

int tree_plan_max_nodes() { return kTreeMax; }

cudaError_t launch_tree_plan(int B, int Tq, int max_depth, const int32_t* parent, const int32_t* ctx_len, int32_t* q_pos, int32_t* path,
                             cudaStream_t s) {
  return launch_step(k_tree_plan, dim3((unsigned)B), dim3(kTreeThreads), 0, s, Tq, max_depth, parent, ctx_len, q_pos, path, status_word());
}

}  // namespace csa2
