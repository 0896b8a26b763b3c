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
// Bound: latency of a chain of dependent loads in the small case (32 sequences of 8 tokens: 5.1 us), the bytes written in
// the large one (160 sequences of up to 32,768 tokens, 31.5 MB of columns: 8.0 us).
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
// The page at place i of the stack: the free list, then the released pages in the order of their sequences.
__device__ __forceinline__ int32_t stack_page(const PagePlanArgs& a, const PageHead& h, const PageRow* rows, int64_t i) {
  if (i < 0 || i >= (int64_t)h.n_free + h.released) return -1;
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

// What thread `t` of `threads` (at most 2^24) writes of sequence b: new places in the table, positions, slots.  A warp takes
// the slots of a page, which is looked up once for all of them.  Columns are below 2^31 and entries below 2^29, so that
// their sums fit 32 bits without a sign; with 64 the fill's instructions took longer than its bytes.
__device__ __forceinline__ void fill_row(const PagePlanArgs& a, const PageHead& h, const PageRow* rows, const PageRow& r, int b,
                                         uint32_t t, uint32_t threads, uint32_t* status) {
  auto new_page = [&](int p) { return stack_page(a, h, rows, (int64_t)h.n_free + h.released - 1 - (r.take + (p - r.held))); };
  int32_t* table = a.page_table + (int64_t)b * a.max_pages;
  for (int64_t k = t; k < (int64_t)r.need - r.held; k += threads) {
    const int32_t page = new_page(r.held + (int)k);
    if (page < 0 || page >= a.n_pages) raise_status(status, CSA2_STATUS_BAD_PAGE);
    table[r.held + k] = page;
  }
  if (a.q_pos) {
    int32_t* out = a.q_pos + (int64_t)b * a.Tq;
    const uint32_t cols = (uint32_t)a.Tq, n = (uint32_t)r.n_new;
    auto at = [&](uint32_t i) { return i < n ? r.len + (int32_t)i : -1; };
    if (a.q_pos4) {        // four at a time: rows start on 16 bytes
      for (uint32_t i = 4 * t; i < cols; i += 4 * threads)
        *reinterpret_cast<int4*>(out + i) = make_int4(at(i), at(i + 1), at(i + 2), at(i + 3));
    } else {
      for (uint32_t i = t; i < cols; i += threads) out[i] = at(i);
    }
  }
  if (a.slots) {
    int64_t* out = a.slots + (int64_t)b * a.max_new;
    const uint32_t lane = threadIdx.x & 31, cols = (uint32_t)a.max_new, e0 = (uint32_t)r.e0, e1 = (uint32_t)r.e1;
    const uint32_t p0 = e0 / kPage, groups = (e0 % kPage + cols + kPage - 1) / kPage;   // column i is place (e0 + i) % 64
    for (uint32_t g = t >> 5; g < groups; g += threads >> 5) {
      const uint32_t p = p0 + g, e = p * kPage + lane;
      int32_t page = -1;
      if (e1 > e0 && p * kPage < e1) {                       // (so p is below `need`)
        // (a page behind `held` may not be in the table yet: another thread writes it)
        page = (int32_t)p < r.held ? table[p] : new_page((int)p);
        if (page < 0 || page >= a.n_pages) {
          if (lane == 0) raise_status(status, CSA2_STATUS_BAD_PAGE);
          page = -1;
        }
      }
#pragma unroll
      for (uint32_t u = 0; u < kPage; u += 32) {
        const uint32_t i = e + u - e0;                       // (before e0 it wraps past every column)
        if (i < cols) out[i] = page >= 0 && e + u < e1 ? (int64_t)page * kPage + lane + u : -1;
      }
    }
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

// fill_here: the columns too (then the rows stay in shared memory).
constexpr int kFillSeqs = 64;
__global__ void __launch_bounds__(kPlanThreads) k_page_plan(PagePlanArgs a, PageHead* head, PageRow* rows, int fill_here, uint32_t* status) {
  __shared__ int64_t s_sums[2][32];
  __shared__ PageHead s_head;
  __shared__ PageRow s_rows[kFillSeqs];
  if (!fill_here) pdl_trigger();   // k_page_fill waits for this kernel; what follows it must not start before both are done
  pdl_wait();
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
  if (fill_here) rows = s_rows;      // (at most kFillSeqs sequences)
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
  // Inclusive prefix sums over the block of two values, and their totals.  (A warp's worth of sequences takes no barrier.)
  auto scan2 = [&](int64_t& x, int64_t& y, int64_t* all_x, int64_t* all_y) {
    x = warp_scan64(x, lane);
    y = warp_scan64(y, lane);
    __syncthreads();
    if (lane == 31) {
      s_sums[0][warp] = x;
      s_sums[1][warp] = y;
    }
    __syncthreads();
    const int64_t wx = warp_scan64(lane < warps ? s_sums[0][lane] : 0, lane), wy = warp_scan64(lane < warps ? s_sums[1][lane] : 0, lane);
    *all_x = __shfl_sync(0xffffffffu, wx, 31);
    *all_y = __shfl_sync(0xffffffffu, wy, 31);
    const int64_t bx = __shfl_sync(0xffffffffu, wx, warp > 0 ? warp - 1 : 0), by = __shfl_sync(0xffffffffu, wy, warp > 0 ? warp - 1 : 0);
    if (warp) {
      x += bx;
      y += by;
    }
  };
  const int32_t n_free = *a.n_free;
  // The first batch of sequences stays in registers; with more, the pages that all of them give back (they are there to
  // be handed out to any) are counted before.
  PageRow r = {};
  if (tid < a.B) r = read(tid, true);
  int64_t back_inc = tid < a.B ? max(0, r.held - r.need) : 0, want_inc = tid < a.B ? max(0, r.need - r.held) : 0;
  int64_t back_all, want_all;
  scan2(back_inc, want_inc, &back_all, &want_all);
  int64_t released = back_all;
  if (a.B > threads) {
    int64_t mine = 0, none = 0, total;
    for (int b = threads + tid; b < a.B; b += threads) {
      const PageRow q = read(b, true);
      mine += max(0, q.held - q.need);
    }
    scan2(mine, none, &total, &none);
    released += total;
  }
  const int64_t avail = (int64_t)n_free + released;
  const bool sane = n_free >= 0 && avail <= a.n_pages;
  if (!sane && tid == 0) raise_status(status, CSA2_STATUS_BAD_COUNT);
  if (tid == 0) s_head = PageHead{n_free, sane ? (int32_t)released : 0, 0, 0};
  __syncthreads();
  int64_t back0 = 0, want0 = 0;
  for (int b0 = 0;;) {
    const int b = b0 + tid;
    if (b < a.B) {
      const int64_t back = max(0, r.held - r.need), want = max(0, r.need - r.held);
      // in order: a sequence gets its pages if they and all that was asked for before it are there
      const bool granted = r.e1 >= 0 && sane && (want == 0 || want0 + want_inc <= avail);
      const int32_t e_last = granted ? r.e1 : r.e0;
      a.seq_len_out[b] = granted ? r.len + r.n_new : r.len;
      a.n_entries[b] = e_last;
      a.first_entry[b] = min(r.e0, e_last);
      if (a.granted) a.granted[b] = granted ? 1 : 0;
      a.held[b] = granted ? r.need : r.held;
      if (granted && want > 0) atomicMax(&s_head.taken, (int32_t)(want0 + want_inc));   // the last one granted has the sum
      if (!granted) r.need = r.held;
      r.n_new = granted ? max(0, r.n_new) : 0;
      r.e1 = e_last;
      r.back = (int32_t)(back0 + back_inc - back);
      r.take = (int32_t)min((int64_t)INT_MAX, want0 + want_inc - want);
      rows[b] = r;
    }
    back0 += back_all;
    want0 += want_all;
    b0 += threads;
    if (b0 >= a.B) break;
    r = PageRow{};
    const bool live = b0 + tid < a.B;
    if (live) r = read(b0 + tid, false);
    back_inc = live ? max(0, r.held - r.need) : 0;
    want_inc = live ? max(0, r.need - r.held) : 0;
    scan2(back_inc, want_inc, &back_all, &want_all);
  }
  __syncthreads();
  const PageHead h = s_head;
  if (tid == 0) {
    if (!fill_here) *head = h;
    if (sane) *a.n_free = h.n_free + h.released - h.taken;
  }
  if (!fill_here) return;
  // ---- few columns: written here, a power of two of warps to a sequence
  int per = 32;
  while (per < threads && per * min(a.B, threads / per) < threads && per * 2 <= threads) per *= 2;
  const int teams = threads / per;
  if (tid < teams * per)
    for (int b = tid / per; b < a.B; b += teams) fill_row(a, h, rows, rows[b], b, tid % per, per, status);
  push_released(a, h, rows, tid, threads, status);
}

// Threads of a block, columns of a thread (16 x 8,192 and 160 x 32,768 columns: with 8 columns 5.7 and 8.0 us, 16 6.4 and
// 9.6, 32 6.8 and 10.2).
constexpr int kFillThreads = 256, kFillPer = 8;

__global__ void __launch_bounds__(kFillThreads) k_page_fill(PagePlanArgs a, const PageHead* head, const PageRow* rows, uint32_t* status) {
  pdl_wait();
  const PageHead h = *head;
  const uint32_t t = blockIdx.x * kFillThreads + threadIdx.x, threads = gridDim.x * kFillThreads;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) fill_row(a, h, rows, rows[b], b, t, threads, status);
  push_released(a, h, rows, t + (int64_t)threads * blockIdx.y, (int64_t)threads * gridDim.y, status);
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

// One block writes the columns itself up to kFillSeqs sequences and kFillHere columns of all together: that saves the
// second launch, 2 us of the host's time, where it takes about as long (one launch, two launches, in us on the GPU:
// 8 x 8 3.3 and 4.7, 32 x 8 5.7 and 5.5, 64 x 8 6.6 and 5.9, 4 x 1,024 4.7 and 4.1).  Beyond that the block is the slower
// one: 32 x 512 7.0 and 5.4, 128 x 8 10.0 and 7.0, 256 x 64 16.8 and 7.6, 600 x 8 35.1 and 10.2.
constexpr int64_t kFillHere = 4096;

cudaError_t launch_page_plan(const PagePlanArgs& a, void* ws, cudaStream_t s) {
  PageHead* head = static_cast<PageHead*>(ws);
  PageRow* rows = reinterpret_cast<PageRow*>(static_cast<char*>(ws) + head_bytes());
  const int64_t cols = std::max<int64_t>(std::max<int64_t>(a.q_pos ? a.Tq : 0, a.slots ? a.max_new : 0), 1);
  const bool here = a.B <= kFillSeqs && cols * a.B <= kFillHere;
  // as many threads as there are sequences, and for the columns up to eight warps to a sequence
  const int64_t warps = (a.B + 31) / 32, want = here ? std::max<int64_t>(warps, a.B * std::min<int64_t>((cols + 63) / 64, 8)) : warps;
  const int threads = (int)std::min<int64_t>(kPlanThreads / 32, want) * 32;
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
