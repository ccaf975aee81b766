// kv_plan: pages, row starts, positions and slots of a step, from the lengths of its sequences.
//
// With P tokens a page, sequence b of len_b kept and n_b new tokens needs need_b = ceil((len_b + n_b) / P) pages.  Those that
// it owns past need_b go back to the stack of free ones, in order of (b, page of b); then the sequences in turn take what they
// lack from its top.  All of it are running sums over the sequences: row starts (of n), places on the
// stack (of pages given back) and ranks from its top (of pages wanted).  Wants are summed whether they are met or not, so
// the sequences that get pages are those whose running sum the stack covers: a prefix, whose ranks need no second sum.
//
// One workgroup: the sums are a few thousand additions, and pages given back must be on the stack before any are taken.  Rows
// follow in the same launch while there are few, else in one of their own.  Bound: latency, of the loads that follow from
// each other (lengths, page, table entry).
#include <algorithm>

#include "w4_internal.h"
#include "w4_kv.h"

namespace w4 {

namespace {

constexpr int kPlanThreads = 1024, kRowThreads = 256;
constexpr int kOneLaunchRows = 4096;  // rows that the first launch writes too, at most

// Inclusive sum over the workgroup's threads; all: over all of them.  lds: one int64 per wave; the caller separates uses.
template <int THREADS>
__device__ __forceinline__ int64_t block_sum(int64_t mine, int64_t& all, int64_t* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t x = __shfl_up((long long)incl, d);
    if (lane >= d) incl += x;
  }
  if (lane == 63) lds[wave] = incl;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    const int64_t x = lds[w];
    if (w < wave) incl += x;
    all += x;
  }
  return incl;
}

// f(b, from, i) for i of 0 .. count - 1 of every lane's sequence b, from being a value of that sequence's: a lane does its
// first one itself, and the wave does the others of each lane that has more.
template <class F>
__device__ __forceinline__ void for_pages(int b, int count, int64_t from, F f) {
  if (count > 0) f(b, from, 0);
  unsigned long long more = __ballot(count > 1);
  while (more) {
    const int l = __builtin_ctzll(more), c = __shfl(count, l);
    const int64_t x = __shfl((long long)from, l);
    const int at = __shfl(b, l);
    for (int i = 1 + (threadIdx.x & 63); i < c; i += 64) f(at, x, i);
    more &= more - 1;
  }
}

// A sequence and what it asks for.
struct Asked {
  int len, n, have, need;  // kept and new tokens; pages owned and needed (have, if it does not fit)
  bool fits;               // its lengths fit the table, its rows the step's
  int rows;                // that it counts for in the starts
};
__device__ __forceinline__ Asked asked(const PlanArgs& g, int b) {
  Asked s;
  s.len = g.kv_len[b], s.n = g.new_len[b];
  s.have = min(max(g.owned[b], 0), g.W);
  s.rows = min(max(s.n, 0), g.T);
  return s;
}
// start: the row that it starts at, at most T
__device__ __forceinline__ void fit(const PlanArgs& g, int start, Asked& s) {
  const int64_t total = (int64_t)s.len + s.n;
  s.fits = s.len >= 0 && s.n >= 0 && total <= (int64_t)g.W * g.page_size && start + (int64_t)s.n <= g.T;
  s.need = s.fits ? (int)((total + g.page_size - 1) / g.page_size) : s.have;
}

// Row t: of sequence b (-1: none), which starts at row `start`.
__device__ __forceinline__ void write_row(const PlanArgs& g, int t, int b, int start, int end) {
  int pos = 0;
  int64_t slot = -1;
  if (b >= 0) {
    const int status = g.status[b], total = g.kv_total[b], i = t - start;
    if (status >= 0) {
      const int len = status == 0 ? total - (end - start) : total;
      pos = (int)((uint32_t)len + (uint32_t)(g.depth ? g.depth[t] : i));
      if (status == 0) {
        const int page = (len + i) / g.page_size, id = g.table[b * g.ldt + page];
        if ((uint32_t)id < (uint32_t)g.pages) slot = (int64_t)id * g.page_size + (len + i - page * g.page_size);
      }
    }
  }
  g.pos[t] = pos;
  g.slot[t] = slot;
}

// The last of n + 1 ascending starts that is not above t, by its index; -1 if that is the last of all.
__device__ __forceinline__ int sequence_of(const int32_t* starts, int n, int t) {
  int lo = 0, hi = n + 1;  // starts[lo] <= t < starts[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (starts[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo == n ? -1 : lo;
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs g, bool rows_too) {
  __shared__ int64_t sums[3][kPlanThreads / 64];
  __shared__ int starts[kPlanThreads + 1];
  __shared__ int last_taken;
  const int tid = threadIdx.x;
  const bool once = g.B <= kPlanThreads;
  const int count = min(max(*g.free_count, 0), g.pages);
  Asked s{};
  int64_t row0 = 0, given = 0, all = 0;
  if (tid == 0) last_taken = 0;
  // starts, and pages that go back
  for (int b0 = 0; b0 < g.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    s = b < g.B ? asked(g, b) : Asked{};
    const int64_t end = row0 + block_sum<kPlanThreads>(s.rows, all, sums[0]);
    row0 += all;
    const int start = (int)min((int64_t)g.T, end - s.rows);
    if (b < g.B) {
      fit(g, start, s);
      g.q_start[b] = start;
      if (once) starts[b] = start;
      if (b == g.B - 1) {
        g.q_start[g.B] = (int)min((int64_t)g.T, end);
        if (once) starts[g.B] = (int)min((int64_t)g.T, end);
      }
    }
    const int back = max(0, s.have - s.need);
    const int64_t at = count + given + block_sum<kPlanThreads>(back, all, sums[1]) - back;
    given += all;
    for_pages(b, back, at | (int64_t)s.need << 32, [&](int of, int64_t x, int i) {
      int32_t* entry = g.table + of * g.ldt + (x >> 32) + i;
      const int64_t to = (x & 0xffffffff) + i;
      if (to < g.pages) g.free[to] = *entry;
      *entry = -1;
    });
    if (!once) __syncthreads();
  }
  __syncthreads();  // the stack holds what was given back
  const int there = (int)min((int64_t)g.pages, count + given);
  // pages that are taken
  int64_t wanted = 0;
  for (int b0 = 0; b0 < g.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    if (!once) {
      s = b < g.B ? asked(g, b) : Asked{};
      if (b < g.B) fit(g, g.q_start[b], s);
    }
    const int want = max(0, s.need - s.have);
    const int64_t end = wanted + block_sum<kPlanThreads>(want, all, sums[2]);
    wanted += all;
    const bool granted = want == 0 || end <= there;
    for_pages(b, granted ? want : 0, (there - 1 - (end - want)) | (int64_t)s.have << 32, [&](int of, int64_t x, int i) {
      g.table[of * g.ldt + (x >> 32) + i] = g.free[(x & 0xffffffff) - i];
    });
    if (granted && want > 0) atomicMax(&last_taken, (int)end);
    if (b < g.B) {
      g.owned[b] = granted ? s.need : s.have;
      g.status[b] = !s.fits ? -1 : granted ? 0 : want;
      g.kv_total[b] = s.fits && granted ? s.len + s.n : s.len;
    }
    if (!once) __syncthreads();
  }
  __syncthreads();
  if (tid == 0) *g.free_count = there - last_taken;
  if (!rows_too) return;
  for (int t = tid; t < g.T; t += kPlanThreads) {
    const int b = once ? sequence_of(starts, g.B, t) : sequence_of(g.q_start, g.B, t);
    const int at = max(b, 0);
    write_row(g, t, b, once ? starts[at] : g.q_start[at], once ? starts[at + 1] : g.q_start[at + 1]);
  }
}

__global__ __launch_bounds__(kRowThreads) void plan_rows_kernel(PlanArgs g) {
  const int t = blockIdx.x * kRowThreads + threadIdx.x;
  if (t >= g.T) return;
  const int b = sequence_of(g.q_start, g.B, t), at = max(b, 0);
  write_row(g, t, b, g.q_start[at], g.q_start[at + 1]);
}

}  // namespace

void launch_plan(const PlanArgs& a, hipStream_t st) {
  const bool rows_too = a.T <= kOneLaunchRows;
  plan_kernel<<<1, kPlanThreads, 0, st>>>(a, rows_too);
  if (!rows_too) plan_rows_kernel<<<(a.T + kRowThreads - 1) / kRowThreads, kRowThreads, 0, st>>>(a);
}

}  // namespace w4
