// kv_plan: pages, row starts, positions and slots of a step, from the lengths of its sequences.
//
// With P tokens a page, sequence b of len_b kept and n_b new tokens needs need_b = ceil((len_b + n_b) / P) pages.  Those that
// it owns past need_b go back to the stack of free ones, in order of (b, page of b); then the sequences in turn take what they
// lack from its top.  All of it are running sums over the sequences: row starts (of n), places on the
// stack (of pages given back) and ranks from its top (of pages wanted).  Wants are summed whether they are met or not, so
// the sequences that get pages are those whose running sum the stack covers: a prefix, whose ranks need no second sum.
//
// One workgroup: the sums are a few thousand additions, and pages given back are taken again in the same call.  (Many workgroups could move
// the pages of a large step: a page that is given back and taken has its old entry for a source, which its rank names.  This is not done.)
// Up to 1024 sequences, a thread each, the sums stay in LDS, and every page that moves and every row finds its sequence there by
// bisection, so that all are under way at once; above, sequences come in rounds of 1024.  Rows follow in the same launch while there are
// few, else in one of their own.
// Bound: latency, of the launch and the loads that follow from each other (lengths, page, table entry).
// Measured: 64 single tokens 4 us where no page moves, 9.9 (10.8 in a replayed graph) with 5000 given back and as many taken; 256
// sequences, 25 k rows, 26 k pages back and taken 21.5 and 4.1 for the rows (through one CU, four loads of a thread under way; one load
// 22 as well: its stores bound it). Above 1024 sequences, in a replayed graph: 2048 single tokens 17 us where no page moves and 35 with 3
// in 10 replaced, 8192 44 and 103: rounds of 1024 one after another.
#include <algorithm>

#include "w4_internal.h"
#include "w4_kv.h"

namespace w4 {

namespace {

constexpr int kPlanThreads = 1024, kRowThreads = 256;
constexpr int kOneLaunchRows = 4096;  // rows that the first launch writes too, at most

// Inclusive sum over kPlanThreads threads; all: over all of them.  lds: one int64 per wave; the caller separates uses.
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
  for (int w = 0; w < kPlanThreads / 64; ++w) {
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

// Inclusive sum over a wave, kept to `most` (below 2^31): adding so is associative, and fits 32 bits.
__device__ __forceinline__ uint32_t wave_sum(uint32_t x, uint32_t most) {
#define W4_STEP(CTRL, ROWS) x = min(most, x + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false))
  W4_STEP(0x111, 0xF);  // row_shr 1, 2, 4, 8: sums of the rows of 16
  W4_STEP(0x112, 0xF);
  W4_STEP(0x114, 0xF);
  W4_STEP(0x118, 0xF);
  W4_STEP(0x142, 0xA);  // row_bcast15 into rows 1 and 3, row_bcast31 into rows 2 and 3
  W4_STEP(0x143, 0xC);
#undef W4_STEP
  return x;
}
// The sums of the waves before this one, and of all; mine: a wave's inclusive sum (its last lane's counts).
template <int WAVES>
__device__ __forceinline__ uint32_t before_wave(const uint32_t* waves, uint32_t most, uint32_t& all) {
  const int wave = threadIdx.x >> 6;
  uint32_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    if (w == wave) before = all;
    all = min(most, all + waves[w]);
  }
  return before;
}

// Up to THREADS sequences.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void plan_few_kernel(PlanArgs g, bool rows_too) {
  constexpr int WAVES = THREADS / 64;
  constexpr uint32_t kMost = 0x7fffffffu;
  constexpr int DEEP = 4;  // pages under way for each thread
  __shared__ uint32_t waves[3][WAVES];
  __shared__ int starts[THREADS + 1], backs[THREADS], wants[THREADS], firsts[THREADS];
  __shared__ uint32_t taken;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = tid;
  const int count = min(max(*g.free_count, 0), g.pages);
  Asked s = b < g.B ? asked(g, b) : Asked{};
  if (tid == 0) taken = 0;
  uint32_t all;
  const uint32_t rows = wave_sum((uint32_t)s.rows, (uint32_t)g.T);
  if (lane == 63) waves[0][wave] = rows;
  __syncthreads();
  // kept to T, an end may be less than a start and its rows, but then all further ones are T
  const uint32_t row0 = before_wave<WAVES>(waves[0], (uint32_t)g.T, all);
  const uint32_t up = (uint32_t)__shfl_up((int)rows, 1);  // by all lanes
  const uint32_t lane_before = lane ? up : 0u;
  const int start = (int)min((uint32_t)g.T, row0 + lane_before);
  if (b < g.B) {
    fit(g, start, s);
    g.q_start[b] = start, starts[b] = start;
  }
  if (tid == 0) g.q_start[g.B] = (int)all, starts[g.B] = (int)all;
  // pages that go back, and pages that are lacked
  const uint32_t back = max(0, s.have - s.need), want = max(0, s.need - s.have);
  const uint32_t back_to = wave_sum(back, kMost), want_to = wave_sum(want, kMost);
  if (lane == 63) waves[1][wave] = back_to, waves[2][wave] = want_to;
  __syncthreads();
  uint32_t given, wanted;
  const uint32_t back0 = before_wave<WAVES>(waves[1], kMost, given), want0 = before_wave<WAVES>(waves[2], kMost, wanted);
  const uint32_t back_end = min(kMost, back0 + back_to), want_end = min(kMost, want0 + want_to);
  backs[tid] = (int)(back_end - min(back, back_end)), wants[tid] = (int)(want_end - min(want, want_end));
  firsts[tid] = min(s.have, s.need);
  const int there = (int)min((uint32_t)g.pages, (uint32_t)count + given);
  const bool granted = want == 0 || want_end <= (uint32_t)there;
  if (granted && want > 0) atomicMax(&taken, want_end);
  if (b < g.B) {
    g.owned[b] = granted ? s.need : s.have;
    g.status[b] = !s.fits ? -1 : granted ? 0 : (int)want;
    g.kv_total[b] = s.fits && granted ? s.len + s.n : s.len;
  }
  __syncthreads();
  // the last of B ascending sums that is not above i: the sequence of page i
  auto of = [&](const int* sums, int i) {
    int lo = 0, hi = g.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (sums[mid] <= i)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  };
  if (given > 0) {
    for (uint32_t i0 = tid; i0 < given; i0 += DEEP * THREADS) {
      int32_t* entry[DEEP];
      int32_t page[DEEP];
#pragma unroll
      for (int e = 0; e < DEEP; ++e) {
        const int i = (int)min(i0 + e * THREADS, given - 1), x = of(backs, i);
        entry[e] = g.table + x * g.ldt + firsts[x] + (i - backs[x]);
        page[e] = *entry[e];
      }
#pragma unroll
      for (int e = 0; e < DEEP; ++e) {
        const uint32_t i = i0 + e * THREADS;
        if (i >= given) break;
        if (count + (int64_t)i < g.pages) g.free[count + i] = page[e];
        *entry[e] = -1;
      }
    }
    __syncthreads();  // the stack holds what was given back
  }
  const uint32_t all_taken = taken;
  for (uint32_t i0 = tid; i0 < all_taken; i0 += DEEP * THREADS) {
    int32_t page[DEEP];
#pragma unroll
    for (int e = 0; e < DEEP; ++e) page[e] = g.free[there - 1 - (int)min(i0 + e * THREADS, all_taken - 1)];
#pragma unroll
    for (int e = 0; e < DEEP; ++e) {
      const uint32_t i = i0 + e * THREADS;
      if (i >= all_taken) break;
      const int x = of(wants, (int)i);
      g.table[x * g.ldt + firsts[x] + ((int)i - wants[x])] = page[e];
    }
  }
  if (tid == 0) *g.free_count = there - (int)all_taken;
  if (!rows_too) return;
  __syncthreads();
  for (int t = tid; t < g.T; t += THREADS) {
    const int x = sequence_of(starts, g.B, t), at = max(x, 0);
    write_row(g, t, x, starts[at], starts[at + 1]);
  }
}

// Any number of sequences.
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs g, bool rows_too) {
  __shared__ int64_t sums[3][kPlanThreads / 64];
  __shared__ int last_taken;
  const int tid = threadIdx.x;
  const int count = min(max(*g.free_count, 0), g.pages);
  int64_t row0 = 0, given = 0, all = 0;
  if (tid == 0) last_taken = 0;
  // starts, and pages that go back
  for (int b0 = 0; b0 < g.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    Asked s = b < g.B ? asked(g, b) : Asked{};
    const int64_t end = row0 + block_sum(s.rows, all, sums[0]);
    row0 += all;
    const int start = (int)min((int64_t)g.T, end - s.rows);
    if (b < g.B) {
      fit(g, start, s);
      g.q_start[b] = start;
      if (b == g.B - 1) g.q_start[g.B] = (int)min((int64_t)g.T, end);
    }
    const int back = max(0, s.have - s.need);
    const int64_t at = min((int64_t)0x7fffffff, count + given + block_sum(back, all, sums[1]) - back);
    given += all;
    for_pages(b, back, at | (int64_t)s.need << 32, [&](int of, int64_t x, int i) {
      int32_t* entry = g.table + of * g.ldt + (x >> 32) + i;
      const int64_t to = (x & 0xffffffff) + i;
      if (to < g.pages) g.free[to] = *entry;
      *entry = -1;
    });
    __syncthreads();
  }
  const int there = (int)min((int64_t)g.pages, count + given);  // the stack holds what was given back
  // pages that are taken
  int64_t wanted = 0;
  for (int b0 = 0; b0 < g.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    Asked s = b < g.B ? asked(g, b) : Asked{};
    if (b < g.B) fit(g, g.q_start[b], s);
    const int want = max(0, s.need - s.have);
    const int64_t end = wanted + block_sum(want, all, sums[2]);
    wanted += all;
    const bool granted = want == 0 || end <= there;
    const int64_t from = granted && want > 0 ? (there - 1 - (end - want)) | (int64_t)s.have << 32 : 0;
    for_pages(b, granted ? want : 0, from, [&](int of, int64_t x, int i) {
      g.table[of * g.ldt + (x >> 32) + i] = g.free[(x & 0xffffffff) - i];
    });
    if (granted && want > 0) atomicMax(&last_taken, (int)end);
    if (b < g.B) {
      g.owned[b] = granted ? s.need : s.have;
      g.status[b] = !s.fits ? -1 : granted ? 0 : want;
      g.kv_total[b] = s.fits && granted ? s.len + s.n : s.len;
    }
    __syncthreads();
  }
  if (tid == 0) *g.free_count = there - last_taken;
  if (!rows_too) return;
  for (int t = tid; t < g.T; t += kPlanThreads) {
    const int b = sequence_of(g.q_start, g.B, t), at = max(b, 0);
    write_row(g, t, b, g.q_start[at], g.q_start[at + 1]);
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
  if (a.B <= 256 && a.T <= 1024)
    plan_few_kernel<256><<<1, 256, 0, st>>>(a, rows_too);
  else if (a.B <= kPlanThreads)
    plan_few_kernel<kPlanThreads><<<1, kPlanThreads, 0, st>>>(a, rows_too);
  else
    plan_kernel<<<1, kPlanThreads, 0, st>>>(a, rows_too);
  if (!rows_too) plan_rows_kernel<<<(a.T + kRowThreads - 1) / kRowThreads, kRowThreads, 0, st>>>(a);
}

}  // namespace w4
