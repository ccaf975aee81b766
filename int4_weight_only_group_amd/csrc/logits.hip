// logits_adjust: penalties for tokens that occur, biases and token masks on rows of f32 logits.
//
// With c the number of times that token v occurs behind the prompt of the row's request:
//   x = l > 0 ? l / r : l r  if v occurs at all (in the prompt or behind it), else l;
//   x = x - f c - p [c > 0];   x = x + bias(v);   x = -infinity if v is masked.
//
// A workgroup takes a slice of the vocabulary of one row.  How often a token occurs, and whether in the prompt, is counted in
// LDS, a word per token of the slice: the whole history is read (from L2: all slices read the same) and what falls into
// the slice is added up there, in any order.  The slice's logits are on their way meanwhile, in registers.  Biases follow at
// the end, on what the row then holds: a slice has few.  Of a token that a list names twice the later entry counts,
// found by a maximum of entry numbers where the counts were.
//
// Bound: HBM, each logit read and written once; for long histories the counting, a token in each slice.  So tokens are loaded
// eight deep, and the code is kept to few registers: waits of many waves cover each other.  (Rows of one request in a
// workgroup that counts once and takes them in turn: 100 rows of 4 requests, 262144 logits, up to 20001 tokens, 64, 68 and 60 us with
// 2, 4 and 6 rows against 59; 32 rows of 4 requests, 151936 logits, 15, 21 and 29 against 12.5: fewer workgroups, loads in turn.)
// Measured: those 64, with biases and masks for half of them, 20.4 us, 3.9 TB/s; with 10 tokens, at 262144 logits, 26.3, 5.1 TB/s;
// the 100 58, 3.7 TB/s; one of 151936 logits and 1570 tokens 4.4.
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int kThreads = 512;
constexpr uint32_t kInPrompt = 0x80000000u;

struct Rows {
  LogitArgs g;
  int slices;
};

__device__ __forceinline__ float adjusted(float x, uint32_t count, float r, float f, float p) {
  if (count == 0) return x;
  x = x > 0.f ? x / r : x * r;
  const int said = (int)(count & ~kInPrompt);
  if (said > 0) x = x - f * (float)said - p;
  return x;
}

// E: fours of logits of a thread; WIDE: rows of aligned fours
template <int E, bool WIDE>
__global__ __launch_bounds__(kThreads) void logits_kernel(Rows a) {
  constexpr int SLICE = 4 * E * kThreads;
  __shared__ __align__(16) uint32_t counts[SLICE];
  const LogitArgs& g = a.g;
  const int m = blockIdx.x / a.slices, v0 = (blockIdx.x - m * a.slices) * SLICE, tid = threadIdx.x;
  const int here = min(SLICE, g.V - v0);
  const float* in = g.logits + m * g.ldl + v0;
  float* out = g.out + m * g.ldo + v0;
  const bool in_place = g.out == g.logits;
  f32x4 x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = (e * kThreads + tid) * 4;
    if (WIDE && i + 4 <= here) {
      x[e] = *reinterpret_cast<const f32x4*>(in + i);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[e][k] = in[min(i + k, here - 1)];
    }
  }
  int req = g.request ? g.request[m] : m;
  if ((uint32_t)req >= (uint32_t)g.requests) req = -1;
  const int group = g.mask ? g.mask_row ? g.mask_row[m] : m : -1;
  const uint32_t* mask = (uint32_t)group < (uint32_t)g.masks ? g.mask + group * g.ld_mask : nullptr;
  const bool count = g.tokens && req >= 0;
  float r = 1.f, f = 0.f, p = 0.f;
  if (count) {
    if (g.repetition) r = g.repetition[req];
    if (g.frequency) f = g.frequency[req];
    if (g.presence) p = g.presence[req];
    for (int i = tid; i < SLICE / 4; i += kThreads) reinterpret_cast<u32x4*>(counts)[i] = u32x4{0, 0, 0, 0};
    __syncthreads();
    const int len = min(max(g.token_len[req], 0), g.max_tokens);
    const int prompt = g.prompt_len ? g.prompt_len[req] : 0;
    const int32_t* tokens = g.tokens + req * g.ld_tokens;
    constexpr int DEEP = 8;
    for (int i0 = 0; i0 < len; i0 += DEEP * kThreads) {
      uint32_t t[DEEP];
#pragma unroll
      for (int e = 0; e < DEEP; ++e) t[e] = (uint32_t)tokens[min(i0 + e * kThreads + tid, len - 1)];
#pragma unroll
      for (int e = 0; e < DEEP; ++e) {
        const int i = i0 + e * kThreads + tid;
        const uint32_t at = t[e] - (uint32_t)v0;  // of an id below 0: 2^31 - v0 at least, which is past the slice
        if (i < len && at < (uint32_t)here) {
          if (i < prompt)
            atomicOr(&counts[at], kInPrompt);
          else
            atomicAdd(&counts[at], 1u);
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = (e * kThreads + tid) * 4;
    if (i >= here) continue;
    bool same = in_place;  // nothing to write
    if (count) {
      const u32x4 c = *reinterpret_cast<const u32x4*>(counts + i);
      same &= (c[0] | c[1] | c[2] | c[3]) == 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) x[e][k] = adjusted(x[e][k], c[k], r, f, p);
    }
    if (mask) {
      const uint32_t bits = mask[(v0 + i) >> 5] >> (i & 31);
      same &= (bits & 15) == 15;
#pragma unroll
      for (int k = 0; k < 4; ++k) x[e][k] = bits >> k & 1 ? x[e][k] : -INFINITY;
    }
    if (same) continue;
    if (WIDE && i + 4 <= here) {
      *reinterpret_cast<f32x4*>(out + i) = x[e];
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < here) out[i + k] = x[e][k];
    }
  }
  if (!g.bias || req < 0) return;
  const int b0 = min(max(g.bias_start[req], 0), g.biases), b1 = min(max(g.bias_start[req + 1], b0), g.biases);
  if (b0 == b1) return;
  __syncthreads();  // the row is written, the counts are read
  auto place = [&](int i) { return (uint32_t)g.bias_id[i] - (uint32_t)v0; };
  for (int i = b0 + tid; i < b1; i += kThreads)
    if (place(i) < (uint32_t)here) counts[place(i)] = 0;
  __syncthreads();
  for (int i = b0 + tid; i < b1; i += kThreads)
    if (place(i) < (uint32_t)here) atomicMax(&counts[place(i)], (uint32_t)i + 1);
  __syncthreads();
  for (int i = b0 + tid; i < b1; i += kThreads) {
    const uint32_t at = place(i);
    if (at < (uint32_t)here && counts[at] == (uint32_t)i + 1)
      if (!mask || mask[(v0 + at) >> 5] >> (at & 31) & 1) out[at] += g.bias[i];
  }
}

int64_t workgroups(const LogitArgs& g, int e) { return g.M * ((g.V + (int64_t)e * 4 * kThreads - 1) / (e * 4 * kThreads)); }

// Slices of 2048, 4096 or 8192 logits: small ones where they fill a round of workgroups at most, since counting takes as long for
// any.  One row of 151936 4.4, 4.8, 5.9 us; 8 of them 5.3, 5.0, 5.7; 64 with 8191 tokens 26.7, 21.1, 20.4.
int fours(const LogitArgs& g) { return workgroups(g, 1) <= 512 ? 1 : workgroups(g, 2) <= 1024 ? 2 : 4; }

template <int E>
void launch_slices(const LogitArgs& g, hipStream_t st) {
  const bool wide = ((uintptr_t)g.logits & 15) == 0 && ((uintptr_t)g.out & 15) == 0 && g.ldl % 4 == 0 && g.ldo % 4 == 0;
  const int64_t n = workgroups(g, E);
  const Rows a{g, (int)(n / g.M)};
  if (wide)
    logits_kernel<E, true><<<(int)n, kThreads, 0, st>>>(a);
  else
    logits_kernel<E, false><<<(int)n, kThreads, 0, st>>>(a);
}

}  // namespace

int64_t logits_workgroups(const LogitArgs& g) { return workgroups(g, fours(g)); }

void launch_logits(const LogitArgs& g, hipStream_t st) {
  const int e = fours(g);
  if (e == 1)
    launch_slices<1>(g, st);
  else if (e == 2)
    launch_slices<2>(g, st);
  else
    launch_slices<4>(g, st);
}

}  // namespace w4
