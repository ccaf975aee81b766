// logits_adjust: penalties for tokens that occur, biases and token masks on rows of f32 logits.
//
// With c the number of times that token v occurs behind the prompt of the row's request:
//   x = l > 0 ? l / r : l r  if v occurs at all (in the prompt or behind it), else l;
//   x = x - f c - p [c > 0];   x = x + bias(v);   x = -infinity if v is masked.
//
// A workgroup takes a slice of the vocabulary of one row.  Its counts lie in LDS, an integer per token of the slice: the
// whole history is read (from L2: the slices of a row read the same) and what falls into the slice is
// counted by LDS additions, whose order does not matter.  The slice's logits are on their way meanwhile, in registers.
// Biases follow at the end, on what the row then holds: a slice has few.  Of a token that a list names twice the later entry counts,
// found by a maximum of entry numbers where the counts were.
#include <algorithm>

#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int kThreads = 256;
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

template <int E, bool WIDE>
__global__ __launch_bounds__(kThreads) void logits_kernel(Rows a) {
  constexpr int SLICE = 4 * E * kThreads;
  __shared__ uint32_t counts[SLICE];
  const LogitArgs& g = a.g;
  const int m = blockIdx.x / a.slices, v0 = (blockIdx.x - m * a.slices) * SLICE, tid = threadIdx.x;
  const int here = min(SLICE, g.V - v0);
  const float* in = g.logits + m * g.ldl + v0;
  float* out = g.out + m * g.ldo + v0;
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
    for (int i = tid; i < len; i += kThreads) {
      const uint32_t at = (uint32_t)tokens[i] - (uint32_t)v0;
      if (at < (uint32_t)here) {
        if (i < prompt)
          atomicOr(&counts[at], kInPrompt);
        else
          atomicAdd(&counts[at], 1u);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = (e * kThreads + tid) * 4;
    if (i >= here) continue;
    if (count) {
      const u32x4 c = *reinterpret_cast<const u32x4*>(counts + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[e][k] = adjusted(x[e][k], c[k], r, f, p);
    }
    if (mask) {
      const uint32_t bits = mask[(v0 + i) >> 5] >> (i & 31);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[e][k] = bits >> k & 1 ? x[e][k] : -INFINITY;
    }
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

constexpr int kWide = 4;  // vector loads of a thread: a slice of 4096 logits

}  // namespace

int64_t logits_workgroups(const LogitArgs& g) { return (int64_t)g.M * ((g.V + (int64_t)kWide * 4 * kThreads - 1) / (kWide * 4 * kThreads)); }

void launch_logits(const LogitArgs& g, hipStream_t st) {
  const bool wide = ((uintptr_t)g.logits & 15) == 0 && ((uintptr_t)g.out & 15) == 0 && g.ldl % 4 == 0 && g.ldo % 4 == 0;
  Rows a{g, (int)((g.V + (int64_t)kWide * 4 * kThreads - 1) / (kWide * 4 * kThreads))};
  const int grid = g.M * a.slices;
  if (wide)
    logits_kernel<kWide, true><<<grid, kThreads, 0, st>>>(a);
  else
    logits_kernel<kWide, false><<<grid, kThreads, 0, st>>>(a);
}

}  // namespace w4
