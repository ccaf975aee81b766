// rope_f16 and kv_append_rope: rotary positions, alone or on the way into a paged cache.
//
// Mathematics.  Pair i of a head's first R dims is the complex number (a, b): dims (i, i + R/2)
// in the half layout, (2i, 2i + 1) in the interleaved one.  It is multiplied by
// mscale * exp(+-i theta), theta = pos * freq[i]:  (a c - b s, b c + a s).  Dims from R on pass.
//
// The angle.  At position 10^5 a product in f32 is off by 4e-3 radians, so pos * freq is formed
// in f64, in turns (theta / 2 pi), and reduced to [-1/2, 1/2] there; the reduced angle is good
// to 1e-10 turns at 10^6 positions, and only then goes to f32 for sincospif.  The f64 work is
// one pair per thread (R/2 per token, shared by all heads through LDS), so it costs little.
//
// Bound: HBM for prompts (each element read once, written once), launch latency for a decode
// step.
#include "w4_internal.h"
#include "w4_kv.h"

namespace w4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens of a workgroup

struct RopeArgs {
  const void* src[3];  // q, k, v rows (heads of one token are contiguous)
  int64_t ld[3];       // elements between tokens
  int heads[3];
  uint16_t* q_out;
  int64_t ldq_out;
  KvCache c;
  const int64_t* slots;
  const int32_t* pos;
  const float* freq;
  float mscale, sign;
  int T, D, R, tokens;  // tokens: of each workgroup
};

// Where 8 (or 1) output values of a head go: f16 for q and an f16 cache, e4m3 with the head's
// scale otherwise; nothing when the token's slot is outside the cache.
struct Dst {
  void* p;  // the head's first element, or nullptr
  bool e4m3;
  float scale;
};

template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (F32) return reinterpret_cast<const float*>(p)[i];
  return (float)reinterpret_cast<const f16*>(p)[i];
}

template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (F32) {
    const f32x4* q = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i);
    const f32x4 lo = q[0], hi = q[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = lo[e], v[4 + e] = hi[e];
  } else {
    const f16x8 h = *reinterpret_cast<const f16x8*>(reinterpret_cast<const f16*>(p) + i);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)h[e];
  }
}

// RN to e4m3 of x / scale, saturated at 448 (NaN stays NaN)
__device__ __forceinline__ float e4m3_range(float x, float scale) {
  x = x / scale;
  x = x > 448.f ? 448.f : x;
  return x < -448.f ? -448.f : x;
}

__device__ __forceinline__ void store8(const Dst& d, int i, const float (&v)[8]) {
  if (d.e4m3) {
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = e4m3_range(v[e], d.scale);
    u32x2 w = {0, 0};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      int x = __builtin_amdgcn_cvt_pk_fp8_f32(s[4 * e], s[4 * e + 1], 0, false);
      x = __builtin_amdgcn_cvt_pk_fp8_f32(s[4 * e + 2], s[4 * e + 3], x, true);
      w[e] = (uint32_t)x;
    }
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint8_t*>(d.p) + i) = w;
  } else {
    f16x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = (f16)v[e];
    *reinterpret_cast<f16x8*>(reinterpret_cast<f16*>(d.p) + i) = h;
  }
}

__device__ __forceinline__ void store1(const Dst& d, int i, float v) {
  if (d.e4m3)
    reinterpret_cast<uint8_t*>(d.p)[i] =
        (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_range(v, d.scale), 0.f, 0, false);
  else
    reinterpret_cast<f16*>(d.p)[i] = (f16)v;
}

// A token's head j (q heads, then k, then v): its source row and where it goes.
__device__ __forceinline__ Dst head_of(const RopeArgs& g, int t, int j, int64_t slot, const void*& src, int64_t& at) {
  const int w = j < g.heads[0] ? 0 : j < g.heads[0] + g.heads[1] ? 1 : 2;
  const int h = j - (w > 0 ? g.heads[0] : 0) - (w > 1 ? g.heads[1] : 0);
  src = w == 0 ? g.src[0] : w == 1 ? g.src[1] : g.src[2];
  at = (int64_t)t * (w == 0 ? g.ld[0] : w == 1 ? g.ld[1] : g.ld[2]) + (int64_t)h * g.D;
  if (w == 0) return {g.q_out + (int64_t)t * g.ldq_out + (int64_t)h * g.D, false, 1.f};
  if (slot < 0 || slot >= (int64_t)g.c.pages * g.c.page_size) return {nullptr, false, 1.f};
  const int page = (int)slot / g.c.page_size, off = (int)slot - page * g.c.page_size;
  const int64_t e = page * g.c.stride_page + h * g.c.stride_head + off * g.c.stride_token;
  void* base = w == 1 ? g.c.k : g.c.v;
  if (!g.c.e4m3) return {reinterpret_cast<f16*>(base) + e, false, 1.f};
  const float* sc = w == 1 ? g.c.k_scale : g.c.v_scale;
  return {reinterpret_cast<uint8_t*>(base) + e, true, sc ? sc[h] : 1.f};
}

enum Mode { kHalf, kInterleaved, kHalfOdd };

// Items of a head: kHalf (R/2 a multiple of 8): R/16 pairs of 8-dim chunks (both sides of the
// pairs in one thread, so y may be x), then the (D - R)/8 chunks that pass.  kInterleaved: D/8
// chunks (a chunk that R ends in passes its tail).  kHalfOdd (any other R): R/2 pairs and
// D - R single dims.  A v head is D/8 chunks that pass.
template <bool F32, int MODE>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs g) {
  __shared__ float2 turn[kMaxTokens * 128];  // [token][pair]: mscale (cos, sin)
  const int t0 = blockIdx.x * g.tokens, nt = min(g.tokens, g.T - t0), half = g.R / 2;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tl = i / half, p = i - tl * half;
    double a = (double)g.pos[t0 + tl] * (double)g.freq[p] * 0.15915494309189535;  // turns
    a -= rint(a);
    float s, c;
    sincospif(2.f * (float)a, &s, &c);
    turn[tl * half + p] = make_float2(c * g.mscale, s * g.mscale * g.sign);
  }
  __syncthreads();
  const int rot_heads = g.heads[0] + g.heads[1];
  const int per = MODE == kHalf ? g.D / 8 - g.R / 16 : MODE == kInterleaved ? g.D / 8 : g.D - half;
  const int n_rot = rot_heads * per, n = n_rot + g.heads[2] * (g.D / 8);
  for (int i = threadIdx.x; i < nt * n; i += kThreads) {
    const int tl = i / n, r = i - tl * n, t = t0 + tl;
    const bool rot = r < n_rot;
    const int j = rot ? r / per : rot_heads + (r - n_rot) / (g.D / 8);
    const int item = rot ? r - j * per : (r - n_rot) % (g.D / 8);
    const void* src;
    int64_t at;
    const Dst d = head_of(g, t, j, g.slots ? g.slots[t] : -1, src, at);
    if (d.p == nullptr) continue;
    const float2* cs = turn + tl * half;
    if (MODE == kHalfOdd && rot) {
      if (item < half) {
        const float a = load1<F32>(src, at + item), b = load1<F32>(src, at + item + half);
        const float2 w = cs[item];
        store1(d, item, a * w.x - b * w.y);
        store1(d, item + half, b * w.x + a * w.y);
      } else {
        store1(d, item + half, load1<F32>(src, at + item + half));
      }
      continue;
    }
    if (MODE == kHalf && rot && item < g.R / 16) {
      float a[8], b[8];
      load8<F32>(src, at + item * 8, a);
      load8<F32>(src, at + item * 8 + half, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 w = cs[item * 8 + e];
        const float x = a[e];
        a[e] = x * w.x - b[e] * w.y;
        b[e] = b[e] * w.x + x * w.y;
      }
      store8(d, item * 8, a);
      store8(d, item * 8 + half, b);
      continue;
    }
    const int c0 = (MODE == kHalf && rot ? item + g.R / 16 : item) * 8;
    float a[8];
    load8<F32>(src, at + c0, a);
    if (MODE == kInterleaved && rot) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (c0 + 2 * e >= g.R) break;
        const float2 w = cs[c0 / 2 + e];
        const float x = a[2 * e];
        a[2 * e] = x * w.x - a[2 * e + 1] * w.y;
        a[2 * e + 1] = a[2 * e + 1] * w.x + x * w.y;
      }
    }
    store8(d, c0, a);
  }
}

void launch(RopeArgs& g, bool f32, bool interleaved, hipStream_t st) {
  const int mode = interleaved ? kInterleaved : (g.R / 2) % 8 == 0 ? kHalf : kHalfOdd;
  g.tokens = 1;
  const int grid = (g.T + g.tokens - 1) / g.tokens;
#define W4_ROPE(F, M) rope_kernel<F, M><<<grid, kThreads, 0, st>>>(g)
  if (f32) {
    if (mode == kHalf) W4_ROPE(true, kHalf);
    else if (mode == kInterleaved) W4_ROPE(true, kInterleaved);
    else W4_ROPE(true, kHalfOdd);
  } else {
    if (mode == kHalf) W4_ROPE(false, kHalf);
    else if (mode == kInterleaved) W4_ROPE(false, kInterleaved);
    else W4_ROPE(false, kHalfOdd);
  }
#undef W4_ROPE
}

}  // namespace

void launch_rope(const void* x, bool f32, int64_t ldx, const int32_t* pos, const float* freq, uint16_t* y, int64_t ldy,
                 int T, int H, int D, int R, bool interleaved, bool inverse, float mscale, hipStream_t st) {
  RopeArgs g{};
  g.src[0] = x, g.ld[0] = ldx, g.heads[0] = H;
  g.q_out = y, g.ldq_out = ldy;
  g.pos = pos, g.freq = freq, g.mscale = mscale, g.sign = inverse ? -1.f : 1.f;
  g.T = T, g.D = D, g.R = R;
  launch(g, f32, interleaved, st);
}

void launch_kv_append(const void* q, int64_t ldq, uint16_t* q_out, int64_t ldqo, int Hq, const void* k, int64_t ldk,
                      const void* v, int64_t ldv, bool f32, const KvCache& c, const int64_t* slots, const int32_t* pos,
                      const float* freq, int T, int R, bool interleaved, float mscale, hipStream_t st) {
  RopeArgs g{};
  g.src[0] = q, g.ld[0] = ldq, g.heads[0] = q ? Hq : 0;
  g.src[1] = k, g.ld[1] = ldk, g.heads[1] = c.heads;
  g.src[2] = v, g.ld[2] = ldv, g.heads[2] = c.heads;
  g.q_out = q_out, g.ldq_out = ldqo;
  g.c = c, g.slots = slots, g.pos = pos, g.freq = freq, g.mscale = mscale, g.sign = 1.f;
  g.T = T, g.D = c.dim, g.R = R;
  launch(g, f32, interleaved, st);
}

}  // namespace w4
