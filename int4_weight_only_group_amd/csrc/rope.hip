// rope_f16 and kv_append_rope: rotary positions, alone or on the way into a paged cache; norm_rope_f16 and
// kv_append_norm_rope: the same behind a norm of each query and key head.
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
// The norm.  x becomes x w / sqrt(mean(x^2) + eps) over the D dims of its head, before it turns.  A head's items lie on
// adjacent lanes, as many as the next power of two has, so that the squares of what the lanes hold anyway
// are summed by lane moves and x is read once.  Where R / 2 is no multiple of 8, pairs do not share chunks of 8 dims: a lane holds a
// chunk all the same, and takes the other halves of its pairs from LDS, where the lanes of its head leave their normed values.
//
// Bound: HBM for prompts (each element read once, written once), the launch and the chain of
// loads for a decode step.  So a thread's first elements, its token's slot and its head's scale
// are all on their way before the angles are formed.
// Measured: 8192 tokens of 16 + 2 + 2 heads of 128 dims, f32, into an f16 cache 23.7 us, 5.3 TB/s;
// 8191 of 16 heads of 80, f16, 10.1 us, 4.2 TB/s; one token 2.4 us.  With norms: 8191 tokens of 16 + 8 + 8 heads of 128 dims, f32, into an f16
// cache 40.0 us, 5.0 TB/s; 8191 of 16 heads of 128, f32, 18.7 (partly from the last-level cache); of 80, f16, interleaved, 17.5 (10 of a head's 16
// lanes hold dims); one token 4.5 in a replayed graph.  (Weights in LDS in place of registers: 43.1, 19.3, 18.8.)
#include "w4_internal.h"
#include "w4_kv.h"

namespace w4 {

namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;  // tokens of a workgroup, at most

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
  int per, n;           // items of a rotated head (norms: lanes, a power of two), of a token
  int items;            // norms: items of a rotated head
  const float* weight[2];  // norms: of q's and k's dims; nullptr: 1
  float eps, per_dim;      // norms: per_dim = 1 / D
  float per_n, per_head, per_chunks;  // 1 / n, 1 / per, 1 / (D / 8)
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
__device__ __forceinline__ f32x8 load8(const void* p, int64_t i) {
  if constexpr (F32) {
    const f32x4* q = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i);
    return __builtin_shufflevector(q[0], q[1], 0, 1, 2, 3, 4, 5, 6, 7);
  }
  return __builtin_convertvector(*reinterpret_cast<const f16x8*>(reinterpret_cast<const f16*>(p) + i), f32x8);
}

// RN to e4m3 of x / scale, saturated at 448 (NaN stays NaN)
__device__ __forceinline__ float e4m3_range(float x, float scale) {
  x = x / scale;
  x = x > 448.f ? 448.f : x;
  return x < -448.f ? -448.f : x;
}

__device__ __forceinline__ void store8(const Dst& d, int i, f32x8 v) {
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
    *reinterpret_cast<f16x8*>(reinterpret_cast<f16*>(d.p) + i) = __builtin_convertvector(v, f16x8);
  }
}

__device__ __forceinline__ void store1(const Dst& d, int i, float v) {
  if (d.e4m3)
    reinterpret_cast<uint8_t*>(d.p)[i] =
        (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_range(v, d.scale), 0.f, 0, false);
  else
    reinterpret_cast<f16*>(d.p)[i] = (f16)v;
}

// i / d for 0 <= i < 2^24 with r = 1 / d in f32: the product is off by less than one
__device__ __forceinline__ int divide(int i, int d, float r) {
  int q = (int)((float)i * r);
  const int rest = i - q * d;
  q += rest >= d;
  return q - (rest < 0);
}

enum Mode { kHalf, kInterleaved, kHalfOdd };

// Items of a head: kHalf (R/2 a multiple of 8): R/16 pairs of 8-dim chunks (both sides of the
// pairs in one thread, so y may be x), then the (D - R)/8 chunks that pass.  kInterleaved: D/8
// chunks (a chunk that R ends in passes its tail).  kHalfOdd (any other R): R/2 pairs and
// D - R single dims.  A v head is D/8 chunks that pass.
int items_of(int mode, int D, int R) {
  return mode == kHalf ? D / 8 - R / 16 : mode == kInterleaved ? D / 8 : D - R / 2;
}

struct Item {
  Dst d;
  int tl, item;  // token of the workgroup, item of the head
  bool rot;      // of a head that turns
  f32x8 a, b;
  f32x8 wa, wb;  // norms: their weights
};

// Sum over aligned groups of n lanes, a power of two up to 32, all of them active; every lane gets it.
__device__ __forceinline__ float lanes_sum(float v, int n) {
  if (n >= 2) v += dpp_f<0xB1>(v);   // quad_perm [1,0,3,2]
  if (n >= 4) v += dpp_f<0x4E>(v);   // quad_perm [2,3,0,1]
  if (n >= 8) v += dpp_f<0x141>(v);  // row_half_mirror
  if (n >= 16) v += dpp_f<0x140>(v);  // row_mirror
  if (n >= 32) v += __shfl_xor(v, 16);
  return v;
}

__device__ __forceinline__ float squares(const f32x8& x) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s += x[e] * x[e];
  return s;
}

// what an item's values are multiplied with for a head whose squares sum up to s
__device__ __forceinline__ float norm_of(const RopeArgs& g, float s) { return 1.f / sqrtf(s * g.per_dim + g.eps); }

template <bool F32, int MODE, bool NORM>
__device__ __forceinline__ void fetch(const RopeArgs& g, int i, int t0, Item& x) {
  const int half = g.R / 2, rot_heads = g.heads[0] + g.heads[1], n_rot = rot_heads * g.per;
  x.tl = divide(i, g.n, g.per_n);
  const int r = i - x.tl * g.n, t = t0 + x.tl;
  const int64_t slot = g.slots ? g.slots[t] : -1;
  x.rot = r < n_rot;
  int j = x.rot ? divide(r, g.per, g.per_head) : divide(r - n_rot, g.D / 8, g.per_chunks);
  x.item = x.rot ? r - j * g.per : r - n_rot - j * (g.D / 8);
  j += x.rot ? 0 : rot_heads;
  // the head: of q, k or v, where it is read and where it goes
  const int w = j < g.heads[0] ? 0 : j < rot_heads ? 1 : 2;
  const int h = j - (w > 0 ? g.heads[0] : 0) - (w > 1 ? g.heads[1] : 0);
  const void *q = g.src[0], *k = g.src[1], *v = g.src[2];
  const int64_t ldq = g.ld[0], ldk = g.ld[1], ldv = g.ld[2];
  const void* src = w == 0 ? q : w == 1 ? k : v;
  const int64_t at = (int64_t)t * (w == 0 ? ldq : w == 1 ? ldk : ldv) + (int64_t)h * g.D;
  if constexpr (NORM) {
    x.d.p = nullptr;
    x.a = 0.f, x.b = 0.f;
    // a lane past the head's items, or past the token's: it only takes part in the sum
    if (x.rot ? x.item >= g.items : w == 2 && h >= g.heads[2]) return;
  }
  const float* weight = nullptr;
  if constexpr (NORM) {
    const float *wq = g.weight[0], *wk = g.weight[1];
    weight = !x.rot ? nullptr : w == 0 ? wq : wk;
    x.wa = 1.f, x.wb = 1.f;
  }
  if (MODE == kHalfOdd && !NORM && x.rot) {
    if (x.item < half) x.a[0] = load1<F32>(src, at + x.item);
    x.b[0] = load1<F32>(src, at + x.item + half);
  } else {
    const bool pair = MODE == kHalf && x.rot && x.item < g.R / 16;
    if (MODE == kHalf && x.rot && !pair) x.item += g.R / 16;
    x.a = load8<F32>(src, at + x.item * 8);
    if (pair) x.b = load8<F32>(src, at + x.item * 8 + half);
    if (NORM && weight) {
      x.wa = load8<true>(weight, x.item * 8);
      if (pair) x.wb = load8<true>(weight, x.item * 8 + half);
    }
  }
  x.d.e4m3 = w > 0 && g.c.e4m3;
  x.d.scale = 1.f;
  x.d.p = nullptr;
  if (w == 0) {
    x.d.p = g.q_out + (int64_t)t * g.ldq_out + (int64_t)h * g.D;
  } else if (slot >= 0 && slot < (int64_t)g.c.pages * g.c.page_size) {
    const int page = (int)slot / g.c.page_size, off = (int)slot - page * g.c.page_size;
    const int64_t e = page * g.c.stride_page + h * g.c.stride_head + off * g.c.stride_token;
    const float *ks = g.c.k_scale, *vs = g.c.v_scale, *sc = w == 1 ? ks : vs;
    void *kc = g.c.k, *vc = g.c.v;
    if (x.d.e4m3 && sc) x.d.scale = sc[h];
    x.d.p = reinterpret_cast<uint8_t*>(w == 1 ? kc : vc) + (x.d.e4m3 ? e : 2 * e);
  }
}

template <bool F32, int MODE, bool NORM>
__device__ __forceinline__ void finish(const RopeArgs& g, const float2* turn, f32x8* staged, Item& x) {
  if constexpr (NORM) {
    const float f = norm_of(g, lanes_sum(squares(x.a) + squares(x.b), g.per));
    if (x.rot) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x.a[e] = x.a[e] * f * x.wa[e], x.b[e] = x.b[e] * f * x.wb[e];
    }
  }
  if (x.d.p == nullptr) return;
  const int half = g.R / 2;
  const float2* cs = turn + x.tl * half;
  if constexpr (MODE == kHalfOdd && NORM) {
    // all lanes of a head are in this wave, and here or not here together (a lane past the head's items holds none of its dims)
    const float* head = reinterpret_cast<const float*>(staged + (threadIdx.x & ~(g.per - 1)));
    if (x.rot) {
      staged[threadIdx.x] = x.a;
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = x.item * 8 + e;
        if (d >= g.R) break;
        const bool first = d < half;
        const float2 w = cs[first ? d : d - half];
        const float other = head[first ? d + half : d - half];
        x.a[e] = x.a[e] * w.x + (first ? -other : other) * w.y;
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();  // read before the next heads are left there
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    store8(x.d, x.item * 8, x.a);
    return;
  }
  if (MODE == kHalfOdd && x.rot) {
    if (x.item < half) {
      const float2 w = cs[x.item];
      store1(x.d, x.item, x.a[0] * w.x - x.b[0] * w.y);
      store1(x.d, x.item + half, x.b[0] * w.x + x.a[0] * w.y);
    } else {
      store1(x.d, x.item + half, x.b[0]);
    }
    return;
  }
  const int c0 = x.item * 8;
  if (MODE == kHalf && x.rot && x.item < g.R / 16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 w = cs[c0 + e];
      const float a = x.a[e];
      x.a[e] = a * w.x - x.b[e] * w.y;
      x.b[e] = x.b[e] * w.x + a * w.y;
    }
    store8(x.d, c0 + half, x.b);
  }
  if (MODE == kInterleaved && x.rot) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (c0 + 2 * e >= g.R) break;
      const float2 w = cs[c0 / 2 + e];
      const float a = x.a[2 * e];
      x.a[2 * e] = a * w.x - x.a[2 * e + 1] * w.y;
      x.a[2 * e + 1] = x.a[2 * e + 1] * w.x + a * w.y;
    }
  }
  store8(x.d, c0, x.a);
}

template <bool F32, int MODE, bool NORM>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs g) {
  __shared__ float2 turn[kMaxTokens * 128];  // [token][pair]: mscale (cos, sin)
  __shared__ f32x8 staged[NORM && MODE == kHalfOdd ? kThreads : 1];  // of each thread: its chunk (as vectors, for their alignment)
  const int t0 = blockIdx.x * g.tokens, nt = min(g.tokens, g.T - t0), half = g.R / 2, n = nt * g.n;
  Item x{};
  int i = threadIdx.x;
  if (i < n) fetch<F32, MODE, NORM>(g, i, t0, x);
  for (int k = threadIdx.x; k < nt * half; k += kThreads) {
    const int tl = k / half, p = k - tl * half;
    double a = (double)g.pos[t0 + tl] * (double)g.freq[p] * 0.15915494309189535;  // turns
    a -= rint(a);
    float s, c;
    sincospif(2.f * (float)a, &s, &c);
    turn[k] = make_float2(c * g.mscale, s * g.mscale * g.sign);
  }
  __syncthreads();
  while (i < n) {
    finish<F32, MODE, NORM>(g, turn, staged, x);
    i += kThreads;
    if (i < n) fetch<F32, MODE, NORM>(g, i, t0, x);
  }
}

void launch(RopeArgs& g, bool f32, bool interleaved, bool norm, hipStream_t st) {
  const int mode = interleaved ? kInterleaved : (g.R / 2) % 8 == 0 ? kHalf : kHalfOdd;
  g.per = g.items = norm && mode == kHalfOdd ? g.D / 8 : items_of(mode, g.D, g.R);
  if (norm)
    for (g.per = 1; g.per < g.items;) g.per *= 2;
  g.n = (g.heads[0] + g.heads[1]) * g.per + g.heads[2] * (g.D / 8);
  if (norm) g.n = (g.n + g.per - 1) / g.per * g.per;  // the groups of the next token's lanes are aligned too
  g.per_n = 1.f / g.n, g.per_head = 1.f / g.per, g.per_chunks = 1.f / (g.D / 8);
  // Where tokens are plenty (8 workgroups a CU stay), narrow ones share a workgroup as long as its threads go about
  // once over their items: 8191 x 16 x 80 of f16 (160 items a token) take 10.5 us two at a time, 12.5 one at a time;
  // 8192 x 20 x 128 of f32 into the cache (176 items) 24.7 and 23.3.  With a norm, up to twice: 8191 x 16 x 128 of f32 (128
  // lanes a token) 19.4 two at a time, 21.2 one at a time; 8191 x 16 x 80 of f16 (256 lanes) 17.7 and 19.1.
  g.tokens = 1;
  while (g.tokens < kMaxTokens && g.n * g.tokens * 2 <= kThreads * (norm ? 8 : 5) / 4 && g.T / g.tokens > 8 * 256) g.tokens *= 2;
  const int grid = (g.T + g.tokens - 1) / g.tokens;
#define W4_ROPE(F, M)                                               \
  if (norm)                                                         \
    rope_kernel<F, M, true><<<grid, kThreads, 0, st>>>(g);          \
  else                                                              \
    rope_kernel<F, M, false><<<grid, kThreads, 0, st>>>(g)
  if (f32) {
    if (mode == kHalf) {
      W4_ROPE(true, kHalf);
    } else if (mode == kInterleaved) {
      W4_ROPE(true, kInterleaved);
    } else {
      W4_ROPE(true, kHalfOdd);
    }
  } else {
    if (mode == kHalf) {
      W4_ROPE(false, kHalf);
    } else if (mode == kInterleaved) {
      W4_ROPE(false, kInterleaved);
    } else {
      W4_ROPE(false, kHalfOdd);
    }
  }
#undef W4_ROPE
}

}  // namespace

void launch_rope(const void* x, bool f32, int64_t ldx, const int32_t* pos, const float* freq, uint16_t* y, int64_t ldy,
                 int T, int H, int D, int R, bool interleaved, bool inverse, float mscale, const HeadNorm* norm,
                 hipStream_t st) {
  RopeArgs g{};
  g.src[0] = x, g.ld[0] = ldx, g.heads[0] = H;
  g.q_out = y, g.ldq_out = ldy;
  g.pos = pos, g.freq = freq, g.mscale = mscale, g.sign = inverse ? -1.f : 1.f;
  g.T = T, g.D = D, g.R = R;
  if (norm) g.weight[0] = norm->q, g.eps = norm->eps, g.per_dim = 1.f / D;
  launch(g, f32, interleaved, norm != nullptr, st);
}

void launch_kv_append(const void* q, int64_t ldq, uint16_t* q_out, int64_t ldqo, int Hq, const void* k, int64_t ldk,
                      const void* v, int64_t ldv, bool f32, const KvCache& c, const int64_t* slots, const int32_t* pos,
                      const float* freq, int T, int R, bool interleaved, float mscale, const HeadNorm* norm,
                      hipStream_t st) {
  RopeArgs g{};
  g.src[0] = q, g.ld[0] = ldq, g.heads[0] = q ? Hq : 0;
  g.src[1] = k, g.ld[1] = ldk, g.heads[1] = c.heads;
  g.src[2] = v, g.ld[2] = ldv, g.heads[2] = c.heads;
  g.q_out = q_out, g.ldq_out = ldqo;
  g.c = c, g.slots = slots, g.pos = pos, g.freq = freq, g.mscale = mscale, g.sign = 1.f;
  g.T = T, g.D = c.dim, g.R = R;
  if (norm) g.weight[0] = norm->q, g.weight[1] = norm->k, g.eps = norm->eps, g.per_dim = 1.f / c.dim;
  launch(g, f32, interleaved, norm != nullptr, st);
}

}  // namespace w4
