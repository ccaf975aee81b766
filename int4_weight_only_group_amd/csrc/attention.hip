// attention_paged: softmax(scale q k^T) v of new tokens over a paged cache.
//
// Query i of a sequence with n new and L cached tokens stands at position p = L - n + i and sees
// the keys max(0, p + 1 - window) <= j <= p.  Keys are taken in blocks; m, the largest score so
// far, and l, the sum of exp(s - m), are kept in f32, and what was summed before is scaled by
// exp(m_old - m_new) whenever m grows:  out = sum_j exp(s_j - m) v_j / l.
#include <cmath>

#include "w4_internal.h"
#include "w4_kv.h"

namespace w4 {

namespace {

// One wave per (token, query head): 64 keys at a time, a key per lane for the scores and
// D/64 dims per lane for the sums over v.
__global__ __launch_bounds__(64) void attention_row_kernel(AttnArgs g) {
  __shared__ float qs[256];
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, D = g.c.dim;
  int b = 0, first = t, n = 1;
  if (g.q_start) {
    int lo = 0, hi = g.B;  // the last sequence that starts at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (g.q_start[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    first = g.q_start[b];
    n = min(g.q_start[b + 1], g.T) - first;
    if (t < first || t >= first + n) return;
  } else {
    if (t >= g.B) return;
    b = t;
  }
  const int64_t most = (int64_t)g.W * g.c.page_size;
  const int L = (int)max((int64_t)0, min((int64_t)g.kv_len[b], most));
  const int p = L - n + (t - first), end = p + 1;  // keys below `end`
  const int beg = g.window > 0 ? max(0, end - g.window) : 0;
  const uint16_t* q = g.q + (int64_t)t * g.ldq + (int64_t)h * D;
  for (int d = lane; d < D; d += 64) qs[d] = (float)__builtin_bit_cast(f16, q[d]);
  __syncthreads();
  const int kvh = h / (g.Hq / g.c.heads);
  const float ks = g.c.e4m3 && g.c.k_scale ? g.c.k_scale[kvh] : 1.f;
  const float vs = g.c.e4m3 && g.c.v_scale ? g.c.v_scale[kvh] : 1.f;
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  bool bad = false;
  for (int j0 = beg; j0 < end; j0 += 64) {
    const int j = j0 + lane;
    int64_t at = -1;
    if (j < end) {
      const int page = g.table[b * g.ldt + j / g.c.page_size];
      if (page < 0 || page >= g.c.pages) bad = true;
      else at = page * g.c.stride_page + kvh * g.c.stride_head + (j % g.c.page_size) * g.c.stride_token;
    }
    float s = -INFINITY;
    if (at >= 0) {
      float sum = 0.f;
      for (int d = 0; d < D; ++d) {
        const float k = g.c.e4m3
                            ? __builtin_amdgcn_cvt_f32_fp8(reinterpret_cast<const uint8_t*>(g.c.k)[at + d], 0)
                            : (float)reinterpret_cast<const f16*>(g.c.k)[at + d];
        sum += qs[d] * k;
      }
      s = sum * (g.scale * ks);
    }
    float mt = s;
    for (int x = 32; x; x >>= 1) mt = fmaxf(mt, __shfl_xor(mt, x));
    const float mn = fmaxf(m, mt), ms = mn == -INFINITY ? 0.f : mn;
    const float e = s == -INFINITY ? 0.f : expf(s - ms);
    float sum = e;
    for (int x = 32; x; x >>= 1) sum += __shfl_xor(sum, x);
    const float al = m == -INFINITY ? 0.f : expf(m - ms);
    l = l * al + sum;
    m = mn;
    for (int i = 0; i < 4; ++i) acc[i] *= al;
    for (int x = 0; x < 64 && j0 + x < end; ++x) {
      const float w = __shfl(e, x);
      const int64_t va = __shfl((long long)at, x);
      if (va < 0) continue;
      for (int i = 0; i < 4; ++i) {
        const int d = lane + 64 * i;
        if (d < D)
          acc[i] += w * (g.c.e4m3
                             ? __builtin_amdgcn_cvt_f32_fp8(reinterpret_cast<const uint8_t*>(g.c.v)[va + d], 0)
                             : (float)reinterpret_cast<const f16*>(g.c.v)[va + d]);
      }
    }
  }
  const float f = __any(bad) ? NAN : l == 0.f ? 0.f : vs / l;
  uint16_t* out = g.out + (int64_t)t * g.ldo + (int64_t)h * D;
  for (int i = 0; i < 4; ++i) {
    const int d = lane + 64 * i;
    if (d < D) out[d] = __builtin_bit_cast(uint16_t, (f16)(acc[i] * f));
  }
}

}  // namespace

size_t attention_ws_bytes(const AttnArgs&) { return 0; }

void launch_attention(const AttnArgs& a, void*, hipStream_t st) {
  attention_row_kernel<<<dim3(a.T, a.Hq), 64, 0, st>>>(a);
}

}  // namespace w4
