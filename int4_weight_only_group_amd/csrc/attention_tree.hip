// attention_paged_tree: attention of drafted tokens that form trees.  A row sees the cached tokens before the new
// ones and, of these, those whose bits are set in its mask.  The mathematics, the kernel for at most 16 rows and the one for
// many are attention_paged's (attention_core.h): tiles of old keys are seen whole, edge tiles take the bits.
//
// Between them, the kernel here: 17 to 64 or 96 rows (tree_most()).  Bound: the waits of a turn, at two waves a SIMD; for the case below
// memory gives 3.0 TB/s of 5.1, and the matrix cores are 13 % busy, the VALU 35: with one buffer K and V have half a turn each to
// arrive.  For one short sequence: latencies one after another, since the first K and V are asked for when the queries and masks are in LDS
// (8 tokens of 8 heads after 1562: 12.6 us, where the kernel for few rows takes 6.5 for as many keys).  Waves take 32-key tiles in LDS of
// their own, as in the kernel for few rows and without barriers, and multiply each with up to four blocks of 16 rows (two at 256 dims), so
// that an operand from K or V serves them all; the queries are in LDS, once per workgroup; two waves of a SIMD cover each other's
// waits.  Tiles that all rows see whole have a loop of their own: with the masks in it the sums of 64 rows do not fit the registers, and what
// is reloaded from scratch waits for every tile in flight (172 us against 58 for the case below).
// A weight is one f16, as in the kernel for many rows: the result's error is 2.5e-4 to 2.9e-4 of its norm, where its own rounding to f16
// is 2.1e-4.  Two f16 a weight, as for few rows, make it 2.1e-4 here too and take their time though the matrix cores are 13 % busy, since a
// wave's splitting and second products stand between its loads: with the join 70.0 us against 60.6 for that case, 53.1 against 47.0 for
// 64 dims in f16, 15.8 against 15.2 for the 8 tokens, 1 % more at 256 dims; in the kernel for many rows 8 to 35 % more (2 sequences of
// 256 tokens, 64 heads on 8: 236 against 175).
// Measured, 16 heads on 8: 16 sequences of 301 to 8192 keys, 7 to 48 tokens (up to 96 rows, two tiles) each, 128 dims, e4m3: 51.5 us and
// 7.8 for the join; 155 MB read for 145, as the second tile's keys come from caches mostly.  With the join: 64 dims 47 from f16, 45 from
// e4m3; 7 to 24 tokens of 256 dims 88 from e4m3, 132 from f16.
#include "attention_core.h"

namespace w4 {

namespace {

template <int DP, bool FP8>
__global__ __launch_bounds__((64 * tree_waves<DP, FP8>()), (tree_per_cu<DP, FP8>() * tree_waves<DP, FP8>() / 4)) void attention_tree_kernel(Plan p) {
  constexpr int NW = tree_waves<DP, FP8>(), KT = kFewKeys, ES = FP8 ? 1 : 2, ROWB = DP * ES;
  constexpr int TILE = few_tile<DP, FP8>(), NB = tree_buffers<DP, FP8>(), RT = tree_blocks<DP>(), ROWS = 16 * RT;
  constexpr int STEPS = DP / 32, DB = DP / 16;
  extern __shared__ __align__(16) unsigned char lds[];
  __shared__ float join[NW][ROWS][2];  // m and l; then what a wave's sums are multiplied with
  __shared__ float row_f[ROWS];
  __shared__ int row_lo[ROWS], row_any[ROWS];
  const AttnArgs& g = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kvh = blockIdx.x % g.c.heads, part = blockIdx.x / g.c.heads;
  const DealtTile d = deal_tiles<NW, KT, KT * NW>(p, part, lds);
  if (d.b < 0) return;
  auto scalar = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  const int b = scalar(d.b), tile = scalar(d.tile), index = scalar(d.index), count = scalar(d.count);
  const Seq s = {scalar(d.s.first), scalar(d.s.n), scalar(d.s.len)};
  const Keys k = keys_of<true>(p, s, 0, 0, KT, KT, KT);
  const int per = ((k.hi - k.lo + count - 1) / count + KT * NW - 1) / (KT * NW) * (KT * NW);
  const int k0 = min(k.hi, k.lo + index * per), k1 = min(k.hi, k0 + per);
  const int tiles = (k1 - k0 + KT - 1) / KT;
  const int mine = tiles > wave ? (tiles - wave + NW - 1) / NW : 0;
  const int D = g.c.dim, r0 = tile * ROWS, rows = min(s.n * p.G - r0, ROWS);
  if (p.part && kvh == 0 && index == 0 && threadIdx.x == 0) p.head[scalar(d.slot)] = {scalar(d.first), count, b, tile};

  WaveTiles<DP, FP8, NW, NB> keys(p, lds, b, kvh, k0, k1, lane, wave);
  constexpr std::false_type K_{};
  constexpr std::true_type V_{};
  // the keys that all rows see: [all0, all1)
  const int all1 = s.len - s.n, all0 = g.window ? s.len - g.window : 0;
  keys.whole_first(all0, all1, mine);
  if (mine > 0) {
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) keys.fetch_ids(i);
  }

  // the queries, zeros past the rows and dims; 16-byte chunk x of row r lies at x ^ k_swz(r)
  unsigned char* q_lds = lds + NW * tree_wave_lds<DP, FP8>();
  for (int i = threadIdx.x; i < ROWS * (DP / 8); i += 64 * NW) {
    const int r = i / (DP / 8), x = i % (DP / 8), at = r0 + min(r, rows - 1), tk = divide(at, p.group);
    f16x8 v = {};
    if (r < rows && 8 * x < D)
      v = *reinterpret_cast<const f16x8*>(g.q + (int64_t)(s.first + tk) * g.ldq + (int64_t)(kvh * p.G + at - tk * p.G) * D + 8 * x);
    *reinterpret_cast<f16x8*>(q_lds + r * DP * 2 + ((x ^ k_swz<DP>(r)) * 16)) = v;
  }
  const int row = lane & 15, grp = lane >> 4;
  // the rows' masks (the words that count), what they see of the old keys, whether they see any
  uint64_t* words = reinterpret_cast<uint64_t*>(q_lds + ROWS * DP * 2);
  for (int r = threadIdx.x; r < ROWS; r += 64 * NW) {
    const TreeRow tree = tree_row(g, s, divide(r0 + min(r, rows - 1), p.group));
    row_lo[r] = tree.lo, row_any[r] = tree.any;
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w) words[r * kTreeWords + w] = 64 * w < tree.n ? tree.bits[w] : 0;
  }
  auto sees_of = [&](int rt, int j0) W4_INLINE {
    TreeRow tree;
    tree.bits = words + (16 * rt + row) * kTreeWords;
    tree.base = s.len - s.n, tree.lo = row_lo[16 * rt + row], tree.n = min(s.n, 64 * kTreeWords);
    return tree_sees(tree, j0);
  };
  const float c = FP8 && g.c.k_scale ? p.c * g.c.k_scale[kvh] : p.c;
  keys.places();
  // Q^T operand of step t: 16-byte chunk 4 t + grp; e4m3: a 16-byte chunk of K feeds two steps, so 8 (t / 2) + 2 grp + t % 2.
  // Four steps go over 256 bytes, so that a further four are a constant away.
  constexpr int QA = STEPS < 4 ? STEPS : 4;
  uint32_t q_at[QA];
#pragma unroll
  for (int t = 0; t < QA; ++t) {
    const int x = FP8 ? 8 * (t / 2) + 2 * grp + (t & 1) : 4 * t + grp;
    q_at[t] = (uint32_t)(uintptr_t)(lds_void_t*)q_lds + row * DP * 2 + ((x ^ k_swz<DP>(row)) * 16);
  }
  __syncthreads();  // the queries are there

  if (mine > 0) {
    wait_vm<0>();
#pragma unroll
    for (int i = 0; i < NB; ++i)
      if (i < mine) keys.fetch(i, K_), keys.fetch(i, V_);
  }
  float m[RT], l[RT];
  f32x4 acc[RT][DB];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = -INFINITY, l[rt] = 0.f;
#pragma unroll
    for (int i = 0; i < DB; ++i) acc[rt][i] = {0.f, 0.f, 0.f, 0.f};
  }
  // What is waited for is followed by V of the same tile and the tiles of NB - 1 further turns (and some page numbers, so that this
  // waits for a little more), if there are as many.
  constexpr int BEHIND = (NB - 1) * 2 * keys.NI;
  auto k_there = [&](int i) W4_INLINE {
    if (NB == 1 || i + NB <= mine) wait_vm<BEHIND + keys.NI>();
    else wait_vm<0>();
  };
  auto v_there = [&](int i) W4_INLINE {
    if (i + NB < mine) wait_vm<BEHIND + keys.NI + 1>();
    else wait_vm<0>();
  };
  auto next_k = [&](int i) W4_INLINE {  // K of turn i has been read
    if (i + NB < mine) {
      wait_lds();
      keys.fetch_ids(i + 2 * NB);
      keys.fetch(i + NB, K_);
    }
  };
  auto next_v = [&](int i) W4_INLINE {
    if (i + NB < mine) {
      wait_lds();
      keys.fetch(i + NB, V_);
    }
  };
  // weights of a block's 32 keys (scores in units of log 2), moving its m, l and sums if need be
  auto weigh = [&](f32x4 (&sc)[2], int rt) W4_INLINE {
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(sc[0][e], sc[1][e]));
    if (__any(above(top, m[rt]))) {
      const float mn = moved(across<true>(top, fmax2), m[rt]);
      const float f = m[rt] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[rt] - mn);
      l[rt] *= f;
#pragma unroll
      for (int i = 0; i < DB; ++i) acc[rt][i] *= f;
      m[rt] = mn;
    }
    const float ms = m[rt] == -INFINITY ? 0.f : m[rt];
    f16x8 w;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * kb + e] = (f16)__builtin_amdgcn_exp2f(sc[kb][e] - ms);
    // l sums the weights as rounded, which are the ones that multiply v
    const u32x4 bits = __builtin_bit_cast(u32x4, w);
    const hf16x2 ones = {(__fp16)1.f, (__fp16)1.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t two = bits[e];
      l[rt] = __builtin_amdgcn_fdot2(__builtin_bit_cast(hf16x2, two), ones, l[rt], false);
    }
    return w;
  };
  auto q_frag = [&](int rt, int st) W4_INLINE {
    return *reinterpret_cast<const lds_f16x8*>(q_at[st % QA] + st / QA * 256 + rt * 16 * DP * 2);
  };
  // f(st, operands of keys 0 .. 15 and 16 .. 31) for each step
  auto over_k = [&](uint32_t buf, auto f) W4_INLINE {
#pragma unroll
    for (int x = 0; x < keys.KA; ++x) {
      const uint32_t at = keys.k_at[x] + buf;
      if constexpr (FP8) {
        const u32x4 a = *reinterpret_cast<const lds_u32x4*>(at), e = *reinterpret_cast<const lds_u32x4*>(at + 16 * ROWB);
        f(2 * x, widen8(a[0], a[1]), widen8(e[0], e[1]));
        f(2 * x + 1, widen8(a[2], a[3]), widen8(e[2], e[3]));
      } else {
        const f16x8 a = *reinterpret_cast<const lds_f16x8*>(at), e = *reinterpret_cast<const lds_f16x8*>(at + 16 * ROWB);
        f(x, a, e);
      }
    }
  };
  // blocks: of 16 rows that there are
  auto go = [&](auto blocks) W4_INLINE {
    constexpr int BL = decltype(blocks)::value;
    int i = 0;
    for (; i < keys.whole; ++i) {  // tiles that all rows see whole
      const uint32_t buf = keys.buffer(i);
      k_there(i);
      f32x4 sc[BL][2];
#pragma unroll
      for (int rt = 0; rt < BL; ++rt) sc[rt][0] = sc[rt][1] = {0.f, 0.f, 0.f, 0.f};
      over_k(buf, [&](int st, const f16x8& k_0, const f16x8& k_1) W4_INLINE {
#pragma unroll
        for (int rt = 0; rt < BL; ++rt) {
          const f16x8 q = q_frag(rt, st);
          sc[rt][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_0, q, sc[rt][0], 0, 0, 0);
          sc[rt][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_1, q, sc[rt][1], 0, 0, 0);
        }
      });
      next_k(i);
      f16x8 w[BL];
#pragma unroll
      for (int rt = 0; rt < BL; ++rt) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[rt][kb][e] = score(sc[rt][kb][e], c);
        w[rt] = weigh(sc[rt], rt);
      }
      v_there(i);
#pragma unroll
      for (int x = 0; x < DB; ++x) {
        const f16x8 v = keys.v_frag(x, buf);
#pragma unroll
        for (int rt = 0; rt < BL; ++rt) acc[rt][x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w[rt], acc[rt][x], 0, 0, 0);
      }
      next_v(i);
    }
    for (; i < mine; ++i) {  // tiles that some row does not see whole, a block of rows after another
      const uint32_t buf = keys.buffer(i);
      const int j0 = keys.first_key(i);
      k_there(i);
      f16x8 w[BL];
#pragma unroll
      for (int rt = 0; rt < BL; ++rt) {
        f32x4 sc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const uint32_t sees = sees_of(rt, j0);
        w[rt] = f16x8{};
        if (!__any(sees != 0)) continue;
        over_k(buf, [&](int st, const f16x8& k_0, const f16x8& k_1) W4_INLINE {
          const f16x8 q = q_frag(rt, st);
          sc[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_0, q, sc[0], 0, 0, 0);
          sc[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_1, q, sc[1], 0, 0, 0);
        });
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int e = 0; e < 4; ++e)  // key j0 + 16 kb + 4 grp + e of row 16 rt + lane % 16
            sc[kb][e] = sees >> (16 * kb + 4 * grp + e) & 1 ? score(sc[kb][e], c) : -INFINITY;
        w[rt] = weigh(sc, rt);
      }
      next_k(i);
      v_there(i);
      uint32_t odd = 0;
#pragma unroll
      for (int x = 0; x < DB; ++x) {
        const f16x8 v = finite(keys.v_frag(x, buf), odd);
#pragma unroll
        for (int rt = 0; rt < BL; ++rt) acc[rt][x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w[rt], acc[rt][x], 0, 0, 0);
      }
      if (__any(odd != 0)) {
#pragma unroll
        for (int rt = 0; rt < BL; ++rt) {
          const uint32_t sees = sees_of(rt, j0);
#pragma unroll 1
          for (int r = 0; r < KT; ++r) {
            const bool see = (sees >> r & 1) != 0;
#pragma unroll
            for (int x = 0; x < DB; ++x) {
              const int byte = (16 * x + 4 * grp) * ES;
              const uint32_t at = keys.vt + buf + r * ROWB + ((byte / 16) ^ v_swz_few<ROWB, FP8>(r)) * 16 + byte % 16;
              f16x4 v;
              if constexpr (FP8) {
                const f16x8 y = widen8(*reinterpret_cast<const lds_i32*>(at), 0);
                v = __builtin_shufflevector(y, y, 0, 1, 2, 3);
              } else {
                v = *reinterpret_cast<const lds_f16x4*>(at);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[rt][x][e] += see ? special_of(v[e]) : 0.f;
            }
          }
        }
      }
      next_v(i);
    }
  };
  if (rows <= 8 * RT)
    go(std::integral_constant<int, RT / 2>{});
  else
    go(std::integral_constant<int, RT>{});

  // join the waves: first (m, l) of each row, then the sums, as many blocks of 16 dims at a time as the tiles' space holds
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    l[rt] = across<true>(l[rt], add2);
    if (grp == 0) join[wave][16 * rt + row][0] = m[rt], join[wave][16 * rt + row][1] = l[rt];
  }
  __syncthreads();  // the tiles have been read, too
  for (int r = threadIdx.x; r < rows; r += 64 * NW) {
    float mt = -INFINITY, lt = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) mt = fmaxf(mt, join[w][r][0]);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = join[w][r][0], f = mw == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mw - mt);
      lt += join[w][r][1] * f;
      join[w][r][0] = f;
    }
    if (count > 1) {
      float* to = part_row(p, part, kvh, r) + D;
      to[0] = mt, to[1] = lt;
    } else {
      row_f[r] = row_any[r] ? (FP8 && g.c.v_scale ? g.c.v_scale[kvh] : 1.f) / lt : 0.f;
    }
  }
  constexpr int BPR = 2 * NB * TILE / (RT * 1024) < DB ? 2 * NB * TILE / (RT * 1024) : DB;  // blocks of dims of a round
  static_assert(BPR >= 1, "a wave's sums fit where its tiles were");
  constexpr int SPAN = BPR * RT * 64;  // four sums each of a wave's round
  f32x4* sums = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int i0 = 0; i0 < DB; i0 += BPR) {
#pragma unroll
    for (int i = 0; i < BPR && i0 + i < DB; ++i)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) sums[wave * SPAN + (i * RT + rt) * 64 + lane] = acc[rt][i0 + i];
    __syncthreads();
    for (int x = threadIdx.x; x < SPAN; x += 64 * NW) {
      const int r = x / 64 % RT * 16 + (x & 15), dim = 16 * (i0 + x / (64 * RT)) + 4 * (x / 16 & 3);
      if (r >= rows || dim >= D) continue;  // the last round may be short
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w) o += sums[w * SPAN + x] * join[w][r][0];
      if (count > 1) {
        *reinterpret_cast<f32x4*>(part_row(p, part, kvh, r) + dim) = o;
      } else {
        const int at = r0 + r, tk = divide(at, p.group);
        f16x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = (f16)(o[e] * row_f[r]);
        *reinterpret_cast<f16x4*>(g.out + (int64_t)(s.first + tk) * g.ldo + (int64_t)(kvh * p.G + at - tk * p.G) * D + dim) = h;
      }
    }
    __syncthreads();
  }
}

template <int DP, bool FP8>
void launch_tree_dim(const Plan& p, hipStream_t st) {
  static std::once_flag flags[kMaxDevices];
  once_per_device(flags, [] {
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(attention_tree_kernel<DP, FP8>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, tree_lds<DP, FP8>());
  });
  attention_tree_kernel<DP, FP8><<<p.parts * p.a.c.heads, 64 * tree_waves<DP, FP8>(), tree_lds<DP, FP8>(), st>>>(p);
}

template <bool FP8>
void launch_tree(const Plan& p, hipStream_t st) {
  const int D = p.a.c.dim;
  if (D <= 64) launch_tree_dim<64, FP8>(p, st);
  else if (D <= 128) launch_tree_dim<128, FP8>(p, st);
  else launch_tree_dim<256, FP8>(p, st);
}

}  // namespace

void launch_attention_tree(const AttnArgs& a, void* ws, hipStream_t st) { launch_as<true>(a, ws, st); }

}  // namespace w4
