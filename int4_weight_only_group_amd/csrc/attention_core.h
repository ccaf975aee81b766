// The kernels of attention_paged and attention_paged_tree: softmax(scale q k^T) v of new tokens over a paged cache.
// attention.hip and attention_tree.hip each compile their own from this file.
//
// Query i of a sequence with n new and L cached tokens stands at position p = L - n + i and sees
// the keys max(0, p + 1 - window) <= j <= p.  Keys are taken in tiles; m, a little below the largest score
// so far, and l, the sum of exp(s - m), are kept in f32 per row, and what was summed before is
// scaled by exp(m_old - m_new) when m moves:  out = sum_j exp(s_j - m) v_j / l.  Scores are kept
// in units of log 2 (the scale carries log2 e), so the exponential is exp2.
//
// Rows.  The G = Hq / Hkv query heads of a kv head read the same keys, so a row is a (token, head
// of the group) pair, numbered token * G + head, and a tile of keys serves them all.
//
// Both kernels compute S^T = K Q^T and O^T = V^T P^T on the matrix cores, with q rows as columns:
// a lane then holds scores of one row only (m, l and the rescaling are per-lane scalars), and the
// accumulator layout of S^T is the operand layout of P^T up to the order of the keys, which V's
// transposing LDS reads follow; the weights never leave their lane.
//
// Keys that no row of the workgroup sees are not read: zeros stand in for them (what a page holds
// past its sequence's end may be anything).  A page number outside the cache gives NaN keys.  A row that sees no key is
// 0; one that sees keys, all with scores of -infinity, has l = 0 and is NaN, as its softmax is.
#pragma once

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "w4_internal.h"
#include "w4_kv.h"

namespace w4 {

namespace {

typedef __attribute__((address_space(3))) void lds_void_t;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) f16x8 lds_f16x8;
typedef __attribute__((address_space(3))) f16x4 lds_f16x4;
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
typedef __attribute__((address_space(3))) int lds_i32;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

// for lambdas: one that is not inlined keeps what it captures in memory
#define W4_INLINE __attribute__((always_inline))

constexpr float kLog2e = 1.44269504088896340736f;
// m is set kLift below a score, and moves only when one is more than kLift + kSlack above it (in powers of two), so that
// most tiles rescale nothing.  Weights stay below 2^15, which f16 holds, and the largest is 2^11 at least, so that
// f16's rounding takes 2^-36 of it at most from weights below f16's normal range: many keys far below one still
// add up right.  (Slack 8 and lift 0, 7 or slack 4 and lift 11 take the same time in every case.)
constexpr float kSlack = 4.f, kLift = 11.f;
// A score, rounded.  Fused with the subtraction of m, the product would not be, while m comes from a rounded one: from 2^23
// on (in powers of two) a weight could then exceed f16, and from 2^27 on vanish or be infinite.  So this is a
// multiplication more per score than a fused one: 503 us against 491 for the chunk of 4096, 120.6 against 118.4 for the
// windowed ragged batch, 31.1 against 30.5 for the 1570-token prompt, the same for decodes.
__device__ __forceinline__ float score(float s, float c) {
  float x = s * c;
  asm("" : "+v"(x));
  return x;
}
// whether m has to move for a score of top (not for one of -infinity before there is an m), and where to
__device__ __forceinline__ bool above(float top, float m) { return top - m > kLift + kSlack; }
__device__ __forceinline__ float moved(float top, float m) { return fmaxf(m, top - kLift); }

alignas(16) __device__ const uint32_t kZeros[4] = {0, 0, 0, 0};
alignas(16) __device__ const uint32_t kNans[4] = {0x7e007e00u, 0x7e007e00u, 0x7e007e00u, 0x7e007e00u};   // f16
alignas(16) __device__ const uint32_t kNans8[4] = {0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu};  // e4m3

// LDS DMA: lane l's 16 (4) bytes land at lds + 16 l (4 l).  Inline asm, because the compiler would
// wait for all of it before every later LDS read; the kernels wait explicitly.  The s_nop covers the
// wait states after the write of m0.
__device__ __forceinline__ void dma16(const void* p, uint32_t lds) {
  asm volatile("s_nop 1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void dma4(const void* p, uint32_t lds) {
  asm volatile("s_nop 1\n\tglobal_load_lds_dword %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}
// the same from a wave-uniform base and a 32-bit offset per lane
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 1\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt holds 0..63");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// f over the lanes l, l ^ 32 (and l ^ 16): every lane gets the result
template <bool QUARTERS, class F>
__device__ __forceinline__ float across(float v, F f) {
  uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  uint32_t a = h[0], b = h[1];
  v = f(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
  if constexpr (QUARTERS) {
    x = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    a = r[0], b = r[1];
    v = f(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
  }
  return v;
}
__device__ __forceinline__ float fmax2(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }

// LDS layout of a tile: key row r holds DP f16 = DP / 8 chunks of 16 bytes; chunk c of it lies at
// chunk c ^ k_swz(r) (K: 16-byte reads of 16 rows at one chunk touch all 64 banks) or c ^ v_swz(r)
// (V: transposing reads of 4 rows x 4 chunks, or 8 rows x 2, do).  With DP = 64 two rows share
// the 256 bytes of the banks, so their parity is part of the bank already.
template <int DP>
__device__ __forceinline__ int k_swz(int r) {
  return DP == 64 ? (r >> 1) & 7 : r & 15;
}
template <int DP>
__device__ __forceinline__ int v_swz(int r) {
  return DP == 64 ? ((r >> 1) & 1) << 2 | ((r >> 2) & 1) << 1 : (r & 3) << 2 | ((r >> 2) & 1) << 1;
}

// n / d for 0 <= n < 2^31: (n * mul) >> shift, mul = floor(2^shift / d) + 1, shift = 31 + ceil(log2 d).
// The product's error is below n / 2^shift < 1 / d, so the floor is exact.
struct Divider {
  uint64_t mul;
  int shift, d;
};
Divider divider(int d) {
  int s = 0;
  while (((int64_t)1 << s) < d) ++s;
  return {(((uint64_t)1 << (31 + s)) / (uint64_t)d) + 1, 31 + s, d};
}
// mul <= 2^32 (d a power of two: 2^31 + 1), so the product is below 2^63 + 2^31
__device__ __forceinline__ int divide(int n, const Divider& d) { return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift); }

struct Plan {
  AttnArgs a;
  Divider page, group;
  int G;
  int splits;       // few rows: parts of the keys of all sequences, about; many rows: of a row tile, at most
  int least;        // few rows: keys of a part at least
  int tiles;        // many rows: row tiles at most
  int parts;        // trees of more rows: parts of all tiles at most (splits: workgroups of a round)
  int start_keys;   // trees of more rows: how many keys a workgroup could take while it starts and ends
  int part_rows;    // rows kept of a part; many rows: of a row tile
  bool skip_short;  // both kernels run: sequences of at most kFewRows rows are the first one's
  float c;          // scale * log2 e
  int4* head;       // of a sequence (few) or row tile (many): first part, parts, ...; see the kernels
  float* part;      // [part][kv head][part_rows][dim + 4]: unscaled sums, m, l; nullptr: no parts
};

// A part's row in the workspace.
__device__ __forceinline__ float* part_row(const Plan& p, int64_t part, int kvh, int row) {
  return p.part + ((part * p.a.c.heads + kvh) * p.part_rows + row) * (p.a.c.dim + 4);
}

constexpr int kFewRows = 16;  // rows of the decode kernel's tile

struct Seq {
  int first, n, len;  // first row, rows, cached tokens
};
__device__ __forceinline__ Seq sequence(const AttnArgs& g, int b) {
  Seq s;
  if (g.q_start) {
    s.first = min(max(g.q_start[b], 0), g.T);
    s.n = min(max(g.q_start[b + 1], s.first), g.T) - s.first;
  } else {
    s.first = b, s.n = 1;
  }
  s.len = min(max(g.kv_len[b], 0), g.W * g.c.page_size);
  return s;
}

// The keys [lo, hi) that the tokens t0 .. t1 of a sequence see (lo rounded down to `align`), in `act`
// parts of `per` keys (the last may be shorter; one part of no keys writes the zeros).  per goes by
// the sequence's length, so that the tiles of a prompt, whose lengths differ, have parts of one length.
struct Keys {
  int lo, hi, per, act;
};
template <bool TREE>
__device__ __forceinline__ Keys keys_of(const Plan& p, const Seq& s, int t0, int t1, int align, int unit, int least) {
  Keys k;
  if constexpr (TREE) t0 = 0, t1 = s.n - 1;  // any row may see any new token
  k.hi = max(0, s.len - s.n + t1 + 1);
  k.lo = p.a.window ? max(0, s.len - s.n + t0 + 1 - p.a.window) : 0;
  // as many keys as the launch allows for, if a sequence has more rows than max_q
  if (TREE && p.a.window) k.lo = max(k.lo, k.hi - p.a.window - p.a.max_q);
  k.lo = min(k.lo / align * align, k.hi);
  const int all = p.a.window ? k.hi - k.lo : s.len;
  k.per = max(least, (max(all, k.hi - k.lo) + p.splits - 1) / p.splits);
  k.per = (k.per + unit - 1) / unit * unit;
  k.act = max(1, (k.hi - k.lo + k.per - 1) / k.per);
  return k;
}

// attention_paged_tree: what a row sees, the keys [lo, base) before the new tokens and, of these, the ones
// whose bits are set.  Its depth is the number of those, less one (0 at least); the window goes by it.
struct TreeRow {
  const uint64_t* bits;
  int base, lo, n;  // n: new tokens that have bits
  bool any;         // it sees a key
};
// the first x of 32 bits
__device__ __forceinline__ uint32_t first_bits(int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1u; }
__device__ __forceinline__ TreeRow tree_row(const AttnArgs& g, const Seq& s, int tok) {
  TreeRow r;
  r.bits = g.mask + (int64_t)(s.first + tok) * g.ldm;
  r.base = s.len - s.n;
  r.n = (int)min((int64_t)s.n, g.ldm * 64);
  int set = 0;
  r.any = false;
  for (int w = 0; w * 64 < r.n; ++w) {
    uint64_t x = r.bits[w];
    if (r.n - w * 64 < 64) x &= (1ull << (r.n - w * 64)) - 1;
    set += __popcll(x);
    const int out = -r.base - w * 64;  // new tokens that are not cached
    if (out > 0) x = out >= 64 ? 0 : x >> out;
    r.any |= x != 0;
  }
  r.lo = g.window ? max(0, r.base + max(set, 1) - g.window) : 0;
  r.any |= r.lo < r.base;
  return r;
}
// which of the keys j0 .. j0 + 31 it sees (j0 and all keys that matter are cached tokens' numbers)
__device__ __forceinline__ uint32_t tree_sees(const TreeRow& r, int j0) {
  const uint32_t old = first_bits(r.base - j0) & ~first_bits(r.lo - j0);
  const int at = j0 - r.base;  // as a number of a new token
  if (at <= -32 || at >= r.n) return old;
  const int from = max(at, 0), w = from >> 6, shift = from & 63;
  uint64_t x = r.bits[w] >> shift;
  if (shift > 32 && (w + 1) * 64 < r.n) x |= r.bits[w + 1] << (64 - shift);
  const uint32_t fresh = (uint32_t)x & first_bits(r.n - from);
  return old | (at < 0 ? fresh << -at : fresh);
}

// 8 and 16 e4m3 codes as f16: exact (every value of the format is an f16)
__device__ __forceinline__ f16x8 widen8(uint32_t lo, uint32_t hi) {
  f16x8 h;
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
  const auto c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
  const auto d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
  h[0] = (f16)a[0], h[1] = (f16)a[1], h[2] = (f16)b[0], h[3] = (f16)b[1];
  h[4] = (f16)c[0], h[5] = (f16)c[1], h[6] = (f16)d[0], h[7] = (f16)d[1];
  return h;
}
__device__ __forceinline__ void widen(const u32x4& v, f16x8 (&h)[2]) {
  h[0] = widen8(v[0], v[1]);
  h[1] = widen8(v[2], v[3]);
}

// A matrix product multiplies a weight of 0 with every v, and 0 * infinity is NaN.  So in tiles that
// some rows do not see whole (edge tiles) the product takes v with 0 for what is not finite, and
// if there was any, it is added afterwards, to the rows that see it (its weight is positive).
// finite: v so cleaned; odd: its cleared elements, as 16-bit masks, are or-ed into it.
__device__ __forceinline__ f16x8 finite(const f16x8& v, uint32_t& odd) {
  u32x4 x = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t top = ((x[i] & 0x7c007c00u) + 0x04000400u) & 0x80008000u;  // exponent all ones
    const uint32_t mask = (top - (top >> 15)) | top;
    odd |= mask;
    x[i] &= ~mask;
  }
  return __builtin_bit_cast(f16x8, x);
}
__device__ __forceinline__ float special_of(f16 v) {  // v if it is not finite, else 0
  return (__builtin_bit_cast(uint16_t, v) & 0x7c00) == 0x7c00 ? (float)v : 0.f;
}

// ------------------------------------------------------------------------- few rows (decode)
// At most 16 rows of a (sequence, kv head): decode, short drafts.  Bound: HBM, by the cache's bytes.
// A workgroup takes a part of one sequence's keys for one kv head; its waves take 32-key tiles in
// turn, each with LDS of its own for one tile and no barrier until the waves' sums are joined.  K of
// tile t + 1 is fetched as soon as K of t has been multiplied, V of t + 1 after V of t, so a wave always
// has half a tile or more in flight; the page numbers run a tile further ahead, through LDS too (in
// registers, the compiler's wait for them would be a wait for everything in flight).  e4m3 tiles stay
// e4m3 in LDS and are widened to f16, exactly, as fragments are read.
//
// Measured: 8 sequences of 61001 to 65536 tokens (16 heads on 2 of 128 dims, 520 MB) 97 us, 5.4 TB/s of the 5.9 that a
// bare DMA of such pages reaches; 64 of 1 to 8192 in e4m3 (16 on 8, 553 MB) 115 us, 4.8 TB/s; one of 1570, 6.4 us and
// 3.5 for the join: the latencies of page number, K, V and sums one after another.  The kernel for many rows takes
// 13.5 us for the last, and for 64 of 8192 in e4m3 278 against 195.
constexpr int kFewKeys = 32;
constexpr int kMinPart = 128;  // keys of a part at least: 64 and 256 take 10.4 and 10.3 us for one of 1570 against 9.9
template <int DP, bool FP8>
constexpr int few_tile() { return kFewKeys * DP * (FP8 ? 1 : 2); }  // bytes of K, and of V
template <int DP, bool FP8>
constexpr int few_waves() { return few_tile<DP, FP8>() > 8192 ? 2 : 4; }
template <int DP, bool FP8>
constexpr int few_lds() { return few_waves<DP, FP8>() * (2 * few_tile<DP, FP8>() + 512); }
// Workgroups of a CU: two at least, so that one starts or ends while the other streams.
template <int DP, bool FP8>
constexpr int few_per_cu() { return few_lds<DP, FP8>() > 40960 ? 2 : 4; }

// Tile rows of ROWB bytes, as above (k_swz, v_swz are for f16: ROWB = 2 DP); the transposing 8-byte
// reads of e4m3 take the 16-byte chunk of 16 rows, {0-3, 16-19} + 4 group for two groups at a time.
template <int ROWB>
__device__ __forceinline__ int k_swz_few(int r) {
  return ROWB == 64 ? (r >> 2) & 3 : ROWB == 128 ? (r >> 1) & 7 : r & 15;
}
template <int ROWB, bool FP8>
__device__ __forceinline__ int v_swz_few(int r) {
  if constexpr (!FP8) return v_swz<ROWB / 2>(r);
  return ROWB == 64    ? ((r >> 2) & 1) | ((r >> 4) & 1) << 1
         : ROWB == 128 ? ((r >> 1) & 3) | ((r >> 4) & 1) << 2
                       : (r & 7) | ((r >> 4) & 1) << 3;
}

// The 32-key tiles that one of a workgroup's NW waves takes, every NW-th of the keys [k0, k1): K and V in LDS of its own,
// NB tiles of each, fetched by LDS DMA, and the operands that the matrix products take from there.  Turn i is tile i, or, once
// whole_first() has been called, one of the `whole` tiles from f0 on first.
template <int DP, bool FP8, int NW, int NB = 1>
struct WaveTiles {
  static constexpr int KT = kFewKeys, ES = FP8 ? 1 : 2, ROWB = DP * ES, TILE = few_tile<DP, FP8>();
  static constexpr int CH = ROWB / 16, RPI = 64 / CH, NI = KT / RPI;  // chunks of a row; rows and count of a DMA instruction
  static constexpr int KA = ROWB / 64;
  static constexpr int IDS = NB == 1 ? 2 : NB == 2 ? 4 : 8;  // turns' page numbers: 2 NB at least
  const Plan& p;
  const int k0, k1, lane, wave;
  const uint32_t kt, vt;
  const int32_t* table;
  const int* ids;
  const uint32_t ids_at;
  const char* bases[2];
  const bool plain;
  const uint32_t token_bytes;
  uint32_t k_at[KA], v_row, v_chunk;
  int f0 = 0, whole = 0;

  // lds: NW NB pairs of tiles, then IDS * 256 bytes of page numbers a wave
  __device__ __forceinline__ WaveTiles(const Plan& p, unsigned char* lds, int b, int kvh, int k0, int k1, int lane, int wave)
      : p(p), k0(k0), k1(k1), lane(lane), wave(wave),
        kt((uint32_t)(uintptr_t)(lds_void_t*)lds + wave * (2 * NB * TILE)), vt(kt + TILE),
        table(p.a.table + (int64_t)b * p.a.ldt), ids(reinterpret_cast<const int*>(lds + NW * 2 * NB * TILE + wave * (IDS * 256))),
        ids_at((uint32_t)(uintptr_t)(lds_void_t*)ids),
        bases{reinterpret_cast<const char*>(p.a.c.k) + kvh * p.a.c.stride_head * ES,
              reinterpret_cast<const char*>(p.a.c.v) + kvh * p.a.c.stride_head * ES},
        // Whole tiles of pages of 16 n tokens: half a tile lies in one page, whose address is scalar; a lane adds its
        // row and chunk.
        plain(p.a.c.dim == DP && p.a.c.page_size % 16 == 0 && (k0 & 15) == 0 && p.a.c.stride_token < (1 << 20)),
        token_bytes((uint32_t)p.a.c.stride_token * ES) {}

  // the tiles that lie within [a, b) come first; all: tiles of this wave
  __device__ __forceinline__ void whole_first(int a, int b, int all) {
    const int at = k0 + wave * KT;  // first key of tile 0
    f0 = min(all, max(0, a - at + KT * NW - 1) / (KT * NW));
    whole = max(0, min(all, b - at < KT ? 0 : (b - at - KT) / (KT * NW) + 1) - f0);
    if (whole == 0) f0 = 0;
  }
  __device__ __forceinline__ int first_key(int i) const {
    i = i < whole ? f0 + i : i - whole < f0 ? i - whole : i;
    return k0 + (i * NW + wave) * KT;
  }
  static __device__ __forceinline__ uint32_t buffer(int i) { return NB == 1 ? 0u : (uint32_t)(i % NB * 2 * TILE); }

  __device__ __forceinline__ void fetch_ids(int t) const {
    const int j = min(first_key(t) + (lane & 31), k1 - 1);
    dma4(table + divide(j, p.page), ids_at + (t & (IDS - 1)) * 256);
  }

  template <class OfV>
  __device__ __forceinline__ void fetch(int t, OfV) const {
    constexpr bool V = OfV::value;
    const KvCache& c = p.a.c;
    const uint32_t st = (V ? vt : kt) + buffer(t);
    const int j0 = first_key(t), *here = ids + (t & (IDS - 1)) * 64;
    int lane_here = lane;  // opaque, or the lanes' offsets move out of the loop and fill registers
    asm volatile("" : "+v"(lane_here));
    auto chunk = [&](int r) {
      const int ch = lane_here % CH;
      return (V ? ch ^ v_swz_few<ROWB, FP8>(r) : ch ^ k_swz_few<ROWB>(r)) * 16;
    };
    if (plain && j0 + KT <= k1) {
      const int id0 = __builtin_amdgcn_readfirstlane(here[0]);
      const int id1 = __builtin_amdgcn_readfirstlane(here[16]);
      if ((uint32_t)id0 < (uint32_t)c.pages && (uint32_t)id1 < (uint32_t)c.pages) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int j = j0 + 16 * half, id = half ? id1 : id0;
          const int64_t at = id * c.stride_page + (j - divide(j, p.page) * c.page_size) * c.stride_token;
          const char* base = bases[V] + at * ES;
#pragma unroll
          for (int i = 0; i < NI / 2; ++i) {
            const int in = i * RPI + lane_here / CH;
            dma16(base + (int64_t)i * RPI * token_bytes, (uint32_t)(lane_here / CH) * token_bytes + chunk(16 * half + in),
                  st + (half * NI / 2 + i) * 1024);
          }
        }
        return;
      }
    }
#pragma unroll 1
    for (int i = 0; i < NI; ++i) {
      const int r = i * RPI + lane_here / CH, at_chunk = chunk(r);
      const int j = j0 + r, page = divide(j, p.page), id = here[r];
      const int64_t at = (id * c.stride_page + (j - page * c.page_size) * c.stride_token) * ES;
      const bool in = j < k1, good = (uint32_t)id < (uint32_t)c.pages;
      const void* from = in && !good && !V                       ? (const void*)(FP8 ? kNans8 : kNans)
                         : in && good && at_chunk < c.dim * ES ? (const void*)(bases[V] + at + at_chunk)
                                                               : (const void*)kZeros;
      dma16(from, st + i * 1024);
    }
  }

  // LDS offsets of a lane's fragments: the swizzles fold into the lane's part
  __device__ __forceinline__ void places() {
    const int row = lane & 15, grp = lane >> 4;
#pragma unroll
    for (int x = 0; x < KA; ++x) k_at[x] = kt + row * ROWB + (((4 * x + grp) ^ k_swz_few<ROWB>(row)) * 16);
    if constexpr (FP8) {  // 8 rows x 16 codes: lane L of 16 points at row L / 2, half L % 2
      const int x = (lane & 15) >> 1, r = (x & 4) * 4 + 4 * grp + (x & 3);
      v_row = vt + r * ROWB + (lane & 1) * 8, v_chunk = v_swz_few<ROWB, FP8>(r);
    } else {
      const int r = 4 * grp + ((lane & 15) >> 2);
      v_row = vt + r * ROWB + (lane & 1) * 8, v_chunk = ((lane & 3) >> 1) ^ v_swz_few<ROWB, FP8>(r);
    }
  }
  // V^T operand: dims 16 i + lane % 16, keys 4 grp .. + 3 and 16 + 4 grp .. + 3
  __device__ __forceinline__ f16x8 v_frag(int i, uint32_t buf = 0) const {
    if constexpr (FP8) {
      const auto v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<lds_i32x2*>(v_row + buf + (i ^ v_chunk) * 16));
      return widen8(v[0], v[1]);
    } else {
      const uint32_t at = v_row + buf + ((2 * i) ^ v_chunk) * 16;
      const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(at));
      const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(at + 16 * ROWB));
      return __builtin_bit_cast(f16x8, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// The keys [lo, hi) that a sequence's rows see (lo rounded down to 16, for whole pages); n < 0: not this
// kernel's sequence.
struct FewKeys {
  int n, lo, hi;
};
__device__ __forceinline__ FewKeys few_keys(const Plan& p, const Seq& s) {
  FewKeys k;
  if (s.n == 0 || (p.skip_short && s.n * p.G > kFewRows)) return {-1, 0, 0};
  k.n = min(s.n, kFewRows / p.G);
  k.hi = max(0, s.len - s.n + k.n);
  k.lo = p.a.window ? min(max(0, s.len - s.n + 1 - p.a.window) & ~15, k.hi) : 0;
  return k;
}
// Parts of a sequence when parts should have about `per` keys.
__device__ __forceinline__ int few_parts(const FewKeys& k, int per) {
  return k.n < 0 ? 0 : max(1, (k.hi - k.lo + per - 1) / per);
}

// Keys of a part, about, where all sequences have `all`.
__device__ __forceinline__ int part_keys(const Plan& p, int64_t all) {
  return (int)min((int64_t)1 << 30, max((int64_t)p.least, (all + p.splits - 1) / p.splits + kFewKeys - 1)) & ~(kFewKeys - 1);
}

// Sum over the workgroup, and over the threads before this one.
template <int NW>
__device__ __forceinline__ int64_t block_scan(int64_t mine, int64_t& before, int64_t* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t incl = mine;
#define W4_STEP(CTRL, ROWS)                                                                                    \
  incl += (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_update_dpp(0, (int)(incl >> 32), CTRL, ROWS, 0xF, false) << 32 | \
                    (uint32_t)__builtin_amdgcn_update_dpp(0, (int)incl, CTRL, ROWS, 0xF, false))
  W4_STEP(0x111, 0xF);  // row_shr 1, 2, 4, 8: sums of the rows of 16
  W4_STEP(0x112, 0xF);
  W4_STEP(0x114, 0xF);
  W4_STEP(0x118, 0xF);
  W4_STEP(0x142, 0xA);  // row_bcast15 into rows 1 and 3, row_bcast31 into rows 2 and 3
  W4_STEP(0x143, 0xC);
#undef W4_STEP
  before = incl - mine;
  if constexpr (NW == 1) return (int64_t)__shfl((long long)incl, 63);
  if (lane == 63) lds[wave] = incl;
  __syncthreads();
  int64_t all = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < wave) before += lds[w];
    all += lds[w];
  }
  return all;
}

// Which sequence and which of its parts the part-th workgroup takes: the keys of all sequences are dealt
// out in parts of about the same length, since lengths differ and the longest sequence alone would
// set the time.  Every workgroup finds its own by a scan over the sequences.  b < 0: past the last.
struct Dealt {
  int b, index, count;
  Seq s;
};
template <int NW>
__device__ __forceinline__ Dealt deal(const Plan& p, int part) {
  __shared__ int64_t sums[2][NW];
  __shared__ Dealt found;
  const int B = p.a.B, each = (B + 64 * NW - 1) / (64 * NW);
  if (B == 1) {
    const Seq s = sequence(p.a, 0);
    const FewKeys k = few_keys(p, s);
    const int n = few_parts(k, part_keys(p, k.hi - k.lo));
    return {part < n ? 0 : -1, part, n, s};
  }
  const int b0 = min(B, (int)threadIdx.x * each), b1 = min(B, b0 + each);
  if (threadIdx.x == 0) found.b = -1;
  int64_t mine = 0, before = 0;
  Seq one{0, 0, 0};  // this thread's sequence when it has at most one
  for (int b = b0; b < b1; ++b) {
    one = sequence(p.a, b);
    const FewKeys k = few_keys(p, one);
    mine += k.hi - k.lo;
  }
  const int64_t all = block_scan<NW>(mine, before, sums[0]);
  const int per = part_keys(p, all);
  auto parts = [&](int b) { return few_parts(few_keys(p, each == 1 ? one : sequence(p.a, b)), per); };
  mine = 0;
  for (int b = b0; b < b1; ++b) mine += parts(b);
  (void)block_scan<NW>(mine, before, sums[1]);
  if (part >= before && part < before + mine) {
    int64_t at = before;
    for (int b = b0; b < b1; ++b) {
      const int n = parts(b);
      if (part < at + n) {
        found = {b, (int)(part - at), n, each == 1 ? one : sequence(p.a, b)};
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  return found;
}

template <int DP, bool FP8, bool TREE>
__global__ __launch_bounds__((64 * few_waves<DP, FP8>()), (few_per_cu<DP, FP8>())) void attention_few_kernel(Plan p) {
  constexpr int NW = few_waves<DP, FP8>(), KT = kFewKeys, ES = FP8 ? 1 : 2, ROWB = DP * ES;
  constexpr int TILE = few_tile<DP, FP8>();
  constexpr int STEPS = DP / 32, DB = DP / 16;
  extern __shared__ __align__(16) unsigned char lds[];
  __shared__ float join[NW][16][2];
  const AttnArgs& g = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kvh = blockIdx.x % g.c.heads, part = blockIdx.x / g.c.heads;
  Dealt mine_is;
  if (p.part) {
    mine_is = deal<NW>(p, part);
    if (mine_is.b < 0) return;
  } else {  // no parts: a workgroup per sequence
    mine_is = {part, 0, 1, sequence(g, part)};
  }
  auto scalar = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  const int b = scalar(mine_is.b), index = scalar(mine_is.index), count = scalar(mine_is.count);
  const Seq s = {scalar(mine_is.s.first), scalar(mine_is.s.n), scalar(mine_is.s.len)};
  const FewKeys k = few_keys(p, s);
  if (k.n < 0) return;
  const int n = k.n, rows = n * p.G;
  const int per = ((k.hi - k.lo + count - 1) / count + KT - 1) & ~(KT - 1);
  const int k0 = min(k.hi, k.lo + index * per), k1 = min(k.hi, k0 + per);
  const int tiles = (k1 - k0 + KT - 1) / KT;
  const int mine = tiles > wave ? (tiles - wave + NW - 1) / NW : 0;
  const int D = g.c.dim;
  if (p.part && kvh == 0 && index == 0 && threadIdx.x == 0) p.head[b] = {part, count, 0, 0};

  WaveTiles<DP, FP8, NW> keys(p, lds, b, kvh, k0, k1, lane, wave);
  constexpr std::false_type K_{};
  constexpr std::true_type V_{};
  if (mine > 0) keys.fetch_ids(0), keys.fetch_ids(1);

  // Q^T operand: lane (row = lane % 16, grp = lane / 16), step t.  f16: dims 32 t + 8 grp ..; e4m3: a
  // 16-byte chunk of K feeds two steps, so dims 16 (4 (t / 2) + grp) + 8 (t % 2) ..
  const int row = lane & 15, grp = lane >> 4;
  const int tok = divide(min(row, rows - 1), p.group);
  f16x8 q[STEPS];
  {
    const uint16_t* src = g.q + (int64_t)(s.first + tok) * g.ldq +
                          (int64_t)(kvh * p.G + min(row, rows - 1) - tok * p.G) * D;
#pragma unroll
    for (int t = 0; t < STEPS; ++t) {
      const int d = FP8 ? 16 * (4 * (t / 2) + grp) + 8 * (t & 1) : 32 * t + 8 * grp;
      f16x8 z = {};
      q[t] = row < rows && d < D ? *reinterpret_cast<const f16x8*>(src + d) : z;
    }
  }
  // the keys that this lane's row sees: [see0, see1); that all rows see: [all0, all1)
  const int see1 = s.len - s.n + tok + 1, see0 = g.window ? see1 - g.window : 0;
  const int all1 = s.len - s.n + !TREE, all0 = g.window ? s.len - s.n + n - g.window : 0;
  TreeRow tree;
  if constexpr (TREE) tree = tree_row(g, s, tok);
  const float c = FP8 && g.c.k_scale ? p.c * g.c.k_scale[kvh] : p.c;
  float m = -INFINITY, l = 0.f;
  f32x4 acc[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i) acc[i] = {0.f, 0.f, 0.f, 0.f};

  keys.places();
  constexpr int KA = ROWB / 64;  // 64-byte blocks of a row: chunks 4 x + grp

  if (mine > 0) {
    wait_vm<0>();
    keys.fetch(0, K_);
    keys.fetch(0, V_);
  }
  for (int t = 0; t < mine; ++t) {
    const int j0 = keys.first_key(t);
    wait_vm<keys.NI>();  // V of this tile may be in flight
    f32x4 sc[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      sc[kb] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < KA; ++x) {
        const uint32_t at = keys.k_at[x] + 16 * kb * ROWB;
        if constexpr (FP8) {
          const u32x4 codes = *reinterpret_cast<const lds_u32x4*>(at);
          sc[kb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(codes[0], codes[1]), q[2 * x], sc[kb], 0, 0, 0);
          sc[kb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(codes[2], codes[3]), q[2 * x + 1], sc[kb], 0, 0, 0);
        } else {
          sc[kb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(*reinterpret_cast<const lds_f16x8*>(at), q[x], sc[kb], 0, 0, 0);
        }
      }
    }
    if (t + 1 < mine) {
      wait_lds();  // K has been read
      keys.fetch_ids(t + 2);
      keys.fetch(t + 1, K_);
    }
    // sc[kb][e]: key j0 + 16 kb + 4 grp + e of this lane's row
    const bool edge = j0 + KT > all1 || j0 < all0;
    uint32_t sees = 0;
    if constexpr (TREE)
      if (edge) sees = tree_sees(tree, j0);
    // whether this lane's row sees key j0 + r
    auto seen = [&](int r) W4_INLINE { return TREE ? (sees >> r & 1) != 0 : j0 + r >= see0 && j0 + r < see1; };
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[kb][e] = score(sc[kb][e], c);
    if (edge) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[kb][e] = seen(16 * kb + 4 * grp + e) ? sc[kb][e] : -INFINITY;
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(sc[0][e], sc[1][e]));
    if (__any(above(top, m))) {
      const float mn = moved(across<true>(top, fmax2), m);
      const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mn);
      l *= f;
#pragma unroll
      for (int i = 0; i < DB; ++i) acc[i] *= f;
      m = mn;
    }
    const float ms = m == -INFINITY ? 0.f : m;
    // weights as the sum of two f16 (22 bits): the matrix cores have time for both products here
    f16x8 w, w_low;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = __builtin_amdgcn_exp2f(sc[kb][e] - ms);
        const f16 high = (f16)x;
        l += x;
        w[4 * kb + e] = high;
        w_low[4 * kb + e] = (f16)(x - (float)high);
      }
    auto add = [&](int i, const f16x8& v) {
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w, acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w_low, acc[i], 0, 0, 0);
    };
    if (t + 1 < mine)
      wait_vm<keys.NI + 1>();  // K and the page numbers of the next tiles may be in flight
    else
      wait_vm<0>();
    if (!edge || (!TREE && n == 1 && j0 >= all0)) {  // no row sees less of the tile's keys (past k1: zeros) than another
#pragma unroll
      for (int i = 0; i < DB; ++i) add(i, keys.v_frag(i));
    } else {
      uint32_t odd = 0;
#pragma unroll
      for (int i = 0; i < DB; ++i) add(i, finite(keys.v_frag(i), odd));
      if (__any(odd != 0)) {
#pragma unroll 1
        for (int r = 0; r < KT; ++r) {
          const bool see = seen(r);
#pragma unroll
          for (int i = 0; i < DB; ++i) {
            const int byte = (16 * i + 4 * grp) * ES;
            const uint32_t at = keys.vt + r * ROWB + ((byte / 16) ^ v_swz_few<ROWB, FP8>(r)) * 16 + byte % 16;
            f16x4 v;
            if constexpr (FP8) {
              const f16x8 x = widen8(*reinterpret_cast<const lds_i32*>(at), 0);
              v = __builtin_shufflevector(x, x, 0, 1, 2, 3);
            } else {
              v = *reinterpret_cast<const lds_f16x4*>(at);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] += see ? special_of(v[e]) : 0.f;
          }
        }
      }
    }
    if (t + 1 < mine) {
      wait_lds();  // V has been read
      keys.fetch(t + 1, V_);
    }
  }

  // join the waves: each leaves (m, l) and its sums in LDS
  l = across<true>(l, add2);
  // sums f32 [16][DP], four dims x of row r at x ^ r (rows of one column would share a bank)
  static_assert(16 * DP * 4 <= 2 * TILE, "a wave's sums fit where its tiles were");
  auto sums_of = [&](int w, int r, int x) { return reinterpret_cast<f32x4*>(lds + w * 2 * TILE + r * DP * 4 + (x ^ r) * 16); };
  wait_lds();
#pragma unroll
  for (int i = 0; i < DB; ++i) *sums_of(wave, row, 4 * i + grp) = acc[i];
  if (grp == 0) join[wave][row][0] = m, join[wave][row][1] = l;
  __syncthreads();
  const float vs = FP8 && g.c.v_scale ? g.c.v_scale[kvh] : 1.f;
  for (int i = threadIdx.x; i < rows * (D / 4); i += 64 * NW) {
    const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
    float mt = -INFINITY, lt = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) mt = fmaxf(mt, join[w][r][0]);
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = join[w][r][0], f = mw == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mw - mt);
      lt += join[w][r][1] * f;
      o += *sums_of(w, r, d / 4) * f;
    }
    if (count > 1) {
      if (r < p.part_rows) {
        float* to = part_row(p, part, kvh, r);
        *reinterpret_cast<f32x4*>(to + d) = o;
        if (d == 0) to[D] = mt, to[D + 1] = lt;
      }
    } else {
      const int tk = divide(r, p.group);
      bool any = s.len - s.n + tk >= 0;
      if constexpr (TREE) any = tree_row(g, s, tk).any;
      const float f = any ? vs / lt : 0.f;
      f16x4 h;
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = (f16)(o[e] * f);
      *reinterpret_cast<f16x4*>(g.out + (int64_t)(s.first + tk) * g.ldo + (int64_t)(kvh * p.G + r - tk * p.G) * D +
                                d) = h;
    }
  }
}

// ------------------------------------------------------------------------------ many rows
// Chunks of prompts.  Bound: the matrix cores.  A workgroup of four waves takes a tile of rows of a (sequence, kv
// head), 32 per wave, and a part of their keys; K and V tiles are double buffered in LDS.  Either four row
// blocks share the key tiles (KS = 1: 128 rows), or two do and two waves each take every other tile, their sums
// being joined in LDS at the end (KS = 2: 64 rows; half the time per workgroup for twice as many, where
// 128 rows leave CUs idle).  32 rows a wave: its sums, queries and scores take 240 registers at 128 dims, so that two
// waves of a SIMD cover each other's waits.  K's and V's fragments come from LDS at the rate that the products
// take them.
//
// Measured, 16 heads on 2 of 128 dims: a chunk of 4096 tokens behind 12288, 501 us, 0.96 PFLOP/s (a library f16 product
// of 8192^3: 1.1), 527 from an e4m3 cache; a prompt of 1570, 30.6 us, of which the longest workgroup's 25 turns of 64 keys
// take 25, 38.3 from e4m3.  16 heads on 8 of 256 dims, 2048 tokens behind 6144: 293 us, 0.82 PFLOP/s, one wave a SIMD
// (the same with four buffers, whose loads have three turns to arrive).
constexpr int kManyWaves = 4;
template <int DP, int KS>
constexpr int many_keys() { return DP == 256 || KS == 2 ? 32 : 64; }  // of a key tile
template <int DP, int KS>
constexpr int many_lds() { return KS * 4 * many_keys<DP, KS>() * DP * 2 + kManyWaves * 1024; }
// Workgroups of a CU: two by their LDS, and by their registers up to 128 dims.  (Three buffers at KS = 2 take the LDS of
// one: a 1570-token prompt in 39 us against 31.7.)
template <int DP>
constexpr int many_per_cu() { return DP == 256 ? 1 : 2; }

__device__ __forceinline__ int tiles_of(const Plan& p, int n) {
  if (p.skip_short && n * p.G <= kFewRows) return 0;
  return (min(n, p.a.max_q) * p.G + p.part_rows - 1) / p.part_rows;  // the launch has tiles for max_q tokens each
}

// The sequence and tile of the tile-th row tile of the batch; b = -1 past the last.  64 sequences at a
// time, one per lane.
__device__ __forceinline__ Seq locate(const Plan& p, int tile, int& b, int& at) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int b0 = 0; b0 < p.a.B; b0 += 64) {
    const Seq s = sequence(p.a, min(b0 + lane, p.a.B - 1));
    const int mine = b0 + lane < p.a.B ? tiles_of(p, s.n) : 0;
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int x = __shfl_up(incl, d);
      if (lane >= d) incl += x;
    }
    const unsigned long long hit = __ballot(base + incl > tile);
    if (hit) {
      const int at_lane = __builtin_ctzll(hit);
      b = b0 + at_lane;
      at = tile - base - (__shfl(incl, at_lane) - __shfl(mine, at_lane));
      b = __builtin_amdgcn_readfirstlane(b);
      at = __builtin_amdgcn_readfirstlane(at);
      return {__builtin_amdgcn_readlane(s.first, at_lane), __builtin_amdgcn_readlane(s.n, at_lane),
              __builtin_amdgcn_readlane(s.len, at_lane)};
    }
    base += __shfl(incl, 63);
  }
  b = -1, at = 0;
  return {0, 0, 0};
}

// Trees: which row tile and which of its parts the part-th workgroup takes.  All rows of a sequence see its old keys, so that a
// tile's work goes by its sequence's length, and the keys of all tiles are dealt out in parts of about the same
// length, which the workgroups choose from the lengths: by the longest sequence's, 16 of 301 to 8192 keys (7 to 48 rows of two
// heads each, on 8 kv heads of 128 dims, e4m3) take 125 us in the kernel for many rows, and so 67.  (Ranges of equal length
// that go on from tile to tile balance better and take longer: a workgroup's second part starts as slowly as its first.)
struct DealtTile {
  int b, tile, slot;        // b < 0: past the last; slot: the tile's number in the batch
  int index, count, first;  // part of the tile, its parts, the first of them
  Seq s;
};
template <int NW, int KT, int UNIT>
__device__ __forceinline__ DealtTile deal_tiles(const Plan& p, int part, unsigned char* lds) {
  __shared__ int64_t sums[3][NW];
  __shared__ DealtTile found;
  const int B = p.a.B, each = (B + 64 * NW - 1) / (64 * NW), lane = threadIdx.x & 63;
  auto keys = [&](const Seq& s) {
    const Keys k = keys_of<true>(p, s, 0, 0, KT, UNIT, UNIT);
    return k.hi - k.lo;
  };
  auto parts_of = [&](int keys, int per) { return max(1, (keys + per - 1) / per); };
  // Keys of a part where all tiles have `all`, f of an equal share of the p.splits workgroups of a round.
  auto share = [&](int64_t all, float f) {
    const int64_t x = (int64_t)((float)all * f / (float)p.splits) + 1;
    return (int)min((int64_t)1 << 30, max((int64_t)kMinPart, (x + UNIT - 1) / UNIT * UNIT));
  };
  // The best of 64 lengths of parts from a half to 4 shares: rounds of the parts they make, times their length and what a
  // workgroup takes to start and end, in keys.  count(per): parts of all tiles.
  auto choose = [&](int64_t all, auto count) {
    const int per = share(all, .5f * __builtin_amdgcn_exp2f((float)lane * (3.f / 63.f)));
    const float rounds = ceilf(count(per) / (float)p.splits);
    float best = rounds * (float)(per + p.start_keys), least = best;
    least = fminf(least, __shfl_xor(least, 32));
    least = fminf(least, __shfl_xor(least, 16));
    least = fminf(least, __shfl_xor(least, 8));
    least = fminf(least, __shfl_xor(least, 4));
    least = fminf(least, __shfl_xor(least, 2));
    least = fminf(least, __shfl_xor(least, 1));
    return __builtin_amdgcn_readlane(per, __builtin_ctzll(__ballot(best == least)));
  };
  auto spare = [&](int tiles) {  // tiles that the launch allows for and the batch does not have
    if (p.part && blockIdx.x == 0)
      for (int i = tiles + threadIdx.x; i < p.tiles; i += 64 * NW) p.head[i] = {0, 0, 0, 0};
  };
  if (B == 1) {
    const Seq s = sequence(p.a, 0);
    const int n = tiles_of(p, s.n), k = keys(s);
    spare(n);
    int per = 1 << 30;
    if (p.part) per = choose((int64_t)n * k, [&](int per) { return (float)n * (float)parts_of(k, per); });
    const int count = parts_of(k, per), tile = part / count;
    return {tile < n ? 0 : -1, tile, tile, part - tile * count, count, tile * count, s};
  }
  const int b0 = min(B, (int)threadIdx.x * each), b1 = min(B, b0 + each);
  if (threadIdx.x == 0) found.b = -1;
  int64_t mine = 0, before = 0;
  Seq one{0, 0, 0};  // this thread's sequence when it has at most one
  int one_keys = 0;
  for (int b = b0; b < b1; ++b) {
    one = sequence(p.a, b);
    one_keys = keys(one);
    mine += (int64_t)tiles_of(p, one.n) * one_keys;
  }
  int per = 1 << 30;
  if (p.part) {
    int2* seqs = reinterpret_cast<int2*>(lds);  // keys, tiles
    if (each == 1 && b0 < B) seqs[b0] = {one_keys, tiles_of(p, one.n)};
    const int64_t all = block_scan<NW>(mine, before, sums[0]);
    if (each == 1)
      per = choose(all, [&](int per) {
        const float f = 1.f / (float)per;
        float n = 0.f;
        for (int b = 0; b < B; ++b) n += (float)seqs[b].y * fmaxf(1.f, ceilf((float)seqs[b].x * f));
        return n;
      });
    else  // many sequences: parts are short beside a round
      per = share(all, .5f);
  }
  mine = 0;
  int64_t tiles = 0, slot;
  for (int b = b0; b < b1; ++b) {
    const Seq s = each == 1 ? one : sequence(p.a, b);
    const int64_t n = tiles_of(p, s.n);
    tiles += n, mine += n * parts_of(keys(s), per);
  }
  (void)block_scan<NW>(mine, before, sums[1]);
  const int64_t total = block_scan<NW>(tiles, slot, sums[2]);
  if (part >= before && part < before + mine) {
    for (int b = b0; b < b1; ++b) {
      const Seq s = each == 1 ? one : sequence(p.a, b);
      const int64_t n = tiles_of(p, s.n);
      const int count = n > 0 ? parts_of(keys(s), per) : 1;
      if (part < before + n * count) {
        const int in = (int)(part - before), tile = in / count;
        // (starts that fall make more tiles than the launch allows for)
        if (slot + tile < p.tiles) found = {b, tile, (int)slot + tile, in - tile * count, count, part - (in - tile * count), s};
        break;
      }
      before += n * count, slot += n;
    }
  }
  spare((int)min(total, (int64_t)p.tiles));
  __syncthreads();
  return found;
}

template <int DP, bool FP8, int KS, bool TREE>
__global__ __launch_bounds__((64 * kManyWaves), (many_per_cu<DP>())) void attention_many_kernel(Plan p) {
  constexpr int NW = kManyWaves, RG = NW / KS, ROWS = 32 * RG;  // row blocks, rows
  constexpr int KT = many_keys<DP, KS>(), TILE = KT * DP * 2, RW = KT / RG;  // RW: rows of a tile that a wave fetches
  constexpr int STEPS = DP / 16, DB = DP / 32, SUB = KT / 32, NB = 2;  // NB: buffers
  extern __shared__ __align__(16) unsigned char lds[];
  const AttnArgs& g = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the last tiles of a sequence see the most keys: they go first
  const int kvh = blockIdx.x % g.c.heads, rest = blockIdx.x / g.c.heads;
  int b, tile, split, slot, part;  // part: its number in the workspace
  Seq s;
  int first = 0, parts = 0;
  if constexpr (TREE) {
    const DealtTile d = deal_tiles<NW, KT, KT * KS>(p, rest, lds);
    if (d.b < 0) return;
    auto scalar = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
    b = scalar(d.b), tile = scalar(d.tile), split = scalar(d.index), slot = scalar(d.slot);
    s = {scalar(d.s.first), scalar(d.s.n), scalar(d.s.len)};
    first = scalar(d.first), parts = scalar(d.count), part = rest;
  } else {
    split = rest % p.splits, slot = p.tiles - 1 - rest / p.splits, part = slot * p.splits + split;
    s = locate(p, slot, b, tile);
    if (b < 0) {
      if (p.part && kvh == 0 && split == 0 && threadIdx.x == 0) p.head[slot] = {0, 0, 0, 0};
      return;
    }
  }
  const int D = g.c.dim, all_rows = s.n * p.G, r0 = tile * ROWS, r1 = min(all_rows, r0 + ROWS);
  Keys k = keys_of<TREE>(p, s, divide(r0, p.group), divide(r1 - 1, p.group), KT, KT, 2 * KT * KS);
  if constexpr (TREE) {
    k.act = parts;
    k.per = ((k.hi - k.lo + parts - 1) / parts + KT * KS - 1) / (KT * KS) * (KT * KS);
  } else {
    if (split >= k.act) return;
    first = slot * p.splits;
  }
  if (p.part && kvh == 0 && split == 0 && threadIdx.x == 0) p.head[slot] = {first, k.act, b, tile};
  const int k0 = TREE ? min(k.hi, k.lo + split * k.per) : k.lo + split * k.per, k1 = min(k.hi, k0 + k.per);
  const int tiles = (k1 - k0 + KT - 1) / KT;
  const int32_t* table = g.table + (int64_t)b * g.ldt;

  // Q^T operand: lane (row = lane % 32, h = lane / 32), step t: dims 16 t + 8 h ..
  const int rg = wave % RG, kg = wave / RG;  // row block; with KS = 2, which of every two key tiles
  const int h = lane >> 5, wr0 = r0 + 32 * rg, wr1 = min(r1, wr0 + 32);
  const bool live = wr0 < r1;  // a wave of no rows helps to fetch
  const int row = min(wr0 + (lane & 31), r1 - 1), tok = divide(row, p.group);
  f16x8 q[STEPS];
  const int at0 = s.len - s.n + 1;  // keys before and at token 0's position
  const int see1 = at0 + tok, see0 = g.window ? see1 - g.window : 0;
  const int tok_a = divide(min(wr0, r1 - 1), p.group), tok_b = divide(max(wr0, wr1) - 1, p.group);
  // keys that any row of the wave sees
  const int any1 = TREE ? s.len : at0 + tok_b, any0 = g.window ? at0 + (TREE ? 0 : tok_a) - g.window : 0;
  TreeRow tree;
  if constexpr (TREE) tree = tree_row(g, s, tok);
  const float c = FP8 && g.c.k_scale ? p.c * g.c.k_scale[kvh] : p.c;
  float m = -INFINITY, l = 0.f;
  f32x16 acc[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[i][e] = 0.f;

  // LDS: NB K tiles, NB V tiles (of each kg), the waves' page numbers.  Offsets of a lane's fragments within a tile:
  // the swizzles fold into the lane's part, up to the chunk bits that count steps (K) or dims blocks (V)
  // below 256 bytes.
  constexpr int SPACE = 2 * NB * TILE;  // of a kg
  const uint32_t lds_at = (uint32_t)(uintptr_t)(lds_void_t*)lds + kg * SPACE;
  auto k_tile = [](int i) { return (uint32_t)(i % NB * TILE); };
  auto v_tile = [](int i) { return (uint32_t)((NB + i % NB) * TILE); };
  constexpr int HALF = 32 * DP * 2;  // bytes of 32 keys
  constexpr int KA = STEPS < 8 ? STEPS : 8, VA = DB < 4 ? DB : 4;
  uint32_t k_at[KA], v_at[VA];
#pragma unroll
  for (int st = 0; st < KA; ++st) {
    const int r = lane & 31;
    k_at[st] = lds_at + (uint32_t)(r * DP * 2 + (((2 * st + h) ^ k_swz<DP>(r)) * 16));
  }
#pragma unroll
  for (int i = 0; i < VA; ++i) {
    const int r = 4 * h + ((lane & 15) >> 2), ch = 4 * i + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    v_at[i] = lds_at + (uint32_t)(r * DP * 2 + ((ch ^ v_swz<DP>(r)) * 16) + (lane & 1) * 8);
  }
  // K operand: key lane % 32 of 32 at LDS offset `at`, dims 16 st + 8 h ..
  auto k_frag = [&](uint32_t at, int st) W4_INLINE {
    return *reinterpret_cast<const lds_f16x8*>(reinterpret_cast<lds_char*>(k_at[st % KA]) + (at + st / KA * 256));
  };
  // V^T operand x of 32 keys at `at`: dims 32 (x / 2) + lane % 32, keys 16 (x % 2) + 4 h .. + 3 and + 8 ..
  auto v_frag = [&](uint32_t at, int x) W4_INLINE {
    lds_char* from = reinterpret_cast<lds_char*>(v_at[x / 2 % VA]) + (at + x / 2 / VA * 256 + 16 * (x & 1) * DP * 2);
    const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(from));
    const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(from + 8 * DP * 2));
    return __builtin_bit_cast(f16x8, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  // ---- whole tiles: [f0, f0 + whole) of this part are seen whole by all rows and come first, in a loop
  // without masks; the tiles at the edges follow.
  int f0 = 0, whole;
  {
    const int end = TREE ? at0 - 1 : at0 + divide(r0, p.group);
    int beg = g.window ? at0 + (TREE ? s.n - 1 : divide(r1 - 1, p.group)) - g.window : 0;
    if constexpr (TREE) {  // depths are known: the deepest row's first key
      if (g.window) {
        __shared__ int deepest;
        if (threadIdx.x == 0) deepest = 0;
        __syncthreads();
        atomicMax(&deepest, tree.lo);
        __syncthreads();
        beg = __builtin_amdgcn_readfirstlane(deepest);
      }
    }
    f0 = max(0, beg - k0 + KT - 1) / KT;
    whole = max(0, max(0, min(end, k1) - k0) / KT - f0);
    if (whole == 0) f0 = 0;
  }
  // in the order that they are taken; this wave takes kg, kg + KS, ...: `turns` of them, `full` in the first loop
  auto tile_at = [&](int i) {
    const int n = i * KS + kg;
    return n < whole ? f0 + n : n - whole < f0 ? n - whole : n;
  };
  auto there = [&](int i) { return i * KS + kg < tiles; };
  const int full = whole / KS, turns = (tiles + KS - 1) / KS;

  // The loop over whole tiles goes by 32 keys and is pipelined: while the softmax of block u runs on the VALU,
  // the matrix cores compute the scores of block u + 1, then the weighted sums of block u - 1.  `sc` are
  // u's scores and `top` their largest of this lane, `w` the weights of u - 1 (scaled by the m of then: when u moves m,
  // the sums are rescaled after the products of u - 1).  Slices of four products carry their share of
  // the VALU work, fragments are read two slices ahead, and between(x) follows slice x.  l sums the
  // weights as rounded, which are the ones that multiply v.  One f16 a weight makes the result's error 2.9e-4 of its norm
  // where its own rounding to f16 is 2.1e-4; two, as for few rows, would make it 2.1e-4 and take 43 % longer
  // for the chunk of 4096, 19 % for the 1570-token prompt.
  f32x16 sc;
  f16x8 w[2];
  float ms = 0.f, top = 0.f;  // ms: m, or 0 before there is one
  auto top_of = [&](const f32x16& x) W4_INLINE {
    float y[6];
#pragma unroll
    for (int e = 0; e < 5; ++e) y[e] = fmaxf(fmaxf(x[3 * e], x[3 * e + 1]), x[3 * e + 2]);
    y[0] = fmaxf(fmaxf(y[0], y[1]), x[15]);
    y[2] = fmaxf(fmaxf(y[2], y[3]), y[4]);
    return score(fmaxf(y[0], y[2]), c);
  };
  constexpr int SLICES = STEPS / 2, EACH = 16 / SLICES;
  f16x8 frags[3][4];  // of three slices in turn
  // of: which of two blocks whose tiles follow each other in LDS this is: 0 reads ahead into 1; -1: alone
  auto block = [&](auto with_qk, auto with_pv, uint32_t k_next, uint32_t v_last, auto between, auto of) W4_INLINE {
    constexpr bool QK = decltype(with_qk)::value, PV = decltype(with_pv)::value;
    constexpr int OF = decltype(of)::value, FROM = OF == 1 ? SLICES : 0;
    auto read = [&](int x) W4_INLINE {  // the fragments of slice x; past the last: of the block that follows
      const uint32_t on = x / SLICES * HALF;
      const int y = x % SLICES;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (QK)
          if (y < SLICES / 2) frags[(FROM + x) % 3][e] = k_frag(k_next + on, 4 * y + e);
        if constexpr (PV)
          if (y >= SLICES / 2) frags[(FROM + x) % 3][e] = v_frag(v_last + on, 4 * (y - SLICES / 2) + e);
      }
    };
    f32x16 next;
    u32x4 nw[2];
    float y[16], f = 1.f;
    auto round_to = [&](int x) W4_INLINE {  // slice x's weights to f16, a slice after their exponentials
#pragma unroll
      for (int e = EACH * x; e < EACH * (x + 1); e += 2) {
        const f16x2 pair = {(f16)y[e], (f16)y[e + 1]};
        nw[e >> 3][e >> 1 & 3] = __builtin_bit_cast(uint32_t, pair);
      }
    };
#pragma unroll
    for (int e = 0; e < 16; ++e) next[e] = 0.f;
    if constexpr (OF != 1) read(0), read(1);
    const bool move = __any(above(top, m));
    if (move) {
      const float mn = moved(across<false>(top, fmax2), m);
      f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      ms = m == -INFINITY ? 0.f : m;
      l *= f;
    }
#pragma unroll
    for (int x = 0; x < SLICES; ++x) {
      if (x + 2 < SLICES || OF == 0) read(x + 2);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int z = 4 * (x % (SLICES / 2)) + e;
        const f16x8& fr = frags[(FROM + x) % 3][e];
        if constexpr (QK)
          if (x < SLICES / 2) next = __builtin_amdgcn_mfma_f32_32x32x16_f16(fr, q[z], next, 0, 0, 0);
        if constexpr (PV)
          if (x >= SLICES / 2) acc[z / 2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fr, w[z & 1], acc[z / 2], 0, 0, 0);
      }
      if (x > 0) round_to(x - 1);
#pragma unroll
      for (int e = EACH * x; e < EACH * (x + 1); ++e) {
        y[e] = __builtin_amdgcn_exp2f(score(sc[e], c) - ms);
        asm volatile("" : "+v"(y[e]));  // in this slice: the compiler would move it behind the last branch
      }
      if constexpr (QK)
        if (x == SLICES - 1) {
          top = top_of(next);
          asm volatile("" : "+v"(top));
        }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // LDS reads
        __builtin_amdgcn_sched_group_barrier(0x402, EACH + 1, 0);  // VALU work
      }
      __builtin_amdgcn_sched_barrier(0);
      between(x);
    }
    round_to(SLICES - 1);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t bits = nw[e >> 2][e & 3];
      const hf16x2 ones = {(__fp16)1.f, (__fp16)1.f};
      l = __builtin_amdgcn_fdot2(__builtin_bit_cast(hf16x2, bits), ones, l, false);
    }
    if (move) {
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] *= f;
    }
    w[0] = __builtin_bit_cast(f16x8, nw[0]), w[1] = __builtin_bit_cast(f16x8, nw[1]);
    sc = next;
  };

  // ---- a tile that some row does not see whole, 32 keys at a time
  auto edge = [&](int i) W4_INLINE {
#pragma unroll 1
    for (int u = 0; u < SUB; ++u) {
      const int j0 = k0 + tile_at(i) * KT + 32 * u;
      if (j0 >= any1 || j0 + 32 <= any0) continue;
      uint32_t sees = 0;
      if constexpr (TREE) {
        sees = tree_sees(tree, j0);
        if (!__any(sees != 0)) continue;
      }
      const uint32_t kt = k_tile(i) + u * HALF, vt = v_tile(i) + u * HALF;
#pragma unroll
      for (int e = 0; e < 16; ++e) sc[e] = 0.f;
#pragma unroll
      for (int st = 0; st < STEPS; ++st)
        sc = __builtin_amdgcn_mfma_f32_32x32x16_f16(k_frag(kt, st), q[st], sc, 0, 0, 0);
      top = -INFINITY;
      // whether this lane's row sees key j0 + r
      auto seen = [&](int r) W4_INLINE { return TREE ? (sees >> r & 1) != 0 : j0 + r >= see0 && j0 + r < see1; };
#pragma unroll
      for (int e = 0; e < 16; ++e) {  // key j0 + 8 (e / 4) + 4 h + e % 4 of this lane's row
        sc[e] = seen(8 * (e >> 2) + 4 * h + (e & 3)) ? score(sc[e], c) : -INFINITY;
        top = fmaxf(top, sc[e]);
      }
      top = across<false>(top, fmax2);
      if (__any(above(top, m))) {
        const float mn = moved(top, m), f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mn);
        l *= f;
#pragma unroll
        for (int x = 0; x < DB; ++x)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[x][e] *= f;
        m = mn;
        ms = m == -INFINITY ? 0.f : m;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        w[e >> 3][e & 7] = (f16)__builtin_amdgcn_exp2f(sc[e] - ms);
        l += (float)w[e >> 3][e & 7];
      }
      uint32_t odd = 0;
#pragma unroll
      for (int x = 0; x < 2 * DB; ++x)
        acc[x / 2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(finite(v_frag(vt, x), odd), w[x & 1], acc[x / 2], 0, 0, 0);
      if (!__any(odd != 0)) continue;
#pragma unroll 1
      for (int r = 0; r < 32; ++r) {
        const bool see = seen(r);
#pragma unroll
        for (int x = 0; x < DB; ++x)
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const f16x4 v = *reinterpret_cast<const lds_f16x4*>(
                lds_at + vt + (uint32_t)(r * DP * 2 + ((4 * x + a) ^ v_swz<DP>(r)) * 16 + 8 * h));
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[x][4 * a + e] += see ? special_of(v[e]) : 0.f;
          }
      }
    }
  };

  // ---- fetching: this wave's RW rows of a tile
  constexpr int ES = FP8 ? 1 : 2, CH = DP * ES / 16, RPI = 64 / CH, NI = RW / RPI;  // chunks of a row; rows and count of a load
  static_assert(RW % RPI == 0, "whole rows of a load");
  const char* bases[2] = {reinterpret_cast<const char*>(g.c.k) + kvh * g.c.stride_head * ES,
                          reinterpret_cast<const char*>(g.c.v) + kvh * g.c.stride_head * ES};
  // Pages of whole RW rows (and no padded dims): this wave's rows of a tile lie in one page, so their offset
  // from the base is scalar and a lane adds its row and chunk.  64 tiles' offsets are computed at once, one
  // per lane; the turn between two tiles then takes two lane reads.  (Scalar address arithmetic at every
  // turn, and per-lane addresses the more so, cost more issue slots than the softmax: 2048 tokens after 6144 take
  // 152 us with pages of 16, 233 with pages of 8 or 100, and 232 at 80, 96 and 112 dims.)
  const bool plain = D == DP && g.c.page_size % RW == 0 && g.c.stride_token < (1 << 20);
  const uint32_t lane_row = (uint32_t)(lane / CH) * (uint32_t)g.c.stride_token * ES;
  const int64_t step_bytes = (int64_t)RPI * g.c.stride_token * ES;  // between the rows of two loads
  int64_t offsets = 0;  // lane i: of tile batch + i; -1: a page outside the cache
  int batch = -64;
  auto offset_of = [&](int i) W4_INLINE {  // k1 > 0
    if ((i & ~63) != batch) {
      batch = i & ~63;
      const int jw = k0 + tile_at(batch + lane) * KT + RW * rg, j = min(jw, k1 - 1);
      const int page = divide(j, p.page), id = table[page];
      offsets = (uint32_t)id < (uint32_t)g.c.pages
                    ? (id * g.c.stride_page + (j - page * g.c.page_size) * g.c.stride_token) * ES
                    : -1;
    }
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(offsets >> 32), i & 63) << 32 |
                     (uint32_t)__builtin_amdgcn_readlane((int)offsets, i & 63));
  };
  // any other page size: page numbers of a tile's rows, through LDS, four tiles of them
  const int* ids = reinterpret_cast<const int*>(lds + KS * SPACE + wave * 1024);
  const uint32_t ids_at = (uint32_t)(uintptr_t)(lds_void_t*)ids;
  auto fetch_ids = [&](int i) W4_INLINE {
    if (plain) return;
    const int j = min(k0 + tile_at(i) * KT + RW * rg + lane % RW, k1 - 1);
    dma4(table + divide(j, p.page), ids_at + (i & 3) * 256);
  };
  u32x4 held[2][NI];  // e4m3: tiles on their way to LDS
  const char* from[2] = {nullptr, nullptr};  // this wave's rows of the plain K and V tiles that ready() found, and where
  uint32_t to[2] = {0, 0};                   // they go
  auto chunk = [&](auto of_v, int r, int ln) W4_INLINE {  // byte of row r that lane's 16 bytes are fetched from
    constexpr bool V = decltype(of_v)::value;
    const int ch = ln % CH;
    return FP8 ? ch * 16 : (V ? ch ^ v_swz<DP>(r) : ch ^ k_swz<DP>(r)) * 16;
  };
  auto fetch_one = [&](auto of_v, int x) W4_INLINE {  // load x of a plain tile
    constexpr bool V = decltype(of_v)::value;
    const uint32_t off = lane_row + chunk(of_v, RW * rg + x * RPI + lane / CH, lane);
    const char* row0 = from[V] + x * step_bytes;
    if constexpr (FP8)
      held[V][x] = *reinterpret_cast<const u32x4*>(row0 + off);
    else
      dma16(row0, off, to[V] + x * 1024);
  };
  // Makes tile i, `off` from the base if plain, ready for fetch_one(0 .. NI - 1), or fetches it whole and says false.
  auto ready = [&](int i, auto of_v, int64_t off) W4_INLINE {
    constexpr bool V = decltype(of_v)::value;
    const uint32_t st = lds_at + (V ? v_tile(i) : k_tile(i)) + rg * (TILE / RG);
    const int jt = k0 + tile_at(i) * KT, jw = jt + RW * rg;
    if (plain && off >= 0 && jt + KT <= k1) {
      from[V] = bases[V] + off;
      to[V] = st;
      return true;
    }
#pragma unroll
    for (int x = 0; x < NI; ++x) {
      const int rw = x * RPI + lane / CH, at_chunk = chunk(of_v, RW * rg + rw, lane), j = jw + rw;
      int64_t at = off + (int64_t)rw * g.c.stride_token * ES;
      bool good = off >= 0;
      if (!plain) {
        const int page = divide(j, p.page), id = ids[(i & 3) * 64 + rw];
        at = (id * g.c.stride_page + (j - page * g.c.page_size) * g.c.stride_token) * ES;
        good = (uint32_t)id < (uint32_t)g.c.pages;
      }
      const bool in = j < k1;
      const void* src = in && !good && !V                 ? (const void*)(FP8 ? kNans8 : kNans)
                        : in && good && at_chunk < D * ES ? (const void*)(bases[V] + at + at_chunk)
                                                          : (const void*)kZeros;
      if constexpr (FP8)
        held[V][x] = *reinterpret_cast<const u32x4*>(src);
      else
        dma16(src, st + x * 1024);
    }
    return false;
  };
  // e4m3: what fetch() holds of tile i, widened, to LDS
  auto land = [&](int i, auto of_v) W4_INLINE {
    constexpr bool V = decltype(of_v)::value;
    unsigned char* st = lds + kg * SPACE + (V ? v_tile(i) : k_tile(i));
#pragma unroll
    for (int x = 0; x < NI; ++x) {
      const int r = RW * rg + x * RPI + lane / CH, ch = lane % CH * 2;
      const int swz = V ? v_swz<DP>(r) : k_swz<DP>(r);
      f16x8 y[2];
      widen(held[V][x], y);
#pragma unroll
      for (int e = 0; e < 2; ++e) *reinterpret_cast<f16x8*>(st + r * DP * 2 + ((ch + e) ^ swz) * 16) = y[e];
    }
  };
  constexpr std::false_type K_{};
  constexpr std::true_type V_{};
  // every wave's part of what was fetched is there, and what was read before has been read
  auto meet = [&]() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
  int held_k = -1, held_v = -1;  // e4m3: the tiles in `held`
  auto put_down = [&]() W4_INLINE {
    if constexpr (FP8) {
      if (held_k >= 0) land(held_k, K_);
      if (held_v >= 0) land(held_v, V_);
      held_k = held_v = -1;
    }
  };
  auto start_k = [&](int i, int64_t off) W4_INLINE {  // says whether fetch_one is to do the rest
    if (!there(i)) return false;
    held_k = i;
    return ready(i, K_, off);
  };
  auto start_v = [&](int i, int64_t off) W4_INLINE {
    if (!there(i)) return false;
    held_v = i;
    return ready(i, V_, off);
  };
  // a tile that is not there has no offset: with no keys at all (k1 = 0), not even of the table's first page
  auto get_k = [&](int i) W4_INLINE {
    if (there(i) && start_k(i, plain ? offset_of(i) : 0)) {
#pragma unroll
      for (int x = 0; x < NI; ++x) fetch_one(K_, x);
    }
  };
  auto get_v = [&](int i) W4_INLINE {
    if (there(i) && start_v(i, plain ? offset_of(i) : 0)) {
#pragma unroll
      for (int x = 0; x < NI; ++x) fetch_one(V_, x);
    }
  };
  // Between the block that reads K of tile t last and the one that reads K of t + 1: K of t is not read any
  // more, nor V of t - 1 (SUB = 2) or t - 2, so the tiles NB further may follow, all of them now, or the plain ones
  // behind the first slices of the next block.  (Issued together, the waves' DMA queues up for the memory
  // path while the matrix cores idle.)
  constexpr int LAG = SUB == 2 ? 1 : 2;  // V is that far behind K
  bool more_k = false, more_v = false;
  int64_t off_v[2] = {0, 0};  // offsets of the next V tiles
  // inner: tile t + NB is a whole one, and phase is t % NB, a constant
  auto turn = [&](int t, auto inner, int phase) W4_INLINE {
    put_down();
    meet();
    if (!plain) {
      fetch_ids(t + NB + 1);
      more_k = start_k(t + NB, 0);
      more_v = start_v(t + NB - LAG, 0);
      return;
    }
    const int64_t off = offset_of(t + NB), now_v = off_v[0];
    if constexpr (LAG == 2) off_v[0] = off_v[1];
    off_v[LAG - 1] = off;
    if (decltype(inner)::value && (off | now_v) >= 0) {
      from[0] = bases[0] + off, from[1] = bases[1] + now_v;
      to[0] = lds_at + k_tile(phase) + rg * (TILE / RG), to[1] = lds_at + v_tile(phase + NB - LAG) + rg * (TILE / RG);
      held_k = t + NB, held_v = t + NB - LAG;
      more_k = more_v = true;
      return;
    }
    more_k = start_k(t + NB, off);
    more_v = start_v(t + NB - LAG, now_v);
  };
  constexpr int PER = (2 * NI + DB - 1) / DB;  // loads behind a slice
  auto rest_k = [&](int x) W4_INLINE {
    if (more_k) {
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (x * PER + e < NI) fetch_one(K_, x * PER + e);
    }
  };
  auto rest_v = [&](int x) W4_INLINE {
    if (more_v) {
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (x * PER + e < NI) fetch_one(V_, x * PER + e);
    }
  };
  auto rest_kv = [&](int x) W4_INLINE { rest_k(x), rest_v(x); };
  auto none = [](int) {};
  auto turn_whole = [&](int t) W4_INLINE {
    turn(t, std::false_type{}, 0);
#pragma unroll
    for (int x = 0; x < DB; ++x) rest_kv(x);
  };
  if (tiles > 0) {
    if (!plain) {
      for (int i = 0; i <= NB; ++i) fetch_ids(i);
      wait_vm<0>();
    }
    get_k(0);
    if constexpr (NB > LAG) get_v(0);
    put_down();
    get_k(1);
    if (plain) off_v[0] = offset_of(NB - LAG), off_v[1] = offset_of(NB - 1);
  }
  {
    const uint16_t* src = g.q + (int64_t)(s.first + tok) * g.ldq + (int64_t)(kvh * p.G + row - tok * p.G) * D;
#pragma unroll
    for (int t = 0; t < STEPS; ++t) {
      const int d = 16 * t + 8 * h;
      f16x8 z = {};
      q[t] = d < D ? *reinterpret_cast<const f16x8*>(src + d) : z;
    }
  }
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  constexpr std::integral_constant<int, -1> alone{};
  if (live && full > 0) {
    if constexpr (FP8) put_down();
    meet();  // K of tile 0 (and 1)
#pragma unroll
    for (int e = 0; e < 16; ++e) sc[e] = 0.f;
#pragma unroll
    for (int st = 0; st < STEPS; ++st)
      sc = __builtin_amdgcn_mfma_f32_32x32x16_f16(k_frag(k_tile(0), st), q[st], sc, 0, 0, 0);
    top = top_of(sc);
    if constexpr (SUB == 2) {
      block(yes, no, k_tile(0) + HALF, 0, none, alone);
      auto step = [&](int t, auto inner, int phase) W4_INLINE {  // phase: t % 2
        turn(t, inner, phase);
        block(yes, yes, k_tile(phase + 1), v_tile(phase), rest_kv, std::integral_constant<int, 0>{});
        block(yes, yes, k_tile(phase + 1) + HALF, v_tile(phase) + HALF, none, std::integral_constant<int, 1>{});
      };
      // as many tiles a round as buffers, so that LDS addresses are a lane's base and a constant
      int t = 0;
      for (; t + 3 < full; t += 2) {
        step(t, yes, 0);
        step(t + 1, yes, 1);
      }
      while (t + 1 < full) {
        step(t++, no, 0);
        if (t + 1 < full) step(t++, no, 1);
      }
      turn_whole(full - 1);
      block(no, yes, 0, v_tile(full - 1), none, alone);
    } else {
      turn_whole(0);
      if (full == 1) {
        block(no, no, 0, 0, none, alone);
      } else {
        block(yes, no, k_tile(1), 0, none, alone);
        auto step = [&](int t, auto inner, int phase) W4_INLINE {  // phase: t % NB
          turn(t, inner, phase);
          block(yes, yes, k_tile(phase + 1), v_tile(phase + NB - 1), rest_kv, alone);
        };
        int t = 1;
        for (; t + 2 * NB - 1 < full; t += NB) {
          step(t, yes, 1);
          step(t + 1, yes, 0);
        }
        while (t + 1 < full) {
          step(t++, no, 1);
          if (t + 1 < full) step(t++, no, 0);
        }
        turn_whole(full - 1);
        block(no, yes, 0, v_tile(full - 2), none, alone);
      }
      put_down();
      meet();  // V of the last
      get_v(full);
    }
#pragma unroll
    for (int x = 0; x < 2 * DB; ++x)
      acc[x / 2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v_frag(v_tile(full - 1) + (SUB - 1) * HALF, x), w[x & 1],
                                                         acc[x / 2], 0, 0, 0);
  } else if (full > 0) {  // a wave of no rows: the same barriers and fetches
    put_down();
    meet();
    for (int t = 0; t < full; ++t) turn_whole(t);
    put_down();
    if constexpr (SUB == 1) {
      meet();
      get_v(full);
    }
  } else if (LAG == NB) {
    get_v(0);
  }
  // on their way or there: K of tiles full .. full + NB - 1, V of full
  for (int i = full; i < turns; ++i) {
    put_down();
    meet();
    if (i > full) get_k(i + NB - 1);
    get_v(i + 1);
    fetch_ids(i + 3);
    if (live && there(i)) edge(i);
  }

  // The sums, acc[i][e]: dim 32 i + 8 (e / 4) + 4 h + e % 4 of this lane's row, go through LDS, 128 dims at a time, so
  // that rows are written whole.  Four dims x of row r of the wave's 32 lie at x ^ r (mod what 128 dims hold).
  l = across<false>(l, add2);
  constexpr int DW = DP < 128 ? DP : 128, XW = DW / 4;  // dims of a round, in fours
  static_assert(ROWS * DW * 4 <= KS * SPACE, "the rows fit where the tiles were");
  unsigned char* mine = lds + rg * 32 * DW * 4;
  auto four_of = [&](int r, int x) W4_INLINE { return reinterpret_cast<f32x4*>(mine + r * DW * 4 + (x ^ (r % XW)) * 16); };
  const int rows = live && kg == 0 ? wr1 - wr0 : 0;
  wait_vm<0>();     // no DMA is on its way to LDS any more
  __syncthreads();  // the tiles have been read
  if constexpr (KS == 2) {  // the second half of the keys' sums are handed over, lane by lane
    static_assert(RG * (DB * 16 + 4) * 256 <= KS * SPACE, "a wave's sums fit where its tiles were");
    f32x4* give = reinterpret_cast<f32x4*>(lds + rg * (DB * 16 + 4) * 256) + lane;
    if (kg == 1) {
#pragma unroll
      for (int i = 0; i < DB * 4; ++i) {
        f32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = acc[i / 4][i % 4 * 4 + e];
        give[i * 64] = o;
      }
      give[DB * 4 * 64] = {m, l, 0.f, 0.f};
    }
    __syncthreads();
    if (kg == 0) {
      const f32x4 ml = give[DB * 4 * 64];
      const float top1 = fmaxf(m, ml[0]);
      // a half that saw none of the row's keys has l = 0 and sums of 0, or NaN from NaN keys
      const float f0 = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - top1);
      const float f1 = ml[0] == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(ml[0] - top1);
      l = l * f0 + ml[1] * f1;
      m = top1;
#pragma unroll
      for (int i = 0; i < DB * 4; ++i) {
        const f32x4 o = give[i * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i / 4][i % 4 * 4 + e] = acc[i / 4][i % 4 * 4 + e] * f0 + o[e] * f1;
      }
    }
    __syncthreads();
    if (kg == 1) return;
  }
  const float f = (TREE ? tree.any : see1 > 0) ? (FP8 && g.c.v_scale ? g.c.v_scale[kvh] : 1.f) / l : 0.f;
#pragma unroll
  for (int d0 = 0; d0 < DP; d0 += DW) {
#pragma unroll
    for (int i = 0; i < DW / 32; ++i)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        f32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = acc[d0 / 32 + i][4 * a + e] * (k.act > 1 ? 1.f : f);
        *four_of(lane & 31, 8 * i + 2 * a + h) = o;
      }
    wait_lds();
    if (k.act > 1) {
      for (int i = lane; i < rows * XW; i += 64) {
        const int r = i / XW, x = i % XW;
        if (d0 + 4 * x < D)
          *reinterpret_cast<f32x4*>(part_row(p, part, kvh, wr0 - r0 + r) + d0 + 4 * x) = *four_of(r, x);
      }
    } else {
      for (int i = lane; i < rows * XW / 2; i += 64) {
        const int r = i / (XW / 2), x = i % (XW / 2) * 2, at = wr0 + r, tk = divide(at, p.group);
        if (d0 + 4 * x < D) {
          const f32x4 o0 = *four_of(r, x), o1 = *four_of(r, x + 1);
          f16x8 o;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = (f16)o0[e], o[4 + e] = (f16)o1[e];
          *reinterpret_cast<f16x8*>(g.out + (int64_t)(s.first + tk) * g.ldo + (int64_t)(kvh * p.G + at - tk * p.G) * D +
                                    d0 + 4 * x) = o;
        }
      }
    }
    wait_lds();
  }
  if (k.act > 1 && h == 0 && lane < rows) {
    float* to_ml = part_row(p, part, kvh, wr0 - r0 + lane) + D;
    to_ml[0] = m, to_ml[1] = l;
  }
}

// ------------------------------------------------------------------------------- the parts
// A row whose keys were in several parts: with M = max m, the sum of 2^(m_s - M) (sums_s, l_s).  Parts come
// in batches, running as in the kernels above, so that a batch's loads are in flight together.  Bound:
// latency (head, then the parts).  A workgroup of four waves takes one row, a quarter of the parts
// each (WIDE), or a row per wave.  3.5 us for 13 parts of one token's 16 rows of 128 dims, 5.2 for 32 parts of 512
// rows.
template <bool FEW, bool WIDE, int EL, bool TREE>
__global__ __launch_bounds__(256) void attention_join_kernel(Plan p) {
  typedef float vec __attribute__((ext_vector_type(EL)));
  constexpr int BATCH = WIDE ? 8 : 4, STEP = WIDE ? 4 : 1;
  __shared__ vec sums[4][64];
  __shared__ float mls[4][2];
  const AttnArgs& g = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), D = g.c.dim, d = lane * EL;
  const int blocks = WIDE ? p.part_rows : (p.part_rows + 3) / 4;  // of an item
  const int item = blockIdx.x / blocks, in = blockIdx.x - item * blocks;
  const int kvh = item % g.c.heads;
  const int4 head = p.head[item / g.c.heads];
  const int b = FEW ? item / g.c.heads : head.z, r0 = FEW ? 0 : head.w * p.part_rows;
  const int count = head.y, first = head.x;
  if (!FEW && count <= 1) return;  // no such tile, or written already
  const Seq s = sequence(g, b);
  const int all_rows = s.n * p.G;
  if (FEW && (s.n == 0 || (p.skip_short && all_rows > kFewRows) || count <= 1)) return;
  const int r = WIDE ? in : in * 4 + wave;
  if (r >= min(all_rows - r0, p.part_rows)) return;  // whole workgroups if WIDE
  vec o = 0.f;
  float l = 0.f, m = -INFINITY;
  for (int x0 = WIDE ? wave : 0; x0 < count; x0 += BATCH * STEP) {
    float om[BATCH], ol[BATCH];
    vec ov[BATCH];
#pragma unroll
    for (int y = 0; y < BATCH; ++y) {
      const int x = x0 + y * STEP;
      om[y] = -INFINITY, ol[y] = 0.f, ov[y] = 0.f;
      if (x < count) {
        const float* from = part_row(p, first + x, kvh, r);
        om[y] = from[D], ol[y] = from[D + 1];
        if (d < D) ov[y] = *reinterpret_cast<const vec*>(from + d);
      }
    }
    float top = m;
#pragma unroll
    for (int y = 0; y < BATCH; ++y) top = fmaxf(top, om[y]);
    const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
    l *= f, o *= f;
#pragma unroll
    for (int y = 0; y < BATCH; ++y) {
      const float fy = om[y] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(om[y] - top);
      // a part that saw none of the row's keys (m at -infinity) has l = 0 and sums of 0, or NaN from NaN keys
      l += om[y] == -INFINITY ? ol[y] : ol[y] * fy;
      o += om[y] == -INFINITY ? ov[y] : ov[y] * fy;
    }
    m = top;
  }
  if constexpr (WIDE) {
    sums[wave][lane] = o;
    if (lane == 0) mls[wave][0] = m, mls[wave][1] = l;
    __syncthreads();
    if (wave != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, mls[w][0]);
    l = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = mls[w][0] == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(mls[w][0] - top);
      l += mls[w][1] * f;
      o += sums[w][lane] * f;
    }
  }
  if (d >= D) return;
  const int row = r0 + r, tok = divide(row, p.group);
  bool any = s.len - s.n + tok >= 0;
  if constexpr (TREE) any = (!g.window && s.len > s.n) || tree_row(g, s, tok).any;
  const float f = any ? (g.c.e4m3 && g.c.v_scale ? g.c.v_scale[kvh] : 1.f) / l : 0.f;
  uint16_t* out = g.out + (int64_t)(s.first + tok) * g.ldo + (int64_t)(kvh * p.G + row - tok * p.G) * D + d;
  typedef uint16_t bits __attribute__((ext_vector_type(EL)));
  bits h;
#pragma unroll
  for (int e = 0; e < EL; ++e) h[e] = __builtin_bit_cast(uint16_t, (f16)(o[e] * f));
  *reinterpret_cast<bits*>(out) = h;
}

// ------------------------------------------------------------------------------- the launch
// Which kernels run: the one for few rows if no sequence has more than 16 rows, by max_q; the
// other if all have the same number (or there is one): both, each leaving the other's sequences, when
// they may differ.  So a single token of a group of more than 16 heads goes to the one for many: eight of 8192 tokens and one
// kv head of 128 dims take 19.2 us with 32 heads, 22.8 with 64, and 16.0 with 16.
struct Launch {
  bool few, many;
  int few_splits, few_parts, few_rows, few_least;  // few_parts 0: one workgroup per (sequence, kv head), no parts
  int many_splits, many_rows, tiles;
  bool tree;       // trees: attention_tree.hip's kernel
  int start_keys;  // trees: see Plan
  int tree_parts;  // trees: of all tiles, at most (many_splits: about)
  size_t few_bytes, many_bytes;
};

constexpr int kCus = 256;

// The decode kernel's workgroups that a CU holds, and their waves.
struct FewShape {
  int per_cu, waves;
};
template <int DP, bool FP8>
FewShape few_shape() { return {few_per_cu<DP, FP8>(), few_waves<DP, FP8>()}; }
FewShape few_shape_of(const AttnArgs& a) {
  const int d = a.c.dim;
  return a.c.e4m3 ? d <= 64 ? few_shape<64, true>() : d <= 128 ? few_shape<128, true>() : few_shape<256, true>()
                  : d <= 64 ? few_shape<64, false>() : d <= 128 ? few_shape<128, false>() : few_shape<256, false>();
}

// Up to how many rows, and words of a mask: 16 sequences of up to 4096 keys, 8 kv heads, in that kernel and in the one for many rows:
// e4m3, 128 dims: 64 rows 39.1 / 46.5 us, 96 rows 46.5 / 48.8, 128 rows 54.2 / 52.6; 256 dims, 96 rows 75.5 / 91.7;
// f16, 128 dims: 64 rows 46.6 / 51.1, 96 rows 52.5 / 52.4, 128 rows 69.8 / 55.5; 256 dims, 64 rows 102 / 97 (two
// sequences 30 / 39), 96 rows 120 / 101; 64 dims, 80 rows 33.7 / 38.6, 128 rows 41.8 / 40.4.  (The number of sequences is not asked:
// with 64 rows of 256 dims in f16 the many lose 5 % by it, the few gain 23.)
int tree_most(const AttnArgs& a) { return a.c.e4m3 || a.c.dim <= 64 ? 96 : 64; }
constexpr int kTreeWords = 2;
template <int DP>
constexpr int tree_blocks() { return DP == 256 ? 2 : 4; }  // of 16 rows
template <int DP, bool FP8>
constexpr int tree_waves() { return few_tile<DP, FP8>() == 8192 ? 8 : 4; }
template <int DP, bool FP8>
constexpr int tree_buffers() { return few_tile<DP, FP8>() > 2048 ? 1 : 2; }
template <int DP, bool FP8>
constexpr int tree_per_cu() { return few_tile<DP, FP8>() <= 4096 ? 2 : 1; }  // workgroups
// a wave's tiles and page numbers; then the queries and masks
template <int DP, bool FP8>
constexpr int tree_wave_lds() {
  return 2 * tree_buffers<DP, FP8>() * few_tile<DP, FP8>() + 256 * WaveTiles<DP, FP8, 1, tree_buffers<DP, FP8>()>::IDS;
}
template <int DP, bool FP8>
constexpr int tree_lds() { return tree_waves<DP, FP8>() * tree_wave_lds<DP, FP8>() + 16 * tree_blocks<DP>() * (DP * 2 + 8 * kTreeWords); }
int tree_rows(const AttnArgs& a) { return 16 * (a.c.dim <= 128 ? tree_blocks<128>() : tree_blocks<256>()); }
int tree_per_cu_of(const AttnArgs& a) {
  const int d = a.c.dim;
  return a.c.e4m3 ? d <= 64 ? tree_per_cu<64, true>() : d <= 128 ? tree_per_cu<128, true>() : tree_per_cu<256, true>()
                  : d <= 64 ? tree_per_cu<64, false>() : d <= 128 ? tree_per_cu<128, false>() : tree_per_cu<256, false>();
}

// Trees of many rows: rows of a tile, and about how many parts there should be of all tiles together, for one round of the
// workgroups that the CUs hold.
template <class F>
void plan_tree(const AttnArgs& a, int64_t most, F row_tiles, Launch& x) {
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.c.heads);
  x.tree = rows <= tree_most(a);
  // The kernel for many rows in tiles of 128: 64 take 140 us against 127 for 4 sequences of 61 to 200 rows of two heads,
  // 256 dims, a window of 4096, 168 and 124 at 128 dims without it in e4m3, 24 and 22 for one of 512 rows and 4096 keys.
  x.many_rows = x.tree ? tree_rows(a) : 128;
  const int per_cu = x.tree ? tree_per_cu_of(a) : a.c.dim <= 128 ? many_per_cu<128>() : many_per_cu<256>();
  // What a workgroup takes to start and end, and its part to be joined, as keys of 128 dims, in either kernel.  With 250, 500, 1000
  // and 2000 of them 16 sequences of 7 to 16 rows of two heads, 256 dims, 301 to 8192 keys, take 130, 130, 122 and 123 us; 4 of 61 to 200 with a
  // window of 4096 127 with 250 and 500, 123 with 1000; some twenty other shapes the same time with any.
  x.start_keys = 1000 * 128 / std::max(a.c.dim, 64);
  const int64_t tiles = row_tiles(x.many_rows), slots = std::max(1, per_cu * kCus / a.c.heads);
  const int64_t keys = a.window ? std::min(most, (int64_t)a.window + a.max_q + 64) : most;
  x.tiles = (int)tiles;
  x.many_splits = (int)slots;
  // at most; whole tiles where they are many rounds
  x.tree_parts = (int)(tiles > 8 * slots ? tiles : std::min(2 * slots + tiles, tiles * ((keys + kMinPart - 1) / kMinPart)));
}

// Lengths are on the device, so that the table's width stands for every sequence's.  Where it is much wider than they
// are, calls are cut for longer ones (16 heads on 2 of 128 dims, tables as wide as needed / of 1024 pages of 16): a
// prompt of 1570 tokens 30.6 / 37.9 us (128 rows in two parts), 300 after 2000 27.7 / 30.3, one token after 200 8.1 /
// 9.7, 64 after 1000 on 8 kv heads 42 / 50 (parts and a join), one after 1570, 4 x 8 after 16384 the same.
Launch plan(const AttnArgs& a) {
  Launch x{};
  const int G = a.Hq / a.c.heads;
  const int64_t most = (int64_t)a.W * a.c.page_size;
  x.few = (int64_t)a.max_q * G <= kFewRows;
  x.many = !x.few;
  if (x.many && !a.mask && a.B > 1 && G <= kFewRows && (int64_t)a.B * a.max_q != a.T) x.few = true;
  const size_t row = (size_t)(a.c.dim + 4) * sizeof(float);
  if (x.few) {
    // at most: 16 tokens' window, from a multiple of 16
    const int64_t keys = a.window ? std::min(most, (int64_t)a.window + 2 * kFewRows) : most;
    x.few_rows = (int)std::min<int64_t>(kFewRows, (int64_t)a.max_q * G);
    // A workgroup per (sequence, kv head) and no join while its waves have three tiles each (250 keys of 2 kv heads:
    // 8.1 us against 10.1, 500: 11.0 and 9.6), or 16 and there is a wave for every SIMD without parts (64 equal
    // sequences of 1000 on 8 kv heads 49.5 us against 58.7; of 1 to 2000, 58.2 and 65.5).
    const FewShape shape = few_shape_of(a);
    const int alone = (int64_t)a.B * a.c.heads * shape.waves >= 4 * kCus ? 16 : 3;
    if (keys > (int64_t)alone * kFewKeys * shape.waves) {
      // one round of the workgroups that the CUs hold, in parts of equal length (their number exceeds
      // few_splits by at most one per sequence); with more sequences than that, two parts each, for balance
      const int slots = kCus * shape.per_cu / a.c.heads;
      x.few_splits = std::max(slots - a.B, 2 * a.B);
      // (keys + per - 1) / per parts of each sequence at most
      // Two tiles of each of four waves where one would make more than a workgroup a CU: one sequence of 20000 on 2 kv
      // heads 16.0 us against 20.0, 8 of 4096 with two rows each 15.8 and 17.3; with two waves (3 of 1500, 256 dims,
      // 8 kv heads) 22.9 and 20.4.
      x.few_least = shape.waves == 4 && a.B * ((keys + kMinPart - 1) / kMinPart) * a.c.heads > kCus ? 2 * kMinPart : kMinPart;
      x.few_parts = (int)std::min<int64_t>((int64_t)x.few_splits + a.B, a.B * ((keys + x.few_least - 1) / x.few_least));
      x.few_bytes = (size_t)a.B * sizeof(int4) + (size_t)x.few_parts * a.c.heads * x.few_rows * row;
    }
  }
  if (x.many) {
    auto row_tiles = [&](int rows) {  // at most: by all rows, and by max_q
      return std::min((int64_t)a.T * G / rows + std::min(a.B, a.T), a.B * (((int64_t)a.max_q * G + rows - 1) / rows));
    };
    // Rows of a tile and parts of a row: what takes least by this sum, in us.  Its terms are measured alone; the sum at 128
    // dims is 35.6 for the 1570-token prompt (30.6 measured), 554 for the chunk of 4096 (501), 21.5 for 300
    // tokens after 2000 (27.7), 18.3 for the drafts (26.9: the join grows with the parts).  A workgroup starts and ends in 5, and goes over 64 keys in `turn`, alone
    // or two on its CU; f32 parts are written and read at 4 TB/s, by one more launch.  Parts fill a round of
    // the workgroups that the CUs hold, or one for each CU: four sequences of 8 new tokens after 16384 (16 heads on 2)
    // take 29 us in 64 parts and 26 in 32, 256 new tokens 55 in 8 and 67 in 4; 200 after 2048 (32 on 8), 36 in
    // 5 that exceed the round, and 27 in 4.  64 rows: a prompt of 1570 tokens 31.6, in 128 rows 39.
    constexpr float kTurn[2][2] = {{.87f, 1.2f}, {1.4f, 2.14f}};
    const int per_cu = a.c.dim <= 128 ? many_per_cu<128>() : many_per_cu<256>();
    float least = INFINITY;
    for (int rows = 64; rows <= 128; rows *= 2) {
      const int64_t tiles = row_tiles(rows), items = tiles * a.c.heads;
      const int64_t keys = a.window ? std::min(most, (int64_t)a.window + rows) : most;
      for (int fill = 0; fill <= per_cu; ++fill) {
        const int64_t splits = std::max<int64_t>(1, std::min((keys + 127) / 128, fill * kCus / items));
        const int64_t wgs = items * splits, round = per_cu * kCus;
        const float turn = kTurn[rows / 128][wgs > kCus && per_cu > 1] * std::max(a.c.dim, 64) / 128;
        const float us = (float)((wgs + round - 1) / round) * (5.f + (float)(keys / splits) / 64.f * turn) +
                         (splits > 1 ? 2.f + (float)wgs * rows * (float)row * 2.f / 4e6f : 0.f);
        if (us >= least) continue;
        least = us;
        x.many_rows = rows, x.tiles = (int)tiles, x.many_splits = (int)splits;
      }
    }
    if (a.mask) plan_tree(a, most, row_tiles, x);
    const int64_t items = (int64_t)x.tiles * a.c.heads;
    if (a.mask) {
      if (x.tree_parts > x.tiles)
        x.many_bytes = (size_t)x.tiles * sizeof(int4) + (size_t)x.tree_parts * a.c.heads * x.many_rows * row;
    } else if (x.many_splits > 1)
      x.many_bytes = (size_t)x.tiles * sizeof(int4) + (size_t)items * x.many_splits * x.many_rows * row;
  }
  return x;
}

// Whether every launch stays below 2^32 threads, which is as many as one takes.
bool launchable(const Launch& x, const AttnArgs& a) {
  constexpr int64_t kMost = ((int64_t)1 << 32) / 256;  // workgroups
  const int64_t heads = a.c.heads;
  if (x.few) {
    if ((x.few_parts ? x.few_parts : a.B) * heads >= kMost) return false;
    if (x.few_parts && a.B * heads * x.few_rows >= kMost) return false;
  }
  if (x.many && a.mask) return (int64_t)x.tree_parts * heads < kMost / 2;  // of 512 threads
  return !x.many || x.tiles * heads * x.many_splits < kMost;  // parts are for few tiles: their join is small
}

template <int DP, bool FP8, bool TREE>
void launch_few(const Plan& p, int items, hipStream_t st) {
  static std::once_flag flags[kMaxDevices];
  once_per_device(flags, [] {
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(attention_few_kernel<DP, FP8, TREE>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, few_lds<DP, FP8>());
  });
  attention_few_kernel<DP, FP8, TREE><<<items, 64 * few_waves<DP, FP8>(), few_lds<DP, FP8>(), st>>>(p);
}

template <int DP, bool FP8, int KS, bool TREE>
void launch_many_ks(const Plan& p, int items, hipStream_t st) {
  static std::once_flag flags[kMaxDevices];
  once_per_device(flags, [] {
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(attention_many_kernel<DP, FP8, KS, TREE>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, many_lds<DP, KS>());
  });
  attention_many_kernel<DP, FP8, KS, TREE><<<TREE ? p.parts * p.a.c.heads : items * p.splits, 64 * kManyWaves, many_lds<DP, KS>(), st>>>(p);
}
template <int DP, bool FP8, bool TREE>
void launch_many(const Plan& p, int items, hipStream_t st) {
  if constexpr (!TREE) {
    if (p.part_rows == 64) return launch_many_ks<DP, FP8, 2, false>(p, items, st);
  }
  launch_many_ks<DP, FP8, 1, TREE>(p, items, st);
}

template <bool FEW, bool WIDE, bool TREE>
void launch_join(const Plan& p, int items, hipStream_t st) {
  const int D = p.a.c.dim, grid = items * (WIDE ? p.part_rows : (p.part_rows + 3) / 4);
  if (D <= 64)
    attention_join_kernel<FEW, WIDE, 1, TREE><<<grid, 256, 0, st>>>(p);
  else if (D <= 128)
    attention_join_kernel<FEW, WIDE, 2, TREE><<<grid, 256, 0, st>>>(p);
  else
    attention_join_kernel<FEW, WIDE, 4, TREE><<<grid, 256, 0, st>>>(p);
}

template <bool FP8>
void launch_tree(const Plan& p, hipStream_t st);  // attention_tree.hip's; no other file has TREE

template <bool FP8, bool TREE>
void launch_dims(const Launch& x, Plan p, char* ws, hipStream_t st) {
  const int D = p.a.c.dim, heads = p.a.c.heads;
  if (x.few) {
    p.splits = x.few_splits, p.least = x.few_least, p.part_rows = x.few_rows;
    p.head = reinterpret_cast<int4*>(ws);
    p.part = x.few_parts ? reinterpret_cast<float*>(ws + (size_t)p.a.B * sizeof(int4)) : nullptr;
    const int items = (x.few_parts ? x.few_parts : p.a.B) * heads;
    if (D <= 64) launch_few<64, FP8, TREE>(p, items, st);
    else if (D <= 128) launch_few<128, FP8, TREE>(p, items, st);
    else launch_few<256, FP8, TREE>(p, items, st);
    if (x.few_parts) launch_join<true, true, TREE>(p, p.a.B * heads, st);
  }
  if (x.many) {
    ws += x.few_bytes;
    p.splits = x.many_splits, p.part_rows = x.many_rows, p.tiles = x.tiles;
    p.head = reinterpret_cast<int4*>(ws);
    p.parts = x.tree_parts, p.start_keys = x.start_keys;
    p.part = (TREE ? x.tree_parts > x.tiles : x.many_splits > 1) ? reinterpret_cast<float*>(ws + (size_t)x.tiles * sizeof(int4)) : nullptr;
    const int items = x.tiles * heads;
    bool between = false;
    if constexpr (TREE)
      if (x.tree) launch_tree<FP8>(p, st), between = true;
    if (between) {
    } else if (D <= 64) {
      launch_many<64, FP8, TREE>(p, items, st);
    } else if (D <= 128) {
      launch_many<128, FP8, TREE>(p, items, st);
    } else {
      launch_many<256, FP8, TREE>(p, items, st);
    }
    // many parts: a workgroup per row
    // (trees: or few rows)
    if (p.part && ((TREE ? x.tree_parts / x.tiles : p.splits) >= 16 || (TREE && items * x.many_rows <= 2048))) launch_join<false, true, TREE>(p, items, st);
    else if (p.part) launch_join<false, false, TREE>(p, items, st);
  }
}

// a.mask: a tree's (TREE) or none
template <bool TREE>
void launch_as(const AttnArgs& a, void* ws, hipStream_t st) {
  const Launch x = plan(a);
  Plan p{};
  p.a = a, p.G = a.Hq / a.c.heads, p.page = divider(a.c.page_size), p.group = divider(p.G);
  p.skip_short = x.few && x.many, p.c = a.scale * kLog2e;
  if (a.c.e4m3)
    launch_dims<true, TREE>(x, p, reinterpret_cast<char*>(ws), st);
  else
    launch_dims<false, TREE>(x, p, reinterpret_cast<char*>(ws), st);
}

}  // namespace

}  // namespace w4
