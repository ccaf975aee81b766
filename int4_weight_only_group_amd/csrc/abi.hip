// The C ABI (include/w4.h): argument checks on the host, then one launch path per call.
// Nothing here allocates device memory or keeps per-call state.
#include <atomic>
#include <cmath>
#include <cstring>

#include "../../include/w4.h"
#include "w4_internal.h"
#include "w4_kv.h"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;

inline bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool al4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
inline bool al2(const void* p) { return ((uintptr_t)p & 1u) == 0; }

std::atomic<int> g_device_ok[w4::kMaxDevices];  // 0 unknown, 1 gfx950, -1 other

int check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= w4::kMaxDevices) {
    (void)hipGetLastError();
    return W4_ERR_DEVICE;
  }
  int c = g_device_ok[dev].load(std::memory_order_relaxed);
  if (c == 0) {
    hipDeviceProp_t p;
    if (hipGetDeviceProperties(&p, dev) != hipSuccess) {
      (void)hipGetLastError();
      c = -1;
    } else {
      c = std::strncmp(p.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
    }
    g_device_ok[dev].store(c, std::memory_order_relaxed);
  }
  return c == 1 ? W4_OK : W4_ERR_DEVICE;
}

// Two-phase workspace protocol.  Returns 1 when the call was a size query (already
// answered), 0 to go on, or a negative status.
int workspace(void* ws, size_t* ws_bytes, size_t need) {
  if (ws == nullptr && ws_bytes != nullptr) {
    *ws_bytes = need;
    return 1;
  }
  if (need == 0) return 0;
  if (ws == nullptr || ws_bytes == nullptr || *ws_bytes < need) return W4_ERR_WORKSPACE;
  if (!al16(ws)) return W4_ERR_ALIGN;
  return 0;
}

int launched() { return hipGetLastError() == hipSuccess ? W4_OK : W4_ERR_LAUNCH; }

// [p, p + bytes) as integers, for overlap checks of device ranges
struct Span {
  uintptr_t lo, hi;
};
inline Span span(const void* p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes}; }
inline bool overlap(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

int check_w4_shape(int64_t N, int64_t K) {
  if (N < 1 || K < 64 || K % 64 != 0 || N > kMaxDim || K > kMaxDim) return W4_ERR_SHAPE;
  if (N * (K / 8) > ((int64_t)1 << 40)) return W4_ERR_SHAPE;
  return W4_OK;
}

// gemm_f16_dequant_next and its symmetric group-128 twin (sym: no biases, K % 128 == 0, one
// scale per 128 codes): gemm_f16's and the dequant's checks, the GEMM's workspace, then the
// overlap checks (the two operations run at once), then one launch path.
int gemm_dequant_next(const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb, float* C, int64_t ldc, int64_t M,
                      int64_t N, int64_t K, void* ws, size_t* ws_bytes, const uint32_t* qw, const uint16_t* scales,
                      const uint16_t* biases, uint16_t* wt, int64_t ldwt, int64_t Nq, int64_t Kq, bool sym,
                      w4_stream_t stream) {
  // the GEMM's checks (gemm_f16) ...
  if (!A || !B || !C || !qw || !scales || !wt) return W4_ERR_NULL;
  if (M < 1 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return W4_ERR_SHAPE;
  if (lda < K || ldb < N || ldc < N || lda > kMaxDim || ldb > kMaxDim || ldc > kMaxDim) return W4_ERR_SHAPE;
  if (!al2(A) || !al2(B) || !al4(C)) return W4_ERR_ALIGN;
  if (w4::gemm_path(A, lda, B, ldb, M, N, K) == w4::kGemmPlain && (M + 15) / 16 > 65535) return W4_ERR_SHAPE;
  // ... and the dequant's (w4_dequant_f16_t, w4_dequant_f16_t_sym128)
  if (int e = check_w4_shape(Nq, Kq)) return e;
  if (sym && Kq % 128 != 0) return W4_ERR_SHAPE;
  if (ldwt < Nq || ldwt > kMaxDim || Nq > 65535 * 64) return W4_ERR_SHAPE;
  if (!al16(qw) || !al16(scales) || (!sym && !al16(biases)) || !al2(wt)) return W4_ERR_ALIGN;
  const size_t need = w4::gemm_ws_bytes(A, lda, B, ldb, M, N, K);
  const int w = workspace(ws, ws_bytes, need);
  if (w < 0) return w;
  if (w == 1) return W4_OK;
  // the two run at once: neither's outputs may overlap the other's operands or outputs
  const int64_t groups = Nq * (Kq / (sym ? 128 : 64));
  const Span a = span(A, ((M - 1) * lda + K) * 2), b = span(B, ((K - 1) * ldb + N) * 2);
  const Span c = span(C, ((M - 1) * ldc + N) * 4), wk = span(ws, need ? (int64_t)need : 0);
  const Span q = span(qw, Nq * Kq / 2), sc = span(scales, groups * 2), bi = span(biases, sym ? 0 : groups * 2),
             t = span(wt, ((Kq - 1) * ldwt + Nq) * 2);
  for (const Span& x : {a, b, c, wk, q, sc, bi})
    if (overlap(t, x)) return W4_ERR_OVERLAP;
  for (const Span& x : {q, sc, bi})
    if (overlap(c, x) || overlap(wk, x)) return W4_ERR_OVERLAP;
  if (int e = check_device()) return e;
  (void)hipGetLastError();
  w4::launch_gemm_dequant(A, lda, B, ldb, C, ldc, (int)M, (int)N, (int)K, ws, qw, scales, biases, wt, ldwt, (int)Nq,
                          (int)Kq, sym, (hipStream_t)stream);
  return launched();
}

constexpr int64_t kMaxTokens = (int64_t)1 << 24, kMaxHeads = 1024, kMaxHeadDim = 256;

// x rows [T][H][D] (f16 or f32, the heads of a token contiguous) and their rotation
int check_rows(const void* x, int64_t ld, int64_t H, int64_t D) {
  if (H < 1 || H > kMaxHeads || ld < H * D || ld > kMaxDim) return W4_ERR_SHAPE;
  if (!al16(x) || ld % 8 != 0) return W4_ERR_ALIGN;
  return W4_OK;
}
int check_rope(int64_t T, int64_t D, int64_t R, int32_t x_type, const int32_t* pos, const float* freq, float mscale) {
  if (!pos || (!freq && R > 0)) return W4_ERR_NULL;
  if (T < 1 || T >= kMaxTokens || D < 8 || D > kMaxHeadDim || D % 8 != 0 || R < 0 || R > D || R % 2 != 0)
    return W4_ERR_SHAPE;
  if ((x_type != W4_F16 && x_type != W4_F32) || !std::isfinite(mscale)) return W4_ERR_SHAPE;
  if (!al4(pos) || !al4(freq)) return W4_ERR_ALIGN;
  return W4_OK;
}

int check_norm(const w4::HeadNorm& n) {
  if (!(n.eps >= 1e-30f && n.eps <= 1e30f)) return W4_ERR_SHAPE;
  return al16(n.q) && al16(n.k) ? W4_OK : W4_ERR_ALIGN;
}

// w4_kv_cache's requirements; on W4_OK c is the kernels' view of it
int check_cache(const w4_kv_cache* h, w4::KvCache& c) {
  if (!h || !h->k || !h->v) return W4_ERR_NULL;
  if (h->type != W4_F16 && h->type != W4_E4M3) return W4_ERR_SHAPE;
  const bool e4m3 = h->type == W4_E4M3;
  const int64_t unit = e4m3 ? 16 : 8, most = ((int64_t)1 << 31) - 1;
  if (h->pages < 1 || h->page_size < 1 || h->pages > most || h->page_size > most / h->pages) return W4_ERR_SHAPE;
  if (h->heads < 1 || h->heads > kMaxHeads || h->dim < 8 || h->dim > kMaxHeadDim || h->dim % unit != 0)
    return W4_ERR_SHAPE;
  for (int64_t s : {h->stride_page, h->stride_head, h->stride_token}) {
    if (s < 0 || s > ((int64_t)1 << 40)) return W4_ERR_SHAPE;
    if (s % unit != 0) return W4_ERR_ALIGN;
  }
  if (!al16(h->k) || !al16(h->v) || !al4(h->k_scale) || !al4(h->v_scale)) return W4_ERR_ALIGN;
  c = {h->k, h->v, h->k_scale, h->v_scale, h->stride_page, h->stride_head, h->stride_token,
       (int)h->pages, (int)h->page_size, (int)h->heads, (int)h->dim, e4m3};
  return W4_OK;
}

}  // namespace

extern "C" {

const char* w4_strerror(int status) {
  switch (status) {
    case W4_OK: return "ok";
    case W4_ERR_NULL: return "a required pointer is NULL";
    case W4_ERR_SHAPE: return "a size is out of the supported range";
    case W4_ERR_ALIGN: return "a pointer or leading dimension is misaligned";
    case W4_ERR_WORKSPACE: return "the workspace is too small";
    case W4_ERR_DEVICE: return "no usable gfx950 device is current";
    case W4_ERR_LAUNCH: return "the HIP runtime rejected a kernel launch";
    case W4_ERR_INTERNAL: return "internal error";
    case W4_ERR_OVERLAP: return "an output of one operation overlaps an operand of the other";
    default: return "unknown status";
  }
}

int w4_pack(const uint8_t* q, uint32_t* qw, int64_t N, int64_t K, w4_stream_t stream) {
  try {
    if (!q || !qw) return W4_ERR_NULL;
    if (int e = check_w4_shape(N, K)) return e;
    if (!al16(q) || !al16(qw)) return W4_ERR_ALIGN;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_pack(q, qw, N, K, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int w4_gemv(const uint32_t* qw, const uint16_t* scales, const uint16_t* biases, const uint16_t* x,
            int64_t ldx, float* y, int64_t ldy, int64_t M, int64_t N, int64_t K, void* ws,
            size_t* ws_bytes, w4_stream_t stream) {
  try {
    if (!qw || !scales || !biases || !x || !y) return W4_ERR_NULL;
    if (int e = check_w4_shape(N, K)) return e;
    if (M < 1 || M > 16 || ldx < K || ldy < N || ldx > kMaxDim || ldy > kMaxDim) return W4_ERR_SHAPE;
    if (!al16(qw) || !al16(scales) || !al16(biases) || !al16(x) || !al4(y) || ldx % 8 != 0)
      return W4_ERR_ALIGN;
    const int w = workspace(ws, ws_bytes, w4::gemv_ws_bytes(M, N, K));
    if (w < 0) return w;
    if (w == 1) return W4_OK;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_gemv(qw, scales, biases, x, ldx, y, ldy, (int)M, (int)N, (int)K,
                    w4::gemv_ws_bytes(M, N, K) ? ws : nullptr, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int w4_quantize(const uint16_t* w, int64_t ldw, uint32_t* qw, uint16_t* scales, uint16_t* biases,
                int64_t N, int64_t K, w4_stream_t stream) {
  try {
    if (!w || !qw || !scales || !biases) return W4_ERR_NULL;
    if (int e = check_w4_shape(N, K)) return e;
    if (ldw < K || ldw > kMaxDim) return W4_ERR_SHAPE;
    if (!al16(w) || ldw % 8 != 0 || !al16(qw) || !al2(scales) || !al2(biases)) return W4_ERR_ALIGN;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_quantize(w, ldw, qw, scales, biases, N, K, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int w4_gemv_sym128(const uint32_t* qw, const uint16_t* scales, const uint16_t* x, int64_t ldx,
                   float* y, int64_t ldy, int64_t M, int64_t N, int64_t K, void* ws, size_t* ws_bytes,
                   w4_stream_t stream) {
  try {
    if (!qw || !scales || !x || !y) return W4_ERR_NULL;
    if (int e = check_w4_shape(N, K)) return e;
    if (K % 128 != 0) return W4_ERR_SHAPE;
    if (M < 1 || M > 16 || ldx < K || ldy < N || ldx > kMaxDim || ldy > kMaxDim) return W4_ERR_SHAPE;
    if (!al16(qw) || !al16(scales) || !al16(x) || !al4(y) || ldx % 8 != 0) return W4_ERR_ALIGN;
    const int w = workspace(ws, ws_bytes, w4::gemv_ws_bytes(M, N, K));
    if (w < 0) return w;
    if (w == 1) return W4_OK;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_gemv_sym128(qw, scales, x, ldx, y, ldy, (int)M, (int)N, (int)K,
                           w4::gemv_ws_bytes(M, N, K) ? ws : nullptr, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int w4_dequant_f16_t_sym128(const uint32_t* qw, const uint16_t* scales, uint16_t* wt, int64_t ldwt,
                            int64_t N, int64_t K, w4_stream_t stream) {
  try {
    if (!qw || !scales || !wt) return W4_ERR_NULL;
    if (int e = check_w4_shape(N, K)) return e;
    if (K % 128 != 0) return W4_ERR_SHAPE;
    if (ldwt < N || ldwt > kMaxDim || N > 65535 * 64) return W4_ERR_SHAPE;
    if (!al16(qw) || !al16(scales) || !al2(wt)) return W4_ERR_ALIGN;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_dequant_t_sym128(qw, scales, wt, ldwt, (int)N, (int)K, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int w4_dequant_f16_t(const uint32_t* qw, const uint16_t* scales, const uint16_t* biases,
                     uint16_t* wt, int64_t ldwt, int64_t N, int64_t K, w4_stream_t stream) {
  try {
    if (!qw || !scales || !biases || !wt) return W4_ERR_NULL;
    if (int e = check_w4_shape(N, K)) return e;
    if (ldwt < N || ldwt > kMaxDim || N > 65535 * 64) return W4_ERR_SHAPE;
    if (!al16(qw) || !al16(scales) || !al16(biases) || !al2(wt)) return W4_ERR_ALIGN;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_dequant_t(qw, scales, biases, wt, ldwt, (int)N, (int)K, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int gemm_f16(const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb, float* C, int64_t ldc,
             int64_t M, int64_t N, int64_t K, void* ws, size_t* ws_bytes, w4_stream_t stream) {
  try {
    if (!A || !B || !C) return W4_ERR_NULL;
    if (M < 1 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return W4_ERR_SHAPE;
    if (lda < K || ldb < N || ldc < N || lda > kMaxDim || ldb > kMaxDim || ldc > kMaxDim)
      return W4_ERR_SHAPE;
    if (!al2(A) || !al2(B) || !al4(C)) return W4_ERR_ALIGN;
    if (w4::gemm_path(A, lda, B, ldb, M, N, K) == w4::kGemmPlain && (M + 15) / 16 > 65535)
      return W4_ERR_SHAPE;
    const int w = workspace(ws, ws_bytes, w4::gemm_ws_bytes(A, lda, B, ldb, M, N, K));
    if (w < 0) return w;
    if (w == 1) return W4_OK;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_gemm(A, lda, B, ldb, C, ldc, (int)M, (int)N, (int)K, ws, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int gemm_f16_dequant_next(const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb, float* C, int64_t ldc,
                          int64_t M, int64_t N, int64_t K, void* ws, size_t* ws_bytes, const uint32_t* qw,
                          const uint16_t* scales, const uint16_t* biases, uint16_t* wt, int64_t ldwt, int64_t Nq,
                          int64_t Kq, w4_stream_t stream) {
  try {
    if (!biases) return W4_ERR_NULL;
    return gemm_dequant_next(A, lda, B, ldb, C, ldc, M, N, K, ws, ws_bytes, qw, scales, biases, wt, ldwt, Nq, Kq,
                             false, stream);
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int gemm_f16_dequant_next_sym128(const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb, float* C,
                                 int64_t ldc, int64_t M, int64_t N, int64_t K, void* ws, size_t* ws_bytes,
                                 const uint32_t* qw, const uint16_t* scales, uint16_t* wt, int64_t ldwt, int64_t Nq,
                                 int64_t Kq, w4_stream_t stream) {
  try {
    return gemm_dequant_next(A, lda, B, ldb, C, ldc, M, N, K, ws, ws_bytes, qw, scales, nullptr, wt, ldwt, Nq, Kq,
                             true, stream);
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int logits_argmax_topk(const float* logits, int64_t ldl, int64_t M, int64_t V, int64_t k,
                       int32_t* idx, float* val, void* ws, size_t* ws_bytes, w4_stream_t stream) {
  try {
    if (!logits || !idx || !val) return W4_ERR_NULL;
    if (M < 1 || M > 65535 || V < 1 || V >= ((int64_t)1 << 31) || k < 1 || k > 256 || k > V ||
        ldl < V)
      return W4_ERR_SHAPE;
    if (w4::topk_chunk(V, (int)k) == 0) return W4_ERR_SHAPE;
    if (!al4(logits) || !al4(idx) || !al4(val)) return W4_ERR_ALIGN;
    const int w = workspace(ws, ws_bytes, w4::topk_ws_bytes(M, V, (int)k));
    if (w < 0) return w;
    if (w == 1) return W4_OK;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_topk(logits, ldl, (int)M, (int)V, (int)k, idx, val, ws, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int w4_gemv_topk(const uint32_t* qw, const uint16_t* scales, const uint16_t* biases, const uint16_t* x,
                 int64_t V, int64_t K, int64_t k, float* logits, int32_t* idx, float* val, void* ws,
                 size_t* ws_bytes, w4_stream_t stream) {
  try {
    if (!qw || !scales || !biases || !x || !logits || !idx || !val) return W4_ERR_NULL;
    if (int e = check_w4_shape(V, K)) return e;
    if (k < 1 || k > 64 || !w4::head_topk_supported(V, K, (int)k)) return W4_ERR_SHAPE;
    if (!al16(qw) || !al16(scales) || !al16(biases) || !al16(x) || !al4(logits) || !al4(idx) || !al4(val))
      return W4_ERR_ALIGN;
    const int w = workspace(ws, ws_bytes, w4::head_topk_ws_bytes(V, K, (int)k));
    if (w < 0) return w;
    if (w == 1) return W4_OK;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_head_topk(qw, scales, biases, x, logits, idx, val, (int)V, (int)K, (int)k, ws, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int logits_argmax_topk_noalloc(const float* logits, int64_t ldl, int64_t M, int64_t V, int64_t k,
                               int32_t* idx, float* val, w4_stream_t stream) {
  try {
    if (!logits || !idx || !val) return W4_ERR_NULL;
    if (M < 1 || M > 65535 || V < 1 || V >= ((int64_t)1 << 31) || k < 1 || k > 256 || k > V ||
        ldl < V)
      return W4_ERR_SHAPE;
    if (w4::topk_chunk(V, (int)k) == 0) return W4_ERR_SHAPE;
    if (!al4(logits) || !al4(idx) || !al4(val)) return W4_ERR_ALIGN;
    if (w4::topk_ws_bytes(M, V, (int)k) > w4::kTopkScratchBytes) return W4_ERR_WORKSPACE;
    if (int e = check_device()) return e;
    void* scratch = w4::topk_scratch();  // this device's copy of the library's array
    if (scratch == nullptr) return W4_ERR_INTERNAL;
    (void)hipGetLastError();
    w4::launch_topk(logits, ldl, (int)M, (int)V, (int)k, idx, val, scratch, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int rope_f16(const void* x, int32_t x_type, int64_t ldx, const int32_t* pos, const float* freq, uint16_t* y,
             int64_t ldy, int64_t T, int64_t H, int64_t D, int64_t R, int32_t interleaved, int32_t inverse,
             float mscale, w4_stream_t stream) {
  try {
    if (!x || !y) return W4_ERR_NULL;
    if (int e = check_rope(T, D, R, x_type, pos, freq, mscale)) return e;
    if (int e = check_rows(x, ldx, H, D)) return e;
    if (int e = check_rows(y, ldy, H, D)) return e;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_rope(x, x_type == W4_F32, ldx, pos, freq, y, ldy, (int)T, (int)H, (int)D, (int)R, interleaved != 0,
                    inverse != 0, mscale, nullptr, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int norm_rope_f16(const void* x, int32_t x_type, int64_t ldx, const float* weight, float eps, const int32_t* pos,
                  const float* freq, uint16_t* y, int64_t ldy, int64_t T, int64_t H, int64_t D, int64_t R,
                  int32_t interleaved, float mscale, w4_stream_t stream) {
  try {
    if (!x || !y) return W4_ERR_NULL;
    if (int e = check_rope(T, D, R, x_type, pos, freq, mscale)) return e;
    const w4::HeadNorm norm{weight, nullptr, eps};
    if (int e = check_norm(norm)) return e;
    if (int e = check_rows(x, ldx, H, D)) return e;
    if (int e = check_rows(y, ldy, H, D)) return e;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_rope(x, x_type == W4_F32, ldx, pos, freq, y, ldy, (int)T, (int)H, (int)D, (int)R, interleaved != 0, false,
                    mscale, &norm, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

}  // extern "C"

namespace {

// kv_append_rope, or kv_append_norm_rope with a norm
int append(const void* q, int64_t ldq, uint16_t* q_out, int64_t ldqo, int64_t Hq, const void* k, int64_t ldk,
           const void* v, int64_t ldv, int32_t x_type, const w4_kv_cache* cache, const int64_t* slot, const int32_t* pos,
           const float* freq, const w4::HeadNorm* norm, int64_t T, int64_t R, int32_t interleaved, float mscale,
           w4_stream_t stream) {
  try {
    if (!k || !v || !slot || (!q) != (!q_out)) return W4_ERR_NULL;
    w4::KvCache c;
    if (int e = check_cache(cache, c)) return e;
    if (int e = check_rope(T, c.dim, R, x_type, pos, freq, mscale)) return e;
    if (int e = check_rows(k, ldk, c.heads, c.dim)) return e;
    if (int e = check_rows(v, ldv, c.heads, c.dim)) return e;
    if (q) {
      if (int e = check_rows(q, ldq, Hq, c.dim)) return e;
      if (int e = check_rows(q_out, ldqo, Hq, c.dim)) return e;
    }
    if (((uintptr_t)slot & 7u) != 0) return W4_ERR_ALIGN;
    if (norm)
      if (int e = check_norm(*norm)) return e;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_kv_append(q, ldq, q_out, ldqo, (int)Hq, k, ldk, v, ldv, x_type == W4_F32, c, slot, pos, freq, (int)T,
                         (int)R, interleaved != 0, mscale, norm, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

// attention_paged, or attention_paged_tree with a mask
int attend(const uint16_t* q, int64_t ldq, const w4_kv_cache* cache, const int32_t* table, int64_t ldt, int64_t W,
           const int32_t* kv_len, const int32_t* q_start, const uint64_t* mask, int64_t ldm, int64_t B, int64_t T,
           int64_t max_q, int64_t Hq, int64_t window, float scale, uint16_t* out, int64_t ldo, void* ws,
           size_t* ws_bytes, w4_stream_t stream) {
  try {
    if (!q || !table || !kv_len || !out) return W4_ERR_NULL;
    w4::KvCache c;
    if (int e = check_cache(cache, c)) return e;
    if (T < 1 || T >= kMaxTokens || B < 1 || B > ((int64_t)1 << 20) || max_q < 1 || max_q > T) return W4_ERR_SHAPE;
    if (!q_start && (B > T || max_q != 1)) return W4_ERR_SHAPE;
    if (W < 1 || W > ((int64_t)1 << 30) / c.page_size || ldt < W || ldt > kMaxDim) return W4_ERR_SHAPE;
    if (Hq < 1 || Hq % c.heads != 0 || Hq > kMaxHeads || T * Hq > kMaxDim || window < 0) return W4_ERR_SHAPE;
    if (!(scale >= 1e-30f && scale <= 1e30f)) return W4_ERR_SHAPE;  // its product with log2 e is a normal number
    if (int e = check_rows(q, ldq, Hq, c.dim)) return e;
    if (int e = check_rows(out, ldo, Hq, c.dim)) return e;
    if (!al4(table) || !al4(kv_len) || !al4(q_start)) return W4_ERR_ALIGN;
    w4::AttnArgs a;
    a.q = q, a.out = out, a.ldq = ldq, a.ldo = ldo, a.c = c;
    a.table = table, a.ldt = ldt, a.kv_len = kv_len, a.q_start = q_start;
    a.W = (int)W, a.B = (int)B, a.T = (int)T, a.max_q = (int)max_q, a.Hq = (int)Hq;
    a.window = window >= ((int64_t)1 << 30) ? 0 : (int)window;  // no sequence is longer
    a.scale = scale;
    if (mask) {
      if (((uintptr_t)mask & 7u) != 0) return W4_ERR_ALIGN;
      if (ldm < (max_q + 63) / 64 || ldm > kMaxDim || (a.window && a.window < max_q)) return W4_ERR_SHAPE;
      a.mask = mask, a.ldm = ldm;
    }
    size_t need = 0;
    if (!w4::attention_ws_bytes(a, need)) return W4_ERR_SHAPE;
    const int w = workspace(ws, ws_bytes, need);
    if (w < 0) return w;
    if (w == 1) return W4_OK;
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    if (mask)
      w4::launch_attention_tree(a, need ? ws : nullptr, (hipStream_t)stream);
    else
      w4::launch_attention(a, need ? ws : nullptr, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

}  // namespace

extern "C" {

int kv_append_rope(const void* q, int64_t ldq, uint16_t* q_out, int64_t ldqo, int64_t Hq, const void* k, int64_t ldk,
                   const void* v, int64_t ldv, int32_t x_type, const w4_kv_cache* cache, const int64_t* slot,
                   const int32_t* pos, const float* freq, int64_t T, int64_t R, int32_t interleaved, float mscale,
                   w4_stream_t stream) {
  return append(q, ldq, q_out, ldqo, Hq, k, ldk, v, ldv, x_type, cache, slot, pos, freq, nullptr, T, R, interleaved,
                mscale, stream);
}

int kv_append_norm_rope(const void* q, int64_t ldq, uint16_t* q_out, int64_t ldqo, int64_t Hq, const void* k, int64_t ldk,
                        const void* v, int64_t ldv, int32_t x_type, const w4_kv_cache* cache, const int64_t* slot,
                        const int32_t* pos, const float* freq, const float* q_weight, const float* k_weight, float eps,
                        int64_t T, int64_t R, int32_t interleaved, float mscale, w4_stream_t stream) {
  const w4::HeadNorm norm{q_weight, k_weight, eps};
  return append(q, ldq, q_out, ldqo, Hq, k, ldk, v, ldv, x_type, cache, slot, pos, freq, &norm, T, R, interleaved, mscale,
                stream);
}

int attention_paged(const uint16_t* q, int64_t ldq, const w4_kv_cache* cache, const int32_t* table, int64_t ldt,
                    int64_t W, const int32_t* kv_len, const int32_t* q_start, int64_t B, int64_t T, int64_t max_q,
                    int64_t Hq, int64_t window, float scale, uint16_t* out, int64_t ldo, void* ws, size_t* ws_bytes,
                    w4_stream_t stream) {
  return attend(q, ldq, cache, table, ldt, W, kv_len, q_start, nullptr, 0, B, T, max_q, Hq, window, scale, out, ldo, ws,
                ws_bytes, stream);
}

int attention_paged_tree(const uint16_t* q, int64_t ldq, const w4_kv_cache* cache, const int32_t* table, int64_t ldt,
                         int64_t W, const int32_t* kv_len, const int32_t* q_start, const uint64_t* mask, int64_t ldm,
                         int64_t B, int64_t T, int64_t max_q, int64_t Hq, int64_t window, float scale, uint16_t* out,
                         int64_t ldo, void* ws, size_t* ws_bytes, w4_stream_t stream) {
  if (!mask) return W4_ERR_NULL;
  return attend(q, ldq, cache, table, ldt, W, kv_len, q_start, mask, ldm, B, T, max_q, Hq, window, scale, out, ldo, ws,
                ws_bytes, stream);
}

int kv_plan(const int32_t* kv_len, const int32_t* new_len, int64_t B, int32_t* table, int64_t ldt, int64_t W,
            int32_t* owned, int32_t* free_pages, int32_t* free_count, int64_t pages, int64_t page_size,
            const int32_t* depth, int64_t T, int32_t* q_start, int32_t* kv_total, int32_t* pos, int64_t* slot,
            int32_t* status, w4_stream_t stream) {
  try {
    if (!kv_len || !new_len || !table || !owned || !free_pages || !free_count || !q_start || !kv_total || !pos || !slot ||
        !status)
      return W4_ERR_NULL;
    if (B < 1 || B > ((int64_t)1 << 20) || T < 1 || T >= kMaxTokens) return W4_ERR_SHAPE;
    if (page_size < 1 || page_size > kMaxDim || W < 1 || W > kMaxDim / page_size || ldt < W || ldt > kMaxDim)
      return W4_ERR_SHAPE;
    if (pages < 1 || pages > (((int64_t)1 << 31) - 1) / page_size || B * W >= (int64_t)1 << 31) return W4_ERR_SHAPE;
    for (const void* p : {(const void*)kv_len, (const void*)new_len, (const void*)table, (const void*)owned,
                          (const void*)free_pages, (const void*)free_count, (const void*)depth, (const void*)q_start,
                          (const void*)kv_total, (const void*)pos, (const void*)status})
      if (!al4(p)) return W4_ERR_ALIGN;
    if (((uintptr_t)slot & 7u) != 0) return W4_ERR_ALIGN;
    if (int e = check_device()) return e;
    w4::PlanArgs a;
    a.kv_len = kv_len, a.new_len = new_len, a.depth = depth;
    a.table = table, a.owned = owned, a.free = free_pages, a.free_count = free_count, a.ldt = ldt;
    a.q_start = q_start, a.kv_total = kv_total, a.pos = pos, a.status = status, a.slot = slot;
    a.B = (int)B, a.W = (int)W, a.pages = (int)pages, a.page_size = (int)page_size, a.T = (int)T;
    (void)hipGetLastError();
    w4::launch_plan(a, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

int logits_adjust(const float* logits, int64_t ldl, int64_t M, int64_t V, const w4_logit_rules* rules, float* out,
                  int64_t ldo, w4_stream_t stream) {
  try {
    if (!logits || !rules || !out) return W4_ERR_NULL;
    const w4_logit_rules& h = *rules;
    const int64_t most = ((int64_t)1 << 31) - 1;
    if ((h.tokens && !h.token_len) || (h.bias && (!h.bias_id || !h.bias_start))) return W4_ERR_NULL;
    if (M < 1 || V < 1 || M > kMaxDim || V > most || ldl < V || ldo < V || ldl > ((int64_t)1 << 40) || ldo > ((int64_t)1 << 40))
      return W4_ERR_SHAPE;
    if (out == logits && ldo != ldl) return W4_ERR_OVERLAP;
    if (h.requests < 1 || h.requests > most || (!h.request && M > h.requests)) return W4_ERR_SHAPE;
    if (h.tokens && (h.max_tokens < 0 || h.max_tokens >= kMaxDim || h.ld_tokens < h.max_tokens || h.ld_tokens > ((int64_t)1 << 40)))
      return W4_ERR_SHAPE;
    if (h.bias && (h.biases < 0 || h.biases >= most)) return W4_ERR_SHAPE;
    if (h.mask && (h.masks < 1 || h.masks > most || h.ld_mask < (V + 31) / 32 || h.ld_mask > ((int64_t)1 << 40) ||
                   (!h.mask_row && M > h.masks)))
      return W4_ERR_SHAPE;
    for (const void* p : {(const void*)logits, (const void*)out, (const void*)h.request, (const void*)h.tokens,
                          (const void*)h.token_len, (const void*)h.prompt_len, (const void*)h.repetition,
                          (const void*)h.frequency, (const void*)h.presence, (const void*)h.bias, (const void*)h.bias_id,
                          (const void*)h.bias_start, (const void*)h.mask, (const void*)h.mask_row})
      if (!al4(p)) return W4_ERR_ALIGN;
    w4::LogitArgs a;
    a.logits = logits, a.out = out, a.ldl = ldl, a.ldo = ldo, a.M = (int)M, a.V = (int)V;
    a.request = h.request, a.requests = (int)h.requests;
    a.tokens = h.tokens, a.ld_tokens = h.ld_tokens, a.max_tokens = h.tokens ? (int)h.max_tokens : 0;
    a.token_len = h.token_len, a.prompt_len = h.prompt_len;
    a.repetition = h.repetition, a.frequency = h.frequency, a.presence = h.presence;
    a.bias = h.bias, a.bias_id = h.bias_id, a.bias_start = h.bias_start, a.biases = h.bias ? (int)h.biases : 0;
    a.mask = h.mask, a.ld_mask = h.ld_mask, a.masks = h.mask ? (int)h.masks : 0, a.mask_row = h.mask_row;
    if (w4::logits_workgroups(a) >= ((int64_t)1 << 23)) return W4_ERR_SHAPE;  // 2^32 threads
    if (int e = check_device()) return e;
    (void)hipGetLastError();
    w4::launch_logits(a, (hipStream_t)stream);
    return launched();
  } catch (...) {
    return W4_ERR_INTERNAL;
  }
}

}  // extern "C"
