"""Group-wise affine int4 weight-only linear layer for MI355X (gfx950).

Thin Python binding over the C ABI in include/w4.h (libw4.so).  Every function here only
checks and marshals torch tensors (dtype, device, strides) and calls the library on the
current HIP stream; all computation happens in the HIP kernels.  There is no CPU fallback.

Weight format: packed codes ``qw`` int32 [N][K/8] (uint32 bit patterns, eight 4-bit codes
per word, low nibble first), ``scales`` and ``biases`` float16 [N][K/64]; the weight is
w[n][k] = scales[n][k//64] * q[n][k] + biases[n][k//64].
"""

from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._lib import KvCache, lib, LIB_PATH  # noqa: F401

__all__ = [
    "W4Error", "w4_pack", "w4_quantize", "w4_gemv", "w4_gemv_sym128", "w4_dequant_f16_t_sym128", "w4_dequant_f16_t", "gemm_f16", "gemm_f16_dequant_next", "gemm_f16_dequant_next_sym128", "logits_argmax_topk",
    "logits_argmax_topk_noalloc", "w4_gemv_topk", "gemv_topk_workspace_bytes",
    "topk_workspace_bytes", "gemm_workspace_bytes", "status_string",
    "rope_frequencies", "rope_f16", "kv_append_rope", "attention_paged", "attention_workspace_bytes",
]

W4_OK, W4_ERR_WORKSPACE = 0, -4


class W4Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


def status_string(status: int) -> str:
    return lib().w4_strerror(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != W4_OK:
        raise W4Error(fn, status)


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


_raw_stream = torch._C._cuda_getCurrentRawStream  # of a device, as an address


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.device.index != torch.cuda.current_device():
        # the library launches on the current device; a pointer of another one would fault
        raise ValueError(f"{name} is on {t.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _rowmajor(t: torch.Tensor, name: str) -> int:
    """Leading dimension of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with contiguous rows (stride(1) == 1)")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _contig(t: torch.Tensor, name: str) -> None:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def w4_pack(q: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """uint8 codes [N][K] -> packed int32 words [N][K/8] (eight codes per word)."""
    _dev(q, "q", torch.uint8)
    _contig(q, "q")
    n, k = q.shape
    if out is None:
        out = torch.empty((n, k // 8), dtype=torch.int32, device=q.device)
    _dev(out, "out", torch.int32)
    _contig(out, "out")
    if tuple(out.shape) != (n, k // 8):
        raise ValueError("out must be [N][K/8]")
    _check("w4_pack", lib().w4_pack(q.data_ptr(), out.data_ptr(), n, k, _stream()))
    return out


def w4_quantize(w: torch.Tensor, out: tuple | None = None):
    """float16 weights [N][K] (rows contiguous) -> (qw int32 [N][K/8], scales float16 [N][K/64],
    biases float16 [N][K/64]): the min/max affine fit per group of 64 (see include/w4.h)."""
    _dev(w, "w", torch.float16)
    if w.dim() != 2:
        raise ValueError("w must be [N][K]")
    ldw = _rowmajor(w, "w")
    n, k = w.shape
    if out is None:
        out = (torch.empty((n, k // 8), dtype=torch.int32, device=w.device),
               torch.empty((n, k // 64), dtype=torch.float16, device=w.device),
               torch.empty((n, k // 64), dtype=torch.float16, device=w.device))
    qw, s, b = out
    _dev(qw, "qw", torch.int32)
    _dev(s, "scales", torch.float16)
    _dev(b, "biases", torch.float16)
    for t, nm in ((qw, "qw"), (s, "scales"), (b, "biases")):
        _contig(t, nm)
    if tuple(qw.shape) != (n, k // 8) or tuple(s.shape) != (n, k // 64) or tuple(b.shape) != (n, k // 64):
        raise ValueError("outputs must be [N][K/8], [N][K/64], [N][K/64]")
    _check("w4_quantize", lib().w4_quantize(w.data_ptr(), ldw, qw.data_ptr(), s.data_ptr(), b.data_ptr(),
                                            n, k, _stream()))
    return qw, s, b


def _w4_args(qw, scales, biases):
    _dev(qw, "qw", torch.int32)
    _dev(scales, "scales", torch.float16)
    _dev(biases, "biases", torch.float16)
    for t, nm in ((qw, "qw"), (scales, "scales"), (biases, "biases")):
        _contig(t, nm)
    n, kw = qw.shape
    k = kw * 8
    if tuple(scales.shape) != (n, k // 64) or tuple(biases.shape) != (n, k // 64):
        raise ValueError("scales and biases must be [N][K/64]")
    return n, k


def w4_gemv(qw: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, x: torch.Tensor,
            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m][n] = sum_k w[n][k] x[m][k] for x float16 [M][K] (M <= 16) -> float32 [M][N].

    Shapes that split K across workgroups need a workspace (see gemv_workspace_bytes); one is
    allocated when none (or too small a one) is given.
    """
    n, k = _w4_args(qw, scales, biases)
    _dev(x, "x", torch.float16)
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError("x must be [M][K]")
    ldx = _rowmajor(x, "x")
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _dev(out, "out", torch.float32)
    if tuple(out.shape) != (m, n):
        raise ValueError("out must be [M][N]")
    ldy = _rowmajor(out, "out")
    need = gemv_workspace_bytes(m, n, k)
    ws_ptr, cap = None, None
    if need:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        ws_ptr = workspace.data_ptr()
        cap = ctypes.byref(ctypes.c_size_t(workspace.numel() * workspace.element_size()))
    _check("w4_gemv", lib().w4_gemv(qw.data_ptr(), scales.data_ptr(), biases.data_ptr(),
                                    x.data_ptr(), ldx, out.data_ptr(), ldy, m, n, k, ws_ptr, cap,
                                    _stream()))
    return out


@functools.lru_cache(maxsize=256)
def gemv_workspace_bytes(m: int, n: int, k: int) -> int:
    """Workspace bytes w4_gemv needs for M rows of x and an [N][K] int4 matrix (0 for most shapes)."""
    need = ctypes.c_size_t(0)
    p = ctypes.c_void_p(16)
    _check("w4_gemv", lib().w4_gemv(p, p, p, p, k, p, n, m, n, k, None, ctypes.byref(need), None))
    return int(need.value)


def w4_dequant_f16_t(qw: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """Transposed f16 scratch: float16 [K][N], out[k][n] = RN16(s*q + b)."""
    n, k = _w4_args(qw, scales, biases)
    if out is None:
        out = torch.empty((k, n), dtype=torch.float16, device=qw.device)
    _dev(out, "out", torch.float16)
    if tuple(out.shape) != (k, n):
        raise ValueError("out must be [K][N]")
    ldwt = _rowmajor(out, "out")
    _check("w4_dequant_f16_t", lib().w4_dequant_f16_t(qw.data_ptr(), scales.data_ptr(),
                                                      biases.data_ptr(), out.data_ptr(), ldwt, n,
                                                      k, _stream()))
    return out


def _sym_args(qw, scales):
    _dev(qw, "qw", torch.int32)
    _dev(scales, "scales", torch.float16)
    _contig(qw, "qw")
    _contig(scales, "scales")
    n, kw = qw.shape
    k = kw * 8
    if k % 128 != 0 or tuple(scales.shape) != (n, k // 128):
        raise ValueError("the symmetric group-128 format needs K % 128 == 0 and scales [N][K/128]")
    return n, k


def w4_gemv_sym128(qw: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Symmetric group-128 GEMV: y[m][n] = sum_k scales[n][k//128] (q[n][k] - 8) x[m][k].

    Takes w4_gemv's workspace (gemv_workspace_bytes; allocated when none or too small a one
    is given)."""
    n, k = _sym_args(qw, scales)
    _dev(x, "x", torch.float16)
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError("x must be [M][K]")
    ldx = _rowmajor(x, "x")
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _dev(out, "out", torch.float32)
    if tuple(out.shape) != (m, n):
        raise ValueError("out must be [M][N]")
    ldy = _rowmajor(out, "out")
    need = gemv_workspace_bytes(m, n, k)
    ws_ptr, cap = None, None
    if need:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        ws_ptr = workspace.data_ptr()
        cap = ctypes.byref(ctypes.c_size_t(workspace.numel() * workspace.element_size()))
    _check("w4_gemv_sym128", lib().w4_gemv_sym128(qw.data_ptr(), scales.data_ptr(), x.data_ptr(), ldx,
                                                  out.data_ptr(), ldy, m, n, k, ws_ptr, cap, _stream()))
    return out


def w4_dequant_f16_t_sym128(qw: torch.Tensor, scales: torch.Tensor,
                            out: torch.Tensor | None = None) -> torch.Tensor:
    """Transposed f16 scratch of the symmetric group-128 format: out[k][n] = RN16(s (q - 8))."""
    n, k = _sym_args(qw, scales)
    if out is None:
        out = torch.empty((k, n), dtype=torch.float16, device=qw.device)
    _dev(out, "out", torch.float16)
    if tuple(out.shape) != (k, n):
        raise ValueError("out must be [K][N]")
    ldwt = _rowmajor(out, "out")
    _check("w4_dequant_f16_t_sym128", lib().w4_dequant_f16_t_sym128(qw.data_ptr(), scales.data_ptr(),
                                                                    out.data_ptr(), ldwt, n, k, _stream()))
    return out


def gemm_f16(a: torch.Tensor, b: torch.Tensor, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C = A @ B: float16 A [M][K], float16 B [K][N] (rows contiguous) -> float32 [M][N].

    Shapes that split K need a workspace (see gemm_workspace_bytes); one is allocated when
    none (or too small a one) is given.
    """
    _dev(a, "a", torch.float16)
    _dev(b, "b", torch.float16)
    lda, ldb = _rowmajor(a, "a"), _rowmajor(b, "b")
    m, k = a.shape
    k2, n = b.shape
    if k != k2:
        raise ValueError("inner dimensions differ")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=a.device)
    _dev(out, "out", torch.float32)
    if tuple(out.shape) != (m, n):
        raise ValueError("out must be [M][N]")
    ldc = _rowmajor(out, "out")
    need = ctypes.c_size_t(0)
    _check("gemm_f16", lib().gemm_f16(a.data_ptr(), lda, b.data_ptr(), ldb, out.data_ptr(), ldc,
                                      m, n, k, None, ctypes.byref(need), None))
    ws_ptr, cap = None, None
    if need.value:
        if workspace is None or workspace.numel() * workspace.element_size() < need.value:
            workspace = torch.empty(need.value, dtype=torch.uint8, device=a.device)
        ws_ptr = workspace.data_ptr()
        cap = ctypes.byref(ctypes.c_size_t(workspace.numel() * workspace.element_size()))
    _check("gemm_f16", lib().gemm_f16(a.data_ptr(), lda, b.data_ptr(), ldb, out.data_ptr(), ldc,
                                      m, n, k, ws_ptr, cap, _stream()))
    return out


def gemm_f16_dequant_next(a: torch.Tensor, b: torch.Tensor, qw: torch.Tensor, scales: torch.Tensor,
                          biases: torch.Tensor, out: torch.Tensor | None = None,
                          wt: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """gemm_f16(a, b) and w4_dequant_f16_t(qw, scales, biases) in one call (the dequant rides
    in the CUs the GEMM's last round leaves idle when it fits there): returns (C, wt)."""
    nq, kq = _w4_args(qw, scales, biases)
    return _gemm_dequant_next("gemm_f16_dequant_next", a, b, qw, scales, biases, nq, kq, out, wt, workspace)


def gemm_f16_dequant_next_sym128(a: torch.Tensor, b: torch.Tensor, qw: torch.Tensor, scales: torch.Tensor,
                                 out: torch.Tensor | None = None, wt: torch.Tensor | None = None,
                                 workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """gemm_f16(a, b) and w4_dequant_f16_t_sym128(qw, scales) in one call: returns (C, wt)."""
    nq, kq = _sym_args(qw, scales)
    return _gemm_dequant_next("gemm_f16_dequant_next_sym128", a, b, qw, scales, None, nq, kq, out, wt, workspace)


def _gemm_dequant_next(fn, a, b, qw, scales, biases, nq, kq, out, wt, workspace):
    _dev(a, "a", torch.float16)
    _dev(b, "b", torch.float16)
    lda, ldb = _rowmajor(a, "a"), _rowmajor(b, "b")
    m, k = a.shape
    k2, n = b.shape
    if k != k2:
        raise ValueError("inner dimensions differ")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=a.device)
    _dev(out, "out", torch.float32)
    if tuple(out.shape) != (m, n):
        raise ValueError("out must be [M][N]")
    if wt is None:
        wt = torch.empty((kq, nq), dtype=torch.float16, device=qw.device)
    _dev(wt, "wt", torch.float16)
    if tuple(wt.shape) != (kq, nq):
        raise ValueError("wt must be [Kq][Nq]")
    ldc, ldwt = _rowmajor(out, "out"), _rowmajor(wt, "wt")
    w4q = [qw.data_ptr(), scales.data_ptr()] + ([biases.data_ptr()] if biases is not None else [])

    def call(ws_ptr, cap, stream):
        return getattr(lib(), fn)(a.data_ptr(), lda, b.data_ptr(), ldb, out.data_ptr(), ldc, m, n, k, ws_ptr, cap,
                                  *w4q, wt.data_ptr(), ldwt, nq, kq, stream)

    need = ctypes.c_size_t(0)
    _check(fn, call(None, ctypes.byref(need), None))
    ws_ptr, cap = None, None
    if need.value:
        if workspace is None or workspace.numel() * workspace.element_size() < need.value:
            workspace = torch.empty(need.value, dtype=torch.uint8, device=a.device)
        ws_ptr = workspace.data_ptr()
        cap = ctypes.byref(ctypes.c_size_t(workspace.numel() * workspace.element_size()))
    _check(fn, call(ws_ptr, cap, _stream()))
    return out, wt


def gemm_workspace_bytes(a: torch.Tensor, b: torch.Tensor) -> int:
    """Workspace bytes gemm_f16 needs for these operands (0 for most shapes)."""
    need = ctypes.c_size_t(0)
    _check("gemm_f16", lib().gemm_f16(a.data_ptr(), _rowmajor(a, "a"), b.data_ptr(), _rowmajor(b, "b"),
                                      ctypes.c_void_p(16), b.shape[1], a.shape[0], b.shape[1], a.shape[1],
                                      None, ctypes.byref(need), None))
    return int(need.value)


def topk_workspace_bytes(m: int, v: int, k: int) -> int:
    n = ctypes.c_size_t(0)
    _check("logits_argmax_topk", lib().logits_argmax_topk(
        ctypes.c_void_p(16), v, m, v, k, ctypes.c_void_p(16), ctypes.c_void_p(16), None,
        ctypes.byref(n), None))
    return int(n.value)


def logits_argmax_topk(logits: torch.Tensor, k: int, idx: torch.Tensor | None = None,
                       val: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Per row the k largest logits (value desc, ties to lower index): (int32 idx, float32 val)."""
    _dev(logits, "logits", torch.float32)
    ldl = _rowmajor(logits, "logits")
    m, v = logits.shape
    if idx is None:
        idx = torch.empty((m, k), dtype=torch.int32, device=logits.device)
    if val is None:
        val = torch.empty((m, k), dtype=torch.float32, device=logits.device)
    _dev(idx, "idx", torch.int32)
    _dev(val, "val", torch.float32)
    _contig(idx, "idx")
    _contig(val, "val")
    if tuple(idx.shape) != (m, k) or tuple(val.shape) != (m, k):
        raise ValueError("idx and val must be [M][k]")
    need = ctypes.c_size_t(0)
    _check("logits_argmax_topk", lib().logits_argmax_topk(
        logits.data_ptr(), ldl, m, v, k, idx.data_ptr(), val.data_ptr(), None,
        ctypes.byref(need), None))
    if need.value and (workspace is None or workspace.numel() * workspace.element_size() < need.value):
        workspace = torch.empty(need.value, dtype=torch.uint8, device=logits.device)
    ws_ptr = workspace.data_ptr() if need.value else None
    cap = ctypes.c_size_t(workspace.numel() * workspace.element_size() if need.value else 0)
    _check("logits_argmax_topk", lib().logits_argmax_topk(
        logits.data_ptr(), ldl, m, v, k, idx.data_ptr(), val.data_ptr(), ws_ptr,
        ctypes.byref(cap) if need.value else None, _stream()))
    return idx, val


def logits_argmax_topk_noalloc(logits: torch.Tensor, k: int, idx: torch.Tensor | None = None,
                               val: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """logits_argmax_topk without a workspace: the library's own per-device scratch array holds
    the candidates (so the call allocates nothing when idx and val are given).  Calls that
    overlap on one device share that array."""
    _dev(logits, "logits", torch.float32)
    ldl = _rowmajor(logits, "logits")
    m, v = logits.shape
    if idx is None:
        idx = torch.empty((m, k), dtype=torch.int32, device=logits.device)
    if val is None:
        val = torch.empty((m, k), dtype=torch.float32, device=logits.device)
    _dev(idx, "idx", torch.int32)
    _dev(val, "val", torch.float32)
    _contig(idx, "idx")
    _contig(val, "val")
    if tuple(idx.shape) != (m, k) or tuple(val.shape) != (m, k):
        raise ValueError("idx and val must be [M][k]")
    _check("logits_argmax_topk_noalloc", lib().logits_argmax_topk_noalloc(
        logits.data_ptr(), ldl, m, v, k, idx.data_ptr(), val.data_ptr(), _stream()))
    return idx, val


def gemv_topk_workspace_bytes(v: int, k_dim: int, k: int) -> int:
    """Workspace bytes w4_gemv_topk needs for a [v][k_dim] head and top-k."""
    n = ctypes.c_size_t(0)
    p = ctypes.c_void_p(16)
    _check("w4_gemv_topk", lib().w4_gemv_topk(p, p, p, p, v, k_dim, k, p, p, p, None, ctypes.byref(n), None))
    return int(n.value)


def w4_gemv_topk(qw: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, x: torch.Tensor, k: int,
                 logits: torch.Tensor | None = None, idx: torch.Tensor | None = None,
                 val: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """The int4 LM head with top-k on the device, one call: x float16 [K] (or [1][K]) -> (logits float32 [V],
    idx int32 [k], val float32 [k]), the k largest logits, value descending, ties to the lower
    index.  One is allocated for each of the outputs and the workspace not given."""
    v, kdim = _w4_args(qw, scales, biases)
    _dev(x, "x", torch.float16)
    _contig(x, "x")
    if x.numel() != kdim or (x.dim() == 2 and x.shape[0] != 1):
        raise ValueError("x must be [K] or [1][K]")
    outs = []
    for t, name, shape, dt in ((logits, "logits", (v,), torch.float32), (idx, "idx", (k,), torch.int32),
                               (val, "val", (k,), torch.float32)):
        if t is None:
            t = torch.empty(shape, dtype=dt, device=x.device)
        _dev(t, name, dt)
        _contig(t, name)
        if t.numel() != shape[0]:
            raise ValueError(f"{name} must hold {shape[0]} elements")
        outs.append(t)
    logits, idx, val = outs
    need = gemv_topk_workspace_bytes(v, kdim, k)
    ws_ptr, cap = None, None  # no workspace at all when none is needed (a null one would be a query)
    if need:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        ws_ptr = workspace.data_ptr()
        cap = ctypes.byref(ctypes.c_size_t(workspace.numel() * workspace.element_size()))
    _check("w4_gemv_topk", lib().w4_gemv_topk(qw.data_ptr(), scales.data_ptr(), biases.data_ptr(), x.data_ptr(),
                                              v, kdim, k, logits.data_ptr(), idx.data_ptr(), val.data_ptr(),
                                              ws_ptr, cap, _stream()))
    return logits, idx, val


# ------------------------------------------------- rotary positions, paged cache, attention

_F16, _F32, _E4M3 = 0, 1, 2


def rope_frequencies(rot: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                     original: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device: str | torch.device = "cuda") -> tuple[torch.Tensor, float]:
    """(freq float32 [rot/2], mscale) for rope_f16 and kv_append_rope: freq[i] = base^(-2i / rot),
    for contexts `factor` times as long as the model was trained on changed by `scaling`:
    "linear" divides every frequency by factor; "ntk" raises the base to
    base * factor^(rot / (rot - 2)), which divides the lowest frequency by factor and leaves the
    highest; "yarn" divides the frequencies that turn less than beta_slow times in `original` positions,
    leaves those that turn more than beta_fast times, blends between in the pair's index, and
    has mscale 0.1 ln(factor) + 1."""
    if rot < 0 or rot % 2 or base <= 1.0 or factor < 1.0:
        raise ValueError("rot must be even and not negative, base > 1, factor >= 1")
    i = torch.arange(rot // 2, dtype=torch.float64)
    mscale = 1.0
    if scaling == "ntk":
        if rot < 4:
            raise ValueError("ntk needs rot >= 4")
        base = base * factor ** (rot / (rot - 2))
    freq = base ** (-2.0 * i / max(rot, 1))
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if original < 1 or not beta_fast > beta_slow > 0:
            raise ValueError("yarn needs original >= 1 and beta_fast > beta_slow > 0")

        def index(turns):  # the (real) index of the pair that turns so often in `original` positions
            return rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))

        lo = max(math.floor(index(beta_fast)), 0)
        hi = min(math.ceil(index(beta_slow)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        freq = freq * (1.0 - ramp) + freq / factor * ramp
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.float().to(device), mscale


# These calls run once or twice per layer and token, so their checks are kept short: _need() looks at a
# tensor once and leaves the wording of a refusal to _dev().


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, dev: int) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev:
        _dev(t, name, dtype)


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, dev: int) -> int:
    """Elements between the tokens of a [tokens][heads][dim] tensor with contiguous heads."""
    _need(t, name, dtype, dev)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens][heads][dim]")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d > 1) or (s1 != d and h > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return s0 if n > 1 else h * d


def _row_dtype(t: torch.Tensor, name: str) -> torch.dtype:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.float32, torch.float16):
        raise TypeError(f"{name} must be torch.float16 or torch.float32, got {t.dtype}")
    return t.dtype


def _vec(t: torch.Tensor, name: str, dtype: torch.dtype, n: int, dev: int) -> int:
    _need(t, name, dtype, dev)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and hold {n} elements")
    return t.data_ptr()


def _freq(t: torch.Tensor, dev: int) -> tuple[int | None, int]:
    """(address, dims that it rotates) of a vector of frequencies"""
    _need(t, "freq", torch.float32, dev)
    if not t.is_contiguous():
        raise ValueError("freq must be contiguous")
    n = t.numel()
    return (t.data_ptr() if n else None), 2 * n


def _kv_cache(k_cache, v_cache, k_scale, v_scale, dev: int) -> KvCache:
    if not isinstance(k_cache, torch.Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    dtype = k_cache.dtype
    if dtype is torch.float16:
        kind = _F16
        if k_scale is not None or v_scale is not None:
            raise ValueError("a float16 cache takes no scales")
    elif dtype is torch.float8_e4m3fn:
        kind = _E4M3
    else:
        raise TypeError(f"the caches must be torch.float16 or torch.float8_e4m3fn, got {dtype}")
    _need(k_cache, "k_cache", dtype, dev)
    _need(v_cache, "v_cache", dtype, dev)
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must both be [pages][kv heads][page size][dim]")
    st, stv = k_cache.stride(), v_cache.stride()
    if (st[3] != 1 and shape[3] > 1) or (st != stv and any(a != b and n > 1 for a, b, n in zip(st, stv, shape))):
        raise ValueError("k_cache and v_cache must have the same strides and a contiguous dim")
    pages, heads, size, dim = shape
    ks = None if k_scale is None else _vec(k_scale, "k_scale", torch.float32, heads, dev)
    vs = None if v_scale is None else _vec(v_scale, "v_scale", torch.float32, heads, dev)
    return KvCache(k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, pages, size, heads, dim,
                   st[0] if pages > 1 else 0, st[1] if heads > 1 else 0, st[2] if size > 1 else 0, kind)


def rope_f16(x: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, *, interleaved: bool = False,
             mscale: float = 1.0, inverse: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotary positions: x float16 or float32 [T][H][D] (heads contiguous), positions int32 [T],
    freq float32 [R/2] (see rope_frequencies) -> float16 [T][H][D] with the first R dims of every
    head rotated by positions * freq, times mscale.  Pairs are (i, i + R/2), or (2i, 2i + 1) if
    interleaved.  inverse rotates back: the gradient of the rotation.  out may be x (float16)."""
    dev = torch.cuda.current_device()
    dtype = _row_dtype(x, "x")
    ldx = _rows(x, "x", dtype, dev)
    t, h, d = x.shape
    if out is None:
        out = torch.empty((t, h, d), dtype=torch.float16, device=x.device)
        ldy = h * d
    else:
        ldy = _rows(out, "out", torch.float16, dev)
        if out.shape != x.shape:
            raise ValueError("out must have x's shape")
    f, rot = _freq(freq, dev)
    _check("rope_f16", lib().rope_f16(x.data_ptr(), _F32 if dtype is torch.float32 else _F16, ldx,
                                      _vec(positions, "positions", torch.int32, t, dev), f, out.data_ptr(), ldy, t, h,
                                      d, rot, interleaved, inverse, mscale, _raw_stream(dev)))
    return out


def kv_append_rope(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   slots: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, *,
                   q: torch.Tensor | None = None, q_out: torch.Tensor | None = None, interleaved: bool = False,
                   mscale: float = 1.0, k_scale: torch.Tensor | None = None,
                   v_scale: torch.Tensor | None = None) -> torch.Tensor | None:
    """New tokens into a paged cache with the rotation on the way (see rope_f16), one launch.

    k, v [T][kv heads][dim] and q [T][heads][dim], all float16 or all float32 (views of the rows
    of one q|k|v product will do); caches [pages][kv heads][page size][dim], any strides with a
    contiguous dim, float16 or float8_e4m3fn (value = code * scale[head], scales float32 [kv heads]);
    slots int64 [T] = page * page size + token of the page, distinct, -1: not written.
    Returns the rotated queries, float16 (None without q)."""
    dev = torch.cuda.current_device()
    c = _kv_cache(k_cache, v_cache, k_scale, v_scale, dev)
    dtype = _row_dtype(k, "k")
    ldk, ldv = _rows(k, "k", dtype, dev), _rows(v, "v", dtype, dev)
    t, heads, d = k.shape
    if v.shape != k.shape or heads != c.heads or d != c.dim:
        raise ValueError("k and v must be [T][kv heads][dim] of the cache")
    ldq = ldqo = hq = 0
    pq = pqo = None
    if q is not None:
        ldq = _rows(q, "q", dtype, dev)
        n, hq, dq = q.shape
        if n != t or dq != d:
            raise ValueError("q must be [T][heads][dim] with k's T and dim")
        if q_out is None:
            q_out = torch.empty((t, hq, d), dtype=torch.float16, device=q.device)
            ldqo = hq * d
        else:
            ldqo = _rows(q_out, "q_out", torch.float16, dev)
            if q_out.shape != q.shape:
                raise ValueError("q_out must have q's shape")
        pq, pqo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    f, rot = _freq(freq, dev)
    _check("kv_append_rope", lib().kv_append_rope(
        pq, ldq, pqo, ldqo, hq, k.data_ptr(), ldk, v.data_ptr(), ldv, _F32 if dtype is torch.float32 else _F16, c,
        _vec(slots, "slots", torch.int64, t, dev), _vec(positions, "positions", torch.int32, t, dev), f, t, rot,
        interleaved, mscale, _raw_stream(dev)))
    return q_out


def attention_workspace_bytes(k_cache: torch.Tensor, b: int, t: int, max_q: int, heads: int, pages_per_seq: int,
                              window: int = 0) -> int:
    """Workspace bytes attention_paged needs for t query rows of b sequences over this cache, with
    tables of pages_per_seq pages."""
    c = _kv_cache(k_cache, k_cache, None, None, torch.cuda.current_device())
    need = ctypes.c_size_t(0)
    p, ld = 16, heads * c.dim
    _check("attention_paged", lib().attention_paged(p, ld, c, p, pages_per_seq, pages_per_seq, p, p, b, t, max_q,
                                                    heads, window, 1.0, p, ld, None, ctypes.byref(need), None))
    return int(need.value)


def attention_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor,
                    kv_len: torch.Tensor, *, q_start: torch.Tensor | None = None, max_q: int | None = None,
                    scale: float | None = None, window: int = 0, k_scale: torch.Tensor | None = None,
                    v_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the new tokens of B sequences over a paged cache that holds them already.

    q float16 [T][heads][dim]: sequence b has the rows q_start[b] .. q_start[b+1] - 1 (q_start
    int32 [B + 1]; None: one row each); kv_len int32 [B]: its cached tokens, the new ones included;
    table int32 [B][pages of a sequence]; caches and scales as for kv_append_rope.  Row i of n
    stands at p = kv_len - n + i and sees the keys max(0, p + 1 - window) .. p (window 0: from 0);
    scale defaults to dim ** -0.5.  max_q: the longest sequence's rows (default: T; give it, 1 for
    decode: it chooses the kernel).  Returns float16 [T][heads][dim]; a row that sees no key is 0,
    rows past the last sequence are not written.  A table much wider than the sequences are long costs time.  out may be q.  One is allocated for out and the workspace
    (attention_workspace_bytes) when not given or too small."""
    dev = torch.cuda.current_device()
    c = _kv_cache(k_cache, v_cache, k_scale, v_scale, dev)
    ldq = _rows(q, "q", torch.float16, dev)
    t, hq, d = q.shape
    if d != c.dim:
        raise ValueError("q must have the cache's dim")
    if out is None:
        out = torch.empty((t, hq, d), dtype=torch.float16, device=q.device)
        ldo = hq * d
    else:
        ldo = _rows(out, "out", torch.float16, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    _need(table, "table", torch.int32, dev)
    ldt = _rowmajor(table, "table")
    b, width = table.shape
    start = None
    if q_start is not None:
        start = _vec(q_start, "q_start", torch.int32, b + 1, dev)
        if max_q is None:
            max_q = t
    elif max_q is None:
        max_q = 1
    if scale is None:
        scale = d ** -0.5
    args = (q.data_ptr(), ldq, c, table.data_ptr(), ldt, width, _vec(kv_len, "kv_len", torch.int32, b, dev), start, b,
            t, max_q, hq, window, scale, out.data_ptr(), ldo)
    fn, stream = lib().attention_paged, _raw_stream(dev)
    status = W4_ERR_WORKSPACE
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous, on the current device")
        status = fn(*args, workspace.data_ptr(), ctypes.c_size_t(workspace.numel() * workspace.element_size()), stream)
    if status == W4_ERR_WORKSPACE:
        size = ctypes.c_size_t(0)
        _check("attention_paged", fn(*args, None, size, None))
        workspace = torch.empty(max(16, size.value), dtype=torch.uint8, device=q.device)
        status = fn(*args, workspace.data_ptr(), size, stream)
    _check("attention_paged", status)
    return out
