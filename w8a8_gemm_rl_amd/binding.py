"""Thin ctypes binding over libqurl_w8a8.so (C ABI in include/qurl_w8a8.h).

Argument marshalling only: torch tensors supply device memory and the current
HIP stream; every step of the computation runs in the library's kernels. If
the shared library is missing this module raises -- there is no fallback.

Function names mirror the C entry points without the ``qr_`` prefix.
"""

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# The in-tree build; QR_LIB_PATH names another build of the same library to
# load instead (the CPU tests use it for the host-sanitizer build).
LIB_PATH = os.environ.get("QR_LIB_PATH") or os.path.join(_HERE, "libqurl_w8a8.so")

QT = {"int8": 0, "fp8": 1}
OUT = {"bf16": 0, "raw": 1}
NORM = {"rms": 0, "layer": 1}
# Formats of a linear's input (the header's QR_ACT_*); "fp4" and "fp8" tokens of an
# MXFP4 product are the block formats.
ACT = {"int8": 0, "fp8": 1, "mxfp8": 2, "mxfp4": 3, "bf16": 4}
STATUS = {
    0: "QR_OK", -1: "QR_ERR_INVALID_ARG", -2: "QR_ERR_UNSUPPORTED", -3: "QR_ERR_WORKSPACE",
    -4: "QR_ERR_HIP", -5: "QR_ERR_NO_DEVICE",
}
# Every function include/qurl_w8a8.h declares.
EXPORTS = [
    "qr_quantize_weights_uaq", "qr_requantize_weights", "qr_quantize_act_per_token",
    "qr_norm_quant", "qr_silu_mul_quant", "qr_acr_tis_loss", "qr_mx_quantize", "qr_mx_gemm",
    "qr_w8a8_gemm", "qr_w8a8_gemm_quant", "qr_linear_fused", "qr_linear_fused_noalloc",
    "qr_workspace_size", "qr_gemm_plan", "qr_tile_name", "qr_num_tiles", "qr_set_plan_override",
    "qr_set_small_m_override", "qr_set_fuse_override", "qr_last_error", "qr_version", "qr_probe_read", "qr_probe_mfma",
    "qr_probe_copy_stream", "qr_mxfp4_quantize", "qr_mx_dequantize", "qr_mxfp4_gemm", "qr_mxfp4_linear",
    "qr_block_norm_quant", "qr_silu_mul_mx", "qr_mxfp4_plan", "qr_vocab_logp", "qr_vocab_logp_grad",
    "qr_vocab_distill", "qr_vocab_distill_grad", "qr_vocab_plan",
]


class QRError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None
_lock = threading.Lock()

_i64, _f32, _vp, _int, _sz = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_SIGS = {
    "qr_quantize_weights_uaq": (_int, [_vp, _i64, _i64, _i64, _f32, _int, _vp, _vp, _vp, _vp, _vp, _vp]),
    "qr_requantize_weights": (_int, [_vp, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp]),
    "qr_quantize_act_per_token": (_int, [_vp, _i64, _i64, _i64, _f32, _int, _vp, _vp, _vp]),
    "qr_norm_quant": (_int, [_vp, _i64, _i64, _i64, _int, _vp, _vp, _f32, _int, _vp, _vp, _vp]),
    "qr_silu_mul_quant": (_int, [_vp, _vp, _i64, _i64, _i64, _i64, _f32, _int, _vp, _vp, _vp]),
    "qr_acr_tis_loss": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _f32, _f32, _vp, _vp, _vp, _vp, _sz,
                               _vp]),
    "qr_mx_quantize": (_int, [_vp, _i64, _i64, _i64, _int, _vp, _vp, _vp]),
    "qr_mx_gemm": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _i64, _vp]),
    "qr_mxfp4_quantize": (_int, [_vp, _i64, _i64, _i64, _int, _vp, _vp, _vp]),
    "qr_mx_dequantize": (_int, [_vp, _vp, _i64, _i64, _int, _vp, _i64, _int, _vp]),
    "qr_mxfp4_gemm": (_int, [_vp, _vp, _int, _vp, _vp, _i64, _i64, _i64, _int, _vp, _i64, _vp, _sz, _vp]),
    "qr_mxfp4_linear": (_int, [_vp, _i64, _int, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _sz, _vp]),
    "qr_block_norm_quant": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _int, _vp, _vp, _vp, _i64, _f32, _vp,
                                   _vp, _f32, _int, _vp, _i64, _vp, _vp, _vp]),
    "qr_silu_mul_mx": (_int, [_vp, _vp, _i64, _i64, _i64, _i64, _int, _vp, _vp, _vp]),
    "qr_vocab_logp": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _f32, _vp, _vp, _vp, _sz, _vp]),
    "qr_vocab_logp_grad": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _f32, _vp, _vp, _vp, _i64, _vp,
                                  _i64, _vp, _sz, _vp]),
    "qr_vocab_distill": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _int, _vp, _i64, _f32, _vp,
                                _vp, _vp, _sz, _vp]),
    "qr_vocab_distill_grad": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _int, _vp, _i64, _f32,
                                     _vp, _vp, _vp, _i64, _vp, _i64, _vp, _sz, _vp]),
    "qr_w8a8_gemm": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _vp, _i64, _vp, _sz, _vp]),
    "qr_w8a8_gemm_quant": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _i64, _i64, _i64,
                                  _f32, _vp, _vp, _vp, _sz, _vp]),
    "qr_linear_fused": (_int, [_vp, _i64, _f32, _vp, _vp, _i64, _i64, _i64, _int, _vp, _i64, _vp, _sz, _vp]),
    "qr_linear_fused_noalloc": (_int, [_vp, _i64, _f32, _vp, _vp, _i64, _i64, _i64, _int, _vp, _i64,
                                       _vp]),
    "qr_workspace_size": (_sz, [ctypes.c_char_p, _i64, _i64, _i64, _int]),
    "qr_gemm_plan": (_int, [_i64, _i64, _i64, _int, ctypes.POINTER(_int), ctypes.POINTER(_int),
                            ctypes.POINTER(_int)]),
    "qr_mxfp4_plan": (_int, [_i64, _i64, _i64, _int] + 4 * [ctypes.POINTER(_int)]),
    "qr_vocab_plan": (_int, [_i64, _i64, _i64] + 3 * [ctypes.POINTER(_int)] + [ctypes.POINTER(_i64)]),
    "qr_tile_name": (ctypes.c_char_p, [_int]),
    "qr_num_tiles": (_int, []),
    "qr_set_plan_override": (_int, [_int, _int, _int]),
    "qr_set_small_m_override": (_int, [_int]),
    "qr_set_fuse_override": (_int, [_int]),
    "qr_last_error": (ctypes.c_char_p, []),
    "qr_probe_read": (_int, [_vp, _sz, _vp, _i64, _vp]),
    "qr_probe_mfma": (_int, [_int, _int, _int, _vp, _vp, ctypes.POINTER(_int), _vp]),
    "qr_probe_copy_stream": (_int, [_int, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _int, _int, _vp, _i64, _vp]),
    "qr_version": (ctypes.c_char_p, []),
}


def lib():
    """Load (once) and return the shared library; raise if it is not built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"{LIB_PATH} is not built: run `python -m w8a8_gemm_rl_amd.build`")
                L = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in _SIGS.items():
                    f = getattr(L, name)
                    f.restype = res
                    f.argtypes = args
                _lib = L
    return _lib


def _check(fn, status):
    if status != 0:
        msg = lib().qr_last_error().decode(errors="replace")
        raise QRError(fn, status, msg)


def _qt(qt):
    if qt not in QT:
        raise ValueError(f"qt must be one of {list(QT)}, got {qt!r}")
    return QT[qt]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must live on a HIP device")


def _rows(t, name):
    """Leading dimension of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    if t.shape[0] <= 1:  # the row stride of a single row is arbitrary
        return max(t.shape[1], 1)
    return t.stride(0)


def code_dtype(qt):
    return torch.int8 if qt == "int8" else torch.float8_e4m3fn


# ----------------------------------------------------------------------------
# Workspace: one scratch buffer per (device, stream), grown on demand. Calls on
# one stream are ordered, so they may share it; calls on different streams may
# run at the same time and get different buffers. A buffer that is outgrown is
# kept alive (never freed): a HIP graph captured earlier may still write into
# it on every replay, and the caching allocator must not hand its memory to
# another tensor.
# ----------------------------------------------------------------------------
_ws = {}
_ws_retired = []


def workspace(nbytes, device):
    if nbytes == 0:
        return None, 0
    dev = torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    key = (idx, torch.cuda.current_stream(idx).cuda_stream)
    buf = _ws.get(key)
    if buf is None or buf.numel() < nbytes:
        if buf is not None:
            _ws_retired.append(buf)
        buf = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=torch.device("cuda", idx))
        _ws[key] = buf
    return buf, buf.numel()


# ----------------------------------------------------------------------------
# Entry points
# ----------------------------------------------------------------------------

def version():
    return lib().qr_version().decode()


def num_tiles():
    return lib().qr_num_tiles()


def tile_name(i):
    r = lib().qr_tile_name(i)
    return None if r is None else r.decode()


def set_plan_override(tile=-1, splitk=0, rows=0):
    _check("qr_set_plan_override", lib().qr_set_plan_override(tile, splitk, rows))


def set_small_m_override(rf=0):
    """One-launch decode path of linear_fused at 1-4 tokens: 0 automatic,
    -1 off, 1..5 blocks of 16 * rf output channels (calling thread only)."""
    _check("qr_set_small_m_override", lib().qr_set_small_m_override(rf))


def set_fuse_override(mode=0):
    """w8a8_gemm_quant: 0 separate launches (default), 1 the one-launch
    grid-barrier path where the plan allows (calling thread only)."""
    _check("qr_set_fuse_override", lib().qr_set_fuse_override(mode))


def gemm_plan(M, N, K, qt):
    """(tile, splitk, rows) of the plan qr_w8a8_gemm uses for this shape."""
    t, s, r = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check("qr_gemm_plan", lib().qr_gemm_plan(M, N, K, _qt(qt), ctypes.byref(t), ctypes.byref(s),
                                              ctypes.byref(r)))
    return t.value, s.value, r.value


def workspace_size(fn, M, N, K, qt):
    """Bytes of workspace `fn` takes for a shape; qt is "int8" or "fp8", for the MXFP4 products the
    tokens' "fp4" or "fp8", for the losses over a vocabulary the list length L (1 for the logp calls)."""
    if fn in ("qr_mxfp4_gemm", "qr_mxfp4_linear"):
        qt = _tokens(qt)
    elif not fn.startswith("qr_vocab_"):
        qt = _qt(qt)
    r = lib().qr_workspace_size(fn.encode(), M, N, K, qt)
    if r == ctypes.c_size_t(-1).value:
        raise QRError("qr_workspace_size", -1, lib().qr_last_error().decode())
    return r


def quantize_weights_uaq(W, s, qt, Wq=None, scale_w=None, W_scaled=None, gamma=None, beta=None):
    """W [N, K] fp32 (rows contiguous) -> (Wq [N, K], scale_w [N]) on W's device."""
    _need_cuda(W, Wq, scale_w, W_scaled, gamma, beta)
    if W.dtype != torch.float32:
        raise ValueError("W must be float32")
    N, K = W.shape
    ldw = _rows(W, "W")
    if Wq is None:
        Wq = torch.empty((N, K), dtype=code_dtype(qt), device=W.device)
    if scale_w is None:
        scale_w = torch.empty(N, dtype=torch.float32, device=W.device)
    if W_scaled is not None and (W_scaled.shape != W.shape or _rows(W_scaled, "W_scaled") != ldw):
        raise ValueError("W_scaled must have W's shape and row stride")
    with torch.cuda.device(W.device):
        st = lib().qr_quantize_weights_uaq(_ptr(W), N, K, ldw, float(s), _qt(qt), _ptr(Wq),
                                           _ptr(scale_w), _ptr(W_scaled), _ptr(gamma), _ptr(beta),
                                           _stream(W.device))
    _check("qr_quantize_weights_uaq", st)
    return Wq, scale_w


def requantize_weights(Wp, qt, Wq, scale_w=None, row_flips=None):
    """Refresh the codes of stored parameters Wp = W / s [N, K] fp32 in place in Wq.

    With row_flips (an int32 device tensor of N entries) entry n receives the
    number of codes of row n whose value changed. Returns (Wq, scale_w).
    """
    _need_cuda(Wp, Wq, scale_w, row_flips)
    if Wp.dtype != torch.float32:
        raise ValueError("Wp must be float32")
    N, K = Wp.shape
    ldw = _rows(Wp, "Wp")
    if Wq.shape != (N, K) or Wq.dtype != code_dtype(qt) or not Wq.is_contiguous():
        raise ValueError("Wq must be a contiguous [N, K] code tensor of the quantized type")
    if scale_w is None:
        scale_w = torch.empty(N, dtype=torch.float32, device=Wp.device)
    if row_flips is not None and (row_flips.dtype != torch.int32 or row_flips.numel() != N
                                  or not row_flips.is_contiguous()):
        raise ValueError("row_flips must be a contiguous int32 tensor of N entries")
    with torch.cuda.device(Wp.device):
        st = lib().qr_requantize_weights(_ptr(Wp), N, K, ldw, _qt(qt), _ptr(Wq), _ptr(scale_w),
                                         _ptr(row_flips), _stream(Wp.device))
    _check("qr_requantize_weights", st)
    return Wq, scale_w


def norm_quant(H, gamma, qt, beta=None, eps=1e-6, kind="rms", Xq=None, scale_x=None):
    """Norm of bf16 rows H [M, K] with the folded gain gamma (= gamma*s, fp32 [K]) and
    optional folded bias beta, fused with per-token quantization -> (Xq, scale_x)."""
    _need_cuda(H, gamma, beta, Xq, scale_x)
    if H.dtype != torch.bfloat16:
        raise ValueError("H must be bfloat16")
    if kind not in NORM:
        raise ValueError(f"kind must be one of {list(NORM)}")
    M, K = H.shape
    ldh = _rows(H, "H")
    for name, t in (("gamma", gamma), ("beta", beta)):
        if t is not None and (t.dtype != torch.float32 or t.numel() != K or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 tensor of K entries")
    if Xq is None:
        Xq = torch.empty((M, K), dtype=code_dtype(qt), device=H.device)
    if scale_x is None:
        scale_x = torch.empty(M, dtype=torch.float32, device=H.device)
    with torch.cuda.device(H.device):
        st = lib().qr_norm_quant(_ptr(H), M, K, ldh, NORM[kind], _ptr(gamma), _ptr(beta),
                                 float(eps), _qt(qt), _ptr(Xq), _ptr(scale_x), _stream(H.device))
    _check("qr_norm_quant", st)
    return Xq, scale_x


def silu_mul_quant(G, U, act_mult, qt, Xq=None, scale_x=None):
    """SiLU(G) * U for bf16 [M, N] views (rows contiguous, any row strides), fused with
    per-token quantization; scale_x carries act_mult -> (Xq, scale_x)."""
    _need_cuda(G, U, Xq, scale_x)
    if G.dtype != torch.bfloat16 or U.dtype != torch.bfloat16:
        raise ValueError("G and U must be bfloat16")
    if G.shape != U.shape:
        raise ValueError("G and U must have one shape")
    M, N = G.shape
    ldg, ldu = _rows(G, "G"), _rows(U, "U")
    if Xq is None:
        Xq = torch.empty((M, N), dtype=code_dtype(qt), device=G.device)
    if scale_x is None:
        scale_x = torch.empty(M, dtype=torch.float32, device=G.device)
    with torch.cuda.device(G.device):
        st = lib().qr_silu_mul_quant(_ptr(G), _ptr(U), M, N, ldg, ldu, float(act_mult), _qt(qt),
                                     _ptr(Xq), _ptr(scale_x), _stream(G.device))
    _check("qr_silu_mul_quant", st)
    return Xq, scale_x


def acr_tis_loss(logp, logp_prox, logp_behav, adv, mask, eps, C, loss=None, grad=None,
                 with_grad=True):
    """Per-token ACR / TIS loss on fp32 [n] tensors and a uint8 mask ->
    (loss [n], grad [n] or None, sums float64 [3] = loss sum, valid, clipped)."""
    ts = (logp, logp_prox, logp_behav, adv)
    _need_cuda(*ts, mask, loss, grad)
    n = logp.numel()
    for t in ts:
        if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous():
            raise ValueError("log-probabilities and advantages must be contiguous float32 of one size")
    if mask.dtype != torch.uint8 or mask.numel() != n or not mask.is_contiguous():
        raise ValueError("mask must be a contiguous uint8 tensor of the same size")
    dev = logp.device
    if loss is None:
        loss = torch.empty(n, dtype=torch.float32, device=dev)
    if grad is None and with_grad:
        grad = torch.empty(n, dtype=torch.float32, device=dev)
    sums = torch.empty(3, dtype=torch.float64, device=dev)
    ws, ws_bytes = workspace(workspace_size("qr_acr_tis_loss", n, 0, 0, "int8"), dev)
    with torch.cuda.device(dev):
        st = lib().qr_acr_tis_loss(*(_ptr(t) for t in ts), _ptr(mask), n, float(eps), float(C),
                                   _ptr(loss), _ptr(grad), _ptr(sums), _ptr(ws), ws_bytes,
                                   _stream(dev))
    _check("qr_acr_tis_loss", st)
    return loss, grad, sums


def mx_quantize(A, codes=None, scales=None):
    """Block-wise FP8 of fp32 or bf16 rows A [R, K] -> (codes [R, K] fp8, E8M0 scales uint8
    [ceil(K/128), R, 4]: scales[p, r, j] belongs to 32-element block 4 p + j of row r)."""
    _need_cuda(A, codes, scales)
    if A.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("A must be float32 or bfloat16")
    R, K = A.shape
    lda = _rows(A, "A")
    if codes is None:
        codes = torch.empty((R, K), dtype=torch.float8_e4m3fn, device=A.device)
    if scales is None:
        scales = torch.empty(((K + 127) // 128, R, 4), dtype=torch.uint8, device=A.device)
    with torch.cuda.device(A.device):
        st = lib().qr_mx_quantize(_ptr(A), R, K, lda, int(A.dtype == torch.bfloat16), _ptr(codes),
                                  _ptr(scales), _stream(A.device))
    _check("qr_mx_quantize", st)
    return codes, scales


def mx_gemm(Xq, sx, Wq, sw, out="bf16", Y=None):
    """Block-wise FP8 product: Y [M, N] = bf16(acc) or the fp32 accumulators."""
    _need_cuda(Xq, sx, Wq, sw, Y)
    M, K = Xq.shape
    N = Wq.shape[0]
    P = (K + 127) // 128
    if Wq.shape[1] != K or sx.shape != (P, M, 4) or sw.shape != (P, N, 4):
        raise ValueError("operand shapes do not match")
    for t in (Xq, sx, Wq, sw):
        if not t.is_contiguous():
            raise ValueError("operands must be contiguous")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16 if out == "bf16" else torch.float32,
                        device=Xq.device)
    ldy = _rows(Y, "Y")
    with torch.cuda.device(Xq.device):
        st = lib().qr_mx_gemm(_ptr(Xq), _ptr(sx), _ptr(Wq), _ptr(sw), M, N, K, OUT[out], _ptr(Y),
                              ldy, _stream(Xq.device))
    _check("qr_mx_gemm", st)
    return Y


def quantize_act_per_token(X, act_mult, qt, Xq=None, scale_x=None):
    """X [M, K] bf16 (rows contiguous, any row stride) -> (Xq [M, K], scale_x [M])."""
    _need_cuda(X, Xq, scale_x)
    if X.dtype != torch.bfloat16:
        raise ValueError("X must be bfloat16")
    M, K = X.shape
    ldx = _rows(X, "X")
    if Xq is None:
        Xq = torch.empty((M, K), dtype=code_dtype(qt), device=X.device)
    if scale_x is None:
        scale_x = torch.empty(M, dtype=torch.float32, device=X.device)
    with torch.cuda.device(X.device):
        st = lib().qr_quantize_act_per_token(_ptr(X), M, K, ldx, float(act_mult), _qt(qt), _ptr(Xq),
                                             _ptr(scale_x), _stream(X.device))
    _check("qr_quantize_act_per_token", st)
    return Xq, scale_x


def w8a8_gemm(Xq, scale_x, Wq, scale_w, qt, out="bf16", Y=None, ws=None):
    """Y = dequant(Xq @ Wq^T): bf16 [M, N], or raw int32 / fp32 accumulators."""
    _need_cuda(Xq, scale_x, Wq, scale_w, Y)
    M, K = Xq.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K:
        raise ValueError("Xq and Wq disagree on K")
    if Y is None:
        dt = torch.bfloat16 if out == "bf16" else (torch.int32 if qt == "int8" else torch.float32)
        Y = torch.empty((M, N), dtype=dt, device=Xq.device)
    ldy = _rows(Y, "Y")
    need = workspace_size("qr_w8a8_gemm", M, N, K, qt)
    if ws is None:
        ws, wsb = workspace(need, Xq.device)
    else:
        wsb = ws.numel() * ws.element_size()
    with torch.cuda.device(Xq.device):
        st = lib().qr_w8a8_gemm(_ptr(Xq), _ptr(scale_x), _ptr(Wq), _ptr(scale_w), M, N, K, _qt(qt),
                                OUT[out], _ptr(Y), ldy, _ptr(ws), wsb, _stream(Xq.device))
    _check("qr_w8a8_gemm", st)
    return Y


_wsq = {}


def quant_workspace(nbytes, device):
    """The binding's workspace for qr_w8a8_gemm_quant: one zeroed buffer per
    (device, stream), separate from the other calls' (its header must stay
    as the fused launches leave it); outgrown buffers are kept alive."""
    if nbytes == 0:
        return None, 0
    dev = torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    key = (idx, torch.cuda.current_stream(idx).cuda_stream)
    buf = _wsq.get(key)
    if buf is None or buf.numel() < nbytes:
        if buf is not None:
            _ws_retired.append(buf)
        buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=torch.device("cuda", idx))
        _wsq[key] = buf
    return buf, buf.numel()


def w8a8_gemm_quant(Xq, scale_x, Wq, scale_w, qt, Y=None, q_cols=None, q_act_mult=1.0,
                    Xq_next=None, scale_x_next=None, ws=None):
    """Y = dequant(Xq @ Wq^T) in bf16, and (q_cols = (c0, c1)) the per-token
    quantization of Y[:, c0:c1] with q_act_mult -> (Y, Xq_next, scale_x_next).
    `ws`, if given, must be a workspace zeroed once when allocated and used
    only by this call."""
    _need_cuda(Xq, scale_x, Wq, scale_w, Y, Xq_next, scale_x_next)
    M, K = Xq.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K:
        raise ValueError("Xq and Wq disagree on K")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=Xq.device)
    ldy = _rows(Y, "Y")
    c0, c1 = (0, 0) if q_cols is None else q_cols
    if q_cols is not None:
        if Xq_next is None:
            Xq_next = torch.empty((M, c1 - c0), dtype=code_dtype(qt), device=Xq.device)
        if scale_x_next is None:
            scale_x_next = torch.empty(M, dtype=torch.float32, device=Xq.device)
    need = workspace_size("qr_w8a8_gemm_quant", M, N, K, qt)
    if ws is None:
        ws, wsb = quant_workspace(need, Xq.device)
    else:
        wsb = ws.numel() * ws.element_size()
    with torch.cuda.device(Xq.device):
        st = lib().qr_w8a8_gemm_quant(_ptr(Xq), _ptr(scale_x), _ptr(Wq), _ptr(scale_w), M, N, K,
                                      _qt(qt), _ptr(Y), ldy, c0, c1 - c0, float(q_act_mult),
                                      _ptr(Xq_next), _ptr(scale_x_next), _ptr(ws), wsb,
                                      _stream(Xq.device))
    _check("qr_w8a8_gemm_quant", st)
    return Y, Xq_next, scale_x_next


def linear_fused(X, act_mult, Wq, scale_w, qt, Y=None, ws=None):
    """One rollout linear: per-token quantization of bf16 X, W8A8 product, bf16 Y."""
    _need_cuda(X, Wq, scale_w, Y)
    if X.dtype != torch.bfloat16:
        raise ValueError("X must be bfloat16")
    M, K = X.shape
    N = Wq.shape[0]
    ldx = _rows(X, "X")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    ldy = _rows(Y, "Y")
    need = workspace_size("qr_linear_fused", M, N, K, qt)
    if ws is None:
        ws, wsb = workspace(need, X.device)
    else:
        wsb = ws.numel() * ws.element_size()
    with torch.cuda.device(X.device):
        st = lib().qr_linear_fused(_ptr(X), ldx, float(act_mult), _ptr(Wq), _ptr(scale_w), M, N, K,
                                   _qt(qt), _ptr(Y), ldy, _ptr(ws), wsb, _stream(X.device))
    _check("qr_linear_fused", st)
    return Y


def linear_fused_noalloc(X, act_mult, Wq, scale_w, qt, Y=None):
    """linear_fused with the library's fixed device scratch instead of a
    workspace: the call allocates nothing (Y must be given to avoid torch's
    own allocation)."""
    _need_cuda(X, Wq, scale_w, Y)
    if X.dtype != torch.bfloat16:
        raise ValueError("X must be bfloat16")
    M, K = X.shape
    N = Wq.shape[0]
    ldx = _rows(X, "X")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    ldy = _rows(Y, "Y")
    with torch.cuda.device(X.device):
        st = lib().qr_linear_fused_noalloc(_ptr(X), ldx, float(act_mult), _ptr(Wq), _ptr(scale_w),
                                           M, N, K, _qt(qt), _ptr(Y), ldy, _stream(X.device))
    _check("qr_linear_fused_noalloc", st)
    return Y


# ----------------------------------------------------------------------------
# MXFP4 operators and block norms. Decode calls are a few microseconds on the GPU, so
# the marshalling here is kept short (one-token mxfp4_linear: 10.8 us of host time with
# this module's general helpers, 7 with these): the stream as a plain handle, no
# device switch where the tensors' device is current, scratch from torch's allocator
# (stream-ordered; a graph's own pool under capture, so captured graphs never share it).
# ----------------------------------------------------------------------------

def _call(fn, idx, *args):
    """Call library function `fn` on the current stream of device `idx`, made current."""
    f = getattr(_lib or lib(), fn)
    if idx == torch._C._cuda_getDevice():
        st = f(*args, torch._C._cuda_getCurrentRawStream(idx))
    else:
        with torch.cuda.device(idx):
            st = f(*args, torch._C._cuda_getCurrentRawStream(idx))
    if st != 0:
        _check(fn, st)


def _one_device(dev, *ts):
    """Every given tensor lives on HIP device `dev`; returns its index."""
    if dev.type != "cuda":
        raise ValueError("tensors must live on a HIP device")
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}: one device expected")
    return dev.index


def _ld(t, name):
    """Row stride of a 2-D tensor with contiguous rows."""
    return t.shape[-1] or 1 if t.is_contiguous() else _rows(t, name)


def _addr(t):
    return None if t is None else t.data_ptr()


def _out(t, like, shape, dtype, name):
    """A new dense output beside `like`, or the caller's after a check of its shape and type."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
    return t


def _mx_codes(codes, scales, name):
    """(rows, K, format) of block-wise codes and their scale panels: uint8 holds two E2M1
    codes a byte."""
    if codes.dim() != 2 or not codes.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D tensor of codes")
    R, K = codes.shape
    if codes.dtype == torch.uint8:
        K, fmt = 2 * K, 3
    elif codes.dtype == torch.float8_e4m3fn:
        fmt = 2
    else:
        raise ValueError(f"{name} must be uint8 (MXFP4) or float8_e4m3fn (block-wise FP8) codes")
    if scales.dtype != torch.uint8 or scales.shape != ((K + 127) // 128, R, 4) or not scales.is_contiguous():
        raise ValueError(f"the scales of {name} must be contiguous uint8 panels {((K + 127) // 128, R, 4)}")
    return R, K, fmt


def _mx_out(like, M, K, fmt, codes, scales):
    """Outputs of a producer with block-wise codes."""
    if fmt == "mxfp4":
        codes = _out(codes, like, (M, K // 2), torch.uint8, "codes")
    else:
        codes = _out(codes, like, (M, K), torch.float8_e4m3fn, "codes")
    return codes, _out(scales, like, ((K + 127) // 128, M, 4), torch.uint8, "scales")


def mxfp4_quantize(A, codes=None, scales=None):
    """MXFP4 of fp32 or bf16 rows A [R, K] -> (codes uint8 [R, K/2], two E2M1 codes a
    byte, E8M0 scales uint8 [ceil(K/128), R, 4])."""
    idx = _one_device(A.device, codes, scales)
    if A.dtype != torch.float32 and A.dtype != torch.bfloat16:
        raise ValueError("A must be float32 or bfloat16")
    lda = _ld(A, "A")
    R, K = A.shape
    if K % 32:
        raise QRError("qr_mxfp4_quantize", -2, f"K={K} is not a multiple of 32")
    codes, scales = _mx_out(A, R, K, "mxfp4", codes, scales)
    _call("qr_mxfp4_quantize", idx, A.data_ptr(), R, K, lda, int(A.dtype == torch.bfloat16),
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def mx_dequantize(codes, scales, out=None, dtype=torch.bfloat16):
    """The values of MXFP4 (uint8) or block-wise FP8 (float8_e4m3fn) codes, bf16 or fp32
    [R, K]; `out` may have any row stride."""
    idx = _one_device(codes.device, scales, out)
    R, K, fmt = _mx_codes(codes, scales, "codes")
    if out is None:
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("dtype must be bfloat16 or float32")
        out, ldo = codes.new_empty((R, K), dtype=dtype), K
    elif out.shape != (R, K) or out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out must be a bfloat16 or float32 tensor of the codes' rows and K")
    else:
        ldo = _ld(out, "out")
    _call("qr_mx_dequantize", idx, codes.data_ptr(), scales.data_ptr(), R, K, fmt, out.data_ptr(), ldo,
          int(out.dtype == torch.bfloat16))
    return out


def _mx4_out(Y, like, M, N, dtype):
    if Y is None:
        return like.new_empty((M, N), dtype=dtype), N
    if Y.shape != (M, N) or Y.dtype != dtype:
        raise ValueError(f"Y must be {dtype} [{M}, {N}]")
    return Y, _ld(Y, "Y")


_mx4_ws = {}


def _mx4_workspace(fn, M, N, K, xfmt, like, ws):
    """(workspace address or None, bytes, its tensor) of a call; sizes are kept per shape."""
    if ws is not None:
        if not ws.is_contiguous():
            raise ValueError("ws must be contiguous")
        return ws.data_ptr(), ws.numel() * ws.element_size(), ws
    need = _mx4_ws.get((fn, M, N, K, xfmt))
    if need is None:
        need = lib().qr_workspace_size(fn.encode(), M, N, K, xfmt)
        if need == ctypes.c_size_t(-1).value:
            raise QRError(fn, -2, lib().qr_last_error().decode())
        if len(_mx4_ws) > 4096:
            _mx4_ws.clear()
        _mx4_ws[(fn, M, N, K, xfmt)] = need
    if need == 0:
        return None, 0, None
    ws = like.new_empty(need, dtype=torch.uint8)
    return ws.data_ptr(), need, ws


def _tokens(x):
    """QR_ACT_* format of an MXFP4 product's tokens."""
    if x == "fp4":
        return 3
    if x == "fp8":
        return 2
    raise ValueError(f"x must be 'fp4' or 'fp8', got {x!r}")


def mxfp4_plan(M, N, K, x="fp4"):
    """(weight rows of a tile, tokens of a tile or 0 for the kernel of few tokens, K splits, whether
    blocks copy into their next tile ahead): the plan mxfp4_gemm uses for this shape."""
    n, m, s, a = (ctypes.c_int() for _ in range(4))
    _check("qr_mxfp4_plan", lib().qr_mxfp4_plan(M, N, K, _tokens(x), *(ctypes.byref(v) for v in (n, m, s, a))))
    return n.value, m.value, s.value, bool(a.value)


def mxfp4_gemm(Xq, sx, Wq, sw, out="bf16", Y=None, ws=None):
    """Product of quantized tokens (uint8 MXFP4 or float8_e4m3fn block-wise codes [M, K] with
    their scale panels) with MXFP4 weights Wq [N, K/2]: bf16 Y [M, N] or the fp32 accumulators.
    `ws`, if given, holds workspace_size("qr_mxfp4_gemm", ...) bytes, 256-byte aligned."""
    idx = _one_device(Xq.device, sx, Wq, sw, Y, ws)
    M, K, xfmt = _mx_codes(Xq, sx, "Xq")
    N, Kw, wfmt = _mx_codes(Wq, sw, "Wq")
    if wfmt != 3 or Kw != K:
        raise ValueError("Wq must be uint8 MXFP4 codes of Xq's K")
    if out not in OUT:
        raise ValueError(f"out must be one of {list(OUT)}")
    Y, ldy = _mx4_out(Y, Xq, M, N, torch.bfloat16 if out == "bf16" else torch.float32)
    wsp, wsb, ws = _mx4_workspace("qr_mxfp4_gemm", M, N, K, xfmt, Xq, ws)
    _call("qr_mxfp4_gemm", idx, Xq.data_ptr(), sx.data_ptr(), xfmt, Wq.data_ptr(), sw.data_ptr(), M, N, K,
          OUT[out], Y.data_ptr(), ldy, wsp, wsb)
    return Y


def mxfp4_linear(X, Wq, sw, x="fp4", Y=None, ws=None):
    """One rollout linear with MXFP4 weights: bf16 X [M, K] (any row stride) quantized block-wise
    to `x` ("fp4" or "fp8"), product, bf16 Y [M, N]. `ws` as for mxfp4_gemm ("qr_mxfp4_linear")."""
    idx = _one_device(X.device, Wq, sw, Y, ws)
    if X.dtype != torch.bfloat16:
        raise ValueError("X must be bfloat16")
    xfmt = _tokens(x)
    ldx = _ld(X, "X")
    M, K = X.shape
    N, Kw, wfmt = _mx_codes(Wq, sw, "Wq")
    if wfmt != 3 or Kw != K:
        raise ValueError("Wq must be uint8 MXFP4 codes of X's K")
    Y, ldy = _mx4_out(Y, X, M, N, torch.bfloat16)
    wsp, wsb, ws = _mx4_workspace("qr_mxfp4_linear", M, N, K, xfmt, X, ws)
    _call("qr_mxfp4_linear", idx, X.data_ptr(), ldx, xfmt, Wq.data_ptr(), sw.data_ptr(), M, N, K,
          Y.data_ptr(), ldy, wsp, wsb)
    return Y


def _gate_ld(gate, shape):
    """Row stride of a gate: 0 says one fp32 value per channel, else rows of bf16 [M, K]. Rows
    that are one row expanded have stride 0 too: refused here like those of Y and H in the
    library, which would take them for the fp32 gate."""
    if gate.dtype == torch.bfloat16 and gate.shape == shape:
        ld = _ld(gate, "gate")
        if ld < shape[1]:
            raise QRError("qr_block_norm_quant", -1, f"a row stride below K={shape[1]} (gate)")
        return ld
    if gate.dtype != torch.float32 or gate.shape != shape[1:] or not gate.is_contiguous():
        raise ValueError("gate must be float32 [K] or bfloat16 [M, K]")
    return 0


def block_norm_quant(Y, H, gamma, fmt, post_gamma=None, gate=None, res_scale=1.0, beta=None,
                     post_beta=None, eps=1e-6, kind="rms", Hout=None, codes=None, scales=None):
    """The step between two blocks: Hout = bf16(res_scale * H + gate * post_norm(Y)), and
    norm(Hout) with gain gamma in format fmt ("int8", "fp8", "mxfp8", "mxfp4" or "bf16") ->
    (Hout, codes, scales); scales is None for "bf16".

    Y, H bf16 [M, K]; gamma, beta, post_gamma, post_beta fp32 [K]; gate None, fp32 [K] or bf16
    [M, K] (rows of their own, not one expanded). Hout may be H or Y (updated in place)."""
    idx = _one_device(Y.device, H, gamma, post_gamma, gate, beta, post_beta, Hout, codes, scales)
    shape = Y.shape
    if Y.dtype != torch.bfloat16 or H.dtype != torch.bfloat16 or H.shape != shape:
        raise ValueError("Y and H must be bfloat16 of one shape")
    if fmt not in ACT:
        raise ValueError(f"fmt must be one of {list(ACT)}, got {fmt!r}")
    if kind not in NORM:
        raise ValueError(f"kind must be one of {list(NORM)}")
    ldy, ldh = _ld(Y, "Y"), _ld(H, "H")
    M, K = shape
    for t in (gamma, post_gamma, beta, post_beta):
        if t is not None and (t.dtype != torch.float32 or t.numel() != K or not t.is_contiguous()):
            raise ValueError("gains and biases must be contiguous float32 tensors of K entries")
    ldgate = 0 if gate is None else _gate_ld(gate, shape)
    if Hout is None:
        Hout, ldo = Y.new_empty(shape), K
    elif Hout.shape != shape or Hout.dtype != torch.bfloat16:
        raise ValueError("Hout must be bfloat16 of Y's shape")
    else:
        ldo = _ld(Hout, "Hout")
    if fmt == "bf16":
        codes, scales = _out(codes, Y, (M, K), torch.bfloat16, "codes"), None
    elif fmt == "int8" or fmt == "fp8":
        codes = _out(codes, Y, (M, K), code_dtype(fmt), "codes")
        scales = _out(scales, Y, (M,), torch.float32, "scales")
    else:
        if K % 32:
            raise QRError("qr_block_norm_quant", -2, f"K={K} is not a multiple of 32")
        codes, scales = _mx_out(Y, M, K, fmt, codes, scales)
    _call("qr_block_norm_quant", idx, Y.data_ptr(), ldy, H.data_ptr(), ldh, M, K, NORM[kind],
          _addr(post_gamma), _addr(post_beta), _addr(gate), ldgate, res_scale, gamma.data_ptr(),
          _addr(beta), eps, ACT[fmt], Hout.data_ptr(), ldo, codes.data_ptr(), _addr(scales))
    return Hout, codes, scales


def silu_mul_mx(G, U, fmt, codes=None, scales=None):
    """SiLU(G) * U for bf16 [M, N] views (rows contiguous, any row strides), quantized block-wise to
    fmt ("mxfp4" or "mxfp8") -> (codes, scales)."""
    idx = _one_device(G.device, U, codes, scales)
    if G.dtype != torch.bfloat16 or U.dtype != torch.bfloat16 or G.shape != U.shape:
        raise ValueError("G and U must be bfloat16 of one shape")
    if fmt not in ("mxfp4", "mxfp8"):
        raise ValueError(f"fmt must be 'mxfp4' or 'mxfp8', got {fmt!r}")
    ldg, ldu = _ld(G, "G"), _ld(U, "U")
    M, N = G.shape
    if N % 32:
        raise QRError("qr_silu_mul_mx", -2, f"N={N} is not a multiple of 32")
    codes, scales = _mx_out(G, M, N, fmt, codes, scales)
    _call("qr_silu_mul_mx", idx, G.data_ptr(), U.data_ptr(), M, N, ldg, ldu, ACT[fmt], codes.data_ptr(),
          scales.data_ptr())
    return codes, scales


# ----------------------------------------------------------------------------
# Losses over a large vocabulary
# ----------------------------------------------------------------------------

def _head_args(X, W):
    """(M, N, K, row strides) of bf16 hidden states X [M, K] and head W [N, K]."""
    if X.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise ValueError("X and W must be bfloat16")
    if X.dim() != 2 or W.dim() != 2:
        raise ValueError("X and W must be 2-D")
    ldx, ldw = _ld(X, "X"), _ld(W, "W")
    if W.shape[1] != X.shape[1]:
        raise ValueError("X and W disagree on K")
    return X.shape[0], W.shape[0], X.shape[1], ldx, ldw


def _per_token(t, M, dtype, name):
    if t.dtype != dtype or t.shape != (M,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {M} entries")


def _list_args(index, teacher, teacher_lse, M):
    """Entries of a token's list."""
    if index.dtype != torch.int64 or index.dim() != 2 or index.shape[0] != M or not index.is_contiguous():
        raise ValueError("index must be a contiguous int64 tensor [M, L]")
    if teacher.dtype not in (torch.float32, torch.bfloat16) or teacher.shape != index.shape \
            or not teacher.is_contiguous():
        raise ValueError("teacher must be a contiguous float32 or bfloat16 tensor of index's shape")
    if teacher_lse is not None:
        _per_token(teacher_lse, M, torch.float32, "teacher_lse")
    return index.shape[1]


def _grads(X, W, need_dX, need_dW, dX, dW):
    """Gradient outputs and their row strides."""
    out = []
    for t, like, need, name in ((dX, X, need_dX, "dX"), (dW, W, need_dW, "dW")):
        if t is None and need:
            t = like.new_empty(like.shape)
        elif t is not None and (t.shape != like.shape or t.dtype != torch.bfloat16):
            raise ValueError(f"{name} must be bfloat16 of the shape of its tensor")
        out += [t, like.shape[1] if t is None else _ld(t, name)]
    if out[0] is None and out[2] is None:
        raise ValueError("neither dX nor dW asked for")
    return out


def vocab_plan(M, N, K):
    """(ids and tokens of a tile of the logits, rows of a tile of dX, ids of a gradient's piece) of the
    plan that the calls use for M >= 1 tokens, N ids and K hidden values."""
    a, b, c, d = ctypes.c_int(), ctypes.c_int(), ctypes.c_int(), ctypes.c_int64()
    _check("qr_vocab_plan", lib().qr_vocab_plan(M, N, K, *(ctypes.byref(v) for v in (a, b, c, d))))
    return a.value, b.value, c.value, d.value


def vocab_logp(X, W, target, scale=1.0, logp=None, lse=None, ws=None):
    """Log-probabilities of one id per token, without the logits: X [M, K] bf16 hidden states, W [N, K]
    bf16 head (rows contiguous, any row strides), target int64 [M] -> (logp fp32 [M], lse fp32 [M]);
    logits are scale * X W^T. Targets outside [0, N) mask their tokens (0). `ws`, if given, holds
    workspace_size("qr_vocab_logp", M, N, K, 1) bytes, 256-byte aligned."""
    idx = _one_device(X.device, W, target, logp, lse, ws)
    M, N, K, ldx, ldw = _head_args(X, W)
    _per_token(target, M, torch.int64, "target")
    logp, lse = _out(logp, X, (M,), torch.float32, "logp"), _out(lse, X, (M,), torch.float32, "lse")
    wsp, wsb, ws = _mx4_workspace("qr_vocab_logp", M, N, K, 1, X, ws)
    _call("qr_vocab_logp", idx, X.data_ptr(), ldx, W.data_ptr(), ldw, M, N, K, target.data_ptr(), scale,
          logp.data_ptr(), lse.data_ptr(), wsp, wsb)
    return logp, lse


def vocab_logp_grad(X, W, target, lse, dlogp, scale=1.0, need_dX=True, need_dW=True, dX=None, dW=None, ws=None):
    """Gradient of vocab_logp: with its lse and dlogp = d loss / d logp (fp32 [M]) -> (dX [M, K],
    dW [N, K]) in bf16, None where not needed. Given dX and dW are overwritten (any row strides).
    `ws` as for vocab_logp ("qr_vocab_logp_grad")."""
    idx = _one_device(X.device, W, target, lse, dlogp, dX, dW, ws)
    M, N, K, ldx, ldw = _head_args(X, W)
    _per_token(target, M, torch.int64, "target")
    _per_token(lse, M, torch.float32, "lse")
    _per_token(dlogp, M, torch.float32, "dlogp")
    dX, lddx, dW, lddw = _grads(X, W, need_dX, need_dW, dX, dW)
    wsp, wsb, ws = _mx4_workspace("qr_vocab_logp_grad", M, N, K, 1, X, ws)
    _call("qr_vocab_logp_grad", idx, X.data_ptr(), ldx, W.data_ptr(), ldw, M, N, K, target.data_ptr(), scale,
          lse.data_ptr(), dlogp.data_ptr(), _addr(dX), lddx, _addr(dW), lddw, wsp, wsb)
    return dX, dW


def vocab_distill(X, W, index, teacher, scale=1.0, teacher_lse=None, loss=None, lse=None, ws=None):
    """Divergence from a teacher's top logits, without the student's logits: token t has the ids
    index[t] (int64 [M, L], ids outside [0, N) are no entries) with the teacher's logits teacher[t]
    (fp32 or bf16 [M, L]), weighted by their softmax, or with teacher_lse (fp32 [M]) by
    exp(scale * teacher - teacher_lse) -> (loss fp32 [M], lse fp32 [M]). X, W, scale and ws as for
    vocab_logp ("qr_vocab_distill", with L)."""
    idx = _one_device(X.device, W, index, teacher, teacher_lse, loss, lse, ws)
    M, N, K, ldx, ldw = _head_args(X, W)
    L = _list_args(index, teacher, teacher_lse, M)
    loss, lse = _out(loss, X, (M,), torch.float32, "loss"), _out(lse, X, (M,), torch.float32, "lse")
    wsp, wsb, ws = _mx4_workspace("qr_vocab_distill", M, N, K, L, X, ws)
    _call("qr_vocab_distill", idx, X.data_ptr(), ldx, W.data_ptr(), ldw, M, N, K, index.data_ptr(),
          teacher.data_ptr(), int(teacher.dtype == torch.bfloat16), _addr(teacher_lse), L, scale,
          loss.data_ptr(), lse.data_ptr(), wsp, wsb)
    return loss, lse


def vocab_distill_grad(X, W, index, teacher, lse, dloss, scale=1.0, teacher_lse=None, need_dX=True, need_dW=True,
                       dX=None, dW=None, ws=None):
    """Gradient of vocab_distill: with its lse and dloss = d objective / d loss (fp32 [M]) -> (dX, dW)
    as vocab_logp_grad."""
    idx = _one_device(X.device, W, index, teacher, teacher_lse, lse, dloss, dX, dW, ws)
    M, N, K, ldx, ldw = _head_args(X, W)
    L = _list_args(index, teacher, teacher_lse, M)
    _per_token(lse, M, torch.float32, "lse")
    _per_token(dloss, M, torch.float32, "dloss")
    dX, lddx, dW, lddw = _grads(X, W, need_dX, need_dW, dX, dW)
    wsp, wsb, ws = _mx4_workspace("qr_vocab_distill_grad", M, N, K, L, X, ws)
    _call("qr_vocab_distill_grad", idx, X.data_ptr(), ldx, W.data_ptr(), ldw, M, N, K, index.data_ptr(),
          teacher.data_ptr(), int(teacher.dtype == torch.bfloat16), _addr(teacher_lse), L, scale,
          lse.data_ptr(), dloss.data_ptr(), _addr(dX), lddx, _addr(dW), lddw, wsp, wsb)
    return dX, dW


# ----------------------------------------------------------------------------
# Measurement helpers (peaks the chip reaches; not part of the linear)
# ----------------------------------------------------------------------------

def probe_read(buf, sink=None):
    """Enqueue one read of the whole byte buffer `buf` (a contiguous device
    tensor whose size is a multiple of 16 bytes); returns the sink tensor."""
    _need_cuda(buf, sink)
    nbytes = buf.numel() * buf.element_size()
    if sink is None:
        sink = torch.empty(2048, dtype=torch.int32, device=buf.device)
    with torch.cuda.device(buf.device):
        st = lib().qr_probe_read(_ptr(buf), nbytes, _ptr(sink), sink.numel(), _stream(buf.device))
    _check("qr_probe_read", st)
    return sink


PROBE_PANEL, PROBE_NO_BARRIER, PROBE_RESIDENT = 1, 2, 4


def probe_copy_stream(tile, Wq, Xq, rows, sink=None, panel=False, barrier=True, resident=False):
    """Enqueue the operand copies GEMM tile `tile` (4, 8 or 10) makes over the
    8-bit code matrices Wq [N, K] and Xq [M, K] (rows contiguous; their row
    strides are passed on) with `rows` weight rows per tile, without the
    matrix work; panel reads Wq's bytes as K panels instead (Wq contiguous),
    barrier=False drops the barrier per K step, resident=True copies K step
    0's bytes at every step (operands resident in L2). Returns the sink
    tensor (one word per block)."""
    _need_cuda(Wq, Xq, sink)
    if Wq.dim() != 2 or Xq.dim() != 2 or Wq.shape[1] != Xq.shape[1]:
        raise ValueError("Wq [N, K] and Xq [M, K] with the same K expected")
    if Wq.element_size() != 1 or Xq.element_size() != 1:
        raise ValueError("8-bit code matrices expected")
    if panel and not Wq.is_contiguous():
        raise ValueError("panel reads need a contiguous Wq")
    (N, K), M = Wq.shape, Xq.shape[0]
    ldw, ldx = _rows(Wq, "Wq"), _rows(Xq, "Xq")
    bm = {4: 256, 8: 128, 10: 256}.get(tile, 1)
    grid = -(-N // max(rows, 1)) * -(-M // bm)
    if sink is None:
        sink = torch.empty(max(grid, 1), dtype=torch.int32, device=Wq.device)
    flags = ((PROBE_PANEL if panel else 0) | (0 if barrier else PROBE_NO_BARRIER)
             | (PROBE_RESIDENT if resident else 0))
    with torch.cuda.device(Wq.device):
        st = lib().qr_probe_copy_stream(tile, _ptr(Wq), N, ldw, _ptr(Xq), M, ldx, K, rows, flags,
                                        _ptr(sink), sink.numel(), _stream(Wq.device))
    _check("qr_probe_copy_stream", st)
    return sink


def probe_mfma(qt, blocks, iters, device="cuda:0", sink=None, ticks=None):
    """Enqueue the MFMA probe; returns (sink, ticks, wall clock rate in kHz)."""
    dev = torch.device(device)
    if sink is None:
        sink = torch.empty(8 * blocks, dtype=torch.int32, device=dev)
    if ticks is None:
        ticks = torch.empty(4 * blocks, dtype=torch.int64, device=dev)
    khz = ctypes.c_int(0)
    with torch.cuda.device(dev):
        st = lib().qr_probe_mfma(_qt(qt), blocks, iters, _ptr(sink), _ptr(ticks), ctypes.byref(khz),
                                 _stream(dev))
    _check("qr_probe_mfma", st)
    return sink, ticks, khz.value
