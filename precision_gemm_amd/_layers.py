"""Binding of the norms (``include/norm.h``), the 4-bit products
(``include/mx4gemm.h``) and the experts' layer of a few tokens (``expert_layer``
of ``include/experts.h``), in the manner of ``_experts.py``: the C names and
argument order without the type arguments, every operand checked before anything
is launched. 4-bit elements and their scales are uint8 tensors (or of torch's
types for them); their leading dimensions and strides count bytes, that of the
scales rows.
"""
from __future__ import annotations

import ctypes

import precision_gemm_amd as _pg

from . import _experts
from ._experts import _at, _first, _in_int, _span, _spans

RMS_NORM_GRAD_MAX_K = 16384
EXPERT_LAYER_MAX_SLOTS = 2048
EXPERT_LAYER_MAX_EXPERTS = 1024
# Kernels of the 4-bit product by number (mx4gemm_kernel of the C header): S
# stream B, T take rows of any alignment, L load straight into LDS.
MX4GEMM_KERNELS = ("S16x16", "S16x32", "S32x16", "S32x32", "S32x64", "T64x64", "T128x128",
                   "L64x64", "L64x128", "L128x128", "L128x128_R2", "L128x256", "L256x256")

torch = _experts.torch
if torch is not None:
    from ._experts import _F32, _FLOATS, _IDS, _INT8, _I32, _TYPES
    _MX4 = tuple(getattr(torch, n) for n in ("uint8", "float4_e2m1fn_x2") if hasattr(torch, n))
    _MX4_SCALE = tuple(getattr(torch, n) for n in ("uint8", "float8_e8m0fnu") if hasattr(torch, n))
    _W_TYPES = {**_TYPES, **{t: 4 for t in _MX4}}
_lib = None  # the loaded library, set by declare()


def declare(lib):
    """Argument types of the library's calls."""
    global _lib
    i, f, p, ll, sz = (ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_longlong,
                       ctypes.c_size_t)
    lib.rms_norm.argtypes = [i, i, p, i, i, p, i, p, f, p, i, p, i, p]
    lib.rms_norm_i8.argtypes = [i, i, p, i, i, p, i, p, f, p, i, p, i, p, p]
    lib.rms_norm_grad.argtypes = [i, i, p, i, i, p, i, p, f, p, i, p, i, p, p, sz, p]
    lib.rms_norm_grad_workspace_size.argtypes = [i, i, i]
    lib.mx4_quantize_rows.argtypes = [i, i, p, i, i, p, i, p, i, p]
    lib.mx4_dequantize_rows.argtypes = [i, i, p, i, p, i, p, i, i, p]
    lib.mx4gemm.argtypes = [i, i, i, p, i, p, i, p, i, p, i, p, p, i, i, p]
    lib.mx4gemm_grouped.argtypes = [i, i, i, i, p, p, i, p, i, p, i, ll, p, i, ll, p, p, i, i, p]
    lib.mx4gemm_select_kernel.argtypes = [i, i, i, i, i, i]
    lib.expert_layer.argtypes = [i, i, i, i, i, p, i, i, p, i, p, p, i, i, ll, p, p, i, ll, p, p,
                                 i, p, sz, p]
    lib.expert_layer_workspace_size.argtypes = [i, i, i, i, i]
    for name in ("rms_norm", "rms_norm_i8", "rms_norm_grad", "mx4_quantize_rows",
                 "mx4_dequantize_rows", "mx4gemm", "mx4gemm_grouped", "expert_layer",
                 "mx4gemm_select_kernel"):
        getattr(lib, name).restype = i
    lib.rms_norm_grad_workspace_size.restype = sz
    lib.expert_layer_workspace_size.restype = sz
    _lib = lib


def _workspace(workspace, device):
    if workspace is None:
        return None, 0
    at = _at("workspace", workspace, (getattr(workspace, "dtype", None),), device, 0, True)
    return at, workspace.numel() * workspace.element_size()


def _bytes(K):
    """Bytes of a row of K 4-bit elements."""
    if K < 0:
        _in_int(K=K)
    return (K + 1) // 2 if K > 0 else 0


def _scales(K, lds, rows):
    """Bytes of the scales of `rows` rows of K elements, lds rows apart."""
    if 0 < K <= _experts._INT_MAX and 0 < rows <= lds <= _experts._INT_MAX:
        return 4 * (((K + 127) // 128 - 1) * lds + rows)
    _in_int(K=K, rows=rows, lds=lds)
    return 0


def rms_norm(M, K, X, ldx, R, ldr, weight, eps, H, ldh, Y, ldy, stream=None, check=True) -> int:
    """C ABI ``rms_norm``: H = X + R, Y = H / sqrt(mean(H^2) + eps) * weight; X,
    R, H and Y of one type (fp32, fp16 or bf16), R and H may be None."""
    d = _first("X", X)
    dt = (X.dtype,)
    return _experts._call(
        _lib.rms_norm, d, stream, check, M, K, _at("X", X, _FLOATS, d, _span(M, K, ldx)),
        _TYPES[X.dtype], ldx, None if R is None else _at("R", R, dt, d, _span(M, K, ldr)), ldr,
        _at("weight", weight, _F32, d, K, True), float(eps),
        None if H is None else _at("H", H, dt, d, _span(M, K, ldh)), ldh,
        _at("Y", Y, dt, d, _span(M, K, ldy)), ldy)


def rms_norm_i8(M, K, X, ldx, R, ldr, weight, eps, H, ldh, Q, ldq, scale, stream=None,
                check=True) -> int:
    """C ABI ``rms_norm_i8``: the same in int8 with one fp32 scale a row."""
    d = _first("X", X)
    dt = (X.dtype,)
    return _experts._call(
        _lib.rms_norm_i8, d, stream, check, M, K, _at("X", X, _FLOATS, d, _span(M, K, ldx)),
        _TYPES[X.dtype], ldx, None if R is None else _at("R", R, dt, d, _span(M, K, ldr)), ldr,
        _at("weight", weight, _F32, d, K, True), float(eps),
        None if H is None else _at("H", H, dt, d, _span(M, K, ldh)), ldh,
        _at("Q", Q, _INT8, d, _span(M, K, ldq)), ldq, _at("scale", scale, _F32, d, M, True))


def rms_norm_grad_workspace_size(M, K, dtype) -> int:
    """C ABI ``rms_norm_grad_workspace_size`` (bytes); dtype: that of dY."""
    return int(_pg._load().rms_norm_grad_workspace_size(M, K, _TYPES[dtype]))


def rms_norm_grad(M, K, dY, lddy, H, ldh, weight, eps, dH, lddh, dX, lddx, dweight, workspace,
                  stream=None, check=True) -> int:
    """C ABI ``rms_norm_grad``: dX and dweight (fp32, or None) from dY and dH
    (or None); workspace: a GPU tensor of any type, or None without dweight."""
    d = _first("dY", dY)
    dt = (dY.dtype,)
    return _experts._call(
        _lib.rms_norm_grad, d, stream, check, M, K, _at("dY", dY, _FLOATS, d, _span(M, K, lddy)),
        _TYPES[dY.dtype], lddy, _at("H", H, dt, d, _span(M, K, ldh)), ldh,
        _at("weight", weight, _F32, d, K, True), float(eps),
        None if dH is None else _at("dH", dH, dt, d, _span(M, K, lddh)), lddh,
        _at("dX", dX, dt, d, _span(M, K, lddx)), lddx,
        None if dweight is None else _at("dweight", dweight, _F32, d, K, True),
        *_workspace(workspace, d))


def mx4_quantize_rows(M, K, X, ldx, Q, ldq, scale, lds, stream=None, check=True) -> int:
    """C ABI ``mx4_quantize_rows``: rows of X (fp32, fp16 or bf16) to 4-bit
    blocks, two elements a byte of Q, with their scales."""
    d = _first("X", X)
    return _experts._call(
        _lib.mx4_quantize_rows, d, stream, check, M, K,
        _at("X", X, _FLOATS, d, _span(M, K, ldx)), _TYPES[X.dtype], ldx,
        _at("Q", Q, _MX4, d, _span(M, _bytes(K), ldq)), ldq,
        _at("scale", scale, _MX4_SCALE, d, _scales(K, lds, M), True), lds)


def mx4_dequantize_rows(M, K, Q, ldq, scale, lds, Y, ldy, stream=None, check=True) -> int:
    """C ABI ``mx4_dequantize_rows``: the blocks' values in Y (fp32, fp16 or
    bf16)."""
    d = _first("Q", Q)
    return _experts._call(
        _lib.mx4_dequantize_rows, d, stream, check, M, K,
        _at("Q", Q, _MX4, d, _span(M, _bytes(K), ldq)), ldq,
        _at("scale", scale, _MX4_SCALE, d, _scales(K, lds, M), True), lds,
        _at("Y", Y, _FLOATS, d, _span(M, K, ldy)), _TYPES[Y.dtype], ldy)


def mx4gemm(M, N, K, A, lda, scaleA, ldsa, B, ldb, scaleB, ldsb, bias, C, ldc, stream=None,
            check=True) -> int:
    """C ABI ``mx4gemm``: C = A B^T + bias, A (M x K) and B (N x K) in 4-bit
    blocks, bias fp32 or None, C fp32, fp16 or bf16."""
    d = _first("A", A)
    width = _bytes(K)
    return _experts._call(
        _lib.mx4gemm, d, stream, check, M, N, K,
        _at("A", A, _MX4, d, _span(M, width, lda)), lda,
        _at("scaleA", scaleA, _MX4_SCALE, d, _scales(K, ldsa, M), True), ldsa,
        _at("B", B, _MX4, d, _span(N, width, ldb)), ldb,
        _at("scaleB", scaleB, _MX4_SCALE, d, _scales(K, ldsb, N), True), ldsb,
        None if bias is None else _at("bias", bias, _F32, d, N, True),
        _at("C", C, _FLOATS, d, _span(M, N, ldc)), _TYPES[C.dtype], ldc)


def mx4gemm_grouped(M, N, K, groups, offsets, A, lda, scaleA, ldsa, B, ldb, strideB, scaleB, ldsb,
                    strideSB, bias, C, ldc, stream=None, check=True) -> int:
    """C ABI ``mx4gemm_grouped``: mx4gemm over rows sorted by group; `offsets`
    holds groups + 1 int32, bias groups x N; strideB and strideSB in bytes."""
    d = _first("offsets", offsets)
    width = _bytes(K)
    _in_int(strideSB=min(strideSB, 0))
    n = _scales(K, ldsb, N)
    return _experts._call(
        _lib.mx4gemm_grouped, d, stream, check, M, N, K, groups,
        _at("offsets", offsets, _I32, d, groups + 1, True),
        _at("A", A, _MX4, d, _span(M, width, lda)), lda,
        _at("scaleA", scaleA, _MX4_SCALE, d, _scales(K, ldsa, M), True), ldsa,
        _at("B", B, _MX4, d, _spans(groups, strideB, N, width, ldb)), ldb, strideB,
        _at("scaleB", scaleB, _MX4_SCALE, d,
            (groups - 1) * strideSB + n if groups > 0 and n > 0 else 0, True), ldsb,
        strideSB,
        None if bias is None else _at("bias", bias, _F32, d, groups * N, True),
        _at("C", C, _FLOATS, d, _span(M, N, ldc)), _TYPES[C.dtype], ldc)


def mx4gemm_select_kernel(M, N, K, groups, aligned, num_cus) -> int:
    """C ABI ``mx4gemm_select_kernel`` (host-side dispatch decision): an index of
    MX4GEMM_KERNELS, or a negative status."""
    return _pg._load().mx4gemm_select_kernel(M, N, K, groups, int(bool(aligned)), num_cus)


def expert_layer_workspace_size(tokens, topk, H, F, dtype) -> int:
    """C ABI ``expert_layer_workspace_size`` (bytes); dtype: that of X."""
    return int(_pg._load().expert_layer_workspace_size(tokens, topk, H, F, _TYPES[dtype]))


def expert_layer(tokens, topk, experts, H, F, X, ldx, ids, weights, W1, ldw1, strideW1, scale1, W2,
                 ldw2, strideW2, scale2, out, ldo, workspace, stream=None, check=True) -> int:
    """C ABI ``expert_layer``: out[t] = sum_j weights[t, j] W2_e (silu(W1_e[:F]
    X[t]) * (W1_e[F:] X[t])), e = ids[t, j]. X and out fp32, fp16 or bf16; W1
    and W2 of that type (scale1 and scale2 None), int8 with fp32 scales a row, or
    4-bit blocks (uint8, strides in bytes) with theirs; weights fp32 or None."""
    d = _first("X", X)
    for name, n in (("tokens", tokens), ("topk", topk), ("experts", experts)):
        if n < 0:
            _in_int(**{name: n})
    slots = tokens * topk
    if slots < 0:
        _in_int(tokens=tokens, topk=topk)
    px = _at("X", X, _FLOATS, d, _span(tokens, H, ldx))
    kinds = (X.dtype,) + _INT8 + _MX4
    _at("W1", W1, kinds, d, 0)
    w_type = _W_TYPES[W1.dtype]
    width1, width2 = (_bytes(H), _bytes(F)) if w_type == 4 else (H, F)
    p1 = _at("W1", W1, kinds, d, _spans(experts, strideW1, 2 * F, width1, ldw1))
    s1 = s2 = None
    if w_type == 3:
        s1 = _at("scale1", scale1, _F32, d, experts * 2 * F, True)
        s2 = _at("scale2", scale2, _F32, d, experts * H, True)
    elif w_type == 4:
        s1 = _at("scale1", scale1, _MX4_SCALE, d, experts * _scales(H, 2 * F, 2 * F), True)
        s2 = _at("scale2", scale2, _MX4_SCALE, d, experts * _scales(F, H, H), True)
    return _experts._call(
        _lib.expert_layer, d, stream, check, tokens, topk, experts, H, F,
        px, _TYPES[X.dtype], ldx,
        _at("ids", ids, _IDS, d, slots, True), ids.element_size(),
        None if weights is None else _at("weights", weights, _F32, d, slots, True),
        p1, w_type, ldw1, strideW1, s1,
        _at("W2", W2, (W1.dtype,), d, _spans(experts, strideW2, H, width2, ldw2)), ldw2,
        strideW2, s2, _at("out", out, (X.dtype,), d, _span(tokens, H, ldo)), ldo,
        *_workspace(workspace, d))
