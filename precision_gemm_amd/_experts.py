"""Binding of the calls around the experts of a mixture layer and of the 8-bit
integer products (``include/i8gemm.h``, ``include/experts.h`` and the grouped
products of ``include/sgemm.h``).

The functions have the C names and argument order, without the type arguments:
those come from the tensors. Operands are GPU tensors on one device; leading
dimensions and strides count elements. Each tensor is taken from its first
element on and has to reach as far as the call will go (the rows behind one
another at the leading dimension, whatever the tensor's own shape); one that is
too short, of another type or on another device is refused with a TypeError or
ValueError before anything is launched. The work runs on `stream`, or else on
the current stream of the operands' device.
"""
from __future__ import annotations

import ctypes

import torch

import precision_gemm_amd as _pg

EXPERT_SORT_MAX_EXPERTS = 1024
I8GEMM_MAX_K = 131071

_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int8: 3}
_FLOATS = (torch.float32, torch.float16, torch.bfloat16)


def declare(lib):
    """Argument types of the library's calls."""
    i, f, p, ll, sz = (ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_longlong,
                       ctypes.c_size_t)
    lib.i8_quantize_rows.argtypes = [i, i, p, i, i, p, i, p, p]
    lib.i8gemm.argtypes = [i, i, i, p, i, p, p, i, p, p, p, i, i, p]
    lib.i8gemm_grouped.argtypes = [i, i, i, i, p, p, i, p, p, i, ll, p, p, p, i, i, p]
    lib.expert_sort.argtypes = [i, i, i, p, i, p, p, p, sz, p]
    lib.expert_sort_workspace_size.argtypes = [i, i, i]
    lib.expert_gather.argtypes = [i, i, i, p, i, i, p, p, i, p]
    lib.expert_combine.argtypes = [i, i, i, p, i, i, p, p, p, i, p]
    lib.expert_combine_grad.argtypes = [i, i, i, p, i, i, p, i, p, p, p, i, p, p]
    lib.sgemm_grouped.argtypes = [i, i, i, i, i, p, f, p, i, p, i, ll, f, p, i, p]
    lib.sgemm_grouped_outer.argtypes = [i, i, i, i, p, f, p, i, p, i, f, p, i, ll, p]
    for name in ("i8_quantize_rows", "i8gemm", "i8gemm_grouped", "expert_sort", "expert_gather",
                 "expert_combine", "expert_combine_grad", "sgemm_grouped", "sgemm_grouped_outer"):
        getattr(lib, name).restype = i
    lib.expert_sort_workspace_size.restype = sz


class _Operands:
    """Checks one call's tensors and hands out their addresses."""

    def __init__(self):
        self.device = None

    def at(self, name, t, dtypes, rows, cols=1, ld=None):
        """Address of `rows` rows of `cols` elements, `ld` apart."""
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a GPU tensor")
        if t.dtype not in dtypes:
            raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
        if self.device is None:
            self.device = t.device
        elif t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the operands before it on {self.device}")
        need = (rows - 1) * (cols if ld is None else ld) + cols if rows > 0 and cols > 0 else 0
        have = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
        if need > have:
            raise ValueError(f"{name} holds {have} elements from its first one on, "
                             f"the call needs {need}")
        return t.data_ptr()

    def groups(self, name, t, dtypes, groups, stride, rows, cols, ld):
        """Address of `groups` matrices, `stride` apart."""
        at = self.at(name, t, dtypes, rows, cols, ld)
        if groups > 1 and rows > 0 and cols > 0:
            need = (groups - 1) * stride + (rows - 1) * ld + cols
            have = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
            if need > have:
                raise ValueError(f"{name} holds {have} elements from its first one on, "
                                 f"the call needs {need}")
        return at

    def call(self, name, stream, check, *args):
        fn = getattr(_pg._load(), name)
        if stream is None:
            stream = torch.cuda.current_stream(self.device).cuda_stream
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        if torch.cuda.current_device() == self.device.index:
            status = fn(*args, stream)
        else:
            with torch.cuda.device(self.device):
                status = fn(*args, stream)
        return _pg._check(status, check)


def i8_quantize_rows(M, K, X, ldx, Q, ldq, scale, stream=None, check=True) -> int:
    """C ABI ``i8_quantize_rows``: rows of X (fp32, fp16 or bf16) to 8-bit
    integers Q with one fp32 scale a row."""
    o = _Operands()
    return o.call("i8_quantize_rows", stream, check, M, K, o.at("X", X, _FLOATS, M, K, ldx),
                  _TYPES[X.dtype], ldx, o.at("Q", Q, (torch.int8,), M, K, ldq), ldq,
                  o.at("scale", scale, (torch.float32,), M))


def i8gemm(M, N, K, A, lda, scaleA, B, ldb, scaleB, bias, C, ldc, stream=None, check=True) -> int:
    """C ABI ``i8gemm``: C = (A B^T) * scaleA[m] * scaleB[n] + bias[n], A (M x
    K) and B (N x K) int8, bias fp32 or None, C fp32, fp16 or bf16."""
    o = _Operands()
    f32 = (torch.float32,)
    return o.call("i8gemm", stream, check, M, N, K, o.at("A", A, (torch.int8,), M, K, lda), lda,
                  o.at("scaleA", scaleA, f32, M), o.at("B", B, (torch.int8,), N, K, ldb), ldb,
                  o.at("scaleB", scaleB, f32, N),
                  None if bias is None else o.at("bias", bias, f32, N),
                  o.at("C", C, _FLOATS, M, N, ldc), _TYPES[C.dtype], ldc)


def i8gemm_grouped(M, N, K, groups, offsets, A, lda, scaleA, B, ldb, strideB, scaleB, bias, C,
                   ldc, stream=None, check=True) -> int:
    """C ABI ``i8gemm_grouped``: i8gemm over rows sorted by group; `offsets`
    holds groups + 1 int32, scaleB and bias groups x N."""
    o = _Operands()
    f32, i8 = (torch.float32,), (torch.int8,)
    return o.call("i8gemm_grouped", stream, check, M, N, K, groups,
                  o.at("offsets", offsets, (torch.int32,), groups + 1),
                  o.at("A", A, i8, M, K, lda), lda, o.at("scaleA", scaleA, f32, M),
                  o.groups("B", B, i8, groups, strideB, N if groups else 0, K, ldb), ldb, strideB,
                  o.at("scaleB", scaleB, f32, groups, N),
                  None if bias is None else o.at("bias", bias, f32, groups, N),
                  o.at("C", C, _FLOATS, M, N, ldc), _TYPES[C.dtype], ldc)


def expert_sort_workspace_size(tokens, topk, experts) -> int:
    """C ABI ``expert_sort_workspace_size`` (bytes)."""
    return int(_pg._load().expert_sort_workspace_size(tokens, topk, experts))


def expert_sort(tokens, topk, experts, ids, offsets, row_of_slot, workspace, stream=None,
                check=True) -> int:
    """C ABI ``expert_sort``: ids (int32 or int64, contiguous) to offsets and
    row_of_slot (int32); workspace: a GPU tensor of any type, or None where
    expert_sort_workspace_size() is 0."""
    o = _Operands()
    p_ids = o.at("ids", ids, (torch.int32, torch.int64), tokens * topk)
    ws, ws_bytes = None, 0
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != o.device:
            raise TypeError("workspace must be a GPU tensor on the operands' device")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    return o.call("expert_sort", stream, check, tokens, topk, experts, p_ids, ids.element_size(),
                  o.at("offsets", offsets, (torch.int32,), experts + 1),
                  o.at("row_of_slot", row_of_slot, (torch.int32,), tokens * topk), ws, ws_bytes)


def expert_gather(tokens, topk, cols, X, ldx, row_of_slot, Y, ldy, stream=None, check=True) -> int:
    """C ABI ``expert_gather``: Y[row_of_slot[t, j]] = X[t]; X and Y of one
    type, fp32, fp16, bf16 or int8."""
    o = _Operands()
    any_type = _FLOATS + (torch.int8,)
    slots = tokens * topk
    return o.call("expert_gather", stream, check, tokens, topk, cols,
                  o.at("X", X, any_type, tokens, cols, ldx), _TYPES[X.dtype], ldx,
                  o.at("row_of_slot", row_of_slot, (torch.int32,), slots),
                  o.at("Y", Y, (X.dtype,), slots, cols, ldy), ldy)


def expert_combine(tokens, topk, cols, Y, ldy, row_of_slot, weights, out, ldo, stream=None,
                   check=True) -> int:
    """C ABI ``expert_combine``: out[t] = sum_j weights[t, j] Y[row_of_slot[t,
    j]]; weights fp32, or None for 1 (the gradient of expert_gather)."""
    o = _Operands()
    slots = tokens * topk
    return o.call("expert_combine", stream, check, tokens, topk, cols,
                  o.at("Y", Y, _FLOATS, slots, cols, ldy), _TYPES[Y.dtype], ldy,
                  o.at("row_of_slot", row_of_slot, (torch.int32,), slots),
                  None if weights is None else o.at("weights", weights, (torch.float32,), slots),
                  o.at("out", out, (Y.dtype,), tokens, cols, ldo), ldo)


def expert_combine_grad(tokens, topk, cols, dout, ldo, Y, ldy, row_of_slot, weights, dY, lddy,
                        dweights, stream=None, check=True) -> int:
    """C ABI ``expert_combine_grad``: dY and dweights (fp32, or None: then Y
    may be None too) from dout."""
    o = _Operands()
    slots = tokens * topk
    f32 = (torch.float32,)
    return o.call("expert_combine_grad", stream, check, tokens, topk, cols,
                  o.at("dout", dout, _FLOATS, tokens, cols, ldo), _TYPES[dout.dtype], ldo,
                  None if Y is None else o.at("Y", Y, (dout.dtype,), slots, cols, ldy), ldy,
                  o.at("row_of_slot", row_of_slot, (torch.int32,), slots),
                  None if weights is None else o.at("weights", weights, f32, slots),
                  o.at("dY", dY, (dout.dtype,), slots, cols, lddy), lddy,
                  None if dweights is None else o.at("dweights", dweights, f32, slots))


def sgemm_grouped(transB, M, N, K, groups, offsets, alpha, A, lda, B, ldb, strideB, beta, C, ldc,
                  stream=None, check=True) -> int:
    """C ABI ``sgemm_grouped``: C[m] = alpha A[m] op(B_g) + beta C[m] for the
    rows offsets[g] <= m < offsets[g + 1] of every group."""
    o = _Operands()
    f32 = (torch.float32,)
    rows, cols = (N, K) if transB else (K, N)
    return o.call("sgemm_grouped", stream, check, int(transB), M, N, K, groups,
                  o.at("offsets", offsets, (torch.int32,), groups + 1), float(alpha),
                  o.at("A", A, f32, M, K, lda), lda,
                  o.groups("B", B, f32, groups, strideB, rows if groups else 0, cols, ldb), ldb,
                  strideB, float(beta), o.at("C", C, f32, M, N, ldc), ldc)


def sgemm_grouped_outer(M, N, K, groups, offsets, alpha, A, lda, B, ldb, beta, C, ldc, strideC,
                        stream=None, check=True) -> int:
    """C ABI ``sgemm_grouped_outer``: C_g = alpha A_g^T B_g + beta C_g over the
    rows offsets[g] <= k < offsets[g + 1] of A (K x M) and B (K x N)."""
    o = _Operands()
    f32 = (torch.float32,)
    return o.call("sgemm_grouped_outer", stream, check, M, N, K, groups,
                  o.at("offsets", offsets, (torch.int32,), groups + 1), float(alpha),
                  o.at("A", A, f32, K, M, lda), lda, o.at("B", B, f32, K, N, ldb), ldb,
                  float(beta), o.groups("C", C, f32, groups, strideC, M if groups else 0, N, ldc),
                  ldc, strideC)
