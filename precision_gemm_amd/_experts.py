"""Binding of the calls around the experts of a mixture layer and of the 8-bit
integer products (``include/i8gemm.h``, ``include/experts.h`` and the grouped
products of ``include/sgemm.h``).

The functions have the C names and argument order, without the type arguments:
those come from the tensors. Operands are GPU tensors on one device; leading
dimensions and strides count elements. Each tensor is taken from its first
element on and has to reach as far as the call will go (the rows behind one
another at the leading dimension, whatever the tensor's own shape); one that is
too short, of another type or on another device is refused with a TypeError or
ValueError before anything is launched, and so is a view with gaps between its
elements for an operand without a leading dimension (ids, row_of_slot, offsets,
weights, scales, bias). The work runs on `stream`, or else on the current stream
of the operands' device.
"""
from __future__ import annotations

import ctypes

import precision_gemm_amd as _pg

try:
    import torch
except ImportError:  # the names are there without it; the calls are not
    torch = None

EXPERT_SORT_MAX_EXPERTS = 1024
I8GEMM_MAX_K = 131071
# Kernels of the 8-bit product by number (i8gemm_kernel of the C header): S
# stream B, T take rows of any alignment, L load straight into LDS.
I8GEMM_KERNELS = ("S16x16", "S16x16_W16", "S16x32", "S32x16", "S32x32", "S32x64", "T64x64",
                  "T128x128", "L32x64", "L64x64_R4", "L64x64", "L64x128", "L128x128", "L128x256",
                  "L256x256")
# The same of the grouped fp32 products (sgemm_grouped_kernel and
# sgemm_grouped_outer_kernel): S stream, T go through LDS.
GROUPED_KERNELS = ("S16x16", "S32x16", "S16x64", "S32x64", "T64x64", "T64x64_ANY", "T64x64_V1",
                   "T128x128")
GROUPED_OUTER_KERNELS = ("S16x16", "S32x32", "T64x64", "T64x64_ANY", "T64x64_V1", "T128x128",
                         "T128x128_ANY")

if torch is not None:
    _FLOATS = (torch.float32, torch.float16, torch.bfloat16)
    _INT8, _F32, _I32 = (torch.int8,), (torch.float32,), (torch.int32,)
    _IDS = (torch.int32, torch.int64)
    _ANY = _FLOATS + _INT8
    _TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int8: 3}
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
_lib = None  # the loaded library, set by declare()


def declare(lib):
    """Argument types of the library's calls."""
    global _lib
    i, f, p, ll, sz = (ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_longlong,
                       ctypes.c_size_t)
    lib.i8_quantize_rows.argtypes = [i, i, p, i, i, p, i, p, p]
    lib.i8gemm.argtypes = [i, i, i, p, i, p, p, i, p, p, p, i, i, p]
    lib.i8gemm_grouped.argtypes = [i, i, i, i, p, p, i, p, p, i, ll, p, p, p, i, i, p]
    lib.i8gemm_select_kernel.argtypes = [i, i, i, i, i, i]
    lib.sgemm_grouped_select_kernel.argtypes = [i, i, i, i, i, i]
    lib.sgemm_grouped_outer_select_kernel.argtypes = [i, i, i, i, i]
    lib.expert_sort.argtypes = [i, i, i, p, i, p, p, p, sz, p]
    lib.expert_sort_workspace_size.argtypes = [i, i, i]
    lib.expert_gather.argtypes = [i, i, i, p, i, i, p, p, i, p]
    lib.expert_combine.argtypes = [i, i, i, p, i, i, p, p, p, i, p]
    lib.expert_combine_grad.argtypes = [i, i, i, p, i, i, p, i, p, p, p, i, p, p]
    lib.sgemm_grouped.argtypes = [i, i, i, i, i, p, f, p, i, p, i, ll, f, p, i, p]
    lib.sgemm_grouped_outer.argtypes = [i, i, i, i, p, f, p, i, p, i, f, p, i, ll, p]
    for name in ("i8_quantize_rows", "i8gemm", "i8gemm_grouped", "expert_sort", "expert_gather",
                 "expert_combine", "expert_combine_grad", "sgemm_grouped", "sgemm_grouped_outer",
                 "i8gemm_select_kernel", "sgemm_grouped_select_kernel",
                 "sgemm_grouped_outer_select_kernel"):
        getattr(lib, name).restype = i
    lib.expert_sort_workspace_size.restype = sz
    _lib = lib


_INT_MAX = 2**31 - 1  # sizes and leading dimensions are C ints


def _in_int(**sizes):
    """Refuses what would reach the library as another number. (Numbers that are
    only negative are the library's to refuse.)"""
    for name, n in sizes.items():
        if not -_INT_MAX <= n <= _INT_MAX:
            raise ValueError(f"{name} is {n}: sizes are below 2**31 and not negative")


def _span(rows, cols, ld):
    """Elements from the first to the last of `rows` rows, `ld` apart."""
    if 0 < rows <= _INT_MAX and 0 < cols <= ld <= _INT_MAX:
        return (rows - 1) * ld + cols
    _in_int(rows=rows, columns=cols, ld=ld)
    return (rows - 1) * ld + cols if rows > 0 and cols > 0 else 0


def _spans(groups, stride, rows, cols, ld):
    """The same for `groups` matrices, `stride` apart."""
    if groups < 0 or stride < 0:
        _in_int(groups=groups, stride=min(stride, 0))
    n = _span(rows, cols, ld)
    return (groups - 1) * stride + n if groups > 0 and n > 0 else 0


def _first(name, t):
    """The device of a call's operands, from one of them, with the library loaded."""
    if torch is None:
        raise ImportError("the expert and 8-bit calls take torch tensors, and torch is missing")
    if _lib is None:
        _pg._load()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor")
    return t.get_device()


def _at(name, t, dtypes, device, need, packed=False):
    """Address of an operand that the call takes `need` elements of; packed: one
    behind the other, as there is no leading dimension to say otherwise."""
    try:
        if t.get_device() == device and t.dtype in dtypes and need <= t.numel() and \
                t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    # not the plain case: a view, or a mistake
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the call's other operands on cuda:{device}")
    have = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
    if need > have:
        raise ValueError(f"{name} holds {have} elements from its first one on, "
                         f"the call needs {need}")
    if packed and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, got shape {tuple(t.shape)} with strides "
                         f"{t.stride()}")
    return t.data_ptr()


def _call(fn, device, stream, check, *args):
    if stream is None:
        stream = _raw_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if torch._C._cuda_getDevice() == device:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    return status if status == 0 else _pg._check(status, check)


def i8_quantize_rows(M, K, X, ldx, Q, ldq, scale, stream=None, check=True) -> int:
    """C ABI ``i8_quantize_rows``: rows of X (fp32, fp16 or bf16) to 8-bit
    integers Q with one fp32 scale a row."""
    d = _first("X", X)
    return _call(_lib.i8_quantize_rows, d, stream, check, M, K,
                 _at("X", X, _FLOATS, d, _span(M, K, ldx)), _TYPES[X.dtype], ldx,
                 _at("Q", Q, _INT8, d, _span(M, K, ldq)), ldq,
                 _at("scale", scale, _F32, d, M, True))


def i8gemm(M, N, K, A, lda, scaleA, B, ldb, scaleB, bias, C, ldc, stream=None, check=True) -> int:
    """C ABI ``i8gemm``: C = (A B^T) * scaleA[m] * scaleB[n] + bias[n], A (M x
    K) and B (N x K) int8, bias fp32 or None, C fp32, fp16 or bf16."""
    d = _first("A", A)
    return _call(_lib.i8gemm, d, stream, check, M, N, K,
                 _at("A", A, _INT8, d, _span(M, K, lda)), lda,
                 _at("scaleA", scaleA, _F32, d, M, True),
                 _at("B", B, _INT8, d, _span(N, K, ldb)), ldb,
                 _at("scaleB", scaleB, _F32, d, N, True),
                 None if bias is None else _at("bias", bias, _F32, d, N, True),
                 _at("C", C, _FLOATS, d, _span(M, N, ldc)), _TYPES[C.dtype], ldc)


def i8gemm_grouped(M, N, K, groups, offsets, A, lda, scaleA, B, ldb, strideB, scaleB, bias, C,
                   ldc, stream=None, check=True) -> int:
    """C ABI ``i8gemm_grouped``: i8gemm over rows sorted by group; `offsets`
    holds groups + 1 int32, scaleB and bias groups x N."""
    d = _first("offsets", offsets)
    return _call(_lib.i8gemm_grouped, d, stream, check, M, N, K, groups,
                 _at("offsets", offsets, _I32, d, groups + 1, True),
                 _at("A", A, _INT8, d, _span(M, K, lda)), lda,
                 _at("scaleA", scaleA, _F32, d, M, True),
                 _at("B", B, _INT8, d, _spans(groups, strideB, N, K, ldb)), ldb, strideB,
                 _at("scaleB", scaleB, _F32, d, groups * N, True),
                 None if bias is None else _at("bias", bias, _F32, d, groups * N, True),
                 _at("C", C, _FLOATS, d, _span(M, N, ldc)), _TYPES[C.dtype], ldc)


def i8gemm_select_kernel(M, N, K, groups, aligned, num_cus) -> int:
    """C ABI ``i8gemm_select_kernel`` (host-side dispatch decision): an index of
    I8GEMM_KERNELS, or a negative status."""
    if _lib is None:
        _pg._load()
    return _lib.i8gemm_select_kernel(M, N, K, groups, int(bool(aligned)), num_cus)


def expert_sort_workspace_size(tokens, topk, experts) -> int:
    """C ABI ``expert_sort_workspace_size`` (bytes)."""
    return int(_pg._load().expert_sort_workspace_size(tokens, topk, experts))


def expert_sort(tokens, topk, experts, ids, offsets, row_of_slot, workspace, stream=None,
                check=True) -> int:
    """C ABI ``expert_sort``: ids (int32 or int64, contiguous) to offsets and
    row_of_slot (int32); workspace: a GPU tensor of any type, or None where
    expert_sort_workspace_size() is 0."""
    d = _first("ids", ids)
    if experts < 0:
        _in_int(experts=experts)
    slots = tokens * topk
    if slots < 0:
        _in_int(tokens=tokens, topk=topk)
    p_ids = _at("ids", ids, _IDS, d, slots, True)
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws = _at("workspace", workspace, (getattr(workspace, "dtype", None),), d, 0, True)
        ws_bytes = workspace.numel() * workspace.element_size()
    return _call(_lib.expert_sort, d, stream, check, tokens, topk, experts, p_ids,
                 ids.element_size(), _at("offsets", offsets, _I32, d, experts + 1, True),
                 _at("row_of_slot", row_of_slot, _I32, d, slots, True), ws, ws_bytes)


def expert_gather(tokens, topk, cols, X, ldx, row_of_slot, Y, ldy, stream=None, check=True) -> int:
    """C ABI ``expert_gather``: Y[row_of_slot[t, j]] = X[t]; X and Y of one
    type, fp32, fp16, bf16 or int8."""
    d = _first("X", X)
    slots = tokens * topk
    if slots < 0:
        _in_int(tokens=tokens, topk=topk)
    return _call(_lib.expert_gather, d, stream, check, tokens, topk, cols,
                 _at("X", X, _ANY, d, _span(tokens, cols, ldx)), _TYPES[X.dtype], ldx,
                 _at("row_of_slot", row_of_slot, _I32, d, slots, True),
                 _at("Y", Y, (X.dtype,), d, _span(slots, cols, ldy)), ldy)


def expert_combine(tokens, topk, cols, Y, ldy, row_of_slot, weights, out, ldo, stream=None,
                   check=True) -> int:
    """C ABI ``expert_combine``: out[t] = sum_j weights[t, j] Y[row_of_slot[t,
    j]]; weights fp32, or None for 1 (the gradient of expert_gather)."""
    d = _first("Y", Y)
    slots = tokens * topk
    if slots < 0:
        _in_int(tokens=tokens, topk=topk)
    return _call(_lib.expert_combine, d, stream, check, tokens, topk, cols,
                 _at("Y", Y, _FLOATS, d, _span(slots, cols, ldy)), _TYPES[Y.dtype], ldy,
                 _at("row_of_slot", row_of_slot, _I32, d, slots, True),
                 None if weights is None else _at("weights", weights, _F32, d, slots, True),
                 _at("out", out, (Y.dtype,), d, _span(tokens, cols, ldo)), ldo)


def expert_combine_grad(tokens, topk, cols, dout, ldo, Y, ldy, row_of_slot, weights, dY, lddy,
                        dweights, stream=None, check=True) -> int:
    """C ABI ``expert_combine_grad``: dY and dweights (fp32, or None: then Y
    may be None too) from dout."""
    d = _first("dout", dout)
    slots = tokens * topk
    if slots < 0:
        _in_int(tokens=tokens, topk=topk)
    return _call(_lib.expert_combine_grad, d, stream, check, tokens, topk, cols,
                 _at("dout", dout, _FLOATS, d, _span(tokens, cols, ldo)), _TYPES[dout.dtype], ldo,
                 None if Y is None else _at("Y", Y, (dout.dtype,), d, _span(slots, cols, ldy)),
                 ldy, _at("row_of_slot", row_of_slot, _I32, d, slots, True),
                 None if weights is None else _at("weights", weights, _F32, d, slots, True),
                 _at("dY", dY, (dout.dtype,), d, _span(slots, cols, lddy)), lddy,
                 None if dweights is None else _at("dweights", dweights, _F32, d, slots, True))


def sgemm_grouped(transB, M, N, K, groups, offsets, alpha, A, lda, B, ldb, strideB, beta, C, ldc,
                  stream=None, check=True) -> int:
    """C ABI ``sgemm_grouped``: C[m] = alpha A[m] op(B_g) + beta C[m] for the
    rows offsets[g] <= m < offsets[g + 1] of every group."""
    d = _first("offsets", offsets)
    rows, cols = (N, K) if transB else (K, N)
    return _call(_lib.sgemm_grouped, d, stream, check, int(transB), M, N, K, groups,
                 _at("offsets", offsets, _I32, d, groups + 1, True), float(alpha),
                 _at("A", A, _F32, d, _span(M, K, lda)), lda,
                 _at("B", B, _F32, d, _spans(groups, strideB, rows, cols, ldb)), ldb, strideB,
                 float(beta), _at("C", C, _F32, d, _span(M, N, ldc)), ldc)


def sgemm_grouped_outer(M, N, K, groups, offsets, alpha, A, lda, B, ldb, beta, C, ldc, strideC,
                        stream=None, check=True) -> int:
    """C ABI ``sgemm_grouped_outer``: C_g = alpha A_g^T B_g + beta C_g over the
    rows offsets[g] <= k < offsets[g + 1] of A (K x M) and B (K x N)."""
    d = _first("offsets", offsets)
    return _call(_lib.sgemm_grouped_outer, d, stream, check, M, N, K, groups,
                 _at("offsets", offsets, _I32, d, groups + 1, True), float(alpha),
                 _at("A", A, _F32, d, _span(K, M, lda)), lda,
                 _at("B", B, _F32, d, _span(K, N, ldb)), ldb, float(beta),
                 _at("C", C, _F32, d, _spans(groups, strideC, M, N, ldc)), ldc, strideC)


def sgemm_grouped_select_kernel(transB, M, N, groups, vec4_ok, num_cus) -> int:
    """C ABI ``sgemm_grouped_select_kernel`` (host-side dispatch decision): an
    index of GROUPED_KERNELS, or a negative status."""
    if _lib is None:
        _pg._load()
    return _lib.sgemm_grouped_select_kernel(int(transB), M, N, groups, int(bool(vec4_ok)), num_cus)


def sgemm_grouped_outer_select_kernel(M, N, groups, vec4_ok, num_cus) -> int:
    """C ABI ``sgemm_grouped_outer_select_kernel``, as above: an index of
    GROUPED_OUTER_KERNELS."""
    if _lib is None:
        _pg._load()
    return _lib.sgemm_grouped_outer_select_kernel(M, N, groups, int(bool(vec4_ok)), num_cus)
