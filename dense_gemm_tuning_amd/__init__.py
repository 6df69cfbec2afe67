"""Python binding of the gfx950 dense GEMM library (``libdgt_gemm.so``).

Argument marshalling only: every function forwards to the C entry point of
the same name in ``include/dgt_gemm.h``; all arithmetic happens in the HIP
kernels behind it.  Pointers are device addresses passed as Python ints,
``stream`` is a ``hipStream_t`` as an int (0 = null stream).  Each function
returns the library's status code (0 = GEMM_OK); ``check`` turns a non-zero
status into an exception.

``gemm(A, B, C, alpha, beta, variant, trans_a=..., trans_b=...)`` is a
convenience for torch tensors on the GPU: it reads shapes, leading dimensions
(``stride(0)``) and ``torch.cuda.current_stream()`` and calls ``gemm_f32`` /
``gemm_bf16`` / ``gemm_f16`` (or ``gemm_ex`` for transposed or explicit-rung
calls).  Torch is used for memory and streams only.

There is no fallback: if the library has not been built, every call raises.
"""

from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib",
                        "libdgt_gemm.so")

GEMM_OK = 0
GEMM_ERR_DIM = -1
GEMM_ERR_LD = -2
GEMM_ERR_NULL = -3
GEMM_ERR_OVERLAP = -4
GEMM_ERR_VARIANT = -5
GEMM_ERR_LAUNCH = -6
GEMM_ERR_ARG = -7
GEMM_ERR_WORKSPACE = -8
GEMM_ERR_SCRATCH = -9
GEMM_ERR_ALIGN = -10
NOALLOC_SCRATCH_BYTES = 64 << 20  # DGT_GEMM_NOALLOC_SCRATCH_BYTES
MX4_MAX_PITCH = 1 << 24  # DGT_GEMM_MX4_MAX_PITCH

VARIANT_AUTO = 0
VARIANT_NAIVE = 1
VARIANT_LDS = 2
VARIANT_MFMA = 3
VARIANT_SKINNY = 4
VARIANT_MFMA_T256 = 5
VARIANT_MFMA_T128 = 6
VARIANT_MFMA_REGS = 7
VARIANTS = {"auto": VARIANT_AUTO, "naive": VARIANT_NAIVE, "lds": VARIANT_LDS,
            "mfma": VARIANT_MFMA, "skinny": VARIANT_SKINNY, "mfma256": VARIANT_MFMA_T256,
            "mfma128": VARIANT_MFMA_T128, "mfma_regs": VARIANT_MFMA_REGS}

# Every symbol the header declares (the tests check the library exports them).
EXPORTS = ("gemm_f32", "gemm_bf16", "gemm_f16", "gemm_f32_variant", "gemm_bf16_variant",
           "gemm_f16_variant", "gemm_ex", "gemm_strided_batched", "gemm_splitk",
           "gemm_splitk_noalloc", "gemm_splitk_slices", "gemm_splitk_workspace_size",
           "gemm_streamk", "gemm_streamk_workspace_size", "gemm_select_variant",
           "gemm_status_string", "gemm_abi_version", "gemm_mx4_code_pitch",
           "gemm_mx4_scale_pitch", "gemm_mx4_quantize", "gemm_mx4_dequantize", "gemm_mx4",
           "gemm_mx4_a16", "gemm_orthogonalize", "gemm_orthogonalize_workspace_size")

DTYPE_F32 = 0
DTYPE_BF16 = 1
DTYPE_F16 = 2

_lib = None


class GemmError(RuntimeError):
    def __init__(self, status: int):
        super().__init__(gemm_status_string(status))
        self.status = status


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"HIP GEMM library not built ({LIB_PATH} missing); run "
                "`python -m dense_gemm_tuning_amd.build` or "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(LIB_PATH)
        i, f, p = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
        core = [i, i, i, f, p, i, p, i, f, p, i, p]
        for name in ("gemm_f32", "gemm_bf16", "gemm_f16"):
            fn = getattr(lib, name)
            fn.restype = i
            fn.argtypes = core
        for name in ("gemm_f32_variant", "gemm_bf16_variant", "gemm_f16_variant"):
            fn = getattr(lib, name)
            fn.restype = i
            fn.argtypes = [i, *core]
        lib.gemm_ex.restype = i
        lib.gemm_ex.argtypes = [i, i, i, i, *core]
        i64 = ctypes.c_int64
        lib.gemm_splitk.restype = i
        lib.gemm_splitk.argtypes = [i, i, i, *core[:11], i, p, i64, p]
        lib.gemm_splitk_noalloc.restype = i
        lib.gemm_splitk_noalloc.argtypes = [i, i, i, *core[:11], i, p]
        lib.gemm_streamk.restype = i
        lib.gemm_streamk.argtypes = [i, i, i, *core[:11], p, i64, p]
        lib.gemm_streamk_workspace_size.restype = i64
        lib.gemm_streamk_workspace_size.argtypes = [i, i, i, i]
        lib.gemm_splitk_slices.restype = i
        lib.gemm_splitk_slices.argtypes = [i, i, i, i, i]
        lib.gemm_splitk_workspace_size.restype = i64
        lib.gemm_splitk_workspace_size.argtypes = [i, i, i, i, i]
        lib.gemm_strided_batched.restype = i
        lib.gemm_strided_batched.argtypes = [i, i, i, i, i, i, i, f, p, i, i64, p, i, i64, f,
                                             p, i, i64, p, i64, i, p]
        lib.gemm_select_variant.restype = i
        lib.gemm_select_variant.argtypes = [i] * 9
        for name in ("gemm_mx4_code_pitch", "gemm_mx4_scale_pitch"):
            fn = getattr(lib, name)
            fn.restype = i64
            fn.argtypes = [i]
        lib.gemm_mx4_quantize.restype = i
        lib.gemm_mx4_quantize.argtypes = [i, i, i, i, p, i, p, i, p, i, p]
        lib.gemm_mx4_dequantize.restype = i
        lib.gemm_mx4_dequantize.argtypes = [i, i, i, p, i, p, i, p, i, p]
        lib.gemm_mx4.restype = i
        lib.gemm_mx4.argtypes = [i, i, i, f, p, i, p, i, p, i, p, i, f, p, i, p, p]
        lib.gemm_mx4_a16.restype = i
        lib.gemm_mx4_a16.argtypes = [i, i, i, i, f, p, i, p, i, p, i, f, p, i, p, p]
        lib.gemm_orthogonalize.restype = i
        lib.gemm_orthogonalize.argtypes = [i, i, i, p, i, i64, p, i, i64, i, i, f, f, f, f, p, i64,
                                           p]
        lib.gemm_orthogonalize_workspace_size.restype = i64
        lib.gemm_orthogonalize_workspace_size.argtypes = [i, i, i]
        lib.gemm_status_string.restype = ctypes.c_char_p
        lib.gemm_status_string.argtypes = [i]
        lib.gemm_abi_version.restype = i
        lib.gemm_abi_version.argtypes = []
        _lib = lib
    return _lib


def library() -> ctypes.CDLL:
    """The loaded ctypes handle (raises if the library is not built)."""
    return _load()


def gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return _load().gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_bf16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return _load().gemm_bf16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_f16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return _load().gemm_f16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_f32_variant(variant, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                     stream=0) -> int:
    return _load().gemm_f32_variant(variant, M, N, K, alpha, A, lda, B, ldb, beta,
                                    C, ldc, stream)


def gemm_bf16_variant(variant, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                      stream=0) -> int:
    return _load().gemm_bf16_variant(variant, M, N, K, alpha, A, lda, B, ldb, beta,
                                     C, ldc, stream)


def gemm_f16_variant(variant, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                     stream=0) -> int:
    return _load().gemm_f16_variant(variant, M, N, K, alpha, A, lda, B, ldb, beta,
                                    C, ldc, stream)


def gemm_ex(dtype, trans_a, trans_b, variant, M, N, K, alpha, A, lda, B, ldb, beta, C,
            ldc, stream=0) -> int:
    return _load().gemm_ex(int(dtype), int(trans_a), int(trans_b), int(variant), M, N, K,
                           alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_strided_batched(dtype, trans_a, trans_b, variant, M, N, K, alpha, A, lda, stride_a,
                         B, ldb, stride_b, beta, C, ldc, stride_c, bias, stride_bias, batch,
                         stream=0) -> int:
    return _load().gemm_strided_batched(int(dtype), int(trans_a), int(trans_b), int(variant),
                                        M, N, K, alpha, A, lda, stride_a, B, ldb, stride_b,
                                        beta, C, ldc, stride_c, bias, stride_bias, batch,
                                        stream)


def gemm_splitk(dtype, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, splits,
                workspace, workspace_bytes, stream=0) -> int:
    return _load().gemm_splitk(int(dtype), int(trans_a), int(trans_b), M, N, K, alpha, A, lda,
                               B, ldb, beta, C, ldc, int(splits), workspace,
                               int(workspace_bytes), stream)


def gemm_splitk_noalloc(dtype, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                        splits, stream=0) -> int:
    return _load().gemm_splitk_noalloc(int(dtype), int(trans_a), int(trans_b), M, N, K, alpha, A,
                                       lda, B, ldb, beta, C, ldc, int(splits), stream)


def gemm_streamk(dtype, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                 workspace, workspace_bytes, stream=0) -> int:
    return _load().gemm_streamk(int(dtype), int(trans_a), int(trans_b), M, N, K, alpha, A, lda,
                                B, ldb, beta, C, ldc, workspace, int(workspace_bytes), stream)


def gemm_streamk_workspace_size(dtype, M, N, K) -> int:
    return _load().gemm_streamk_workspace_size(int(dtype), M, N, K)


def gemm_splitk_slices(dtype, M, N, K, splits) -> int:
    return _load().gemm_splitk_slices(int(dtype), M, N, K, int(splits))


def gemm_splitk_workspace_size(dtype, M, N, K, splits) -> int:
    return _load().gemm_splitk_workspace_size(int(dtype), M, N, K, int(splits))


def gemm_select_variant(dtype, trans_a, trans_b, M, N, K, lda, ldb, ldc) -> int:
    """dtype: DTYPE_F32, DTYPE_BF16 or DTYPE_F16; trans_a, trans_b: 0 or 1."""
    return _load().gemm_select_variant(int(dtype), int(trans_a), int(trans_b), M, N, K,
                                       lda, ldb, ldc)


def gemm_mx4_code_pitch(K) -> int:
    return _load().gemm_mx4_code_pitch(K)


def gemm_mx4_scale_pitch(K) -> int:
    return _load().gemm_mx4_scale_pitch(K)


def gemm_mx4_quantize(dtype, trans, M, K, X, ldx, Q, ldq, S, lds, stream=0) -> int:
    return _load().gemm_mx4_quantize(int(dtype), int(trans), M, K, X, ldx, Q, ldq, S, lds, stream)


def gemm_mx4_dequantize(dtype, M, K, Q, ldq, S, lds, Y, ldy, stream=0) -> int:
    return _load().gemm_mx4_dequantize(int(dtype), M, K, Q, ldq, S, lds, Y, ldy, stream)


def gemm_mx4(M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, beta, C, ldc, bias=0,
             stream=0) -> int:
    return _load().gemm_mx4(M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, beta, C, ldc,
                            bias, stream)


def gemm_mx4_a16(dtype, M, N, K, alpha, A, lda, B, ldb, SB, ldsb, beta, C, ldc, bias=0,
                 stream=0) -> int:
    return _load().gemm_mx4_a16(int(dtype), M, N, K, alpha, A, lda, B, ldb, SB, ldsb, beta, C, ldc,
                                bias, stream)


def gemm_orthogonalize(dtype, M, N, G, ldg, stride_g, O, ldo, stride_o, batch, steps, a, b, c, eps,
                       workspace, workspace_bytes, stream=0) -> int:
    return _load().gemm_orthogonalize(int(dtype), M, N, G, ldg, stride_g, O, ldo, stride_o, batch,
                                      int(steps), a, b, c, eps, workspace, int(workspace_bytes),
                                      stream)


def gemm_orthogonalize_workspace_size(M, N, batch) -> int:
    return _load().gemm_orthogonalize_workspace_size(M, N, batch)


def gemm_status_string(status: int) -> str:
    return _load().gemm_status_string(status).decode()


def gemm_abi_version() -> int:
    return _load().gemm_abi_version()


def check(status: int) -> None:
    if status != GEMM_OK:
        raise GemmError(status)


def _ld(t) -> int:
    """Row pitch of a 2-D tensor; for an empty or single-row operand the pitch
    is never used (torch may report 0), so report a legal one."""
    rows, cols = t.shape
    if rows <= 1 or t.numel() == 0:
        return max(t.stride(0), cols, 1)
    return t.stride(0)


def _check_layout(named, dims=(2,)):
    """Structure checks of the torch-facing calls, run before anything reaches
    the library: each (name, tensor) has a dimension count in ``dims`` and,
    unless it is empty or has a single column, unit stride along its last axis
    (row-major rows).  A column-strided view would otherwise pass the leading-dimension check and
    read the wrong elements."""
    for name, t in named:
        if t.dim() not in dims:
            raise ValueError(f"{name} must have {' or '.join(map(str, dims))} dimensions, "
                             f"got {t.dim()}")
        if t.numel() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must be row-major with unit column stride")


def _check_device(named, device):
    """Every non-empty (name, tensor) must live on the GPU ``device``: a host
    tensor would hand a host pointer to a kernel."""
    for name, t in named:
        if t.numel() > 0 and (not t.is_cuda or t.device != device):
            raise ValueError(f"{name} must be a GPU tensor on {device}, got {t.device}")


def _dtype_code(A, B, C):
    import torch
    if A.dtype != B.dtype or A.dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise TypeError("A and B must both be float32, both bfloat16 or both float16")
    if C.dtype != torch.float32:
        raise TypeError("C must be float32")
    return {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16,
            torch.float16: DTYPE_F16}[A.dtype]


def _stream_handle(stream):
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return stream


def gemm(A, B, C, alpha: float = 1.0, beta: float = 0.0, variant=VARIANT_AUTO,
         stream=None, trans_a: bool = False, trans_b: bool = False) -> int:
    """C <- alpha*op(A)*op(B) + beta*C on torch tensors (row-major, unit column
    stride).  op(X) is X, or X transposed when trans_x: then A is the stored
    K x M tensor, B the stored N x K tensor.

    A and B are float32, bfloat16 or float16 (16-bit bits are passed as-is),
    C float32.  ``variant`` is a ladder rung (enum gemm_variant) or its name
    in VARIANTS: "auto", "naive", "lds", "mfma", "skinny", "mfma256" /
    "mfma128" for the DMA kernels with a fixed workgroup tile, or
    "mfma_regs" for the register-staged MFMA kernel.
    Returns the status code; the work is queued on ``stream`` (default: torch's
    current stream) and not waited for.
    """
    if isinstance(variant, str):
        variant = VARIANTS[variant]
    dtype = _dtype_code(A, B, C)
    named = (("A", A), ("B", B), ("C", C))
    _check_layout(named)
    M, K = A.shape[::-1] if trans_a else A.shape
    K2, N = B.shape[::-1] if trans_b else B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, "
                         f"C {tuple(C.shape)}")
    _check_device(named, C.device)
    stream = _stream_handle(stream)
    lda, ldb, ldc = _ld(A), _ld(B), _ld(C)
    args = (M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(), ldb,
            float(beta), C.data_ptr(), ldc, stream)
    if trans_a or trans_b:
        return gemm_ex(dtype, trans_a, trans_b, variant, *args)
    auto_fn, var_fn = {DTYPE_F32: (gemm_f32, gemm_f32_variant),
                       DTYPE_BF16: (gemm_bf16, gemm_bf16_variant),
                       DTYPE_F16: (gemm_f16, gemm_f16_variant)}[dtype]
    if variant == VARIANT_AUTO:
        return auto_fn(*args)
    return var_fn(variant, *args)


def gemm_batched(A, B, C, alpha: float = 1.0, beta: float = 0.0, bias=None,
                 variant=VARIANT_AUTO, stream=None, trans_a: bool = False,
                 trans_b: bool = False) -> int:
    """C[z] <- alpha*op(A[z])*op(B[z]) + beta*C[z] + bias[z] on torch tensors.

    A, B and C are 3-D (batch first; a batch stride of 0, e.g. from
    ``expand``, shares one matrix) or 2-D for an operand shared by every
    problem; each matrix is row-major with unit column stride.  bias is None,
    a 1-D tensor of N floats or a [1, N] tensor (shared by every problem), or
    a [batch, N] tensor (one row per problem).  Every tensor must be on C's
    GPU.  Returns the status code of gemm_strided_batched.
    """
    import torch

    if isinstance(variant, str):
        variant = VARIANTS[variant]
    dtype = _dtype_code(A, B, C)
    if C.dim() != 3:
        raise TypeError("C must be a 3-D float32 tensor")
    _check_layout((("A", A), ("B", B)), dims=(2, 3))
    _check_layout((("C", C),), dims=(3,))
    batch = C.shape[0]

    def mat(t, name):
        if t.dim() == 2:
            return t, 0
        if t.shape[0] not in (batch, 1):
            raise ValueError(f"{name} must be 2-D or [batch, rows, cols]")
        return t[0] if t.shape[0] == 1 else t, (0 if t.shape[0] == 1 else t.stride(0))

    def pitch(t):
        return _ld(t if t.dim() == 2 else t[0])

    A2, sa = mat(A, "A")
    B2, sb = mat(B, "B")
    a_rows, a_cols = A2.shape[-2:]
    b_rows, b_cols = B2.shape[-2:]
    M, K = (a_cols, a_rows) if trans_a else (a_rows, a_cols)
    K2, N = (b_cols, b_rows) if trans_b else (b_rows, b_cols)
    if K2 != K or tuple(C.shape[1:]) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, "
                         f"C {tuple(C.shape)}")
    bias_ptr, sbias = 0, 0
    if bias is not None:
        if bias.dtype != torch.float32 or bias.dim() not in (1, 2) or bias.shape[-1] != N:
            raise ValueError("bias must be float32 [N], [1, N] or [batch, N]")
        if bias.dim() == 2 and bias.shape[0] not in (1, batch):
            raise ValueError(f"a 2-D bias must have 1 or batch = {batch} rows, "
                             f"got {bias.shape[0]}")
        _check_layout((("bias", bias),), dims=(1, 2))
        bias_ptr = bias.data_ptr()
        # one row shared by every problem reads with stride 0; otherwise row z
        # starts bias.stride(0) floats after row z - 1
        sbias = bias.stride(0) if bias.dim() == 2 and bias.shape[0] > 1 else 0
    _check_device((("A", A), ("B", B), ("C", C)) + ((("bias", bias),) if bias is not None
                                                     else ()), C.device)
    return gemm_strided_batched(dtype, trans_a, trans_b, variant, M, N, K, float(alpha),
                                A2.data_ptr(), pitch(A2), sa, B2.data_ptr(), pitch(B2), sb,
                                float(beta), C.data_ptr(), pitch(C), C.stride(0),
                                bias_ptr, sbias, batch, _stream_handle(stream))


def gemm_split(A, B, C, alpha: float = 1.0, beta: float = 0.0, splits: int = 0,
               workspace=None, stream=None, trans_a: bool = False,
               trans_b: bool = False) -> int:
    """Split-K form of ``gemm`` on torch tensors (gemm_splitk).  ``workspace``
    is a device tensor of at least gemm_splitk_workspace_size bytes; when None
    one is allocated here with torch (the library itself allocates nothing);
    a caller's workspace must be a contiguous GPU tensor on C's device.
    Returns the status code."""
    import torch

    dtype = _dtype_code(A, B, C)
    named = (("A", A), ("B", B), ("C", C))
    _check_layout(named)
    M, K = A.shape[::-1] if trans_a else A.shape
    K2, N = B.shape[::-1] if trans_b else B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, "
                         f"C {tuple(C.shape)}")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _check_device(named + ((("workspace", workspace),) if workspace is not None else ()),
                  C.device)
    need = gemm_splitk_workspace_size(dtype, M, N, K, splits)
    if need < 0:
        return need
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=C.device)
    ws_ptr, ws_bytes = 0, 0
    if workspace is not None:
        ws_ptr = workspace.data_ptr() if workspace.numel() > 0 else 0
        ws_bytes = workspace.numel() * workspace.element_size()
    return gemm_splitk(dtype, trans_a, trans_b, M, N, K, float(alpha), A.data_ptr(), _ld(A),
                       B.data_ptr(), _ld(B), float(beta), C.data_ptr(), _ld(C), splits,
                       ws_ptr, ws_bytes, _stream_handle(stream))


def gemm_stream(A, B, C, alpha: float = 1.0, beta: float = 0.0, workspace=None, stream=None,
                trans_a: bool = False, trans_b: bool = False) -> int:
    """Stream-K form of ``gemm`` on torch tensors (gemm_streamk).  ``workspace``
    is a device tensor of at least gemm_streamk_workspace_size bytes; when
    None one is allocated here with torch (the library itself allocates
    nothing); a caller's workspace must be a contiguous GPU tensor on C's
    device.  Shapes stream-K does not cover run as ``gemm``.  Returns the
    status code."""
    import torch

    dtype = _dtype_code(A, B, C)
    named = (("A", A), ("B", B), ("C", C))
    _check_layout(named)
    M, K = A.shape[::-1] if trans_a else A.shape
    K2, N = B.shape[::-1] if trans_b else B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, "
                         f"C {tuple(C.shape)}")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _check_device(named + ((("workspace", workspace),) if workspace is not None else ()),
                  C.device)
    need = gemm_streamk_workspace_size(dtype, M, N, K)
    if need < 0:
        return need
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=C.device)
    ws_ptr, ws_bytes = 0, 0
    if workspace is not None:
        ws_ptr = workspace.data_ptr() if workspace.numel() > 0 else 0
        ws_bytes = workspace.numel() * workspace.element_size()
    return gemm_streamk(dtype, trans_a, trans_b, M, N, K, float(alpha), A.data_ptr(), _ld(A),
                        B.data_ptr(), _ld(B), float(beta), C.data_ptr(), _ld(C), ws_ptr,
                        ws_bytes, _stream_handle(stream))


# The calls below are made for decode steps of a few microseconds, so their
# checks read every tensor attribute once and ask the library nothing.

_INT_MAX = 2 ** 31 - 1  # the C entry points take sizes and pitches as int
_torch = None  # the module, from the first torch-facing call below on
_FLOAT_CODES = {}  # torch dtype -> enum gemm_dtype


def _use_torch():
    """torch, without an import statement's cost in every call."""
    global _torch
    if _torch is None:
        import torch
        _FLOAT_CODES.update({torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16,
                             torch.float16: DTYPE_F16})
        _torch = torch
    return _torch


def _float_code(t, name):
    if _torch is None:
        _use_torch()
    code = _FLOAT_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return code


def _matrix(t, name):
    """(rows, columns, row pitch) of a row-major 2-D tensor; for an empty or
    single-row one, whose pitch is never used, a legal pitch."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {len(shape)}")
    rows, cols = shape
    pitch, step = t.stride()
    if step != 1 and cols > 1 and rows > 0:
        raise ValueError(f"{name} must be row-major with unit column stride")
    if rows <= 1 or cols == 0:
        pitch = max(cols, 1)
    if rows > _INT_MAX or cols > _INT_MAX or pitch > _INT_MAX:
        raise ValueError(f"{name}: sizes and row pitch must be below 2^31, got {rows} x {cols}, "
                         f"pitch {pitch}")
    return rows, cols, pitch


def _bytes(t, name, rows):
    """(columns, pitch) of MX4 codes or scales of ``rows`` rows."""
    if t.dtype is not (_torch or _use_torch()).uint8:
        raise TypeError(f"{name} must be uint8, got {t.dtype}")
    have, cols, pitch = _matrix(t, name)
    if have != rows:
        raise ValueError(f"{name} must have {rows} rows, got {have}")
    if rows <= 1 or cols == 0:
        pitch = max(16, (cols + 15) // 16 * 16)
    return cols, pitch


def _fits(K, cols_q, cols_s, name):
    """Rows of ``cols_q`` code and ``cols_s`` scale bytes hold K elements.  Wider
    ones are padded storage, unless both widths are what mx4_empty makes for
    more elements: then the operand is one of another K (its blocks past K would go
    unread, or unwritten)."""
    need_q, need_s = (K + 31) // 32 * 16, (K + 511) // 512 * 16  # gemm_mx4_*_pitch
    if cols_q < need_q or cols_s < need_s:
        raise ValueError(f"{name}: {K} elements need rows of {need_q} code and {need_s} scale "
                         f"bytes, got {cols_q} and {cols_s}")
    if cols_q != need_q and cols_q % 16 == 0 and cols_s == (cols_q + 255) // 256 * 16:
        raise ValueError(f"{name}: an operand of {2 * cols_q - 31} to {2 * cols_q} elements a row, "
                         f"not of {K} (of padded storage pass [:, :{need_q}] of the codes)")


def _on_device(index, named):
    """Every non-empty (name, tensor) on GPU ``index`` (-1: the host)."""
    for name, t in named:
        if t.get_device() == index >= 0:
            continue
        if t.numel() > 0:
            at = "" if index < 0 else f" on cuda:{index}"
            raise ValueError(f"{name} must be a GPU tensor{at}, got {t.device}")


def _call_on(index, stream, fn, *args):
    """fn(*args, stream handle) with GPU ``index`` current and, by default, the
    stream current there (the tensors may live on another GPU than the one the
    caller has current)."""
    torch = _torch or _use_torch()
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        at = getattr(stream, "device", None)
        if at is not None and at.index != index:
            raise ValueError(f"stream is on {at}, the tensors on cuda:{index}")
        handle = getattr(stream, "cuda_stream", stream)
    if torch.cuda.current_device() == index:
        return fn(*args, handle)
    with torch.cuda.device(index):
        return fn(*args, handle)


def mx4_empty(rows: int, K: int, device="cuda"):
    """Uninitialised storage of a rows x K MX4 operand: (codes, scales), two
    uint8 tensors of the smallest row pitches."""
    import torch
    if K > _INT_MAX:
        raise ValueError(f"K must be below 2^31, got {K}")
    return (torch.empty(rows, gemm_mx4_code_pitch(K), dtype=torch.uint8, device=device),
            torch.empty(rows, gemm_mx4_scale_pitch(K), dtype=torch.uint8, device=device))


def quantize_mx4(X, Q, S, trans: bool = False, stream=None) -> int:
    """(Q, S) <- op(X) in MX4 blocks along its columns (gemm_mx4_quantize);
    op(X) is X, or X transposed when ``trans``.  X is float32, bfloat16 or
    float16, row-major; Q and S as ``mx4_empty`` makes them for op(X), or views
    of wider storage.  Blocks run along the summation index of the product the
    operand is for.  Returns the status code."""
    dtype = _float_code(X, "X")
    rows, cols, ldx = _matrix(X, "X")
    M, K = (cols, rows) if trans else (rows, cols)
    cols_q, ldq = _bytes(Q, "Q (codes)", M)
    cols_s, lds = _bytes(S, "S (scales)", M)
    _fits(K, cols_q, cols_s, "Q, S")
    index = Q.get_device()
    _on_device(index, (("X", X), ("Q", Q), ("S", S)))
    if M == 0 or K == 0:
        return GEMM_OK
    return _call_on(index, stream, _load().gemm_mx4_quantize, dtype, int(trans), M, K,
                    X.data_ptr(), ldx, Q.data_ptr(), ldq, S.data_ptr(), lds)


def dequantize_mx4(Q, S, Y, stream=None) -> int:
    """Y [rows, K] <- the values of an MX4 operand (gemm_mx4_dequantize), Y
    float32, bfloat16 or float16, row-major.  Returns the status code."""
    dtype = _float_code(Y, "Y")
    M, K, ldy = _matrix(Y, "Y")
    cols_q, ldq = _bytes(Q, "Q (codes)", M)
    cols_s, lds = _bytes(S, "S (scales)", M)
    _fits(K, cols_q, cols_s, "Q, S")
    index = Y.get_device()
    _on_device(index, (("Q", Q), ("S", S), ("Y", Y)))
    if M == 0 or K == 0:
        return GEMM_OK
    return _call_on(index, stream, _load().gemm_mx4_dequantize, dtype, M, K, Q.data_ptr(), ldq,
                    S.data_ptr(), lds, Y.data_ptr(), ldy)


def gemm_quantized(A, SA, B, SB, C, alpha: float = 1.0, beta: float = 0.0, bias=None,
                   stream=None) -> int:
    """C <- alpha*A*B^T + beta*C + bias with B an MX4 operand of N rows (codes
    B, scales SB) and A either one of M rows (codes A, scales SA: gemm_mx4) or
    a bfloat16 / float16 [M, K] tensor with SA None (gemm_mx4_a16).  C is
    float32 [M, N], row-major; bias None or float32 [N].  With 16-bit A, K is
    A's, and B and SB of the widths of another K are refused.  With MX4 A the
    summation runs over every stored element: codes past a ragged K are zeros
    (quantize_mx4 writes them so).  Returns the status code."""
    torch = _torch or _use_torch()
    if C.dtype is not torch.float32:
        raise TypeError("C must be float32")
    M, N, ldc = _matrix(C, "C")
    rows_a, cols_a, lda = _matrix(A, "A")
    cols_b, ldb = _bytes(B, "B (codes)", N)
    cols_sb, ldsb = _bytes(SB, "SB (scales)", N)
    index = C.get_device()
    if SA is None:
        if A.dtype is torch.float32 or A.dtype is torch.uint8:
            raise TypeError("A must be bfloat16 or float16, or MX4 codes with their scales SA")
        dtype = _float_code(A, "A")
        K = cols_a
        if rows_a != M:
            raise ValueError(f"shape mismatch: A {tuple(A.shape)}, C {tuple(C.shape)}")
    else:
        _, lda = _bytes(A, "A (codes)", M)
        cols_sa, ldsa = _bytes(SA, "SA (scales)", M)
        K = 2 * cols_a
        if cols_a != cols_b or cols_a % 16 != 0:
            raise ValueError("A and B must have code rows of one length, a multiple of 16 bytes, "
                             f"got {cols_a} and {cols_b}")
        _fits(K, cols_a, cols_sa, "A, SA")
    _fits(K, cols_b, cols_sb, "B, SB")
    bias_ptr = 0
    if bias is not None:
        if bias.dtype is not torch.float32 or bias.dim() != 1 or bias.shape[0] != N:
            raise ValueError("bias must be float32 [N]")
        if N > 1 and bias.stride(0) != 1:
            raise ValueError("bias must be contiguous")
        bias_ptr = bias.data_ptr()
        _on_device(index, (("bias", bias),))
    _on_device(index, (("A", A), ("B", B), ("SB", SB), ("C", C)))
    if SA is not None:
        _on_device(index, (("SA", SA),))
    if M == 0 or N == 0:
        return GEMM_OK
    if SA is None:
        return _call_on(index, stream, _load().gemm_mx4_a16, dtype, M, N, K, float(alpha),
                        A.data_ptr(), lda, B.data_ptr(), ldb, SB.data_ptr(), ldsb, float(beta),
                        C.data_ptr(), ldc,
                        bias_ptr)
    return _call_on(index, stream, _load().gemm_mx4, M, N, K, float(alpha), A.data_ptr(), lda,
                    SA.data_ptr(), ldsa, B.data_ptr(), ldb, SB.data_ptr(), ldsb, float(beta),
                    C.data_ptr(), ldc, bias_ptr)


def orthogonalize(G, O, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315),
                  eps: float = 1e-7, workspace=None, stream=None) -> int:
    """O <- G orthogonalised by ``steps`` Newton-Schulz steps
    X <- a*X + (b*S + c*S*S)*X from X = G / (|G| + eps) (gemm_orthogonalize;
    the default coefficients are the quintic's that Muon uses).  G is float32,
    bfloat16 or float16 and O bfloat16, both [M, N] or [batch, M, N] with
    row-major matrices, M at most 2^26 and N at most 2^24; O may be G.
    ``workspace`` is a contiguous GPU tensor of at least
    gemm_orthogonalize_workspace_size bytes that no other call uses at the same
    time; when None one is allocated here with torch, for the stream the work
    runs on.  Returns the status code."""
    torch = _torch or _use_torch()
    dtype = _float_code(G, "G")
    if O.dtype is not torch.bfloat16:
        raise TypeError("O must be bfloat16")
    _check_layout((("G", G), ("O", O)), dims=(2, 3))
    if G.shape != O.shape:
        raise ValueError(f"shape mismatch: G {tuple(G.shape)}, O {tuple(O.shape)}")
    named = [("G", G), ("O", O)]
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        named.append(("workspace", workspace))
    batch = G.shape[0] if G.dim() == 3 else 1
    if batch > _INT_MAX or abs(int(steps)) > _INT_MAX:
        raise ValueError(f"batch and steps must be below 2^31, got {batch} and {steps}")
    index = O.get_device()
    _on_device(index, named)
    if G.numel() == 0:
        return GEMM_OK
    M, N = G.shape[-2:]

    def mat(t):
        return (t[0], t.stride(0) if batch > 1 else 0) if t.dim() == 3 else (t, 0)

    (G2, sg), (O2, so) = mat(G), mat(O)
    (_, _, ldg), (_, _, ldo) = _matrix(G2, "G"), _matrix(O2, "O")
    need = gemm_orthogonalize_workspace_size(M, N, batch)
    if need < 0:
        return need
    if workspace is None:
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=O.device)
        else:  # in that stream's order, so that a later call cannot get it too early
            if hasattr(stream, "cuda_stream"):
                on = stream
            elif stream == 0:  # ExternalStream takes 0 for "any stream of the pool"
                on = torch.cuda.default_stream(O.device)
            else:
                on = torch.cuda.ExternalStream(stream, device=O.device)
            with torch.cuda.stream(on):
                workspace = torch.empty(need, dtype=torch.uint8, device=O.device)
    a, b, c = (float(x) for x in coefficients)
    return _call_on(index, stream, _load().gemm_orthogonalize, dtype, M, N, G2.data_ptr(), ldg,
                    sg, O2.data_ptr(), ldo, so, batch, int(steps), a, b, c, float(eps),
                    workspace.data_ptr(), workspace.numel() * workspace.element_size())
