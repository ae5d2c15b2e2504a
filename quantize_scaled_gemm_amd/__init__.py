"""Python binding of libqsg.so (FP8 quantization and scaled FP8 GEMM on
MI355X / gfx950).

Argument marshalling only: every function below has the name of the C entry
point it calls (declared in include/qsg.h), turns torch tensors into device
pointers, sizes and leading dimensions, passes the current HIP stream, and
raises ``QsgError`` on a non-zero status.  All computation happens in the HIP
kernels of the library.  There is no fallback: if the library is missing or
fails to load, every call raises.
"""

import ctypes
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libqsg.so")

# enums of include/qsg.h
E4M3, E5M2 = 0, 1
F32, BF16 = 0, 1
TENSORWISE, DELAYED, MXFP8, BLOCK_1X128, BLOCK_128X128 = 0, 1, 2, 3, 4
MX_CEIL, MX_OCP_FLOOR = 0, 1
AMAX_MAX = 0

FMT = {"e4m3": E4M3, "e5m2": E5M2}

ENTRY_POINTS = (
    "qsg_version",
    "qsg_status_string",
    "qsg_last_error",
    "qsg_amax",
    "qsg_compute_scale",
    "qsg_cast_transpose",
    "qsg_cast_transpose_delayed",
    "qsg_cast_transpose_delayed_noalloc",
    "qsg_amax_update",
    "qsg_quantize",
    "qsg_scaled_gemm",
    "qsg_scaled_gemm_accumulate",
    "qsg_act_fp8_store_fwd",
    "qsg_act_fp8_store_bwd",
    "qsg_wgrad_bf16",
    "qsg_quantize_nvfp4",
    "qsg_gemm_nvfp4",
    "qsg_quantize_int8_workspace",
    "qsg_quantize_int8",
    "qsg_gemm_int8",
    "qsg_wgrad_int8",
    "qsg_swiglu_int8_store_fwd",
    "qsg_swiglu_int8_store_bwd",
    "qsg_rmsnorm_quantize",
    "qsg_rmsnorm_bwd_workspace",
    "qsg_rmsnorm_bwd",
    "qsg_grad_plan",
    "qsg_grad_sumsq",
    "qsg_grad_clip",
)


class QsgError(RuntimeError):
    pass


class Recipe(ctypes.Structure):
    _fields_ = [("scaling", ctypes.c_int32), ("fmt", ctypes.c_int32),
                ("margin", ctypes.c_int32), ("mx_rule", ctypes.c_int32)]


class Grad(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib = None


def load_library(path=LIB_PATH):
    """Load libqsg.so (once) and declare the argument types."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise QsgError(f"{path} is not built: run `python -m quantize_scaled_gemm_amd.build`")
    lib = ctypes.CDLL(path)
    P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
    lib.qsg_version.restype = I
    lib.qsg_version.argtypes = []
    lib.qsg_status_string.restype = ctypes.c_char_p
    lib.qsg_status_string.argtypes = [I]
    lib.qsg_last_error.restype = ctypes.c_char_p
    lib.qsg_last_error.argtypes = []
    lib.qsg_amax.restype = I
    lib.qsg_amax.argtypes = [P, I, I64, I64, I64, F, P]
    lib.qsg_compute_scale.restype = I
    lib.qsg_compute_scale.argtypes = [F, I, I, F, F, P]
    lib.qsg_cast_transpose.restype = I
    lib.qsg_cast_transpose.argtypes = [P, I, I64, I64, I64, I, F, P, P, F, P]
    lib.qsg_cast_transpose_delayed.restype = I
    lib.qsg_cast_transpose_delayed.argtypes = [P, I, I64, I64, I64, I, I, F, I64, I64, F, F, P, P, F, P, P]
    lib.qsg_cast_transpose_delayed_noalloc.restype = I
    lib.qsg_cast_transpose_delayed_noalloc.argtypes = [P, I, I64, I64, I64, I, I, F, I64, I64, F, F, P, P, F, P]
    lib.qsg_amax_update.restype = I
    lib.qsg_amax_update.argtypes = [F, I64, I64, F, I, I, I, F, F, P]
    lib.qsg_quantize.restype = I
    lib.qsg_quantize.argtypes = [P, I, I64, I64, I64, ctypes.POINTER(Recipe), P, P, P, P, P]
    lib.qsg_scaled_gemm.restype = I
    lib.qsg_scaled_gemm.argtypes = [P, I, I, P, P, I, I, P, I64, I64, I64, I64, I64, P, I, I64, P]
    lib.qsg_scaled_gemm_accumulate.restype = I
    lib.qsg_wgrad_bf16.restype = I
    lib.qsg_wgrad_bf16.argtypes = [P, I64, I64, I64, P, I64, I64, P, I, I64, I, P]
    lib.qsg_act_fp8_store_fwd.restype = I
    lib.qsg_act_fp8_store_fwd.argtypes = [P, I64, I64, I64, I, F, P, P, F, P]
    lib.qsg_act_fp8_store_bwd.restype = I
    lib.qsg_act_fp8_store_bwd.argtypes = [P, I64, I64, I64, I, P, F, P, P]
    lib.qsg_scaled_gemm_accumulate.argtypes = [P, I, I, P, P, I, I, P, I64, I64, I64, I64, I64, P, I64, P]
    lib.qsg_quantize_nvfp4.argtypes = [P, I, I64, I64, I64, P, P, P, P, P, P]
    lib.qsg_gemm_nvfp4.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, I64, P, I, I64, P]
    R = ctypes.POINTER(Recipe)
    lib.qsg_rmsnorm_quantize.argtypes = [P, P, I, I64, I64, I64, I64, P, I, ctypes.c_float, R, F, P, I64, F, P, P, P,
                                         P, P, F, P]
    lib.qsg_rmsnorm_bwd_workspace.restype = I64
    lib.qsg_rmsnorm_bwd_workspace.argtypes = [I64, I64]
    lib.qsg_rmsnorm_bwd.argtypes = [P, P, P, I, I64, I64, I64, I64, I64, P, I, F, P, I64, F, I, P, P]
    lib.qsg_grad_plan.argtypes = [ctypes.POINTER(Grad), I64, ctypes.POINTER(Grad), ctypes.POINTER(I64)]
    lib.qsg_grad_sumsq.argtypes = [P, I64, P, P, P]
    lib.qsg_grad_clip.argtypes = [P, I64, P, ctypes.c_float, P, P]
    lib.qsg_quantize_int8_workspace.restype = I64
    lib.qsg_quantize_int8_workspace.argtypes = [I64, I64]
    lib.qsg_quantize_int8.argtypes = [P, I, I64, I64, I64, P, P, P, P, P, P]
    lib.qsg_gemm_int8.argtypes = [P, P, P, P, I64, I64, I64, I64, I64, P, I, P, I, I64, P]
    lib.qsg_wgrad_int8.argtypes = [P, I64, I64, I64, P, P, I64, I64, P, I, I64, I, P]
    lib.qsg_swiglu_int8_store_fwd.argtypes = [P, I, I64, I64, I64, P, P, P, P, P, P]
    lib.qsg_swiglu_int8_store_bwd.argtypes = [P, I, I64, I64, I64, P, P, P, I64, P, P]
    _lib = lib
    return lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise QsgError("tensors passed to libqsg must live on the GPU")
    return t.data_ptr()


def _dtype_code(t):
    import torch

    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise QsgError(f"unsupported input dtype {t.dtype}")


def _matrix(t):
    """(rows, cols, ld) of a 2-D row-major tensor view (unit column stride)."""
    if t.dim() != 2:
        raise QsgError("expected a 2-D tensor")
    rows, cols = t.shape
    if t.numel() == 0:
        return rows, cols, max(cols, 1)
    if cols > 1 and t.stride(1) != 1:
        raise QsgError("the last dimension must be contiguous")
    ld = t.stride(0) if rows > 1 else max(cols, 1)
    return rows, cols, max(ld, cols)


def _buffer(t, name, numel, dtype, required=True):
    """Check a buffer the library reads or writes densely: on the GPU,
    contiguous, exactly ``numel`` elements of ``dtype`` ("u8", "i8", "f32", "bf16", "f64").
    Raw integer pointers are passed through unchecked (the C ABI's own
    contract applies to them)."""
    if t is None:
        if required:
            raise QsgError(f"{name} is required")
        return
    if isinstance(t, int):
        return
    import torch

    want = {"u8": torch.uint8, "i8": torch.int8, "f32": torch.float32, "bf16": torch.bfloat16,
            "f64": torch.float64}[dtype]
    if not t.is_cuda:
        raise QsgError(f"{name} must live on the GPU")
    if t.dtype != want:
        raise QsgError(f"{name} must be {dtype} (got {t.dtype})")
    if t.numel() != numel:
        raise QsgError(f"{name} must hold exactly {numel} elements (got {t.numel()}, shape {tuple(t.shape)})")
    if numel > 0 and not t.is_contiguous():
        raise QsgError(f"{name} must be contiguous")


def _scale_layout(kind, rows, K):
    """(numel, dtype) of a scale tensor of the given kind for an operand of
    `rows` rows and contraction length K (include/qsg.h, qsg_scaling), or
    None when K breaks the kind's block rule (the library then reports the
    shape error)."""
    if kind in (TENSORWISE, DELAYED):
        return 1, "f32"
    if kind == MXFP8:
        return (rows * (K // 32), "u8") if K % 32 == 0 else None
    if kind == BLOCK_1X128:
        return (rows * (K // 128), "f32") if K % 128 == 0 else None
    if kind == BLOCK_128X128:
        return (((rows + 127) // 128) * (K // 128), "f32") if K % 128 == 0 else None
    return None


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch

    # the current stream's handle without the Stream object around it, which costs more than a launch
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _check(rc):
    if rc != 0:
        lib = load_library()
        msg = lib.qsg_last_error().decode()
        raise QsgError(f"{lib.qsg_status_string(rc).decode()} ({rc}): {msg}")


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def qsg_version():
    return load_library().qsg_version()


def qsg_amax(x, amax, stream=None):
    """amax (1 fp32 on the GPU) = max |x|."""
    rows, cols, ld = _matrix(x)
    _buffer(amax, "amax", 1, "f32")
    _check(load_library().qsg_amax(_ptr(x), _dtype_code(x), rows, cols, ld, _ptr(amax), _stream(stream)))


def qsg_compute_scale(amax, fmt, margin, scale, scale_inv, stream=None):
    for t, n in ((amax, "amax"), (scale, "scale"), (scale_inv, "scale_inv")):
        _buffer(t, n, 1, "f32")
    _check(load_library().qsg_compute_scale(_ptr(amax), fmt, margin, _ptr(scale), _ptr(scale_inv),
                                            _stream(stream)))


def qsg_cast_transpose(x, fmt, scale, q=None, qt=None, amax_out=None, stream=None):
    rows, cols, ld = _matrix(x)
    _buffer(scale, "scale", 1, "f32")
    _buffer(q, "q", rows * cols, "u8", required=False)
    _buffer(qt, "qt", rows * cols, "u8", required=False)
    _buffer(amax_out, "amax_out", 1, "f32", required=False)
    _check(load_library().qsg_cast_transpose(_ptr(x), _dtype_code(x), rows, cols, ld, fmt, _ptr(scale),
                                             _ptr(q), _ptr(qt), _ptr(amax_out), _stream(stream)))


DELAYED_WORKSPACE_BYTES = 4224  # QSG_DELAYED_WORKSPACE_BYTES of include/qsg.h


def qsg_cast_transpose_delayed(x, fmt, margin, history, step, scale, scale_inv, q=None, qt=None, amax_out=None,
                               workspace=None, stream=None):
    """One delayed-scaling step of x in one launch: q / qt with the scale in
    force, amax into history[step mod len], scale / scale_inv for the next
    step.  workspace: DELAYED_WORKSPACE_BYTES zeroed bytes on the GPU, reused
    from call to call (every call leaves it zero)."""
    rows, cols, ld = _matrix(x)
    _buffer(history, "history", history.numel(), "f32")
    for t, n in ((scale, "scale"), (scale_inv, "scale_inv")):
        _buffer(t, n, 1, "f32")
    _buffer(q, "q", rows * cols, "u8", required=False)
    _buffer(qt, "qt", rows * cols, "u8", required=False)
    _buffer(amax_out, "amax_out", 1, "f32", required=False)
    if workspace is None:
        raise QsgError("workspace is required")
    if not isinstance(workspace, int):
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise QsgError("workspace must be a contiguous GPU tensor")
        if workspace.numel() * workspace.element_size() < DELAYED_WORKSPACE_BYTES:
            raise QsgError(f"workspace must hold at least {DELAYED_WORKSPACE_BYTES} bytes")
    _check(load_library().qsg_cast_transpose_delayed(_ptr(x), _dtype_code(x), rows, cols, ld, fmt, margin,
                                                     _ptr(history), history.numel(), step, _ptr(scale),
                                                     _ptr(scale_inv), _ptr(q), _ptr(qt), _ptr(amax_out),
                                                     _ptr(workspace), _stream(stream)))


def qsg_cast_transpose_delayed_noalloc(x, fmt, margin, history, step, scale, scale_inv, q=None, qt=None,
                                       amax_out=None, stream=None):
    """qsg_cast_transpose_delayed with the library's own per-GPU workspace
    (no allocation; overlapping calls on one GPU race)."""
    rows, cols, ld = _matrix(x)
    _buffer(history, "history", history.numel(), "f32")
    for t, n in ((scale, "scale"), (scale_inv, "scale_inv")):
        _buffer(t, n, 1, "f32")
    _buffer(q, "q", rows * cols, "u8", required=False)
    _buffer(qt, "qt", rows * cols, "u8", required=False)
    _buffer(amax_out, "amax_out", 1, "f32", required=False)
    _check(load_library().qsg_cast_transpose_delayed_noalloc(_ptr(x), _dtype_code(x), rows, cols, ld, fmt, margin,
                                                             _ptr(history), history.numel(), step, _ptr(scale),
                                                             _ptr(scale_inv), _ptr(q), _ptr(qt), _ptr(amax_out),
                                                             _stream(stream)))


def qsg_amax_update(history, step, amax, fmt, margin, scale, scale_inv, algo=AMAX_MAX, stream=None):
    _buffer(history, "history", history.numel(), "f32")
    for t, n in ((amax, "amax"), (scale, "scale"), (scale_inv, "scale_inv")):
        _buffer(t, n, 1, "f32")
    _check(load_library().qsg_amax_update(_ptr(history), history.numel(), step, _ptr(amax), algo, fmt,
                                          margin, _ptr(scale), _ptr(scale_inv), _stream(stream)))


def qsg_quantize(x, scaling, fmt, q=None, s=None, qt=None, st=None, margin=0, mx_rule=MX_CEIL,
                 stream=None):
    rows, cols, ld = _matrix(x)
    _buffer(q, "q", rows * cols, "u8", required=False)
    _buffer(qt, "qt", rows * cols, "u8", required=False)
    if scaling == TENSORWISE:
        _buffer(s, "s", 3, "f32")
    elif scaling in (MXFP8, BLOCK_1X128, BLOCK_128X128):
        # row-wise copy: blocks along cols; column-wise copy: blocks along rows
        if scaling == BLOCK_128X128:
            ok = rows % 128 == 0 and cols % 128 == 0
            row = col = ((rows // 128) * (cols // 128), "f32") if ok else None
        else:
            row, col = _scale_layout(scaling, rows, cols), _scale_layout(scaling, cols, rows)
        if row is not None and q is not None:
            _buffer(s, "s", row[0], row[1])
        if col is not None and qt is not None:
            _buffer(st, "st", col[0], col[1])
    rec = Recipe(scaling, fmt, margin, mx_rule)
    _check(load_library().qsg_quantize(_ptr(x), _dtype_code(x), rows, cols, ld, ctypes.byref(rec),
                                       _ptr(q), _ptr(s), _ptr(qt), _ptr(st), _stream(stream)))


def _gemm_operands(a, b):
    import torch

    for t, name in ((a, "A"), (b, "B")):
        if t.dtype != torch.uint8:
            raise QsgError(f"{name} must hold FP8 bytes as uint8 (got {t.dtype})")
        if not t.is_cuda:
            raise QsgError(f"{name} must live on the GPU")


def _gemm_scales(ka, sa, M, kb, sb, N, K):
    for kind, t, rows, name in ((ka, sa, M, "sa"), (kb, sb, N, "sb")):
        lay = _scale_layout(kind, rows, K)
        if lay is not None:
            _buffer(t, name, lay[0], lay[1])


def qsg_scaled_gemm(a, fa, ka, sa, b, fb, kb, sb, c, stream=None):
    """C (M x N) = (A sa)(B sb)^T; A is M x K and B is N x K (uint8 FP8 bytes)."""
    M, K, lda = _matrix(a)
    N, Kb, ldb = _matrix(b)
    if Kb != K:
        raise QsgError(f"K mismatch: A has {K}, B has {Kb}")
    Mc, Nc, ldc = _matrix(c)
    if (Mc, Nc) != (M, N):
        raise QsgError(f"C is {Mc}x{Nc}, expected {M}x{N}")
    _gemm_operands(a, b)
    _gemm_scales(ka, sa, M, kb, sb, N, K)
    _check(load_library().qsg_scaled_gemm(_ptr(a), fa, ka, _ptr(sa), _ptr(b), fb, kb, _ptr(sb), M, N, K,
                                          lda, ldb, _ptr(c), _dtype_code(c), ldc, _stream(stream)))


def qsg_scaled_gemm_accumulate(a, fa, ka, sa, b, fb, kb, sb, c, stream=None):
    """C (M x N, fp32) = fp32(C + (A sa)(B sb)^T), in place."""
    import torch

    M, K, lda = _matrix(a)
    N, Kb, ldb = _matrix(b)
    if Kb != K:
        raise QsgError(f"K mismatch: A has {K}, B has {Kb}")
    Mc, Nc, ldc = _matrix(c)
    if (Mc, Nc) != (M, N):
        raise QsgError(f"C is {Mc}x{Nc}, expected {M}x{N}")
    if c.dtype != torch.float32:
        raise QsgError("qsg_scaled_gemm_accumulate accumulates into an fp32 C")
    _gemm_operands(a, b)
    _gemm_scales(ka, sa, M, kb, sb, N, K)
    _check(load_library().qsg_scaled_gemm_accumulate(_ptr(a), fa, ka, _ptr(sa), _ptr(b), fb, kb, _ptr(sb), M, N,
                                                     K, lda, ldb, _ptr(c), ldc, _stream(stream)))


def qsg_act_fp8_store_fwd(h, fmt, scale, a, q, amax_out=None, stream=None):
    """a = bf16(gelu(h)); q = FP8 of h * scale (h bf16, a and q dense)."""
    rows, cols, ld = _matrix(h)
    if _dtype_code(h) != BF16:
        raise QsgError("qsg_act_fp8_store_fwd takes a bf16 input")
    _buffer(scale, "scale", 1, "f32")
    _buffer(a, "a", rows * cols, "bf16")
    _buffer(q, "q", rows * cols, "u8")
    _buffer(amax_out, "amax_out", 1, "f32", required=False)
    _check(load_library().qsg_act_fp8_store_fwd(_ptr(h), rows, cols, ld, fmt, _ptr(scale), _ptr(a), _ptr(q),
                                                _ptr(amax_out), _stream(stream)))


def qsg_act_fp8_store_bwd(da, fmt, q, scale_inv, dh, stream=None):
    """dh = bf16(da * gelu'(dec(q) * scale_inv)) (da bf16, q and dh dense)."""
    rows, cols, ld = _matrix(da)
    if _dtype_code(da) != BF16:
        raise QsgError("qsg_act_fp8_store_bwd takes a bf16 gradient")
    _buffer(q, "q", rows * cols, "u8")
    _buffer(scale_inv, "scale_inv", 1, "f32")
    _buffer(dh, "dh", rows * cols, "bf16")
    _check(load_library().qsg_act_fp8_store_bwd(_ptr(da), rows, cols, ld, fmt, _ptr(q), _ptr(scale_inv), _ptr(dh),
                                                _stream(stream)))


def qsg_wgrad_bf16(dy, x, c, accumulate=False, stream=None):
    """C (N x K) = dY^T X, or C += dY^T X for an fp32 C (dY T x N, X T x K, bf16)."""
    T, N, lddy = _matrix(dy)
    Tx, K, ldx = _matrix(x)
    if Tx != T:
        raise QsgError(f"token count mismatch: dY has {T}, X has {Tx}")
    if _dtype_code(dy) != BF16 or _dtype_code(x) != BF16:
        raise QsgError("qsg_wgrad_bf16 takes bf16 operands")
    Nc, Kc, ldc = _matrix(c)
    if (Nc, Kc) != (N, K):
        raise QsgError(f"C is {Nc}x{Kc}, expected {N}x{K}")
    _check(load_library().qsg_wgrad_bf16(_ptr(dy), T, N, lddy, _ptr(x), K, ldx, _ptr(c), _dtype_code(c), ldc,
                                         1 if accumulate else 0, _stream(stream)))


def qsg_quantize_nvfp4(x, tensor_scale, q=None, s=None, qt=None, st=None, stream=None):
    """NVFP4 copies of x: tensor_scale (3 fp32: amax, s_enc, s_dec); row-wise
    q (rows x cols/2 packed E2M1) with s (rows x cols/16 E4M3 bytes) and/or
    column-wise qt (cols x rows/2) with st (cols x rows/16)."""
    rows, cols, ld = _matrix(x)
    _buffer(tensor_scale, "tensor_scale", 3, "f32")
    if q is not None and cols % 16 == 0:
        _buffer(q, "q", rows * (cols // 2), "u8")
        _buffer(s, "s", rows * (cols // 16), "u8")
    if qt is not None and rows % 16 == 0:
        _buffer(qt, "qt", cols * (rows // 2), "u8")
        _buffer(st, "st", cols * (rows // 16), "u8")
    _check(load_library().qsg_quantize_nvfp4(_ptr(x), _dtype_code(x), rows, cols, ld, _ptr(tensor_scale),
                                             _ptr(q), _ptr(s), _ptr(qt), _ptr(st), _stream(stream)))


def qsg_gemm_nvfp4(a, sa, ts_a, b, sb, ts_b, c, stream=None):
    """C (M x N) = s_dec_a s_dec_b (A Sa)(B Sb)^T on NVFP4 operands: a is
    M x K/2 packed bytes, b is N x K/2, sa / sb their E4M3 block scales
    (M x K/16, N x K/16), ts_a / ts_b their 3-float tensor scales (element 2,
    s_dec, is what the library reads)."""
    M, Kh, lda = _matrix(a)
    N, Khb, ldb = _matrix(b)
    if Khb != Kh:
        raise QsgError(f"K mismatch: A has {2 * Kh}, B has {2 * Khb}")
    K = 2 * Kh
    Mc, Nc, ldc = _matrix(c)
    if (Mc, Nc) != (M, N):
        raise QsgError(f"C is {Mc}x{Nc}, expected {M}x{N}")
    _gemm_operands(a, b)
    if K % 16 == 0:
        _buffer(sa, "sa", M * (K // 16), "u8")
        _buffer(sb, "sb", N * (K // 16), "u8")
    _buffer(ts_a, "ts_a", 3, "f32")
    _buffer(ts_b, "ts_b", 3, "f32")
    sdec_a = _ptr(ts_a) + 8 if not isinstance(ts_a, int) else ts_a
    sdec_b = _ptr(ts_b) + 8 if not isinstance(ts_b, int) else ts_b
    _check(load_library().qsg_gemm_nvfp4(_ptr(a), _ptr(sa), sdec_a, _ptr(b), _ptr(sb), sdec_b, M, N, K, lda, ldb,
                                         _ptr(c), _dtype_code(c), ldc, _stream(stream)))


# The calls below take many tensors and are made for single tokens too, so
# each tensor is asked for as little as accepts it; what is not accepted goes
# to the checks above for the words of its refusal.
_FLOATS = {}  # torch dtype -> (code of the ABI, name); both filled on first use
_NAMES = {}   # torch dtype -> name of any type that a buffer may have


def _float_code(t):
    """(code, name) of a float type of the ABI."""
    e = _FLOATS.get(t.dtype)
    if e is None:
        _dtype_code(t)  # refuses other types
        import torch

        _FLOATS.update({torch.bfloat16: (BF16, "bf16"), torch.float32: (F32, "f32")})
        _NAMES.update({torch.bfloat16: "bf16", torch.float32: "f32", torch.uint8: "u8", torch.float64: "f64",
                       torch.int8: "i8"})
        e = _FLOATS[t.dtype]
    return e


def _rows(t, name):
    """(pointer, rows, cols, ld) of a view whose rows do not overlap."""
    if not t.is_cuda:
        raise QsgError(f"{name} must live on the GPU")
    if t.is_contiguous() and t.dim() == 2:
        rows, cols = t.shape
        return t.data_ptr(), rows, cols, cols or 1
    rows, cols, ld = _matrix(t)
    if rows > 1 and cols > 0 and t.stride(0) < cols:
        raise QsgError(f"{name}: the rows overlap (stride {t.stride(0)} for {cols} columns)")
    return t.data_ptr(), rows, cols, ld


def _same_matrix(t, name, shape, dtype):
    """(pointer, ld) of a matrix of this shape and type, or of none."""
    if t is None:
        return None, 0
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda:
        return t.data_ptr(), shape[1] or 1
    p, rows, cols, ld = _rows(t, name)
    if t.shape != shape:
        raise QsgError(f"{name} is {rows}x{cols}, expected {shape[0]}x{shape[1]}")
    if t.dtype is not dtype:
        raise QsgError(f"{name} must be {dtype} (got {t.dtype})")
    return p, ld


def _dense(t, name, numel, dtype):
    """Pointer of a required buffer that _buffer accepts."""
    if isinstance(t, int):
        return t
    if t is None or _NAMES.get(t.dtype) != dtype or t.numel() != numel or not (t.is_contiguous() and t.is_cuda):
        _buffer(t, name, numel, dtype)
    return t.data_ptr()


def _workspace(t, nbytes):
    if isinstance(t, int) or (t is None and nbytes == 0):
        return t
    if t is None:
        raise QsgError("workspace is required")
    if not t.is_cuda or not t.is_contiguous():
        raise QsgError("workspace must be a contiguous GPU tensor")
    if t.numel() * t.element_size() < nbytes:
        raise QsgError(f"workspace must hold at least {nbytes} bytes")
    return t.data_ptr()


def qsg_rmsnorm_quantize(x, gamma, eps, scaling=None, fmt=E4M3, residual=None, h=None, rstd=None, y=None, q=None,
                         s=None, qt=None, st=None, scale=None, amax_out=None, margin=0, mx_rule=MX_CEIL, stream=None):
    """h = x + residual; y = RMS norm of h times gamma; FP8 copies of y under a
    recipe (scaling None: y only).  x, residual and h are 2-D with a unit
    column stride; h may be x or residual itself.  gamma (cols) is fp32 or
    bf16, rstd (rows) fp32; DELAYED takes its scale and returns amax_out."""
    px, rows, cols, ld = _rows(x, "x")
    dt, dname = _float_code(x)
    gt, gname = _float_code(gamma)
    numel, shape, dtype = rows * cols, x.shape, x.dtype
    pr, ldr = _same_matrix(residual, "residual", shape, dtype)
    ph, ldh = _same_matrix(h, "h", shape, dtype)
    pg = _dense(gamma, "gamma", cols, gname)
    prstd = None if rstd is None else _dense(rstd, "rstd", rows, "f32")
    py = None if y is None else _dense(y, "y", numel, dname)
    pq = None if q is None else _dense(q, "q", numel, "u8")
    pqt = None if qt is None else _dense(qt, "qt", numel, "u8")
    pa = None if amax_out is None else _dense(amax_out, "amax_out", 1, "f32")
    psc = ps = pst = rec = None
    if scaling is not None:
        rec = Recipe(scaling, fmt, margin, mx_rule)
        if scaling == DELAYED:
            psc = _dense(scale, "scale", 1, "f32")
        elif scaling == TENSORWISE:
            ps = _dense(s, "s", 3, "f32")
        elif scaling == MXFP8 or scaling == BLOCK_1X128:
            # a shape that breaks the block rule has no layout, and the library refuses it
            if q is not None:
                row = _scale_layout(scaling, rows, cols)
                ps = _dense(s, "s", row[0], row[1]) if row else _ptr(s)
            if qt is not None:
                col = _scale_layout(scaling, cols, rows)
                pst = _dense(st, "st", col[0], col[1]) if col else _ptr(st)
    _check(load_library().qsg_rmsnorm_quantize(px, pr, dt, rows, cols, ld, ldr, pg, gt, eps, rec, psc, ph, ldh, prstd,
                                               py, pq, ps, pqt, pst, pa, _stream(stream)))


def qsg_rmsnorm_bwd_workspace(rows, cols):
    """Bytes of the workspace of qsg_rmsnorm_bwd."""
    n = load_library().qsg_rmsnorm_bwd_workspace(rows, cols)
    if n < 0:
        _check(n)
    return n


def qsg_rmsnorm_bwd(dy, h, gamma, rstd, dx, dres=None, dgamma=None, accumulate=False, workspace=None, stream=None):
    """dx = gradient of x (and of the residual) from dy, the gradient of y, plus
    dres, the gradient that reaches h directly; dgamma (cols fp32) written or
    accumulated.  workspace: qsg_rmsnorm_bwd_workspace(rows, cols) bytes."""
    pdy, rows, cols, lddy = _rows(dy, "dy")
    dt = _float_code(dy)[0]
    gt, gname = _float_code(gamma)
    shape, dtype = dy.shape, dy.dtype
    ph, ldh = _same_matrix(h, "h", shape, dtype)
    pdx, lddx = _same_matrix(dx, "dx", shape, dtype)
    pdr, lddres = _same_matrix(dres, "dres", shape, dtype)
    pg = _dense(gamma, "gamma", cols, gname)
    prstd = _dense(rstd, "rstd", rows, "f32")
    pdg = None if dgamma is None else _dense(dgamma, "dgamma", cols, "f32")
    pw = _workspace(workspace, qsg_rmsnorm_bwd_workspace(rows, cols))
    _check(load_library().qsg_rmsnorm_bwd(pdy, ph, pdr, dt, rows, cols, lddy, ldh, lddres, pg, gt, prstd, pdx, lddx,
                                          pdg, 1 if accumulate else 0, pw, _stream(stream)))


GRAD_WORKSPACE_BYTES = 8192  # QSG_GRAD_WORKSPACE_BYTES of include/qsg.h


class GradPlan:
    """The chunk table of a list of gradients, on the GPU (``table``,
    ``n_chunks``), with the tensors that it points into.  It has to live until
    a captured graph that reads it is replayed no more."""

    def __init__(self, table, n_chunks, grads, outs, stream=None):
        self.table, self.n_chunks, self.grads, self.outs = table, n_chunks, grads, outs
        self.streams = {stream}  # handles: where the table was allocated, and every one recorded below

    def read_on(self, stream):
        """A launch on this stream reads the table: its memory, once freed, is
        not given away before that launch is done."""
        if not isinstance(self.table, int):
            import torch

            self.table.record_stream(torch.cuda.ExternalStream(stream, device=self.table.device))
        self.streams.add(stream)


def qsg_grad_plan(grads, outs=None):
    """GradPlan of contiguous fp32 or bf16 gradients of any shapes; clipped
    values go to ``outs`` (same shapes and types; default: in place), none of
    which may overlap another tensor (a gradient twice in place).  It is made
    once for gradients that stay where they are, and keeps them alive."""
    import torch

    grads = list(grads)
    outs = grads if outs is None else list(outs)
    if len(outs) != len(grads):
        raise QsgError(f"{len(grads)} gradients, but {len(outs)} outputs")
    for k, (g, o) in enumerate(zip(grads, outs)):
        for t, name in ((g, "gradient"), (o, "output")):
            if not t.is_cuda:
                raise QsgError(f"{name} {k} must live on the GPU")
            if not t.is_contiguous():
                raise QsgError(f"{name} {k} must be contiguous")
            if t.device != grads[0].device:
                raise QsgError(f"{name} {k} is on {t.device}, the first gradient on {grads[0].device}")
        if o.shape != g.shape or o.dtype != g.dtype:
            raise QsgError(f"output {k} must have the shape and type of its gradient")
    entries = (Grad * max(1, len(grads)))()
    for k, (g, o) in enumerate(zip(grads, outs)):
        entries[k] = Grad(g.data_ptr(), o.data_ptr(), g.numel(), _dtype_code(g), 0)
    n = ctypes.c_int64(0)
    lib = load_library()
    _check(lib.qsg_grad_plan(entries, len(grads), None, ctypes.byref(n)))
    chunks = (Grad * max(1, n.value))()
    _check(lib.qsg_grad_plan(entries, len(grads), chunks, ctypes.byref(n)))
    host = torch.frombuffer(chunks, dtype=torch.uint8)
    table = host.to(grads[0].device if grads else "cuda")
    return GradPlan(table, n.value, grads, outs, torch.cuda.current_stream(table.device).cuda_stream)


def qsg_grad_sumsq(plan, sumsq, workspace, stream=None):
    """sumsq (1 fp64 on the GPU) = sum of the squares of the plan's gradients.
    workspace: GRAD_WORKSPACE_BYTES bytes on the GPU."""
    on = _stream(stream)
    _check(load_library().qsg_grad_sumsq(_ptr(plan.table), plan.n_chunks, _dense(sumsq, "sumsq", 1, "f64"),
                                         _workspace(workspace, GRAD_WORKSPACE_BYTES), on))
    if on not in plan.streams:
        plan.read_on(on)


def qsg_grad_clip(plan, sumsq, max_norm, norm_out=None, stream=None):
    """The plan's outputs = gradients * min(1, max_norm / (norm + 1e-6)) with
    norm = sqrt(sumsq), written to norm_out (1 fp32) if given."""
    on = _stream(stream)
    _check(load_library().qsg_grad_clip(_ptr(plan.table), plan.n_chunks, _dense(sumsq, "sumsq", 1, "f64"),
                                        max_norm, None if norm_out is None else _dense(norm_out, "norm_out", 1, "f32"),
                                        on))
    if on not in plan.streams:
        plan.read_on(on)


# ---------------------------------------------------------------------------
# INT8
# ---------------------------------------------------------------------------
# Each tensor is asked for as little as accepts it, and has to be on the device
# of the call's first one, which _launch compares with the current device; what
# is not accepted goes to the checks above for the words of its refusal.
def _refuse_device(t, name, dev):
    raise QsgError(f"{name} is on device {t.get_device()}, the call's first tensor on device {dev}")


def _view(t, name, dev):
    """(pointer, rows, cols, ld) of a view whose rows do not overlap."""
    if t.get_device() == dev >= 0 and t.is_contiguous():
        shape = t.shape
        if len(shape) == 2:
            return t.data_ptr(), shape[0], shape[1], shape[1] or 1
    r = _rows(t, name)
    if t.get_device() != dev:
        _refuse_device(t, name, dev)
    return r


def _packed(t, name, numel, dtype, dev):
    """Pointer of a required buffer that _buffer accepts."""
    if isinstance(t, int):
        return t
    if (t is None or _NAMES.get(t.dtype) != dtype or t.numel() != numel or t.get_device() != dev
            or not t.is_contiguous()):
        _buffer(t, name, numel, dtype)
        if t.get_device() != dev:
            _refuse_device(t, name, dev)
    return t.data_ptr()


def _pair(codes, numel, cname, scales, n, sname, dev):
    """Pointers of codes and the scales that belong to them, or of neither."""
    if codes is None and scales is None:
        return None, None
    return _packed(codes, cname, numel, "i8", dev), _packed(scales, sname, n, "f32", dev)


def _codes(t, name, dev):
    """(pointer, rows, cols, ld) of an INT8 operand."""
    r = _view(t, name, dev)
    if _NAMES.get(t.dtype) != "i8":
        import torch

        if t.dtype is not torch.int8:
            raise QsgError(f"{name} must hold INT8 codes as int8 (got {t.dtype})")
    return r


def _launch_stream(stream, dev):
    """The stream's handle; the library launches on the current device."""
    import torch

    now = torch.cuda.current_device()
    if now != dev:
        raise QsgError(f"the tensors are on device {dev}, the current device is {now}")
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(now)


def qsg_quantize_int8_workspace(rows, cols):
    """Bytes of the workspace of qsg_quantize_int8 with a transposed copy."""
    n = load_library().qsg_quantize_int8_workspace(rows, cols)
    if n < 0:
        _check(n)
    return n


def qsg_quantize_int8(x, q=None, s=None, qt=None, st=None, workspace=None, stream=None):
    """INT8 copies of x (rows x cols): row-wise q (int8) with one fp32 scale for
    each row in s, and / or transposed qt (cols x rows) with one for each column
    in st, for which workspace holds qsg_quantize_int8_workspace(rows, cols)
    bytes."""
    dev = x.get_device()
    px, rows, cols, ld = _view(x, "x", dev)
    dt = _float_code(x)[0]
    pq, ps = _pair(q, rows * cols, "q", s, rows, "s", dev)
    pqt = pst = pw = None
    if qt is not None or st is not None:
        pqt, pst = _pair(qt, rows * cols, "qt", st, cols, "st", dev)
        pw = _workspace(workspace, qsg_quantize_int8_workspace(rows, cols))
        if pw is not None and not isinstance(workspace, int) and workspace.get_device() != dev:
            _refuse_device(workspace, "workspace", dev)
    _check(load_library().qsg_quantize_int8(px, dt, rows, cols, ld, pq, ps, pqt, pst, pw, _launch_stream(stream, dev)))


def qsg_gemm_int8(a, sa, b, sb, c, bias=None, stream=None):
    """C (M x N) = (A B^T) sa[:, None] sb (+ bias): A is M x K and B is N x K
    (int8), sa (M) and sb (N) fp32 scales, bias N values of fp32 or bf16."""
    dev = a.get_device()
    ct = _float_code(c)[0]
    pa, M, K, lda = _codes(a, "A", dev)
    pb, N, Kb, ldb = _codes(b, "B", dev)
    if Kb != K:
        raise QsgError(f"K mismatch: A has {K}, B has {Kb}")
    pc, Mc, Nc, ldc = _view(c, "C", dev)
    if Mc != M or Nc != N:
        raise QsgError(f"C is {Mc}x{Nc}, expected {M}x{N}")
    psa, psb = _packed(sa, "sa", M, "f32", dev), _packed(sb, "sb", N, "f32", dev)
    pbias, bt = None, 0
    if bias is not None:
        bt, bname = _float_code(bias)
        pbias = _packed(bias, "bias", N, bname, dev)
    _check(load_library().qsg_gemm_int8(pa, psa, pb, psb, M, N, K, lda, ldb, pbias, bt, pc, ct, ldc,
                                        _launch_stream(stream, dev)))


def qsg_wgrad_int8(dy, q, s, c, accumulate=False, stream=None):
    """C (N x K) = dY^T bf16(q s[:, None]), or C += for an fp32 C: dY T x N
    (bf16), q T x K (int8) with T fp32 scales in s."""
    dev = dy.get_device()
    pdy, T, N, lddy = _view(dy, "dY", dev)
    if _float_code(dy)[0] != BF16:
        raise QsgError("qsg_wgrad_int8 takes a bf16 dY")
    pq, Tq, K, ldq = _codes(q, "q", dev)
    if Tq != T:
        raise QsgError(f"token count mismatch: dY has {T}, q has {Tq}")
    pc, Nc, Kc, ldc = _view(c, "C", dev)
    if Nc != N or Kc != K:
        raise QsgError(f"C is {Nc}x{Kc}, expected {N}x{K}")
    ct = _float_code(c)[0]
    ps = _packed(s, "s", T, "f32", dev)
    _check(load_library().qsg_wgrad_int8(pdy, T, N, lddy, pq, ps, K, ldq, pc, ct, ldc, 1 if accumulate else 0,
                                         _launch_stream(stream, dev)))


def qsg_swiglu_int8_store_fwd(gu, a=None, aq=None, sa=None, ck=None, cs=None, stream=None):
    """a = silu(g) u of gu = [g, u] (rows x 2 cols): a (rows x cols, the type of
    gu) and / or its INT8 copy (aq, sa as qsg_quantize_int8); ck (rows x 2 cols,
    int8) and cs (rows x 2 ceil(cols / 128)) keep g and u for backward."""
    dev = gu.get_device()
    p, rows, both, ld = _view(gu, "gu", dev)
    if both % 2:
        raise QsgError(f"gu has {both} columns: those of g, then as many of u are expected")
    cols = both // 2
    dt, dname = _float_code(gu)
    pa = None if a is None else _packed(a, "a", rows * cols, dname, dev)
    paq, psa = _pair(aq, rows * cols, "aq", sa, rows, "sa", dev)
    pck, pcs = _pair(ck, rows * both, "ck", cs, rows * 2 * -(-cols // 128), "cs", dev)
    _check(load_library().qsg_swiglu_int8_store_fwd(p, dt, rows, cols, ld, pa, paq, psa, pck, pcs,
                                                    _launch_stream(stream, dev)))


def qsg_swiglu_int8_store_bwd(da, ck, cs, dgu, a=None, stream=None):
    """dgu = [dg, du] (rows x 2 cols) from da (rows x cols) and what the forward
    pass kept; a (rows x cols) is computed again on request.  One type for da,
    dgu and a."""
    dev = da.get_device()
    p, rows, cols, ldda = _view(da, "da", dev)
    dt, dname = _float_code(da)
    if dgu is None:
        raise QsgError("dgu is required")
    po, ro, co, lddgu = _view(dgu, "dgu", dev)
    if ro != rows or co != 2 * cols:
        raise QsgError(f"dgu is {ro}x{co}, expected {rows}x{2 * cols}")
    if dgu.dtype is not da.dtype:
        raise QsgError(f"dgu must be {da.dtype} (got {dgu.dtype})")
    pck = _packed(ck, "ck", rows * 2 * cols, "i8", dev)
    pcs = _packed(cs, "cs", rows * 2 * -(-cols // 128), "f32", dev)
    pa = None if a is None else _packed(a, "a", rows * cols, dname, dev)
    _check(load_library().qsg_swiglu_int8_store_bwd(p, dt, rows, cols, ldda, pck, pcs, po, lddgu, pa,
                                                    _launch_stream(stream, dev)))
