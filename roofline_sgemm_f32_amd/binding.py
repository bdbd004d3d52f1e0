"""ctypes binding over libsgemm.so (declared in include/sgemm.h).

Argument marshalling only: every step of the product runs in the library's
HIP kernels.  PyTorch supplies device memory and the stream.  If the library
has not been built, the first call raises; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(HERE, "libsgemm.so")
_lib = None

# sgemm_variant_t
VARIANTS = {
    "auto": 0,
    "k1_coalesced": 1,
    "k2_lds_tiled32": 2,
    "k3_regtile_db": 3,
    "k4_mfma": 4,
    "k2_lds_tiled16": 5,
    "k2_lds_tiled32_pad1": 6,
    "k0_naive": 7,
    "k2_lds_tiled16_pad1": 8,
    "k4_mfma_tile128": 9,
    "k4_mfma_tile64": 10,
    "k4_mfma_tile128x256": 11,
}

# sgemm_status_t
STATUS = {
    0: "SGEMM_OK", 1: "SGEMM_ERR_DIM", 2: "SGEMM_ERR_LD", 3: "SGEMM_ERR_NULLPTR",
    4: "SGEMM_ERR_VARIANT", 5: "SGEMM_ERR_ALIAS", 6: "SGEMM_ERR_LAUNCH",
    7: "SGEMM_ERR_UNSUPPORTED", 8: "SGEMM_ERR_ARG", 9: "SGEMM_ERR_SCRATCH",
}

EXPORTS = ["sgemm_f32", "sgemm_f32_variant", "sgemm_copy_f32", "sgemm_copy_f32_launch",
           "sgemm_status_string", "sgemm_variant_name", "sgemm_auto_variant",
           "sgemm_last_hip_error", "sgemm_abi_version", "sgemm_probe_valu_f32",
           "sgemm_probe_mfma_f32", "sgemm_f32_ex", "sgemm_f32_colmajor", "sgemm_f32_ex_split",
           "sgemm_split_plan", "sgemm_plan_config", "sgemm_f32_ex_split_noalloc",
           "sgemm_glu_f32", "sgemm_glu_backward_f32", "sgemm_q4", "sgemm_q4_glu"]

MAX_SPLITS = 64
STATIC_SCRATCH_BYTES = 64 * 1024 * 1024  # SGEMM_STATIC_SCRATCH_BYTES

OP_N, OP_T = 0, 1

# sgemm_act_t
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4}


# Importing this module does not import torch: the feed-forward functions,
# whose calls take microseconds, do so once, through _use_torch, which sets
# these (sgemm_type_t of the tensor types; a device's current stream's handle).
torch = None
_FLOATS = {}
_raw_stream = None


class SgemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


def library_path() -> str:
    return _LIB_PATH


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libsgemm.so; raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m roofline_sgemm_f32_amd.build`"
                           " (there is no non-HIP fallback)")
    lib = ctypes.CDLL(p)
    i64, vp, cint = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    gemm = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    lib.sgemm_f32.argtypes = gemm
    lib.sgemm_f32.restype = cint
    lib.sgemm_f32_variant.argtypes = [cint, *gemm]
    lib.sgemm_f32_variant.restype = cint
    f32 = ctypes.c_float
    ex = [cint, cint, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
    lib.sgemm_f32_ex.argtypes = ex
    lib.sgemm_f32_ex.restype = cint
    lib.sgemm_f32_colmajor.argtypes = ex
    lib.sgemm_f32_colmajor.restype = cint
    lib.sgemm_f32_ex_split.argtypes = [*ex[:-1], cint, vp]
    lib.sgemm_f32_ex_split.restype = cint
    lib.sgemm_f32_ex_split_noalloc.argtypes = [*ex[:-1], cint, vp]
    lib.sgemm_f32_ex_split_noalloc.restype = cint
    lib.sgemm_split_plan.argtypes = [cint, cint, i64, i64, i64, vp, i64, vp, i64, cint,
                                     ctypes.POINTER(i64)]
    lib.sgemm_split_plan.restype = cint
    ip = ctypes.POINTER(cint)
    lib.sgemm_plan_config.argtypes = [cint, cint, i64, i64, i64, vp, i64, vp, i64, ip, ip, ip, ip,
                                      ip, ctypes.POINTER(i64)]
    lib.sgemm_plan_config.restype = cint
    lib.sgemm_glu_f32.argtypes = [cint, cint, i64, i64, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp,
                                  i64, vp]
    lib.sgemm_glu_f32.restype = cint
    lib.sgemm_glu_backward_f32.argtypes = [cint, cint, i64, i64, i64, vp, i64, vp, vp, i64, vp, vp,
                                           i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, i64, f32, vp]
    lib.sgemm_glu_backward_f32.restype = cint
    lib.sgemm_q4.argtypes = [cint, cint, i64, i64, i64, vp, i64, vp, i64, i64, vp, i64, vp, i64,
                             vp, i64, vp]
    lib.sgemm_q4.restype = cint
    lib.sgemm_q4_glu.argtypes = [cint, cint, cint, i64, i64, i64, vp, i64, vp, vp, i64, i64, vp, vp,
                                 i64, vp, vp, i64, vp, i64, vp]
    lib.sgemm_q4_glu.restype = cint
    lib.sgemm_copy_f32.argtypes = [vp, vp, i64, vp]
    lib.sgemm_copy_f32.restype = cint
    lib.sgemm_copy_f32_launch.argtypes = [vp, vp, i64, cint, i64, vp]
    lib.sgemm_copy_f32_launch.restype = cint
    lib.sgemm_status_string.argtypes = [cint]
    lib.sgemm_status_string.restype = ctypes.c_char_p
    lib.sgemm_variant_name.argtypes = [cint]
    lib.sgemm_variant_name.restype = ctypes.c_char_p
    lib.sgemm_auto_variant.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64]
    lib.sgemm_auto_variant.restype = cint
    lib.sgemm_last_hip_error.argtypes = []
    lib.sgemm_last_hip_error.restype = cint
    lib.sgemm_probe_valu_f32.argtypes = [vp, i64, cint, i64, ctypes.c_float, ctypes.c_float, vp]
    lib.sgemm_probe_valu_f32.restype = cint
    lib.sgemm_probe_mfma_f32.argtypes = [vp, vp, vp, i64, i64, vp]
    lib.sgemm_probe_mfma_f32.restype = cint
    lib.sgemm_abi_version.argtypes = []
    lib.sgemm_abi_version.restype = cint
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().sgemm_status_string(int(status)).decode()


def variant_name(variant: int) -> str | None:
    r = load().sgemm_variant_name(int(variant))
    return r.decode() if r is not None else None


def _variant_id(variant) -> int:
    if isinstance(variant, str):
        if variant not in VARIANTS:
            raise ValueError(f"unknown variant {variant!r}; one of {sorted(VARIANTS)}")
        return VARIANTS[variant]
    return int(variant)


def sgemm_f32_variant(variant, M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    """Raw entry point: integer pointers and sizes; returns the status code."""
    return load().sgemm_f32_variant(_variant_id(variant), M, N, K, A, lda, B, ldb, C, ldc, stream)


def sgemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    return load().sgemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream)


def _ld(t, name):
    import torch
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    return max(t.stride(0), t.shape[1], 1) if t.shape[0] > 1 else max(t.shape[1], 1)


def _stream_handle(device):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def sgemm(A, B, out=None, variant="auto"):
    """C = A @ B for float32 CUDA (ROCm) tensors, computed by libsgemm on the
    current stream.  Row-major views with any row stride >= the row length
    are accepted; ``out`` (M x N, written, never read) may be supplied."""
    import torch
    if A.device.type != "cuda" or B.device.type != "cuda":
        raise ValueError("operands must be GPU tensors")
    M, K = A.shape
    K2, N = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {tuple(B.shape)}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    elif out.shape != (M, N):
        raise ValueError("out has the wrong shape")
    lda, ldb, ldc = _ld(A, "A"), _ld(B, "B"), _ld(out, "out")
    st = sgemm_f32_variant(variant, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb,
                           out.data_ptr(), ldc, _stream_handle(A.device))
    if st != 0:
        raise SgemmError(st, "sgemm_f32_variant")
    return out


def sgemm_ex(A, B, out=None, transa=False, transb=False, alpha=1.0, beta=0.0, splits=None,
             noalloc=False):
    """C = alpha op(A) op(B) + beta C (row-major float32 GPU tensors).  A is
    M x K, or K x M with transa (op(A) = A^T); B is K x N, or N x K with
    transb.  ``out`` holds C (read only when beta != 0); it is allocated when
    omitted (then beta must be 0).  ``splits`` (sgemm_f32_ex_split): None or
    0 chooses the K split by shape, 1 never splits, 2..64 asks for at most
    that many K chunks.  ``noalloc`` calls sgemm_f32_ex_split_noalloc, whose
    scratch is the library's static device array (the library then
    allocates nothing)."""
    import torch
    if A.device.type != "cuda" or B.device.type != "cuda":
        raise ValueError("operands must be GPU tensors")
    M, K = (A.shape[1], A.shape[0]) if transa else tuple(A.shape)
    Kb, N = (B.shape[1], B.shape[0]) if transb else tuple(B.shape)
    if Kb != K:
        raise ValueError("inner dimensions differ")
    if out is None:
        if beta != 0:
            raise ValueError("beta != 0 needs out")
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    elif tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    args = (int(transa), int(transb), M, N, K, alpha, A.data_ptr(), _ld(A, "A"), B.data_ptr(),
            _ld(B, "B"), beta, out.data_ptr(), _ld(out, "out"))
    if noalloc:
        name = "sgemm_f32_ex_split_noalloc"
        st = load().sgemm_f32_ex_split_noalloc(*args, int(splits or 0), _stream_handle(A.device))
    elif splits is None:
        name = "sgemm_f32_ex"
        st = load().sgemm_f32_ex(*args, _stream_handle(A.device))
    else:
        name = "sgemm_f32_ex_split"
        st = load().sgemm_f32_ex_split(*args, int(splits), _stream_handle(A.device))
    if st != 0:
        raise SgemmError(st, name)
    return out


def split_plan(M, N, K, transa=False, transb=False, lda=None, ldb=None, A_ptr=0, B_ptr=0,
               splits=0):
    """(chunks, kchunk) of the K split sgemm_f32_ex_split would run (host
    only; the pointers enter only through their 16-byte alignment)."""
    lda = (max(M, 1) if transa else max(K, 1)) if lda is None else lda
    ldb = (max(K, 1) if transb else max(N, 1)) if ldb is None else ldb
    kc = ctypes.c_int64(0)
    r = load().sgemm_split_plan(int(transa), int(transb), M, N, K, A_ptr or None, lda,
                                B_ptr or None, ldb, int(splits), ctypes.byref(kc))
    if r < 0:
        raise SgemmError(-r, "sgemm_split_plan")
    return r, kc.value


def plan_config(M, N, K, transa=False, transb=False, lda=None, ldb=None, A_ptr=0, B_ptr=0):
    """The kernel configuration a shape-chosen call runs (host only): dict
    with engine ("mfma", "thin" or None), tile (tile_m, tile_n), k_groups,
    packed, splits, kchunk; splits 0 when neither kernel is launched."""
    lda = (max(M, 1) if transa else max(K, 1)) if lda is None else lda
    ldb = (max(K, 1) if transb else max(N, 1)) if ldb is None else ldb
    en, tm, tn, wk, pk = (ctypes.c_int(0) for _ in range(5))
    kc = ctypes.c_int64(0)
    r = load().sgemm_plan_config(int(transa), int(transb), M, N, K, A_ptr or None, lda,
                                 B_ptr or None, ldb, ctypes.byref(en), ctypes.byref(tm),
                                 ctypes.byref(tn), ctypes.byref(wk), ctypes.byref(pk),
                                 ctypes.byref(kc))
    if r < 0:
        raise SgemmError(-r, "sgemm_plan_config")
    return {"engine": {1: "mfma", 2: "thin"}.get(en.value), "tile": (tm.value, tn.value),
            "k_groups": wk.value, "packed": bool(pk.value), "splits": r, "kchunk": kc.value}


def _ld_col(t, name):
    """Leading dimension of a column-major 2-D view (unit row stride)."""
    import torch
    if t.dtype != torch.float32 or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D float32 tensor")
    if t.shape[0] > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be column-major (unit row stride)")
    return max(t.stride(1), t.shape[0], 1) if t.shape[1] > 1 else max(t.shape[0], 1)


def sgemm_colmajor(A, B, out, transa=False, transb=False, alpha=1.0, beta=0.0):
    """The column-major (BLAS) convention on column-major tensor views
    (stride(0) == 1): out (m x n) = alpha op(A) op(B) + beta out."""
    m, n = out.shape
    k = A.shape[0] if transa else A.shape[1]
    st = load().sgemm_f32_colmajor(int(transa), int(transb), m, n, k, alpha, A.data_ptr(),
                                   _ld_col(A, "A"), B.data_ptr(), _ld_col(B, "B"), beta,
                                   out.data_ptr(), _ld_col(out, "out"), _stream_handle(out.device))
    if st != 0:
        raise SgemmError(st, "sgemm_f32_colmajor")
    return out


def _use_torch() -> None:
    global torch, _raw_stream
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if _raw_stream is None:  # the public way, 2 us slower
        def _raw_stream(dev):
            return torch.cuda.current_stream(dev).cuda_stream
    _FLOATS.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})


def _act_id(act) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}; one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def _rows(t, name, shape=None, dtypes=None):
    """Leading dimension of a 2-D row-major GPU tensor, checked."""
    try:  # the usual case in few steps: these calls take microseconds
        (rows, cols), (ld, step) = t.shape, t.stride()
        if (t.is_cuda and (t.dtype in dtypes if dtypes else t.dtype == torch.float32)
                and (shape is None or (rows, cols) == shape) and (step == 1 or cols == 1)):
            if rows > 1 and ld >= cols > 0:
                return ld
            if rows == 1 and cols > 0:
                return cols
    except (AttributeError, ValueError):
        pass
    return _rows_checked(t, name, shape, dtypes)


def _rows_checked(t, name, shape, dtypes):
    dtypes = dtypes or (torch.float32,)
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a tensor of {' or '.join(str(d) for d in dtypes)}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must have a row stride of at least its row length")
    return max(t.stride(0), t.shape[1], 1) if t.shape[0] > 1 else max(t.shape[1], 1)


def _pair_ld(a, b, name, shape, dtypes=None):
    """The leading dimension two tensors share (the C entry points take one)."""
    la, lb = _rows(a, f"{name}[0]", shape, dtypes), _rows(b, f"{name}[1]", shape, dtypes)
    if la != lb:
        raise ValueError(f"{name}: the two tensors must have the same row stride ({la} and {lb})")
    return la


def _call(fn, where, X, others, *args):
    """Call an entry point on the device of its tensors and that device's
    current stream."""
    dev = X.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{where}: tensors on {t.device} and {X.device}")
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):  # the default stream is the current device's
            st = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        st = fn(*args, _raw_stream(dev))
    if st != 0:
        raise SgemmError(st, where)


def _dim(t, i) -> int:
    """Size i of a 2-D tensor; 0 of anything else, which the checks then name."""
    return t.shape[i] if isinstance(t, torch.Tensor) and t.dim() == 2 else 0


def _two(pair, name):
    """The two tensors of a pair that come together."""
    if not isinstance(pair, (tuple, list)) or len(pair) != 2 or any(t is None for t in pair):
        raise ValueError(f"{name} must be a pair of tensors")
    return pair


def _halves(rows, cols, like):
    """Two rows x cols float32 tensors, the column halves of one buffer."""
    buf = torch.empty((rows, 2 * cols), dtype=torch.float32, device=like.device)
    return buf[:, :cols], buf[:, cols:]


def glu(X, Wg, Wu, act="silu", transw=False, out=None, save=False):
    """The gated feed-forward block H = act(X Wg) * (X Wu), float32, on the
    current stream.  X is M x K; Wg and Wu are K x F, or F x K with ``transw``
    (the layout of a linear layer), with the same row stride.  ``act``: silu,
    gelu, gelu_tanh, relu or sigmoid.  Returns H (M x F, ``out`` when given);
    with ``save`` true (H, G, U), with G = X Wg and U = X Wu, which
    glu_backward takes.  ``save`` may also be the pair (G, U) to write."""
    _FLOATS or _use_torch()
    a = _act_id(act)
    ldx = _rows(X, "X")
    M, K = X.shape
    F = _dim(Wg, 0 if transw else 1)
    ldw = _pair_ld(Wg, Wu, "weights", (F, K) if transw else (K, F))
    if out is None:
        H, ldh = torch.empty((M, F), dtype=torch.float32, device=X.device), max(F, 1)
    else:
        H, ldh = out, _rows(out, "out", (M, F))
    G = U = None
    ldgu = 1
    if isinstance(save, (tuple, list)):
        G, U = _two(save, "save")
    elif save:
        G, U = _halves(M, F, X)
    if G is not None:
        ldgu = _pair_ld(G, U, "save", (M, F))
    null = G is None or M == 0 or F == 0
    _call(load().sgemm_glu_f32, "sgemm_glu_f32", X, (Wg, Wu, H, G, U), a, int(transw), M, F, K,
          X.data_ptr(), ldx, Wg.data_ptr(), Wu.data_ptr(), ldw, H.data_ptr(), ldh,
          None if null else G.data_ptr(), None if null else U.data_ptr(), ldgu)
    return H if G is None else (H, G, U)


def glu_backward(dH, X, Wg, Wu, G, U, act="silu", transw=False, need_dx=True, need_dw=True,
                 dX=None, dW=None, beta=0.0, inplace=False):
    """Gradients of glu: from dH (M x F) and the G and U of the forward pass,
    (dX, dWg, dWu), None for those not asked for (``need_dx``, ``need_dw``).
    ``dX`` and ``dW`` = (dWg, dWu) may be supplied; with ``beta`` the weight
    gradients are added to beta times what dW holds.  ``inplace`` overwrites
    G and U with dG and dU instead of allocating M x 2F floats for them."""
    _FLOATS or _use_torch()
    a = _act_id(act)
    ldx = _rows(X, "X")
    M, K = X.shape
    F = _dim(Wg, 0 if transw else 1)
    wshape = (F, K) if transw else (K, F)
    ldw = _pair_ld(Wg, Wu, "weights", wshape)
    ldgu = _pair_ld(G, U, "G, U", (M, F))
    lddh = _rows(dH, "dH", (M, F))
    dG, dU = (G, U) if inplace else _halves(M, F, X)
    lddgu = _pair_ld(dG, dU, "dG, dU", (M, F))
    lddx = lddw = 1
    if need_dx:
        dX = torch.empty((M, K), dtype=torch.float32, device=X.device) if dX is None else dX
        lddx = _rows(dX, "dX", (M, K))
    else:
        dX = None
    dWg = dWu = None
    if need_dw:
        if dW is None:
            if beta != 0:
                raise ValueError("beta != 0 needs dW")
            if transw:
                buf = torch.empty((2 * F, K), dtype=torch.float32, device=X.device)
                dW = buf[:F], buf[F:]
            else:
                dW = _halves(K, F, X)
        dWg, dWu = _two(dW, "dW")
        lddw = _pair_ld(dWg, dWu, "dW", wshape)
    # Empty tensors have no address; the entry point takes null for "skip".
    x_null, w_null = dX is None or dX.numel() == 0, dWg is None or dWg.numel() == 0
    _call(load().sgemm_glu_backward_f32, "sgemm_glu_backward_f32", X,
          (Wg, Wu, G, U, dH, dX, dWg, dWu), a, int(transw), M, F, K, X.data_ptr(), ldx,
          Wg.data_ptr(), Wu.data_ptr(), ldw, G.data_ptr(), U.data_ptr(), ldgu, dH.data_ptr(), lddh,
          dG.data_ptr(), dU.data_ptr(), lddgu, None if x_null else dX.data_ptr(), lddx,
          None if w_null else dWg.data_ptr(), None if w_null else dWu.data_ptr(), lddw, beta)
    return dX, dWg, dWu


def _q4_weight(w, scales, zeros, N, K, group, name):
    """Strides of one packed weight (bytes, scales, zero points), checked."""
    groups = -(-K // group)
    ldw = _rows(w, f"{name} weights", (N, (K + 1) // 2), (torch.uint8,))
    lds = _rows(scales, f"{name} scales", (N, groups), _FLOATS)
    ldz = _rows(zeros, f"{name} zeros", (N, groups), (torch.uint8,)) if zeros is not None else 1
    return ldw, lds, ldz


def _q4_group(group) -> int:
    if group < 32 or group & (group - 1):
        raise ValueError("group must be a power of two, 32 or more")
    return int(group)


def q4_matmul(X, w, scales, zeros=None, group=128, out=None):
    """Y[m, n] = sum_k X[m, k] scales[n, k // group] (q[n, k] - zeros[n, k // group])
    on the current stream, with 4-bit q packed two to a byte along K, low half
    first (``w``: uint8, N x ceil(K / 2)).  X is M x K float32, float16 or
    bfloat16, and so is Y; ``scales`` is N x ceil(K / group) of any of these
    types, ``zeros`` uint8 of that shape (None: 8).  ``group`` is a power of
    two, 32 or more.  Sums are kept in float32 and rounded once."""
    _FLOATS or _use_torch()
    group = _q4_group(group)
    ldx = _rows(X, "X", None, _FLOATS)
    M, K = X.shape
    N = _dim(w, 0)
    ldw, lds, ldz = _q4_weight(w, scales, zeros, N, K, group, "q4")
    if out is None:
        Y, ldy = torch.empty((M, N), dtype=X.dtype, device=X.device), max(N, 1)
    else:
        Y, ldy = out, _rows(out, "out", (M, N), (X.dtype,))
    _call(load().sgemm_q4, "sgemm_q4", X, (w, scales, zeros, Y), _FLOATS[X.dtype],
          _FLOATS[scales.dtype], M, N, K, X.data_ptr(), ldx, w.data_ptr(), ldw, group,
          scales.data_ptr(), lds, zeros.data_ptr() if zeros is not None else None, ldz, Y.data_ptr(),
          ldy)
    return Y


def q4_glu(X, gate_w, gate_scales, up_w, up_scales, gate_zeros=None, up_zeros=None, group=128,
           act="silu", out=None):
    """The gated feed-forward block with 4-bit weights, H = act(G) * U, where G
    and U are q4_matmul's products of X with the gate and the up weights (the
    same shapes, types and row strides); G and U stay in float32."""
    _FLOATS or _use_torch()
    a, group = _act_id(act), _q4_group(group)
    ldx = _rows(X, "X", None, _FLOATS)
    M, K = X.shape
    F = _dim(gate_w, 0)
    if (gate_zeros is None) != (up_zeros is None):
        raise ValueError("gate_zeros and up_zeros must be given together")
    ld = _q4_weight(gate_w, gate_scales, gate_zeros, F, K, group, "gate")
    if _q4_weight(up_w, up_scales, up_zeros, F, K, group, "up") != ld:
        raise ValueError("gate and up weights must have the same row strides")
    if gate_scales.dtype != up_scales.dtype:
        raise TypeError("gate and up scales must have the same type")
    if out is None:
        H, ldh = torch.empty((M, F), dtype=X.dtype, device=X.device), max(F, 1)
    else:
        H, ldh = out, _rows(out, "out", (M, F), (X.dtype,))
    _call(load().sgemm_q4_glu, "sgemm_q4_glu", X,
          (gate_w, gate_scales, up_w, up_scales, gate_zeros, up_zeros, H), a, _FLOATS[X.dtype],
          _FLOATS[gate_scales.dtype], M, F, K, X.data_ptr(), ldx, gate_w.data_ptr(), up_w.data_ptr(),
          ld[0], group, gate_scales.data_ptr(), up_scales.data_ptr(), ld[1],
          gate_zeros.data_ptr() if gate_zeros is not None else None,
          up_zeros.data_ptr() if up_zeros is not None else None, ld[2], H.data_ptr(), ldh)
    return H


def copy_f32(dst, src):
    """dst[:] = src[:] (float32 GPU tensors, contiguous) with the copy probe."""
    n = src.numel()
    if dst.numel() != n or not (dst.is_contiguous() and src.is_contiguous()):
        raise ValueError("copy needs contiguous tensors of equal size")
    st = load().sgemm_copy_f32(dst.data_ptr(), src.data_ptr(), n, _stream_handle(src.device))
    if st != 0:
        raise SgemmError(st, "sgemm_copy_f32")
    return dst


def copy_f32_launch(dst, src, block: int, grid: int):
    """The copy probe with an explicit workgroup size and count."""
    n = src.numel()
    if dst.numel() != n or not (dst.is_contiguous() and src.is_contiguous()):
        raise ValueError("copy needs contiguous tensors of equal size")
    st = load().sgemm_copy_f32_launch(dst.data_ptr(), src.data_ptr(), n, block, grid,
                                      _stream_handle(src.device))
    if st != 0:
        raise SgemmError(st, "sgemm_copy_f32_launch")
    return dst


VALU_CHAINS = 32
MFMA_WAVES_PER_BLOCK = 4
MFMA_ACC_PER_WAVE = 4


def probe_valu(blocks: int, block: int, iters: int, x: float, y: float, out=None):
    """Run the VALU multiply-add probe; returns the (blocks*block, VALU_CHAINS)
    output tensor (final chain values).  Work: blocks*block*iters*VALU_CHAINS*2
    FLOP."""
    import torch
    if out is None:
        out = torch.empty((blocks * block, VALU_CHAINS), dtype=torch.float32, device="cuda")
    elif out.numel() < blocks * block * VALU_CHAINS or not out.is_contiguous():
        raise ValueError("out too small or not contiguous")
    st = load().sgemm_probe_valu_f32(out.data_ptr(), blocks, block, iters, x, y,
                                     _stream_handle(out.device))
    if st != 0:
        raise SgemmError(st, "sgemm_probe_valu_f32")
    return out


def probe_mfma(a_vals, b_vals, blocks: int, iters: int, out=None):
    """Run the matrix-core probe; returns (blocks*4, 4, 32, 32) accumulators.
    Work: blocks*16*iters*4096 FLOP."""
    import torch
    n = blocks * MFMA_WAVES_PER_BLOCK * MFMA_ACC_PER_WAVE
    if out is None:
        out = torch.empty((blocks * MFMA_WAVES_PER_BLOCK, MFMA_ACC_PER_WAVE, 32, 32),
                          dtype=torch.float32, device="cuda")
    elif out.numel() < n * 1024 or not out.is_contiguous():
        raise ValueError("out too small or not contiguous")
    for v in (a_vals, b_vals):
        if v.numel() != 64 or v.dtype != torch.float32 or v.device.type != "cuda" or not v.is_contiguous():
            raise ValueError("a_vals and b_vals must be 64 contiguous float32 GPU values")
    st = load().sgemm_probe_mfma_f32(out.data_ptr(), a_vals.data_ptr(), b_vals.data_ptr(), blocks,
                                     iters, _stream_handle(out.device))
    if st != 0:
        raise SgemmError(st, "sgemm_probe_mfma_f32")
    return out
