"""Thin ctypes binding of ``libtp.so`` (declared in include/tp.h).

Argument marshalling only: torch tensors are passed as raw device pointers,
the caller's current CUDA stream as the stream handle, and every status code
is turned into a ``TPError``.  All computation happens in the library's CUDA
kernels; there is no fallback — if the library has not been built, ``lib()``
raises.
"""

import ctypes
import importlib.util
import os
import warnings


class _Torch:
    """torch, imported when it is first used: what counts bytes and operations
    needs only ctypes."""

    def __getattr__(self, name):
        global torch
        import torch
        return getattr(torch, name)


torch = _Torch()
PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtp.so")

F32, BF16, FP8 = 0, 1, 2
GELU, SWIGLU = 0, 1
FUSED, MATERIALISED, OVERLAP, SP = 0, 1, 2, 3
SCOPE_MLP, SCOPE_ATTN, SCOPE_LAYER = 0, 1, 2
FP8_ROW, FP8_BLOCK = 0, 1
FP8_FORMS = ("thin", "narrow", "wide")

STATUS = {0: "TP_OK", 1: "TP_ERR_NULL", 2: "TP_ERR_SHAPE", 3: "TP_ERR_DTYPE",
          4: "TP_ERR_WORKSPACE", 5: "TP_ERR_UNSUPPORTED", 6: "TP_ERR_CUDA",
          7: "TP_ERR_DEVICE_TIMEOUT", 8: "TP_ERR_ARG", 9: "TP_ERR_RANGE"}


class TPError(RuntimeError):
    def __init__(self, code, where, detail=""):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}{detail}")


class MlpDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("h", ctypes.c_int64),
                ("h_ffn", ctypes.c_int64), ("n", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("mode", ctypes.c_int32), ("dropout_p", ctypes.c_float),
                ("seed", ctypes.c_uint64)]


class AttnDesc(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("s", ctypes.c_int64),
                ("h", ctypes.c_int64), ("n_q", ctypes.c_int32),
                ("n_kv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("n", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("mode", ctypes.c_int32)]


class CommReport(ctypes.Structure):
    _fields_ = [(k, ctypes.c_uint64) for k in (
        "reductions_fwd", "reductions_bwd", "payload_bytes", "ring_bytes_num",
        "ring_bytes_den", "page2_bytes", "total_payload", "total_ring_num",
        "total_page2", "sp_rs_bytes_num", "sp_ag_bytes_num", "sp_bytes_den",
        "sp_reduce_scatters", "sp_all_gathers", "sp_total_num")]


class ActDesc(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("s", ctypes.c_int64),
                ("h", ctypes.c_int64), ("h_ffn", ctypes.c_int64),
                ("n_q", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("n", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("dropout", ctypes.c_int32), ("seq_parallel", ctypes.c_int32)]


class ActReport(ctypes.Structure):
    _fields_ = [(k, ctypes.c_uint64) for k in (
        "mlp_x", "mlp_hidden", "mlp_act", "mlp_mask", "attn_x", "attn_q",
        "attn_kv", "attn_scores", "attn_lse", "attn_o", "norm_x", "norm_rstd",
        "mlp_bytes", "attn_bytes_pages", "attn_bytes_flash",
        "layer_bytes_flash")]


class LayerDesc(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("s", ctypes.c_int64),
                ("h", ctypes.c_int64), ("h_ffn", ctypes.c_int64),
                ("n_q", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("n", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("mode", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class ProfileEntry(ctypes.Structure):
    _fields_ = [("launches", ctypes.c_uint64), ("ms", ctypes.c_double),
                ("flops", ctypes.c_double), ("bytes", ctypes.c_double)]


KERNEL_FAMILIES = ["gemm_tc", "gemm_simt", "attn_fwd", "attn_bwd_dkdv",
                   "attn_bwd_dq", "reduce", "elementwise", "rmsnorm",
                   "gemm_tc_fp8", "quantize_fp8"]

_P = ctypes.c_void_p
_I64, _I32, _F, _SZ, _U64 = (ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                             ctypes.c_size_t, ctypes.c_uint64)
_MP = ctypes.POINTER(MlpDesc)
_AP = ctypes.POINTER(AttnDesc)
_LP = ctypes.POINTER(LayerDesc)
_U64P = ctypes.POINTER(ctypes.c_uint64)

# name -> (restype, argtypes); mirrors include/tp.h
SIGNATURES = {
    "tp_mlp_workspace_bytes": (_SZ, [_MP]),
    "tp_mlp_bwd_scratch_bytes": (_SZ, [_MP]),
    "tp_mlp_fwd": (_I32, [_MP, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "tp_mlp_bwd": (_I32, [_MP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                          _P, _SZ, _P]),
    "tp_attn_workspace_bytes": (_SZ, [_AP]),
    "tp_attn_bwd_scratch_bytes": (_SZ, [_AP]),
    "tp_attn_set_ds_budget": (_SZ, [_SZ]),
    "tp_attn_fwd": (_I32, [_AP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "tp_attn_bwd": (_I32, [_AP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                           _P, _P, _P, _P, _SZ, _P]),
    "tp_layer_workspace_bytes": (_SZ, [_LP]),
    "tp_layer_bwd_scratch_bytes": (_SZ, [_LP]),
    "tp_layer_fwd": (_I32, [_LP] + [_P] * 11 + [_SZ, _P]),
    "tp_layer_bwd": (_I32, [_LP] + [_P] * 21 + [_SZ, _P]),
    "tp_rmsnorm_fwd": (_I32, [_I64, _I64, _F, _I32, _P, _P, _P, _P, _P]),
    "tp_rmsnorm_bwd_scratch_bytes": (_SZ, [_I64, _I64]),
    "tp_rmsnorm_bwd": (_I32, [_I64, _I64, _F, _I32, _P, _P, _P, _P, _P, _P,
                              _P, _P, _SZ, _P]),
    "tp_rmsnorm_bwd_noalloc": (_I32, [_I64, _I64, _F, _I32, _P, _P, _P, _P,
                                      _P, _P, _P, _P]),
    "tp_comm_bytes": (_I32, [_I32, _I64, _I64, _I32, _I32,
                             ctypes.POINTER(CommReport)]),
    "tp_act_memory": (_I32, [ctypes.POINTER(ActDesc),
                             ctypes.POINTER(ActReport)]),
    "tp_quantize_fp8": (_I32, [_I64, _P, _P, _P, _P, _P]),
    "tp_gemm_fp8": (_I32, [_I64, _I64, _I64, _P, _I64, _P, _P, _I64, _P, _P,
                           _I64, _P]),
    "tp_quantize_fp8_block": (_I32, [_I32, _I32, _I64, _I64, _P, _I64] +
                              [_P, _I64, _P, _I64] * 2 + [_P]),
    "tp_swiglu_fp8_fwd": (_I32, [_I64, _I64, _P, _I64] +
                          [_P, _I64, _P, _I64] * 2 + [_P]),
    "tp_swiglu_fp8_bwd": (_I32, [_I64, _I64, _P, _I64, _P, _I64] +
                          [_P, _I64, _P, _I64] * 2 + [_P]),
    "tp_add_rmsnorm_fp8_fwd": (_I32, [_I64, _I64, _F, _P, _P, _P, _P, _P, _P,
                                      _P, _I64, _P, _I64, _P]),
    "tp_gemm_fp8_block": (_I32, [_I64, _I64, _I64] +
                          [_P, _I64, _P, _I64, _I32] * 2 +
                          [_I32, _P, _I64, _P]),
    "tp_gemm_fp8_block_form": (_I32, [_I64, _I64, _I64, _I32, _I32] +
                               [ctypes.POINTER(_I32)] * 3),
    "tp_mlp_flops": (_I32, [_MP, _U64P, _U64P]),
    "tp_attn_flops": (_I32, [_AP, _U64P, _U64P]),
    "tp_gemm": (_I32, [_I32, _I64, _I64, _I64, _P, _I64, _I32, _P, _I64, _I32,
                       _P, _I64, _P]),
    "tp_profile_enable": (_I32, [_I32]),
    "tp_profile_reset": (_I32, []),
    "tp_profile_read": (_I32, [_I32, ctypes.POINTER(ProfileEntry)]),
    "tp_device_status": (_I32, [_P]),
    "tp_status_string": (ctypes.c_char_p, [_I32]),
    "tp_launch_count": (_U64, []),
    "tp_last_cuda_error": (_I32, [ctypes.POINTER(ctypes.c_char_p)]),
    "tp_selftest_wait_timeout": (_I32, [_P]),
    "tp_num_sms": (_I32, []),
}

_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "megatron_tensor_transformer_gate_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def check(code, where):
    if code != 0:
        detail = ""
        if code == 6:   # TP_ERR_CUDA: name the CUDA error behind it
            name = ctypes.c_char_p()
            err = lib().tp_last_cuda_error(ctypes.byref(name))
            detail = f" ({err}: {(name.value or b'').decode()})"
        raise TPError(code, where, detail)


def ptr(t):
    """Device (or host) address of a tensor, or None."""
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def raw_stream(stream, dev):
    """The stream's handle, the current one of device ``dev`` if None (read
    without making a torch.cuda.Stream, which costs as much as a launch)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(dev)


def stream_handle(stream=None):
    return ctypes.c_void_p(raw_stream(stream, torch.cuda.current_device()))


def dtype_code(t):
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


# ------------------------------------------------------------ accounting --
def comm_bytes(scope, T, h, n, dtype):
    r = CommReport()
    check(lib().tp_comm_bytes(scope, T, h, n, dtype, ctypes.byref(r)),
          "tp_comm_bytes")
    return {k: getattr(r, k) for k, _ in CommReport._fields_}


def quantize_fp8(x, q, scale, amax_work, stream=None):
    """E4M3 codes of the bf16 tensor x into q (uint8, same numel); the
    per-tensor scale into the one-element fp32 tensor ``scale``."""
    check(lib().tp_quantize_fp8(x.numel(), ptr(x), ptr(q), ptr(scale),
                                ptr(amax_work), stream_handle(stream)),
          "tp_quantize_fp8")


def selftest_wait_timeout(stream=None):
    """Enqueue the kernel whose bounded wait runs out (about 2 s)."""
    check(lib().tp_selftest_wait_timeout(stream_handle(stream)),
          "tp_selftest_wait_timeout")


def gemm_fp8(qa, scale_a, qb, scale_b, C, stream=None):
    """C[M, N] = qa·qbᵀ / (scale_a·scale_b) on E4M3 codes (K-major both)."""
    M, N = C.shape
    K = qa.shape[1]
    check(lib().tp_gemm_fp8(M, N, K, ptr(qa), qa.stride(0), ptr(scale_a),
                            ptr(qb), qb.stride(0), ptr(scale_b), ptr(C),
                            C.stride(0), stream_handle(stream)),
          "tp_gemm_fp8")


# ------------------------------------------------ FP8 with a scale per block --
# A block-scaled matrix is a pair (q, s): codes q [rows, cols] (float8_e4m3fn
# or uint8, unit column stride, rows 16-byte aligned) and fp32 scales s with
# one row for each 128 columns, [⌈cols/128⌉, rows] (a scale for each row) or
# [⌈cols/128⌉, ⌈rows/128⌉] (one for each 128×128 block).
def fp8_block_empty(rows, cols, group=FP8_ROW, device="cuda"):
    """Room for a block-scaled [rows, cols] matrix: (q, s)."""
    q = torch.empty((rows, (cols + 15) // 16 * 16), dtype=torch.float8_e4m3fn,
                    device=device)[:, :cols]
    s = torch.empty(((cols + 127) // 128,
                     rows if group == FP8_ROW else (rows + 127) // 128),
                    dtype=torch.float32, device=device)
    return q, s


# The checks of a call run before every launch, which for a generated token is
# most of its time.  csrc/pycall.cpp makes them for arguments in their ordinary
# form and calls the C entry (2.7 to 4 µs a call); where it finds anything else
# it answers None, and the functions below check again and say what is wrong.
# Where it is not built for this Python and torch they make every call.
_tpcall = None   # that module, or its stand-in


class _EveryCallInPython:
    @staticmethod
    def quantize(*_):
        return None

    swiglu = swiglu_bwd = norm = gemm = quantize


def _load():
    global _tpcall
    L = lib()
    torch.Tensor   # the module links against torch's libraries as loaded
    try:
        from .build import pycall_path
        spec = importlib.util.spec_from_file_location(__package__ + "._tpcall",
                                                      pycall_path())
        fast = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(fast)
        fast.bind(*(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in
                    ("tp_quantize_fp8_block", "tp_swiglu_fp8_fwd",
                     "tp_swiglu_fp8_bwd", "tp_add_rmsnorm_fp8_fwd",
                     "tp_gemm_fp8_block")))
    except ImportError as e:
        warnings.warn("the block-scaled calls' module is not built for this "
                      f"Python and torch, each call takes longer: {e}")
        fast = _EveryCallInPython
    _tpcall = fast
    return fast


def _shape(t):
    return tuple(t.shape)


def _refuse_matrix(t, what):
    if t.dim() != 2:
        raise ValueError(f"{what}: a matrix, got {_shape(t)}")
    if not t.is_cuda:
        raise ValueError(f"{what}: not on a GPU")
    raise ValueError(f"{what}: columns must be adjacent, strides {t.stride()}")


def _matrix(t, what):
    """(rows, cols, row stride, device) of a matrix on the current device with
    adjacent columns."""
    dev = t.get_device()
    if t.dim() != 2 or dev < 0:
        _refuse_matrix(t, what)
    rows, cols = t.shape
    ld, unit = t.stride()
    if unit != 1 and cols != 1:
        _refuse_matrix(t, what)
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{what} is on cuda:{dev}, the current device is "
                         f"cuda:{torch._C._cuda_getDevice()}")
    return rows, cols, ld if rows > 1 else cols, dev


def _refuse_dense(t, what, dtype, shape, dev):
    if t.dtype != dtype:
        raise TypeError(f"{what}: {dtype}, got {t.dtype}")
    if _shape(t) != shape:
        raise ValueError(f"{what}: shape {shape}, got {_shape(t)}")
    if t.get_device() != dev:
        raise ValueError(f"{what}: on {t.device}, not cuda:{dev}")
    raise ValueError(f"{what}: dense rows, strides {t.stride()}")


def _dense(t, what, dtype, shape, dev):
    """Address of a dense tensor of this type, shape and device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or \
            not t.is_contiguous():
        _refuse_dense(t, what, dtype, shape, dev)
    return t.data_ptr()


def _refuse_pair(q, s, what, rows, cols, dev):
    if s is None:
        raise ValueError(f"{what}: codes without scales")
    if not _is_code(q):
        raise TypeError(f"{what}: E4M3 codes, got {q.dtype}")
    if s.dtype != torch.float32:
        raise TypeError(f"{what} scales: float32, got {s.dtype}")
    if _shape(q) != (rows, cols):
        raise ValueError(f"{what}: shape {(rows, cols)}, got {_shape(q)}")
    for t, w in ((q, what), (s, what + " scales")):
        if t.get_device() != dev:
            raise ValueError(f"{w}: on {t.device}, not cuda:{dev}")
        if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] != 1):
            _refuse_matrix(t, w)
    raise ValueError(f"{what} scales: {_shape(s)} for codes {(rows, cols)}")


def _is_code(q):
    return q.dtype is torch.float8_e4m3fn or q.dtype is torch.uint8


def _fp8_pair(q, s, what, rows, cols, dev):
    """(address, ldq, address of the scales, lds, group) of a block-scaled
    matrix of this shape on this device."""
    kb, rb = (cols + 127) >> 7, (rows + 127) >> 7
    if s is None or q.shape != (rows, cols) or not _is_code(q) or \
            s.dtype is not torch.float32 or q.get_device() != dev or \
            s.get_device() != dev or s.dim() != 2:
        _refuse_pair(q, s, what, rows, cols, dev)
    ld, unit = q.stride()
    lds, sunit = s.stride()
    sb, sr = s.shape
    if (unit != 1 and cols != 1) or (sunit != 1 and sr != 1) or sb != kb or \
            (sr != rows and sr != rb):
        _refuse_pair(q, s, what, rows, cols, dev)
    # a single row's stride is free: what the kernels ask for
    if rows == 1:
        ld = (cols + 15) & ~15
    return (q.data_ptr(), ld, s.data_ptr(), lds if sb > 1 else sr,
            FP8_ROW if sr == rows else FP8_BLOCK)


_NO_PAIR = (None, 0, None, 0)


def _fp8_outs(rows, cols, dev, q, s, qt, st):
    """The eight output arguments and the group of a quantizing call."""
    if qt is None:
        if q is None:
            raise ValueError("neither q nor qt given")
        a = _fp8_pair(q, s, "q", rows, cols, dev)
        return a[:4] + _NO_PAIR, a[4]
    b = _fp8_pair(qt, st, "qt", cols, rows, dev)
    if q is None:
        return _NO_PAIR + b[:4], b[4]
    a = _fp8_pair(q, s, "q", rows, cols, dev)
    # of a single row, 1×128 groups and 128×128 blocks have one layout
    ga, gb = a[4] if rows > 1 else b[4], b[4] if cols > 1 else a[4]
    if ga != gb:
        raise ValueError("q and qt have scales of different groups")
    return a[:4] + b[:4], ga


def _done(rc, where):
    """Whether _tpcall made the call (an error of it is raised)."""
    if rc:
        check(rc, where)
    return rc is not None


def quantize_fp8_block(x, q=None, s=None, qt=None, st=None, stream=None):
    """Block-scaled E4M3 codes of x (bf16 or fp32 [rows, cols]) into (q, s),
    of its transpose into (qt, st); the scales' shape says whether a scale
    belongs to 128 elements of a row or to a 128×128 block."""
    if _done((_tpcall or _load()).quantize(x, q, s, qt, st, stream),
             "tp_quantize_fp8_block"):
        return
    rows, cols, ld, dev = _matrix(x, "x")
    outs, group = _fp8_outs(rows, cols, dev, q, s, qt, st)
    check(lib().tp_quantize_fp8_block(dtype_code(x), group, rows, cols,
                                      x.data_ptr(), ld, *outs,
                                      raw_stream(stream, dev)),
          "tp_quantize_fp8_block")


def _row_group(group, what):
    if group != FP8_ROW:
        raise ValueError(f"{what} writes a scale for each row")


def _gate_up(gu):
    T, f2, ld, dev = _matrix(gu, "gu")
    if gu.dtype is not torch.bfloat16:
        raise TypeError(f"gu: bfloat16, got {gu.dtype}")
    if f2 % 2:
        raise ValueError(f"gu: an even number of columns, got {f2}")
    return T, f2 // 2, ld, dev


def swiglu_fp8_fwd(gu, q=None, s=None, qt=None, st=None, stream=None):
    """Codes of SiLU(G)⊙U ([T, f]) into (q, s), of its transpose into
    (qt, st); gu is [G | U], bf16 [T, 2f]."""
    if _done((_tpcall or _load()).swiglu(gu, q, s, qt, st, stream),
             "tp_swiglu_fp8_fwd"):
        return
    T, f, ld, dev = _gate_up(gu)
    outs, group = _fp8_outs(T, f, dev, q, s, qt, st)
    if group != FP8_ROW and T > 1:
        _row_group(group, "swiglu_fp8_fwd")
    check(lib().tp_swiglu_fp8_fwd(T, f, gu.data_ptr(), ld, *outs,
                                  raw_stream(stream, dev)),
          "tp_swiglu_fp8_fwd")


def swiglu_fp8_bwd(dA, gu, q=None, s=None, qt=None, st=None, stream=None):
    """Codes of [dG | dU] ([T, 2f]) into (q, s), of its transpose into
    (qt, st), from dA (bf16 [T, f]) and the forward's gu."""
    if _done((_tpcall or _load()).swiglu_bwd(dA, gu, q, s, qt, st, stream),
             "tp_swiglu_fp8_bwd"):
        return
    T, f, ld, dev = _gate_up(gu)
    rows, cols, ldda, _ = _matrix(dA, "dA")
    if dA.dtype is not torch.bfloat16:
        raise TypeError(f"dA: bfloat16, got {dA.dtype}")
    if rows != T or cols != f:
        raise ValueError(f"dA: shape {(T, f)}, got {(rows, cols)}")
    outs, group = _fp8_outs(T, 2 * f, dev, q, s, qt, st)
    if group != FP8_ROW and T > 1:
        _row_group(group, "swiglu_fp8_bwd")
    check(lib().tp_swiglu_fp8_bwd(T, f, dA.data_ptr(), ldda, gu.data_ptr(),
                                  ld, *outs, raw_stream(stream, dev)),
          "tp_swiglu_fp8_bwd")


def add_rmsnorm_fp8_fwd(x, r, gamma, x1, q, s, rstd, y=None, eps=1e-5,
                        stream=None):
    """x1 = x + r (r None: x1 is x and may be None), the codes of
    RMSNorm(x1)·γ into (q, s), rstd [T] fp32, and y (bf16, optional); x1 may
    be x or r."""
    if _done((_tpcall or _load()).norm(x, r, gamma, x1, q, s, rstd, y, eps,
                                       stream), "tp_add_rmsnorm_fp8_fwd"):
        return
    T, h, _, dev = _matrix(x, "x")
    bf16, shape = torch.bfloat16, (T, h)
    px = _dense(x, "x", bf16, shape, dev)
    pr = None if r is None else _dense(r, "r", bf16, shape, dev)
    p1 = None if x1 is None else _dense(x1, "x1", bf16, shape, dev)
    py = None if y is None else _dense(y, "y", bf16, shape, dev)
    pg = _dense(gamma, "gamma", bf16, (h,), dev)
    prs = _dense(rstd, "rstd", torch.float32, (T,), dev)
    if p1 is None and pr is not None:
        raise ValueError("x1: where the sum with r goes")
    pq, ldq, ps, lds, group = _fp8_pair(q, s, "q", T, h, dev)
    if group != FP8_ROW and T > 1:
        _row_group(group, "add_rmsnorm_fp8_fwd")
    check(lib().tp_add_rmsnorm_fp8_fwd(T, h, eps, px, pr, pg, p1, py, prs, pq,
                                       ldq, ps, lds, raw_stream(stream, dev)),
          "tp_add_rmsnorm_fp8_fwd")


def gemm_fp8_block(qa, sa, qb, sb, C, stream=None):
    """C[M, N] (bf16 or fp32) = A·Bᵀ of the block-scaled A = (qa, sa) [M, K]
    and B = (qb, sb) [N, K].  The K blocks' sums are added in an order fixed by
    the sizes (gemm_fp8_block_form): a row's last bits may differ between
    batches of different sizes."""
    if _done((_tpcall or _load()).gemm(qa, sa, qb, sb, C, stream),
             "tp_gemm_fp8_block"):
        return
    M, N, ldc, dev = _matrix(C, "C")
    K = qa.shape[-1]
    pa, lda, psa, ldsa, ga = _fp8_pair(qa, sa, "qa", M, K, dev)
    pb, ldb, psb, ldsb, gb = _fp8_pair(qb, sb, "qb", N, K, dev)
    check(lib().tp_gemm_fp8_block(M, N, K, pa, lda, psa, ldsa, ga, pb, ldb,
                                  psb, ldsb, gb, dtype_code(C), C.data_ptr(),
                                  ldc, raw_stream(stream, dev)),
          "tp_gemm_fp8_block")


def gemm_fp8_block_form(M, N, K, b_group=FP8_BLOCK, sms=0):
    """(form, rows of A a tile, parts of K) that gemm_fp8_block takes for these
    sizes on a device of ``sms`` SMs (0: the current one's)."""
    out = [_I32() for _ in range(3)]
    check(lib().tp_gemm_fp8_block_form(M, N, K, b_group, sms,
                                       *map(ctypes.byref, out)),
          "tp_gemm_fp8_block_form")
    return FP8_FORMS[out[0].value], out[1].value, out[2].value


def act_memory(b, s, h, h_ffn, n_q, n_kv, d, n, dtype=BF16, act=SWIGLU,
               dropout=False, seq_parallel=False):
    """Saved activations per rank (elements by tensor, bytes by block)."""
    r = ActReport()
    desc = ActDesc(b, s, h, h_ffn, n_q, n_kv, d, n, dtype, act, int(dropout),
                   int(seq_parallel))
    check(lib().tp_act_memory(ctypes.byref(desc), ctypes.byref(r)),
          "tp_act_memory")
    return {k: getattr(r, k) for k, _ in ActReport._fields_}


def mlp_flops(desc):
    f, b = ctypes.c_uint64(), ctypes.c_uint64()
    check(lib().tp_mlp_flops(ctypes.byref(desc), ctypes.byref(f),
                             ctypes.byref(b)), "tp_mlp_flops")
    return f.value, b.value


def attn_flops(desc):
    f, b = ctypes.c_uint64(), ctypes.c_uint64()
    check(lib().tp_attn_flops(ctypes.byref(desc), ctypes.byref(f),
                              ctypes.byref(b)), "tp_attn_flops")
    return f.value, b.value


# ------------------------------------------------------------------ GEMM --
def gemm(A, B, C, a_mn_major=False, b_mn_major=False, stream=None):
    """C[M, N] = A·Bᵀ with the operand layouts of tp_gemm."""
    M, N = C.shape
    K = A.shape[0] if a_mn_major else A.shape[1]
    check(lib().tp_gemm(dtype_code(C), M, N, K, ptr(A), A.stride(0),
                        int(a_mn_major), ptr(B), B.stride(0), int(b_mn_major),
                        ptr(C), C.stride(0), stream_handle(stream)),
          "tp_gemm")


# ------------------------------------------------------------------- MLP --
def mlp_desc(T, h, h_ffn, n, dtype=BF16, act=GELU, mode=FUSED, dropout_p=0.0,
             seed=0):
    return MlpDesc(T, h, h_ffn, n, dtype, act, mode, dropout_p, seed)


def mlp_workspace_bytes(desc):
    return lib().tp_mlp_workspace_bytes(ctypes.byref(desc))


def mlp_bwd_scratch_bytes(desc):
    return lib().tp_mlp_bwd_scratch_bytes(ctypes.byref(desc))


def mlp_fwd(desc, X, W1, W2, Out, ws, b1=None, b2=None, R=None, stream=None):
    check(lib().tp_mlp_fwd(ctypes.byref(desc), ptr(X), ptr(W1), ptr(b1),
                           ptr(W2), ptr(b2), ptr(R), ptr(Out), ptr(ws),
                           ws.numel() * ws.element_size(),
                           stream_handle(stream)), "tp_mlp_fwd")


def mlp_bwd(desc, dOut, X, W1, W2, ws, dX, dW1, dW2, scratch, db1=None,
            db2=None, dres=None, stream=None):
    check(lib().tp_mlp_bwd(ctypes.byref(desc), ptr(dOut), ptr(X), ptr(W1),
                           ptr(W2), ptr(ws), ptr(dres), ptr(dX), ptr(dW1),
                           ptr(db1), ptr(dW2), ptr(db2), ptr(scratch),
                           scratch.numel() * scratch.element_size(),
                           stream_handle(stream)), "tp_mlp_bwd")


# ------------------------------------------------------------- attention --
def attn_desc(b, s, h, n_q, n_kv, d, n, dtype=BF16, causal=True, mode=FUSED):
    return AttnDesc(b, s, h, n_q, n_kv, d, n, dtype, int(causal), mode)


def attn_workspace_bytes(desc):
    return lib().tp_attn_workspace_bytes(ctypes.byref(desc))


def attn_bwd_scratch_bytes(desc):
    return lib().tp_attn_bwd_scratch_bytes(ctypes.byref(desc))


def attn_set_ds_budget(nbytes):
    """Bound on the attention backward's dS tile bytes per pass (0 = the
    default); returns the previous bound."""
    return lib().tp_attn_set_ds_budget(nbytes)


def attn_fwd(desc, X, Wq, Wk, Wv, Wo, Out, ws, bo=None, R=None, stream=None):
    check(lib().tp_attn_fwd(ctypes.byref(desc), ptr(X), ptr(Wq), ptr(Wk),
                            ptr(Wv), ptr(Wo), ptr(bo), ptr(R), ptr(Out),
                            ptr(ws), ws.numel() * ws.element_size(),
                            stream_handle(stream)), "tp_attn_fwd")


def attn_bwd(desc, dOut, X, Wq, Wk, Wv, Wo, ws, dX, dWq, dWk, dWv, dWo,
             scratch, dbo=None, dres=None, stream=None):
    check(lib().tp_attn_bwd(ctypes.byref(desc), ptr(dOut), ptr(X), ptr(Wq),
                            ptr(Wk), ptr(Wv), ptr(Wo), ptr(ws), ptr(dres),
                            ptr(dX), ptr(dWq), ptr(dWk), ptr(dWv), ptr(dWo),
                            ptr(dbo), ptr(scratch),
                            scratch.numel() * scratch.element_size(),
                            stream_handle(stream)), "tp_attn_bwd")


# --------------------------------------------------------------- RMSNorm --
# ----------------------------------------------------------------- layer --
def layer_desc(b, s, h, h_ffn, n_q, n_kv, d, n, dtype=BF16, mode=FUSED,
               eps=1e-5):
    return LayerDesc(b, s, h, h_ffn, n_q, n_kv, d, n, dtype, mode, eps)


def layer_workspace_bytes(desc):
    return lib().tp_layer_workspace_bytes(ctypes.byref(desc))


def layer_bwd_scratch_bytes(desc):
    return lib().tp_layer_bwd_scratch_bytes(ctypes.byref(desc))


def layer_fwd(desc, x, P, out, ws, stream=None):
    """out = x1 + MLP(RMSNorm₂(x1)), x1 = x + Attn(RMSNorm₁(x)); P holds g1,
    Wq, Wk, Wv, Wo, g2, W1, W2."""
    check(lib().tp_layer_fwd(
        ctypes.byref(desc), ptr(x), *(ptr(P[k]) for k in
                                      ("g1", "Wq", "Wk", "Wv", "Wo", "g2",
                                       "W1", "W2")),
        ptr(out), ptr(ws), ws.numel() * ws.element_size(),
        stream_handle(stream)), "tp_layer_fwd")


def layer_bwd(desc, dout, x, P, ws, grads, scratch, stream=None):
    """grads: dX, dg1, dWq, dWk, dWv, dWo, dg2, dW1, dW2 (overwritten)."""
    names = ("g1", "Wq", "Wk", "Wv", "Wo", "g2", "W1", "W2")
    check(lib().tp_layer_bwd(
        ctypes.byref(desc), ptr(dout), ptr(x), *(ptr(P[k]) for k in names),
        ptr(ws), ptr(grads["dX"]), *(ptr(grads["d" + k]) for k in names),
        ptr(scratch), scratch.numel() * scratch.element_size(),
        stream_handle(stream)), "tp_layer_bwd")


def rmsnorm_fwd(x, gamma, y, rstd, eps=1e-5, stream=None):
    T, h = x.shape
    check(lib().tp_rmsnorm_fwd(T, h, eps, dtype_code(x), ptr(x), ptr(gamma),
                               ptr(y), ptr(rstd), stream_handle(stream)),
          "tp_rmsnorm_fwd")


def rmsnorm_bwd_scratch_bytes(T, h):
    return lib().tp_rmsnorm_bwd_scratch_bytes(T, h)


def rmsnorm_bwd(dy, x, gamma, rstd, dx, dgamma, scratch, dres=None, eps=1e-5,
                stream=None):
    T, h = x.shape
    check(lib().tp_rmsnorm_bwd(T, h, eps, dtype_code(x), ptr(dy), ptr(x),
                               ptr(gamma), ptr(rstd), ptr(dres), ptr(dx),
                               ptr(dgamma), ptr(scratch),
                               scratch.numel() * scratch.element_size(),
                               stream_handle(stream)), "tp_rmsnorm_bwd")


def rmsnorm_bwd_noalloc(dy, x, gamma, rstd, dx, dgamma, dres=None, eps=1e-5,
                        stream=None):
    """RMSNorm backward without caller scratch (see tp_rmsnorm_bwd_noalloc)."""
    T, h = x.shape
    check(lib().tp_rmsnorm_bwd_noalloc(T, h, eps, dtype_code(x), ptr(dy),
                                       ptr(x), ptr(gamma), ptr(rstd),
                                       ptr(dres), ptr(dx), ptr(dgamma),
                                       stream_handle(stream)),
          "tp_rmsnorm_bwd_noalloc")


def device_status(stream=None):
    check(lib().tp_device_status(stream_handle(stream)), "tp_device_status")


def launch_count():
    return lib().tp_launch_count()


# ------------------------------------------------------------- profiling --
def profile_enable(max_launches):
    check(lib().tp_profile_enable(max_launches), "tp_profile_enable")


def profile_reset():
    check(lib().tp_profile_reset(), "tp_profile_reset")


def profile_read():
    """{family: {launches, ms, flops, bytes}} for every kernel family."""
    out = {}
    for i, name in enumerate(KERNEL_FAMILIES):
        e = ProfileEntry()
        check(lib().tp_profile_read(i, ctypes.byref(e)), "tp_profile_read")
        out[name] = {"launches": e.launches, "ms": e.ms, "flops": e.flops,
                     "bytes": e.bytes}
    return out
