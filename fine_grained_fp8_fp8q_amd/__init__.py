"""fine_grained_fp8_fp8q_amd -- fine-grained FP8 (E4M3) linear-layer hot path
for AMD Instinct MI355X (gfx950).

Thin ctypes binding over the C ABI of ``libfp8q.so`` (declared in
``include/fp8q.h``).  Every step of the path runs in the library's HIP
kernels; this module only checks tensor types, allocates outputs with torch
(device memory and the current stream are torch's) and marshals arguments.
There is no fallback: if the library is missing or the device is not gfx950
the calls raise.

Functions (names follow the C ABI without the ``fp8q_`` prefix):

* ``quantize_act(x, tile_axis="row"|"token_t", scale_mode="free"|"pow2")``
  -> (codes uint8, scales float32)
* ``quantize_weight(w, scale_mode="free"|"pow2")`` -> (codes, scales)
* ``quantize_linear(x, w, act_scale_mode=..., weight_scale_mode=...)`` ->
  (a_codes, a_scales, w_codes, w_scales) in one launch
* ``gemm(a, a_scales, w, w_scales, out_dtype=torch.bfloat16|torch.float32)``
* ``grouped_gemm(a, a_scales, offsets, w, w_scales, out_dtype=...)``
* ``wgrad(dy_t, dy_scales, x_t, x_scales)``

  The three GEMMs call ``fp8q_gemm`` / ``fp8q_grouped_gemm`` / ``fp8q_wgrad``
  (partials at float32 grade); ``acc="fp8_mfma"``, ``"fp8_mfma_scaled"`` or
  ``"fp32_pow2"`` calls the ``_ex`` entry point with that accumulation form.
* ``gemm_quantized(a, a_scales, w, w_scales, scale_mode=...)`` -> (codes, scales)
  of C rounded to BF16 and quantized per 1x128 tile along N
* ``gather_rows(codes, scales, index)`` -> (codes, scales) of rows ``index``
* ``swiglu_quantize(x, scale_mode=..., cache=False, cache_scale_mode="pow2")``
  -> (codes, scales[, cache_codes, cache_scales])
* the expert layer around the GEMMs: ``moe_sort`` (routing table),
  ``moe_combine`` / ``moe_combine_backward`` (weighted sum of a token's
  expert rows and its gradient), ``swiglu_backward`` (from the BF16 input or
  its FP8 cache) and ``grouped_wgrad`` (every expert's weight gradient)
* between a block's linear layers: ``rmsnorm_quantize`` (residual addition,
  RMS norm and 1x128 quantization), ``rmsnorm_backward``,
  ``rmsnorm_quantize_t`` (the normalised rows in token-axis tiles, by a routing
  table's token list if given), ``moe_route`` (the router's choice of experts)
  and ``moe_route_backward``
"""

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8q.so")

OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_ALIGN, ERR_LAUNCH, ERR_DEVICE = range(6)
SCALE_FREE, SCALE_POW2 = 0, 1
OUT_F32, OUT_BF16 = 0, 1
ACC_FP32, ACC_FP8_MFMA, ACC_FP8_MFMA_SCALED, ACC_FP32_POW2 = 0, 1, 2, 3
TILE_ROW, TILE_TOKEN_T = 0, 1
INDEX_I32, INDEX_I64 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP_TWO = 0, 1

SYMBOLS = ("fp8q_quantize_act", "fp8q_quantize_weight", "fp8q_quantize_linear", "fp8q_quantize_weight_t", "fp8q_gemm",
           "fp8q_gemm_ex", "fp8q_gemm_quantized", "fp8q_grouped_gemm", "fp8q_grouped_gemm_ex", "fp8q_wgrad",
           "fp8q_wgrad_ex", "fp8q_gather_rows", "fp8q_swiglu_quantize", "fp8q_moe_sort", "fp8q_moe_combine",
           "fp8q_moe_combine_backward", "fp8q_swiglu_backward", "fp8q_grouped_wgrad", "fp8q_grouped_wgrad_ex",
           "fp8q_rmsnorm_quantize", "fp8q_rmsnorm_backward", "fp8q_rmsnorm_quantize_t", "fp8q_moe_route",
           "fp8q_moe_route_backward", "fp8q_rmsnorm_backward_workspace",
           "fp8q_moe_sort_workspace", "fp8q_set_gemm_small_limit", "fp8q_status_string")

_lib = None


class Fp8qError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def load_library(path=None):
    """Load libfp8q.so (built in place by ``build.py``) and declare signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m fine_grained_fp8_fp8q_amd.build`")
    lib = ctypes.CDLL(p)
    vp, i64, i32, ip = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    lib.fp8q_quantize_act.argtypes = [vp, i64, i64, i64, ip, ip, vp, i64, vp, vp]
    lib.fp8q_quantize_weight.argtypes = [vp, i64, i64, i64, ip, vp, i64, vp, vp]
    lib.fp8q_quantize_linear.argtypes = [vp, i64, i64, i64, ip, vp, i64, vp, vp, i64, i64, ip, vp, i64, vp, vp]
    lib.fp8q_quantize_weight_t.argtypes = [vp, i64, i64, i64, ip, vp, i64, vp, vp, i64, vp, vp]
    lib.fp8q_gemm.argtypes = [vp, vp, vp, vp, i64, i64, i64, ip, vp, i64, vp]
    lib.fp8q_gemm_ex.argtypes = [vp, vp, vp, vp, i64, i64, i64, ip, ip, vp, i64, vp]
    lib.fp8q_gemm_quantized.argtypes = [vp, vp, vp, vp, i64, i64, i64, ip, ip, vp, i64, vp, vp]
    lib.fp8q_grouped_gemm.argtypes = [vp, vp, vp, i32, i64, vp, vp, i64, i64, ip, vp, i64, vp]
    lib.fp8q_grouped_gemm_ex.argtypes = [vp, vp, vp, i32, i64, vp, vp, i64, i64, ip, ip, vp, i64, vp]
    lib.fp8q_wgrad.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, i64, vp]
    lib.fp8q_wgrad_ex.argtypes = [vp, vp, vp, vp, i64, i64, i64, ip, vp, i64, vp]
    lib.fp8q_gather_rows.argtypes = [vp, i64, i64, i64, vp, vp, i64, vp, i64, vp, vp]
    lib.fp8q_swiglu_quantize.argtypes = [vp, i64, i64, i64, ip, vp, i64, vp, ip, vp, i64, vp, vp]
    lib.fp8q_moe_sort.argtypes = [vp, ip, i64, i64, i64, i64, i32, i32, i64, vp, vp, vp, vp, i64, vp]
    lib.fp8q_moe_combine.argtypes = [vp, ip, i64, i64, i64, vp, vp, i64, i64, ip, vp, i64, vp]
    lib.fp8q_moe_combine_backward.argtypes = [vp, ip, i64, i64, i64, vp, ip, i64, i64, vp, vp, i64, vp, vp, i64, ip,
                                              vp, i64, vp, vp, vp]
    lib.fp8q_swiglu_backward.argtypes = [vp, vp, i64, i64, i64, vp, i64, vp, i64, ip, vp, i64, vp, vp, i64, vp]
    lib.fp8q_grouped_wgrad.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, i64, vp]
    lib.fp8q_grouped_wgrad_ex.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, ip, vp, i64, vp]
    f64 = ctypes.c_double
    lib.fp8q_rmsnorm_quantize.argtypes = [vp, ip, i64, i64, i64, vp, ip, i64, vp, i64, vp, ip, f64, vp, i64, ip, vp, i64, vp, vp, vp]
    lib.fp8q_rmsnorm_backward.argtypes = [vp, ip, i64, i64, i64, vp, ip, i64, vp, vp, ip, vp, i64, vp, ip, i64, ip, vp, i64, vp, vp,
                                          vp, i64, vp]
    lib.fp8q_rmsnorm_quantize_t.argtypes = [vp, ip, i64, i64, i64, vp, vp, ip, vp, i64, ip, vp, i64, vp, vp]
    lib.fp8q_moe_route.argtypes = [vp, ip, i64, i64, i64, vp, ip, i32, i32, ip, i64, ip, f64, ip, vp, vp, vp, vp, vp]
    lib.fp8q_moe_route_backward.argtypes = [vp, vp, ip, i64, i64, vp, ip, i64, i64, ip, ip, f64, vp, vp, ip, i64, vp]
    lib.fp8q_rmsnorm_backward_workspace.argtypes = [i64, i64]
    lib.fp8q_rmsnorm_backward_workspace.restype = i64
    lib.fp8q_moe_sort_workspace.argtypes = [i64, i64, i32]
    lib.fp8q_moe_sort_workspace.restype = i64
    lib.fp8q_set_gemm_small_limit.argtypes = [i64]
    lib.fp8q_set_gemm_small_limit.restype = i64
    for name in SYMBOLS[:-4]:
        getattr(lib, name).restype = ctypes.c_int
    lib.fp8q_status_string.argtypes = [ctypes.c_int]
    lib.fp8q_status_string.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


def status_string(status):
    return load_library().fp8q_status_string(int(status)).decode()


def _check(status, where):
    if status != OK:
        raise Fp8qError(status, where)


# ------------------------------------------------------- torch plumbing ----

def _torch():
    import torch
    return torch


def _stream(t):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None and t.numel() else ctypes.c_void_p(0)


def _need(t, dtype, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _row_major(t, name):
    """Row stride of a 2-D tensor with contiguous rows (any stride is fine for
    an empty one: nothing is read through it; a single column has no column
    stride)."""
    if t.dim() != 2 or (t.numel() and t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")
    return t.stride(0) if t.numel() else max(t.shape[1], 1)


def _pad16(n):
    return (n + 15) // 16 * 16


_SCALE_MODES = {"free": SCALE_FREE, "pow2": SCALE_POW2}


def _scale_mode(mode):
    return _SCALE_MODES[mode]


def _alloc_codes(rows, cols, device):
    """uint8 [rows, cols] view of a buffer whose row stride is a multiple of 16."""
    torch = _torch()
    buf = torch.empty((rows, _pad16(max(cols, 1))), dtype=torch.uint8, device=device)
    return buf[:, :cols]


# ------------------------------------------------------------ the calls ----

def quantize_act(x, tile_axis="row", scale_mode="free"):
    """BF16 [rows, cols] -> (codes, scales).

    tile_axis="row": 1x128 tiles along cols; codes [rows, cols],
    scales [rows, ceil(cols/128)].  tile_axis="token_t": 128x1 tiles along
    rows; codes [cols, rows] (transposed), scales [cols, ceil(rows/128)].
    """
    torch = _torch()
    _need(x, torch.bfloat16, "x")
    ldx = _row_major(x, "x")
    rows, cols = x.shape
    axis = {"row": TILE_ROW, "token_t": TILE_TOKEN_T}[tile_axis]
    if axis == TILE_ROW:
        codes = _alloc_codes(rows, cols, x.device)
        scales = torch.empty((rows, (cols + 127) // 128), dtype=torch.float32, device=x.device)
    else:
        codes = _alloc_codes(cols, rows, x.device)
        scales = torch.empty((cols, (rows + 127) // 128), dtype=torch.float32, device=x.device)
    st = load_library().fp8q_quantize_act(_ptr(x), rows, cols, ldx, axis, _scale_mode(scale_mode),
                                          _ptr(codes), codes.stride(0) if codes.numel() else 16,
                                          _ptr(scales), _stream(x))
    _check(st, "fp8q_quantize_act")
    return codes, scales


def quantize_weight(w, scale_mode="free"):
    """BF16 [N, K] -> (codes [N, K], scales [ceil(N/128), ceil(K/128)])."""
    torch = _torch()
    _need(w, torch.bfloat16, "w")
    ldw = _row_major(w, "w")
    n, k = w.shape
    codes = _alloc_codes(n, k, w.device)
    scales = torch.empty(((n + 127) // 128, (k + 127) // 128), dtype=torch.float32, device=w.device)
    st = load_library().fp8q_quantize_weight(_ptr(w), n, k, ldw, _scale_mode(scale_mode), _ptr(codes),
                                             codes.stride(0) if codes.numel() else 16, _ptr(scales),
                                             _stream(w))
    _check(st, "fp8q_quantize_weight")
    return codes, scales


def quantize_linear(x, w, act_scale_mode="free", weight_scale_mode="free"):
    """Both operands of a linear layer in one launch: the activation x
    [M, K] per 1x128 tile and the weight w [N, K] per 128x128 block, bit for
    bit ``quantize_act(x)`` and ``quantize_weight(w)``."""
    torch = _torch()
    _need(x, torch.bfloat16, "x")
    _need(w, torch.bfloat16, "w")
    ldx = _row_major(x, "x")
    ldw = _row_major(w, "w")
    m, k = x.shape
    n = w.shape[0]
    if w.shape[1] != k:
        raise ValueError("x and w must have the same K")
    nb = (k + 127) // 128
    ac = _alloc_codes(m, k, x.device)
    as_ = torch.empty((m, nb), dtype=torch.float32, device=x.device)
    wc = _alloc_codes(n, k, x.device)
    ws = torch.empty(((n + 127) // 128, nb), dtype=torch.float32, device=x.device)
    st = load_library().fp8q_quantize_linear(
        _ptr(x), m, k, ldx if x.numel() else k, _scale_mode(act_scale_mode), _ptr(ac),
        ac.stride(0) if ac.numel() else _pad16(max(k, 1)), _ptr(as_), _ptr(w), n, ldw if w.numel() else k,
        _scale_mode(weight_scale_mode), _ptr(wc), wc.stride(0) if wc.numel() else _pad16(max(k, 1)), _ptr(ws),
        _stream(x))
    _check(st, "fp8q_quantize_linear")
    return ac, as_, wc, ws


def quantize_weight_t(w, scale_mode="free", both=True):
    """BF16 [N, K] -> (codes, scales, codes_t, scales_t): the 128x128 block
    quantization of w and its transpose (codes_t [K, N], scales_t
    [ceil(K/128), ceil(N/128)]) from one pass; with both=False only the
    transposed pair is written and codes, scales are None.  The transposed
    pair is the W operand of the activation-gradient GEMM (see dgrad)."""
    torch = _torch()
    _need(w, torch.bfloat16, "w")
    ldw = _row_major(w, "w")
    n, k = w.shape
    codes = _alloc_codes(n, k, w.device) if both else None
    scales = torch.empty(((n + 127) // 128, (k + 127) // 128), dtype=torch.float32, device=w.device) \
        if both else None
    codes_t = _alloc_codes(k, n, w.device)
    scales_t = torch.empty(((k + 127) // 128, (n + 127) // 128), dtype=torch.float32, device=w.device)
    st = load_library().fp8q_quantize_weight_t(
        _ptr(w), n, k, ldw, _scale_mode(scale_mode),
        _ptr(codes) if both else None, (codes.stride(0) if codes.numel() else 16) if both else 16,
        _ptr(scales) if both else None,
        _ptr(codes_t), codes_t.stride(0) if codes_t.numel() else 16, _ptr(scales_t), _stream(w))
    _check(st, "fp8q_quantize_weight_t")
    return codes, scales, codes_t, scales_t


def _out_code(dtype):
    torch = _torch()
    if dtype == torch.bfloat16:
        return OUT_BF16
    if dtype == torch.float32:
        return OUT_F32
    raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")


def _acc_code(acc):
    """"fp32" (default; partials at float32 grade), "fp8_mfma" (partials
    formed inside the FP8 matrix core, ~14-bit alignment in groups of 8),
    "fp8_mfma_scaled" (power-of-two scales applied by the matrix core, all K
    blocks accumulated there: no promotion) or "fp32_pow2" (power-of-two
    scales applied exactly while widening to BF16, float32 grade, all K
    blocks accumulated in the BF16 matrix core: no fold)."""
    try:
        return {"fp32": ACC_FP32, "fp8_mfma": ACC_FP8_MFMA, "fp8_mfma_scaled": ACC_FP8_MFMA_SCALED,
                "fp32_pow2": ACC_FP32_POW2}[acc]
    except KeyError:
        raise ValueError('acc must be "fp32", "fp8_mfma", "fp8_mfma_scaled" or "fp32_pow2"') from None


def _contig_codes(t, name):
    torch = _torch()
    _need(t, torch.uint8, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (K-contiguous rows, no padding)")


def _contig_f32(t, name):
    torch = _torch()
    _need(t, torch.float32, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def gemm(a, a_scales, w, w_scales, out_dtype=None, out=None, acc="fp32"):
    """C[M, N] = block-scaled A . W^T from E4M3 codes and float32 scales."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    for t, n in ((a, "a"), (w, "w")):
        _contig_codes(t, n)
    for t, n in ((a_scales, "a_scales"), (w_scales, "w_scales")):
        _contig_f32(t, n)
    m, k = a.shape
    n = w.shape[0]
    if w.shape[1] != k or a_scales.shape != (m, k // 128) or w_scales.shape != ((n + 127) // 128, k // 128):
        raise ValueError("operand shapes do not match")
    c = out if out is not None else torch.empty((m, n), dtype=out_dtype, device=a.device)
    lib, code = load_library(), _acc_code(acc)
    if code == ACC_FP32:
        st = lib.fp8q_gemm(_ptr(a), _ptr(a_scales), _ptr(w), _ptr(w_scales), m, n, k, _out_code(c.dtype), _ptr(c),
                           c.stride(0), _stream(a))
    else:
        st = lib.fp8q_gemm_ex(_ptr(a), _ptr(a_scales), _ptr(w), _ptr(w_scales), m, n, k, _out_code(c.dtype), code,
                              _ptr(c), c.stride(0), _stream(a))
    _check(st, "fp8q_gemm")
    return c


def set_gemm_small_limit(max_outputs):
    """Outputs (M * N) up to which the float32-grade dense GEMM uses 32 x 32
    split-K tiles; a negative value restores the default.  Returns the
    previous setting (-1 for the default)."""
    return int(load_library().fp8q_set_gemm_small_limit(int(max_outputs)))


def gemm_quantized(a, a_scales, w, w_scales, scale_mode="free", acc="fp32"):
    """C = A . W^T (as ``gemm``) rounded to BF16 and quantized per 1x128
    tile along N in the epilogue: (codes uint8 [M, N], scales float32
    [M, ceil(N/128)]), bit for bit ``quantize_act(gemm(..., bfloat16))``."""
    torch = _torch()
    _contig_codes(a, "a")
    _contig_codes(w, "w")
    _contig_f32(a_scales, "a_scales")
    _contig_f32(w_scales, "w_scales")
    m, k = a.shape
    n = w.shape[0]
    if w.shape[1] != k:
        raise ValueError("a and w must have the same K")
    codes = _alloc_codes(m, n, a.device)
    scales = torch.empty((m, (n + 127) // 128), dtype=torch.float32, device=a.device)
    st = load_library().fp8q_gemm_quantized(_ptr(a), _ptr(a_scales), _ptr(w), _ptr(w_scales), m, n, k,
                                            _acc_code(acc), _scale_mode(scale_mode), _ptr(codes),
                                            codes.stride(0) if codes.numel() else _pad16(max(n, 1)),
                                            _ptr(scales), _stream(a))
    _check(st, "fp8q_gemm_quantized")
    return codes, scales


def dgrad(dy, dy_scales, w_t, w_t_scales, out_dtype=None, out=None, acc="fp32"):
    """dX[M, K] = dY[M, N] . W[N, K] from dY quantized in 1x128 tiles along N
    and the transposed weight pair of quantize_weight_t: the block-scaled
    GEMM with reduction axis N (fp8q_gemm on those operands)."""
    return gemm(dy, dy_scales, w_t, w_t_scales, out_dtype=out_dtype, out=out, acc=acc)


def grouped_gemm(a, a_scales, offsets, w, w_scales, out_dtype=None, out=None, acc="fp32"):
    """Per-expert block-scaled GEMM; rows [offsets[g], offsets[g+1]) use w[g].

    offsets: int32 device tensor [G+1].  Rows of the output not covered by any
    group are left as allocated (uninitialised unless ``out`` is given).
    """
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    _contig_codes(a, "a")
    _contig_codes(w, "w")
    _contig_f32(a_scales, "a_scales")
    _contig_f32(w_scales, "w_scales")
    _need(offsets, torch.int32, "offsets")
    rows_cap, k = a.shape
    g, n, kw = w.shape
    if kw != k or offsets.numel() != g + 1:
        raise ValueError("operand shapes do not match")
    c = out if out is not None else torch.empty((rows_cap, n), dtype=out_dtype, device=a.device)
    lib, code = load_library(), _acc_code(acc)
    if code == ACC_FP32:
        st = lib.fp8q_grouped_gemm(_ptr(a), _ptr(a_scales), _ptr(offsets), g, rows_cap, _ptr(w), _ptr(w_scales), n,
                                   k, _out_code(c.dtype), _ptr(c), c.stride(0), _stream(a))
    else:
        st = lib.fp8q_grouped_gemm_ex(_ptr(a), _ptr(a_scales), _ptr(offsets), g, rows_cap, _ptr(w),
                                      _ptr(w_scales), n, k, _out_code(c.dtype), code, _ptr(c), c.stride(0),
                                      _stream(a))
    _check(st, "fp8q_grouped_gemm")
    return c


def wgrad(dy_t, dy_scales, x_t, x_scales, out=None, acc="fp32"):
    """dW[Nout, Kin] = dY^T X (float32) from token-axis-quantized operands."""
    torch = _torch()
    _contig_codes(dy_t, "dy_t")
    _contig_codes(x_t, "x_t")
    _contig_f32(dy_scales, "dy_scales")
    _contig_f32(x_scales, "x_scales")
    nout, t = dy_t.shape
    kin = x_t.shape[0]
    if x_t.shape[1] != t:
        raise ValueError("operand shapes do not match")
    dw = out if out is not None else torch.empty((nout, kin), dtype=torch.float32, device=dy_t.device)
    lib, code = load_library(), _acc_code(acc)
    if code == ACC_FP32:
        st = lib.fp8q_wgrad(_ptr(dy_t), _ptr(dy_scales), _ptr(x_t), _ptr(x_scales), nout, kin, t, _ptr(dw),
                            dw.stride(0), _stream(dy_t))
    else:
        st = lib.fp8q_wgrad_ex(_ptr(dy_t), _ptr(dy_scales), _ptr(x_t), _ptr(x_scales), nout, kin, t, code,
                               _ptr(dw), dw.stride(0), _stream(dy_t))
    _check(st, "fp8q_wgrad")
    return dw


def gather_rows(codes, scales, index):
    """FP8 dispatch gather: (codes[index], scales[index]) as new tensors.

    codes uint8 [rows, cols] with contiguous rows (e.g. ``quantize_act``
    output), scales float32 [rows, ceil(cols/128)] contiguous, index int32
    [n] on the GPU.  An index outside [0, rows) yields a zero row and a zero
    scale (the library does not check indices on the host).
    """
    torch = _torch()
    _need(codes, torch.uint8, "codes")
    ldc = _row_major(codes, "codes")
    _contig_f32(scales, "scales")
    _need(index, torch.int32, "index")
    if index.dim() != 1 or not index.is_contiguous():
        raise ValueError("index must be a contiguous 1-D int32 tensor")
    rows, cols = codes.shape
    nb = (cols + 127) // 128
    if tuple(scales.shape) != (rows, nb):
        raise ValueError(f"scales must be [{rows}, {nb}], got {tuple(scales.shape)}")
    n = index.numel()
    out = _alloc_codes(n, cols, codes.device)
    out_s = torch.empty((n, nb), dtype=torch.float32, device=codes.device)
    st = load_library().fp8q_gather_rows(_ptr(codes), rows, cols, ldc if codes.numel() else cols,
                                         _ptr(scales), _ptr(index), n, _ptr(out),
                                         out.stride(0) if out.numel() else _pad16(max(cols, 1)),
                                         _ptr(out_s), _stream(codes))
    _check(st, "fp8q_gather_rows")
    return out, out_s


def swiglu_quantize(x, scale_mode="free", cache=False, cache_scale_mode="pow2"):
    """SwiGLU of x = [gate | up] (BF16 [rows, 2*inter]), quantized 1x128.

    Returns (codes [rows, inter], scales [rows, ceil(inter/128)]); with
    cache=True also the 1x128 quantization of x itself (cache_scale_mode,
    inter a multiple of 128): (codes, scales, cache_codes [rows, 2*inter],
    cache_scales [rows, 2*inter/128]).
    """
    torch = _torch()
    _need(x, torch.bfloat16, "x")
    ldx = _row_major(x, "x")
    rows, two_inter = x.shape
    if two_inter % 2:
        raise ValueError("x must have an even number of columns (gate | up)")
    inter = two_inter // 2
    codes = _alloc_codes(rows, inter, x.device)
    scales = torch.empty((rows, (inter + 127) // 128), dtype=torch.float32, device=x.device)
    cc = cs = None
    if cache:
        cc = _alloc_codes(rows, two_inter, x.device)
        cs = torch.empty((rows, (two_inter + 127) // 128), dtype=torch.float32, device=x.device)
    st = load_library().fp8q_swiglu_quantize(
        _ptr(x), rows, inter, ldx if x.numel() else two_inter, _scale_mode(scale_mode), _ptr(codes),
        codes.stride(0) if codes.numel() else _pad16(max(inter, 1)), _ptr(scales),
        _scale_mode(cache_scale_mode), _ptr(cc) if cache else ctypes.c_void_p(0),
        cc.stride(0) if cache and cc.numel() else _pad16(max(two_inter, 1)),
        _ptr(cs) if cache else ctypes.c_void_p(0), _stream(x))
    _check(st, "fp8q_swiglu_quantize")
    return (codes, scales, cc, cs) if cache else (codes, scales)


# ------------------------------------- the expert layer around the GEMMs ----

# These calls are also made for a single token, where the host's part of a
# call is most of its time: each argument is looked at once, and the stream is
# asked for by its raw handle.

def _one_device(first, *others):
    """The device of the tensors given (None among them is skipped)."""
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on one device, got {first.device} and {t.device}")
    return first.device


_stream_handle = None


def _raw_stream(dev):
    """Handle of the current stream of dev; asked for without making a
    torch.cuda.Stream of it (1.8 us) where torch has the call for that."""
    global _stream_handle
    if _stream_handle is None:
        torch = _torch()
        _stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _stream_handle(dev.index)


def _call(dev, name, *args):
    """Calls the entry point on the current stream of dev, which becomes the
    current device for the call where it is not."""
    torch = _torch()
    fn = getattr(_lib or load_library(), name)
    if dev.index == torch.cuda.current_device():
        st = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev))
    if st != OK:
        raise Fp8qError(st, name)


def _addr(t):
    """Address of a tensor's data, None (NULL) for none; 0 (NULL) for an empty one."""
    return None if t is None else t.data_ptr()


_empty_strided = None


def _new(rows, cols, dtype, dev, ld=0):
    """A new [rows, cols] tensor, dense or with the row stride given (0.3 us less than torch.empty)."""
    global _empty_strided
    if _empty_strided is None:
        _empty_strided = _torch().empty_strided
    return _empty_strided((rows, cols), (ld or cols or 1, 1), dtype=dtype, device=dev)


def _new_codes(rows, cols, dev):
    """A new uint8 [rows, cols] tensor whose row stride is a multiple of 16, and that stride."""
    ld = _pad16(max(cols, 1))
    return _new(rows, cols, _torch().uint8, dev, ld), ld


def _rows_of(t, name, dtypes):
    """(rows, columns, row stride, address) of a 2-D GPU tensor with
    contiguous rows and one of the types given.  The stride of a single row
    says nothing; one below the width (an expanded or overlapping tensor) is
    left for the library to refuse."""
    if not isinstance(t, _types()[0]):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1 and shape[0]):
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")
    rows, cols = shape
    if rows and cols:
        return rows, cols, stride[0] if rows > 1 else cols, t.data_ptr()
    return rows, cols, max(cols, 1), None


_torch_types = None


def _types():
    """(torch.Tensor, (float32, bfloat16) in the order of OUT_F32 and OUT_BF16, int32)."""
    global _torch_types
    if _torch_types is None:
        torch = _torch()
        _torch_types = torch.Tensor, (torch.float32, torch.bfloat16), torch.int32
    return _torch_types


def _pair_table(row_of, weights):
    """Checks row_of and weights: contiguous [tokens, topk]."""
    tensor, (f32, _), i32 = _types()
    if not isinstance(row_of, tensor) or row_of.dtype != i32 or row_of.dim() != 2 or not row_of.is_contiguous():
        _need(row_of, i32, "row_of")
        raise ValueError("row_of must be a contiguous int32 [tokens, topk] tensor")
    shape = row_of.shape
    if weights is not None and (not isinstance(weights, tensor) or weights.dtype != f32 or weights.shape != shape or
                                not weights.is_contiguous()):
        _contig_f32(weights, "weights")
        raise ValueError("weights must have the shape of row_of")
    return shape


def moe_sort(experts, num_hosted, first=0, align=1, rows_cap=None):
    """Routing table of the experts first .. first + num_hosted - 1 from the
    expert of every (token, choice) pair, int32 or int64 [tokens, topk].

    Returns (offsets int32 [num_hosted + 1], token int32 [rows_cap], row_of
    int32 [tokens, topk]): the groups' row ranges (padded to multiples of
    align), the token of every row (-1 for padding and behind the last group;
    ``gather_rows`` takes it as its index) and the row of every pair (-1: not
    hosted here, or dropped).  rows_cap defaults to the smallest multiple of
    align that drops no pair whatever the routing; pairs past a smaller one
    are dropped.
    """
    torch = _torch()
    tokens, topk, ld, experts_p = _rows_of(experts, "experts", (torch.int32, torch.int64))
    # (num_hosted and align go over as 32-bit integers, first as a 64-bit one)
    if not 0 <= num_hosted < 1 << 31 or not 0 <= first < 1 << 31 or not 1 <= align < 1 << 31:
        raise ValueError("num_hosted and first must not be negative, align must be at least 1, all below 2^31")
    pairs = tokens * topk
    if rows_cap is None:
        rows_cap = (pairs + num_hosted * (align - 1) + align - 1) // align * align
    elif rows_cap < 0:
        raise ValueError("rows_cap must not be negative")
    # one allocation: [offsets | token | row_of | workspace], each part 16-byte aligned
    n0, n1 = (num_hosted + 4) // 4 * 4, (rows_cap + 3) // 4 * 4
    need = (_lib or load_library()).fp8q_moe_sort_workspace(tokens, topk, num_hosted)
    n2 = (pairs + 3) // 4 * 4
    buf = torch.empty(n0 + n1 + n2 + need // 4, dtype=torch.int32, device=experts.device)
    if num_hosted == 0:  # nothing is launched: every pair is without a row
        buf.fill_(-1)
        buf[0] = 0
    p = buf.data_ptr()
    _call(experts.device, "fp8q_moe_sort", experts_p, INDEX_I64 if experts.dtype == torch.int64 else INDEX_I32, tokens,
          topk, ld, first, num_hosted, align, rows_cap, p, p + 4 * n0, p + 4 * (n0 + n1),
          p + 4 * (n0 + n1 + n2) if need else None, need)
    return (buf.as_strided((num_hosted + 1,), (1,)), buf.as_strided((rows_cap,), (1,), n0),
            buf.as_strided((tokens, topk), (topk or 1, 1), n0 + n1))


def moe_combine(y, row_of, weights=None, out_dtype=None, out=None):
    """out[t] = sum_j weights[t, j] * y[row_of[t, j]] in float32, rounded once.

    y BF16 or float32 [rows_cap, N], row_of int32 [tokens, topk] (rows outside
    y add nothing), weights float32 like row_of or None for the plain sum
    (the gradient of the row gather).  out_dtype torch.bfloat16 (default) or
    torch.float32.
    """
    types = _types()[1]
    cap, n, ld, y_p = _rows_of(y, "y", types)
    tokens, topk = _pair_table(row_of, weights)
    if out is None:
        dev = _one_device(y, row_of, weights)
        out_dtype = out_dtype or types[OUT_BF16]
        if out_dtype not in types:
            raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
        out, ldo = _new(tokens, n, out_dtype, dev), max(n, 1)
    else:
        ot, on, ldo, _ = _rows_of(out, "out", types)
        dev = _one_device(y, row_of, weights, out)
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out has another type than out_dtype")
        if (ot, on) != (tokens, n):
            raise ValueError(f"out must be [{tokens}, {n}], got [{ot}, {on}]")
    _call(dev, "fp8q_moe_combine", y_p, types.index(y.dtype), cap, n, ld, _addr(row_of), _addr(weights), tokens, topk,
          types.index(out.dtype), _addr(out), ldo)
    return out


def moe_combine_backward(dout, y, row_of, weights=None, token=None, bf16=True, quantize=False, scale_mode="free",
                         want_dweights=True):
    """Gradient of ``moe_combine`` for dout (BF16 or float32 [tokens, N]).

    Returns (dy, codes, scales, dweights), None for what was not asked for:
    dy BF16 [rows_cap, N] (bf16=True), its 1x128 quantization (quantize=True)
    and float32 dweights [tokens, topk].  token is ``moe_sort``'s: rows
    without a pair are zero; without it they are left uninitialised.
    """
    torch = _torch()
    types = _types()[1]
    dt, dn, ldd, dout_p = _rows_of(dout, "dout", types)
    cap, n, ldy, y_p = _rows_of(y, "y", types)
    tokens, topk = _pair_table(row_of, weights)
    if (dt, dn) != (tokens, n):
        raise ValueError(f"dout must be [{tokens}, {n}], got [{dt}, {dn}]")
    if token is not None:
        if not isinstance(token, torch.Tensor) or token.dtype != torch.int32 or token.shape != (cap,) or \
                not token.is_contiguous():
            _need(token, torch.int32, "token")
            raise ValueError(f"token must be a contiguous int32 tensor of {cap} rows")
    dev = _one_device(y, dout, row_of, weights, token)
    dy = _new(cap, n, torch.bfloat16, dev) if bf16 else None
    codes = scales = dw = None
    ldc = n
    if quantize:
        codes, ldc = _new_codes(cap, n, dev)
        scales = _new(cap, (n + 127) // 128, torch.float32, dev)
    if want_dweights:
        dw = _new(tokens, topk, torch.float32, dev)
    _call(dev, "fp8q_moe_combine_backward", dout_p, types.index(dout.dtype), tokens, n, ldd, y_p, types.index(y.dtype), cap,
          ldy, _addr(row_of), _addr(weights), topk, _addr(token), _addr(dy), max(n, 1), _scale_mode(scale_mode), _addr(codes), ldc,
          _addr(scales), _addr(dw))
    return dy, codes, scales, dw


def swiglu_backward(x, dy, x_scales=None, bf16=True, quantize=False, scale_mode="pow2", want_y=False):
    """Gradient of SwiGLU for x = [gate | up] and dy (BF16 [rows, inter]).

    x is BF16 [rows, 2*inter], or uint8 E4M3 codes with x_scales [rows,
    2*inter/128] (the cache of ``swiglu_quantize(cache=True)``).  Returns (dx,
    y, codes, scales), None for what was not asked for: dx BF16 [rows,
    2*inter] (bf16=True), the recomputed y BF16 [rows, inter] (want_y=True)
    and the 1x128 quantization of dx (quantize=True; inter a multiple of 128).
    """
    torch = _torch()
    rows, two_inter, ldx, x_p = _rows_of(x, "x", (torch.bfloat16,) if x_scales is None else (torch.uint8,))
    dr, inter, lddy, dy_p = _rows_of(dy, "dy", (torch.bfloat16,))
    if two_inter != 2 * inter or dr != rows:
        raise ValueError(f"x must be [rows, 2*inter] and dy [rows, inter], got [{rows}, {two_inter}] and [{dr}, {inter}]")
    if inter % 128 and (x_scales is not None or quantize):
        raise ValueError("inter must be a multiple of 128 for the FP8 cache and for a quantized dx")
    if x_scales is not None:
        _contig_f32(x_scales, "x_scales")
        if tuple(x_scales.shape) != (rows, two_inter // 128):
            raise ValueError(f"x_scales must be [{rows}, {two_inter // 128}], got {tuple(x_scales.shape)}")
    if not (bf16 or quantize or want_y):
        raise ValueError("nothing to compute: ask for bf16, quantize or want_y")
    dev = _one_device(x, dy, x_scales)
    dx = _new(rows, two_inter, torch.bfloat16, dev) if bf16 else None
    y = _new(rows, inter, torch.bfloat16, dev) if want_y else None
    codes = scales = None
    ldc = two_inter
    if quantize:
        codes, ldc = _new_codes(rows, two_inter, dev)
        scales = _new(rows, two_inter // 128, torch.float32, dev)
    _call(dev, "fp8q_swiglu_backward", x_p, _addr(x_scales), rows, inter, ldx, dy_p, lddy, _addr(dx), max(two_inter, 1),
          _scale_mode(scale_mode), _addr(codes), ldc, _addr(scales), _addr(y), max(inter, 1))
    return dx, y, codes, scales


def grouped_wgrad(dy_t, dy_scales, x_t, x_scales, offsets, out=None, acc="fp32"):
    """dW[g] = dY_g^T X_g (float32 [G, Nout, Kin]) over each group's rows of
    the sorted token axis, from token-axis-quantized operands [Nout, rows_cap]
    and [Kin, rows_cap].

    offsets: int32 device tensor [G+1] of multiples of 128 (``moe_sort`` with
    align=128).  An empty group gives zeros.
    """
    torch = _torch()
    u8, f32 = (torch.uint8,), (torch.float32,)
    nout, cap, ld0, dy_p = _rows_of(dy_t, "dy_t", u8)
    kin, xcap, ld1, x_p = _rows_of(x_t, "x_t", u8)
    if cap != xcap:
        raise ValueError("operand shapes do not match")
    if cap % 128:
        raise ValueError("the token axis must be a multiple of 128")
    sr, sc, ld2, dys_p = _rows_of(dy_scales, "dy_scales", f32)
    xr, xc, ld3, xs_p = _rows_of(x_scales, "x_scales", f32)
    nb = cap // 128
    if (sr, sc, xr, xc) != (nout, nb, kin, nb):
        raise ValueError("scales must be [rows of the codes, tokens/128]")
    if cap and (ld0, ld1, ld2, ld3) != (cap, cap, nb, nb):
        raise ValueError("codes and scales must be contiguous")
    if not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int32 or not offsets.is_cuda or \
            offsets.dim() != 1 or not offsets.is_contiguous() or not offsets.numel():
        _need(offsets, torch.int32, "offsets")
        raise ValueError("offsets must be a contiguous int32 [G+1] tensor")
    g = offsets.numel() - 1
    ldw = max(kin, 1)
    if out is None:
        dw = dy_scales.new_empty((g, nout, kin))
    else:
        dw = out
        _need(dw, torch.float32, "out")
        if tuple(dw.shape) != (g, nout, kin):
            raise ValueError(f"out must be [{g}, {nout}, {kin}], got {tuple(dw.shape)}")
        if dw.numel():
            ldw = dw.stride(1) if nout > 1 else dw.stride(0) if g > 1 else kin
            if (kin > 1 and dw.stride(2) != 1) or ldw < kin or (g > 1 and dw.stride(0) != nout * ldw):
                raise ValueError("out must have contiguous rows and matrices that follow one another")
    dev = _one_device(dy_t, dy_scales, x_t, x_scales, offsets, dw)
    code = _acc_code(acc)
    args = (dy_p, dys_p, x_p, xs_p, offsets.data_ptr(), g, cap, nout, kin)
    if code == ACC_FP32:
        _call(dev, "fp8q_grouped_wgrad", *args, _addr(dw), ldw)
    else:
        _call(dev, "fp8q_grouped_wgrad_ex", *args, code, _addr(dw), ldw)
    return dw


# ------------------------------------- between a block's linear layers ----

def _vector(t, n, dtypes, name):
    """Address of a contiguous GPU vector of n elements and one of the types given."""
    if not isinstance(t, _types()[0]):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n}")
    return t.data_ptr()


def _on16(t, addr):
    """t and its address, or those of a copy that begins on a 16-byte boundary:
    micro-batches slice per-row vectors anywhere, the library reads them from there."""
    if addr is None or addr & 15 == 0:
        return t, addr
    t = t.clone()
    return t, t.data_ptr()


def rmsnorm_quantize(x, weight, residual=None, eps=1e-6, bf16=False, quantize=True, scale_mode="free", h_out=None):
    """Residual addition, RMS norm and 1x128 quantization of its output.

    x BF16 or float32 [rows, N], weight BF16 or float32 [N].  With a residual
    (BF16 or float32 [rows, N]) h = x + residual is rounded to its type and
    normalised, without one x is.  Returns (y, codes, scales, rstd, h), None
    for what was not asked for: y BF16 [rows, N] (bf16=True), its codes and
    scales (quantize=True), rstd = 1 / rms float32 [rows], and h like residual
    (None without one), written to h_out if given, which may be residual
    itself.
    """
    torch = _torch()
    f32, b16 = types = _types()[1]
    rows, n, ldx, x_p = _rows_of(x, "x", types)
    w_p = _vector(weight, n, types, "weight")
    h, res_p, ldr, ldh, stream = None, None, n, n, OUT_BF16
    if residual is not None:
        rr, rn, ldr, res_p = _rows_of(residual, "residual", types)
        if (rr, rn) != (rows, n):
            raise ValueError(f"residual must be [{rows}, {n}], got [{rr}, {rn}]")
        stream = types.index(residual.dtype)
        if h_out is not None:
            hr, hn, ldh, _ = _rows_of(h_out, "h_out", (residual.dtype,))
            if (hr, hn) != (rows, n):
                raise ValueError(f"h_out must be [{rows}, {n}], got [{hr}, {hn}]")
            h = h_out
    elif h_out is not None:
        raise ValueError("h_out goes with a residual")
    dev = _one_device(x, weight, residual, h_out)
    if residual is not None and h is None:
        h = _new(rows, n, residual.dtype, dev)
    y = _new(rows, n, b16, dev) if bf16 else None
    codes = scales = None
    ldc = n
    if quantize:
        codes, ldc = _new_codes(rows, n, dev)
        scales = _new(rows, (n + 127) // 128, f32, dev)
    rstd = torch.empty_strided((rows,), (1,), dtype=f32, device=dev)
    _call(dev, "fp8q_rmsnorm_quantize", x_p, types.index(x.dtype), rows, n, ldx, res_p, stream, ldr, _addr(h), ldh, w_p,
          types.index(weight.dtype), eps, _addr(y), n, _scale_mode(scale_mode), _addr(codes), ldc, _addr(scales), _addr(rstd))
    return y, codes, scales, rstd, h


def rmsnorm_backward(dy, h, rstd, weight, dres=None, out_dtype=None, quantize=False, scale_mode="free", want_dx=True, want_dweight=True):
    """Gradient of the norm for dy (BF16 or float32 [rows, N]), from the h it
    normalised (x without a residual), rstd and weight of ``rmsnorm_quantize``.

    dres, the gradient that reaches h past the norm, is added to dx and has
    its type out_dtype (torch.bfloat16 by default, dres's type with one).
    Returns (dx, codes, scales, dweight), None for what was not asked for: dx
    [rows, N] (want_dx), the 1x128 quantization of its BF16 rounding
    (quantize) and float32 dweight [N] (want_dweight).  rstd may be a slice of
    a batch's anywhere (off a 16-byte boundary it is copied first).
    """
    torch = _torch()
    f32, b16 = types = _types()[1]
    rows, n, ldd, dy_p = _rows_of(dy, "dy", types)
    hr, hn, ldh, h_p = _rows_of(h, "h", types)
    if (hr, hn) != (rows, n):
        raise ValueError(f"h must be [{rows}, {n}], got [{hr}, {hn}]")
    rstd_p, w_p = _vector(rstd, rows, (f32,), "rstd"), _vector(weight, n, types, "weight")
    rstd, rstd_p = _on16(rstd, rstd_p)
    res_p, ldr = None, n
    if dres is not None:
        rr, rn, ldr, res_p = _rows_of(dres, "dres", types if out_dtype is None else (out_dtype,))
        if (rr, rn) != (rows, n):
            raise ValueError(f"dres must be [{rows}, {n}], got [{rr}, {rn}]")
        out_dtype = dres.dtype
    out_dtype = out_dtype or b16
    if out_dtype not in types:
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    if not (want_dx or quantize or want_dweight):
        raise ValueError("nothing to compute: ask for dx, quantize or dweight")
    dev = _one_device(dy, h, rstd, weight, dres)
    dx = _new(rows, n, out_dtype, dev) if want_dx else None
    codes = scales = dw = work = None
    ldc, need = n, 0
    if quantize:
        codes, ldc = _new_codes(rows, n, dev)
        scales = _new(rows, (n + 127) // 128, f32, dev)
    if want_dweight:
        # (two allocations: a gradient that is kept should not keep the workspace)
        dw = torch.empty_strided((n,), (1,), dtype=f32, device=dev)
        need = (_lib or load_library()).fp8q_rmsnorm_backward_workspace(rows, n)
        work = torch.empty_strided((need // 4,), (1,), dtype=f32, device=dev)
    _call(dev, "fp8q_rmsnorm_backward", dy_p, types.index(dy.dtype), rows, n, ldd, h_p, types.index(h.dtype), ldh, rstd_p, w_p,
          types.index(weight.dtype), res_p, ldr, _addr(dx), types.index(out_dtype), n, _scale_mode(scale_mode), _addr(codes), ldc,
          _addr(scales), _addr(dw), _addr(work), need)
    return dx, codes, scales, dw


def rmsnorm_quantize_t(h, rstd, weight, index=None, scale_mode="free"):
    """The norm's output once more, from h, rstd and weight as for
    ``rmsnorm_backward``, in 128x1 token-axis tiles: (codes [N, rows],
    scales [N, ceil(rows/128)]), bit for bit ``quantize_act(y, "token_t")``
    of the y that ``rmsnorm_quantize`` forms.

    index: int32 [rows], the row of h behind every row of the token axis
    (``moe_sort``'s token; outside h: zeros).  Default: every row of h.  rstd
    and index may be slices anywhere, as for ``rmsnorm_backward``.
    """
    types = _types()[1]
    hr, n, ldh, h_p = _rows_of(h, "h", types)
    rstd_p, w_p = _vector(rstd, hr, types[:1], "rstd"), _vector(weight, n, types, "weight")
    rstd, rstd_p = _on16(rstd, rstd_p)
    rows, i_p = hr, None
    if index is not None:
        rows = index.numel() if isinstance(index, _types()[0]) else 0
        index, i_p = _on16(index, _vector(index, rows, _types()[2:], "index"))
    dev = _one_device(h, rstd, weight, index)
    codes, ldc = _new_codes(n, rows, dev)
    scales = _new(n, (rows + 127) // 128, types[0], dev)
    _call(dev, "fp8q_rmsnorm_quantize_t", h_p, types.index(h.dtype), hr, n, ldh, rstd_p, w_p, types.index(weight.dtype), i_p, rows,
          _scale_mode(scale_mode), _addr(codes), ldc, _addr(scales))
    return codes, scales


_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}


def _score(score):
    try:
        return _SCORES[score]
    except KeyError:
        raise ValueError('score must be "softmax" or "sigmoid"') from None


def moe_route(logits, topk, bias=None, score="sigmoid", groups=1, top_groups=1, group_score="top2", renormalize=True, scale=1.0,
              index_dtype=None, want_scores=False, load=None):
    """The router's choice: the topk experts of every token and their weights.

    logits BF16 or float32 [tokens, E]; score "sigmoid" or "softmax".  The
    choice goes by score + bias (float32 [E]), or by the logits without one,
    within the top_groups best of `groups` groups of consecutive experts (by
    their best expert, group_score "max", or their two best, "top2"); ties go
    to the lower index.  Weights are scale * score, divided by their sum if
    renormalize.  Experts whose logit or bias is -inf or NaN are never chosen;
    what a token lacks is expert -1 with weight 0 (``moe_sort`` skips it).

    Returns (experts int32 or index_dtype [tokens, topk], best first, weights
    float32 [tokens, topk], scores float32 [tokens, E] with want_scores, else
    None).  load: int32 [E], to which each expert's number of pairs is added.
    """
    torch = _torch()
    tensor, types, i32 = _types()
    tokens, n, ld, logits_p = _rows_of(logits, "logits", types)
    bias_p = None if bias is None else _vector(bias, n, types[:1], "bias")
    load_p = None if load is None else _vector(load, n, (i32,), "load")
    index_dtype = index_dtype or i32
    if index_dtype not in (i32, torch.int64):
        raise TypeError("index_dtype must be torch.int32 or torch.int64")
    # (topk and the groups go over as 64- and 32-bit integers)
    if not 0 <= topk <= n or not 1 <= top_groups <= groups < 1 << 31:
        raise ValueError("topk must be in 0 .. experts, top_groups in 1 .. groups")
    if group_score not in ("max", "top2"):
        raise ValueError('group_score must be "max" or "top2"')
    dev = _one_device(logits, bias, load)
    experts = _new(tokens, topk, index_dtype, dev)
    weights = _new(tokens, topk, types[0], dev)
    scores = _new(tokens, n, types[0], dev) if want_scores else None
    _call(dev, "fp8q_moe_route", logits_p, types.index(logits.dtype), tokens, n, ld, bias_p, _score(score), groups, top_groups,
          GROUP_MAX if group_score == "max" else GROUP_TOP_TWO, topk, bool(renormalize), scale,
          INDEX_I32 if index_dtype == i32 else INDEX_I64, _addr(experts), _addr(weights), _addr(scores), load_p)
    return experts, weights, scores


def moe_route_backward(dweights, experts, logits, score="sigmoid", renormalize=True, scale=1.0, dscores=None, out_dtype=None):
    """Gradient of ``moe_route``'s weights with respect to the logits, the
    choice held fixed: dweights float32 and experts (int32 or int64) [tokens,
    topk], logits, score, renormalize and scale as there.  dscores: float32
    [tokens, E], added as the gradient of the scores.  Returns dlogits
    [tokens, E], out_dtype or the logits' type.  dweights and experts may be
    rows of a batch's anywhere, as rstd for ``rmsnorm_backward``.
    """
    torch = _torch()
    tensor, types, i32 = _types()
    tokens, n, ld, logits_p = _rows_of(logits, "logits", types)
    _contig_f32(dweights, "dweights")
    if not isinstance(experts, tensor) or experts.dtype not in (i32, torch.int64):
        raise TypeError("experts must be an int32 or int64 torch.Tensor")
    shape = tuple(dweights.shape)
    if len(shape) != 2 or shape[0] != tokens or tuple(experts.shape) != shape or not experts.is_contiguous():
        raise ValueError(f"dweights and experts must be contiguous [{tokens}, topk] tensors")
    if shape[1] > n:
        raise ValueError("more choices than experts")
    if dscores is not None:
        _contig_f32(dscores, "dscores")
        if tuple(dscores.shape) != (tokens, n):
            raise ValueError(f"dscores must be [{tokens}, {n}], got {tuple(dscores.shape)}")
    out_dtype = out_dtype or logits.dtype
    if out_dtype not in types:
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    dev = _one_device(logits, dweights, experts, dscores)
    dlogits = _new(tokens, n, out_dtype, dev)
    (dweights, dw_p), (experts, e_p) = _on16(dweights, dweights.data_ptr()), _on16(experts, experts.data_ptr())
    _call(dev, "fp8q_moe_route_backward", dw_p, e_p, INDEX_I32 if experts.dtype == i32 else INDEX_I64, tokens,
          shape[1], logits_p, types.index(logits.dtype), n, ld, _score(score), bool(renormalize), scale, _addr(dscores), _addr(dlogits),
          types.index(out_dtype), n)
    return dlogits
