"""int4_weight_only_amd -- Python binding of libw4.so, the MI355X (gfx950) group-wise INT4
weight-only linear layer.

The binding only marshals arguments: it checks tensor dtypes/devices/shapes, allocates outputs
with torch (device memory is torch's), passes raw pointers and the current HIP stream to the C
ABI declared in include/w4.h, and turns a nonzero status into an exception.  Every step of the
computation runs in the library's HIP kernels; there is no CPU or PyTorch fallback: if libw4.so is
missing or cannot be loaded, importing this package raises.

bf16 tensors are passed as torch.bfloat16 (their bits are the uint16 patterns of the ABI).
"""
import ctypes
import os

import torch

__all__ = [
    "W4_SYM", "W4_ASYM", "W4_OUT_BF16", "W4_OUT_F32", "W4Error", "packed_layout", "w4_pack",
    "w4_gemv", "w4_gemv_ws", "w4_gemv_work_bytes", "w4_gemv_glu", "w4_gemm", "act_quant_int8", "w4a8_gemv", "w4a8_gemm", "w4a8_linear",
    "w4_qat_repack", "gptq_hessian", "gptq_factor", "gptq_quantize", "gptq_quantize_noalloc",
    "gptq",
    "w4_linear",
    "W4_ROPE_HALF", "W4_ROPE_INTERLEAVED", "W4_ROPE_PLAIN", "W4_ROPE_LINEAR", "W4_ROPE_NTK",
    "W4_ROPE_YARN", "w4_rope_frequencies", "w4_rope_append", "w4_attn_decode",
    "w4_attn_decode_work_bytes", "w4_attn_prefill", "w4_attn_prefill_work_bytes",
    "w4_residual_norm",
    "library_path",
]

W4_SYM, W4_ASYM = 0, 1
W4_OUT_BF16, W4_OUT_F32 = 0, 1
W4_ROPE_HALF, W4_ROPE_INTERLEAVED = 0, 1
W4_ROPE_PLAIN, W4_ROPE_LINEAR, W4_ROPE_NTK, W4_ROPE_YARN = 0, 1, 2, 3
GEMV_MAX_M = 64

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libw4.so")


class _KvCache(ctypes.Structure):
    """w4_kv_cache of include/w4.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_table", ctypes.c_void_p), ("n_seqs", ctypes.c_int64),
                ("table_cols", ctypes.c_int64), ("ld_table", ctypes.c_int64),
                ("kv_len", ctypes.c_void_p)]


class W4Error(RuntimeError):
    def __init__(self, fn, status, text):
        super().__init__(f"{fn} failed with status {status}: {text}")
        self.status = status


def _load(path):
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} not found at {path}; build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'` or "
                          "`python int4_weight_only_amd/build.py`")
    lib = ctypes.CDLL(path)
    i64, p, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    lib.w4_packed_layout.argtypes = [i64, i64, i32, ctypes.POINTER(i64), ctypes.POINTER(i64),
                                     ctypes.POINTER(ctypes.c_size_t)]
    lib.w4_pack.argtypes = [p, i64, i64, i64, i32, i32, p, p, p, p]
    lib.w4_qat_repack.argtypes = [p, i64, i64, i64, p, p, p, p]
    lib.w4_gptq_hessian.argtypes = [p, i64, i64, i64, p, p]
    lib.w4_gptq_factor.argtypes = [p, i64, ctypes.c_float, p, p, p, p]
    lib.w4_gptq_quantize.argtypes = [p, i64, i64, i64, p, p, i32, i32, p, p, p, p, p, p]
    lib.w4_gptq_quantize_noalloc.argtypes = [p, i64, i64, i64, p, p, i32, i32, p, p, p, p, p]
    lin = [p, i64, i64, p, p, p, p, i64, i64, i32, p, i64, i32]
    lib.w4_gemv.argtypes = lin + [p]
    lib.w4_gemv_ws.argtypes = lin + [p, ctypes.c_size_t, p]
    lib.w4_gemv_work_bytes.argtypes = [i64, i64, i64, i32]
    lib.w4_gemv_work_bytes.restype = ctypes.c_size_t
    lib.w4_gemv_glu.argtypes = lin + [p]
    lib.w4_gemm.argtypes = lin + [p]
    lib.act_quant_int8.argtypes = [p, i64, i64, i64, p, i64, p, p, p]
    lib.w4a8_gemv.argtypes = [p, p, i64, i64, p, p, p, i64, i64, p, i64, i32, p, p]
    lib.w4a8_gemm.argtypes = lib.w4a8_gemv.argtypes
    lib.w4a8_linear.argtypes = [p, i64, i64, p, p, p, i64, i64, p, i64, i32, p, p, p]
    cache, f32, f64 = ctypes.POINTER(_KvCache), ctypes.c_float, ctypes.c_double
    lib.w4_rope_frequencies.argtypes = [i32, i32, f64, f64, f64, p, p]
    lib.w4_rope_append.argtypes = [p, i64, i64, i32, p, p, i32, i32, f32, cache, p, i64, p]
    attn = [f32, i64, i64, p, i64, i32, p, p, ctypes.c_size_t, p]
    lib.w4_attn_decode.argtypes = [p, i64, i32, cache] + attn
    lib.w4_attn_decode_work_bytes.argtypes = [i32, cache, i64, i64]
    lib.w4_attn_decode_work_bytes.restype = ctypes.c_size_t
    lib.w4_attn_prefill.argtypes = [p, i64, i64, i32, p, cache] + attn
    lib.w4_attn_prefill_work_bytes.argtypes = [i64, i32, cache, i64, i64]
    lib.w4_attn_prefill_work_bytes.restype = ctypes.c_size_t
    lib.w4_residual_norm.argtypes = [p, i64, p, i64, i32, i64, i64, p, p, f32, p, i64, f32, f32,
                                     p, i64, p, i64, p]
    for f in ("w4_rope_frequencies", "w4_rope_append", "w4_attn_decode", "w4_attn_prefill",
              "w4_residual_norm"):
        getattr(lib, f).restype = i32
    for f in ("w4_packed_layout", "w4_pack", "w4_qat_repack", "w4_gptq_hessian", "w4_gptq_factor",
              "w4_gptq_quantize", "w4_gptq_quantize_noalloc", "w4_gemv", "w4_gemv_ws",
              "w4_gemv_glu", "w4_gemm",
              "act_quant_int8", "w4a8_gemv", "w4a8_gemm", "w4a8_linear"):
        getattr(lib, f).restype = i32
    lib.w4_status_string.argtypes = [i32]
    lib.w4_status_string.restype = ctypes.c_char_p
    lib.w4_last_hip_error.argtypes = []
    lib.w4_last_hip_error.restype = ctypes.c_char_p
    return lib


_lib = _load(_LIB_PATH)


def library_path():
    return _LIB_PATH


def _select_library(path):
    """Bind every entry point of this module to another build of the library (the tests use the
    build with the kernel-choice hook, libw4_hooks.so); returns the path bound before."""
    global _lib, _LIB_PATH
    prev = _LIB_PATH
    _lib = _load(path)
    _LIB_PATH = path
    return prev


def _check(fn, status):
    if status != 0:
        text = _lib.w4_status_string(status).decode()
        if status == 7:  # W4_ERR_HIP
            text += ": " + _lib.w4_last_hip_error().decode()
        raise W4Error(fn, status, text)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    """The current stream of a device, as an address (without a torch.cuda.Stream object, whose
    making costs a small call a tenth of its time)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _need(t, name, dtype, device=None, dim=None):
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda
            and (device is None or t.device == device) and (dim is None or t.ndim == dim)
            and (t.ndim == 0 or t.stride(-1) == 1)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dims, got {t.dim()}")
    if t.dim() > 0 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dim")


def _check_out_shape(out, rows, cols, name="out"):
    """A caller-supplied output must hold `rows` x `cols` elements at its own row stride: the
    kernels write rows 0 .. rows-1, columns 0 .. cols-1, with ldy = out.stride(0)."""
    if out.shape[0] < rows or out.shape[1] < cols:
        raise ValueError(f"{name} has shape {tuple(out.shape)}, needs at least ({rows}, {cols})")
    if rows > 1 and out.stride(0) < cols:
        raise ValueError(f"{name} rows overlap: stride {out.stride(0)} < {cols} columns")


def _out(out, rows, cols, tdtype, dev):
    if out is None:
        return torch.empty((rows, cols), dtype=tdtype, device=dev)
    _need(out, "out", tdtype, dev, 2)
    _check_out_shape(out, rows, cols)
    return out


def packed_layout(d_out, d_in, group_size):
    """(k_pad, n_groups, qweight_bytes) of the packed format (host-only query)."""
    kp, ng, nb = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_size_t()
    _check("w4_packed_layout", _lib.w4_packed_layout(d_out, d_in, group_size, ctypes.byref(kp),
                                                     ctypes.byref(ng), ctypes.byref(nb)))
    return kp.value, ng.value, nb.value


def w4_pack(w, group_size, mode, d_in=None):
    """RTN-pack an fp32 weight [d_out][ldw] (first d_in columns) on the GPU.
    Returns (qweight uint8 [d_out][k_pad/2], scales bf16 [d_out][G], zeros bf16 or None)."""
    _need(w, "w", torch.float32, dim=2)
    d_out, ldw = w.shape
    d_in = ldw if d_in is None else d_in
    k_pad, n_groups, _ = packed_layout(d_out, d_in, group_size)
    dev = w.device
    qweight = torch.empty((d_out, k_pad // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((d_out, n_groups), dtype=torch.bfloat16, device=dev)
    zeros = torch.empty_like(scales) if mode == W4_ASYM else None
    _check("w4_pack", _lib.w4_pack(_ptr(w), d_out, d_in, w.stride(0), group_size, mode,
                                   _ptr(qweight), _ptr(scales), _ptr(zeros), _stream(dev)))
    return qweight, scales, zeros


def w4_qat_repack(w, d_in=None, want_m=False):
    """Pack a bf16 weight [d_out][ldw] (first d_in columns) that lies on the 4-bit grid per group
    of 32 columns, keeping its levels (the g32 symmetric format).  Returns (qweight, scales), plus
    m uint8 [d_out][G] (the divisor kept per group, 0 off the grid) when want_m."""
    _need(w, "w", torch.bfloat16, dim=2)
    d_out, ldw = w.shape
    d_in = ldw if d_in is None else d_in
    k_pad, n_groups, _ = packed_layout(d_out, d_in, 32)
    dev = w.device
    qweight = torch.empty((d_out, k_pad // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((d_out, n_groups), dtype=torch.bfloat16, device=dev)
    m = torch.empty((d_out, n_groups), dtype=torch.uint8, device=dev) if want_m else None
    _check("w4_qat_repack", _lib.w4_qat_repack(_ptr(w), d_out, d_in, w.stride(0), _ptr(qweight),
                                               _ptr(scales), _ptr(m), _stream(dev)))
    return (qweight, scales, m) if want_m else (qweight, scales)


def gptq_hessian(x, d_in=None):
    """H = (2/N) X^T X, fp32 [d_in][d_in], from bf16 calibration activations x [N][ldx]."""
    _need(x, "x", torch.bfloat16, dim=2)
    N = x.shape[0]
    d_in = x.shape[1] if d_in is None else d_in
    h = torch.empty((d_in, d_in), dtype=torch.float32, device=x.device)
    _check("w4_gptq_hessian", _lib.w4_gptq_hessian(_ptr(x), N, d_in, x.stride(0), _ptr(h),
                                                   _stream(x.device)))
    return h


def gptq_factor(h, alpha=0.01):
    """Dead columns, damping and U with (H + lambda I)^-1 = U^T U.  h fp32 [d_in][d_in] is used as
    the working matrix and destroyed.  Returns (u fp32 [d_in][d_in], dead uint8 [d_in])."""
    _need(h, "h", torch.float32, dim=2)
    d_in = h.shape[0]
    if h.shape[1] != d_in or not h.is_contiguous():
        raise ValueError("h must be a contiguous square matrix")
    u = torch.empty_like(h)
    work = torch.empty_like(h)
    dead = torch.empty((d_in,), dtype=torch.uint8, device=h.device)
    _check("w4_gptq_factor", _lib.w4_gptq_factor(_ptr(h), d_in, float(alpha), _ptr(u), _ptr(work),
                                                 _ptr(dead), _stream(h.device)))
    return u, dead


def gptq_quantize(w, u, dead, group_size, mode, d_in=None):
    """The GPTQ column loop on fp32 weights w [d_out][ldw] (used as the working copy and
    destroyed).  Returns (qweight, scales, zeros or None, row_loss fp32 [d_out])."""
    _need(w, "w", torch.float32, dim=2)
    dev = w.device
    _need(u, "u", torch.float32, dev, 2)
    if dead is not None:
        _need(dead, "dead", torch.uint8, dev, 1)
    d_out, ldw = w.shape
    d_in = ldw if d_in is None else d_in
    if tuple(u.shape) != (d_in, d_in) or not u.is_contiguous():
        raise ValueError(f"u must be contiguous [{d_in}][{d_in}]")
    k_pad, n_groups, _ = packed_layout(d_out, d_in, group_size)
    qweight = torch.empty((d_out, k_pad // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((d_out, n_groups), dtype=torch.bfloat16, device=dev)
    zeros = torch.empty_like(scales) if mode == W4_ASYM else None
    work = torch.empty((d_out, 32), dtype=torch.float32, device=dev)
    row_loss = torch.empty((d_out,), dtype=torch.float32, device=dev)
    _check("w4_gptq_quantize", _lib.w4_gptq_quantize(
        _ptr(w), d_out, d_in, w.stride(0), _ptr(u), _ptr(dead), group_size, mode, _ptr(qweight),
        _ptr(scales), _ptr(zeros), _ptr(work), _ptr(row_loss), _stream(dev)))
    return qweight, scales, zeros, row_loss


def gptq_quantize_noalloc(w, u, dead, group_size, mode, d_in=None, row_loss=None, out=None):
    """gptq_quantize for callers that cannot allocate: the block errors live in the library's own
    device array (calls that overlap on one GPU race), and the outputs are the caller's
    out=(qweight, scales, zeros or None) and row_loss (nothing is allocated here either when
    they are given).  Returns (qweight, scales, zeros or None, row_loss or None)."""
    _need(w, "w", torch.float32, dim=2)
    dev = w.device
    _need(u, "u", torch.float32, dev, 2)
    if dead is not None:
        _need(dead, "dead", torch.uint8, dev, 1)
    d_out, ldw = w.shape
    d_in = ldw if d_in is None else d_in
    if tuple(u.shape) != (d_in, d_in) or not u.is_contiguous():
        raise ValueError(f"u must be contiguous [{d_in}][{d_in}]")
    k_pad, n_groups, _ = packed_layout(d_out, d_in, group_size)
    if out is None:
        qweight = torch.empty((d_out, k_pad // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((d_out, n_groups), dtype=torch.bfloat16, device=dev)
        zeros = torch.empty_like(scales) if mode == W4_ASYM else None
    else:
        qweight, scales, zeros = out
        _need(qweight, "qweight", torch.uint8, dev, 2)
        _need(scales, "scales", torch.bfloat16, dev, 2)
        if tuple(qweight.shape) != (d_out, k_pad // 2) or not qweight.is_contiguous():
            raise ValueError(f"qweight must be contiguous [{d_out}][{k_pad // 2}]")
        for name, t in (("scales", scales), ("zeros", zeros)):
            if t is not None and (tuple(t.shape) != (d_out, n_groups) or not t.is_contiguous()):
                raise ValueError(f"{name} must be contiguous [{d_out}][{n_groups}]")
    if row_loss is not None:
        _need(row_loss, "row_loss", torch.float32, dev, 1)
        if row_loss.shape[0] < d_out:
            raise ValueError(f"row_loss must hold {d_out} values")
    _check("w4_gptq_quantize_noalloc", _lib.w4_gptq_quantize_noalloc(
        _ptr(w), d_out, d_in, w.stride(0), _ptr(u), _ptr(dead), group_size, mode, _ptr(qweight),
        _ptr(scales), _ptr(zeros), _ptr(row_loss), _stream(dev)))
    return qweight, scales, zeros, row_loss


def gptq(w, x, group_size, mode, alpha=0.01, d_in=None):
    """GPTQ of fp32 weights w [d_out][>= d_in] with bf16 calibration activations x [N][>= d_in]
    (w is not modified).  Returns (qweight, scales, zeros or None, row_loss)."""
    d_in = w.shape[1] if d_in is None else d_in
    h = gptq_hessian(x, d_in)
    u, dead = gptq_factor(h, alpha)
    return gptq_quantize(w.clone(), u, dead, group_size, mode, d_in)


def _linear(fn_name, x, qweight, scales, zeros, bias, d_in, group_size, out_dtype, out,
            extra=()):
    _need(x, "x", torch.bfloat16, dim=2)
    dev = x.device
    _need(qweight, "qweight", torch.uint8, dev, 2)
    _need(scales, "scales", torch.bfloat16, dev, 2)
    if zeros is not None:
        _need(zeros, "zeros", torch.bfloat16, dev, 2)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, dev, 1)
    M = x.shape[0]
    d_out = qweight.shape[0]
    k_pad, n_groups, _ = packed_layout(d_out, d_in, group_size)
    if tuple(qweight.shape) != (d_out, k_pad // 2) or not qweight.is_contiguous():
        raise ValueError(f"qweight must be contiguous [{d_out}][{k_pad // 2}]")
    for name, t in (("scales", scales), ("zeros", zeros)):
        if t is not None and (tuple(t.shape) != (d_out, n_groups) or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous [{d_out}][{n_groups}]")
    if bias is not None and bias.shape[0] != d_out:
        raise ValueError(f"bias must have {d_out} elements")
    if x.shape[1] < d_in:
        raise ValueError(f"x has {x.shape[1]} columns, fewer than d_in={d_in}")
    tdtype = torch.float32 if out_dtype == W4_OUT_F32 else torch.bfloat16
    out = _out(out, M, d_out, tdtype, dev)
    fn = getattr(_lib, fn_name)
    args = [_ptr(x), M, x.stride(0), _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(bias),
            d_out, d_in, group_size, _ptr(out), out.stride(0), out_dtype]
    _check(fn_name, fn(*args, *extra, _stream(dev)))
    return out


def w4_gemv_work_bytes(M, d_out, d_in, group_size):
    """Bytes of workspace w4_gemv_ws needs for these sizes (0: none)."""
    return int(_lib.w4_gemv_work_bytes(M, d_out, d_in, group_size))


def w4_gemv_ws(x, qweight, scales, zeros, bias, d_in, group_size, out_dtype=W4_OUT_BF16,
               out=None, work=None):
    """w4_gemv with a workspace (a device uint8 tensor of at least w4_gemv_work_bytes bytes; one
    is allocated with torch when work is None): the reduction over d_in split over column slices
    on matrices with few, long rows per compute unit."""
    need = w4_gemv_work_bytes(x.shape[0], qweight.shape[0], d_in, group_size)
    if work is None:
        work = torch.zeros(max(need, 16), dtype=torch.uint8, device=x.device)
    _need(work, "work", torch.uint8, x.device, 1)
    return _linear("w4_gemv_ws", x, qweight, scales, zeros, bias, d_in, group_size, out_dtype,
                   out, extra=(_ptr(work), work.numel()))


def w4_gemv(x, qweight, scales, zeros, bias, d_in, group_size, out_dtype=W4_OUT_BF16, out=None):
    """Decode W4A16 linear, 1 <= M <= 64: y[M][d_out] = x . W_hat^T (+ b)."""
    return _linear("w4_gemv", x, qweight, scales, zeros, bias, d_in, group_size, out_dtype, out)


def w4_gemv_glu(x, qweight, scales, zeros, bias, d_in, group_size, out_dtype=W4_OUT_BF16,
                out=None):
    """Gate/up GEMV with the SiLU(gate) * up epilogue: qweight holds 2 d_ff rows (gate rows, then
    up rows), bias 2 d_ff values or None; returns h [M][d_ff]."""
    _need(x, "x", torch.bfloat16, dim=2)
    dev = x.device
    _need(qweight, "qweight", torch.uint8, dev, 2)
    _need(scales, "scales", torch.bfloat16, dev, 2)
    if zeros is not None:
        _need(zeros, "zeros", torch.bfloat16, dev, 2)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, dev, 1)
    M = x.shape[0]
    rows = qweight.shape[0]
    if rows % 2:
        raise ValueError("a fused gate/up weight has an even number of rows")
    d_ff = rows // 2
    k_pad, n_groups, _ = packed_layout(rows, d_in, group_size)
    if tuple(qweight.shape) != (rows, k_pad // 2) or not qweight.is_contiguous():
        raise ValueError(f"qweight must be contiguous [{rows}][{k_pad // 2}]")
    for name, t in (("scales", scales), ("zeros", zeros)):
        if t is not None and (tuple(t.shape) != (rows, n_groups) or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous [{rows}][{n_groups}]")
    if bias is not None and bias.shape[0] != rows:
        raise ValueError(f"bias must have {rows} elements")
    if x.shape[1] < d_in:
        raise ValueError(f"x has {x.shape[1]} columns, fewer than d_in={d_in}")
    tdtype = torch.float32 if out_dtype == W4_OUT_F32 else torch.bfloat16
    out = _out(out, M, d_ff, tdtype, dev)
    _check("w4_gemv_glu", _lib.w4_gemv_glu(_ptr(x), M, x.stride(0), _ptr(qweight), _ptr(scales),
                                           _ptr(zeros), _ptr(bias), d_ff, d_in, group_size,
                                           _ptr(out), out.stride(0), out_dtype, _stream(dev)))
    return out


def w4_gemm(x, qweight, scales, zeros, bias, d_in, group_size, out_dtype=W4_OUT_BF16, out=None):
    """Prefill W4A16 linear, any M >= 1 (bf16 matrix cores)."""
    return _linear("w4_gemm", x, qweight, scales, zeros, bias, d_in, group_size, out_dtype, out)


def w4_linear(x, qweight, scales, zeros, bias, d_in, group_size, out_dtype=W4_OUT_BF16,
              out=None):
    """Dispatch by token count: the decode kernel for M <= 64, the matrix-core GEMM above."""
    fn = w4_gemv if x.shape[0] <= GEMV_MAX_M else w4_gemm
    return fn(x, qweight, scales, zeros, bias, d_in, group_size, out_dtype, out)


def act_quant_int8(x, K=None, with_sum=True, out=None):
    """Per-token int8 quantization.  Returns (q int8 [M][ldq], s_x fp32 [M], q_sum int32 [M] or
    None); ldq is K rounded up to 16 (columns >= K are left unset).  out=(q, s_x) reuses
    caller tensors of those shapes."""
    _need(x, "x", torch.bfloat16, dim=2)
    M = x.shape[0]
    K = x.shape[1] if K is None else K
    dev = x.device
    ldq = (K + 15) // 16 * 16
    if out is None:
        q = torch.empty((M, ldq), dtype=torch.int8, device=dev)
        s_x = torch.empty((M,), dtype=torch.float32, device=dev)
    else:
        q, s_x = out
        _need(q, "q", torch.int8, dev, 2)
        _need(s_x, "s_x", torch.float32, dev, 1)
        if q.shape[0] != M or q.shape[1] < K or q.stride(1) != 1 or s_x.shape[0] != M:
            raise ValueError("out must be (q [M][>= K] row-major, s_x [M])")
        ldq = q.stride(0)
    q_sum = torch.empty((M,), dtype=torch.int32, device=dev) if with_sum else None
    _check("act_quant_int8", _lib.act_quant_int8(_ptr(x), M, K, x.stride(0), _ptr(q), ldq,
                                                 _ptr(s_x), _ptr(q_sum), _stream(dev)))
    return q, s_x, q_sum


def w4a8_gemv(q, s_x, qweight, s_w, bias, d_in, out_dtype=W4_OUT_BF16, want_acc=False,
              out=None):
    """W4A8 decode linear (M <= 64).  Returns y, or (y, acc int32 [M][d_out]) when want_acc."""
    return _w4a8("w4a8_gemv", q, s_x, qweight, s_w, bias, d_in, out_dtype, want_acc, out)


def w4a8_gemm(q, s_x, qweight, s_w, bias, d_in, out_dtype=W4_OUT_BF16, want_acc=False,
              out=None):
    """W4A8 prefill linear on the int8 matrix cores (any M), the arguments and result of
    w4a8_gemv.  Returns y, or (y, acc int32 [M][d_out]) when want_acc."""
    return _w4a8("w4a8_gemm", q, s_x, qweight, s_w, bias, d_in, out_dtype, want_acc, out)


def _w4a8(name, q, s_x, qweight, s_w, bias, d_in, out_dtype, want_acc, out):
    _need(q, "q", torch.int8, dim=2)
    dev = q.device
    _need(s_x, "s_x", torch.float32, dev, 1)
    _need(qweight, "qweight", torch.uint8, dev, 2)
    s_w = s_w.reshape(-1)
    _need(s_w, "s_w", torch.bfloat16, dev, 1)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, dev, 1)
    M = q.shape[0]
    d_out = qweight.shape[0]
    k_pad, _, _ = packed_layout(d_out, d_in, 0)
    if tuple(qweight.shape) != (d_out, k_pad // 2) or not qweight.is_contiguous():
        raise ValueError(f"qweight must be contiguous [{d_out}][{k_pad // 2}]")
    if s_w.shape[0] != d_out or (bias is not None and bias.shape[0] != d_out):
        raise ValueError(f"s_w and bias must have {d_out} elements")
    if s_x.shape[0] != M or q.shape[1] < d_in:
        raise ValueError("q must be [M][>= d_in] and s_x [M]")
    tdtype = torch.float32 if out_dtype == W4_OUT_F32 else torch.bfloat16
    out = _out(out, M, d_out, tdtype, dev)
    acc = torch.empty((M, d_out), dtype=torch.int32, device=dev) if want_acc else None
    _check(name, getattr(_lib, name)(_ptr(q), _ptr(s_x), M, q.stride(0), _ptr(qweight),
                                     _ptr(s_w), _ptr(bias), d_out, d_in, _ptr(out),
                                     out.stride(0), out_dtype, _ptr(acc), _stream(dev)))
    return (out, acc) if want_acc else out


def w4a8_linear(x, qweight, s_w, bias, d_in, out_dtype=W4_OUT_BF16, want_acc=False,
                want_scales=False, out=None):
    """W4A8 decode linear on bf16 activations, quantized per token inside the kernel (the result
    of act_quant_int8 + w4a8_gemv in one launch).  Returns y, then acc int32 [M][d_out] if
    want_acc, then s_x fp32 [M] if want_scales."""
    _need(x, "x", torch.bfloat16, dim=2)
    dev = x.device
    _need(qweight, "qweight", torch.uint8, dev, 2)
    s_w = s_w.reshape(-1)
    _need(s_w, "s_w", torch.bfloat16, dev, 1)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, dev, 1)
    M = x.shape[0]
    d_out = qweight.shape[0]
    k_pad, _, _ = packed_layout(d_out, d_in, 0)
    if tuple(qweight.shape) != (d_out, k_pad // 2) or not qweight.is_contiguous():
        raise ValueError(f"qweight must be contiguous [{d_out}][{k_pad // 2}]")
    if s_w.shape[0] != d_out or (bias is not None and bias.shape[0] != d_out):
        raise ValueError(f"s_w and bias must have {d_out} elements")
    if x.shape[1] < d_in:
        raise ValueError(f"x has {x.shape[1]} columns, fewer than d_in={d_in}")
    tdtype = torch.float32 if out_dtype == W4_OUT_F32 else torch.bfloat16
    out = _out(out, M, d_out, tdtype, dev)
    acc = torch.empty((M, d_out), dtype=torch.int32, device=dev) if want_acc else None
    s_x = torch.empty(M, dtype=torch.float32, device=dev) if want_scales else None
    _check("w4a8_linear", _lib.w4a8_linear(_ptr(x), M, x.stride(0), _ptr(qweight), _ptr(s_w),
                                           _ptr(bias), d_out, d_in, _ptr(out), out.stride(0),
                                           out_dtype, _ptr(s_x), _ptr(acc), _stream(dev)))
    res = (out,) + ((acc,) if want_acc else ()) + ((s_x,) if want_scales else ())
    return res if len(res) > 1 else out


def w4_rope_frequencies(rot_dim, scaling=W4_ROPE_PLAIN, base=10000.0, factor=1.0, context=1.0):
    """(inv_freq fp32 [rot_dim / 2], amplitude) of rotary positions for a context scaling (host
    only; move inv_freq to the GPU once)."""
    inv_freq = torch.empty(max(rot_dim, 2) // 2, dtype=torch.float32, device="cpu")
    amplitude = ctypes.c_float()
    _check("w4_rope_frequencies", _lib.w4_rope_frequencies(
        rot_dim, scaling, base, factor, context, _ptr(inv_freq), ctypes.byref(amplitude)))
    return inv_freq, amplitude.value


def _kv_cache(k_cache, v_cache, page_table, kv_len, dev):
    """The ABI's view of a cache [n_pages][page_size][n_kv_heads][head_dim] (any strides with the
    last dim contiguous; another order of slots and heads is a permuted view)."""
    if not (k_cache.dtype is v_cache.dtype is torch.bfloat16
            and page_table.dtype is kv_len.dtype is torch.int32
            and k_cache.device == v_cache.device == page_table.device == kv_len.device == dev
            and k_cache.is_cuda):
        _need(k_cache, "k_cache", torch.bfloat16, dev)
        _need(v_cache, "v_cache", torch.bfloat16, dev)
        _need(page_table, "page_table", torch.int32, dev)
        _need(kv_len, "kv_len", torch.int32, dev)
    try:
        n_pages, page_size, n_kv, D = shape = k_cache.shape
        n_seqs, cols = page_table.shape
        n_lens, = kv_len.shape
    except ValueError:
        raise ValueError("k_cache and v_cache must have 4 dims, page_table 2 and kv_len 1") from None
    sp, ss, sh, sd = strides = k_cache.stride()
    if v_cache.shape != shape or v_cache.stride() != strides or n_pages == 1 or page_size == 1 \
            or n_kv == 1:
        # the stride of a dimension of one element says nothing
        if v_cache.shape != shape or any(n > 1 and x != y for n, x, y in
                                         zip(shape, strides, v_cache.stride())):
            raise ValueError("k_cache and v_cache must have the same shape and strides")
        sp, ss, sh = (x if n > 1 else 0 for n, x in zip(shape, strides[:3]))
    ld, one = page_table.stride()
    if (sd != 1 and D > 1) or (one != 1 and cols > 1) or (n_lens > 1 and kv_len.stride(0) != 1):
        raise ValueError("k_cache, v_cache, page_table and kv_len must be contiguous along their "
                         "last dim")
    if n_lens != n_seqs:
        raise ValueError(f"kv_len must have {n_seqs} elements")
    return _KvCache(k_cache.data_ptr(), v_cache.data_ptr(), n_pages, sp, ss, sh, page_size, n_kv,
                    D, page_table.data_ptr(), n_seqs, cols, ld if n_seqs > 1 else cols,
                    kv_len.data_ptr())


def _need_q_start(q_start, n_seqs, dev):
    _need(q_start, "q_start", torch.int32, dev, 1)
    if q_start.shape[0] != n_seqs + 1:
        raise ValueError(f"q_start must have {n_seqs + 1} elements")


def w4_rope_append(qkv, n_heads, k_cache, v_cache, page_table, kv_len, inv_freq, q_start=None,
                   layout=W4_ROPE_HALF, factor=1.0, out=None):
    """Rotary positions on the fused projection qkv bf16 [T][(n_heads + 2 n_kv) head_dim]; the
    rotated keys and the values are written to the cache, the rotated queries returned
    ([T][n_heads * head_dim]).  kv_len counts the T tokens already; q_start int32 [n_seqs + 1] gives
    each sequence's rows (None: one token per sequence).  out must not overlap qkv."""
    _need(qkv, "qkv", torch.bfloat16, dim=2)
    dev = qkv.device
    _need(inv_freq, "inv_freq", torch.float32, dev, 1)
    cache = _kv_cache(k_cache, v_cache, page_table, kv_len, dev)
    if q_start is not None:
        _need_q_start(q_start, cache.n_seqs, dev)
    T, width = qkv.shape
    if width < (n_heads + 2 * cache.n_kv_heads) * cache.head_dim:
        raise ValueError(f"qkv has {width} columns, fewer than its heads")
    out = _out(out, T, n_heads * cache.head_dim, torch.bfloat16, dev)
    _check("w4_rope_append", _lib.w4_rope_append(
        _ptr(qkv), T, qkv.stride(0) if T > 1 else width, n_heads, _ptr(q_start), _ptr(inv_freq),
        2 * inv_freq.shape[0], layout, factor, ctypes.byref(cache), _ptr(out),
        out.stride(0) if T > 1 else out.shape[1], _stream(dev)))
    return out


def _attention(name, q, k_cache, v_cache, page_table, kv_len, q_start, scale, window, sinks,
               out_dtype, out, want_lse, work):
    _need(q, "q", torch.bfloat16, dim=2)
    dev = q.device
    cache = _kv_cache(k_cache, v_cache, page_table, kv_len, dev)
    T, width = q.shape
    D = cache.head_dim
    if width % D != 0:
        raise ValueError(f"q has {width} columns, not a multiple of head_dim={D}")
    n_heads = width // D
    lead = [_ptr(q), q.stride(0) if T > 1 else width, n_heads]
    if q_start is None:
        if T != cache.n_seqs:
            raise ValueError(f"q must have one row for each of {cache.n_seqs} sequences")
        need = _lib.w4_attn_decode_work_bytes(n_heads, ctypes.byref(cache), window, sinks)
    else:
        _need_q_start(q_start, cache.n_seqs, dev)
        lead = [lead[0], T, lead[1], n_heads, _ptr(q_start)]
        need = _lib.w4_attn_prefill_work_bytes(T, n_heads, ctypes.byref(cache), window, sinks)
    if work is None:
        if need:
            work = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need(work, "work", torch.uint8, dev, 1)
    tdtype = torch.float32 if out_dtype == W4_OUT_F32 else torch.bfloat16
    out = _out(out, T, width, tdtype, dev)
    lse = torch.empty((T, n_heads), dtype=torch.float32, device=dev) if want_lse else None
    _check(name, getattr(_lib, name)(
        *lead, ctypes.byref(cache), D ** -0.5 if scale is None else scale, window, sinks,
        _ptr(out), out.stride(0) if T > 1 else width, out_dtype, _ptr(lse), _ptr(work),
        0 if work is None else work.numel(), _stream(dev)))
    return (out, lse) if want_lse else out


def w4_attn_decode(q, k_cache, v_cache, page_table, kv_len, scale=None, window=0, sinks=0,
                   out_dtype=W4_OUT_BF16, out=None, want_lse=False, work=None):
    """Attention of one new token per sequence (q bf16 [n_seqs][n_heads * head_dim], at position
    kv_len - 1) over the paged cache; scale None: 1 / sqrt(head_dim).  Returns y [n_seqs][width],
    or (y, lse fp32 [n_seqs][n_heads]) when want_lse.  work: a uint8 tensor of at least
    w4_attn_decode_work_bytes bytes (None: one is allocated where needed)."""
    return _attention("w4_attn_decode", q, k_cache, v_cache, page_table, kv_len, None, scale,
                      window, sinks, out_dtype, out, want_lse, work)


def w4_attn_prefill(q, k_cache, v_cache, page_table, kv_len, q_start, scale=None, window=0,
                    sinks=0, out_dtype=W4_OUT_BF16, out=None, want_lse=False, work=None):
    """w4_attn_decode for T tokens of n_seqs sequences, the rows q_start[b] .. q_start[b + 1] - 1 of
    q being the last tokens of sequence b: prompts, chunks, or several new tokens each."""
    if q_start is None:
        raise TypeError("q_start must be a torch.Tensor")
    return _attention("w4_attn_prefill", q, k_cache, v_cache, page_table, kv_len, q_start, scale,
                      window, sinks, out_dtype, out, want_lse, work)


def w4_attn_decode_work_bytes(n_heads, k_cache, v_cache, page_table, kv_len, window=0, sinks=0):
    """Bytes of workspace w4_attn_decode needs for these sizes (0: none)."""
    cache = _kv_cache(k_cache, v_cache, page_table, kv_len, k_cache.device)
    return int(_lib.w4_attn_decode_work_bytes(n_heads, ctypes.byref(cache), window, sinks))


def w4_attn_prefill_work_bytes(T, n_heads, k_cache, v_cache, page_table, kv_len, window=0,
                               sinks=0):
    """Bytes of workspace w4_attn_prefill needs for these sizes (0: none)."""
    cache = _kv_cache(k_cache, v_cache, page_table, kv_len, k_cache.device)
    return int(_lib.w4_attn_prefill_work_bytes(T, n_heads, ctypes.byref(cache), window, sinks))


def w4_residual_norm(x, residual, w_pre, w_post=None, gate=None, alpha=1.0, eps=1e-6,
                     weight_offset=0.0, out=None, residual_out=None):
    """The seam between two blocks: residual_out = residual + alpha * gate * n with n = x or
    rms(x, w_post), and y = rms(residual_out, w_pre).  x bf16 [T][d] (None: y = rms(residual,
    w_pre) alone), residual bf16 or fp32 [T][d], gate bf16 [d] or [T][d].  residual_out may be
    `residual` itself.  Returns (y bf16 [T][d], residual_out)."""
    if not isinstance(residual, torch.Tensor) or residual.dtype not in (torch.bfloat16,
                                                                         torch.float32):
        raise TypeError("residual must be a torch.bfloat16 or torch.float32 tensor")
    _need(residual, "residual", residual.dtype, dim=2)
    dev = residual.device
    T, d = residual.shape
    _need(w_pre, "w_pre", torch.bfloat16, dev, 1)
    if w_post is not None:
        _need(w_post, "w_post", torch.bfloat16, dev, 1)
    if w_pre.shape[0] != d or (w_post is not None and w_post.shape[0] != d):
        raise ValueError(f"w_pre and w_post must have {d} elements")
    ldx = ldg = ldro = 0
    if x is not None:
        _need(x, "x", torch.bfloat16, dev, 2)
        if tuple(x.shape) != (T, d):
            raise ValueError(f"x must be [{T}][{d}]")
        ldx = x.stride(0) if T > 1 else d
        residual_out = _out(residual_out, T, d, residual.dtype, dev)
        ldro = residual_out.stride(0) if T > 1 else d
    elif residual_out is not None:
        raise ValueError("residual_out needs x")
    if gate is not None:
        _need(gate, "gate", torch.bfloat16, dev)
        if tuple(gate.shape) not in ((d,), (T, d)):
            raise ValueError(f"gate must be [{d}] or [{T}][{d}]")
        ldg = gate.stride(0) if gate.dim() == 2 and T > 1 else 0
    y = _out(out, T, d, torch.bfloat16, dev)
    _check("w4_residual_norm", _lib.w4_residual_norm(
        _ptr(x), ldx, _ptr(residual), residual.stride(0) if T > 1 else d,
        W4_OUT_F32 if residual.dtype == torch.float32 else W4_OUT_BF16, T, d, _ptr(w_post),
        _ptr(w_pre), weight_offset, _ptr(gate), ldg, alpha, eps, _ptr(residual_out), ldro,
        _ptr(y), y.stride(0) if T > 1 else d, _stream(dev)))
    return y, (residual if x is None else residual_out)
