"""GB300 (sm_103a) MoE expert layer: dispatch -> grouped expert FFN -> combine.

Thin ctypes binding of libmoe_gb300.so (declared in include/moe.h).  Every
step of the layer runs in the library's CUDA kernels; this module only
marshals arguments.  PyTorch is used for device memory and streams.  There
is no CPU fallback: if the library is missing or the GPU is not an sm_103
part, calls raise.

Low-level names mirror the C ABI (moe_plan, moe_ffn_fwd, moe_ffn_bwd, ...)
and take raw integers for pointers.  The helpers below them (Shape,
alloc_plan, workspace, plan, ffn_fwd, ffn_bwd) take torch tensors.
"""

import ctypes
import os

__all__ = [
    "MOE_OK", "MOE_ACT_SWIGLU", "MOE_ACT_CLAMPED_GLU", "MOE_BF16", "MOE_FP32", "MoeShape",
    "MoePlan", "MoeBias", "MoeError", "lib", "library_path", "moe_workspace_size", "moe_saved_size",
    "moe_plan", "moe_ffn_fwd", "moe_ffn_bwd", "moe_get_device_error", "moe_status_string",
    "moe_set_wait_timeout_ns", "moe_kernel_launch_count", "moe_profile_enable",
    "moe_profile_read", "moe_profile_kernel_name", "Shape", "alloc_plan", "workspace", "plan", "ffn_fwd", "ffn_bwd",
    "bias_struct", "check_device_error", "moe_gather_rows", "moe_combine_rows", "gather_rows",
    "combine_rows", "moe_rms_norm_workspace_size", "moe_rms_norm_fwd", "moe_rms_norm_bwd",
    "rms_norm_workspace", "rms_norm_fwd", "rms_norm_bwd", "MoeGrad",
    "moe_grad_clip_workspace_size", "moe_grad_clip", "grad_table", "grad_clip_workspace",
    "grad_clip", "moe_mx_quantize", "moe_mx_dequantize", "mx_alloc", "mx_quantize",
    "mx_dequantize", "MoeMxWeights", "moe_few_workspace_size", "moe_ffn_few", "few_workspace",
    "mx_struct", "ffn_few", "moe_join_norm_workspace_size", "moe_join_norm_fwd",
    "moe_join_norm_bwd", "join_norm_workspace", "join_norm_fwd", "join_norm_bwd",
    "moe_route_bwd_workspace_size", "moe_route_bwd", "route_bwd_workspace", "route_bwd",
    "moe_orthogonalize_workspace_size", "moe_orthogonalize", "orthogonalize_workspace",
    "orthogonalize",
]

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_BAD_INDEX = 4
MOE_ERR_TIMEOUT = 5
MOE_ERR_CUDA = 6
MOE_ACT_SWIGLU = 0
MOE_ACT_CLAMPED_GLU = 1
MOE_GATE_UP_CONCAT = 0
MOE_GATE_UP_INTERLEAVED = 1
MOE_BF16 = 0
MOE_FP32 = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libmoe_gb300.so")


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("act", ctypes.c_int32),
                ("clamp_limit", ctypes.c_float), ("alpha", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("gate_up_layout", ctypes.c_int32),
                ("out_fp32", ctypes.c_int32)]


class MoePlan(ctypes.Structure):
    _fields_ = [("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("inv", ctypes.c_void_p)]


class MoeBias(ctypes.Structure):
    """moe_bias_t: optional per-expert biases and their gradient outputs."""
    _fields_ = [("b_gate_up", ctypes.c_void_p), ("b_down", ctypes.c_void_p),
                ("db_gate_up", ctypes.c_void_p), ("db_down", ctypes.c_void_p)]


class MoeGrad(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


class MoeMxWeights(ctypes.Structure):
    _fields_ = [("codes_gate_up", ctypes.c_void_p), ("scales_gate_up", ctypes.c_void_p),
                ("codes_down", ctypes.c_void_p), ("scales_down", ctypes.c_void_p)]


class MoeError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, moe_status_string(status), status))


_lib = None


def lib():
    """Load libmoe_gb300.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError("libmoe_gb300.so is not built (run dispatch_gemm_combine_gb300._build"
                           ".build() or __graft_entry__.build())")
    L = ctypes.CDLL(library_path)
    P = ctypes.c_void_p
    S = ctypes.POINTER(MoeShape)
    PL = ctypes.POINTER(MoePlan)
    L.moe_workspace_size.argtypes = [S, ctypes.c_int]
    L.moe_workspace_size.restype = ctypes.c_size_t
    L.moe_saved_size.argtypes = [S]
    L.moe_saved_size.restype = ctypes.c_size_t
    L.moe_plan.argtypes = [S, P, PL, P, ctypes.c_size_t, P]
    L.moe_plan.restype = ctypes.c_int
    L.moe_route.argtypes = [S, P, P, P, PL, P, ctypes.c_size_t, P]
    L.moe_route.restype = ctypes.c_int
    B = ctypes.POINTER(MoeBias)
    L.moe_ffn_fwd.argtypes = [S, P, P, P, P, P, B, PL, P, P, P, ctypes.c_size_t, P]
    L.moe_ffn_fwd.restype = ctypes.c_int
    L.moe_ffn_bwd.argtypes = [S, P, P, P, P, P, P, B, PL, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.moe_ffn_bwd.restype = ctypes.c_int
    L.moe_get_device_error.argtypes = [P, P]
    L.moe_get_device_error.restype = ctypes.c_int
    L.moe_status_string.argtypes = [ctypes.c_int]
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    L.moe_set_wait_timeout_ns.restype = ctypes.c_uint64
    L.moe_kernel_launch_count.argtypes = []
    L.moe_kernel_launch_count.restype = ctypes.c_uint64
    L.moe_profile_enable.argtypes = [ctypes.c_int]
    L.moe_profile_enable.restype = ctypes.c_int
    L.moe_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double),
                                   ctypes.POINTER(ctypes.c_uint64), ctypes.c_int]
    L.moe_profile_read.restype = ctypes.c_int
    L.moe_profile_kernel_name.argtypes = [ctypes.c_int]
    L.moe_profile_kernel_name.restype = ctypes.c_char_p
    L.moe_gather_rows.argtypes = [P, ctypes.c_int64, ctypes.c_int32, P, ctypes.c_int64,
                                  ctypes.c_int64, P, P]
    L.moe_gather_rows.restype = ctypes.c_int
    L.moe_combine_rows.argtypes = [S, P, P, P, ctypes.c_int32, P, P]
    L.moe_combine_rows.restype = ctypes.c_int
    I64, I32, F32, SZ = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    L.moe_rms_norm_workspace_size.argtypes = [I64, I32]
    L.moe_rms_norm_workspace_size.restype = SZ
    L.moe_rms_norm_fwd.argtypes = [I64, I32, I32, P, P, P, F32, P, P, P, P, P]
    L.moe_rms_norm_fwd.restype = ctypes.c_int
    L.moe_rms_norm_bwd.argtypes = [I64, I32, I32, P, P, P, P, P, P, P, P, SZ, P]
    L.moe_rms_norm_bwd.restype = ctypes.c_int
    G = ctypes.POINTER(MoeGrad)
    L.moe_grad_clip_workspace_size.argtypes = [G, I64]
    L.moe_grad_clip_workspace_size.restype = SZ
    L.moe_grad_clip.argtypes = [G, I64, F32, P, P, SZ, P]
    L.moe_grad_clip.restype = ctypes.c_int
    L.moe_mx_quantize.argtypes = [P, I32, I64, I64, I64, P, P, P]
    L.moe_mx_quantize.restype = ctypes.c_int
    L.moe_mx_dequantize.argtypes = [P, P, I64, I64, I64, I32, P, P]
    L.moe_mx_dequantize.restype = ctypes.c_int
    L.moe_few_workspace_size.argtypes = [S]
    L.moe_few_workspace_size.restype = SZ
    L.moe_ffn_few.argtypes = [S, P, P, P, P, P, P, ctypes.POINTER(MoeMxWeights), B, P, P, SZ, P]
    L.moe_ffn_few.restype = ctypes.c_int
    L.moe_join_norm_fwd.argtypes = [I64, I32, I32, P, P, I32, P, P, F32, P, F32, P, P, P, P, P, P]
    L.moe_join_norm_fwd.restype = ctypes.c_int
    L.moe_join_norm_workspace_size.argtypes = [I64, I32]
    L.moe_join_norm_workspace_size.restype = SZ
    L.moe_join_norm_bwd.argtypes = ([I64, I32, I32] + [P] * 9 + [F32] + [P] * 6 + [SZ, P])
    L.moe_join_norm_bwd.restype = ctypes.c_int
    L.moe_route_bwd_workspace_size.argtypes = [S]
    L.moe_route_bwd_workspace_size.restype = SZ
    L.moe_route_bwd.argtypes = [S, P, P, P, P, P, F32, F32, P, P, P, SZ, P]
    L.moe_route_bwd.restype = ctypes.c_int
    L.moe_orthogonalize_workspace_size.argtypes = [I64, I64, I64]
    L.moe_orthogonalize_workspace_size.restype = SZ
    L.moe_orthogonalize.argtypes = [I64, I64, I64, I32, P, I64, I64, I32, P, F32, F32, P, I64, I64, P,
                                    SZ, P]
    L.moe_orthogonalize.restype = ctypes.c_int
    _lib = L
    return L


# ---------------------------------------------------------------- raw C ABI
def moe_workspace_size(shape, which):
    return lib().moe_workspace_size(ctypes.byref(shape), which)


def moe_saved_size(shape):
    return lib().moe_saved_size(ctypes.byref(shape))


def moe_plan(shape, topk_idx, plan, ws, ws_bytes, stream):
    return lib().moe_plan(ctypes.byref(shape), topk_idx, ctypes.byref(plan), ws, ws_bytes, stream)


def _byref(st):
    return ctypes.byref(st) if st is not None else None


def moe_ffn_fwd(shape, x, topk_idx, topk_w, w_gate_up, w_down, bias, plan, y, saved, ws,
                ws_bytes, stream):
    return lib().moe_ffn_fwd(ctypes.byref(shape), x, topk_idx, topk_w, w_gate_up, w_down,
                             _byref(bias), _byref(plan), y, saved, ws, ws_bytes, stream)


def moe_ffn_bwd(shape, dy, x, topk_idx, topk_w, w_gate_up, w_down, bias, plan, saved, dx,
                d_topk_w, dw_gate_up, dw_down, ws, ws_bytes, stream):
    return lib().moe_ffn_bwd(ctypes.byref(shape), dy, x, topk_idx, topk_w, w_gate_up, w_down,
                             _byref(bias), _byref(plan), saved, dx, d_topk_w, dw_gate_up,
                             dw_down, ws, ws_bytes, stream)


def moe_get_device_error(ws, stream):
    return lib().moe_get_device_error(ws, stream)


def moe_status_string(status):
    return lib().moe_status_string(status).decode()


def moe_set_wait_timeout_ns(ns):
    return lib().moe_set_wait_timeout_ns(ns)


def moe_kernel_launch_count():
    return lib().moe_kernel_launch_count()


def moe_profile_enable(on):
    return lib().moe_profile_enable(1 if on else 0)


def moe_profile_kernel_name(kind):
    n = lib().moe_profile_kernel_name(kind)
    return None if n is None else n.decode()


def moe_profile_read():
    """{kernel kind name: (total ms, launches)} since the last read."""
    n = 64
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_uint64 * n)()
    k = lib().moe_profile_read(ms, cnt, n)
    return {moe_profile_kernel_name(i): (ms[i], cnt[i]) for i in range(min(k, n))}


def moe_gather_rows(index, n, div, src, src_rows, row_bytes, dst, stream):
    return lib().moe_gather_rows(index, n, div, src, src_rows, row_bytes, dst, stream)


def moe_combine_rows(shape, inv, topk_w, src, src_fp32, dst, stream):
    return lib().moe_combine_rows(ctypes.byref(shape), inv, topk_w, src, 1 if src_fp32 else 0,
                                  dst, stream)


def moe_plan_noalloc(shape, topk_idx, plan, stream):
    """moe_plan without a workspace, for callers that cannot allocate device
    memory when they build a plan; its scratch is a fixed array inside the
    library (see include/moe.h for the size limit and the sharing rules)."""
    fn = lib().moe_plan_noalloc
    fn.argtypes = [ctypes.POINTER(MoeShape), ctypes.c_void_p, ctypes.POINTER(MoePlan),
                   ctypes.c_void_p]
    fn.restype = ctypes.c_int
    return fn(ctypes.byref(shape), topk_idx, ctypes.byref(plan), stream)


def moe_rms_norm_workspace_size(T, H):
    return lib().moe_rms_norm_workspace_size(T, H)


def moe_rms_norm_fwd(T, H, dtype, x, residual, weight, eps, y, y_scale, total, rstd, stream):
    return lib().moe_rms_norm_fwd(T, H, dtype, x, residual, weight, eps, y, y_scale, total, rstd,
                                  stream)


def moe_rms_norm_bwd(T, H, dtype, dy, d_total, total, rstd, weight, dx, dweight, ws, ws_bytes,
                     stream):
    return lib().moe_rms_norm_bwd(T, H, dtype, dy, d_total, total, rstd, weight, dx, dweight, ws,
                                  ws_bytes, stream)


def moe_grad_clip_workspace_size(grads, n):
    return lib().moe_grad_clip_workspace_size(grads, n)


def moe_grad_clip(grads, n, max_norm, norm_out, ws, ws_bytes, stream):
    return lib().moe_grad_clip(grads, n, max_norm, norm_out, ws, ws_bytes, stream)


def moe_mx_quantize(w, dtype, E, K, N, codes, scales, stream):
    return lib().moe_mx_quantize(w, dtype, E, K, N, codes, scales, stream)


def moe_mx_dequantize(codes, scales, E, K, N, dtype, w, stream):
    return lib().moe_mx_dequantize(codes, scales, E, K, N, dtype, w, stream)


def moe_few_workspace_size(shape):
    return lib().moe_few_workspace_size(ctypes.byref(shape))


def moe_ffn_few(shape, x, x_scale, topk_idx, topk_w, w_gate_up, w_down, mx, bias, y, ws, ws_bytes,
                stream):
    return lib().moe_ffn_few(ctypes.byref(shape), x, x_scale, topk_idx, topk_w, w_gate_up, w_down,
                             _byref(mx), _byref(bias), y, ws, ws_bytes, stream)


def moe_join_norm_fwd(T, H, dtype, y, residual, post_norm, post_weight, gate, residual_scale,
                      weight, eps, total, n, n_scale, rstd_post, rstd, stream):
    return lib().moe_join_norm_fwd(T, H, dtype, y, residual, post_norm, post_weight, gate,
                                   residual_scale, weight, eps, total, n, n_scale, rstd_post, rstd,
                                   stream)


def moe_join_norm_workspace_size(T, H):
    return lib().moe_join_norm_workspace_size(T, H)


def moe_join_norm_bwd(T, H, dtype, dn, d_total, total, rstd, weight, y, rstd_post, post_weight, gate,
                      residual_scale, dy, d_residual, d_gate, d_post_weight, d_weight, ws, ws_bytes,
                      stream):
    return lib().moe_join_norm_bwd(T, H, dtype, dn, d_total, total, rstd, weight, y, rstd_post,
                                   post_weight, gate, residual_scale, dy, d_residual, d_gate,
                                   d_post_weight, d_weight, ws, ws_bytes, stream)


def moe_route_bwd_workspace_size(shape):
    return lib().moe_route_bwd_workspace_size(ctypes.byref(shape))


def moe_route_bwd(shape, logits, topk_idx, topk_w, counts, d_topk_w, balance, z, d_logits, losses,
                  ws, ws_bytes, stream):
    return lib().moe_route_bwd(ctypes.byref(shape), logits, topk_idx, topk_w, counts, d_topk_w,
                               balance, z, d_logits, losses, ws, ws_bytes, stream)


def moe_orthogonalize_workspace_size(E, M, N):
    return lib().moe_orthogonalize_workspace_size(E, M, N)


def moe_orthogonalize(E, M, N, dtype, g, g_ld, g_stride, steps, coefs, eps, scale, out, out_ld,
                      out_stride, ws, ws_bytes, stream):
    """coefs: None, or a ctypes array of 3 * steps floats."""
    return lib().moe_orthogonalize(E, M, N, dtype, g, g_ld, g_stride, steps, coefs, eps, scale, out,
                                   out_ld, out_stride, ws, ws_bytes, stream)


# ---------------------------------------------------------------- torch helpers
def Shape(T, H, I, E, k, act=MOE_ACT_SWIGLU, dtype=MOE_BF16, clamp_limit=7.0, alpha=1.702,
          gate_up_layout=0, out_fp32=0):
    return MoeShape(T, H, I, E, k, act, clamp_limit, alpha, dtype, gate_up_layout,
                    1 if out_fp32 else 0)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    # the raw handle of torch.cuda.current_stream(), without the Stream object (the
    # tensors of the call are on the GPU, so torch's part of it is awake)
    from torch import _C
    return _C._cuda_getCurrentRawStream(_C._cuda_getDevice())


def _check(status, where):
    if status != MOE_OK:
        raise MoeError(status, where)


def alloc_plan(shape, device="cuda"):
    """int32 device tensors for a plan plus the MoePlan struct pointing at them."""
    import torch
    Tk = max(1, shape.T * shape.k)
    t = {"counts": torch.empty(shape.E, dtype=torch.int32, device=device),
         "offsets": torch.empty(shape.E + 1, dtype=torch.int32, device=device),
         "perm": torch.empty(Tk, dtype=torch.int32, device=device),
         "inv": torch.empty(Tk, dtype=torch.int32, device=device)}
    st = MoePlan(t["counts"].data_ptr(), t["offsets"].data_ptr(), t["perm"].data_ptr(),
                 t["inv"].data_ptr())
    return t, st


def workspace(shape, which, device="cuda"):
    """Zero-filled workspace for call kind `which` (0 plan, 1 fwd, 2 bwd, 3 bwd
    without a saved context)."""
    import torch
    n = moe_workspace_size(shape, which)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def saved_buffer(shape, device="cuda"):
    import torch
    return torch.empty(moe_saved_size(shape), dtype=torch.uint8, device=device)


def route(shape, logits, topk_idx, topk_w, plan_struct=None, ws=None, stream=None):
    """Top-k ids and weights of fp32 logits [T,E] (and the plan, given one)."""
    _check(lib().moe_route(ctypes.byref(shape), _ptr(logits), _ptr(topk_idx), _ptr(topk_w),
                           ctypes.byref(plan_struct) if plan_struct is not None else None,
                           _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "moe_route")


def bias_struct(b_gate_up=None, b_down=None, db_gate_up=None, db_down=None):
    """MoeBias over torch tensors (None = absent), or None when all are absent."""
    ts = (b_gate_up, b_down, db_gate_up, db_down)
    if all(t is None for t in ts):
        return None
    s = MoeBias(*[_ptr(t) for t in ts])
    s.tensors = ts                   # they live as long as the struct
    return s


def plan(shape, topk_idx, plan_struct, ws, stream=None):
    _check(moe_plan(shape, _ptr(topk_idx), plan_struct, _ptr(ws), ws.numel(), _stream(stream)),
           "moe_plan")


def ffn_fwd(shape, x, topk_idx, topk_w, w_gate_up, w_down, y, ws, plan_struct=None, saved=None,
            stream=None, bias=None):
    """bias: a MoeBias (see bias_struct) or None."""
    _check(moe_ffn_fwd(shape, _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(w_gate_up),
                       _ptr(w_down), bias, plan_struct, _ptr(y), _ptr(saved), _ptr(ws),
                       ws.numel(), _stream(stream)), "moe_ffn_fwd")


def ffn_bwd(shape, dy, x, topk_idx, topk_w, w_gate_up, w_down, plan_struct, saved, dx, d_topk_w,
            dw_gate_up, dw_down, ws, stream=None, bias=None):
    """bias: a MoeBias (see bias_struct; it also names the bias-gradient
    outputs) or None."""
    _check(moe_ffn_bwd(shape, _ptr(dy), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(w_gate_up),
                       _ptr(w_down), bias, plan_struct, _ptr(saved), _ptr(dx), _ptr(d_topk_w),
                       _ptr(dw_gate_up), _ptr(dw_down), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_ffn_bwd")


def gather_rows(index, div, src, dst, stream=None):
    """dst[r] = src[index[r] // div] for every row r of dst (torch tensors on
    the device; src and dst rows of equal byte size, index int32)."""
    n = index.numel()
    row_bytes = dst.element_size() * (dst.numel() // max(1, dst.shape[0])) if dst.dim() else 0
    if dst.shape[0] != n:
        raise ValueError("gather_rows: dst has %d rows for %d indices" % (dst.shape[0], n))
    src_rows = src.shape[0] if src.dim() else 1
    if n and src.element_size() * (src.numel() // max(1, src_rows)) != row_bytes:
        raise ValueError("gather_rows: src and dst rows differ in size")
    _check(moe_gather_rows(_ptr(index), n, div, _ptr(src), src_rows, row_bytes, _ptr(dst),
                           _stream(stream)), "moe_gather_rows")


def combine_rows(shape, inv, src, dst, topk_w=None, stream=None):
    """dst[t] = sum_j (topk_w[t, j] or 1) * src[inv[t*k + j]] (torch tensors;
    src fp32 or the storage dtype, dst as shape.out_fp32 says)."""
    import torch
    _check(moe_combine_rows(shape, _ptr(inv), _ptr(topk_w), _ptr(src), src.dtype == torch.float32,
                            _ptr(dst), _stream(stream)), "moe_combine_rows")


def _storage_dtype(where, t):
    import torch
    if t.dtype is torch.bfloat16:
        return MOE_BF16
    if t.dtype is torch.float32:
        return MOE_FP32
    raise ValueError("%s: bfloat16 or float32 expected, got %s" % (where, t.dtype))


def _dense(where, name, t, shape, dtype):
    """The tensor's address, after a check that it is what the call reads or
    writes: this shape and dtype, dense and row-major, on the GPU.  None passes."""
    if t is None:
        return None
    if t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.shape == shape:
        return t.data_ptr()
    raise ValueError("%s: %s must be a dense %s tensor of shape %s on the GPU, got %s %s%s" % (
        where, name, dtype, tuple(shape), t.dtype, tuple(t.shape),
        "" if t.is_contiguous() else " (strided)"))


def _ws(where, ws):
    """(address, bytes) of a workspace, after a check that it is on the GPU and dense."""
    if ws is None:
        return None, 0
    if ws.is_cuda and ws.is_contiguous():
        return ws.data_ptr(), ws.numel() * ws.element_size()
    raise ValueError("%s: the workspace must be a dense tensor on the GPU" % where)


def rms_norm_workspace(T, H, device="cuda"):
    """Zero-filled workspace of rms_norm_bwd for at most T rows of H columns."""
    import torch
    n = moe_rms_norm_workspace_size(T, H)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_rms_norm_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def rms_norm_fwd(x, weight, y, eps=1e-6, residual=None, total=None, rstd=None, y_scale=None,
                 stream=None):
    """y = rms_norm(x + residual) * weight over the last axis of x [T,H].  y is
    in x's dtype, or with y_scale [T,H/32] (uint8) e4m3 codes [T,H] (uint8 or
    float8_e4m3fn); total [T,H] and rstd [T] (fp32) receive x + residual and
    1 / rms, which the backward wants."""
    import torch
    T, H = x.shape
    w, dt, shape = "rms_norm_fwd", x.dtype, x.shape
    code = _storage_dtype(w, x)
    ydt = dt
    if y_scale is not None:
        ydt = torch.float8_e4m3fn if y.dtype is torch.float8_e4m3fn else torch.uint8
    _check(lib().moe_rms_norm_fwd(
        T, H, code, _dense(w, "x", x, shape, dt), _dense(w, "residual", residual, shape, dt),
        _dense(w, "weight", weight, (H,), dt), eps, _dense(w, "y", y, shape, ydt),
        _dense(w, "y_scale", y_scale, (T, H // 32), torch.uint8),
        _dense(w, "total", total, shape, dt), _dense(w, "rstd", rstd, (T,), torch.float32),
        _stream(stream)), "moe_rms_norm_fwd")


def rms_norm_bwd(dy, total, rstd, weight, dx, dweight=None, d_total=None, ws=None, stream=None):
    """Gradient of rms_norm_fwd: dx [T,H] (of x and of the residual) and dweight
    [H] (fp32, None for a frozen weight), from dy, the forward's total and rstd,
    and d_total, the gradient that reaches total from elsewhere (or None).  ws:
    rms_norm_workspace(T, H), needed with dweight."""
    import torch
    T, H = dy.shape
    w, dt, shape = "rms_norm_bwd", dy.dtype, dy.shape
    code = _storage_dtype(w, dy)
    _check(lib().moe_rms_norm_bwd(
        T, H, code, _dense(w, "dy", dy, shape, dt), _dense(w, "d_total", d_total, shape, dt),
        _dense(w, "total", total, shape, dt), _dense(w, "rstd", rstd, (T,), torch.float32),
        _dense(w, "weight", weight, (H,), dt), _dense(w, "dx", dx, shape, dt),
        _dense(w, "dweight", dweight, (H,), torch.float32), *_ws(w, ws), _stream(stream)),
        "moe_rms_norm_bwd")


def grad_table(grads, out=None):
    """The list of gradients that grad_clip works on: an array of MoeGrad over
    dense tensors (bf16 or fp32, mixed as they come).  out: the tensors that
    receive the scaled gradients, None for in place, False for the norm alone.
    The table keeps addresses, not tensors: build it again when they move."""
    grads = list(grads)
    out = grads if out is None else ([None] * len(grads) if out is False else list(out))
    if len(out) != len(grads):
        raise ValueError("grad_table: %d outputs for %d gradients" % (len(out), len(grads)))
    t = (MoeGrad * max(1, len(grads)))()
    for i, (g, o) in enumerate(zip(grads, out)):
        code = _storage_dtype("grad_table", g)
        t[i] = MoeGrad(_dense("grad_table", "gradient %d" % i, g, g.shape, g.dtype),
                       _dense("grad_table", "output %d" % i, o, g.shape, g.dtype), g.numel(), code)
    t.count = len(grads)
    return t


def grad_clip_workspace(table, device="cuda"):
    """Zero-filled workspace of grad_clip for this table."""
    import torch
    n = moe_grad_clip_workspace_size(table, table.count)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_grad_clip_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def grad_clip(table, max_norm, norm, ws, stream=None):
    """Scale the table's gradients so that their global norm is at most max_norm.
    norm [2] (fp32, on the GPU) receives the norm before and the factor applied
    (1 where nothing is clipped, or where the norm is not finite)."""
    import torch
    _check(lib().moe_grad_clip(table, table.count, max_norm,
                               _dense("grad_clip", "norm", norm, (2,), torch.float32),
                               *_ws("grad_clip", ws), _stream(stream)), "moe_grad_clip")


def mx_alloc(E, K, N, device="cuda"):
    """(codes [E,N,K/2], scales [E,N,K/32]), uint8, for weights [E,K,N]."""
    import torch
    return (torch.empty((E, N, K // 2), dtype=torch.uint8, device=device),
            torch.empty((E, N, K // 32), dtype=torch.uint8, device=device))


def mx_quantize(w, codes, scales, stream=None):
    """Microscaled 4-bit codes and scale bytes (mx_alloc) of weights w [E,K,N]."""
    import torch
    E, K, N = w.shape
    f = "mx_quantize"
    _check(lib().moe_mx_quantize(
        _dense(f, "w", w, w.shape, w.dtype), _storage_dtype(f, w), E, K, N,
        _dense(f, "codes", codes, (E, N, K // 2), torch.uint8),
        _dense(f, "scales", scales, (E, N, K // 32), torch.uint8), _stream(stream)),
        "moe_mx_quantize")


def mx_dequantize(codes, scales, w, stream=None):
    """The values of microscaled codes, into w [E,K,N] (bf16 or fp32)."""
    import torch
    E, K, N = w.shape
    f = "mx_dequantize"
    _check(lib().moe_mx_dequantize(
        _dense(f, "codes", codes, (E, N, K // 2), torch.uint8),
        _dense(f, "scales", scales, (E, N, K // 32), torch.uint8), E, K, N, _storage_dtype(f, w),
        _dense(f, "w", w, w.shape, w.dtype), _stream(stream)), "moe_mx_dequantize")


def few_workspace(shape, device="cuda"):
    """Zero-filled workspace of ffn_few for this shape (T <= 128)."""
    import torch
    n = moe_few_workspace_size(shape)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_few_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def mx_struct(codes_gate_up, scales_gate_up, codes_down, scales_down):
    """MoeMxWeights over the tensors mx_quantize filled for w_gate_up and w_down
    (ffn_few checks their shapes)."""
    import torch
    ts = (codes_gate_up, scales_gate_up, codes_down, scales_down)
    s = MoeMxWeights(*[_dense("mx_struct", f[0], t, t.shape, torch.uint8)
                       for f, t in zip(MoeMxWeights._fields_, ts)])
    s.tensors = ts                   # they live as long as the struct
    s.shapes = tuple(t.shape for t in ts)
    return s


def _check_mx(where, mx, E, H, I):
    """The shapes of mx_struct's tensors are those of a layer with these sizes."""
    if mx.shapes != ((E, 2 * I, H // 2), (E, 2 * I, H // 32), (E, H, I // 2), (E, H, I // 32)):
        raise ValueError("%s: 4-bit weights of shapes %s are not those of a layer with %d experts, H = %d, I = %d"
                         % (where, [tuple(s) for s in mx.shapes], E, H, I))


def ffn_few(shape, x, topk_idx, topk_w, w_gate_up, w_down, y, ws, stream=None, bias=None,
            x_scale=None, mx=None):
    """y = layer(x) for at most 128 tokens (inference).  x [T,H] in the storage
    dtype, or e4m3 codes (uint8 or float8_e4m3fn) with x_scale [T,H/32]; the
    weights as ffn_fwd takes them, or None for both with mx (see mx_struct);
    bias: see bias_struct; ws: few_workspace(shape)."""
    import torch
    f, T, H, I, E, k = "ffn_few", shape.T, shape.H, shape.I, shape.E, shape.k
    dt = torch.float32 if shape.dtype == MOE_FP32 else torch.bfloat16
    xdt = dt
    if x_scale is not None:
        xdt = torch.float8_e4m3fn if x.dtype is torch.float8_e4m3fn else torch.uint8
    if hasattr(mx, "shapes"):        # (a struct filled by hand names no tensors)
        _check_mx(f, mx, E, H, I)
    if hasattr(bias, "tensors"):
        _dense(f, "b_gate_up", bias.tensors[0], (E, 2 * I), dt)
        _dense(f, "b_down", bias.tensors[1], (E, H), dt)
    _check(lib().moe_ffn_few(
        ctypes.byref(shape), _dense(f, "x", x, (T, H), xdt),
        _dense(f, "x_scale", x_scale, (T, H // 32), torch.uint8),
        _dense(f, "topk_idx", topk_idx, (T, k), torch.int32),
        _dense(f, "topk_w", topk_w, (T, k), torch.float32),
        _dense(f, "w_gate_up", w_gate_up, (E, H, 2 * I), dt),
        _dense(f, "w_down", w_down, (E, I, H), dt), _byref(mx), _byref(bias),
        _dense(f, "y", y, (T, H), torch.float32 if shape.out_fp32 else dt), *_ws(f, ws),
        _stream(stream)), "moe_ffn_few")


def join_norm_workspace(T, H, device="cuda"):
    """Zero-filled workspace of join_norm_bwd for at most T rows of H columns."""
    import torch
    n = moe_join_norm_workspace_size(T, H)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_join_norm_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def join_norm_fwd(y, residual, total, post_norm=True, post_weight=None, gate=None, residual_scale=1.0,
                  weight=None, n=None, n_scale=None, eps=1e-6, rstd_post=None, rstd=None, stream=None):
    """A block's output y [T,H] joins the residual stream:
        total = residual_scale * residual + gate * (rms_norm(y) * post_weight)
    (post_norm=False: y * post_weight without the norm; gate [T] fp32, one factor per
    token; either may be None), and the norm before the next block:
        n = rms_norm(total) * weight
    (both None where none follows), in y's dtype, or with n_scale [T,H/32] (uint8) as
    e4m3 codes (uint8 or float8_e4m3fn).  rstd_post and rstd [T] (fp32) receive both
    norms' 1 / rms for the backward."""
    import torch
    T, H = y.shape
    f, dt, shape = "join_norm_fwd", y.dtype, y.shape
    code = _storage_dtype(f, y)
    ndt = dt
    if n_scale is not None and n is not None:
        ndt = torch.float8_e4m3fn if n.dtype is torch.float8_e4m3fn else torch.uint8
    _check(lib().moe_join_norm_fwd(
        T, H, code, _dense(f, "y", y, shape, dt), _dense(f, "residual", residual, shape, dt),
        1 if post_norm else 0, _dense(f, "post_weight", post_weight, (H,), dt),
        _dense(f, "gate", gate, (T,), torch.float32), residual_scale,
        _dense(f, "weight", weight, (H,), dt), eps, _dense(f, "total", total, shape, dt),
        _dense(f, "n", n, shape, ndt), _dense(f, "n_scale", n_scale, (T, H // 32), torch.uint8),
        _dense(f, "rstd_post", rstd_post, (T,), torch.float32),
        _dense(f, "rstd", rstd, (T,), torch.float32), _stream(stream)), "moe_join_norm_fwd")


def join_norm_bwd(y, dy, d_residual, d_total=None, dn=None, total=None, weight=None, rstd=None,
                  post_norm=True, post_weight=None, rstd_post=None, gate=None, residual_scale=1.0,
                  d_gate=None, d_post_weight=None, d_weight=None, ws=None, stream=None):
    """Gradient of join_norm_fwd: dy and d_residual [T,H] from dn (the gradient of n;
    None where no norm followed) and d_total (the gradient that reaches total from
    elsewhere, or None), with what the forward had and gave.  d_gate [T],
    d_post_weight [H] and d_weight [H] (fp32) are optional; ws: join_norm_workspace(T, H),
    needed with either weight's gradient."""
    import torch
    T, H = y.shape
    f, dt, shape = "join_norm_bwd", y.dtype, y.shape
    code = _storage_dtype(f, y)
    if bool(post_norm) != (rstd_post is not None):
        raise ValueError("join_norm_bwd: rstd_post is given with a post norm, and only then")
    _check(lib().moe_join_norm_bwd(
        T, H, code, _dense(f, "dn", dn, shape, dt), _dense(f, "d_total", d_total, shape, dt),
        _dense(f, "total", total, shape, dt), _dense(f, "rstd", rstd, (T,), torch.float32),
        _dense(f, "weight", weight, (H,), dt), _dense(f, "y", y, shape, dt),
        _dense(f, "rstd_post", rstd_post, (T,), torch.float32),
        _dense(f, "post_weight", post_weight, (H,), dt), _dense(f, "gate", gate, (T,), torch.float32),
        residual_scale, _dense(f, "dy", dy, shape, dt),
        _dense(f, "d_residual", d_residual, shape, dt),
        _dense(f, "d_gate", d_gate, (T,), torch.float32),
        _dense(f, "d_post_weight", d_post_weight, (H,), torch.float32),
        _dense(f, "d_weight", d_weight, (H,), torch.float32), *_ws(f, ws), _stream(stream)),
        "moe_join_norm_bwd")


def route_bwd_workspace(shape, device="cuda"):
    """Zero-filled workspace of route_bwd for this shape (T, E and k count)."""
    import torch
    n = moe_route_bwd_workspace_size(shape)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_route_bwd_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def route_bwd(shape, logits, d_logits, ws, topk_idx=None, topk_w=None, d_topk_w=None, counts=None,
              balance=0.0, z=0.0, losses=None, stream=None):
    """d_logits [T,E] (fp32): the gradient of <d_topk_w, topk_w> with respect to the
    logits that route() took, plus balance times that of the load-balancing loss and z
    times that of the z-loss (include/moe.h); losses [2] (fp32) receives both.  counts:
    the plan's."""
    import torch
    f, T, E, k, f32 = "route_bwd", shape.T, shape.E, shape.k, torch.float32
    _check(lib().moe_route_bwd(
        ctypes.byref(shape), _dense(f, "logits", logits, (T, E), f32),
        _dense(f, "topk_idx", topk_idx, (T, k), torch.int32), _dense(f, "topk_w", topk_w, (T, k), f32),
        _dense(f, "counts", counts, (E,), torch.int32), _dense(f, "d_topk_w", d_topk_w, (T, k), f32),
        balance, z, _dense(f, "d_logits", d_logits, (T, E), f32), _dense(f, "losses", losses, (2,), f32),
        *_ws(f, ws), _stream(stream)), "moe_route_bwd")


def _matrices(where, name, t, dtype):
    """(address, row stride, matrix stride) of [M,N] or [E,M,N], after a check that it
    is of this dtype, on the GPU, with its rows' elements side by side."""
    if t.dtype is not dtype or not t.is_cuda or t.dim() not in (2, 3):
        raise ValueError("%s: %s must be a %s tensor [M,N] or [E,M,N] on the GPU, got %s %s" % (
            where, name, dtype, t.dtype, tuple(t.shape)))
    M, N = t.shape[-2:]
    ld = t.stride(-2) if M > 1 else N
    if (N > 1 and t.stride(-1) != 1) or ld < N:
        raise ValueError("%s: %s's rows must be contiguous and apart, got strides %s" % (
            where, name, tuple(t.stride())))
    return t.data_ptr(), ld, t.stride(0) if t.dim() == 3 and t.shape[0] > 1 else M * ld


def orthogonalize_workspace(g, device=None):
    """Zero-filled workspace of orthogonalize for g [M,N] or [E,M,N] (fewer matrices
    of that size take no more)."""
    import torch
    E = g.shape[0] if g.dim() == 3 else 1
    n = moe_orthogonalize_workspace_size(E, *g.shape[-2:])
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_orthogonalize_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=g.device if device is None else device)


def orthogonalize(g, out, ws, steps=5, coefs=None, eps=1e-7, scale=1.0, stream=None):
    """out = scale * (g made orthogonal by `steps` Newton-Schulz products), for each
    matrix of g [M,N] or [E,M,N] (bf16 or fp32); out of the same shape, bf16.  Rows may
    lie apart: the gate half of dw_gate_up is dw_gate_up[:, :, :I].  coefs: (c0, c1, c2)
    for every step, or a list of `steps` of them; ws: orthogonalize_workspace(g).  The
    steps run in fp16 with fp32 sums: what that costs is told in include/moe.h (1e-3 in
    the 2-norm for a Gaussian g, up to 8e-2 for one of rank 4)."""
    import torch
    f = "orthogonalize"
    code = _storage_dtype(f, g)
    if out.shape != g.shape:
        raise ValueError("orthogonalize: out has shape %s for %s" % (tuple(out.shape), tuple(g.shape)))
    if coefs is not None:
        if len(coefs) == 0 or not 1 <= steps <= 32:
            raise ValueError("orthogonalize: 1 to 32 steps with three coefficients each")
        rows = [tuple(c) for c in coefs] if hasattr(coefs[0], "__len__") else [tuple(coefs)] * steps
        if len(rows) != steps or any(len(c) != 3 for c in rows):
            raise ValueError("orthogonalize: three coefficients, or %d times three" % steps)
        coefs = (ctypes.c_float * (3 * steps))(*[v for c in rows for v in c])
    _check(lib().moe_orthogonalize(
        g.shape[0] if g.dim() == 3 else 1, g.shape[-2], g.shape[-1], code,
        *_matrices(f, "g", g, g.dtype), steps, coefs, eps, scale,
        *_matrices(f, "out", out, torch.bfloat16), *_ws(f, ws), _stream(stream)), "moe_orthogonalize")


def check_device_error(ws, stream=None):
    """Synchronise and raise MoeError if a kernel recorded a device-side error."""
    _check(moe_get_device_error(_ptr(ws), _stream(stream)), "device")
