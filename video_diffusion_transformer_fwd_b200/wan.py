"""ctypes binding of libwan (the C ABI declared in include/wan.h).

Argument marshalling only: the raw entry points keep the C names
(``wan_block_forward`` and so on) and take integer device addresses; the
torch helpers below them pull ``data_ptr()`` and the current CUDA stream out
of tensors and raise ``WanError`` on a nonzero status. Every computation runs
inside the library. Loading fails loudly if ``libwan.so`` has not been built.
"""
from __future__ import annotations

import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libwan.so")

WAN_OK, WAN_EINVAL, WAN_EALIGN, WAN_EUNSUPPORTED, WAN_ECUDA, WAN_ETIMEOUT, WAN_EBOUNDS = 0, -1, -2, -3, -4, -5, -6
WAN_F32, WAN_BF16, WAN_FP8, WAN_FP8_ATTN = 0, 1, 2, 3
WAN_ACT_NONE, WAN_ACT_GELU_TANH, WAN_ACT_SILU, WAN_ACT_RELU = range(4)
WAN_NOALLOC_WORKSPACE_BYTES = 16 << 20
(WAN_WS_ACT, WAN_WS_QKV, WAN_WS_O, WAN_WS_QC, WAN_WS_KVC, WAN_WS_OC, WAN_WS_H, WAN_WS_MOD,
 WAN_WS_STATS, WAN_WS_A8, WAN_WS_ASCALE, WAN_WS_ATTN8) = range(12)
(WAN_K_GEMM_TC, WAN_K_GEMM_SIMT, WAN_K_ATTN_SELF, WAN_K_ATTN_CROSS, WAN_K_ATTN_SIMT, WAN_K_LAYERNORM,
 WAN_K_QKNORM_ROPE, WAN_K_EULER, WAN_K_MISC, WAN_K_ATTN_TC, WAN_K_MODEL, WAN_K_QUANT) = range(12)
WAN_K_COUNT = 12
KERNEL_CLASS_NAMES = ("gemm_tc", "gemm_simt", "attn_self", "attn_cross", "attn_simt", "layernorm",
                      "qknorm_rope", "euler_cfg", "misc", "attn_tc", "model", "quant")
STATUS_NAMES = {0: "WAN_OK", -1: "WAN_EINVAL", -2: "WAN_EALIGN", -3: "WAN_EUNSUPPORTED",
                -4: "WAN_ECUDA", -5: "WAN_ETIMEOUT", -6: "WAN_EBOUNDS"}


class WanError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


class wan_dims(ctypes.Structure):
    _fields_ = [("F", ctypes.c_int), ("H", ctypes.c_int), ("W", ctypes.c_int),
                ("dim", ctypes.c_int), ("heads", ctypes.c_int), ("ffn_dim", ctypes.c_int),
                ("text_len", ctypes.c_int), ("eps", ctypes.c_float), ("dtype", ctypes.c_int),
                ("e0_per_token", ctypes.c_int)]


WEIGHT_FIELDS = ("modulation", "wq", "bq", "wk", "bk", "wv", "bv", "wo", "bo", "gq", "gk",
                 "g3", "b3", "cwq", "cbq", "cwk", "cbk", "cwv", "cbv", "cwo", "cbo",
                 "cgq", "cgk", "w1", "b1", "w2", "b2", "w_scales")
# the ten projection matrices, in the order of wan_block_weights.w_scales
FP8_MATRICES = ("wq", "wk", "wv", "wo", "cwq", "cwk", "cwv", "cwo", "w1", "w2")


class wan_block_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in WEIGHT_FIELDS]


class wan_model_dims(ctypes.Structure):
    _fields_ = [("C_in", ctypes.c_int), ("C_out", ctypes.c_int), ("F", ctypes.c_int),
                ("H", ctypes.c_int), ("W", ctypes.c_int), ("dim", ctypes.c_int),
                ("heads", ctypes.c_int), ("ffn_dim", ctypes.c_int), ("text_len", ctypes.c_int),
                ("text_dim", ctypes.c_int), ("freq_dim", ctypes.c_int), ("eps", ctypes.c_float),
                ("dtype", ctypes.c_int), ("t_per_token", ctypes.c_int)]


MODEL_WEIGHT_FIELDS = ("patch_w", "patch_b", "text_w1", "text_b1", "text_w2", "text_b2",
                       "time_w1", "time_b1", "time_w2", "time_b2", "proj_w", "proj_b",
                       "head_mod", "head_w", "head_b")


class wan_model_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in MODEL_WEIGHT_FIELDS]


class wan_linear_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("a", "w", "a_scale", "w_scale", "bias", "residual", "out")] +
                [(n, ctypes.c_int64) for n in ("lda", "ldw", "ldr", "ldo")] +
                [(n, ctypes.c_int) for n in ("M", "N", "K", "dtype", "w_scale_rows", "activation", "res_dtype",
                                             "out_dtype")])


class wan_rmsnorm_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "residual", "gain", "h_out", "y", "row_scale")] +
                [(n, ctypes.c_int64) for n in ("ldx", "ldr", "ldh", "ldy")] +
                [(n, ctypes.c_int) for n in ("rows", "D", "x_dtype", "res_dtype", "y_dtype")] +
                [("eps", ctypes.c_float)])


# the same layouts for struct.pack: a small call is bound by its host work, and
# one packed argument costs a quarter of twenty converted ones
_LINEAR_ARGS, _RMSNORM_ARGS = struct.Struct("@7P4q8i"), struct.Struct("@6P4q5if")

_c_int, _vp, _sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t

_SIGS = {
    "wan_last_error": (ctypes.c_char_p, []),
    "wan_rope_freqs": (_c_int, [_c_int, _c_int, ctypes.c_double, _vp, _vp]),
    "wan_block_workspace_bytes": (_sz, [ctypes.POINTER(wan_dims), _c_int]),
    "wan_block_workspace_offset": (_sz, [ctypes.POINTER(wan_dims), _c_int, _c_int]),
    "wan_block_forward": (_c_int, [ctypes.POINTER(wan_dims), _c_int, _vp, _vp, _vp, _vp,
                                   ctypes.POINTER(wan_block_weights), _vp, _c_int, _vp, _sz, _vp]),
    "wan_block_forward_noalloc": (_c_int, [ctypes.POINTER(wan_dims), _c_int, _vp, _vp, _vp, _vp,
                                           ctypes.POINTER(wan_block_weights), _vp, _c_int, _vp]),
    "wan_block_sp_workspace_bytes": (_sz, [ctypes.POINTER(wan_dims), _c_int, _c_int]),
    "wan_block_sp_qkv": (_c_int, [ctypes.POINTER(wan_dims), _c_int, _c_int, _c_int, _vp, _vp,
                                  ctypes.POINTER(wan_block_weights), _vp, _c_int, _vp, _vp, _sz, _vp]),
    "wan_block_sp_finish": (_c_int, [ctypes.POINTER(wan_dims), _c_int, _c_int, _vp, _vp, _vp, _vp,
                                     ctypes.POINTER(wan_block_weights), _vp, _vp, _sz, _vp]),
    "wan_permute_chunks": (_c_int, [_vp, _vp, _c_int, ctypes.POINTER(ctypes.c_int),
                                    ctypes.POINTER(ctypes.c_int), _sz, _vp]),
    "wan_attention": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp,
                               _vp, ctypes.c_float, ctypes.POINTER(ctypes.c_int), _vp, _c_int, _vp]),
    "wan_euler_cfg_step": (_c_int, [_vp, _vp, _vp, _c_int, _sz, ctypes.c_float, ctypes.c_float,
                                    ctypes.c_float, _vp]),
    "wan_device_status": (_c_int, [_vp]),
    "wan_debug_bounds": (_c_int, []),
    "wan_profile_enable": (_c_int, [_c_int]),
    "wan_selftest_watchdog": (_c_int, [_vp]),
    "wan_profile_read": (_c_int, [_c_int, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_double)]),
    "wan_model_workspace_bytes": (_sz, [ctypes.POINTER(wan_model_dims), _c_int]),
    "wan_quantize_fp8": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "wan_linear_fp8": (_c_int, [_c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "wan_linear": (_c_int, [_vp, _vp]),
    "wan_rmsnorm": (_c_int, [_vp, _vp]),
    "wan_attention_8bit_workspace_bytes": (_sz, [_c_int, _c_int, _c_int, _c_int]),
    "wan_unipc_coefficients": (_c_int, [ctypes.POINTER(ctypes.c_double), _c_int, _c_int, _c_int, _c_int,
                                        ctypes.POINTER(ctypes.c_double)]),
    "wan_unipc_step": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _sz, ctypes.c_float, ctypes.c_float,
                                ctypes.POINTER(ctypes.c_double), _vp]),
    "wan_attention_8bit": (_c_int, [_c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp, ctypes.c_float,
                                    _vp, _sz, _vp]),
    "wan_model_forward": (_c_int, [ctypes.POINTER(wan_model_dims), _c_int, _vp, _vp, _vp, _vp,
                                   ctypes.POINTER(wan_model_weights),
                                   ctypes.POINTER(wan_block_weights), _c_int, _vp, _c_int, _vp,
                                   _vp, _sz, _vp]),
}

_lib = None


def load(path: str | None = None):
    """Load libwan.so (raises if it is missing: there is no fallback). The
    environment variable WAN_LIBRARY may name another build of the library
    (the debug build, ``build_lib.build(debug=True)``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or os.environ.get("WAN_LIBRARY") or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libwan.so not built at {path}; run "
                           "`python -m video_diffusion_transformer_fwd_b200.build_lib`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def wan_last_error() -> bytes:
    return load().wan_last_error()


def last_error() -> str:
    return wan_last_error().decode()


def check(rc: int):
    if rc != WAN_OK:
        raise WanError(rc, last_error())


# ---------------------------------------------------------------- raw C entry points
def wan_rope_freqs(head_dim, max_pos, theta, table, stream):
    return load().wan_rope_freqs(head_dim, max_pos, theta, table, stream)


def wan_block_workspace_bytes(dims, B):
    return load().wan_block_workspace_bytes(ctypes.byref(dims), B)


def wan_block_workspace_offset(dims, B, which):
    return load().wan_block_workspace_offset(ctypes.byref(dims), B, which)


def wan_block_forward(dims, B, x, ctx, ctx_lens, e0, weights, rope, rope_max_pos, workspace,
                      ws_bytes, stream):
    return load().wan_block_forward(ctypes.byref(dims), B, x, ctx, ctx_lens, e0,
                                    ctypes.byref(weights), rope, rope_max_pos, workspace,
                                    ws_bytes, stream)


def wan_block_forward_noalloc(dims, B, x, ctx, ctx_lens, e0, weights, rope, rope_max_pos, stream):
    return load().wan_block_forward_noalloc(ctypes.byref(dims), B, x, ctx, ctx_lens, e0,
                                            ctypes.byref(weights), rope, rope_max_pos, stream)


def wan_block_sp_workspace_bytes(dims, B, rows):
    return load().wan_block_sp_workspace_bytes(ctypes.byref(dims), B, rows)


def wan_block_sp_qkv(dims, B, rows, tok0, x, e0, weights, rope, rope_max_pos, qkv, workspace, ws_bytes,
                     stream):
    return load().wan_block_sp_qkv(ctypes.byref(dims), B, rows, tok0, x, e0, ctypes.byref(weights), rope,
                                   rope_max_pos, qkv, workspace, ws_bytes, stream)


def wan_block_sp_finish(dims, B, rows, x, ctx, ctx_lens, e0, weights, o, workspace, ws_bytes, stream):
    return load().wan_block_sp_finish(ctypes.byref(dims), B, rows, x, ctx, ctx_lens, e0, ctypes.byref(weights),
                                      o, workspace, ws_bytes, stream)


def wan_permute_chunks(src, dst, ndim, dims, perm, chunk_bytes, stream):
    d = (ctypes.c_int * max(ndim, 1))(*dims)
    p = (ctypes.c_int * max(ndim, 1))(*perm)
    return load().wan_permute_chunks(src, dst, ndim, d, p, chunk_bytes, stream)


def wan_attention(B, heads, Lq, Lk, head_dim, dtype, q, k, v, o, k_lens, scale, grid, rope,
                  rope_max_pos, stream):
    g = None if grid is None else (ctypes.c_int * 3)(*grid)
    return load().wan_attention(B, heads, Lq, Lk, head_dim, dtype, q, k, v, o, k_lens, scale,
                                g, rope, rope_max_pos, stream)


def wan_euler_cfg_step(x, v_cond, v_uncond, v_dtype, n, guide_scale, sigma, sigma_next, stream):
    return load().wan_euler_cfg_step(x, v_cond, v_uncond, v_dtype, n, guide_scale, sigma,
                                     sigma_next, stream)


def wan_model_workspace_bytes(dims, B):
    return load().wan_model_workspace_bytes(ctypes.byref(dims), B)


def wan_model_forward(dims, B, latent, t, text, ctx_lens, weights, blocks, num_blocks, rope,
                      rope_max_pos, out, workspace, ws_bytes, stream):
    return load().wan_model_forward(ctypes.byref(dims), B, latent, t, text, ctx_lens,
                                    ctypes.byref(weights), blocks, num_blocks, rope, rope_max_pos,
                                    out, workspace, ws_bytes, stream)


def wan_quantize_fp8(src, src_dtype, rows, cols, per_row, q, scale, stream):
    return load().wan_quantize_fp8(src, src_dtype, rows, cols, per_row, q, scale, stream)


def wan_linear_fp8(M, N, K, a, a_scale, w, w_scale, bias, out, stream):
    return load().wan_linear_fp8(M, N, K, a, a_scale, w, w_scale, bias, out, stream)


def wan_linear(args, stream):
    """args: a wan_linear_args, or None."""
    return load().wan_linear(None if args is None else ctypes.addressof(args), stream)


def wan_rmsnorm(args, stream):
    """args: a wan_rmsnorm_args, or None."""
    return load().wan_rmsnorm(None if args is None else ctypes.addressof(args), stream)


def wan_attention_8bit_workspace_bytes(B, heads, Lq, Lk):
    return load().wan_attention_8bit_workspace_bytes(B, heads, Lq, Lk)


def wan_attention_8bit(B, heads, Lq, Lk, q, k, v, o, k_lens, scale, workspace, ws_bytes, stream):
    return load().wan_attention_8bit(B, heads, Lq, Lk, q, k, v, o, k_lens, scale, workspace, ws_bytes,
                                     stream)


def wan_unipc_coefficients(sigmas, num_sigmas, step, order, lower_order_final, coef):
    return load().wan_unipc_coefficients(sigmas, num_sigmas, step, order, lower_order_final, coef)


def wan_unipc_step(x, last, m_out, m_prev1, m_prev2, v_cond, v_uncond, v_dtype, n, guide_scale, sigma, coef,
                   stream):
    return load().wan_unipc_step(x, last, m_out, m_prev1, m_prev2, v_cond, v_uncond, v_dtype, n, guide_scale,
                                 sigma, coef, stream)


def wan_debug_bounds():
    return load().wan_debug_bounds()


def wan_device_status(stream):
    return load().wan_device_status(stream)


def wan_selftest_watchdog(stream):
    return load().wan_selftest_watchdog(stream)


def wan_profile_enable(on):
    return load().wan_profile_enable(on)


def wan_profile_read(kernel_class, launches, total_ms):
    return load().wan_profile_read(kernel_class, launches, total_ms)


def profile_read():
    """{class name: (launches, total device ms)} of the current record."""
    out = {}
    for c in range(WAN_K_COUNT):
        n = ctypes.c_int(0)
        ms = ctypes.c_double(0.0)
        check(wan_profile_read(c, ctypes.byref(n), ctypes.byref(ms)))
        out[KERNEL_CLASS_NAMES[c]] = (n.value, ms.value)
    return out


# ---------------------------------------------------------------- torch helpers
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def dtype_code(t) -> int:
    torch, dt = _torch(), t.dtype
    if dt == torch.bfloat16:
        return WAN_BF16
    if dt == torch.float32:
        return WAN_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


DTYPE_CODES = {"bf16": WAN_BF16, "f32": WAN_F32, "fp8": WAN_FP8, "fp8attn": WAN_FP8_ATTN}


def make_dims(F, H, W, dim, heads, ffn_dim, text_len, eps=1e-6, dtype="bf16", e0_per_token=False) -> wan_dims:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return wan_dims(F, H, W, dim, heads, ffn_dim, text_len, eps, code, 1 if e0_per_token else 0)


def dims_of(cfg) -> wan_dims:
    return make_dims(cfg.F, cfg.H, cfg.W, cfg.dim, cfg.heads, cfg.ffn_dim, cfg.text_len,
                     cfg.eps, cfg.dtype)


def make_weights(w: dict) -> wan_block_weights:
    for n in WEIGHT_FIELDS:
        if w.get(n) is not None and not w[n].is_contiguous():
            raise ValueError(f"weight {n} must be contiguous")
    return wan_block_weights(*[_ptr(w.get(n)) for n in WEIGHT_FIELDS])


def quantize_fp8(t, per_row=True, stream=None):
    """e4m3 codes (uint8, same shape) and float32 scales ([rows] or [1]) of a
    float32 / bf16 tensor; rows are the last axis."""
    torch = _torch()
    cols = t.shape[-1] if t.dim() else 1
    rows = t.numel() // cols if cols else 0
    q = torch.empty(t.shape, dtype=torch.uint8, device=t.device)
    sc = torch.empty((rows if per_row else 1,), dtype=torch.float32, device=t.device)
    check(wan_quantize_fp8(t.data_ptr(), dtype_code(t), rows, cols, 1 if per_row else 0,
                           q.data_ptr(), sc.data_ptr(), _stream(stream)))
    return q, sc


def linear_fp8(a, a_scale, w, w_scale, bias=None, out=None, stream=None):
    """out = (a w^T) a_scale[m] w_scale + bias, float32 [M, N]."""
    torch = _torch()
    M, K = a.shape
    N = w.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=a.device)
    check(wan_linear_fp8(M, N, K, a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
                         _ptr(bias), out.data_ptr(), _stream(stream)))
    return out


ACTIVATIONS = {"none": WAN_ACT_NONE, "gelu_tanh": WAN_ACT_GELU_TANH, "silu": WAN_ACT_SILU, "relu": WAN_ACT_RELU}


class _Types:
    """Type codes of torch dtypes (with torch imported on first use)."""
    codes = None

    @classmethod
    def get(cls):
        if cls.codes is None:
            torch = _torch()
            cls.codes = {torch.float32: WAN_F32, torch.bfloat16: WAN_BF16, torch.uint8: WAN_FP8,
                         torch.float8_e4m3fn: WAN_FP8}
        return cls.codes


def _float_code(codes, t):
    """dtype_code through the dict."""
    code = codes.get(t.dtype, WAN_FP8)
    return dtype_code(t) if code == WAN_FP8 else code


# Small calls are bound by the host: the helpers of wan_rmsnorm and wan_linear
# look at each tensor once and make one library call.
def _matrix(t, name, shape, rows, dev):
    """Address and row stride (in elements) of t, which must have this shape, as
    a matrix of its last axis (rows: the product of the other axes)."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if len(shape) != 2:
        t = t.view(rows, shape[-1])
    ld, unit = t.stride()
    if unit != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return t.data_ptr(), (ld if rows > 1 else shape[-1])


def _vector(t, name, n, dtype, dev):
    """Address of a contiguous vector of n elements."""
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    return t.data_ptr()


def _raw_stream(stream, dev):
    """Handle of the stream, by default of the current one of device dev."""
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    return stream.cuda_stream


def _empty_on(stream, shape, dtype, device):
    """torch.empty whose memory belongs to the stream that writes it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def rmsnorm(x, gain=None, residual=None, eps=1e-6, out_dtype=None, out=None, row_scale=None, h_out=None, stream=None):
    """RMS norm over the last axis with the residual's addition (wan_rmsnorm):
    h = x + residual, y = h / sqrt(mean(h^2) + eps) * gain.

    x [..., D] and residual [..., D] are bf16 or float32, gain float32 [D].
    ``out_dtype`` is "bf16", "f32" or "fp8" (e4m3 codes, uint8, with one
    float32 scale per row); by default the type of ``out``, or of x. Outputs
    that are not given are allocated. Rows may be strided (2-D tensors).
    Forward only: no gradient is recorded.
    Returns (y, row_scale, h): row_scale is None unless y holds codes, h is x
    itself without a residual and has the residual's type with one."""
    torch, codes = _torch(), _Types.codes or _Types.get()
    dev, shape = x.get_device(), x.shape
    if dev < 0:
        raise ValueError("x is not on a CUDA device")
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return rmsnorm(x, gain, residual, eps, out_dtype, out, row_scale, h_out, stream)
    if not shape or not shape[-1]:
        raise ValueError("x needs a last axis to normalise")
    D = shape[-1]
    rows = x.numel() // D
    xc = _float_code(codes, x)
    if out is None:
        code = xc if out_dtype is None else DTYPE_CODES[out_dtype]
        out = _empty_on(stream, shape, {WAN_FP8: torch.uint8, WAN_BF16: torch.bfloat16, WAN_F32: torch.float32}[code], x.device)
    else:
        code = codes.get(out.dtype)
        if code is None or (out_dtype is not None and DTYPE_CODES[out_dtype] != code):
            raise ValueError(f"out has type {out.dtype}")
    xp, ldx = _matrix(x, "x", shape, rows, dev)
    yp, ldy = _matrix(out, "out", shape, rows, dev)
    gp = 0 if gain is None else _vector(gain, "gain", D, torch.float32, dev)
    sp = 0
    if code == WAN_FP8:
        if row_scale is None:
            row_scale = _empty_on(stream, shape[:-1], torch.float32, x.device)
        sp = _vector(row_scale, "row_scale", rows, torch.float32, dev)
    elif row_scale is not None:
        raise ValueError("row_scale goes with e4m3 codes")
    rc, rp, ldr, hp, ldh = WAN_F32, 0, 0, 0, 0
    if residual is not None:
        rc = _float_code(codes, residual)
        rp, ldr = _matrix(residual, "residual", shape, rows, dev)
        if h_out is None:
            h_out = _empty_on(stream, shape, residual.dtype, x.device)
        elif h_out.dtype != residual.dtype:
            raise ValueError("h_out has the residual's type")
        hp, ldh = _matrix(h_out, "h_out", shape, rows, dev)
    elif h_out is not None:
        raise ValueError("h_out needs a residual")
    check(load().wan_rmsnorm(_RMSNORM_ARGS.pack(xp, rp, gp, hp, yp, sp, ldx, ldr, ldh, ldy, rows, D, xc, rc, code, eps),
                             _raw_stream(stream, dev)))
    return out, row_scale, (x if residual is None else h_out)


def linear(a, w, bias=None, activation="none", residual=None, a_scale=None, w_scale=None, out=None, out_dtype=None,
           stream=None):
    """Linear layer with bias, activation and residual (wan_linear):
    act(a w^T [a_scale w_scale] + bias) + residual, from one row to many.

    a [..., K] and w [N, K] are bf16, or e4m3 codes (uint8 or float8_e4m3fn)
    with float32 scales: a_scale one per row of a, w_scale one for w or one
    per row of w. bias is bf16 [N]; ``activation`` "none", "gelu_tanh", "silu"
    or "relu"; residual [..., N] bf16 or float32 and may be ``out`` itself.
    ``out_dtype`` is "bf16" or "f32" (by default the type of ``out``, of the
    residual, or bf16). Rows may be strided (2-D tensors); those of a and w
    start on 16-byte boundaries. Forward only: no gradient is recorded.
    Returns out [..., N]."""
    torch, codes = _torch(), _Types.codes or _Types.get()
    dev = a.get_device()
    if dev < 0:
        raise ValueError("a is not on a CUDA device")
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return linear(a, w, bias, activation, residual, a_scale, w_scale, out, out_dtype, stream)
    code = codes.get(a.dtype)
    if code is None or codes.get(w.dtype) != code:
        raise ValueError(f"a has type {a.dtype}, w {w.dtype}")
    ash, wsh = a.shape, w.shape
    if len(wsh) != 2 or not ash or ash[-1] != wsh[1]:
        raise ValueError(f"a {tuple(ash)} does not fit w {tuple(wsh)}")
    N, K = wsh
    shape = ash[:-1] + (N,)
    if out is None:
        dt = {"bf16": torch.bfloat16, "f32": torch.float32, None: torch.bfloat16 if residual is None else residual.dtype}[out_dtype]
        out = _empty_on(stream, shape, dt, a.device)
    elif out_dtype is not None and dtype_code(out) != DTYPE_CODES[out_dtype]:
        raise ValueError(f"out has type {out.dtype}, not {out_dtype}")
    if not N:
        return out
    M = a.numel() // K if K else out.numel() // N
    ap, lda = _matrix(a, "a", ash, M, dev)
    wp, ldw = _matrix(w, "w", wsh, N, dev)
    op, ldo = _matrix(out, "out", shape, M, dev)
    per_row, asp, wsp = 0, 0, 0
    if code == WAN_FP8:
        if a_scale is None or w_scale is None:
            raise ValueError("e4m3 operands need a_scale and w_scale")
        per_row = 1 if N > 1 and w_scale.numel() == N else 0
        asp = _vector(a_scale, "a_scale", M, torch.float32, dev)
        wsp = _vector(w_scale, "w_scale", N if per_row else 1, torch.float32, dev)
    elif a_scale is not None or w_scale is not None:
        raise ValueError("bf16 operands have no scales")
    bp = 0 if bias is None else _vector(bias, "bias", N, torch.bfloat16, dev)
    rc, rp, ldr = WAN_F32, 0, 0
    if residual is not None:
        rc = _float_code(codes, residual)
        rp, ldr = _matrix(residual, "residual", shape, M, dev)
    check(load().wan_linear(_LINEAR_ARGS.pack(ap, wp, asp, wsp, bp, rp, op, lda, ldw, ldr, ldo, M, N, K, code, per_row,
                                              ACTIVATIONS[activation], rc, _float_code(codes, out)),
                            _raw_stream(stream, dev)))
    return out


def quantize_block_weights(w: dict, stream=None) -> dict:
    """An FP8 copy of a bf16 block weight dict: the ten projection matrices
    become e4m3 codes and ``w_scales`` holds their ten per-tensor scales."""
    torch = _torch()
    out = dict(w)
    scales = torch.empty(10, dtype=torch.float32, device=w["wq"].device)
    for i, n in enumerate(FP8_MATRICES):
        q, sc = quantize_fp8(w[n], per_row=False, stream=stream)
        out[n] = q
        scales[i:i + 1].copy_(sc)
    out["w_scales"] = scales
    return out


def rope_freqs(head_dim, max_pos=1024, theta=1e4, device="cuda", stream=None):
    torch = _torch()
    t = torch.empty((max_pos, head_dim // 2, 2), dtype=torch.float32, device=device)
    check(wan_rope_freqs(head_dim, max_pos, theta, t.data_ptr(), _stream(stream)))
    return t


def workspace_bytes(dims: wan_dims, B: int) -> int:
    n = wan_block_workspace_bytes(dims, B)
    if n == 0 and B > 0:
        raise WanError(WAN_EINVAL, last_error())
    return n


def alloc_workspace(dims: wan_dims, B: int, device="cuda"):
    torch = _torch()
    n = wan_block_workspace_bytes(dims, B)
    if n == 0:
        raise WanError(WAN_EINVAL, last_error())
    return torch.empty(n, dtype=torch.uint8, device=device)


def workspace_view(ws, dims: wan_dims, B: int, which: int, shape, dtype):
    """A tensor view of one workspace buffer (see WAN_WS_* in include/wan.h)."""
    torch = _torch()
    off = wan_block_workspace_offset(dims, B, which)
    n = 1
    for s in shape:
        n *= s
    es = torch.empty((), dtype=dtype).element_size()
    return ws[off:off + n * es].view(dtype).view(*shape)


def block_forward(dims: wan_dims, x, ctx, e0, weights, rope, workspace, ctx_lens=None,
                  stream=None, cweights=None):
    """One block in place on x ([B, L, dim] float32). ``weights`` is a dict of
    device tensors (see WEIGHT_FIELDS) or a prebuilt wan_block_weights."""
    B = x.shape[0]
    cw = weights if isinstance(weights, wan_block_weights) else make_weights(weights)
    check(wan_block_forward(dims, B, x.data_ptr(), _ptr(ctx), _ptr(ctx_lens), e0.data_ptr(), cw,
                            rope.data_ptr(), rope.shape[0], workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), _stream(stream)))
    return x


def attention(q, k, v, k_lens=None, scale=0.0, grid=None, rope=None, out=None, stream=None):
    """q [B, Lq, n, d], k/v [B, Lk, n, d] (bf16 or f32). With ``grid`` the
    3D RoPE is applied to q and k in place first."""
    torch = _torch()
    B, Lq, n, d = q.shape
    Lk = k.shape[1]
    o = torch.empty_like(q) if out is None else out
    check(wan_attention(B, n, Lq, Lk, d, dtype_code(q), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                        o.data_ptr(), _ptr(k_lens), scale, grid, _ptr(rope),
                        0 if rope is None else rope.shape[0], _stream(stream)))
    return o


def attention_8bit(q, k, v, k_lens=None, scale=0.0, out=None, workspace=None, stream=None):
    """8-bit attention: q [B, Lq, n, 128], k / v [B, Lk, n, 128] bf16."""
    torch = _torch()
    B, Lq, n, d = q.shape
    Lk = k.shape[1]
    o = torch.empty_like(q) if out is None else out
    if workspace is None:
        workspace = torch.empty(max(wan_attention_8bit_workspace_bytes(B, n, Lq, Lk), 1), dtype=torch.uint8,
                                device=q.device)
    check(wan_attention_8bit(B, n, Lq, Lk, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(k_lens),
                             scale, workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return o


def euler_cfg_step(x, v_cond, v_uncond, guide_scale, sigma, sigma_next, stream=None):
    check(wan_euler_cfg_step(x.data_ptr(), v_cond.data_ptr(), _ptr(v_uncond), dtype_code(v_cond),
                             x.numel(), guide_scale, sigma, sigma_next, _stream(stream)))
    return x


def device_status(stream=None) -> int:
    return wan_device_status(_stream(stream))


def make_model_dims(C_in, C_out, F, H, W, dim, heads, ffn_dim, text_len, text_dim, freq_dim=256,
                    eps=1e-6, dtype="bf16", t_per_token=False) -> wan_model_dims:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return wan_model_dims(C_in, C_out, F, H, W, dim, heads, ffn_dim, text_len, text_dim, freq_dim,
                          eps, code, 1 if t_per_token else 0)


def make_model_weights(w: dict) -> wan_model_weights:
    for n in MODEL_WEIGHT_FIELDS:
        if w.get(n) is not None and not w[n].is_contiguous():
            raise ValueError(f"weight {n} must be contiguous")
    return wan_model_weights(*[_ptr(w.get(n)) for n in MODEL_WEIGHT_FIELDS])


def make_block_array(blocks) -> ctypes.Array:
    """A C array of wan_block_weights from a list of weight dicts (or structs)."""
    arr = (wan_block_weights * len(blocks))()
    for i, b in enumerate(blocks):
        arr[i] = b if isinstance(b, wan_block_weights) else make_weights(b)
    return arr


def alloc_model_workspace(dims: wan_model_dims, B: int, device="cuda"):
    torch = _torch()
    n = wan_model_workspace_bytes(dims, B)
    if n == 0:
        raise WanError(WAN_EINVAL, last_error())
    return torch.empty(n, dtype=torch.uint8, device=device)


def model_forward(dims: wan_model_dims, latent, t, text, weights, blocks, rope, workspace,
                  ctx_lens=None, out=None, stream=None):
    """Velocity of the whole model: latent [B, C_in, F, H, W] float32, t [B]
    (or [B, L] with dims.t_per_token) float32 timesteps (device), text [B, text_len, text_dim] in the compute
    dtype. ``blocks`` is a list of block weight dicts or a make_block_array()
    result. Returns out [B, C_out, F, H, W] float32."""
    torch = _torch()
    B = latent.shape[0]
    if out is None:
        out = torch.empty((B, dims.C_out, dims.F, dims.H, dims.W), dtype=torch.float32,
                          device=latent.device)
    mw = weights if isinstance(weights, wan_model_weights) else make_model_weights(weights)
    arr = blocks if isinstance(blocks, ctypes.Array) else make_block_array(blocks)
    check(wan_model_forward(dims, B, latent.data_ptr(), t.data_ptr(), _ptr(text), _ptr(ctx_lens),
                            mw, arr, len(arr), rope.data_ptr(), rope.shape[0],
                            out.data_ptr(), workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


class UniPCSampler:
    """State of the UniPC sampler over one latent (see wan_unipc_step): the
    schedule, the step index, the corrected previous sample and a ring of
    three data predictions. ``x`` (float32, device) is updated in place."""

    def __init__(self, x, sigmas, order=2, lower_order_final=True):
        torch = _torch()
        self.x = x
        self.sigmas = [float(s) for s in sigmas]
        self.n = len(self.sigmas) - 1
        self.order, self.lof = order, lower_order_final
        self.i = 0
        self.last = torch.empty_like(x)
        self.ring = [torch.empty_like(x) for _ in range(3)]
        self._sig = (ctypes.c_double * len(self.sigmas))(*self.sigmas)
        self._coef = (ctypes.c_double * 8)()

    @property
    def sigma(self) -> float:
        return self.sigmas[self.i]

    def coefficients(self, step=None):
        check(wan_unipc_coefficients(self._sig, len(self.sigmas), self.i if step is None else step, self.order,
                                     1 if self.lof else 0, self._coef))
        return list(self._coef)

    def step(self, v_cond, v_uncond=None, guide_scale=1.0, stream=None):
        if self.i >= self.n:
            raise RuntimeError("UniPC schedule finished")
        self.coefficients()
        i = self.i
        m_out = self.ring[i % 3]
        m1 = self.ring[(i - 1) % 3] if i >= 1 else None
        m2 = self.ring[(i - 2) % 3] if i >= 2 else None
        check(wan_unipc_step(self.x.data_ptr(), self.last.data_ptr(), m_out.data_ptr(), _ptr(m1), _ptr(m2),
                             v_cond.data_ptr(), _ptr(v_uncond), dtype_code(v_cond), self.x.numel(), guide_scale,
                             self.sigmas[i], self._coef, _stream(stream)))
        self.i += 1
        return self.x
