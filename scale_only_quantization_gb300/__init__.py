"""Python binding of the scale-only QAD MoE library (libqad_gb300.so, sm_103a).

Argument marshalling only: every step of the layer runs in the library's CUDA kernels.
Each function below has the name and argument order of the C entry point in
include/qad.h; tensors are torch tensors on the current CUDA device (their data pointers
are passed), the stream defaults to torch's current stream, and a non-zero status
raises QADError.  There is no CPU fallback: if the library is not built the functions
raise.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqad_gb300.so")

QAD_OK, QAD_ERR_INVALID_ARG, QAD_ERR_UNSUPPORTED, QAD_ERR_WORKSPACE, QAD_ERR_CUDA, QAD_ERR_DEVICE = 0, -1, -2, -3, -4, -5
QAD_ERR_SCRATCH_LIMIT = -6
QAD_NOALLOC_MAX_EXPERTS, QAD_NOALLOC_MAX_PAIRS = 256, 262144
QAD_FMT_NVFP4, QAD_FMT_INT4_G128, QAD_FMT_FP8_ROW, QAD_FMT_NVFP4A16, QAD_FMT_W8A8, QAD_FMT_W4AFP8 = range(6)
QAD_FMT_NVFP4_E4M3 = 6
QAD_DEV_BAD_INDEX, QAD_DEV_DUP_INDEX, QAD_DEV_TIMEOUT = 1, 2, 4
QAD_FLAG_STASH_H, QAD_FLAG_NO_QUANT, QAD_FLAG_RECOMPUTE, QAD_FLAG_NATIVE_FP8 = 1, 2, 4, 8
QAD_FLAG_SMEM_DEQUANT, QAD_FLAG_DEQUANT_DUMP = 16, 32
VIEWS = ["HEADER", "OFFSETS", "COUNTS", "ROW_TOKEN", "ROW_SLOT", "ROW_OF", "W13_HAT", "W2_HAT", "A1", "Z1", "H",
         "H_HAT", "Y", "DY", "DZ1", "DA1", "XQ", "W13_CODES", "W2_CODES", "A1_CODES", "H_CODES", "A_SCALE",
         "H_SCALE", "S13_DEPLOYED", "S2_DEPLOYED"]
VIEW = {n: i for i, n in enumerate(VIEWS)}
KERNELS = 28
QAD_ACT_NONE, QAD_ACT_E4M3, QAD_ACT_INT8 = range(3)
QAD_RMSNORM_MAX_D, QAD_DISTILL_MAX_D, QAD_DISTILL_MAX_K = 16384, 16384, 1024
QAD_MOE_FEW_MAX_T, QAD_MOE_FEW_MAX_D = 64, 8192
QAD_F32, QAD_BF16 = range(2)
QAD_LOGPROBS_MAX_K = 1024

EXPORTS = ["qad_fakequant_fwd", "qad_moe_workspace_bytes", "qad_moe_fwd", "qad_moe_bwd_dgrad",
           "qad_moe_bwd_scalegrad", "qad_check_device_error", "qad_status_string", "qad_moe_debug_view",
           "qad_profile_enable", "qad_profile_reset", "qad_profile_read", "qad_kernel_name", "qad_launch_count",
           "qad_debug_quotient", "qad_route_permute_noalloc", "qad_debug_wait_timeout", "qad_debug_stuck_copy",
           "qad_moe_combine", "qad_nvfp4_deploy_scales", "qad_rmsnorm_workspace_bytes", "qad_rmsnorm_fwd", "qad_rmsnorm_bwd",
           "qad_linear_ce_workspace_bytes", "qad_linear_ce_fwd", "qad_linear_ce_fwd_bwd", "qad_distill_topk_fwd",
           "qad_distill_topk_fwd_bwd", "qad_moe_few_workspace_bytes", "qad_moe_few_fwd", "qad_token_logprobs",
           "qad_token_logprobs_bwd", "qad_grad_norm_workspace_bytes", "qad_grad_norm", "qad_grad_clip", "qad_adamw_step"]


class QADError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, status_string(status), status))


class MoEShape(ctypes.Structure):
    """qad_moe_shape: T tokens, hidden d, expert FFN F, E experts, top-k, format, flags."""
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("F", ctypes.c_int64), ("E", ctypes.c_int64),
                ("topk", ctypes.c_int32), ("fmt", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Tensor(ctypes.Structure):
    """qad_tensor: one entry of a list of tensors."""
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class TensorList:
    """Tensors as the optimizer calls take them (qad_tensor[]); holds the tensors, so that their memory stays."""

    def __init__(self, tensors):
        import torch
        kinds = {torch.float32: QAD_F32, torch.bfloat16: QAD_BF16}
        self.tensors = list(tensors)
        self.n = len(self.tensors)
        self.array = (Tensor * max(1, self.n))()
        for a, t in zip(self.array, self.tensors):
            if t.dtype not in kinds or not t.is_contiguous():
                raise ValueError("a list takes contiguous fp32 and bf16 tensors, got %s %s with strides %s" % (
                    t.dtype, tuple(t.shape), t.stride()))
            a.data, a.numel, a.dtype = t.data_ptr(), t.numel(), kinds[t.dtype]


def tensor_list(tensors):
    """A TensorList of `tensors`: made once where the tensors stay (a captured step, preallocated gradients)."""
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


_lib = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F32 = ctypes.c_float
_F64 = ctypes.c_double
_SHAPE = ctypes.POINTER(MoEShape)


def lib():
    """Load libqad_gb300.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libqad_gb300.so is not built: run `python -m scale_only_quantization_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "qad_fakequant_fwd": (ctypes.c_int, [ctypes.c_int, _P, _P, _P, _I64, _I64, _I64, _P]),
            "qad_moe_workspace_bytes": (ctypes.c_size_t, [_SHAPE]),
            "qad_moe_fwd": (ctypes.c_int, [_SHAPE, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
            "qad_moe_bwd_dgrad": (ctypes.c_int, [_SHAPE, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
            "qad_moe_bwd_scalegrad": (ctypes.c_int, [_SHAPE, _P, _P, _P, _P, _P, _P, ctypes.c_int, _P,
                                                     ctypes.c_size_t, _P]),
            "qad_check_device_error": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_int32)]),
            "qad_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "qad_moe_debug_view": (ctypes.c_int, [_SHAPE, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t),
                                                  ctypes.POINTER(ctypes.c_int64)]),
            "qad_profile_enable": (ctypes.c_int, [ctypes.c_int]),
            "qad_profile_reset": (ctypes.c_int, []),
            "qad_profile_read": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int64),
                                                ctypes.c_int]),
            "qad_kernel_name": (ctypes.c_char_p, [ctypes.c_int]),
            "qad_launch_count": (ctypes.c_int64, []),
            "qad_debug_quotient": (ctypes.c_int, [_P, _P, _P, _P, _I64, ctypes.c_int32, _P]),
            "qad_debug_wait_timeout": (ctypes.c_int, [_P, _I64, _P]),
            "qad_debug_stuck_copy": (ctypes.c_int, [_I64, _I64]),
            "qad_route_permute_noalloc": (ctypes.c_int, [_P, _I64, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P,
                                                         _P, _P, _P]),
            "qad_moe_combine": (ctypes.c_int, [_P, _P, _P, _P, _I64, ctypes.c_int32, _I64, _P]),
            "qad_nvfp4_deploy_scales": (ctypes.c_int, [_P, _P, _I64, _I64, _P]),
            "qad_rmsnorm_workspace_bytes": (ctypes.c_size_t, [_I64, _I64]),
            "qad_rmsnorm_fwd": (ctypes.c_int, [_P, _P, _P, _F32, ctypes.c_int] + [_P] * 6 + [_I64] * 4 + [_P]),
            "qad_rmsnorm_bwd": (ctypes.c_int, [_P] * 7 + [_I64] * 3 + [_P, ctypes.c_size_t, _P]),
            "qad_linear_ce_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, ctypes.c_int, ctypes.c_int]),
            "qad_linear_ce_fwd": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _P,
                                                 ctypes.c_size_t, _P]),
            "qad_linear_ce_fwd_bwd": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, ctypes.c_int, _I64,
                                                     _I64, _I64, _P, ctypes.c_size_t, _P]),
            "qad_distill_topk_fwd": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _P, _P, _F32, _P, _I64, _I64, _I64, _I64,
                                                    _P, _P]),
            "qad_distill_topk_fwd_bwd": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _P, _P, _F32, _P, _P, _P, ctypes.c_int,
                                                        _I64, _I64, _I64, _I64, _P, _P]),
            "qad_moe_few_workspace_bytes": (ctypes.c_size_t, [_SHAPE]),
            "qad_moe_few_fwd": (ctypes.c_int, [_SHAPE] + [_P] * 9 + [ctypes.c_size_t, _P]),
            "qad_token_logprobs": (ctypes.c_int, [_P, ctypes.c_int, _I64, _P, _F32] + [_P] * 5 + [_I64] * 3 + [_P, _P]),
            "qad_token_logprobs_bwd": (ctypes.c_int, [_P, ctypes.c_int, _I64, _P, _F32] + [_P] * 5 + [_I64] * 3 + [_P]),
            "qad_grad_norm_workspace_bytes": (ctypes.c_size_t, []),
            "qad_grad_norm": (ctypes.c_int, [_P, _I64, _P, _P, ctypes.c_size_t, _P]),
            "qad_grad_clip": (ctypes.c_int, [_P, _P, _I64, _P, _F32, _P]),
            "qad_adamw_step": (ctypes.c_int, [_P] * 4 + [_I64, _P, _F64, _F64, _F32, _F32, _F32, _P, _F32, _P, _P,
                                              ctypes.c_size_t, _P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def status_string(status):
    return lib().qad_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else t.data_ptr()  # argtypes makes the pointer: an object per argument costs ~0.2 us


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


_raw_stream = None


def _current_stream():
    """Handle of torch's current stream on the current device, without building a Stream object per call."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        torch.cuda.current_stream()  # CUDA is initialised, or this raises
        get, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        if get is not None and dev is not None:
            _raw_stream = lambda: get(dev())  # noqa: E731
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(rc, where):
    if rc != QAD_OK:
        raise QADError(rc, where)
    return rc


def shape(T, d, F, E, topk, fmt, flags=0):
    return MoEShape(int(T), int(d), int(F), int(E), int(topk), int(fmt), int(flags), 0)


def qad_fakequant_fwd(fmt, w, scale, w_hat, E, N, K, stream=None):
    return _check(lib().qad_fakequant_fwd(int(fmt), _ptr(w), _ptr(scale), _ptr(w_hat), int(E), int(N), int(K),
                                          _stream(stream)), "qad_fakequant_fwd")


def qad_nvfp4_deploy_scales(s, s_q, n_mat, per_mat, stream=None):
    return _check(lib().qad_nvfp4_deploy_scales(_ptr(s), _ptr(s_q), int(n_mat), int(per_mat), _stream(stream)),
                  "qad_nvfp4_deploy_scales")


def qad_moe_workspace_bytes(s):
    return int(lib().qad_moe_workspace_bytes(ctypes.byref(s)))


def qad_moe_fwd(s, x, topk_idx, topk_w, w13, s13, w2, s2, out, ws, stream=None):
    return _check(lib().qad_moe_fwd(ctypes.byref(s), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(w13), _ptr(s13),
                                    _ptr(w2), _ptr(s2), _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream(stream)), "qad_moe_fwd")


def qad_moe_bwd_dgrad(s, dout, topk_w, w13, s13, w2, s2, dx, dprobs, ws, stream=None):
    return _check(lib().qad_moe_bwd_dgrad(ctypes.byref(s), _ptr(dout), _ptr(topk_w), _ptr(w13), _ptr(s13), _ptr(w2),
                                          _ptr(s2), _ptr(dx), _ptr(dprobs), _ptr(ws),
                                          ws.numel() * ws.element_size(), _stream(stream)), "qad_moe_bwd_dgrad")


def qad_moe_bwd_scalegrad(s, w13, s13, w2, s2, ds13, ds2, accumulate, ws, stream=None):
    return _check(lib().qad_moe_bwd_scalegrad(ctypes.byref(s), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), _ptr(ds13),
                                              _ptr(ds2), int(accumulate), _ptr(ws), ws.numel() * ws.element_size(),
                                              _stream(stream)), "qad_moe_bwd_scalegrad")


def qad_check_device_error(ws, stream=None):
    """Returns the device error word (0 = none); synchronises the stream."""
    code = ctypes.c_int32(0)
    rc = lib().qad_check_device_error(_ptr(ws), _stream(stream), ctypes.byref(code))
    if rc not in (QAD_OK, QAD_ERR_DEVICE):
        raise QADError(rc, "qad_check_device_error")
    return int(code.value)


def qad_moe_debug_view(s, which):
    """(byte offset, element count) of workspace region `which` (a VIEWS name or index)."""
    off, n = ctypes.c_size_t(0), ctypes.c_int64(0)
    w = VIEW[which] if isinstance(which, str) else int(which)
    _check(lib().qad_moe_debug_view(ctypes.byref(s), w, ctypes.byref(off), ctypes.byref(n)), "qad_moe_debug_view")
    return int(off.value), int(n.value)


def qad_profile_enable(on):
    return _check(lib().qad_profile_enable(int(bool(on))), "qad_profile_enable")


def qad_profile_reset():
    return _check(lib().qad_profile_reset(), "qad_profile_reset")


def qad_profile_read():
    """{kernel name: (total ms, launches)} since the last reset; synchronises the device."""
    ms = (ctypes.c_float * KERNELS)()
    n = (ctypes.c_int64 * KERNELS)()
    _check(lib().qad_profile_read(ms, n, KERNELS), "qad_profile_read")
    return {lib().qad_kernel_name(i).decode(): (float(ms[i]), int(n[i])) for i in range(KERNELS)}


def qad_kernel_name(i):
    return lib().qad_kernel_name(int(i)).decode()


def qad_launch_count():
    return int(lib().qad_launch_count())


def qad_debug_quotient(w, s, x_fast, x_ieee, n, mode=0, stream=None):
    return _check(lib().qad_debug_quotient(_ptr(w), _ptr(s), _ptr(x_fast), _ptr(x_ieee), int(n), int(mode),
                                           _stream(stream)), "qad_debug_quotient")


def qad_route_permute_noalloc(topk_idx, T, topk, E, row_token, row_slot, row_of, offsets, counts, header,
                              stream=None):
    """Routing maps without any device allocation by the library (see include/qad.h)."""
    return _check(lib().qad_route_permute_noalloc(_ptr(topk_idx), int(T), int(topk), int(E), _ptr(row_token),
                                                  _ptr(row_slot), _ptr(row_of), _ptr(offsets), _ptr(counts),
                                                  _ptr(header), _stream(stream)), "qad_route_permute_noalloc")


def qad_moe_combine(rows, row_of, p, out, T, topk, d, stream=None):
    return _check(lib().qad_moe_combine(_ptr(rows), _ptr(row_of), _ptr(p), _ptr(out), int(T), int(topk), int(d),
                                        _stream(stream)), "qad_moe_combine")


def qad_rmsnorm_workspace_bytes(T, d):
    return int(lib().qad_rmsnorm_workspace_bytes(int(T), int(d)))


def qad_rmsnorm_fwd(x, res, gamma, eps, act, res_out, y, y_hat, codes, scale, rstd, T, d, ldx, ldres, stream=None):
    """Residual addition + RMSNorm with an optional 8-bit output (see include/qad.h)."""
    return _check(lib().qad_rmsnorm_fwd(_ptr(x), _ptr(res), _ptr(gamma), float(eps), int(act), _ptr(res_out), _ptr(y),
                                        _ptr(y_hat), _ptr(codes), _ptr(scale), _ptr(rstd), int(T), int(d), int(ldx),
                                        int(ldres), _stream(stream)), "qad_rmsnorm_fwd")


def qad_rmsnorm_bwd(dy, dres, r, gamma, rstd, dx, dgamma, T, d, ldr, ws=None, stream=None):
    return _check(lib().qad_rmsnorm_bwd(_ptr(dy), _ptr(dres), _ptr(r), _ptr(gamma), _ptr(rstd), _ptr(dx),
                                        _ptr(dgamma), int(T), int(d), int(ldr), _ptr(ws), _nbytes(ws),
                                        _stream(stream)), "qad_rmsnorm_bwd")


def qad_linear_ce_workspace_bytes(N, d, V, dh, dw):
    return int(lib().qad_linear_ce_workspace_bytes(int(N), int(d), int(V), int(bool(dh)), int(bool(dw))))


def qad_linear_ce_fwd(h, ldh, w, ldw, target, loss, lse, N, d, V, ws, stream=None):
    """Cross entropy of hidden states against the head w, without keeping the logits (see include/qad.h)."""
    return _check(lib().qad_linear_ce_fwd(_ptr(h), int(ldh), _ptr(w), int(ldw), _ptr(target), _ptr(loss), _ptr(lse),
                                          int(N), int(d), int(V), _ptr(ws), _nbytes(ws), _stream(stream)),
                  "qad_linear_ce_fwd")


def qad_linear_ce_fwd_bwd(h, ldh, w, ldw, target, g, loss, lse, dh, dw, accumulate, N, d, V, ws, stream=None):
    return _check(lib().qad_linear_ce_fwd_bwd(_ptr(h), int(ldh), _ptr(w), int(ldw), _ptr(target), _ptr(g), _ptr(loss),
                                              _ptr(lse), _ptr(dh), _ptr(dw), int(accumulate), int(N), int(d), int(V),
                                              _ptr(ws), _nbytes(ws), _stream(stream)), "qad_linear_ce_fwd_bwd")


def qad_distill_topk_fwd(h, ldh, w, ldw, idx, t_logit, mix, inv_temp, loss, N, d, V, K, err=None, stream=None):
    """Divergence from the teacher's top K logits over the teacher's own tokens (see include/qad.h)."""
    return _check(lib().qad_distill_topk_fwd(_ptr(h), int(ldh), _ptr(w), int(ldw), _ptr(idx), _ptr(t_logit), _ptr(mix),
                                             float(inv_temp), _ptr(loss), int(N), int(d), int(V), int(K), _ptr(err),
                                             _stream(stream)), "qad_distill_topk_fwd")


def qad_distill_topk_fwd_bwd(h, ldh, w, ldw, idx, t_logit, mix, inv_temp, g, loss, dh, accumulate, N, d, V, K,
                             err=None, stream=None):
    return _check(lib().qad_distill_topk_fwd_bwd(_ptr(h), int(ldh), _ptr(w), int(ldw), _ptr(idx), _ptr(t_logit),
                                                 _ptr(mix), float(inv_temp), _ptr(g), _ptr(loss), _ptr(dh),
                                                 int(accumulate), int(N), int(d), int(V), int(K), _ptr(err),
                                                 _stream(stream)), "qad_distill_topk_fwd_bwd")


def qad_moe_few_workspace_bytes(s):
    return int(lib().qad_moe_few_workspace_bytes(ctypes.byref(s)))


def qad_moe_few_fwd(s, x, topk_idx, topk_w, w13, s13, w2, s2, out, ws, stream=None):
    """The layer's forward for at most QAD_MOE_FEW_MAX_T tokens, nothing kept for a backward (see include/qad.h)."""
    return _check(lib().qad_moe_few_fwd(ctypes.byref(s), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(w13), _ptr(s13),
                                        _ptr(w2), _ptr(s2), _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream)),
                  "qad_moe_few_fwd")


def qad_token_logprobs(z, dtype, ldz, token, inv_temp, logp, lse, entropy, top_idx, top_logit, N, V, K, err=None,
                       stream=None):
    """Log probabilities of given tokens, entropy and top alternatives of logits (see include/qad.h)."""
    return _check(lib().qad_token_logprobs(_ptr(z), int(dtype), int(ldz), _ptr(token), float(inv_temp), _ptr(logp),
                                           _ptr(lse), _ptr(entropy), _ptr(top_idx), _ptr(top_logit), int(N), int(V),
                                           int(K), _ptr(err), _stream(stream)), "qad_token_logprobs")


def qad_token_logprobs_bwd(z, dtype, ldz, token, inv_temp, lse, entropy, g_logp, g_entropy, dz, lddz, N, V, stream=None):
    return _check(lib().qad_token_logprobs_bwd(_ptr(z), int(dtype), int(ldz), _ptr(token), float(inv_temp), _ptr(lse),
                                               _ptr(entropy), _ptr(g_logp), _ptr(g_entropy), _ptr(dz), int(lddz), int(N),
                                               int(V), _stream(stream)), "qad_token_logprobs_bwd")


def qad_grad_norm_workspace_bytes():
    return int(lib().qad_grad_norm_workspace_bytes())


def qad_grad_norm(grads, norm, ws, stream=None):
    """The norm over all tensors of a list (a TensorList, or the tensors themselves)."""
    g = tensor_list(grads)
    return _check(lib().qad_grad_norm(g.array, g.n, _ptr(norm), _ptr(ws), _nbytes(ws), _stream(stream)), "qad_grad_norm")


def qad_grad_clip(grads, out, norm, max_norm, stream=None):
    """Gradients times min(1, max_norm / (norm + 1e-6)); out None: in place."""
    g, o = tensor_list(grads), None if out is None else tensor_list(out)
    if o is not None and o.n != g.n:
        raise ValueError("%d gradients and %d outputs" % (g.n, o.n))
    return _check(lib().qad_grad_clip(g.array, None if o is None else o.array, g.n, _ptr(norm), float(max_norm),
                                      _stream(stream)), "qad_grad_clip")


def qad_adamw_step(params, grads, exp_avg, exp_avg_sq, lr, beta1, beta2, eps, decay, floor, norm, max_norm, steps, ws,
                   stream=None):
    """One AdamW step over lists of tensors, clipped by the norm if one is given (see include/qad.h)."""
    p, g, m, v = (tensor_list(a) for a in (params, grads, exp_avg, exp_avg_sq))
    if not p.n == g.n == m.n == v.n or (lr is not None and lr.numel() != g.n):
        raise ValueError("the lists differ in length: %d parameters, %d gradients, %d and %d moments, %s rates" % (
            p.n, g.n, m.n, v.n, None if lr is None else lr.numel()))
    return _check(lib().qad_adamw_step(p.array, g.array, m.array, v.array, g.n, _ptr(lr), float(beta1), float(beta2),
                                       float(eps), float(decay), float(floor), _ptr(norm), float(max_norm), _ptr(steps),
                                       _ptr(ws), _nbytes(ws), _stream(stream)), "qad_adamw_step")


def qad_debug_wait_timeout(err_word, budget_cycles, stream=None):
    return _check(lib().qad_debug_wait_timeout(_ptr(err_word), int(budget_cycles), _stream(stream)),
                  "qad_debug_wait_timeout")


def qad_debug_stuck_copy(row, budget_cycles=0):
    return _check(lib().qad_debug_stuck_copy(int(row), int(budget_cycles)), "qad_debug_stuck_copy")


def workspace_view(ws, s, which, dtype):
    """A torch view of workspace region `which` with element type `dtype` (flat)."""
    import torch
    off, n = qad_moe_debug_view(s, which)
    itemsize = torch.tensor([], dtype=dtype).element_size()
    return ws.view(torch.uint8)[off: off + n * itemsize].view(dtype)
