"""The layer as a torch.autograd.Function and an nn.Module, over the C ABI.

Scale-only QAD ("MCoreQAD Backend", opening section; AngelSlim mcore_qad walkthrough,
nxmr.cn/news/131691, sections 二.3-二.4): the routed-expert weights are frozen, the forward
sees their fake-quantized copies, and the quantizer scales are the only trainable
parameters.  So the backward returns no gradient for the weights or the routing indices,
dx for the hidden states, dprobs for the routing weights (their gradient reaches the router)
and ds13 / ds2 for the scales.

Marshalling only: the forward is qad_moe_fwd, the backward qad_moe_bwd_dgrad followed by
qad_moe_bwd_scalegrad, all on torch's current stream.  The workspace, which carries the
stashed stages from the forward to the backward, lives in the autograd context.

What stands around the layer in a training step: QADRMSNorm (residual addition, norm and the 8-bit
form of its output) before it, QADHeadLoss (cross entropy and distillation on the frozen head) at the
end.
"""
import torch
from torch.autograd.function import once_differentiable

from . import (QAD_ACT_NONE, qad_distill_topk_fwd, qad_distill_topk_fwd_bwd, qad_linear_ce_fwd, qad_linear_ce_fwd_bwd,
               qad_linear_ce_workspace_bytes, qad_moe_bwd_dgrad, qad_moe_bwd_scalegrad, qad_moe_fwd,
               qad_moe_workspace_bytes, qad_rmsnorm_bwd, qad_rmsnorm_fwd, qad_rmsnorm_workspace_bytes, shape)


class QADMoEFunction(torch.autograd.Function):
    """out = MoE(x; topk_idx, topk_w, W13_hat(s13), W2_hat(s2)).

    x [T, d] bf16; topk_idx [T, k] int32; topk_w [T, k] fp32; w13 [E, 2F, d] bf16 (gate rows,
    then up rows); s13 fp32 [E, 2F, d / B]; w2 [E, d, F] bf16; s2 fp32 [E, d, F / B]; fmt a
    qad_fmt; flags QAD_FLAG_* bits.  All tensors contiguous on the current CUDA device.
    """

    @staticmethod
    def forward(ctx, x, topk_idx, topk_w, w13, s13, w2, s2, fmt, flags):
        T, d = x.shape
        E, two_f, _ = w13.shape
        k = topk_idx.shape[1]
        s = shape(T, d, two_f // 2, E, k, fmt, flags)
        ws = torch.empty(qad_moe_workspace_bytes(s), dtype=torch.uint8, device=x.device)
        out = torch.empty_like(x)
        qad_moe_fwd(s, x, topk_idx, topk_w, w13, s13, w2, s2, out, ws)
        ctx.save_for_backward(topk_w, w13, s13, w2, s2)
        ctx.layer_shape = s
        ctx.ws = ws
        ctx.mark_non_differentiable(topk_idx)
        return out

    @staticmethod
    def backward(ctx, dout):
        topk_w, w13, s13, w2, s2 = ctx.saved_tensors
        s, ws = ctx.layer_shape, ctx.ws
        dout = dout.contiguous()
        dx = torch.empty_like(dout)
        dprobs = torch.empty_like(topk_w) if ctx.needs_input_grad[2] else None
        qad_moe_bwd_dgrad(s, dout, topk_w, w13, s13, w2, s2, dx, dprobs, ws)
        ds13 = ds2 = None
        if ctx.needs_input_grad[4] or ctx.needs_input_grad[6]:
            ds13 = torch.empty_like(s13)
            ds2 = torch.empty_like(s2)
            qad_moe_bwd_scalegrad(s, w13, s13, w2, s2, ds13, ds2, 0, ws)
        ctx.ws = None
        return (dx if ctx.needs_input_grad[0] else None, None, dprobs, None, ds13, None, ds2, None, None)


class QADMoE(torch.nn.Module):
    """The routed experts of one MoE layer: frozen bf16 weights (buffers) and learnable fp32
    scales (parameters), initialised by the caller."""

    def __init__(self, w13, s13, w2, s2, fmt, flags=0):
        super().__init__()
        self.register_buffer("w13", w13.contiguous())
        self.register_buffer("w2", w2.contiguous())
        self.s13 = torch.nn.Parameter(s13.contiguous())
        self.s2 = torch.nn.Parameter(s2.contiguous())
        self.fmt = int(fmt)
        self.flags = int(flags)

    def forward(self, x, topk_idx, topk_w):
        return QADMoEFunction.apply(x.contiguous(), topk_idx.contiguous(), topk_w.contiguous(), self.w13, self.s13,
                                    self.w2, self.s2, self.fmt, self.flags)


def _packed(t):
    """t, contiguous and on a 16-byte boundary: contiguous() alone returns a view such as ids[1:] where it lies."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _rows(t, d, what):
    """t as [rows, d] bf16 rows that the library can read: unit column stride, 16-byte aligned rows."""
    if t.dtype != torch.bfloat16 or t.shape[-1] != d:
        raise ValueError("%s must be bf16 with %d columns, got %s %s" % (what, d, t.dtype, tuple(t.shape)))
    t = t.reshape(-1, d)
    if t.stride(1) != 1 or t.stride(0) % 8 or t.stride(0) < d or t.data_ptr() % 16:
        t = _packed(t)
    return t


class QADRMSNormFunction(torch.autograd.Function):
    """(y, r, codes, scale) = residual addition + RMSNorm of x with the per-row activation quantizer `act`.

    r = bf16(x + res) is the residual stream; y = bf16(r * rstd * gamma) is what the router and the layer
    read; codes [.., d] uint8 and scale [rows] fp32 are its 8-bit form (None with QAD_ACT_NONE).  The
    backward is straight through the quantizer: dx for x and res, dgamma.
    """

    @staticmethod
    def forward(ctx, x, res, gamma, eps, act):
        d = gamma.numel()
        x2 = _rows(x, d, "x")
        res2 = None if res is None else _rows(res, d, "res")
        if res2 is not None and res2.shape != x2.shape:
            raise ValueError("x and res differ in shape")
        T = x2.shape[0]
        dev = x.device
        r = torch.empty((T, d), dtype=torch.bfloat16, device=dev)
        y = torch.empty_like(r)
        rstd = torch.empty(T, dtype=torch.float32, device=dev)
        codes = torch.empty((T, d), dtype=torch.uint8, device=dev) if act != QAD_ACT_NONE else None
        scale = torch.empty(T, dtype=torch.float32, device=dev) if act != QAD_ACT_NONE else None
        gamma = _packed(gamma)
        qad_rmsnorm_fwd(x2, res2, gamma, eps, act, r, y, None, codes, scale, rstd, T, d, x2.stride(0) if T > 1 else d,
                        res2.stride(0) if res2 is not None and T > 1 else d)
        ctx.save_for_backward(r, gamma, rstd)
        ctx.set_materialize_grads(False)  # an output that nothing reads costs the backward nothing
        ctx.res_shape = None if res is None else res.shape
        ctx.shape = x.shape
        if codes is not None:
            ctx.mark_non_differentiable(codes, scale)
            codes = codes.view(x.shape)
        return y.view(x.shape), r.view(x.shape), codes, scale

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dr, _codes, _scale):
        r, gamma, rstd = ctx.saved_tensors
        T, d = r.shape
        need = ctx.needs_input_grad[2]
        if dy is None and dr is None:
            return None, None, None, None, None
        if dy is None:  # only the residual stream goes on
            dx, dgamma = dr, torch.zeros_like(gamma) if need else None
        else:
            dx = torch.empty_like(r)
            dgamma = torch.empty(d, dtype=torch.float32, device=r.device) if need else None
            ws = torch.empty(qad_rmsnorm_workspace_bytes(T, d), dtype=torch.uint8, device=r.device) if need else None
            qad_rmsnorm_bwd(_packed(dy.reshape(T, d)), None if dr is None else _packed(dr.reshape(T, d)), r, gamma, rstd, dx,
                            dgamma, T, d, d, ws)
            dgamma = dgamma.to(gamma.dtype) if need else None
        return (dx.reshape(ctx.shape), None if ctx.res_shape is None else dx.reshape(ctx.res_shape), dgamma, None, None)


class QADRMSNorm(torch.nn.Module):
    """RMSNorm before a quantized layer: forward(x, res=None) -> (y, r), or (y, r, codes, scale) with a per-row
    activation grid (QAD_ACT_E4M3, QAD_ACT_INT8).  The weight is kept in high precision; frozen unless trained."""

    def __init__(self, weight, eps=1e-6, act=QAD_ACT_NONE, trained=False):
        super().__init__()
        self.weight = torch.nn.Parameter(_packed(weight.to(torch.bfloat16)), requires_grad=trained)
        self.eps = float(eps)
        self.act = int(act)

    def forward(self, x, res=None):
        y, r, codes, scale = QADRMSNormFunction.apply(x, res, self.weight, self.eps, self.act)
        return (y, r) if self.act == QAD_ACT_NONE else (y, r, codes, scale)


def _tokens(t, V):
    """t as int32: a 64-bit token keeps its side of the vocabulary [0, V) instead of wrapping into it."""
    return t if t.dtype == torch.int32 else t.clamp(-1, V).to(torch.int32)


class QADHeadLossFunction(torch.autograd.Function):
    """total = sum_i g_lm[i] * CE_i + sum_i g_kd[i] * KD_i of hidden states h against the frozen head w.

    CE_i is the cross entropy over the whole vocabulary (rows with target < 0 carry none), KD_i the
    divergence over the teacher's top tokens idx [N, K] with logits t [N, K], softened by tau, mixed
    forward and reverse by mix [N] (None: forward).  Either part is left out when its target or idx is
    None.  The hidden-state gradient is formed in the forward, where the logits are, and scaled by the
    upstream gradient in the backward; an h that needs none (detach it under no_grad) costs the losses alone.
    err int32 [1]: a device error word that the calls' is OR-ed into.  Returns (total, CE [N] or None, KD [N] or None).
    """

    @staticmethod
    def forward(ctx, h, w, target, g_lm, idx, t, g_kd, tau, mix, err):
        V, d = w.shape
        if w.dtype != torch.bfloat16 or not w.is_contiguous():
            raise ValueError("the head must be a contiguous bf16 [V, d]")
        h2 = _rows(h, d, "h")
        N, dev = h2.shape[0], h.device
        ld = h2.stride(0) if N > 1 else d
        grad = ctx.needs_input_grad[0]
        dh = torch.empty((N, d), dtype=torch.bfloat16, device=dev) if grad else None
        total = ce = kd = None
        if target is not None:
            target = _packed(_tokens(target.reshape(-1), V))
            g_lm = _packed(g_lm.to(torch.float32))
            if target.numel() != N or g_lm.numel() != N:
                raise ValueError("one target and one weight per row of h")
            ce, lse = torch.empty(N, dtype=torch.float32, device=dev), torch.empty(N, dtype=torch.float32, device=dev)
            ws = torch.empty(qad_linear_ce_workspace_bytes(N, d, V, grad, 0) // 4, dtype=torch.int32, device=dev)
            if grad:
                qad_linear_ce_fwd_bwd(h2, ld, w, d, target, g_lm, ce, lse, dh, None, 0, N, d, V, ws)
            else:
                qad_linear_ce_fwd(h2, ld, w, d, target, ce, lse, N, d, V, ws)
            err.bitwise_or_(ws[:1])
            total = torch.dot(ce, g_lm)
        if idx is not None:
            K = idx.shape[-1]
            idx = _packed(_tokens(idx.reshape(N, K), V))
            t = _packed(t.reshape(N, K).to(torch.float32))
            g_kd = _packed(g_kd.to(torch.float32))
            mix = None if mix is None else _packed(mix.to(torch.float32))
            if g_kd.numel() != N or (mix is not None and mix.numel() != N):
                raise ValueError("one distillation weight (and mix) per row of h")
            kd = torch.empty(N, dtype=torch.float32, device=dev)
            if grad:
                qad_distill_topk_fwd_bwd(h2, ld, w, d, idx, t, mix, 1.0 / tau, g_kd, kd, dh, int(target is not None), N,
                                         d, V, K, err)
            else:
                qad_distill_topk_fwd(h2, ld, w, d, idx, t, mix, 1.0 / tau, kd, N, d, V, K, err)
            total = torch.dot(kd, g_kd) if total is None else total + torch.dot(kd, g_kd)
        if total is None:
            raise ValueError("neither targets nor teacher logits")
        if grad:
            ctx.save_for_backward(dh)
        ctx.shape = h.shape
        ctx.mark_non_differentiable(*[x for x in (ce, kd) if x is not None])
        return total, ce, kd

    @staticmethod
    @once_differentiable
    def backward(ctx, dtotal, _ce, _kd):
        (dh,) = ctx.saved_tensors
        # as a 1 x 1 tensor the factor stays fp32 (a scalar tensor would be rounded to dh's bf16 first); one rounding
        dh = torch.mul(dh, dtotal.to(torch.float32).view(1, 1), out=torch.empty_like(dh))
        return (dh.view(ctx.shape), None, None, None, None, None, None, None, None, None)


class QADHeadLoss(torch.nn.Module):
    """The loss of a scale-only QAD step on the frozen output head (AngelSlim mcore_qad walkthrough,
    section 二.5): total = lm_weight * lm + distill_weight * distill, each a mean over its tokens.

    forward(h, target=None, teacher_idx=None, teacher_logits=None, mix=None) -> (total, lm, distill): lm is
    the cross entropy over the rows with a target, distill the divergence over the teacher's top tokens, over the
    rows that keep one (a teacher_idx in the vocabulary whose logit is not -inf): padding does not dilute either mean.
    A target or teacher token past the vocabulary carries nothing, as a negative one does, and sets a bit that
    device_error() returns.
    """

    def __init__(self, w, lm_weight=1.0, distill_weight=1.0, tau=1.0):
        super().__init__()
        self.register_buffer("w", _packed(w.to(torch.bfloat16)))
        self._err = {}  # device -> error word; not a buffer, which data parallelism would overwrite with rank 0's
        self.lm_weight, self.distill_weight, self.tau = float(lm_weight), float(distill_weight), float(tau)

    def device_error(self):
        """The QAD_DEV_* bits of the calls since it was last read (0: none), and clears them; waits for the device."""
        code = 0
        for err in self._err.values():
            code |= int(err.item())
            err.zero_()
        return code

    def forward(self, h, target=None, teacher_idx=None, teacher_logits=None, mix=None):
        N, V = h.numel() // h.shape[-1], self.w.shape[0]
        g_lm = g_kd = None
        # few operations: small steps wait for their launches
        if target is not None:
            target = _tokens(target.reshape(-1), V)
            live = target.clamp(0, V - 1) == target
            lm_rows = live.sum().clamp_min_(1)
            g_lm = live / lm_rows
            if self.lm_weight != 1.0:
                g_lm.mul_(self.lm_weight)
        if teacher_idx is not None:
            K = teacher_idx.shape[-1]
            teacher_idx, teacher_logits = _tokens(teacher_idx.reshape(N, K), V), teacher_logits.reshape(N, K)
            kept = ((teacher_idx.clamp(0, V - 1) == teacher_idx) & (teacher_logits != -torch.inf)).any(1)
            kd_rows = kept.sum().clamp_min_(1)
            g_kd = kept / kd_rows
            if self.distill_weight != 1.0:
                g_kd.mul_(self.distill_weight)
        if not torch.is_grad_enabled():
            h = h.detach()
        if h.device not in self._err:
            self._err[h.device] = torch.zeros(1, dtype=torch.int32, device=h.device)
        total, ce, kd = QADHeadLossFunction.apply(h, self.w, target, g_lm, teacher_idx, teacher_logits, g_kd, self.tau,
                                                  mix, self._err[h.device])
        return total, None if ce is None else ce.sum() / lm_rows, None if kd is None else kd.sum() / kd_rows
