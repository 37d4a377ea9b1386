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
end, QADTokenLogprobs for what is read off logits the caller holds (the teacher's top alternatives), and
QADAdamW for the step of the scales.  QADMoE.few is the layer's forward for a few tokens (generation).
"""
import math

import torch
from torch.autograd.function import once_differentiable

from . import (QAD_ACT_NONE, qad_distill_topk_fwd, qad_distill_topk_fwd_bwd, qad_linear_ce_fwd, qad_linear_ce_fwd_bwd,
               qad_linear_ce_workspace_bytes, qad_moe_bwd_dgrad, qad_moe_bwd_scalegrad, qad_moe_few_fwd,
               qad_moe_few_workspace_bytes, qad_moe_fwd, qad_moe_workspace_bytes, qad_nvfp4_deploy_scales,
               qad_rmsnorm_bwd, qad_rmsnorm_fwd, qad_rmsnorm_workspace_bytes, qad_adamw_step, qad_grad_norm,
               qad_grad_norm_workspace_bytes, qad_token_logprobs, qad_token_logprobs_bwd, shape, tensor_list, QAD_BF16,
               QAD_F32, QAD_FLAG_NO_QUANT, QAD_FMT_NVFP4_E4M3)


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
        self._err = {}  # device -> error word of few(), as QADHeadLoss keeps it

    def device_error(self):
        """The QAD_DEV_* bits of few()'s calls since it was last read (0: none), and clears them; waits for the device.
        QAD_DEV_TIMEOUT: an output is invalid."""
        return QADHeadLoss.device_error(self)

    def forward(self, x, topk_idx, topk_w):
        return QADMoEFunction.apply(x.contiguous(), topk_idx.contiguous(), topk_w.contiguous(), self.w13, self.s13,
                                    self.w2, self.s2, self.fmt, self.flags)

    @torch.no_grad()
    def few(self, x, topk_idx, topk_w, quant=None):
        """The layer's output for at most QAD_MOE_FEW_MAX_T tokens, without a gradient: what a generation loop calls.
        quant False: the unquantized teacher; None: by the module's QAD_FLAG_NO_QUANT.  device_error() has what went
        wrong."""
        if quant is None:
            quant = not self.flags & QAD_FLAG_NO_QUANT
        E, two_f, d = self.w13.shape
        T, k = topk_idx.shape
        if x.dtype != torch.bfloat16 or topk_idx.dtype != torch.int32 or topk_w.dtype != torch.float32 or \
                x.shape != (T, d) or topk_w.shape != (T, k):
            raise ValueError("x bf16 [T, %d], topk_idx int32 [T, k] and topk_w fp32 [T, k], got %s %s, %s %s, %s %s" % (
                d, x.dtype, tuple(x.shape), topk_idx.dtype, tuple(topk_idx.shape), topk_w.dtype, tuple(topk_w.shape)))
        if {x.device, topk_idx.device, topk_w.device} != {self.w13.device}:
            raise ValueError("x, topk_idx and topk_w lie on the weights' device, %s" % self.w13.device)
        s = shape(T, d, two_f // 2, E, k, self.fmt, 0 if quant else QAD_FLAG_NO_QUANT)
        s13, s2 = self.s13, self.s2
        with torch.cuda.device(self.w13.device):
            if quant and self.fmt == QAD_FMT_NVFP4_E4M3:  # a program that generates much keeps these between updates
                s13, s2 = torch.empty_like(self.s13), torch.empty_like(self.s2)
                for a, b in ((self.s13, s13), (self.s2, s2)):
                    qad_nvfp4_deploy_scales(a, b, E, a.numel() // E)
            ws = torch.empty((qad_moe_few_workspace_bytes(s) + 3) // 4, dtype=torch.int32, device=x.device)
            out = torch.empty((T, d), dtype=torch.bfloat16, device=x.device)
            qad_moe_few_fwd(s, _packed(x), _packed(topk_idx), _packed(topk_w), self.w13, s13, self.w2, s2, out, ws)
            _error_word(self._err, x.device).bitwise_or_(ws[:1])
        return out


def _error_word(words, device):
    """The device's error word in `words` (device -> word), made at its first use: an ordinary tensor also where that is in
    inference mode, since it is written and cleared outside as well."""
    if device not in words:
        with torch.inference_mode(False):
            words[device] = torch.zeros(1, dtype=torch.int32, device=device)
    return words[device]


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
        total, ce, kd = QADHeadLossFunction.apply(h, self.w, target, g_lm, teacher_idx, teacher_logits, g_kd, self.tau,
                                                  mix, _error_word(self._err, h.device))
        return total, None if ce is None else ce.sum() / lm_rows, None if kd is None else kd.sum() / kd_rows


class QADTokenLogprobsFunction(torch.autograd.Function):
    """(logp, entropy, lse, top_idx, top_logit) of logits z [N, V] at temperature tau; the gradient is that of logp and
    entropy."""

    @staticmethod
    def forward(ctx, z, token, tau, top, err):
        N, V = z.shape
        kinds = {torch.bfloat16: QAD_BF16, torch.float32: QAD_F32}
        if z.dtype not in kinds:
            raise ValueError("logits must be bf16 or fp32, got %s" % z.dtype)
        if N and V and (z.stride(1) != 1 or z.stride(0) < V or z.data_ptr() % 16):
            z = _packed(z)
        if token is not None:
            token = _packed(_tokens(token.reshape(-1), V))
            if token.numel() != N:
                raise ValueError("one token per row of z")
            if token.device != z.device:
                raise ValueError("tokens on %s, logits on %s" % (token.device, z.device))
        ld = z.stride(0) if N > 1 else V
        lse, entropy = (torch.empty(N, dtype=torch.float32, device=z.device) for _ in range(2))
        logp = None if token is None else torch.empty_like(lse)
        top_idx = torch.empty((N, top), dtype=torch.int32, device=z.device) if top else None
        top_logit = torch.empty((N, top), dtype=torch.float32, device=z.device) if top else None
        with torch.cuda.device(z.device):
            qad_token_logprobs(z, kinds[z.dtype], ld, token, 1.0 / tau, logp, lse, entropy, top_idx, top_logit, N, V, top,
                               err)
        ctx.save_for_backward(z, lse, entropy, *(() if token is None else (token,)))
        ctx.tau, ctx.ld, ctx.kind = tau, ld, kinds[z.dtype]
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(lse, *((top_idx, top_logit) if top else ()))
        return logp, entropy, lse, top_idx, top_logit

    @staticmethod
    @once_differentiable
    def backward(ctx, g_logp, g_entropy, _lse, _idx, _logit):
        if g_logp is None and g_entropy is None:
            return None, None, None, None, None
        z, lse, entropy, *token = ctx.saved_tensors
        N, V = z.shape
        dz = torch.empty((N, V), dtype=z.dtype, device=z.device)
        g_logp, g_entropy = (None if g is None else g.to(torch.float32).contiguous() for g in (g_logp, g_entropy))
        with torch.cuda.device(z.device):
            qad_token_logprobs_bwd(z, ctx.kind, ctx.ld, token[0] if token else None, 1.0 / ctx.tau, lse, entropy, g_logp,
                                   g_entropy, dz, V, N, V)
        return dz, None, None, None, None


class QADTokenLogprobs(torch.nn.Module):
    """What is read off logits: forward(z, token=None) -> (logp, entropy, lse, top_idx, top_logit).

    logp [N] is the log probability of each row's token at temperature tau (None without tokens, 0 where the token is
    negative); top_idx and top_logit [N, top] the row's largest logits, which are teacher_idx and teacher_logits of
    QADHeadLoss (None with top 0).  logp and entropy have a gradient.  A token past the vocabulary sets a bit that
    device_error() returns.  Logits that do not start on a 16-byte boundary (z[1:] of an odd vocabulary) are copied first.
    """

    def __init__(self, tau=1.0, top=0):
        super().__init__()
        self.tau, self.top = float(tau), int(top)
        self._err = {}  # device -> error word, as QADHeadLoss keeps it

    device_error = QADHeadLoss.device_error

    def forward(self, z, token=None):
        return QADTokenLogprobsFunction.apply(z, token, self.tau, self.top, _error_word(self._err, z.device))


class QADAdamW(torch.optim.Optimizer):
    """AdamW of the quantizer scales with clipping by the norm over all gradients, in four launches at most for up to 480
    tensors of the same settings ("MCoreQAD Backend", YAML optim: lr, betas, weight decay, grad_clip).

    Parameters are fp32; groups may set lr, betas, eps, weight_decay and floor, the lower bound that keeps a scale
    positive (-inf: none).  max_norm None: no clipping (the norm is taken all the same).  Every parameter needs a gradient
    (fp32 or bf16) at each step; a step whose norm is not finite changes nothing, the count of steps neither.  last_norm
    [1] is the norm before clipping.  State: exp_avg, exp_avg_sq and step (an int64 on the device that parameters of the
    same settings and the same number of steps share).  A step may be captured once one has been taken eagerly; its
    replays read the rates that write_rates() has written, until other settings change or the parameters' memory does.
    """

    def __init__(self, params, lr=2e-4, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0, floor=-math.inf, max_norm=1.0):
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, floor=floor))
        self.max_norm = max_norm
        self.last_norm = None
        self._ws = self._plan = None

    def _make_plan(self):
        """Parameters of equal settings and as many steps behind them go together: (settings, parameters, their lists,
        rates, steps).  Each part counts in a tensor of its own: two of them with one counter would count twice."""
        every = [p for group in self.param_groups for p in group["params"]]
        dev = every[0].device if every else None
        for p in every:
            if p.dtype != torch.float32 or not p.is_contiguous() or not p.is_cuda or p.device != dev:
                raise ValueError("parameters are contiguous fp32 tensors of one CUDA device, got %s on %s" % (p.dtype, p.device))
            st = self.state[p]
            if "exp_avg" in st and {st["exp_avg"].device, st["exp_avg_sq"].device} != {dev}:
                raise ValueError("parameters on %s, their moments on %s: load the state again" % (dev, st["exp_avg"].device))
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a first step, or one of changed settings or parameters, is not captured: step once before")
        sets, counts, counters = {}, {}, set()
        for group in self.param_groups:
            key = (*group["betas"], group["eps"], group["weight_decay"], group["floor"])
            for p in group["params"]:
                step = self.state[p].get("step")
                if step is not None and id(step) not in counts:
                    counts[id(step)] = int(step)
                sets.setdefault((key, 0 if step is None else counts[id(step)]), []).append((p, group))
        plan = []
        for (key, _), members in sets.items():
            ps = [p for p, _ in members]
            for p in ps:
                st = self.state[p]
                if "exp_avg" not in st:
                    st["exp_avg"], st["exp_avg_sq"] = torch.zeros_like(p), torch.zeros_like(p)
            steps = next((self.state[p]["step"] for p in ps if "step" in self.state[p]), None)
            steps = torch.zeros(1, dtype=torch.int64, device=dev) if steps is None else steps.to(dev, torch.int64).view(1)
            if steps.data_ptr() in counters:
                steps = steps.clone()
            counters.add(steps.data_ptr())
            for p in ps:
                self.state[p]["step"] = steps
            lists = [tensor_list(x) for x in ([p.detach() for p in ps], [self.state[p]["exp_avg"] for p in ps],
                                              [self.state[p]["exp_avg_sq"] for p in ps])]
            plan.append(dict(key=key, members=members, lists=lists, steps=steps, lr=None,
                             rates=torch.empty(len(ps), dtype=torch.float32, device=dev)))
        if plan and (self._ws is None or self._ws.device != dev):
            self._ws = torch.empty(qad_grad_norm_workspace_bytes(), dtype=torch.uint8, device=dev)
            self.last_norm = torch.zeros(1, device=dev)
        return plan

    def __getstate__(self):
        return dict(super().__getstate__(), max_norm=self.max_norm)

    def __setstate__(self, state):
        """Of a copied or unpickled optimizer, and of load_state_dict(): the plan is made again."""
        super().__setstate__(state)
        self._plan = None
        for name in ("_ws", "last_norm"):
            self.__dict__.setdefault(name, None)

    def add_param_group(self, group):
        super().add_param_group(group)
        self._plan = None

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        # a plan holds as long as the settings and the parameters' memory stay
        settings = [(*g["betas"], g["eps"], g["weight_decay"], g["floor"], *[p.data_ptr() for p in g["params"]])
                    for g in self.param_groups]
        if self._plan is None or settings != self._settings:
            self._plan, self._settings = self._make_plan(), settings
        grads = []
        for part in self._plan:
            if any(p.grad is None for p, _ in part["members"]):
                raise ValueError("every parameter needs a gradient")
            if any(p.grad.device != self._ws.device for p, _ in part["members"]):
                raise ValueError("gradients lie on the parameters' device, %s" % self._ws.device)
            grads.append([_packed(p.grad) for p, _ in part["members"]])
        with torch.cuda.device(self._ws.device if grads else None):
            self._launch(grads)
        return loss

    def write_rates(self):
        """Writes the groups' rates to where the steps read them, on the current stream and without waiting for it.  step()
        does it; a program that replays a captured step calls it whenever its schedule has moved them."""
        for part in self._plan or ():
            lr = [float(group["lr"]) for _, group in part["members"]]
            if lr != part["lr"]:
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("rates have changed: call write_rates() before the capture")
                part["rates"].copy_(torch.tensor(lr, dtype=torch.float32, pin_memory=True), non_blocking=True)
                part["lr"] = lr

    def _launch(self, grads):
        self.write_rates()
        if grads:  # without clipping too: a step whose norm is not finite is left out
            qad_grad_norm([g for part in grads for g in part], self.last_norm, self._ws)
        max_norm = math.inf if self.max_norm is None else self.max_norm
        for part, gs in zip(self._plan, grads):
            b1, b2, eps, decay, floor = part["key"]
            p, m, v = part["lists"]
            qad_adamw_step(p, gs, m, v, part["rates"], b1, b2, eps, decay, floor, self.last_norm, max_norm, part["steps"],
                           self._ws)
            # written behind autograd's back: a graph that saved one of them must not be used
            torch.autograd.graph.increment_version([x for x, _ in part["members"]])
