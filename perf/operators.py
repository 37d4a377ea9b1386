"""Operators around the expert layer, as they are timed and compared: each case as its plain form in elementary torch
operations (own = False) or through the library's entry points (own = True).

  norm     residual addition + root-mean-square norm, with an 8-bit output and its scales; its gradient
  ce       softmax cross entropy of hidden states against a head [V, d], without keeping the logits; its gradients
  distill  distillation from a teacher's top logits over the teacher's own tokens; its gradient
"""
import math

import torch

own = False

EPS = 1e-6
QMAX = {"e4m3": 448.0, "int8": 127.0}


def listed():
    return [
        # one token of a generation loop entering an fp8 expert layer: latency is all
        dict(name="norm_token_e4m3", op="norm", T=1, d=2048, ldx=2048, res=True, quant="e4m3"),
        # the hidden states of one micro-batch (8 x 2048 tokens) before an fp8 expert layer
        dict(name="norm_batch_e4m3", op="norm", T=16384, d=2048, ldx=2048, res=True, quant="e4m3"),
        # INT8 fake-quantized input of a GPT-OSS-wide layer, an odd row count, x a slice of a wider projection
        dict(name="norm_slice_int8", op="norm", T=1003, d=2880, ldx=5776, res=False, quant="int8"),
        # the training backward of the micro-batch: residual gradient joined, norm weight trained
        dict(name="norm_batch_grad", op="norm_grad", T=16384, d=2048, ldr=2048, dres=True),
        # scoring a handful of answer tokens: the head is streamed once
        dict(name="ce_score_8", op="ce", N=8, d=2048, V=151936, grad=False, dw=False),
        # a tiny model's step over a 32000-token vocabulary
        dict(name="ce_tiny_step", op="ce", N=512, d=256, V=32000, grad=True, dw=False),
        # the language-model loss of half a micro-batch with a frozen head: loss and hidden-state gradient
        dict(name="ce_batch_step", op="ce", N=8192, d=2048, V=151936, grad=True, dw=False),
        # odd token count and odd vocabulary, the head trained as well
        dict(name="ce_head_trained", op="ce", N=2047, d=2880, V=50257, grad=True, dw=True),
        # a tiny model's distillation step from the teacher's top 16
        dict(name="distill_tiny_step", op="distill", N=64, d=256, V=32000, K=16, mixed=False, tau=1.0, grad=True),
        # self-distillation from the teacher's top 64 over a quarter micro-batch
        dict(name="distill_batch_step", op="distill", N=4096, d=2048, V=151936, K=64, mixed=False, tau=1.0, grad=True),
        # held-out divergence only, a number of kept logits that is no power of two
        dict(name="distill_eval", op="distill", N=1000, d=2880, V=50257, K=100, mixed=False, tau=1.0, grad=False),
        # a whole micro-batch of a wider model, forward and reverse divergence mixed per token, softened
        dict(name="distill_wide_step", op="distill", N=16384, d=4096, V=151936, K=32, mixed=True, tau=2.0, grad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return max(lo, 16 * (_log_int(rng, lo, hi) // 16))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "ce", "ce", "distill", "distill"])
    while True:
        if op == "norm":
            d = _width(rng, 64, 8192)
            c = dict(op=op, T=_log_int(rng, 1, 32768), d=d, ldx=d + 16 * rng.choice([0, 0, 1, 9]),
                     res=rng.random() < 0.7, quant=rng.choice(["none", "e4m3", "int8"]))
            fits = c["T"] * d <= 1 << 26
        elif op == "norm_grad":
            d = _width(rng, 64, 8192)
            c = dict(op=op, T=_log_int(rng, 1, 32768), d=d, ldr=d + 16 * rng.choice([0, 0, 3]),
                     dres=rng.random() < 0.7)
            fits = c["T"] * d <= 1 << 26
        elif op == "ce":
            grad = rng.random() < 0.7
            c = dict(op=op, N=_log_int(rng, 1, 8192), d=_width(rng, 64, 4096), V=_log_int(rng, 1000, 160000),
                     grad=grad, dw=grad and rng.random() < 0.4)
            fits = c["N"] * c["d"] * c["V"] <= 8192 * 2048 * 151936 // 2
        else:
            c = dict(op=op, N=_log_int(rng, 1, 16384), d=_width(rng, 64, 4096), V=_log_int(rng, 1000, 160000),
                     K=_log_int(rng, 4, 128), mixed=rng.random() < 0.5, tau=rng.choice([1.0, 2.0, 4.0]),
                     grad=rng.random() < 0.7)
            fits = c["N"] * c["d"] * c["K"] <= 16384 * 4096 * 32
        if fits:
            return c


# ------------------------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    """Inputs, output buffers and workspaces that a training or scoring program keeps from step to step."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda")

    bf = torch.bfloat16
    s = dict(case)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        T, d = case["T"], case["d"]
        # hidden states with a few channels far above the rest, as residual streams have them
        gain = torch.where(rand(d) < 0.01, 20.0, 1.0)
        s["gamma"] = (1 + 0.1 * randn(d)).to(bf)
        if op == "norm":
            s["x"] = (randn(T, case["ldx"])).to(bf)[:, :d]
            s["res"] = (randn(T, d) * gain).to(bf) if case["res"] else None
            s["r"] = torch.empty((T, d), dtype=bf, device="cuda") if case["res"] else None
            s["y"] = torch.empty((T, d), dtype=bf, device="cuda")
            s["codes"] = torch.empty((T, d), dtype=torch.uint8, device="cuda")
            s["scale"] = torch.empty(T, device="cuda")
            s["rstd"] = torch.empty(T, device="cuda")
        else:
            s["r"] = (randn(T, case["ldr"])).to(bf)[:, :d]
            s["r"].mul_(gain.to(bf))
            s["rstd"] = torch.rsqrt(s["r"].float().square().mean(1) + EPS)
            s["dy"] = (randn(T, d) * 1e-3).to(bf)
            s["dres"] = (randn(T, d) * 1e-3).to(bf) if case["dres"] else None
            s["dx"] = torch.empty((T, d), dtype=bf, device="cuda")
            s["dgamma"] = torch.empty(d, device="cuda")
        return s
    N, d, V = case["N"], case["d"], case["V"]
    s["w"] = (0.02 * randn(V, d)).to(bf)
    # each row's weight in the total loss: a mean over the tokens, weighted
    s["g"] = (0.5 + rand(N)) / N
    s["dh"] = torch.empty((N, d), dtype=bf, device="cuda")
    s["loss"] = torch.empty(N, device="cuda")
    if op == "ce":
        t = ints(0, V, N)
        # hidden states that favour the next token by 0 to 12 nats: from unsure to certain
        wt = s["w"][t].float()
        s["h"] = (randn(N, d) + 12 * rand(N, 1) / wt.square().sum(1, keepdim=True) * wt).to(bf)
        drop = (rand(N) < 1 / 16) & (torch.arange(N, device="cuda") > 0)  # prompt tokens carry no loss
        s["target"] = torch.where(drop, -1, t).to(torch.int32)
        s["lse"] = torch.empty(N, device="cuda")
        s["dw"] = torch.empty((V, d), dtype=bf, device="cuda") if case["dw"] else None
    else:
        K = case["K"]
        s["h"] = randn(N, d).to(bf)
        # K distinct tokens a row (gaps below V / K), and a teacher near the student, as self-distillation has it
        s["idx"] = ((ints(0, V, N, 1) + torch.cumsum(ints(1, max(2, V // K), N, K), 1)) % V).to(torch.int32)
        z = torch.bmm(s["w"][s["idx"].long()], s["h"].unsqueeze(2)).squeeze(2).float()
        s["t"] = z + randn(N, K) + 4 * rand(N, 1)
        if K > 8:  # some rows keep fewer tokens than K
            short = (rand(N, 1) < 0.1) & (torch.arange(K, device="cuda") >= K - 2)
            s["idx"] = torch.where(short, -1, s["idx"]).to(torch.int32)
        s["mix"] = rand(N) if case["mixed"] else None
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ one pass


def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _workspace(s, nbytes, *shape):
    """The workspace of a state: taken at its first pass and kept."""
    if "ws" not in s:
        s["ws"] = torch.empty(nbytes(*shape), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s):
    import scale_only_quantization_gb300 as Q
    op = s["op"]
    if op == "norm":
        kind = {"none": Q.QAD_ACT_NONE, "e4m3": Q.QAD_ACT_E4M3, "int8": Q.QAD_ACT_INT8}[s["quant"]]
        e4m3, int8 = s["quant"] == "e4m3", s["quant"] == "int8"
        # e4m3: the norm's output for the router and its codes for the experts; int8: the fake-quantized output
        Q.qad_rmsnorm_fwd(s["x"], s["res"], s["gamma"], EPS, kind, s["r"], None if int8 else s["y"],
                          s["y"] if int8 else None, s["codes"] if e4m3 else None,
                          s["scale"] if kind != Q.QAD_ACT_NONE else None, s["rstd"], s["T"], s["d"], s["ldx"], s["d"])
        out = dict(y=s["y"], rstd=s["rstd"])
        if s["res"] is not None:
            out["r"] = s["r"]
        if kind != Q.QAD_ACT_NONE:
            out["scale"] = s["scale"]
        if e4m3:
            out["q"] = s["codes"].view(torch.float8_e4m3fn)
        return out
    if op == "norm_grad":
        ws = _workspace(s, Q.qad_rmsnorm_workspace_bytes, s["T"], s["d"])
        Q.qad_rmsnorm_bwd(s["dy"], s["dres"], s["r"], s["gamma"], s["rstd"], s["dx"], s["dgamma"], s["T"], s["d"],
                          s["ldr"], ws)
        return dict(dx=s["dx"], dgamma=s["dgamma"])
    N, d, V = s["N"], s["d"], s["V"]
    if op == "ce":
        ws = _workspace(s, Q.qad_linear_ce_workspace_bytes, N, d, V, int(s["grad"]), int(s["dw"] is not None))
        if not s["grad"]:
            Q.qad_linear_ce_fwd(s["h"], d, s["w"], d, s["target"], s["loss"], s["lse"], N, d, V, ws)
            return dict(loss=s["loss"], lse=s["lse"])
        Q.qad_linear_ce_fwd_bwd(s["h"], d, s["w"], d, s["target"], s["g"], s["loss"], s["lse"], s["dh"], s["dw"], 0, N,
                                d, V, ws)
        out = dict(loss=s["loss"], lse=s["lse"], dh=s["dh"])
        return dict(out, dw=s["dw"]) if s["dw"] is not None else out
    if not s["grad"]:
        Q.qad_distill_topk_fwd(s["h"], d, s["w"], d, s["idx"], s["t"], s["mix"], 1 / s["tau"], s["loss"], N, d, V,
                               s["K"], s["err"])
        return dict(loss=s["loss"])
    Q.qad_distill_topk_fwd_bwd(s["h"], d, s["w"], d, s["idx"], s["t"], s["mix"], 1 / s["tau"], s["g"], s["loss"],
                               s["dh"], 0, N, d, V, s["K"], s["err"])
    return dict(loss=s["loss"], dh=s["dh"])


def _plain_norm(s):
    x, gamma = s["x"].float(), s["gamma"].float()
    r = x if s["res"] is None else (x + s["res"].float()).to(torch.bfloat16).float()  # the residual stream is bf16
    rstd = 1 / torch.sqrt((r * r).mean(1) + EPS)
    y = (r * rstd[:, None] * gamma).to(torch.bfloat16)  # what the layer and its quantizer read
    out = dict(rstd=rstd)
    if s["res"] is not None:
        out["r"] = r.to(torch.bfloat16)
    if s["quant"] == "none":
        return dict(out, y=y)
    scale = y.float().abs().amax(1) / QMAX[s["quant"]]
    q = torch.where(scale[:, None] > 0, y.float() / scale[:, None], 0.0)
    if s["quant"] == "e4m3":
        return dict(out, y=y, scale=scale, q=q.clamp(-448, 448).to(torch.float8_e4m3fn))
    q = q.round().clamp(-128, 127)
    return dict(out, y=(q * scale[:, None]).to(torch.bfloat16), scale=scale)


def _plain_norm_grad(s):
    r, rstd, dy = s["r"].float(), s["rstd"][:, None], s["dy"].float()
    n = r * rstd
    dn = dy * s["gamma"].float()
    dx = rstd * (dn - n * (dn * n).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.to(torch.bfloat16), dgamma=(dy * n).sum(0))


def _plain_ce(s):
    h, w, t = s["h"].float(), s["w"].float(), s["target"].long()
    z = h @ w.T
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(1)
    valid = t >= 0
    at = t.clamp_min(0)
    rows = torch.arange(s["N"], device=t.device)
    loss = torch.where(valid, lse - z[rows, at], 0.0)
    if not s["grad"]:
        return dict(loss=loss, lse=lse)
    p = e / total
    p[rows, at] -= 1
    p *= torch.where(valid, s["g"], 0.0)[:, None]
    out = dict(loss=loss, lse=lse, dh=(p @ w).to(torch.bfloat16))
    return dict(out, dw=(p.T @ h).to(torch.bfloat16)) if s["dw"] is not None else out


def _plain_distill(s):
    beta = 1 / s["tau"]
    keep = s["idx"] >= 0
    wk = s["w"][s["idx"].long().clamp_min(0)].float()
    z = torch.bmm(wk, s["h"].float().unsqueeze(2)).squeeze(2)
    # a row's last kept slots may be empty; every row here keeps one at least
    zs = torch.where(keep, z * beta, -torch.inf)
    ts = torch.where(keep, s["t"] * beta, -torch.inf)
    zs, ts = zs - zs.amax(1, keepdim=True), ts - ts.amax(1, keepdim=True)
    ez, et = torch.exp(zs), torch.exp(ts)
    sz, st = ez.sum(1, keepdim=True), et.sum(1, keepdim=True)
    q, p = ez / sz, et / st
    diff = torch.where(keep, (zs - torch.log(sz)) - (ts - torch.log(st)), 0.0)  # log q - log p
    # sum p (log p - log q) = sum p (exp(diff) - 1 - diff), every term of one sign: nothing cancels between near models
    kl, rkl = (p * (torch.expm1(diff) - diff)).sum(1), (q * (torch.expm1(-diff) + diff)).sum(1)
    m = torch.zeros_like(kl) if s["mix"] is None else s["mix"]
    loss = (1 - m) * kl + m * rkl
    if not s["grad"]:
        return dict(loss=loss)
    dz = (1 - m)[:, None] * (q - p) + m[:, None] * q * (diff - rkl[:, None])
    dz = dz * (beta * s["g"])[:, None]
    return dict(loss=loss, dh=torch.bmm(dz.unsqueeze(1), wk).squeeze(1).to(torch.bfloat16))


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "ce": _plain_ce, "distill": _plain_distill}


# ------------------------------------------------------------------------------------------------ work


def work(case):
    op = case["op"]
    if op == "norm":
        T, d = case["T"], case["d"]
        n = 2 + (4 if case["res"] else 0) + 2 + (1 if case["quant"] == "e4m3" else 0)
        return dict(bytes=T * d * n + 2 * d + 8 * T, flops=T * d * 6)
    if op == "norm_grad":
        T, d = case["T"], case["d"]
        return dict(bytes=T * d * (6 + (2 if case["dres"] else 0)) + 6 * d + 4 * T, flops=T * d * 10)
    N, d, V = case["N"], case["d"], case["V"]
    if op == "ce":
        # the logits once; with gradients the probabilities' product with the head, and with the hidden states
        products = 1 + int(case["grad"]) + int(case["dw"])
        return dict(bytes=2 * V * d * (2 if case["dw"] else 1) + N * d * (4 if case["grad"] else 2) + 16 * N,
                    flops=2 * products * N * V * d)
    K = case["K"]
    rows = V * -math.expm1(-N * K / V)  # rows of the head that some token names
    return dict(bytes=int(2 * rows * d) + N * d * (4 if case["grad"] else 2) + 8 * N * K + 12 * N,
                flops=(4 if case["grad"] else 2) * N * K * d)


# ------------------------------------------------------------------------------------------------ 64 bits


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits (linear algebra by torch's float64 products)."""
    if case["op"] == "ce" and case["N"] * case["d"] * case["V"] > 8192 * 2048 * 151936:
        return None
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "norm":
        r = s["x"].to(f)
        out = {}
        if s["res"] is not None:
            out["r"] = r + s["res"].to(f)
            r = out["r"].to(torch.bfloat16).to(f)
        out["rstd"] = (r.pow(2).sum(1) / case["d"] + EPS).pow(-0.5)
        y = torch.einsum("td,t,d->td", r, out["rstd"], s["gamma"].to(f))
        if case["quant"] == "none":
            return dict(out, y=y)
        y16 = y.to(torch.bfloat16).to(f)
        out["scale"] = y16.abs().max(1).values / QMAX[case["quant"]]
        if case["quant"] == "e4m3":
            return dict(out, y=y, q=y16 / out["scale"].clamp_min(1e-300)[:, None])
        return dict(out, y=(y16 / out["scale"].clamp_min(1e-300)[:, None]).round() * out["scale"][:, None])
    if case["op"] == "norm_grad":
        r, inv, dy, gamma = s["r"].to(f), s["rstd"].to(f)[:, None], s["dy"].to(f), s["gamma"].to(f)
        inner = (r * dy * gamma).sum(1, keepdim=True)
        dx = inv * dy * gamma - inv.pow(3) * r * inner / case["d"]
        dx = dx if s["dres"] is None else dx + s["dres"].to(f)
        return dict(dx=dx, dgamma=torch.einsum("td,td,t->d", dy, r, inv[:, 0]))
    if case["op"] == "ce":
        h, w = s["h"].to(f), s["w"].to(f)
        z = torch.matmul(h, w.t())
        lse = torch.logsumexp(z, 1)
        live = s["target"] >= 0
        t = torch.where(live, s["target"], 0).long()[:, None]
        loss = (lse - z.gather(1, t)[:, 0]) * live
        if not case["grad"]:
            return dict(loss=loss, lse=lse)
        z.sub_(lse[:, None]).exp_()
        z.scatter_add_(1, t, torch.full_like(t, -1, dtype=f))
        z.mul_((s["g"].to(f) * live)[:, None])
        out = dict(loss=loss, lse=lse, dh=torch.matmul(z, w))
        return dict(out, dw=torch.matmul(z.t(), h)) if case["dw"] else out
    keep = s["idx"] >= 0
    wk = s["w"][torch.where(keep, s["idx"], 0).long()].to(f)
    z = (wk @ s["h"].to(f)[:, :, None])[:, :, 0] / case["tau"]
    t = s["t"].to(f) / case["tau"]
    hide = torch.where(keep, 0.0, -1e30).to(f)
    lq, lp = torch.log_softmax(z + hide, 1), torch.log_softmax(t + hide, 1)
    q, p = lq.exp(), lp.exp()
    gap = (lp - lq) * keep
    kl, rkl = (p * gap).sum(1), -(q * gap).sum(1)
    m = torch.zeros_like(kl) if s["mix"] is None else s["mix"].to(f)
    loss = kl + m * (rkl - kl)
    if not case["grad"]:
        return dict(loss=loss)
    dz = ((1 - m)[:, None] * (q - p) - m[:, None] * q * (gap + rkl[:, None])) * s["g"].to(f)[:, None] / case["tau"]
    return dict(loss=loss, dh=(dz[:, None, :] @ wk)[:, 0])
