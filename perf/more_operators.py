"""Operators that a step of on-policy distillation needs beside the layer's training calls, as they are timed and
compared: each case as its plain form in elementary torch operations (own = False) or through the library's entry
points (own = True).

  few           the whole expert layer for a few tokens: the student writes its own text
  logprobs      log probabilities of given tokens, entropy and top alternatives of logits: the teacher reads it
  logprobs_grad their gradient with respect to the logits
  clip          the norm over all scale gradients, and the clipped gradients
  adamw         the step of the scales: the norm, clipping and AdamW over all tensors
"""
import math

import torch

own = False

# the library's numbers of its formats: element grid of the weights, elements per weight scale (0: a row), grid of
# the activations
FORMATS = {"nvfp4": (0, "e2m1", 16, "e2m1"), "w4a16": (1, "int4", 128, None), "fp8": (2, "e4m3", 0, "e4m3"),
           "nvfp4a16": (3, "e2m1", 16, None), "w8a8": (4, "int8", 0, "int8"), "w4afp8": (5, "int4", 128, "e4m3"),
           "nvfp4_deployed": (6, "e2m1", 16, "e2m1g")}
QMAX = {"e2m1": 6.0, "int4": 7.0, "e4m3": 448.0, "int8": 127.0}
BETAS, ADAM_EPS, DECAY, FLOOR = (0.9, 0.95), 1e-8, 0.01, 1e-6


def listed():
    return [
        # one token of a generation loop through a Qwen3-30B-A3B layer: eight experts' weights are all there is to read
        dict(name="few_token_nvfp4", op="few", T=1, d=2048, F=768, E=128, k=8, fmt="nvfp4", zipf=False),
        # a handful of sequences side by side in a GPT-OSS-wide layer with some experts much in demand
        dict(name="few_wide_fp8", op="few", T=5, d=2880, F=2880, E=32, k=4, fmt="fp8", zipf=True),
        # a batch of 32 rollouts: nearly every expert is asked for
        dict(name="few_batch_w4a16", op="few", T=32, d=2048, F=768, E=128, k=8, fmt="w4a16", zipf=False),
        # the logits of one sampled token: its probability, and the alternatives an interface shows
        dict(name="logprobs_token", op="logprobs", N=1, V=151936, ldz=151936, dtype="fp32", K=20, tau=0.6),
        # a teacher reading 1000 tokens over a vocabulary of odd size, rows at any alignment
        dict(name="logprobs_odd", op="logprobs", N=1000, V=50257, ldz=50257, dtype="bf16", K=100, tau=1.0),
        # a teacher reading two sequences of 2048: the top logits that the distillation loss takes
        dict(name="logprobs_teacher", op="logprobs", N=4096, V=151936, ldz=151936, dtype="bf16", K=64, tau=1.0),
        # a policy gradient with an entropy bonus on a tiny model's fp32 logits, softened, a slice of padded rows
        dict(name="logprobs_grad_tiny", op="logprobs_grad", N=512, V=32000, ldz=32064, dtype="fp32", tau=2.0),
        # the same for two sequences of 2048 over the large vocabulary
        dict(name="logprobs_grad_batch", op="logprobs_grad", N=4096, V=151936, ldz=151936, dtype="bf16", tau=1.0),
        # gradients of a small model's scales: launches are all
        dict(name="clip_tiny", op="clip", layers=2, E=4, d=256, F=128, B=16, norms=True),
        # eight Qwen3-30B-A3B layers' block scales: 302 million gradients
        dict(name="clip_model", op="clip", layers=8, E=128, d=2048, F=768, B=16, norms=False),
        # the optimizer step of the small model
        dict(name="adamw_tiny", op="adamw", layers=2, E=4, d=256, F=128, B=16, norms=True),
        # the optimizer step of four of the large layers, their norms trained as well
        dict(name="adamw_model", op="adamw", layers=4, E=128, d=2048, F=768, B=16, norms=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, m=16):
    return max(lo, m * (_log_int(rng, lo, hi) // m))


def draw(rng):
    op = rng.choice(["few", "few", "logprobs", "logprobs", "logprobs_grad", "clip", "adamw"])
    while True:
        if op == "few":
            fmt = rng.choice(sorted(FORMATS))
            m = 128 if FORMATS[fmt][2] == 128 else 16
            E = _log_int(rng, 4, 128)
            c = dict(op=op, T=_log_int(rng, 1, 64), d=_width(rng, 256, 4096, m), F=_width(rng, 128, 4096, m), E=E,
                     k=rng.randint(1, min(8, E)), fmt=fmt, zipf=rng.random() < 0.5)
            size = 3 * c["d"] * c["F"]
            fits = E * size <= 128 * 3 * 2048 * 768 and c["T"] * c["k"] * size <= 256 * 3 * 2048 * 768
        elif op in ("logprobs", "logprobs_grad"):
            V = _log_int(rng, 1000, 160000)
            c = dict(op=op, N=_log_int(rng, 1, 4096), V=V, ldz=V + rng.choice([0, 0, 47, -V % 64]),
                     dtype=rng.choice(["bf16", "fp32"]), tau=rng.choice([0.6, 1.0, 2.0]))
            if op == "logprobs":
                c["K"] = rng.choice([0, _log_int(rng, 1, 128), _log_int(rng, 1, 128)])
            fits = c["N"] * V * (2 if c["dtype"] == "fp32" else 1) <= 4096 * 151936
        else:
            B = rng.choice([16, 128, 0])
            c = dict(op=op, layers=_log_int(rng, 1, 20 if op == "clip" else 7), E=_log_int(rng, 1, 128),
                     d=_width(rng, 128, 4096, 128), F=_width(rng, 128, 2048, 128), B=B, norms=rng.random() < 0.5)
            fits = sum(_sizes(c)) <= (288 << 20 if op == "clip" else 144 << 20)
        if fits:
            return c


def _sizes(case):
    """Elements of each parameter: per layer the scales of both expert stacks, and the norm's weight if it is trained."""
    E, d, F, B = case["E"], case["d"], case["F"], case["B"]
    layer = [E * 2 * F * (d // B if B else 1), E * d * (F // B if B else 1)] + ([d] if case["norms"] else [])
    return layer * case["layers"]


# ------------------------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    """Inputs, weights, output buffers and workspaces that a training or generating program keeps from step to step."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    bf = torch.bfloat16
    s = dict(case)
    op = case["op"]
    if op == "few":
        T, d, F, E, k = (case[n] for n in ("T", "d", "F", "E", "k"))
        _, grid, block, act = FORMATS[case["fmt"]]
        for w, sc, n, m in (("w13", "s13", 2 * F, d), ("w2", "s2", d, F)):
            s[w] = torch.empty((E, n, m), dtype=bf, device="cuda")
            b = block or m
            s[sc] = torch.empty((E, n, m // b), device="cuda")
            for e in range(E):
                we = (0.02 * randn(n, m)).to(bf)
                s[w][e] = we
                # the scales' usual start, a little off as training leaves them
                s[sc][e] = we.float().abs().view(n, m // b, b).amax(2) / QMAX[grid] * (0.9 + 0.2 * rand(n, m // b))
            if act == "e2m1g":  # generating with deployed scales: made once, an E4M3 number times one of the matrix
                top = s[sc].amax((1, 2), keepdim=True) / 448.0
                s[sc] = (s[sc] / top).to(torch.float8_e4m3fn).float() * top
        s["x"] = randn(T, d).to(bf)
        # routing without replacement; with zipf some experts are asked for far more often than others
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        keys = torch.log(rand(T, E).clamp_min(1e-20)) * (rank ** 1.2 if case["zipf"] else 1.0)
        s["idx"] = torch.topk(keys, k, 1).indices.to(torch.int32)
        s["p"] = torch.softmax(randn(T, k), 1)
        s["out"] = torch.empty((T, d), dtype=bf, device="cuda")
        return s
    if op in ("logprobs", "logprobs_grad"):
        N, V, ldz = case["N"], case["V"], case["ldz"]
        dt = bf if case["dtype"] == "bf16" else torch.float32
        z = randn(N, ldz).mul_(2.5)
        # from unsure to certain: each row has a few tokens well above the rest
        at = torch.randint(0, V, (N, 8), generator=g, device="cuda")
        z.scatter_add_(1, at, 14 * rand(N, 8) * rand(N, 1))
        z[:, V - V // 500:] = -torch.inf  # a vocabulary padded behind its last word
        s["z"] = z.to(dt)[:, :V]
        t = torch.where(rand(N) < 0.8, at[:, 0], torch.randint(0, V - V // 500, (N,), generator=g, device="cuda"))
        t = t.clamp_max(V - V // 500 - 1)
        drop = (rand(N) < 1 / 16) & (torch.arange(N, device="cuda") > 0)  # prompt tokens are not asked for
        s["token"] = torch.where(drop, -1, t).to(torch.int32)
        if op == "logprobs":
            for name in ("logp", "lse", "entropy"):
                s[name] = torch.empty(N, device="cuda")
            s["top_idx"] = torch.empty((N, case["K"]), dtype=torch.int32, device="cuda")
            s["top_logit"] = torch.empty((N, case["K"]), device="cuda")
            s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
            return s
        s["lse"], s["entropy"] = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
        for i in range(0, N, 512):  # what the forward call left, in 64 bits
            x = s["z"][i:i + 512].double() / case["tau"]
            l = torch.logsumexp(x, 1, keepdim=True)
            s["lse"][i:i + 512] = l[:, 0]
            s["entropy"][i:i + 512] = -(torch.exp(x - l) * (x - l).clamp_min(-1e4)).sum(1)
        s["g_logp"], s["g_ent"] = randn(N) / N, 0.01 * (0.5 + rand(N)) / N
        s["dz"] = torch.empty((N, V), dtype=dt, device="cuda")
        return s
    sizes = _sizes(case)
    # gradients of very different sizes from tensor to tensor; a few large ones in each
    like = [torch.empty(n, dtype=bf if case["norms"] and i % 3 == 2 else torch.float32, device="cuda")
            for i, n in enumerate(sizes)]
    s["grads"] = [(randn(n) * (1 + 30 * (rand(n) < 1e-4)) * 10 ** (-1 - 3 * rand(1)) / math.sqrt(n)).to(t.dtype)
                  for n, t in zip(sizes, like)]
    s["norm"] = torch.empty(1, device="cuda")
    s["max_norm"] = 0.01
    if op == "clip":
        s["out"] = like
        return s
    s["params"] = [0.003 * (0.5 + rand(n)) for n in sizes]
    s["m"] = [0.1 * t.float() * (1 + randn(n)) for n, t in zip(sizes, s["grads"])]
    s["v"] = [t.float().square() * (0.05 + rand(n)) for n, t in zip(sizes, s["grads"])]
    s["lr"] = 2e-4 * 0.003 * (0.5 + rand(len(sizes)))
    s["steps"] = torch.full((1,), 7, dtype=torch.int64, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ one pass


def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _kept(s, name, make):
    """A workspace or list of the state: made at its first pass and kept."""
    if name not in s:
        s[name] = make()
    return s[name]


def _run_own(s):
    import scale_only_quantization_gb300 as Q
    op = s["op"]

    def space(nbytes, *shape):
        return _kept(s, "ws", lambda: torch.empty(nbytes(*shape), dtype=torch.uint8, device="cuda"))

    if op == "few":
        shape = _kept(s, "shape", lambda: Q.shape(s["T"], s["d"], s["F"], s["E"], s["k"], FORMATS[s["fmt"]][0]))
        Q.qad_moe_few_fwd(shape, s["x"], s["idx"], s["p"], s["w13"], s["s13"], s["w2"], s["s2"], s["out"],
                          space(Q.qad_moe_few_workspace_bytes, shape))
        return dict(out=s["out"])
    if op == "logprobs":
        kind = Q.QAD_BF16 if s["dtype"] == "bf16" else Q.QAD_F32
        K = s["K"]
        Q.qad_token_logprobs(s["z"], kind, s["ldz"], s["token"], 1 / s["tau"], s["logp"], s["lse"], s["entropy"],
                             s["top_idx"] if K else None, s["top_logit"] if K else None, s["N"], s["V"], K, s["err"])
        out = dict(logp=s["logp"], lse=s["lse"], entropy=s["entropy"])
        return dict(out, top_idx=s["top_idx"], top_logit=s["top_logit"]) if K else out
    if op == "logprobs_grad":
        kind = Q.QAD_BF16 if s["dtype"] == "bf16" else Q.QAD_F32
        Q.qad_token_logprobs_bwd(s["z"], kind, s["ldz"], s["token"], 1 / s["tau"], s["lse"], s["entropy"], s["g_logp"],
                                 s["g_ent"], s["dz"], s["V"], s["N"], s["V"])
        return dict(dz=s["dz"])
    ws = space(Q.qad_grad_norm_workspace_bytes)
    grads = _kept(s, "grad_list", lambda: Q.tensor_list(s["grads"]))
    Q.qad_grad_norm(grads, s["norm"], ws)
    if op == "clip":
        Q.qad_grad_clip(grads, _kept(s, "out_list", lambda: Q.tensor_list(s["out"])), s["norm"], s["max_norm"])
        return dict(norm=s["norm"], out=s["out"])
    lists = _kept(s, "lists", lambda: [Q.tensor_list(s[name]) for name in ("params", "m", "v")])
    Q.qad_adamw_step(lists[0], grads, lists[1], lists[2], s["lr"], BETAS[0], BETAS[1], ADAM_EPS, DECAY, FLOOR, s["norm"],
                     s["max_norm"], s["steps"], ws)
    return dict(norm=s["norm"], params=s["params"], m=s["m"], v=s["v"])


def _grid(x, kind):
    """x rounded to the nearest value of the grid (ties to the even code), saturating."""
    if kind == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    if kind in ("int4", "int8"):
        lo, hi = (-8, 7) if kind == "int4" else (-128, 127)
        return x.round().clamp(lo, hi)
    a = x.abs()
    steps = (a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float()
    return torch.copysign(0.5 * steps + (a > 2.5).float() + (a >= 3.5).float() + 2 * (a > 5).float(), x)


def _fake(v, scale, kind):
    """bf16(q(v / s) * s) over the last axis, s one number per block of it: what the layer's quantizers make."""
    shape = v.shape
    v = v.float().view(*scale.shape, -1)
    sc = scale.unsqueeze(-1)
    x = torch.where(sc > 0, v / sc, 0.0)
    return (_grid(x, kind) * sc).to(torch.bfloat16).float().view(shape)


def _over(a, q):
    """fp32(a / q): by way of 64 bits, as torch may multiply by a rounded reciprocal in 32."""
    return (a.double() / q).float()


def _fake_act(v, kind):
    if kind is None:
        return v
    n, m = v.shape
    if kind in ("e4m3", "int8"):
        return _fake(v, _over(v.abs().amax(1, keepdim=True), QMAX[kind]), kind)
    scale = _over(v.abs().view(n, m // 16, 16).amax(2), 6.0)
    if kind == "e2m1g":
        top = _over(scale.amax(1, keepdim=True), 448.0)
        scale = torch.where(top > 0, (scale / top).to(torch.float8_e4m3fn).float() * top, 0.0)
    return _fake(v, scale, "e2m1")


def _plain_few(s):
    _, grid, _, act = FORMATS[s["fmt"]]
    T, k, F = s["T"], s["k"], s["F"]
    e = s["idx"].long().reshape(-1)
    a = _fake_act(s["x"].float(), act).repeat_interleave(k, 0)
    # z1, h and y are bf16 in the layer's definition: what its quantizers and its combine read
    z = torch.bmm(_fake(s["w13"][e], s["s13"][e], grid), a.unsqueeze(2)).squeeze(2).to(torch.bfloat16).float()
    gate, up = z[:, :F], z[:, F:]
    h = _fake_act((gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16).float(), act)
    y = torch.bmm(_fake(s["w2"][e], s["s2"][e], grid), h.unsqueeze(2)).squeeze(2).to(torch.bfloat16).float()
    return dict(out=(y.view(T, k, -1) * s["p"].unsqueeze(2)).sum(1).to(torch.bfloat16))


def _plain_logprobs(s):
    z, K = s["z"].float(), s["K"]
    x = z / s["tau"]
    x = x - x.amax(1, keepdim=True)
    e = torch.exp(x)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    lse = (z.amax(1, keepdim=True) / s["tau"] + log_total).squeeze(1)
    entropy = (log_total - (e * x.clamp_min(-1e30)).sum(1, keepdim=True) / total).squeeze(1)
    t = s["token"].long()
    at = x.gather(1, t.clamp_min(0).unsqueeze(1))
    out = dict(logp=torch.where(t >= 0, (at - log_total).squeeze(1), 0.0), lse=lse, entropy=entropy)
    if not K:
        return out
    # the value's order as a whole number, ties to the lowest index: one key for both
    del x, e
    bits = (z + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = torch.topk((order << 32) - torch.arange(s["V"], device=z.device), K, 1).values
    idx = torch.remainder(-key, 1 << 32)
    return dict(out, top_idx=idx.to(torch.int32), top_logit=z.gather(1, idx))


def _plain_logprobs_grad(s):
    t = s["token"].long()
    logp = s["z"].float() / s["tau"] - s["lse"].unsqueeze(1)
    p = torch.exp(logp)
    g = torch.where(t >= 0, s["g_logp"], 0.0).unsqueeze(1)
    dz = -p * (g + s["g_ent"].unsqueeze(1) * (logp.clamp_min(-1e30) + s["entropy"].unsqueeze(1)))
    dz.scatter_add_(1, t.clamp_min(0).unsqueeze(1), g)
    return dict(dz=(dz / s["tau"]).to(s["z"].dtype))


def _norm_and_factor(s):
    total = torch.stack([t.double().square().sum() for t in s["grads"]]).sum().sqrt()
    return total, (s["max_norm"] / (total + 1e-6)).clamp_max(1.0).float()


def _plain_clip(s):
    total, factor = _norm_and_factor(s)
    return dict(norm=total.float().view(1), out=[(t.float() * factor).to(t.dtype) for t in s["grads"]])


def _adamw(p, t, m, v, lr, steps, factor):
    t = t.float() * factor
    m.mul_(BETAS[0]).add_(t * (1 - BETAS[0]))
    v.mul_(BETAS[1]).add_(t * t * (1 - BETAS[1]))
    c1, c2 = 1 - BETAS[0] ** steps.double(), 1 - BETAS[1] ** steps.double()
    step = lr / c1.float() * m / (torch.sqrt(v / c2.float()) + ADAM_EPS)
    p.copy_((p - lr * DECAY * p - step).clamp_min(FLOOR))


def _plain_adamw(s):
    total, factor = _norm_and_factor(s)
    s["steps"] += 1
    [_adamw(p, t, m, v, lr, s["steps"], factor) for p, t, m, v, lr in zip(s["params"], s["grads"], s["m"], s["v"], s["lr"])]
    return dict(norm=total.float().view(1), params=s["params"], m=s["m"], v=s["v"])


_PLAIN = {"few": _plain_few, "logprobs": _plain_logprobs, "logprobs_grad": _plain_logprobs_grad, "clip": _plain_clip,
          "adamw": _plain_adamw}


# ------------------------------------------------------------------------------------------------ work


def work(case):
    op = case["op"]
    if op == "few":
        T, d, F, E, k = (case[n] for n in ("T", "d", "F", "E", "k"))
        share = [r ** -1.2 if case["zipf"] else 1.0 for r in range(1, E + 1)]
        # experts that some token names, about; a weight's own two bytes and its part of a scale
        experts = sum(1 - (1 - min(1.0, k * v / sum(share))) ** T for v in share)
        block = FORMATS[case["fmt"]][2]
        per = 3 * d * F * (2 + (4 / block if block else 0)) + (0 if block else 4 * (2 * F + d))
        return dict(bytes=int(max(experts, min(k, E)) * per) + 4 * T * d + 8 * T * k, flops=6 * T * k * d * F)
    if op in ("logprobs", "logprobs_grad"):
        n = case["N"] * case["V"] * (2 if case["dtype"] == "bf16" else 4)
        if op == "logprobs":
            return dict(bytes=n + case["N"] * (16 + 8 * case["K"]), flops=5 * case["N"] * case["V"])
        return dict(bytes=2 * n + 20 * case["N"], flops=6 * case["N"] * case["V"])
    sizes = _sizes(case)
    grads = sum(n * (2 if case["norms"] and i % 3 == 2 else 4) for i, n in enumerate(sizes))
    if op == "clip":
        return dict(bytes=2 * grads + 4, flops=3 * sum(sizes))
    return dict(bytes=grads + 24 * sum(sizes) + 4 * len(sizes), flops=16 * sum(sizes))


# ------------------------------------------------------------------------------------------------ 64 bits


def _near(x, kind):
    """The grid again, in 64 bits: on each binade a rounding to whole multiples of its step."""
    if kind in ("int4", "int8"):
        return torch.clamp(torch.round(x), *((-8, 7) if kind == "int4" else (-128, 127)))
    low, bits, top = (0, 1, 6.0) if kind == "e2m1" else (-6, 3, 448.0)
    step = torch.ldexp(torch.ones_like(x), (torch.frexp(x).exponent - 1).clamp_min(low) - bits)
    return torch.clamp(torch.round(x / step) * step, -top, top)


def _quantized(v, scale, kind):
    """v in 64 bits through the quantizer whose steps are fp32: the quotient, and the product that is rounded to bf16."""
    b = v.shape[-1] // scale.shape[-1]
    sc = scale.double().repeat_interleave(b, -1)
    x = (v / torch.where(sc == 0, 1.0, sc)).float().double()
    return (_near(x, kind) * sc).float().to(torch.bfloat16).double()


def _quantized_act(v, kind):
    if kind is None:
        return v
    b = 16 if kind.startswith("e2m1") else v.shape[-1]
    scale = (v.abs().unflatten(-1, (-1, b)).amax(-1) / QMAX[kind[:4]]).float()
    if kind == "e2m1g":
        top = (scale.double().amax(-1, keepdim=True) / 448).float().double()
        code = _near((scale.double() / torch.where(top == 0, 1.0, top)).float().double(), "e4m3")
        scale = (code * top).float()
    return _quantized(v, scale, kind[:4])


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits; what the layer's definition holds in bf16 is rounded there."""
    s = prepare(case, seed)
    f = torch.float64
    op = case["op"]
    if op == "few":
        _, grid, _, act = FORMATS[case["fmt"]]
        x, out = _quantized_act(s["x"].to(f), act), torch.zeros((case["T"], case["d"]), dtype=f, device="cuda")
        for e in s["idx"].unique().tolist():  # one expert after another
            t, j = (s["idx"] == e).nonzero(as_tuple=True)
            z = (x[t] @ _quantized(s["w13"][e].to(f), s["s13"][e], grid).T).to(torch.bfloat16).to(f)
            h = z[:, :case["F"]] * torch.sigmoid(z[:, :case["F"]]) * z[:, case["F"]:]
            h = _quantized_act(h.to(torch.bfloat16).to(f), act)
            y = (h @ _quantized(s["w2"][e].to(f), s["s2"][e], grid).T).to(torch.bfloat16).to(f)
            out.index_add_(0, t, y * s["p"][t, j].to(f)[:, None])
        return dict(out=out)
    if op == "logprobs":
        parts = []
        for i in range(0, case["N"], 256):
            z = s["z"][i:i + 256].to(f)
            l = torch.log_softmax(z / case["tau"], 1)
            t = s["token"][i:i + 256].long()
            part = dict(logp=l.gather(1, t.clamp_min(0)[:, None])[:, 0] * (t >= 0),
                        lse=torch.logsumexp(z / case["tau"], 1), entropy=torch.special.entr(l.exp()).sum(1))
            if case["K"]:
                value, at = torch.sort(z, dim=1, descending=True, stable=True)
                part.update(top_idx=at[:, :case["K"]].to(torch.int32), top_logit=value[:, :case["K"]])
            parts.append(part)
        return {name: torch.cat([q[name] for q in parts]) for name in parts[0]}
    if op == "logprobs_grad":
        dz = torch.empty((case["N"], case["V"]), dtype=f, device="cuda")
        for i in range(0, case["N"], 256):
            at = slice(i, i + 256)
            x = s["z"][at].to(f) / case["tau"]
            p = torch.softmax(x, 1)
            t = s["token"][at].long()
            hit = torch.nn.functional.one_hot(t.clamp_min(0), case["V"]) * (t >= 0)[:, None]
            spread = torch.special.entr(p).sum(1, keepdim=True)
            d = s["g_logp"][at].to(f)[:, None] * (hit - p * (t >= 0)[:, None])
            d += s["g_ent"][at].to(f)[:, None] * (torch.special.entr(p) - p * spread)
            dz[at] = d / case["tau"]
        return dict(dz=dz)
    grads = [t.to(f) for t in s["grads"]]
    norm = math.sqrt(math.fsum(float((t ** 2).sum()) for t in grads))
    factor = min(1.0, s["max_norm"] / (norm + 1e-6))
    total = torch.tensor([norm], dtype=f, device="cuda")
    if op == "clip":
        return dict(norm=total, out=[t * factor for t in grads])
    n = int(s["steps"]) + 1
    new = dict(norm=total, params=[], m=[], v=[])
    for p, t, m, v, lr in zip(s["params"], grads, s["m"], s["v"], s["lr"].tolist()):
        t = t * factor
        m = torch.lerp(t, m.to(f), BETAS[0])
        v = torch.lerp(t * t, v.to(f), BETAS[1])
        mh, vh = m / (1 - BETAS[0] ** n), v / (1 - BETAS[1] ** n)
        new["params"].append((p.to(f) * (1 - lr * DECAY) - lr * mh / (vh ** 0.5 + ADAM_EPS)).clamp(min=FLOOR))
        new["m"].append(m)
        new["v"].append(v)
    return new
