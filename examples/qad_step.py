"""A scale-only QAD training run of a small mixture-of-experts model, end to end on the library's calls:

  embedding -> [residual RMSNorm -> router -> routed experts, fake-quantized] x layers -> residual RMSNorm
  -> cross entropy on the frozen head + distillation from the unquantized model's top logits -> scale gradients

Only the quantizer scales are trained; the teacher is the same frozen model with the quantizers off
("MCoreQAD Backend", opening section).

    python examples/qad_step.py [--fmt N] [--steps N] [--d N] [--layers N] [--vocab N] [--tokens N] [--topk N]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import scale_only_quantization_gb300 as Q  # noqa: E402
import synth  # noqa: E402
from scale_only_quantization_gb300.autograd import QADHeadLoss, QADMoE, QADMoEFunction, QADRMSNorm  # noqa: E402


class Model(torch.nn.Module):
    """Random frozen weights; one router [E, d] and one expert stack per layer."""

    def __init__(self, fmt, d=256, F=128, E=8, topk=2, layers=2, vocab=4001, lm_weight=0.01, seed=0,
                 device="cuda"):
        super().__init__()
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        bf = torch.bfloat16

        def rand(*shape):
            return torch.randn(shape, generator=g, device=device)

        self.topk = topk
        self.register_buffer("embed", rand(vocab, d).to(bf))
        self.norms = torch.nn.ModuleList(QADRMSNorm(1 + 0.1 * rand(d)) for _ in range(layers + 1))
        self.routers = [(rand(E, d) * d ** -0.5).to(bf) for _ in range(layers)]
        self.experts = torch.nn.ModuleList()
        for i in range(layers):
            inp = synth.make_inputs(dict(E=E, d=d, F=F, topk=topk, T=1, fmt=fmt), seed=seed + i, device=device)
            # weights large enough for the experts to move the residual stream
            w13, w2 = (inp["w13"].float() * (50 / d ** 0.5)).to(bf), (inp["w2"].float() * (50 / F ** 0.5)).to(bf)
            self.experts.append(QADMoE(w13, synth.init_scales(w13, fmt, g), w2, synth.init_scales(w2, fmt, g), fmt))
        self.head = QADHeadLoss((rand(vocab, d) * 2 * d ** -0.5).to(bf), lm_weight=lm_weight, distill_weight=1.0)

    def hidden(self, tokens, quantized=True):
        x, res = self.embed[tokens], None
        for norm, router, moe in zip(self.norms, self.routers, self.experts):
            y, res = norm(x, res)
            p, idx = torch.topk(y.float() @ router.float().T, self.topk, dim=1)
            p, idx = torch.softmax(p, dim=1), idx.to(torch.int32).contiguous()
            if quantized:
                x = moe(y, idx, p)
            else:
                x = QADMoEFunction.apply(y, idx, p, moe.w13, moe.s13, moe.w2, moe.s2, moe.fmt, Q.QAD_FLAG_NO_QUANT)
        return self.norms[-1](x, res)[0]

    @torch.no_grad()
    def teacher(self, tokens, k):
        """The unquantized model's top k logits and their tokens."""
        z = self.hidden(tokens, quantized=False).float() @ self.head.w.float().T
        t, idx = torch.topk(z, k, dim=1)
        return idx.to(torch.int32).contiguous(), t.contiguous()


def train(fmt=Q.QAD_FMT_NVFP4, steps=20, tokens=512, topk=32, lr=0.005, log=print, **model):
    """Trains the scales for `steps` steps on random tokens; returns the (total, lm, distill) of every step."""
    m = Model(fmt, **model)
    scales = [p for p in m.parameters() if p.requires_grad]
    # a step of Adam moves a parameter by about its rate: `lr` is a fraction of the tensor's typical scale
    opt = torch.optim.AdamW([dict(params=[s], lr=lr * float(s.detach().mean())) for s in scales], weight_decay=0.0,
                            betas=(0.9, 0.95))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    vocab = m.embed.shape[0]
    x = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    idx, t = m.teacher(x, topk)
    target = idx[:, 0].clone()  # no corpus here: the token that the unquantized model would write
    target[: tokens // 8] = -1  # a prompt: no language-model loss
    history = []
    for step in range(steps):
        opt.zero_grad(set_to_none=True)
        total, lm, kd = m.head(m.hidden(x), target, idx, t)
        total.backward()
        torch.nn.utils.clip_grad_norm_(scales, 1.0)
        opt.step()
        history.append(tuple(float(v.detach()) for v in (total, lm, kd)))
        if log:
            log("step %2d  total %.5f  lm %.5f  distill %.5f" % ((step,) + history[-1]))
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--fmt", type=int, default=Q.QAD_FMT_NVFP4, help="a qad_fmt number")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--topk", type=int, default=32, help="teacher logits kept per token")
    ap.add_argument("--d", type=int, default=256)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--vocab", type=int, default=4001)
    a = ap.parse_args()
    from scale_only_quantization_gb300 import build
    build.build()
    train(a.fmt, a.steps, a.tokens, a.topk, d=a.d, layers=a.layers, vocab=a.vocab)
