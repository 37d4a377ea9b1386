"""The autograd views of the norm and the head loss, and the example that trains a small model with them."""
import os
import sys

import pytest
import torch

import scale_only_quantization_gb300 as Q

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _build():
    from scale_only_quantization_gb300 import build
    build.build()


def test_modules_hold_frozen_weights():
    from scale_only_quantization_gb300.autograd import QADHeadLoss, QADRMSNorm
    n = QADRMSNorm(torch.ones(64))
    assert not n.weight.requires_grad and n.weight.dtype == torch.bfloat16
    assert QADRMSNorm(torch.ones(64), trained=True).weight.requires_grad
    h = QADHeadLoss(torch.randn(10, 64))
    assert list(h.parameters()) == [] and h.w.dtype == torch.bfloat16


def test_rows_are_checked():
    from scale_only_quantization_gb300.autograd import _rows
    x = torch.zeros((6, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        _rows(x.float(), 64, "x")
    with pytest.raises(ValueError):
        _rows(x, 32, "x")
    assert _rows(x[:, 8:40], 32, "x").stride(0) == 64            # a slice of aligned rows is read in place
    assert _rows(x[:, 1:33], 32, "x").is_contiguous()            # an unaligned one is copied
    assert _rows(x.t()[:, :6], 6, "x").is_contiguous()
    assert _rows(x.view(2, 3, 64), 64, "x").shape == (6, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("act", [Q.QAD_ACT_NONE, Q.QAD_ACT_E4M3])
def test_norm_gradients_equal_the_abi_calls(act):
    from scale_only_quantization_gb300.autograd import QADRMSNorm
    _build()
    T, d = 50, 272
    bf = torch.bfloat16
    x, res, dy, dr = (torch.randn((2, T // 2, d), device="cuda").to(bf) for _ in range(4))
    n = QADRMSNorm(1 + 0.1 * torch.randn(d, device="cuda"), act=act, trained=True)
    x.requires_grad_(True)
    res.requires_grad_(True)
    out = n(x, res)
    torch.autograd.backward([out[0], out[1]], [dy, dr])
    r, y = torch.empty((T, d), dtype=bf, device="cuda"), torch.empty((T, d), dtype=bf, device="cuda")
    rstd = torch.empty(T, device="cuda")
    Q.qad_rmsnorm_fwd(x.detach(), res.detach(), n.weight.detach(), 1e-6, 0, r, y, None, None, None, rstd, T, d, d, d)
    dx, dg = torch.empty_like(r), torch.empty(d, device="cuda")
    ws = torch.empty(Q.qad_rmsnorm_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    Q.qad_rmsnorm_bwd(dy, dr, r, n.weight.detach(), rstd, dx, dg, T, d, d, ws)
    assert torch.equal(out[0].view(T, d), y) and torch.equal(out[1].view(T, d), r)
    assert torch.equal(x.grad.view(T, d), dx) and torch.equal(res.grad.view(T, d), dx)
    assert torch.equal(n.weight.grad, dg.to(bf))
    if act:
        assert out[2].shape == x.shape and out[3].shape == (T,)


@pytest.mark.gpu
def test_head_loss_against_torch():
    """total, its parts and dh against fp64 torch autograd of the same definition; dh within its bf16 roundings (of the
    softmax, of each part's sum and of their total: 4 x 2^-8 of the terms' size)."""
    from scale_only_quantization_gb300.autograd import QADHeadLoss
    _build()
    N, d, V, K = 60, 128, 900, 16
    bf = torch.bfloat16
    w = (torch.randn((V, d), device="cuda") * d ** -0.5).to(bf)
    h = torch.randn((N, d), device="cuda").to(bf).requires_grad_(True)
    target = torch.randint(0, V, (N,), device="cuda")
    target[:7] = -1
    idx = torch.stack([torch.randperm(V, device="cuda")[:K] for _ in range(N)]).to(torch.int32)
    t = torch.randn((N, K), device="cuda") * 2
    loss = QADHeadLoss(w, lm_weight=0.3, distill_weight=0.7, tau=2.0)
    total, lm, kd = loss(h, target, idx, t)
    (3.0 * total).backward()
    h64 = h.detach().double().requires_grad_(True)
    z = h64 @ w.double().T
    live = target >= 0
    lm64 = torch.nn.functional.cross_entropy(z[live], target[live])
    lq = torch.log_softmax(z.gather(1, idx.long()) / 2, 1)
    lp = torch.log_softmax(t.double() / 2, 1)
    kd64 = (lp.exp() * (lp - lq)).sum(1).mean()
    tot64 = 0.3 * lm64 + 0.7 * kd64
    (3.0 * tot64).backward()
    for a, b in ((lm, lm64), (kd, kd64), (total, tot64)):
        assert abs(float((a - b).detach())) < 1e-5
    size = (3 * (0.3 / 53 + 0.7 / N)) * w.double().abs().amax(0)
    assert torch.all((h.grad.double() - h64.grad).abs() <= 4 * 2.0 ** -8 * (h64.grad.abs() + size))
    # either part alone
    only = QADHeadLoss(w)(h.detach(), target)
    assert only[2] is None and abs(float((only[1] - lm64).detach())) < 1e-5
    only = QADHeadLoss(w, tau=2.0)(h.detach(), None, idx, t)
    assert only[1] is None and abs(float((only[2] - kd64).detach())) < 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [Q.QAD_FMT_NVFP4, Q.QAD_FMT_INT4_G128])
def test_example_trains_the_scales(fmt):
    """The divergence from the unquantized model falls when only the scales move (4-bit weights: 8-bit ones start
    within the noise of a few tokens routed otherwise)."""
    _build()
    import qad_step
    hist = qad_step.train(fmt, steps=12, tokens=256, log=None)
    kd = [h[2] for h in hist]
    assert all(x == x and x < 1e3 for h in hist for x in h)
    assert kd[0] > 0 and min(kd[-3:]) < 0.95 * kd[0]


@pytest.mark.gpu
def test_norm_and_losses_in_a_cuda_graph():
    """The calls allocate nothing and read nothing back: a captured step replays with the same results."""
    _build()
    N, d, V, K = 200, 256, 3000, 16
    bf = torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w, gamma = rand(N, d).to(bf), (rand(V, d) * d ** -0.5).to(bf), (1 + 0.1 * rand(d)).to(bf)
    target = torch.randint(0, V, (N,), generator=g, device="cuda").to(torch.int32)
    idx = torch.randint(0, V, (N, K), generator=g, device="cuda").to(torch.int32)
    t = rand(N, K)
    y, dh = torch.empty_like(x), torch.empty_like(x)
    ce, lse, kd = (torch.empty(N, device="cuda") for _ in range(3))
    ws = torch.empty(Q.qad_linear_ce_workspace_bytes(N, d, V, 1, 0), dtype=torch.uint8, device="cuda")

    def step():
        Q.qad_rmsnorm_fwd(x, None, gamma, 1e-6, 0, None, y, None, None, None, None, N, d, d, d)
        Q.qad_linear_ce_fwd_bwd(y, d, w, d, target, None, ce, lse, dh, None, 0, N, d, V, ws)
        Q.qad_distill_topk_fwd_bwd(y, d, w, d, idx, t, None, 1.0, None, kd, dh, 1, N, d, V, K)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    ref = [v.clone() for v in (y, ce, lse, kd, dh)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in (y, ce, lse, kd, dh):
        v.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    for v, r in zip((y, ce, lse, kd, dh), ref):
        assert torch.equal(v, r)


@pytest.mark.gpu
def test_head_loss_of_no_rows():
    from scale_only_quantization_gb300.autograd import QADHeadLoss
    _build()
    head = QADHeadLoss(torch.randn((100, 64), device="cuda"))
    h = torch.empty((0, 64), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    total, lm, _ = head(h, torch.empty(0, dtype=torch.int64, device="cuda"))
    total.backward()
    assert float(total.detach()) == 0 and float(lm.detach()) == 0 and h.grad.shape == (0, 64)


@pytest.mark.gpu
def test_head_loss_reports_tokens_past_the_vocabulary():
    """A target or teacher token that is not in the vocabulary: its row carries nothing, the mean is over the others, and
    the module's error word says so until it is read."""
    from scale_only_quantization_gb300.autograd import QADHeadLoss
    _build()
    N, d, V, K = 40, 64, 300, 8
    w = (torch.randn((V, d), device="cuda") * d ** -0.5).to(torch.bfloat16)
    h = torch.randn((N, d), device="cuda").to(torch.bfloat16).requires_grad_(True)
    target = torch.randint(0, V, (N,), device="cuda")
    idx = torch.randint(0, V, (N, K), device="cuda", dtype=torch.int32)
    t = torch.randn((N, K), device="cuda")
    head = QADHeadLoss(w)
    for want in (0, Q.QAD_DEV_BAD_INDEX, 0):
        tg, ix = target.clone(), idx.clone()
        if want:
            tg[3], tg[9] = V, 2 ** 30
        total, lm, kd = head(h, tg, ix, t)
        assert head.device_error() == want
        z = h.detach().double() @ w.double().T
        live = tg < V
        ref = torch.nn.functional.cross_entropy(z[live], tg[live])
        assert abs(float(lm.detach()) - float(ref)) < 1e-5
        if want:
            total.backward()
            assert torch.isfinite(h.grad.float()).all()
    ix = idx.clone()
    ix[5, 2] = V
    head(h, None, ix, t)
    with torch.no_grad():
        head(h, target, idx, t)          # a clean call does not clear what an earlier one reported
    assert head.device_error() == Q.QAD_DEV_BAD_INDEX
    assert head.device_error() == 0      # read and cleared


def test_views_off_a_16_byte_boundary_are_copied():
    """contiguous() returns a contiguous view as it is, wherever it starts."""
    from scale_only_quantization_gb300.autograd import _packed, _rows
    ids = torch.arange(41, dtype=torch.int32)
    for v in (ids[1:], torch.arange(9.0)[3:], torch.arange(16, dtype=torch.uint8)[5:].view(torch.uint8)):
        p = _packed(v)
        assert p.data_ptr() % 16 == 0 and p.is_contiguous() and torch.equal(p, v)
    assert _packed(ids).data_ptr() == ids.data_ptr()             # an aligned one is read in place
    flat = torch.arange(6 * 64 + 8, dtype=torch.float32).to(torch.bfloat16)
    x = flat[1: 1 + 6 * 64].view(6, 64)
    r = _rows(x, 64, "x")
    assert x.is_contiguous() and x.data_ptr() % 16 and r.data_ptr() % 16 == 0 and torch.equal(r, x)


@pytest.mark.gpu
def test_shifted_targets_and_other_misaligned_views():
    """target = ids[1:] in int32, and every other input as a view that starts off a 16-byte boundary."""
    from scale_only_quantization_gb300.autograd import QADHeadLoss, QADRMSNorm
    _build()
    N, d, V, K = 33, 64, 300, 8
    bf = torch.bfloat16

    def off(t):  # the same values, one element into a buffer of their own
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:] = t.reshape(-1)
        return b[1:].view(t.shape)

    w = (torch.randn((V, d), device="cuda") * d ** -0.5).to(bf)
    h = torch.randn((N, d), device="cuda").to(bf)
    ids = torch.randint(0, V, (N + 1,), device="cuda", dtype=torch.int32)
    idx = torch.randint(0, V, (N, K), device="cuda", dtype=torch.int32)
    t, mix = torch.randn((N, K), device="cuda"), torch.rand(N, device="cuda")
    head = QADHeadLoss(w)
    a, b = h.clone().requires_grad_(True), off(h).requires_grad_(True)
    ta = head(a, ids[1:].clone(), idx, t, mix)
    tb = QADHeadLoss(off(w))(b, ids[1:], off(idx), off(t), off(mix))
    ta[0].backward()
    tb[0].backward()
    assert all(torch.equal(x, y) for x, y in zip(ta, tb)) and torch.equal(a.grad, b.grad)
    norm = QADRMSNorm(1 + 0.1 * torch.randn(d, device="cuda"), trained=True)
    norm2 = QADRMSNorm(off(norm.weight.detach()), trained=True)
    a, b, g = h.clone().requires_grad_(True), off(h).requires_grad_(True), torch.randn((N, d), device="cuda").to(bf)
    ya, yb = norm(a, h), norm2(b, off(h))
    torch.autograd.backward([ya[0], ya[1]], [g, h])
    torch.autograd.backward([yb[0], yb[1]], [off(g), off(h)])
    assert torch.equal(ya[0], yb[0]) and torch.equal(a.grad, b.grad) and torch.equal(norm.weight.grad, norm2.weight.grad)


@pytest.mark.gpu
def test_distillation_mean_is_over_the_rows_that_keep_a_token():
    """Padding rows (no teacher token) neither shrink the distillation loss nor its gradient."""
    from scale_only_quantization_gb300.autograd import QADHeadLoss
    _build()
    N, d, V, K = 30, 64, 300, 8
    w = (torch.randn((V, d), device="cuda") * d ** -0.5).to(torch.bfloat16)
    h = torch.randn((N, d), device="cuda").to(torch.bfloat16)
    idx = torch.randint(0, V, (N, K), device="cuda", dtype=torch.int32)
    t = torch.randn((N, K), device="cuda") * 2
    idx[20:25] = -1
    t[25:28] = -float("inf")
    idx[28:, :] = V          # not in the vocabulary: not kept either
    head = QADHeadLoss(w, distill_weight=0.5)
    a, b = h.clone().requires_grad_(True), h[:20].clone().requires_grad_(True)
    ta, tb = head(a, None, idx, t), head(b, None, idx[:20], t[:20])
    ta[0].backward()
    tb[0].backward()
    assert abs(float(ta[2] - tb[2])) <= 1e-6 * float(tb[2]) and abs(float((ta[0] - tb[0]).detach())) <= 1e-6
    assert torch.all(a.grad[20:] == 0)
    assert torch.all((a.grad[:20].double() - b.grad.double()).abs() <= 2.0 ** -7 * b.grad.double().abs())
    none = head(h, None, torch.full_like(idx, -1), t)
    assert float(none[0]) == 0 and float(none[2]) == 0
    other = head(h.view(5, 6, d), None, idx.view(5, 6, K), t)       # the same rows in other shapes
    assert torch.equal(other[0], ta[0].detach())


@pytest.mark.gpu
def test_upstream_gradient_is_applied_in_fp32():
    """(loss / 3).backward(): the stored gradient times 1/3 in fp32, rounded to bf16 once."""
    from scale_only_quantization_gb300.autograd import QADHeadLoss
    _build()
    N, d, V = 50, 128, 500
    w = (torch.randn((V, d), device="cuda") * d ** -0.5).to(torch.bfloat16)
    h = torch.randn((N, d), device="cuda").to(torch.bfloat16)
    target = torch.randint(0, V, (N,), device="cuda")
    head = QADHeadLoss(w)
    a, b = h.clone().requires_grad_(True), h.clone().requires_grad_(True)
    head(a, target)[0].backward()
    (head(b, target)[0] / 3).backward()
    assert torch.equal(b.grad, (a.grad.float() * (torch.ones((), device="cuda") / 3)).to(torch.bfloat16))
    assert b.grad.dtype == torch.bfloat16


@pytest.mark.gpu
def test_second_derivatives_are_refused():
    """The gradients are kernels' outputs: asking to differentiate them again raises instead of returning a gradient
    that does not depend on the hidden states."""
    from scale_only_quantization_gb300.autograd import QADHeadLoss, QADRMSNorm
    _build()
    d, V = 64, 100
    h = torch.randn((5, d), device="cuda").to(torch.bfloat16).requires_grad_(True)
    w = torch.randn((V, d), device="cuda") * d ** -0.5
    target = torch.randint(0, V, (5,), device="cuda")
    for loss in (QADHeadLoss(w)(h, target)[0].square(), QADRMSNorm(torch.ones(d, device="cuda"))(h)[0].float().square().sum()):
        (g,) = torch.autograd.grad(loss, h, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.float().sum(), h)


@pytest.mark.gpu
def test_norm_with_one_output_unused(monkeypatch):
    """A gradient that does not arrive is not made up as zeros and read: with r unused the call gets none, with y unused
    dx is r's gradient as it came."""
    from scale_only_quantization_gb300 import autograd as A
    _build()
    calls = []
    bwd = A.qad_rmsnorm_bwd
    monkeypatch.setattr(A, "qad_rmsnorm_bwd", lambda *a, **k: (calls.append(a), bwd(*a, **k)))
    d = 272
    x, res, g = (torch.randn((2, 20, d), device="cuda").to(torch.bfloat16) for _ in range(3))
    norm = A.QADRMSNorm(1 + 0.1 * torch.randn(d, device="cuda"), trained=True)

    def grads(which):
        a, b = x.clone().requires_grad_(True), res.clone().requires_grad_(True)
        norm.weight.grad = None
        out = norm(a, b)
        if which == "both":
            torch.autograd.backward([out[0], out[1]], [g, torch.zeros_like(g)])
        else:
            out[which].backward(g)
        return a.grad, b.grad, norm.weight.grad

    only_y, both, only_r = grads(0), grads("both"), grads(1)
    assert all(torch.equal(p, q) for p, q in zip(only_y, both))
    assert calls[0][1] is None and calls[1][1] is not None and len(calls) == 2
    assert torch.equal(only_r[0], g) and torch.equal(only_r[1], g) and torch.all(only_r[2] == 0)
    # the residual may come in another view of the same rows
    a, b = x.clone().requires_grad_(True), res.reshape(40, d).clone().requires_grad_(True)
    norm(a, b)[0].backward(g)
    assert torch.equal(a.grad, only_y[0]) and torch.equal(b.grad.view_as(res), only_y[1])


@pytest.mark.gpu
def test_no_gradient_asked_none_computed(monkeypatch):
    """Under no_grad, or with hidden states that need none, the head loss makes the forward calls; the numbers are the
    same bits."""
    from scale_only_quantization_gb300 import autograd as A
    _build()
    N, d, V, K = 40, 64, 300, 8
    w = (torch.randn((V, d), device="cuda") * d ** -0.5).to(torch.bfloat16)
    h = torch.randn((N, d), device="cuda").to(torch.bfloat16)
    target = torch.randint(0, V, (N,), device="cuda")
    target[:3] = -1
    idx = torch.randint(0, V, (N, K), device="cuda", dtype=torch.int32)
    t = torch.randn((N, K), device="cuda")
    head = A.QADHeadLoss(w, 0.3, 0.7)
    want = [v.detach() for v in head(h.clone().requires_grad_(True), target, idx, t)]

    def refuse(*a, **k):
        raise AssertionError("a gradient was computed")
    monkeypatch.setattr(A, "qad_linear_ce_fwd_bwd", refuse)
    monkeypatch.setattr(A, "qad_distill_topk_fwd_bwd", refuse)
    got = head(h, target, idx, t)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.no_grad():
        got = head(h.clone().requires_grad_(True), target, idx, t)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not got[0].requires_grad


def test_the_error_word_is_the_rank_s_own():
    """Data parallelism broadcasts a module's buffers from rank 0 before each forward: the error word is none."""
    from scale_only_quantization_gb300.autograd import QADHeadLoss
    h = QADHeadLoss(torch.randn(10, 64))
    assert [n for n, _ in h.named_buffers()] == ["w"] and list(h.state_dict()) == ["w"]
    assert h.device_error() == 0


def test_wide_tokens_do_not_wrap_into_the_vocabulary():
    from scale_only_quantization_gb300.autograd import _tokens
    t = torch.tensor([0, 99, 100, -1, -100, 2 ** 32 + 5, -(2 ** 32) + 5, 2 ** 62])
    assert _tokens(t, 100).tolist() == [0, 99, 100, -1, -1, 100, -1, 100] and _tokens(t, 100).dtype == torch.int32
    t = t[:5].to(torch.int32)
    assert _tokens(t, 100) is t


@pytest.mark.gpu
def test_head_loss_of_wide_tokens():
    """A 64-bit token whose low word names a word of the vocabulary is past it all the same."""
    from scale_only_quantization_gb300.autograd import QADHeadLoss
    _build()
    N, d, V, K = 20, 64, 300, 8
    h = torch.randn((N, d), device="cuda").to(torch.bfloat16)
    target = torch.randint(0, V, (N,), device="cuda")
    idx = torch.randint(0, V, (N, K), device="cuda")
    t = torch.randn((N, K), device="cuda")
    head = QADHeadLoss(torch.randn((V, d), device="cuda") * d ** -0.5)
    a = [target.clone(), idx.clone()]
    a[0][4], a[1][6, 2] = -1, -1
    want = head(h, a[0], a[1], t)
    assert head.device_error() == 0
    a[0][4], a[1][6, 2] = 2 ** 32 + 5, 2 ** 32 + 5
    got = head(h, a[0], a[1], t)
    assert all(torch.equal(x, y) for x, y in zip(want, got)) and head.device_error() == Q.QAD_DEV_BAD_INDEX
