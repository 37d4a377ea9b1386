"""Top-k distillation (qad_distill_topk_*) against its definition in 64 bits.

Bounds (u = 2^-24): a student logit is a chain of at most d fp32 additions, |dz| <= d u sum |h w| =: e.  The loss moves
by at most 2 b e (KL: sum |q - p| <= 2) or 2 b e max |x| (RKL), plus fp32 roundings of its K positive terms.  dz moves
by at most 4 b e (1 + max |x|) and a few u, times b g sum |w|; dh is rounded to bf16 once (2^-8).
"""
import pytest
import torch

import scale_only_quantization_gb300 as Q

U = 2.0 ** -24


def _lib():
    from scale_only_quantization_gb300 import build
    build.build()
    return Q.lib()


def test_refusals_before_any_launch():
    L = _lib()
    P = 1 << 20
    names = ("h", "ldh", "w", "ldw", "idx", "t", "mix", "b", "g", "loss", "dh", "acc", "N", "d", "V", "K", "err", "st")
    base = dict(h=P, ldh=64, w=P, ldw=64, idx=P, t=P, mix=None, b=1.0, g=None, loss=P, dh=P, acc=0, N=4, d=64, V=100, K=8,
                err=None, st=None)
    both = lambda **k: L.qad_distill_topk_fwd_bwd(*[{**base, **k}[n] for n in names])  # noqa: E731
    fwd = lambda **k: L.qad_distill_topk_fwd(*[{**base, **k}[n] for n in names if n not in ("g", "dh", "acc")])  # noqa: E731
    bad, uns = Q.QAD_ERR_INVALID_ARG, Q.QAD_ERR_UNSUPPORTED
    for f in (both, fwd):
        assert f(N=0, h=None, w=None) == Q.QAD_OK
        assert f(N=-1) == bad and f(V=0) == bad and f(K=0) == bad and f(d=0) == bad
        assert f(b=0.0) == bad and f(b=-1.0) == bad and f(b=float("inf")) == bad and f(b=float("nan")) == bad
        assert f(d=72, ldh=72, ldw=72) == uns and f(K=1025) == uns and f(d=16400, ldh=16400, ldw=16400) == uns
        assert f(ldh=56) == bad and f(ldw=68) == bad
        for p in ("h", "w", "idx", "t", "loss"):
            assert f(**{p: None}) == bad and f(**{p: P + 2}) == bad
        assert f(mix=P + 2) == bad and f(err=P + 2) == bad
    assert both(dh=None) == bad and both(g=P + 2) == bad


def make(N, d, V, K, seed=0, mixed=False, ldh=None, ldw=None, near=1.0, size=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    h, w = (size * rand(N, ldh or d)).to(bf), (rand(V, ldw or d) / d ** 0.5).to(bf)
    idx = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(N)]).to(torch.int32)
    z = (w[idx.long(), :d].double() @ h[:, :d].double()[:, :, None])[:, :, 0]
    t = (z + near * rand(N, K)).float()
    mix = torch.rand(N, generator=g, device="cuda") if mixed else None
    gr = torch.rand(N, generator=g, device="cuda") + 0.5
    return dict(h=h, w=w, idx=idx, t=t, mix=mix, g=gr, N=N, d=d, V=V, K=K)


def run(c, beta=1.0, grad=True, accumulate=None, err=None):
    loss = torch.full((c["N"],), float("nan"), device="cuda")
    dh = torch.full((c["N"], c["d"]), float("nan"), dtype=torch.bfloat16, device="cuda") if accumulate is None else accumulate
    a = (c["h"], c["h"].stride(0), c["w"], c["w"].stride(0), c["idx"], c["t"], c["mix"], beta)
    z = (c["N"], c["d"], c["V"], c["K"], err)
    if grad:
        Q.qad_distill_topk_fwd_bwd(*a, c["g"], loss, dh, int(accumulate is not None), *z)
    else:
        Q.qad_distill_topk_fwd(*a, loss, *z)
    torch.cuda.synchronize()
    return loss, dh


def exact(c, beta=1.0, h=None):
    d, V = c["d"], c["V"]
    idx, t = c["idx"].long(), c["t"].double() * beta
    keep = (idx >= 0) & (idx < V) & (t > -float("inf"))
    wk = c["w"][idx.clamp(0, V - 1), :d].double() * keep[:, :, None]
    h = c["h"][:, :d].double() if h is None else h
    z = (wk @ h[:, :, None])[:, :, 0] * beta
    ninf = torch.full_like(z, -1e300)
    lq = torch.log_softmax(torch.where(keep, z, ninf), 1)
    lp = torch.log_softmax(torch.where(keep, t, ninf), 1)
    zero = torch.zeros_like(z)
    q, p = torch.where(keep, lq.exp(), zero), torch.where(keep, lp.exp(), zero)
    x = torch.where(keep, lq - lp, zero)
    rkl = (q * x).sum(1)
    m = torch.zeros_like(rkl) if c["mix"] is None else c["mix"].double()
    loss = (1 - m) * -(p * x).sum(1) + m * rkl
    dz = beta * c["g"].double()[:, None] * ((1 - m)[:, None] * (q - p) + m[:, None] * q * (x - rkl[:, None]))
    e = d * U * (wk.abs() @ h.abs()[:, :, None])[:, :, 0].amax(1) * beta
    xm = 1 + x.abs().amax(1)
    tol_loss = 4 * e * xm + 1e-6 + 2e-6 * xm * loss.abs()
    tol_dh = (beta * c["g"].double() * (8 * e * xm + 1e-6 * xm))[:, None] * wk.abs().sum(1)
    return loss, (dz[:, None, :] @ wk)[:, 0], tol_loss, tol_dh


def check(c, beta=1.0):
    loss, dh = run(c, beta)
    l64, d64, tl, td = exact(c, beta)
    assert torch.all((loss.double() - l64).abs() <= tl), float(((loss.double() - l64).abs() / tl).max())
    assert torch.all((dh.double() - d64).abs() <= 2.0 ** -8 * d64.abs() + td)
    assert torch.equal(run(c, beta, grad=False)[0], loss)
    return loss, dh


@pytest.mark.gpu
@pytest.mark.parametrize("beta", [1.0, 0.5])
@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("N, d, V, K", [(1, 16, 5, 1), (1, 256, 1000, 5), (3, 272, 777, 33), (65, 2048, 4096, 64), (9, 2880, 999, 100),
                                        (2, 4096, 2000, 128), (2, 8192, 300, 300), (4, 64, 2000, 1024), (1, 16384, 64, 17)])
def test_against_64_bits(N, d, V, K, mixed, beta):
    _lib()
    check(make(N, d, V, K, seed=N + d + K, mixed=mixed), beta)


@pytest.mark.gpu
@pytest.mark.parametrize("near, size", [(0.01, 1.0), (3.0, 1.0), (30.0, 1.0), (1.0, 40.0), (0.0, 1.0)])
def test_near_far_and_equal_distributions(near, size):
    """From a teacher a hundredth of a nat away to one on other tokens altogether."""
    _lib()
    check(make(33, 256, 500, 16, seed=3, mixed=True, near=near, size=size))


@pytest.mark.gpu
def test_strided_rows_of_hidden_states_and_head():
    _lib()
    check(make(21, 272, 300, 20, seed=4, mixed=True, ldh=560, ldw=296))


@pytest.mark.gpu
def test_slots_that_do_not_count():
    """Empty slots (idx < 0, t = -inf), a row that keeps none, one that keeps one, and indices past the vocabulary,
    which are reported; NaN in a slot that does not count changes nothing."""
    _lib()
    c = make(8, 256, 500, 12, seed=6, mixed=True)
    c["idx"][0, 3:] = -1
    c["t"][1, 5] = -float("inf")
    c["idx"][2, :] = -1
    c["t"][3, :] = -float("inf")
    c["idx"][4, 1:] = -5
    c["t"][0, 4] = float("nan")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, dh = run(c, err=err)
    assert Q.qad_check_device_error(err) == 0
    e = {**c, "t": torch.where(torch.isnan(c["t"]), 0.0, c["t"])}
    l64, d64, tl, td = exact(e)
    empty = torch.tensor([False, False, True, True, False, False, False, False], device="cuda")
    assert torch.all(loss[empty] == 0) and torch.all(dh[empty] == 0)
    assert abs(float(loss[4])) <= 1e-6 and torch.all(dh[4].abs() <= 1e-5)
    live = ~empty
    assert torch.all((loss.double() - l64).abs()[live] <= tl[live])
    assert torch.all((dh.double() - d64).abs()[live] <= (2.0 ** -8 * d64.abs() + td)[live])
    c["idx"][5, 2] = 500
    c["idx"][6, 0] = 2 ** 31 - 1
    loss, dh = run(c, err=err)
    assert Q.qad_check_device_error(err) == Q.QAD_DEV_BAD_INDEX
    l64, d64, tl, td = exact({**c, "t": e["t"]})
    assert torch.all((loss.double() - l64).abs()[live] <= tl[live])


@pytest.mark.gpu
def test_nan_stays_in_its_row():
    _lib()
    c = make(6, 256, 400, 16, seed=8)
    loss, dh = run(c)
    c["h"][2, 5] = float("nan")
    c["t"][4, 1] = float("nan")
    l2, d2 = run(c)
    for i in (0, 1, 3, 5):
        assert torch.equal(loss[i], l2[i]) and torch.equal(dh[i], d2[i])
    assert torch.isnan(l2[2]) and torch.isnan(l2[4])


@pytest.mark.gpu
def test_accumulates_onto_a_gradient():
    """accumulate adds in fp32 and rounds once."""
    _lib()
    c = make(17, 256, 300, 16, seed=9)
    _, d64, _, td = exact(c)
    base = torch.randn((17, 256), device="cuda").to(torch.bfloat16)
    _, dh = run(c, accumulate=base.clone())
    ref = base.double() + d64
    assert torch.all((dh.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + td + 2 * U * (base.double().abs() + d64.abs()))


@pytest.mark.gpu
def test_gradient_against_differences():
    """(L(h + s v) - L(h - s v)) / 2s of the 64-bit loss against <dh, v>, up to dh's bf16 rounding."""
    _lib()
    c = make(5, 256, 300, 24, seed=10, mixed=True)
    _, dh = run(c, 0.5)
    h = c["h"].double()
    s = 1e-5
    for seed in range(3):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        v = torch.randn(h.shape, generator=g, device="cuda", dtype=torch.float64)
        num = c["g"].double() * (exact(c, 0.5, h + s * v)[0] - exact(c, 0.5, h - s * v)[0]) / (2 * s)
        assert torch.all((num - (dh.double() * v).sum(1)).abs() <= 2.0 ** -8 * (dh.double() * v).abs().sum(1) + 1e-5)


@pytest.mark.gpu
def test_repeatable_on_another_stream():
    _lib()
    c = make(70, 512, 900, 40, seed=12)
    a = run(c)
    with torch.cuda.stream(torch.cuda.Stream()):
        b = run(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("N, d, V, K", [(1, 2048, 500, 64), (152, 512, 600, 24), (153, 512, 600, 24), (2000, 64, 200, 9), (700, 1024, 900, 40)])
def test_row_counts_below_and_above_the_sms(N, d, V, K, mixed):
    _lib()
    check(make(N, d, V, K, seed=N, mixed=mixed))


@pytest.mark.gpu
def test_a_later_logit_far_above_the_first():
    """The sums' reference is the first batch's largest logit; one 100 nats above it replaces it."""
    _lib()
    c = make(30, 256, 400, 24, seed=21, mixed=True)
    for i in range(30):  # make slot 5 + i % 19 the row's own direction, so that its logit is the largest by far
        c["w"][int(c["idx"][i, 5 + i % 19])] = c["h"][i] * 0.5
    check(c)


@pytest.mark.gpu
def test_nan_in_a_head_row_reaches_the_rows_that_name_it_only():
    _lib()
    c = make(12, 256, 400, 16, seed=22)
    c["idx"] = torch.stack([torch.arange(16, device="cuda", dtype=torch.int32) + 16 * (i % 6) for i in range(12)])
    c["idx"][3, 4] = -1
    loss, dh = run(c)
    c["w"][17] = float("nan")            # named by rows 1 and 7
    c["w"][16 * 3 + 4] = float("nan")    # row 9's, and in row 3 a slot that does not count
    c["w"][399] = float("inf")           # nobody's
    l2, d2 = run(c)
    for i in range(12):
        if i in (1, 7, 9):
            assert torch.isnan(l2[i])
        else:
            assert torch.equal(loss[i], l2[i]) and torch.equal(dh[i], d2[i])


@pytest.mark.gpu
@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("N, d, K, row", [(400, 2048, 20, 250), (200, 4096, 9, 0), (1500, 256, 40, 1499), (40, 8192, 5, 3)])
def test_a_copy_that_never_comes_is_reported(N, d, K, row, mixed):
    """One token row's copies left out: the wait gives up (0.5 ms here), the rows of its block are NaN in loss and dh, with
    or without an error word to say so, other rows have their bits, and the next call is clean."""
    _lib()
    c = make(N, d, 300, K, seed=40, mixed=mixed)
    loss, dh = run(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    Q.qad_debug_stuck_copy(row, 1_000_000)
    try:
        got = [run(c, err=err), run(c)]
    finally:
        Q.qad_debug_stuck_copy(-1)
    assert Q.qad_check_device_error(err) == Q.QAD_DEV_TIMEOUT
    for l2, d2 in got:
        gone = torch.isnan(l2)
        assert gone[row] and torch.equal(gone, torch.isnan(d2).all(1)) and torch.equal(gone, torch.isnan(d2).any(1))
        assert int(gone.sum()) <= 8 * -(-N // 152) + 8
        assert torch.equal(l2[~gone], loss[~gone]) and torch.equal(d2[~gone], dh[~gone])
    err.zero_()
    l2, d2 = run(c, err=err)
    assert Q.qad_check_device_error(err) == 0 and torch.equal(l2, loss) and torch.equal(d2, dh)


@pytest.mark.gpu
@pytest.mark.parametrize("beta", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("low", [-1e4, -1e30, torch.finfo(torch.float32).min])
def test_teacher_logits_of_the_lowest_value(low, beta):
    """A finite teacher logit counts however low it is and whatever the temperature: p = 0 there, the student's
    probability is taken over it.  With the forward divergence alone, and in rows of a mix whose share of the reverse
    one is 0, loss and gradient stay finite and are those of the definition."""
    _lib()
    c = make(24, 256, 400, 12, seed=31, mixed=True)
    c["t"][::2, 7:] = low
    c["t"][1::4, :3] = low
    for mix in (None, torch.zeros(24, device="cuda")):
        e = {**c, "mix": mix}
        loss, dh = run(e, beta)
        l64, d64, _, _ = exact(e, beta)
        assert torch.isfinite(loss).all() and torch.isfinite(dh.float()).all()
        # a logit is 4 packed products, a sum and 5 steps of a reduction: 10 roundings of at most sum |h w|
        w = c["w"][c["idx"].long()].double().abs()
        err = 10 * U * (w @ c["h"].double().abs()[:, :, None])[:, :, 0].amax(1)
        assert torch.all((loss.double() - l64).abs() <= 2 * beta * err + 4e-6 * (1 + l64.abs()))
        assert torch.all((dh.double() - d64).norm(dim=1) <= 1e-2 * d64.norm(dim=1))  # bf16: 2^-8 of an element
        assert torch.equal(run(e, beta, grad=False)[0], loss)


def bounds(c, beta):
    """exact()'s loss and dh with each slot's error weighted by its own probability.  A logit is at most 16 packed products,
    a sum, 5 steps of a reduction and 16 warps' sums: 38 roundings of sum |h w|, 40 here (e).  x moves by 2 b e and the
    roundings of z, t and their differences (dx); KL's derivative with respect to x_k is q - p, RKL's q (x - RKL), and
    terms with |x| >= 1/2 are differences of probabilities.  dz's factors: exp by the intrinsic (2 ulp and 1.2 ulp per
    unit of its argument), K fp32 additions of the three sums, whose own references are the first slot's x."""
    d, V, K = c["d"], c["V"], c["K"]
    idx, t = c["idx"].long(), c["t"].double() * beta
    keep = (idx >= 0) & (idx < V) & (t > -float("inf"))
    wk = c["w"][idx.clamp(0, V - 1), :d].double() * keep[:, :, None]
    h = c["h"][:, :d].double()
    z = (wk @ h[:, :, None])[:, :, 0] * beta
    e = 40 * U * (wk.abs() @ h.abs()[:, :, None])[:, :, 0].amax(1, keepdim=True) * beta
    ninf = torch.full_like(z, -1e300)
    lq = torch.log_softmax(torch.where(keep, z, ninf), 1)
    lp = torch.log_softmax(torch.where(keep, t, ninf), 1)
    zero = torch.zeros_like(z)
    q, p, x = (torch.where(keep, v, zero) for v in (lq.exp(), lp.exp(), lq - lp))
    rkl = (q * x).sum(1, keepdim=True)
    m = torch.zeros_like(rkl) if c["mix"] is None else c["mix"].double()[:, None]
    big = lambda v: torch.where(keep, v.abs(), zero).amax(1, keepdim=True)  # noqa: E731
    dx = 2 * e + 16 * U * (big(z) + big(t) + big(x) + 1)
    kl = -(p * x).sum(1, keepdim=True)
    loss = (1 - m) * kl + m * rkl
    tol_loss = (1 - m) * ((q - p).abs() * dx + (p + q) * dx * dx) + m * q * ((x - rkl).abs() * dx + dx * dx * (1 + x.abs()))
    tol_loss = tol_loss + torch.where(x.abs() > 0.4, (p + q) * (1 + x.abs()) * (dx + 2e-6), zero)
    tol_loss = tol_loss.sum(1) + 2e-5 * loss[:, 0].abs() + 1e-12
    first = x.gather(1, keep.to(torch.int8).argmax(1, keepdim=True))
    eps = 2 * e + 4e-6 + 2e-7 * (z - torch.where(keep, z, ninf).amax(1, keepdim=True)).abs() + (K + 10) * U
    gb = beta * c["g"].double()[:, None]
    dz = gb * ((1 - m) * (q - p) + m * q * (x - rkl))
    tol_dz = gb * ((1 - m) * (q * eps + p * (4e-6 + K * U)) + m * q * (eps * ((x - first).abs() + (rkl - first).abs()) + 2 * dx))
    dh, slack = (dz[:, None, :] @ wk)[:, 0], (tol_dz[:, None, :] @ wk.abs())[:, 0]
    return loss[:, 0], dh, tol_loss, slack


def check_closely(c, beta=1.0, gradient=True):
    """Every row's loss and gradient within bounds() (bf16: 2^-8 of an element more), and bounds that would reject a
    missing or a turned gradient in every row."""
    loss, dh = run(c, beta)
    l64, d64, tl, slack = bounds(c, beta)
    tol = 2.0 ** -8 * d64.abs() + slack
    if gradient:
        assert torch.all((d64.abs() > tol).any(1)) and torch.all(slack.norm(dim=1) < 0.5 * d64.norm(dim=1))
    assert torch.all((loss.double() - l64).abs() <= tl), float(((loss.double() - l64).abs() / tl).max())
    assert torch.all((dh.double() - d64).abs() <= tol), float(((dh.double() - d64).abs() / tol).max())
    assert torch.all((dh.double() - d64).norm(dim=1) <= 2.0 ** -8 * d64.norm(dim=1) + slack.norm(dim=1))
    assert torch.equal(run(c, beta, grad=False)[0], loss)


@pytest.mark.gpu
@pytest.mark.parametrize("beta", [1.0, 0.5])
@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("N, d, V, K", [(3, 272, 777, 33), (65, 2048, 4096, 64), (9, 2880, 999, 100), (2, 4096, 2000, 128), (2, 8192, 300, 300),
                                        (4, 64, 2000, 1024), (2, 16384, 64, 17)])
def test_closely_against_64_bits(N, d, V, K, mixed, beta):
    _lib()
    check_closely(make(N, d, V, K, seed=N + d + K, mixed=mixed), beta)


@pytest.mark.gpu
@pytest.mark.parametrize("near, size", [(0.01, 1.0), (0.1, 1.0), (3.0, 1.0), (30.0, 1.0), (1.0, 40.0), (0.0, 1.0)])
def test_near_far_and_equal_distributions_closely(near, size):
    """The loss keeps its relative precision down to a teacher a hundredth of a nat away; where the distributions are
    equal, or both one token's, there is no gradient to hold apart from its bounds."""
    _lib()
    check_closely(make(33, 256, 500, 16, seed=3, mixed=True, near=near, size=size), gradient=near > 0 and size == 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("mixed", [False, True])
def test_a_later_logit_far_above_the_first_closely(mixed):
    """The sums' reference is replaced and the sums scaled: all of the student's weight is on the later slot."""
    _lib()
    c = make(30, 256, 400, 24, seed=21, mixed=mixed)
    for i in range(30):
        c["w"][int(c["idx"][i, 5 + i % 19])] = c["h"][i] * 0.5
    check_closely(c, gradient=not mixed)


@pytest.mark.gpu
@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("N, d, K", [(9800, 256, 11), (6100, 512, 11), (4900, 1024, 11), (2450, 2048, 11), (1230, 4096, 11), (1230, 8192, 5),
                                     (1230, 16384, 5)])
def test_teams_with_many_rows(N, d, K, mixed):
    """Eight rows or more for every team of every width: the rows' slots and the ring's stages are used again and again."""
    _lib()
    check_closely(make(N, d, 300, K, seed=N, mixed=mixed))
