"""Linear cross entropy (qad_linear_ce_*) against its definition in 64 bits.

Bounds: a logit is an fp32 accumulation of d bf16 products, |dz| <= d 2^-23 max_v sum |h w| =: e (2^-23: the tensor
cores may truncate).  The loss moves by at most 2 e and a few fp32 units of its terms.  exp(z - ref) is rounded to bf16
once before the product with the head (2^-8 of every term) and the gradient once at the end (2^-8), so
|ddh| <= g (2^-8 + 4 e) sum_v q |w_v| + g 4 e |w_t| + 2^-8 |dh|, and dw alike with q_iv - 1[v = t] rounded.
"""
import pytest
import torch

import scale_only_quantization_gb300 as Q


def _lib():
    from scale_only_quantization_gb300 import build
    build.build()
    return Q.lib()


def test_refusals_before_any_launch():
    L = _lib()
    P = 1 << 20
    need = {g: Q.qad_linear_ce_workspace_bytes(4, 64, 100, *g) for g in ((0, 0), (1, 0), (0, 1), (1, 1))}
    assert all(n > 0 and n % 1024 == 0 for n in need.values())
    names = ("h", "ldh", "w", "ldw", "t", "g", "loss", "lse", "dh", "dw", "acc", "N", "d", "V", "ws", "n", "st")
    base = dict(h=P, ldh=64, w=P, ldw=64, t=P, g=None, loss=P, lse=P, dh=P, dw=P, acc=0, N=4, d=64, V=100, ws=P, n=1 << 30,
                st=None)
    both = lambda **k: L.qad_linear_ce_fwd_bwd(*[{**base, **k}[m] for m in names])  # noqa: E731
    fwd = lambda **k: L.qad_linear_ce_fwd(*[{**base, **k}[m] for m in names if m not in ("g", "dh", "dw", "acc")])  # noqa: E731
    bad, uns = Q.QAD_ERR_INVALID_ARG, Q.QAD_ERR_UNSUPPORTED
    for f in (both, fwd):
        assert f(N=-1) == bad and f(V=0) == bad and f(d=0) == bad
        assert f(d=72, ldh=72, ldw=72) == uns and f(V=1 << 30) == uns and f(N=1 << 30) == uns
        assert f(ws=None) == bad and f(ws=P + 16) == bad and f(ldh=56) == bad and f(ldw=68) == bad
        for p in ("h", "w", "t", "loss", "lse"):
            assert f(**{p: None}) == bad and f(**{p: P + 2}) == bad
    assert fwd(n=need[0, 0] - 1) == Q.QAD_ERR_WORKSPACE
    assert both(n=need[1, 1] - 1) == Q.QAD_ERR_WORKSPACE and both(dw=None, n=need[1, 0] - 1) == Q.QAD_ERR_WORKSPACE
    assert both(dh=None, dw=None) == bad and both(dh=P + 2) == bad and both(dw=P + 2) == bad and both(g=P + 4) == bad
    assert Q.qad_linear_ce_workspace_bytes(4, 72, 100, 1, 0) == 0


def test_workspace_is_bounded_in_the_vocabulary():
    """The stored piece of exp(logits) stays within 1 GB however many tokens and words there are."""
    for N, V in [(1, 1), (8192, 151936), (32768, 151936), (100000, 256000), (8, 1 << 20)]:
        fwd, grad = (Q.qad_linear_ce_workspace_bytes(N, 2048, V, g, 0) for g in (0, 1))
        assert grad - fwd <= (1 << 30) + 4 * N * 2048 + 4096


def make(N, d, V, seed=0, ldh=None, ldw=None, boost=6.0, size=1.0, drop=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    w = (rand(V, ldw or d) / d ** 0.5).to(bf)
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    h = size * rand(N, ldh or d)
    h[:, :d] += boost * torch.rand((N, 1), generator=g, device="cuda") * w[t, :d].float()
    gr = torch.rand(N, generator=g, device="cuda") + 0.5
    target = torch.where(torch.rand(N, generator=g, device="cuda") < drop, -1, t).to(torch.int32)
    return dict(h=h.to(bf), w=w, target=target, g=gr, N=N, d=d, V=V)


def run(c, dh=True, dw=False, accumulate=None, fwd_only=False):
    N, d, V = c["N"], c["d"], c["V"]
    nan = float("nan")
    o = dict(loss=torch.full((N,), nan, device="cuda"), lse=torch.full((N,), nan, device="cuda"))
    o["dh"] = (torch.full((N, d), nan, dtype=torch.bfloat16, device="cuda") if accumulate is None else accumulate) if dh else None
    o["dw"] = torch.full((V, d), nan, dtype=torch.bfloat16, device="cuda") if dw else None
    n = Q.qad_linear_ce_workspace_bytes(N, d, V, int(dh and not fwd_only), int(dw and not fwd_only))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # nothing of the workspace may be taken as set
    a = (c["h"], c["h"].stride(0), c["w"], c["w"].stride(0), c["target"])
    if fwd_only:
        Q.qad_linear_ce_fwd(*a, o["loss"], o["lse"], N, d, V, ws)
    else:
        Q.qad_linear_ce_fwd_bwd(*a, c["g"], o["loss"], o["lse"], o["dh"], o["dw"], int(accumulate is not None), N, d, V, ws)
    o["err"] = Q.qad_check_device_error(ws)
    return o


def exact(c, h=None):
    d, V = c["d"], c["V"]
    h = c["h"][:, :d].double() if h is None else h
    w = c["w"][:, :d].double()
    z = h @ w.T
    lse = torch.logsumexp(z, 1)
    t = c["target"].long()
    live = (t >= 0) & (t < V)
    at = torch.where(live, t, 0)[:, None]
    loss = torch.where(live, lse - z.gather(1, at)[:, 0], 0.0)
    q = (z - lse[:, None]).exp()
    g = torch.where(live, c["g"].double(), 0.0)[:, None]
    gz = q.clone()
    gz.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
    gz *= g
    e = (d * 2.0 ** -23 * (h.abs() @ w.abs().T).amax(1))[:, None]
    tol = dict(loss=2 * e[:, 0] + 2e-6 * (1 + lse.abs()), lse=2 * e[:, 0] + 2e-6 * (1 + lse.abs()))
    dh, dw = gz @ w, gz.T @ h
    tol["dh"] = g * ((2.0 ** -8 + 4 * e + 1e-5) * (q @ w.abs()) + (4 * e + 1e-5) * w[at[:, 0]].abs()) + 2.0 ** -8 * dh.abs()
    tol["dw"] = ((2.0 ** -8 + 1e-5) * gz.abs() + 4 * g * e * q).T @ h.abs() + 2.0 ** -8 * dw.abs() + 1e-12
    onehot = torch.zeros_like(q).scatter_(1, at, 1.0) * g
    tol["dw"] += (4 * e * onehot).T @ h.abs()
    return dict(loss=loss, lse=lse, dh=dh, dw=dw), tol


def check(c, dh=True, dw=False):
    o = run(c, dh, dw)
    ref, tol = exact(c)
    assert o["err"] == 0
    for n in ("loss", "lse") + (("dh",) if dh else ()) + (("dw",) if dw else ()):
        bad = (o[n].double() - ref[n]).abs() - tol[n]
        assert torch.all(bad <= 0), (n, float(bad.max()))
    f = run(c, fwd_only=True)
    assert torch.equal(f["loss"], o["loss"]) and torch.equal(f["lse"], o["lse"])
    return o


SIZES = [(1, 16, 1), (1, 64, 2), (1, 256, 1000), (5, 272, 257), (255, 256, 256), (256, 512, 255), (257, 144, 511), (300, 256, 5003),
         (513, 2048, 1025), (33, 2880, 2049)]


@pytest.mark.gpu
@pytest.mark.parametrize("N, d, V", SIZES)
def test_loss_and_hidden_gradient_against_64_bits(N, d, V):
    _lib()
    check(make(N, d, V, seed=N + d + V))


@pytest.mark.gpu
@pytest.mark.parametrize("N, d, V", SIZES)
def test_head_gradient_against_64_bits(N, d, V):
    _lib()
    check(make(N, d, V, seed=N + d + V, drop=0.2), dw=True)
    if N < 300:
        check(make(N, d, V, seed=N + d, drop=0.2), dh=False, dw=True)


@pytest.mark.gpu
def test_many_pieces_of_the_vocabulary(monkeypatch):
    """A row count whose pieces do not hold the whole vocabulary: three pieces, the last one ragged, against the
    same rows in a call of their own (one piece)."""
    _lib()
    N, d, V = 20000, 64, 60001
    c = make(N, d, V, seed=1, drop=0.1)
    assert Q.qad_linear_ce_workspace_bytes(N, d, V, 1, 0) < 2 * N * V
    o = run(c, dw=True)
    part = {**c, "N": 300, "h": c["h"][-300:], "target": c["target"][-300:], "g": c["g"][-300:]}
    ref, tol = exact(part)
    for n in ("loss", "lse", "dh"):
        assert torch.all((o[n][-300:].double() - ref[n]).abs() <= tol[n])
    # the head's gradient: some of its rows, over all tokens
    rows = torch.tensor([0, 1, 25599, 25600, 40000, 60000], device="cuda")
    h, w = c["h"].double(), c["w"].double()
    live = c["target"] >= 0
    gz = (h @ w[rows].T - o["lse"].double()[:, None]).exp()
    gz -= (c["target"].long()[:, None] == rows[None]).double()
    gz *= torch.where(live, c["g"].double(), 0.0)[:, None]
    dw = gz.T @ h
    size = gz.abs().T @ h.abs()
    assert torch.all((o["dw"][rows].double() - dw).abs() <= 2.0 ** -8 * dw.abs() + (2.0 ** -8 + 2e-4) * size + 1e-9)


@pytest.mark.gpu
def test_strided_rows_of_hidden_states_and_head():
    _lib()
    check(make(70, 272, 600, seed=4, ldh=560, ldw=296), dw=True)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1.0, 30.0, 300.0])
def test_large_logits(size):
    """Logits hundreds of nats apart: rows whose target is far below the largest logit take the second sweep."""
    _lib()
    c = make(300, 256, 2000, seed=5, boost=0.0, size=size)
    o = run(c, dw=True)
    ref, tol = exact(c)
    for n in ("loss", "lse", "dh", "dw"):
        assert torch.isfinite(o[n]).all()
        assert torch.all((o[n].double() - ref[n]).abs() <= tol[n]), n


@pytest.mark.gpu
def test_sure_predictions_keep_their_precision():
    """Losses down to e^-30: the loss and the gradient keep their relative precision (no cancellation against lse)."""
    _lib()
    N, d, V = 64, 256, 3000
    c = make(N, d, V, seed=6, boost=0.0, size=0.2)
    t = c["target"].long()
    c["h"] = (c["h"].float() + torch.linspace(5, 38, N, device="cuda")[:, None] * c["w"][t].float()).to(torch.bfloat16)
    o = run(c)
    ref, _ = exact(c)
    # log1p of the sum over the other tokens: lse - z_t cancels below 1e-14, in 64 bits too
    z = c["h"].double() @ c["w"].double().T
    z -= z.gather(1, t[:, None])
    loss = torch.log1p(z.exp().scatter(1, t[:, None], 0.0).sum(1))
    assert float(loss.min()) < 1e-9
    assert torch.all((o["loss"].double() - loss).abs() <= 1e-3 * loss)
    rel = (o["dh"].double() - ref["dh"]).norm(dim=1) / ref["dh"].norm(dim=1)
    assert float(rel.max()) < 1e-2


@pytest.mark.gpu
def test_rows_without_a_target():
    """target < 0: loss and gradient 0, lse still written; a target past the vocabulary is reported and treated the same."""
    _lib()
    c = make(40, 256, 700, seed=7)
    c["target"][::3] = -1
    c["target"][1] = -100
    o = check(c, dw=True)
    assert torch.all(o["loss"][::3] == 0) and torch.all(o["dh"][::3] == 0) and torch.isfinite(o["lse"]).all()
    c["target"][2] = 700
    c["target"][5] = 2 ** 31 - 1
    o = run(c, dw=True)
    assert o["err"] == Q.QAD_DEV_BAD_INDEX
    ref, tol = exact(c)
    for n in ("loss", "lse", "dh", "dw"):
        assert torch.all((o[n].double() - ref[n]).abs() <= tol[n]), n
    c["target"][:] = -1
    o = run(c, dw=True)
    assert torch.all(o["loss"] == 0) and torch.all(o["dh"] == 0) and torch.all(o["dw"] == 0)


@pytest.mark.gpu
def test_nan_stays_in_its_row():
    _lib()
    c = make(300, 256, 700, seed=8)
    a = run(c)
    c["h"][2, 5] = float("nan")
    c["target"][7] = -1
    c["h"][7, 1] = float("inf")
    b = run(c)
    rows = [i for i in range(300) if i not in (2, 7)]
    for n in ("loss", "lse", "dh"):
        assert torch.equal(a[n][rows], b[n][rows])
    assert torch.isnan(b["loss"][2]) and torch.all(b["dh"][7] == 0)


@pytest.mark.gpu
def test_accumulates_onto_a_gradient_and_weights_default_to_one():
    _lib()
    c = make(50, 256, 700, seed=9)
    ref, tol = exact(c)
    base = torch.randn((50, 256), device="cuda").to(torch.bfloat16)
    o = run(c, accumulate=base.clone())
    s = base.double() + ref["dh"]
    assert torch.all((o["dh"].double() - s).abs() <= tol["dh"] + 2.0 ** -8 * s.abs())
    one = {**c, "g": torch.ones(50, device="cuda")}
    a = run(one)
    b = run({**c, "g": None})
    assert torch.equal(a["dh"], b["dh"])


@pytest.mark.gpu
def test_gradient_against_differences():
    _lib()
    c = make(6, 256, 300, seed=10)
    o = run(c)
    h = c["h"].double()
    s = 1e-5
    for seed in range(3):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        v = torch.randn(h.shape, generator=g, device="cuda", dtype=torch.float64)
        num = c["g"].double() * (exact(c, h + s * v)[0]["loss"] - exact(c, h - s * v)[0]["loss"]) / (2 * s)
        _, tol = exact(c)
        assert torch.all((num - (o["dh"].double() * v).sum(1)).abs() <= (tol["dh"] * v.abs()).sum(1) + 1e-6)


@pytest.mark.gpu
def test_no_rows():
    """N = 0 is a valid call: the head's gradient is zero."""
    _lib()
    w = torch.randn((300, 64), device="cuda").to(torch.bfloat16)
    dw = torch.full_like(w, float("nan"))
    e = torch.empty(0, device="cuda")
    ws = torch.empty(Q.qad_linear_ce_workspace_bytes(0, 64, 300, 0, 1), dtype=torch.uint8, device="cuda")
    Q.qad_linear_ce_fwd_bwd(e, 64, w, 64, e, None, e, e, None, dw, 0, 0, 64, 300, ws)
    torch.cuda.synchronize()
    assert torch.all(dw == 0)


@pytest.mark.gpu
def test_repeatable_on_another_stream():
    _lib()
    c = make(700, 512, 3000, seed=12)
    a = run(c, dw=True)
    with torch.cuda.stream(torch.cuda.Stream()):
        b = run(c, dw=True)
    torch.cuda.synchronize()
    for n in ("loss", "lse", "dh", "dw"):
        assert torch.equal(a[n], b[n])


@pytest.mark.gpu
@pytest.mark.parametrize("N, d, V", [(64, 512, 700), (127, 272, 3001), (128, 256, 5000), (129, 256, 5000), (700, 320, 40000)])
def test_row_counts_around_the_transposed_products(N, d, V):
    """Up to 128 rows the products are taken transposed; many words for few columns split the contraction into many slabs."""
    _lib()
    check(make(N, d, V, seed=N, drop=0.1), dw=True)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 40, 128])
def test_large_logits_of_few_rows(N):
    """The second sweep of the transposed products: targets hundreds of nats below the largest logit."""
    _lib()
    c = make(N, 256, 2000, seed=15, boost=0.0, size=200.0)
    o = run(c, dw=True)
    ref, tol = exact(c)
    assert float(ref["loss"].max()) > 100.0
    for n in ("loss", "lse", "dh", "dw"):
        assert torch.isfinite(o[n]).all()
        assert torch.all((o[n].double() - ref[n]).abs() <= tol[n]), n


@pytest.mark.gpu
def test_neighbouring_calls_share_a_workspace():
    """Calls of different sizes follow each other on one workspace without a wait between them."""
    _lib()
    cs = [make(N, 256, V, seed=N, drop=0.1) for N, V in ((300, 5000), (20, 9000), (600, 777), (1, 9000))]
    want = [run(c) for c in cs]
    ws = torch.empty(max(Q.qad_linear_ce_workspace_bytes(c["N"], 256, c["V"], 1, 0) for c in cs), dtype=torch.uint8,
                     device="cuda")
    outs = []
    for c in cs:
        N = c["N"]
        o = dict(loss=torch.empty(N, device="cuda"), lse=torch.empty(N, device="cuda"),
                 dh=torch.empty((N, 256), dtype=torch.bfloat16, device="cuda"))
        Q.qad_linear_ce_fwd_bwd(c["h"], 256, c["w"], 256, c["target"], c["g"], o["loss"], o["lse"], o["dh"], None, 0, N,
                                256, c["V"], ws)
        outs.append(o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for n in o:
            assert torch.equal(o[n], w[n])


@pytest.mark.gpu
def test_no_rows_with_a_hidden_gradient_only():
    """N = 0 with dh alone: an empty tensor has no address, and the call has nothing to write."""
    _lib()
    w = torch.randn((300, 64), device="cuda").to(torch.bfloat16)
    e = torch.empty(0, device="cuda")
    ws = torch.full((Q.qad_linear_ce_workspace_bytes(0, 64, 300, 1, 0),), 0xFF, dtype=torch.uint8, device="cuda")
    Q.qad_linear_ce_fwd_bwd(e, 64, w, 64, e, None, e, e, e, None, 0, 0, 64, 300, ws)
    assert Q.qad_check_device_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N", [3, 150])
def test_normaliser_of_a_target_far_below(N):
    """lse does not pass through the target's logit: with logits 0, 1, 2, ... and a target at -2^20 (all products exact
    in fp32) it keeps its precision, whose ulp at 2^20 would be 1/8; a target at -inf leaves it finite."""
    _lib()
    V, d = 300, 16
    w = torch.zeros((V, d), device="cuda", dtype=torch.bfloat16)
    w[:, 0] = torch.arange(V, device="cuda") % 8
    w[7, 0], w[7, 1] = 0.0, -(2.0 ** 20)
    w[9, 0], w[9, 2] = 0.0, -3e38
    h = torch.zeros((N, d), device="cuda", dtype=torch.bfloat16)
    h[:, 0] = 1.0
    h[0::3, 1] = 1.0     # the target's logit is -2^20
    h[1::3, 2] = 8.0     # ... below fp32's range
    target = torch.full((N,), 7, dtype=torch.int32, device="cuda")
    target[1::3] = 9
    target[2::3] = 8
    c = dict(h=h, w=w, target=target, g=torch.ones(N, device="cuda"), N=N, d=d, V=V)
    o = run(c)
    z = h.double() @ w.double().T
    lse = torch.logsumexp(z, 1)
    assert torch.all((o["lse"].double() - lse).abs() <= 2e-6 * (1 + lse.abs()))
    want = lse - z.gather(1, target.long()[:, None])[:, 0]
    assert torch.isinf(o["loss"][1::3]).all()
    ok = torch.arange(N, device="cuda") % 3 != 1
    assert torch.all((o["loss"].double() - want).abs()[ok] <= 2e-6 * (1 + want.abs()[ok]))


def test_partial_sums_are_bounded_in_the_vocabulary():
    """What the loss alone needs besides a few words per row does not grow with tokens times words."""
    for N, V in [(1, 1), (128, 1 << 20), (128, (1 << 30) - 1), (8192, 151936), (32768, 151936), (100000, 256000), (1 << 20, 256000)]:
        assert Q.qad_linear_ce_workspace_bytes(N, 2048, V, 0, 0) <= (32 << 20) + 64 * N + 16384


@pytest.mark.gpu
def test_pieces_of_few_rows():
    """A vocabulary that 128 rows take in two pieces, the second one short: the sums of both, and some of the gradient."""
    _lib()
    N, d, V = 20, 16, 3500001
    c = make(N, d, V, seed=3, drop=0.1)
    o = run(c)
    ref, tol = exact(c)
    assert o["err"] == 0
    for n in ("loss", "lse", "dh"):
        assert torch.all((o[n].double() - ref[n]).abs() <= tol[n]), n


def _one_row_far_below(N, d, V, row, seed):
    """Inputs in which exactly one row's target lies more than 60 nats below its largest logit."""
    c = make(N, d, V, seed=seed, drop=0.1)
    c["h"][row] = (c["h"][row].float() * 40).to(torch.bfloat16)
    z = c["h"][row].double() @ c["w"].double().T
    c["target"][row] = int(z.argmin())
    assert float(z.max() - z.min()) > 100
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("N, row", [(1000, 700), (1000, 999), (300, 0), (2600, 1300)])
def test_second_sweep_of_one_tile_of_rows(N, row):
    """One row asks for the second sweep: it and the rows of its tile are right, the others keep the bits that they have
    when nobody asks; a second such row in another tile changes nothing for the first."""
    _lib()
    d, V = 256, 3001
    c = _one_row_far_below(N, d, V, row, seed=N + row)
    o = run(c, dw=True)
    ref, tol = exact(c)
    assert o["err"] == 0
    for n in ("loss", "lse", "dh", "dw"):
        assert torch.all((o[n].double() - ref[n]).abs() <= tol[n]), n
    calm = {**c, "target": c["target"].clone()}
    calm["target"][row] = int((c["h"][row].double() @ c["w"].double().T).argmax())
    a = run(calm)
    rest = torch.arange(N, device="cuda") != row
    for n in ("loss", "lse", "dh"):
        assert torch.equal(a[n][rest], o[n][rest]), n
    again = _one_row_far_below(N, d, V, (row + 300) % N, seed=N + row)
    two = {**c, "h": again["h"].clone(), "target": again["target"].clone()}
    two["h"][row], two["target"][row] = c["h"][row], c["target"][row]
    b = run(two)
    assert torch.equal(b["loss"][row], o["loss"][row]) and torch.equal(b["dh"][row], o["dh"][row])
    ref, tol = exact(two)
    for n in ("loss", "lse", "dh"):
        assert torch.all((b[n].double() - ref[n]).abs() <= tol[n]), n


@pytest.mark.gpu
def test_second_sweep_of_many_pieces():
    """The tiles that ask, over three pieces of the vocabulary."""
    _lib()
    N, d, V, row = 20000, 64, 60001, 12345
    c = _one_row_far_below(N, d, V, row, seed=2)
    o = run(c)
    at = slice(row - 40, row + 40)
    part = {**c, "N": 80, "h": c["h"][at], "target": c["target"][at], "g": c["g"][at]}
    ref, tol = exact(part)
    for n in ("loss", "lse", "dh"):
        assert torch.all((o[n][at].double() - ref[n]).abs() <= tol[n]), n


@pytest.mark.gpu
def test_one_row_does_not_double_the_step():
    """The second sweep is of the row's tile only: with 16 tiles of rows the call takes well under half as long again
    (twice, were all rows swept)."""
    _lib()
    N, d, V = 4096, 512, 50000
    slow = _one_row_far_below(N, d, V, 2000, seed=1)
    fast = {**slow, "target": slow["target"].clone()}
    fast["target"][2000] = int((slow["h"][2000].double() @ slow["w"].double().T).argmax())
    ws = torch.empty(Q.qad_linear_ce_workspace_bytes(N, d, V, 1, 0), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    dh = torch.empty((N, d), dtype=torch.bfloat16, device="cuda")

    def time(c):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        for _ in range(10):
            Q.qad_linear_ce_fwd_bwd(c["h"], d, c["w"], d, c["target"], c["g"], loss, lse, dh, None, 0, N, d, V, ws)
        e[1].record()
        torch.cuda.synchronize()
        return e[0].elapsed_time(e[1])

    both = [(time(fast), time(slow)) for _ in range(8)][1:]
    assert min(b for _, b in both) < 1.5 * min(a for a, _ in both), both
