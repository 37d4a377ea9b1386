"""Log probabilities, entropy and top alternatives of logits (qad_token_logprobs) and their gradient, against 64 bits.

Tolerances.  S = sum of 2^y over V logits: each thread adds ceil(V / 512) terms (16 of them at a time in two lanes),
then 5 + 16 (+ 8) sums join: n = V / 512 + 64 roundings of 2^-24 at most, one of y itself (|y| of the terms that matter:
at most log2 V + 40) and two of the exponential: rel(S) <= (n + 64) * 2^-24 =: e.  The logarithm and the last additions
round once each.  U / S is off by at most (e + 2^-22) * (40 + ln V).
"""
import math

import pytest
import torch

import scale_only_quantization_gb300 as Q

U24 = 2.0 ** -24
KINDS = {torch.float32: Q.QAD_F32, torch.bfloat16: Q.QAD_BF16}


def _build():
    from scale_only_quantization_gb300 import build
    build.build()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _logits(N, V, ld, dtype, seed, offset=0):
    g = _gen(seed)
    big = torch.randn((N, ld + offset), generator=g, device="cuda") * 3
    z = big.to(dtype)[:, offset:offset + V]
    token = torch.randint(0, V, (N,), generator=g, device="cuda").to(torch.int32)
    return z, token


def _forward(z, token, K, tau=1.0, ld=None):
    N, V = z.shape
    ld = z.stride(0) if ld is None else ld
    f = lambda *s: torch.full(s, 777.0, device="cuda")  # noqa: E731
    out = dict(logp=f(N) if token is not None else None, lse=f(N), entropy=f(N),
               idx=torch.full((N, K), -777, dtype=torch.int32, device="cuda") if K else None, top=f(N, K) if K else None)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    Q.qad_token_logprobs(z, KINDS[z.dtype], ld, token, 1 / tau, out["logp"], out["lse"], out["entropy"], out["idx"],
                         out["top"], N, V, K, err)
    out["err"] = int(err)
    return out


def _reference(z, token, K, tau=1.0):
    x = z.double() / tau
    lse = torch.logsumexp(x, 1)
    l = torch.log_softmax(x, 1)
    ent = -(l.exp() * l.clamp_min(-1e300)).sum(1)
    logp = None
    if token is not None:
        t = token.long().clamp(0, z.shape[1] - 1)
        logp = torch.where(token >= 0, l.gather(1, t[:, None])[:, 0], 0.0)
    top, idx = torch.sort(z.double() + 0.0, dim=1, descending=True, stable=True)
    return dict(lse=lse, entropy=ent, logp=logp, idx=idx[:, :K].to(torch.int32), top=top[:, :K])


def _check(z, token, K, tau=1.0):
    got, ref = _forward(z, token, K, tau), _reference(z, token, K, tau)
    V = z.shape[1]
    e = (V / 512 + 128) * U24
    big = ref["lse"].abs() + z.double().abs().amax(1) / tau
    assert torch.all((got["lse"] - ref["lse"]).abs() <= e + 4 * U24 * big)
    assert torch.all((got["entropy"] - ref["entropy"]).abs() <= (2 * e + 4 * U24) * (40 + math.log(V)))
    if token is not None:
        assert torch.all((got["logp"] - ref["logp"]).abs() <= e + 4 * U24 * (big + ref["logp"].abs()))
    if K:
        assert torch.equal(got["idx"], ref["idx"])
        assert torch.equal(got["top"].double() + 0.0, ref["top"])
    assert got["err"] == 0
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V,ld,K", [(1, 1, 1, 1), (3, 7, 7, 7), (5, 130, 136, 0), (2, 1000, 1001, 100), (9, 8191, 8191, 16),
                                      (40, 8193, 8200, 64), (1, 151936, 151936, 20), (7, 50257, 50257, 100),
                                      (400, 32000, 32000, 8), (2, 200000, 200000, 600), (3, 1024, 1024, 1024),
                                      (1, 40000, 40000, 1024), (20, 32000, 32000, 513), (160, 151936, 151936, 64),
                                      (1, 33, 40, 33), (33, 100003, 100003, 256)])
def test_matches_64_bits(N, V, ld, K, dtype):
    _build()
    z, token = _logits(N, V, ld, dtype, N + V + K)
    token[N // 2] = -1 if N > 1 else token[0]
    _check(z, token, K, tau=0.7 if K % 2 else 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("offset,ld", [(8, 5003), (16, 5000), (8, 5001), (24, 5007)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_at_any_alignment(dtype, offset, ld):
    """A slice of columns, odd strides: the rows start at every place relative to 16 bytes, and the rest of the buffer
    holds NaN, which must not be read into a result."""
    _build()
    N, V = 17, 4999
    buf = torch.full((N * (ld + offset) + 64,), float("nan"), dtype=dtype, device="cuda")
    z = torch.as_strided(buf, (N, V), (ld + offset, 1), offset)
    z.copy_(torch.randn((N, V), generator=_gen(1), device="cuda") * 3)
    token = torch.arange(N, device="cuda", dtype=torch.int32) * 293
    got = _forward(z, token, 12, ld=ld + offset)
    same = _forward(z.contiguous(), token, 12)
    ref = _reference(z.contiguous(), token, 12)
    assert torch.equal(got["idx"], ref["idx"]) and torch.equal(same["idx"], ref["idx"])
    for name in ("logp", "lse", "entropy"):
        assert torch.all((got[name] - ref[name]).abs() <= 100 * (5000 / 512 + 128) * U24)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [1, 50, 300, 1000])
@pytest.mark.parametrize("rows", ["constant", "rising", "falling", "few values", "zeros of both signs", "late peak"])
def test_orders_and_ties(rows, K):
    """Rows in which very many logits pass the threshold, and equal ones that stand by their index."""
    _build()
    N, V = 4, 30011
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    if rows == "constant":
        z = torch.full((N, V), -2.5, device="cuda")
    elif rows == "rising":
        z = (i * 1e-4).expand(N, V)
    elif rows == "falling":
        z = (-i * 1e-4).expand(N, V)
    elif rows == "few values":
        z = torch.randint(-2, 3, (N, V), generator=_gen(2), device="cuda").float()
    elif rows == "zeros of both signs":
        z = torch.where(torch.rand((N, V), generator=_gen(3), device="cuda") < 0.5, 0.0, -0.0)
    else:
        z = torch.where(i > V - 2000, 20 + i * 1e-3, -i * 1e-3).expand(N, V)
    token = torch.tensor([0, V - 1, 17, -1], dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        _check(z.to(dtype).contiguous(), token, K)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_lowest_infinite_and_nan(dtype):
    _build()
    V, K = 9001, 6
    inf, low = float("inf"), torch.finfo(dtype).min
    z = (torch.randn((9, V), generator=_gen(4), device="cuda") * 2).to(dtype)
    token = torch.full((9,), 5, dtype=torch.int32, device="cuda")
    z[0, 100:] = -inf                       # most of a row masked
    z[1] = -inf                             # all of it
    z[2] = -inf
    z[2, [7000, 30, 8999]] = torch.tensor([1.0, 1.0, 0.5], device="cuda", dtype=dtype)
    z[3] = low                              # finite all the same: a uniform row
    z[4] = low
    z[4, 77] = 0.0
    z[5, 4000] = float("nan")
    z[6, 8000] = inf
    z[7] = float("nan")
    z[8, 5] = -inf                          # the token itself masked
    got = _forward(z, token, K)
    ref = _reference(z[[0, 2, 3, 4, 8]], token[[0, 2, 3, 4, 8]], K)
    tol = (V / 512 + 128) * U24
    for a, b in enumerate([0, 2, 3, 4, 8]):
        for name in ("lse", "entropy", "logp"):
            x, y = float(got[name][b]), float(ref[name][a])
            if b == 2 and name == "logp" or b == 8 and name == "logp":
                assert x == -inf
            else:
                assert abs(x - y) <= 100 * tol + 4 * U24 * abs(y), (b, name, x, y)
    assert torch.equal(got["idx"][[0, 2, 3, 4, 8]], ref["idx"]) and torch.equal(got["top"][[0, 2, 3, 4, 8]].double(), ref["top"])
    assert got["idx"][2].tolist() == [30, 7000, 8999, 0, 1, 2]
    assert float(got["lse"][1]) == -inf and float(got["entropy"][1]) == 0 and float(got["logp"][1]) == -inf
    assert got["idx"][1].tolist() == list(range(K)) and torch.all(got["top"][1] == -inf)
    for b in (5, 6, 7):
        assert all(math.isnan(float(got[name][b])) for name in ("lse", "entropy", "logp"))
    assert 4000 not in got["idx"][5].tolist() and int(got["idx"][6][0]) == 8000 and float(got["top"][6][0]) == inf
    assert got["idx"][7].tolist() == [-1] * K and torch.all(got["top"][7] == -inf)
    # the gradients of the masked rows
    dz = _backward(z, token, got, torch.ones(9, device="cuda"), torch.ones(9, device="cuda"))
    assert torch.all(dz[1] == 0) and torch.all(dz[0, 100:] == 0) and torch.isfinite(dz[[0, 1, 3, 4]].float()).all()


@pytest.mark.gpu
def test_outputs_left_out_and_tokens_past_the_vocabulary():
    _build()
    z, token = _logits(6, 999, 999, torch.float32, 5)
    full = _forward(z, token, 9)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse, idx, top = torch.empty(6, device="cuda"), torch.empty((6, 9), dtype=torch.int32, device="cuda"), torch.empty((6, 9), device="cuda")
    Q.qad_token_logprobs(z, 0, 999, None, 1.0, None, lse, None, None, None, 6, 999, 0)
    assert torch.all((lse - full["lse"]).abs() <= 300 * U24 + 2 * U24 * full["lse"].abs())
    Q.qad_token_logprobs(z, 0, 999, None, 1.0, None, None, None, idx, None, 6, 999, 9)
    Q.qad_token_logprobs(z, 0, 999, None, 1.0, None, None, None, None, top, 6, 999, 9)
    assert torch.equal(idx, full["idx"]) and torch.equal(top, full["top"])
    token[2], token[4] = 999, 2 ** 31 - 1
    got = _forward(z, token, 0)
    assert got["err"] == Q.QAD_DEV_BAD_INDEX and float(got["logp"][2]) == 0 and float(got["logp"][4]) == 0
    assert torch.equal(got["logp"][[0, 1, 3, 5]], _forward(z, token.clamp_max(998), 0)["logp"][[0, 1, 3, 5]])
    Q.qad_token_logprobs(z, 0, 999, token, 1.0, None, lse, None, None, None, 6, 999, 0, err)
    assert int(err) == Q.QAD_DEV_BAD_INDEX
    Q.qad_token_logprobs(z[:0], 0, 999, token, 1.0, None, lse, None, None, None, 0, 999, 0)  # no rows


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^31 logits: the last rows."""
    _build()
    N, V = 16000, 151936
    z = torch.empty((N, V), dtype=torch.bfloat16, device="cuda")
    for i in range(0, N, 1000):
        z[i:i + 1000] = torch.randn((1000, V), generator=_gen(i), device="cuda")
    token = torch.randint(0, V, (N,), generator=_gen(1), device="cuda").to(torch.int32)
    got = _forward(z, token, 4)
    ref = _reference(z[-3:], token[-3:], 4)
    assert torch.equal(got["idx"][-3:], ref["idx"])
    assert torch.all((got["logp"][-3:] - ref["logp"]).abs() <= 1e-4)
    g = torch.ones(N, device="cuda")
    Q.qad_token_logprobs_bwd(z, 1, V, token, 1.0, got["lse"], got["entropy"], g, None, z, V, N, V)  # in place
    p = torch.exp(ref["logp"])
    at = z[-3:].gather(1, token[-3:].long()[:, None])[:, 0]
    assert torch.all((at.double() - (1 - p)).abs() <= 2.0 ** -8 + 1e-4)


# ------------------------------------------------------------------------------------------------ gradient


def _backward(z, token, fwd, g_logp, g_ent, tau=1.0, lddz=None):
    N, V = z.shape
    lddz = V if lddz is None else lddz
    dz = torch.full((N, lddz), 777.0, dtype=z.dtype, device="cuda")
    Q.qad_token_logprobs_bwd(z, KINDS[z.dtype], z.stride(0), token, 1 / tau, fwd["lse"], fwd["entropy"], g_logp, g_ent,
                             dz, lddz, N, V)
    if lddz > V:
        assert torch.all(dz[:, V:] == 777.0)
    return dz[:, :V]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V,ld,lddz,part", [(1, 1, 1, 1, "both"), (3, 7, 9, 7, "both"), (5, 1000, 1000, 1000, "logp"),
                                              (5, 1000, 1001, 1003, "entropy"), (33, 4097, 4097, 4097, "both"),
                                              (7, 50257, 50257, 50257, "both"), (7, 50257, 50264, 50272, "both"),
                                              (2, 151936, 151936, 151936, "both")])
def test_gradient_matches_the_formula(N, V, ld, lddz, part, dtype):
    """dz = b (g (1[v = t] - p) - h p (log p + H)) in 64 bits, from the same lse and H.

    log p is off by 2^-24 (|b z| + |lse|) (one fused rounding, and lse's own), p by that and 4 roundings relatively."""
    _build()
    tau = 0.7
    z, token = _logits(N, V, ld, dtype, N + V)
    if N > 1:
        token[1] = -1
    fwd = _forward(z, token, 0, tau)
    g = _gen(9)
    gl = torch.randn(N, generator=g, device="cuda") if part != "entropy" else None
    ge = torch.randn(N, generator=g, device="cuda") if part != "logp" else None
    dz = _backward(z, token, fwd, gl, ge, tau, lddz)
    b = float(torch.tensor(1 / tau, dtype=torch.float32))
    x = z.double() * b
    lp = x - fwd["lse"].double()[:, None]
    p = lp.exp()
    gg = torch.zeros(N, 1, dtype=torch.float64, device="cuda") if gl is None else (gl.double() * (token >= 0))[:, None]
    hh = torch.zeros(N, 1, dtype=torch.float64, device="cuda") if ge is None else ge.double()[:, None]
    H = fwd["entropy"].double()[:, None]
    hit = torch.zeros_like(x).scatter_(1, token.long().clamp_min(0)[:, None], 1.0)
    ref = b * (gg * (hit - p) - hh * p * (lp + H))
    off = 2 * U24 * (x.abs() + fwd["lse"].double().abs()[:, None]) + 8 * U24
    tol = b * p * (gg.abs() + hh.abs() * (lp.abs() + H)) * (off + 8 * U24) + b * p * hh.abs() * off
    tol = tol + 4 * U24 * b * gg.abs() * hit + 1e-37
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert torch.all((dz.double() - ref).abs() <= tol)


@pytest.mark.gpu
def test_gradient_against_differences():
    """d(g logp + h H) along random directions by central differences of the forward call in fp32: the step 2^-5 leaves
    a third-order error of 2^-10 |u|^3 / 6 and 2^-23 * 20 / 2^-4 of rounding."""
    _build()
    N, V, eps = 8, 300, 2.0 ** -5
    z, token = _logits(N, V, V, torch.float32, 3)
    g = _gen(4)
    gl, ge = torch.randn(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
    dz = _backward(z, token, _forward(z, token, 0), gl, ge)

    def value(x):
        f = _forward(x, token, 0)
        return gl.double() * f["logp"].double() + ge.double() * f["entropy"].double()

    for _ in range(4):
        u = torch.randn((N, V), generator=g, device="cuda").clamp(-2, 2)
        diff = (value(z + eps * u) - value(z - eps * u)) / (2 * eps)
        along = (dz.double() * u.double()).sum(1)
        assert torch.all((diff - along).abs() <= (gl.abs() + 8 * ge.abs()) * 2.0 ** -10 * 8 + 1e-3)


@pytest.mark.gpu
def test_gradient_in_place_and_autograd():
    from scale_only_quantization_gb300.autograd import QADTokenLogprobs
    _build()
    N, V = 12, 5003
    z, token = _logits(N, V, V, torch.float32, 6)
    fwd = _forward(z, token, 0)
    gl, ge = torch.randn(N, device="cuda"), torch.randn(N, device="cuda")
    ref = _backward(z, token, fwd, gl, ge)
    own = z.clone()
    Q.qad_token_logprobs_bwd(own, 0, V, token, 1.0, fwd["lse"], fwd["entropy"], gl, ge, own, V, N, V)
    assert torch.equal(own, ref)
    # autograd: a loss on both outputs, one of them alone, 64-bit tokens, a strided view
    read = QADTokenLogprobs(tau=2.0, top=5)
    leaf = z.clone().requires_grad_(True)
    logp, ent, lse, idx, top = read(leaf, token.long())
    (logp * gl).sum().backward(retain_graph=True)
    g64 = z.double().requires_grad_(True)
    l = torch.log_softmax(g64 / 2, 1)
    (l.gather(1, token.long()[:, None])[:, 0] * gl.double()).sum().backward()
    assert torch.all((leaf.grad.double() - g64.grad).abs() <= 1e-5 * gl.abs().double()[:, None])
    leaf.grad = None
    (ent * ge).sum().backward()
    g64.grad = None
    l = torch.log_softmax(g64 / 2, 1)
    ((-(l.exp() * l).sum(1)) * ge.double()).sum().backward()
    assert torch.all((leaf.grad.double() - g64.grad).abs() <= 1e-4 * ge.abs().double()[:, None])
    assert not (lse.requires_grad or idx.requires_grad or top.requires_grad)
    assert torch.equal(top, torch.topk(z, 5, dim=1).values) and read.device_error() == 0
    wide = torch.randn((N, 2 * V), device="cuda")
    assert torch.equal(read(wide[:, 1:V + 1])[3], read(wide[:, 1:V + 1].contiguous())[3])
    tok = token.long()
    tok[0] = 2 ** 40
    logp = read(z, tok)[0]
    assert float(logp[0]) == 0 and read.device_error() == Q.QAD_DEV_BAD_INDEX and read.device_error() == 0
    with pytest.raises(ValueError):
        read(z.double(), token)
    with pytest.raises(ValueError):
        read(z, token[:3])
    empty = read(torch.empty((0, 50), device="cuda", requires_grad=True), torch.empty(0, dtype=torch.int64, device="cuda"))
    empty[0].sum().backward()
    assert empty[3].shape == (0, 5)


@pytest.mark.gpu
def test_captured_with_new_inputs():
    _build()
    z, token = _logits(3, 20011, 20011, torch.bfloat16, 7)
    out = {k: v for k, v in _forward(z, token, 10).items()}
    dz = torch.empty_like(z)
    g = torch.ones(3, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.qad_token_logprobs(z, 1, 20011, token, 1.0, out["logp"], out["lse"], out["entropy"], out["idx"], out["top"], 3,
                             20011, 10, err)
        Q.qad_token_logprobs_bwd(z, 1, 20011, token, 1.0, out["lse"], out["entropy"], g, g, dz, 20011, 3, 20011)
    for seed in (8, 9):
        z.copy_(_logits(3, 20011, 20011, torch.bfloat16, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        again = _forward(z, token, 10)
        assert all(torch.equal(out[k], again[k]) for k in ("logp", "lse", "entropy", "idx", "top"))
        assert torch.equal(dz, _backward(z, token, again, g, g))


def test_refusals():
    """Checked on the host before anything is launched (no GPU is touched)."""
    _build()
    L = Q.lib()
    P = 1 << 20
    good = [P, 0, 100, P, 1.0, P, P, P, P, P, 4, 100, 8, P, None]
    call = lambda args: L.qad_token_logprobs(*args)  # noqa: E731

    def put(base, **at):
        args = list(base)
        for k, v in at.items():
            args[int(k[1:])] = v
        return args

    inv, unsup = Q.QAD_ERR_INVALID_ARG, Q.QAD_ERR_UNSUPPORTED
    for bad in (dict(a0=None), dict(a0=P + 4), dict(a1=2), dict(a1=-1), dict(a2=99), dict(a4=0.0), dict(a4=-1.0),
                dict(a4=float("nan")), dict(a4=float("inf")), dict(a3=None), dict(a3=P + 2), dict(a5=P + 1), dict(a10=-1),
                dict(a11=0, a12=0), dict(a12=-1), dict(a12=0), dict(a8=None, a9=None), dict(a13=P + 1), dict(a9=P + 2)):
        assert call(put(good, **bad)) == inv, bad
    assert call(put(good, a5=None, a6=None, a7=None, a8=None, a9=None, a12=0)) == inv
    assert call(put(good, a12=101)) == unsup and call(put(good, a2=5000, a11=5000, a12=1025)) == unsup
    assert call(put(good, a2=1 << 30, a11=1 << 30)) == unsup and call(put(good, a10=1 << 30)) == unsup
    assert call(put(good, a10=0)) == Q.QAD_OK and call(put(good, a0=None, a10=0)) == Q.QAD_OK
    back = [P, 0, 100, P, 1.0, P, P, P, P, P + 4096, 100, 4, 100, None]
    call = lambda args: L.qad_token_logprobs_bwd(*args)  # noqa: E731
    for bad in (dict(a0=None), dict(a1=2), dict(a2=99), dict(a3=None), dict(a5=None), dict(a6=None), dict(a7=None, a8=None),
                dict(a9=None), dict(a9=P + 8), dict(a10=99), dict(a9=P, a10=104), dict(a7=P + 2), dict(a4=-1.0)):
        assert call(put(back, **bad)) == inv, bad
    assert call(put(back, a11=0)) == Q.QAD_OK


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused():
    from scale_only_quantization_gb300.autograd import QADTokenLogprobs
    _build()
    with pytest.raises(ValueError):
        QADTokenLogprobs()(torch.zeros(2, 64, device="cuda"), torch.zeros(2, dtype=torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [-1e5, -1e9, -1e10, -3e10, -1e20, -1e30, -1e35])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tau", [1.0, 0.6, 2.0 ** 20])
def test_low_finite_fills(tau, dtype, fill):
    """Masks of finite numbers: most of a row, its front, single logits left, a whole row, two levels of them.  A fill's
    probability is 0 beside logits of ordinary size (of a size that the temperature leaves ordinary), so that the bounds
    are those of the live logits; in a row of nothing else log p = -ln V has no part of the fill's size."""
    _build()
    V, K = 20011, 4
    z = (torch.randn((6, V), generator=_gen(21), device="cuda") * 2 * tau).to(dtype)
    z[0, 40:] = fill
    z[1, :V - 7] = fill
    z[2, 1::2] = fill
    z[3] = fill
    z[4] = fill
    z[4, 12345] = tau
    z[5, :9000] = fill
    z[5, 9000:18000] = 2 * fill
    live = z.double() > 0.5 * fill
    live[3] = True
    token = torch.tensor([3, V - 2, 10, 77, 12345, 19000], dtype=torch.int32, device="cuda")
    got, ref = _forward(z, token, K, tau), _reference(z, token, K, tau)
    if fill < -1e3 * tau:
        e = (V / 512 + 128) * U24
        big = (z.double().abs() * live).amax(1) / tau + ref["lse"].abs()
        assert torch.all((got["lse"] - ref["lse"]).abs() <= e + 4 * U24 * big)
        assert torch.all((got["entropy"] - ref["entropy"]).abs() <= (2 * e + 4 * U24) * (40 + math.log(V)))
        big[3] = math.log(V)
        assert torch.all((got["logp"] - ref["logp"]).abs() <= e + 4 * U24 * big)
        dz = _backward(z, token, got, torch.ones(6, device="cuda"), torch.ones(6, device="cuda"), tau)
        rows = [0, 1, 2, 4, 5]  # the uniform row: lse holds nothing smaller than the fill's own rounding
        assert torch.isfinite(dz[rows].float()).all() and torch.all(dz[rows][~live[rows]] == 0)
    assert torch.equal(got["idx"], ref["idx"]) and torch.equal(got["top"].double() + 0.0, ref["top"])
    assert all(torch.isfinite(got[name]).all() for name in ("lse", "entropy", "logp"))


@pytest.mark.gpu
@pytest.mark.parametrize("tau", [1e30, 1e37, 1e38, 2e38])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_smallest_inverse_temperatures(tau, dtype):
    """1 / tau down to fp32's subnormal numbers, logits of up to the largest finite ones: the span of a row can pass what
    fp32 holds.  b itself is given as fp32, and the reference takes that number; its product with log2(e) is rounded once
    more, to 2^-149 where it is subnormal, which the exponents |z| <= 3.4e38 multiply."""
    _build()
    V = 5003
    b = float(torch.tensor(1 / tau, dtype=torch.float32))
    top = torch.finfo(dtype).max
    z = (torch.rand((4, V), generator=_gen(22), device="cuda", dtype=torch.float64) * 2 - 1)
    z = torch.stack([z[0] * 5, z[1] * min(tau, 1e38) * 3, z[2] * 3.3e38, z[3] * 3.3e38]).to(dtype)
    z[3] = torch.sort(z[3].float()).values.to(dtype)  # rising: the reference moves at nearly every step
    if tau < 1e37:
        z = z[:2]
    assert torch.all(z.abs() <= top)
    N = z.shape[0]
    token = torch.tensor([0, 17, 2, V - 1], dtype=torch.int32, device="cuda")[:N]
    got = _forward(z, token, 3, tau)
    ref = _reference(z, token, 3, 1 / b)
    e = (V / 512 + 128) * U24
    big = z.double().abs().amax(1)
    off = e + 8 * U24 * big * b + 4 * 2.0 ** -149 * big
    for name in ("lse", "entropy", "logp"):
        assert torch.all((got[name] - ref[name]).abs() <= (2 * off) * (1 if name != "entropy" else 40 + math.log(V))), name
    assert torch.equal(got["idx"], ref["idx"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tau", [0.6, 0.7, 3.0])
def test_gradient_of_rows_of_large_logits_is_finite(tau, dtype):
    """Rows of one low number (a padded row): b z - lse is what lse's rounding leaves, of any size and sign, so that p is
    not known; it is a probability all the same, and a row whose gradients are 0 stays 0."""
    _build()
    V = 1003
    fills = [-1e8, -1e10, -1e20, -1e30, float(torch.finfo(dtype).min) * 0.5, 3e10, 1e30]
    z = torch.tensor(fills, device="cuda").to(dtype)[:, None].expand(-1, V).contiguous()
    n = len(fills)
    token = torch.arange(n, device="cuda", dtype=torch.int32)
    got = _forward(z, token, 0, tau)
    one, zero = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    dz = _backward(z, token, got, one, one, tau).double()
    # |dz| <= b (g + h p |log p + H|), |p log p| <= 1/e
    assert torch.all(dz.abs() <= 1 / tau * (2 + math.log(V)) * 1.01)
    assert torch.all(_backward(z, token, got, zero, zero, tau) == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_of_a_masked_target_is_zero_there(dtype):
    _build()
    V = 5003
    z = torch.randn((3, V), generator=_gen(23), device="cuda").to(dtype)
    z[0, 5] = -float("inf")
    z[1, 10:] = -float("inf")
    z[2, 4000] = -float("inf")
    token = torch.tensor([5, 4999, 4001], dtype=torch.int32, device="cuda")
    got = _forward(z, token, 0)
    assert float(got["logp"][0]) == float(got["logp"][1]) == -float("inf")
    g, h = torch.full((3,), 2.0, device="cuda"), torch.full((3,), 0.5, device="cuda")
    dz = _backward(z, token, got, g, h)
    assert torch.all(dz[torch.isinf(z)] == 0) and torch.isfinite(dz.float()).all()
    assert float(dz[2, 4001]) > 1.9
    # the other logits: log p is off by 2^-23 (|z| + |lse|) <= 2^-18, p and log p + H follow it
    p = torch.softmax(z[0].double(), 0)
    lp = torch.log(p).clamp_min(-1e4)
    ref = -2.0 * p - 0.5 * p * (lp + float(got["entropy"][0]))
    assert torch.all((dz[0].double() - ref).abs() <= (2.0 ** -8 if dtype == torch.bfloat16 else 0) * ref.abs() + 2.0 ** -18 * p * 20)
