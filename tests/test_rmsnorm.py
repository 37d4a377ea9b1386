"""Residual RMSNorm (qad_rmsnorm_fwd / _bwd) against its definition in 64 bits.

Bounds, from the arithmetic (u = 2^-24 for fp32, 2^-8 for bf16): r is one fp32 sum rounded to bf16, so exact;
the mean square adds at most ~100 positive terms in a chain per lane and tree (100 u), rstd halves that and adds a few
units (1e-5 covers it); y is rounded to bf16 once.  The 8-bit outputs are compared bit for bit with the oracle's
activation quantizer applied to the y that the kernel wrote.
"""
import numpy as np
import pytest
import torch

import scale_only_quantization_gb300 as Q
from oracle import quant as OQ
import synth

ACTS = {Q.QAD_ACT_E4M3: Q.QAD_FMT_FP8_ROW, Q.QAD_ACT_INT8: Q.QAD_FMT_W8A8}
EPS = 1e-6


def _lib():
    from scale_only_quantization_gb300 import build
    build.build()
    return Q.lib()


def test_refusals_before_any_launch():
    L = _lib()
    P = 1 << 20
    fwd = lambda **k: L.qad_rmsnorm_fwd(*[{**dict(x=P, res=None, gamma=P, eps=EPS, act=0, r=None, y=P, yh=None, c=None,  # noqa: E731
                                                  s=None, rstd=None, T=4, d=64, ldx=64, ldres=0, st=None), **k}[n]
                                          for n in ("x", "res", "gamma", "eps", "act", "r", "y", "yh", "c", "s", "rstd",
                                                    "T", "d", "ldx", "ldres", "st")])
    bad = Q.QAD_ERR_INVALID_ARG
    assert fwd(T=0, x=None, gamma=None, y=None) == Q.QAD_OK
    assert fwd(T=-1) == bad and fwd(d=0) == bad and fwd(act=3) == bad and fwd(act=-1) == bad
    assert fwd(eps=-1.0) == bad and fwd(eps=float("nan")) == bad
    assert fwd(d=72) == Q.QAD_ERR_UNSUPPORTED and fwd(d=16400) == Q.QAD_ERR_UNSUPPORTED
    assert fwd(x=None) == bad and fwd(x=P + 2) == bad and fwd(gamma=P + 8) == bad and fwd(y=P + 4) == bad
    assert fwd(ldx=56) == bad and fwd(ldx=68) == bad
    assert fwd(res=P, ldres=32) == bad and fwd(res=P + 2, ldres=64) == bad
    assert fwd(y=None) == bad                                       # no output at all
    assert fwd(c=P) == bad and fwd(s=P) == bad and fwd(yh=P) == bad  # quantized outputs without a grid
    assert fwd(act=Q.QAD_ACT_E4M3, c=P) == bad                      # codes without scales
    bwd = lambda **k: L.qad_rmsnorm_bwd(*[{**dict(dy=P, dres=None, r=P, gamma=P, rstd=P, dx=P, dg=None, T=4, d=64,  # noqa: E731
                                                  ldr=64, ws=None, n=0, st=None), **k}[m]
                                          for m in ("dy", "dres", "r", "gamma", "rstd", "dx", "dg", "T", "d", "ldr",
                                                    "ws", "n", "st")])
    assert bwd(T=0) == Q.QAD_OK and bwd(T=-1) == bad and bwd(d=24) == Q.QAD_ERR_UNSUPPORTED
    assert bwd(dy=None) == bad and bwd(dx=P + 2) == bad and bwd(ldr=60) == bad and bwd(dres=P + 2) == bad
    assert bwd(dg=P) == bad and bwd(dg=P, ws=P + 16, n=1 << 20) == bad
    need = Q.qad_rmsnorm_workspace_bytes(4, 64)
    assert need > 0 and bwd(dg=P, ws=P, n=need - 1) == Q.QAD_ERR_WORKSPACE
    assert Q.qad_rmsnorm_workspace_bytes(4, 24) == 0 and Q.qad_rmsnorm_workspace_bytes(-1, 64) == 0


def _run(T, d, act, res=True, ldx=None, ldres=None, seed=0, inplace=False, x=None, scale_out=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ldx, ldres = ldx or d, ldres or d
    bf = torch.bfloat16
    if x is None:
        x = torch.randn((T, ldx), generator=g, device="cuda").to(bf)
    r_in = (3 * torch.randn((T, ldres), generator=g, device="cuda")).to(bf) if res else None
    gamma = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(bf)
    nan = float("nan")
    o = dict(y=torch.full((T, d), nan, dtype=bf, device="cuda"), rstd=torch.full((T,), nan, device="cuda"))
    if act:
        o.update(y_hat=torch.full((T, d), nan, dtype=bf, device="cuda"), scale=torch.full((T,), nan, device="cuda"),
                 codes=torch.zeros((T, d), dtype=torch.uint8, device="cuda"))
    res_copy = r_in.clone() if res else None
    o["r"] = r_in if inplace else torch.full((T, d), nan, dtype=bf, device="cuda")
    Q.qad_rmsnorm_fwd(x, r_in, gamma, EPS, act, o["r"], o["y"], o.get("y_hat"), o.get("codes"), o.get("scale"),
                      o["rstd"], T, d, ldx, ldres)
    torch.cuda.synchronize()
    return x[:, :d], (res_copy[:, :d] if res else None), gamma, o


def _check(x, res, gamma, o, act):
    r = x.double() if res is None else (x.float() + res.float()).to(torch.bfloat16).double()
    assert torch.equal(o["r"][:, : x.shape[1]].double(), r)
    rstd = (r.square().mean(1) + EPS).rsqrt()
    assert torch.all((o["rstd"].double() - rstd).abs() <= 1e-5 * rstd)
    y = r * rstd[:, None] * gamma.double()
    assert torch.all((o["y"].double() - y).abs() <= (2.0 ** -8 + 2e-5) * y.abs() + 1e-38)
    if not act:
        return
    fmt, yb = ACTS[act], OQ.bf16_to_f64(synth.to_numpy_bits(o["y"]))
    qmax = 448.0 if act == Q.QAD_ACT_E4M3 else 127.0
    s = (np.abs(yb).max(axis=1).astype(np.float32) / np.float32(qmax)).astype(np.float32)
    assert np.array_equal(synth.to_numpy(o["scale"]), s)
    yh = OQ.fakequant_act(fmt, yb)
    assert np.array_equal(synth.to_numpy_bits(o["y_hat"]), OQ.f64_to_bf16_bits(yh))
    # codes stand for the same values: code * scale rounds to y_hat
    c = o["codes"]
    val = c.view(torch.float8_e4m3fn).float() if act == Q.QAD_ACT_E4M3 else c.view(torch.int8).float()
    assert torch.equal((val * o["scale"][:, None]).to(torch.bfloat16), o["y_hat"])


@pytest.mark.gpu
@pytest.mark.parametrize("act", [Q.QAD_ACT_NONE, Q.QAD_ACT_E4M3, Q.QAD_ACT_INT8])
@pytest.mark.parametrize("T, d", [(1, 16), (1, 2048), (3, 272), (5, 256), (7, 512), (130, 2064), (33, 2880), (2, 4096),
                                  (9, 4112), (3, 8192), (2, 8208), (2, 16384), (1000, 48)])
def test_forward_against_64_bits(T, d, act):
    _lib()
    _check(*_run(T, d, act, seed=T + d), act)


@pytest.mark.gpu
@pytest.mark.parametrize("act", [Q.QAD_ACT_NONE, Q.QAD_ACT_E4M3])
def test_forward_strides_without_residual_and_in_place(act):
    _lib()
    _check(*_run(37, 272, act, ldx=560, ldres=288), act)
    _check(*_run(37, 2048, act, res=False, ldx=2056), act)
    _check(*_run(37, 2048, act, inplace=True), act)


@pytest.mark.gpu
@pytest.mark.parametrize("act", [Q.QAD_ACT_E4M3, Q.QAD_ACT_INT8])
def test_forward_of_zero_rows_tiny_rows_and_large_rows(act):
    """A row of zeros gives zeros and scale 0; rows at the ends of bf16's range stay finite."""
    _lib()
    d = 256
    x = torch.randn((4, d), device="cuda").to(torch.bfloat16)
    x[0] = 0
    x[1] *= 2.0 ** -60
    x[2] *= 2.0 ** 60
    x, res, gamma, o = _run(4, d, act, res=False, x=x)
    assert torch.all(o["y"][0] == 0) and float(o["scale"][0]) == 0 and torch.all(o["y_hat"][0] == 0)
    _check(x, res, gamma, o, act)


@pytest.mark.gpu
def test_forward_nan_and_inf_stay_in_their_rows():
    _lib()
    x = torch.randn((6, 512), device="cuda").to(torch.bfloat16)
    clean = _run(6, 512, Q.QAD_ACT_E4M3, res=False, x=x.clone())[3]
    x[2, 17] = float("nan")
    x[4, 3] = float("inf")
    o = _run(6, 512, Q.QAD_ACT_E4M3, res=False, x=x)[3]
    for i in (0, 1, 3, 5):
        for n in ("y", "y_hat", "codes", "scale", "rstd"):
            assert torch.equal(o[n][i], clean[n][i])
    assert torch.isnan(o["y"][2]).all()


def _bwd(T, d, dres, seed, ldr=None, dgamma=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ldr = ldr or d
    bf = torch.bfloat16
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    r, dy = (2 * rand(T, ldr)).to(bf), rand(T, d).to(bf)
    e = rand(T, d).to(bf) if dres else None
    gamma = (1 + 0.2 * rand(d)).to(bf)
    rstd = (r[:, :d].double().square().mean(1) + EPS).rsqrt().float()
    dx = torch.full((T, d), float("nan"), dtype=bf, device="cuda")
    dg = torch.full((d,), float("nan"), device="cuda") if dgamma else None
    ws = torch.empty(Q.qad_rmsnorm_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    Q.qad_rmsnorm_bwd(dy, e, r, gamma, rstd, dx, dg, T, d, ldr, ws if dgamma else None)
    torch.cuda.synchronize()
    return r[:, :d], dy, e, gamma, rstd, dx, dg


@pytest.mark.gpu
@pytest.mark.parametrize("dres", [False, True])
@pytest.mark.parametrize("T, d", [(1, 16), (1, 2048), (5, 272), (1215, 256), (1300, 512), (2500, 1040), (61, 2880),
                                  (17, 4096), (9, 8192), (5, 16384), (20000, 64)])
def test_backward_against_64_bits(T, d, dres):
    """dx: a handful of fp32 roundings of terms of the sizes below, then one bf16 rounding; dgamma: fp32 sums of T
    terms over up to 1216 groups."""
    _lib()
    r, dy, e, gamma, rstd, dx, dg = _bwd(T, d, dres, seed=T + d)
    r, dy, gamma, rstd = r.double(), dy.double(), gamma.double(), rstd.double()[:, None]
    n, dn = r * rstd, dy * gamma
    ref = rstd * (dn - n * (dn * n).mean(1, keepdim=True))
    size = rstd * (dn.abs() + n.abs() * (dn * n).abs().mean(1, keepdim=True))
    if dres:
        ref, size = ref + e.double(), size + e.double().abs()
    assert torch.all((dx.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2e-5 * size)
    terms = dy * n
    assert torch.all((dg.double() - terms.sum(0)).abs() <= 2e-5 * terms.abs().sum(0))


@pytest.mark.gpu
def test_backward_strided_without_norm_weight_gradient_and_repeatable():
    _lib()
    a = _bwd(300, 2048, True, seed=1, ldr=2080)
    b = _bwd(300, 2048, True, seed=1, ldr=2080)
    c = _bwd(300, 2048, True, seed=1, ldr=2080, dgamma=False)
    assert torch.equal(a[5], b[5]) and torch.equal(a[6], b[6]) and torch.equal(a[5], c[5])


@pytest.mark.gpu
def test_backward_against_differences():
    """Directional derivatives of the 64-bit forward: <dy, y(r + h v) - y(r - h v)> / 2h = <dx, v> up to the bf16
    rounding of dx (2^-8 |dx| . |v|) and the differences' own error (h^2)."""
    _lib()
    r, dy, _, gamma, rstd, dx, dg = _bwd(4, 256, False, seed=5)
    r, dy, gamma = r.double(), dy.double(), gamma.double()
    y = lambda a, b: a * (a.square().mean(1, keepdim=True) + EPS).rsqrt() * b  # noqa: E731
    h = 1e-4
    for seed in range(3):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        v = torch.randn(r.shape, generator=g, device="cuda", dtype=torch.float64)
        num = (dy * (y(r + h * v, gamma) - y(r - h * v, gamma))).sum() / (2 * h)
        assert abs(float(num - (dx.double() * v).sum())) <= float(2.0 ** -8 * (dx.double() * v).abs().sum()) + 1e-5
        u = v[0]
        num = (dy * (y(r, gamma + h * u) - y(r, gamma - h * u))).sum() / (2 * h)
        assert abs(float(num - (dg.double() * u).sum())) <= 1e-4 * float((dg.double() * u).abs().sum()) + 1e-6


@pytest.mark.gpu
def test_norm_feeds_the_layer_quantizer():
    """The fused codes are those that the fp8 layer makes of the same y: its per-token scales and routed codes."""
    _lib()
    inp = synth.make_inputs(synth.workload("tiny_nvfp4", fmt=synth.FMT_FP8_ROW), seed=2, device="cuda")
    T, d, F, E, k = (inp[n] for n in ("T", "d", "F", "E", "topk"))
    _, _, _, o = _run(T, d, Q.QAD_ACT_E4M3, seed=11)
    s = Q.shape(T, d, F, E, k, Q.QAD_FMT_FP8_ROW, Q.QAD_FLAG_NATIVE_FP8)
    ws = torch.empty(Q.qad_moe_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    out = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    Q.qad_moe_fwd(s, o["y"], inp["topk_idx"], inp["topk_w"], inp["w13"], inp["s13"], inp["w2"], inp["s2"], out, ws)
    assert Q.qad_check_device_error(ws) == 0
    assert torch.equal(Q.workspace_view(ws, s, "A_SCALE", torch.float32), o["scale"])
    row_of = Q.workspace_view(ws, s, "ROW_OF", torch.int32).view(T, k)
    codes = Q.workspace_view(ws, s, "A1_CODES", torch.uint8).view(-1, d)
    assert torch.equal(codes[row_of[:, 0].long()], o["codes"])


@pytest.mark.gpu
def test_on_another_stream():
    _lib()
    st = torch.cuda.Stream()
    x = torch.randn((64, 256), device="cuda").to(torch.bfloat16)
    gamma = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    torch.cuda.synchronize()
    Q.qad_rmsnorm_fwd(x, None, gamma, EPS, 0, None, y, None, None, None, None, 64, 256, 256, 0, stream=st)
    st.synchronize()
    Q.qad_rmsnorm_fwd(x, None, gamma, EPS, 0, None, y2, None, None, None, None, 64, 256, 256, 0)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)


@pytest.mark.gpu
def test_no_rows_give_a_zero_weight_gradient():
    _lib()
    e = torch.empty(0, device="cuda")
    dg = torch.full((64,), float("nan"), device="cuda")
    Q.qad_rmsnorm_bwd(e, None, e, e, e, e, dg, 0, 64, 64)
    torch.cuda.synchronize()
    assert torch.all(dg == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [256, 272, 2048, 2880, 4096])
def test_statistics_have_the_unfused_bits(d):
    """rstd and y are those of elementary fp32 operations, bit for bit: 128 chains of squares (element i in chain i %
    128), the four chains of a group one after the other, the 32 groups pairwise, then one product with 1 / d, one root,
    one reciprocal and two products."""
    _lib()
    x, res, gamma, o = _run(200, d, 0, seed=d)
    r = (x.float() + res.float()).to(torch.bfloat16).float()
    sq = torch.zeros((200, -(-d // 128) * 128), device="cuda")
    sq[:, :d] = r * r
    chains = torch.zeros((200, 128), device="cuda")
    for part in sq.split(128, dim=1):
        chains = chains + part
    c = chains.view(200, 32, 4)
    s = ((c[:, :, 0] + c[:, :, 1]) + c[:, :, 2]) + c[:, :, 3]
    while s.shape[1] > 1:
        s = s[:, 0::2] + s[:, 1::2]
    inv = torch.tensor(1.0, device="cuda") / d
    rstd = 1 / torch.sqrt(s[:, 0] * inv + EPS)
    y = (r * rstd[:, None] * gamma.float()).to(torch.bfloat16)
    assert torch.equal(o["rstd"], rstd) and torch.equal(o["y"], y)


@pytest.mark.gpu
@pytest.mark.parametrize("act", [Q.QAD_ACT_E4M3, Q.QAD_ACT_INT8])
@pytest.mark.parametrize("d", [48, 512, 1024, 2048, 4112, 8208])
def test_nan_and_infinity_reach_the_8bit_outputs(d, act):
    """A row whose y holds a NaN has no 8-bit form: scale NaN, and with it every y_hat and E4M3 code; an infinite y
    makes the scale infinite and its own code NaN.  Rows beside it keep their bits."""
    _lib()
    x = torch.randn((7, d), device="cuda").to(torch.bfloat16)
    clean = _run(7, d, act, res=False, x=x.clone())[3]
    x[2, d // 3] = float("nan")
    x[4, d - 1] = float("inf")
    x[5, 0] = -float("inf")
    o = _run(7, d, act, res=False, x=x)[3]
    for i in (0, 1, 3, 6):
        for n in ("y", "y_hat", "codes", "scale", "rstd"):
            assert torch.equal(o[n][i], clean[n][i])
    for i in (2, 4, 5):
        assert torch.isnan(o["y"][i]).any()
        assert torch.isnan(o["scale"][i]) and torch.isnan(o["y_hat"][i]).all()
        if act == Q.QAD_ACT_E4M3:
            assert torch.isnan(o["codes"][i].view(torch.float8_e4m3fn).float()).all()
    # finite r, a norm weight that carries y past bf16's range
    x = torch.ones((2, d), device="cuda", dtype=torch.bfloat16)
    x[1, 5] = 2.0
    gamma = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    gamma[5] = 3.3e38
    y, yh = torch.empty_like(x), torch.empty_like(x)
    codes, scale = torch.empty((2, d), dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
    Q.qad_rmsnorm_fwd(x, None, gamma, EPS, act, None, y, yh, codes, scale, None, 2, d, d, d)
    torch.cuda.synchronize()
    assert torch.isfinite(y[0]).all() and torch.isfinite(scale[0]) and torch.isfinite(yh[0, 0])
    assert torch.isinf(y[1, 5]) and torch.isinf(scale[1]) and torch.isnan(yh[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [48, 1024, 2048, 4112, 8208])
def test_no_epsilon(d):
    """eps = 0 (or one far below the row): a row of zeros gives y = 0, rows whose squares leave fp32's range at the
    bottom keep their norm, down to where 1 / rms itself does; the backward of such rows is finite."""
    _lib()
    bf = torch.bfloat16
    x = torch.randn((6, d), device="cuda").to(bf)
    x[0] = 0
    for i, e in ((1, -50), (2, -70), (3, -100), (4, 70)):
        x[i] = (x[i].float() * 2.0 ** e).to(bf)
    gamma = (1 + 0.2 * torch.randn(d, device="cuda")).to(bf)
    for eps in (0.0, 1e-38):
        y, rstd, scale = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
        codes = torch.empty((6, d), dtype=torch.uint8, device="cuda")
        Q.qad_rmsnorm_fwd(x, None, gamma, eps, Q.QAD_ACT_E4M3, None, y, None, codes, scale, rstd, 6, d, d, d)
        torch.cuda.synchronize()
        assert torch.all(y[0] == 0) and float(scale[0]) == 0 and torch.all(codes[0] & 0x7F == 0)
        assert torch.isfinite(rstd).all()
        eps32 = float(torch.tensor(eps))
        want = (x.double().square().mean(1) + eps32).rsqrt()
        rows = slice(1, 6) if eps == 0 else slice(0, 6)
        assert torch.all((rstd.double() - want).abs()[rows] <= 1e-5 * want[rows])
        ref = x.double() * torch.where(torch.isinf(want), 0.0, want)[:, None] * gamma.double()
        assert torch.all((y.double() - ref).abs() <= (2.0 ** -8 + 2e-5) * ref.abs() + 1e-38)
        dy, dx = torch.randn((6, d), device="cuda").to(bf), torch.empty_like(x)
        Q.qad_rmsnorm_bwd(dy, None, x, gamma, rstd, dx, None, 6, d, d)
        torch.cuda.synchronize()
        assert torch.isfinite(dx).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T, d, row", [(6000, 528, 4000), (6000, 1040, 5), (3000, 4096, 2999), (700, 2880, 0)])
def test_a_copy_that_never_comes_is_reported(T, d, row):
    """The backward's ring with one row's copies left out: its wait gives up (0.5 ms here), the rows of its block and
    the weight gradient are NaN, the error word says timeout, other rows have their bits, and the next call on the same
    workspace is clean."""
    _lib()
    clean = _bwd(T, d, True, seed=T)
    r, dy, e, gamma, rstd = clean[:5]
    ws = torch.full((Q.qad_rmsnorm_workspace_bytes(T, d),), 0xFF, dtype=torch.uint8, device="cuda")

    def call(with_ws=True):
        dx = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
        dg = torch.zeros(d, device="cuda") if with_ws else None
        Q.qad_rmsnorm_bwd(dy, e, r, gamma, rstd, dx, dg, T, d, d, ws if with_ws else None)
        return (Q.qad_check_device_error(ws) if with_ws else torch.cuda.synchronize()), dx, dg

    with pytest.raises(Q.QADError):
        Q.qad_debug_stuck_copy(0, -1)
    Q.qad_debug_stuck_copy(row, 1_000_000)
    try:
        err, dx, dg = call()
        _, dx2, _ = call(with_ws=False)
    finally:
        Q.qad_debug_stuck_copy(-1)
    assert err == Q.QAD_DEV_TIMEOUT and torch.isnan(dg).all()
    for out in (dx, dx2):
        gone = torch.isnan(out).any(1)
        assert gone[row] and torch.isnan(out[row]).all()
        assert int(gone.sum()) <= -(-T // 304) + 8 and torch.equal(out[~gone], clean[5][~gone])
    err, dx, dg = call()
    assert err == 0 and torch.equal(dx, clean[5]) and torch.equal(dg, clean[6])


@pytest.mark.gpu
@pytest.mark.parametrize("dres", [False, True])
@pytest.mark.parametrize("T, d", [(12000, 528), (12000, 768), (12000, 1024), (6000, 1040), (6000, 2048), (3000, 2064), (3000, 2880), (3000, 4096),
                                  (3000, 4112), (3000, 8208)])
def test_backward_of_many_rows(T, d, dres):
    """Nine rows or more for every group of warps: the ring's stages are filled again and its phases turn over.  Bounds
    as above, and a relative one per row, which bf16's rounding takes half of."""
    _lib()
    r, dy, e, gamma, rstd, dx, dg = _bwd(T, d, dres, seed=T + d)
    r, dy, gamma, rstd = r.double(), dy.double(), gamma.double(), rstd.double()[:, None]
    n, dn = r * rstd, dy * gamma
    ref = rstd * (dn - n * (dn * n).mean(1, keepdim=True))
    size = rstd * (dn.abs() + n.abs() * (dn * n).abs().mean(1, keepdim=True))
    if dres:
        ref, size = ref + e.double(), size + e.double().abs()
    assert torch.all((dx.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2e-5 * size)
    assert torch.all((dx.double() - ref).norm(dim=1) <= 2.0 ** -7 * ref.norm(dim=1))
    terms = dy * n
    assert torch.all((dg.double() - terms.sum(0)).abs() <= 2e-5 * terms.abs().sum(0))


@pytest.mark.gpu
@pytest.mark.parametrize("T, d", [(1000, 256), (6000, 1024), (3000, 4096), (700, 8192)])
def test_backward_in_place(T, d):
    """dx may be dy or dres: the same bits as in a buffer of its own."""
    _lib()
    r, dy, e, gamma, rstd, dx, dg = _bwd(T, d, True, seed=T)
    for which in (0, 1):
        a = [dy.clone(), e.clone()]
        dg2 = torch.empty_like(dg)
        ws = torch.empty(Q.qad_rmsnorm_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
        Q.qad_rmsnorm_bwd(a[0], a[1], r, gamma, rstd, a[which], dg2, T, d, d, ws)
        assert Q.qad_check_device_error(ws) == 0
        assert torch.equal(a[which], dx) and torch.equal(dg2, dg) and torch.equal(a[1 - which], (e, dy)[which])
