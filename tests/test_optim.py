"""Norm, clipping and AdamW over lists of tensors against 64 bits, and their refusals.

Tolerances: the norm adds squares of 16 values in fp32 (17 roundings) and the rest in 64 bits: sqrt halves the error,
and the result is rounded: (9 + 1) * 2^-24.  The clip factor divides and adds once more (4 * 2^-24 in all with the norm
given), a product rounds once.  AdamW: m and v three roundings of terms of their own size; the step's quotient about ten.
"""
import ctypes
import math

import pytest
import torch

import scale_only_quantization_gb300 as Q

U24 = 2.0 ** -24
SIZES = [0, 1, 3, 7, 1023, 1024, 1025, 16384, 16385, 70001, 0, 300000]


def _build():
    from scale_only_quantization_gb300 import build
    build.build()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _grads(sizes, seed=0, kinds=(torch.float32, torch.float32, torch.bfloat16)):
    g = _gen(seed)
    return [(torch.randn(n, generator=g, device="cuda") * 10.0 ** (i % 5 - 3)).to(kinds[i % len(kinds)])
            for i, n in enumerate(sizes)]


def _ws():
    return torch.full((Q.qad_grad_norm_workspace_bytes(),), 0xAB, dtype=torch.uint8, device="cuda")


def _norm(grads, ws=None):
    out = torch.full((1,), -1.0, device="cuda")
    Q.qad_grad_norm(grads, out, _ws() if ws is None else ws)
    return out


def _norm64(grads):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in grads))


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [SIZES, [5], [0], [], [1] * 700, [1000] * 481 + [50000], [4_000_001, 3], [0] * 500 + [9]])
def test_norm(sizes):
    _build()
    grads = _grads(sizes, len(sizes))
    a, b = _norm(grads), _norm(grads)
    ref = _norm64(grads)
    assert abs(float(a) - ref) <= 10 * U24 * ref
    assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1e-44, 1e-30, 1e-16, 1e16, 1e25, 3e38])
def test_norm_of_values_whose_squares_leave_the_range(size):
    _build()
    grads = [torch.full((777,), size, device="cuda"), torch.full((3,), -size, device="cuda"), torch.zeros(40, device="cuda")]
    ref = _norm64(grads)
    got = float(_norm(grads))
    if ref > torch.finfo(torch.float32).max:
        assert got == math.inf
    else:
        assert abs(got - ref) <= 10 * U24 * ref + 2.0 ** -150
    mixed = [torch.full((5000,), 1e-25, device="cuda"), torch.tensor([1e22, 1.0], device="cuda")]
    assert abs(float(_norm(mixed)) - 1e22) <= 10 * U24 * 1e22


@pytest.mark.gpu
def test_norm_that_is_not_finite():
    _build()
    for bad in (float("inf"), float("-inf"), float("nan")):
        for dtype in (torch.float32, torch.bfloat16):
            grads = _grads([1000, 70001], 1, (dtype,))
            grads[1][69999] = bad
            got = float(_norm(grads))
            assert math.isnan(got) if bad != bad else got == math.inf


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("sizes", [SIZES, [3], [2000] * 500, []])
def test_clip(sizes, in_place):
    _build()
    for max_norm in (0.0, 1e-3, 1.0, 1e9):
        grads = _grads(sizes, 2)
        keep = [g.clone() for g in grads]
        norm = _norm(grads)
        out = grads if in_place else [torch.full_like(g, 5.0) for g in grads]
        Q.qad_grad_clip(grads, None if in_place else out, norm, max_norm)
        f = min(1.0, max_norm / (float(norm) + 1e-6))
        for g, k, o in zip(grads, keep, out):
            half = U24 if g.dtype == torch.float32 else 2.0 ** -8
            assert torch.all((o.double() - k.double() * f).abs() <= (4 * U24 + half) * k.double().abs() * f + 1e-44)
            if f == 1.0:
                assert torch.equal(o, k)
            if not in_place:
                assert torch.equal(g, k)


@pytest.mark.gpu
def test_clip_by_a_norm_that_is_not_finite():
    _build()
    g = _grads([100], 3)
    out = [torch.empty_like(g[0])]
    Q.qad_grad_clip(g, out, torch.full((1,), float("nan"), device="cuda"), 1.0)
    assert torch.isnan(out[0]).all()
    Q.qad_grad_clip(g, out, torch.full((1,), float("inf"), device="cuda"), 1.0)
    assert torch.all(out[0] == 0)


def _state(sizes, seed, kinds=(torch.float32, torch.float32, torch.bfloat16)):
    g = _gen(seed)
    rand = lambda n: torch.rand(n, generator=g, device="cuda")  # noqa: E731
    grads = _grads(sizes, seed + 1, kinds)
    return dict(p=[0.01 * (0.5 + rand(n)) for n in sizes], g=grads, m=[t.float() * rand(t.numel()) for t in grads],
                v=[t.float().square() * rand(t.numel()) for t in grads],
                lr=1e-4 * (0.5 + rand(max(1, len(sizes))))[:len(sizes)],
                steps=torch.full((1,), 4, dtype=torch.int64, device="cuda"))


def _step(s, norm=None, max_norm=0.0, b1=0.9, b2=0.95, eps=1e-8, decay=0.1, floor=-math.inf, ws=None):
    Q.qad_adamw_step(s["p"], s["g"], s["m"], s["v"], s["lr"], b1, b2, eps, decay, floor, norm, max_norm, s["steps"],
                     _ws() if ws is None else ws)


def _check_step(before, after, c, b1=0.9, b2=0.95, eps=1e-8, decay=0.1, floor=-math.inf):
    t = int(before["steps"]) + 1
    assert int(after["steps"]) == t
    for i, g in enumerate(before["g"]):
        p, m, v, g = (x.double() for x in (before["p"][i], before["m"][i], before["v"][i], g))
        lr = float(before["lr"][i])
        m1, v1 = b1 * m + (1 - b1) * c * g, b2 * v + (1 - b2) * (c * g) ** 2
        dm = 8 * U24 * (b1 * m.abs() + (1 - b1) * (c * g).abs()) + 1e-44
        assert torch.all((after["m"][i].double() - m1).abs() <= dm)
        assert torch.all((after["v"][i].double() - v1).abs() <= 16 * U24 * v1 + 1e-43)
        step = lr * m1 / (1 - b1 ** t) / ((v1 / (1 - b2 ** t)).sqrt() + eps)
        ref = (p - lr * decay * p - step).clamp_min(floor)
        slack = lr / (1 - b1 ** t) * dm / ((v1 / (1 - b2 ** t)).sqrt() + eps)
        assert torch.all((after["p"][i].double() - ref).abs() <= 3 * U24 * p.abs() + 24 * U24 * step.abs() + 2 * slack + 1e-44)


def _copy(s):
    return {k: [x.clone() for x in v] if isinstance(v, list) else v.clone() for k, v in s.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [SIZES, [1], [], [300] * 485, [0, 0]])
@pytest.mark.parametrize("clip", [None, 0.01, 1e9])
def test_adamw(sizes, clip):
    _build()
    s = _state(sizes, 5)
    before = _copy(s)
    norm = None if clip is None else _norm(s["g"])
    _step(s, norm, clip or 0.0, floor=0.0075)
    c = 1.0 if clip is None else min(1.0, clip / (float(norm) + 1e-6))
    _check_step(before, s, c, floor=0.0075)
    assert all(torch.equal(a, b) for a, b in zip(s["g"], before["g"]))


@pytest.mark.gpu
def test_adamw_from_nothing_and_without_a_denominator():
    """The first step, beta 0, zero gradients with eps: 0 / eps; the parameters move by nothing but their decay."""
    _build()
    s = _state([1000, 5], 6)
    s["steps"].zero_()
    for i in range(2):
        s["m"][i].zero_()
        s["v"][i].zero_()
    s["g"][1].zero_()
    before = _copy(s)
    _step(s, b1=0.0, b2=0.0)
    _check_step(before, s, 1.0, b1=0.0, b2=0.0)
    assert torch.all((s["p"][1] - before["p"][1] * (1 - before["lr"][1] * 0.1)).abs() <= 3 * U24 * before["p"][1])


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_norm_that_is_not_finite_leaves_everything(bad):
    _build()
    s = _state(SIZES, 7)
    before = _copy(s)
    _step(s, torch.full((1,), bad, device="cuda"), 1.0)
    assert int(s["steps"]) == 4
    for k in ("p", "m", "v"):
        assert all(torch.equal(a, b) for a, b in zip(s[k], before[k]))
    _step(s, torch.full((1,), 1.0, device="cuda"), 1.0)  # the next one counts
    assert int(s["steps"]) == 5


@pytest.mark.gpu
def test_a_nan_gradient_without_a_norm_stays_one():
    _build()
    s = _state([50, 60], 8, (torch.float32,))
    s["g"][0][7] = float("nan")
    _step(s, floor=0.001)
    assert torch.isnan(s["p"][0][7]) and int(torch.isnan(s["p"][0]).sum()) == 1 and torch.isfinite(s["p"][1]).all()


@pytest.mark.gpu
def test_captured_step_reads_rates_and_gradients_again():
    _build()
    s = _state([5000, 33, 70000], 9)
    ws, norm = _ws(), torch.zeros(1, device="cuda")
    lists = [Q.tensor_list(s[k]) for k in ("p", "g", "m", "v")]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        Q.qad_grad_norm(lists[1], norm, ws)
        Q.qad_adamw_step(lists[0], lists[1], lists[2], lists[3], s["lr"], 0.9, 0.95, 1e-8, 0.1, -math.inf, norm, 0.5,
                         s["steps"], ws)
    for k in range(3):
        s["lr"].mul_(0.5)
        for g in s["g"]:
            g.mul_(0.25)
        before = _copy(s)
        graph.replay()
        torch.cuda.synchronize()
        _check_step(before, s, min(1.0, 0.5 / (float(norm) + 1e-6)))


@pytest.mark.gpu
def test_optimizer():
    """QADAdamW against torch.optim.AdamW behind clip_grad_norm_, in 64 bits: 20 steps, groups with rates and floors of
    their own, a saved and loaded state in between."""
    from scale_only_quantization_gb300.autograd import QADAdamW
    _build()
    g = _gen(10)
    init = [torch.rand(n, generator=g, device="cuda") + 0.5 for n in (1000, 7, 40000)]
    ps = [torch.nn.Parameter(t.clone()) for t in init]
    rs = [torch.nn.Parameter(t.double()) for t in init]
    make = lambda x: [dict(params=x[:1], lr=1e-2), dict(params=x[1:], lr=3e-3, weight_decay=0.1)]  # noqa: E731
    opt = QADAdamW(make(ps), max_norm=0.5)
    ref = torch.optim.AdamW(make(rs), betas=(0.9, 0.95), weight_decay=0.0)
    for k in range(20):
        for p, r in zip(ps, rs):
            r.grad = torch.randn(p.shape, generator=g, device="cuda", dtype=torch.float64) * 0.1
            p.grad = r.grad.float()
        total = torch.nn.utils.clip_grad_norm_(rs, 0.5)
        opt.param_groups[0]["lr"] = ref.param_groups[0]["lr"] = 1e-2 / (1 + k)
        opt.step()
        ref.step()
        assert abs(float(opt.last_norm) - float(total)) <= 1e-6 * float(total)
        if k == 10:
            state = opt.state_dict()
            opt = QADAdamW(make(ps), max_norm=0.5)
            opt.load_state_dict(state)
    assert int(opt.state[ps[2]]["step"]) == 20
    for p, r in zip(ps, rs):  # 20 steps, each with errors of a few 2^-24 of the step (1e-2 at most) and of p
        assert torch.all((p.detach().double() - r.detach()).abs() <= 20 * (4 * U24 * 2 + 64 * U24 * 1e-2))
    floored = QADAdamW([torch.nn.Parameter(torch.full((5,), 1e-3, device="cuda"))], lr=1.0, floor=1e-4, max_norm=None)
    floored.param_groups[0]["params"][0].grad = torch.ones(5, device="cuda")
    floored.step()
    assert torch.all(floored.param_groups[0]["params"][0] == torch.tensor(1e-4, device="cuda"))
    with pytest.raises(ValueError):
        ps[0].grad = None
        opt.step()
    with pytest.raises(ValueError):
        bad = QADAdamW([torch.nn.Parameter(torch.ones(3, device="cuda", dtype=torch.bfloat16))])
        bad.param_groups[0]["params"][0].grad = torch.ones(3, device="cuda", dtype=torch.bfloat16)
        bad.step()


@pytest.mark.gpu
def test_optimizer_settings_that_part_and_groups_that_join():
    """Two groups step together, then one's decay changes, then a third joins: each counts its own steps, as
    torch.optim.AdamW does."""
    from scale_only_quantization_gb300.autograd import QADAdamW
    _build()
    g = _gen(12)
    init = [torch.rand(n, generator=g, device="cuda") + 0.5 for n in (100, 33, 257)]
    ps = [torch.nn.Parameter(t.clone()) for t in init]
    rs = [torch.nn.Parameter(t.double()) for t in init]
    make = lambda x: [dict(params=[x[0]], lr=1e-2), dict(params=[x[1]], lr=1e-2)]  # noqa: E731
    opt = QADAdamW(make(ps), max_norm=None)
    ref = torch.optim.AdamW(make(rs), betas=(0.9, 0.95), weight_decay=0.0)
    for k in range(9):
        if k == 3:
            for o in (opt, ref):
                o.param_groups[1]["weight_decay"] = 0.1
        if k == 6:
            opt.add_param_group(dict(params=[ps[2]], lr=1e-2))
            ref.add_param_group(dict(params=[rs[2]], lr=1e-2))
        for p, r in zip(ps, rs):
            r.grad = torch.randn(p.shape, generator=g, device="cuda", dtype=torch.float64) * 0.1
            p.grad = r.grad.float()
        opt.step()
        ref.step()
    assert [int(opt.state[p]["step"]) for p in ps] == [9, 9, 3]
    for p, r in zip(ps, rs):  # 9 steps, each with errors of a few 2^-24 of the step (1e-2) and of p
        assert torch.all((p.detach().double() - r.detach()).abs() <= 9 * (4 * U24 * 2 + 64 * U24 * 1e-2))


@pytest.mark.gpu
def test_rollout_teacher_and_step_together():
    """The operators as an on-policy step uses them: the quantized model writes, the unquantized one reads, the scales
    move; every scale gets a finite gradient and stays at or above the floor."""
    import os
    import sys
    _build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import qad_step
    m = qad_step.Model(Q.QAD_FMT_NVFP4, d=128, F=128, E=4, layers=1, vocab=1001)
    g = _gen(11)
    start = torch.randint(0, 1001, (9,), generator=g, device="cuda")
    tokens, logp = m.rollout(start, 5, g)
    assert tokens.shape == (9, 5) and logp.shape == (9, 4) and torch.all(logp <= 0) and torch.isfinite(logp).all()
    assert torch.equal(tokens[:, 0], start) and int(tokens.min()) >= 0 and int(tokens.max()) < 1001
    idx, t = m.teacher(tokens.reshape(-1), 16)
    z = m.hidden(tokens.reshape(-1), quantized=False).float() @ m.head.w.float().T
    assert torch.equal(t, torch.topk(z, 16, dim=1).values)
    hist = qad_step.train(Q.QAD_FMT_NVFP4, steps=3, tokens=64, rollout=8, log=None, d=128, F=128, E=4, layers=1, vocab=1001)
    assert len(hist) == 3 and all(x == x and x < 1e3 for h in hist for x in h)


def test_refusals():
    """Checked on the host before anything is launched (no GPU is touched)."""
    _build()
    L = Q.lib()
    P = 1 << 20
    n = Q.qad_grad_norm_workspace_bytes()
    inv = Q.QAD_ERR_INVALID_ARG

    def lst(*items):
        a = (Q.Tensor * max(1, len(items)))()
        for t, it in zip(a, items):
            t.data, t.numel, t.dtype, t.reserved = it
        return a

    ok = lst((P, 8, 0, 0), (P, 4, 1, 0))
    f32 = lst((P, 8, 0, 0), (P, 4, 0, 0))
    for bad in (lst((P + 4, 8, 0, 0)), lst((None, 8, 0, 0)), lst((P, -1, 0, 0)), lst((P, 8, 2, 0)), lst((P, 8, 0, 1))):
        assert L.qad_grad_norm(bad, 1, P, P, n, None) == inv
        assert L.qad_grad_clip(bad, None, 1, P, 1.0, None) == inv
        assert L.qad_adamw_step(bad, ok, f32, f32, 1, P, 0.9, 0.9, 1e-8, 0.0, 0.0, None, 0.0, P, P, n, None) == inv
    assert L.qad_grad_norm(None, 2, P, P, n, None) == inv and L.qad_grad_norm(ok, -1, P, P, n, None) == inv
    assert L.qad_grad_norm(ok, 2, None, P, n, None) == inv and L.qad_grad_norm(ok, 2, P + 2, P, n, None) == inv
    assert L.qad_grad_norm(ok, 2, P, P + 16, n, None) == inv and L.qad_grad_norm(ok, 2, P, None, n, None) == inv
    assert L.qad_grad_norm(ok, 2, P, P, n - 1, None) == Q.QAD_ERR_WORKSPACE
    assert L.qad_grad_norm(lst((P, 1 << 40, 0, 0)), 1, P, P, n, None) == Q.QAD_ERR_UNSUPPORTED
    assert L.qad_grad_clip(ok, f32, 2, P, 1.0, None) == inv                        # other types
    assert L.qad_grad_clip(ok, lst((P, 8, 0, 0), (P, 5, 1, 0)), 2, P, 1.0, None) == inv
    assert L.qad_grad_clip(ok, None, 2, None, 1.0, None) == inv and L.qad_grad_clip(ok, None, 2, P, -1.0, None) == inv
    assert L.qad_grad_clip(ok, None, 2, P, float("nan"), None) == inv
    good = [f32, ok, f32, f32, 2, P, 0.9, 0.95, 1e-8, 0.0, 0.0, P, 1.0, P, P, n, None]
    for i, v in [(0, ok), (2, ok), (3, ok), (0, None), (1, None), (4, -1), (5, None), (5, P + 2), (6, 1.0), (6, -0.1), (7, 1.0),
                 (6, float("nan")), (8, -1.0), (9, -1.0), (10, float("nan")), (11, P + 2), (12, -1.0), (13, None),
                 (13, P + 4), (14, None), (14, P + 128)]:
        args = list(good)
        args[i] = v
        assert L.qad_adamw_step(*args) == inv, (i, v)
    assert L.qad_adamw_step(*good[:15], n - 1, None) == Q.QAD_ERR_WORKSPACE
    with pytest.raises(ValueError):
        Q.tensor_list([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(ValueError):
        Q.tensor_list([torch.zeros((4, 4))[:, :2]])
    three, two = Q.tensor_list([torch.zeros(4)] * 3), Q.tensor_list([torch.zeros(4)] * 2)
    with pytest.raises(ValueError):
        Q.qad_grad_clip(three, two, None, 1.0)
    with pytest.raises(ValueError):
        Q.qad_adamw_step(three, three, two, three, None, 0.9, 0.9, 0.0, 0.0, 0.0, None, 0.0, None, None)
    assert ctypes.sizeof(Q.Tensor) == 24


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [-1, -2, -5, -(1 << 63), (1 << 63) - 1])
def test_a_step_count_below_zero_or_past_the_last_leaves_everything(steps):
    _build()
    s = _state([1000, 7], 13)
    s["steps"].fill_(steps)
    before = _copy(s)
    _step(s, _norm(s["g"]), 1.0)
    assert int(s["steps"]) == steps
    for k in ("p", "m", "v"):
        assert all(torch.equal(a, b) for a, b in zip(s[k], before[k]))


@pytest.mark.gpu
def test_a_large_step_count():
    """The powers of beta are 0 by then."""
    _build()
    s = _state([1000, 7], 14)
    s["steps"].fill_(10 ** 12)
    before = _copy(s)
    _step(s)
    _check_step(before, s, 1.0)


class _NoLaunches:
    """The optimizer's launches replaced by records of what they would have been given."""

    def __init__(self, monkeypatch):
        from scale_only_quantization_gb300 import autograd
        self.norms, self.steps = [], []
        monkeypatch.setattr(autograd, "qad_grad_norm", lambda grads, norm, ws: self.norms.append((grads, norm, ws)))
        monkeypatch.setattr(autograd, "qad_adamw_step", lambda *args: self.steps.append(args))


def _filled(ps):
    for p in ps:
        p.grad = torch.ones_like(p)


def test_optimizer_of_tensors_on_the_host_is_refused(monkeypatch):
    import contextlib
    from scale_only_quantization_gb300.autograd import QADAdamW
    _build()
    calls = _NoLaunches(monkeypatch)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    ps = [torch.nn.Parameter(torch.ones(3))]
    opt = QADAdamW(ps)
    _filled(ps)
    with pytest.raises(ValueError):
        opt.step()
    assert not calls.norms and not calls.steps


@pytest.mark.gpu
def test_optimizer_of_tensors_that_moved_is_refused(monkeypatch):
    """Parameters, moments or gradients that lie elsewhere since the last step: nothing is launched on them."""
    from scale_only_quantization_gb300.autograd import QADAdamW
    _build()
    for moved in ("parameters", "one parameter", "moments", "gradient"):
        ps = [torch.nn.Parameter(torch.ones(n, device="cuda")) for n in (5, 6)]
        opt = QADAdamW(ps)
        _filled(ps)
        opt.step()
        with monkeypatch.context() as m:
            calls = _NoLaunches(m)
            if moved == "parameters":
                for p in ps:
                    p.data = p.data.cpu()
                    p.grad = torch.ones_like(p)
            elif moved == "one parameter":
                ps[1].data = ps[1].data.cpu()
                ps[1].grad = torch.ones_like(ps[1])
            elif moved == "moments":
                state = opt.state_dict()
                opt.load_state_dict(state)
                opt.state[ps[0]]["exp_avg"] = opt.state[ps[0]]["exp_avg"].cpu()
            else:
                keep = ps[1].data
                ps[1].grad = None
                ps[1].data = keep.cpu()
                ps[1].grad = torch.ones(6)
                ps[1].data = keep
            with pytest.raises(ValueError):
                opt.step()
            assert not calls.norms and not calls.steps


@pytest.mark.gpu
def test_rates_are_rewritten_in_place(monkeypatch):
    """A schedule writes new rates where the last step read them, which a captured step reads again."""
    from scale_only_quantization_gb300.autograd import QADAdamW
    _build()
    ps = [torch.nn.Parameter(torch.ones(n, device="cuda")) for n in (5, 6)]
    opt = QADAdamW([dict(params=ps[:1], lr=0.5), dict(params=ps[1:], lr=0.25)])
    _filled(ps)
    calls = _NoLaunches(monkeypatch)
    opt.step()
    rates = calls.steps[0][4]
    assert rates.tolist() == [0.5, 0.25]
    opt.param_groups[1]["lr"] = 0.125
    opt.step()
    assert calls.steps[1][4].data_ptr() == rates.data_ptr() and rates.tolist() == [0.5, 0.125]


@pytest.mark.gpu
def test_a_schedule_does_not_wait_for_the_device():
    from scale_only_quantization_gb300.autograd import QADAdamW
    _build()
    ps = [torch.nn.Parameter(torch.ones(n, device="cuda")) for n in (5, 6)]
    opt = QADAdamW(ps, lr=0.5)
    _filled(ps)
    opt.step()
    torch.cuda.synchronize()
    mode = torch.cuda.get_sync_debug_mode()
    torch.cuda.set_sync_debug_mode("error")
    try:
        for k in range(3):
            opt.param_groups[0]["lr"] = 0.25 / (1 + k)
            opt.step()
    finally:
        torch.cuda.set_sync_debug_mode(mode)
    assert int(opt.state[ps[0]]["step"]) == 4


@pytest.mark.gpu
def test_captured_optimizer_step_under_a_schedule():
    """A captured step() replayed under a schedule equals eager steps under it; a first step, or one whose rates have not
    been written, is not captured."""
    from scale_only_quantization_gb300.autograd import QADAdamW
    _build()
    g = _gen(41)
    init = [torch.rand(n, generator=g, device="cuda") + 0.5 for n in (1000, 7)]
    grads = [torch.randn(n, generator=g, device="cuda") for n in (1000, 7)]
    ps = [[torch.nn.Parameter(t.clone()) for t in init] for _ in range(2)]
    opts = [QADAdamW(p, lr=1e-2) for p in ps]
    for p in ps:
        for q, t in zip(p, grads):
            q.grad = t.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(graph, stream=st):
            opts[0].step()
    with torch.cuda.stream(st):
        opts[0].step()
    opts[1].step()
    torch.cuda.synchronize()
    opts[0].param_groups[0]["lr"] = 5e-3
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(graph, stream=st):
            opts[0].step()
    with torch.cuda.stream(st):
        opts[0].write_rates()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        opts[0].step()
    for k in range(4):
        for o in opts:
            o.param_groups[0]["lr"] = 5e-3 / (1 + k)
        with torch.cuda.stream(st):
            opts[0].write_rates()
            graph.replay()
        opts[1].step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*ps))
    assert int(opts[0].state[ps[0][0]]["step"]) == 5


@pytest.mark.gpu
def test_a_backward_pass_over_parameters_that_moved_is_refused():
    from scale_only_quantization_gb300.autograd import QADAdamW
    _build()
    p = torch.nn.Parameter(torch.full((5,), 2.0, device="cuda"))
    opt = QADAdamW([p])
    p.grad = torch.ones_like(p)
    early = (p * p).sum()
    opt.step()
    with pytest.raises(RuntimeError):
        early.backward()
    p.grad = None
    (p * p).sum().backward()
    assert torch.equal(p.grad, 2 * p.detach())


@pytest.mark.gpu
def test_a_copied_optimizer_goes_on():
    import copy
    import io
    from scale_only_quantization_gb300.autograd import QADAdamW
    _build()
    p = torch.nn.Parameter(torch.linspace(0.5, 1, 100, device="cuda"))
    opt = QADAdamW([p], lr=1e-2, max_norm=0.5)
    p.grad = torch.linspace(-1, 2, 100, device="cuda")
    opt.step()
    file = io.BytesIO()
    torch.save(opt, file)
    file.seek(0)
    others = [copy.deepcopy(opt), torch.load(file, weights_only=False)]
    opt.step()
    for other in others:
        q = other.param_groups[0]["params"][0]
        assert q.data_ptr() != p.data_ptr() and other.max_norm == 0.5
        q.grad = p.grad.clone()
        other.step()
        assert torch.equal(q, p) and int(other.state[q]["step"]) == 2 and torch.equal(other.last_norm, opt.last_norm)


@pytest.mark.gpu
def test_without_clipping_the_norm_is_kept_and_checked():
    from scale_only_quantization_gb300.autograd import QADAdamW
    _build()
    ps = [torch.nn.Parameter(torch.ones(n, device="cuda")) for n in (5, 4)]
    opt = QADAdamW(ps, lr=0.1, max_norm=None)
    _filled(ps)
    opt.step()
    assert float(opt.last_norm) == 3.0
    after = [p.detach().clone() for p in ps]
    assert torch.all((after[0] - 0.9).abs() <= 1e-6)  # lr m / sqrt(v) with m and v of one gradient of 1: not clipped
    for bad in (float("nan"), float("inf")):
        ps[1].grad[2] = bad
        opt.step()
        assert int(opt.state[ps[0]]["step"]) == 1 and all(torch.equal(p, a) for p, a in zip(ps, after))


@pytest.mark.gpu
def test_norm_of_a_large_tensor_behind_many_empty_ones():
    """The tensors that come first do not decide how many blocks the others get: the same time in either order, within
    what launches and noise may differ (one block for all took over a hundred times as long)."""
    _build()
    big, one, none = torch.ones(1 << 26, device="cuda"), torch.ones(1, device="cuda"), torch.empty(0, device="cuda")
    ws, norm = _ws(), torch.zeros(1, device="cuda")

    def spent(tensors):
        grads, best = Q.tensor_list(tensors), math.inf
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            Q.qad_grad_norm(grads, norm, ws)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
            assert abs(float(norm) - 8192.0) <= 8192 * 10 * U24 + 1e-3
        return best

    assert spent([one] + [none] * 500 + [big]) <= 5 * spent([big] + [none] * 500 + [one])


@pytest.mark.gpu
def test_clip_without_a_bound_by_a_norm_that_is_infinite():
    """max_norm is infinite too: the finite gradients become 0 all the same, the others NaN (inf times 0)."""
    _build()
    g = [torch.tensor([1.0, -2.0, float("inf"), 0.0], device="cuda"), torch.ones(9, device="cuda", dtype=torch.bfloat16)]
    Q.qad_grad_clip(g, None, torch.full((1,), float("inf"), device="cuda"), float("inf"))
    assert g[0][[0, 1, 3]].tolist() == [0, 0, 0] and math.isnan(float(g[0][2])) and torch.all(g[1] == 0)
    h = [torch.tensor([1.0, -2.0], device="cuda")]
    Q.qad_grad_clip(h, None, _norm(h), float("inf"))
    assert h[0].tolist() == [1.0, -2.0]
