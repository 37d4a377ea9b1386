"""The layer for a few tokens (qad_moe_few_fwd) against the oracle, and its refusals.

Tolerance, element by element, from what the call may do differently from the oracle's 64-bit sums:
  - fp32 sums of K products: SUM * sum |a w| with SUM = 32 * 2^-24 (K / 16 products of 16 in turn on each of up to 8
    warps, rounding errors of either sign);
  - sigmoid from the fast exponential and reciprocal: H off by 2^-20 of itself;
  - so Z1 and H may round to the neighbouring bf16 value and H's code to the neighbouring code.  Where that can happen
    is found by running the oracle's own steps on gate and up sums moved to the ends of their error intervals; H_hat's
    largest change, times |W2_hat|, is allowed on Y;
  - Y may round to its neighbour (2 half steps, 2^-7 |Y|); out is rounded once (2^-8 |out|; the oracle's is not).
"""
import ctypes

import numpy as np
import pytest
import torch

import scale_only_quantization_gb300 as Q
import synth
from gpu_util import bits, vals
from oracle import moe as OM
from oracle import quant as OQ

SUM = 32 * 2.0 ** -24


def _build():
    from scale_only_quantization_gb300 import build
    build.build()


def _inputs(T, d, F, E, k, fmt, seed=0, routing="uniform"):
    cfg = dict(T=T, d=d, F=F, E=E, topk=k, fmt=fmt, routing=routing)
    return synth.make_inputs(cfg, seed=seed, device="cuda")


def _scales(inp):
    """The scales as the call takes them: deployed ones where the format has them."""
    if inp["fmt"] != Q.QAD_FMT_NVFP4_E4M3:
        return inp["s13"], inp["s2"]
    out = []
    for s in (inp["s13"], inp["s2"]):
        q = torch.empty_like(s)
        Q.qad_nvfp4_deploy_scales(s, q, inp["E"], s.numel() // inp["E"])
        out.append(q)
    return out


def _few(inp, flags=0, out=None, ws=None, w13=None, w2=None):
    s = Q.shape(inp["T"], inp["d"], inp["F"], inp["E"], inp["topk"], inp["fmt"], flags)
    n = Q.qad_moe_few_workspace_bytes(s)
    assert n > 0
    if ws is None:
        ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")  # what it held before does not matter
    if out is None:
        out = torch.full((inp["T"], inp["d"]), float("nan"), dtype=torch.bfloat16, device="cuda")
    s13, s2 = _scales(inp)
    Q.qad_moe_few_fwd(s, inp["x"], inp["topk_idx"], inp["topk_w"], inp["w13"] if w13 is None else w13, s13,
                      inp["w2"] if w2 is None else w2, s2, out, ws)
    return out, ws


def _oracle(inp, quant=True):
    """(out before its last rounding, the bound of the difference)."""
    fmt, F = inp["fmt"], inp["F"]
    x, idx, p = bits(inp["x"]), synth.to_numpy(inp["topk_idx"]), synth.to_numpy(inp["topk_w"]).astype(np.float64)
    fwd = OM.moe_forward(fmt, x, idx, p, bits(inp["w13"]), synth.to_numpy(inp["s13"]), bits(inp["w2"]),
                         synth.to_numpy(inp["s2"]), quant=quant)
    rt = fwd["route"]
    off, row_of = rt["offsets"], rt["row_of"]
    z = OM.grouped_gemm_nt(fwd["a1"], fwd["w13h"], off)
    dz = SUM * OM.grouped_gemm_nt(np.abs(fwd["a1"]), np.abs(fwd["w13h"]), off)
    moved = np.zeros_like(fwd["hh"])
    for sg in (-1, 1):
        for su in (-1, 1):
            for sh in (-1, 1):
                zz = OQ.round_bf16(z + dz * np.concatenate([np.full(F, sg), np.full(F, su)])[None, :])
                h = OQ.round_bf16(OM.swiglu(zz) * (1 + sh * 2.0 ** -20))
                hh = OQ.fakequant_act(fmt, h) if quant else h
                moved = np.maximum(moved, np.abs(hh - fwd["hh"]))
    dy = OM.grouped_gemm_nt(moved + SUM * np.abs(fwd["hh"]), np.abs(fwd["w2h"]), off) + 2.0 ** -7 * np.abs(fwd["y"])
    ref = OM.combine(fwd["y"], p, row_of)
    tol = OM.combine(dy, np.abs(p), row_of)
    return ref, tol + 2.0 ** -8 * (np.abs(ref) + tol) + 1e-30, fwd


SHAPES = [
    (1, 256, 128, 4, 2),
    (7, 384, 256, 8, 3),      # K of three quarters of a team's chunks
    (33, 128, 128, 3, 3),     # every token at every expert: passes of 8, 8, 8, 8 and 1
    (64, 128, 256, 40, 5),
    (2, 1024, 384, 16, 8),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", range(7))
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_the_oracle(shape, fmt):
    _build()
    T, d, F, E, k = shape
    inp = _inputs(T, d, F, E, k, fmt, seed=T + fmt, routing="zipf" if T == 64 else "uniform")
    out, ws = _few(inp)
    ref, tol, _ = _oracle(inp)
    assert Q.qad_check_device_error(ws) == 0
    assert np.all(np.abs(vals(out) - ref) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("shape,fmt", [((3, 16, 16, 5, 2), 0), ((5, 272, 144, 6, 2), 2), ((2, 2880, 2880, 4, 2), 3),
                                       ((64, 16, 16, 1024, 32), 4), ((1, 8192, 16, 2, 1), 6), ((1, 16, 8192, 2, 2), 2),
                                       ((9, 80, 48, 1, 1), 0), ((4, 2048, 768, 16, 8), 0), ((64, 256, 128, 4, 4), 5)])
def test_odd_sizes(shape, fmt):
    """Sizes that fill no chunk, the largest and the smallest, one expert, 1024 experts with 32 slots."""
    _build()
    T, d, F, E, k = shape
    inp = _inputs(T, d, F, E, k, fmt, seed=d + F)
    out, ws = _few(inp)
    ref, tol, _ = _oracle(inp)
    assert Q.qad_check_device_error(ws) == 0
    assert np.all(np.abs(vals(out) - ref) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
def test_unquantized_teacher(fmt):
    _build()
    inp = _inputs(6, 256, 384, 8, 4, fmt, seed=3)
    inp["s13"].fill_(float("nan"))  # not read
    inp["s2"].fill_(float("nan"))
    out, ws = _few(inp, Q.QAD_FLAG_NO_QUANT)
    ref, tol, _ = _oracle(inp, quant=False)
    assert Q.qad_check_device_error(ws) == 0
    assert np.all(np.abs(vals(out) - ref) <= tol)


@pytest.mark.gpu
def test_bad_and_repeated_indices_are_dropped():
    _build()
    inp = _inputs(12, 256, 128, 6, 4, 0, seed=5)
    idx = inp["topk_idx"]
    idx[2, 1] = 6
    idx[3, 0] = -1
    idx[4, 3] = idx[4, 0]
    idx[7] = torch.tensor([5, 5, 5, 5])
    idx[9] = torch.tensor([-5, 100, 1 << 30, -(1 << 31)])
    out, ws = _few(inp)
    assert Q.qad_check_device_error(ws) == Q.QAD_DEV_BAD_INDEX | Q.QAD_DEV_DUP_INDEX
    ref, tol, fwd = _oracle(inp)
    assert fwd["route"]["error"] == 3
    assert np.all(np.abs(vals(out) - ref) <= tol)
    assert not np.any(vals(out)[9])
    # no pair left at all, then a clean call on the same workspace
    idx.fill_(-1)
    out, ws = _few(inp, ws=ws)
    assert Q.qad_check_device_error(ws) == Q.QAD_DEV_BAD_INDEX and not np.any(vals(out))
    idx.copy_(torch.arange(4, device="cuda").expand(12, 4))
    out, ws = _few(inp, ws=ws)
    assert Q.qad_check_device_error(ws) == 0
    ref, tol, _ = _oracle(inp)
    assert np.all(np.abs(vals(out) - ref) <= tol)


@pytest.mark.gpu
def test_no_tokens_and_rows_behind_the_last():
    _build()
    inp = _inputs(3, 256, 128, 4, 2, 0, seed=6)
    guard = torch.full((5, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    _few(inp, out=guard)
    assert torch.all(guard[3:] == 7.0)
    none = dict(inp, T=0)
    guard.fill_(7.0)
    _, ws = _few(none, out=guard)
    assert torch.all(guard == 7.0) and Q.qad_check_device_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_weights_off_a_32_byte_boundary_give_the_same_bits(fmt):
    _build()
    inp = _inputs(5, 256, 128, 4, 2, fmt, seed=7)
    ref, _ = _few(inp)
    moved = []
    for w in (inp["w13"], inp["w2"]):
        flat = torch.empty(w.numel() + 64, dtype=torch.bfloat16, device="cuda")
        at = 8 if flat.data_ptr() % 32 == 0 else 0
        moved.append(flat[at:at + w.numel()].copy_(w.reshape(-1)))
        assert moved[-1].data_ptr() % 32 == 16
    out, _ = _few(inp, w13=moved[0], w2=moved[1])
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))


@pytest.mark.gpu
def test_a_row_that_is_not_finite_stays_alone():
    """A NaN or an infinity in one token's row does not reach the others, also not through a pass they share."""
    _build()
    inp = _inputs(9, 256, 128, 2, 2, Q.QAD_FMT_INT4_G128, seed=8)
    ref, _ = _few(inp)
    inp["x"][4, 17] = float("nan")
    inp["x"][6, 3] = float("inf")
    out, ws = _few(inp)
    assert Q.qad_check_device_error(ws) == 0
    rest = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(out[rest], ref[rest])
    assert torch.isnan(out[4]).all() and not torch.isfinite(out[6]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 2, 6])
def test_agrees_with_the_training_forward(fmt):
    """The same definition as qad_moe_fwd: the outputs differ by roundings that fall the other way (both are within the
    oracle's bound, so within twice that of one another)."""
    _build()
    inp = _inputs(16, 512, 256, 8, 4, fmt, seed=9)
    out, _ = _few(inp)
    s = Q.shape(16, 512, 256, 8, 4, fmt)
    ws = torch.empty(Q.qad_moe_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    full = torch.empty_like(out)
    Q.qad_moe_fwd(s, inp["x"], inp["topk_idx"], inp["topk_w"], inp["w13"], inp["s13"], inp["w2"], inp["s2"], full, ws)
    _, tol, _ = _oracle(inp)
    assert np.all(np.abs(vals(out) - vals(full)) <= 2 * tol)


@pytest.mark.gpu
def test_zero_scales_and_zero_rows():
    _build()
    inp = _inputs(4, 256, 128, 4, 2, 0, seed=10)
    inp["w13"][1].zero_()
    inp["s13"][1].zero_()
    inp["s2"][2, :8].zero_()
    inp["x"][2].zero_()
    out, _ = _few(inp)
    ref, tol, _ = _oracle(inp)
    assert np.all(np.abs(vals(out) - ref) <= tol)
    assert not np.any(vals(out)[2])


@pytest.mark.gpu
def test_captured_and_two_streams_at_once():
    """Two captured calls on workspaces of their own replay at the same time, with new routing, as eager calls do."""
    _build()
    a, b = _inputs(8, 512, 256, 16, 4, 0, seed=11), _inputs(3, 512, 256, 16, 4, 2, seed=12)
    want, ws = [], []
    for inp in (a, b):
        out, w = _few(inp)
        want.append(out.clone())
        ws.append(w)
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in want]
    graphs = []
    for inp, o, w, st in zip((a, b), outs, ws, streams):
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            _few(inp, out=o, ws=w)
        graphs.append(g)
    idx = a["topk_idx"].clone()
    for _ in range(3):
        for o in outs:
            o.fill_(0)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                for _ in range(4):
                    g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        a["topk_idx"].copy_((idx + 1) % 16)
        want[0] = _few(a)[0].clone()
        torch.cuda.synchronize()
        idx = a["topk_idx"].clone()


@pytest.mark.gpu
def test_module():
    from scale_only_quantization_gb300.autograd import QADMoE
    _build()
    for fmt in (0, 6):
        inp = _inputs(5, 256, 128, 4, 2, fmt, seed=13)
        moe = QADMoE(inp["w13"], inp["s13"], inp["w2"], inp["s2"], fmt)
        out = moe.few(inp["x"], inp["topk_idx"], inp["topk_w"])
        assert torch.equal(out, _few(inp)[0]) and not out.requires_grad
        teacher = moe.few(inp["x"], inp["topk_idx"], inp["topk_w"], quant=False)
        assert torch.equal(teacher, _few(inp, Q.QAD_FLAG_NO_QUANT)[0])
        with pytest.raises(ValueError):
            moe.few(inp["x"].float(), inp["topk_idx"], inp["topk_w"])
        with pytest.raises(ValueError):
            moe.few(inp["x"], inp["topk_idx"].long(), inp["topk_w"])
        with pytest.raises(ValueError):
            moe.few(inp["x"], inp["topk_idx"].cpu(), inp["topk_w"])
        with pytest.raises(Q.QADError):
            many = inp["x"].repeat(13, 1)
            moe.few(many, inp["topk_idx"].repeat(13, 1), inp["topk_w"].repeat(13, 1))


def test_refusals():
    """Checked on the host before anything is launched (no GPU is touched)."""
    _build()
    L = Q.lib()
    size = lambda *a: Q.qad_moe_few_workspace_bytes(Q.shape(*a))  # noqa: E731
    assert size(1, 256, 128, 4, 2, 0) > 0 and size(0, 256, 128, 4, 2, 0) > 0 and size(64, 8192, 8192, 4, 2, 0) > 0
    assert size(65, 256, 128, 4, 2, 0) == 0 and size(-1, 256, 128, 4, 2, 0) == 0
    assert size(1, 8208, 128, 4, 2, 0) == 0 and size(1, 256, 8208, 4, 2, 0) == 0
    assert size(1, 264, 128, 4, 2, 0) == 0 and size(1, 272, 128, 4, 2, 1) == 0 and size(1, 256, 128, 4, 5, 0) == 0
    assert size(1, 256, 128, 1025, 2, 0) == 0 and size(1, 256, 128, 40, 33, 0) == 0 and size(1, 256, 128, 4, 2, 7) == 0
    for flag in (Q.QAD_FLAG_STASH_H, Q.QAD_FLAG_RECOMPUTE, Q.QAD_FLAG_SMEM_DEQUANT):
        assert size(1, 256, 128, 4, 2, 0, flag) == 0
    assert size(1, 256, 128, 4, 2, 2, Q.QAD_FLAG_NATIVE_FP8) == 0
    assert size(1, 256, 128, 4, 2, 0, Q.QAD_FLAG_NO_QUANT) > 0
    P = 1 << 20  # an aligned stand-in address
    s = Q.shape(1, 256, 128, 4, 2, 0)
    n = Q.qad_moe_few_workspace_bytes(s)
    good = [P] * 9 + [n, None]
    call = lambda args, sh=s: L.qad_moe_few_fwd(ctypes.byref(sh), *args)  # noqa: E731
    for i in range(9):
        for bad in (None, P + 8):
            args = list(good)
            args[i] = bad
            assert call(args) == Q.QAD_ERR_INVALID_ARG, i
    assert call([P] * 8 + [P + 128, n, None]) == Q.QAD_ERR_INVALID_ARG  # the workspace: 256 bytes
    assert call([P] * 9 + [n - 1, None]) == Q.QAD_ERR_WORKSPACE
    assert call(good, Q.shape(65, 256, 128, 4, 2, 0)) == Q.QAD_ERR_UNSUPPORTED
    assert call(good, Q.shape(1, 256, 128, 4, 2, 0, Q.QAD_FLAG_RECOMPUTE)) == Q.QAD_ERR_INVALID_ARG
    assert L.qad_moe_few_fwd(None, *good) == Q.QAD_ERR_INVALID_ARG
    assert Q.qad_moe_few_workspace_bytes(Q.shape(1, 256, 128, 4, 2, 0)) % 1024 == 0


@pytest.mark.gpu
def test_threads_and_captures_of_two_sizes_of_one_format():
    """One format's kernel takes 190 KB of shared memory for one token of 2048 and 157 KB for eight: neither call's limit
    reaches the other's launch, from two host threads or between a capture and its graph."""
    import threading
    _build()
    one, eight = _inputs(1, 2048, 128, 8, 2, 0, seed=31), _inputs(8, 2048, 128, 8, 2, 0, seed=32)
    want = [_few(one)[0].clone(), _few(eight)[0].clone()]
    torch.cuda.synchronize()
    failed = []

    def work(inp, ref):
        try:
            st = torch.cuda.Stream()
            out, ws = torch.empty_like(ref), None
            with torch.cuda.stream(st):
                for _ in range(3000):
                    out, ws = _few(inp, out=out, ws=ws)
            st.synchronize()
            assert torch.equal(out, ref)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in 3 * list(zip((one, eight), want))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    outs = [torch.zeros_like(w) for w in want]
    wss = [_few(inp)[1] for inp in (one, eight)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for inp, o, w in zip((one, eight), outs, wss):
            _few(inp, out=o, ws=w)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.gpu
@pytest.mark.parametrize("d,E,T,most", [(8192, 4, 7, 8), (6144, 4, 7, 8), (8192, 1024, 5, 8)])
def test_fewer_tokens_do_not_read_the_weights_more_often(d, E, T, most):
    """With rows this wide fewer than 8 columns fit; T tokens of one expert take no more passes than 8 do (7 tokens in
    columns of 3 took three passes, where 8 in columns of 4 take two)."""
    _build()
    times = []
    for n in (T, most):
        inp = _inputs(n, d, 1024, 4, 1, 0, seed=34)
        inp["topk_idx"].zero_()
        if E > 4:  # experts that nobody names are not read, and their weights need not be there
            inp = dict(inp, E=E)
        out, ws = _few(inp)
        best = 1e9
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            _few(inp, out=out, ws=ws)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert times[0] <= 1.12 * times[1], times


@pytest.mark.gpu
@pytest.mark.parametrize("shape,fmt", [((64, 2048, 128, 8, 4), 0), ((64, 2048, 128, 8, 4), 5), ((32, 1536, 256, 4, 2), 2),
                                       ((5, 2880, 144, 6, 4), 2), ((8, 2048, 768, 8, 2), 1), ((5, 8192, 128, 2, 1), 0),
                                       ((6, 8192, 128, 2, 1), 4), ((7, 8192, 128, 2, 1), 0), ((9, 8192, 128, 2, 2), 6),
                                       ((7, 128, 8192, 2, 1), 1), ((8, 6144, 128, 3, 2), 3), ((7, 6144, 128, 3, 2), 2),
                                       ((5, 8192, 128, 1024, 2), 0)])  # its indices stay below 8: no others' weights are read
def test_short_rings_and_few_columns(shape, fmt):
    """Rows whose staging leaves the rings two chunks (8 tokens of 1400 and more), and rows so wide that fewer than 8
    tokens are served at once (above about 5100): the routing without barriers is then off for some token counts."""
    _build()
    T, d, F, E, k = shape
    inp = _inputs(T, d, F, min(E, 8), k, fmt, seed=T + d + F)
    if k == 1:
        inp["topk_idx"].fill_(1)
    ref, tol, _ = _oracle(inp)
    inp = dict(inp, E=E)
    out, ws = _few(inp)
    assert Q.qad_check_device_error(ws) == 0
    assert np.all(np.abs(vals(out) - ref) <= tol)
    for _ in range(3):  # the same bits again
        assert torch.equal(_few(inp)[0], out)


@pytest.mark.gpu
def test_module_flags_and_error_word():
    """few() is the layer that the module is: quantized or not as its flags say, unless the call says; what the call's
    error word held is there to be read."""
    from scale_only_quantization_gb300.autograd import QADMoE
    _build()
    inp = _inputs(5, 256, 128, 4, 2, 0, seed=33)
    args = (inp["x"], inp["topk_idx"], inp["topk_w"])
    plain = QADMoE(inp["w13"], inp["s13"], inp["w2"], inp["s2"], 0, Q.QAD_FLAG_NO_QUANT)
    quant = QADMoE(inp["w13"], inp["s13"], inp["w2"], inp["s2"], 0, Q.QAD_FLAG_RECOMPUTE)
    off, on = _few(inp, Q.QAD_FLAG_NO_QUANT)[0], _few(inp)[0]
    assert not torch.equal(off, on)
    assert torch.equal(plain.few(*args), off) and torch.equal(quant.few(*args), on)
    assert torch.equal(plain.few(*args, quant=True), on) and torch.equal(quant.few(*args, quant=False), off)
    assert quant.device_error() == 0 and plain.device_error() == 0
    idx = inp["topk_idx"].clone()
    idx[1, 0] = 4
    quant.few(inp["x"], idx, inp["topk_w"])
    idx[1, 0] = idx[1, 1]
    quant.few(inp["x"], idx, inp["topk_w"])
    quant.few(*args)
    assert quant.device_error() == Q.QAD_DEV_BAD_INDEX | Q.QAD_DEV_DUP_INDEX and quant.device_error() == 0
    assert quant.few(inp["x"][:0], idx[:0], inp["topk_w"][:0]).shape == (0, 256) and quant.device_error() == 0


@pytest.mark.gpu
def test_error_words_of_modules_first_used_in_inference_mode():
    """A generation loop runs in inference mode; its errors are read, and its modules used, outside as well."""
    from scale_only_quantization_gb300.autograd import QADHeadLoss, QADMoE, QADTokenLogprobs
    _build()
    inp = _inputs(5, 256, 128, 4, 2, 0, seed=35)
    moe, read = QADMoE(inp["w13"], inp["s13"], inp["w2"], inp["s2"], 0), QADTokenLogprobs()
    head = QADHeadLoss(torch.randn((64, 256), device="cuda"))
    bad = inp["topk_idx"].clone()
    bad[0, 0] = 4
    z, token = torch.randn((3, 64), device="cuda"), torch.tensor([1, 64, 2], device="cuda")
    h = torch.randn((3, 256), device="cuda").to(torch.bfloat16)
    with torch.inference_mode():
        moe.few(inp["x"], bad, inp["topk_w"])
        read(z, token)
        head(h, token)
    for m in (moe, read, head):
        assert m.device_error() == Q.QAD_DEV_BAD_INDEX and m.device_error() == 0
    moe.few(inp["x"], inp["topk_idx"], inp["topk_w"])
    read(z, token)
    head(h, token)
    assert moe.device_error() == 0 and read.device_error() == head.device_error() == Q.QAD_DEV_BAD_INDEX
    with torch.inference_mode():
        assert moe.device_error() == 0
