"""The sequence operators on the GPU against their definitions in 64 bits (tests/seq_oracle.py),
at the sizes, layouts and masks where they can go wrong."""
import math

import pytest
import torch

import seq_oracle as O
from gpu_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _normal(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(O.TYPES[dtype])


def _padded(t, left, right):
    """The same rows inside wider ones: (view on the GPU, the whole)."""
    wide = torch.full((t.shape[0], left + t.shape[1] + right), float("nan"), dtype=t.dtype)
    wide[:, left:left + t.shape[1]] = t
    wide = wide.cuda()
    return wide[:, left:left + t.shape[1]], wide


def _within(got, ref, tol, what):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((got - ref).abs() / tol)[bad].max()),
                           bad.nonzero()[0].tolist())


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


# lengths: single tokens, empty sequences, lengths around the window and around the kernels' runs
LENS = [[1], [0, 5, 0, 0, 2, 1], [3, 2, 9, 1, 40], [17, 64, 0, 31], [8, 8, 8], [0, 0],
        [1] * 70 + [0] * 3 + [130]]


# ------------------------------------------------------------------------------------------
# causal depthwise layer
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,D,W,lens,pad,silu", [
    ("bf16", 64, 4, 0, 0, True), ("f16", 72, 4, 1, 8, True), ("f32", 68, 3, 1, 4, False),
    ("bf16", 1000, 4, 2, 0, True), ("f16", 67, 4, 2, 3, True), ("f32", 1, 2, 3, 0, True),
    ("bf16", 2056, 4, 3, 8, True), ("f16", 8, 8, 2, 0, False), ("f32", 33, 7, 6, 1, True),
    ("bf16", 130, 5, 4, 5, True), ("f16", 16, 6, 5, 0, True), ("bf16", 24, 2, 6, 8, True)])
def test_dw1d_prompts(dtype, D, W, lens, pad, silu):
    import depthwise_pointwise_convolution_amd as F
    g = _gen(D * 100 + W)
    lens = LENS[lens]
    B, T = len(lens), sum(lens)
    cu = _offsets(lens)
    x = _normal(g, T, D, dtype=dtype)
    w, bias = _normal(g, D, W, dtype=dtype, std=0.5), _normal(g, D, std=0.2)
    nslots = B + 2
    slots = torch.randperm(nslots, generator=g)[:B].to(torch.int32)
    if B > 2:
        slots[1] = -1  # a sequence that keeps nothing
    carry = torch.randint(0, 2, (B,), generator=g, dtype=torch.int32)
    state = _normal(g, nslots, W - 1, D, dtype=dtype)
    ref, tol, sref, written = O.dw1d(dtype, x, w, bias, cu, slots.tolist(), carry.tolist(), state, silu)
    xg, _ = _padded(x, pad, pad)
    yg, whole = _padded(torch.full((T, D), float("nan"), dtype=O.TYPES[dtype]), pad, pad)
    sg = state.cuda()
    prob = F.dw1d_problem(dtype, D, W, tokens=T, seqs=B, slots=nslots, silu=silu, ldx=xg.stride(0) if T else 0,
                          ldy=yg.stride(0) if T else 0)
    F.fcm_dw1d_fwd(prob, xg, w.cuda(), bias.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), slots.cuda(),
                   carry.cuda(), sg, yg)
    torch.cuda.synchronize()
    assert bool(written.all()) or T == 0
    _within(yg, ref, tol, "y")
    assert torch.equal(sg.cpu().double(), sref)
    if pad:
        assert whole[:, :pad].isnan().all() and whole[:, pad + D:].isnan().all()
    # without a state every sequence starts from zero
    ref, tol, _, _ = O.dw1d(dtype, x, w, None, cu, slots.tolist(), carry.tolist(), None, silu)
    prob.slots = 0
    F.fcm_dw1d_fwd(prob, xg, w.cuda(), None, torch.tensor(cu, dtype=torch.int32).cuda(), None, None, None, yg)
    _within(yg, ref, tol, "y without state")


@pytest.mark.parametrize("dtype,B,D,W,pad", [
    ("bf16", 1, 64, 4, 0), ("f16", 5, 72, 4, 8), ("f32", 3, 67, 3, 1), ("bf16", 33, 2056, 4, 0),
    ("f16", 2, 9, 8, 3), ("f32", 7, 1024, 2, 4)])
def test_dw1d_tokens_continue_prompts(dtype, B, D, W, pad):
    import depthwise_pointwise_convolution_amd as F
    g = _gen(B * 1000 + D)
    w, bias = _normal(g, D, W, dtype=dtype, std=0.5), _normal(g, D, std=0.2)
    nslots = B + 3
    slots = torch.randperm(nslots, generator=g)[:B].to(torch.int32)
    if B > 2:
        slots[0], slots[B - 1] = -1, nslots  # idle rows
    state = _normal(g, nslots, W - 1, D, dtype=dtype)
    sg, sref = state.cuda(), state
    prob = F.dw1d_problem(dtype, D, W, tokens=B, seqs=B, slots=nslots, ldx=D + 2 * pad)
    for step in range(W + 1):
        x = _normal(g, B, D, dtype=dtype)
        live = [0 <= s < nslots for s in slots.tolist()]
        ref, tol, sref, _ = O.dw1d(dtype, x, w, bias, list(range(B + 1)), slots.tolist(), [1] * B, sref, True)
        ref[[not v for v in live]] = 0
        xg, _ = _padded(x, pad, pad)
        y = torch.full((B, D), float("nan"), dtype=O.TYPES[dtype], device="cuda")
        F.fcm_dw1d_step(prob, xg, w.cuda(), bias.cuda(), slots.cuda(), sg, y)
        _within(y, ref, tol, f"y of step {step}")
        assert torch.equal(sg.cpu().double(), sref)


# ------------------------------------------------------------------------------------------
# selective scan
# ------------------------------------------------------------------------------------------
def _scan_inputs(g, dtype, T, D, N, G, B, nslots, gate):
    v = {"x": _normal(g, T, D, dtype=dtype), "dt": _normal(g, T, D, dtype=dtype),
         "Bm": _normal(g, T, G * N, dtype=dtype), "Cm": _normal(g, T, G * N, dtype=dtype),
         "z": _normal(g, T, D, dtype=dtype, std=2.0) if gate else None,
         "A": -torch.rand(D, N, generator=g) * 8 - 0.01, "skip": _normal(g, D), "dt_bias": _normal(g, D) - 3.0,
         "state": _normal(g, nslots, D, N)}
    return v


def _run_scan(F, v, dtype, cu, slots, carry, G, pads, softplus=True, step=False, repeat=1):
    T, D = v["x"].shape
    N = v["A"].shape[1]
    strided = {k: _padded(v[k], p, p)[0] for k, p in zip(("x", "dt", "Bm", "Cm"), pads)}
    zg = _padded(v["z"], pads[0], pads[1])[0] if v["z"] is not None else None
    y, whole = _padded(torch.full((T, D), float("nan"), dtype=O.TYPES[dtype]), pads[1], pads[0])
    ld = {k: (t.stride(0) if T else 0) for k, t in strided.items()}
    state = v["state"].cuda() if v["state"] is not None else None
    prob = F.scan_problem(dtype, D, N, groups=G, tokens=T, seqs=len(slots), softplus=softplus,
                          slots=0 if state is None else state.shape[0], ldx=ld["x"], lddt=ld["dt"], ldb=ld["Bm"],
                          ldc=ld["Cm"], ldz=zg.stride(0) if zg is not None and T else 0, ldy=y.stride(0) if T else 0)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    sl = torch.tensor(slots, dtype=torch.int32).cuda() if state is not None else None
    common = (strided["x"], strided["dt"], dev(v["A"]), strided["Bm"], strided["Cm"], dev(v["skip"]),
              dev(v["dt_bias"]), zg)
    if step:
        F.fcm_scan_step(prob, *common, sl, state, y)
    else:
        ws = torch.full((max(16, F.fcm_scan_workspace(prob)) // 4,), float("nan"), device="cuda")
        ca = torch.tensor(carry, dtype=torch.int32).cuda() if state is not None else None
        F.fcm_scan_fwd(prob, *common, torch.tensor(cu, dtype=torch.int32).cuda(), sl, ca, state, ws, y)
    torch.cuda.synchronize()
    for p, side in ((pads[1], whole[:, :pads[1]]), (pads[0], whole[:, pads[1] + D:])):
        assert p == 0 or bool(side.isnan().all())
    return y, state


@pytest.mark.parametrize("dtype,D,N,G,lens,gate,pads", [
    ("bf16", 64, 16, 1, 0, True, (0, 0, 0, 0)), ("f16", 72, 16, 1, 1, True, (8, 0, 3, 1)),
    ("f32", 68, 16, 2, 2, True, (4, 0, 0, 5)), ("bf16", 130, 16, 1, 3, False, (0, 1, 0, 0)),
    ("f16", 67, 8, 1, 2, True, (3, 0, 8, 8)), ("f32", 1, 1, 1, 3, False, (0, 0, 0, 0)),
    ("bf16", 48, 5, 3, 4, True, (0, 8, 1, 1)), ("f32", 66, 24, 2, 3, True, (0, 0, 0, 0)),
    ("f16", 40, 32, 1, 1, False, (0, 0, 0, 0)), ("bf16", 65, 33, 1, 2, True, (1, 1, 1, 1)),
    ("f32", 20, 64, 1, 3, True, (0, 0, 0, 0)), ("bf16", 128, 64, 2, 4, True, (0, 0, 0, 0)),
    ("f16", 64, 16, 1, 5, True, (0, 0, 0, 0)), ("bf16", 32, 16, 2, 6, True, (0, 0, 0, 0))])
def test_scan_prompts(dtype, D, N, G, lens, gate, pads):
    import depthwise_pointwise_convolution_amd as F
    g = _gen(D * 100 + N)
    lens = LENS[lens]
    B, T, cu = len(lens), sum(lens), _offsets(lens)
    v = _scan_inputs(g, dtype, T, D, N, G, B, B + 2, gate)
    slots = torch.randperm(B + 2, generator=g)[:B].tolist()
    if B > 2:
        slots[1] = -1
    carry = torch.randint(0, 2, (B,), generator=g).tolist()
    args = [v[k] for k in ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias", "z")]
    ref, tol, sref, stol, _ = O.scan(dtype, *args, cu, slots, carry, v["state"], G, True)
    y, state = _run_scan(F, v, dtype, cu, slots, carry, G, pads)
    _within(y, ref, tol, "y")
    _within(state, sref, stol, "state")


@pytest.mark.parametrize("dtype,D,N,lens", [
    ("f32", 24, 16, [1500]), ("bf16", 72, 16, [700, 0, 1, 513, 1025]), ("f16", 16, 8, [2047, 129]),
    ("f32", 9, 24, [600, 300]), ("bf16", 12, 64, [257, 640])])
def test_scan_long_prompts_and_slow_decay(dtype, D, N, lens):
    # states that hardly decay, so that what a chunk hands on reaches the end of the sequence
    import depthwise_pointwise_convolution_amd as F
    g = _gen(D + N + len(lens))
    B, T, cu = len(lens), sum(lens), _offsets(lens)
    v = _scan_inputs(g, dtype, T, D, N, 1, B, B, True)
    v["A"][:, ::2] *= 2.0 ** -8
    v["dt_bias"] -= 2.0
    v["state"] *= 50.0
    slots, carry = list(range(B))[::-1], [1] * B
    args = [v[k] for k in ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias", "z")]
    ref, tol, sref, stol, _ = O.scan(dtype, *args, cu, slots, carry, v["state"], 1, True)
    y, state = _run_scan(F, v, dtype, cu, slots, carry, 1, (0, 0, 0, 0))
    _within(y, ref, tol, "y")
    _within(state, sref, stol, "state")


def test_scan_without_options():
    # no softplus, no bias, no skip, no gate, no state
    import depthwise_pointwise_convolution_amd as F
    g = _gen(3)
    lens = [5, 0, 300, 1]
    cu = _offsets(lens)
    v = _scan_inputs(g, "f32", sum(lens), 36, 16, 1, 4, 4, False)
    v["dt"] = v["dt"].abs() * 0.2
    v["skip"] = v["dt_bias"] = v["state"] = None
    args = [v[k] for k in ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias", "z")]
    ref, tol, _, _, _ = O.scan("f32", *args, cu, [0] * 4, [0] * 4, None, 1, False)
    y, _ = _run_scan(F, v, "f32", cu, [0] * 4, [0] * 4, 1, (0, 0, 0, 0), softplus=False)
    _within(y, ref, tol, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_step_sizes_from_tiny_to_large(dtype):
    # softplus far on both sides: steps near exp(-30) keep their relative precision, steps near 60
    # make the decay underflow to zero
    import depthwise_pointwise_convolution_amd as F
    g = _gen(8)
    T, D, N = 61, 40, 16
    v = _scan_inputs(g, dtype, T, D, N, 1, 1, 1, True)
    v["dt"] = torch.linspace(-30, 60, T)[:, None].expand(T, D).to(O.TYPES[dtype]).contiguous()
    v["dt_bias"] = None
    v["z"] = torch.linspace(-100, 100, T)[:, None].expand(T, D).to(O.TYPES[dtype]).contiguous()
    args = [v[k] for k in ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias", "z")]
    ref, tol, sref, stol, _ = O.scan(dtype, *args, [0, T], [0], [1], v["state"], 1, True)
    y, state = _run_scan(F, v, dtype, [0, T], [0], [1], 1, (0, 0, 0, 0))
    _within(y, ref, tol + 2.0 ** -120, "y")
    _within(state, sref, stol + 2.0 ** -120, "state")


@pytest.mark.parametrize("dtype,B,D,N,G,gate,pads", [
    ("bf16", 1, 64, 16, 1, True, (0, 0, 0, 0)), ("f16", 9, 72, 16, 2, True, (8, 0, 1, 3)),
    ("f32", 5, 67, 16, 1, False, (0, 0, 0, 0)), ("bf16", 37, 130, 16, 1, True, (0, 0, 8, 8)),
    ("f32", 3, 21, 5, 3, True, (1, 0, 0, 0)), ("f16", 4, 40, 24, 1, True, (0, 0, 0, 0)),
    ("bf16", 2, 33, 64, 1, True, (0, 0, 0, 0)), ("f32", 130, 8, 32, 1, True, (0, 0, 0, 0)),
    ("f16", 2, 10, 1, 1, False, (0, 0, 0, 0)), ("bf16", 3, 1100, 8, 1, True, (0, 0, 0, 0))])
def test_scan_tokens(dtype, B, D, N, G, gate, pads):
    import depthwise_pointwise_convolution_amd as F
    g = _gen(B * 1000 + D)
    v = _scan_inputs(g, dtype, B, D, N, G, B, B + 3, gate)
    slots = torch.randperm(B + 3, generator=g)[:B].tolist()
    if B > 2:
        slots[0], slots[B - 1] = -5, B + 3
    args = [v[k] for k in ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias", "z")]
    ref, tol, sref, stol, _ = O.scan(dtype, *args, list(range(B + 1)), slots, [1] * B, v["state"], G, True)
    for b in range(B):
        if not 0 <= slots[b] < B + 3:
            ref[b] = 0
    y, state = _run_scan(F, v, dtype, None, slots, None, G, pads, step=True)
    _within(y, ref, tol, "y")
    _within(state, sref, stol, "state")


def test_prompt_in_parts_and_token_by_token():
    # one prompt whole, in three calls, and token by token: the same outputs and state
    import depthwise_pointwise_convolution_amd as F
    g = _gen(12)
    T, D, N = 70, 64, 16
    v = _scan_inputs(g, "f32", T, D, N, 1, 1, 1, True)
    args = [v[k] for k in ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias", "z")]
    ref, tol, sref, stol, _ = O.scan("f32", *args, [0, T], [0], [1], v["state"], 1, True)
    for cuts in ([0, 1, 33, 70], list(range(71))):
        state, ys = v["state"], []
        for a, b in zip(cuts, cuts[1:]):
            part = {k: (t[a:b].contiguous() if k in ("x", "dt", "Bm", "Cm", "z") else t) for k, t in v.items()}
            part["state"] = state
            y, s = _run_scan(F, part, "f32", [0, b - a], [0], [1], 1, (0, 0, 0, 0), step=b - a == 1)
            state = s.cpu()
            ys.append(y.cpu())
        _within(torch.cat(ys), ref, tol, "y in parts")
        _within(state, sref, stol, "state in parts")


# ------------------------------------------------------------------------------------------
# 4-bit pointwise layer
# ------------------------------------------------------------------------------------------
def _q4_inputs(g, dtype, M, C, K, group, zeros):
    groups = -(-C // group)
    return {"x": _normal(g, M, C, dtype=dtype),
            "q": torch.randint(0, 256, (K, C // 2), generator=g, dtype=torch.uint8),
            "scales": (torch.rand(K, groups, generator=g) * 0.02 + 0.001).to(O.TYPES[dtype]),
            "zeros": torch.randint(0, 16, (K, groups), generator=g, dtype=torch.uint8) if zeros else None,
            "bias": _normal(g, K)}


Q4_SIZES = [("bf16", 1, 128, 16, 128, False), ("f16", 1, 8, 1, 32, True), ("bf16", 2, 136, 17, 128, True),
            ("f16", 3, 1000, 37, 32, True), ("bf16", 4, 2048, 65, 64, True), ("f16", 5, 264, 100, 64, False),
            ("bf16", 8, 1096, 31, 128, True), ("f16", 16, 4096, 48, 128, True), ("bf16", 17, 512, 130, 32, True),
            ("f16", 33, 96, 64, 64, True), ("bf16", 64, 640, 80, 128, False), ("f16", 130, 40, 33, 32, True),
            ("bf16", 7, 8200, 19, 128, True), ("f16", 12, 4128, 16, 64, True), ("bf16", 1, 16384, 5, 128, True),
            ("f16", 9, 24, 2000, 32, False)]


@pytest.mark.parametrize("dtype,M,C,K,group,zeros", Q4_SIZES)
def test_q4_against_64_bits(dtype, M, C, K, group, zeros):
    import depthwise_pointwise_convolution_amd as F
    g = _gen(M * 7 + C + K)
    v = _q4_inputs(g, dtype, M, C, K, group, zeros)
    for act, bias, pad in (("none", None, 0), ("relu", v["bias"], 8), ("relu6", v["bias"], 0)):
        ref, tol = O.q4(dtype, v["x"], v["q"], v["scales"], v["zeros"], bias, group, act)
        xg, _ = _padded(v["x"], pad, pad)
        if pad:  # x starts 16-byte aligned inside its wider rows
            assert xg.data_ptr() % 16 == 0
        y, whole = _padded(torch.full((M, K), float("nan"), dtype=O.TYPES[dtype]), pad // 8, pad // 4)
        prob = F.q4_problem(dtype, M, C, K, group=group, act=act, ldx=xg.stride(0), ldy=y.stride(0))
        F.fcm_q4_fwd(prob, xg, v["q"].cuda(), v["scales"].cuda(), None if v["zeros"] is None else v["zeros"].cuda(),
                     None if bias is None else bias.cuda(), y)
        _within(y, ref, tol, f"y with {act}")
        assert pad == 0 or (whole[:, :1].isnan().all() and whole[:, 1 + K:].isnan().all())


@pytest.mark.parametrize("dtype,M,C,K,group,zeros", Q4_SIZES)
def test_q4_integers_are_exact(dtype, M, C, K, group, zeros):
    # whole-number inputs and scales that are powers of two: every sum is exact in 32 bits
    import depthwise_pointwise_convolution_amd as F
    g = _gen(M + C * 3 + K)
    v = _q4_inputs(g, dtype, M, C, K, group, zeros)
    x = torch.randint(-2, 3, (M, C), generator=g).to(O.TYPES[dtype])
    scales = (2.0 ** torch.randint(-6, -2, v["scales"].shape, generator=g)).to(O.TYPES[dtype])
    ref, _ = O.q4(dtype, x, v["q"], scales, v["zeros"], None, group, "none")
    y = torch.full((M, K), float("nan"), dtype=O.TYPES[dtype], device="cuda")
    F.fcm_q4_fwd(F.q4_problem(dtype, M, C, K, group=group), x.cuda(), v["q"].cuda(), scales.cuda(),
                 None if v["zeros"] is None else v["zeros"].cuda(), None, y)
    assert torch.equal(y.cpu(), ref.float().to(O.TYPES[dtype]))


def test_q4_unaligned_weights_and_values_that_are_not_finite():
    import depthwise_pointwise_convolution_amd as F
    g = _gen(4)
    M, C, K = 6, 256, 40
    v = _q4_inputs(g, "bf16", M, C, K, 64, True)
    q = torch.zeros(K * C // 2 + 4, dtype=torch.uint8)
    q[4:] = v["q"].reshape(-1)
    x = v["x"].clone()
    x[2, 7], x[4, 9] = float("inf"), float("nan")
    y = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    F.fcm_q4_fwd(F.q4_problem("bf16", M, C, K, group=64), x.cuda(), q.cuda()[4:], v["scales"].cuda(),
                 v["zeros"].cuda(), None, y)
    ref, tol = O.q4("bf16", v["x"], v["q"], v["scales"], v["zeros"], None, 64, "none")
    rows = [0, 1, 3, 5]
    _within(y[rows], ref[rows], tol[rows], "rows without such values")
    assert not y[2].isfinite().any() and y[4].isnan().all()


# ------------------------------------------------------------------------------------------
# beam search
# ------------------------------------------------------------------------------------------
def _beam_case(g, dtype, R, W, V, eos):
    # logits on a grid: many are equal, in all types exactly
    logits = (torch.randn(R * W, V, generator=g) * 24).round() / 8
    logits[torch.rand(R * W, V, generator=g) < 0.1] = -math.inf
    scores = -torch.rand(R * W, generator=g) * 4
    done = (torch.rand(R * W, generator=g) < 0.2).to(torch.int32) if eos >= 0 else None
    return logits.to(O.TYPES[dtype]), scores, done


def _run_beam(F, dtype, logits, scores, done, R, W, eos, pad=0):
    V = logits.shape[1]
    lg, _ = _padded(logits, pad, pad)
    prob = F.beam_problem(dtype, R, W, V, eos=eos, ldl=lg.stride(0))
    n = R * W
    ws = torch.full((F.fcm_beam_workspace(prob) // 4 + 4,), float("nan"), device="cuda")
    nxt = torch.full((n,), float("nan"), device="cuda")
    par, tok, dn = (torch.full((n,), -7, dtype=torch.int32, device="cuda") for _ in range(3))
    F.fcm_beam_select(prob, lg, scores.cuda(), None if done is None else done.cuda(), ws, nxt, par, tok, dn)
    torch.cuda.synchronize()
    return prob, nxt.cpu(), par.cpu(), tok.cpu(), dn.cpu()


def _same_beams(got, ref, V):
    _, nxt, par, tok, dn = got
    best, parent, token, ended = ref
    assert par.tolist() == parent.tolist() and tok.tolist() == token.tolist()
    assert [bool(v) for v in dn] == [bool(v) for v in ended]
    assert torch.equal(nxt.isinf(), best.isinf())
    ok = ~best.isinf()
    # one rounding to 32 bits; the log-sum-exp has V exponentials of arguments up to |l - top|
    # that are rounded once: the error of their mean is far below 2^-20
    assert ((nxt.double() - best)[ok].abs() <= 2.0 ** -20 + 2.0 ** -23 * best[ok].abs()).all()


@pytest.mark.parametrize("dtype,R,W,V,eos,pad", [
    ("f32", 1, 1, 1, -1, 0), ("f32", 1, 4, 3, 2, 0), ("f16", 2, 8, 5, 0, 3), ("bf16", 3, 4, 1000, 2, 8),
    ("f32", 2, 5, 4099, 7, 0), ("f16", 1, 8, 32001, 2, 1), ("bf16", 5, 2, 20000, -1, 0), ("f32", 1, 32, 700, 3, 0),
    ("f16", 2, 32, 9000, 1, 0), ("f32", 7, 3, 2048, 2047, 4), ("bf16", 1, 16, 65537, 5, 0)])
def test_beam_selection(dtype, R, W, V, eos, pad):
    import depthwise_pointwise_convolution_amd as F
    g = _gen(R * 10 + W + V)
    logits, scores, done = _beam_case(g, dtype, R, W, V, eos)
    ref = O.beam(logits, scores, done, W, eos)
    _same_beams(_run_beam(F, dtype, logits, scores, done, R, W, eos, pad), ref, V)


@pytest.mark.parametrize("dtype,W,V", [("f32", 4, 50), ("bf16", 6, 5000), ("f16", 3, 40000)])
def test_beam_selection_at_its_edges(dtype, W, V):
    # requests: the first step of a search (all beams but one at -inf); rows that are masked
    # altogether; fewer tokens than beams left; all logits equal; NaN and infinite logits; all done
    import depthwise_pointwise_convolution_amd as F
    g = _gen(W + V)
    R, eos = 7, 4
    logits, scores, done = _beam_case(g, "f32", R, W, V, eos)
    done[:] = 0
    scores[1:W] = -math.inf
    logits[W:2 * W] = -math.inf
    logits[2 * W:3 * W] = -math.inf
    logits[2 * W, 11], logits[2 * W + 1, 3] = 1.0, 2.0
    logits[3 * W:4 * W] = 0.25
    scores[3 * W:4 * W] = -1.0
    logits[4 * W, ::3] = math.nan
    logits[4 * W + 1, 7] = math.inf
    done[5 * W:6 * W] = 1
    scores[6 * W:] = -math.inf
    logits = logits.to(O.TYPES[dtype])
    if dtype != "f32":
        logits[4 * W + 1, 7] = math.inf
    ref = O.beam(logits, scores, done, W, eos)
    _same_beams(_run_beam(F, dtype, logits, scores, done, R, W, eos), ref, V)


@pytest.mark.parametrize("W,shapes", [(1, [(8,)]), (4, [(64, 16), (3, 40)]), (8, [(40000,), (5,), (7, 3)]),
                                      (32, [(33,), (1024,)])])
def test_beam_reorder(W, shapes):
    import depthwise_pointwise_convolution_amd as F
    g = _gen(W)
    R = 6
    n = R * W
    parent = torch.randint(0, W, (n,), generator=g, dtype=torch.int32)
    parent[:W] = 0                                            # one beam has every child
    parent[W:2 * W] = torch.arange(W)                         # nothing moves
    parent[2 * W:3 * W] = torch.arange(W - 1, -1, -1)         # a permutation: nothing is copied
    slots = torch.randperm(n + 5, generator=g)[:n].to(torch.int32)
    pools = [torch.randn(n + 5, *s, generator=g) for s in shapes]
    pools.append(torch.randn(n + 5, 24, generator=g).to(torch.bfloat16))
    # slots whose bytes are no multiple of a word, below and above what a workgroup copies
    pools.append(torch.randn(n + 5, 8193, generator=g).to(torch.bfloat16))
    pools.append(torch.randint(0, 256, (n + 5, 16403), generator=g, dtype=torch.uint8))
    pools.append(torch.randint(0, 256, (n + 5, 7), generator=g, dtype=torch.uint8))
    want, wpools = O.reorder(parent.tolist(), slots.tolist(), W, pools)
    got = [p.cuda() for p in pools]
    out = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    prob = F.beam_problem("f32", R, W, 100)
    F.fcm_beam_reorder(prob, parent.cuda(), slots.cuda(), out, got)
    assert out.tolist() == want
    for a, b in zip(got, wpools):
        assert torch.equal(a.cpu(), b)


# ------------------------------------------------------------------------------------------
# streams and graphs
# ------------------------------------------------------------------------------------------
def _token_pass(F, dtype="bf16", B=3, D=256, N=16, K=96, V=500):
    """One decoding pass through all operators on buffers of its own: (run, outputs)."""
    g = _gen(77)
    c = lambda *s, **k: _normal(g, *s, **k).cuda()  # noqa: E731
    t = O.TYPES[dtype]
    x, w, win = c(B, D, dtype=dtype), c(D, 4, dtype=dtype), c(B, 3, D, dtype=dtype)
    dt, bc, A = c(B, D, dtype=dtype), c(B, 2 * N, dtype=dtype), -torch.rand(D, N).cuda()
    st = c(B, D, N)
    v = {k: (a.cuda() if a is not None else None) for k, a in _q4_inputs(g, dtype, B, D, V, 64, True).items()}
    u, y = torch.empty(B, D, dtype=t, device="cuda"), torch.empty(B, D, dtype=t, device="cuda")
    lo = torch.empty(B, V, dtype=t, device="cuda")
    p1 = F.dw1d_problem(dtype, D, 4, tokens=B, seqs=B, slots=B)
    p2 = F.scan_problem(dtype, D, N, tokens=B, seqs=B, slots=B, ldb=2 * N, ldc=2 * N)
    p3 = F.q4_problem(dtype, B, D, V, group=64)
    p4 = F.beam_problem(dtype, 1, B, V, eos=1)
    ws = torch.empty(F.fcm_beam_workspace(p4), dtype=torch.uint8, device="cuda")
    scores, nxt = -torch.arange(B).float().cuda(), torch.empty(B, device="cuda")
    par, tok, dn, sl = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(4))
    slots = torch.arange(B, dtype=torch.int32).cuda()

    def run():
        F.fcm_dw1d_step(p1, x, w, None, slots, win, u)
        F.fcm_scan_step(p2, u, dt, A, bc, bc[:, N:], None, None, None, slots, st, y)
        F.fcm_q4_fwd(p3, y, v["q"], v["scales"], v["zeros"], None, lo)
        F.fcm_beam_select(p4, lo, scores, None, ws, nxt, par, tok, dn)
        F.fcm_beam_reorder(p4, par, slots, sl, [win, st])
    return run, [win, st, u, y, lo, nxt, par, tok, dn, sl]


def test_operators_on_another_stream_and_in_a_graph():
    import depthwise_pointwise_convolution_amd as F
    run, out = _token_pass(F)
    torch.cuda.synchronize()
    start = [out[0].clone(), out[1].clone()]
    want = []
    for _ in range(4):
        run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    for mode in ("stream", "graph"):
        out[0].copy_(start[0])
        out[1].copy_(start[1])
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        if mode == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
            out[0].copy_(start[0])
            out[1].copy_(start[1])
            torch.cuda.synchronize()
        for k in range(4):
            if mode == "graph":
                graph.replay()
                (torch.ones(1000, device="cuda") * 2).sum().item()  # the program's own work between
            else:
                with torch.cuda.stream(s):
                    run()
            torch.cuda.synchronize()
            for a, b in zip(out, want[k]):
                assert torch.equal(a, b), (mode, k)


def test_results_do_not_depend_on_the_run():
    import depthwise_pointwise_convolution_amd as F
    g = _gen(5)
    lens = [300, 41]
    v = _scan_inputs(g, "f32", 341, 96, 16, 1, 2, 2, True)
    first = _run_scan(F, v, "f32", _offsets(lens), [0, 1], [1, 0], 1, (0, 0, 0, 0))
    again = _run_scan(F, v, "f32", _offsets(lens), [0, 1], [1, 0], 1, (0, 0, 0, 0))
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------------------------------------
# offsets past 32 bits, and the operators together
# ------------------------------------------------------------------------------------------
def test_states_and_rows_past_32_bits():
    import depthwise_pointwise_convolution_amd as F
    g = _gen(6)
    D, N, slots = 2048, 16, 70000  # a pool of 9 GB
    assert slots * D * N * 4 > 2 ** 33
    v = _scan_inputs(g, "bf16", 2, D, N, 1, 2, 2, True)
    pool = torch.empty(slots, D, N, device="cuda")
    where = [slots - 1, slots // 2 + 7]
    pool[where] = v["state"].cuda()
    small, big = dict(v), dict(v, state=None)
    want, ws = _run_scan(F, small, "bf16", None, [0, 1], None, 1, (0, 0, 0, 0), step=True)
    prob = F.scan_problem("bf16", D, N, tokens=2, seqs=2, slots=slots)
    y = torch.empty(2, D, dtype=torch.bfloat16, device="cuda")
    dev = [big[k].cuda() for k in ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias", "z")]
    F.fcm_scan_step(prob, *dev, torch.tensor(where, dtype=torch.int32).cuda(), pool, y)
    assert torch.equal(y, want) and torch.equal(pool[where], ws)
    # beams over the same pool
    prob = F.beam_problem("f32", 1, 2, 100)
    parent = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    F.fcm_beam_reorder(prob, parent, torch.tensor(where, dtype=torch.int32).cuda(), out, [pool])
    assert out.tolist() == where and torch.equal(pool[where[1]], pool[where[0]])
    del pool
    # rows that lie 2^31 bytes apart
    T, ld = 4, 2 ** 30 + 64
    wide = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").as_strided((T, 64), (ld, 1))
    x = _normal(g, T, 64, dtype="bf16")
    wide.copy_(x)
    w = _normal(g, 64, 4, dtype="bf16")
    prob = F.dw1d_problem("bf16", 64, 4, tokens=T, seqs=1, ldx=ld)
    y = torch.empty(T, 64, dtype=torch.bfloat16, device="cuda")
    F.fcm_dw1d_fwd(prob, wide, w.cuda(), None, torch.tensor([0, T], dtype=torch.int32).cuda(), None, None, None, y)
    ref, tol, _, _ = O.dw1d("bf16", x, w, None, [0, T], [0], [0], None, True)
    _within(y, ref, tol, "rows far apart")
    logits, scores, _ = _beam_case(g, "bf16", 1, T, 64, -1)
    wide.copy_(logits)
    prob = F.beam_problem("bf16", 1, T, 64, ldl=ld)
    out = [torch.empty(T, dtype=t, device="cuda") for t in (torch.float32,) + (torch.int32,) * 3]
    F.fcm_beam_select(prob, wide, scores.cuda(), None,
                      torch.empty(F.fcm_beam_workspace(prob), dtype=torch.uint8, device="cuda"), *out)
    ref = O.beam(logits, scores, None, T, -1)
    assert out[1].tolist() == ref[1].tolist() and out[2].tolist() == ref[2].tolist()


def test_a_rate_of_minus_infinity_forgets_and_no_step_keeps():
    import depthwise_pointwise_convolution_amd as F
    g = _gen(9)
    T, D, N = 6, 8, 16
    v = _scan_inputs(g, "f32", T, D, N, 1, 1, 1, False)
    v["A"][:, 0] = -math.inf
    v["dt_bias"] = None
    v["dt"] = v["dt"].abs()
    y, state = _run_scan(F, v, "f32", [0, T], [0], [1], 1, (0, 0, 0, 0), softplus=False)
    assert y.isfinite().all() and state.isfinite().all()
    last = (v["dt"][-1] * v["x"][-1] * v["Bm"][-1, 0]).double()
    _within(state[0, :, 0], last, 4 * O.U * last.abs(), "state that forgets")
    v["dt"] = torch.zeros_like(v["dt"])
    _, state = _run_scan(F, v, "f32", [0, T], [0], [1], 1, (0, 0, 0, 0), softplus=False)
    assert torch.equal(state.cpu(), v["state"])


def test_example_decodes_and_its_scores_hold():
    # every beam's score, summed over single-token steps with reordered states, against one prompt
    # run over the beam's tokens.  Both round activations to bf16 (2^-8) at some ten places a layer
    # in different orders; logits are of order 1, so a token's log-probability moves by a few 2^-8
    # and the sum over 12 tokens by well under 0.5 (a wrong state changes it by several units)
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import state_space_decode as E
    worst = E.main(["--dim", "128", "--layers", "2", "--vocab", "501", "--requests", "3", "--beams", "4",
                    "--tokens", "12", "--check"])
    assert worst < 0.5


# ------------------------------------------------------------------------------------------
# large strides and values that are not finite
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("M,C,ldx,group", [(32, 136, 2 ** 25 + 2 ** 22, 32), (20, 1000, 2 ** 26 - 8, 128),
                                           (18, 24, 2 ** 26 - 8, 64), (5, 136, 2 ** 26 - 8, 64)])
def test_q4_rows_far_apart(M, C, ldx, group):
    # a tile's rows span more than 2^31 bytes: channels behind the last are zero, whatever lies between the
    # rows.  Whole numbers and scales that are powers of two: exact
    import depthwise_pointwise_convolution_amd as F
    g = _gen(C + M)
    K = 40
    v = _q4_inputs(g, "bf16", M, C, K, group, True)
    x = torch.randint(-2, 3, (M, C), generator=g).to(torch.bfloat16)
    scales = (2.0 ** torch.randint(-6, -2, v["scales"].shape, generator=g)).to(torch.bfloat16)
    wide = torch.full(((M - 1) * ldx + C,), 512.0, dtype=torch.bfloat16, device="cuda").as_strided((M, C), (ldx, 1))
    wide.copy_(x)
    ref, _ = O.q4("bf16", x, v["q"], scales, v["zeros"], None, group, "none")
    y = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    F.fcm_q4_fwd(F.q4_problem("bf16", M, C, K, group=group, ldx=ldx), wide, v["q"].cuda(), scales.cuda(),
                 v["zeros"].cuda(), None, y)
    assert torch.equal(y.cpu(), ref.float().to(torch.bfloat16))


@pytest.mark.parametrize("C,group", [(136, 32), (1000, 64), (264, 64)])
def test_q4_scales_that_are_not_finite_stay_in_their_channel(C, group):
    # groups that a last step of 128 channels has room for but C has not
    import depthwise_pointwise_convolution_amd as F
    g = _gen(C)
    M, K = 5, 70
    v = _q4_inputs(g, "bf16", M, C, K, group, True)
    for k in range(0, K, 16):  # the first channel of every tile
        v["scales"][k, 0] = float("inf") if k % 32 else float("nan")
    y = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    F.fcm_q4_fwd(F.q4_problem("bf16", M, C, K, group=group), v["x"].cuda(), v["q"].cuda(), v["scales"].cuda(),
                 v["zeros"].cuda(), None, y)
    rest = [k for k in range(K) if k % 16]
    ref, tol = O.q4("bf16", v["x"], v["q"][rest], v["scales"][rest], v["zeros"][rest], None, group, "none")
    _within(y[:, rest], ref, tol, "channels with finite scales")
    assert not y[:, ::16].isfinite().any()


@pytest.mark.parametrize("dtype,N,lens", [("f32", 16, [3]), ("bf16", 16, [40, 0, 7]), ("f32", 5, [9, 2]), ("f16", 24, [70])])
@pytest.mark.parametrize("step", [False, True])
def test_a_rate_that_is_no_number_shows(dtype, N, lens, step):
    # (a maximum with the lowest float would make a NaN weight forget and answer with finite values)
    import depthwise_pointwise_convolution_amd as F
    g = _gen(N)
    lens = [1] * len(lens) if step else lens
    B, T, cu, D = len(lens), sum(lens), _offsets(lens), 40
    v = _scan_inputs(g, dtype, T, D, N, 1, B, B, False)
    v["A"][7, N - 2] = float("nan")
    y, state = _run_scan(F, v, dtype, cu, list(range(B)), [1] * B, 1, (0, 0, 0, 0), step=step)
    other = [d for d in range(D) if d != 7]
    assert y[:, 7].isnan().all() and y[:, other].isfinite().all()
    ran = [b for b in range(B) if lens[b]]
    assert state[ran, 7, N - 2].isnan().all()
    state[ran, 7, N - 2] = 0
    assert state.isfinite().all()


@pytest.mark.parametrize("dtype,N", [("f32", 16), ("bf16", 8), ("f16", 24)])
@pytest.mark.parametrize("lens", [[5, 3], [1], [0, 13, 6], [70, 2]])
def test_an_infinite_state_stays_infinite(dtype, N, lens):
    # the last row of a sequence is its only infinite one: nothing behind it may touch the state
    import depthwise_pointwise_convolution_amd as F
    g = _gen(N + len(lens))
    B, T, cu, D = len(lens), sum(lens), _offsets(lens), 24
    v = _scan_inputs(g, dtype, T, D, N, 1, B, B, False)
    v["x"] = v["x"].abs() + 0.5
    for b in range(B):
        if lens[b]:
            v["Bm"][cu[b + 1] - 1, N - 1] = math.inf if b % 2 else -math.inf
    v["Cm"] = v["Cm"].abs() + 0.5
    _, state = _run_scan(F, v, dtype, cu, list(range(B)), [1] * B, 1, (0, 0, 0, 0))
    args = [v[k] for k in ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias", "z")]
    _, _, sref, stol, _ = O.scan(dtype, *args, cu, list(range(B)), [1] * B, v["state"], 1, True)
    far = sref.isinf()
    assert far.any() and torch.equal(state.cpu().double()[far], sref[far])
    stol[far], sref[far] = 0, 0
    state[far.cuda()] = 0
    _within(state, sref, stol, "the other states")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("W,V", [(3, 50), (4, 3000), (2, 40000)])
def test_beams_over_rows_of_extreme_values(dtype, W, V):
    # a row that is masked with the type's lowest value altogether is V equal tokens, one with two infinite
    # logits is two: their log-sum-exps differ from those values by log V and log 2, which a sum beside
    # 3e38 loses also in 64 bits
    import depthwise_pointwise_convolution_amd as F
    t = O.TYPES[dtype]
    g = _gen(V)
    R = 3
    logits = torch.randn(R * W, V, generator=g).to(t)
    logits[0] = torch.finfo(t).min
    logits[W + 1, [2, V - 1]] = math.inf
    logits[2 * W:] = torch.finfo(t).min
    scores = -0.1 - torch.arange(R * W).float() / 64
    _, nxt, par, tok, _ = _run_beam(F, dtype, logits, scores, None, R, W, -1)
    l = logits.double().clamp(max=torch.finfo(torch.float32).max)
    top = l.max(-1, keepdim=True).values
    logp = (l - top) - torch.log(torch.exp(l - top).sum(-1, keepdim=True))
    best, at = torch.sort((scores.double()[:, None] + logp).reshape(R, W * V), descending=True, stable=True)
    best, at = best[:, :W].reshape(-1), at[:, :W].reshape(-1)
    assert par.tolist() == (at // V).tolist() and tok.tolist() == (at % V).tolist()
    assert ((nxt.double() - best).abs() <= 2.0 ** -20 + 2.0 ** -23 * best.abs()).all()
