"""The kernels that large sizes select, on the smallest sizes that select them, with ragged ends, against the
definitions in 64 bits (on some channels: each stands for itself).  The rules that select them are repeated
here and held against the sources, so that a case which no longer reaches its kernel shows."""
import os
import re

import pytest
import torch

import seq_oracle as O
from gpu_util import gpu_available
from test_seq_gpu import _gen, _normal, _offsets, _q4_inputs, _run_scan, _scan_inputs, _within

gpu = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def on_gpu(f):
    for m in gpu:
        f = m(f)
    return f


def _source(name):
    import depthwise_pointwise_convolution_amd as F
    with open(os.path.join(os.path.dirname(F.__file__), "csrc", "kernels", name)) as f:
        return re.sub(r"\s+", " ", f.read())


def _some(D, *always, count=24):
    """Channels to check: the first and last, others in between, and `always`."""
    return sorted({0, 1, 63, 64, D - 1, D - 2, *always, *torch.randperm(D, generator=_gen(D))[:count].tolist()} &
                  set(range(D)))


# ------------------------------------------------------------------------------------------
# scan of prompts: one lane a channel, every chunk length, tiles that a chunk does not fit in
# ------------------------------------------------------------------------------------------
#: dtype, D, N, groups, lengths, gate -> lanes of a channel, tokens of a chunk, of a tile
SCANS = [
    ("bf16", 4096, 16, 1, [60, 0, 121, 19], True, 1, 16, 128), ("f16", 4100, 8, 1, [500, 1, 299], True, 1, 32, 256),
    ("f32", 2050, 16, 2, [3001, 2999], True, 1, 64, 128), ("bf16", 1026, 5, 1, [997, 0, 0, 66], False, 1, 16, 256),
    ("bf16", 4096, 64, 1, [3070, 1, 65], True, 4, 64, 32), ("f16", 4160, 40, 1, [130, 3003], False, 4, 64, 40),
    ("f32", 4096, 24, 1, [3135], True, 2, 64, 84), ("f16", 64, 16, 1, [17003], True, 1, 128, 128),
    ("bf16", 2048, 1, 2, [777, 778], True, 1, 32, 256)]


def _waves(T, D, G):
    return T * ((D // G + 63) // 64) * G // 4096


@pytest.mark.parametrize("case", SCANS, ids=str)
def test_scan_cases_reach_their_kernels(case):
    import depthwise_pointwise_convolution_amd as F
    dtype, D, N, G, lens, _, lanes, length, tile = case
    T, B = sum(lens), len(lens)
    text = _source("scan.hip")
    # fwd_states: few sends up to 16 states to more lanes
    assert "const bool few = token_waves(a.tokens, a.D, a.groups) < 3;" in text
    assert N > 16 or _waves(T, D, G) >= 3
    NP, Q = next((p, q) for most, p, q in ((8, 8, 1), (16, 16, 1), (24, 12, 2), (32, 16, 2), (48, 12, 4), (64, 16, 4))
                 if N <= most)
    for most, p, q in ((8, 8, 1), (16, 16, 1), (24, 12, 2), (32, 16, 2), (48, 12, 4)):
        assert re.search(rf"if \(a\.N <= {most}\) return (few \? run_fwd<T, 4, \d>\(a, s\) : )?run_fwd<T, {p}, {q}>", text), most
    assert (Q, 16384 // (2 * NP * Q * 4) // 4 * 4) == (lanes, tile)
    assert "return 16384 / (2 * NS * 4) / kTurn * kTurn;" in text and "kTurn = 4;" in text
    # the workspace tells the chunks' length
    try:
        size = F.fcm_scan_workspace(F.scan_problem(dtype, D, N, groups=G, tokens=T, seqs=B))
    except F.FcmError as e:
        pytest.skip(f"libfcm.so not built: {e}")
    assert size == (T // length + B) * D * (N + 1) * 4


def _channels_of(v, D, G, N, sub):
    """The inputs of the channels `sub` of one group each, and that group's B and C."""
    per = D // G
    for g in range(G):
        mine = [d for d in sub if d // per == g]
        if mine:
            part = {k: v[k][:, mine] for k in ("x", "dt", "z") if v[k] is not None}
            part |= {k: v[k][mine] for k in ("A", "skip", "dt_bias")}
            part |= {k: v[k][:, g * N:(g + 1) * N] for k in ("Bm", "Cm")}
            yield mine, {**part, "z": part.get("z"), "state": v["state"][:, mine]}


def _check_scan(dtype, v, D, N, G, lens, slots, carry, sub, y, state, idle=()):
    for mine, p in _channels_of(v, D, G, N, sub):
        args = [p[k] for k in ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias", "z")]
        ref, tol, sref, stol, _ = O.scan(dtype, *args, _offsets(lens), slots, carry, p["state"], 1, True)
        for b in idle:
            ref[b] = 0
        _within(y[:, mine], ref, tol, "y")
        _within(state[:, mine], sref, stol, "state")


@on_gpu
@pytest.mark.parametrize("case", SCANS, ids=str)
def test_scan_of_many_tokens(case):
    import depthwise_pointwise_convolution_amd as F
    dtype, D, N, G, lens, gate, *_ = case
    g = _gen(D + N)
    B, T, cu = len(lens), sum(lens), _offsets(lens)
    v = _scan_inputs(g, dtype, T, D, N, G, B, B + 1, gate)
    v["A"][:, ::2] *= 2.0 ** -6  # slow decays among them: what a chunk hands on is seen far behind
    slots = torch.randperm(B + 1, generator=g)[:B].tolist()
    if B > 2:
        slots[1] = -1
    carry = [1] + torch.randint(0, 2, (B - 1,), generator=g).tolist()
    pads = (0, 0, 0, 0) if D % 8 == 0 else (2, 0, 3, 1)
    y, state = _run_scan(F, v, dtype, cu, slots, carry, G, pads)
    assert not y.isnan().any() and not state.isnan().any()
    per = D // G
    _check_scan(dtype, v, D, N, G, lens, slots, carry, _some(D, per - 1, per, 255, 256), y, state)


@on_gpu
def test_scan_of_one_long_prompt_among_short_ones():
    # the limit on chunks is one of all sequences together: here one has a thousand
    import depthwise_pointwise_convolution_amd as F
    g = _gen(31)
    D, N, lens = 64, 16, [1, 7997, 0, 2]
    B, T, cu = 4, sum(lens), _offsets(lens)
    size = F.fcm_scan_workspace(F.scan_problem("bf16", D, N, tokens=T, seqs=B))
    assert size == (T // 8 + B) * D * (N + 1) * 4
    v = _scan_inputs(g, "bf16", T, D, N, 1, B, B, True)
    v["A"][:, ::2] *= 2.0 ** -8
    y, state = _run_scan(F, v, "bf16", cu, [0, 1, 2, 3], [1] * B, 1, (0, 0, 0, 0))
    _check_scan("bf16", v, D, N, 1, lens, [0, 1, 2, 3], [1] * B, list(range(D)), y, state)


# ------------------------------------------------------------------------------------------
# scan of tokens: two rows a thread
# ------------------------------------------------------------------------------------------
#: dtype, batch, D, N, groups
STEPS = [("bf16", 65, 4096, 16, 1), ("f16", 257, 4100, 4, 1), ("f32", 131, 4098, 8, 2), ("bf16", 33, 4104, 32, 1),
         ("f16", 17, 4096, 64, 1), ("f32", 19, 4097, 48, 1), ("bf16", 65, 4100, 12, 1)]


@pytest.mark.parametrize("case", STEPS, ids=str)
def test_token_cases_take_two_rows_a_thread(case):
    _, B, D, N, _ = case
    text = _source("scan.hip")
    Q = next(q for most, q in ((4, 1), (8, 2), (16, 4), (32, 8), (64, 16)) if N <= most)
    assert "(long long)a.seqs * cblocks >= 4096" in text and "if (a.N <= 16) return run_step4<T, 4>" in text
    assert N % 4 == 0 and B * -(-D // (256 // Q)) >= 4096 and B % 2 == 1


@on_gpu
@pytest.mark.parametrize("case", STEPS, ids=str)
def test_scan_of_a_token_of_many_sequences(case):
    import depthwise_pointwise_convolution_amd as F
    dtype, B, D, N, G = case
    g = _gen(B + D)
    v = _scan_inputs(g, dtype, B, D, N, G, B, B + 3, True)
    slots = torch.randperm(B + 3, generator=g)[:B].tolist()
    idle = [0, 5, 6, B - 1]  # the first and second of a pair, a whole one's two, the odd one at the end
    for i, b in enumerate(idle):
        slots[b] = -1 if i % 2 else B + 3
    y, state = _run_scan(F, v, dtype, None, slots, None, G, (0, 0, 0, 0), step=True)
    assert not y.isnan().any()
    _check_scan(dtype, v, D, N, G, [1] * B, slots, [1] * B, _some(D, D // G - 1, D // G), y, state, idle)


# ------------------------------------------------------------------------------------------
# 4-bit layer: two and four 16-channel tiles a workgroup
# ------------------------------------------------------------------------------------------
#: dtype, M, C, K, group, zeros -> 16-channel tiles of a workgroup.  C is a multiple of 128 (wide loads) or
#: not, and below or above the 1024 channels whose scales are staged at a time
Q4S = [("bf16", 1, 384, 16393, 128, True, 2), ("f16", 1, 1288, 16390, 32, False, 2), ("bf16", 5, 1280, 16399, 64, True, 2),
       ("f16", 8, 200, 16401, 128, True, 2), ("bf16", 16, 1280, 16393, 32, True, 2), ("f16", 12, 1160, 16417, 64, True, 2),
       ("bf16", 17, 1280, 16395, 64, False, 2), ("f16", 29, 136, 16393, 32, True, 2), ("f16", 45, 384, 8203, 128, True, 2),
       ("bf16", 16, 384, 49153, 64, True, 4), ("f16", 9, 1280, 49169, 32, True, 4), ("bf16", 13, 256, 49207, 128, False, 4)]


@pytest.mark.parametrize("case", Q4S, ids=str)
def test_4_bit_cases_reach_their_kernels(case):
    _, M, C, K, _, _, tiles = case
    text = _source("q4.hip")
    assert "if (rows >= 3072) return go(integral_constant<int, 4>(), integral_constant<int, 4>());" in text
    assert "if (rows >= 1024) return go(integral_constant<int, 2>(), integral_constant<int, 4>());" in text
    assert "if constexpr (NI == 4 && MT == 1 && WIDE)" in text
    NI, MT = next(v for most, v in ((4, (1, 1)), (8, (2, 1)), (16, (4, 1)), (1 << 20, (4, 2))) if M <= most)
    rows = -(-K // 16) * -(-M // (4 * NI * MT))
    four = (NI, MT) == (4, 1) and C % 128 == 0 and rows >= 3072
    assert rows >= 1024 and (4 if four else 2) == tiles
    assert K % (16 * tiles) != 0


@on_gpu
@pytest.mark.parametrize("case", Q4S, ids=str)
def test_4_bit_layer_of_many_channels(case):
    import depthwise_pointwise_convolution_amd as F
    dtype, M, C, K, group, zeros, tiles = case
    g = _gen(K + C)
    v = _q4_inputs(g, dtype, M, C, K, group, zeros)
    some = _some(K, *range(K - 16 * tiles - 2, K), 16 * tiles - 1, 16 * tiles, count=300)
    # random values, and whole numbers with scales that are powers of two, whose sums are exact
    x = torch.randint(-2, 3, (M, C), generator=g).to(O.TYPES[dtype])
    scales = (2.0 ** torch.randint(-6, -2, v["scales"].shape, generator=g)).to(O.TYPES[dtype])
    for exact, xs, ss, bias in ((False, v["x"], v["scales"], v["bias"]), (True, x, scales, None)):
        y = torch.full((M, K), float("nan"), dtype=O.TYPES[dtype], device="cuda")
        F.fcm_q4_fwd(F.q4_problem(dtype, M, C, K, group=group), xs.cuda(), v["q"].cuda(), ss.cuda(),
                     None if v["zeros"] is None else v["zeros"].cuda(), None if bias is None else bias.cuda(), y)
        assert not y.isnan().any()
        ref, tol = O.q4(dtype, xs, v["q"][some], ss[some], None if v["zeros"] is None else v["zeros"][some],
                        None if bias is None else bias[some], group, "none")
        if exact:
            assert torch.equal(y[:, some].cpu(), ref.float().to(O.TYPES[dtype]))
        else:
            _within(y[:, some], ref, tol, "y")


# ------------------------------------------------------------------------------------------
# depthwise layer: outputs past the L2s
# ------------------------------------------------------------------------------------------
#: dtype, D, W, lengths
LAYERS = [("bf16", 4096, 4, [1000, 0, 2, 3097]), ("f16", 8200, 3, [2051]), ("f32", 4100, 7, [1, 1023, 1025])]


@pytest.mark.parametrize("case", LAYERS, ids=str)
def test_depthwise_cases_stream_their_outputs(case):
    dtype, D, _, lens = case
    assert "const bool past_l2 = (long long)a.tokens * a.D * (int)sizeof(T) > (32ll << 20);" in _source("dw1d.hip")
    size = {"f32": 4}.get(dtype, 2)
    assert sum(lens) * D * size > 32 << 20 and D * size % 16 == 0 and sum(lens) % 8 != 0


@on_gpu
@pytest.mark.parametrize("case", LAYERS, ids=str)
def test_depthwise_layer_of_many_tokens(case):
    import depthwise_pointwise_convolution_amd as F
    dtype, D, W, lens = case
    g = _gen(D)
    B, T, cu = len(lens), sum(lens), _offsets(lens)
    x, w, bias = _normal(g, T, D, dtype=dtype), _normal(g, D, W, dtype=dtype, std=0.5), _normal(g, D, std=0.2)
    state = _normal(g, B, W - 1, D, dtype=dtype)
    slots, carry = list(range(B))[::-1], [b % 2 for b in range(B)]
    i32 = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    # rows that go on behind the channels, which have to stay as they are
    pad = 16 // x.element_size()
    whole = torch.full((T, D + pad), float("nan"), dtype=O.TYPES[dtype], device="cuda")
    y, sg = whole[:, :D], state.cuda()
    F.fcm_dw1d_fwd(F.dw1d_problem(dtype, D, W, tokens=T, seqs=B, slots=B, ldy=D + pad), x.cuda(), w.cuda(), bias.cuda(),
                   i32(cu), i32(slots), i32(carry), sg, y)
    assert not y.isnan().any() and whole[:, D:].isnan().all()
    sub = _some(D, 255, 256, 2047, 2048, count=40)
    ref, tol, sref, _ = O.dw1d(dtype, x[:, sub], w[sub], bias[sub], cu, slots, carry, state[:, :, sub], True)
    _within(y[:, sub], ref, tol, "y")
    assert torch.equal(sg[:, :, sub].cpu().double(), sref)
