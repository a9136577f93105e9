"""Refusals of the sequence operators: every bad argument is told on the host, by status and text,
before anything is enqueued (so no GPU is needed)."""
import os

import pytest

BASE = 1 << 20  # an aligned address that is never followed


def _F():
    import depthwise_pointwise_convolution_amd as F
    try:
        F.lib()
    except F.FcmError as e:
        pytest.skip(f"libfcm.so not built: {e}")
    return F


def _refused(call, status, word):
    F = _F()
    with pytest.raises(F.FcmError) as e:
        call()
    assert e.value.status == status, str(e.value)
    assert word in str(e.value), str(e.value)
    assert word in F.fcm_last_error()


def _dw1d(F, prob=None, x=BASE, w=BASE, bias=None, cu=BASE, slots=BASE, carry=None, state=BASE, y=2 * BASE, **k):
    k = {"dtype": "bf16", "D": 64, "W": 4, "tokens": 8, "seqs": 2, "slots": 2, **k}
    return lambda: F.fcm_dw1d_fwd(prob or F.dw1d_problem(**k), x, w, bias, cu, slots, carry, state, y, stream=0)


@pytest.mark.parametrize("change,status,word", [
    ({"x": None}, 1, "x is NULL"), ({"w": None}, 1, "w is NULL"), ({"cu": None}, 1, "cu is NULL"),
    ({"y": None}, 1, "y is NULL"), ({"x": BASE + 1}, 1, "misaligned"), ({"bias": BASE + 2}, 1, "misaligned"),
    ({"carry": BASE + 2}, 1, "misaligned"), ({"state": None}, 1, "need a state"),
    ({"slots": None, "seqs": 5}, 1, "misaligned"), ({"ldx": 63}, 1, "stride"), ({"ldy": 8}, 1, "stride"),
    ({"ldx": -64}, 1, "stride"), ({"D": 0}, 1, "positive"), ({"W": 0}, 1, "positive"), ({"tokens": -1}, 1, "negative"),
    ({"seqs": -1}, 1, "negative"), ({"W": 9}, 2, "2 to 8 taps"), ({"W": 1}, 2, "2 to 8 taps"),
    ({"dtype": 3}, 2, "int8"), ({"dtype": 9}, 1, "fcm_dtype"), ({"D": 1 << 25}, 2, "2^24"),
    ({"tokens": (1 << 31) - 1}, 1, "2^30"), ({"state": BASE + 1}, 1, "misaligned")])
def test_dw1d_refusals(change, status, word):
    F = _F()
    if change.get("slots", 0) is None:
        # slots == NULL: sequence b lives in slot b, so there have to be that many
        prob = F.dw1d_problem("bf16", 64, 4, tokens=8, seqs=5, slots=2)
        _refused(_dw1d(F, prob=prob, slots=None), 1, "at least seqs slots")
        return
    _refused(_dw1d(F, **change), status, word)


def test_step_refusals():
    F = _F()
    p = F.dw1d_problem("f16", 64, 4, tokens=3, seqs=2, slots=4)
    _refused(lambda: F.fcm_dw1d_step(p, BASE, BASE, None, BASE, BASE, BASE, stream=0), 1, "tokens == seqs")
    p = F.dw1d_problem("f16", 64, 4, tokens=2, seqs=2, slots=4)
    _refused(lambda: F.fcm_dw1d_step(p, BASE, BASE, None, BASE, None, BASE, stream=0), 1, "state is NULL")
    p = F.scan_problem("f16", 64, 16, tokens=3, seqs=2, slots=4)
    _refused(lambda: F.fcm_scan_step(p, *[BASE] * 7, None, BASE, BASE, BASE, stream=0), 1, "tokens == seqs")
    p = F.scan_problem("f16", 64, 16, tokens=2, seqs=2, slots=1)
    _refused(lambda: F.fcm_scan_step(p, *[BASE] * 7, None, None, BASE, BASE, stream=0), 1, "at least seqs slots")


SCAN = ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias", "z", "cu", "slots", "carry", "state", "workspace", "y")


@pytest.mark.parametrize("change,status,word", [
    ({k: None}, 1, f"{k} is NULL") for k in ("x", "dt", "A", "Bm", "Cm", "cu", "y")] + [
    ({"A": BASE + 2}, 1, "misaligned"), ({"z": BASE + 1}, 1, "misaligned"), ({"skip": BASE + 1}, 1, "misaligned"),
    ({"state": None}, 1, "need a state"), ({"ldb": 15}, 1, "stride"), ({"ldz": 1}, 1, "stride"),
    ({"N": 0}, 1, "positive"), ({"N": 65}, 2, "64 states"), ({"groups": 3}, 1, "divide"), ({"groups": -1}, 1, "negative"),
    ({"dtype": 3}, 2, "int8"), ({"tokens": -1}, 1, "negative")])
def test_scan_refusals(change, status, word):
    F = _F()
    ptr = {**{k: BASE for k in SCAN}, **{k: v for k, v in change.items() if k in SCAN}}
    k = {"dtype": "bf16", "D": 64, "N": 16, "tokens": 8, "seqs": 2, "slots": 2,
         **{n: v for n, v in change.items() if n not in SCAN}}
    _refused(lambda: F.fcm_scan_fwd(F.scan_problem(**k), *[ptr[n] for n in SCAN], stream=0), status, word)


def test_workspace_of_a_bad_problem():
    F = _F()
    _refused(lambda: F.fcm_scan_workspace(F.scan_problem("f16", 64, 99)), 1, "64 states")
    _refused(lambda: F.fcm_beam_workspace(F.beam_problem("f16", 1, 40, 100)), 1, "32 beams")


@pytest.mark.parametrize("t", ["x", b"x", 1.0, [0]])
def test_only_tensors_and_addresses_are_pointers(t):
    F = _F()
    with pytest.raises(AttributeError):
        F._ptr(t)
    assert F._ptr(None) is None and F._ptr(4096) == 4096


@pytest.mark.parametrize("T,B,D,N,G", [(1, 1, 64, 16, 1), (9, 3, 64, 16, 1), (100, 7, 300, 5, 3), (2048, 1, 2048, 16, 1),
                                       (777, 4, 1026, 24, 2), (8192, 11, 4096, 16, 1), (16000, 1, 256, 64, 1),
                                       (65536, 2, 128, 8, 1), (500, 500, 64, 16, 1)])
def test_scan_workspace_holds_the_chunks_of_any_split(T, B, D, N, G):
    # the workspace has tokens // len + seqs chunks of (N + 1) * D floats, len a power of two; however
    # the tokens are divided among the sequences, their chunks (one at least each) fit
    import random
    F = _F()
    size = F.fcm_scan_workspace(F.scan_problem("bf16", D, N, groups=G, tokens=T, seqs=B))
    if size == 0:
        return
    chunks, rest = divmod(size, (N + 1) * D * 4)
    lens = [1 << k for k in range(3, 20) if T // (1 << k) + B == chunks]
    assert rest == 0 and lens, (size, chunks)
    r = random.Random(T)
    for _ in range(50):
        cuts = sorted(r.choice((0, T, r.randrange(T + 1))) for _ in range(B - 1))
        parts = [b - a for a, b in zip([0] + cuts, cuts + [T])]
        assert sum(max(1, -(-n // lens[0])) for n in parts) <= chunks


Q4 = ("x", "q", "scales", "zeros", "bias", "y")


@pytest.mark.parametrize("change,status,word", [
    ({"x": None}, 1, "x is NULL"), ({"q": None}, 1, "q is NULL"), ({"scales": None}, 1, "scales is NULL"),
    ({"y": None}, 1, "y is NULL"), ({"x": BASE + 8}, 1, "misaligned"), ({"q": BASE + 2}, 1, "misaligned"),
    ({"scales": BASE + 1}, 1, "misaligned"), ({"bias": BASE + 2}, 1, "misaligned"), ({"C": 60}, 2, "multiple of 8"),
    ({"group": 16}, 2, "32, 64 or 128"), ({"dtype": "f32"}, 2, "16-bit"), ({"act": 7}, 1, "fcm_act"),
    ({"ldx": 132}, 1, "multiple of 8"), ({"ldy": 10}, 1, "stride"), ({"M": -1}, 1, "not negative"),
    ({"K": 0}, 1, "positive"), ({"C": 0}, 1, "positive")])
def test_q4_refusals(change, status, word):
    F = _F()
    ptr = {**{k: BASE for k in Q4}, **{k: v for k, v in change.items() if k in Q4}}
    k = {"dtype": "bf16", "M": 2, "C": 128, "K": 64, "group": 64,
         **{n: v for n, v in change.items() if n not in Q4}}
    _refused(lambda: F.fcm_q4_fwd(F.q4_problem(**k), *[ptr[n] for n in Q4], stream=0), status, word)


BEAM = ("logits", "scores", "done", "workspace", "next_scores", "parent", "token", "next_done")


@pytest.mark.parametrize("change,status,word", [
    ({k: None}, 1, f"{k} is NULL") for k in ("logits", "scores", "workspace", "next_scores", "parent", "token")] + [
    ({"workspace": BASE + 8}, 1, "misaligned"), ({"beams": 0}, 1, "positive"), ({"beams": 33}, 2, "32 beams"),
    ({"vocab": 0}, 1, "positive"), ({"eos": 100}, 1, "eos"), ({"eos": -1}, 1, "need an eos"),
    ({"ldl": 99}, 1, "stride"), ({"requests": -1}, 1, "not negative"),
    ({"beams": 32, "vocab": 1 << 27, "eos": 1}, 2, "2^31"), ({"dtype": 3}, 2, "int8")])
def test_beam_refusals(change, status, word):
    F = _F()
    ptr = {**{k: BASE for k in BEAM}, **{k: v for k, v in change.items() if k in BEAM}}
    k = {"dtype": "f16", "requests": 2, "beams": 4, "vocab": 100, "eos": 2,
         **{n: v for n, v in change.items() if n not in BEAM}}
    _refused(lambda: F.fcm_beam_select(F.beam_problem(**k), *[ptr[n] for n in BEAM], stream=0), status, word)


class _Pool:
    """What fcm_beam_reorder asks of a state tensor."""

    def __init__(self, at, slots, width, size=4):
        self.at, self.shape, self.width, self.size = at, (slots, width), width, size

    def data_ptr(self):
        return self.at

    def stride(self, _):
        return self.width

    def element_size(self):
        return self.size


@pytest.mark.parametrize("change,word", [
    ({"parent": None}, "parent is NULL"), ({"slots": None}, "slots is NULL"), ({"next_slots": None}, "next_slots is NULL"),
    ({"next_slots": BASE}, "distinct"), ({"pools": [_Pool(BASE, 4, 0)]}, "slot's bytes"),
    ({"pools": [_Pool(BASE, 4, 1 << 39)]}, "slot's bytes"), ({"pools": [_Pool(BASE, 4, 8)] * 9}, "npools"), ({"pools": [_Pool(None, 4, 8)]}, "a pool is NULL")])
def test_beam_reorder_refusals(change, word):
    F = _F()
    a = {"parent": BASE, "slots": BASE, "next_slots": 2 * BASE, "pools": [], **change}
    prob = F.beam_problem("f32", 1, 4, 100)
    _refused(lambda: F.fcm_beam_reorder(prob, a["parent"], a["slots"], a["next_slots"], a["pools"], stream=0), 1, word)


def test_empty_batches_are_no_work():
    F = _F()
    F.fcm_dw1d_fwd(F.dw1d_problem("f16", 64, 4, tokens=0, seqs=0), None, BASE, None, BASE, None, None, None, None,
                   stream=0)
    F.fcm_scan_fwd(F.scan_problem("f16", 64, 16, tokens=0, seqs=0), None, None, BASE, None, None, None, None, None,
                   BASE, None, None, None, None, None, stream=0)
    F.fcm_q4_fwd(F.q4_problem("f16", 0, 64, 64), None, BASE, BASE, None, None, None, stream=0)
    F.fcm_beam_select(F.beam_problem("f16", 0, 4, 64), *[None] * 8, stream=0)
    F.fcm_beam_reorder(F.beam_problem("f16", 0, 4, 64), None, None, None, [], stream=0)


def test_null_problem():
    F = _F()
    L = F.lib()
    for name, n in (("fcm_dw1d_fwd", 9), ("fcm_dw1d_step", 7), ("fcm_scan_fwd", 15), ("fcm_scan_step", 12),
                    ("fcm_q4_fwd", 7), ("fcm_beam_select", 9)):
        assert getattr(L, name)(None, *[BASE] * n) == F.FCM_ERR_INVALID_ARG, name
        assert "problem is NULL" in F.fcm_last_error()


def test_sequence_sources_are_built():
    from depthwise_pointwise_convolution_amd import build
    have = {s for s, _ in build.SOURCES}
    on_disk = {"kernels/" + f for f in os.listdir(os.path.join(build.CSRC, "kernels")) if f.endswith(".hip")}
    assert on_disk <= have


# ------------------------------------------------------------------------------------------
# the convenience wrappers' own checks, on the CPU
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("C,group,symmetric", [(64, 32, False), (200, 64, False), (136, 128, True), (32, 32, True)])
def test_quantized_weights_are_within_half_a_step(C, group, symmetric):
    import torch
    from depthwise_pointwise_convolution_amd.sequence import Q4Linear, quantize_q4
    g = torch.Generator().manual_seed(C)
    w = (torch.randn(9, C, generator=g) * 0.1).to(torch.float16)
    w[3] = 0
    w[4] = w[4].abs()
    q, scales, zeros = quantize_q4(w, group, symmetric)
    back = Q4Linear(q, scales, zeros, group=group).weight()
    step = scales.float()[:, torch.arange(C) // group]
    # half a step, and where the rounded scale falls short of the span or the zero is rounded, up to
    # 15 codes times the scale's rounding (2^-11), or another half step at the far end
    assert ((back - w.float()).abs() <= step * (1.0 if not symmetric else 0.5) + step * 15 * 2.0 ** -11 + 1e-9).all()
    assert (back[3] == 0).all()
    assert (zeros is None) == symmetric


def test_wrappers_refuse_wrong_shapes_and_types():
    import torch
    from depthwise_pointwise_convolution_amd.sequence import BeamSearch, Q4Linear, StateSpaceBlock, quantize_q4
    z = torch.zeros
    q, s = z(8, 32, dtype=torch.uint8), z(8, 1, dtype=torch.float16)
    for bad in (lambda: quantize_q4(z(8, 64)), lambda: quantize_q4(z(8, 60, dtype=torch.float16)),
                lambda: quantize_q4(z(8, 64, dtype=torch.float16), 16),
                lambda: Q4Linear(q.int(), s), lambda: Q4Linear(q, s.float()), lambda: Q4Linear(q, s, group=32),
                lambda: Q4Linear(q, s, zeros=z(8, 2, dtype=torch.uint8)), lambda: Q4Linear(q, s, bias=z(7)),
                lambda: Q4Linear(q, s, act="gelu"), lambda: Q4Linear(q, s)(z(2, 63, dtype=torch.float16)),
                lambda: Q4Linear(q, s)(z(2, 64)), lambda: Q4Linear(q, s)(z(64, 2, dtype=torch.float16).t()),
                lambda: StateSpaceBlock(None, z(8, 4), None, None, None, None, z(7, 16), None, None, 1),
                lambda: StateSpaceBlock(None, z(8, 4), z(7), None, None, None, z(8, 16), None, None, 1),
                lambda: BeamSearch(2, 3, 10, z(5, dtype=torch.int32)),
                lambda: BeamSearch(2, 3, 10, z(6)),
                lambda: BeamSearch(1, 2, 10, z(2, dtype=torch.int32)).advance(z(2, 9), []),
                lambda: BeamSearch(1, 2, 10, z(2, dtype=torch.int32)).advance(z(3, 10), [])):
        with pytest.raises(ValueError):
            bad()


def test_a_vocabulary_whose_places_overflow_is_refused():
    # a row is cut into 64 splits at most, of whole blocks of 1024 tokens, so places up to a split
    # and a block behind the vocabulary are computed in 32 bits
    F = _F()
    most = 2 ** 31 - 2 ** 25
    per = -(-(-(-most // 1024)) // 64) * 1024  # tokens of a split
    assert most + per - 1 < 2 ** 31 and -(-most // per) * per + 1024 < 2 ** 31
    assert F.fcm_beam_workspace(F.beam_problem("f16", 1, 1, most)) == -(-most // per) * (8 + 8)
    for vocab in (most + 1, 2 ** 31 - 2 ** 16, 2 ** 31 - 1):
        prob = F.beam_problem("f16", 1, 1, vocab)
        _refused(lambda: F.fcm_beam_select(prob, *[BASE] * 8, stream=0), 2, "vocab")
        with pytest.raises(F.FcmError):
            F.fcm_beam_workspace(prob)


@pytest.mark.parametrize("T,B,D,N,G", [(1 << 24, 4096, 1 << 12, 1, 1 << 12), (1 << 24, 1 << 15, 1 << 10, 4, 1 << 9),
                                       (1 << 29, 1 << 19, 64, 1, 64), (1 << 26, 1 << 15, 256, 64, 1),
                                       (1 << 20, 1 << 11, 1 << 14, 16, 1), (1 << 22, 1, 1 << 12, 1, 1 << 12)])
def test_a_scan_of_any_size_is_a_launch(T, B, D, N, G):
    # a launch has fewer than 2^32 threads: 64 at least for each chunk of a channel group, at most four
    # lanes a channel
    F = _F()
    size = F.fcm_scan_workspace(F.scan_problem("bf16", D, N, groups=G, tokens=T, seqs=B))
    chunks, rest = divmod(size, (N + 1) * D * 4)
    lanes = 1 if N <= 16 else 2 if N <= 32 else 4
    assert rest == 0 and chunks * G * -(-(D // G) * lanes // 64) * 64 < 2 ** 32


def test_launches_past_2_to_the_32_threads_are_refused():
    F = _F()
    # selection: a wave for each split of at least 1024 tokens
    prob = F.beam_problem("f16", 1 << 20, 1, 1 << 16, eos=1)
    _refused(lambda: F.fcm_beam_select(prob, *[BASE] * 8, stream=0), 2, "requests * beams * vocab")
    prob = F.beam_problem("f16", (1 << 20) - 1, 1, 1 << 16)
    assert F.fcm_beam_workspace(prob) == ((1 << 20) - 1) * 64 * 16
    # reordering: 256 threads for each 16 KB of each beam's states
    prob = F.beam_problem("f16", 1 << 10, 8, 100)
    pool = _Pool(BASE, 4, 1 << 23)
    _refused(lambda: F.fcm_beam_reorder(prob, BASE, BASE, 2 * BASE, [pool], stream=0), 2, "states")
