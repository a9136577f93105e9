"""Refusals of the gated delta rule, the microscaled 4-bit calls and the verification of drafted tokens: every bad
argument is told on the host, by status and text, before anything is enqueued (so no GPU is needed)."""
import math

import pytest

from test_seq_abi import BASE, _F, _refused

DELTA = ("q", "k", "v", "a", "b", "A", "dt_bias", "norm", "z", "cu", "slots", "carry", "state", "workspace", "y")
DELTA_STEP = ("q", "k", "v", "a", "b", "A", "dt_bias", "norm", "z", "slots", "state", "y")


def _delta(names, change):
    F = _F()
    ptr = {**{k: BASE for k in names}, **{k: v for k, v in change.items() if k in names}}
    k = {"dtype": "bf16", "Hk": 2, "Hv": 4, "Dk": 64, "Dv": 32, "tokens": 2, "seqs": 2, "slots": 2,
         **{n: v for n, v in change.items() if n not in names}}
    call = F.fcm_delta_fwd if names is DELTA else F.fcm_delta_step
    return lambda: call(F.delta_problem(**k), *[ptr[n] for n in names], stream=0)


@pytest.mark.parametrize("change,status,word", [
    ({k: None}, 1, f"{k} is NULL") for k in ("q", "k", "v", "a", "b", "A", "cu", "workspace", "y")] + [
    ({k: BASE + 1}, 1, "misaligned") for k in ("q", "k", "v", "a", "b", "A", "dt_bias", "norm", "z", "cu", "slots",
                                               "carry", "state", "workspace", "y")] + [
    ({"workspace": BASE + 8}, 1, "misaligned"), ({"state": None}, 1, "need a state"), ({"Hk": 3}, 1, "divide"),
    ({"Hk": 0}, 1, "positive"), ({"Dk": 0}, 1, "positive"), ({"Dv": -1}, 1, "positive"), ({"Dk": 257}, 2, "256"),
    ({"Dv": 257}, 2, "256"), ({"Hk": 1, "Hv": 1 << 17}, 2, "2^16"), ({"eps": 0.0}, 1, "eps"), ({"eps": -1.0}, 1, "eps"),
    ({"eps": math.nan}, 1, "eps"), ({"eps": math.inf}, 1, "eps"), ({"scale": math.inf}, 1, "scale"),
    ({"scale": math.nan}, 1, "scale"), ({"dtype": 3}, 2, "int8"), ({"dtype": 9}, 1, "fcm_dtype"), ({"tokens": -1}, 1, "negative"),
    ({"seqs": -1}, 1, "negative"), ({"slots": None, "seqs": 3}, 1, "at least seqs slots"), ({"ldq": 127}, 1, "stride"),
    ({"ldk": 1}, 1, "stride"), ({"ldv": 127}, 1, "stride"), ({"lda": 3}, 1, "stride"), ({"ldb": 3}, 1, "stride"),
    ({"ldz": 100}, 1, "stride"), ({"ldy": -128}, 1, "stride"), ({"ldy": (1 << 40) + 1}, 1, "2^40"), ({"ldy": 1 << 22}, 2, "2^22"), ({"ldv": 1 << 30}, 2, "2^22"),
    ({"tokens": (1 << 31) - 1}, 1, "2^30"), ({"tokens": 1 << 29, "Hv": 1 << 14}, 2, "one launch"),
    ({"seqs": 1 << 24, "slots": 1 << 24}, 2, "one launch")])
def test_delta_refusals(change, status, word):
    change = dict(change)
    if "slots" in change and change["slots"] is not None and change["slots"] != BASE + 1:
        n = change.pop("slots")
        F = _F()
        k = {"dtype": "bf16", "Hk": 2, "Hv": 4, "Dk": 64, "Dv": 32, "tokens": 2, "seqs": 2, **change, "slots": n}
        _refused(lambda: F.fcm_delta_fwd(F.delta_problem(**k), *[BASE] * 15, stream=0), status, word)
        return
    _refused(_delta(DELTA, change), status, word)


@pytest.mark.parametrize("change,status,word", [
    ({k: None}, 1, f"{k} is NULL") for k in ("q", "k", "v", "a", "b", "A", "state", "y")] + [
    ({"tokens": 3}, 1, "tokens == seqs"), ({"slots": None, "tokens": 3, "seqs": 3}, 1, "at least seqs slots"),
    ({"Dk": 300}, 2, "256"), ({"state": BASE + 2}, 1, "misaligned")])
def test_delta_step_refusals(change, status, word):
    _refused(_delta(DELTA_STEP, change), status, word)


def test_delta_flags_are_checked():
    F = _F()
    for name in ("qk_norm", "softplus"):
        p = F.delta_problem("f16", 1, 1, 64, 64, tokens=1, seqs=1, slots=1)
        setattr(p, name, 2)
        _refused(lambda: F.fcm_delta_workspace(p), 1, name)


@pytest.mark.parametrize("T,B", [(0, 1), (1, 1), (64, 1), (65, 1), (777, 4), (8192, 11), (500, 500), (64 * 7, 7)])
def test_delta_places_hold_the_chunks_of_any_split(T, B):
    # sequence b's chunks start at cu[b] // 64 + b: however the tokens are divided they do not meet, and the last is
    # below tokens // 64 + seqs + 1
    import random
    F = _F()
    size = F.fcm_delta_workspace(F.delta_problem("bf16", 1, 2, 64, 32, tokens=T, seqs=B, slots=B))
    more = F.fcm_delta_workspace(F.delta_problem("bf16", 1, 2, 64, 32, tokens=T, seqs=B + 1, slots=B + 1))
    one = more - size  # a place
    assert size >= (T // 64 + B + 1) * one and one > 0
    r = random.Random(T)
    for _ in range(100):
        cuts = sorted(r.choice((0, T, r.randrange(T + 1))) for _ in range(B - 1))
        cu = [0] + cuts + [T]
        at = -1
        for b in range(B):
            first = cu[b] // 64 + b
            assert first > at
            at = max(first, first + -(-(cu[b + 1] - cu[b]) // 64) - 1)
        assert at < T // 64 + B + 1


@pytest.mark.parametrize("change,status,word", [
    ({"x": None}, 1, "x is NULL"), ({"q": None}, 1, "q is NULL"), ({"scales": None}, 1, "scales is NULL"),
    ({"x": BASE + 1}, 1, "misaligned"), ({"q": BASE + 4}, 1, "misaligned"), ({"C": 48}, 2, "multiple of 32"),
    ({"C": 0}, 1, "positive"), ({"M": -1}, 1, "not negative"), ({"C": 1 << 21}, 2, "2^20"), ({"ldx": 63}, 1, "stride"),
    ({"dtype": 3}, 2, "int8"), ({"M": 1 << 30, "C": 1 << 10}, 2, "2^36")])
def test_mx4_quantize_refusals(change, status, word):
    F = _F()
    ptr = {k: change.get(k, BASE) for k in ("x", "q", "scales")}
    k = {"dtype": "bf16", "M": 2, "C": 64, **{n: v for n, v in change.items() if n not in ptr}}
    _refused(lambda: F.fcm_mx4_quantize(F.mx4_problem(**k), ptr["x"], ptr["q"], ptr["scales"], stream=0), status, word)
    if "ldx" in k:
        k["ldy"] = k.pop("ldx")
    word = word.replace("x is", "y is")
    _refused(lambda: F.fcm_mx4_dequantize(F.mx4_problem(**k), ptr["q"], ptr["scales"], ptr["x"], stream=0), status, word)


MX4 = ("x", "q", "scales", "bias", "y")
MX4X4 = ("xq", "xscales", "q", "scales", "bias", "y")


@pytest.mark.parametrize("names,change,status,word", [
    (MX4, {k: None}, 1, f"{k} is NULL") for k in ("x", "q", "scales", "y")] + [
    (MX4X4, {k: None}, 1, f"{k} is NULL") for k in ("xq", "xscales", "q", "scales", "y")] + [
    (MX4, {"x": BASE + 8}, 1, "misaligned"), (MX4, {"q": BASE + 8}, 1, "misaligned"), (MX4X4, {"xq": BASE + 8}, 1, "misaligned"),
    (MX4, {"bias": BASE + 2}, 1, "misaligned"), (MX4X4, {"y": BASE + 1}, 1, "misaligned"), (MX4, {"ldx": 132}, 1, "multiple of 8"),
    (MX4, {"ldx": 1 << 26}, 2, "2^26"), (MX4, {"ldy": 10}, 1, "stride"), (MX4X4, {"ldy": 10}, 1, "stride"),
    (MX4, {"dtype": "f32"}, 2, "16-bit"), (MX4X4, {"dtype": "f32"}, 2, "16-bit"), (MX4, {"act": 7}, 1, "fcm_act"),
    (MX4, {"C": 40}, 2, "multiple of 32"), (MX4, {"K": 0}, 1, "positive"), (MX4X4, {"M": (1 << 20) + 1}, 2, "2^20"),
    (MX4X4, {"M": 1 << 20, "K": 1 << 24}, 2, "one launch")])
def test_mx4_refusals(names, change, status, word):
    F = _F()
    ptr = {**{k: BASE for k in names}, **{k: v for k, v in change.items() if k in names}}
    k = {"dtype": "bf16", "M": 2, "C": 128, "K": 64, **{n: v for n, v in change.items() if n not in names}}
    call = F.fcm_mx4_fwd if names is MX4 else F.fcm_mx4x4_fwd
    _refused(lambda: call(F.mx4_problem(**k), *[ptr[n] for n in names], stream=0), status, word)


DRAFT = ("target", "draft", "tokens", "counts", "uniform", "workspace", "accepted", "next")


@pytest.mark.parametrize("change,status,word", [
    ({k: None}, 1, f"{k} is NULL") for k in ("target", "tokens", "uniform", "workspace", "accepted", "next")] + [
    ({k: BASE + 1}, 1, "misaligned") for k in ("target", "draft", "tokens", "counts", "uniform", "accepted", "next")] + [
    ({"workspace": BASE + 8}, 1, "misaligned"), ({"drafts": 0}, 1, "positive"), ({"drafts": 65}, 2, "64"), ({"vocab": 0}, 1, "positive"),
    ({"requests": -1}, 1, "not negative"), ({"vocab": (1 << 31) - 1}, 2, "2^31 - 2^25"), ({"temperature": -1.0}, 1, "temperature"),
    ({"temperature": math.inf}, 1, "temperature"), ({"temperature": math.nan}, 1, "temperature"), ({"ldt": 99}, 1, "stride"),
    ({"ldd": 1}, 1, "stride"), ({"dtype": 3}, 2, "int8"), ({"requests": 1 << 25}, 2, "2^24"),
    ({"requests": 1 << 20, "vocab": 1 << 24}, 2, "one launch")])
def test_draft_refusals(change, status, word):
    F = _F()
    ptr = {**{k: BASE for k in DRAFT}, **{k: v for k, v in change.items() if k in DRAFT}}
    k = {"dtype": "f16", "requests": 2, "drafts": 4, "vocab": 100, **{n: v for n, v in change.items() if n not in DRAFT}}
    _refused(lambda: F.fcm_draft_verify(F.draft_problem(**k), *[ptr[n] for n in DRAFT], stream=0), status, word)


def test_workspace_of_a_bad_problem():
    F = _F()
    _refused(lambda: F.fcm_delta_workspace(F.delta_problem("f16", 1, 1, 999, 64)), 1, "256")
    _refused(lambda: F.fcm_draft_workspace(F.draft_problem("f16", 1, 99, 64)), 1, "64")
    assert F.fcm_delta_workspace(F.delta_problem("f16", 1, 1, 64, 64, tokens=0, seqs=0)) > 0


def test_nothing_to_do():
    # no sequences, rows or requests: accepted without a launch
    F = _F()
    F.fcm_delta_fwd(F.delta_problem("f16", 1, 1, 64, 64, tokens=0, seqs=0), *[BASE] * 15, stream=0)
    F.fcm_delta_step(F.delta_problem("f16", 1, 1, 64, 64, tokens=0, seqs=0), *[BASE] * 12, stream=0)
    F.fcm_mx4_quantize(F.mx4_problem("f16", 0, 64), None, None, None, stream=0)
    F.fcm_mx4_dequantize(F.mx4_problem("f16", 0, 64), None, None, None, stream=0)
    F.fcm_mx4_fwd(F.mx4_problem("f16", 0, 64, 8), None, BASE, BASE, None, None, stream=0)
    F.fcm_mx4x4_fwd(F.mx4_problem("f16", 0, 64, 8), None, None, BASE, BASE, None, None, stream=0)
    F.fcm_draft_verify(F.draft_problem("f16", 0, 4, 64), *[None] * 8, stream=0)
