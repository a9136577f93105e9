"""The recurrent operators' wrappers with their launches stubbed (no GPU): what they pass on, on which
stream, and what they refuse."""
import contextlib

import pytest
import torch

import depthwise_pointwise_convolution_amd.sequence as S

z = torch.zeros
BF = torch.bfloat16
NAMES = {"fcm_dw1d_fwd": 8, "fcm_dw1d_step": 6, "fcm_delta_fwd": 15, "fcm_delta_step": 12, "fcm_mx4_quantize": 3,
         "fcm_mx4_dequantize": 3, "fcm_mx4_fwd": 5, "fcm_mx4x4_fwd": 6, "fcm_draft_verify": 8}


@pytest.fixture
def calls(monkeypatch):
    """(name, problem, pointer arguments, stream) of the launches."""
    got = []

    def stub(name):
        def launch(prob, *args, stream=None):
            assert len(args) == NAMES[name]
            got.append((name, prob, args, torch.cuda.current_stream() if stream is None else stream))
        return launch

    for name in NAMES:
        monkeypatch.setattr(S, name, stub(name))
    monkeypatch.setattr(S, "fcm_delta_workspace", lambda prob: 64)
    monkeypatch.setattr(S, "fcm_draft_workspace", lambda prob: 64)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    monkeypatch.setattr(S, "_on_gpu", lambda t: True)
    return got


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def linear(C, K, dtype=BF, **k):
    return S.MX4Linear(z(K, C // 2, dtype=torch.uint8), z(K, C // 32, dtype=torch.uint8), dtype=dtype, **k)


def block(Hk=1, Hv=2, Dk=4, Dv=8, dim=32, W=4, slots=3, in_proj=None, **k):
    mixed, inner = 2 * Hk * Dk + Hv * Dv, Hv * Dv
    parts = {"conv_w": z(mixed, W, dtype=BF), "conv_b": None, "A": z(Hv), "dt_bias": z(Hv), "norm": z(Dv), **k}
    return S.DeltaRuleBlock(in_proj or linear(dim, mixed + inner + 2 * Hv), parts["conv_w"], parts["conv_b"], parts["A"],
                            parts["dt_bias"], parts["norm"], lambda y: y, Hk, Dk, Dv, slots)


class Stream:
    def __init__(self):
        self.waited = []

    def wait_stream(self, other):
        self.waited.append(other)


@pytest.mark.parametrize("what", ["prompt", "step", "linear", "4-bit tokens", "quantize", "verify"])
def test_a_stream_takes_the_whole_call(calls, monkeypatch, what):
    caller, other = Stream(), Stream()
    now, seen = [caller], []

    @contextlib.contextmanager
    def use(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", use)
    b, lin, both = block(), linear(64, 8), linear(64, 8, quantize_input=True)
    for name in ("empty", "rand"):
        def made(*a, real=getattr(torch, name), **k):
            seen.append(now[-1])
            return real(*a, **k)
        monkeypatch.setattr(torch, name, made)
    if what == "prompt":
        b.prompt(z(5, 32, dtype=BF), ints(0, 2, 5), ints(0, 1), stream=other)
    elif what == "step":
        b.step(z(2, 32, dtype=BF), ints(0, 1), stream=other)
    elif what == "linear":
        lin(z(4, 66, dtype=BF)[:, 1:65], stream=other)
    elif what == "4-bit tokens":
        both(z(4, 64, dtype=BF), stream=other)
    elif what == "quantize":
        S.quantize_mx4(z(4, 64), stream=other)
    else:
        S.DraftVerifier(2, 3, 10)(z(8, 10), z(2, 3, dtype=torch.int32), stream=other)
    assert calls and seen
    assert all(s is other for s in seen + [c[3] for c in calls])
    assert other.waited == [caller] and now == [caller]


def test_a_block_hands_on_its_parts(calls):
    for T, run in ((5, lambda b, x: b.prompt(x, ints(0, 2, 5), ints(0, 1), ints(1, 0))),
                   (1, lambda b, x: b.prompt(x, ints(0, 1), ints(2))), (3, lambda b, x: b.step(x, ints(0, -1, 2)))):
        calls.clear()
        Hk, Hv, Dk, Dv = 2, 6, 4, 8
        mixed, inner = 2 * Hk * Dk + Hv * Dv, Hv * Dv
        wide = torch.arange(T * (mixed + inner + 2 * Hv), dtype=torch.float32).to(BF).reshape(T, -1)
        b = block(Hk, Hv, Dk, Dv, in_proj=lambda x: wide)
        y = run(b, z(T, 32, dtype=BF))
        (_, conv, cargs, _), (_, prob, args, _) = calls
        assert y.shape == (T, inner)
        assert (conv.D, conv.tokens, conv.ldx) == (mixed, T, wide.shape[1] if T > 1 else 0)
        assert (prob.Hk, prob.Hv, prob.Dk, prob.Dv, prob.tokens, prob.slots) == (Hk, Hv, Dk, Dv, T, 3)
        q, k, v, a, bb, A, dt_bias, norm, zz = args[:9]
        u = cargs[-1]
        for t, at, n in ((q, 0, Hk * Dk), (k, Hk * Dk, Hk * Dk), (v, 2 * Hk * Dk, inner)):
            assert t.data_ptr() == u.data_ptr() + 2 * at and t.shape == (T, n)
        for t, at, n in ((zz, mixed, inner), (a, mixed + inner, Hv), (bb, mixed + inner + Hv, Hv)):
            assert t.data_ptr() == wide.data_ptr() + 2 * at and t.shape == (T, n)
        for ld, n in (("ldq", mixed), ("ldk", mixed), ("ldv", mixed), ("lda", wide.shape[1]), ("ldb", wide.shape[1]),
                      ("ldz", wide.shape[1])):
            assert getattr(prob, ld) == (n if T > 1 else 0), ld
        assert any(t is b.state for t in args) and any(t is b.window for t in cargs)


def test_rows_the_product_cannot_take_are_laid_out(calls):
    lin = linear(64, 8)
    rows = torch.arange(400, dtype=torch.float32).to(BF)
    for x in (rows[1:257].reshape(4, 64), rows[:264].reshape(4, 66)[:, :64], rows[:64][None].expand(4, 64),
              rows.as_strided((4, 64), (8, 1))):
        calls.clear()
        lin(x)
        (_, prob, args, _), = calls
        assert args[0].data_ptr() % 16 == 0 and prob.ldx % 8 == 0 and torch.equal(args[0], x)
        assert (prob.ldx or 64) >= 64
    calls.clear()
    wide = z(4, 96, dtype=BF)
    lin(wide[:, :64])
    assert calls[0][1].ldx == 96 and calls[0][2][0].data_ptr() == wide.data_ptr()


def test_tokens_in_codes_are_quantised_first(calls):
    out = z(4, 24, dtype=BF)[:, 8:16]
    lin = linear(64, 8, quantize_input=True, act="relu")
    assert lin(z(4, 64, dtype=BF), out=out) is out
    (first, quant, qargs, _), (second, prob, args, _) = calls
    assert (first, second) == ("fcm_mx4_quantize", "fcm_mx4x4_fwd")
    assert args[0] is qargs[1] and args[1] is qargs[2] and args[5] is out
    assert (quant.M, quant.C, prob.M, prob.C, prob.K, prob.ldy) == (4, 64, 4, 64, 8, 24)


def test_rows_that_stand_and_those_behind():
    verify = S.DraftVerifier(3, 4, 10)
    cu, slots = verify.kept(ints(0, 4, 2), ints(7, 3, 5))
    assert cu.tolist() == [0, 1, 5, 10, 10, 13, 15] and slots.tolist() == [7, -1, 3, -1, 5, -1]
    assert cu.dtype == slots.dtype == torch.int32 and cu.is_contiguous() and slots.is_contiguous()
    cu, slots = S.DraftVerifier(0, 4, 10).kept(ints(), ints())
    assert cu.tolist() == [0] and slots.numel() == 0


def test_refusals(calls):
    lin, b, verify = linear(64, 8), block(), S.DraftVerifier(2, 3, 10)
    x, p, i = z(2, 64, dtype=BF), z(2, 32, dtype=BF), z(2, 3, dtype=torch.int32)
    u8 = torch.uint8
    for call, what in [
            (lambda: S.MX4Linear(z(8, 24, dtype=u8), z(8, 1, dtype=u8)), "multiple of 32"),
            (lambda: S.MX4Linear(z(8, 0, dtype=u8), z(8, 0, dtype=u8)), "multiple of 32"),
            (lambda: S.MX4Linear(z(8, 32, dtype=u8), z(8, 1, dtype=u8)), "scales"),
            (lambda: S.MX4Linear(z(8, 32, dtype=u8), z(8, 2, dtype=BF)), "scales"),
            (lambda: S.MX4Linear(z(8, 32, dtype=u8), z(8, 2, dtype=u8), bias=z(7)), "bias"),
            (lambda: S.MX4Linear(z(8, 32, dtype=u8), z(8, 2, dtype=u8), act="tanh"), "act"),
            (lambda: linear(64, 8, dtype=torch.float32), "dtype"),
            (lambda: S.quantize_mx4(z(2, 48)), "multiple of 32"), (lambda: S.quantize_mx4(z(64)), "multiple of 32"),
            (lambda: S.quantize_mx4(z(64, 2).t()), "contiguous"),
            (lambda: S.quantize_mx4(z(2, 64, dtype=torch.float64)), "float32"),
            (lambda: lin(x.half()), "bfloat16"), (lambda: lin(z(2, 32, dtype=BF)), r"\[rows, 64\]"),
            (lambda: lin(x, out=z(1, 8, dtype=BF)), "out"), (lambda: lin(x, out=z(2, 8)), "out"),
            (lambda: block(A=z(3)), "value heads|conv_w"), (lambda: block(Hk=2, Hv=3), "key heads"),
            (lambda: block(norm=z(7)), "norm"), (lambda: block(dt_bias=z(2, dtype=BF)), "dt_bias"),
            (lambda: block(conv_w=z(25, 4, dtype=BF)), "conv_w"), (lambda: block(conv_b=z(3)), "conv_b"),
            (lambda: b.prompt(p, ints(0, 2), ints(0, 1)), "cu"),
            (lambda: b.prompt(p, torch.tensor([0, 2]), ints(0)), "cu"),
            (lambda: b.prompt(p, ints(0, 2), torch.tensor([0])), "slots"),
            (lambda: b.prompt(p, ints(0, 2), ints(0), ints(1, 1)), "carry"),
            (lambda: b.step(p, torch.tensor([0, 1])), "slots"), (lambda: b.step(p, ints(0)), "in_proj|slots"),
            (lambda: block(in_proj=lambda v: z(2, 43, dtype=BF)).step(p, ints(0, 1)), "in_proj"),
            (lambda: block(in_proj=lambda v: z(1, 44, dtype=BF)).step(p, ints(0, 1)), "in_proj"),
            (lambda: block(in_proj=lambda v: z(2, 44)).step(p, ints(0, 1)), "in_proj"),
            (lambda: verify(z(7, 10), i), "8 rows"), (lambda: verify(z(8, 9), i), r"\[rows, 10\]"),
            (lambda: verify(z(8, 10), i.long()), "tokens"), (lambda: verify(z(8, 10), i[:1]), "tokens"),
            (lambda: verify(z(8, 10), i, z(6, 10, dtype=BF)), "draft"), (lambda: verify(z(8, 10), i, z(8, 10)), "draft"),
            (lambda: verify(z(8, 10), i, counts=ints(1)), "counts"),
            (lambda: verify(z(8, 10), i, uniform=z(6)), "uniform"),
            (lambda: verify(z(8, 10), i, uniform=z(8, dtype=BF)), "uniform"),
            (lambda: verify(z(8, 10, dtype=torch.float64), i), "float32"),
            (lambda: verify.kept(ints(1), ints(0, 1)), "accepted"), (lambda: verify.kept(ints(1, 1), ints(0)), "slots"),
            (lambda: S.DraftVerifier(2, 0, 10), "positive")]:
        with pytest.raises(ValueError, match=what):
            call()
    assert not [c for c in calls if c[0] not in ("fcm_dw1d_step", "fcm_dw1d_fwd")]


def test_tensors_on_different_devices_are_refused(calls):
    # ("meta" stands for another device than the one of the weights)
    def away(*s, dtype=BF):
        return torch.empty(*s, dtype=dtype, device="meta")

    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    lin, b, verify = linear(64, 8), block(), S.DraftVerifier(2, 3, 10)
    x, p, i = z(2, 64, dtype=BF), z(2, 32, dtype=BF), z(2, 3, dtype=i32)
    for call in (lambda: lin(away(2, 64)), lambda: lin(x, out=away(2, 8)),
                 lambda: S.MX4Linear(z(8, 32, dtype=u8), away(8, 2, dtype=u8)),
                 lambda: S.MX4Linear(z(8, 32, dtype=u8), z(8, 2, dtype=u8), bias=away(8, dtype=f32)),
                 lambda: b.prompt(p, away(2, dtype=i32), ints(0)), lambda: b.prompt(p, ints(0, 2), away(1, dtype=i32)),
                 lambda: b.prompt(p, ints(0, 2), ints(0), carry=away(1, dtype=i32)),
                 lambda: b.step(p, away(2, dtype=i32)), lambda: block(in_proj=lambda v: away(2, 44)).step(p, ints(0, 1)),
                 lambda: block(A=away(2, dtype=f32)), lambda: block(norm=away(8, dtype=f32)),
                 lambda: block(dt_bias=away(2, dtype=f32)), lambda: verify(z(8, 10), away(2, 3, dtype=i32)),
                 lambda: verify(z(8, 10), i, away(6, 10, dtype=f32)),
                 lambda: verify(z(8, 10), i, counts=away(2, dtype=i32)),
                 lambda: verify(z(8, 10), i, uniform=away(8, dtype=f32)),
                 lambda: verify.kept(ints(1, 1), away(2, dtype=i32))):
        with pytest.raises(ValueError, match="must be on"):
            call()


def test_tensors_that_are_not_on_the_gpu_are_refused(calls, monkeypatch):
    # a kernel that follows a host address faults
    lin, b = linear(64, 8), block()
    monkeypatch.undo()
    for call in (lambda: lin(z(2, 64, dtype=BF)), lin.weight, lambda: b.prompt(z(2, 32, dtype=BF), ints(0, 2), ints(0)),
                 lambda: b.step(z(2, 32, dtype=BF), ints(0, 1)), lambda: S.quantize_mx4(z(2, 64)),
                 lambda: S.MX4Linear.from_weight(z(2, 64)),
                 lambda: S.DraftVerifier(2, 3, 10)(z(8, 10), z(2, 3, dtype=torch.int32))):
        with pytest.raises(ValueError, match="GPU"):
            call()
