"""The gated delta rule's norm is of the 32-bit outputs: y is rounded once, and no type's range cuts what goes into it."""
import pytest
import torch

from recurrent_oracle import delta
from seq_oracle import TINY, U, half, silu
from test_delta_gpu import _call, _inputs

pytestmark = pytest.mark.gpu


def _want(dtype, c, spans, slot_of, carry, Dk, Dv, eps):
    """(y, its bound): the recurrence's outputs without their rounding, then the norm and the gate in 64 bits."""
    o, tol, *_ = delta(dtype, c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], None, None, spans, slot_of,
                       carry, c["state"], Dk ** -0.5, eps)
    # (the oracle ends with  tol = t + half * (|o| + t) + TINY)
    tol = ((tol - TINY[dtype] - half(dtype) * o.abs()) / (1 + half(dtype))).clamp(min=0)
    f = (o.square().mean(-1, keepdim=True) + eps).rsqrt()
    off = f * tol.square().mean(-1, keepdim=True).sqrt() + (Dv + 8) * U  # of the factor, relative
    norm, z = c["norm"].double(), c["z"].double()
    y, tol = o * f * norm, (tol * (1 + off) + o.abs() * off) * f * norm.abs()
    g = silu(z)
    tol = tol * g.abs() + y.abs() * (12 * U * z.abs() * torch.sigmoid(z) + 2 * U * z.abs() * g.abs() + 2.0 ** -120)
    y = y * g
    return y, tol + half(dtype) * (y.abs() + tol) + TINY[dtype]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("values,states,eps", [(1.0, 1.0, 1e-6), (1.0, 1e6, 1e-6), (6e4, 1e5, 1e-6), (1e-3, 1e-4, 1e-6),
                                               (1e-6, 1e-6, 1e-6), (1e-4, 1e-5, 1e-12)])
@pytest.mark.parametrize("lens,Hk,Hv,Dk,Dv", [([100, 17, 16, 3], 1, 2, 64, 128), ([130], 2, 2, 40, 36),
                                              ([18, 65], 1, 1, 128, 31)])
def test_norm_of_32_bit_outputs(dtype, values, states, eps, lens, Hk, Hv, Dk, Dv):
    T, B = sum(lens), len(lens)
    c = _inputs(T + Dv, dtype, T, B, Hk, Hv, Dk, Dv, B)
    c["v"] = (c["v"].float().clamp(-1, 1) * values).to(c["v"].dtype)
    c["state"] *= states
    slot_of, carry = list(range(B)), [1] * B
    ends = [sum(lens[:i]) for i in range(B + 1)]
    y, ytol = _want(dtype, c, list(zip(ends, ends[1:])), slot_of, carry, Dk, Dv, eps)
    got, _, _ = _call(c, dtype, lens, slot_of, carry, Hk, Hv, Dk, Dv, {}, eps=eps)
    got = got.double().reshape(T, Hv, Dv)
    assert torch.isfinite(got).all()
    d = (got - y).abs()
    assert (d <= ytol).all(), (float((d / ytol).max()), int((d > ytol).sum()))


@pytest.mark.parametrize("pad", [0, 1])
def test_many_sequences_with_a_norm(pad):
    # two tiles of columns a slice
    lens, Hk, Hv, Dk, Dv = [17, 30, 2, 66] * 32, 2, 4, 64, 48
    T, B = sum(lens), len(lens)
    c = _inputs(1, "f16", T, B, Hk, Hv, Dk, Dv, B)
    c["state"] *= 1e6
    ends = torch.tensor([0] + lens).cumsum(0).tolist()
    y, ytol = _want("f16", c, list(zip(ends, ends[1:])), list(range(B)), [1] * B, Dk, Dv, 1e-6)
    got, _, _ = _call(c, "f16", lens, list(range(B)), [1] * B, Hk, Hv, Dk, Dv, {}, pad=pad)
    assert ((got.double().reshape(T, Hv, Dv) - y).abs() <= ytol).all()


def test_outputs_behind_the_2_to_the_31st():
    # the last sequence's rows, whose 32-bit outputs lie behind 2^31 elements, are bit for bit those of it alone
    import depthwise_pointwise_convolution_amd as F
    Hk, Hv, Dk, Dv, last = 1, 64, 32, 256, 100
    T = 2 ** 31 // (Hv * Dv) + 2 * last
    g = torch.Generator(device="cuda").manual_seed(1)
    x = {n: torch.randn(T, w, device="cuda", generator=g, dtype=torch.bfloat16)
         for n, w in (("q", Hk * Dk), ("k", Hk * Dk), ("v", Hv * Dv), ("a", Hv), ("b", Hv), ("z", Hv * Dv))}
    A, norm = -torch.ones(Hv, device="cuda"), torch.ones(Dv, device="cuda")
    got = []
    for rows in (T, last):
        d = {n: v[-rows:] for n, v in x.items()}
        p = F.delta_problem("bf16", Hk, Hv, Dk, Dv, tokens=rows, seqs=2, slots=2)
        ws = torch.empty(F.fcm_delta_workspace(p), dtype=torch.uint8, device="cuda")
        state = torch.ones(2, Hv, Dk, Dv, device="cuda")
        y = torch.empty(rows, Hv * Dv, dtype=torch.bfloat16, device="cuda")
        cu = torch.tensor([0, rows - last, rows], dtype=torch.int32).cuda()
        F.fcm_delta_fwd(p, d["q"], d["k"], d["v"], d["a"], d["b"], A, None, norm, d["z"], cu, None,
                        torch.ones(2, dtype=torch.int32).cuda(), state, ws, y)
        torch.cuda.synchronize()
        got.append((y[-last:].clone(), state[1].clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.isfinite(got[0][0].float()).all()


def test_two_at_once():
    # two prompts' calls on streams of their own, each with its workspace, give what they give one after the other
    import depthwise_pointwise_convolution_amd as F
    Hk, Hv, Dk, Dv, lens = 2, 4, 64, 64, [300, 5, 200]
    T, B = sum(lens), len(lens)
    cu = torch.tensor([0, 300, 305, 505], dtype=torch.int32).cuda()
    p = F.delta_problem("f16", Hk, Hv, Dk, Dv, tokens=T, seqs=B, slots=B)
    cases = [{n: t.cuda() for n, t in _inputs(seed, "f16", T, B, Hk, Hv, Dk, Dv, B).items()} for seed in (1, 2)]
    out = [[(torch.empty(T, Hv * Dv, dtype=torch.float16, device="cuda"), c["state"].clone(),
             torch.empty(F.fcm_delta_workspace(p), dtype=torch.uint8, device="cuda")) for c in cases] for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for together in (False, True):
        for c, (y, state, ws), s in zip(cases, out[together], streams):
            F.fcm_delta_fwd(p, c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], c["norm"], c["z"], cu, None,
                            None, state, ws, y, stream=s.cuda_stream if together else None)
            if not together:
                torch.cuda.synchronize()
    torch.cuda.synchronize()
    for (y, state, _), (z, other, _) in zip(*out):
        assert torch.equal(y, z) and torch.equal(state, other)
