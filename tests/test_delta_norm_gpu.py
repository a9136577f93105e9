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
