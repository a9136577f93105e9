"""The recurrent operators' wrappers on the GPU, and the operators together."""
import os
import sys

import pytest
import torch

from gpu_util import gpu_available
from recurrent_oracle import delta

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

BF = torch.bfloat16


def _linear(S, g, C, K, **k):
    return S.MX4Linear.from_weight((torch.randn(K, C, generator=g) * C ** -0.5).cuda(), **k)


def _block(S, dim=128, Hk=2, Hv=4, Dk=32, Dv=64, slots=6, seed=1):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).cuda()  # noqa: E731
    mixed, inner = 2 * Hk * Dk + Hv * Dv, Hv * Dv
    return S.DeltaRuleBlock(_linear(S, g, dim, mixed + inner + 2 * Hv), n(mixed, 4, std=0.5).to(BF), n(mixed, std=0.1),
                            -torch.exp(n(Hv)), n(Hv) - 2, 1 + n(Dv, std=0.1), _linear(S, g, inner, dim), Hk, Dk, Dv,
                            slots)


@pytest.mark.parametrize("how", ["stream", "handle", "default stream's handle"])
def test_wrappers_on_a_stream_give_what_they_give_without(how):
    # bit for bit: the same kernels on the same inputs
    import depthwise_pointwise_convolution_amd.sequence as S
    g = torch.Generator().manual_seed(2)
    x = torch.randn(700, 128, generator=g).to(BF).cuda()
    cu = torch.tensor([0, 300, 300, 700], dtype=torch.int32).cuda()
    slots = torch.tensor([4, 1, 0], dtype=torch.int32).cuda()
    tokens = torch.randn(3, 128, generator=g).to(BF).cuda()
    odd = torch.randn(15, 130, generator=g).to(BF).cuda()[:, 1:129]  # laid out anew by the 4-bit layer
    drafts = torch.randint(0, 100, (3, 4), generator=g, dtype=torch.int32).cuda()
    uniform = torch.rand(15, generator=g).cuda()
    head, both = _linear(S, g, 128, 100), _linear(S, g, 128, 100, quantize_input=True, act="relu")
    got = []
    for given in (False, True):
        kw = {}
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        if given:
            kw["stream"] = {"stream": s, "handle": s.cuda_stream, "default stream's handle": 0}[how]
        b = _block(S)
        out = [b.prompt(x, cu, slots, **kw), b.step(tokens, slots, **kw), head(odd, **kw), both(odd, **kw),
               *S.quantize_mx4(odd, **kw)]
        torch.cuda.synchronize()
        out += list(S.DraftVerifier(3, 4, 100)(out[2], drafts, head(odd[:12]), uniform=uniform, **kw))
        torch.cuda.synchronize()
        got.append([t.clone() for t in out + [b.window, b.state]])
    for i, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a, b), i


def test_weights_of_a_layer():
    # weight() is what the codes stand for: within a quarter of the value or of the scale, and the largest of a
    # block, which may end at 6 of up to 8 steps, within a quarter as well
    import depthwise_pointwise_convolution_amd.sequence as S
    g = torch.Generator().manual_seed(3)
    w = torch.randn(70, 96, generator=g).cuda()
    lin = S.MX4Linear.from_weight(w, dtype=torch.float16)
    got, scale = lin.weight(), torch.exp2(lin.scales.float() - 127).repeat_interleave(32, 1)
    assert ((got - w).abs() <= torch.maximum(w.abs(), scale) / 4).all()
    assert lin.dtype == torch.float16 and S.MX4Linear.from_weight(w.half()).dtype == torch.float16
    assert S.MX4Linear.from_weight(w).dtype == BF and lin(w[:3].half()).dtype == torch.float16


@pytest.mark.parametrize("lens,carry", [((5, 1, 0, 9), (0, 1, 1, 1)), ((200, 3, 64), (1, 0, 1)), ((), ())])
def test_a_blocks_rule_and_states(lens, carry):
    # what goes into the out-projection, and the states, against the recurrence on what the depthwise layer gave
    import depthwise_pointwise_convolution_amd as F
    import depthwise_pointwise_convolution_amd.sequence as S
    g = torch.Generator().manual_seed(4)
    T, B, b = sum(lens), len(lens), _block(S)
    x = torch.randn(T + 2, 128, generator=g).to(BF).cuda()  # (two rows of padding behind)
    cu = torch.tensor([0, *lens]).cumsum(0).to(torch.int32).cuda()
    slots = torch.tensor([4, 1, 0, 3][:B], dtype=torch.int32).cuda()
    goes_on = torch.tensor(carry, dtype=torch.int32).cuda()
    b.window.copy_(torch.randn(b.window.shape, generator=g))
    b.state.copy_(torch.randn(b.state.shape, generator=g))
    window, state = b.window.clone(), b.state.cpu().clone()
    seen = []
    project, b.out_proj = b.out_proj, lambda y: (seen.append(y.clone()), project(y))[1]
    b.prompt(x, cu, slots, goes_on)
    p = b.in_proj(x)
    u = torch.zeros(T + 2, b.mixed, dtype=BF, device="cuda")
    F.fcm_dw1d_fwd(F.dw1d_problem("bf16", b.mixed, 4, tokens=T + 2, seqs=B, slots=6, ldx=p.stride(0)), p, b.conv_w, b.conv_b,
                   cu, slots, goes_on, window, u)
    assert torch.equal(window, b.window)
    keys, at = b.keys, b.mixed + b.inner
    u, p = u.cpu(), p.cpu()
    head = lambda t, n: t.reshape(T + 2, n, -1)  # noqa: E731
    offsets = cu.tolist()
    y, ytol, want, stol, written = delta(
        "bf16", head(u[:, :keys], 2), head(u[:, keys:2 * keys], 2), head(u[:, 2 * keys:], 4), p[:, at:at + 4], p[:, at + 4:],
        b.A.cpu(), b.dt_bias.cpu(), b.norm.cpu(), head(p[:, b.mixed:at], 4), list(zip(offsets, offsets[1:])),
        slots.tolist(), list(carry), state, 32 ** -0.5, 1e-6)
    got = seen[0].cpu().reshape(T + 2, 4, 64).double()
    assert written.sum() == T
    assert ((got - y).abs() <= ytol)[written].all()
    assert ((b.state.cpu().double() - want).abs() <= stol).all()


def _example():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import draft_decode
    return draft_decode


def test_drafts_change_the_passes_and_not_the_tokens():
    # a row's result is the same whatever stands behind it and wherever its sequence was cut: the tokens with drafts
    # that stand now and then are those with drafts that never do
    ex = _example()
    R, D, N, V = 3, 4, 14, 500
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, V, (n,), generator=g).cuda() for n in (1, 30, 70)]
    never = lambda last, out: torch.full((R, D), -1, dtype=torch.int32, device="cuda")  # noqa: E731
    alone, slow = ex.decode(ex.Model(128, 2, V, R, seed=6), prompts, D, N + D, never)
    assert slow == N + D

    def known(last, out):
        # the known tokens, with a wrong one in the place that the request and what it has so far name
        rows = [alone[r][len(o):len(o) + D] + [0] * (D - len(alone[r][len(o):len(o) + D])) for r, o in enumerate(out)]
        rows = torch.tensor(rows, dtype=torch.int32)
        for r, o in enumerate(out):
            at = (len(o) + r) % (D + 2)
            if at < D:
                rows[r, at] = (rows[r, at] + 1) % V
        return rows.cuda()

    fast, passes = ex.decode(ex.Model(128, 2, V, R, seed=6), prompts, D, N, known)
    assert fast == [t[:N] for t in alone]
    assert passes < N


def test_the_example_runs():
    ex = _example()
    assert ex.main(["--dim", "128", "--layers", "2", "--vocab", "300", "--tokens", "8", "--check"]) == 0
    ex.main(["--dim", "128", "--layers", "2", "--vocab", "300", "--tokens", "8", "--temperature", "0.9"])


def test_steps_and_verifications_in_a_graph():
    # captured and replayed, against the same calls run eagerly
    import depthwise_pointwise_convolution_amd.sequence as S
    g = torch.Generator().manual_seed(7)
    R, D, V = 3, 4, 200
    x = torch.randn(R * (D + 1), 128, generator=g).to(BF).cuda()
    one = torch.randn(R, 128, generator=g).to(BF).cuda()
    tokens = torch.randint(0, V, (R, D), generator=g, dtype=torch.int32).cuda()
    uniform = (torch.rand(R * (D + 1), generator=g) * 0.3).cuda()
    slots = torch.arange(R, dtype=torch.int32).cuda()
    cu = torch.arange(0, R * (D + 1) + 1, D + 1, dtype=torch.int32).cuda()
    ones = torch.ones(2 * R, dtype=torch.int32).cuda()
    head, both = _linear(S, g, 128, V), _linear(S, g, 128, 128, quantize_input=True)
    verify = S.DraftVerifier(R, D, V)

    def run(b):
        logits = head(b.prompt(x, cu, slots + R, ones[:R]))
        accepted, following = verify(logits, tokens, uniform=uniform)
        y = b.prompt(x, *verify.kept(accepted, slots), ones)
        return [logits, accepted, following, y[:1], b.step(both(one), slots)]

    b = _block(S)
    want = []
    for _ in range(4):
        out = run(b)
        torch.cuda.synchronize()
        want.append([t.clone() for t in out + [b.window, b.state]])
    fresh = _block(S)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(fresh)
    for k in range(4):
        graph.replay()
        (torch.ones(1000, device="cuda") * 2).sum().item()
        torch.cuda.synchronize()
        for i, (a, c) in enumerate(zip(out + [fresh.window, fresh.state], want[k])):
            assert torch.equal(a, c), (k, i)


def test_nothing_to_do():
    import depthwise_pointwise_convolution_amd.sequence as S
    g = torch.Generator().manual_seed(8)
    b, head, both = _block(S), _linear(S, g, 128, 70), _linear(S, g, 128, 70, quantize_input=True)
    b.state.fill_(1.0)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    x = torch.zeros(0, 128, dtype=BF, device="cuda")
    assert b.prompt(x, torch.zeros(1, dtype=torch.int32, device="cuda"), none).shape == (0, 128)
    assert b.step(x, none).shape == (0, 128)
    # (an empty prompt that carries nothing on starts its slot from zero, one that does leaves it)
    zeros = torch.zeros(3, dtype=torch.int32, device="cuda")
    b.prompt(x, zeros, torch.tensor([1, 4], dtype=torch.int32).cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda())
    assert (b.state[1] == 0).all() and (b.state[[0, 2, 3, 4, 5]] == 1).all()
    assert head(x).shape == (0, 70) and both(x).shape == (0, 70)
    accepted, following = S.DraftVerifier(0, 4, 70)(head(x), none)
    assert accepted.shape == following.shape == (0,)
    assert S.quantize_mx4(x)[0].shape == (0, 64)
