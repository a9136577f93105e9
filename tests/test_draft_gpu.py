"""Verification of drafted tokens on the GPU: the answers that the definition allows."""
import math

import pytest
import torch

from recurrent_oracle import verify
from seq_oracle import TYPES

pytestmark = pytest.mark.gpu


def _run(dtype, target, draft, tokens, counts, uniform, heat, pad=0):
    """target [B, N+1, V], draft [B, N, V] or None."""
    import depthwise_pointwise_convolution_amd as F
    B, N1, V = target.shape
    N = N1 - 1

    def rows(t):
        wide = torch.full((t.shape[0] * t.shape[1], V + pad), math.inf, dtype=t.dtype, device="cuda")
        wide[:, :V] = t.reshape(-1, V).cuda()
        return wide

    p = F.draft_problem(dtype, B, N, V, temperature=heat, ldt=V + pad, ldd=V + pad)
    ws = torch.full((max(16, F.fcm_draft_workspace(p)),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((2, B + 1), -7, dtype=torch.int32, device="cuda")
    F.fcm_draft_verify(p, rows(target), rows(draft) if draft is not None else None, tokens.to(torch.int32).cuda(),
                       counts.to(torch.int32).cuda() if counts is not None else None,
                       uniform.cuda() if uniform is not None else None, ws, out[0], out[1])
    torch.cuda.synchronize()
    assert (out[:, B] == -7).all()
    return list(zip(out[0, :B].tolist(), out[1, :B].tolist()))


def _inputs(seed, dtype, B, N, V, heat, near=0.5):
    g = torch.Generator().manual_seed(seed)
    target = torch.randn(B, N + 1, V, generator=g) * 2
    target = target.masked_fill(torch.rand(B, N + 1, V, generator=g) < 0.1, -math.inf)
    draft = target[:, :N] + near * torch.randn(B, N, V, generator=g)
    target, draft = target.to(TYPES[dtype]), draft.to(TYPES[dtype])
    noise = -torch.log(-torch.log(torch.rand(B, N, V, generator=g).clamp(1e-6, 1 - 1e-6)))
    tokens = (draft.float() / heat + noise if heat > 0 else draft.float()).argmax(-1)
    return target, draft, tokens, torch.rand(B, N + 1, generator=g)


def _compare(got, target, draft, tokens, counts, uniform, heat):
    N = target.shape[1] - 1
    for r, answer in enumerate(got):
        n = N if counts is None else max(0, min(N, int(counts[r])))
        allowed = verify(target[r], draft[r] if draft is not None else None, tokens[r], n,
                         uniform[r] if uniform is not None else None, heat)
        assert answer in allowed, (r, answer, allowed)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,N,V,heat,near", [
    (1, 1, 1, 1.0, 0.5), (3, 2, 7, 1.0, 0.5), (4, 4, 1000, 0.7, 0.3), (2, 3, 1024, 1.3, 2.0), (5, 5, 4097, 1.0, 0.5),
    (2, 8, 33333, 0.9, 0.2), (1, 2, 200000, 1.0, 0.1), (3, 3, 65, 0.0, 0.1), (4, 4, 5000, 0.0, 0.02), (2, 64, 40, 1.0, 0.05),
    (40, 2, 300, 1.0, 1.0)])
@pytest.mark.parametrize("with_draft", [True, False])
def test_answers(dtype, B, N, V, heat, near, with_draft):
    target, draft, tokens, uniform = _inputs(B + N + V, dtype, B, N, V, heat, near)
    if not with_draft:
        draft = None
    counts = (torch.arange(B) * 3 + N) % (N + 2) if B > 2 else None
    got = _run(dtype, target, draft, tokens, counts, uniform if heat > 0 else None, heat, pad=V % 3)
    _compare(got, target, draft, tokens, counts, uniform, heat)


def test_the_distribution():
    # 4000 requests over the same small rows: accepted and drawn tokens follow the target's probabilities.  The
    # share of a token of probability p is off by four standard deviations sqrt(p (1-p) / n) in one of 16000.
    g = torch.Generator().manual_seed(0)
    n, V = 4000, 6
    row, other = torch.randn(V, generator=g), torch.randn(V, generator=g)
    target = row.expand(n, 2, V).contiguous()
    draft = other.expand(n, 1, V).contiguous()
    tokens = torch.multinomial(torch.softmax(other, 0), n, True, generator=g)[:, None]
    uniform = torch.rand(n, 2, generator=g)
    got = _run("f32", target, draft, tokens, None, uniform, 1.0)
    _compare(got, target, draft, tokens, None, uniform, 1.0)
    first = torch.tensor([int(tokens[i, 0]) if k > 0 else t for i, (k, t) in enumerate(got)])
    p = torch.softmax(row.double(), 0)
    share = torch.bincount(first, minlength=V).double() / n
    assert ((share - p).abs() <= 4.5 * (p * (1 - p) / n).sqrt()).all()


@pytest.mark.parametrize("heat", [1.0, 0.0])
def test_rows_and_tokens_at_their_ends(heat):
    V, N = 300, 3
    target, draft, tokens, uniform = _inputs(1, "f32", 10, N, V, 1.0)
    tokens = target[:, :N].argmax(-1)
    uniform[:, :N] *= 0.1
    target[0, 1] = -math.inf               # a row that leaves nothing
    target[1, 3] = -math.inf               # the one behind the last token
    draft[2, 1] = -math.inf                # a draft's row without any
    target[3, 0, 7] = math.inf             # larger than all
    target[4, 2, 5] = math.nan             # not a token
    tokens[5, 1] = V                       # no token of the vocabulary
    tokens[6, 0] = -1
    draft[7] = target[7, :N]               # the draft is the target
    target[8, 1] = torch.finfo(torch.float32).min  # a mask of the lowest value, everywhere
    target[9, 0, 20:] = torch.finfo(torch.float32).min
    for d in (draft, None):
        got = _run("f32", target, d, tokens, None, uniform, heat)
        _compare(got, target, d, tokens, None, uniform, heat)
    assert got[0] == (1, -1) and got[1][1] == -1 or heat == 1.0 and got[0][1] == -1


@pytest.mark.parametrize("r", [0.0, 1.0 - 2.0 ** -24, 1.0, 2.0])
def test_numbers_at_their_ends(r):
    V = 5000
    target, draft, tokens, uniform = _inputs(2, "f16", 4, 2, V, 1.0)
    uniform[:, 2] = r
    got = _run("f16", target, draft, tokens, None, uniform, 1.0)
    _compare(got, target, draft, tokens, None, uniform, 1.0)
    uniform[:, :2] = r
    got = _run("f16", target, draft, tokens, None, uniform, 1.0)
    _compare(got, target, draft, tokens, None, uniform, 1.0)


@pytest.mark.parametrize("heat", [1e-30, 1e-3, 1e30])
def test_temperatures_at_their_ends(heat):
    target, draft, tokens, uniform = _inputs(3, "f32", 4, 3, 500, 1.0)
    got = _run("f32", target, draft, tokens, None, uniform, heat)
    _compare(got, target, draft, tokens, None, uniform, heat)


def test_a_draft_without_logits_that_always_fails():
    # of one token with all of the target's probability but another one drafted, the target's is drawn
    target = torch.full((3, 2, 50), -math.inf)
    target[:, :, 11] = 3.0
    got = _run("f32", target, None, torch.tensor([[4], [11], [49]]), None, torch.full((3, 2), 0.5), 1.0)
    assert got == [(0, 11), (1, 11), (0, 11)]


def test_captured():
    import depthwise_pointwise_convolution_amd as F
    target, draft, tokens, uniform = _inputs(4, "bf16", 6, 4, 3000, 1.0)
    t, d = target.reshape(-1, 3000).cuda(), draft.reshape(-1, 3000).cuda()
    x, u = tokens.to(torch.int32).cuda(), uniform.cuda()
    p = F.draft_problem("bf16", 6, 4, 3000)
    ws = torch.empty(F.fcm_draft_workspace(p), dtype=torch.uint8, device="cuda")
    out = torch.zeros(2, 6, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    F.fcm_draft_verify(p, t, d, x, None, u, ws, out[0], out[1])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        F.fcm_draft_verify(p, t, d, x, None, u, ws, out[0], out[1])
    g = torch.Generator().manual_seed(5)
    for _ in range(3):
        uniform = torch.rand(6, 5, generator=g)
        u.copy_(uniform)
        ws.random_(0, 255)
        graph.replay()
        torch.cuda.synchronize()
        _compare(list(zip(*out.tolist())), target, draft, tokens, None, uniform, 1.0)


@pytest.mark.parametrize("heat", [1.0, 0.0])
def test_rows_far_apart(heat):
    # rows 2^30 elements apart: what dense ones give
    import depthwise_pointwise_convolution_amd as F
    B, N, V, far = 2, 2, 1000, 2 ** 30
    target, draft, tokens, uniform = _inputs(12, "bf16", B, N, V, heat)
    wide = torch.empty((B * (N + 1) - 1) * far + 2 * V, dtype=torch.bfloat16, device="cuda")
    t, d = wide.as_strided((B * (N + 1), V), (far, 1)), wide.as_strided((B * N, V), (far, 1), V)
    t.copy_(target.reshape(-1, V))
    d.copy_(draft.reshape(-1, V))
    p = F.draft_problem("bf16", B, N, V, temperature=heat, ldt=far, ldd=far)
    ws = torch.empty(F.fcm_draft_workspace(p), dtype=torch.uint8, device="cuda")
    out = torch.zeros(2, B, dtype=torch.int32, device="cuda")
    F.fcm_draft_verify(p, t, d, tokens.to(torch.int32).cuda(), None, uniform.cuda(), ws, out[0], out[1])
    torch.cuda.synchronize()
    _compare(list(zip(*out.tolist())), target, draft, tokens, None, uniform, heat)


def test_two_at_once():
    # two calls on streams of their own, each with its workspace
    import depthwise_pointwise_convolution_amd.sequence as S
    B, N, V = 6, 4, 20000
    cases = [_inputs(seed, "bf16", B, N, V, 1.0) for seed in (21, 22)]
    on = [tuple(c.cuda() for c in (t.reshape(-1, V), x.to(torch.int32), d.reshape(-1, V), u)) for t, d, x, u in cases]
    verify = S.DraftVerifier(B, N, V)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [verify(t, x, d, uniform=u, stream=s) for (t, x, d, u), s in zip(on, streams)]
    torch.cuda.synchronize()
    for (a, n), (target, draft, tokens, uniform) in zip(got, cases):
        _compare(list(zip(a.tolist(), n.tolist())), target, draft, tokens, None, uniform, 1.0)
