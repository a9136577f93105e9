"""The sequence operators' wrappers on the GPU."""
import pytest
import torch

from gpu_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

BF = torch.bfloat16


def _linear(S, g, C, K, group=64):
    return S.Q4Linear.from_weight((torch.randn(K, C, generator=g) * C ** -0.5).to(BF).cuda(), group=group)


def _block(S, dim=128, inner=256, N=16, rank=8, slots=6, seed=1):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).cuda()  # noqa: E731
    return S.StateSpaceBlock(_linear(S, g, dim, 2 * inner), n(inner, 4, std=0.5).to(BF), n(inner, std=0.1),
                             _linear(S, g, inner, rank + 2 * N), _linear(S, g, rank, inner), n(inner) - 3,
                             -torch.rand(inner, N, generator=g).cuda() - 0.1, n(inner), _linear(S, g, inner, dim), slots)


@pytest.mark.parametrize("how", ["stream", "handle", "default stream's handle"])
def test_wrappers_on_a_stream_give_what_they_give_without(how):
    # bit for bit: the same kernels on the same inputs
    import depthwise_pointwise_convolution_amd.sequence as S
    g = torch.Generator().manual_seed(2)
    x = torch.randn(700, 128, generator=g).to(BF).cuda()
    cu = torch.tensor([0, 300, 300, 700], dtype=torch.int32).cuda()
    slots = torch.tensor([4, 1, 0], dtype=torch.int32).cuda()
    tokens = torch.randn(3, 128, generator=g).to(BF).cuda()
    odd = torch.randn(5, 130, generator=g).to(BF).cuda()[:, 1:129]  # laid out anew by the 4-bit layer
    head = _linear(S, g, 128, 1000)
    got = []
    for given in (False, True):
        kw = {}
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        if given:
            kw["stream"] = {"stream": s, "handle": s.cuda_stream, "default stream's handle": 0}[how]
        b = _block(S)
        search = S.BeamSearch(1, 3, 1000, slots)
        out = [b.prompt(x, cu, slots, **kw), b.step(tokens, slots, **kw), head(odd, **kw)]
        logits = head(out[1], **kw) if not given else None
        if given and how != "default stream's handle":
            with torch.cuda.stream(s):
                logits = head(out[1])
        elif given:
            logits = head(out[1])
        out += list(search.advance(logits, [b.window, b.state], **kw))
        if given:
            torch.cuda.current_stream().wait_stream(s)
        out += [search.scores, search.slots, b.window, b.state]
        torch.cuda.synchronize()
        got.append([t.clone() for t in out])
    for i, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a, b), i


def test_broadcast_rows_give_what_their_copies_give():
    import depthwise_pointwise_convolution_amd.sequence as S
    g = torch.Generator().manual_seed(3)
    lin = _linear(S, g, 128, 500)
    row = torch.randn(1, 128, generator=g).to(BF).cuda()
    y = lin(row.expand(7, 128))
    assert torch.equal(y, lin(row.repeat(7, 1)))
    slots = torch.arange(4, dtype=torch.int32).cuda()
    one, all_ = S.BeamSearch(1, 4, 500, slots), S.BeamSearch(1, 4, 500, slots)
    pools = [torch.randn(4, 8, generator=g).cuda()]
    a, b = one.advance(y[:1].expand(4, 500), pools), all_.advance(y[:4], [pools[0].clone()])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(one.scores, all_.scores)
