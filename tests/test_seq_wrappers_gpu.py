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


def test_beams_traced_back_by_the_steps_results():
    # the tokens of every beam, gathered step by step and from the kept parents and tokens at the end
    import depthwise_pointwise_convolution_amd.sequence as S
    g = torch.Generator().manual_seed(4)
    R, W, V, steps = 2, 3, 300, 6
    search = S.BeamSearch(R, W, V, torch.arange(R * W, dtype=torch.int32).cuda())
    base = torch.arange(R).repeat_interleave(W).cuda() * W
    history, kept = torch.zeros(R * W, 0, dtype=torch.int32).cuda(), []
    for _ in range(steps):
        parent, token = search.advance(torch.randn(R * W, V, generator=g).cuda(), [])
        history = torch.cat([history[base + parent], token[:, None]], 1)
        kept.append((parent, token))
    at = torch.arange(R * W).cuda()
    back = []
    for parent, token in reversed(kept):
        back.insert(0, token[at])
        at = base[at] + parent[at]
    assert torch.equal(torch.stack(back, 1), history)


def test_a_block_and_a_search_in_a_graph():
    # two steps (the search's buffers alternate) captured and replayed, against the same steps run eagerly
    import depthwise_pointwise_convolution_amd.sequence as S
    g = torch.Generator().manual_seed(5)
    W, V = 3, 200
    x = torch.randn(W, 128, generator=g).to(BF).cuda()
    head = _linear(S, g, 128, V)
    slots = torch.arange(W, dtype=torch.int32).cuda()

    def start():
        return _block(S, slots=W), S.BeamSearch(1, W, V, slots)

    def two(b, search):
        out = []
        for _ in range(2):
            out += list(search.advance(head(b.step(x, search.slots)), [b.window, b.state]))
        return out

    b, search = start()
    want = []
    for _ in range(4):
        out = two(b, search)
        torch.cuda.synchronize()
        want.append([t.clone() for t in out + [search.scores, search.slots, b.state]])
    b, search = start()
    two(b, search)  # (the workspace and the kernels are there before the capture)
    torch.cuda.synchronize()
    fresh, fresh_search = start()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = two(fresh, fresh_search)
    for k in range(4):
        graph.replay()
        (torch.ones(1000, device="cuda") * 2).sum().item()
        torch.cuda.synchronize()
        for i, (a, c) in enumerate(zip(out + [fresh_search.scores, fresh_search.slots, fresh.state], want[k])):
            assert torch.equal(a, c), (k, i)
