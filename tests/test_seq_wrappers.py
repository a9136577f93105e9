"""The sequence operators' wrappers with their launches stubbed (no GPU): what they pass on, on which
stream, and what they refuse."""
import contextlib

import pytest
import torch

import depthwise_pointwise_convolution_amd.sequence as S

z = torch.zeros
BF = torch.bfloat16


class Calls(list):
    """(name, problem, pointer arguments, stream) of the launches."""


@pytest.fixture
def calls(monkeypatch):
    got = Calls()

    def stub(name):
        def launch(prob, *args, stream=None):
            n = {"fcm_dw1d_fwd": 8, "fcm_dw1d_step": 6, "fcm_scan_fwd": 14, "fcm_scan_step": 11, "fcm_q4_fwd": 6,
                 "fcm_beam_select": 8, "fcm_beam_reorder": 4}[name]
            if len(args) > n:
                args, stream = args[:n], args[n]
            # the stream it runs on: the one passed, or what is current by then
            got.append((name, prob, args, torch.cuda.current_stream() if stream is None else stream))
        return launch

    for name in ("fcm_dw1d_fwd", "fcm_dw1d_step", "fcm_scan_fwd", "fcm_scan_step", "fcm_q4_fwd", "fcm_beam_select",
                 "fcm_beam_reorder"):
        monkeypatch.setattr(S, name, stub(name))
    monkeypatch.setattr(S, "fcm_scan_workspace", lambda prob: 64)
    monkeypatch.setattr(S, "fcm_beam_workspace", lambda prob: 64)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    # CPU tensors stand for those of the GPU
    monkeypatch.setattr(S, "_on_gpu", lambda t: True, raising=False)
    return got


def linear(C, K, dtype=BF):
    return S.Q4Linear(z(K, C // 2, dtype=torch.uint8), z(K, -(-C // 32), dtype=dtype), group=32)


def block(inner=16, N=4, rank=8, dim=24, dtype=BF, **k):
    parts = {"in_proj": linear(dim, 2 * inner, dtype), "x_proj": linear(inner, rank + 2 * N, dtype),
             "dt_proj": linear(rank, inner, dtype), "out_proj": linear(inner, dim, dtype), **k}
    return S.StateSpaceBlock(parts["in_proj"], z(inner, 4, dtype=dtype), None, parts["x_proj"], parts["dt_proj"], None,
                             z(inner, N), None, parts["out_proj"], slots=3)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


# ------------------------------------------------------------------------------------------
# streams
# ------------------------------------------------------------------------------------------
class Stream:
    def __init__(self, name):
        self.name, self.waited = name, []

    def wait_stream(self, other):
        self.waited.append(other)


@pytest.fixture
def streams(monkeypatch):
    """(the caller's stream, another one, what is the current one)."""
    now = [Stream("caller")]

    @contextlib.contextmanager
    def use(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", use)
    return now[0], Stream("other"), now


@pytest.mark.parametrize("what", ["prompt", "step", "linear", "advance"])
def test_a_stream_takes_the_whole_call(calls, streams, monkeypatch, what):
    # projections, allocations and launches: all on the stream that was given, behind the caller's
    caller, other, now = streams
    seen = []

    def watched(f):
        def call(x):
            seen.append(now[-1])
            return f(x)
        return call

    for name in ("empty", "empty_like"):
        def made(*a, real=getattr(torch, name), **k):
            seen.append(now[-1])
            return real(*a, **k)
        monkeypatch.setattr(torch, name, made)
    b = block(in_proj=watched(linear(24, 32)), x_proj=watched(linear(16, 16)), dt_proj=watched(linear(8, 16)),
              out_proj=watched(linear(16, 24)))
    search = S.BeamSearch(1, 2, 10, ints(0, 1))
    lin = linear(64, 8)
    seen.clear()
    if what == "prompt":
        b.prompt(z(5, 24, dtype=BF), ints(0, 2, 5), ints(0, 1), stream=other)
    elif what == "step":
        b.step(z(2, 24, dtype=BF), ints(0, 1), stream=other)
    elif what == "linear":
        # (an input that has to be laid out first)
        lin(z(4, 66, dtype=BF)[:, 1:65], stream=other)
    else:
        search.advance(z(2, 10), [z(2, 8)], stream=other)
    assert calls
    seen += [c[3] for c in calls]
    assert all(s is other for s in seen), [s.name for s in seen]
    assert other.waited == [caller] and now == [caller]


# ------------------------------------------------------------------------------------------
# broadcast inputs
# ------------------------------------------------------------------------------------------
def _strided_rows(prob, ld, t, rows, width):
    """Whether the launch reads `rows` rows of `t` inside its storage."""
    pitch = getattr(prob, ld) or width
    last = t.storage_offset() + (rows - 1) * pitch + width
    return last * t.element_size() <= t.untyped_storage().nbytes()


def test_broadcast_rows_are_laid_out(calls):
    # a stride of 0 means densely packed rows in the library: one row that stands for several, and
    # rows that overlap, are copied before
    row = torch.arange(64, dtype=BF)[None]
    lin = linear(64, 8)
    for x in (row.expand(4, 64), torch.arange(100, dtype=BF).as_strided((4, 64), (8, 1))):
        calls.clear()
        lin(x)
        (_, prob, args, _), = calls
        assert prob.M == 4 and _strided_rows(prob, "ldx", args[0], 4, 64)
        assert torch.equal(args[0], x)
    # a first step's logits: the same row for every beam
    search = S.BeamSearch(2, 3, 10, ints(*range(6)))
    logits = torch.randn(1, 10).expand(6, 10)
    calls.clear()
    search.advance(logits, [])
    prob, args = calls[0][1:3]
    assert _strided_rows(prob, "ldl", args[0], 6, 10) and torch.equal(args[0], logits)
    # one column: its rows may stand anywhere
    search = S.BeamSearch(1, 4, 1, ints(*range(4)))
    calls.clear()
    search.advance(z(1, 1).expand(4, 1), [])
    assert _strided_rows(calls[0][1], "ldl", calls[0][2][0], 4, 1)


def test_strided_rows_are_taken_as_they_are(calls):
    wide = z(4, 96, dtype=BF)
    linear(64, 8)(wide[:, :64])
    assert calls[0][1].ldx == 96 and calls[0][2][0].data_ptr() == wide.data_ptr()


# ------------------------------------------------------------------------------------------
# outputs
# ------------------------------------------------------------------------------------------
def test_an_output_that_the_kernel_would_miss_is_refused(calls):
    lin, x = linear(64, 8), z(4, 64, dtype=BF)
    for x_, out in ((x, z(2, 8, dtype=BF)), (x, z(4, 9, dtype=BF)), (x, z(4, 8)),
                    (x, z(8, 4, dtype=BF).t()), (x, z(1, 8, dtype=BF).expand(4, 8)),
                    (x, z(60, dtype=BF).as_strided((4, 8), (4, 1))),
                    (x[:1], z(8, 2, dtype=BF)[:, 1:2].t())):
        with pytest.raises(ValueError, match="out"):
            lin(x_, out=out)
    assert not calls


def test_outputs_that_fit_are_written_in_place(calls):
    lin, x = linear(64, 8), z(4, 64, dtype=BF)
    wide = z(4, 24, dtype=BF)
    for x_, out in ((x, wide[:, 8:16]), (x, z(4, 8, dtype=BF)), (x, z(6, 8, dtype=BF)), (x[:1], z(1, 8, dtype=BF)), (x[:1], wide[2:3, 3:11]),
                    (x[:0], z(0, 8, dtype=BF))):
        calls.clear()
        assert lin(x_, out=out) is out
        assert calls[0][2][5].data_ptr() == out.data_ptr()
    one = linear(64, 1)
    out = z(1, 7, dtype=BF)[:, 2:3]
    assert one(x[:1], out=out) is out


# ------------------------------------------------------------------------------------------
# what a block's projections give
# ------------------------------------------------------------------------------------------
def _gives(t):
    return lambda x: t


@pytest.mark.parametrize("name,bad", [
    ("in_proj", z(2, 16, dtype=BF)), ("in_proj", z(2, 33, dtype=BF)), ("in_proj", z(1, 32, dtype=BF)),
    ("in_proj", z(2, 32)), ("in_proj", z(32, 2, dtype=BF).t()), ("in_proj", z(2, 64, dtype=BF)[:, ::2]),
    ("in_proj", z(64, dtype=BF)), ("x_proj", z(1, 16, dtype=BF)), ("x_proj", z(2, 16)), ("x_proj", z(2, 8, dtype=BF)),
    ("x_proj", z(2, 32, dtype=BF)[:, ::2]), ("x_proj", z(32, dtype=BF)), ("dt_proj", z(2, 15, dtype=BF)),
    ("dt_proj", z(1, 16, dtype=BF)), ("dt_proj", z(2, 16)), ("dt_proj", z(16, 2, dtype=BF).t())])
def test_projections_of_another_form_are_refused(calls, name, bad):
    # (their memory is handed to the kernels, which would read past it or other values than meant)
    b = block(**{name: _gives(bad)})
    with pytest.raises(ValueError, match=name):
        b.prompt(z(2, 24, dtype=BF), ints(0, 2), ints(0))
    with pytest.raises(ValueError, match=name):
        b.step(z(2, 24, dtype=BF), ints(0, 1))


def test_projections_that_broadcast_a_row_are_laid_out(calls):
    rows = {"in_proj": z(1, 32, dtype=BF).expand(3, 32), "x_proj": z(1, 16, dtype=BF).expand(3, 16),
            "dt_proj": z(1, 16, dtype=BF).expand(3, 16)}
    b = block(**{k: _gives(v) for k, v in rows.items()})
    b.step(z(3, 24, dtype=BF), ints(0, 1, 2))
    b.prompt(z(3, 24, dtype=BF), ints(0, 2, 3), ints(0, 1))
    for name, prob, args, _ in calls:
        if name.startswith("fcm_dw1d"):
            assert _strided_rows(prob, "ldx", args[0], 3, 16)
        if name.startswith("fcm_scan"):
            for ld, at, width in (("ldx", 0, 16), ("lddt", 1, 16), ("ldb", 3, 4), ("ldc", 4, 4), ("ldz", 7, 16)):
                assert _strided_rows(prob, ld, args[at], 3, width), ld


# ------------------------------------------------------------------------------------------
# where tensors are
# ------------------------------------------------------------------------------------------
def test_tensors_that_are_not_on_the_gpu_are_refused(calls, monkeypatch):
    # a kernel that follows a host address faults
    lin, b, search = linear(64, 8), block(), S.BeamSearch(1, 2, 10, ints(0, 1))
    monkeypatch.undo()
    for call in (lambda: lin(z(2, 64, dtype=BF)), lambda: b.prompt(z(2, 24, dtype=BF), ints(0, 2), ints(0)),
                 lambda: b.step(z(2, 24, dtype=BF), ints(0, 1)), lambda: search.advance(z(2, 10), [])):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_tensors_on_different_devices_are_refused(calls):
    # ("meta" stands for another device than the one of the weights)
    def away(*s, dtype=BF):
        return torch.empty(*s, dtype=dtype, device="meta")

    i32 = {"dtype": torch.int32}
    lin, b, search = linear(64, 8), block(), S.BeamSearch(1, 2, 10, ints(0, 1))
    x, p = z(2, 64, dtype=BF), z(2, 24, dtype=BF)
    q, s = z(8, 32, dtype=torch.uint8), z(8, 2, dtype=BF)
    for call in (lambda: lin(away(2, 64)), lambda: lin(x, out=away(2, 8)),
                 lambda: S.Q4Linear(q, away(8, 2), group=32),
                 lambda: S.Q4Linear(q, s, zeros=away(8, 2, dtype=torch.uint8), group=32),
                 lambda: S.Q4Linear(q, s, bias=away(8, dtype=torch.float32), group=32),
                 lambda: b.prompt(p, away(2, **i32), ints(0)), lambda: b.prompt(p, ints(0, 2), away(1, **i32)),
                 lambda: b.prompt(p, ints(0, 2), ints(0), carry=away(1, **i32)), lambda: b.step(p, away(2, **i32)),
                 lambda: block(in_proj=_gives(away(2, 32))).step(p, ints(0, 1)),
                 lambda: block(x_proj=_gives(away(2, 16))).step(p, ints(0, 1)),
                 lambda: block(dt_proj=_gives(away(2, 16))).step(p, ints(0, 1)),
                 lambda: S.StateSpaceBlock(None, z(8, 4), None, None, None, None, away(8, 4, dtype=torch.float32), None,
                                           None, 1),
                 lambda: S.StateSpaceBlock(None, z(8, 4), away(8, dtype=torch.float32), None, None, None, z(8, 4), None,
                                           None, 1),
                 lambda: search.advance(away(2, 10), []), lambda: search.advance(z(2, 10), [away(2, 8)])):
        with pytest.raises(ValueError, match="must be on"):
            call()


# ------------------------------------------------------------------------------------------
# state arrays of the binding's reordering
# ------------------------------------------------------------------------------------------
@pytest.fixture
def reorder(monkeypatch):
    """fcm_beam_reorder of these pools, with the library's function stubbed: the (pool, slot bytes, slots)
    it would be given."""
    import depthwise_pointwise_convolution_amd as F
    got = []

    class Lib:
        @staticmethod
        def fcm_beam_reorder(prob, parent, slots, out, n, ptrs, bytes_, slots_, stream):
            got.append([(ptrs[i], bytes_[i], slots_[i]) for i in range(n)])
            return 0

    monkeypatch.setattr(F, "lib", lambda: Lib)
    return lambda *pools: (got.clear(), F.fcm_beam_reorder(None, 1, 2, 3, list(pools), stream=0), got[0])[2]


def test_state_arrays_with_gaps_are_refused(reorder):
    # a slot is as many bytes as slots are apart: with gaps in it, or before the first slot's start, the last
    # slot's copy would end behind the array
    base = z(6, 12)
    for bad in (base[:, 4:], base[:, ::2], base.reshape(6, 3, 4)[:, :, :2], base.reshape(6, 3, 4)[:, 1:],
                base[:, 8:].unsqueeze(1).expand(6, 3, 4), z(1, 12).expand(6, 12), base.t()[:, :5],
                z(30).as_strided((4, 2, 2), (4, 3, 1))):
        with pytest.raises(ValueError, match="slots"):
            reorder(z(6, 4), bad)


def test_state_arrays_without_gaps_are_taken(reorder):
    base = z(6, 3, 4)
    for good in (base, base[1:4], base.transpose(1, 2), base.reshape(6, 12)[2:], z(6, dtype=BF), base[:1],
                 z(6, 1, 5, 1), z(6, 2, 3, 4).permute(0, 3, 1, 2)):
        size = good[0].numel() * good.element_size()
        assert reorder(good) == [(good.data_ptr(), size, good.shape[0])]
    # the only slot of an array, whatever its distance to a next one
    assert reorder(z(6, 12)[:1, :4])[0][1] == 16


# ------------------------------------------------------------------------------------------
# a search's results
# ------------------------------------------------------------------------------------------
def test_each_step_of_a_search_has_its_own_results(calls, monkeypatch):
    # parents and tokens are what a caller keeps of every step to trace the beams back by
    step = iter(range(1, 9))

    def select(prob, logits, scores, done, ws, nxt, parent, token, next_done, *stream):
        n = next(step)
        nxt.fill_(-n), parent.fill_(n), token.fill_(10 * n), next_done.fill_(n)

    def reorder(prob, parent, slots, next_slots, pools, *stream):
        next_slots.copy_(slots + 1)

    monkeypatch.setattr(S, "fcm_beam_select", select)
    monkeypatch.setattr(S, "fcm_beam_reorder", reorder)
    search = S.BeamSearch(1, 2, 10, ints(0, 1), eos=3)
    kept = [(search.advance(z(2, 10), [z(4, 8)]), search.scores, search.done, search.slots) for _ in range(4)]
    for n, ((parent, token), _, _, _) in enumerate(kept, 1):
        assert parent.tolist() == [n] * 2 and token.tolist() == [10 * n] * 2
    for n, (_, scores, done, slots) in list(enumerate(kept, 1))[-2:]:
        assert scores.tolist() == [-n] * 2 and done.tolist() == [n] * 2 and slots.tolist() == [n, n + 1]
    assert search.parent is kept[-1][0][0] and search.token is kept[-1][0][1]


def test_intermediates_lie_beside_the_states(calls):
    # an in-projection that also moves its input: what the kernels write is not where that input is
    x = torch.empty(2, 24, dtype=BF, device="meta")
    b = block(in_proj=_gives(z(2, 32, dtype=BF)))
    b.step(x, ints(0, 1))
    b.prompt(x, ints(0, 2), ints(0))
    for name, _, args, _ in calls:
        assert all(a is None or a.device.type == "cpu" for a in args), name
