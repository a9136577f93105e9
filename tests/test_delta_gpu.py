"""Gated delta rule on the GPU against the recurrence in 64 bits."""
import math

import pytest
import torch

from recurrent_oracle import delta
from seq_oracle import TYPES

pytestmark = pytest.mark.gpu


def _inputs(seed, dtype, T, B, Hk, Hv, Dk, Dv, slots, qk_norm=True):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g) * std

    dt, std = TYPES[dtype], 1.0 if qk_norm else Dk ** -0.5
    c = {"q": normal(T, Hk, Dk, std=std).to(dt), "k": normal(T, Hk, Dk, std=std).to(dt), "v": normal(T, Hv, Dv).to(dt),
         "a": normal(T, Hv, std=1.5).to(dt), "b": normal(T, Hv, std=2.0).to(dt), "A": -torch.exp(normal(Hv)),
         "dt_bias": normal(Hv), "norm": 1 + normal(Dv, std=0.2), "z": normal(T, Hv, Dv).to(dt),
         "state": normal(slots, Hv, Dk, Dv)}
    if not qk_norm:  # beta |k|^2 <= 2 bounds the recurrence
        length = c["k"].float().norm(dim=-1, keepdim=True)
        c["k"] = (c["k"].float() / length.clamp(min=1.0)).to(dt)
    return c


def _gpu(t, pad=0):
    """On the GPU, with rows `pad` elements further apart than dense ones."""
    if t is None:
        return None, 0
    t = t.reshape(t.shape[0], -1) if t.dim() > 1 else t
    if not pad:
        return t.cuda(), 0
    wide = torch.full((t.shape[0], t.shape[1] + pad), math.nan, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]], t.shape[1] + pad


def _call(c, dtype, lens, slot_of, carry, Hk, Hv, Dk, Dv, opts, pad=0, state=True, eps=1e-6, step=False):
    import depthwise_pointwise_convolution_amd as F
    T, B = c["q"].shape[0], len(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    d, ld = {}, {}
    for name in "qkvabz":
        d[name], ld["ld" + name] = _gpu(c[name], pad)
    for name in ("A", "dt_bias", "norm"):
        d[name] = c[name].cuda() if c[name] is not None else None
    y, ld["ldy"] = _gpu(torch.full((T, Hv * Dv), 7.0).to(TYPES[dtype]), pad)
    pool = c["state"].cuda() if state else None
    slots = torch.tensor(slot_of, dtype=torch.int32).cuda() if slot_of is not None else None
    p = F.delta_problem(dtype, Hk, Hv, Dk, Dv, tokens=T, seqs=B, slots=c["state"].shape[0] if state else 0, eps=eps, **opts, **ld)
    if step:
        F.fcm_delta_step(p, d["q"], d["k"], d["v"], d["a"], d["b"], d["A"], d["dt_bias"], d["norm"], d["z"], slots, pool, y)
    else:
        ws = torch.full((F.fcm_delta_workspace(p),), 255, dtype=torch.uint8, device="cuda")
        F.fcm_delta_fwd(p, d["q"], d["k"], d["v"], d["a"], d["b"], d["A"], d["dt_bias"], d["norm"], d["z"],
                        torch.tensor(cu, dtype=torch.int32).cuda(), slots,
                        torch.tensor(carry, dtype=torch.int32).cuda() if carry is not None else None, pool, ws, y)
    torch.cuda.synchronize()
    return y.cpu(), pool.cpu() if state else None, [(cu[i], cu[i + 1]) for i in range(B)]


def _check(got, pool, want, T, Hv, Dv, dtype):
    y, ytol, new, ntol, written = want
    got = got.double().reshape(T, Hv, Dv)
    d = (got - y).abs()
    bad = (d > ytol) & written[:, None, None]
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), float((d / ytol)[written].max()))
    assert (got[~written] == torch.tensor(7.0).to(TYPES[dtype]).double()).all()
    if new is not None:
        d = (pool.double() - new).abs()
        assert (d <= ntol + 2 ** -23 * new.abs()).all(), float((d / (ntol + 2 ** -23 * new.abs() + 1e-300)).max())


CASES = [
    # dtype, lengths, Hk, Hv, Dk, Dv, options
    ("bf16", [1], 1, 1, 128, 128, {}),
    ("bf16", [64], 2, 4, 128, 128, {}),
    ("bf16", [65, 0, 200, 3], 2, 2, 128, 128, {"norm": False}),
    ("bf16", [130, 63, 64, 1], 1, 3, 64, 128, {"gate": False}),
    ("f16", [100, 29], 2, 4, 128, 64, {}),
    ("f16", [5] * 7, 1, 2, 128, 128, {}),
    ("f32", [77, 1, 130], 1, 2, 72, 100, {"norm": False, "gate": False}),
    ("f32", [70], 1, 1, 256, 256, {}),
    ("f32", [129], 1, 1, 32, 16, {"qk_norm": False}),
    ("bf16", [90], 1, 2, 256, 192, {"qk_norm": False, "norm": False}),
    ("f16", [33, 66], 3, 3, 24, 40, {}),
    ("bf16", [67], 1, 1, 1, 1, {"norm": False}),
    ("f16", [66], 1, 2, 7, 5, {}),
    ("f32", [68], 1, 1, 33, 17, {"softplus": False}),
    ("bf16", [2, 3], 1, 2, 130, 255, {}),
    ("f16", [300], 1, 1, 256, 250, {"norm": False}),
]


@pytest.mark.parametrize("dtype,lens,Hk,Hv,Dk,Dv,opts", CASES)
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_prompts(dtype, lens, Hk, Hv, Dk, Dv, opts, pad):
    opts = dict(opts)
    T, B = sum(lens), len(lens)
    c = _inputs(11 * T + Dk + Dv + pad, dtype, T, B, Hk, Hv, Dk, Dv, B + 2, opts.get("qk_norm", True))
    if not opts.pop("norm", True):
        c["norm"] = None
    if not opts.pop("gate", True):
        c["z"] = None
    if not opts.get("softplus", True):
        c["a"], c["dt_bias"] = c["a"].abs(), None
    slot_of = [B + 1 - i for i in range(B)]
    carry = [(i + 1) % 2 for i in range(B)]
    got, pool, spans = _call(c, dtype, lens, slot_of, carry, Hk, Hv, Dk, Dv, opts, pad)
    want = delta(dtype, c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], c["norm"], c["z"], spans, slot_of,
                 carry, c["state"], Dk ** -0.5, 1e-6, opts.get("qk_norm", True), opts.get("softplus", True))
    _check(got, pool, want, T, Hv, Dv, dtype)


@pytest.mark.parametrize("dtype,Dk,Dv,opts,pad", [
    ("bf16", 32, 32, {}, 0), ("f16", 128, 30, {"gate": False}, 2), ("f32", 64, 31, {"norm": False}, 0),
    ("bf16", 136, 32, {"norm": False}, 1), ("f32", 20, 32, {}, 4)])
def test_prompts_of_many_sequences(dtype, Dk, Dv, opts, pad):
    # so many sequences and heads that a slice has two tiles of columns
    opts, lens = dict(opts), ([1, 9, 66, 0, 17, 3, 30, 2] * 16)[:128]
    T, B = sum(lens), len(lens)
    c = _inputs(Dk + Dv, dtype, T, B, 2, 4, Dk, Dv, B)
    if not opts.pop("norm", True):
        c["norm"] = None
    if not opts.pop("gate", True):
        c["z"] = None
    slot_of, carry = [B - 1 - i for i in range(B)], [i % 3 for i in range(B)]
    got, pool, spans = _call(c, dtype, lens, slot_of, carry, 2, 4, Dk, Dv, opts, pad)
    want = delta(dtype, c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], c["norm"], c["z"], spans, slot_of,
                 carry, c["state"], Dk ** -0.5, 1e-6)
    _check(got, pool, want, T, 4, Dv, dtype)


@pytest.mark.parametrize("dtype,Hk,Hv,Dk,Dv,opts", [
    ("bf16", 2, 4, 128, 128, {}), ("f16", 1, 2, 64, 128, {"norm": False}), ("f32", 1, 1, 256, 256, {}),
    ("bf16", 1, 3, 128, 64, {"gate": False}), ("f32", 2, 2, 72, 100, {"qk_norm": False}), ("f16", 1, 1, 1, 1, {"norm": False}),
    ("bf16", 1, 2, 33, 17, {}), ("f16", 1, 1, 5, 255, {}), ("f32", 1, 1, 250, 3, {"softplus": False})])
@pytest.mark.parametrize("pad", [0, 3])
def test_tokens(dtype, Hk, Hv, Dk, Dv, opts, pad):
    opts, B = dict(opts), 5
    c = _inputs(Dk + 7 * Dv + pad, dtype, B, B, Hk, Hv, Dk, Dv, B + 2, opts.get("qk_norm", True))
    if not opts.pop("norm", True):
        c["norm"] = None
    if not opts.pop("gate", True):
        c["z"] = None
    if not opts.get("softplus", True):
        c["a"], c["dt_bias"] = c["a"].abs(), None
    slot_of = [4, -1, 6, 0, 7]  # two idle rows
    got, pool, spans = _call(c, dtype, [1] * B, slot_of, None, Hk, Hv, Dk, Dv, opts, pad, step=True)
    want = delta(dtype, c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], c["norm"], c["z"], spans, slot_of,
                 [1] * B, c["state"], Dk ** -0.5, 1e-6, opts.get("qk_norm", True), opts.get("softplus", True), chunk=1)
    want[0][[1, 4]] = 0
    want[1][[1, 4]] = 0
    _check(got, pool, want, B, Hv, Dv, dtype)


def test_nothing_carried():
    # no state array: every sequence starts from zero and nothing is stored
    lens = [70, 5]
    c = _inputs(3, "bf16", 75, 2, 1, 2, 64, 64, 2)
    got, _, spans = _call(c, "bf16", lens, None, None, 1, 2, 64, 64, {}, state=False)
    want = delta("bf16", c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], c["norm"], c["z"], spans, [0, 1],
                 [0, 0], None, 64 ** -0.5, 1e-6)
    _check(got, None, want, 75, 2, 64, "bf16")


def test_rows_behind_the_last_sequence_are_left():
    c = _inputs(4, "f16", 90, 2, 1, 2, 64, 64, 2)
    got, pool, spans = _call(c, "f16", [40, 30], [1, 0], [1, 1], 1, 2, 64, 64, {})
    want = delta("f16", c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], c["norm"], c["z"], spans, [1, 0],
                 [1, 1], c["state"], 64 ** -0.5, 1e-6)
    _check(got, pool, want, 90, 2, 64, "f16")


@pytest.mark.parametrize("A,a", [(-math.inf, 0.0), (-1e30, 1.0), (0.0, 1.0), (-1e-30, 0.0), (-50.0, 8.0)])
def test_rates_at_their_ends(A, a):
    # forgetting at once, never, and powers far below the smallest float
    c = _inputs(5, "f32", 100, 1, 1, 1, 32, 32, 1)
    c["A"][:] = A
    c["a"] = torch.where(torch.arange(100)[:, None] % 7 == 0, torch.tensor(a), c["a"])
    got, pool, spans = _call(c, "f32", [100], [0], [1], 1, 1, 32, 32, {})
    c["A"] = c["A"].clamp(min=-1e30)
    want = delta("f32", c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], c["norm"], c["z"], spans, [0], [1],
                 c["state"], 32 ** -0.5, 1e-6)
    _check(got, pool, want, 100, 1, 32, "f32")


def test_equal_keys():
    # the hardest system: every key the same, hardly any decay, rates near 1
    c = _inputs(6, "f32", 150, 1, 1, 1, 64, 64, 1)
    c["k"][:] = c["k"][0]
    c["b"][:] = 9.0
    c["A"][:] = -1e-3
    got, pool, spans = _call(c, "f32", [150], [0], [1], 1, 1, 64, 64, {})
    want = delta("f32", c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], c["norm"], c["z"], spans, [0], [1],
                 c["state"], 64 ** -0.5, 1e-6)
    _check(got, pool, want, 150, 1, 64, "f32")


def test_a_bad_value_stays_in_its_head_and_sequence():
    lens = [70, 70]
    c = _inputs(7, "bf16", 140, 2, 1, 2, 64, 64, 2)
    clean, cpool, _ = _call(c, "bf16", lens, [0, 1], [1, 1], 1, 2, 64, 64, {})
    c["v"][80, 1, 5] = math.nan
    c["v"][90, 1, 6] = math.inf
    got, pool, _ = _call(c, "bf16", lens, [0, 1], [1, 1], 1, 2, 64, 64, {})
    got, clean = got.reshape(140, 2, 64), clean.reshape(140, 2, 64)
    assert torch.equal(got[:, 0], clean[:, 0]) and torch.equal(got[:70], clean[:70])
    assert torch.equal(pool[0], cpool[0]) and torch.equal(pool[1, 0], cpool[1, 0])
    assert not torch.isfinite(got[80:, 1, 5]).any()


def test_prompt_in_parts_and_tokens_give_the_same():
    # one prompt whole, in two calls, and token by token
    T, dtype = 75, "f32"
    c = _inputs(8, dtype, T, 1, 1, 2, 64, 32, 1)
    whole, pool, spans = _call(c, dtype, [T], [0], [1], 1, 2, 64, 32, {})
    want = delta(dtype, c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], c["norm"], c["z"], spans, [0], [1],
                 c["state"], 64 ** -0.5, 1e-6)
    rows = []
    part = {**c}
    for s, e in [(0, 41)] + [(t, t + 1) for t in range(41, T)]:
        cut = {n: v[s:e] if n in "qkvabz" else v for n, v in part.items()}
        y, part["state"], _ = _call(cut, dtype, [e - s], [0], [1], 1, 2, 64, 32, {}, step=e - s == 1)
        rows.append(y)
    # two ways of the same sums: each within its bound, and the second one's runs over more chunks
    _check(whole, pool, want, T, 2, 32, dtype)
    d = (torch.cat(rows).double().reshape(T, 2, 32) - want[0]).abs()
    assert (d <= 40 * want[1]).all()


def test_captured():
    import depthwise_pointwise_convolution_amd as F
    c = _inputs(9, "bf16", 100, 2, 1, 2, 64, 64, 2)
    d = {n: c[n].reshape(c[n].shape[0], -1).cuda() if c[n].dim() > 1 and n != "state" else c[n].cuda() for n in c}
    cu = torch.tensor([0, 60, 100], dtype=torch.int32).cuda()
    slots, carry = torch.tensor([1, 0], dtype=torch.int32).cuda(), torch.ones(2, dtype=torch.int32).cuda()
    p = F.delta_problem("bf16", 1, 2, 64, 64, tokens=100, seqs=2, slots=2)
    t = F.delta_problem("bf16", 1, 2, 64, 64, tokens=2, seqs=2, slots=2)
    ws = torch.empty(F.fcm_delta_workspace(p), dtype=torch.uint8, device="cuda")
    y, y1 = torch.empty(100, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 128, dtype=torch.bfloat16, device="cuda")

    def both():
        F.fcm_delta_fwd(p, d["q"], d["k"], d["v"], d["a"], d["b"], d["A"], d["dt_bias"], d["norm"], d["z"], cu, slots,
                        carry, d["state"], ws, y)
        F.fcm_delta_step(t, d["q"], d["k"], d["v"], d["a"], d["b"], d["A"], d["dt_bias"], d["norm"], d["z"], slots,
                         d["state"], y1)

    first = d["state"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    wanted = []
    d["state"].copy_(first)
    for _ in range(3):
        both()
        wanted.append([x.clone() for x in (y, y1, d["state"])])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    d["state"].copy_(first)
    for w in wanted:
        y.zero_()
        ws.random_(0, 255)
        graph.replay()
        torch.cuda.synchronize()
        for got, x in zip((y, y1, d["state"]), w):
            assert torch.equal(got, x)


@pytest.mark.parametrize("cu", [[0, 30, 75], [0, 10, 75], [-9, 30, 2 ** 31 - 1], [-2 ** 31, 10, 99]])
def test_offsets_beyond_the_rows_are_cut(cu):
    # bit for bit what the offsets cut to 0 .. 50 give: which sequences are short goes by those too
    import depthwise_pointwise_convolution_amd as F
    T, B, Hk, Hv, Dk, Dv = 50, 2, 1, 2, 64, 32
    c = _inputs(31, "bf16", T, B, Hk, Hv, Dk, Dv, B)
    got = []
    for offsets in (cu, [min(max(v, 0), T) for v in cu]):
        d = {n: t.cuda() for n, t in c.items()}
        y = torch.full((T, Hv, Dv), 7.0, dtype=torch.bfloat16, device="cuda")
        p = F.delta_problem("bf16", Hk, Hv, Dk, Dv, tokens=T, seqs=B, slots=B)
        ws = torch.full((F.fcm_delta_workspace(p),), 255, dtype=torch.uint8, device="cuda")
        F.fcm_delta_fwd(p, d["q"], d["k"], d["v"], d["a"], d["b"], d["A"], d["dt_bias"], d["norm"], d["z"],
                        torch.tensor(offsets, dtype=torch.int32).cuda(), None, torch.ones(B, dtype=torch.int32).cuda(),
                        d["state"], ws, y)
        torch.cuda.synchronize()
        got.append((y.cpu(), d["state"].cpu()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.isfinite(got[0][0].float()).all()


@pytest.mark.parametrize("step", [True, False])
def test_rows_and_states_far_apart(step):
    # rows 2^30 elements apart, states behind the 2^31st element: bit for bit what dense ones give
    import depthwise_pointwise_convolution_amd as F
    T, Hk, Hv, Dk, Dv, far = 4 if step else 20, 1, 2, 128, 128, 2 ** 30 if step else 2 ** 28
    slots = 2 ** 31 // (Hv * Dk * Dv) + 2
    c = _inputs(32, "bf16", T, 1, Hk, Hv, Dk, Dv, T)
    pool = torch.empty(slots, Hv, Dk, Dv, device="cuda")
    got = []
    for apart in (False, True):
        d = {n: t.cuda().reshape(t.shape[0], -1) if n in "qkvabz" else t.cuda() for n, t in c.items()}
        ld, state = {}, d["state"]
        which = torch.arange(T if step else 1, dtype=torch.int32)
        if apart:
            wide = torch.empty((T - 1) * far + 1024, dtype=torch.bfloat16, device="cuda")
            at = 0
            for n in "qkab" + ("vz" if step else ""):
                w = d[n].shape[1]
                rows = wide.as_strided((T, w), (far, 1), at)
                rows.copy_(d[n])
                d[n], ld["ld" + n], at = rows, far, at + w
            which = slots - 1 - which
            pool[which.long().cuda()] = state[:len(which)]
            state = pool
        y = torch.empty(T, Hv * Dv, dtype=torch.bfloat16, device="cuda")
        p = F.delta_problem("bf16", Hk, Hv, Dk, Dv, tokens=T, seqs=T if step else 1, slots=state.shape[0], **ld)
        args = [d[n] for n in ("q", "k", "v", "a", "b", "A", "dt_bias", "norm", "z")]
        if step:
            F.fcm_delta_step(p, *args, which.cuda(), state, y)
        else:
            ws = torch.empty(F.fcm_delta_workspace(p), dtype=torch.uint8, device="cuda")
            F.fcm_delta_fwd(p, *args, torch.tensor([0, T], dtype=torch.int32).cuda(), which.cuda(),
                            torch.ones(1, dtype=torch.int32).cuda(), state, ws, y)
        torch.cuda.synchronize()
        got.append((y.cpu(), state[which.long().cuda()].cpu()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("Hk,Hv", [(1, 4), (2, 10), (1, 9)])
def test_key_heads_shared_by_many(Hk, Hv):
    lens, Dk, Dv = [70, 3, 40], 40, 24
    T, B = sum(lens), len(lens)
    c = _inputs(41 + Hv, "bf16", T, B, Hk, Hv, Dk, Dv, B)
    got, pool, spans = _call(c, "bf16", lens, [2, 0, 1], [1, 0, 1], Hk, Hv, Dk, Dv, {})
    want = delta("bf16", c["q"], c["k"], c["v"], c["a"], c["b"], c["A"], c["dt_bias"], c["norm"], c["z"], spans, [2, 0, 1],
                 [1, 0, 1], c["state"], Dk ** -0.5, 1e-6)
    _check(got, pool, want, T, Hv, Dv, "bf16")
