"""Convenience wrappers over the sequence operators: 4-bit pointwise layers, a state-space block
with its carried states, and beam search.  Shapes, types and strides are checked here; the
computation runs in the library's kernels.

A block is  in-projection -> causal depthwise layer -> (step, B, C) projection -> selective scan
gated by the in-projection's other half -> out-projection:

    block = StateSpaceBlock(..., slots=16)
    y = block.prompt(x, cu, slots)        # packed prompts [tokens, dim]
    y = block.step(x, slots)              # one token of each sequence [batch, dim]

Every call works on torch's current stream.  With ``stream`` (a torch stream or a raw handle) all of
it, the projections and what it allocates among it, works on that stream instead, behind what the
current stream holds at the call; whoever uses the results or the states on another stream waits for it.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import (ACT_CODES, beam_problem, dw1d_problem, fcm_beam_reorder, fcm_beam_select,
               fcm_beam_workspace, fcm_dw1d_fwd, fcm_dw1d_step, fcm_q4_fwd, fcm_scan_fwd,
               fcm_scan_step, fcm_scan_workspace, q4_problem, scan_problem)

DTYPE_NAMES = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _on_gpu(t: torch.Tensor) -> bool:
    """On the GPU whose stream the launches go to."""
    return t.is_cuda and t.get_device() == torch.cuda.current_device()


# (The checks of every step write their messages only where they refuse: a formatted shape or device
# costs as much as the rest of a check.)
def _beside(t: torch.Tensor, device: torch.device, name: str):
    """(a kernel that is given an address of another device, or of the host, faults)"""
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _rows(t: torch.Tensor, width: int, dtype: torch.dtype, name: str, device: torch.device):
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != width:
        raise ValueError(f"{name} must be [rows, {width}]")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    one, (apart, step) = shape[0] <= 1, t.stride()
    if step != 1 and not one:
        raise ValueError(f"{name}'s channels must be contiguous")
    # (rows that overlap, as a broadcast one does, have no row stride that the library takes)
    return t if (one or apart >= width) and (step == 1 or width == 1) else t.contiguous()


def _out(t: torch.Tensor, rows: int, width: int, dtype: torch.dtype, device: torch.device):
    """An output is written where it lies (its first `rows` rows), so its rows have to be apart and their
    channels dense."""
    _beside(t, device, "out")
    _need(t.dim() == 2 and t.shape[0] >= rows and t.shape[1] == width and t.dtype == dtype,
          f"out must be [{rows}, {width}] {dtype}")
    _need(width == 1 or t.stride(1) == 1, "out's channels must be contiguous")
    _need(t.shape[0] <= 1 or t.stride(0) >= width, "out's rows must not overlap")


def _stride(t: torch.Tensor) -> int:
    """Row stride; a single row has none that matters."""
    return t.stride(0) if t.shape[0] > 1 else 0


def _on(stream, call, *tensors):
    """`call` with all its work on `stream`.  The allocator hands memory out by stream: what `call`
    makes belongs to `stream` (which has to outlive it), the caller's `tensors` may be freed while it still uses them, and so may the
    results while the current stream does; each is told of the other."""
    if not hasattr(stream, "wait_stream"):  # a raw handle, 0 the default stream's
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    here = torch.cuda.current_stream()
    if stream == here:
        return call()
    stream.wait_stream(here)
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        result = call()
    for t in result if isinstance(result, tuple) else (result,):
        if t.is_cuda:
            t.record_stream(here)
    return result


def quantize_q4(weight: torch.Tensor, group: int = 128, symmetric: bool = False):
    """Codes, scales and zeros of a [K, C] weight for :class:`Q4Linear`: in each group of channels the
    15 steps of a code span its smallest to largest weight (zero included), or, if symmetric, codes
    1..15 span minus to plus the largest magnitude about a zero of 8 (zeros is then None).  The error of a
    weight is at most half a step, plus a step's rounding to the storage type."""
    _need(weight.dim() == 2 and weight.dtype in (torch.float16, torch.bfloat16),
          "weight must be [K, C] in a 16-bit type")
    _need(group in (32, 64, 128) and weight.shape[1] % 8 == 0,
          "groups have 32, 64 or 128 channels, C a multiple of 8")
    K, C = weight.shape
    groups = -(-C // group)
    w = torch.nn.functional.pad(weight.float(), (0, groups * group - C)).reshape(K, groups, group)
    if symmetric:
        scale = (w.abs().amax(-1) / 7).to(weight.dtype)
        zero = torch.full_like(scale, 8, dtype=torch.float32)
    else:
        low, high = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        scale = ((high - low) / 15).to(weight.dtype)
        zero = torch.where(scale > 0, (-low / scale.float()).round(), torch.zeros_like(low))
        zero = zero.clamp(0, 15)
    step = torch.where(scale > 0, scale.float(), torch.ones_like(scale, dtype=torch.float32))
    q = ((w / step[..., None]).round() + zero[..., None]).clamp(0, 15).to(torch.uint8)
    q = q.reshape(K, groups * group)[:, :C]
    q = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    return q, scale, None if symmetric else zero.to(torch.uint8)


class Q4Linear:
    """y = act(x W^T + bias) with W in 4-bit codes: q [K, C/2] uint8, scales [K, ceil(C/group)] in
    the activations' type, zeros the same in uint8 or None (8), bias [K] float32 or None."""

    def __init__(self, q, scales, zeros=None, bias=None, group: int = 128, act: str = "none"):
        _need(q.dim() == 2 and q.dtype == torch.uint8 and q.is_contiguous(), "q must be [K, C/2] uint8")
        self.K, self.C = q.shape[0], q.shape[1] * 2
        groups = -(-self.C // group)
        _need(scales.dtype in (torch.float16, torch.bfloat16) and scales.is_contiguous() and
              tuple(scales.shape) == (self.K, groups), f"scales must be [{self.K}, {groups}], 16-bit")
        _need(zeros is None or (zeros.dtype == torch.uint8 and zeros.is_contiguous() and
                                tuple(zeros.shape) == (self.K, groups)),
              f"zeros must be [{self.K}, {groups}] uint8")
        _need(bias is None or (bias.dtype == torch.float32 and tuple(bias.shape) == (self.K,) and
                               bias.is_contiguous()), f"bias must be [{self.K}] float32")
        for name, v in (("scales", scales), ("zeros", zeros), ("bias", bias)):
            if v is not None:
                _beside(v, q.device, name)
        _need(act in ACT_CODES, f"act must be one of {sorted(ACT_CODES)}")
        self.q, self.scales, self.zeros, self.bias = q, scales, zeros, bias
        self.group, self.act, self.dtype = group, act, scales.dtype

    @classmethod
    def from_weight(cls, weight, bias=None, group: int = 128, act: str = "none",
                    symmetric: bool = False) -> "Q4Linear":
        return cls(*quantize_q4(weight, group, symmetric), bias=bias, group=group, act=act)

    def weight(self) -> torch.Tensor:
        """The [K, C] weight the codes stand for, in float32."""
        q = torch.stack([self.q & 15, self.q >> 4], -1).reshape(self.K, self.C).float()
        at = torch.arange(self.C, device=q.device) // self.group
        zero = 8.0 if self.zeros is None else self.zeros.float()[:, at]
        return (q - zero) * self.scales.float()[:, at]

    def __call__(self, x, out=None, stream=None) -> torch.Tensor:
        if stream is not None:
            return _on(stream, lambda: self(x, out), x, out)
        _need(_on_gpu(self.q), "the weights must be on the current GPU")
        x = _rows(x, self.C, self.dtype, "x", self.q.device)
        if x.data_ptr() % 16 or _stride(x) % 8:
            x = x.contiguous()
        M = x.shape[0]
        if out is None:
            out = torch.empty(M, self.K, dtype=self.dtype, device=x.device)
        else:
            _out(out, M, self.K, self.dtype, x.device)
        fcm_q4_fwd(q4_problem(DTYPE_NAMES[self.dtype], M, self.C, self.K, group=self.group,
                              act=self.act, ldx=_stride(x), ldy=_stride(out)),
                   x, self.q, self.scales, self.zeros, self.bias, out)
        return out


class StateSpaceBlock:
    """A state-space block and the states of `slots` sequences.  dim: the model's width, inner: the
    block's channels, N states of a channel, rank: width of the step's low-rank projection.

    in_proj: dim -> 2*inner (scan input, gate); conv_w [inner, W], conv_b [inner] float32;
    x_proj: inner -> rank + 2*N (step, B, C); dt_proj: rank -> inner; dt_bias [inner] float32;
    A [inner, N] float32, negative; skip [inner] float32; out_proj: inner -> dim.  The projections
    are callables on [rows, channels] such as :class:`Q4Linear`."""

    def __init__(self, in_proj, conv_w, conv_b, x_proj, dt_proj, dt_bias, A, skip, out_proj,
                 slots: int):
        self.inner, self.W = conv_w.shape
        self.N = A.shape[1]
        self.dtype = conv_w.dtype
        _need(self.dtype in DTYPE_NAMES, "conv_w must be float32, float16 or bfloat16")
        _need(tuple(A.shape) == (self.inner, self.N) and A.dtype == torch.float32 and
              A.is_contiguous(), f"A must be [{self.inner}, N] float32")
        for name, v in (("conv_b", conv_b), ("dt_bias", dt_bias), ("skip", skip)):
            _need(v is None or (tuple(v.shape) == (self.inner,) and v.dtype == torch.float32 and
                                v.is_contiguous()), f"{name} must be [{self.inner}] float32")
        for name, v in (("A", A), ("conv_b", conv_b), ("dt_bias", dt_bias), ("skip", skip)):
            if v is not None:
                _beside(v, conv_w.device, name)
        self.in_proj, self.x_proj, self.dt_proj, self.out_proj = in_proj, x_proj, dt_proj, out_proj
        self.conv_w, self.conv_b, self.dt_bias, self.A, self.skip = (
            conv_w.contiguous(), conv_b, dt_bias, A, skip)
        self.slots = slots
        self.window = torch.zeros(slots, self.W - 1, self.inner, dtype=self.dtype,
                                  device=conv_w.device)
        self.state = torch.zeros(slots, self.inner, self.N, device=conv_w.device)
        self.name = DTYPE_NAMES[self.dtype]

    def _projected(self, p, rows: int, width: int, name: str):
        """What a projection gave, in the form the kernels take its rows."""
        p = _rows(p, width, self.dtype, name, self.window.device)
        if p.shape[0] != rows:
            raise ValueError(f"{name} must have {rows} rows")
        return p

    def _halves(self, x):
        """(scan input, gate): the in-projection's two halves."""
        xz = self._projected(self.in_proj(x), x.shape[0], 2 * self.inner, "in_proj's result")
        return xz[:, :self.inner], xz[:, self.inner:]

    def _parts(self, u):
        """(step, B, C) of the depthwise layer's output."""
        p = self.x_proj(u)
        _need(p.dim() == 2 and p.shape[1] > 2 * self.N, "x_proj must give the step's rows and then B and C")
        rank = p.shape[1] - 2 * self.N
        p = self._projected(p, u.shape[0], p.shape[1], "x_proj's result")
        dt = self._projected(self.dt_proj(p[:, :rank]), u.shape[0], self.inner, "dt_proj's result")
        return dt, p[:, rank:rank + self.N], p[:, rank + self.N:]

    def _index(self, t, n: int, name: str):
        if t is None:
            return
        _beside(t, self.window.device, name)
        if t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous():
            raise ValueError(f"{name} must be [{n}] int32")

    def prompt(self, x, cu, slots, carry=None, stream=None) -> torch.Tensor:
        """x: [tokens, dim], sequence b in rows cu[b] .. cu[b+1]-1 and state slot slots[b]; with
        carry[b] != 0 it continues from there."""
        if stream is not None:
            return _on(stream, lambda: self.prompt(x, cu, slots, carry), x, cu, slots, carry)
        _need(_on_gpu(self.window), "the block must be on the current GPU")
        T, B = x.shape[0], slots.shape[0]
        self._index(cu, B + 1, "cu")
        self._index(slots, B, "slots")
        self._index(carry, B, "carry")
        xs, z = self._halves(x)
        u = torch.empty(T, self.inner, dtype=self.dtype, device=self.window.device)
        fcm_dw1d_fwd(dw1d_problem(self.name, self.inner, self.W, tokens=T, seqs=B,
                                  slots=self.slots, ldx=_stride(xs)),
                     xs, self.conv_w, self.conv_b, cu, slots, carry, self.window, u)
        dt, b, c = self._parts(u)
        y = torch.empty_like(u)
        prob = scan_problem(self.name, self.inner, self.N, tokens=T, seqs=B, slots=self.slots,
                            lddt=_stride(dt), ldb=_stride(b), ldc=_stride(c), ldz=_stride(z))
        ws = torch.empty(max(16, fcm_scan_workspace(prob)), dtype=torch.uint8,
                         device=self.window.device)
        fcm_scan_fwd(prob, u, dt, self.A, b, c, self.skip, self.dt_bias, z, cu, slots, carry,
                     self.state, ws, y)
        return self.out_proj(y)

    def step(self, x, slots, stream=None) -> torch.Tensor:
        """x: [batch, dim], one token of the sequence in slots[b] (outside [0, slots): an idle row)."""
        if stream is not None:
            return _on(stream, lambda: self.step(x, slots), x, slots)
        _need(_on_gpu(self.window), "the block must be on the current GPU")
        B = x.shape[0]
        self._index(slots, B, "slots")
        xs, z = self._halves(x)
        u = torch.empty(B, self.inner, dtype=self.dtype, device=self.window.device)
        fcm_dw1d_step(dw1d_problem(self.name, self.inner, self.W, tokens=B, seqs=B,
                                   slots=self.slots, ldx=_stride(xs)),
                      xs, self.conv_w, self.conv_b, slots, self.window, u)
        dt, b, c = self._parts(u)
        y = torch.empty_like(u)
        fcm_scan_step(scan_problem(self.name, self.inner, self.N, tokens=B, seqs=B,
                                   slots=self.slots, lddt=_stride(dt), ldb=_stride(b),
                                   ldc=_stride(c), ldz=_stride(z)),
                      u, dt, self.A, b, c, self.skip, self.dt_bias, z, slots, self.state, y)
        return self.out_proj(y)


class BeamSearch:
    """Beams of `requests` searches: their scores, done flags and state slots, moved on by each
    :meth:`advance`.  Beam i starts in state slot slots[i]; at first only the first beam of a request
    counts (the others would repeat it)."""

    def __init__(self, requests: int, beams: int, vocab: int, slots: torch.Tensor, eos: int = -1):
        n = requests * beams
        _need(slots.dtype == torch.int32 and tuple(slots.shape) == (n,) and slots.is_contiguous(),
              f"slots must be [{n}] int32")
        dev = slots.device
        self.requests, self.beams, self.vocab, self.eos = requests, beams, vocab, eos
        self.scores = torch.full((requests, beams), float("-inf"), device=dev)
        self.scores[:, 0] = 0
        self.scores = self.scores.reshape(-1)
        self.done = torch.zeros(n, dtype=torch.int32, device=dev)
        self.slots = slots.clone()
        self.parent = torch.zeros(n, dtype=torch.int32, device=dev)
        self.token = torch.zeros(n, dtype=torch.int32, device=dev)
        self._next = (torch.empty_like(self.scores), torch.empty_like(self.done),
                      torch.empty_like(self.slots))
        self._ws: Optional[torch.Tensor] = None
        self._key = self._prob = None  # the last logits' form and their problem

    def advance(self, logits: torch.Tensor, pools: Sequence[torch.Tensor], stream=None):
        """Takes the logits [requests*beams, vocab] of the beams' last tokens, picks the next beams,
        and moves the states in `pools` ([slots, ...], contiguous) to them.  Returns (parent, token),
        tensors of this step's own, to trace the beams back by; scores, done and slots are the new beams'
        (two sets of buffers in turn, so that two steps can be captured and replayed as one graph: the
        call after the next writes over them)."""
        if stream is not None:
            return _on(stream, lambda: self.advance(logits, pools), logits, *pools)
        n = self.requests * self.beams
        _need(logits.dtype in DTYPE_NAMES, "logits must be float32, float16 or bfloat16")
        _need(_on_gpu(self.slots), "the search must be on the current GPU")
        logits = _rows(logits, self.vocab, logits.dtype, "logits", self.slots.device)
        if logits.shape[0] != n:
            raise ValueError(f"logits must have {n} rows")
        for p in pools:
            _beside(p, logits.device, "a state pool")
            _need(p.is_contiguous(), "state pools must be contiguous")
        key = (logits.dtype, self.eos, _stride(logits))
        if key != self._key:
            self._key, self._prob = key, beam_problem(DTYPE_NAMES[logits.dtype], self.requests, self.beams,
                                                      self.vocab, eos=self.eos, ldl=key[2])
        prob = self._prob
        if self._ws is None:
            self._ws = torch.empty(max(16, fcm_beam_workspace(prob)), dtype=torch.uint8,
                                   device=logits.device)
        scores, done, slots = self._next
        self.parent, self.token = torch.empty_like(slots), torch.empty_like(slots)
        fcm_beam_select(prob, logits, self.scores, self.done if self.eos >= 0 else None, self._ws,
                        scores, self.parent, self.token, done)
        for i in range(0, len(pools), 8) or (0,):
            fcm_beam_reorder(prob, self.parent, self.slots, slots, list(pools[i:i + 8]))
        self._next = (self.scores, self.done, self.slots)
        self.scores, self.done, self.slots = scores, done, slots
        return self.parent, self.token
